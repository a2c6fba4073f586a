// The softmax of a 128-key tile on the tensor-core attention kernels with bf16
// P, in halves of 64 columns, and the driver's tensor-map encoder.
#pragma once

#include <cuda.h>
#include <math.h>

#include "common.cuh"

namespace specv {
namespace {

// 64 consecutive fp32 TMEM columns of this thread's lane.
__device__ __forceinline__ void load64(uint32_t taddr, uint32_t (&v)[64]) {
    uint32_t (&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(&v[0]);
    uint32_t (&hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(&v[32]);
    tmem_ld32(taddr, lo);
    tmem_ld32(taddr + 32, hi);
    tmem_wait_ld();
}

// Scores of 64 columns with the invisible ones at -inf; returns their maximum.
// vis: bit c set when column c is visible.
__device__ __forceinline__ float mask_max64(uint32_t (&r)[64], uint64_t vis) {
    if (vis != ~0ull) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
            r[c] = ((vis >> c) & 1ull) ? r[c] : __float_as_uint(-INFINITY);
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c2 = 0; c2 < 32; ++c2)
        mx[c2 & 3] =
            fmax3(mx[c2 & 3], __uint_as_float(r[2 * c2]), __uint_as_float(r[2 * c2 + 1]));
    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// Scores of 64 columns (raw fp32 bits from TMEM, rewritten in place) in log2
// units with the invisible ones at -inf; returns their maximum.  vis: bit c
// set when column c is visible.
__device__ __forceinline__ float scale_mask64(uint32_t (&r)[64], float sl2, uint64_t vis) {
#pragma unroll
    for (int c = 0; c < 64; c += 2) {
        float v0, v1;
        f2_split(f2_mul(f2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), f2(sl2, sl2)),
                 v0, v1);
        r[c] = __float_as_uint(v0);
        r[c + 1] = __float_as_uint(v1);
    }
    return mask_max64(r, vis);
}

// p = 2^(v - m) of 64 columns (fp32 bits), packed to bf16 (F16: fp16) pairs;
// returns their sum.
template <bool F16>
__device__ __forceinline__ float exp_pack64(const uint32_t (&v)[64], float m, uint32_t (&pk)[32]) {
    const uint64_t neg_m = f2(-m, -m);
    uint64_t ps[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < 64; c += 2) {
        float e0, e1;
        f2_split(f2_add(f2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), neg_m), e0, e1);
        e0 = fast_exp2(e0);
        e1 = fast_exp2(e1);
        ps[(c >> 1) & 1] = f2_add(ps[(c >> 1) & 1], f2(e0, e1));
        pk[c >> 1] = F16 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
    }
    float a0, a1, b0, b1;
    f2_split(ps[0], a0, a1);
    f2_split(ps[1], b0, b1);
    return (a0 + b0) + (a1 + b1);
}

// Visible columns [c0, c0 + 64) of a 128-key tile for a query row: the
// context keys (with a window: the sinks and the keys from `low` on), then the
// drafts of the row's bits, limited to the tile's keys.
template <bool WIN>
__device__ __forceinline__ uint64_t visible64(int key0, int c0, int nvalid, int ctx,
                                              uint64_t mrow, int low, int sinks) {
    const int kc0 = key0 + c0, nv = nvalid - c0, nctx = ctx - kc0;
    auto below = [](int n) { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1; };
    const uint64_t valid = below(nv);
    uint64_t cbits = below(nctx);
    if (WIN) cbits &= below(sinks - kc0) | ~below(low - kc0);
    const uint64_t dbits = nctx >= 64    ? 0ull
                           : nctx >= 0   ? mrow << nctx
                           : nctx > -64  ? mrow >> -nctx
                                         : 0ull;
    return (cbits | dbits) & valid;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn get_encode_fn() {
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    }
    return fn;
}

}  // namespace
}  // namespace specv
