// Log probabilities of given tokens, the entropy of their rows and the top
// alternatives, in one pass over the logits.
//
// With z = x / T of a row's V logits, m their maximum and y = (x - m) log2(e) / T:
//   l = sum 2^y,  a = sum 2^y y,   lse = m / T + ln l,
//   logprob = z_token - lse,       entropy = ln l - ln 2 * a / l
// (the entropy as a difference of two terms of its own size, not of lse and a
// mean of z).  x - m comes before the product, so an exponent near zero is
// exact; l and a are held in fp32 per thread over a few hundred terms and
// merged by their maxima, the logarithm and what is written are taken in 64 bits.
//
// What bounds it: the logits are read once.  An element costs ~5 issue slots
// (widen, subtract, scale, clamp, 2^y, two sums), about half of what an SM has
// while the memory delivers its bf16 elements.
//
// A row goes to S CTAs (one where there are rows enough), each over a
// contiguous part in rounds of 256 threads x 64 bytes, the next round's loads
// in flight.  With S > 1 the CTA that takes the row's last ticket merges the
// parts; no CTA waits on another.
//
// Top alternatives, K <= 32.  In a part's first round the K-th largest of the
// 256 threads' maxima (value, then lower index) is a bound that K elements
// reach: only those at or above it go to a list in shared memory, at most
// (K - 1) * 32 + 1 of them whatever the values, about K for values in no
// order.  Later rounds append what exceeds the K-th best so far; a list past
// 128 entries is ranked (each entry counts the better ones) and cut to K, and
// a round that would overflow it takes a bound of its own first.
#include <limits.h>
#include <math.h>

#include "common.cuh"

namespace specv {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;          // 16-byte loads of a thread per round
constexpr int kCap = 2048;        // list entries
constexpr int kSoft = 128;        // list length that is cut to K
constexpr int kMaxParts = 32;
constexpr float kFarBelow = -1000.f;  // 2^y is +0 there; keeps -inf out of products

template <typename T> constexpr int per_vec() { return 16 / (int)sizeof(T); }

// Larger value, or the same at a lower index.
__device__ __forceinline__ bool better(float v, int i, float bv, int bi) {
    return v > bv || (v == bv && i < bi);
}

// maximum that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Stats {
    float m = -INFINITY, l = 0.f, a = 0.f;
    // sums rebased to maximum `to` >= m
    __device__ void rebase(float to, float c) {
        if (l != 0.f) {
            const float d = max_nan((m - to) * c, kFarBelow), s = fast_exp2(d);
            a = s * fmaf(l, d, a);
            l *= s;
        }
        m = to;
    }
    __device__ void merge(Stats o, float c) {
        const float to = fmaxf(m, o.m);
        if (m < to) rebase(to, c);
        if (o.m < to) o.rebase(to, c);
        l += o.l;
        a += o.a;
    }
};

template <typename T> __device__ __forceinline__ void widen(const uint4& r, float (&x)[per_vec<T>()]);
template <> __device__ __forceinline__ void widen<float>(const uint4& r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
}
template <> __device__ __forceinline__ void widen<__nv_bfloat16>(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Vector v of a row: elements v * EPV - off .. of [0, V), -inf outside.  The
// vectors lie on the 16-byte grid of memory; one that is not whole is read
// element by element, so nothing outside the row is.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* row, int64_t V, int off, int64_t v) {
    constexpr int EPV = per_vec<T>();
    const int64_t e = v * EPV - off;
    if (e >= 0 && e + EPV <= V) {
        uint4 r;
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                     : "l"(row + e));
        return r;
    }
    alignas(16) T x[EPV];
#pragma unroll
    for (int i = 0; i < EPV; ++i)
        x[i] = e + i >= 0 && e + i < V ? row[e + i] : Elem<T>::from_f32(-INFINITY);
    return *reinterpret_cast<const uint4*>(x);
}

struct Shared {
    float v[kCap];
    int i[kCap];
    float tv[kThreads];  // the threads' maxima
    int ti[kThreads];
    float best_v[32];
    int best_i[32];
    Stats stats[kThreads / 32];
    float bound_v;
    int bound_i;
    int count, last;
};

// Ranks the first `count` entries of the list and leaves its K best, sorted, at
// the front (every thread calls it; the list is complete and visible).
__device__ __forceinline__ int cut(Shared& s, int count, int K) {
    const int tid = threadIdx.x;
    for (int e = tid; e < count; e += kThreads) {
        const float v = s.v[e];
        const int i = s.i[e];
        int rank = 0;
        for (int o = 0; o < count; ++o) rank += better(s.v[o], s.i[o], v, i);
        if (rank < K) {
            s.best_v[rank] = v;
            s.best_i[rank] = i;
        }
    }
    __syncthreads();
    const int kept = count < K ? count : K;
    if (tid < kept) {
        s.v[tid] = s.best_v[tid];
        s.i[tid] = s.best_i[tid];
    }
    if (tid == 0) s.count = kept;
    __syncthreads();
    return kept;
}

// What is written for a row: stats complete, the sorted alternatives in s.
template <typename T>
__device__ __forceinline__ void write_row(const LogprobArgs& a, Shared& s, const Stats& st, int64_t row,
                                          const T* x, int found) {
    const int tid = threadIdx.x;
    const bool none = st.l == 0.f;  // every logit is -inf
    const double lnl = log((double)st.l), t = a.temperature;
    const double lse = none ? 0.0 : (double)st.m / t + lnl;
    if (tid == 0) {
        const int tok = a.tokens[row];
        float lp = -INFINITY;
        if (tok < 0 || tok >= a.V) raise_device_error(a.dev_err, SPEC_DEVERR_TOKEN);
        else if (!none) lp = (float)((double)Elem<T>::to_f32(x[tok]) / t - lse);
        a.logprob[row] = lp;
        if (a.entropy)
            a.entropy[row] = none ? 0.f : (float)(lnl - 0.69314718055994530942 * ((double)st.a / st.l));
    }
    if (tid < a.K) {
        const bool have = tid < found;
        if (a.top_ids) a.top_ids[row * a.K + tid] = have ? s.i[tid] : -1;
        if (a.top_logprobs)
            a.top_logprobs[row * a.K + tid] = have ? (float)((double)s.v[tid] / t - lse) : -INFINITY;
    }
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, 4) logprob_kernel(const LogprobArgs a) {
    constexpr int EPV = per_vec<T>();
    __shared__ Shared s;
    const int tid = threadIdx.x, S = a.parts, K = a.K;
    const int64_t row = blockIdx.x / S;
    const int part = blockIdx.x - (int)row * S;
    if (tid == 0) s.count = 0;
    grid_dep_launch_dependents();
    grid_dep_wait();
    if (a.lens && (int)(row % a.n) >= a.lens[row / a.n]) return;

    const T* x = static_cast<const T*>(a.logits) + row * a.V;
    const int off = (int)(((uint64_t)row * (uint64_t)a.V) % EPV);
    const int64_t vecs = (a.V + off + EPV - 1) / EPV, per = (vecs + S - 1) / S;
    const int64_t v0 = part * per, v1 = v0 + per < vecs ? v0 + per : vecs;
    const float c = a.c;
    Stats st;
    uint64_t l2 = f2(0.f, 0.f), a2 = l2;
    float m = -INFINITY;
    float tau = -INFINITY;  // the K-th best of the rounds before (-inf: fewer than K)

    uint4 cur[kVecs], nxt[kVecs];
    auto fetch = [&](uint4 (&r)[kVecs], int64_t v) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            const int64_t at = v + u * kThreads + tid;
            r[u] = at < v1 ? load_vec(x, a.V, off, at)
                           : (sizeof(T) == 4 ? make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u)
                                             : make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u));
        }
    };
    fetch(cur, v0);
    for (int64_t v = v0; v < v1; v += kVecs * kThreads) {
        fetch(nxt, v + kVecs * kThreads);
        float bm = -INFINITY;
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
            float e[EPV];
            widen<T>(cur[u], e);
#pragma unroll
            for (int j = 0; j < EPV; j += 2) bm = fmax3(bm, e[j], e[j + 1]);
        }
        if (bm > m) {
            Stats old;
            old.m = m;
            float p, q;
            f2_split(l2, p, q);
            old.l = p + q;
            f2_split(a2, p, q);
            old.a = p + q;
            old.rebase(bm, c);
            m = bm;
            l2 = f2(old.l, 0.f);
            a2 = f2(old.a, 0.f);
        }
        {
            const float mm = m == -INFINITY ? 0.f : m;
            const uint64_t neg = f2(-mm, -mm), cc = f2(c, c);
#pragma unroll
            for (int u = 0; u < kVecs; ++u) {
                float e[EPV];
                widen<T>(cur[u], e);
#pragma unroll
                for (int j = 0; j < EPV; j += 2) {
                    float y0, y1;
                    f2_split(f2_mul(f2_add(f2(e[j], e[j + 1]), neg), cc), y0, y1);
                    y0 = max_nan(y0, kFarBelow);
                    y1 = max_nan(y1, kFarBelow);
                    const uint64_t w = f2(fast_exp2(y0), fast_exp2(y1));
                    l2 = f2_add(l2, w);
                    a2 = f2_fma(w, f2(y0, y1), a2);
                }
            }
        }
        if (TOP) {
            const bool first = v == v0;
            const int base = (int)(v * EPV - off);  // first element of the round
            // appends this round's elements that `want` takes; the last place taken
            auto append = [&](auto want) {
                int place = -1;
#pragma unroll
                for (int u = 0; u < kVecs; ++u) {
                    float e[EPV];
                    widen<T>(cur[u], e);
                    const int at = base + (u * kThreads + tid) * EPV;
#pragma unroll
                    for (int j = 0; j < EPV; ++j)
                        if (want(e[j], at + j)) {
                            place = atomicAdd(&s.count, 1);
                            if (place < kCap) {
                                s.v[place] = e[j];
                                s.i[place] = at + j;
                            }
                        }
                }
                return place;
            };
            int place = -1;
            if (!first && bm > tau) place = append([&](float e, int) { return e > tau; });
            if (__syncthreads_or(first || place >= kSoft)) {
                int count = first ? 0 : s.count;
                if (first || count > kCap) {
                    // entries of earlier rounds (fewer than kSoft) stand in front
                    const int before = first ? 0 : __syncthreads_count(tid < kSoft && s.i[tid] < base);
                    int bi = INT_MAX;
#pragma unroll
                    for (int u = kVecs - 1; u >= 0; --u) {
                        float e[EPV];
                        widen<T>(cur[u], e);
#pragma unroll
                        for (int j = EPV - 1; j >= 0; --j)
                            if (e[j] == bm) bi = base + (u * kThreads + tid) * EPV + j;
                    }
                    s.tv[tid] = bm;
                    s.ti[tid] = bi;
                    if (tid == 0) {
                        s.count = before;
                        s.bound_v = -INFINITY;
                        s.bound_i = INT_MAX;
                    }
                    __syncthreads();
                    int rank = 0;
                    for (int o = 0; o < kThreads; ++o) rank += better(s.tv[o], s.ti[o], bm, bi);
                    if (rank == K - 1 && bm > -INFINITY) {
                        s.bound_v = bm;
                        s.bound_i = bi;
                    }
                    __syncthreads();
                    const float bv = s.bound_v;
                    const int bx = s.bound_i;
                    if (bm > tau && bm >= bv)
                        append([&](float e, int i) { return e > tau && !better(bv, bx, e, i); });
                    __syncthreads();
                    count = s.count;
                }
                cut(s, count, K);
                tau = count >= K ? s.v[K - 1] : -INFINITY;
                __syncthreads();  // before the next round appends
            }
        }
#pragma unroll
        for (int u = 0; u < kVecs; ++u) cur[u] = nxt[u];
    }
    st.m = m;
    {
        float p, q;
        f2_split(l2, p, q);
        st.l = p + q;
        f2_split(a2, p, q);
        st.a = p + q;
    }
    // the CTA's sums
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Stats other;
        other.m = __shfl_xor_sync(0xffffffffu, st.m, o);
        other.l = __shfl_xor_sync(0xffffffffu, st.l, o);
        other.a = __shfl_xor_sync(0xffffffffu, st.a, o);
        st.merge(other, c);
    }
    if ((tid & 31) == 0) s.stats[tid >> 5] = st;
    __syncthreads();
    st = s.stats[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) st.merge(s.stats[w], c);
    int found = 0;
    if (TOP) found = cut(s, s.count, K);

    if (S == 1) {
        write_row<T>(a, s, st, row, x, found);
        return;
    }
    // ---- parts: leave this one's record; the last CTA of the row merges them
    const int64_t rec = row * S + part;
    float* pst = a.part_stats + rec * 4;
    if (TOP && tid < K) {
        a.part_v[rec * K + tid] = tid < found ? s.v[tid] : -INFINITY;
        a.part_i[rec * K + tid] = tid < found ? s.i[tid] : -1;
    }
    if (tid == 0) *reinterpret_cast<float4*>(pst) = make_float4(st.m, st.l, st.a, 0.f);
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        s.last = atomicAdd(&a.tickets[row], 1) == S - 1;
        s.count = 0;
    }
    __syncthreads();
    if (!s.last) return;
    __threadfence();
    if (tid == 0) a.tickets[row] = 0;
    if (TOP) {
        for (int e = tid; e < S * K; e += kThreads) {
            const int i = __ldcg(a.part_i + row * S * K + e);
            if (i >= 0) {
                const int place = atomicAdd(&s.count, 1);
                s.v[place] = __ldcg(a.part_v + row * S * K + e);
                s.i[place] = i;
            }
        }
    }
    st = Stats();
    for (int p = 0; p < S; ++p) {
        const float4 r = __ldcg(reinterpret_cast<const float4*>(a.part_stats) + row * S + p);
        Stats o;
        o.m = r.x;
        o.l = r.y;
        o.a = r.z;
        st.merge(o, c);
    }
    __syncthreads();
    if (TOP) found = cut(s, s.count, K);
    write_row<T>(a, s, st, row, x, found);
}

}  // namespace

// Parts of a row: four CTAs an SM where the rows alone are fewer, a round of
// loads at least for each part.
int logprob_parts(const LogprobArgs& a, int num_sms, int max_tickets) {
    const int64_t rows = (int64_t)a.B * a.n;
    const int64_t round = kThreads * kVecs * (a.dtype == SPEC_DTYPE_F32 ? 4 : 8);
    const int64_t most = (a.V + round - 1) / round, want = (4 * (int64_t)num_sms + rows - 1) / rows;
    int64_t s = want < most ? want : most;
    if (s > kMaxParts) s = kMaxParts;
    return rows > max_tickets ? 1 : (int)s;
}

size_t logprob_workspace_bytes(const LogprobArgs& a) {
    return a.parts > 1 ? (size_t)a.B * a.n * a.parts * (16 + 8 * (size_t)a.K) : 0;
}

cudaError_t launch_logprobs(LogprobArgs a, void* workspace, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.B * a.n;
    a.part_stats = static_cast<float*>(workspace);
    a.part_v = a.part_stats + rows * a.parts * 4;
    a.part_i = reinterpret_cast<int32_t*>(a.part_v + rows * a.parts * a.K);
    const dim3 grid((unsigned)(rows * a.parts)), block(kThreads);
    if (a.dtype == SPEC_DTYPE_F32)
        return a.K ? launch_dependent(logprob_kernel<float, true>, grid, block, 0, stream, a)
                   : launch_dependent(logprob_kernel<float, false>, grid, block, 0, stream, a);
    return a.K ? launch_dependent(logprob_kernel<__nv_bfloat16, true>, grid, block, 0, stream, a)
               : launch_dependent(logprob_kernel<__nv_bfloat16, false>, grid, block, 0, stream, a);
}

}  // namespace specv
