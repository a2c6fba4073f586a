// Log probabilities of given tokens, the entropy of their rows and the top
// alternatives, in one pass over the logits.
//
// With z = x / T of a row's V logits, m their maximum and y = (x - m) log2(e) / T:
//   l = sum 2^y,  a = sum 2^y y,   lse = m / T + ln l,
//   logprob = z_token - lse,       entropy = ln l - ln 2 * a / l
// (the entropy as a difference of two terms of its own size, not of lse and a
// mean of z).  x - m comes before the product, so an exponent near zero is
// exact; l and a are held in fp32 per thread over a few hundred terms and
// merged by their maxima.
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
// Top alternatives, K <= 32.  In a part's first round the K-th largest of the maxima of
// 64 groups of threads is a bound that K elements reach: only those at or above it go to
// a list in shared memory, about K + a few for values in no order, and later rounds append
// what exceeds it.  After 1, 2, 4 rounds and then every kCheck the threads meet; a list past
// K + kSlack entries is ranked (each entry counts the better ones) and cut to K, whose last
// is the bound from then on: a thread that appends costs its warp half a round.  Where the
// list overflowed meanwhile (many equal or rising values) the rounds since are read once
// more, each with a bound over the 256 threads' maxima by value and index, which at most
// (K - 1) * 32 + 1 elements of a round reach, whatever they are.
// The rare parts are rolled loops, in line: unrolled, the kernel had 78 KB of code; as
// function calls they made the compiler wait for the next round's loads at every call.
//
// Measured, bf16: 2048 rows of 152064 with 5 alternatives 133 us (4.7 TB/s; the bytes' floor
// 92), without any 104; 32 sequences of up to 5 rows of 128256 with 20 alternatives 20.7,
// without 11; 5 fp32 rows of 1000 5.5.  What is left of the alternatives is the appends (12
// of 133 us, 4 of 20.7), the meetings and, in parts, the merge.  Alternatives: meeting in
// every round 1.5 times as long (rows of 152064), no cut before the end 155 us, cuts at
// 2 K + 16 entries 3 us more, the round's maximum over widened values 2.
#include <float.h>
#include <limits.h>
#include <math.h>

#include "common.cuh"

namespace specv {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;          // 16-byte loads of a thread per round
constexpr int kCap = 2048;        // list entries
constexpr int kSlack = 8;         // entries beyond K that cut the list to K
constexpr int kCheck = 4;         // most rounds between two looks at the list
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
};

// The sums of a warp's lanes, in every lane.
__device__ __forceinline__ Stats warp_total(Stats v, float c) {
    const float to = warp_max(v.m);
    if (v.m < to) v.rebase(to, c);
    v.m = to;
    v.l = warp_sum(v.l);
    v.a = warp_sum(v.a);
    return v;
}

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

// Largest element of N vectors.  (bf16: in pairs as they lie, so that the values need not be
// widened for it)
template <typename T, int N> __device__ __forceinline__ float max_of(const uint4 (&r)[N]) {
    auto two = [](uint32_t a, uint32_t b) {
        uint32_t m;
        if constexpr (sizeof(T) == 4) m = __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
        else asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
        return m;
    };
    uint32_t m = two(two(r[0].x, r[0].y), two(r[0].z, r[0].w));
#pragma unroll
    for (int u = 1; u < N; ++u) m = two(m, two(two(r[u].x, r[u].y), two(r[u].z, r[u].w)));
    return sizeof(T) == 4 ? __uint_as_float(m)
                          : fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}

// Vector v of a row: elements v * EPV - off .. of [0, V), -inf outside and for v >= end.
// The vectors lie on the 16-byte grid of memory; one that is not whole is read element by
// element, so nothing outside the row is.
template <typename T>
__device__ __forceinline__ uint4 load_edge(const T* row, int V, int off, int v, int end) {
    constexpr int EPV = per_vec<T>(), EPW = EPV / 4;
    const int64_t e = (int64_t)v * EPV - off;
    if (v < end && e >= 0 && e + EPV <= V) return __ldg(reinterpret_cast<const uint4*>(row + e));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll 1
    for (int i = 0; i < EPV; ++i) {
        const T x = v < end && e + i >= 0 && e + i < V ? row[e + i] : Elem<T>::from_f32(-INFINITY);
        uint32_t bits;
        if constexpr (sizeof(T) == 4) bits = __float_as_uint(x);
        else bits = (uint32_t)__bfloat16_as_ushort(x) << (16 * (i & 1));
        const int j = i / EPW;
        w[0] |= j == 0 ? bits : 0;
        w[1] |= j == 1 ? bits : 0;
        w[2] |= j == 2 ? bits : 0;
        w[3] |= j == 3 ? bits : 0;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

struct Shared {
    float v[kCap];
    int i[kCap];
    alignas(16) float tv[kThreads];  // maxima of the groups or threads
    int ti[kThreads];
    float best_v[32];
    int best_i[32];
    float4 stats[kThreads / 32];
    float bound_v;
    int bound_i;
    int count, last;
};

// Ranks the first `count` entries of the list and leaves its K best, sorted, at
// the front (every thread calls it; the list is complete and visible).
__device__ __forceinline__ int cut(Shared& s, int count, int K) {
    const int tid = threadIdx.x;
#pragma unroll 1
    for (int e = tid; e < count; e += kThreads) {
        const float v = s.v[e];
        const int i = s.i[e];
        int rank = 0;
#pragma unroll 4
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

// Appends the elements of a thread's round (vectors cur, elements from `first` on) that
// exceed `above` (ABOVE), reach bv (REACH), or both, an equal of bv at index bx at the
// latest (BOTH).  Most calls find one element: a vector whose maximum is too small is not
// looked into.
enum { ABOVE, REACH, BOTH };
template <typename T, int HOW>
__device__ __forceinline__ void append(Shared& s, const uint4 (&cur)[kVecs], int first, float above,
                                       float bv, int bx) {
    constexpr int EPV = per_vec<T>(), EPW = EPV / 4;  // elements of a vector, of a word
    const float least = HOW == ABOVE ? above : bv;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
        const uint4 one[1] = {cur[u]};
        const float vm = max_of<T>(one);
        if (HOW == ABOVE ? !(vm > least) : !(vm >= least)) continue;
        float e[EPV];
        widen<T>(cur[u], e);
        const int at = first + u * kThreads * EPV;
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < EPV; ++j)
            bits |= (uint32_t)(HOW == ABOVE   ? e[j] > above
                               : HOW == REACH ? e[j] >= bv
                                              : e[j] > above && !better(bv, bx, e[j], at + j))
                    << j;
#pragma unroll 1
        for (; bits; bits &= bits - 1) {
            const int j = __ffs(bits) - 1, q = j / EPW;
            const uint32_t w = q == 0 ? cur[u].x : q == 1 ? cur[u].y : q == 2 ? cur[u].z : cur[u].w;
            const int place = atomicAdd(&s.count, 1);
            if (place < kCap) {
                s.v[place] = __uint_as_float(EPW == 1 ? w : j & 1 ? w & 0xffff0000u : w << 16);
                s.i[place] = at + j;
            }
        }
    }
}

// Index of the first element of a thread's round that equals v.
template <typename T>
__device__ __forceinline__ int index_of(uint4 c0, uint4 c1, uint4 c2, uint4 c3, int first, float v) {
    constexpr int EPV = per_vec<T>(), EPW = EPV / 4;
#pragma unroll 1
    for (int e = 0; e < kVecs * EPV; ++e) {
        const int u = e / EPV, j = e % EPV / EPW, h = e % EPW;
        const uint4 r = u == 0 ? c0 : u == 1 ? c1 : u == 2 ? c2 : c3;
        const uint32_t w = j == 0 ? r.x : j == 1 ? r.y : j == 2 ? r.z : r.w;
        if (__uint_as_float(EPW == 1 ? w : h ? w & 0xffff0000u : w << 16) == v)
            return first + u * kThreads * EPV + e % EPV;
    }
    return INT_MAX;
}

// What is written for a row: stats complete, the sorted alternatives in s.  (fp32: on this
// GPU a 64-bit logarithm by every warp took longer than the row.)
template <typename T>
__device__ __forceinline__ void write_row(const LogprobArgs& a, Shared& s, const Stats& st, int64_t row,
                                          float token, int found) {
    const int tid = threadIdx.x;
    if (tid >= 32) return;
    const bool none = st.l == 0.f;  // every logit is -inf
    const float lnl = logf(st.l);
    // z - lse = (x - m) / T - ln l, from the difference on
    auto lp = [&](float x) { return none ? -INFINITY : (x - st.m) * a.inv_t - lnl; };
    if (tid == 0) {
        a.logprob[row] = lp(token);
        if (a.entropy) a.entropy[row] = none ? 0.f : lnl - 0.69314718055994530942f * (st.a / st.l);
    }
    if (tid < a.K) {
        const bool have = tid < found;
        if (a.top_ids) a.top_ids[row * a.K + tid] = have ? s.i[tid] : -1;
        if (a.top_logprobs) a.top_logprobs[row * a.K + tid] = have ? lp(s.v[tid]) : -INFINITY;
    }
}

// The K-th largest of the maxima of 64 groups of four threads (bm: a thread's), which K
// elements reach; -inf if there are fewer.
__device__ __forceinline__ float bound_of_groups(Shared& s, float bm, int K) {
    const int tid = threadIdx.x;
    float g = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
    g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
    if ((tid & 3) == 0) s.tv[tid >> 2] = g;
    __syncthreads();
    if (tid < 64) {
        const float mine = s.tv[tid];
        int rank = 0;
#pragma unroll 4
        for (int o = 0; o < 64; o += 4) {
            const float4 q = *reinterpret_cast<const float4*>(&s.tv[o]);
            rank += (q.x > mine || (q.x == mine && o < tid)) + (q.y > mine || (q.y == mine && o + 1 < tid)) +
                    (q.z > mine || (q.z == mine && o + 2 < tid)) +
                    (q.w > mine || (q.w == mine && o + 3 < tid));
        }
        if (rank == K - 1) s.bound_v = mine;
    }
    __syncthreads();
    return s.bound_v;
}

template <typename T, bool TOP, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) logprob_kernel(const LogprobArgs a) {
    constexpr int EPV = per_vec<T>();
    __shared__ Shared s;
    const int tid = threadIdx.x, S = a.parts, K = a.K;
    const int row = blockIdx.x / (uint32_t)S, part = blockIdx.x - row * S;
    if (tid == 0) {
        s.count = 0;
        s.bound_v = -INFINITY;
    }
    grid_dep_launch_dependents();
    grid_dep_wait();
    if (a.lens) {
        const int b = (uint32_t)row / (uint32_t)a.n;
        if (row - b * a.n >= __ldg(a.lens + b)) return;
    }

    const T* x = static_cast<const T*>(a.logits) + (int64_t)row * a.V;
    // vectors of 16 bytes on memory's grid (indexes inside a row are 32-bit)
    const int V = (int)a.V, off = (int)(((uint64_t)row * (uint64_t)a.V) % EPV);
    constexpr int kRound = kVecs * kThreads;
    const int vecs = (int)(((int64_t)V + off + EPV - 1) / EPV);
    const int per = S == 1 ? vecs : a.part_rounds * kRound;
    const int v0 = part * per, v1 = part == S - 1 ? vecs : v0 + per;
    const float c = a.c;
    uint64_t l2 = f2(0.f, 0.f), a2 = l2;
    float m = -INFINITY;
    // what an element has to exceed: K elements of the rounds before reach it
    float tau = -INFINITY;
    int checked = v0;  // first vector of the rounds since the list was looked at

    uint4 cur[kVecs], nxt[kVecs];
    // (of a round that lies whole inside the row no vector is looked at singly)
    auto fetch = [&](uint4 (&r)[kVecs], int v) {
        if (v + kVecs * kThreads <= v1 && (v > 0 || off == 0) && (int64_t)(v + kVecs * kThreads) * EPV - off <= V) {
            const uint4* p = reinterpret_cast<const uint4*>(x - off) + v + tid;
#pragma unroll
            for (int u = 0; u < kVecs; ++u)
                asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(r[u].x), "=r"(r[u].y), "=r"(r[u].z), "=r"(r[u].w)
                             : "l"(p + u * kThreads));
        } else {
#pragma unroll
            for (int u = 0; u < kVecs; ++u)
                r[u] = load_edge<T>(x, V, off, v + u * kThreads + tid, v1);
        }
    };
    // the given token and, once it is known, its logit (thread 0)
    const int tok = tid == 0 ? __ldg(a.tokens + row) : 0;
    float token = -INFINITY;
    fetch(cur, v0);
#pragma unroll 1
    for (int v = v0; v < v1; v += kVecs * kThreads) {
        if (v + kVecs * kThreads < v1) fetch(nxt, v + kVecs * kThreads);
        const float bm = max_of<T>(cur);
        if (bm > m) {
            float p, q;
            Stats old;
            old.m = m;
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
        if (v == v0 && tid == 0) {
            if (tok >= 0 && tok < V) token = Elem<T>::to_f32(x[tok]);
            else if (part == 0) raise_device_error(a.dev_err, SPEC_DEVERR_TOKEN);
        }
        if (TOP) {
            const int at = (v + tid) * EPV - off;
            if (v == v0) {
                const float bv = bound_of_groups(s, bm, K);
                // (-inf is no alternative)
                if (bm >= bv) append<T, REACH>(s, cur, at, -INFINITY, fmaxf(bv, -FLT_MAX), INT_MAX);
                tau = bv;
            } else if (bm > tau) {
                append<T, ABOVE>(s, cur, at, tau, -INFINITY, INT_MAX);
            }
            const bool end = v + kRound >= v1;
            if (end || v == v0 || v + kRound - checked >= min(kCheck * kRound, checked - v0)) {
                __syncthreads();
                int count = s.count;
                if (count > kCap) {
                    // entries from before (at most K + kSlack) stand in front
                    const int before =
                        v == v0 ? 0 : __syncthreads_count(tid < K + kSlack && s.i[tid] < checked * EPV - off);
                    if (v == v0) tau = -INFINITY;
                    __syncthreads();
                    if (tid == 0) s.count = before;
#pragma unroll 1
                    for (int w = checked; w <= v; w += kRound) {
                        fetch(cur, w);
                        const int first = (w + tid) * EPV - off;
                        const float top = max_of<T>(cur);
                        const int bi = index_of<T>(cur[0], cur[1], cur[2], cur[3], first, top);
                        s.tv[tid] = top;
                        s.ti[tid] = bi;
                        if (tid == 0) {
                            s.bound_v = -INFINITY;
                            s.bound_i = INT_MAX;
                        }
                        __syncthreads();
                        int rank = 0;
#pragma unroll 1
                        for (int o = 0; o < kThreads; ++o) rank += better(s.tv[o], s.ti[o], top, bi);
                        if (rank == K - 1 && top > -INFINITY) {
                            s.bound_v = top;
                            s.bound_i = bi;
                        }
                        __syncthreads();
                        append<T, BOTH>(s, cur, first, tau, s.bound_v, s.bound_i);
                        __syncthreads();
                        count = s.count;
                        cut(s, count, K);
                        if (count >= K) tau = s.v[K - 1];
                        __syncthreads();
                    }
                } else if (count > K + kSlack && !end) {
                    cut(s, count, K);
                    tau = s.v[K - 1];
                    __syncthreads();  // before the next round appends
                }
                checked = v + kRound;
            }
        }
#pragma unroll
        for (int u = 0; u < kVecs; ++u) cur[u] = nxt[u];
    }
    Stats st;
    st.m = m;
    {
        float p, q;
        f2_split(l2, p, q);
        st.l = p + q;
        f2_split(a2, p, q);
        st.a = p + q;
    }
    // the CTA's sums
    st = warp_total(st, c);
    if ((tid & 31) == 0) s.stats[tid >> 5] = make_float4(st.m, st.l, st.a, 0.f);
    __syncthreads();
    // sums in `from` of n parts (a warp: all that is needed further on)
    auto gather = [&](const float4* from, int n) {
        Stats sum;
        if ((tid & 31) < n) {
            const float4 r = __ldcg(from + (tid & 31));
            sum.m = r.x;
            sum.l = r.y;
            sum.a = r.z;
        }
        return warp_total(sum, c);
    };
    if (tid < 32) {
        const float4 r = tid < kThreads / 32 ? s.stats[tid] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        st.m = r.x;
        st.l = r.y;
        st.a = r.z;
        st = warp_total(st, c);
    }
    int found = 0;
    if (TOP) found = cut(s, s.count, K);
    if (S > 1) {
        // ---- parts: leave this one's record; the last CTA of the row merges them
        const int64_t rec = (int64_t)row * S + part;
        if (TOP && tid < K) {
            a.part_v[rec * K + tid] = tid < found ? s.v[tid] : -INFINITY;
            a.part_i[rec * K + tid] = tid < found ? s.i[tid] : -1;
        }
        if (tid == 0) reinterpret_cast<float4*>(a.part_stats)[rec] = make_float4(st.m, st.l, st.a, 0.f);
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
        // the parts' alternatives, up to four a thread, through a bound of their own
        constexpr int kMine = kMaxParts * 32 / kThreads;
        float w[kMine], bm = -INFINITY;
        int id[kMine];
        if (TOP) {
#pragma unroll
            for (int u = 0; u < kMine; ++u) {
                const int e = u * kThreads + tid;
                w[u] = -INFINITY;
                if (e < S * K) {
                    w[u] = __ldcg(a.part_v + (int64_t)row * S * K + e);
                    id[u] = __ldcg(a.part_i + (int64_t)row * S * K + e);
                }
                bm = fmaxf(bm, w[u]);
            }
        }
        if (tid < 32) st = gather(reinterpret_cast<const float4*>(a.part_stats) + (int64_t)row * S, S);
        if (TOP) {
            if (tid == 0) s.bound_v = -INFINITY;
            const float bv = bound_of_groups(s, bm, K);
#pragma unroll
            for (int u = 0; u < kMine; ++u)
                if (w[u] >= bv && w[u] > -INFINITY) {
                    const int place = atomicAdd(&s.count, 1);
                    s.v[place] = w[u];
                    s.i[place] = id[u];
                }
            __syncthreads();
            found = cut(s, s.count, K);
        }
    }
    write_row<T>(a, s, st, row, token, found);
}

}  // namespace

// Rounds that a row takes at least (one more where it begins inside a vector).
static int64_t rounds_of(const LogprobArgs& a) {
    const int64_t round = kThreads * kVecs * (a.dtype == SPEC_DTYPE_F32 ? 4 : 8);
    return (a.V + round - 1) / round;
}

// Parts of a row: four CTAs an SM where the rows alone are fewer, each of whole rounds and
// as many as the others but for the last.
int logprob_parts(const LogprobArgs& a, int num_sms, int max_tickets) {
    const int64_t rows = (int64_t)a.B * a.n, most = rounds_of(a);
    const int64_t want = (4 * (int64_t)num_sms + rows - 1) / rows;
    if (rows > max_tickets) return 1;
    int64_t s = want < most ? want : most;
    if (s > kMaxParts) s = kMaxParts;
    const int64_t rounds = (most + s - 1) / s;
    return (int)((most + rounds - 1) / rounds);
}

size_t logprob_workspace_bytes(const LogprobArgs& a) {
    return a.parts > 1 ? (size_t)a.B * a.n * a.parts * (16 + 8 * (size_t)a.K) : 0;
}

cudaError_t launch_logprobs(LogprobArgs a, void* workspace, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.B * a.n;
    // (parts - 1) part_rounds < rounds_of(a): no part is empty
    a.part_rounds = (int)((rounds_of(a) + a.parts - 1) / a.parts);
    a.part_stats = static_cast<float*>(workspace);
    a.part_v = a.part_stats + rows * a.parts * 4;
    a.part_i = reinterpret_cast<int32_t*>(a.part_v + rows * a.parts * a.K);
    const dim3 grid((unsigned)(rows * a.parts)), block(kThreads);
    // CTAs of an SM: four (64 registers) hide more of the loads.  Rows in parts with
    // alternatives are faster with three: fewer of the given rows may be in use, and four
    // of those on one SM are what the others wait for.  2048 rows of 152064, 5 alternatives:
    // 132 us with four, 143 with three; 32 x up to 5 rows of 128256, 20 alternatives: 23.2, 20.4.
    const bool f32 = a.dtype == SPEC_DTYPE_F32, three = a.K && !f32 && a.parts > 1;
    auto* kern = f32 ? (a.K ? logprob_kernel<float, true, 4> : logprob_kernel<float, false, 4>)
                 : three ? logprob_kernel<__nv_bfloat16, true, 3>
                 : a.K   ? logprob_kernel<__nv_bfloat16, true, 4>
                         : logprob_kernel<__nv_bfloat16, false, 4>;
    return launch_dependent(kern, grid, block, 0, stream, a);
}

}  // namespace specv
