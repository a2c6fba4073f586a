// Internal launch interface between the C-ABI shim (spec_abi.cu) and the
// kernel translation units.  Host-visible only; no torch types anywhere.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "spec_verify.h"

namespace specv {

// Geometry and pointers of one verification-attention call.
struct AttnArgs {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const uint16_t* k_scale;  // fp16 bits, INT8 caches only
    const uint16_t* v_scale;
    const int32_t* block_table;
    const int32_t* ctx_lens;
    int32_t B, k, Hq, Hkv, D, P, num_pages, max_pages;
    int32_t q_dtype, kv_dtype;
    float scale;
    void* out;
    float* lse;
    int* dev_err;       // device error word
    int* seg_counters;  // [B*Hkv] zeroed arrival counters (fused split-KV merge)
    // [B, k] draft-visibility bits (bit t of row i: query i sees draft t), or
    // null for the causal chain (bits 0..i)
    const uint64_t* tree_mask;
    // tensor-core kernels: tiles charged per segment when the tile list is
    // split over the persistent CTAs (TileSplit); < 0 = the kernel's default
    int32_t split_alpha = -1;
    // sliding window (0 = none): a key before the drafts is visible to query i
    // when it is one of the first `sinks` or lies less than `window` positions
    // before the query (see window_low)
    int32_t window = 0, sinks = 0;
    // e4m3 cache: fp32 scales per (page, kv-head), [num_pages, Hkv]
    const float* k_page_scale = nullptr;
    const float* v_page_scale = nullptr;
};

// Draft bits visible to query i of sequence b: the tree row's first k (further
// bits name no draft: they must not count into its depth), or the causal chain.
__host__ __device__ inline uint64_t draft_bits(const AttnArgs& a, int b, int i) {
#ifdef __CUDA_ARCH__
    if (a.tree_mask) return __ldg(a.tree_mask + (int64_t)b * a.k + i) & (~0ull >> (64 - a.k));
#else
    if (a.tree_mask) return a.tree_mask[(int64_t)b * a.k + i] & (~0ull >> (64 - a.k));
#endif
    return i >= 63 ? ~0ull : ((1ull << (i + 1)) - 1);
}

// Ancestors of a query among the drafts: its position is ctx + depth.
__host__ __device__ inline int draft_depth(uint64_t bits) {
#ifdef __CUDA_ARCH__
    const int n = __popcll(bits);
#else
    const int n = __builtin_popcountll(bits);
#endif
    return n > 0 ? n - 1 : 0;
}

// First key that the window of a query at position pos reaches (0 without a window).
__host__ __device__ inline int window_low(const AttnArgs& a, int pos) {
    return a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
}

// Draft bits of query i at context ctx with the window applied to a chain (a
// tree's window covers all its nodes: the entry point refuses a narrower one).
__host__ __device__ inline uint64_t window_bits(const AttnArgs& a, uint64_t bits, int i, int ctx) {
    if (a.window <= 0 || a.tree_mask || i < a.window) return bits;
    uint64_t near = ~0ull << (i - a.window + 1);
    if (a.sinks > ctx) near |= a.sinks - ctx >= 64 ? ~0ull : (1ull << (a.sinks - ctx)) - 1;
    return bits & near;
}

// The keys that no query of a sequence sees, between its sinks and the first
// query's window, are skipped in whole units (tiles of a kernel): a sequence
// of L keys is the units [0, head) and [head + skip, ceil(L / unit)).
struct WindowSpan {
    int head, skip;
};
__host__ __device__ inline WindowSpan window_span(const AttnArgs& a, int ctx, int unit) {
    WindowSpan w;
    const int low = window_low(a, ctx);
    w.head = (int)(((int64_t)(a.sinks < low ? a.sinks : low) + unit - 1) / unit);
    w.skip = low / unit - w.head;
    if (w.skip < 0) w.skip = 0;
    return w;
}

// ---- SIMT kernel (CUDA cores; any supported dtype / shape) ----
struct SimtPlan {
    int32_t chunk;       // keys per split chunk (multiple of 16)
    int32_t max_chunks;  // chunks per sequence at the longest possible context
    int32_t row_groups;  // query-row groups per (sequence, kv-head)
    int32_t rows_per_group;
};
SimtPlan simt_plan(const AttnArgs& a, int num_sms, int forced_chunk);
size_t simt_workspace_bytes(const AttnArgs& a, const SimtPlan& p);
cudaError_t launch_attn_simt(const AttnArgs& a, const SimtPlan& p, void* workspace,
                             cudaStream_t stream);

// ---- single-pass SIMT kernel for short contexts (one launch, no split) ----
// Longest context it holds (the whole block table of a sequence), or 0 when
// the call does not fit its shared-memory plan.
int small_attn_max_keys(const AttnArgs& a);
// CTAs (one cluster) per (sequence, kv-head, row group) the automatic choice takes.
int small_attn_cluster_size(const AttnArgs& a, int num_sms);
// `cluster` = CTAs per unit, 1..8, or 0 for the automatic choice (which falls
// back to one CTA when the device cannot place the cluster; a forced size
// returns the launch error instead).
cudaError_t launch_attn_small(const AttnArgs& a, int num_sms, int cluster, cudaStream_t stream);

// ---- tensor-core kernel (tcgen05 + TMA, persistent, split-KV stream-K) ----
bool tc_supported(const AttnArgs& a);
size_t tc_workspace_bytes(const AttnArgs& a, int num_ctas);
cudaError_t launch_attn_tc(const AttnArgs& a, int num_ctas, void* workspace, cudaStream_t stream);

// Merge of the split-KV partials written by a tensor-core kernel (its tiles
// over `num_ctas` persistent CTAs, split by TileSplit with `alpha` tiles
// charged per segment; partial slots [2*C][128][D]; per CTA boundary the
// segment record {b, kv-head, tile-in-segment, tiles} and the CTA's first
// tile; per sequence the tile prefix, in the kernel's tile units).
cudaError_t launch_combine_stream_k(const AttnArgs& a, int num_ctas, int alpha,
                                    const float* part_o, const float* part_lse,
                                    const int4* seg_rec, const int* seg_pre, cudaStream_t stream);

// ---- tensor-core kernel with 128-key tiles: bf16, head_dim 128, up to 128
// query rows per kv-head (two softmax sets); workspace as tc_workspace_bytes ----
bool tc2_supported(const AttnArgs& a);
cudaError_t launch_attn_tc2(const AttnArgs& a, int num_ctas, void* workspace, cudaStream_t stream);

// Most units that a segment's keys can fill, by the block table's width and the
// window: the host does not know the lengths, so a call without a window of short
// sequences in a wide table counts as one of long segments.
inline int64_t max_units(const AttnArgs& a, int unit) {
    const int64_t all = ((int64_t)a.max_pages * a.P + unit - 1) / unit;
    if (a.window <= 0) return all;
    const int64_t seen = ((int64_t)a.sinks + unit - 1) / unit +
                         ((int64_t)a.window + a.k + unit - 2) / unit + 1;
    return all < seen ? all : seen;
}

// How a call of short segments goes without cutting any (and so without the
// combine): cutting costs a launch, the partials and a piece's end, `worth` tiles'
// time together.
//  * kOwnCta: as many segments as CTAs or fewer, a CTA each.  A segment of t tiles
//    then takes t (1 - segments / CTAs) tiles' time longer than its share.  Past 12
//    tiles unequal lengths outweigh it.
//  * kRounded: more segments; the CTAs' ranges end at the segment's end nearest to
//    an even split, up to a segment away from it at both ends together.  Worth it up
//    to `base` tiles per segment and `more` / 4 for every segment that a CTA takes.
enum { kCut, kOwnCta, kRounded };
inline int whole_segments(const AttnArgs& a, int num_ctas, int unit, int worth, int base,
                          int more) {
    const int64_t segs = (int64_t)a.B * a.Hkv, t = max_units(a, unit);
    if (segs > num_ctas)
        return (t - base) * 4 * num_ctas <= (int64_t)more * segs ? kRounded : kCut;
    return t <= 12 && t * (num_ctas - segs) <= (int64_t)worth * num_ctas ? kOwnCta : kCut;
}

// ---- tensor-core kernel over an e4m3 cache (codes fed to the MMAs as stored;
// same shapes as the 128-key bf16 kernel); workspace as tc_workspace_bytes ----
bool f8_supported(const AttnArgs& a);
cudaError_t launch_attn_f8(const AttnArgs& a, int num_ctas, void* workspace, cudaStream_t stream);

// ---- tensor-core kernel for groups of sequences that share a prefix (bf16, i8
// or e4m3 cache), and the launch that joins its pieces ----
bool shared_supported(const AttnArgs& a, int groups);
bool shared_pays(const AttnArgs& a, int groups, int sms);
size_t shared_workspace_bytes(const AttnArgs& a, int groups, int num_ctas);
cudaError_t launch_attn_shared(const AttnArgs& a, const int32_t* group_starts,
                               const int32_t* shared_lens, int groups, int num_ctas, void* workspace,
                               cudaStream_t stream);

// ---- warp-MMA kernel for k*G <= 16 query rows (mma.sync m16n8k16, TMA pages) ----
bool mma_supported(const AttnArgs& a);
cudaError_t launch_attn_mma(const AttnArgs& a, int num_ctas, void* workspace, cudaStream_t stream);

// ---- greedy acceptance ----
struct AcceptArgs {
    const void* logits;
    int32_t dtype;
    const int32_t* draft;
    int32_t B, k;
    int64_t V;
    int32_t* accepted_len;
    int32_t* next_token;
    // tree acceptance (null for the chain rule): parent [B, k] in [-1, i),
    // accepted node path [B, k] (-1 padded; may be null), device error word
    const int32_t* parent = nullptr;
    int32_t* path = nullptr;
    int* dev_err = nullptr;
};
size_t accept_workspace_bytes(const AcceptArgs& a);
// `tickets` must hold B zeroed int32 (self-resetting across calls).
cudaError_t launch_accept(const AcceptArgs& a, void* workspace, int32_t* tickets,
                          cudaStream_t stream);

// ---- rejection-sampling acceptance (two launches; see accept_rejection.cu) ----
size_t rejection_workspace_bytes(int B, int k, int64_t V);
// `tickets` must hold B zeroed int32 (self-resetting across calls).
cudaError_t launch_accept_rejection(const void* target, const void* draft, int32_t dtype,
                                    const int32_t* draft_tokens, int B, int k, int64_t V,
                                    float temperature, uint64_t seed, int32_t* accepted_len,
                                    int32_t* next_token, void* workspace, int32_t* tickets,
                                    int* dev_err, cudaStream_t stream);

// ---- drafts' K/V append (INT8 quantisation) and the commit ----
cudaError_t launch_kv_append(const void* k_new, const void* v_new, int32_t src_dtype,
                             void* k_cache, void* v_cache, uint16_t* k_scale, uint16_t* v_scale,
                             int32_t cache_dtype, const int32_t* block_table,
                             const int32_t* ctx_lens, int B, int n, int Hkv, int D, int P,
                             int num_pages, int max_pages, int* dev_err, cudaStream_t stream);
// ---- delta + run-length page codec (codec.cu) ----
size_t codec_decode_smem(int P, int D);
cudaError_t launch_codec_encode(const void* codes, int64_t nblk, int P, int D, void* pairs,
                                int32_t* npairs, cudaStream_t stream);
cudaError_t launch_codec_decode(const void* pairs, const int32_t* npairs, int64_t nblk, int P,
                                int D, void* codes, int* dev_err, cudaStream_t stream);

// ---- rotary positions with the append (rope_append.cu) ----
struct RopeAppendArgs {
    const void* q;  // null when Hq = 0
    const void* k_new;
    const void* v_new;
    void* q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements between tokens
    int32_t src_dtype;
    void* k_cache;
    void* v_cache;
    void* k_scale;  // fp16 per (page, kv-head, slot) for i8, fp32 per (page, kv-head) for e4m3
    void* v_scale;
    int32_t cache_dtype;
    const int32_t* block_table;
    const int32_t* ctx_lens;
    const int32_t* positions;  // [B, n] or null: ctx + t
    const int32_t* new_lens;   // [B] or null: n
    const uint64_t* table;     // [rot / 2] 64-bit fractions of a turn per position
    int32_t rot, interleaved;
    float amplitude;
    int32_t B, n, Hq, Hkv, D, P, num_pages, max_pages;
    int* dev_err;
};
cudaError_t launch_rope_append(const RopeAppendArgs& a, int num_sms, cudaStream_t stream);

// ---- the cache read back (kv_gather.cu) ----
struct GatherArgs {
    const void* k_cache;
    const void* v_cache;
    const void* k_scale;
    const void* v_scale;
    int32_t cache_dtype;
    const int32_t* block_table;
    const int32_t* starts;  // [B] or null: 0
    const int32_t* lens;
    void* k_out;
    void* v_out;
    int32_t out_dtype;
    int32_t B, max_len, Hkv, D, P, num_pages, max_pages;
    int* dev_err;
};
cudaError_t launch_kv_gather(const GatherArgs& a, cudaStream_t stream);

// ---- log probabilities, entropy, top alternatives (logprobs.cu) ----
struct LogprobArgs {
    const void* logits;
    int32_t dtype;
    const int32_t* tokens;
    const int32_t* lens;  // [B] or null: n
    int32_t B, n;
    int64_t V;
    float inv_t;  // 1 / temperature
    float c;      // log2(e) / temperature
    int32_t K;
    float* logprob;
    float* entropy;       // or null
    int32_t* top_ids;     // [B, n, K] or null
    float* top_logprobs;  // [B, n, K] or null
    int32_t parts = 1;    // CTAs of a row (logprob_parts)
    int32_t part_rounds;  // rounds of loads of each
    int32_t* tickets;     // [B * n] zeroed when parts > 1 (self-resetting)
    float* part_stats;    // workspace
    float* part_v;
    int32_t* part_i;
    int* dev_err;
};
int logprob_parts(const LogprobArgs& a, int num_sms, int max_tickets);
size_t logprob_workspace_bytes(const LogprobArgs& a);
cudaError_t launch_logprobs(LogprobArgs a, int num_sms, void* workspace, cudaStream_t stream);

// ---- pages held by several rows, and the accepted path of a tree (kv_pages.cu) ----
struct ForkArgs {
    void* k_cache;
    void* v_cache;
    void* k_scale;
    void* v_scale;
    int32_t cache_dtype, elem;  // bytes of an element
    int32_t* block_table;
    int32_t* ctx_lens;
    int32_t* page_refs;
    const int32_t* parents;
    const int32_t* children;
    int32_t n, room, rows, Hkv, D, P, num_pages, max_pages;
    uint32_t* free_bits;  // workspace
    uint32_t* one_bits;
    int32_t* free_count;
    int32_t* need;
    int32_t* src;
    int* dev_err;
};
size_t fork_workspace_bytes(int num_pages, int n);
cudaError_t launch_kv_fork(ForkArgs a, void* workspace, cudaStream_t stream);

struct ReleaseArgs {
    int32_t* block_table;
    int32_t* ctx_lens;
    int32_t* page_refs;
    const int32_t* rows;
    const int32_t* keep_lens;  // [n] or null: 0
    int32_t n, batch, P, num_pages, max_pages;
    int* dev_err;
};
cudaError_t launch_kv_release(const ReleaseArgs& a, cudaStream_t stream);

struct CompactArgs {
    void* k_cache;
    void* v_cache;
    void* k_scale;
    void* v_scale;
    int32_t cache_dtype, elem;
    const int32_t* block_table;
    const int32_t* ctx_lens;
    const int32_t* path;
    const int32_t* accepted;
    int32_t B, k, Hkv, D, P, num_pages, max_pages;
    int* dev_err;
};
cudaError_t launch_kv_compact(const CompactArgs& a, cudaStream_t stream);

cudaError_t launch_commit(int32_t* ctx_lens, const int32_t* accepted_len, int B, int extra,
                          cudaStream_t stream);

// Sets the thread-local error message of the C ABI; returns `code`.
int set_error(int code, const char* msg);

}  // namespace specv
