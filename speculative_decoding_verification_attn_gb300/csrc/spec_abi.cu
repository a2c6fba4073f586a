// C ABI of the verification hot path: argument validation, the per-device
// workspace, path selection and launches on the caller's stream.  Every
// entry point returns a status code; on an error nothing is enqueued and the
// thread-local message says why.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <atomic>
#include <initializer_list>
#include <mutex>
#include <string>
#include <vector>

#include "kernels.h"
#include "workspace.h"

namespace {

thread_local std::string g_err;

int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_err = buf;
    return code;
}

int cuda_fail(cudaError_t e, const char* what) {
    return fail(SPEC_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

std::atomic<int64_t> g_opt_path{0}, g_opt_ctas{0}, g_opt_validate{0}, g_opt_simt_chunk{0},
    g_opt_split{0}, g_opt_small_cluster{0};

// Per-device workspace: [error word | acceptance tickets | segment counters |
// scratch].  The header is zeroed at allocation; tickets and counters are
// reset by the kernels that use them.
constexpr size_t kHeader = 128 * 1024;
constexpr size_t kTicketsOff = 256, kCountersOff = 64 * 1024;
constexpr int kMaxTickets = (int)((kCountersOff - kTicketsOff) / 4);
constexpr int kMaxCounters = (int)((kHeader - kCountersOff) / 4);
struct Workspace {
    void* base = nullptr;
    size_t bytes = 0;
    int sms = 0;
    // outgrown buffers: graphs captured before the growth still point into
    // them, so they stay until spec_release
    std::vector<void*> retired;
};
std::mutex g_ws_mu;
std::vector<Workspace> g_ws;

// Returns the current device's workspace with at least `scratch` bytes of
// scratch space (allocating or growing it), or sets an error.
int get_workspace(size_t scratch, cudaStream_t stream, Workspace** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    std::lock_guard<std::mutex> lk(g_ws_mu);
    if ((int)g_ws.size() <= dev) g_ws.resize(dev + 1);
    Workspace& w = g_ws[dev];
    if (w.sms == 0) {
        e = cudaDeviceGetAttribute(&w.sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    }
    const size_t need = kHeader + ((scratch + 255) & ~size_t(255));
    if (w.bytes < need) {
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(stream, &cap) == cudaSuccess &&
            cap != cudaStreamCaptureStatusNone)
            return fail(SPEC_ERR_UNSUPPORTED, "the workspace would grow during a stream capture: "
                        "make one such call before capturing");
        (void)cudaGetLastError();
        try {
            w.retired.reserve(w.retired.size() + 1);
        } catch (...) {
            return fail(SPEC_ERR_CUDA, "out of host memory");
        }
        void* fresh = nullptr;
        const size_t grow = specv::grow_buffer(need, w.bytes, [&](size_t bytes) {
            e = cudaMalloc(&fresh, bytes);
            if (e != cudaSuccess) (void)cudaGetLastError();  // not the next launch's
            return e == cudaSuccess;
        });
        if (!grow) return cuda_fail(e, "cudaMalloc(workspace)");
        e = cudaMemset(fresh, 0, kHeader);
        if (e == cudaSuccess) e = cudaDeviceSynchronize();
        if (e != cudaSuccess) {
            cudaFree(fresh);
            return cuda_fail(e, "cudaMemset(workspace)");
        }
        if (w.base) w.retired.push_back(w.base);
        w.base = fresh;
        w.bytes = grow;
    }
    *out = &w;
    return SPEC_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether the product of sizes >= 1 reaches `limit`; no step of it overflows.
bool reaches(int64_t limit, std::initializer_list<int64_t> sizes) {
    int64_t p = 1;
    for (const int64_t s : sizes) {
        if (p >= (limit + s - 1) / s) return true;
        p *= s;
    }
    return false;
}

int dtype_size(int32_t dt) {
    switch (dt) {
    case SPEC_DTYPE_F32: return 4;
    case SPEC_DTYPE_BF16: return 2;
    case SPEC_DTYPE_F16: return 2;
    case SPEC_DTYPE_I8: return 1;
    case SPEC_DTYPE_E4M3: return 1;
    default: return 0;
    }
}

// Host-side check of block_table / ctx_lens (SPEC_OPT_VALIDATE): of the entries
// that a kernel looks at, which with a window are those of pages that hold a
// sink or a key of the first query's window (or later).
int validate_tables(const specv::AttnArgs& a, cudaStream_t stream) {
    std::vector<int32_t> ctx, bt;
    try {
        ctx.resize(a.B);
        bt.resize((size_t)a.B * a.max_pages);
    } catch (...) {
        return fail(SPEC_ERR_CUDA, "validate: out of host memory");
    }
    cudaError_t e = cudaMemcpyAsync(ctx.data(), a.ctx_lens, sizeof(int32_t) * a.B,
                                    cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess)
        e = cudaMemcpyAsync(bt.data(), a.block_table, sizeof(int32_t) * bt.size(),
                            cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return cuda_fail(e, "validate: copy tables");
    for (int b = 0; b < a.B; ++b) {
        const int64_t L = (int64_t)ctx[b] + a.k;
        if (ctx[b] < 0 || L > (int64_t)a.max_pages * a.P)
            return fail(SPEC_ERR_INVALID, "ctx_lens[%d]=%d: ctx + num_draft exceeds the %d pages "
                        "of the block table", b, ctx[b], a.max_pages);
        const int64_t n = (L + a.P - 1) / a.P, low = specv::window_low(a, ctx[b]);
        for (int64_t p = 0; p < n; ++p) {
            if (p * a.P >= a.sinks && (p + 1) * a.P <= low) continue;  // no query sees it
            const int32_t id = bt[(size_t)b * a.max_pages + p];
            if (id < 0 || id >= a.num_pages)
                return fail(SPEC_ERR_INVALID, "block_table[%d][%lld]=%d outside [0, %d)", b,
                            (long long)p, id, a.num_pages);
        }
    }
    return SPEC_OK;
}

}  // namespace

namespace specv {
// Records `msg` as this thread's last error and returns `code` (for entry
// points defined in other translation units).
int set_error(int code, const char* msg) { return fail(code, "%s", msg); }
}  // namespace specv

extern "C" {

int spec_version(void) { return 100; }

const char* spec_last_error(void) { return g_err.c_str(); }

int spec_set_option(int32_t option, int64_t value) {
    switch (option) {
    case SPEC_OPT_ATTN_PATH:
        if (value < 0 || value > 5)
            return fail(SPEC_ERR_INVALID, "attn path must be 0, 1, 2, 3, 4 or 5");
        g_opt_path = value;
        return SPEC_OK;
    case SPEC_OPT_NUM_CTAS:
        if (value < 0 || value > 65535) return fail(SPEC_ERR_INVALID, "num_ctas out of range");
        g_opt_ctas = value;
        return SPEC_OK;
    case SPEC_OPT_VALIDATE:
        g_opt_validate = value ? 1 : 0;
        return SPEC_OK;
    case SPEC_OPT_SIMT_CHUNK:
        if (value < 0 || value > (1 << 30)) return fail(SPEC_ERR_INVALID, "chunk out of range");
        g_opt_simt_chunk = value;
        return SPEC_OK;
    case SPEC_OPT_SPLIT_WEIGHT:
        if (value < 0 || value > 257) return fail(SPEC_ERR_INVALID, "split weight out of range");
        g_opt_split = value;
        return SPEC_OK;
    case SPEC_OPT_SMALL_CLUSTER:
        if (value < 0 || value > 8) return fail(SPEC_ERR_INVALID, "small cluster must be 0..8");
        g_opt_small_cluster = value;
        return SPEC_OK;
    default:
        return fail(SPEC_ERR_INVALID, "unknown option %d", option);
    }
}

}  // extern "C"

namespace {

// The words of a call's scales: i8 fp16 per (page, kv-head, slot), e4m3 fp32
// per (page, kv-head).
int check_scales(int32_t dtype, const void* k_scale, const void* v_scale) {
    if (dtype == SPEC_DTYPE_I8 && (!k_scale || !v_scale))
        return fail(SPEC_ERR_INVALID, "an I8 cache needs k_scale and v_scale");
    if (dtype == SPEC_DTYPE_E4M3) {
        if (!k_scale || !v_scale)
            return fail(SPEC_ERR_INVALID, "an E4M3 cache needs k_scale and v_scale");
        if ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3)
            return fail(SPEC_ERR_INVALID, "E4M3 scales must be 4-byte aligned");
    }
    return SPEC_OK;
}

int verify_attn_impl(const void* q, const void* k_cache, const void* v_cache, const void* k_scale,
                     const void* v_scale, const int32_t* block_table, const int32_t* ctx_lens,
                     const uint64_t* tree_mask, int32_t batch, int32_t num_draft,
                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                     int32_t page_size, int32_t num_pages, int32_t max_pages_per_seq,
                     int32_t q_dtype, int32_t kv_dtype, float scale, int32_t window,
                     int32_t num_sinks, void* out, float* lse, void* stream,
                     const int32_t* group_starts = nullptr, const int32_t* shared_lens = nullptr,
                     int32_t num_groups = 0) {
    g_err.clear();
    if (batch < 0) return fail(SPEC_ERR_INVALID, "batch < 0");
    if (num_draft < 1 || num_draft > 64) return fail(SPEC_ERR_INVALID, "num_draft must be in [1, 64]");
    if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads)
        return fail(SPEC_ERR_INVALID, "num_q_heads must be a positive multiple of num_kv_heads");
    if (head_dim < 32 || head_dim > 256 || head_dim % 32)
        return fail(SPEC_ERR_INVALID, "head_dim must be a multiple of 32 in [32, 256]");
    if (page_size < 1) return fail(SPEC_ERR_INVALID, "page_size < 1");
    if (num_pages < 1 || max_pages_per_seq < 1)
        return fail(SPEC_ERR_INVALID, "num_pages and max_pages_per_seq must be >= 1");
    if (q_dtype != SPEC_DTYPE_F32 && q_dtype != SPEC_DTYPE_BF16)
        return fail(SPEC_ERR_INVALID, "q_dtype must be F32 or BF16");
    if (kv_dtype != SPEC_DTYPE_F32 && kv_dtype != SPEC_DTYPE_BF16 && kv_dtype != SPEC_DTYPE_I8 &&
        kv_dtype != SPEC_DTYPE_E4M3)
        return fail(SPEC_ERR_INVALID, "kv_dtype must be F32, BF16, I8 or E4M3");
    if (!(scale == scale)) return fail(SPEC_ERR_INVALID, "scale is NaN");
    if (batch == 0) return SPEC_OK;
    // the kernels walk keys 0 .. num_draft - 1 at least, whatever ctx_lens says
    if ((int64_t)max_pages_per_seq * page_size < num_draft)
        return fail(SPEC_ERR_INVALID, "the block table's %d pages of %d do not hold num_draft = %d "
                    "keys", max_pages_per_seq, page_size, num_draft);
    if (!q || !k_cache || !v_cache || !block_table || !ctx_lens || !out)
        return fail(SPEC_ERR_INVALID, "null tensor pointer");
    int rc = check_scales(kv_dtype, k_scale, v_scale);
    if (rc) return rc;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return fail(SPEC_ERR_INVALID, "q, caches and out must be 16-byte aligned");
    if (reaches(1LL << 40, {num_pages, num_kv_heads, page_size, head_dim}))
        return fail(SPEC_ERR_INVALID, "cache too large");
    const int64_t R = (int64_t)num_draft * (num_q_heads / num_kv_heads);
    (void)dtype_size;

    specv::AttnArgs a;
    a.q = q; a.k_cache = k_cache; a.v_cache = v_cache;
    const bool paged = kv_dtype == SPEC_DTYPE_E4M3;  // one fp32 scale per (page, kv-head)
    a.k_scale = paged ? nullptr : static_cast<const uint16_t*>(k_scale);
    a.v_scale = paged ? nullptr : static_cast<const uint16_t*>(v_scale);
    a.k_page_scale = paged ? static_cast<const float*>(k_scale) : nullptr;
    a.v_page_scale = paged ? static_cast<const float*>(v_scale) : nullptr;
    a.window = window; a.sinks = num_sinks;
    a.block_table = block_table; a.ctx_lens = ctx_lens;
    a.B = batch; a.k = num_draft; a.Hq = num_q_heads; a.Hkv = num_kv_heads; a.D = head_dim;
    a.P = page_size; a.num_pages = num_pages; a.max_pages = max_pages_per_seq;
    a.q_dtype = q_dtype; a.kv_dtype = kv_dtype; a.scale = scale;
    a.out = out; a.lse = lse;
    a.dev_err = nullptr; a.seg_counters = nullptr;
    a.tree_mask = tree_mask;
    const int64_t split_opt = g_opt_split.load();
    a.split_alpha = split_opt > 0 ? (int32_t)(split_opt - 1) : -1;
    cudaStream_t st = static_cast<cudaStream_t>(stream);

    Workspace* ws = nullptr;
    rc = get_workspace(0, st, &ws);
    if (rc) return rc;

    // kernels: 1 SIMT (chunked), 2 tcgen05 (64-key tiles), 3 warp MMA,
    // 4 single-pass SIMT, 5 tcgen05 (128-key tiles; an e4m3 cache has a kernel
    // of its own there and takes it wherever the shape fits).  Automatic: a bf16
    // cache with head_dim 128 takes the 128-key tcgen05 kernel, except that
    // with <= 16 query rows per kv-head the warp-MMA kernel (whose pieces of
    // a split segment cost less) keeps the calls with more segments than SMs
    // and tables shorter than 3072 keys (about 24 tiles per segment, the
    // point where the two cross over when measured); the INT8 cache takes
    // the 64-key tcgen05 kernel; every other shape the single-pass SIMT
    // kernel when a whole sequence fits its shared memory, else the chunked one
    const int64_t path = g_opt_path.load();
    const bool win = window > 0;
    const bool tc_ok = specv::tc_supported(a), mma_ok = !win && specv::mma_supported(a);
    const bool f8_ok = specv::f8_supported(a);
    const bool tc2_ok = f8_ok || specv::tc2_supported(a);
    const bool small_ok = !win && specv::small_attn_max_keys(a) > 0;
    // groups with shared prefixes: a tensor-core kernel of its own, where it saves
    // more than it costs or path 5 asks for it (any other forced kernel reads each
    // sequence by itself)
    const bool groups = (path == 0 || path == 5) && specv::shared_supported(a, num_groups) &&
                        (path == 5 || specv::shared_pays(a, num_groups, ws->sms));
    int kernel;
    if (path == 1 || groups) kernel = 1;
    else if (path >= 2) {
        if ((path == 2 && !tc_ok) || (path == 3 && !mma_ok) || (path == 4 && !small_ok) ||
            (path == 5 && !tc2_ok))
            return fail(SPEC_ERR_UNSUPPORTED, "forced attention kernel %d does not support this "
                        "shape/dtype", (int)path);
        kernel = (int)path;
    } else {
        const bool many_short = (int64_t)batch * num_kv_heads > ws->sms &&
                                (int64_t)max_pages_per_seq * page_size < 3072;
        const bool tc2_auto = tc2_ok && kv_dtype != SPEC_DTYPE_I8;
        kernel = mma_ok && (many_short || !tc2_auto) ? 3 : tc2_auto ? 5 : tc_ok ? 2 : small_ok ? 4 : 1;
    }
    if (kernel == 3 && (int64_t)batch * num_kv_heads > kMaxCounters)
        return fail(SPEC_ERR_UNSUPPORTED, "batch * num_kv_heads > %d for the warp-MMA kernel",
                    kMaxCounters);
    const bool use_tc = kernel == 2 || kernel == 3 || kernel == 5;
    if (g_opt_validate.load()) {
        rc = validate_tables(a, st);
        if (rc) return rc;
    }
    cudaError_t e;
    if (groups) {
        int ctas = (int)g_opt_ctas.load();
        if (ctas <= 0) ctas = ws->sms;
        rc = get_workspace(specv::shared_workspace_bytes(a, num_groups, ctas), st, &ws);
        if (rc) return rc;
        a.dev_err = static_cast<int*>(ws->base);
        e = specv::launch_attn_shared(a, group_starts, shared_lens, num_groups, ctas,
                                      static_cast<char*>(ws->base) + kHeader, st);
        if (e != cudaSuccess) return cuda_fail(e, "verify_attn (shared prefixes) launch");
        return SPEC_OK;
    }
    if (use_tc) {
        int ctas = (int)g_opt_ctas.load();
        if (ctas <= 0) ctas = ws->sms;
        rc = get_workspace(specv::tc_workspace_bytes(a, ctas), st, &ws);
        if (rc) return rc;
        a.dev_err = static_cast<int*>(ws->base);
        a.seg_counters = reinterpret_cast<int*>(static_cast<char*>(ws->base) + kCountersOff);
        void* wsp = static_cast<char*>(ws->base) + kHeader;
        e = kernel == 3   ? specv::launch_attn_mma(a, ctas, wsp, st)
            : f8_ok       ? specv::launch_attn_f8(a, ctas, wsp, st)
            : kernel == 5 ? specv::launch_attn_tc2(a, ctas, wsp, st)
                          : specv::launch_attn_tc(a, ctas, wsp, st);
        if (e != cudaSuccess) return cuda_fail(e, "verify_attn (tensor-core) launch");
    } else if (kernel == 4) {
        a.dev_err = static_cast<int*>(ws->base);
        e = specv::launch_attn_small(a, ws->sms, (int)g_opt_small_cluster.load(), st);
        if (e != cudaSuccess) return cuda_fail(e, "verify_attn (single-pass SIMT) launch");
    } else {
        const specv::SimtPlan p = specv::simt_plan(a, ws->sms, (int)g_opt_simt_chunk.load());
        const int64_t gy = (int64_t)batch * num_kv_heads * p.row_groups;
        if (gy > 65535 || R > (1 << 20))
            return fail(SPEC_ERR_UNSUPPORTED, "batch * num_kv_heads too large for the SIMT path");
        rc = get_workspace(specv::simt_workspace_bytes(a, p), st, &ws);
        if (rc) return rc;
        a.dev_err = static_cast<int*>(ws->base);
        e = specv::launch_attn_simt(a, p, static_cast<char*>(ws->base) + kHeader, st);
        if (e != cudaSuccess) return cuda_fail(e, "verify_attn (SIMT) launch");
    }
    return SPEC_OK;
}

}  // namespace

extern "C" {

int spec_verify_attn(const void* q, const void* k_cache, const void* v_cache, const void* k_scale,
                     const void* v_scale, const int32_t* block_table, const int32_t* ctx_lens,
                     int32_t batch, int32_t num_draft, int32_t num_q_heads, int32_t num_kv_heads,
                     int32_t head_dim, int32_t page_size, int32_t num_pages,
                     int32_t max_pages_per_seq, int32_t q_dtype, int32_t kv_dtype, float scale,
                     void* out, float* lse, void* stream) {
    return verify_attn_impl(q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens, nullptr,
                            batch, num_draft, num_q_heads, num_kv_heads, head_dim, page_size,
                            num_pages, max_pages_per_seq, q_dtype, kv_dtype, scale, 0, 0, out,
                            lse, stream);
}

int spec_verify_attn_window(const void* q, const void* k_cache, const void* v_cache,
                            const void* k_scale, const void* v_scale, const int32_t* block_table,
                            const int32_t* ctx_lens, const uint64_t* tree_mask, int32_t batch,
                            int32_t num_draft, int32_t num_q_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t page_size, int32_t num_pages,
                            int32_t max_pages_per_seq, int32_t q_dtype, int32_t kv_dtype,
                            float scale, int32_t window, int32_t num_sinks, void* out, float* lse,
                            void* stream) {
    g_err.clear();
    if (window < 1) return fail(SPEC_ERR_INVALID, "window must be >= 1");
    if (num_sinks < 0) return fail(SPEC_ERR_INVALID, "num_sinks must be >= 0");
    if (tree_mask && window < num_draft)
        return fail(SPEC_ERR_INVALID, "a tree's window must hold all its nodes: window >= num_draft");
    return verify_attn_impl(q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens,
                            tree_mask, batch, num_draft, num_q_heads, num_kv_heads, head_dim,
                            page_size, num_pages, max_pages_per_seq, q_dtype, kv_dtype, scale,
                            window, num_sinks, out, lse, stream);
}

int spec_verify_attn_shared(const void* q, const void* k_cache, const void* v_cache,
                            const void* k_scale, const void* v_scale, const int32_t* block_table,
                            const int32_t* ctx_lens, const uint64_t* tree_mask,
                            const int32_t* group_starts, const int32_t* shared_lens,
                            int32_t num_groups, int32_t batch, int32_t num_draft,
                            int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                            int32_t page_size, int32_t num_pages, int32_t max_pages_per_seq,
                            int32_t q_dtype, int32_t kv_dtype, float scale, void* out, float* lse,
                            void* stream) {
    g_err.clear();
    if (num_groups < 0) return fail(SPEC_ERR_INVALID, "num_groups < 0");
    if (num_groups > 0 && batch > 0 && (!group_starts || !shared_lens))
        return fail(SPEC_ERR_INVALID, "group_starts or shared_lens is NULL");
    return verify_attn_impl(q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens,
                            tree_mask, batch, num_draft, num_q_heads, num_kv_heads, head_dim,
                            page_size, num_pages, max_pages_per_seq, q_dtype, kv_dtype, scale, 0,
                            0, out, lse, stream, group_starts, shared_lens, num_groups);
}

int spec_verify_attn_tree(const void* q, const void* k_cache, const void* v_cache,
                          const void* k_scale, const void* v_scale, const int32_t* block_table,
                          const int32_t* ctx_lens, const uint64_t* tree_mask, int32_t batch,
                          int32_t num_draft, int32_t num_q_heads, int32_t num_kv_heads,
                          int32_t head_dim, int32_t page_size, int32_t num_pages,
                          int32_t max_pages_per_seq, int32_t q_dtype, int32_t kv_dtype,
                          float scale, void* out, float* lse, void* stream) {
    if (batch > 0 && !tree_mask) return fail(SPEC_ERR_INVALID, "tree_mask is NULL");
    return verify_attn_impl(q, k_cache, v_cache, k_scale, v_scale, block_table, ctx_lens,
                            tree_mask, batch, num_draft, num_q_heads, num_kv_heads, head_dim,
                            page_size, num_pages, max_pages_per_seq, q_dtype, kv_dtype, scale,
                            0, 0, out, lse, stream);
}

}  // extern "C"

namespace {

int accept_greedy_impl(const void* logits, int32_t logits_dtype, const int32_t* draft_tokens,
                       const int32_t* parents, int32_t batch, int32_t num_draft, int64_t vocab,
                       int32_t* accepted_len, int32_t* next_token, int32_t* path, void* stream) {
    g_err.clear();
    if (batch < 0) return fail(SPEC_ERR_INVALID, "batch < 0");
    if (num_draft < 1 || num_draft > 64) return fail(SPEC_ERR_INVALID, "num_draft must be in [1, 64]");
    if (vocab < 1 || vocab >= (1LL << 31)) return fail(SPEC_ERR_INVALID, "vocab must be in [1, 2^31)");
    if (logits_dtype != SPEC_DTYPE_F32 && logits_dtype != SPEC_DTYPE_BF16)
        return fail(SPEC_ERR_INVALID, "logits_dtype must be F32 or BF16");
    if (batch == 0) return SPEC_OK;
    if (batch > kMaxTickets) return fail(SPEC_ERR_UNSUPPORTED, "batch > %d", kMaxTickets);
    if (!logits || !draft_tokens || !accepted_len || !next_token)
        return fail(SPEC_ERR_INVALID, "null tensor pointer");
    if (!aligned16(logits)) return fail(SPEC_ERR_INVALID, "logits must be 16-byte aligned");
    specv::AcceptArgs a;
    a.logits = logits; a.dtype = logits_dtype; a.draft = draft_tokens; a.B = batch;
    a.k = num_draft; a.V = vocab; a.accepted_len = accepted_len; a.next_token = next_token;
    a.parent = parents; a.path = path;
    const int64_t blocks = (int64_t)batch * (num_draft + 1) * ((vocab + 8191) / 8192);
    if (blocks >= (1LL << 31)) return fail(SPEC_ERR_UNSUPPORTED, "logits too large");
    Workspace* ws = nullptr;
    int rc = get_workspace(specv::accept_workspace_bytes(a), static_cast<cudaStream_t>(stream),
                           &ws);
    if (rc) return rc;
    a.dev_err = static_cast<int*>(ws->base);
    int32_t* tickets = reinterpret_cast<int32_t*>(static_cast<char*>(ws->base) + kTicketsOff);
    cudaError_t e = specv::launch_accept(a, static_cast<char*>(ws->base) + kHeader, tickets,
                                         static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "accept_greedy launch");
    return SPEC_OK;
}

}  // namespace

extern "C" {

int spec_accept_greedy(const void* logits, int32_t logits_dtype, const int32_t* draft_tokens,
                       int32_t batch, int32_t num_draft, int64_t vocab, int32_t* accepted_len,
                       int32_t* next_token, void* stream) {
    return accept_greedy_impl(logits, logits_dtype, draft_tokens, nullptr, batch, num_draft, vocab,
                              accepted_len, next_token, nullptr, stream);
}

int spec_accept_tree(const void* logits, int32_t logits_dtype, const int32_t* draft_tokens,
                     const int32_t* parents, int32_t batch, int32_t num_draft, int64_t vocab,
                     int32_t* accepted_len, int32_t* next_token, int32_t* path, void* stream) {
    if (batch > 0 && !parents) return fail(SPEC_ERR_INVALID, "parents is NULL");
    return accept_greedy_impl(logits, logits_dtype, draft_tokens, parents, batch, num_draft,
                              vocab, accepted_len, next_token, path, stream);
}

int spec_accept_rejection(const void* target_logits, const void* draft_logits,
                          int32_t logits_dtype, const int32_t* draft_tokens, int32_t batch,
                          int32_t num_draft, int64_t vocab, float temperature, uint64_t seed,
                          int32_t* accepted_len, int32_t* next_token, void* stream) {
    g_err.clear();
    if (batch < 0) return fail(SPEC_ERR_INVALID, "batch < 0");
    if (num_draft < 1 || num_draft > 64) return fail(SPEC_ERR_INVALID, "num_draft must be in [1, 64]");
    if (vocab < 1 || vocab >= (1LL << 31)) return fail(SPEC_ERR_INVALID, "vocab must be in [1, 2^31)");
    if (logits_dtype != SPEC_DTYPE_F32 && logits_dtype != SPEC_DTYPE_BF16)
        return fail(SPEC_ERR_INVALID, "logits_dtype must be F32 or BF16");
    if (!(temperature > 0.f) || !(temperature < INFINITY))
        return fail(SPEC_ERR_INVALID, "temperature must be positive and finite");
    if (batch == 0) return SPEC_OK;
    if (batch > kMaxTickets) return fail(SPEC_ERR_UNSUPPORTED, "batch > %d", kMaxTickets);
    if (!target_logits || !draft_logits || !draft_tokens || !accepted_len || !next_token)
        return fail(SPEC_ERR_INVALID, "null tensor pointer");
    if (!aligned16(target_logits) || !aligned16(draft_logits))
        return fail(SPEC_ERR_INVALID, "logits must be 16-byte aligned");
    const int64_t units = (int64_t)batch * (2 * num_draft + 1) * ((vocab + 2047) / 2048);
    if (units >= (1LL << 31)) return fail(SPEC_ERR_UNSUPPORTED, "logits too large");
    Workspace* ws = nullptr;
    int rc = get_workspace(specv::rejection_workspace_bytes(batch, num_draft, vocab),
                           static_cast<cudaStream_t>(stream), &ws);
    if (rc) return rc;
    int32_t* tickets = reinterpret_cast<int32_t*>(static_cast<char*>(ws->base) + kTicketsOff);
    cudaError_t e = specv::launch_accept_rejection(
        target_logits, draft_logits, logits_dtype, draft_tokens, batch, num_draft, vocab,
        temperature, seed, accepted_len, next_token, static_cast<char*>(ws->base) + kHeader,
        tickets, static_cast<int*>(ws->base), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "accept_rejection launch");
    return SPEC_OK;
}

int spec_kv_append(const void* k_new, const void* v_new, int32_t src_dtype, void* k_cache,
                   void* v_cache, void* k_scale, void* v_scale, int32_t cache_dtype,
                   const int32_t* block_table, const int32_t* ctx_lens, int32_t batch,
                   int32_t num_new, int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                   int32_t num_pages, int32_t max_pages_per_seq, void* stream) {
    g_err.clear();
    if (batch < 0) return fail(SPEC_ERR_INVALID, "batch < 0");
    if (num_new < 1) return fail(SPEC_ERR_INVALID, "num_new must be >= 1");
    if (num_kv_heads < 1) return fail(SPEC_ERR_INVALID, "num_kv_heads must be >= 1");
    if (head_dim < 32 || head_dim > 256 || head_dim % 32)
        return fail(SPEC_ERR_INVALID, "head_dim must be a multiple of 32 in [32, 256]");
    if (page_size < 1) return fail(SPEC_ERR_INVALID, "page_size < 1");
    if (num_pages < 1 || max_pages_per_seq < 1)
        return fail(SPEC_ERR_INVALID, "num_pages and max_pages_per_seq must be >= 1");
    if (src_dtype != SPEC_DTYPE_F32 && src_dtype != SPEC_DTYPE_BF16)
        return fail(SPEC_ERR_INVALID, "src_dtype must be F32 or BF16");
    if (cache_dtype != SPEC_DTYPE_F32 && cache_dtype != SPEC_DTYPE_BF16 &&
        cache_dtype != SPEC_DTYPE_I8 && cache_dtype != SPEC_DTYPE_E4M3)
        return fail(SPEC_ERR_INVALID, "cache_dtype must be F32, BF16, I8 or E4M3");
    if (batch == 0) return SPEC_OK;
    if (!k_new || !v_new || !k_cache || !v_cache || !block_table || !ctx_lens)
        return fail(SPEC_ERR_INVALID, "null tensor pointer");
    int rc = check_scales(cache_dtype, k_scale, v_scale);
    if (rc) return rc;
    if (cache_dtype == SPEC_DTYPE_E4M3) {
        // pages share a scale: the page form of the rotary append, nothing rotated
        const int64_t stride = (int64_t)num_kv_heads * head_dim;
        return spec_rope_append(nullptr, k_new, v_new, nullptr, 0, stride, stride, 0, src_dtype,
                                k_cache, v_cache, k_scale, v_scale, cache_dtype, block_table,
                                ctx_lens, nullptr, nullptr, nullptr, 0, 0, 1.f, batch, num_new, 0,
                                num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq,
                                stream);
    }
    if (reaches(1LL << 33, {batch, num_new, num_kv_heads}))
        return fail(SPEC_ERR_UNSUPPORTED, "too many rows");
    Workspace* ws = nullptr;
    rc = get_workspace(0, static_cast<cudaStream_t>(stream), &ws);
    if (rc) return rc;
    cudaError_t e = specv::launch_kv_append(
        k_new, v_new, src_dtype, k_cache, v_cache, static_cast<uint16_t*>(k_scale),
        static_cast<uint16_t*>(v_scale), cache_dtype, block_table, ctx_lens, batch, num_new,
        num_kv_heads, head_dim, page_size, num_pages, max_pages_per_seq,
        static_cast<int*>(ws->base), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kv_append launch");
    return SPEC_OK;
}

int spec_rope_append(const void* q, const void* k_new, const void* v_new, void* q_out,
                     int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t q_out_stride,
                     int32_t src_dtype, void* k_cache, void* v_cache, void* k_scale, void* v_scale,
                     int32_t cache_dtype, const int32_t* block_table, const int32_t* ctx_lens,
                     const int32_t* positions, const int32_t* new_lens, const uint64_t* rope_table,
                     int32_t rotary_dim, int32_t interleaved, float amplitude, int32_t batch,
                     int32_t num_new, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                     int32_t page_size, int32_t num_pages, int32_t max_pages_per_seq,
                     void* stream) {
    g_err.clear();
    if (batch < 0) return fail(SPEC_ERR_INVALID, "batch < 0");
    if (num_new < 1) return fail(SPEC_ERR_INVALID, "num_new must be >= 1");
    if (num_kv_heads < 1) return fail(SPEC_ERR_INVALID, "num_kv_heads must be >= 1");
    if (num_q_heads < 0) return fail(SPEC_ERR_INVALID, "num_q_heads must be >= 0");
    if (head_dim < 32 || head_dim > 256 || head_dim % 32)
        return fail(SPEC_ERR_INVALID, "head_dim must be a multiple of 32 in [32, 256]");
    if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 16)
        return fail(SPEC_ERR_INVALID, "rotary_dim must be a multiple of 16 in [0, head_dim]");
    if (page_size < 1) return fail(SPEC_ERR_INVALID, "page_size < 1");
    if (num_pages < 1 || max_pages_per_seq < 1)
        return fail(SPEC_ERR_INVALID, "num_pages and max_pages_per_seq must be >= 1");
    if (src_dtype != SPEC_DTYPE_F32 && src_dtype != SPEC_DTYPE_BF16)
        return fail(SPEC_ERR_INVALID, "src_dtype must be F32 or BF16");
    if (cache_dtype != SPEC_DTYPE_F32 && cache_dtype != SPEC_DTYPE_BF16 &&
        cache_dtype != SPEC_DTYPE_I8 && cache_dtype != SPEC_DTYPE_E4M3)
        return fail(SPEC_ERR_INVALID, "cache_dtype must be F32, BF16, I8 or E4M3");
    if (!(amplitude > -INFINITY && amplitude < INFINITY))
        return fail(SPEC_ERR_INVALID, "amplitude must be finite");
    const int64_t kv_row = (int64_t)num_kv_heads * head_dim, q_row = (int64_t)num_q_heads * head_dim;
    if (k_stride < kv_row || v_stride < kv_row || (num_q_heads && (q_stride < q_row ||
                                                                   q_out_stride < q_row)))
        return fail(SPEC_ERR_INVALID, "a token stride is shorter than the token's row");
    if (batch == 0) return SPEC_OK;
    if (!k_new || !v_new || !k_cache || !v_cache || !block_table || !ctx_lens ||
        (num_q_heads && (!q || !q_out)) || (rotary_dim && !rope_table))
        return fail(SPEC_ERR_INVALID, "null tensor pointer");
    int rc = check_scales(cache_dtype, k_scale, v_scale);
    if (rc) return rc;
    const int64_t step = src_dtype == SPEC_DTYPE_F32 ? 4 : 8;  // elements of 16 bytes
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (num_q_heads && (!aligned16(q) || !aligned16(q_out) || q_stride % step ||
                         q_out_stride % step)) ||
        k_stride % step || v_stride % step)
        return fail(SPEC_ERR_INVALID, "tensors and token strides must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(rope_table) & 7))
        return fail(SPEC_ERR_INVALID, "rope_table must be 8-byte aligned");
    // every launch index and in-kernel product below stays inside 31 bits
    if (reaches(1LL << 31, {batch, num_new, num_q_heads + 2 * (int64_t)num_kv_heads}) ||
        reaches(1LL << 40, {num_pages, num_kv_heads, page_size}))
        return fail(SPEC_ERR_UNSUPPORTED, "too many rows");
    Workspace* ws = nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = get_workspace(0, st, &ws);
    if (rc) return rc;
    specv::RopeAppendArgs a;
    a.q = q; a.k_new = k_new; a.v_new = v_new; a.q_out = q_out;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.q_out_stride = q_out_stride; a.src_dtype = src_dtype;
    a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
    a.cache_dtype = cache_dtype; a.block_table = block_table; a.ctx_lens = ctx_lens;
    a.positions = positions; a.new_lens = new_lens; a.table = rope_table;
    a.rot = rotary_dim; a.interleaved = interleaved != 0; a.amplitude = amplitude;
    a.B = batch; a.n = num_new; a.Hq = num_q_heads; a.Hkv = num_kv_heads; a.D = head_dim;
    a.P = page_size; a.num_pages = num_pages; a.max_pages = max_pages_per_seq;
    a.dev_err = static_cast<int*>(ws->base);
    cudaError_t e = specv::launch_rope_append(a, ws->sms, st);
    if (e != cudaSuccess) return cuda_fail(e, "rope_append launch");
    return SPEC_OK;
}

int spec_rope_table(int32_t rotary_dim, double theta, int32_t scaling, double factor,
                    double original_len, double fast_turns, double slow_turns, uint64_t* table,
                    float* amplitude) {
    g_err.clear();
    if (rotary_dim < 2 || rotary_dim > 256 || rotary_dim % 2)
        return fail(SPEC_ERR_INVALID, "rotary_dim must be even and in [2, 256]");
    if (!(theta > 1.0 && theta < INFINITY)) return fail(SPEC_ERR_INVALID, "theta must be > 1");
    const bool by_index = scaling == (SPEC_ROPE_YARN | SPEC_ROPE_RAMP_BY_INDEX);
    if (by_index) scaling = SPEC_ROPE_YARN;
    if (scaling < SPEC_ROPE_PLAIN || scaling > SPEC_ROPE_YARN)
        return fail(SPEC_ERR_INVALID, "unknown scaling %d", scaling);
    if (scaling != SPEC_ROPE_PLAIN && !(factor >= 1.0 && factor < INFINITY))
        return fail(SPEC_ERR_INVALID, "factor must be >= 1");
    if (scaling == SPEC_ROPE_NTK && rotary_dim < 4)
        return fail(SPEC_ERR_INVALID, "SPEC_ROPE_NTK needs rotary_dim >= 4");
    if (scaling == SPEC_ROPE_YARN &&
        !(original_len > 0 && original_len < INFINITY && slow_turns >= 0 &&
          fast_turns > slow_turns && fast_turns < INFINITY))
        return fail(SPEC_ERR_INVALID, "SPEC_ROPE_YARN needs original_len > 0 and "
                    "0 <= slow_turns < fast_turns");
    if (!table || !amplitude) return fail(SPEC_ERR_INVALID, "null table or amplitude");
    const double two_pi = 6.283185307179586476925286766559;
    const double d = rotary_dim;
    const double base = scaling == SPEC_ROPE_NTK ? theta * pow(factor, d / (d - 2)) : theta;
    // the ramp over the index: from pair `first` (kept) to pair `last` (all scaled)
    double first = 0, last = 0;
    if (by_index) {
        auto border = [&](double turns) {  // slow_turns may be 0: no pair turns so little
            return turns > 0 ? d / 2 * log(original_len / (two_pi * turns)) / log(theta) : d;
        };
        first = fmin(fmax(floor(border(fast_turns)), 0.0), d - 1);
        last = fmin(fmax(ceil(border(slow_turns)), 0.0), d - 1);
        if (last <= first) last = first + 0.001;  // a step
    }
    for (int j = 0; j < rotary_dim / 2; ++j) {
        double f = pow(base, -2.0 * j / d);
        if (scaling == SPEC_ROPE_LINEAR) f /= factor;
        if (scaling == SPEC_ROPE_YARN) {
            double keep =
                by_index ? 1 - (j - first) / (last - first)
                         : (original_len * f / two_pi - slow_turns) / (fast_turns - slow_turns);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            f = keep * f + (1 - keep) * f / factor;
        }
        // f <= 1 radian per position: the fraction of a turn stays below 2^62
        table[j] = (uint64_t)(f / two_pi * 18446744073709551616.0);
    }
    *amplitude = scaling == SPEC_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.f;
    return SPEC_OK;
}

int spec_kv_gather(const void* k_cache, const void* v_cache, const void* k_scale,
                   const void* v_scale, int32_t cache_dtype, const int32_t* block_table,
                   const int32_t* starts, const int32_t* lens, int32_t batch, int32_t max_len,
                   int32_t num_kv_heads, int32_t head_dim, int32_t page_size, int32_t num_pages,
                   int32_t max_pages_per_seq, int32_t out_dtype, void* k_out, void* v_out,
                   void* stream) {
    g_err.clear();
    if (batch < 0) return fail(SPEC_ERR_INVALID, "batch < 0");
    if (max_len < 0) return fail(SPEC_ERR_INVALID, "max_len < 0");
    if (num_kv_heads < 1) return fail(SPEC_ERR_INVALID, "num_kv_heads must be >= 1");
    if (head_dim < 32 || head_dim > 256 || head_dim % 32)
        return fail(SPEC_ERR_INVALID, "head_dim must be a multiple of 32 in [32, 256]");
    if (page_size < 1) return fail(SPEC_ERR_INVALID, "page_size < 1");
    if (num_pages < 1 || max_pages_per_seq < 1)
        return fail(SPEC_ERR_INVALID, "num_pages and max_pages_per_seq must be >= 1");
    if (out_dtype != SPEC_DTYPE_F32 && out_dtype != SPEC_DTYPE_BF16)
        return fail(SPEC_ERR_INVALID, "out_dtype must be F32 or BF16");
    if (cache_dtype != SPEC_DTYPE_F32 && cache_dtype != SPEC_DTYPE_BF16 &&
        cache_dtype != SPEC_DTYPE_I8 && cache_dtype != SPEC_DTYPE_E4M3)
        return fail(SPEC_ERR_INVALID, "cache_dtype must be F32, BF16, I8 or E4M3");
    if (batch == 0 || max_len == 0) return SPEC_OK;
    if (!k_cache || !v_cache || !block_table || !lens || !k_out || !v_out)
        return fail(SPEC_ERR_INVALID, "null tensor pointer");
    int rc = check_scales(cache_dtype, k_scale, v_scale);
    if (rc) return rc;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_out) || !aligned16(v_out))
        return fail(SPEC_ERR_INVALID, "caches and outputs must be 16-byte aligned");
    if (batch > 65535 || reaches(1LL << 31, {max_len, num_kv_heads, head_dim / 16}))
        return fail(SPEC_ERR_UNSUPPORTED, "too many rows");
    Workspace* ws = nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = get_workspace(0, st, &ws);
    if (rc) return rc;
    specv::GatherArgs a;
    a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
    a.cache_dtype = cache_dtype; a.block_table = block_table; a.starts = starts; a.lens = lens;
    a.k_out = k_out; a.v_out = v_out; a.out_dtype = out_dtype;
    a.B = batch; a.max_len = max_len; a.Hkv = num_kv_heads; a.D = head_dim; a.P = page_size;
    a.num_pages = num_pages; a.max_pages = max_pages_per_seq;
    a.dev_err = static_cast<int*>(ws->base);
    cudaError_t e = specv::launch_kv_gather(a, st);
    if (e != cudaSuccess) return cuda_fail(e, "kv_gather launch");
    return SPEC_OK;
}

// Entries of a table row that a block walks, a few thousand further at a time, in 32 bits.
constexpr int32_t kMaxTableWidth = 1 << 30;

// Sizes, types and pointers of a paged cache that a call writes.
static int check_cache(const void* k_cache, const void* v_cache, const void* k_scale,
                       const void* v_scale, int32_t cache_dtype, int32_t num_kv_heads,
                       int32_t head_dim, int32_t page_size, int32_t num_pages,
                       int32_t max_pages_per_seq, bool empty) {
    if (num_kv_heads < 1) return fail(SPEC_ERR_INVALID, "num_kv_heads must be >= 1");
    if (head_dim < 32 || head_dim > 256 || head_dim % 32)
        return fail(SPEC_ERR_INVALID, "head_dim must be a multiple of 32 in [32, 256]");
    if (page_size < 1) return fail(SPEC_ERR_INVALID, "page_size < 1");
    if (num_pages < 1 || max_pages_per_seq < 1)
        return fail(SPEC_ERR_INVALID, "num_pages and max_pages_per_seq must be >= 1");
    if (cache_dtype != SPEC_DTYPE_F32 && cache_dtype != SPEC_DTYPE_BF16 &&
        cache_dtype != SPEC_DTYPE_I8 && cache_dtype != SPEC_DTYPE_E4M3)
        return fail(SPEC_ERR_INVALID, "cache_dtype must be F32, BF16, I8 or E4M3");
    if (empty) return SPEC_OK;
    if (!k_cache || !v_cache) return fail(SPEC_ERR_INVALID, "null tensor pointer");
    const int rc = check_scales(cache_dtype, k_scale, v_scale);
    if (rc) return rc;
    if (!aligned16(k_cache) || !aligned16(v_cache))
        return fail(SPEC_ERR_INVALID, "caches must be 16-byte aligned");
    if (reaches(1LL << 40, {num_pages, num_kv_heads, page_size, head_dim}))
        return fail(SPEC_ERR_INVALID, "cache too large");
    // (indexes inside a page are 32-bit)
    if (reaches(1LL << 30, {num_kv_heads, page_size, head_dim}))
        return fail(SPEC_ERR_UNSUPPORTED, "page too large");
    return SPEC_OK;
}

int spec_kv_compact(void* k_cache, void* v_cache, void* k_scale, void* v_scale,
                    int32_t cache_dtype, const int32_t* block_table, const int32_t* ctx_lens,
                    const int32_t* path, const int32_t* accepted_len, int32_t batch,
                    int32_t num_draft, int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                    int32_t num_pages, int32_t max_pages_per_seq, void* stream) {
    g_err.clear();
    if (batch < 0) return fail(SPEC_ERR_INVALID, "batch < 0");
    if (num_draft < 1 || num_draft > 64) return fail(SPEC_ERR_INVALID, "num_draft must be in [1, 64]");
    int rc = check_cache(k_cache, v_cache, k_scale, v_scale, cache_dtype, num_kv_heads, head_dim,
                         page_size, num_pages, max_pages_per_seq, batch == 0);
    if (rc || batch == 0) return rc;
    if (!block_table || !ctx_lens || !path || !accepted_len)
        return fail(SPEC_ERR_INVALID, "null tensor pointer");
    if (batch > 65535) return fail(SPEC_ERR_UNSUPPORTED, "batch > 65535");
    Workspace* ws = nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = get_workspace(0, st, &ws);
    if (rc) return rc;
    specv::CompactArgs a;
    a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
    a.cache_dtype = cache_dtype; a.elem = dtype_size(cache_dtype);
    a.block_table = block_table; a.ctx_lens = ctx_lens; a.path = path; a.accepted = accepted_len;
    a.B = batch; a.k = num_draft; a.Hkv = num_kv_heads; a.D = head_dim; a.P = page_size;
    a.num_pages = num_pages; a.max_pages = max_pages_per_seq;
    a.dev_err = static_cast<int*>(ws->base);
    cudaError_t e = specv::launch_kv_compact(a, st);
    if (e != cudaSuccess) return cuda_fail(e, "kv_compact launch");
    return SPEC_OK;
}

int spec_kv_fork(void* k_cache, void* v_cache, void* k_scale, void* v_scale, int32_t cache_dtype,
                 int32_t* block_table, int32_t* ctx_lens, int32_t* page_refs,
                 const int32_t* parents, const int32_t* children, int32_t num_pairs, int32_t room,
                 int32_t num_rows, int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                 int32_t num_pages, int32_t max_pages_per_seq, void* stream) {
    g_err.clear();
    if (num_pairs < 0) return fail(SPEC_ERR_INVALID, "num_pairs < 0");
    if (room < 0) return fail(SPEC_ERR_INVALID, "room < 0");
    if (num_rows < 1) return fail(SPEC_ERR_INVALID, "num_rows must be >= 1");
    int rc = check_cache(k_cache, v_cache, k_scale, v_scale, cache_dtype, num_kv_heads, head_dim,
                         page_size, num_pages, max_pages_per_seq, num_pairs == 0);
    if (rc || num_pairs == 0) return rc;
    if (!block_table || !ctx_lens || !page_refs || !parents || !children)
        return fail(SPEC_ERR_INVALID, "null tensor pointer");
    if (num_pairs >= 1 << 24) return fail(SPEC_ERR_UNSUPPORTED, "num_pairs must be < 2^24");
    if (max_pages_per_seq > kMaxTableWidth)
        return fail(SPEC_ERR_UNSUPPORTED, "max_pages_per_seq must be <= 2^30");
    Workspace* ws = nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = get_workspace(specv::fork_workspace_bytes(num_pages, num_pairs), st, &ws);
    if (rc) return rc;
    specv::ForkArgs a;
    a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale;
    a.cache_dtype = cache_dtype; a.elem = dtype_size(cache_dtype);
    a.block_table = block_table; a.ctx_lens = ctx_lens; a.page_refs = page_refs;
    a.parents = parents; a.children = children; a.n = num_pairs; a.room = room; a.rows = num_rows;
    a.Hkv = num_kv_heads; a.D = head_dim; a.P = page_size; a.num_pages = num_pages;
    a.max_pages = max_pages_per_seq;
    a.dev_err = static_cast<int*>(ws->base);
    cudaError_t e = specv::launch_kv_fork(a, static_cast<char*>(ws->base) + kHeader, st);
    if (e != cudaSuccess) return cuda_fail(e, "kv_fork launch");
    return SPEC_OK;
}

int spec_kv_release(int32_t* block_table, int32_t* ctx_lens, int32_t* page_refs,
                    const int32_t* rows, const int32_t* keep_lens, int32_t num, int32_t num_rows,
                    int32_t page_size, int32_t num_pages, int32_t max_pages_per_seq, void* stream) {
    g_err.clear();
    if (num < 0) return fail(SPEC_ERR_INVALID, "num < 0");
    if (num_rows < 1) return fail(SPEC_ERR_INVALID, "num_rows must be >= 1");
    if (page_size < 1) return fail(SPEC_ERR_INVALID, "page_size < 1");
    if (num_pages < 1 || max_pages_per_seq < 1)
        return fail(SPEC_ERR_INVALID, "num_pages and max_pages_per_seq must be >= 1");
    if (num == 0) return SPEC_OK;
    if (!block_table || !ctx_lens || !page_refs || !rows)
        return fail(SPEC_ERR_INVALID, "null tensor pointer");
    // (each row looks for itself among the others)
    if (num >= 1 << 24) return fail(SPEC_ERR_UNSUPPORTED, "num must be < 2^24");
    if (max_pages_per_seq > kMaxTableWidth)
        return fail(SPEC_ERR_UNSUPPORTED, "max_pages_per_seq must be <= 2^30");
    Workspace* ws = nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int rc = get_workspace(0, st, &ws);
    if (rc) return rc;
    specv::ReleaseArgs a;
    a.block_table = block_table; a.ctx_lens = ctx_lens; a.page_refs = page_refs; a.rows = rows;
    a.keep_lens = keep_lens; a.n = num; a.batch = num_rows; a.P = page_size;
    a.num_pages = num_pages; a.max_pages = max_pages_per_seq;
    a.dev_err = static_cast<int*>(ws->base);
    cudaError_t e = specv::launch_kv_release(a, st);
    if (e != cudaSuccess) return cuda_fail(e, "kv_release launch");
    return SPEC_OK;
}

int spec_token_logprobs(const void* logits, int32_t logits_dtype, const int32_t* tokens,
                        const int32_t* lens, int32_t batch, int32_t num_rows, int64_t vocab,
                        float temperature, int32_t num_top, float* logprob, float* entropy,
                        int32_t* top_ids, float* top_logprobs, void* stream) {
    g_err.clear();
    if (batch < 0) return fail(SPEC_ERR_INVALID, "batch < 0");
    if (num_rows < 1) return fail(SPEC_ERR_INVALID, "num_rows must be >= 1");
    if (vocab < 1 || vocab >= (1LL << 31) - (1 << 16))
        return fail(SPEC_ERR_INVALID, "vocab must be in [1, 2^31 - 2^16)");
    if (logits_dtype != SPEC_DTYPE_F32 && logits_dtype != SPEC_DTYPE_BF16)
        return fail(SPEC_ERR_INVALID, "logits_dtype must be F32 or BF16");
    if (!(temperature >= 1e-30f) || !(temperature < INFINITY))
        return fail(SPEC_ERR_INVALID, "temperature must be positive (1e-30 at least) and finite");
    if (num_top < 0 || num_top > 32) return fail(SPEC_ERR_INVALID, "num_top must be in [0, 32]");
    if (batch == 0) return SPEC_OK;
    if (!logits || !tokens || !logprob) return fail(SPEC_ERR_INVALID, "null tensor pointer");
    if (num_top && !top_ids && !top_logprobs)
        return fail(SPEC_ERR_INVALID, "num_top > 0 needs top_ids or top_logprobs");
    if (!aligned16(logits)) return fail(SPEC_ERR_INVALID, "logits must be 16-byte aligned");
    if (reaches(1LL << 26, {batch, num_rows})) return fail(SPEC_ERR_UNSUPPORTED, "too many rows");
    Workspace* ws = nullptr;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int rc = get_workspace(0, st, &ws);
    if (rc) return rc;
    specv::LogprobArgs a;
    a.logits = logits; a.dtype = logits_dtype; a.tokens = tokens; a.lens = lens;
    a.B = batch; a.n = num_rows; a.V = vocab;
    a.inv_t = (float)(1.0 / (double)temperature);
    a.c = (float)(1.4426950408889634074 / (double)temperature);
    a.K = num_top; a.logprob = logprob; a.entropy = entropy; a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.parts = specv::logprob_parts(a, ws->sms, kMaxTickets);
    rc = get_workspace(specv::logprob_workspace_bytes(a), st, &ws);
    if (rc) return rc;
    a.tickets = reinterpret_cast<int32_t*>(static_cast<char*>(ws->base) + kTicketsOff);
    a.dev_err = static_cast<int*>(ws->base);
    cudaError_t e = specv::launch_logprobs(a, ws->sms, static_cast<char*>(ws->base) + kHeader, st);
    if (e != cudaSuccess) return cuda_fail(e, "token_logprobs launch");
    return SPEC_OK;
}

static int codec_args(int64_t num_blocks, int32_t page_size, int32_t head_dim) {
    if (num_blocks < 0) return fail(SPEC_ERR_INVALID, "num_blocks < 0");
    if (head_dim < 32 || head_dim > 256 || head_dim % 32)
        return fail(SPEC_ERR_INVALID, "head_dim must be a multiple of 32 in [32, 256]");
    if (page_size < 1 || (int64_t)page_size * head_dim > 16384)
        return fail(SPEC_ERR_INVALID, "page_size must be >= 1 with page_size * head_dim <= 16384");
    if (num_blocks / 8 >= (1LL << 31)) return fail(SPEC_ERR_UNSUPPORTED, "too many blocks");
    return SPEC_OK;
}

int spec_codec_encode(const void* codes, int64_t num_blocks, int32_t page_size, int32_t head_dim,
                      void* pairs, int32_t* num_pairs, void* stream) {
    g_err.clear();
    int rc = codec_args(num_blocks, page_size, head_dim);
    if (rc) return rc;
    if (num_blocks == 0) return SPEC_OK;
    if (!codes || !pairs || !num_pairs) return fail(SPEC_ERR_INVALID, "null tensor pointer");
    cudaError_t e = specv::launch_codec_encode(codes, num_blocks, page_size, head_dim, pairs,
                                               num_pairs, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "codec_encode launch");
    return SPEC_OK;
}

int spec_codec_decode(const void* pairs, const int32_t* num_pairs, int64_t num_blocks,
                      int32_t page_size, int32_t head_dim, void* codes, void* stream) {
    g_err.clear();
    int rc = codec_args(num_blocks, page_size, head_dim);
    if (rc) return rc;
    if (num_blocks == 0) return SPEC_OK;
    if (!codes || !pairs || !num_pairs) return fail(SPEC_ERR_INVALID, "null tensor pointer");
    if ((reinterpret_cast<uintptr_t>(pairs) & 15) || (reinterpret_cast<uintptr_t>(codes) & 15))
        return fail(SPEC_ERR_INVALID, "pairs and codes must be 16-byte aligned");
    Workspace* ws = nullptr;
    rc = get_workspace(0, static_cast<cudaStream_t>(stream), &ws);
    if (rc) return rc;
    cudaError_t e = specv::launch_codec_decode(pairs, num_pairs, num_blocks, page_size, head_dim,
                                               codes, static_cast<int*>(ws->base),
                                               static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "codec_decode launch");
    return SPEC_OK;
}

int spec_commit(int32_t* ctx_lens, const int32_t* accepted_len, int32_t batch, int32_t extra,
                void* stream) {
    g_err.clear();
    if (batch < 0) return fail(SPEC_ERR_INVALID, "batch < 0");
    if (batch == 0) return SPEC_OK;
    if (!ctx_lens || !accepted_len) return fail(SPEC_ERR_INVALID, "null tensor pointer");
    cudaError_t e = specv::launch_commit(ctx_lens, accepted_len, batch, extra,
                                         static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "commit launch");
    return SPEC_OK;
}

int spec_device_error(int32_t* flags) {
    g_err.clear();
    if (!flags) return fail(SPEC_ERR_INVALID, "flags is NULL");
    Workspace* ws = nullptr;
    int rc = get_workspace(0, nullptr, &ws);
    if (rc) return rc;
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
    int all = 0;
    auto read = [&](void* base) {  // a word of a buffer, read and cleared
        int v = 0;
        e = cudaMemcpy(&v, base, sizeof(int), cudaMemcpyDeviceToHost);
        if (e == cudaSuccess && v) e = cudaMemset(base, 0, sizeof(int));
        all |= v;
        return e == cudaSuccess;
    };
    std::lock_guard<std::mutex> lk(g_ws_mu);
    bool ok = read(ws->base);
    for (size_t i = 0; ok && i < ws->retired.size(); ++i) ok = read(ws->retired[i]);
    if (ok) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "read device error word");
    *flags = all;
    return SPEC_OK;
}

int spec_release(void) {
    g_err.clear();
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    std::lock_guard<std::mutex> lk(g_ws_mu);
    if ((int)g_ws.size() > dev && g_ws[dev].base) {
        e = cudaDeviceSynchronize();
        if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
        cudaFree(g_ws[dev].base);
        for (void* p : g_ws[dev].retired) cudaFree(p);
        g_ws[dev].retired.clear();
        g_ws[dev].base = nullptr;
        g_ws[dev].bytes = 0;
    }
    return SPEC_OK;
}

}  // extern "C"

// ---------------------------------------------------------------- tensor-descriptor form
//
// The same two calls taking self-describing tensors (pointer, element type,
// rank, shape, strides in elements): the descriptors are checked against
// one another and forwarded to the flat entry points above.  The kernels
// read dense row-major tensors, so any other stride is refused (-2).

namespace {

// Dense row-major strides of `t` (in elements) match the given ones?
bool dense(const spec_tensor_t& t) {
    int64_t s = 1;
    for (int d = t.ndim - 1; d >= 0; --d) {
        if (t.shape[d] != 1 && t.stride[d] != s) return false;
        s *= t.shape[d];
    }
    return true;
}

// Checks rank, element type, shape (-1 = any), alignment and density of a
// descriptor; returns 0 or sets the error.
int check_tensor(const spec_tensor_t* t, const char* name, int ndim, std::initializer_list<int32_t> dtypes,
                 std::initializer_list<int64_t> shape, bool need16 = false) {
    if (!t) return fail(SPEC_ERR_INVALID, "%s: null descriptor", name);
    if (t->ndim != ndim) return fail(SPEC_ERR_INVALID, "%s: rank %d, expected %d", name, t->ndim, ndim);
    bool ok = false;
    for (int32_t dt : dtypes) ok = ok || t->dtype == dt;
    if (!ok) return fail(SPEC_ERR_INVALID, "%s: unsupported element type %d", name, t->dtype);
    int d = 0;
    for (int64_t want : shape) {
        if (t->shape[d] < 0 || (want >= 0 && t->shape[d] != want))
            return fail(SPEC_ERR_INVALID, "%s: dimension %d is %lld, expected %lld", name, d,
                        (long long)t->shape[d], (long long)want);
        ++d;
    }
    if (need16 && (reinterpret_cast<uintptr_t>(t->data) & 15))
        return fail(SPEC_ERR_INVALID, "%s: data must be 16-byte aligned", name);
    if (!dense(*t))
        return fail(SPEC_ERR_UNSUPPORTED, "%s: only dense row-major strides are supported", name);
    return SPEC_OK;
}

bool fits_i32(int64_t v) { return v >= 0 && v < (1LL << 31); }

}  // namespace

extern "C" {

int spec_verify_attn_tensors(const spec_tensor_t* q, const spec_tensor_t* k_cache,
                             const spec_tensor_t* v_cache, const spec_tensor_t* k_scale,
                             const spec_tensor_t* v_scale, const spec_tensor_t* block_table,
                             const spec_tensor_t* ctx_lens, int32_t num_draft, float scale,
                             spec_tensor_t* out, spec_tensor_t* lse, void* stream) {
    g_err.clear();
    int rc = check_tensor(q, "q", 4, {SPEC_DTYPE_F32, SPEC_DTYPE_BF16}, {-1, num_draft, -1, -1}, true);
    if (rc) return rc;
    const int64_t B = q->shape[0], Hq = q->shape[2], D = q->shape[3];
    rc = check_tensor(k_cache, "k_cache", 4, 
                      {SPEC_DTYPE_F32, SPEC_DTYPE_BF16, SPEC_DTYPE_I8, SPEC_DTYPE_E4M3},
                      {-1, -1, -1, D}, true);
    if (rc) return rc;
    const int64_t NP = k_cache->shape[0], Hkv = k_cache->shape[1], P = k_cache->shape[2];
    rc = check_tensor(v_cache, "v_cache", 4, {k_cache->dtype}, {NP, Hkv, P, D}, true);
    if (rc) return rc;
    const bool i8 = k_cache->dtype == SPEC_DTYPE_I8, e4m3 = k_cache->dtype == SPEC_DTYPE_E4M3;
    if (i8) {
        rc = check_tensor(k_scale, "k_scale", 3, {SPEC_DTYPE_F16}, {NP, Hkv, P});
        if (!rc) rc = check_tensor(v_scale, "v_scale", 3, {SPEC_DTYPE_F16}, {NP, Hkv, P});
        if (rc) return rc;
    }
    if (e4m3) {
        rc = check_tensor(k_scale, "k_scale", 2, {SPEC_DTYPE_F32}, {NP, Hkv});
        if (!rc) rc = check_tensor(v_scale, "v_scale", 2, {SPEC_DTYPE_F32}, {NP, Hkv});
        if (rc) return rc;
    }
    rc = check_tensor(block_table, "block_table", 2, {SPEC_DTYPE_I32}, {B, -1});
    if (!rc) rc = check_tensor(ctx_lens, "ctx_lens", 1, {SPEC_DTYPE_I32}, {B});
    if (!rc) rc = check_tensor(out, "out", 4, {q->dtype}, {B, num_draft, Hq, D}, true);
    if (!rc && lse) rc = check_tensor(lse, "lse", 3, {SPEC_DTYPE_F32}, {B, num_draft, Hq});
    if (rc) return rc;
    const int64_t MP = block_table->shape[1];
    if (!fits_i32(B) || !fits_i32(Hq) || !fits_i32(D) || !fits_i32(NP) || !fits_i32(Hkv) ||
        !fits_i32(P) || !fits_i32(MP))
        return fail(SPEC_ERR_INVALID, "a dimension does not fit int32");
    const bool scaled = i8 || e4m3;
    return spec_verify_attn(q->data, k_cache->data, v_cache->data,
                            scaled ? k_scale->data : nullptr, scaled ? v_scale->data : nullptr,
                            static_cast<const int32_t*>(block_table->data),
                            static_cast<const int32_t*>(ctx_lens->data), (int32_t)B, num_draft,
                            (int32_t)Hq, (int32_t)Hkv, (int32_t)D, (int32_t)P, (int32_t)NP,
                            (int32_t)MP, q->dtype, k_cache->dtype, scale, out->data,
                            lse ? static_cast<float*>(lse->data) : nullptr, stream);
}

int spec_accept_greedy_tensors(const spec_tensor_t* logits, const spec_tensor_t* draft_tokens,
                               int32_t num_draft, spec_tensor_t* accepted_len,
                               spec_tensor_t* next_token, void* stream) {
    g_err.clear();
    int rc = check_tensor(logits, "logits", 3, {SPEC_DTYPE_F32, SPEC_DTYPE_BF16},
                          {-1, (int64_t)num_draft + 1, -1}, true);
    if (rc) return rc;
    const int64_t B = logits->shape[0];
    rc = check_tensor(draft_tokens, "draft_tokens", 2, {SPEC_DTYPE_I32}, {B, num_draft});
    if (!rc) rc = check_tensor(accepted_len, "accepted_len", 1, {SPEC_DTYPE_I32}, {B});
    if (!rc) rc = check_tensor(next_token, "next_token", 1, {SPEC_DTYPE_I32}, {B});
    if (rc) return rc;
    if (!fits_i32(B)) return fail(SPEC_ERR_INVALID, "batch does not fit int32");
    return spec_accept_greedy(logits->data, logits->dtype,
                              static_cast<const int32_t*>(draft_tokens->data), (int32_t)B,
                              num_draft, logits->shape[2],
                              static_cast<int32_t*>(accepted_len->data),
                              static_cast<int32_t*>(next_token->data), stream);
}

}  // extern "C"
