// decode.cu -- entry points of the decode over 16-bit and E4M3 caches (the
// kernels are in decode_split.cuh).
#include "decode_split.cuh"

using namespace pkv;

extern "C" size_t paged_decode_workspace_size(int32_t batch_size, int32_t q_len_per_req,
                                              int32_t num_qo_heads, int32_t num_kv_heads,
                                              int32_t head_dim, int32_t max_seq_len,
                                              int32_t page_size, int32_t window_left) {
    DecodePlan pl;
    if (plan_decode(batch_size, q_len_per_req, num_qo_heads, num_kv_heads, head_dim, max_seq_len,
                    page_size, window_left, pl) != PKV_OK)
        return 0;
    return pl.ws_bytes;
}

// What a window with first tokens or a cache with block scales adds.
struct DecodeExt {
    int32_t first_tokens = 0;
    const float *k_scales = nullptr, *v_scales = nullptr;
    int64_t scale_page_stride = 0;
    int32_t scale_block = 0;
};

static int decode_impl(const void *query, const void *k_cache, const void *v_cache,
                            int64_t page_stride, int64_t max_num_pages, void *workspace,
                            size_t workspace_bytes, const int32_t *block_tables,
                            int32_t block_table_stride, const uint32_t *seq_lens,
                            int32_t batch_size, int32_t max_seq_len, float bmm1_scale,
                            float bmm2_scale, int32_t window_left, const float *sinks,
                            int32_t q_len_per_req, const int32_t *cum_seq_lens_q, int64_t num_tokens,
                            int32_t num_qo_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t page_size, int32_t layout, int32_t dtype,
                            void *out, float *lse, int32_t *err_word, void *stream,
                            const float *bmm1_dev = nullptr, const float *bmm2_dev = nullptr,
                            bool enable_pdl = false, const DecodeExt *ext = nullptr) {
    if (layout != PKV_NHD && layout != PKV_HND) return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_F16 && dtype != PKV_BF16 && dtype != PKV_F16_E4M3 && dtype != PKV_BF16_E4M3)
        return PKV_ERR_INVALID_ARG;
    const bool kv8 = dtype == PKV_F16_E4M3 || dtype == PKV_BF16_E4M3;  // 8-bit cache, 16-bit query/out
    const bool bf16 = dtype == PKV_BF16 || dtype == PKV_BF16_E4M3;
    DecodePlan pl;
    const int first_tokens = ext ? ext->first_tokens : 0;
    int rc = plan_decode(batch_size, q_len_per_req, num_qo_heads, num_kv_heads, head_dim,
                         max_seq_len, page_size, window_left, pl, false, first_tokens);
    if (rc != PKV_OK) return rc;
    const bool scaled = ext && (ext->k_scales || ext->v_scales || ext->scale_block);
    if (scaled) {
        if (!kv8) return PKV_ERR_INVALID_ARG;  // scales belong to an 8-bit cache
        const int bs = ilog2_exact(ext->scale_block);
        if (bs < 3 || ext->scale_block > page_size) return PKV_ERR_INVALID_ARG;
        if (ext->scale_page_stride < static_cast<int64_t>(num_kv_heads) * (page_size >> bs)) return PKV_ERR_INVALID_ARG;
    }
    if (kv8) {
        // the E4M3 plan's longer splits, whenever they fit the workspace that
        // paged_decode_workspace_size (which knows no element type) sized
        DecodePlan p8;
        if (plan_decode(batch_size, q_len_per_req, num_qo_heads, num_kv_heads, head_dim, max_seq_len,
                        page_size, window_left, p8, true, first_tokens) == PKV_OK &&
            p8.ws_bytes <= pl.ws_bytes)
            pl = p8;
    }
    if (page_stride < static_cast<int64_t>(num_kv_heads) * page_size * head_dim || max_num_pages < 0 ||
        static_cast<int64_t>(block_table_stride) * page_size < max_seq_len)
        return PKV_ERR_INVALID_ARG;
    if (batch_size == 0) return PKV_OK;
    if (!query || !k_cache || !v_cache || !block_tables || !seq_lens || !out) return PKV_ERR_NULL;
    if (scaled && (!ext->k_scales || !ext->v_scales)) return PKV_ERR_NULL;
    if (scaled && ((reinterpret_cast<uintptr_t>(ext->k_scales) | reinterpret_cast<uintptr_t>(ext->v_scales)) & 3))
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        (page_stride % (kv8 ? 16 : 8)))  // 16-byte page starts
        return PKV_ERR_INVALID_ARG;
    if (pl.ws_bytes > 0) {
        if (!workspace) return PKV_ERR_NULL;
        if (workspace_bytes < pl.ws_bytes || (reinterpret_cast<uintptr_t>(workspace) & 255))
            return PKV_ERR_WORKSPACE;
    }
    DecodeParams p;
    p.q = query;
    p.k = k_cache;
    p.v = v_cache;
    p.page_stride = page_stride;
    p.max_num_pages = max_num_pages;
    p.block_tables = block_tables;
    p.bt_stride = block_table_stride;
    p.seq_lens = seq_lens;
    p.B = batch_size;
    p.max_seq_len = max_seq_len;
    p.scale_log2 = bmm1_scale * kLog2e;
    p.bmm2 = bmm2_scale;
    p.bmm1_dev = bmm1_dev;
    p.bmm2_dev = bmm2_dev;
    p.window_left = window_left;
    p.sinks = sinks;
    p.Q = q_len_per_req;
    p.cu_q = cum_seq_lens_q;
    p.num_tokens = num_tokens;
    p.kv_extent = max_num_pages > 0 ? (max_num_pages - 1) * page_stride +
                                          static_cast<int64_t>(num_kv_heads) * page_size * head_dim
                                    : 0;
    p.ws_rows = static_cast<int64_t>(batch_size) * num_kv_heads * pl.n_split_max * pl.R;
    p.Hqo = num_qo_heads;
    p.Hkv = num_kv_heads;
    p.group = num_qo_heads / num_kv_heads;
    p.R = pl.R;
    p.page_shift = ilog2_exact(page_size);
    p.chunk = pl.chunk;
    p.n_split_max = pl.n_split_max;
    p.out = out;
    p.lse = lse;
    p.ws_o = pl.ws_bytes ? static_cast<float *>(workspace) : nullptr;
    p.ws_lse = pl.ws_bytes ? reinterpret_cast<float *>(static_cast<char *>(workspace) + pl.ws_o_bytes)
                           : nullptr;
    p.err = err_word;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.first_tokens = first_tokens;
    p.k_scales = p.v_scales = nullptr;
    p.scale_stride = 0;
    p.block_shift = p.pages_cap = p.scales_cap = 0;
    if (ext) {  // (also without scales and window: a NaN key then has the same effect)
        // a split of `chunk` keys may start and end inside a page (block), in
        // both parts of its run
        p.pages_cap = ((pl.chunk >> p.page_shift) + 5) & ~1;  // (even: the scale list after it is 8-byte aligned)
        if (scaled) {
            p.k_scales = ext->k_scales;
            p.v_scales = ext->v_scales;
            p.scale_stride = ext->scale_page_stride;
            p.block_shift = ilog2_exact(ext->scale_block);
            p.scales_cap = (pl.chunk >> p.block_shift) + 4;
        }
        return run_decode_ext(p, pl, layout, bf16, kv8, enable_pdl, st);
    }
    return bf16 ? run_decode<__nv_bfloat16>(p, pl, layout, kv8, enable_pdl, st)
                : run_decode<__half>(p, pl, layout, kv8, enable_pdl, st);
}

extern "C" int paged_decode(const void *query, const void *k_cache, const void *v_cache,
                            int64_t page_stride, int64_t max_num_pages, void *workspace,
                            size_t workspace_bytes, const int32_t *block_tables,
                            int32_t block_table_stride, const uint32_t *seq_lens,
                            int32_t batch_size, int32_t max_seq_len, float bmm1_scale,
                            float bmm2_scale, int32_t window_left, const float *sinks,
                            int32_t q_len_per_req, int32_t num_qo_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t page_size, int32_t layout, int32_t dtype,
                            void *out, float *lse, int32_t *err_word, void *stream) {
    const CallRange nvtx_range("paged_decode");
    return decode_impl(query, k_cache, v_cache, page_stride, max_num_pages, workspace, workspace_bytes,
                       block_tables, block_table_stride, seq_lens, batch_size, max_seq_len, bmm1_scale,
                       bmm2_scale, window_left, sinks, q_len_per_req, nullptr,
                       static_cast<int64_t>(batch_size) * q_len_per_req, num_qo_heads, num_kv_heads, head_dim,
                       page_size, layout, dtype, out, lse, err_word, stream);
}

extern "C" int paged_decode_varlen(const void *query, int64_t num_tokens, const void *k_cache,
                                   const void *v_cache, int64_t page_stride, int64_t max_num_pages,
                                   void *workspace, size_t workspace_bytes, const int32_t *block_tables,
                                   int32_t block_table_stride, const uint32_t *seq_lens, int32_t batch_size,
                                   int32_t max_seq_len, float bmm1_scale, float bmm2_scale,
                                   int32_t window_left, const float *sinks, int32_t max_q_len,
                                   const int32_t *cum_seq_lens_q, int32_t num_qo_heads, int32_t num_kv_heads,
                                   int32_t head_dim, int32_t page_size, int32_t layout, int32_t dtype,
                                   void *out, float *lse, int32_t *err_word, void *stream) {
    const CallRange nvtx_range("paged_decode_varlen");
    if (num_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (batch_size > 0 && num_tokens > 0 && !cum_seq_lens_q) return PKV_ERR_NULL;
    if (num_tokens == 0) return PKV_OK;
    return decode_impl(query, k_cache, v_cache, page_stride, max_num_pages, workspace, workspace_bytes,
                       block_tables, block_table_stride, seq_lens, batch_size, max_seq_len, bmm1_scale,
                       bmm2_scale, window_left, sinks, max_q_len, cum_seq_lens_q, num_tokens, num_qo_heads,
                       num_kv_heads, head_dim, page_size, layout, dtype, out, lse, err_word, stream);
}

extern "C" int paged_decode_ex(const void *query, int64_t num_tokens, const void *k_cache,
                               const void *v_cache, int64_t page_stride, int64_t max_num_pages,
                               void *workspace, size_t workspace_bytes, const int32_t *block_tables,
                               int32_t block_table_stride, const uint32_t *seq_lens, int32_t batch_size,
                               int32_t max_seq_len, float bmm1_scale, float bmm2_scale,
                               const float *bmm1_scale_dev, const float *bmm2_scale_dev, int32_t window_left,
                               const float *sinks, int32_t max_q_len, const int32_t *cum_seq_lens_q,
                               int32_t num_qo_heads, int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                               int32_t layout, int32_t dtype, int32_t enable_pdl, void *out, float *lse,
                               int32_t *err_word, void *stream) {
    const CallRange nvtx_range("paged_decode_ex");
    if (num_tokens < 0 || max_q_len < 1) return PKV_ERR_INVALID_ARG;
    if (!cum_seq_lens_q && num_tokens < static_cast<int64_t>(batch_size) * max_q_len) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    return decode_impl(query, k_cache, v_cache, page_stride, max_num_pages, workspace, workspace_bytes,
                       block_tables, block_table_stride, seq_lens, batch_size, max_seq_len, bmm1_scale,
                       bmm2_scale, window_left, sinks, max_q_len, cum_seq_lens_q,
                       cum_seq_lens_q ? num_tokens : static_cast<int64_t>(batch_size) * max_q_len, num_qo_heads,
                       num_kv_heads, head_dim, page_size, layout, dtype, out, lse, err_word, stream,
                       bmm1_scale_dev, bmm2_scale_dev, enable_pdl != 0);
}

// ---- a window with first tokens; an E4M3 cache with block scales ----------------

extern "C" size_t paged_decode_window_workspace_size(int32_t batch_size, int32_t q_len_per_req, int32_t num_qo_heads,
                                                     int32_t num_kv_heads, int32_t head_dim, int32_t max_seq_len,
                                                     int32_t page_size, int32_t window_left, int32_t first_tokens) {
    DecodePlan pl;
    if (plan_decode(batch_size, q_len_per_req, num_qo_heads, num_kv_heads, head_dim, max_seq_len, page_size,
                    window_left, pl, false, first_tokens) != PKV_OK)
        return 0;
    return pl.ws_bytes;
}

extern "C" int paged_decode_window(const void *query, int64_t num_tokens, const void *k_cache, const void *v_cache,
                                   int64_t page_stride, int64_t max_num_pages, const float *k_scales,
                                   const float *v_scales, int64_t scale_page_stride, int32_t scale_block,
                                   void *workspace, size_t workspace_bytes, const int32_t *block_tables,
                                   int32_t block_table_stride, const uint32_t *seq_lens, int32_t batch_size,
                                   int32_t max_seq_len, float bmm1_scale, float bmm2_scale,
                                   const float *bmm1_scale_dev, const float *bmm2_scale_dev, int32_t window_left,
                                   int32_t first_tokens, const float *sinks, int32_t max_q_len,
                                   const int32_t *cum_seq_lens_q, int32_t num_qo_heads, int32_t num_kv_heads,
                                   int32_t head_dim, int32_t page_size, int32_t layout, int32_t dtype,
                                   int32_t enable_pdl, void *out, float *lse, int32_t *err_word, void *stream) {
    const CallRange nvtx_range("paged_decode_window");
    if (num_tokens < 0 || max_q_len < 1 || first_tokens < 0 || window_left < -1) return PKV_ERR_INVALID_ARG;
    if (max_seq_len > (1 << 30)) return PKV_ERR_UNSUPPORTED;
    if (window_left > max_seq_len && max_seq_len >= 0) window_left = max_seq_len;  // every key either way
    if (!cum_seq_lens_q && num_tokens < static_cast<int64_t>(batch_size) * max_q_len) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    DecodeExt ext;
    ext.first_tokens = first_tokens;
    ext.k_scales = k_scales;
    ext.v_scales = v_scales;
    ext.scale_page_stride = scale_page_stride;
    ext.scale_block = scale_block;
    return decode_impl(query, k_cache, v_cache, page_stride, max_num_pages, workspace, workspace_bytes, block_tables,
                       block_table_stride, seq_lens, batch_size, max_seq_len, bmm1_scale, bmm2_scale, window_left,
                       sinks, max_q_len, cum_seq_lens_q,
                       cum_seq_lens_q ? num_tokens : static_cast<int64_t>(batch_size) * max_q_len, num_qo_heads,
                       num_kv_heads, head_dim, page_size, layout, dtype, out, lse, err_word, stream, bmm1_scale_dev,
                       bmm2_scale_dev, enable_pdl != 0, &ext);
}

// ---- decode with a library-owned scratch array ------------------------------
//
// For callers that cannot allocate device memory where they call decode: a
// plugin running inside another runtime's execution step (that runtime owns
// the device memory and forbids allocation there), a latency-critical loop
// that cannot afford cudaMalloc's implicit device-wide synchronisation, or
// a process that reserves all device memory up front.  The split partials
// live in a fixed array in this library's own device image instead of a
// caller workspace.
#include <cudaTypedefs.h>

#include <mutex>

namespace pkv {

constexpr size_t kNoAllocScratchBytes = static_cast<size_t>(PKV_NOALLOC_SCRATCH_BYTES);
constexpr int kNoAllocCachedContexts = 64;

// One copy per device that loads the library, held until the process exits.
static __device__ __align__(256) unsigned char g_decode_scratch[kNoAllocScratchBytes];

// Unique id of the calling thread's current CUDA context (driver entry points
// fetched through the runtime: the library does not link libcuda).  False
// when no context is current yet.
static bool current_context_id(unsigned long long *id) {
    static std::once_flag once;
    static PFN_cuCtxGetCurrent_v4000 get_current = nullptr;
    static PFN_cuCtxGetId_v12000 get_id = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 4000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            get_current = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(p);
        if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(p);
    });
    CUcontext ctx = nullptr;
    if (!get_current || !get_id || get_current(&ctx) != CUDA_SUCCESS || !ctx) return false;
    return get_id(ctx, id) == CUDA_SUCCESS;
}

// Device address of g_decode_scratch in the current context.  In host code
// the symbol is only a host-side stand-in, so the address is looked up with
// cudaGetSymbolAddress and cached per CUDA context, keyed by the context's
// unique id: after a device reset (or under another context of the same
// device) the library's module is loaded again and the array may move; the
// new context has a new id, so its address is looked up afresh.
static void *noalloc_scratch_ptr() {
    static std::mutex mu;
    static unsigned long long ids[kNoAllocCachedContexts];
    static void *ptrs[kNoAllocCachedContexts];
    static int used = 0, next = 0;
    unsigned long long id = 0;
    const bool have_id = current_context_id(&id);
    std::lock_guard<std::mutex> lock(mu);
    if (have_id)
        for (int i = 0; i < used; ++i)
            if (ids[i] == id) return ptrs[i];
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_decode_scratch) != cudaSuccess || !p) return nullptr;
    // (the lookup above made the primary context current if none was)
    if (!have_id && !current_context_id(&id)) return p;  // not cached: looked up again next call
    const int slot = used < kNoAllocCachedContexts ? used++ : (next++ % kNoAllocCachedContexts);
    ids[slot] = id;
    ptrs[slot] = p;
    return p;
}

}  // namespace pkv

extern "C" int paged_decode_noalloc(const void *query, const void *k_cache, const void *v_cache,
                                    int64_t page_stride, int64_t max_num_pages,
                                    const int32_t *block_tables, int32_t block_table_stride,
                                    const uint32_t *seq_lens, int32_t batch_size,
                                    int32_t max_seq_len, float bmm1_scale, float bmm2_scale,
                                    int32_t window_left, const float *sinks,
                                    int32_t q_len_per_req, int32_t num_qo_heads,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                                    int32_t layout, int32_t dtype, void *out, float *lse,
                                    int32_t *err_word, void *stream) {
    const CallRange nvtx_range("paged_decode_noalloc");
    DecodePlan pl;
    int rc = plan_decode(batch_size, q_len_per_req, num_qo_heads, num_kv_heads, head_dim,
                         max_seq_len, page_size, window_left, pl);
    if (rc != PKV_OK) return rc;
    if (pl.ws_bytes > kNoAllocScratchBytes) return PKV_ERR_WORKSPACE;
    void *scratch = nullptr;
    if (pl.ws_bytes > 0) {
        scratch = noalloc_scratch_ptr();
        if (!scratch) return PKV_ERR_CUDA;
    }
    return paged_decode(query, k_cache, v_cache, page_stride, max_num_pages, scratch,
                        scratch ? kNoAllocScratchBytes : 0, block_tables, block_table_stride,
                        seq_lens, batch_size, max_seq_len, bmm1_scale, bmm2_scale, window_left,
                        sinks, q_len_per_req, num_qo_heads, num_kv_heads, head_dim, page_size,
                        layout, dtype, out, lse, err_word, stream);
}
