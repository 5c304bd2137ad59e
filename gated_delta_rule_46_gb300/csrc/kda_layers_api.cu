// kda_layers_api.cu -- the extern "C" entry points declared in
// include/kda_layers.h and include/kda_pages.h: argument validation on the host, kernel selection and
// launches on the caller's stream.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "kda_layers.cuh"
#include "kda_pages.cuh"
#include "kda_testing.h"

namespace kda {
static std::atomic<int> g_layers_expire{0};
void set_layers_expire(int mask) { g_layers_expire.store(mask); }
bool take_layers_expire(int bit) { return g_layers_expire.fetch_and(~bit) & bit; }

int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (dev < 64 && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 148;
    if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}
}  // namespace kda

namespace {

constexpr int64_t kMax31 = int64_t(1) << 31;

bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool dtype_ok(kda_dtype_t t) { return t == KDA_F32 || t == KDA_BF16; }
int64_t elem(kda_dtype_t t) { return t == KDA_BF16 ? 2 : 4; }
bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// float32 and int32 values, and the status word
template <typename... P>
bool words(const P *...p) { return (aligned(p, 4) && ...); }
kda_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// log2 of a page size, or -1 where it is not a power of two up to 1024
int page_shift(int page_size) {
    for (int s = 0; s <= 10; ++s)
        if (page_size == (1 << s)) return s;
    return -1;
}

// the same of a block of tokens that shares a scale
int block_shift(int block, int page_size) {
    return block >= 16 && block <= 128 && block <= page_size ? page_shift(block) : -1;
}

// a workspace of `need` bytes, where any are needed
bool workspace_ok(const void *workspace, size_t bytes, size_t need) {
    return aligned(workspace, 16) && (need == 0 || (workspace && bytes >= need));
}

bool pools_ok(void *const *pools, const int64_t *page_bytes, int n) {
    if (n > 0 && (!pools || !page_bytes)) return false;
    for (int i = 0; i < n; ++i)
        if (page_bytes[i] < 0 || (page_bytes[i] > 0 && !pools[i])) return false;
    return true;
}

// rows of a page table whose entries can be counted in 31 bits
bool table_ok(int num_rows, int max_pages) { return (int64_t)num_rows * max_pages < kMax31; }

}  // namespace

extern "C" {

kda_status_t kda_linear(const void *x, int64_t ldx, const void *w, const float *bias, const void *residual,
                        void *out, int64_t M, int64_t N, int64_t K, kda_act_t act, kda_dtype_t out_dtype,
                        uint32_t *status, kda_stream_t stream) {
    if (M < 0 || N < 0 || K <= 0 || ldx < K) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(out_dtype) || act < KDA_ACT_NONE || act > KDA_ACT_SIGMOID) return KDA_ERR_UNSUPPORTED;
    if (M >= kMax31 || N >= kMax31 || K >= kMax31) return KDA_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return KDA_OK;
    if (!x || !w || !out) return KDA_ERR_INVALID_ARG;
    if (!aligned(x, 2) || !aligned(w, 2) || !words(bias, status) || !aligned(out, elem(out_dtype)) ||
        !aligned(residual, elem(out_dtype)))
        return KDA_ERR_INVALID_ARG;
    const kda::LinearParams p{static_cast<const __nv_bfloat16 *>(x), ldx, static_cast<const __nv_bfloat16 *>(w),
                              bias, residual, out, M, N, K, act, out_dtype == KDA_F32, status};
    return from_cuda(kda::launch_linear(p, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t kda_testing_linear_row_tiles(int64_t M, int64_t K, kda_dtype_t out_dtype) {
    return M > 0 && K > 0 && dtype_ok(out_dtype) ? kda::linear_row_tiles(M) : 0;
}

size_t kda_decay_prefill_workspace_size(int64_t total_tokens, int num_seqs, int H, int dk, int dv,
                                        kda_dtype_t dtype) {
    if (total_tokens <= 0 || total_tokens >= kMax31 || num_seqs <= 0 || H <= 0 || (int64_t)num_seqs * H >= kMax31 ||
        !dtype_ok(dtype) || !dim_ok(dk) || !dim_ok(dv))
        return 0;
    size_t bytes = kda::decay_prefill_simt_workspace(total_tokens, num_seqs, H, dk, dv);
    if (dtype == KDA_BF16) {
        const size_t tc = kda::decay_prefill_tc_workspace(total_tokens, num_seqs, H, dk, dv);
        if (tc > bytes) bytes = tc;
    }
    return (bytes + 255) & ~size_t(255);
}

kda_status_t kda_decay_prefill(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                               int64_t ldv, const float *log_decay, const int32_t *cu_seqlens, int num_seqs,
                               int64_t total_tokens, int H, int dk, int dv, kda_dtype_t dtype, float scale,
                               const float *initial_state, float *final_state, void *out, void *workspace,
                               size_t workspace_bytes, uint32_t *status, kda_stream_t stream) {
    if (num_seqs < 0 || total_tokens < 0 || H <= 0 || dk <= 0 || dv <= 0) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || !dim_ok(dk) || !dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if (total_tokens >= kMax31 || (int64_t)num_seqs * H >= kMax31 || (int64_t)H * dk >= kMax31 ||
        (int64_t)H * dv >= kMax31)
        return KDA_ERR_UNSUPPORTED;
    if (ldq < (int64_t)H * dk || ldk < (int64_t)H * dk || ldv < (int64_t)H * dv) return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0) return KDA_OK;
    if (!log_decay || !cu_seqlens) return KDA_ERR_INVALID_ARG;
    if (total_tokens > 0 && (!q || !k || !v || !out)) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, elem(dtype)) || !aligned(k, elem(dtype)) || !aligned(v, elem(dtype)) ||
        !aligned(out, elem(dtype)) || !aligned(initial_state, 16) || !aligned(final_state, 16) ||
        !aligned(workspace, 16) || !words(log_decay, cu_seqlens, status))
        return KDA_ERR_INVALID_ARG;
    const kda::DecayParams p{q, k, v, ldq, ldk, ldv, log_decay, cu_seqlens, num_seqs, H, total_tokens, scale,
                             initial_state, final_state, out, status};
    // TMA copies start on 16-byte boundaries
    if (dtype == KDA_BF16 && total_tokens > 0 && aligned(q, 16) && aligned(k, 16) &&
        aligned(v, 16) && aligned(out, 16) && ldq % 8 == 0 && ldk % 8 == 0 && ldv % 8 == 0)
        return from_cuda(kda::launch_decay_prefill_tc(p, dk, dv, workspace, workspace_bytes,
                                                      reinterpret_cast<cudaStream_t>(stream)));
    return from_cuda(kda::launch_decay_prefill_simt(p, dk, dv, dtype == KDA_BF16, workspace, workspace_bytes,
                                                    reinterpret_cast<cudaStream_t>(stream)));
}

kda_status_t kda_decay_decode(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                              int64_t ldv, const float *log_decay, float *state_pool, int pool_size,
                              const int32_t *slot_ids, void *out, int N, int H, int dk, int dv,
                              kda_dtype_t dtype, float scale, uint32_t *status, kda_stream_t stream) {
    if (N < 0 || pool_size < 0 || H <= 0 || dk <= 0 || dv <= 0) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || !dim_ok(dk) || !dim_ok(dv)) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)N * H >= kMax31 || (int64_t)H * dk >= kMax31 || (int64_t)H * dv >= kMax31)
        return KDA_ERR_UNSUPPORTED;
    if (ldq < (int64_t)H * dk || ldk < (int64_t)H * dk || ldv < (int64_t)H * dv) return KDA_ERR_INVALID_ARG;
    if (N == 0) return KDA_OK;
    if (!slot_ids && pool_size < N) return KDA_ERR_INVALID_ARG;
    if (!q || !k || !v || !log_decay || !state_pool || !out) return KDA_ERR_INVALID_ARG;
    if (!aligned(q, elem(dtype)) || !aligned(k, elem(dtype)) || !aligned(v, elem(dtype)) ||
        !aligned(out, elem(dtype)) || !aligned(state_pool, 16) || !words(log_decay, slot_ids, status))
        return KDA_ERR_INVALID_ARG;
    const kda::DecayStepParams p{q, k, v, ldq, ldk, ldv, log_decay, state_pool, pool_size, slot_ids,
                                 out, N, H, scale, status};
    return from_cuda(kda::launch_decay_decode(p, dk, dv, dtype == KDA_BF16,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

kda_status_t kda_paged_append(const void *k, int64_t ldk, const void *v, int64_t ldv, void *k_cache,
                              void *v_cache, int num_pages, int page_size, const int32_t *page_table,
                              int max_pages, const int32_t *start_pos, const int32_t *cu_seqlens,
                              int num_seqs, int64_t total_tokens, int Hkv, int d, kda_dtype_t dtype,
                              uint32_t *status, kda_stream_t stream) {
    if (num_pages < 0 || max_pages < 0 || num_seqs < 0 || total_tokens < 0 || Hkv <= 0 || d <= 0)
        return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || !dim_ok(d) || page_shift(page_size) < 0) return KDA_ERR_UNSUPPORTED;
    if (total_tokens >= kMax31 || (int64_t)Hkv * d >= kMax31) return KDA_ERR_UNSUPPORTED;
    if (ldk < (int64_t)Hkv * d || ldv < (int64_t)Hkv * d) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens && total_tokens != num_seqs) return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
    if (!k || !v || !k_cache || !v_cache || !page_table || !start_pos) return KDA_ERR_INVALID_ARG;
    const int64_t e = elem(dtype);
    if (!aligned(k, e) || !aligned(v, e) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !words(page_table, start_pos, cu_seqlens, status))
        return KDA_ERR_INVALID_ARG;
    const kda::AppendParams p{k, v, ldk * e, ldv * e, k_cache, v_cache, num_pages, page_shift(page_size),
                              page_table, max_pages, start_pos, cu_seqlens, num_seqs, Hkv, total_tokens,
                              (int)(d * e), 0, status};
    const bool vec16 = aligned(k, 16) && aligned(v, 16) && (ldk * e) % 16 == 0 && (ldv * e) % 16 == 0;
    return from_cuda(kda::launch_paged_append(p, vec16, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_paged_decode_workspace_size(int num_seqs, int64_t max_tokens, int Hq, int Hkv, int d,
                                       kda_dtype_t dtype) {
    if (num_seqs <= 0 || max_tokens < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || !dim_ok(d) || !dtype_ok(dtype)) return 0;
    return (kda::paged_decode_workspace_bytes(num_seqs, max_tokens, Hq, Hkv, d) + 255) & ~size_t(255);
}

kda_status_t kda_paged_decode(const void *q, int64_t ldq, const void *k_cache, const void *v_cache,
                              int num_pages, int page_size, const int32_t *page_table, int max_pages,
                              const int32_t *seq_lens, int num_seqs, int Hq, int Hkv, int d,
                              kda_dtype_t dtype, float scale, void *out, float *lse, void *workspace,
                              size_t workspace_bytes, uint32_t *status, kda_stream_t stream) {
    if (num_pages < 0 || max_pages < 0 || num_seqs < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv)
        return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || !dim_ok(d) || page_shift(page_size) < 0) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)num_seqs * Hq >= kMax31 || (int64_t)Hq * d >= kMax31 ||
        (int64_t)max_pages * page_size > (int64_t(1) << 30))
        return KDA_ERR_UNSUPPORTED;
    if (ldq < (int64_t)Hq * d) return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0) return KDA_OK;
    if (!q || !seq_lens || !out) return KDA_ERR_INVALID_ARG;
    // (a page's id is read before it is compared with num_pages)
    if (max_pages > 0 && (!page_table || (num_pages > 0 && (!k_cache || !v_cache)))) return KDA_ERR_INVALID_ARG;
    const int64_t e = elem(dtype);
    if (!aligned(q, e) || !aligned(out, e) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !words(page_table, seq_lens, lse, status))
        return KDA_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) ||
        workspace_bytes < kda_paged_decode_workspace_size(num_seqs, (int64_t)max_pages * page_size, Hq, Hkv, d, dtype))
        return KDA_ERR_INVALID_ARG;
    kda::PagedParams p{q, ldq, k_cache, v_cache, num_pages, page_shift(page_size), page_table, max_pages,
                             seq_lens, num_seqs, Hq, Hkv, Hq / Hkv, scale, out, lse,
                             static_cast<float *>(workspace), false, 0, status};
    return from_cuda(kda::launch_paged_decode(p, d, dtype == KDA_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status_t kda_paged_append_q8(const void *k, int64_t ldk, const void *v, int64_t ldv, void *k_cache,
                                 void *v_cache, float *k_scale, float *v_scale, int num_pages, int page_size,
                                 int block, const int32_t *page_table, int max_pages, const int32_t *start_pos,
                                 const int32_t *cu_seqlens, int num_seqs, int64_t total_tokens, int Hkv, int d,
                                 kda_dtype_t dtype, uint32_t *status, kda_stream_t stream) {
    if (num_pages < 0 || max_pages < 0 || num_seqs < 0 || total_tokens < 0 || Hkv <= 0 || d <= 0)
        return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || !dim_ok(d) || page_shift(page_size) < 0 || block_shift(block, page_size) < 0)
        return KDA_ERR_UNSUPPORTED;
    if (total_tokens >= kMax31 || (int64_t)Hkv * d >= kMax31) return KDA_ERR_UNSUPPORTED;
    if (ldk < (int64_t)Hkv * d || ldv < (int64_t)Hkv * d) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens && total_tokens != num_seqs) return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_tokens == 0) return KDA_OK;
    if (!k || !v || !k_cache || !v_cache || !k_scale || !v_scale || !page_table || !start_pos) return KDA_ERR_INVALID_ARG;
    const int64_t e = elem(dtype);
    if (!aligned(k, e) || !aligned(v, e) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !words(k_scale, v_scale, page_table, start_pos, cu_seqlens, status))
        return KDA_ERR_INVALID_ARG;
    const kda::AppendQ8Params p{k, v, ldk, ldv, static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache),
                                k_scale, v_scale, num_pages, page_shift(page_size), block_shift(block, page_size),
                                page_table, max_pages, start_pos, cu_seqlens, num_seqs, Hkv, total_tokens, status};
    const bool vec16 = aligned(k, 16) && aligned(v, 16) && (ldk * e) % 16 == 0 && (ldv * e) % 16 == 0;
    return from_cuda(kda::launch_paged_append_q8(p, d, dtype == KDA_BF16, vec16, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_paged_decode_q8_workspace_size(int num_seqs, int64_t max_tokens, int Hq, int Hkv, int d,
                                          kda_dtype_t dtype) {
    if (num_seqs <= 0 || max_tokens < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || !dim_ok(d) || !dtype_ok(dtype)) return 0;
    return (kda::paged_decode_q8_workspace_bytes(num_seqs, max_tokens, Hq, Hkv, d) + 255) & ~size_t(255);
}

kda_status_t kda_paged_decode_q8(const void *q, int64_t ldq, const void *k_cache, const void *v_cache,
                                 const float *k_scale, const float *v_scale, int num_pages, int page_size, int block,
                                 const int32_t *page_table, int max_pages, const int32_t *seq_lens, int num_seqs,
                                 int Hq, int Hkv, int d, kda_dtype_t dtype, float scale, void *out, float *lse,
                                 void *workspace, size_t workspace_bytes, uint32_t *status, kda_stream_t stream) {
    if (num_pages < 0 || max_pages < 0 || num_seqs < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv)
        return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || !dim_ok(d) || page_shift(page_size) < 0 || block_shift(block, page_size) < 0)
        return KDA_ERR_UNSUPPORTED;
    if ((int64_t)num_seqs * Hq >= kMax31 || (int64_t)Hq * d >= kMax31 ||
        (int64_t)max_pages * page_size > (int64_t(1) << 30))
        return KDA_ERR_UNSUPPORTED;
    if (ldq < (int64_t)Hq * d) return KDA_ERR_INVALID_ARG;
    if (num_seqs == 0) return KDA_OK;
    if (!q || !seq_lens || !out) return KDA_ERR_INVALID_ARG;
    if (max_pages > 0 && (!page_table || (num_pages > 0 && (!k_cache || !v_cache || !k_scale || !v_scale))))
        return KDA_ERR_INVALID_ARG;
    const int64_t e = elem(dtype);
    if (!aligned(q, e) || !aligned(out, e) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !words(k_scale, v_scale, page_table, seq_lens, lse, status))
        return KDA_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes,
                      kda_paged_decode_q8_workspace_size(num_seqs, (int64_t)max_pages * page_size, Hq, Hkv, d, dtype)))
        return KDA_ERR_INVALID_ARG;
    kda::PagedQ8Params p{{q, ldq, k_cache, v_cache, num_pages, page_shift(page_size), page_table, max_pages,
                          seq_lens, num_seqs, Hq, Hkv, Hq / Hkv, scale, out, lse,
                          static_cast<float *>(workspace), false, 0, status},
                         k_scale, v_scale, block_shift(block, page_size)};
    return from_cuda(kda::launch_paged_decode_q8(p, d, dtype == KDA_BF16, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_pages_resize_workspace_size(int num_rows, int max_pages, int num_pages) {
    if (num_rows < 0 || max_pages < 0 || num_pages < 0 || !table_ok(num_rows, max_pages)) return 0;
    return (kda::pages_resize_workspace_bytes(num_pages) + 255) & ~size_t(255);
}

kda_status_t kda_pages_resize(int32_t *page_table, int num_rows, int max_pages, int32_t *held, int32_t *refs,
                              int num_pages, const int32_t *tokens, int page_size, void *workspace,
                              size_t workspace_bytes, uint32_t *status, kda_stream_t stream) {
    if (num_rows < 0 || max_pages < 0 || num_pages < 0) return KDA_ERR_INVALID_ARG;
    if (page_shift(page_size) < 0 || !table_ok(num_rows, max_pages)) return KDA_ERR_UNSUPPORTED;
    if (num_rows == 0) return KDA_OK;
    if (!held || !tokens || (max_pages > 0 && !page_table) || (num_pages > 0 && !refs)) return KDA_ERR_INVALID_ARG;
    if (!words(page_table, held, refs, tokens, status) ||
        !workspace_ok(workspace, workspace_bytes, kda::pages_resize_workspace_bytes(num_pages)))
        return KDA_ERR_INVALID_ARG;
    const kda::PageTable p{page_table, num_rows, max_pages, held, refs, num_pages, page_shift(page_size), status};
    return from_cuda(kda::launch_pages_resize(p, tokens, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_pages_fork_workspace_size(int num_rows, int max_pages, int num_forks) {
    if (num_rows < 0 || max_pages < 0 || num_forks < 0 || !table_ok(num_rows, max_pages)) return 0;
    return (kda::pages_fork_workspace_bytes(num_rows, num_forks) + 255) & ~size_t(255);
}

kda_status_t kda_pages_fork(void *const *pools, const int64_t *page_bytes, int num_pools, int32_t *page_table,
                            int num_rows, int max_pages, int32_t *held, int32_t *refs, int num_pages, int32_t *lens,
                            const int32_t *src, const int32_t *dst, int num_forks, int page_size, void *workspace,
                            size_t workspace_bytes, uint32_t *status, kda_stream_t stream) {
    if (num_pools < 0 || num_rows < 0 || max_pages < 0 || num_pages < 0 || num_forks < 0) return KDA_ERR_INVALID_ARG;
    if (page_shift(page_size) < 0 || !table_ok(num_rows, max_pages)) return KDA_ERR_UNSUPPORTED;
    if (!pools_ok(pools, page_bytes, num_pools)) return KDA_ERR_INVALID_ARG;
    if (num_forks == 0) return KDA_OK;
    if (!src || !dst || (num_rows > 0 && (!held || !lens)) || ((int64_t)num_rows * max_pages > 0 && !page_table) ||
        (num_pages > 0 && !refs) || !workspace)
        return KDA_ERR_INVALID_ARG;
    if (!words(page_table, held, refs, lens, src, dst, status) || !aligned(workspace, 16) ||
        workspace_bytes < kda::pages_fork_workspace_bytes(num_rows, num_forks))
        return KDA_ERR_INVALID_ARG;
    const kda::PageTable p{page_table, num_rows, max_pages, held, refs, num_pages, page_shift(page_size), status};
    return from_cuda(kda::launch_pages_fork(pools, page_bytes, num_pools, p, lens, src, dst, num_forks, workspace,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_pages_compact_workspace_size(int num_pages) {
    if (num_pages < 0) return 0;
    return (kda::pages_compact_workspace_bytes(num_pages) + 255) & ~size_t(255);
}

kda_status_t kda_pages_compact(void *const *pools, const int64_t *page_bytes, int num_pools, int32_t *page_table,
                               int num_rows, int max_pages, int32_t *refs, int num_pages, int32_t *page_map,
                               int32_t *live, void *workspace, size_t workspace_bytes, uint32_t *status,
                               kda_stream_t stream) {
    if (num_pools < 0 || num_rows < 0 || max_pages < 0 || num_pages < 0) return KDA_ERR_INVALID_ARG;
    if (!pools_ok(pools, page_bytes, num_pools)) return KDA_ERR_INVALID_ARG;
    if (!live || !workspace || ((int64_t)num_rows * max_pages > 0 && !page_table) || (num_pages > 0 && (!refs || !page_map)))
        return KDA_ERR_INVALID_ARG;
    if (!words(page_table, refs, page_map, live, status) || !aligned(workspace, 16) ||
        workspace_bytes < kda::pages_compact_workspace_bytes(num_pages))
        return KDA_ERR_INVALID_ARG;
    const kda::PageTable p{page_table, num_rows, max_pages, nullptr, refs, num_pages, 0, status};
    return from_cuda(kda::launch_pages_compact(pools, page_bytes, num_pools, p, page_map, live, workspace,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
