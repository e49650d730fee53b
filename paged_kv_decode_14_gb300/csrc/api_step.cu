// Entry points of a serving step that stays on the GPU (masked attention over the cache, block tables, accepted
// paths): argument checks and dispatch.  Declarations and contracts: include/pagedkv.h.
#include <cmath>

#include "api_checks.cuh"

namespace pkv {
cudaError_t launch_masked(const pkv_cache& c, const pkv_rows* q, const pkv_rows* out, float* lse, int64_t num_q_rows,
                          const int32_t* tables, int max_blocks, const int32_t* ctx_lens, const int32_t* q_lens,
                          const int64_t* q_starts, int num_seqs, int max_q_len, int window, int sinks, const int32_t* tree,
                          int tree_words, float scale, void* workspace, cudaStream_t st);
size_t masked_workspace_bytes();
bool block_tables_fit(int num_seqs);
cudaError_t launch_block_tables(int32_t* table, int max_blocks, int32_t* lens, const int32_t* grow, int num_seqs,
                                int32_t* free_blocks, int32_t* free_count, int64_t num_blocks, int64_t* slots,
                                int32_t* positions, int32_t* granted, int64_t* row_starts, int64_t num_rows, bool pad,
                                int* err, cudaStream_t st);
cudaError_t launch_keep_path(const pkv_cache& c, const int32_t* tables, int max_blocks, const int32_t* ctx_lens,
                             const int32_t* q_lens, const int32_t* path, int max_path, const int32_t* path_lens,
                             int num_seqs, int* err, cudaStream_t st);

namespace {

// What both masked attentions check; *empty: nothing to do.
pkv_status check_masked(const pkv_cache* cache, const pkv_rows* q, const pkv_rows* out, int64_t num_q_rows,
                        const int32_t* tables, int32_t max_blocks, const int32_t* ctx_lens, const int32_t* q_lens,
                        int32_t num_seqs, int32_t max_q_len, float scale, const void* workspace, size_t workspace_bytes,
                        bool* empty) {
    *empty = false;
    const pkv_status s = check_cache(cache);
    if (s != PKV_OK) return s;
    if (num_seqs < 0 || num_q_rows < 0 || max_q_len < 1) return PKV_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return PKV_ERR_INVALID_ARG;
    // (positions and queries of a block behind the last stay below 2^31)
    if (num_q_rows > 0x7fffff00 || max_q_len > 0x7fffff00 - 256) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_q_rows == 0) {
        *empty = true;
        return PKV_OK;
    }
    if (!tables || !ctx_lens || !q_lens || max_blocks <= 0) return PKV_ERR_INVALID_ARG;
    if (!rows_ok(q, num_q_rows, 2, cache->head_dim, false) || !rows_ok(out, num_q_rows, 2, cache->head_dim, true))
        return PKV_ERR_INVALID_ARG;
    if (q->num_heads != out->num_heads || q->num_heads % cache->num_kv_heads) return PKV_ERR_INVALID_ARG;
    if (q->num_heads / cache->num_kv_heads > 128) return PKV_ERR_UNSUPPORTED;
    // (the tensor copies take positive strides only)
    if ((num_q_rows > 1 && q->token_stride <= 0) || (q->num_heads > 1 && q->head_stride <= 0)) return PKV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < pkv_masked_workspace_size()) return PKV_ERR_WORKSPACE;
    if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    return PKV_OK;
}

pkv_status update_tables(int32_t* block_tables, int32_t max_blocks_per_seq, int32_t* context_lens, const int32_t* grow,
                         int32_t num_seqs, int32_t* free_blocks, int32_t* free_count, int64_t num_blocks, int64_t* slots,
                         int32_t* positions, int32_t* granted, int64_t* row_starts, int64_t num_rows, bool pad,
                         int32_t* device_error, cudaStream_t st) {
    if (num_seqs < 0 || num_rows < 0 || num_blocks <= 0 || max_blocks_per_seq <= 0) return PKV_ERR_INVALID_ARG;
    if (!block_tables_fit(num_seqs) || num_rows > 0x7fffff00 || num_blocks > 0x7fffffff ||
        (int64_t)max_blocks_per_seq * kBlock > 0x7fffffff)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) {
        if (!pad || num_rows == 0) return PKV_OK;
        if (!slots) return PKV_ERR_INVALID_ARG;
        cudaError_t e = cudaMemsetAsync(slots, 0xff, (size_t)num_rows * sizeof(*slots), st);
        if (e == cudaSuccess && positions) e = cudaMemsetAsync(positions, 0, (size_t)num_rows * sizeof(*positions), st);
        return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
    }
    if (!block_tables || !context_lens || !grow || !free_blocks || !free_count || (num_rows > 0 && !slots))
        return PKV_ERR_INVALID_ARG;
    return launch_block_tables(block_tables, max_blocks_per_seq, context_lens, grow, num_seqs, free_blocks, free_count,
                               num_blocks, slots, positions, granted, row_starts, num_rows, pad, device_error,
                               st) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

PKV_API size_t pkv_masked_workspace_size(void) { return masked_workspace_bytes(); }

PKV_API pkv_status pkv_paged_attention_window(const pkv_cache* cache, const pkv_rows* q, const pkv_rows* out, float* lse,
                                              int64_t num_q_rows, const int32_t* block_tables, int32_t max_blocks_per_seq,
                                              const int32_t* context_lens, const int32_t* q_lens, const int64_t* q_starts,
                                              int32_t num_seqs, int32_t max_q_len, int32_t window, int32_t sinks,
                                              float scale, void* workspace, size_t workspace_bytes, void* stream) {
    bool empty;
    if (window < 1 || sinks < 0) return PKV_ERR_INVALID_ARG;
    const pkv_status s = check_masked(cache, q, out, num_q_rows, block_tables, max_blocks_per_seq, context_lens, q_lens,
                                      num_seqs, max_q_len, scale, workspace, workspace_bytes, &empty);
    if (s != PKV_OK || empty) return s;
    return launch_masked(*cache, q, out, lse, num_q_rows, block_tables, max_blocks_per_seq, context_lens, q_lens, q_starts,
                         num_seqs, max_q_len, window, sinks, nullptr, 0, scale, workspace,
                         (cudaStream_t)stream) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

PKV_API pkv_status pkv_paged_attention_tree(const pkv_cache* cache, const pkv_rows* q, const pkv_rows* out, float* lse,
                                            int64_t num_q_rows, const int32_t* block_tables, int32_t max_blocks_per_seq,
                                            const int32_t* context_lens, const int32_t* q_lens, const int64_t* q_starts,
                                            int32_t num_seqs, int32_t max_q_len, const int32_t* tree_mask,
                                            int32_t mask_words, float scale, void* workspace, size_t workspace_bytes,
                                            void* stream) {
    bool empty;
    if (max_q_len < 1 || mask_words < 0 || (int64_t)mask_words * 32 < max_q_len) return PKV_ERR_INVALID_ARG;
    const pkv_status s = check_masked(cache, q, out, num_q_rows, block_tables, max_blocks_per_seq, context_lens, q_lens,
                                      num_seqs, max_q_len, scale, workspace, workspace_bytes, &empty);
    if (s != PKV_OK || empty) return s;
    if (!tree_mask) return PKV_ERR_INVALID_ARG;
    return launch_masked(*cache, q, out, lse, num_q_rows, block_tables, max_blocks_per_seq, context_lens, q_lens, q_starts,
                         num_seqs, max_q_len, 1, 0, tree_mask, mask_words, scale, workspace,
                         (cudaStream_t)stream) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

PKV_API pkv_status pkv_block_tables_update(int32_t* block_tables, int32_t max_blocks_per_seq, int32_t* context_lens,
                                           const int32_t* grow, int32_t num_seqs, int32_t* free_blocks,
                                           int32_t* free_count, int64_t num_blocks, int64_t* slots, int32_t* positions,
                                           int32_t* granted, int64_t* row_starts, int64_t num_rows,
                                           int32_t* device_error, void* stream) {
    return update_tables(block_tables, max_blocks_per_seq, context_lens, grow, num_seqs, free_blocks, free_count, num_blocks,
                         slots, positions, granted, row_starts, num_rows, false, device_error, (cudaStream_t)stream);
}

PKV_API pkv_status pkv_block_tables_update_padded(int32_t* block_tables, int32_t max_blocks_per_seq,
                                                  int32_t* context_lens, const int32_t* grow, int32_t num_seqs,
                                                  int32_t* free_blocks, int32_t* free_count, int64_t num_blocks,
                                                  int64_t* slots, int32_t* positions, int32_t* granted,
                                                  int64_t* row_starts, int64_t num_rows, int32_t* device_error,
                                                  void* stream) {
    return update_tables(block_tables, max_blocks_per_seq, context_lens, grow, num_seqs, free_blocks, free_count, num_blocks,
                         slots, positions, granted, row_starts, num_rows, true, device_error, (cudaStream_t)stream);
}

PKV_API pkv_status pkv_paged_kv_keep_path(const pkv_cache* cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                                          const int32_t* context_lens, const int32_t* q_lens, const int32_t* path,
                                          int32_t max_path, const int32_t* path_lens, int32_t num_seqs,
                                          int32_t* device_error, void* stream) {
    const pkv_status s = check_cache(cache);
    if (s != PKV_OK) return s;
    if (num_seqs < 0 || max_path < 0) return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0) return PKV_OK;
    if (!block_tables || !context_lens || !q_lens || !path_lens || (max_path > 0 && !path) || max_blocks_per_seq <= 0)
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)num_seqs * cache->num_kv_heads > 0x7fffffff / 2 || max_path > 0x7fffffff / 16 - 128) return PKV_ERR_UNSUPPORTED;
    return launch_keep_path(*cache, block_tables, max_blocks_per_seq, context_lens, q_lens, path, max_path, path_lens,
                            num_seqs, device_error, (cudaStream_t)stream) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

}  // extern "C"
