// Entry points over rows of projections: argument checks and dispatch.
// Declarations and contracts: include/pagedkv.h.
#include <cmath>

#include "common.cuh"

namespace pkv {
pkv_status check_cache(const pkv_cache* c);
int num_sms_current();
cudaError_t launch_qk_norm_rope(const pkv_rows* q_in, const pkv_rows* q_out, const pkv_rows* k_in,
                                const pkv_rows* k_out, int dtype, int D, int64_t T, const int32_t* positions,
                                const pkv_rope* rope, bool inverse, const void* qw, const void* kw, float eps,
                                cudaStream_t st, int num_sms);
cudaError_t launch_append_norm_rope(const pkv_cache& c, const pkv_rows* q_in, const pkv_rows* q_out, const pkv_rows* k,
                                    const pkv_rows* v, const pkv_rows* k_out, const int64_t* slots, int64_t T,
                                    const int32_t* positions, const pkv_rope* rope, const void* qw, const void* kw,
                                    float eps, bool fresh, int* err, cudaStream_t st, int num_sms);
cudaError_t launch_cache_read(const pkv_cache& c, const int32_t* tables, int max_blocks, const int32_t* starts,
                              const int32_t* lens, int num_seqs, int64_t num_rows, const pkv_rows* k,
                              const pkv_rows* v, int dtype, int* err, cudaStream_t st);
cudaError_t launch_prompt(const pkv_rows* q, const pkv_rows* k, const pkv_rows* v, const pkv_rows* out, float* lse,
                          int dtype, int head_dim, int64_t num_q_rows, int64_t num_kv_rows, const int32_t* q_lens,
                          const int32_t* kv_lens, const int64_t* q_starts, const int64_t* kv_starts, int num_seqs,
                          int max_q_len, float scale, void* workspace, int* err, cudaStream_t st);
size_t prompt_workspace_bytes();

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Rows the kernels may touch in 16-byte pieces; out: no two of them share memory (all heads of a token lie
// between two tokens' starts, or all tokens of a head between two heads').
bool rows_ok(const pkv_rows* r, int64_t tokens, int elem_bytes, int head_dim, bool out) {
    if (!r || !r->data || r->num_heads < 1 || !aligned16(r->data)) return false;
    if (tokens > 1 && (r->token_stride * elem_bytes) % 16) return false;
    if (r->num_heads > 1 && (r->head_stride * elem_bytes) % 16) return false;
    if (!out || (tokens <= 1 && r->num_heads == 1)) return true;
    const __int128 ts = tokens > 1 ? r->token_stride : 0, hs = r->num_heads > 1 ? r->head_stride : 0;
    const __int128 t = ts < 0 ? -ts : ts, h = hs < 0 ? -hs : hs;
    if ((tokens > 1 && t < head_dim) || (r->num_heads > 1 && h < head_dim)) return false;
    return tokens == 1 || r->num_heads == 1 || t >= h * (r->num_heads - 1) + head_dim || h >= t * (tokens - 1) + head_dim;
}

bool rope_ok(const pkv_rope* r, int head_dim, const int32_t* positions) {
    if (!r || r->rotary_dim == 0) return true;
    if (r->rotary_dim < 0 || r->rotary_dim % 2 || r->rotary_dim > head_dim || r->rotary_dim > 2 * PKV_ROPE_MAX_PAIRS)
        return false;
    if (!positions || !std::isfinite(r->magnitude)) return false;
    for (int i = 0; i < r->rotary_dim / 2; ++i)
        if (!(std::fabs(r->inv_freq[i]) < 1e9)) return false;
    return true;
}

bool norm_ok(const void* qw, const void* kw, float eps) {
    if (!(eps >= 0.f)) return !qw && !kw && eps == eps;
    return eps < INFINITY && aligned16(qw) && aligned16(kw);
}

int elem_bytes_of(int dtype) { return dtype == PKV_FP32 ? 4 : 2; }

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

PKV_API pkv_status pkv_rope_init(pkv_rope* rope, int32_t rotary_dim, int32_t interleaved, double theta,
                                 int32_t scaling, double factor, int64_t original_len, double low, double high) {
    if (!rope || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > 2 * PKV_ROPE_MAX_PAIRS) return PKV_ERR_INVALID_ARG;
    if (!(theta > 1.0) || !std::isfinite(theta)) return PKV_ERR_INVALID_ARG;
    if (scaling < PKV_ROPE_NONE || scaling > PKV_ROPE_RAMP) return PKV_ERR_INVALID_ARG;
    if (scaling != PKV_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return PKV_ERR_INVALID_ARG;
    if (scaling == PKV_ROPE_NTK && rotary_dim < 4) return PKV_ERR_INVALID_ARG;
    const bool banded = scaling == PKV_ROPE_BANDS || scaling == PKV_ROPE_RAMP;
    if (banded && (original_len < 1 || !(low > 0.0) || !(high > low) || !std::isfinite(high))) return PKV_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586477, rd = rotary_dim;
    *rope = pkv_rope{};
    rope->rotary_dim = rotary_dim;
    rope->interleaved = interleaved != 0;
    rope->magnitude = scaling == PKV_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    const double base = scaling == PKV_ROPE_NTK ? theta * std::pow(factor, rd / (rd - 2.0)) : theta;
    const auto idx = [&](double turns) {
        return rd * std::log((double)original_len / (two_pi * turns)) / (2.0 * std::log(theta));
    };
    const double lo = banded ? std::fmax(0.0, std::floor(idx(high))) : 0.0;
    const double hi = banded ? std::fmin(rd - 1.0, std::ceil(idx(low))) : 0.0;
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rd);
        if (scaling == PKV_ROPE_LINEAR) {
            f /= factor;
        } else if (scaling == PKV_ROPE_BANDS) {
            const double r = (double)original_len * f / two_pi;
            const double t = std::fmin(1.0, std::fmax(0.0, (r - low) / (high - low)));
            f *= t + (1.0 - t) / factor;
        } else if (scaling == PKV_ROPE_RAMP) {
            const double u = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 0.001)));
            f *= (1.0 - u) + u / factor;
        }
        rope->inv_freq[i] = f;
    }
    return PKV_OK;
}

PKV_API pkv_status pkv_qk_norm_rope(const pkv_rows* q_in, const pkv_rows* q_out, const pkv_rows* k_in,
                                    const pkv_rows* k_out, int32_t dtype, int32_t head_dim, int64_t num_tokens,
                                    const int32_t* positions, const pkv_rope* rope, int32_t inverse,
                                    const void* q_weight, const void* k_weight, float norm_eps, void* stream) {
    if (dtype < PKV_BF16 || dtype > PKV_FP32) return PKV_ERR_INVALID_ARG;
    const int e = elem_bytes_of(dtype);
    if (head_dim <= 0 || num_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (head_dim > 256 || (head_dim * e) % 16 || num_tokens > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
    if (!k_in != !k_out) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!rope_ok(rope, head_dim, positions) || !norm_ok(q_weight, k_weight, norm_eps)) return PKV_ERR_INVALID_ARG;
    if (inverse && norm_eps >= 0.f) return PKV_ERR_INVALID_ARG;
    if (!rows_ok(q_in, num_tokens, e, head_dim, false) || !rows_ok(q_out, num_tokens, e, head_dim, true))
        return PKV_ERR_INVALID_ARG;
    if (q_in->num_heads != q_out->num_heads) return PKV_ERR_INVALID_ARG;
    if (k_in) {
        if (!rows_ok(k_in, num_tokens, e, head_dim, false) || !rows_ok(k_out, num_tokens, e, head_dim, true))
            return PKV_ERR_INVALID_ARG;
        if (k_in->num_heads != k_out->num_heads) return PKV_ERR_INVALID_ARG;
    }
    const int sms = num_sms_current();
    if (sms <= 0) return PKV_ERR_CUDA;
    return launch_qk_norm_rope(q_in, q_out, k_in, k_out, dtype, head_dim, num_tokens, positions, rope, inverse != 0,
                               q_weight, k_weight, norm_eps, (cudaStream_t)stream, sms) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

PKV_API pkv_status pkv_paged_kv_append_norm_rope(const pkv_cache* cache, const pkv_rows* q_in, const pkv_rows* q_out,
                                                 const pkv_rows* k, const pkv_rows* v, const pkv_rows* k_out,
                                                 const int64_t* slot_mapping, int64_t num_tokens,
                                                 const int32_t* positions, const pkv_rope* rope, const void* q_weight,
                                                 const void* k_weight, float norm_eps,
                                                 int32_t fp8_scales_from_values, int32_t* device_error, void* stream) {
    const pkv_status s = check_cache(cache);
    if (s != PKV_OK) return s;
    const int D = cache->head_dim;
    if (num_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (num_tokens > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
    if (!q_in != !q_out) return PKV_ERR_INVALID_ARG;
    if (fp8_scales_from_values && cache->kv_dtype != PKV_KV_FP8_E4M3) return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!rope_ok(rope, D, positions) || !norm_ok(q_weight, k_weight, norm_eps)) return PKV_ERR_INVALID_ARG;
    if (!slot_mapping || !rows_ok(k, num_tokens, 2, D, false) || !rows_ok(v, num_tokens, 2, D, false))
        return PKV_ERR_INVALID_ARG;
    if (k->num_heads != cache->num_kv_heads || v->num_heads != cache->num_kv_heads) return PKV_ERR_INVALID_ARG;
    if (k_out && (!rows_ok(k_out, num_tokens, 2, D, true) || k_out->num_heads != cache->num_kv_heads))
        return PKV_ERR_INVALID_ARG;
    if (q_in) {
        if (!rows_ok(q_in, num_tokens, 2, D, false) || !rows_ok(q_out, num_tokens, 2, D, true)) return PKV_ERR_INVALID_ARG;
        if (q_in->num_heads != q_out->num_heads || q_in->num_heads % cache->num_kv_heads) return PKV_ERR_INVALID_ARG;
    }
    const int sms = num_sms_current();
    if (sms <= 0) return PKV_ERR_CUDA;
    return launch_append_norm_rope(*cache, q_in, q_out, k, v, k_out, slot_mapping, num_tokens, positions, rope, q_weight,
                                   k_weight, norm_eps, fp8_scales_from_values != 0, device_error, (cudaStream_t)stream,
                                   sms) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

PKV_API pkv_status pkv_paged_kv_read(const pkv_cache* cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                                     const int32_t* starts, const int32_t* lens, int32_t num_seqs, int64_t num_rows,
                                     const pkv_rows* k_out, const pkv_rows* v_out, int32_t dtype,
                                     int32_t* device_error, void* stream) {
    const pkv_status s = check_cache(cache);
    if (s != PKV_OK) return s;
    if (dtype < PKV_BF16 || dtype > PKV_FP32 || num_seqs < 0 || num_rows < 0) return PKV_ERR_INVALID_ARG;
    const int e = elem_bytes_of(dtype), D = cache->head_dim;
    for (const pkv_rows* r : {k_out, v_out}) {
        if (!r || num_rows == 0) continue;
        if (!rows_ok(r, num_rows, e, D, true) || r->num_heads != cache->num_kv_heads) return PKV_ERR_INVALID_ARG;
    }
    if (num_seqs == 0 || num_rows == 0 || (!k_out && !v_out)) return PKV_OK;
    if (!block_tables || !lens || max_blocks_per_seq <= 0) return PKV_ERR_INVALID_ARG;
    if (num_rows / kBlock + 2 * (int64_t)num_seqs > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
    return launch_cache_read(*cache, block_tables, max_blocks_per_seq, starts, lens, num_seqs, num_rows, k_out, v_out,
                             dtype, device_error, (cudaStream_t)stream) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

PKV_API size_t pkv_prompt_workspace_size(void) { return prompt_workspace_bytes(); }

PKV_API pkv_status pkv_prompt_attention(const pkv_rows* q, const pkv_rows* k, const pkv_rows* v, const pkv_rows* out,
                                        float* lse, int32_t dtype, int32_t head_dim, int64_t num_q_rows,
                                        int64_t num_kv_rows, const int32_t* q_lens, const int32_t* kv_lens,
                                        const int64_t* q_starts, const int64_t* kv_starts, int32_t num_seqs,
                                        int32_t max_q_len, float scale, void* workspace, size_t workspace_bytes,
                                        int32_t* device_error, void* stream) {
    if (dtype < PKV_BF16 || dtype > PKV_FP32 || num_seqs < 0 || num_q_rows < 0 || num_kv_rows < 0)
        return PKV_ERR_INVALID_ARG;
    if (dtype == PKV_FP32 || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
    if (num_q_rows > 0x7fffff00 || num_kv_rows > 0x7fffff00) return PKV_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || !std::isfinite(scale) || max_q_len < 1) return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_q_rows == 0) return PKV_OK;
    if (!q_lens || !kv_lens) return PKV_ERR_INVALID_ARG;
    if (!rows_ok(q, num_q_rows, 2, head_dim, false) || !rows_ok(out, num_q_rows, 2, head_dim, true))
        return PKV_ERR_INVALID_ARG;
    if (!k || !v || k->num_heads < 1 || v->num_heads != k->num_heads || q->num_heads != out->num_heads ||
        q->num_heads % k->num_heads)
        return PKV_ERR_INVALID_ARG;
    if (num_kv_rows > 0 && (!rows_ok(k, num_kv_rows, 2, head_dim, false) || !rows_ok(v, num_kv_rows, 2, head_dim, false)))
        return PKV_ERR_INVALID_ARG;
    if (q->num_heads / k->num_heads > 128) return PKV_ERR_UNSUPPORTED;
    // (the tensor copies take positive strides only)
    for (const pkv_rows* r : {q, k, v}) {
        const int64_t n = r == q ? num_q_rows : num_kv_rows;
        if ((n > 1 && r->token_stride <= 0) || (n > 0 && r->num_heads > 1 && r->head_stride <= 0))
            return PKV_ERR_INVALID_ARG;
    }
    if (!aligned16(workspace)) return PKV_ERR_INVALID_ARG;
    if (workspace && workspace_bytes < pkv_prompt_workspace_size()) return PKV_ERR_WORKSPACE;
    return launch_prompt(q, k, v, out, lse, dtype, head_dim, num_q_rows, num_kv_rows, q_lens, kv_lens, q_starts,
                         kv_starts, num_seqs, max_q_len, scale, workspace, device_error, (cudaStream_t)stream) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

}  // extern "C"
