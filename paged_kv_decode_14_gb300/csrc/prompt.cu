// Causal attention of packed prompts whose keys and values are rows, not
// pages.  Contract: include/pagedkv.h, pkv_prompt_attention.
//
// One warp per (query row, head): lanes hold D / 32 dimensions, keys one by
// one with the running maximum and sum of the softmax in fp32.
#include "rows.cuh"

namespace pkv {
namespace prompt {

using rows::View;

struct Arg {
    View q, k, v, out;
    float* lse;
    const int32_t *q_lens, *kv_lens;
    const int64_t *q_starts, *kv_starts;
    int* err;
    int64_t num_q_rows, num_kv_rows;
    int num_seqs, max_q_len, group;
    float scale;
};

template <typename T>
__device__ __forceinline__ float get(const uint8_t* p, int d);
template <>
__device__ __forceinline__ float get<__nv_bfloat16>(const uint8_t* p, int d) {
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[d]);
}
template <>
__device__ __forceinline__ float get<__half>(const uint8_t* p, int d) {
    return __half2float(reinterpret_cast<const __half*>(p)[d]);
}

template <typename T, int D>
__global__ void __launch_bounds__(256) prompt_kernel(const __grid_constant__ Arg a) {
    griddep_wait();
    const int b = blockIdx.x / a.max_q_len, i = blockIdx.x % a.max_q_len;
    const int Q = a.q_lens[b], L = a.kv_lens[b];
    int64_t q0 = 0, k0 = 0;
    if (a.q_starts) q0 = a.q_starts[b];
    else for (int x = 0; x < b; ++x) q0 += max(a.q_lens[x], 0);
    if (a.kv_starts) k0 = a.kv_starts[b];
    else for (int x = 0; x < b; ++x) k0 += max(a.kv_lens[x], 0);
    if (Q < 0 || Q > a.max_q_len || L < 0 || q0 < 0 || k0 < 0 || q0 + Q > a.num_q_rows || k0 + L > a.num_kv_rows) {
        if (threadIdx.x == 0) raise_error(a.err, PKV_DEVERR_LENGTH);
        return;
    }
    if (i >= Q) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int vis = max(0, L - Q + i + 1);
    for (int h = warp; h < a.q.heads; h += 8) {
        const uint8_t* q = a.q.row(q0 + i, h);
        float x[D / 32], o[D / 32];
        for (int e = 0; e < D / 32; ++e) {
            x[e] = get<T>(q, lane + 32 * e) * a.scale;
            o[e] = 0.f;
        }
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < vis; ++j) {
            const uint8_t* k = a.k.row(k0 + j, h / a.group);
            float s = 0.f;
            for (int e = 0; e < D / 32; ++e) s = fmaf(x[e], get<T>(k, lane + 32 * e), s);
            for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
            const uint8_t* v = a.v.row(k0 + j, h / a.group);
            const float mn = fmaxf(m, s), c = m == mn ? 1.f : expf(m - mn), p = expf(s - mn);
            m = mn;
            l = l * c + p;
            for (int e = 0; e < D / 32; ++e) o[e] = fmaf(p, get<T>(v, lane + 32 * e), o[e] * c);
        }
        T* out = reinterpret_cast<T*>(a.out.row(q0 + i, h));
        for (int e = 0; e < D / 32; ++e) out[lane + 32 * e] = T(vis ? o[e] / l : 0.f);
        if (a.lse && lane == 0) a.lse[(q0 + i) * a.q.heads + h] = vis ? m + logf(l) : -INFINITY;
    }
}

}  // namespace prompt

cudaError_t launch_prompt(const pkv_rows* q, const pkv_rows* k, const pkv_rows* v, const pkv_rows* out, float* lse,
                          int dtype, int head_dim, int64_t num_q_rows, int64_t num_kv_rows, const int32_t* q_lens,
                          const int32_t* kv_lens, const int64_t* q_starts, const int64_t* kv_starts, int num_seqs,
                          int max_q_len, float scale, int* err, cudaStream_t st) {
    using namespace prompt;
    auto view = [&](const pkv_rows* r) {
        View x = {(uint8_t*)r->data, r->token_stride * 2, r->head_stride * 2, r->num_heads};
        return x;
    };
    Arg a = {view(q), view(k), view(v), view(out), lse, q_lens, kv_lens, q_starts, kv_starts, err, num_q_rows,
             num_kv_rows, num_seqs, max_q_len, q->num_heads / k->num_heads, scale};
    const int64_t grid = (int64_t)num_seqs * max_q_len;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    auto go = [&](auto kern) { return launch_pdl(kern, dim3((unsigned)grid), dim3(256), (size_t)0, st, a); };
    if (dtype == PKV_BF16) return head_dim == 128 ? go(prompt_kernel<__nv_bfloat16, 128>) : go(prompt_kernel<__nv_bfloat16, 64>);
    return head_dim == 128 ? go(prompt_kernel<__half, 128>) : go(prompt_kernel<__half, 64>);
}

}  // namespace pkv
