// Per-head RMS norm and rotary position embedding of query and key rows.
// Contract: include/pagedkv.h, pkv_qk_norm_rope.
//
// Per row x of head_dim D, in fp32 (statistics, angles and products), rounded once:
//   y = x / sqrt(mean(x^2) + eps) * w                       (where a norm is asked for)
//   (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s)            for every pair (a, b) of the rotated part
// A row is read and written once, so the bound is HBM for many tokens and the
// launch's latency for few (8192 tokens of 40 heads of 128 bf16: half of a head
// rotated in the interleaved layout 29 us = 5.8 TB/s, with a norm and the whole
// head rotated 32 us, with a norm and pairs across a part of a head 40 to 49 us;
// 32 tokens: 3.5 us).
#include "rows.cuh"

namespace pkv {
namespace rows {

// Warp w of W takes an equal range of the row groups.  No early trigger: an attention launched
// behind this kernel reads its q rows before its own dependency wait.
template <typename T, int GS, int KIND, bool NORM>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_rope_kernel(const View qi, const View qo, const View ki,
                                                                   const View ko, const T* __restrict__ qw,
                                                                   const T* __restrict__ kw, float eps, int D,
                                                                   const __grid_constant__ Rope rope,
                                                                   const int32_t* __restrict__ positions, int64_t tokens,
                                                                   int64_t units, int warp_smem) {
    extern __shared__ __align__(16) uint8_t rows_shared[];
    griddep_wait();
    const int w = blockIdx.x * kWarps + (threadIdx.x >> 5), W = gridDim.x * kWarps;
    warp_rows<T, GS, KIND, NORM>(qi, qo, ki, ko, qw, kw, eps, D, rope, positions, tokens, units * w / W,
                          units * (w + 1) / W, rows_shared + (threadIdx.x >> 5) * warp_smem);
}

}  // namespace rows

using namespace rows;

template <typename T, int GS>
static cudaError_t launch_rows(const View& qi, const View& qo, const View& ki, const View& ko, const void* qw,
                               const void* kw, float eps, int D, const Rope& rope, const int32_t* positions, int64_t T_,
                               int num_sms, cudaStream_t st) {
    const int64_t units = row_units(T_, qi.heads, ki.heads, 32 / GS);
    const size_t smem = rows_smem<T, GS>(rope, D);
    return for_kind(rope_kind<T>(rope, GS), eps >= 0.f, [&](auto kind, auto norm) {
        static std::atomic<uint64_t> set{0};
        return launch_pdl_bigsmem(set, qk_norm_rope_kernel<T, GS, decltype(kind)::value, decltype(norm)::value>,
                                  dim3(rows_ctas(units, num_sms)), dim3(kThreads), DynSmem(smem, rows_smem_most<T, GS>()), st, qi,
                                  qo, ki, ko, (const T*)qw, (const T*)kw, eps, D, rope, positions, T_, units, (int)(smem / kWarps));
    });
}

cudaError_t launch_qk_norm_rope(const pkv_rows* q_in, const pkv_rows* q_out, const pkv_rows* k_in,
                                const pkv_rows* k_out, int dtype, int D, int64_t T, const int32_t* positions,
                                const pkv_rope* rope, bool inverse, const void* qw, const void* kw, float eps,
                                cudaStream_t st, int num_sms) {
    const int e = dtype == PKV_FP32 ? 4 : 2;
    const View qi = view(q_in, e), qo = view(q_out, e), ki = view(k_in, e), ko = view(k_out, e);
    const Rope r = rope_arg(rope, inverse);
#define PKV_ROWS(T_, GS) launch_rows<T_, GS>(qi, qo, ki, ko, qw, kw, eps, D, r, positions, T, num_sms, st)
#define PKV_ROWS_OF(T_) \
    (lanes_of<T_>(D) == 4 ? PKV_ROWS(T_, 4) : lanes_of<T_>(D) == 8 ? PKV_ROWS(T_, 8) : PKV_ROWS(T_, 16))
    if (dtype == PKV_BF16) return PKV_ROWS_OF(__nv_bfloat16);
    if (dtype == PKV_FP16) return PKV_ROWS_OF(__half);
    return lanes_of<float>(D) == 32 ? PKV_ROWS(float, 32) : PKV_ROWS_OF(float);
#undef PKV_ROWS_OF
#undef PKV_ROWS
}

}  // namespace pkv
