// Per-head RMS norm and rotary position embedding of query and key rows, and
// the same pass writing keys and values into the paged cache.  Contracts:
// include/pagedkv.h, pkv_qk_norm_rope and pkv_paged_kv_append_norm_rope.
//
// Per row x of head_dim D, in fp32 (statistics, angles and products), rounded once:
//   y = x / sqrt(mean(x^2) + eps) * w                       (where a norm is asked for)
//   (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s)            for every pair (a, b) of the rotated part
// A row is read and written once, so the bound is HBM for many tokens and the
// launch's latency for few.
#include "rows.cuh"

namespace pkv {
namespace rows {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 3;                // rows whose loads a thread has in flight

// Norm and rotation of `total` rows of one token, GS lanes a row: rows
// 0 .. q_in.heads - 1 are q's heads, the others k's.  Loads of the first
// kUnroll rows a group handles are issued before the angles are computed.
template <typename T, int GS, int CPL>
__device__ __forceinline__ void token_rows(const View& qi, const View& qo, const View& ki, const View& ko,
                                           const T* qw, const T* kw, bool norm, float eps, int D, const Rope& rope,
                                           const int32_t* positions, int64_t t, float2* cs, float* stage) {
    constexpr int N = Chunk<T>::N, RPW = 32 / GS, RPP = kWarps * RPW;
    const int tid = threadIdx.x, lane = tid & (GS - 1), group = tid / GS;
    const int nch = D / N, total = qi.heads + ki.heads;
    uint4 raw[kUnroll][CPL];
    auto load = [&](int r, uint4 (&v)[CPL]) {
        const uint8_t* p = r < qi.heads ? qi.row(t, r) : ki.row(t, r - qi.heads);
#pragma unroll
        for (int j = 0; j < CPL; ++j)
            v[j] = r < total && lane + j * GS < nch ? *reinterpret_cast<const uint4*>(p + (lane + j * GS) * 16)
                                                    : make_uint4(0, 0, 0, 0);
    };
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) load(group + u * RPP, raw[u]);
    uint4 wq[CPL], wk[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
        const int ch = lane + j * GS;
        wq[j] = qw && ch < nch ? *reinterpret_cast<const uint4*>(qw + ch * N) : make_uint4(0, 0, 0, 0);
        wk[j] = kw && ch < nch ? *reinterpret_cast<const uint4*>(kw + ch * N) : make_uint4(0, 0, 0, 0);
    }
    if (rope.pairs > 0) {
        const int pos = positions[t];
        for (int i = tid; i < rope.pairs; i += kThreads) cs[i] = angle(rope, i, pos);
    }
    __syncthreads();
    Rotator<T, GS, CPL> rot;
    rot.load(rope, cs, lane);
    const float inv_dim = 1.f / (float)D;
    for (int r0 = 0; r0 < total; r0 += kUnroll * RPP) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = r0 + u * RPP + group;
            if (r0 + u * RPP >= total) break;              // (uniform: whole warps go on to the shuffles)
            float x[CPL][N];
#pragma unroll
            for (int j = 0; j < CPL; ++j) Chunk<T>::unpack(raw[u][j], x[j]);
            const bool isq = r < qi.heads;
            if (norm) rms_norm<T, GS, CPL>(x, isq ? wq : wk, (isq ? qw : kw) != nullptr, eps, inv_dim);
            rot.apply(x, stage + group * D);
            if (r < total) {
                uint8_t* p = isq ? qo.row(t, r) : ko.row(t, r - qi.heads);
#pragma unroll
                for (int j = 0; j < CPL; ++j)
                    if (lane + j * GS < nch)
                        *reinterpret_cast<uint4*>(p + (lane + j * GS) * 16) = Chunk<T>::pack(x[j]);
            }
            if (r0 + kUnroll * RPP < total) load(r + kUnroll * RPP, raw[u]);
        }
    }
}

// One CTA per token.  No early trigger: an attention launched behind this
// kernel reads its q rows before its own dependency wait.
template <typename T, int GS, int CPL>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const View qi, const View qo, const View ki,
                                                                const View ko, const T* __restrict__ qw,
                                                                const T* __restrict__ kw, int norm, float eps, int D,
                                                                const __grid_constant__ Rope rope,
                                                                const int32_t* __restrict__ positions) {
    extern __shared__ float stage[];
    __shared__ float2 cs[PKV_ROPE_MAX_PAIRS];
    griddep_wait();
    token_rows<T, GS, CPL>(qi, qo, ki, ko, qw, kw, norm != 0, eps, D, rope, positions, blockIdx.x, cs, stage);
}

// Shared memory of the rotate-half pairs that no whole number of 16-byte chunks lies between.
template <typename T, int GS>
__host__ inline size_t stage_bytes(const Rope& r, int D) {
    return r.pairs > 0 && !r.interleaved && r.pairs % Chunk<T>::N ? (size_t)(kThreads / GS) * D * sizeof(float) : 0;
}

// ------------------------------------------------------------------ append

struct AppendArg {
    View q_in, q_out, k, v, k_out;           // k_out.data: nullptr if not wanted
    const __nv_bfloat16 *qw, *kw;
    const int64_t* slots;
    const int32_t* positions;
    int64_t T, num_blocks;
    uint8_t *k_cache, *v_cache;
    float *k_scales, *v_scales;
    int* err;
    float eps;
    int norm, D, Hkv;
    int windows, heads_per_cta, head_ctas;   // K/V part of the grid: windows x head_ctas CTAs
    int q_ctas;                              // CTAs of the q part (one per token, or none)
};

// FP8 codes of 8 values (IEEE division by the page's scale, nearest even, saturating).
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float scale) {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t word = 0;
#pragma unroll
        for (int h = 0; h < 4; ++h)
            word |= (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(x[4 * j + h], scale), __NV_SATFINITE, __NV_E4M3) << (8 * h);
        w[j] = word;
    }
    return make_uint2(w[0], w[1]);
}

// The K/V part: a CTA takes 16 consecutive tokens of the call (a window) and
// some kv-heads.  With given scales (or a bf16 cache) every token stands alone.
//
// Scales from the values need all of a started block's tokens at once.  The
// CTA of the window that holds the block's offset-0 token (the owner) gathers
// them: the run of consecutive slots after it, and, if that run is short of
// the whole block, any other token of the call in the block (one scan of the
// slots).  A token whose chain of consecutive slots leads back to an offset-0
// token, or whose block's offset-0 slot is found by the same scan, is left to
// that owner; any other token continues an older block and is encoded alone
// with the block's scale.  So one launch does what needs every value of a
// block before any is encoded, without atomics: the result is deterministic.
template <int E, int D, bool FRESH>
__device__ __forceinline__ void append_window(const AppendArg& a, const Rope& rope, float2* cs, float* stage) {
    constexpr int LPR = D / 8;                              // lanes per row
    constexpr int ROWS = kThreads / LPR;                    // rows at once: 16 (D = 128) or 32 (D = 64)
    constexpr int HPR = ROWS / 16;                          // kv-heads at once
    __shared__ int64_t member[16];                          // token of row i (-1: none)
    __shared__ int64_t wslot[16];
    __shared__ int kind[16];                                // FRESH: 0 alone, 1 owner, 2 left to an owner / none
    __shared__ unsigned long long found;
    __shared__ float amax[2][kWarps];
    const int tid = threadIdx.x;
    const int w = blockIdx.x / a.head_ctas, hc = blockIdx.x % a.head_ctas;
    const int64_t t0 = (int64_t)w * 16;
    const int i = (tid / LPR) & 15, hsub = tid / (LPR * 16), lane = tid & (LPR - 1);
    const int g_first = hc * a.heads_per_cta, g_last = min(a.Hkv, g_first + a.heads_per_cta);
    if (tid < 16) {
        const int64_t t = t0 + tid;
        int64_t s = t < a.T ? a.slots[t] : -1;
        if (s >= a.num_blocks * kBlock) {
            if (hc == 0) raise_error(a.err, PKV_DEVERR_SLOT);
            s = -1;
        }
        wslot[tid] = s;
        member[tid] = t < a.T ? t : -1;
        kind[tid] = 0;
    }
    __syncthreads();

    // one pass over up to 16 rows (member[], and their slots: all of block `blk` with off = row when
    // fresh, else wslot[])
    auto pass = [&](bool fresh, int64_t fresh_blk) {
        const int64_t t = member[i];
        const int64_t s = fresh ? (t >= 0 ? fresh_blk * kBlock + i : -1) : (t >= 0 ? wslot[i] : -1);
        for (int x = tid; x < 16 * rope.pairs; x += kThreads) {
            const int r = x / rope.pairs, p = x - r * rope.pairs;
            const int64_t tr = member[r];
            cs[r * rope.pairs + p] = angle(rope, p, tr >= 0 ? a.positions[tr] : 0);
        }
        __syncthreads();
        Rotator<__nv_bfloat16, LPR, 1> rot;
        rot.load(rope, cs + i * rope.pairs, lane);
        for (int g0 = g_first; g0 < g_last; g0 += HPR) {
            const int g = g0 + hsub;
            const bool ok = t >= 0 && g < g_last;
            float k[1][8], v[8];
            {
                const uint4 kr = ok ? *reinterpret_cast<const uint4*>(a.k.row(t, g) + lane * 16) : make_uint4(0, 0, 0, 0);
                const uint4 vr = ok ? *reinterpret_cast<const uint4*>(a.v.row(t, g) + lane * 16) : make_uint4(0, 0, 0, 0);
                Chunk<__nv_bfloat16>::unpack(kr, k[0]);
                Chunk<__nv_bfloat16>::unpack(vr, v);
            }
            if (a.norm) {
                uint4 kw[1] = {a.kw ? *reinterpret_cast<const uint4*>(a.kw + lane * 8) : make_uint4(0, 0, 0, 0)};
                rms_norm<__nv_bfloat16, LPR, 1>(k, kw, a.kw != nullptr, a.eps, 1.f / (float)D);
            }
            rot.apply(k, stage + (tid / LPR) * D);
            if (ok && a.k_out.data)
                *reinterpret_cast<uint4*>(a.k_out.row(t, g) + lane * 16) = Chunk<__nv_bfloat16>::pack(k[0]);
            float ksc = 1.f, vsc = 1.f;
            const int64_t blk = s >= 0 ? s / kBlock : 0;
            const int off = (int)(s & (kBlock - 1));
            if constexpr (E == 1) {
                if (FRESH && fresh) {
                    // the block's largest |k| and |v| (NaN ignored): lanes, then the head's warps
                    float mk = 0.f, mv = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        mk = fmaxf(mk, fabsf(k[0][e]));
                        mv = fmaxf(mv, fabsf(v[e]));
                    }
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) {
                        mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
                        mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
                    }
                    const int warp = tid >> 5, wph = kWarps / HPR;   // warps of one head: 16 rows
                    if ((tid & 31) == 0) {
                        amax[0][warp] = mk;
                        amax[1][warp] = mv;
                    }
                    __syncthreads();
                    mk = mv = 0.f;
                    for (int x = 0; x < wph; ++x) {
                        mk = fmaxf(mk, amax[0][hsub * wph + x]);
                        mv = fmaxf(mv, amax[1][hsub * wph + x]);
                    }
                    __syncthreads();
                    ksc = mk > 0.f ? __fdiv_rn(mk, 448.0f) : 1.0f;
                    vsc = mv > 0.f ? __fdiv_rn(mv, 448.0f) : 1.0f;
                    if (i == 0 && lane == 0 && g < g_last) {
                        a.k_scales[fresh_blk * a.Hkv + g] = ksc;
                        a.v_scales[fresh_blk * a.Hkv + g] = vsc;
                    }
                } else if (ok && s >= 0) {
                    ksc = a.k_scales[blk * a.Hkv + g];
                    vsc = a.v_scales[blk * a.Hkv + g];
                }
            }
            if (ok && s >= 0) {
                const size_t page = ((size_t)blk * a.Hkv + g) * (size_t)(kBlock * D * E);
                if constexpr (E == 2) {
                    const size_t at = page + ((off >> 3) * LPR + lane) * 128 + (off & 7) * 16;
                    *reinterpret_cast<uint4*>(a.k_cache + at) = Chunk<__nv_bfloat16>::pack(k[0]);
                    *reinterpret_cast<uint4*>(a.v_cache + at) = Chunk<__nv_bfloat16>::pack(v);
                } else {
                    const size_t at = page + ((off >> 3) * (LPR / 2) + (lane >> 1)) * 128 + (off & 7) * 16 + (lane & 1) * 8;
                    *reinterpret_cast<uint2*>(a.k_cache + at) = encode8(k[0], ksc);
                    *reinterpret_cast<uint2*>(a.v_cache + at) = encode8(v, vsc);
                }
            }
        }
        __syncthreads();                                    // cs, member and stage may change now
    };

    if constexpr (!FRESH) {
        pass(false, 0);
    } else {
        // a token of this window: the owner of a block, left to one, or alone
        if (tid < 16 && wslot[tid] >= 0) {
            const int64_t t = t0 + tid, s = wslot[tid];
            const int off = (int)(s & (kBlock - 1));
            if (off == 0) {
                kind[tid] = 1;
            } else {
                bool chain = t >= off;
                for (int x = 1; chain && x <= off; ++x) chain = a.slots[t - x] == s - x;
                kind[tid] = chain ? 2 : 3;                  // 3: undecided until the scan
            }
        }
        __syncthreads();
        for (int x = 0; x < 16; ++x) {
            if (kind[x] != 3) continue;
            if (tid == 0) found = 0;
            __syncthreads();
            const int64_t head = wslot[x] & ~(int64_t)(kBlock - 1);
            for (int64_t y = tid; y < a.T; y += kThreads)
                if (a.slots[y] == head) found = 1;
            __syncthreads();
            if (tid == 0) kind[x] = found ? 2 : 0;
            __syncthreads();
        }
        // tokens that stand alone (their blocks keep their scales); tokens without a slot only have
        // their rotated K row written
        if (tid < 16) member[tid] = t0 + tid < a.T && kind[tid] == 0 ? t0 + tid : -1;
        __syncthreads();
        int alone = 0;
        for (int x = 0; x < 16; ++x) alone |= member[x] >= 0;
        if (alone) pass(false, 0);
        for (int x = 0; x < 16; ++x) {
            if (kind[x] != 1) continue;
            const int64_t t = t0 + x, s = wslot[x];
            __syncthreads();
            if (tid < 16) {
                bool in = t + tid < a.T;
                for (int y = 1; in && y <= tid; ++y) in = a.slots[t + y] == s + y;
                member[tid] = in ? t + tid : -1;
            }
            __syncthreads();
            if (member[15] < 0) {
                // the run is short of the block: the block's other tokens may be anywhere in the call
                for (int64_t y = tid; y < a.T; y += kThreads) {
                    const int64_t z = a.slots[y] - s;
                    if (z > 0 && z < kBlock) member[z] = y;
                }
                __syncthreads();
            }
            pass(true, s / kBlock);
        }
    }
}

template <int E, int D, bool FRESH>
__global__ void __launch_bounds__(kThreads) append_norm_rope_kernel(const __grid_constant__ AppendArg a,
                                                                    const __grid_constant__ Rope rope) {
    extern __shared__ float stage[];                        // [rows at once][D], unaligned pairs only
    __shared__ float2 cs[16 * (D / 2)];
    griddep_wait();
    const int kv_ctas = a.windows * a.head_ctas;
    if ((int64_t)blockIdx.x < kv_ctas) {
        append_window<E, D, FRESH>(a, rope, cs, stage);
    } else {
        View none = a.q_in;
        none.heads = 0;
        token_rows<__nv_bfloat16, D / 8, 1>(a.q_in, a.q_out, none, none, a.qw, nullptr, a.norm != 0, a.eps, D, rope,
                                            a.positions, (int64_t)blockIdx.x - kv_ctas, cs, stage);
    }
}

}  // namespace rows

using namespace rows;

static View view(const pkv_rows* r, int e) {
    View v = {};
    if (r) {
        v.data = (uint8_t*)r->data;
        v.ts = r->token_stride * e;
        v.hs = r->head_stride * e;
        v.heads = r->num_heads;
    }
    return v;
}

template <typename T, int GS, int CPL>
static cudaError_t launch_rows(const View& qi, const View& qo, const View& ki, const View& ko, const void* qw,
                               const void* kw, float eps, int D, const Rope& rope, const int32_t* positions, int64_t T_,
                               cudaStream_t st) {
    return launch_pdl(qk_norm_rope_kernel<T, GS, CPL>, dim3((unsigned)T_), dim3(kThreads), stage_bytes<T, GS>(rope, D),
                      st, qi, qo, ki, ko, (const T*)qw, (const T*)kw, eps >= 0.f ? 1 : 0, eps, D, rope, positions);
}

cudaError_t launch_qk_norm_rope(const pkv_rows* q_in, const pkv_rows* q_out, const pkv_rows* k_in,
                                const pkv_rows* k_out, int dtype, int D, int64_t T, const int32_t* positions,
                                const pkv_rope* rope, bool inverse, const void* qw, const void* kw, float eps,
                                cudaStream_t st) {
    const int e = dtype == PKV_FP32 ? 4 : 2;
    const View qi = view(q_in, e), qo = view(q_out, e), ki = view(k_in, e), ko = view(k_out, e);
    const Rope r = rope_arg(rope, inverse);
    const int chunks = D * e / 16;
#define PKV_ROWS(T_, GS, CPL) launch_rows<T_, GS, CPL>(qi, qo, ki, ko, qw, kw, eps, D, r, positions, T, st)
#define PKV_ROWS_OF(T_) (chunks <= 8 ? PKV_ROWS(T_, 8, 1) : chunks <= 16 ? PKV_ROWS(T_, 16, 1) : PKV_ROWS(T_, 32, 1))
    if (dtype == PKV_BF16) return PKV_ROWS_OF(__nv_bfloat16);
    if (dtype == PKV_FP16) return PKV_ROWS_OF(__half);
    return chunks > 32 ? PKV_ROWS(float, 32, 2) : PKV_ROWS_OF(float);
#undef PKV_ROWS_OF
#undef PKV_ROWS
}

cudaError_t launch_append_norm_rope(const pkv_cache& c, const pkv_rows* q_in, const pkv_rows* q_out, const pkv_rows* k,
                                    const pkv_rows* v, const pkv_rows* k_out, const int64_t* slots, int64_t T,
                                    const int32_t* positions, const pkv_rope* rope, const void* qw, const void* kw,
                                    float eps, bool fresh, int* err, cudaStream_t st, int num_sms) {
    AppendArg a = {};
    a.q_in = view(q_in, 2);
    a.q_out = view(q_out, 2);
    a.k = view(k, 2);
    a.v = view(v, 2);
    a.k_out = view(k_out, 2);
    a.qw = (const __nv_bfloat16*)qw;
    a.kw = (const __nv_bfloat16*)kw;
    a.slots = slots;
    a.positions = positions;
    a.T = T;
    a.num_blocks = c.num_blocks;
    a.k_cache = (uint8_t*)c.k_cache;
    a.v_cache = (uint8_t*)c.v_cache;
    a.k_scales = const_cast<float*>(c.k_scales);
    a.v_scales = const_cast<float*>(c.v_scales);
    a.err = err;
    a.eps = eps;
    a.norm = eps >= 0.f;
    a.D = c.head_dim;
    a.Hkv = c.num_kv_heads;
    const bool fp8 = c.kv_dtype == PKV_KV_FP8_E4M3;
    const Rope r = rope_arg(rope, false);
    a.windows = (int)((T + 15) / 16);
    const int at_once = c.head_dim == 128 ? 1 : 2;
    a.heads_per_cta = at_once;
    while (a.heads_per_cta < a.Hkv && (int64_t)a.windows * ((a.Hkv + a.heads_per_cta - 1) / a.heads_per_cta) > 8 * num_sms)
        a.heads_per_cta *= 2;
    a.head_ctas = (a.Hkv + a.heads_per_cta - 1) / a.heads_per_cta;
    a.q_ctas = q_in ? (int)T : 0;
    const int64_t grid = (int64_t)a.windows * a.head_ctas + a.q_ctas;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    auto go = [&](auto kern, size_t smem) {
        return launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), smem, st, a, r);
    };
    if (c.head_dim == 128) {
        const size_t smem = stage_bytes<__nv_bfloat16, 16>(r, 128);
        return !fp8 ? go(append_norm_rope_kernel<2, 128, false>, smem)
                    : fresh ? go(append_norm_rope_kernel<1, 128, true>, smem) : go(append_norm_rope_kernel<1, 128, false>, smem);
    }
    const size_t smem = stage_bytes<__nv_bfloat16, 8>(r, 64);
    return !fp8 ? go(append_norm_rope_kernel<2, 64, false>, smem)
                : fresh ? go(append_norm_rope_kernel<1, 64, true>, smem) : go(append_norm_rope_kernel<1, 64, false>, smem);
}

}  // namespace pkv
