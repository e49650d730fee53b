// The norm and rotation of rows (see rows.cuh) in the pass that writes keys and
// values into the paged cache.  Contract: include/pagedkv.h,
// pkv_paged_kv_append_norm_rope.
//
// One launch of two kinds of CTAs: some take the query rows, one warp's share
// each, the others 16 tokens' key and value rows.  Every row is read and
// written once, so the bound is HBM for many tokens and the launch's latency
// for few.  Measured: 7.7k prompt tokens of 32/8 heads of 128 into an FP8 cache,
// 48.5 us = 3.6 TB/s, a bf16 one 44 us; a decode step of 32 tokens 5.0 us, and 16.7
// us where FP8 scales come from the values (a scan of the slots for every token
// whose block's first slot is not in its window).  Prompts are held up by a
// window's chain slots -> rows -> angles, which the 16 resident warps of an SM hide
// by half (with replays of one call 51 us; the q CTAs first 61, both kinds mixed
// 56, rows prefetched to L2 before the slots are known 55).
#include "rows.cuh"

namespace pkv {
namespace rows {

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
    int D, Hkv;
    int windows, heads_per_cta, head_ctas;   // K/V part of the grid: windows x head_ctas CTAs
    int q_ctas, q_smem;                      // CTAs of the q part; a warp's shared memory there
};

// FP8 codes of values divided by a page's scale: e4m3, nearest even, saturating,
// of the IEEE quotient.  The division is done only where it can matter: with r
// = 1 / scale, x r (1 - 2^-21) and x r (1 + 2^-21) enclose both the quotient and
// its rounding (three roundings of 2^-24 each are below 2^-21), conversion is
// monotonic, so where both ends have the same code that is the quotient's; in
// about one of 2^16 values they differ.  (16 divisions a thread were a third of
// the instructions of an FP8 append.)
struct Encoder {
    float scale, lo, hi;
    bool plain;                       // the enclosure does not hold: scale out of 2^+-100, or not a number
    __device__ __forceinline__ explicit Encoder(float s) : scale(s) {
        const float r = __frcp_rn(s);
        lo = r * (1.f - 0x1p-21f);
        hi = r * (1.f + 0x1p-21f);
        plain = !(fabsf(s) > 0x1p-100f && fabsf(s) < 0x1p100f);
    }
    static __device__ __forceinline__ uint32_t codes(float a, float b, float c, float d) {
        return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
               (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
    }
    __device__ __forceinline__ uint2 operator()(const float (&x)[8]) const {
        const uint2 a = make_uint2(codes(x[0] * lo, x[1] * lo, x[2] * lo, x[3] * lo),
                                   codes(x[4] * lo, x[5] * lo, x[6] * lo, x[7] * lo));
        const uint2 b = make_uint2(codes(x[0] * hi, x[1] * hi, x[2] * hi, x[3] * hi),
                                   codes(x[4] * hi, x[5] * hi, x[6] * hi, x[7] * hi));
        if (a.x == b.x && a.y == b.y && !plain) return a;
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = __fdiv_rn(x[e], scale);
        return make_uint2(codes(q[0], q[1], q[2], q[3]), codes(q[4], q[5], q[6], q[7]));
    }
};

// f(token, slot) for every token of the call, by the CTA's threads; 8 loads in flight a thread (a scan
// with one took 30 us for 7.7k tokens, on the path of every prompt's last block).
template <typename F>
__device__ __forceinline__ void scan_slots(const AppendArg& a, int tid, F f) {
    for (int64_t y0 = tid; y0 < a.T; y0 += 8 * kThreads) {
        int64_t z[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) z[u] = y0 + u * kThreads < a.T ? a.slots[y0 + u * kThreads] : -1;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (z[u] >= 0) f(y0 + u * kThreads, z[u]);
    }
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
template <int E, int D, bool FRESH, int KIND, bool NORM>
__device__ __forceinline__ void append_window(const AppendArg& a, const Rope& rope, float2* cs, float* stage) {
    constexpr int LPR = lanes_of<__nv_bfloat16>(D);         // lanes per row: 8 (D = 128) or 4 (D = 64)
    constexpr int ROWS = kThreads / LPR;                    // rows at once: 32 or 64
    constexpr int HPR = ROWS / 16;                          // kv-heads at once
    __shared__ int64_t member[16];                          // token of row i (-1: none)
    __shared__ int64_t near[48];                            // slots of tokens t0 - 16 .. t0 + 31
    int64_t* wslot = near + 16;                             // the window's own (-1: none to write)
    __shared__ int kind[16];                                // FRESH: 0 alone, 1 owner, 2 left to an owner / none
    __shared__ unsigned long long found;
    __shared__ float amax[2][2][kWarps];                    // (by turns: one barrier a head)
    __shared__ int32_t near_pos[48];                        // positions of tokens t0 - 16 .. t0 + 31
    const int tid = threadIdx.x;
    const int w = blockIdx.x / a.head_ctas, hc = blockIdx.x % a.head_ctas;
    const int64_t t0 = (int64_t)w * 16;
    const int i = (tid / LPR) & 15, hsub = tid / (LPR * 16), lane = tid & (LPR - 1);
    const int g_first = hc * a.heads_per_cta, g_last = min(a.Hkv, g_first + a.heads_per_cta);
    if (tid < 48 && (FRESH || (tid >= 16 && tid < 32))) {
        const int64_t t = t0 - 16 + tid;
        int64_t s = t >= 0 && t < a.T ? a.slots[t] : -1;
        if (s >= a.num_blocks * kBlock) {
            if (hc == 0 && tid >= 16 && tid < 32) raise_error(a.err, PKV_DEVERR_SLOT);
            s = -1;
        }
        near[tid] = s;
        near_pos[tid] = rope.pairs > 0 && t >= 0 && t < a.T ? a.positions[t] : 0;
        if (tid >= 16 && tid < 32) {
            member[tid - 16] = t < a.T ? t : -1;
            kind[tid - 16] = 0;
        }
    }
    __syncthreads();

    // one pass over up to 16 rows (member[], and their slots: all of block `blk` with off = row when
    // fresh, else wslot[])
    auto pass = [&](bool fresh, int64_t fresh_blk) {
        const int64_t t = member[i];
        const int64_t s = fresh ? (t >= 0 ? fresh_blk * kBlock + i : -1) : (t >= 0 ? wslot[i] : -1);
        // the first head's rows are under way while the angles are computed, the next head's while one is
        // normed, rotated and encoded
        uint4 kr[kSets], vr[kSets];
        auto fetch = [&](int g) {
            const bool in = t >= 0 && g < g_last;
            const uint8_t *kp = in ? a.k.row(t, g) + lane * 16 : nullptr, *vp = in ? a.v.row(t, g) + lane * 16 : nullptr;
#pragma unroll
            for (int j = 0; j < kSets; ++j) {
                kr[j] = in ? *reinterpret_cast<const uint4*>(kp + j * LPR * 16) : make_uint4(0, 0, 0, 0);
                vr[j] = in ? *reinterpret_cast<const uint4*>(vp + j * LPR * 16) : make_uint4(0, 0, 0, 0);
            }
        };
        fetch(g_first + hsub);
        uint4 kw[kSets];
#pragma unroll
        for (int j = 0; j < kSets; ++j)
            kw[j] = NORM && a.kw ? *reinterpret_cast<const uint4*>(a.kw + (lane + j * LPR) * 8) : make_uint4(0, 0, 0, 0);
        for (int x = tid; x < 16 * rope.pairs; x += kThreads) {
            const int r = x / rope.pairs, p = x - r * rope.pairs;
            const int64_t tr = member[r], d = tr - t0 + 16;
            if (tr >= 0) cs[x] = angle(rope, p, d >= 0 && d < 48 ? near_pos[d] : a.positions[tr]);
        }
        __syncthreads();
        Rotator<__nv_bfloat16, LPR, KIND> rot;
        rot.init(rope, lane);
        rot.load(cs + i * rope.pairs);
        int turn = 0;
        for (int g0 = g_first; g0 < g_last; g0 += HPR, turn ^= 1) {
            const int g = g0 + hsub;
            const bool ok = t >= 0 && g < g_last;
            float k[kSets][8], v[kSets][8];
            uint4 vraw[kSets];
#pragma unroll
            for (int j = 0; j < kSets; ++j) {
                Chunk<__nv_bfloat16>::unpack(kr[j], k[j]);
                Chunk<__nv_bfloat16>::unpack(vr[j], v[j]);
                vraw[j] = vr[j];
            }
            fetch(g + HPR);
            if constexpr (NORM) rms_norm<__nv_bfloat16, LPR>(k, kw, a.kw != nullptr, a.eps, 1.f / (float)D);
            rot.apply(k, stage + (tid / LPR) * D);
            if (ok && a.k_out.data) {
                uint8_t* kp = a.k_out.row(t, g) + lane * 16;
#pragma unroll
                for (int j = 0; j < kSets; ++j)
                    *reinterpret_cast<uint4*>(kp + j * LPR * 16) = Chunk<__nv_bfloat16>::pack(k[j]);
            }
            float ksc = 1.f, vsc = 1.f;
            const int64_t blk = s >= 0 ? s / kBlock : 0;
            const int off = (int)(s & (kBlock - 1));
            if constexpr (E == 1) {
                if (FRESH && fresh) {
                    // the block's largest |k| and |v| (NaN ignored): lanes, then the head's warps
                    float mk = 0.f, mv = 0.f;
#pragma unroll
                    for (int j = 0; j < kSets; ++j)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            mk = fmaxf(mk, fabsf(k[j][e]));
                            mv = fmaxf(mv, fabsf(v[j][e]));
                        }
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) {
                        mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
                        mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
                    }
                    const int warp = tid >> 5, wph = kWarps / HPR;   // warps of one head: 16 rows
                    if ((tid & 31) == 0) {
                        amax[turn][0][warp] = mk;
                        amax[turn][1][warp] = mv;
                    }
                    __syncthreads();
                    mk = mv = 0.f;
                    for (int x = 0; x < wph; ++x) {
                        mk = fmaxf(mk, amax[turn][0][hsub * wph + x]);
                        mv = fmaxf(mv, amax[turn][1][hsub * wph + x]);
                    }
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
                const uint32_t row = (uint32_t)(off >> 3) * (D * E / 16) * 128 + (off & 7) * 16;
                uint8_t *kc = a.k_cache + page + row, *vc = a.v_cache + page + row;
                const Encoder ke(ksc), ve(vsc);
#pragma unroll
                for (int j = 0; j < kSets; ++j) {
                    const int ch = lane + j * LPR;          // 16 bytes of the bf16 row
                    if constexpr (E == 2) {
                        *reinterpret_cast<uint4*>(kc + ch * 128) = Chunk<__nv_bfloat16>::pack(k[j]);
                        *reinterpret_cast<uint4*>(vc + ch * 128) = vraw[j];
                    } else {
                        *reinterpret_cast<uint2*>(kc + (ch >> 1) * 128 + (ch & 1) * 8) = ke(k[j]);
                        *reinterpret_cast<uint2*>(vc + (ch >> 1) * 128 + (ch & 1) * 8) = ve(v[j]);
                    }
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
            const int64_t s = wslot[tid];
            const int off = (int)(s & (kBlock - 1));
            bool chain = true;
            for (int x = 1; x <= off; ++x) chain = chain && wslot[tid - x] == s - x;
            kind[tid] = off == 0 ? 1 : chain ? 2 : 3;       // 3: undecided until the scan
        }
        __syncthreads();
        for (int x = 0; x < 16; ++x) {
            if (kind[x] != 3) continue;
            if (tid == 0) found = 0;
            __syncthreads();
            const int64_t head = wslot[x] & ~(int64_t)(kBlock - 1);
            scan_slots(a, tid, [&](int64_t, int64_t z) {
                if (z == head) found = 1;
            });
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
            bool in = true;
            if (tid < 16) {
                for (int y = 1; y <= tid; ++y) in = in && wslot[x + y] == s + y;
                member[tid] = in ? t + tid : -1;
            }
            // (the barrier carries the answer: a read of member[15] behind it could meet the scan's write)
            if (__syncthreads_or(!in)) {
                // the run is short of the block: the block's other tokens may be anywhere in the call
                scan_slots(a, tid, [&](int64_t y, int64_t z) {
                    z -= s;
                    if (z > 0 && z < kBlock) member[z] = y;
                });
                __syncthreads();
            }
            pass(true, s / kBlock);
        }
    }
}

template <int E, int D, bool FRESH, int KIND, bool NORM>
__global__ void __launch_bounds__(kThreads, 2) append_norm_rope_kernel(const __grid_constant__ AppendArg a,
                                                                       const __grid_constant__ Rope rope) {
    // K/V part: (cos, sin) of 16 tokens' pairs, then (unaligned pairs) the rows at once in fp32; q part: see warp_rows
    extern __shared__ __align__(16) uint8_t rows_shared[];
    griddep_wait();
    const int kv_ctas = a.windows * a.head_ctas;
    if ((int)blockIdx.x < kv_ctas) {
        append_window<E, D, FRESH, KIND, NORM>(a, rope, reinterpret_cast<float2*>(rows_shared),
                                   reinterpret_cast<float*>(rows_shared + 16 * 8 * rope.pairs));
    } else {
        constexpr int GS = lanes_of<__nv_bfloat16>(D), RPW = 32 / GS;
        View none = a.q_in;
        none.heads = 0;
        const int64_t w = (int64_t)(blockIdx.x - kv_ctas) * kWarps + (threadIdx.x >> 5), W = (int64_t)a.q_ctas * kWarps;
        const int64_t units = a.T * ((a.q_in.heads + RPW - 1) / RPW);
        warp_rows<__nv_bfloat16, GS, KIND, NORM>(a.q_in, a.q_out, none, none, a.qw, nullptr, a.eps, D, rope,
                                        a.positions, a.T, units * w / W, units * (w + 1) / W,
                                        rows_shared + (threadIdx.x >> 5) * a.q_smem);
    }
}

}  // namespace rows

using namespace rows;

template <int E, int D, bool FRESH, int KIND, bool NORM>
static cudaError_t launch_one(unsigned grid, size_t smem, cudaStream_t st, const AppendArg& a, const Rope& r) {
    static std::atomic<uint64_t> set{0};
    constexpr int GS = lanes_of<__nv_bfloat16>(D);
    // (the K/V part's most: 16 tokens' (cos, sin), and the rows at once in fp32)
    constexpr size_t kv = 16 * 8 * (D / 2) + kThreads / GS * D * 4, q = rows_smem_most<__nv_bfloat16, GS>();
    return launch_pdl_bigsmem(set, append_norm_rope_kernel<E, D, FRESH, KIND, NORM>, dim3(grid), dim3(kThreads),
                              DynSmem(smem, kv > q ? kv : q), st, a, r);
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
    a.D = c.head_dim;
    a.Hkv = c.num_kv_heads;
    const bool fp8 = c.kv_dtype == PKV_KV_FP8_E4M3;
    const Rope r = rope_arg(rope, false);
    a.windows = (int)((T + 15) / 16);
    const int gs = lanes_of<__nv_bfloat16>(c.head_dim);
    const int at_once = kThreads / gs / 16;
    a.heads_per_cta = at_once;
    while (a.heads_per_cta < a.Hkv && (int64_t)a.windows * ((a.Hkv + a.heads_per_cta - 1) / a.heads_per_cta) > 4 * num_sms)
        a.heads_per_cta *= 2;
    a.head_ctas = (a.Hkv + a.heads_per_cta - 1) / a.heads_per_cta;
    a.q_ctas = q_in ? (int)rows_ctas(row_units(T, q_in->num_heads, 0, 32 / gs), num_sms) : 0;
    const int64_t grid = (int64_t)a.windows * a.head_ctas + a.q_ctas;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    const bool staged = r.pairs > 0 && !r.interleaved && r.pairs % 8;
    const size_t kv_smem = (size_t)16 * 8 * r.pairs + (staged ? (size_t)kThreads / gs * c.head_dim * 4 : 0);
    const size_t q_smem = !q_in ? 0 : gs == 8 ? rows_smem<__nv_bfloat16, 8>(r, 128) : rows_smem<__nv_bfloat16, 4>(r, 64);
    a.q_smem = (int)(q_smem / kWarps);
    const size_t smem = std::max(kv_smem, q_smem);
    return for_kind(rope_kind<__nv_bfloat16>(r, gs), eps >= 0.f, [&](auto kind, auto norm) {
        constexpr int K = decltype(kind)::value;
        constexpr bool N = decltype(norm)::value;
        const unsigned n = (unsigned)grid;
        if (c.head_dim == 128)
            return !fp8 ? launch_one<2, 128, false, K, N>(n, smem, st, a, r)
                        : fresh ? launch_one<1, 128, true, K, N>(n, smem, st, a, r)
                                : launch_one<1, 128, false, K, N>(n, smem, st, a, r);
        return !fp8 ? launch_one<2, 64, false, K, N>(n, smem, st, a, r)
                    : fresh ? launch_one<1, 64, true, K, N>(n, smem, st, a, r)
                            : launch_one<1, 64, false, K, N>(n, smem, st, a, r);
    });
}

}  // namespace pkv
