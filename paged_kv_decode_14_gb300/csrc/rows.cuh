// Rows of projections (queries, keys, values): strided views in three types,
// per-head RMS norms and rotary positions, shared by the kernels that read or
// write such rows.
#pragma once

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"

namespace pkv {
namespace rows {

// One tensor of rows: element (token t, head h, dim d) is d elements past
// data + t * ts + h * hs (byte strides).
struct View {
    uint8_t* data;
    int64_t ts, hs;
    int heads;
    __device__ __forceinline__ uint8_t* row(int64_t t, int h) const { return data + t * ts + h * hs; }
};

// 32 bytes to a 32-byte aligned address.
__device__ __forceinline__ void store32(uint8_t* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// Rows of which every 32-byte piece is 32-byte aligned.
__host__ inline bool wide(const View& v) {
    return (((uintptr_t)v.data | (uintptr_t)v.ts | (uintptr_t)v.hs) & 31) == 0;
}

// The rotation of a launch.  turn[i] is pair i's advance per position as a
// fraction of a full turn in 64-bit fixed point, so position * turn wraps at
// whole turns by itself: the angle of any 32-bit position is good to 2^-31 of a
// turn (its top 32 bits are used; the advance is off by 2^-64, see turn_of) with
// one integer multiply and no 64-bit floating point (whose rate on this chip is
// a small fraction of the integer rate).  It is then rounded to fp32.
struct Rope {
    uint64_t turn[PKV_ROPE_MAX_PAIRS];
    float magnitude;
    int pairs;          // 0: no rotation
    int interleaved;    // pairs (2i, 2i + 1) instead of (i, i + pairs)
    int negate;         // rotate by the negated angle
};

// (cos, sin) of pair i at position pos, times the magnitude.
__device__ __forceinline__ float2 angle(const Rope& r, int i, int pos) {
    const uint64_t a = (uint64_t)(int64_t)pos * r.turn[i];
    // the top 32 bits, as a signed fraction of a turn: [-1/2, 1/2)
    const float half_turns = (float)(int32_t)(uint32_t)(a >> 32) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * r.magnitude, (r.negate ? -s : s) * r.magnitude);
}

// 16 bytes of a row <-> fp32.
template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = bf16_lo(w[j]);
            x[2 * j + 1] = bf16_hi(w[j]);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float* x) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Chunk<__half> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            x[2 * j] = f.x;
            x[2 * j + 1] = f.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float* x) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 p = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Chunk<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 v, float* x) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float* x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

// A row is held by a group of GS lanes, two 16-byte chunks a lane: chunk c by
// lane c % GS in register set c / GS.  (Two chunks: the usual rotate-half pair,
// which spans half a head, then lies in one lane's two sets.)
constexpr int kSets = 2;
template <typename T>
__host__ __device__ constexpr int lanes_of(int dim) {      // the fewest that hold a row
    return dim / Chunk<T>::N <= 8 ? 4 : dim / Chunk<T>::N <= 16 ? 8 : dim / Chunk<T>::N <= 32 ? 16 : 32;
}

// How a kernel rotates: pairs inside a lane's chunk (interleaved), pairs in a
// lane's two sets (rotate-half over the whole head), pairs whole chunks apart,
// anything else (or nothing).
enum Kind { kInside = 0, kSetPairs = 1, kChunks = 2, kGeneral = 3 };
template <typename T>
__host__ inline Kind rope_kind(const Rope& r, int lanes) {
    if (r.pairs == 0) return kGeneral;
    if (r.interleaved) return kInside;
    if (r.pairs == lanes * Chunk<T>::N) return kSetPairs;
    return r.pairs % Chunk<T>::N == 0 ? kChunks : kGeneral;
}

// Rotates rows: (a, b) -> (a c - b s, b c + a s) for the two elements of a pair.
// A lane's elements keep their places for every row, so the (cos, sin) of its
// elements are loaded once a token and serve all its heads.
template <typename T, int GS, int KIND>
struct Rotator {
    static constexpr int N = Chunk<T>::N;
    static constexpr int S = KIND == kSetPairs ? 1 : kSets, M = KIND == kInside ? N / 2 : N;   // (cos, sin) held
    float c[S][M], s[S][M];           // s: negative for a pair's first element (kInside, kSetPairs: the pair's)
    int lane, pairs;
    int part[kSets];                  // rotated elements of a chunk

    __device__ __forceinline__ void init(const Rope& r, int lane_) {
        lane = lane_;
        pairs = r.pairs;
#pragma unroll
        for (int j = 0; j < kSets; ++j) part[j] = min(max(2 * pairs - (lane + j * GS) * N, 0), N);
    }
    // cs: (cos, sin) of a token's pairs
    __device__ __forceinline__ void load(const float2* cs) {
#pragma unroll
        for (int j = 0; j < S; ++j)
#pragma unroll
            for (int e = 0; e < M; ++e) {
                const int el = KIND == kInside ? 2 * e : e;
                if (KIND != kSetPairs && el >= part[j]) continue;
                const int d = (lane + j * GS) * N + el;
                const bool first = KIND == kInside || KIND == kSetPairs || d < pairs;
                const float2 v = cs[KIND == kInside ? d >> 1 : first ? d : d - pairs];
                c[j][e] = v.x;
                s[j][e] = first && (KIND == kChunks || KIND == kGeneral) ? -v.y : v.y;
            }
    }
    // stage: this group's row of D floats in shared memory (kGeneral, which covers rotate-half only)
    __device__ __forceinline__ void apply(float (&x)[kSets][N], float* stage) const {
        if constexpr (KIND == kInside) {
#pragma unroll
            for (int j = 0; j < kSets; ++j)
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    if (e >= part[j]) continue;
                    const float a = x[j][e], b = x[j][e + 1];
                    x[j][e] = fmaf(a, c[j][e / 2], -b * s[j][e / 2]);
                    x[j][e + 1] = fmaf(b, c[j][e / 2], a * s[j][e / 2]);
                }
        } else if constexpr (KIND == kSetPairs) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float a = x[0][e], b = x[1][e];
                x[0][e] = fmaf(a, c[0][e], -b * s[0][e]);
                x[1][e] = fmaf(b, c[0][e], a * s[0][e]);
            }
        } else if constexpr (KIND == kChunks) {
            const int pc = pairs / N;                      // chunks between a pair's elements
            float y[kSets][N];
#pragma unroll
            for (int j = 0; j < kSets; ++j) {
                const int ch = lane + j * GS, p = ch < pc ? ch + pc : ch - pc;   // the partner chunk
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float u = __shfl_sync(0xffffffffu, x[0][e], p & (GS - 1), GS);
                    const float v = __shfl_sync(0xffffffffu, x[1][e], p & (GS - 1), GS);
                    y[j][e] = (p / GS) & 1 ? v : u;
                }
            }
#pragma unroll
            for (int j = 0; j < kSets; ++j)
                if (part[j] > 0)                           // (whole chunks)
#pragma unroll
                    for (int e = 0; e < N; ++e) x[j][e] = fmaf(x[j][e], c[j][e], y[j][e] * s[j][e]);
        } else {
            if (pairs == 0) return;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kSets; ++j)
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (e < part[j]) stage[(lane + j * GS) * N + e] = x[j][e];
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kSets; ++j)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    if (e >= part[j]) continue;
                    const int d = (lane + j * GS) * N + e;
                    x[j][e] = fmaf(x[j][e], c[j][e], stage[d < pairs ? d + pairs : d - pairs] * s[j][e]);
                }
        }
    }
};

// x *= w / sqrt(mean(x^2) + eps) over the row held by a group of GS lanes
// (lanes past the row hold zeros); sums and statistics in fp32.  Squares leave
// fp32's range long before the values do (from 2^64 up, from 2^-75 down): where
// some row's mean is out of the range that is sure to be right, the warp takes
// its rows times a power of two that brings the row's largest value, or
// sqrt(eps), near 1 (1 for the rows that were in range: the same bits).  The
// vote costs 1 to 2 % (8192 tokens of 40 heads of 128 bf16 31.2 -> 31.8 us).
template <typename T, int GS>
__device__ __forceinline__ void rms_norm(float (&x)[kSets][Chunk<T>::N], const uint4 (&w)[kSets], bool weighted,
                                         float eps, float inv_dim) {
    constexpr int N = Chunk<T>::N;
    auto mean_square = [&](float plus) {
        float ss[kSets] = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < N; ++e)
#pragma unroll
            for (int j = 0; j < kSets; ++j) ss[j] = fmaf(x[j][e], x[j][e], ss[j]);
        float sum = ss[0] + ss[1];
#pragma unroll
        for (int o = GS / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o, GS);
        return fmaf(sum, inv_dim, plus);
    };
    const float mean = mean_square(eps);
    float inv = rsqrtf(mean);                              // (under way while the warp votes)
    const bool sure = __float_as_uint(mean) - __float_as_uint(0x1p-100f) <= 220u << 23;   // 2^-100 .. 2^120
    if (!__all_sync(0xffffffffu, sure)) {
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e)
#pragma unroll
            for (int j = 0; j < kSets; ++j) top = fmaxf(top, fabsf(x[j][e]));
#pragma unroll
        for (int o = GS / 2; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o, GS));
        top = fmaxf(top, sqrtf(eps));
        // (an infinite row, and one of zeros without eps, stay as the formula has them)
        const bool plain = sure || !(top > 0.f) || !(top < INFINITY);
        const float f = plain ? 1.f : __uint_as_float((uint32_t)max(254 - (int)(__float_as_uint(top) >> 23), 1) << 23);
#pragma unroll
        for (int e = 0; e < N; ++e)
#pragma unroll
            for (int j = 0; j < kSets; ++j) x[j][e] *= f;
        inv = rsqrtf(mean_square(eps * f * f));
    }
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
        float g[N];
        if (weighted) Chunk<T>::unpack(w[j], g);
#pragma unroll
        for (int e = 0; e < N; ++e) x[j][e] = weighted ? x[j][e] * inv * g[e] : x[j][e] * inv;
    }
}

// Host: radians per position -> the fraction of a turn, in units of 2^-64.  The
// position multiplies its error, and 53 bits of the product f / 2 pi, or of 1 / 2 pi
// itself, would leave 2^-25 of a turn at position 2^31 for f = 1 (a whole turn
// for f near 1e9): the product and its rounding error are both kept.
__host__ inline uint64_t turn_of(double f) {
    constexpr double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;   // 1 / 2 pi
    const double x = std::fabs(f);
    const volatile double product = x * hi;                // (rounded here: not to be fused into what uses it)
    const double p = product, e = std::fma(x, hi, -p) + x * lo;
    const double part = (p - std::floor(p)) * 0x1p32, top = std::floor(part);  // (exact)
    const uint64_t t = ((uint64_t)top << 32) + (uint64_t)(int64_t)std::nearbyint((part - top) * 0x1p32 + e * 0x1p64);
    return f < 0 ? 0 - t : t;
}

// Host: the kernel's form of a rotation.
__host__ inline Rope rope_arg(const pkv_rope* r, bool negate) {
    Rope a = {};
    a.magnitude = 1.f;
    if (!r || r->rotary_dim == 0) return a;
    a.pairs = r->rotary_dim / 2;
    a.interleaved = r->interleaved != 0;
    a.magnitude = r->magnitude;
    a.negate = negate;
    for (int i = 0; i < a.pairs; ++i) a.turn[i] = turn_of(r->inv_freq[i]);
    return a;
}

// ------------------------------------------------------------------ a warp's share of the rows

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;                 // row groups whose loads a warp has in flight
constexpr int kWarpsPerSm = 32;

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// A warp's shared memory: the ring of row groups in flight, the (cos, sin) of
// one token's pairs, and (unaligned rotate-half pairs) a group's rows in fp32.
constexpr int kRing = kAhead * kSets * 512;
template <typename T, int GS>
__host__ inline size_t rows_smem(const Rope& r, int D) {
    const size_t stage = r.pairs > 0 && !r.interleaved && r.pairs % Chunk<T>::N ? (size_t)(32 / GS) * D * 4 : 0;
    return kWarps * (kRing + (((size_t)r.pairs * 8 + 15) / 16 * 16) + (stage + 15) / 16 * 16);
}
// The most of it: a row fills its lanes' chunks, all of it rotated.
template <typename T, int GS>
__host__ constexpr size_t rows_smem_most() {
    constexpr size_t D = GS * kSets * Chunk<T>::N;
    return kWarps * (kRing + D / 2 * 8 + 32 / GS * D * 4);
}

// Where a warp is in its share: a group of 32 / GS rows of one tensor's heads,
// of one token.  A token's groups are q's, then k's.
template <int GS>
struct Cursor {
    static constexpr int RPW = 32 / GS;
    const uint8_t* p;       // this lane's first 16 bytes of its row
    int64_t t;
    int64_t step;           // bytes to the next group's row
    int rows;               // heads from this lane's row on (<= 0: none)
    int left;               // groups left of this tensor's heads
    bool k;                 // in k's heads
    __device__ __forceinline__ void open(const View& v, int64_t t_, int g, int l, int sub) {
        t = t_;
        p = v.row(t, g * RPW + sub) + l * 16;
        step = v.hs * RPW;
        rows = v.heads - g * RPW - sub;
        left = (v.heads + RPW - 1) / RPW - g;
    }
    __device__ __forceinline__ void start(const View& q, const View& kk, int64_t u, int l, int sub) {
        const int gq = (q.heads + RPW - 1) / RPW, gk = (kk.heads + RPW - 1) / RPW;
        const int64_t tt = u / (gq + gk);
        const int g = (int)(u - tt * (gq + gk));
        k = g >= gq;
        open(k ? kk : q, tt, k ? g - gq : g, l, sub);
    }
    __device__ __forceinline__ void next(const View& q, const View& kk, int l, int sub) {
        p += step;
        rows -= RPW;
        if (--left > 0) return;
        const bool to_k = !k && kk.heads > 0;
        const int64_t tt = to_k ? t : t + 1;
        k = to_k;
        open(to_k ? kk : q, tt, 0, l, sub);
    }
};

// The norm and rotation of one warp's share of the rows, GS lanes a row: row
// groups [u, end) of all tokens' groups laid end to end.  A lane copies its own
// 16 bytes of a row to shared memory kAhead groups before it uses them
// (cp.async), so the bytes in flight do not cost registers and warps never wait
// for each other.  What bounds it beside HBM is the instructions of a group, so
// pointers step from head to head.  (8192 tokens of 40 heads of 128 bf16, 168
// MB: direct loads, a CTA a token with its angles behind a barrier, 52 us; this
// with the addresses computed from scratch, 39 us; as it is, 33 us, each as a graph
// of its own; in a graph of twelve calls, without such a graph's 4 us, 29 us = 5.8 TB/s.)
template <typename T, int GS, int KIND, bool NORM>
__device__ __forceinline__ void warp_rows(const View& qi, const View& qo, const View& ki, const View& ko, const T* qw,
                                          const T* kw, float eps, int D, const Rope& rope,
                                          const int32_t* positions, int64_t tokens, int64_t u, int64_t end,
                                          uint8_t* smem) {
    constexpr int N = Chunk<T>::N;
    if (u >= end) return;
    const int lane = threadIdx.x & 31, l = lane & (GS - 1), sub = lane / GS;
    const int nch = D / N;
    float2* cs = reinterpret_cast<float2*>(smem + kRing);
    float* stage = reinterpret_cast<float*>(smem + kRing + (rope.pairs * 8 + 15) / 16 * 16) + sub * D;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + lane * 16, ring_end = ring + kRing;
    Cursor<GS> from, to;
    from.start(qi, ki, u, l, sub);
    to.start(qo, ko, u, l, sub);
    const int count = (int)(end - u);
    int fetched = 0;
    uint32_t fill = ring, use = ring;
    auto fetch = [&] {
        if (fetched < count) {
#pragma unroll
            for (int j = 0; j < kSets; ++j)
                if (l + j * GS < nch && from.rows > 0) cp_async_16(fill + j * 512, from.p + j * GS * 16);
            ++fetched;
            from.next(qi, ki, l, sub);
        }
        cp_async_commit();
        fill += kSets * 512;
        if (fill == ring_end) fill = ring;
    };
#pragma unroll 1
    for (int x = 0; x < kAhead; ++x) fetch();
    uint4 wq[kSets], wk[kSets];
#pragma unroll
    for (int j = 0; j < kSets; ++j) {
        const int ch = l + j * GS;
        wq[j] = NORM && qw && ch < nch ? *reinterpret_cast<const uint4*>(qw + ch * N) : make_uint4(0, 0, 0, 0);
        wk[j] = NORM && kw && ch < nch ? *reinterpret_cast<const uint4*>(kw + ch * N) : make_uint4(0, 0, 0, 0);
    }
    Rotator<T, GS, KIND> rot;
    rot.init(rope, l);
    const float inv_dim = 1.f / (float)D;
    int64_t have = -1;                                     // the token whose angles rot holds
    int pos = rope.pairs > 0 ? positions[to.t] : 0;
    for (int n = 0; n < count; ++n) {
        if (rope.pairs > 0 && to.t != have) {
            have = to.t;
            __syncwarp();
            for (int i = lane; i < rope.pairs; i += 32) cs[i] = angle(rope, i, pos);
            __syncwarp();
            rot.load(cs);
            if (have + 1 < tokens) pos = positions[have + 1];   // (the next token's, long before it is needed)
        }
        cp_async_wait<kAhead - 1>();                       // (a lane reads what it copied itself)
        float x[kSets][N];
#pragma unroll
        for (int j = 0; j < kSets; ++j) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (l + j * GS < nch && to.rows > 0)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                             : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                             : "r"(use + j * 512)
                             : "memory");
            Chunk<T>::unpack(v, x[j]);
        }
        if constexpr (NORM) rms_norm<T, GS>(x, to.k ? wk : wq, (to.k ? kw : qw) != nullptr, eps, inv_dim);
        rot.apply(x, stage);
#pragma unroll
        for (int j = 0; j < kSets; ++j)
            if (l + j * GS < nch && to.rows > 0)
                *reinterpret_cast<uint4*>(const_cast<uint8_t*>(to.p) + j * GS * 16) = Chunk<T>::pack(x[j]);
        use += kSets * 512;
        if (use == ring_end) use = ring;
        to.next(qo, ko, l, sub);
        fetch();
    }
    cp_async_wait<0>();
}

// Row groups of `tokens` tokens with these heads.
__host__ inline int64_t row_units(int64_t tokens, int q_heads, int k_heads, int rpw) {
    return tokens * ((q_heads + rpw - 1) / rpw + (k_heads + rpw - 1) / rpw);
}

// CTAs for `units` row groups: every warp one group at least, 32 warps an SM at most (of which 16 to 32 are
// resident, by the instance's registers: the rest follow as the first end).
__host__ inline unsigned rows_ctas(int64_t units, int num_sms) {
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>((units + kWarps - 1) / kWarps, (int64_t)num_sms * kWarpsPerSm / kWarps));
}

// ------------------------------------------------------------------ host

__host__ inline View view(const pkv_rows* r, int e) {
    View v = {};
    if (r) {
        v.data = (uint8_t*)r->data;
        v.ts = r->token_stride * e;
        v.hs = r->head_stride * e;
        v.heads = r->num_heads;
    }
    return v;
}

// f with the launch's kind of rotation and whether it has a norm, as constants.
template <typename F>
__host__ inline cudaError_t for_kind(Kind k, bool norm, F f) {
    auto g = [&](auto n) {
        switch (k) {
            case kInside: return f(std::integral_constant<int, kInside>(), n);
            case kSetPairs: return f(std::integral_constant<int, kSetPairs>(), n);
            case kChunks: return f(std::integral_constant<int, kChunks>(), n);
            default: return f(std::integral_constant<int, kGeneral>(), n);
        }
    };
    return norm ? g(std::true_type()) : g(std::false_type());
}

}  // namespace rows
}  // namespace pkv
