// Rows of projections (queries, keys, values): strided views in three types,
// per-head RMS norms and rotary positions, shared by the kernels that read or
// write such rows.
#pragma once

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

// The rotation of a launch.  turn[i] is pair i's advance per position as a
// fraction of a full turn in 64-bit fixed point, so position * turn wraps at
// whole turns by itself: the angle of any 32-bit position keeps 32 fraction
// bits with one integer multiply and no 64-bit floating point (whose rate on
// this chip is a small fraction of the integer rate).
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

// Rotates rows held across the GS lanes of a group, CPL chunks of 16 bytes
// a lane (chunk c of a row: lane c % GS, register set c / GS).
//   (a, b) -> (a c - b s, b c + a s) for the two elements of a pair.
// A lane's elements keep their places for every row, so the (cos, sin) of its
// elements sit in registers for all heads of a token.
template <typename T, int GS, int CPL>
struct Rotator {
    static constexpr int N = Chunk<T>::N;
    float c[CPL][N], s[CPL][N];       // s: negative for a pair's first element
    int lane, pairs, rd;
    bool inter, aligned;              // aligned: a pair's two elements lie whole chunks apart

    // cs: (cos, sin) of the token's pairs in shared memory
    __device__ __forceinline__ void load(const Rope& r, const float2* cs, int lane_) {
        lane = lane_;
        pairs = r.pairs;
        rd = 2 * r.pairs;
        inter = r.interleaved != 0;
        aligned = pairs % N == 0;
#pragma unroll
        for (int j = 0; j < CPL; ++j)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int d = (lane + j * GS) * N + e;
                c[j][e] = 1.f;
                s[j][e] = 0.f;
                if (d < rd) {
                    const int i = inter ? d >> 1 : d < pairs ? d : d - pairs;
                    const bool first = inter ? !(d & 1) : d < pairs;
                    const float2 v = cs[i];
                    c[j][e] = v.x;
                    s[j][e] = first ? -v.y : v.y;
                }
            }
    }
    // stage: this group's [rows of D floats] in shared memory (unaligned rotate-half pairs only)
    __device__ __forceinline__ void apply(float (&x)[CPL][N], float* stage) const {
        if (rd == 0) return;
        if (inter) {
#pragma unroll
            for (int j = 0; j < CPL; ++j)
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    if ((lane + j * GS) * N + e >= rd) continue;
                    const float a = x[j][e], b = x[j][e + 1];
                    x[j][e] = fmaf(a, c[j][e], b * s[j][e]);
                    x[j][e + 1] = fmaf(b, c[j][e + 1], a * s[j][e + 1]);
                }
        } else if (aligned) {
            const int pc = pairs / N;                      // chunks between a pair's elements
            float y[CPL][N];
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const int ch = lane + j * GS, p = ch < pc ? ch + pc : ch - pc;   // the partner chunk
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    if constexpr (CPL == 1) {
                        y[j][e] = __shfl_sync(0xffffffffu, x[0][e], p & (GS - 1), GS);
                    } else {
                        const float u = __shfl_sync(0xffffffffu, x[0][e], p & (GS - 1), GS);
                        const float v = __shfl_sync(0xffffffffu, x[1][e], p & (GS - 1), GS);
                        y[j][e] = (p / GS) & 1 ? v : u;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < CPL; ++j)
                if (lane + j * GS < 2 * pc)
#pragma unroll
                    for (int e = 0; e < N; ++e) x[j][e] = fmaf(x[j][e], c[j][e], y[j][e] * s[j][e]);
        } else {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < CPL; ++j)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const int d = (lane + j * GS) * N + e;
                    if (d < rd) stage[d] = x[j][e];
                }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < CPL; ++j)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const int d = (lane + j * GS) * N + e;
                    if (d < rd) x[j][e] = fmaf(x[j][e], c[j][e], stage[d < pairs ? d + pairs : d - pairs] * s[j][e]);
                }
        }
    }
};

// x *= w / sqrt(mean(x^2) + eps) over the row held by a group of GS lanes
// (lanes past the row hold zeros); sums and statistics in fp32.
template <typename T, int GS, int CPL>
__device__ __forceinline__ void rms_norm(float (&x)[CPL][Chunk<T>::N], const uint4 (&w)[CPL], bool weighted, float eps,
                                         float inv_dim) {
    constexpr int N = Chunk<T>::N;
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < CPL; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e) ss = fmaf(x[j][e], x[j][e], ss);
#pragma unroll
    for (int o = GS / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, GS);
    const float inv = rsqrtf(fmaf(ss, inv_dim, eps));
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
        float g[N];
        if (weighted) Chunk<T>::unpack(w[j], g);
#pragma unroll
        for (int e = 0; e < N; ++e) x[j][e] = weighted ? x[j][e] * inv * g[e] : x[j][e] * inv;
    }
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
    for (int i = 0; i < a.pairs; ++i) {
        // radians per position -> the fraction of a turn, in units of 2^-64
        const double t = r->inv_freq[i] * 0.15915494309189533577;
        double f = t - (double)(long long)t;
        if (f < 0) f += 1.0;
        // (scaled by 2^63, not 2^64: a conversion to a signed 64-bit value is defined there;
        // a tiny negative fraction rounds up to a whole turn, which is none)
        a.turn[i] = f >= 1.0 ? 0 : (uint64_t)(int64_t)(f * 0x1p63) << 1;
    }
    return a;
}

}  // namespace rows
}  // namespace pkv
