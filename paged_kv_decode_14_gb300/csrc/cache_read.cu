// Paged cache -> rows: the inverse of the appends.  Contract:
// include/pagedkv.h, pkv_paged_kv_read.
//
// Pure data movement (FP8: one multiply a value), so the bound is HBM: each
// cache byte read once, each row byte written once.  A CTA takes one page
// position of one sequence, all its kv-heads (adjacent in the cache: one
// contiguous piece of a block's K and of its V).  Inside a page a 16-byte
// chunk holds consecutive elements of one token, and the 8 chunks of 8 tokens
// are adjacent; a warp takes 4 tokens x 8 chunks of the head dimension, so
// its loads cover whole 64-byte pieces and its stores whole 128-byte (or
// longer) pieces of rows.  Measured: 64k FP8 tokens of 8 heads of 128 to bf16,
// 430 MB, 69.5 us = 6.2 TB/s; from a bf16 cache, 573 MB, 93.7 us = 6.1 TB/s.  (K and
// V in CTAs of their own, 16-byte stores: 87 us against 74, replays of one call.)
#include <type_traits>

#include "rows.cuh"

namespace pkv {
namespace cache_read {

using rows::View;

constexpr int kThreads = 256;
constexpr int kLoads = 3;              // 16-byte loads a thread has in flight (with 6 resident CTAs an SM)

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

struct Arg {
    const uint8_t *k_cache, *v_cache;
    const float *k_scales, *v_scales;
    View k, v;                         // data nullptr: not wanted
    const int32_t *tables, *lens, *starts;
    int* err;
    int64_t num_blocks, num_rows;
    int num_seqs, max_blocks, Hkv;
    bool wide;                         // the rows' 32-byte pieces are aligned
};

// n elements of T (a whole cache chunk), 32 bytes at a time where the rows allow it: two 16-byte
// stores of a sector reach L2 as two partial writes.
template <typename T>
__device__ __forceinline__ void store_chunk(uint8_t* dst, const float* x, int n, bool wide) {
#pragma unroll
    for (int e = 0; e < 16; e += 2 * rows::Chunk<T>::N) {
        if (e >= n) continue;
        const uint4 a = rows::Chunk<T>::pack(x + e);
        if (e + rows::Chunk<T>::N >= n) {                  // (16 bytes in all)
            *reinterpret_cast<uint4*>(dst + e * sizeof(T)) = a;
            continue;
        }
        const uint4 b = rows::Chunk<T>::pack(x + e + rows::Chunk<T>::N);
        if (wide) {
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            rows::store32(dst + e * sizeof(T), w);
        } else {
            *reinterpret_cast<uint4*>(dst + e * sizeof(T)) = a;
            *reinterpret_cast<uint4*>(dst + e * sizeof(T) + 16) = b;
        }
    }
}

// Cache chunk x of a block: K's, then V's, head by head; within a page a warp
// takes 8 chunks of the head dimension x 4 tokens (NCH = 4: 4 x 8).
struct At {
    int g, ch, off;
    bool v;
};
template <int NCH>
__device__ __forceinline__ At place(int x, int total) {
    constexpr int CW = NCH < 8 ? NCH : 8, TW = 32 / CW;
    At a;
    a.v = x >= total;
    x -= a.v ? total : 0;
    a.g = x / (kBlock * NCH);
    const int y = x % (kBlock * NCH), l = y % 32, w = y / 32;
    a.ch = (w % (NCH / CW)) * CW + l % CW;
    a.off = (w / (NCH / CW)) * TW + l / CW;
    return a;
}

// E: bytes of a cache element (2: bf16, 1: e4m3)
template <typename T, int E, int D>
__global__ void __launch_bounds__(kThreads, 6) read_kernel(const __grid_constant__ Arg a) {
    constexpr int C = 16 / E, NCH = D / C;                 // elements a chunk, chunks a row
    constexpr int PAGE = kBlock * D * E;
    __shared__ int s_seq, s_page;
    __shared__ int64_t s_row;
    griddep_wait();                                        // (no early trigger: an append reads its rows before its own wait)
    // this CTA's unit: the page position `blockIdx.x` of the sequences' pages laid end to end
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int64_t unit = blockIdx.x, row = 0;
        int seq = -1, page = 0;
        for (int b0 = 0; b0 < a.num_seqs; b0 += 32) {
            const int b = b0 + lane;
            int n = b < a.num_seqs ? a.lens[b] : 0;
            const int st = b < a.num_seqs && a.starts ? a.starts[b] : 0;
            if (n < 0 || st < 0 || (n > 0 && ((int64_t)st + n + kBlock - 1) / kBlock > a.max_blocks)) {
                raise_error(a.err, PKV_DEVERR_LENGTH);     // (the grid has a spare CTA per such sequence: one sees it)
                n = max(n, 0);                             // (its rows stay reserved, its pages are not read)
            }
            const bool bad = n > 0 && (st < 0 || ((int64_t)st + n + kBlock - 1) / kBlock > a.max_blocks);
            int64_t pages = n > 0 && !bad ? ((int64_t)st + n - 1) / kBlock - st / kBlock + 1 : 0;
            int64_t pu = pages, pr = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, pu, o), y = __shfl_up_sync(0xffffffffu, pr, o);
                if (lane >= o) {
                    pu += x;
                    pr += y;
                }
            }
            const unsigned hit = __ballot_sync(0xffffffffu, pu > unit);
            if (hit) {
                const int l = __ffs(hit) - 1;
                seq = b0 + l;
                page = (int)(unit - __shfl_sync(0xffffffffu, pu - pages, l));
                row += __shfl_sync(0xffffffffu, pr - n, l);
                break;
            }
            unit -= __shfl_sync(0xffffffffu, pu, 31);
            row += __shfl_sync(0xffffffffu, pr, 31);
        }
        if (lane == 0) {
            s_seq = seq;
            s_page = page;
            s_row = row;
        }
    }
    __syncthreads();
    const int b = s_seq;
    if (b < 0) return;
    const int64_t n = a.lens[b], st = a.starts ? a.starts[b] : 0;
    const int64_t pg = st / kBlock + s_page;               // page of the sequence
    const int32_t blk = a.tables[(size_t)b * a.max_blocks + pg];
    if (blk < 0 || blk >= a.num_blocks) {
        if (threadIdx.x == 0) raise_error(a.err, PKV_DEVERR_BLOCK_ID);
        return;
    }
    // tokens [lo, hi) of the page are wanted; token off's row is row0 + off
    const int lo = (int)max(st - pg * kBlock, (int64_t)0), hi = (int)min(st + n - pg * kBlock, (int64_t)kBlock);
    const int64_t row0 = s_row + pg * kBlock - st;
    if (row0 + hi > a.num_rows && threadIdx.x == 0) raise_error(a.err, PKV_DEVERR_LENGTH);
    // chunks of K, then of V (or of the one that is wanted)
    const int total = a.Hkv * kBlock * NCH, first = a.k.data ? 0 : total,
              last = a.v.data ? 2 * total : total;
    const size_t block = (size_t)blk * a.Hkv;
    for (int x0 = first + threadIdx.x; x0 < last; x0 += kLoads * kThreads) {
        uint4 raw[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const At at = place<NCH>(x0 + u * kThreads, total);
            if (x0 + u * kThreads < last && at.off >= lo && at.off < hi)
                raw[u] = ld_stream((at.v ? a.v_cache : a.k_cache) + (block + at.g) * PAGE + ((at.off >> 3) * NCH + at.ch) * 128 +
                                   (at.off & 7) * 16);
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const At at = place<NCH>(x0 + u * kThreads, total);
            if (x0 + u * kThreads >= last || at.off < lo || at.off >= hi || row0 + at.off >= a.num_rows) continue;
            const View& out = at.v ? a.v : a.k;
            uint8_t* dst = out.row(row0 + at.off, at.g) + at.ch * C * sizeof(T);
            float v[16];
            if constexpr (E == 2) {
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    *reinterpret_cast<uint4*>(dst) = raw[u];
                } else {
                    rows::Chunk<__nv_bfloat16>::unpack(raw[u], v);
                    store_chunk<T>(dst, v, 8, a.wide);
                }
            } else {
                const float sc = (at.v ? a.v_scales : a.k_scales)[block + at.g];
                const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 p = e4m3x2_to_float2(w[j]), q = e4m3x2_to_float2(w[j] >> 16);
                    v[4 * j] = p.x * sc;
                    v[4 * j + 1] = p.y * sc;
                    v[4 * j + 2] = q.x * sc;
                    v[4 * j + 3] = q.y * sc;
                }
                store_chunk<T>(dst, v, 16, a.wide);
            }
        }
    }
}

}  // namespace cache_read

cudaError_t launch_cache_read(const pkv_cache& c, const int32_t* tables, int max_blocks, const int32_t* starts,
                              const int32_t* lens, int num_seqs, int64_t num_rows, const pkv_rows* k,
                              const pkv_rows* v, int dtype, int* err, cudaStream_t st) {
    using namespace cache_read;
    const int e = dtype == PKV_FP32 ? 4 : 2;
    auto view = [&](const pkv_rows* r) {
        View x = {};
        if (r) {
            x.data = (uint8_t*)r->data;
            x.ts = r->token_stride * e;
            x.hs = r->head_stride * e;
            x.heads = r->num_heads;
        }
        return x;
    };
    Arg a = {(const uint8_t*)c.k_cache, (const uint8_t*)c.v_cache, c.k_scales, c.v_scales, view(k), view(v), tables,
             lens, starts, err, c.num_blocks, num_rows, num_seqs, max_blocks, c.num_kv_heads, true};
    a.wide = (!k || rows::wide(a.k)) && (!v || rows::wide(a.v));
    // every sequence's rows touch at most ceil(len / 16) pages, one more where it starts inside a page
    const int64_t units = num_rows / kBlock + (int64_t)num_seqs * (starts ? 2 : 1);
    if (units > 0x7fffffff) return cudaErrorInvalidValue;
    auto go = [&](auto kern) { return launch_pdl(kern, dim3((unsigned)units), dim3(kThreads), (size_t)0, st, a); };
    auto of = [&](auto zero) {
        using T = decltype(zero);
        if (c.kv_dtype == PKV_KV_FP8_E4M3)
            return c.head_dim == 128 ? go(read_kernel<T, 1, 128>) : go(read_kernel<T, 1, 64>);
        return c.head_dim == 128 ? go(read_kernel<T, 2, 128>) : go(read_kernel<T, 2, 64>);
    };
    if (dtype == PKV_BF16) return of(__nv_bfloat16());
    if (dtype == PKV_FP16) return of(__half());
    return of(float());
}

}  // namespace pkv
