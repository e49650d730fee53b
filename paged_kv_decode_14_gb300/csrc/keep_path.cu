// The accepted path of a tree of drafted tokens moved to the places behind the context.  Contract:
// include/pagedkv.h, pkv_paged_kv_keep_path.
//
// Cache row base + path[i] -> base + i for i < n, base = L - Q, within one sequence.  path ascends strictly, so
// path[i] >= i: rows taken in ascending order, a batch read before it is written, never overwrite a row that is
// still to be read.  A warp takes one (sequence, kv-head, K or V), a lane a 16-byte chunk of a row.
//
// bf16 codes, and e4m3 codes that stay in their block, move as they are.  An e4m3 row that changes its block changes
// its scale: code * scale of the old block, divided by the new one's (both in IEEE fp32), to the nearest code.
//
// A few KB a sequence: what it costs is the chain of dependent reads (lengths, path, table, rows) and the launch: 3.4 us for
// the paths of 32 trees of up to 24 nodes (bf16, 8 heads of 128), 5.4 us for 256 trees of up to 64 (FP8, recoded).
#include "common.cuh"

namespace pkv {
namespace keep {

constexpr int kThreads = 128;
constexpr int kLoads = 4;                  // chunks a lane holds of a batch

struct Arg {
    uint8_t *k, *v;
    const float *k_scales, *v_scales;      // nullptr: bf16
    const int32_t *tables, *ctx_lens, *q_lens, *path, *path_lens;
    int* err;
    int64_t num_blocks;
    int num_seqs, max_blocks, max_path, Hkv, head_dim;
};

__device__ __forceinline__ uint32_t recode4(uint32_t w, float from, float to) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float2 x = e4m3x2_to_float2(w >> (8 * i));
        const float2 y = make_float2(__fdiv_rn(__fmul_rn(x.x, from), to), __fdiv_rn(__fmul_rn(x.y, from), to));
        r |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (8 * i);
    }
    return r;
}

__global__ void __launch_bounds__(kThreads) keep_kernel(const Arg a) {
    griddep_wait();
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int heads = 2 * a.Hkv, b = (int)(unit / heads), h = (int)(unit % heads);
    if (b >= a.num_seqs) return;
    const int L = a.ctx_lens[b], Q = a.q_lens[b], n = a.path_lens[b];
    const int32_t* path = a.path + (int64_t)b * a.max_path;
    bool bad = Q < 0 || L < Q || n < 0 || n > Q || n > a.max_path || (L > 0 && (L - 1) / kBlock >= a.max_blocks);
    if (!bad)
        for (int i = lane; i < n; i += 32) bad |= path[i] >= Q || path[i] <= (i > 0 ? path[i - 1] : -1);
    if (__any_sync(0xffffffffu, bad)) {
        if (lane == 0) raise_error(a.err, PKV_DEVERR_LENGTH);
        return;
    }
    const bool is_v = h >= a.Hkv, fp8 = a.k_scales != nullptr;
    const int g = is_v ? h - a.Hkv : h, e = fp8 ? 1 : 2;
    const int chunks = a.head_dim * e / 16;               // of a row: 4 to 16, a power of two
    const int64_t page = (int64_t)kBlock * a.head_dim * e;
    uint8_t* cache = is_v ? a.v : a.k;
    const float* scales = is_v ? a.v_scales : a.k_scales;
    const int32_t* table = a.tables + (int64_t)b * a.max_blocks;
    const int base = L - Q;
    // a chunk's place in the cache, by block and token of the block
    auto place = [&](int id, int off, int ch) {
        return cache + ((int64_t)id * a.Hkv + g) * page + (((off / 8) * chunks + ch) * 8 + off % 8) * 16;
    };
    for (int x0 = 0; x0 < n * chunks; x0 += 32 * kLoads) {
        uint4 v[kLoads];
        uint8_t* to[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int x = x0 + j * 32 + lane, i = x / chunks, ch = x % chunks;
            to[j] = nullptr;
            if (i >= n || path[i] == i) continue;
            const int src = base + path[i], dst = base + i;
            const int id0 = table[src / kBlock], id1 = table[dst / kBlock];
            if (id0 < 0 || id0 >= a.num_blocks || id1 < 0 || id1 >= a.num_blocks) {
                raise_error(a.err, PKV_DEVERR_BLOCK_ID);
                continue;
            }
            v[j] = *reinterpret_cast<const uint4*>(place(id0, src % kBlock, ch));
            to[j] = place(id1, dst % kBlock, ch);
            if (fp8 && id0 != id1) {
                const float f = scales[(int64_t)id0 * a.Hkv + g], t = scales[(int64_t)id1 * a.Hkv + g];
                v[j] = make_uint4(recode4(v[j].x, f, t), recode4(v[j].y, f, t), recode4(v[j].z, f, t), recode4(v[j].w, f, t));
            }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (to[j]) *reinterpret_cast<uint4*>(to[j]) = v[j];
        __syncwarp();
    }
}

}  // namespace keep

cudaError_t launch_keep_path(const pkv_cache& c, const int32_t* tables, int max_blocks, const int32_t* ctx_lens,
                             const int32_t* q_lens, const int32_t* path, int max_path, const int32_t* path_lens,
                             int num_seqs, int* err, cudaStream_t st) {
    using namespace keep;
    const bool fp8 = c.kv_dtype == PKV_KV_FP8_E4M3;
    const Arg a{(uint8_t*)c.k_cache, (uint8_t*)c.v_cache, fp8 ? c.k_scales : nullptr, fp8 ? c.v_scales : nullptr, tables,
                ctx_lens, q_lens, path, path_lens, err, c.num_blocks, num_seqs, max_blocks, max_path, c.num_kv_heads,
                c.head_dim};
    const int64_t units = (int64_t)num_seqs * c.num_kv_heads * 2, ctas = (units + kThreads / 32 - 1) / (kThreads / 32);
    return launch_pdl(keep_kernel, dim3((unsigned)ctas), dim3(kThreads), (size_t)0, st, a);
}

}  // namespace pkv
