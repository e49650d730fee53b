// Block tables, slots and positions from request lengths, and the pool of free blocks behind them.  Contract:
// include/pagedkv.h, pkv_block_tables_update.
//
// With had_b and has_b the blocks of request b before and after, D the blocks that all dropping requests give back
// and N_b = sum over b' <= b of max(has - had, 0):
//   the i-th block given back (last request first, its last block first) goes to stack[count + i]
//   the k-th block needed (first request first, its first block first) is stack[count + D - 1 - k]
// so everything follows from three sums over the requests, and a call with the negated changes puts the pool back
// exactly.  No data to speak of moves: the time is a chain of dependent reads (lengths, table entries or the
// stack, then the writes) and one launch.  One cluster does it, of one CTA or, where there are many rows to write, eight:
// every CTA forms the sums for itself, and the cluster's barrier stands between the reads of the old state, the
// blocks given back and the blocks taken.
//
// Measured (a call that changes and one that takes it back, in a graph): 256 requests by one token 11.9 us, 1024 15 us,
// 8192 61 us; 96 requests of which some bring prompts of up to 1801 tokens and 24 leave 26.9 us.  One call on its own
// is about the latency of its launch, of a first fetch of its instructions and of five to seven reads that wait for one
// another.
#include <cooperative_groups.h>

#include "common.cuh"

namespace pkv {
namespace tables {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kMaxSeqs = 8192;             // requests a call takes: their state is held in shared memory
constexpr int kCluster = 8;
// Rows above which the cluster has kCluster CTAs (a call and one that takes its changes back, with 1 and 8 CTAs: 2048 rows
// 11.8 and 12.0 us, 4096 rows 12.6 and 11.5, 131072 rows 99 and 40).
constexpr int kManyRows = 2048;
// Blocks up to which a request's dropped blocks are one thread's work, not a warp's: a token's or a tree's worth.
constexpr int kFew = 4;
constexpr int kLoads = 4;                  // entries a lane has in flight where a warp gives a request's blocks back

struct Arg {
    int32_t* table;
    int32_t* lens;
    const int32_t* grow;
    int32_t* free_blocks;
    int32_t* free_count;
    int64_t* slots;
    int32_t* positions;
    int32_t* granted;
    int64_t* row_starts;
    int* err;
    int64_t num_blocks, num_rows;
    int num_seqs, max_blocks;
    bool pad;                              // rows behind the last request's: slot -1, position 0 (else left alone)
};

// Shared memory, by request: tokens before; change (0: refused or none); blocks given back by later
// requests; blocks needed by earlier ones; first row; rows (of a refused request too).
struct Shared {
    int *len, *change, *back, *need, *row, *rows;
    __device__ explicit Shared(int* p, int n) : len(p), change(p + n), back(p + 2 * n), need(p + 3 * n), row(p + 4 * n), rows(p + 5 * n) {}
};
constexpr int kArrays = 6;

__device__ __forceinline__ int blocks(int tokens) { return (int)(((unsigned)tokens + kBlock - 1) / kBlock); }

// Exclusive sums over the CTA's threads of N values, and their sums.
template <int N>
__device__ __forceinline__ void scan(int64_t (&v)[N], int64_t (&total)[N], int64_t (*part)[3]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = v[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t p = __shfl_up_sync(0xffffffffu, x[i], o);
            if (lane >= o) x[i] += p;
        }
        if (lane == 31) part[warp][i] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t mine = part[lane][i];                // (32 warps; every warp sums them for itself)
        int64_t u = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t p = __shfl_up_sync(0xffffffffu, u, o);
            if (lane >= o) u += p;
        }
        total[i] = __shfl_sync(0xffffffffu, u, 31);
        v[i] = x[i] - v[i] + __shfl_sync(0xffffffffu, u - mine, warp);
    }
    __syncthreads();
}

// The last i of [0, n) with at[i] <= x (at ascending, at[0] <= x).
__device__ __forceinline__ int find(const int* at, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (at[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads, 1) update_kernel(const Arg a) {
    extern __shared__ int smem[];
    __shared__ int64_t part[32][3];
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.num_seqs;
    const Shared s(smem, n);
    griddep_wait();
    int errors = 0;
    int count = *a.free_count;
    if (count < 0 || count > a.num_blocks) {              // nothing can be given or taken back
        errors |= PKV_DEVERR_LENGTH;
        count = -1;
    }

    // lengths and changes; a change that cannot be is none
    for (int b = tid; b < n; b += kThreads) {
        const int len = a.lens[b], g = a.grow[b];
        int change = g;
        const int64_t after = (int64_t)len + g;
        if (len < 0 || after < 0 || blocks(len) > a.max_blocks || after > (int64_t)a.max_blocks * kBlock || count < 0) {
            if (g != 0 || len < 0) errors |= PKV_DEVERR_LENGTH;
            change = 0;
        }
        s.len[b] = max(len, 0);
        s.change[b] = change;
        s.rows[b] = max(g, 0);
        s.back[b] = 0;
    }
    __syncthreads();
    // blocks that come back: the table's entries that are blocks are counted (a thread a request that drops few: with a
    // warp for each, 8192 requests by one token and back took 300 us, not 60)
    bool drops = false;
    for (int b = tid; b < n; b += kThreads) drops |= s.change[b] < 0;
    const bool any_drop = __syncthreads_or(drops);
    auto is_block = [&](int id) { return id >= 0 && id < a.num_blocks; };
    auto dropped = [&](int b) { return b < n && s.change[b] < 0 ? blocks(s.len[b]) - blocks(s.len[b] + s.change[b]) : 0; };
    // f(b), by a whole warp, for the requests b = first, first + step, ... that drop more than a few blocks
    auto warps = [&](int first, int step, auto f) {
        for (int b = first; b < n; b += 32 * step) {
            unsigned m = __ballot_sync(0xffffffffu, dropped(b + lane * step) > kFew);
            for (; m; m &= m - 1) f(b + (__ffs(m) - 1) * step);
        }
    };
    if (any_drop) {
        for (int b = tid; b < n; b += kThreads) {
            const int few = dropped(b);
            if (few == 0 || few > kFew) continue;
            int c = 0;
            for (int j = blocks(s.len[b]) - few; j < blocks(s.len[b]); ++j) {
                const int id = a.table[(int64_t)b * a.max_blocks + j];
                c += is_block(id);
                if (id >= a.num_blocks) errors |= PKV_DEVERR_BLOCK_ID;
            }
            s.back[b] = c;
        }
        warps(warp, kThreads / 32, [&](int b) {
            const int j1 = blocks(s.len[b]);
            int c = 0;
            for (int j = blocks(s.len[b] + s.change[b]) + lane; j < j1; j += 32 * kLoads) {
                int id[kLoads];
#pragma unroll
                for (int y = 0; y < kLoads; ++y) id[y] = j + 32 * y < j1 ? a.table[(int64_t)b * a.max_blocks + j + 32 * y] : -1;
#pragma unroll
                for (int y = 0; y < kLoads; ++y) {
                    c += is_block(id[y]);
                    if (id[y] >= a.num_blocks) errors |= PKV_DEVERR_BLOCK_ID;
                }
            }
            c = __reduce_add_sync(0xffffffffu, c);
            if (lane == 0) s.back[b] = c;
        });
        __syncthreads();
    }
    // sums, each thread over consecutive requests: rows, blocks that come back, blocks needed
    const int each = (n + kThreads - 1) / kThreads, b0 = min(tid * each, n), b1 = min(b0 + each, n);
    auto need_of = [&](int b) { return s.change[b] > 0 ? blocks(s.len[b] + s.change[b]) - blocks(s.len[b]) : 0; };
    int64_t at[3] = {0, 0, 0}, all[3];
    for (int b = b0; b < b1; ++b) {
        at[0] += s.rows[b];
        at[1] += s.back[b];
        at[2] += need_of(b);
    }
    scan(at, all, part);
    const int64_t all_rows = all[0];
    int64_t all_need = all[2];
    if (all_rows > a.num_rows) {                          // the requests whose rows do not fit get nothing
        errors |= PKV_DEVERR_LENGTH;
        int64_t rows = at[0], need[1] = {0}, sum[1];
        for (int b = b0; b < b1; ++b) {
            rows += s.rows[b];
            if (s.change[b] > 0 && rows > a.num_rows) s.change[b] = 0;
            need[0] += need_of(b);
        }
        scan(need, sum, part);
        at[2] = need[0];
        all_need = sum[0];
    }
    // More come back than the stack has room for: some block is in the tables or on the stack twice.  Which of them can not be
    // told here, so that no request drops any.
    const bool keep = count >= 0 && all[1] > a.num_blocks - count;
    if (keep) {
        errors |= PKV_DEVERR_BLOCK_ID;
        at[1] = 0;
    }
    const int64_t all_back = keep ? 0 : all[1];
    const int top = count < 0 ? 0 : (int)(count + all_back);
    int taken = 0;                                        // blocks needed by the requests that get theirs, up to here
    for (int b = b0; b < b1; ++b) {
        s.row[b] = (int)min(at[0], (int64_t)0x7fffffff);
        at[0] += s.rows[b];
        if (!keep) at[1] += s.back[b];
        else if (s.change[b] < 0) s.change[b] = 0;
        s.back[b] = (int)(all_back - at[1]);              // of later requests
        s.need[b] = (int)min(at[2], (int64_t)0x7fffffff);
        const int c = need_of(b);
        at[2] += c;
        if (c > 0 && at[2] > top) {                       // not enough are free
            errors |= PKV_DEVERR_NO_BLOCKS;
            s.change[b] = 0;
        } else if (c > 0) {
            taken = (int)at[2];
        }
    }
    if (all_need <= top) {
        taken = (int)all_need;
    } else {
        taken = __reduce_max_sync(0xffffffffu, taken);
        if (lane == 0) part[warp][0] = taken;
        __syncthreads();
        taken = __reduce_max_sync(0xffffffffu, (int)part[lane][0]);
    }
    __syncthreads();

    if (ctas > 1) cluster.sync();                         // every CTA has read the old state
    if (any_drop && !keep) {
        // last block first: a request's entries are taken from its end
        for (int b = rank * kThreads + tid; b < n; b += kThreads * ctas) {
            const int few = dropped(b);
            if (few == 0 || few > kFew) continue;
            int at = s.back[b];
            for (int j = blocks(s.len[b]) - 1, k = 0; k < few; --j, ++k) {
                int32_t* e = a.table + (int64_t)b * a.max_blocks + j;
                const int id = *e;
                if (is_block(id)) {
                    a.free_blocks[count + at] = id;
                    ++at;
                }
                *e = -1;
            }
        }
        warps(warp * ctas + rank, kThreads / 32 * ctas, [&](int b) {
            const int j0 = blocks(s.len[b] + s.change[b]);
            int at = s.back[b];
            for (int j = blocks(s.len[b]) - 1 - lane; __any_sync(0xffffffffu, j >= j0); j -= 32 * kLoads) {
                int32_t* e = a.table + (int64_t)b * a.max_blocks + j;
                int id[kLoads];
#pragma unroll
                for (int y = 0; y < kLoads; ++y) id[y] = j - 32 * y >= j0 ? e[-32 * y] : -1;
#pragma unroll
                for (int y = 0; y < kLoads; ++y) {
                    const bool give = is_block(id[y]);
                    const unsigned m = __ballot_sync(0xffffffffu, give);
                    const int place = at + __popc(m & ((1u << lane) - 1u));
                    if (give) a.free_blocks[count + place] = id[y];
                    if (j - 32 * y >= j0) e[-32 * y] = -1;
                    at += __popc(m);
                }
            }
        });
        __threadfence();
        if (ctas > 1) cluster.sync();                     // the stack is whole
        else __syncthreads();
    }
    const int64_t first = (int64_t)rank * kThreads + tid, stride = (int64_t)ctas * kThreads;
    auto block_of = [&](int b, int j) -> int {            // request b's block j, which is new
        const int id = __ldcg(a.free_blocks + top - 1 - (s.need[b] + j - blocks(s.len[b])));
        if (is_block(id)) return id;
        errors |= PKV_DEVERR_BLOCK_ID;
        return -1;
    };
    for (int64_t k = first; k < taken; k += stride) {
        // (requests without new blocks share their place with the next that has some: the last with it)
        const int b = find(s.need, n, (int)k);
        const int j = blocks(s.len[b]) + (int)k - s.need[b];
        if (s.change[b] > 0 && j < blocks(s.len[b] + s.change[b])) a.table[(int64_t)b * a.max_blocks + j] = block_of(b, j);
    }
    const int64_t shown = min(all_rows, a.num_rows);
#pragma unroll 4
    for (int64_t r = first; r < shown; r += stride) {
        const int b = find(s.row, n, (int)r);
        const int64_t at = (int64_t)s.len[b] + (r - s.row[b]);
        int64_t slot = -1;
        if (s.change[b] > 0) {
            const int j = (int)(at / kBlock), had = blocks(s.len[b]);
            int id = j < had ? a.table[(int64_t)b * a.max_blocks + j] : block_of(b, j);
            if (!is_block(id)) {
                errors |= PKV_DEVERR_BLOCK_ID;
                id = -1;
            }
            if (id >= 0) slot = (int64_t)id * kBlock + at % kBlock;
        }
        a.slots[r] = slot;
        if (a.positions) a.positions[r] = (int)at;
    }
    if (a.pad)
        for (int64_t r = shown + first; r < a.num_rows; r += stride) {
            a.slots[r] = -1;
            if (a.positions) a.positions[r] = 0;
        }
    for (int64_t b = first; b < n; b += stride) {
        if (s.change[b] != 0) a.lens[b] = s.len[b] + s.change[b];
        if (a.granted) a.granted[b] = max(s.change[b], 0);
        if (a.row_starts) a.row_starts[b] = s.row[b];
    }
    if (first == 0 && count >= 0) *a.free_count = top - taken;
    // The append and the attention behind this kernel read slots, lengths and tables before their dependency wait: they
    // start when every CTA here has ended (there is no early trigger), and what it wrote is in L2 by then.
    __threadfence();
    errors = (int)__reduce_or_sync(0xffffffffu, (unsigned)errors);
    if (errors && lane == 0) raise_error(a.err, errors);
}

}  // namespace tables

bool block_tables_fit(int num_seqs) { return num_seqs <= tables::kMaxSeqs; }

cudaError_t launch_block_tables(int32_t* table, int max_blocks, int32_t* lens, const int32_t* grow, int num_seqs,
                                int32_t* free_blocks, int32_t* free_count, int64_t num_blocks, int64_t* slots,
                                int32_t* positions, int32_t* granted, int64_t* row_starts, int64_t num_rows, bool pad,
                                int* err, cudaStream_t st) {
    using namespace tables;
    static std::atomic<uint64_t> set{0};
    const Arg a{table, lens, grow, free_blocks, free_count, slots, positions, granted, row_starts, err, num_blocks,
                num_rows, num_seqs, max_blocks, pad};
    const size_t bytes = (size_t)num_seqs * kArrays * sizeof(int), most = (size_t)kMaxSeqs * kArrays * sizeof(int);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (!bit || !(set.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(update_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    const unsigned ctas = num_rows > kManyRows ? kCluster : 1;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, update_kernel, a);
}

}  // namespace pkv
