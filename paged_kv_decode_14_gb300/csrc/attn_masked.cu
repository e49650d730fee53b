// Attention over the paged cache with a mask: a sliding window with first tokens that stay visible, or a tree of
// drafted tokens.  Contracts: include/pagedkv.h, pkv_paged_attention_window and pkv_paged_attention_tree.
//
// For query i of sequence b at position p = L - Q + i and query head h (kv-head h / G):
//   out = sum_j w_j v_j,  w = softmax over the visible j of scale * q . k_j,  lse = ln sum_j exp(scale * q . k_j)
//   window: j is visible iff j <= p and (j > p - window or j < sinks)
//   tree:   j is visible iff j < L - Q, or bit j - (L - Q) of row i of the mask is set
//
// A work item is some queries of one sequence times the heads of HG adjacent kv-heads (HG = 4, 2 or 1).  A row tile has 128
// rows, 128 / HG for each kv-head: PB = floor(128 / (HG G)) queries times its G heads.  The item's keys are a list of
// pages: those of the sinks that lie before the window, then those from the first query's window to the last query.  A
// key's place v in that list and its position differ by one jump behind the sinks, so what a row sees is at most two
// intervals of v, or one and the tree's bits, and pages that no row sees are never touched (their table entries may
// be anything).
//
// Per key tile (8 / HG pages of each kv-head, 128 columns: page after page, the heads of a page side by side, which is
// how they lie in the cache) and chain:
//   S[128 rows, 128 columns] = Q . K^T        (B: pages as they lie in the cache)
//   P = 2^(S scale log2(e) - m), l += sum P   (one thread per row = TMEM lane; P = 0 in other heads' columns)
//   O[128 rows, D] += P . V                   (A = P in TMEM, bf16; B MN-major: pages as they lie)
// With HG = 4 a decode step's few rows are spread over all four quarters of the lanes, and a row has 32 columns of a
// tile to work on instead of 128.
// There are two chains, each with its own S, O, m and l in tensor memory and four softmax warps.  With HG = 1 an item may
// have two row tiles, one a chain, and every key tile serves both.  Otherwise the chains take the key tiles in turns:
// while one's softmax runs the other's products do; their O, m and l are joined at the end of the piece.  m is set by the
// maximum of a row's first visible keys; P is computed against it without a maximum, and only where the P of 64 keys add
// up to 2^14 (bf16 has fp32's range) m rises.
//
// P is rounded to bf16 (8 significant bits; l is summed from the fp32 P): the error it leaves in out is of the size
// of out's own rounding to bf16, so that out's error (relative to its norm) is 0.0023 where P in fp32 gives 0.0017.  P in two
// bf16 parts, as pkv_paged_attention has it, gives 0.0017 too, but takes the decode step below from 30.0 to 31.6 us, the FP8
// streams from 223 to 248, the trees from 63 to 69 (FP8 193 to 238), prompts from 115 to 130 and FP8 chunks from 180 to 216:
// not taken.  fp16 would hold 11 bits, but not V's range.
// FP8 caches: S on e4m3 MMAs, the K pages as they are; a row of q is scaled by a power of two to a maximum in [128,
// 256) and split into two e4m3 terms (exact but for elements below 2^-10 of the row's largest, which are good to 2^-17 of
// it).  V is widened to bf16 in shared memory (exact).  A page's k scale multiplies its S and its v scale its P, in fp32.
//
// Work is cut into equal ranges of key tiles over all items, one range per CTA; an item that a range's end cuts leaves
// partial (O, m, l) in the workspace, and whichever CTA finishes its part last joins them, in the keys' order.
//
// Roles (512 threads): warps 0-3 and 4-7 the softmax of chains 0 and 1, and the results; warps 8-11 make V
// ready; warp 12 the producer; warps 13 and 14 the MMA issuers of the chains; warp 15 the plan.  Every wait is bounded.
//
// Measured (32/8 heads of 128, inputs past L2, back to back in a graph; copies run at 6786 GB/s, bf16 products at 1965
// TFLOP/s): a decode step of 32 sequences, window 1024: 30 us for 133 MB (0.65 of the copy rate); 2048 sequences of 300
// keys: 392 us (0.86).  128 FP8 streams, window 4096: 224 us (0.68).  Trees of 9 to 24 nodes over 32 contexts of 512 to
// 4072: 65 us (0.74); of 64 nodes over 16 FP8 contexts of 8k to 16k: 194 us (0.58 of the product rate).  Four 2k prompts,
// window 512: 116 us, FP8 chunks, window 2048: 177 us (0.27 and 0.35 of the product rate, by the visible pairs; the tiles at
// a window's two ends are computed whole).
// What bounds it: with few rows the copies and, FP8, the widening (1600 of a tile's 2050 clocks); with many the chain S ->
// P -> P . V of a row tile, 3600 clocks for a key tile of both chains, of which 2560 are reads and writes of shared memory (128
// bytes a clock; Q is read once for each half of S), and 9000 at a change of item.  Beside both, five roles' code shares an
// instruction cache (4 to 12 % of its requests miss), and times depend on how the code comes out: whatever was unrolled or
// doubled (a masked copy of the softmax, 64 columns an epilogue step) made it slower, and loops outside the inner ones are
// kept rolled.
#include <cuda.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "rows.cuh"
#include "tc_rows.cuh"

namespace pkv {
int num_sms_current();

namespace masked {

using namespace tcrow;
using rows::View;

constexpr int kRows = 128;                 // rows of a row tile (MMA M)
constexpr int kUnits = 8;                  // pages of one kv-head in a key tile
constexpr int kCols = kUnits * kBlock;     // columns of a key tile
constexpr int kThreads = 512;
// Registers a thread: the launch gives every thread 128, and the roles' shares add up to as many.
constexpr int kRegsSoftmax = 160, kRegsReady = 112, kRegsOther = 80;
static_assert(2 * kRegsSoftmax + kRegsReady + kRegsOther == 4 * 128, "register file");
constexpr int kReady = 8, kProducer = 12, kMma = 13, kPlan = 15;
constexpr int kPieces = 4;                 // pieces of work planned ahead
constexpr int kMaxCtas = 160;              // CTAs of a launch (two workspace slots each)
// what an item costs beside its key tiles, in units (key tiles of one row tile): four 2k prompts take 117 us with 4, 149 with
// 2 and 119 with 8
constexpr int kItemUnits = 4;
// What a piece's wait limit grows by for each of its key tiles, in ns: they take 1 to 2 us, and with values that are not finite
// alone some 50.
constexpr uint64_t kTileLimit = 100000;
constexpr uint32_t kWaitHint = 20000;     // ns that a wait may sleep before it looks at the abort flag
constexpr int kAhead = 3;                  // tiles that an FP8 page's scales are fetched ahead
// What cutting an item costs, in units.  Where there is a CTA for every item and none is longer than its share by more than
// this, each is dealt whole: 32 requests of 256 keys, two kv-heads an item, 14.8 us against 24.0 with their items cut.
constexpr int kCutUnits = 8;
constexpr int kMinUnits = 4;               // units that a CTA has at least
constexpr int kFp8Tiles = 16;              // key tiles a CTA (of one kv-head) that count as much FP8 work
constexpr int kMaxLen = 0x7ffffe00;        // of a context: places of its last tile stay below 2^31

struct Arg {
    CUtensorMap q;
    const uint8_t *k_cache, *v_cache;
    const float *k_scales, *v_scales;
    const int32_t *tables, *ctx_lens, *q_lens;
    const int64_t* q_starts;
    const uint32_t* tree;                  // nullptr: a window
    View out;
    float* lse;
    int* err;
    int* tickets;                          // [CTA][8]
    float* partials;                       // [CTA][2] slots
    uint64_t wait_limit_ns;
    const int* hold;
    int64_t num_blocks, num_q_rows;
    int max_blocks, num_seqs, max_q_len, Hq, Hkv, group;
    int pb;                                // queries of a row tile
    int tree_words, window, sinks;
    float scale_log2;
};

// A partial slot: O as [D / 4][256 rows][4] fp32, then m and l, [256] each.
__host__ __device__ constexpr int slot_floats(int D) { return 2 * kRows * (D + 2); }

// A piece of work: key tiles [t0, t1) of queries q0 .. q0 + nq - 1 of a sequence, kv-heads from g on.
struct Piece {
    int64_t row;            // q's row of query 0
    int b, g, q0, nq, t0, t1;
    int first;              // position of query q0
    int L, Q;
    int sp, np, jump;       // the list: sp first pages, then (from position sp * 16 + jump on) the others, np in all
    int c0, parts;          // the CTAs that hold parts of the item: c0 .. c0 + parts - 1
    int two;                // two row tiles
    int end;                // no more work (the other fields are unset)
    unsigned bad;           // bit i: tiles [i << shift, (i + 1) << shift) hold values that the guard of V took out
    // the shift: as many marks as there are tiles, up to 32
    __device__ __forceinline__ int mark_shift() const { return max(0, 27 - __clz(max(tiles() - 1, 1))); }
    __device__ __forceinline__ int tiles() const { return t1 - t0; }
    // tiles of chain i, the first of them, and the step from one to the next
    __device__ __forceinline__ int count(int i) const { return two ? t1 - t0 : (t1 - t0 + 1 - i) >> 1; }
    __device__ __forceinline__ int begin(int i) const { return two ? 0 : i; }
    __device__ __forceinline__ int step() const { return two ? 1 : 2; }
    __device__ __forceinline__ int page(int idx) const { return idx < sp ? idx : idx + jump / kBlock; }
    // one past the last v that any query of [a, z) of the piece's queries sees
    __device__ __forceinline__ int seen_end(const Arg& p, int z) const { return p.tree ? L : first + z - jump; }
};
static_assert(sizeof(Piece) % 8 == 0, "aligned ring entries");

// What one query sees, in places of the list: [0, ns), [wl, wh], and (tree) bits from place `base` on.
struct Sight {
    int ns, wl, wh;
    __device__ __forceinline__ void window(const Arg& a, const Piece& p, int pos) {
        ns = min(a.sinks, pos + 1);
        wl = max(0, pos - a.window + 1) - p.jump;
        wh = pos - p.jump;
    }
    __device__ __forceinline__ void tree(const Piece& p) {
        ns = wl = 0;
        wh = p.L - p.Q - 1;
    }
    __device__ __forceinline__ bool has(int v) const { return v < ns || (v >= wl && v <= wh); }
};

// Bits j .. j + 31 of a row of `words` mask words (j from -31 up); bits at and past n are clear.
__device__ __forceinline__ uint32_t tree_bits(const uint32_t* row, int words, int j, int n) {
    const int w = j >> 5, s = j & 31;
    const uint32_t lo = w >= 0 && w < words ? row[w] : 0u, hi = w + 1 >= 0 && w + 1 < words ? row[w + 1] : 0u;
    const uint32_t x = __funnelshift_r(lo, hi, s);
    return n - j >= 32 ? x : n - j <= 0 ? 0u : x & ((1u << (n - j)) - 1u);
}

// What all rows of an item see, and what any does.
template <int HG>
struct Guard {
    int ns_all, wl_all, wh_all, ns_any, wl_any, wh_any;
    __device__ __forceinline__ bool any(int v) const { return v < ns_any || (v >= wl_any && v <= wh_any); }
    __device__ __forceinline__ bool all(int v) const { return HG == 1 && (v < ns_all || (v >= wl_all && v <= wh_all)); }
    // all of v .. v + n - 1 are seen by some row (whole: by every row of the tile)
    __device__ __forceinline__ bool any_of(int v, int n) const {
        return v + n <= ns_any || (v >= wl_any && v + n - 1 <= wh_any);
    }
    __device__ __forceinline__ bool all_of(int v, int n) const {
        return HG == 1 && (v + n <= ns_all || (v >= wl_all && v + n - 1 <= wh_all));
    }
};

template <int HG>
__device__ __forceinline__ Guard<HG> guard_of(const Arg& a, const Piece& p) {
    if (a.tree) return Guard<HG>{0, 0, p.L - p.Q - 1, 0, 0, p.L - 1};
    Sight f, l;
    f.window(a, p, p.first);
    l.window(a, p, p.first + p.nq - 1);
    return Guard<HG>{f.ns, l.wl, f.wh, l.ns, f.wl, l.wh};
}

template <int D, bool FP8, int HG>
struct Cfg {
    static constexpr int TP = kUnits / HG;                // pages of a tile (of each head)
    static constexpr int KEYS = TP * kBlock;              // keys of a tile
    static constexpr int RQ = kRows / HG;                 // rows of a row tile that a head has
    // A tile's products and softmax go by halves of its columns where a row works on all of them (trees of 64 nodes 248 -> 230
    // us, prompts 125 -> 119: products of one half run under the softmax of the other); else whole.
    static constexpr int HALVES = HG == 1 ? 2 : 1, HCOLS = kCols / HALVES;
    static constexpr int SLAB = kRows * 128;              // Q: bytes of a 64-dimension slab
    static constexpr int SLABS = D / 64;
    static constexpr int QTILE = SLABS * SLAB;
    static constexpr int NCH = D / 8;                     // 16-byte chunks of a bf16 row
    static constexpr int PAGE = kBlock * D * 2;           // a page as bf16 operand
    static constexpr int LAND = FP8 ? PAGE / 2 : PAGE;    // a page of the cache
    static constexpr int KTILE = kUnits * LAND;
    static constexpr int VTILE = kUnits * PAGE;           // (FP8: a page lands in the upper half of its place)
    static constexpr int NSK = FP8 ? (D == 128 ? 3 : 6) : (D == 128 ? 2 : 5);     // K ring depth
    static constexpr int NSV = D == 128 ? 3 : FP8 ? 6 : 5;                        // V ring depth
    static constexpr int NSC = D == 128 ? 8 : 16;         // scale ring: a tile's are read until its V slot is free
    static_assert(NSC > NSV + kAhead, "scale ring");
    static constexpr int NQS = 4;                         // ring of the rows' powers of two (FP8)
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + 2 * QTILE;
    static constexpr int OFF_V = OFF_K + NSK * KTILE;
    static constexpr int OFF_BAR = OFF_V + NSV * VTILE;
    static constexpr int KFULL = 0, KEMPTY = NSK, VFULL = 2 * NSK, VREADY = VFULL + NSV, VEMPTY = VREADY + NSV,
                         SFULL = VEMPTY + NSV, PFULL = SFULL + 4, PVDONE = SFULL + 8, QFULL = SFULL + 12, QREADY = SFULL + 14,
                         QEMPTY = SFULL + 16, ODONE = SFULL + 18, OFREE = SFULL + 20, LREADY = SFULL + 21,
                         PCFULL = SFULL + 22, PCEMPTY = PCFULL + kPieces,
                         Q1FULL = PCEMPTY + kPieces, DRAIN = Q1FULL + 1;
    static constexpr int NBAR = DRAIN + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;   // tmem address, abort flags
    static constexpr int OFF_ML = OFF_MISC + 16;          // float[chain][m, l][kRows]
    static constexpr int OFF_PIECE = OFF_ML + 4 * 4 * kRows;
    static constexpr int OFF_SC = OFF_PIECE + kPieces * (int)sizeof(Piece);       // FP8: float[NSC][k scales 8, v scales 8]
    static constexpr int OFF_QS = OFF_SC + (FP8 ? NSC * 64 : 0);                  // FP8: float[NQS][kRows]
    static constexpr int SMEM = OFF_QS + (FP8 ? NQS * 4 * kRows : 0);
    static constexpr int COL_O = 2 * kCols;
    static constexpr int TMEM_COLS = 512;
    static_assert(OFF_PIECE % 8 == 0, "alignment");
    static_assert(COL_O + 2 * D <= TMEM_COLS, "tensor memory budget");
    static_assert(SMEM <= 232448, "shared memory budget");
};

// ------------------------------------------------------------------ plan

struct Seq {
    int64_t row;
    int Q, L;               // 0 queries where the lengths are bad
};

// The plan of a launch, made by one warp of every CTA alike.  An item's units are its key tiles times its row tiles
// and kItemUnits; all items' units, in the order sequence, query block, kv-heads, are cut into equal ranges, one per
// CTA, and a CTA has the tiles whose first unit lies in its range.  (Loops are kept rolled: this code runs once, from a
// cold instruction cache.)
template <int HG>
struct Plan {
    static constexpr int TP = kUnits / HG;
    const Arg& a;
    const int lane;
    int groups;             // of HG kv-heads
    int total, u, u1;       // all units; the CTA's place and end
    int share, longer;      // units of a CTA, and how many CTAs have one more
    bool flat;              // a CTA has one item or none: an item counts one unit
    int b, blk, g;          // the item at u, its first unit
    int start;
    Seq s;
    int64_t packed;         // rows before sequence b

    __device__ __forceinline__ Plan(const Arg& a_, int lane_) : a(a_), lane(lane_), groups(a_.Hkv / HG) {}
    __device__ __forceinline__ int per() const { return HG == 1 ? 2 * a.pb : a.pb; }
    __device__ __forceinline__ Seq load(int i, int64_t rows, bool report) const {
        Seq x{a.q_starts ? a.q_starts[i] : rows, a.q_lens[i], a.ctx_lens[i]};
        if (x.Q < 0 || x.Q > a.max_q_len || x.L < x.Q || x.L > kMaxLen || x.row < 0 || x.row > a.num_q_rows - x.Q ||
            (x.Q > 0 && (x.L - 1) / kBlock >= a.max_blocks)) {
            if (report && (x.Q != 0 || x.L < 0)) raise_error(a.err, PKV_DEVERR_LENGTH);
            x.Q = 0;
        }
        return x;
    }
    // the geometry of query block `block` of a sequence; its key tiles, and the units of one
    __device__ __forceinline__ int span(const Seq& x, int block, Piece& p, int& tiles, int& each) const {
        p.q0 = block * per();
        p.nq = min(per(), x.Q - p.q0);
        p.first = x.L - x.Q + p.q0;
        p.sp = p.jump = 0;
        p.np = (x.L + kBlock - 1) / kBlock;
        if (!a.tree) {
            const int wp = max(0, p.first - a.window + 1) / kBlock;
            p.sp = min((min(a.sinks, x.L) + kBlock - 1) / kBlock, wp);
            p.jump = (wp - p.sp) * kBlock;
            p.np = (p.first + p.nq - 1) / kBlock + 1 - (wp - p.sp);
        }
        tiles = (p.np + TP - 1) / TP;
        each = HG == 1 && p.nq > a.pb ? 2 : 1;
        return flat ? 1 : tiles * each + kItemUnits;
    }
    template <typename V>
    __device__ __forceinline__ V scan(V x) const {        // the sum over earlier lanes
        V y = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const V z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        return y - x;
    }
    __device__ __forceinline__ int range(int c) const { return share * c + min(c, longer); }
    __device__ __forceinline__ int cta_of(int unit) const {
        const int head = (share + 1) * longer;
        const bool in = unit < head;
        return (in ? 0 : longer) + (int)((uint32_t)(in ? unit : unit - head) / (uint32_t)(in ? share + 1 : share));
    }
    __device__ __forceinline__ void begin() {
        // a lane stands for some sequences, or where there are few, `each_seq` lanes for one, with equal shares of its blocks
        const int chunk = (a.num_seqs + 31) / 32;
        const int lg = a.num_seqs > 16 ? 0 : 5 - (32 - __clz(a.num_seqs - 1)), each_seq = 1 << lg, seg = lane & (each_seq - 1);
        const int b0 = min((lane >> lg) * chunk, a.num_seqs), b1 = min(b0 + chunk, a.num_seqs);
        int64_t rows = 0;
        if (!a.q_starts) {
#pragma unroll 1
            for (int i = b0; i < b1; ++i) rows += max(a.q_lens[i], 0);
            rows = scan(seg == 0 ? rows : (int64_t)0);
            rows = __shfl_sync(0xffffffffu, rows, lane - seg);
        }
        // units of this lane's sequences; the second time, the item of them that holds unit `u`
        int64_t mine = 0, before = 0;
        int fb = 0, fblk = 0, fg = 0, fs = 0, most = 0;
        int64_t fp = 0, items = 0;
        total = u = u1 = 0;
        flat = false;
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {
            const bool here = turn == 1 && u >= before && u < before + mine;
            if (turn == 0 || here) {
                int64_t at = rows, r = before;
                bool found = false;
#pragma unroll 1
                for (int i = b0; i < b1 && !found; ++i) {
                    const Seq x = load(i, at, turn == 0);
                    const int n = (x.Q + per() - 1) / per(), some = (n + each_seq - 1) >> lg;
#pragma unroll 1
                    for (int k = seg * some; k < min((seg + 1) * some, n) && !found; ++k) {
                        Piece p;
                        int tiles, each;
                        const int w = span(x, k, p, tiles, each);
                        const int64_t all = (int64_t)w * groups;
                        most = max(most, w);
                        items += groups;
                        if (turn == 1 && u < r + all) {
                            fb = i;
                            fblk = k;
                            fg = (int)((uint32_t)(u - (int)r) / (uint32_t)w);
                            fs = (int)r + fg * w;
                            fp = at;
                            found = true;
                        }
                        r += all;
                    }
                    at += max(a.q_lens[i], 0);
                }
                if (turn == 0) mine = r;
            }
            if (turn == 0) {
                before = scan(mine);
                const int64_t sum = __shfl_sync(0xffffffffu, before + mine, 31);
                if (sum > 0x7ffffff0) {                   // (some 15 s of a GPU's work; units are counted in 32 bits)
                    raise_error(a.err, PKV_DEVERR_LENGTH);
                    return;
                }
                total = (int)sum;
                int ctas = max(1, min((int)gridDim.x, total / kMinUnits));
                const int n = (int)__reduce_add_sync(0xffffffffu, (unsigned)min(items, (int64_t)1 << 16));
                most = __reduce_max_sync(0xffffffffu, most);
                flat = n <= (int)gridDim.x && most <= total / ctas + kCutUnits;
                if (flat) {
                    mine = items;
                    before = scan(mine);
                    total = ctas = n;
                }
                if ((int)blockIdx.x >= ctas || total == 0) return;
                share = (int)((uint32_t)total / (uint32_t)ctas);
                longer = total - share * ctas;
                u = range(blockIdx.x);
                u1 = range(blockIdx.x + 1);
            } else {
                const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
                b = __shfl_sync(0xffffffffu, fb, from);
                blk = __shfl_sync(0xffffffffu, fblk, from);
                g = __shfl_sync(0xffffffffu, fg, from);
                start = __shfl_sync(0xffffffffu, fs, from);
                packed = __shfl_sync(0xffffffffu, fp, from);
            }
        }
        s = load(b, packed, false);
    }
    // The next piece with tiles; the same in every lane.
    __device__ __forceinline__ bool next(Piece& p) {
        bool some = false;
#pragma unroll 1
        while (u < u1 && !some) {
            int tiles, each;
            const int w = span(s, blk, p, tiles, each);
            const int keys = start + kItemUnits;          // the first tile's first unit
            auto tile_at = [&](int x) { return flat ? (x > start ? tiles : 0) : x <= keys ? 0 : min(tiles, (x - keys + each - 1) >> (each - 1)); };
            p.t0 = tile_at(u);
            p.t1 = tile_at(u1);
            some = p.t1 > p.t0;
            p.row = s.row;
            p.b = b;
            p.g = g * HG;
            p.L = s.L;
            p.Q = s.Q;
            p.two = each == 2;
            p.end = 0;
            p.c0 = blockIdx.x;
            p.parts = 1;
            if (some && !flat && (p.t0 > 0 || p.t1 < tiles)) {
                if (p.t0 > 0) p.c0 = cta_of(keys);
                p.parts = (p.t1 < tiles ? cta_of(keys + (tiles - 1) * each) : (int)blockIdx.x) - p.c0 + 1;
            }
            // on to the next item
            start += w;
            u = start;
            if (++g == groups) {
                g = 0;
                if (++blk * per() >= s.Q) {
                    blk = 0;
#pragma unroll 1
                    do {
                        packed += max(a.q_lens[b], 0);
                        if (++b >= a.num_seqs) {
                            u = u1;
                            break;
                        }
                        s = load(b, packed, false);
                    } while (s.Q == 0);
                }
            }
        }
        return some;
    }
};

// ------------------------------------------------------------------ numbers

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
constexpr float kHigh = 0x1p14f;           // sum of 64 P at which m rises
// |m| from which its roundings (half of fp32's step at m each, up to three of them) may leave P, l or O their range:
// 2^29, three times 16 octaves above kHigh or below 1
constexpr float kLimit = 0x1p29f;

// Four e4m3 codes as bf16, exactly: the code's exponent and mantissa moved to bf16's places mean the value times
// 2^-120 (subnormals too).  NaN codes become 480 here: the caller looks for them.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t a = __byte_perm(w, 0, 0x1404), b = __byte_perm(w, 0, 0x3424);
    const uint32_t x = (a & 0x80008000u) | ((a >> 4) & 0x07f007f0u), y = (b & 0x80008000u) | ((b >> 4) & 0x07f007f0u);
    const uint32_t f = 0x7b807b80u;        // 2^120
    asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(lo) : "r"(x), "r"(f));
    asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(hi) : "r"(y), "r"(f));
}
// A bit set where one of two bf16 is infinite or NaN: an exponent of all ones carries.
__device__ __forceinline__ uint32_t inf_words(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// Two bf16 (of a word) times f as e4m3 codes, and what they leave as e4m3 codes.
__device__ __forceinline__ void split2(uint32_t w, float f, uint32_t& hi, uint32_t& lo) {
    const float2 x = make_float2(bf16_lo(w) * f, bf16_hi(w) * f);
    hi = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
    const float2 y = e4m3x2_to_float2(hi);
    lo = __nv_cvt_float2_to_fp8x2(make_float2(x.x - y.x, x.y - y.y), __NV_SATFINITE, __NV_E4M3);
}

// ------------------------------------------------------------------ kernel

template <int D>
__device__ __forceinline__ float* part_slot(const Arg& a, int cta, bool starts) {
    return a.partials + ((size_t)cta * 2 + (starts ? 1 : 0)) * slot_floats(D);
}

template <int D, bool FP8, int HG>
__global__ void __launch_bounds__(kThreads, 1) masked_kernel(const __grid_constant__ Arg a) {
    using K = Cfg<D, FP8, HG>;
    extern __shared__ __align__(1024) uint8_t smem[];     // (the swizzle needs it; checked below)
    const uint32_t sb = smem_u32(smem);
    // (the warp's number by a shuffle: known to be uniform, and with it the roles' control flow)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    auto bar = [&](int i) -> uint32_t { return sb + K::OFF_BAR + 8 * i; };
    constexpr int NSK = K::NSK, NSV = K::NSV, RQ = K::RQ;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + K::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + K::OFF_MISC + 4);
    volatile int* drain_flag = reinterpret_cast<volatile int*>(smem + K::OFF_MISC + 8);   // (drain waits at the end)
    float* ml = reinterpret_cast<float*>(smem + K::OFF_ML);
    float* scales = reinterpret_cast<float*>(smem + K::OFF_SC);
    float* q_scale = reinterpret_cast<float*>(smem + K::OFF_QS);
    Piece* ring = reinterpret_cast<Piece*>(smem + K::OFF_PIECE);
    // every wait and every TMEM access is warp-uniform (tcgen05.ld / st are .aligned)
    // (Their limit is kept by the plan's warp, which waits for every piece's end: where one takes that long it sets the abort
    // flag.  A clock in each of the sixty waits made the code a fifth longer.)
    auto wait_all = [&](uint32_t bb, uint32_t parity) {
        bool there = mbar_try_wait(bb, parity);
        while (!there && !*abort_flag) there = mbar_try_wait_hint(bb, parity, kWaitHint);
        return (bool)__all_sync(0xffffffffu, there);
    };

    if (tid == 0) {
        for (int i = 0; i < NSK; ++i) {
            mbar_init(bar(K::KFULL + i), 1);
            mbar_init(bar(K::KEMPTY + i), 2);             // one of each chain
        }
        for (int i = 0; i < NSV; ++i) {
            mbar_init(bar(K::VFULL + i), 1);
            mbar_init(bar(K::VREADY + i), 4);             // one arrival a warp that makes it ready
            mbar_init(bar(K::VEMPTY + i), 2);
        }
        for (int i = 0; i < 2; ++i) {
            for (int h = 0; h < 2; ++h) {                 // by chain and half of a tile's columns
                mbar_init(bar(K::SFULL + 2 * i + h), 1);
                mbar_init(bar(K::PFULL + 2 * i + h), 4);  // one arrival a softmax warp
                mbar_init(bar(K::PVDONE + 2 * i + h), 1);
            }
            mbar_init(bar(K::QFULL + i), 1);
            mbar_init(bar(K::QREADY + i), 4);
            mbar_init(bar(K::QEMPTY + i), 2);
            mbar_init(bar(K::ODONE + i), 1);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(bar(K::PCFULL + i), 1);
            mbar_init(bar(K::PCEMPTY + i), 15);           // every warp but the plan's, which writes them
        }
        mbar_init(bar(K::OFREE), 8);                      // every softmax warp, after a piece of both chains
        mbar_init(bar(K::LREADY), 8);
        mbar_init(bar(K::Q1FULL), 1);
        mbar_init(bar(K::DRAIN), 2);
        *abort_flag = 0;
        *drain_flag = 0;
        mbar_fence_init();
    }
    if (warp == kProducer && lane == 0) asm volatile("prefetch.tensormap [%0];\n" ::"l"(&a.q) : "memory");
    if (warp == kMma) {
        tmem_alloc(smem_u32(tmem_slot), K::TMEM_COLS);
        tmem_relinquish();
    }
    if ((sb & 1023) != 0 && tid == 0) {
        raise_error(a.err, PKV_DEVERR_TIMEOUT);           // (never: the declaration above aligns it)
        *abort_flag = 1;
    }
    // every role goes through here, from its own code path (non-.aligned barrier); the tensor memory's address
    auto enter = [&]() -> uint32_t {
        griddep_wait();                                   // (no early trigger: pkv_paged_attention reads its q before its own wait)
        tc_fence_before();
        cta_bar_sync();
        tc_fence_after();
        return *tmem_slot;
    };

    // The pieces of work: the n-th (nullptr: a wait gave up), until its release by every warp.
    auto piece_at = [&](int n) -> const Piece* {
        return wait_all(bar(K::PCFULL + n % kPieces), (n / kPieces) & 1) ? ring + n % kPieces : nullptr;
    };
    auto release = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(K::PCEMPTY + n % kPieces));
    };

    // (The softmax's code comes last: it is the longest, with all that runs rarely in it.  With it before the other roles',
    // FP8 chunks took 180 us, not 176, and 128 FP8 streams 225.5, not 224.)
    if (warp >= kProducer) {
        regs_dec<kRegsOther>();
        if (warp == kPlan) {
            // -------------------------------------------- the plan (begun while the others set up)
            griddep_wait();
            Plan<HG> plan(a, lane);
            plan.begin();
            Piece p = {};
            p.end = !plan.next(p);
            enter();
            // every warp is done with piece x: the only wait that keeps the time
            auto done = [&](int x) -> bool {
                const Ctl clock{abort_flag, a.err, a.wait_limit_ns + ring[x % kPieces].tiles() * kTileLimit};
                return __all_sync(0xffffffffu, wait(bar(K::PCEMPTY + x % kPieces), (x / kPieces) & 1, clock));
            };
            for (int n = 0;; ++n) {
                if (n >= kPieces && !done(n - kPieces)) break;
                if (lane == 0) {
                    ring[n % kPieces] = p;
                    mbar_arrive(bar(K::PCFULL + n % kPieces));
                }
                __syncwarp();
                if (p.end) {
                    for (int x = max(n - kPieces, 0); x < n && done(x); ++x) {}
                    break;
                }
                p.end = !plan.next(p);
            }
        } else if (warp == kProducer) {
            enter();
            // -------------------------------------------- Q tiles, K and V pages in order
            bool ok = true;
            int nt = 0, nq = 0, nq1 = 0, npc = 0;         // key tiles; Q tiles, those of chain 1; pieces
            int nk = 0, nv = 0;                           // copies issued: K and V tiles
            if (a.hold != nullptr && lane == 0) {
                // (tests of the timeout path only) wait, bounded, for a flag that nothing sets
                const uint64_t h0 = globaltimer_ns();
                while (ok && *reinterpret_cast<const volatile int*>(a.hold) == 0) {
                    if (*abort_flag || globaltimer_ns() - h0 > a.wait_limit_ns) {
                        if (!*abort_flag) raise_error(a.err, PKV_DEVERR_TIMEOUT);
                        *abort_flag = 1;
                        ok = false;
                    }
                    __nanosleep(256);
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            // lanes 0-7 stand for a tile's units of K, 8-15 for those of V
            // (pages leave L2 first: with them in its way the kernel's own code came from DRAM, 41 us for a decode step against 38)
            const uint64_t evict = policy_evict_first();
            const int u8 = lane & 7, upg = u8 / HG, uh = u8 % HG;
            const bool is_v = lane >= 8;
            for (int n = 0; ok; ++n) {
                const Piece* p = piece_at(n);
                if (!p || p->end) break;
                const int32_t* table = a.tables + (int64_t)p->b * a.max_blocks;
                const int np = p->np, g = p->g + uh;
                // 32 entries of the list at a time, a lane each (a bad id is reported, and block 0 read in its place)
                auto blocks = [&](int first) -> int {
                    const int idx = first + lane;
                    const int id = idx < min(np, p->t1 * K::TP) ? table[p->page(idx)] : 0;
                    if (id >= 0 && id < a.num_blocks) return id;
                    raise_error(a.err, PKV_DEVERR_BLOCK_ID);
                    return 0;
                };
                const int first = p->t0 * K::TP;
                int held = first, ids = blocks(first), ids1 = blocks(first + 32);       // entries from `held` on, and the next 32
                // the block of this lane's unit of tile t, which lies among them
                auto block = [&](int t) -> int {
                    const int at = t * K::TP + upg - held;
                    int id = __shfl_sync(0xffffffffu, ids, at & 31);
                    if (__any_sync(0xffffffffu, at >= 32)) {
                        const int x = __shfl_sync(0xffffffffu, ids1, at & 31);
                        id = at < 32 ? id : x;
                    }
                    return id;
                };
                // (FP8) scales on their way into the ring, kAhead tiles before they are needed
                auto fetch = [&](int t, int slot) {
                    if (!FP8) return;
                    const int id = block(t);
                    if (lane < 16 && t < p->t1 && t * K::TP + upg < np)
                        cp_async_4(sb + K::OFF_SC + ((slot % K::NSC) * 16 + lane) * 4,
                                   (is_v ? a.v_scales : a.k_scales) + (int64_t)id * a.Hkv + g);
                    asm volatile("cp.async.commit_group;\n" ::: "memory");
                };
                for (int i = 0; i < (p->two ? 2 : 1) && ok; ++i, ++nq) {
                    const int slot = nq & 1;
                    if (nq >= 2 && !(ok = wait_all(bar(K::QEMPTY + slot), ((nq - 2) >> 1) & 1))) break;
                    // (bf16: a barrier each slot, for the issuers, who see every tile.  FP8: those of chain 0's, by turns, and one of
                    // chain 1's, for the warps that split them, who see no others: no barrier's phases run ahead unseen)
                    const uint32_t full = bar(!FP8 ? K::QFULL + slot : i == 0 ? K::QFULL + (n & 1) : K::Q1FULL);
                    if (lane == 0) mbar_arrive_expect_tx(full, HG * K::SLABS * a.pb * a.group * 128);
                    nq1 += i;
                    npc += i == 0;
                    __syncwarp();
                    if (lane < HG * K::SLABS) {           // (a lane for each head's slab)
                        const int sl = lane % K::SLABS, hq = lane / K::SLABS;
                        tensor_g2s(sb + K::OFF_Q + slot * K::QTILE + sl * K::SLAB + hq * RQ * 128, &a.q, sl * 64,
                                   (p->g + hq) * a.group, (int)(p->row + p->q0 + i * a.pb), full);
                    }
                }
#pragma unroll 1
                for (int x = 0; x < kAhead; ++x) fetch(p->t0 + x, nt + x);
#pragma unroll 1
                for (int t = p->t0; t < p->t1 && ok; ++t, ++nt) {
                    const int sk = nt % NSK, sv = nt % NSV, pages = min(K::TP, np - t * K::TP);
                    if (t * K::TP - held >= 32) {
                        held += 32;
                        ids = ids1;
                        ids1 = blocks(held + 32);
                    }
                    const int64_t src = ((int64_t)block(t) * a.Hkv + g) * K::LAND;
                    if (nt >= NSK && !(ok = wait_all(bar(K::KEMPTY + sk), ((nt - NSK) / NSK) & 1))) break;
                    fetch(t + kAhead, nt + kAhead);
                    if (FP8) asm volatile("cp.async.wait_group %0;\n" ::"n"(kAhead) : "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(bar(K::KFULL + sk), pages * HG * K::LAND);
                    __syncwarp();
                    // (a page's HG heads lie side by side)
                    if (!is_v && uh == 0 && upg < pages)
                        bulk_g2s_hint(sb + K::OFF_K + sk * K::KTILE + u8 * K::LAND, a.k_cache + src, HG * K::LAND, bar(K::KFULL + sk),
                                      evict);
                    ++nk;
                    if (nt >= NSV && !(ok = wait_all(bar(K::VEMPTY + sv), ((nt - NSV) / NSV) & 1))) break;
                    if (lane == 0) mbar_arrive_expect_tx(bar(K::VFULL + sv), pages * HG * K::LAND);
                    __syncwarp();
                    if (is_v && lane < 16 && upg < pages) {
                        if (FP8)
                            bulk_g2s_hint(sb + K::OFF_V + sv * K::VTILE + u8 * K::PAGE + K::LAND, a.v_cache + src, K::LAND,
                                          bar(K::VFULL + sv), evict);
                        else if (uh == 0)
                            bulk_g2s_hint(sb + K::OFF_V + sv * K::VTILE + u8 * K::PAGE, a.v_cache + src, HG * K::PAGE,
                                          bar(K::VFULL + sv), evict);
                    }
                    ++nv;
                }
                // (what a piece fetched past its end is not read: its slots are the next piece's, fetched again)
                if (FP8) cp_async_wait_all();
                release(n);
            }
            if (lane == 0) {
                // drain: every copy in flight lands before the CTA exits
                const Ctl drain{drain_flag, a.err, a.wait_limit_ns};
                for (int t = max(0, nk - NSK); t < nk; ++t) wait(bar(K::KFULL + t % NSK), (t / NSK) & 1, drain);
                for (int t = max(0, nv - NSV); t < nv; ++t) wait(bar(K::VFULL + t % NSV), (t / NSV) & 1, drain);
                for (int t = max(0, (FP8 ? npc : nq) - 2); t < (FP8 ? npc : nq); ++t)
                    wait(bar(K::QFULL + (t & 1)), (t >> 1) & 1, drain);
                if (FP8 && nq1 > 0) wait(bar(K::Q1FULL), (nq1 - 1) & 1, drain);
            }
            __syncwarp();
        } else if (warp == kMma || warp == kMma + 1) {
            // -------------------------------------------- MMA issuer of chain i
            const uint32_t tmem = enter();
            const int i = warp - kMma;
            const bool lead = elect_one();
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);       // (known to be uniform)
            const uint32_t s_i = tm + __shfl_sync(0xffffffffu, i, 0) * kCols;
            const uint32_t o_i = tm + K::COL_O + __shfl_sync(0xffffffffu, i, 0) * D;
            constexpr uint32_t idS = FP8 ? idesc_e4m3_f32(kRows, K::HCOLS) : idesc_bf16_f32(kRows, K::HCOLS, false, false);
            constexpr uint32_t idPV = idesc_bf16_f32(kRows, D, false, true);
            int pcnt = 0, bcnt = 0;                       // this chain's tiles; pieces of both chains
            int tbase = 0, qbase = 0;                     // the CTA's key tiles and Q tiles up to the next piece
            // K, V and Q tiles seen: every one, in order, by both chains (a barrier's parity tells neighbouring phases apart, no
            // more).  (Slots and parities are counted, not divided: this warp's own instructions are on the chain's path.)
            struct Ring {
                int at, slot, used;                       // tiles seen; the next one's slot; that of the last one seen
                uint32_t parity;
            };
            Ring rk = {}, rv = {}, rq = {};
            struct Work {
                int cnt, x0, step, t0, both, ends;
                int whole;                                // tiles of the piece of which some row sees the last page
                int base, q;                              // the CTA's numbers of its first tile and of the chain's Q tile
            };
            // the tiles up to `target`; what the other chain alone uses is given back as soon as it is there
            auto see = [&](Ring& r, int target, bool mine, int ring_n, int full, int empty) -> bool {
                while (r.at <= target) {
                    if (!wait_all(bar(full + r.slot), r.parity)) return false;
                    if (lead && !(mine && r.at == target)) mbar_arrive(bar(empty + r.slot));
                    r.used = r.slot;
                    ++r.at;
                    if (++r.slot == ring_n) {
                        r.slot = 0;
                        r.parity ^= 1;
                    }
                }
                return true;
            };
            constexpr int QRDY = FP8 ? K::QREADY : K::QFULL;
            auto see_k = [&](int t, bool mine) { return see(rk, t, mine, NSK, K::KFULL, K::KEMPTY); };
            auto see_v = [&](int t, bool mine) { return see(rv, t, mine, NSV, K::VREADY, K::VEMPTY); };
            auto see_q = [&](int t, bool mine) { return see(rq, t, mine, 2, QRDY, K::QEMPTY); };
            int n = 0;
            // The next piece, if there is one and (or else, with `any`, the next that does) it has tiles of this chain.
            auto next = [&](Work& x, bool any) -> bool {
                for (;; ++n) {
                    const Piece* at = piece_at(n);
                    if (!at || at->end) return false;
                    x.cnt = at->count(i);
                    if (x.cnt == 0 && !any) return false;
                    x.x0 = at->begin(i);
                    x.step = at->step();
                    x.t0 = at->t0;
                    x.both = !at->two && at->count(1) > 0;
                    x.ends = at->seen_end(a, min(at->nq, at->two ? (i + 1) * a.pb : a.pb));
                    x.whole = (x.ends - x.t0 * K::KEYS + kBlock - 1) / kBlock / K::TP;
                    x.base = tbase;
                    x.q = qbase + (at->two ? i : 0);
                    tbase += at->tiles();
                    qbase += at->two ? 2 : 1;
                    release(n);
                    if (x.cnt > 0) break;
                    if (!see_q(qbase - 1, false) || !see_k(tbase - 1, false) || !see_v(tbase - 1, false)) return false;
                }
                ++n;
                return true;
            };
            // Half h of S of tile j of this chain's in a piece (its K and Q seen).  (A descriptor is the first one's with a
            // constant added: made anew for each, the issue of a product took longer than the product.)
            auto issue_s = [&](const Work& x, int j, auto half) {
                constexpr int h = decltype(half)::value;
                const int sk = rk.used;                   // (no tile behind it has been seen yet)
                const uint32_t kbase = __shfl_sync(0xffffffffu, sb + K::OFF_K + sk * K::KTILE, 0) + h * (K::KTILE / K::HALVES);
                const uint32_t q_s = __shfl_sync(0xffffffffu, sb + K::OFF_Q + (x.q & 1) * K::QTILE, 0);
                constexpr uint32_t dst = h * K::HCOLS;
                if constexpr (FP8) {
                    constexpr uint32_t LO = D == 128 ? K::SLAB : 512;
                    const uint64_t dq = smem_desc(q_s, 128, 1024), dk = smem_desc(kbase, 128, D * 8);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)      // the first term's, then the second's
                        mma_ss_f8(lead, s_i + dst, dq + (((k / (D / 32)) * LO + (k % (D / 32)) * 256) >> 4),
                                  dk + (((k % (D / 32)) * 256) >> 4), idS, k > 0 ? 1u : 0u);
                } else {
                    const uint64_t dq = desc_sw128(q_s, 16, 1024), dk = smem_desc(kbase, 128, K::NCH * 128);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_ss(lead, s_i + dst, dq + (((k / 4) * K::SLAB + (k % 4) * 32) >> 4), dk + ((k * 256) >> 4), idS,
                               k > 0 ? 1u : 0u);
                }
                commit(lead, bar(K::SFULL + 2 * i + h));
                if (h == K::HALVES - 1) {
                    commit(lead, bar(K::KEMPTY + sk));
                    if (j + 1 == x.cnt) commit(lead, bar(K::QEMPTY + (x.q & 1)));
                }
            };
            // One loop: by halves, P . V of the chain's present tile, if there is one, each with the same half of S of the next
            // tile behind it, if there is one in the piece; then both halves of S of a new piece's first.  One thread's
            // products are done in order: S of a half may overwrite the P there.
            Work p = {}, q = {};
            int j = 0, jq = 0;
            bool now = false, ok = true;                  // now: S of tile j of piece p has been issued
#pragma unroll 1
            while (ok) {
                bool then, fresh = false;
                if (now && j + 1 < p.cnt) {
                    q = p;
                    jq = j + 1;
                    then = true;
                } else {
                    then = next(q, !now);                 // (in time for the present piece's last tile, if it is there)
                    jq = 0;
                    fresh = true;
                    if (!then && !now) break;
                }
                const int x = p.x0 + j * p.step;
                if (now) {
                    if (!see_v(p.base + x, true)) break;
                    // a piece's first PV starts O afresh: the other chain too has read the last result that they shared
                    if (j == 0 && bcnt > 0 && !wait_all(bar(K::OFREE), (bcnt - 1) & 1)) break;
                }
                const int sv = rv.used;
                const uint32_t vbase = __shfl_sync(0xffffffffu, sb + K::OFF_V + sv * K::VTILE, 0);
                // units up to the last page that a row sees
                const int steps = x < p.whole ? kUnits : HG * min(max((p.ends - (p.t0 + x) * K::KEYS + kBlock - 1) / kBlock, 1), K::TP);
                constexpr int HALVES = K::HALVES, EACH = kUnits / HALVES;
                // a turn: P . V of half h, if there is a present tile, and S of it, if it belongs to the same piece; the second
                // time (a new piece), S of both
                auto turn = [&](auto half) -> bool {
                    constexpr int h = decltype(half)::value;
                    if (now) {
                        if (!wait_all(bar(K::PFULL + 2 * i + h), pcnt & 1)) return false;
                        tc_fence_after();
                        const uint64_t dv = smem_desc(vbase, K::NCH * 128, 128);
                        if (steps == kUnits) {
#pragma unroll
                            for (int k = 0; k < EACH; ++k)
                                mma_ts(lead, o_i, s_i + h * K::HCOLS + k * 8, dv + (((EACH * h + k) * K::PAGE) >> 4), idPV,
                                       h > 0 || k > 0 ? 1u : j > 0 ? 1u : 0u);
                        } else {
#pragma unroll 1
                            for (int k = 0; k < min(EACH, steps - EACH * h); ++k)
                                mma_ts(lead, o_i, s_i + h * K::HCOLS + k * 8, dv + (((EACH * h + k) * K::PAGE) >> 4), idPV,
                                       j > 0 || h > 0 || k > 0 ? 1u : 0u);
                        }
                        if (HALVES > 1) commit(lead, bar(K::PVDONE + 2 * i + h));
                        if (h == HALVES - 1) {
                            if (j + 1 == p.cnt) commit(lead, bar(K::ODONE + i));
                            commit(lead, bar(K::VEMPTY + sv));
                        }
                    }
                    return true;
                };
                using H0 = std::integral_constant<int, 0>;
                using H1 = std::integral_constant<int, HALVES - 1>;
                if (!(ok = turn(H0{}))) break;
                // (the next S's K is waited for while P . V runs: before it, a late K kept V from being given back)
                if (then && !fresh && !(ok = see_k(q.base + q.x0 + jq * q.step, true))) break;
                // (a new piece's Q and K: bf16 by halves, before the last P; else, as FP8's softmax warps split Q behind it, after)
                constexpr bool EARLY = !FP8 && HALVES > 1;
                if (EARLY && then && fresh && !(ok = see_q(q.q, true) && see_k(q.base + q.x0, true))) break;
                if (HALVES > 1) {
                    if (then && !fresh) issue_s(q, jq, H0{});
                    if (!(ok = turn(H1{}))) break;
                }
                if (!EARLY && then && fresh && !(ok = see_q(q.q, true) && see_k(q.base + q.x0, true))) break;
                if (then && fresh) tc_fence_after();
                if (then && (fresh && HALVES > 1)) issue_s(q, jq, H0{});
                if (then) issue_s(q, jq, H1{});
                if (now) {
                    bcnt += j + 1 == p.cnt && p.both;
                    ++pcnt;
                }
                now = then;
                p = q;
                j = jq;
            }
            commit(lead, bar(K::DRAIN));
            // every MMA issued has completed before TMEM is freed
            const Ctl drain{drain_flag, a.err, a.wait_limit_ns};
            wait(bar(K::DRAIN), 0, drain);
            __syncwarp();
        }
    } else if (warp >= kReady) {
        // ------------------------------------------------ V made ready
        regs_dec<kRegsReady>();
        enter();
        const int w = warp - kReady;

        // V is made harmless to rows that do not see it: a weight of 0 times NaN or infinity is NaN.  Keys that no row sees
        // are cleared, and non-finite values become 0 where some rows do not see them (HG > 1: everywhere, for other
        // heads' rows have weight 0 for them) and are added back, row by row, in the epilogue (from global memory:
        // rare).
        // (FP8) `pages` of the two pages of V from `at` on, each in the upper half of its place and widened over it; their
        // first keys at v and v1.  vs: their scales; where one is not finite, all its page's codes count as NaN (and it, as 1)
        auto widen_pages = [&](uint8_t* at, const Guard<HG>& gd, int v, int v1, int pages, const float* vs) -> bool {
            constexpr int N = D / 32;                     // 16-byte chunks of codes a lane and page
            // (a lane's chunk j % N of page j / N: its key of the page, and where it goes)
            auto key_of = [&](int j) { return (lane & 7) + ((lane + 32 * (j % N)) >> 3) / (D / 16) * 8; };
            auto place = [&](int j) {
                const int q = (lane + 32 * (j % N)) >> 3;
                return at + j / N * K::PAGE + q / (D / 16) * (K::NCH * 128) + 2 * (q % (D / 16)) * 128 + (lane & 7) * 16;
            };
            uint32_t nan = 0;                             // a lane's chunks that hold NaN codes
#pragma unroll 1
            for (int pg = 0; pg < pages; ++pg) {          // (rolled, for the instruction cache)
                uint4 raw[N];
#pragma unroll
                for (int j = 0; j < N; ++j)
                    raw[j] = *reinterpret_cast<const uint4*>(at + pg * K::PAGE + K::LAND + (lane + 32 * j) * 16);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    uint32_t o[8];
                    widen4(raw[j].x, o[0], o[1]);
                    widen4(raw[j].y, o[2], o[3]);
                    widen4(raw[j].z, o[4], o[5]);
                    widen4(raw[j].w, o[6], o[7]);
                    if (nan_codes(raw[j].x) | nan_codes(raw[j].y) | nan_codes(raw[j].z) | nan_codes(raw[j].w)) nan |= 1u << (pg * N + j);
                    uint8_t* dst = place(j) + pg * K::PAGE;
                    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(dst + 128) = make_uint4(o[4], o[5], o[6], o[7]);
                }
            }
            const bool fin0 = fabsf(vs[0]) < INFINITY, fin1 = pages < 2 || fabsf(vs[1]) < INFINITY;
            if (!gd.any_of(v, kBlock) || (pages > 1 && !gd.any_of(v1, kBlock))) {
#pragma unroll 1
                for (int j = 0; j < pages * N; ++j) {
                    if (gd.any((j < N ? v : v1) + key_of(j))) continue;
                    *reinterpret_cast<uint4*>(place(j)) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(place(j) + 128) = make_uint4(0, 0, 0, 0);
                    nan &= ~(1u << j);
                }
            }
            bool found = false;
            if (nan != 0 || !fin0 || !fin1) {
                // (rare) a lane's own chunks again: a NaN code is the only one that has become +-480
#pragma unroll 1
                for (int j = 0; j < pages * N; ++j) {
                    const int key = (j < N ? v : v1) + key_of(j);
                    const bool fin = j < N ? fin0 : fin1, leave = gd.all(key) && fin;
                    if (!gd.any(key) || ((nan >> j & 1) == 0 && fin)) continue;
                    uint16_t* e = reinterpret_cast<uint16_t*>(place(j));
#pragma unroll 1
                    for (int y = 0; y < 16; ++y) {
                        uint16_t& x = e[y / 8 * 64 + y % 8];
                        if ((x & 0x7fff) == 0x43f0 || !fin) x = leave ? 0x7fc0 : 0;
                    }
                    found |= !leave;
                }
            }
            return found;
        };
        auto guard_group = [&](uint8_t* at, const Guard<HG>& gd, int v) -> bool {     // 8 keys of bf16 V
            constexpr int N = K::NCH / 4;
            uint4* e = reinterpret_cast<uint4*>(at + lane * 16);
            const int key = v + (lane & 7);
            if (!gd.any(key)) {
#pragma unroll
                for (int j = 0; j < N; ++j) e[32 * j] = make_uint4(0, 0, 0, 0);
                return false;
            }
            uint32_t bad = 0;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const uint4 x = e[32 * j];
                bad |= inf_words(x.x) | inf_words(x.y) | inf_words(x.z) | inf_words(x.w);
            }
            if (bad == 0 || gd.all(key)) return false;
#pragma unroll 1
            for (int j = 0; j < 4 * N; ++j) {
                uint32_t* y = reinterpret_cast<uint32_t*>(e + 32 * (j / 4)) + j % 4;
                const uint32_t hit = inf_words(*y);
                *y &= ~((hit >> 15) * 0xffffu);
            }
            return true;
        };
        // One warp's share of tile x of piece n, the CTA's gt-th: its units 2 w and 2 w + 1.
        auto ready_v = [&](const Piece& p, int n, int x, int gt) {
            const int sv = gt % NSV, v0 = (p.t0 + x) * K::KEYS, pages = min(K::TP, p.np - (p.t0 + x) * K::TP);
            uint8_t* base = smem + K::OFF_V + sv * K::VTILE;
            const Guard<HG> gd = guard_of<HG>(a, p);
            bool found = false;
            if constexpr (FP8) {
                const int pg = 2 * w / HG, pg1 = (2 * w + 1) / HG;
                if (pg < pages)
                    found = widen_pages(base + 2 * w * K::PAGE, gd, v0 + pg * kBlock, v0 + pg1 * kBlock, pg1 < pages ? 2 : 1,
                                        scales + gt % K::NSC * 16 + 8 + 2 * w);
                fence_proxy_async_smem();
            } else {
                bool touched = false;
#pragma unroll 1
                for (int y = 4 * w; y < 4 * w + 4; ++y) {
                    const int pg = y / 2 / HG, v = v0 + pg * kBlock + (y & 1) * 8;
                    if (pg >= pages || gd.all_of(v, 8)) continue;
                    const bool f = guard_group(base + y * (K::NCH * 128), gd, v);
                    found |= f;
                    touched |= f || !gd.any_of(v, 8);
                }
                if (__any_sync(0xffffffffu, touched)) fence_proxy_async_smem();
            }
            if (__any_sync(0xffffffffu, found) && lane == 0) atomicOr(&ring[n % kPieces].bad, 1u << (x >> p.mark_shift()));
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(K::VREADY + sv));
        };
        bool ok = true;
        int gt = 0;                                       // key tiles
        for (int n = 0; ok; ++n) {
            const Piece* p = piece_at(n);
            if (!p || p->end) break;
            const int tiles = p->tiles();
#pragma unroll 1
            for (int x = 0; x < tiles && ok; ++x, ++gt) {
                if (!(ok = wait_all(bar(K::VFULL + gt % NSV), (gt / NSV) & 1))) break;
                ready_v(*p, n, x, gt);
            }
            release(n);
        }
    } else {
        // ------------------------------------------------ softmax of chain i, thread r = row r
        regs_inc<kRegsSoftmax>();
        const uint32_t tmem = enter();
        const int i = warp >> 2, r = tid & (kRows - 1), hw = (warp & 3) * HG / 4;      // hw: the row's head of the HG
        const int G = a.group, rr = r % RQ, pos = rr / G, hl = rr - pos * G;
        const uint32_t lbase = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t scol = tmem + lbase + i * kCols;   // S / P
        const uint32_t ocol = tmem + lbase + K::COL_O + i * D;
        // What the guard took out of V, added to a row's results where its lane has just written them (rare): the keys
        // of the piece's marked parts are looked through, for 8 dimensions after the other, 8 keys' loads in flight.  (A value
        // at a time over all keys took 20 ms for one NaN in each of 64 streams of 4096 keys, a call of 0.16 to 0.19 ms; now it
        // takes 0.19 to 0.26.  No shuffles or votes: with them in this code every call took 0.8 us longer.)
        auto add_back = [&](const Piece& p, unsigned bad, int qi, int d0, int d1, uint8_t* out, float* part) {
            using Eight = std::conditional_t<FP8, uint2, uint4>;
            constexpr int E = 8, C = FP8 ? 16 : 8;        // elements at a time, and of a 16-byte chunk
            Sight see;
            const uint32_t* tree = nullptr;
            if (a.tree) {
                see.tree(p);
                tree = a.tree + (p.row + p.q0 + qi) * (int64_t)a.tree_words;
            } else {
                see.window(a, p, p.first + qi);
            }
            const int shift = p.mark_shift();
#pragma unroll 1
            for (int d = d0; d < d1; d += E) {
                float add[E] = {};
#pragma unroll 1
                for (unsigned marks = bad; marks; marks &= marks - 1) {
                    const int x = (__ffs(marks) - 1) << shift;
                    const int end = min((p.t0 + min(x + (1 << shift), p.tiles())) * K::TP, p.np) * kBlock;
#pragma unroll 1
                    for (int v = (p.t0 + x) * K::KEYS; v < end; v += 8) {
                        const int id = a.tables[(int64_t)p.b * a.max_blocks + p.page(v / kBlock)];
                        if (id < 0 || id >= a.num_blocks) continue;
                        const int64_t page = (int64_t)id * a.Hkv + p.g + hw;
                        const uint8_t* at = a.v_cache + page * K::LAND + (v % kBlock / 8 * (D / C) + d / C) * 128 + d % C;
                        auto load = [&](int y) { return *reinterpret_cast<const Eight*>(at + y * 16); };
                        const float sc = FP8 ? a.v_scales[page] : 1.f;
                        auto hit = [](const Eight& w) {
                            if constexpr (FP8) return nan_codes(w.x) | nan_codes(w.y);
                            else return inf_words(w.x) | inf_words(w.y) | inf_words(w.z) | inf_words(w.w);
                        };
                        Eight w[8];
#pragma unroll
                        for (int y = 0; y < 8; ++y) w[y] = load(y);
                        uint32_t any = fabsf(sc) < INFINITY ? 0u : 1u;
#pragma unroll
                        for (int y = 0; y < 8; ++y) any |= hit(w[y]);
                        if (any == 0) continue;
#pragma unroll 1
                        for (int y = 0; y < 8; ++y) {
                            const bool has = see.has(v + y) || (tree && v + y >= p.L - p.Q &&
                                                                (tree_bits(tree, a.tree_words, v + y - (p.L - p.Q), p.Q) & 1u));
                            if (!has) continue;
                            const Eight z = load(y);
                            const uint32_t* c = &z.x;
#pragma unroll
                            for (int e = 0; e < E; e += 2) {
                                const float2 f = FP8 ? e4m3x2_to_float2(c[e / 4] >> (e % 4 * 8))
                                                     : make_float2(bf16_lo(c[FP8 ? 0 : e / 2]), bf16_hi(c[FP8 ? 0 : e / 2]));
                                if (!(fabsf(f.x) < INFINITY && fabsf(sc) < INFINITY)) add[e] += f.x * sc;
                                if (!(fabsf(f.y) < INFINITY && fabsf(sc) < INFINITY)) add[e + 1] += f.y * sc;
                            }
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (add[e] == 0.f) continue;
                    if (part) {
                        part[(size_t)((d + e) / 4) * 2 * kRows * 4 + e % 4] += add[e];
                    } else {
                        __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(out) + d + e;
                        *o = __float2bfloat16_rn(__bfloat162float(*o) + add[e]);
                    }
                }
            }
        };
        // the weight of a part with reference m and sum l beside the largest reference `top` of the parts.  (A part
        // that saw nothing holds zeros, or NaN)
        auto weight = [](float m, float l, float top) {
            return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2_fast(m - top);
        };
        auto finish_lse = [](float m, float l) {
            return m == -INFINITY && l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.693147180559945f;
        };
        // The results of a piece: part ct of its rows' results (two row tiles: row tile ct; one: columns from ct * D / 2 on), from
        // this chain's O or (both) from both.  (In loops, one copy: it runs once a piece, from an instruction cache
        // that holds the inner loops by then.)
        auto finish = [&](const Piece& p, int ct, bool both, float m, float l) {
            const bool whole = p.parts == 1;
            float* slot = part_slot<D>(a, blockIdx.x, p.t0 == 0);
            const int qi = (p.two ? ct * a.pb : 0) + pos;
            const bool row_ok = pos < a.pb && qi < p.nq;
            if (!__any_sync(0xffffffffu, row_ok)) return;
            const int d0 = p.two ? 0 : ct * (D / 2), d1 = p.two ? D : d0 + D / 2;
            const uint32_t oa = tmem + lbase + K::COL_O + (both ? 0 : i * D), ob = tmem + lbase + K::COL_O + D;
            float fa = 1.f, fb = 0.f;
            if (both) {
                const float m0 = ml[r], l0 = ml[kRows + r], m1 = ml[2 * kRows + r], l1 = ml[3 * kRows + r];
                m = fmaxf(m0, m1);
                fa = weight(m0, l0, m);
                fb = weight(m1, l1, m);
                l = l0 * fa + l1 * fb;
                if (m0 == -INFINITY) fa = 1.f;
                if (m1 == -INFINITY) fb = 1.f;
            }
            const bool none = m == -INFINITY && l == 0.f;          // a row that saw nothing
            const int64_t row = p.row + p.q0 + qi;
            const int h = (p.g + hw) * G + hl;
            uint8_t* dst = row_ok ? a.out.row(row, h) : nullptr;
            float* part = slot + ((p.two ? ct * kRows : 0) + r) * 4;
            if (row_ok && !whole) {
                slot[(size_t)2 * kRows * D + ct * kRows + r] = m;
                slot[(size_t)2 * kRows * (D + 1) + ct * kRows + r] = l;
            } else if (row_ok && a.lse && (p.two || ct == 0)) {
                a.lse[row * a.Hq + h] = finish_lse(m, l);
            }
            const float inv = none ? 0.f : __fdividef(1.f, l);
            if (whole) {
                fa *= inv;
                fb *= inv;
            }
            uint32_t x[32], y[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = 0;
            tmem_ld32_async(oa + d0, x);
#pragma unroll 1
            for (int c = d0; c < d1; c += 32) {
                if (both) {
                    tmem_ld32_async(ob + c, y);
                    tmem_wait_ld_into(y);
                }
                tmem_wait_ld_into(x);
                float o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(x[e]) * fa + __uint_as_float(y[e]) * fb;
                tmem_ld32_async(oa + min(c + 32, D - 32), x);      // (behind the last, for nothing)
                if (row_ok && whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t v[4];
#pragma unroll
                        for (int f = 0; f < 4; ++f) v[f] = pack_bf16(o[e + 2 * f], o[e + 2 * f + 1]);
                        *reinterpret_cast<uint4*>(dst + (c + e) * 2) = none ? make_uint4(0, 0, 0, 0) : make_uint4(v[0], v[1], v[2], v[3]);
                    }
                } else if (row_ok) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(part + (size_t)((c + e) / 4) * 2 * kRows * 4) =
                            make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
                __syncwarp();
            }
            tmem_wait_ld_into(x);
        };
        // A cut piece's part ct is in memory: the last of the item's CTAs to get here (with these lanes' rows) joins
        // them, in order.
        auto join = [&](const Piece& p, int ct) {
            const int w = warp & 3;
            const int mine = min(32, min(a.pb, p.nq - (p.two ? ct * a.pb : 0)) * G - (w * 32) % RQ);     // valid rows among the lanes
            if (mine <= 0) return;
            __threadfence();
            __syncwarp();
            int old = 0;
            int* ticket = a.tickets + p.c0 * 8 + ct * 4 + w;
            if (lane == 0) old = atom_add_acq_rel_gpu(ticket, 1);
            if (__shfl_sync(0xffffffffu, old, 0) != p.parts - 1) return;
            if (lane == 0) *ticket = 0;
            fence_acquire_gpu();
            // Lanes are rows, or where there are few, rows times groups of columns; eight 16-byte pieces of a part in flight.
            const int d0 = p.two ? 0 : ct * (D / 2), n4 = (p.two ? D : D / 2) / 4, rt = p.two ? ct * kRows : 0;
            const int lg = 32 - __clz(mine - 1), R = w * 32 + (lane & ((1 << lg) - 1)), rp = R % RQ / G;
            if (R >= w * 32 + mine) return;
            auto at = [&](int x) { return part_slot<D>(a, p.c0 + x, x == 0); };
            auto m_of = [&](int x) { return __ldcg(at(x) + (size_t)2 * kRows * D + ct * kRows + R); };
            auto l_of = [&](int x) { return __ldcg(at(x) + (size_t)2 * kRows * (D + 1) + ct * kRows + R); };
            const int64_t orow = p.row + p.q0 + (p.two ? ct * a.pb : 0) + rp;
            const int oh = (p.g + hw) * G + R % RQ - rp * G, step = 32 >> lg;
            uint8_t* dst = a.out.row(orow, oh);
#pragma unroll 1
            for (int q0 = lane >> lg; q0 < n4; q0 += 8 * step) {
                float o[32] = {}, top = -INFINITY, l = 0.f;
#pragma unroll 1
                for (int x = 0; x < p.parts; x += 2) {    // two parts' loads in flight
                    float mx[2], lx[2];
                    float4 u[2][8];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const bool is = x + y < p.parts;
                        const int z = is ? x + y : x;
                        mx[y] = is ? m_of(z) : -INFINITY;
                        lx[y] = is ? l_of(z) : 0.f;
                        const float4* s = reinterpret_cast<const float4*>(at(z)) + (size_t)(d0 / 4) * 2 * kRows + rt + R;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            u[y][e] = is && q0 + e * step < n4 ? __ldcg(s + (size_t)(q0 + e * step) * 2 * kRows)
                                                              : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                    const float was = top;
                    top = fmaxf(top, fmaxf(mx[0], mx[1]));
                    const float fo = was == -INFINITY ? 1.f : exp2_fast(was - top);
                    float f[2];
                    l *= fo;
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        f[y] = weight(mx[y], lx[y], top);
                        l += f[y] * lx[y];
                        if (mx[y] == -INFINITY) f[y] = 1.f;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        o[4 * e] = o[4 * e] * fo + u[0][e].x * f[0] + u[1][e].x * f[1];
                        o[4 * e + 1] = o[4 * e + 1] * fo + u[0][e].y * f[0] + u[1][e].y * f[1];
                        o[4 * e + 2] = o[4 * e + 2] * fo + u[0][e].z * f[0] + u[1][e].z * f[1];
                        o[4 * e + 3] = o[4 * e + 3] * fo + u[0][e].w * f[0] + u[1][e].w * f[1];
                    }
                }
                const bool none = top == -INFINITY && l == 0.f;
                const float il = none ? 0.f : __fdividef(1.f, l);
                if (q0 == 0 && a.lse && (p.two || ct == 0)) a.lse[orow * a.Hq + oh] = finish_lse(top, l);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (q0 + e * step < n4) {
                        uint2 v = make_uint2(0, 0);
                        if (!none) v = make_uint2(pack_bf16(o[4 * e] * il, o[4 * e + 1] * il), pack_bf16(o[4 * e + 2] * il, o[4 * e + 3] * il));
                        *reinterpret_cast<uint2*>(dst + (d0 + (q0 + e * step) * 4) * 2) = v;
                    }
            }
        };
        // (FP8) this warp's rows of Q tile qt, in place, 16 at a time, half a row a lane: groups of 8 rows are 1024 bytes of a
        // slab; the first term's codes go where the first slab was (D = 64: to the first half of each 1024 bytes), the
        // second's to the other.
        auto split_q = [&](int qt) {
            uint8_t* tile = smem + K::OFF_Q + (qt & 1) * K::QTILE;
            constexpr int N = D / 16;                     // 16-byte chunks of half a row
            constexpr int LO = D == 128 ? K::SLAB : 512;
            const int half = lane >> 4, w32 = (warp & 3) * 32;
#pragma unroll 1
            for (int row = w32 + (lane & 15); row < w32 + 32; row += 16) {
                uint32_t top = 0;
                uint4 x[N];
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    const int ch = half * N + c;          // (dimensions 8 ch .. 8 ch + 7)
                    x[c] = *reinterpret_cast<const uint4*>(tile + (ch / 8) * K::SLAB + row * 128 + (((ch & 7) ^ (row & 7)) * 16));
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[c].x & 0x7fff7fffu, x[c].y & 0x7fff7fffu),
                                                 __vmaxu2(x[c].z & 0x7fff7fffu, x[c].w & 0x7fff7fffu)));
                }
                top = max(top & 0xffffu, top >> 16);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
                // 2^(134 - exponent) takes the largest element to [128, 256); kept inside fp32's normal range (a row below
                // 2^-113 counts as smaller beside any scale); infinities and NaN make the row NaN
                const int ex = min(max((int)(top >> 7), 14), 254);
                const float f = __uint_as_float((uint32_t)(261 - ex) << 23);
                const float inv = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(ex - 7) << 23);
                uint8_t* dst = tile + (row / 8) * 1024 + (row & 7) * 16 + half * (N / 2) * 128;
#pragma unroll
                for (int c = 0; c < N / 2; ++c) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint4 y = x[2 * c + e / 2];
                        uint32_t h0, h1, l0, l1;
                        split2(e & 1 ? y.z : y.x, f, h0, l0);
                        split2(e & 1 ? y.w : y.y, f, h1, l1);
                        hi[e] = h0 | h1 << 16;
                        lo[e] = l0 | l1 << 16;
                    }
                    x[2 * c] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    x[2 * c + 1] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                __syncwarp();
#pragma unroll
                for (int c = 0; c < N / 2; ++c) {
                    *reinterpret_cast<uint4*>(dst + c * 128) = x[2 * c];
                    *reinterpret_cast<uint4*>(dst + LO + c * 128) = x[2 * c + 1];
                }
                if (half == 0) q_scale[qt % K::NQS * kRows + row] = inv;
            }
            fence_proxy_async_smem();
        };
        constexpr int HALVES = K::HALVES, STEP = K::KEYS / HALVES, PAGES = STEP / kBlock;      // keys and pages (of each head)
        bool ok = true;
        int scnt = 0, tbase = 0, qbase = 0;               // this chain's tiles; the CTA's tiles and Q tiles
        int pieces = 0, pieces1 = 0, bcnt = 0;            // the CTA's pieces; those of chain 1; those of both chains
        int q1 = 0;                                       // chain 1: its Q tiles
        // (FP8) piece n's Q, whose first tile is the CTA's qt-th: chain 0's row tile by its warps, and chain 1's
        auto ready_q = [&](int n, int qt) {
            const Piece* p = piece_at(n);
            if (!p || p->end || (i == 1 && !p->two)) return;
            qt += i;
            ok = i == 0 ? wait_all(bar(K::QFULL + (n & 1)), (n >> 1) & 1) : wait_all(bar(K::Q1FULL), q1 & 1);
            if (!ok) return;
            ++q1;
            if (__any_sync(0xffffffffu, pos < a.pb && (p->two ? i * a.pb : 0) + pos < p->nq)) split_q(qt);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(K::QREADY + (qt & 1)));
        };
#pragma unroll 1
        for (int n = FP8 ? -1 : 0; ok; ++n) {             // (from -1: the first piece's Q, by the one copy of that code)
            const Piece* p = n < 0 ? nullptr : piece_at(n);
            if (n >= 0 && (!p || p->end)) break;
            const int cnt = p ? p->count(i) : 0;
            const int base = tbase, qt = qbase + (p && p->two ? i : 0);
            if (p) {
                tbase += p->tiles();
                qbase += p->two ? 2 : 1;
            }
            float m = 0.f, l = 0.f;                       // the reference maximum (exp2 units); the sum of P
            if (cnt > 0) {
                const int x0 = p->begin(i), step = p->step(), t0 = p->t0;
                const int qi = (p->two ? i * a.pb : 0) + pos;  // the row's query, from the piece's first on
                const bool row_ok = pos < a.pb && qi < p->nq;
                const bool live = __any_sync(0xffffffffu, row_ok);
                // (rows of no query see everything, so that they ask for no mask)
                Sight see{0, -0x40000000, 0x3fffffff};
                const uint32_t* tree = nullptr;
                if (row_ok) {
                    if (a.tree) {
                        see.tree(*p);
                        tree = a.tree + (p->row + p->q0 + qi) * (int64_t)a.tree_words;
                    } else {
                        see.window(a, *p, p->first + qi);
                    }
                }
                const int tree0 = p->L - p->Q, tree_n = p->Q;
                const int ends = p->seen_end(a, min(p->nq, p->two ? (i + 1) * a.pb : a.pb));
                m = row_ok ? -INFINITY : 0.f;
                float sc = a.scale_log2;
                // (by halves: while P of one is made, the other's P . V and next S run)
#pragma unroll 1
                for (int hh = 0; hh < HALVES * cnt; ++hh) {
                    const int j = hh / HALVES, h = hh % HALVES, x = x0 + j * step;
                    const int v0 = (t0 + x) * K::KEYS + h * STEP;          // the half's first key
                    if (!(ok = wait_all(bar(K::SFULL + 2 * i + h), scnt & 1))) break;
                    // (what no row sees behind the first half is not read by the PV)
                    if (live && !(h > 0 && v0 >= ends)) {
                        tc_fence_after();
                        if (FP8 && hh == 0) {
                            sc = a.scale_log2 * q_scale[qt % K::NQS * kRows + r];
                            if (sc == 0.f) sc = 0x1p-149f;         // (a row of zeros, a tiny scale: -inf * 0 would be NaN)
                        }
                        const bool masked =
                            !__all_sync(0xffffffffu, (v0 >= see.wl && v0 + STEP - 1 <= see.wh) || v0 + STEP <= see.ns);
                        // S and P of page pg of the half: columns of this row's head
                        auto s_col = [&](int pg) { return scol + h * K::HCOLS + (pg * HG + hw) * kBlock; };
                        auto p_col = [&](int pg, int head) { return scol + h * K::HCOLS + (pg * HG + head) * 8; };
                        // FP8: factors of S and of P, a page each
                        float ks[PAGES], vs[PAGES];
                        const float* ks_at = scales + ((base + x) % K::NSC) * 16 + h * PAGES * HG + hw;
                        if constexpr (FP8) {
#pragma unroll
                            for (int pg = 0; pg < PAGES; ++pg) {
                                ks[pg] = masked ? 1.f : ks_at[pg * HG];
                                vs[pg] = ks_at[8 + pg * HG];
                                vs[pg] = fabsf(vs[pg]) < INFINITY ? vs[pg] : 1.f;          // (V has no finite values then)
                            }
                        }
                        // Keys that some row does not see: their S becomes -inf there, in tensor memory (FP8: the page's scale
                        // is multiplied in on the way), and what follows knows no masks.  (A second copy of it with masks,
                        // though hardly ever run, made every tile a third slower: the inner loops no longer fit the
                        // instruction cache.)
                        if (masked) {
#pragma unroll 1
                            for (int pg = 0; pg < PAGES; ++pg) {
                                // the visible ones of the page's 16 keys
                                const int v = v0 + pg * kBlock, n_s = see.ns - v, lo = max(see.wl - v, 0), hi = min(see.wh - v, 31);
                                uint32_t w = n_s >= 16 ? 0xffffu : n_s > 0 ? (1u << n_s) - 1u : 0u;
                                if (lo <= hi) w |= (0xffffffffu << lo) & (0xffffffffu >> (31 - hi));
                                if (tree && v + 31 >= tree0) w |= tree_bits(tree, a.tree_words, v - tree0, tree_n);
                                if (!FP8 && __all_sync(0xffffffffu, (w & 0xffffu) == 0xffffu)) continue;
                                float f[16];
                                tmem_ld16(s_col(pg), f);
                                uint32_t t[16];
#pragma unroll
                                for (int y = 0; y < 16; ++y)
                                    t[y] = w >> y & 1 ? __float_as_uint(FP8 ? f[y] * ks_at[pg * HG] : f[y]) : 0xff800000u;
                                tmem_st16u(s_col(pg), t);
                            }
                            tmem_wait_st();
                        }
                        bool again = false;
#pragma unroll 1
                        for (;;) {
                            if (again || !__all_sync(0xffffffffu, m > -INFINITY)) {
                                // no reference yet (a piece's first tile): the largest that is visible (O and l are 0 so far);
                                // or (rare) one that is too small: m rises by a whole number of octaves, and O and l are
                                // scaled down by as many (exact but for what falls below fp32's range)
                                float top = -INFINITY;
#pragma unroll 1
                                for (int pg = 0; pg < PAGES; ++pg) {
                                    float f[16], t = -INFINITY;
                                    tmem_ld16(s_col(pg), f);
#pragma unroll
                                    for (int y = 0; y < 16; ++y) t = fmaxf(t, FP8 && !masked ? f[y] * ks_at[pg * HG] : f[y]);
                                    top = fmaxf(top, t);
                                }
                                const float target = row_ok ? top * sc : -INFINITY;
                                if (!again) {
                                    if (m == -INFINITY) m = target;
                                } else {
                                    const float inc = target > m ? ceilf(target - m) : 0.f;
                                    const int e = (int)fminf(inc, 127.f);
                                    const float alpha = e < 127 ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.f;
                                    if (hh > 0) {         // the last P . V may still add to O
                                        if (HALVES > 1) wait_all(bar(K::PVDONE + 2 * i + 1 - h), (h ? scnt : scnt - 1) & 1);
                                        tc_fence_after();
#pragma unroll 1
                                        for (int c = 0; c < D; c += 16) {
                                            float o[16];
                                            tmem_ld16(ocol + c, o);
                                            uint32_t v[16];
#pragma unroll
                                            for (int y = 0; y < 16; ++y) v[y] = __float_as_uint(o[y] * alpha);
                                            tmem_st16u(ocol + c, v);
                                        }
                                        tmem_wait_st();
                                    }
                                    l *= alpha;
                                    m += inc;
                                }
                                // (too far below 0 is only seen here: m rises)
                                if (row_ok && m <= -kLimit && m > -INFINITY) raise_error(a.err, PKV_DEVERR_RANGE);
                            }
                            // P, two per packed fp32 operation (the even key in the low half), and their sum.  (Rows with
                            // nothing visible so far keep m = -inf: all their S are.)
                            uint32_t v[STEP / 2];
                            uint64_t ca = 0, cb = 0;
                            const float nm = m == -INFINITY ? 0.f : -m;
                            const uint64_t nm2 = f2pack(__float_as_uint(nm), __float_as_uint(nm));
                            // 16 keys in s[o .. o + 15]: page pg
                            auto emit16 = [&](const uint32_t* s, int pg) {
                                const float f = FP8 ? sc * ks[pg] : sc;
                                const uint64_t sc2 = f2pack(__float_as_uint(f), __float_as_uint(f));
                                const uint64_t vs2 = FP8 ? f2pack(__float_as_uint(vs[pg]), __float_as_uint(vs[pg])) : 0;
#pragma unroll
                                for (int y = 0; y < 16; y += 2) {
                                    float p0, p1;
                                    f2unpack(f2fma(f2pack(s[y], s[y + 1]), sc2, nm2), p0, p1);
                                    p0 = exp2_fast(p0);
                                    p1 = exp2_fast(p1);
                                    uint64_t p2 = f2pack(__float_as_uint(p0), __float_as_uint(p1));
                                    if ((y >> 1) & 1) cb = f2add(cb, p2);
                                    else ca = f2add(ca, p2);
                                    if constexpr (FP8) f2unpack(f2mul(p2, vs2), p0, p1);
                                    v[pg * 8 + (y >> 1)] = pack_bf16(p0, p1);
                                }
                            };
                            uint32_t s0[32], s1[32];
                            if constexpr (HG == 1) {
                                tmem_ld32_async(s_col(0), s0);
                                tmem_ld32_async(s_col(2), s1);
                            } else {
                                tmem_ld16_at<0>(s_col(0), s0);
                                tmem_ld16_at<16>(s_col(1), s0);
                                if constexpr (PAGES > 2) {
                                    tmem_ld16_at<0>(s_col(2), s1);
                                    tmem_ld16_at<16>(s_col(3), s1);
                                }
                            }
                            tmem_wait_ld_into(s0);
                            emit16(s0, 0);
                            emit16(s0 + 16, 1);
                            if constexpr (PAGES > 2) {
                                tmem_wait_ld_into(s1);
                                emit16(s1, 2);
                                emit16(s1 + 16, 3);
                            }
                            float a0, a1;
                            f2unpack(f2add(ca, cb), a0, a1);
                            if (__any_sync(0xffffffffu, row_ok && !(a0 + a1 < kHigh)) && !again) {
                                again = true;             // once more with m raised (NaN logits pass then)
                                continue;
                            }
                            if constexpr (HG == 1) {
                                tmem_st32u(p_col(0, 0), v);
                            } else {
#pragma unroll
                                for (int pg = 0; pg < PAGES; ++pg) {
                                    uint32_t d8[8], z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                                    for (int y = 0; y < 8; ++y) d8[y] = v[pg * 8 + y];
                                    tmem_st8(p_col(pg, hw), d8);
#pragma unroll
                                    for (int y = 1; y < HG; ++y) tmem_st8(p_col(pg, (hw + y) % HG), z);
                                }
                            }
                            l += a0 + a1;                 // (behind the store)
                            tmem_wait_st();
                            break;
                        }
                        tc_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(K::PFULL + 2 * i + h));
                    scnt += h == HALVES - 1;
                }
                if (!ok) break;
                // (a reference so large that fp32 cannot place the weights beside it is reported)
                const float size = fabsf(m);
                if (row_ok && size >= kLimit && size < INFINITY) raise_error(a.err, PKV_DEVERR_RANGE);
            }
            // (while the last P . V runs)
            if (FP8) ready_q(n + 1, qbase);
            if (!ok) break;
            if (cnt == 0) {
                if (n >= 0) {
                    ++pieces;
                    release(n);
                }
                continue;
            }
            // the results; with both chains, half the columns each, from both O, m and l
            const bool both = !p->two && p->count(1) > 0;
            if (both) {
                // (m and l lie in shared memory until both chains have read the last ones)
                if (bcnt > 0 && !(ok = wait_all(bar(K::OFREE), (bcnt - 1) & 1))) break;
                ml[(2 * i) * kRows + r] = m;
                ml[(2 * i + 1) * kRows + r] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(K::LREADY));
                if (!(ok = wait_all(bar(K::LREADY), bcnt & 1))) break;
                ++bcnt;
            }
            if ((both || i == 0) && !(ok = wait_all(bar(K::ODONE), pieces & 1))) break;
            if ((both || i == 1) && !(ok = wait_all(bar(K::ODONE + 1), pieces1 & 1))) break;
            tc_fence_after();
            const int ct0 = p->two || both ? i : 0, ct1 = p->two || both ? i + 1 : 2;
#pragma unroll 1
            for (int ct = ct0; ct < ct1; ++ct) finish(*p, ct, both, m, l);
            // O read: the next piece's first PV may overwrite it (in the chain itself, its P come after this)
            tc_fence_before();
            __syncwarp();
            if (both && lane == 0) mbar_arrive(bar(K::OFREE));
            const unsigned bad = *const_cast<const volatile unsigned*>(&p->bad);
            if (bad != 0) {
#pragma unroll 1
                for (int ct = ct0; ct < ct1; ++ct) {
                    const int qi = (p->two ? ct * a.pb : 0) + pos;
                    const int d0 = p->two ? 0 : ct * (D / 2), d1 = p->two ? D : d0 + D / 2;
                    float* part = part_slot<D>(a, blockIdx.x, p->t0 == 0) + ((p->two ? ct * kRows : 0) + r) * 4;
                    if (pos < a.pb && qi < p->nq)
                        add_back(*p, bad, qi, d0, d1, a.out.row(p->row + p->q0 + qi, (p->g + hw) * G + hl),
                                 p->parts == 1 ? nullptr : part);
                }
                __syncwarp();
            }
            if (p->parts > 1) {
#pragma unroll 1
                for (int ct = ct0; ct < ct1; ++ct) join(*p, ct);
            }
            ++pieces;
            pieces1 += p->two || both;
            release(n);
        }
    }

    // (results are in L2 when the CTA ends: pkv_paged_attention reads its q before its dependency wait)
    if (warp < kReady) __threadfence();
    // teardown: every role arrives from its own code path (non-.aligned barrier)
    __syncwarp();
    tc_fence_before();
    cta_bar_sync();
    if (warp == kMma) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(*tmem_slot, K::TMEM_COLS);
    }
}

// ------------------------------------------------------------------ host

constexpr size_t kTicketOff = 256;         // behind the error word
constexpr size_t kPartOff = kTicketOff + (size_t)kMaxCtas * 8 * sizeof(int);

template <int D, bool FP8, int HG>
cudaError_t launch(const Arg& a, unsigned grid, cudaStream_t st) {
    static std::atomic<uint64_t> set{0};
    return launch_pdl_bigsmem(set, masked_kernel<D, FP8, HG>, dim3(grid), dim3(kThreads), (size_t)Cfg<D, FP8, HG>::SMEM, st,
                              a);
}
template <int D, bool FP8>
cudaError_t launch_hg(const Arg& a, int hg, unsigned grid, cudaStream_t st) {
    return hg == 4 ? launch<D, FP8, 4>(a, grid, st) : hg == 2 ? launch<D, FP8, 2>(a, grid, st) : launch<D, FP8, 1>(a, grid, st);
}

}  // namespace masked

size_t masked_workspace_bytes() {
    return masked::kPartOff + (size_t)masked::kMaxCtas * 2 * masked::slot_floats(128) * sizeof(float);
}

cudaError_t launch_masked(const pkv_cache& c, const pkv_rows* q, const pkv_rows* out, float* lse, int64_t num_q_rows,
                          const int32_t* tables, int max_blocks, const int32_t* ctx_lens, const int32_t* q_lens,
                          const int64_t* q_starts, int num_seqs, int max_q_len, int window, int sinks, const int32_t* tree,
                          int tree_words, float scale, void* workspace, cudaStream_t st) {
    using namespace masked;
    const int sms = num_sms_current();
    if (sms <= 0 || !encoder()) return cudaErrorUnknown;
    const int G = q->num_heads / c.num_kv_heads;
    Arg a = {};
    const unsigned grid = (unsigned)std::min(sms, kMaxCtas);
    // As many kv-heads an item as their rows fit in a row tile (96 requests of 1024 keys, one query each, 32/8 heads of 128:
    // 70 us with 4, 82 with 1; FP8 66 and 93) ...
    const bool fp8 = c.kv_dtype == PKV_KV_FP8_E4M3;
    const int rows = std::min<int64_t>((int64_t)max_q_len * G, kRows);
    int hg = rows <= kRows / 4 && c.num_kv_heads % 4 == 0 ? 4 : rows <= kRows / 2 && c.num_kv_heads % 2 == 0 ? 2 : 1;
    // ... but fewer while there is still a CTA for every item (there are no more queries than a row tile has), as uncut items
    // need no join and cut ones a smaller: 1 request of 256, 4096 or 32k keys 11, 18 or 39 us with 1 against 16, 28 or 62
    // with 4; 32 of 1024 keys 29 with 2, 35 with 4.  Not for much FP8 work in 8 items and more, by the longest context that
    // there can be: there HG = 4's quicker tiles count for more (4 of 32k keys 77 us with 4, 91 with 1; below the limit, 16 of
    // 1024 keys 32 and 23).
    const int64_t keys = std::min<int64_t>((int64_t)max_blocks * kBlock, tree ? INT32_MAX : (int64_t)window + sinks + max_q_len);
    const int64_t heads = (int64_t)num_seqs * c.num_kv_heads;
    if (!(fp8 && heads / hg >= 8 && heads * keys > (int64_t)grid * kFp8Tiles * kCols))
        while (hg > 1 && heads * 2 / hg <= grid) hg /= 2;
    a.pb = kRows / hg / G;
    if (!make_map(&a.q, q, q->data, PKV_BF16, c.head_dim, num_q_rows, G, a.pb)) return cudaErrorInvalidValue;
    a.k_cache = (const uint8_t*)c.k_cache;
    a.v_cache = (const uint8_t*)c.v_cache;
    a.k_scales = c.k_scales;
    a.v_scales = c.v_scales;
    a.tables = tables;
    a.ctx_lens = ctx_lens;
    a.q_lens = q_lens;
    a.q_starts = q_starts;
    a.tree = (const uint32_t*)tree;
    a.out = View{(uint8_t*)out->data, out->token_stride * 2, out->head_stride * 2, out->num_heads};
    a.lse = lse;
    a.err = (int*)workspace;
    a.tickets = (int*)((uint8_t*)workspace + kTicketOff);
    a.partials = (float*)((uint8_t*)workspace + kPartOff);
    AttnParams dbg = {};
    fill_debug(dbg);
    a.wait_limit_ns = dbg.wait_limit_ns;
    a.hold = dbg.hold;
    a.num_blocks = c.num_blocks;
    a.num_q_rows = num_q_rows;
    a.max_blocks = max_blocks;
    a.num_seqs = num_seqs;
    a.max_q_len = max_q_len;
    a.Hq = q->num_heads;
    a.Hkv = c.num_kv_heads;
    a.group = G;
    a.tree_words = tree_words;
    a.window = window;
    a.sinks = sinks;
    a.scale_log2 = std::min(scale * kLog2e, FLT_MAX);     // (not infinite, so that a logit of 0 stays 0)
    if (fp8)
        return c.head_dim == 128 ? launch_hg<128, true>(a, hg, grid, st) : launch_hg<64, true>(a, hg, grid, st);
    return c.head_dim == 128 ? launch_hg<128, false>(a, hg, grid, st) : launch_hg<64, false>(a, hg, grid, st);
}

}  // namespace pkv
