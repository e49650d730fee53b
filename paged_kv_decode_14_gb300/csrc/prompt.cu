// Causal attention of packed prompts whose keys and values are rows, not
// pages, on the 5th-generation tensor cores.  Contract: include/pagedkv.h,
// pkv_prompt_attention.
//
// A work item is up to 256 query rows of one (sequence, kv-head): 2 x PB
// consecutive query positions, PB = floor(128 / G), times the G heads of the
// group, as two 128-row tiles (row r of a tile = position r / G, head r % G),
// so every key tile a CTA loads serves both.  Per key tile t (128 keys) and
// row tile i, with the reference maximum m of each row:
//   S_i[128 rows, 128 keys] = Q_i . K_t^T      (A and B K-major in shared memory)
//   P_i = 2^(S_i scale log2(e) - m), l += sum P_i    (one thread per row = TMEM lane)
//   O_i[128 rows, D] += P_i . V_t              (A = P from TMEM, B MN-major in shared memory)
// and out = O / l at the end.  m is set by the maximum of the row's first 32 keys
// (of its first tile where they are masked); after that no maximum is taken.  P
// is rounded to the inputs' type because both operands of one MMA have the same
// type.  bf16: m is four octaves above that maximum, and P below 2 has a clear
// top exponent bit, so one OR over the packed P of 64 keys tells whether any
// reaches 2.  fp16, whose range is short: m is nine octaves below it, and the
// largest bit pattern of 64 P tells whether any reaches 2^13, so that weights
// keep 11 bits down to 2^-22 of the one that set m.  Only then (a logit 5 or 4
// octaves above that one) m rises, by whole octaves (O and l are rescaled by
// exact powers of 2), and those P are computed again.
//
// Q, K and V tiles arrive by tensor copies (TMA) in the 128-byte swizzle,
// straight from strided rows: K-major operands for Q and K, an MN-major one
// for V, without a pass over the data.
//
// Roles (512 threads): warps 0-3 the softmax of row tile 0, warps 4-7 of row
// tile 1, warps 8-11 the epilogue of both, warp 12 the producer, warps 13 and
// 14 the MMA issuers of row tiles 0 and 1, warp 15 the plan and the V guard.
// Per tile issuer i runs  PV_i(t), first 64 keys as soon as their P is written,
// PV_i(t) rest, S_i(t + 1), as one block, in turns with the other (0, 1, 0, 1,
// ...): left alone, the MMAs of both interleave, both S finish together and the
// tensor core idles through two simultaneous softmaxes; in turns the row tiles
// stay half a period apart (8192 tokens of 32 heads, when this was measured:
// 361 us; the first half's PV ahead of the turn 395; no turns 440).  The last
// tile of an item is followed by the next item's first S.  One thread's tcgen05
// operations complete in order, so when S_i(t + 1) signals, PV_i(t) is done and
// O_i may be rescaled, and S_i(t + 1) overwrites P_i(t) only after PV_i(t) has
// read it.
//
// The V guard makes keys that some rows do not see harmless: a weight of 0
// times NaN or infinity is NaN, so rows of V past the sequence's end are
// cleared in shared memory, and non-finite values among the keys that only
// part of the item's rows see are replaced by 0 there and added back, row by
// row, when the result is written (from global memory: rare).
//
// The items that do not fill a round (few rows over many keys: all of them) have
// their key tiles laid end to end and cut into equal ranges, one per CTA; a cut
// item leaves partial (O, m, l) in the workspace, joined in order by a second
// kernel.  Every wait is bounded.
//
// Bound: a key tile of both row tiles takes about 2830 clocks, of which the MMAs
// are 2080 (the rest is the chain softmax -> PV -> next S of a row tile), and a
// change of item about 5000.  Measured (32/8 heads of 128, bf16): 8192 tokens
// 366 us = 1500 TFLOP/s over the visible pairs, 0.78 of the measured burst rate
// (354 to 374 over boxes: the power cap); 4 x 2048 tokens 130 us; 512-token chunks
// over 3 to 4 thousand keys 173 us; up to 33 rows over 32k keys (fp16) 72 us = 3.7
// TB/s.  All for logits of standard deviation 1: at 2, 3 and 5 a row of some warp
// is past m in many steps, and 4 x 2048 tokens take 228, 273 and 303 us.  At the
// clock that explains 8192 tokens, the tiles and changes of item of the busiest CTA
// leave some 20 us of 4 x 2048 and of the chunks unexplained (among it the first
// plan and chain, 8 us in a launch of one tile, and the join's launch).
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "rows.cuh"
#include "tc_ptx.cuh"

namespace pkv {
int num_sms_current();

namespace prompt {

using namespace ptx;
using rows::store32;
using rows::View;

constexpr int kRows = 128;                 // rows of a row tile (MMA M)
constexpr int kKeys = 128;                 // keys of a key tile
constexpr int kThreads = 512;
// Registers a thread: the launch gives every thread 128, and the roles' shares add up to as many.
constexpr int kRegsSoftmax = 160, kRegsEpilogue = 112, kRegsOther = 80;
static_assert(2 * kRegsSoftmax + kRegsEpilogue + kRegsOther == 4 * 128, "register file");
constexpr int kProducer = 12, kMma = 13, kGuard = 15;   // (0-7: softmax, 8-11: epilogue)
constexpr int kMinTiles = 2;               // key tiles that a CTA of a split range has at least
constexpr int kCutCost = 10;               // what cutting a round of items costs, in key tiles (about 14 us)
constexpr int kFlags = 8;                  // items whose "non-finite V" flags are kept
constexpr int kMaxSplit = 160;             // CTAs of a split launch (two workspace slots each)
constexpr int kPieces = 4;                 // pieces of work the producer may be ahead

struct Join;
struct Arg {
    CUtensorMap q, k, v;
    View vrows, out;                       // V rows again, for the guard's slow path
    float* lse;
    const int32_t *q_lens, *kv_lens;
    const int64_t *q_starts, *kv_starts;
    int* err;
    float* partials;                       // split launches: [CTA][2] slots
    Join* joins;                           // and [CTA]
    uint64_t wait_limit_ns;
    const int* hold;
    int64_t num_q_rows, num_kv_rows;
    int num_seqs, max_q_len, Hq, Hkv, group;
    int pb;                                // query positions of a row tile
    uint32_t per_mul, per_shift;           // n / (2 pb) = (n * per_mul) >> per_shift for n < 2^31
    int split;                             // the items that do not come out even are cut along the keys
    int wide;                              // out's rows are 32-byte aligned
    float scale_log2;
};

// A partial slot: O as [D / 4][256 rows][4] fp32, then m and l, [256] each.
__host__ __device__ constexpr int slot_floats(int D) { return 2 * kRows * (D + 2); }

struct Seq {
    int64_t q0, k0;         // first rows
    int Q, L;               // 0 queries where the lengths are bad
};

// A piece of work: key tiles [t0, t1) of query block qb of sequence s, kv-head g.
struct Piece {
    Seq s;
    int g, q0, nq, T, t0, t1;
    bool two;               // row tile 1 holds rows
    bool whole;             // all of the item's tiles: the result is written at once
    bool end;               // no more work (the other fields are unset)
};
static_assert(sizeof(Piece) % 8 == 0, "aligned ring entries");

// What a CTA leaves for the join: the item that its last piece starts and others go on with.
struct Join {
    Piece p;
    int parts;              // CTAs that hold parts of it, from this one on; 0: none
    int pad;
};

template <int D>
struct Cfg {
    static constexpr int SLABS = D / 64;                  // 128-byte wide slabs of a row
    static constexpr int SLAB = kRows * 128;              // bytes of one slab of a tile
    static constexpr int TILE = SLABS * SLAB;
    static constexpr int NSK = D == 128 ? 2 : 4;          // K ring depth
    static constexpr int NSV = D == 128 ? 3 : 4;          // V ring depth
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + 2 * TILE;
    static constexpr int OFF_V = OFF_K + NSK * TILE;
    static constexpr int OFF_BAR = OFF_V + NSV * TILE;
    // barriers: KFULL[NSK] KEMPTY[NSK] VFULL[NSV] VREADY[NSV] VEMPTY[NSV], then pairs by row tile
    static constexpr int KFULL = 0, KEMPTY = NSK, VFULL = 2 * NSK, VREADY = VFULL + NSV, VEMPTY = VREADY + NSV,
                         SFULL = VEMPTY + NSV, PFA = SFULL + 2, PFB = SFULL + 4, QFULL = SFULL + 6,
                         QEMPTY = SFULL + 8, ODONE = SFULL + 10, OFREE = SFULL + 12, LREADY = SFULL + 14,
                         PVA = SFULL + 16, TURN = SFULL + 18, PCFULL = SFULL + 20, PCEMPTY = PCFULL + kPieces,
                         DRAIN = PCEMPTY + kPieces;
    static constexpr int NBAR = DRAIN + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;   // tmem address, abort flags
    static constexpr int OFF_FLAG = OFF_MISC + 16;        // int[kFlags]
    static constexpr int OFF_INV = OFF_FLAG + 4 * kFlags;     // float[2][kRows]: 1 / l
    static constexpr int OFF_PIECE = OFF_INV + 8 * kRows;     // Piece[kPieces]
    static constexpr int SMEM = OFF_PIECE + kPieces * (int)sizeof(Piece);
    static constexpr int COL_O = 2 * kKeys;
    static constexpr int TMEM_COLS = 512;
    static_assert(COL_O + 2 * D <= TMEM_COLS, "tensor memory budget");
    static_assert(SMEM <= 232448, "shared memory budget");
};

// ------------------------------------------------------------------ work

// The plan of a launch, made by one warp of every CTA alike (its V guard).  Items are dealt in the order of their key tiles, most
// first, whatever sequence they are of: the first `whole` of them as a whole,
// every CTA the same number in serpentine rounds; and (split launches) the key
// tiles of the rest, fewer items than CTAs, laid end to end and cut into equal
// ranges.  So long and short sequences, a last round that is not full and few
// rows over long contexts all leave the CTAs within a tile or so of each other.
// (4 prompts of 2048: in the order of the sequences 172 us, by tiles 152.)
//
// The items of a sequence with at least tau tiles are its last blocks, and
// their number has a closed form, so no list is kept: a lane stands for `chunk`
// consecutive sequences (one where there are at most 32).
struct Plan {
    const Arg& a;
    int lane, chunk, grid;
    int64_t rows_q, rows_k;     // packed rows before this lane's sequences
    Seq one;                    // this lane's sequence, where it has one
    int items, whole;           // all items; those dealt as a whole
    int tau, base, upto;        // the level being dealt: its tiles, items with more, items with as many or more
    int units, ctas;            // the rest: key tiles, CTAs that share them
    int each_cta, longer;       // a CTA's units, and how many CTAs have one more
    int mine, before;           // of them this lane's and earlier lanes'

    __device__ __forceinline__ Plan(const Arg& a_, int lane_, int grid_) : a(a_), lane(lane_), grid(grid_) {}
    __device__ __forceinline__ int per() const { return 2 * a.pb; }
    __device__ __forceinline__ int div_per(uint32_t n) const { return (int)(((uint64_t)n * a.per_mul) >> a.per_shift); }
    __device__ __forceinline__ int blocks(const Seq& s) const { return div_per(s.Q + per() - 1); }
    // key tiles of query block blk: up to its last row's limit
    __device__ __forceinline__ int tiles(const Seq& s, int blk) const {
        const int keys = s.L - s.Q + min((blk + 1) * per(), s.Q);
        return keys > 0 ? (keys + kKeys - 1) / kKeys : 0;
    }
    // query blocks with at least t tiles
    __device__ __forceinline__ int blocks_of(const Seq& s, int t) const {
        const int n = blocks(s);
        if (t <= 0) return n;
        if (t > (s.L + kKeys - 1) / kKeys) return 0;
        const int need = (t - 1) * kKeys + 1 - s.L + s.Q;    // queries up to the block's end, at least (<= Q)
        return need <= 0 ? n : n - div_per(need - 1);
    }
    // f(sequence number, sequence) for this lane's sequences; bad lengths and rows outside the tensors: Q = 0
    template <typename F>
    __device__ __forceinline__ void each(F f, bool report = false) const {
        const int b0 = lane * chunk;
        if (chunk == 1 && !report) {
            if (b0 < a.num_seqs) f(b0, one);
            return;
        }
        int64_t q = rows_q, k = rows_k;
        for (int b = b0; b < min(b0 + chunk, a.num_seqs); ++b) {
            Seq s;
            s.Q = a.q_lens[b];
            s.L = a.kv_lens[b];
            s.q0 = a.q_starts ? a.q_starts[b] : q;
            s.k0 = a.kv_starts ? a.kv_starts[b] : k;
            q += max(s.Q, 0);
            k += max(s.L, 0);
            if (s.Q < 0 || s.Q > a.max_q_len || s.L < 0 || s.q0 < 0 || s.k0 < 0 || s.q0 > a.num_q_rows - s.Q ||
                s.k0 > a.num_kv_rows - s.L) {
                if (report && (s.Q != 0 || s.L < 0)) raise_error(a.err, PKV_DEVERR_LENGTH);
                s.Q = 0;
                s.L = max(s.L, 0);
            }
            f(b, s);
        }
    }
    template <typename V>
    __device__ __forceinline__ V scan(V x) const {           // the sum over earlier lanes
        V y = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const V z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        return y - x;
    }
    __device__ __forceinline__ int count(int t) const {      // items with at least t tiles
        int n = 0;
        each([&](int, const Seq& s) { n += blocks_of(s, t); });
        return __reduce_add_sync(0xffffffffu, n) * a.Hkv;
    }
    // The level that holds this item: the most tiles t with more than `item` items of at least t, at
    // or below the present level (the next one, mostly; else a search -- stepping through 64 levels
    // took a join of 8k rows 170 us).  One call of count: every copy of its code comes from L2.
    __device__ __forceinline__ void level(int item) {
        if (item < upto) return;
        int lo = 0, hi = tau - 1;                            // (count(0) is all of them, count(tau) is upto)
        base = upto;
        upto = items;
        for (int t = hi; lo < hi; t = (lo + hi + 1) >> 1) {
            const int n = count(t);
            if (n > item) {
                lo = t;
                upto = n;
            } else {
                hi = t - 1;
                base = n;
            }
        }
        tau = lo;
    }
    // before the first level: above the most tiles of any item
    __device__ __forceinline__ void top() {
        int m = -1, n = 0;
        each([&](int, const Seq& s) {
            if (s.Q > 0) m = max(m, tiles(s, blocks(s) - 1));
            n += blocks(s);
        });
        items = __reduce_add_sync(0xffffffffu, n) * a.Hkv;
        tau = __reduce_max_sync(0xffffffffu, m) + 1;
        base = upto = 0;
    }
    __device__ __forceinline__ void begin() {
        chunk = (a.num_seqs + 31) / 32;
        rows_q = rows_k = 0;
        int64_t q = 0, k = 0;
        for (int b = lane * chunk; b < min((lane + 1) * chunk, a.num_seqs); ++b) {
            q += max(a.q_lens[b], 0);
            k += max(a.kv_lens[b], 0);
        }
        rows_q = scan(q);
        rows_k = scan(k);
        one = Seq{0, 0, 0, 0};
        each([&](int, const Seq& s) { one = s; }, true);     // (reads the lengths)
        top();
        whole = a.split ? items / grid * grid : items;
        units = ctas = 0;
    }
    // the rest's shares; leaves the level at the rest's first item's
    __device__ __forceinline__ void begin_rest() {
        if (whole == items) return;                          // (also the second time)
        level(whole);
        int n = 0;
        rest([&](int, const Seq&, int, int, int w) { n += w; });
        before = scan(n);
        mine = n;
        units = __reduce_add_sync(0xffffffffu, n);
        ctas = min(grid, max(units / kMinTiles, items - whole));
        each_cta = units / ctas;                             // (every item has a unit: at least 1)
        longer = units - each_cta * ctas;
        // a round of whole items takes as long as its first, the longest; cutting it takes an equal
        // share, and about kCutCost tiles more for the parts and their join
        if (tau <= units / grid + kCutCost) {
            ctas = 0;
            whole = items;
        }
    }
    // f(sequence number, sequence, block, first head, units of the block's heads from there on) for the
    // rest's items among this lane's, given the level of the first of them
    template <typename F>
    __device__ __forceinline__ void rest(F f) const {
        int n = 0;
        each([&](int, const Seq& s) { n += (blocks_of(s, tau) - blocks_of(s, tau + 1)) * a.Hkv; });
        int left = whole - base - scan(n);                   // of this level dealt as a whole, from this lane on
        each([&](int b, const Seq& s) {
            const int more = blocks_of(s, tau + 1), level_items = (blocks_of(s, tau) - more) * a.Hkv;
            const int taken = more * a.Hkv + min(max(left, 0), level_items);
            left -= level_items;
            int g = taken % a.Hkv;
            for (int blk = blocks(s) - 1 - taken / a.Hkv; blk >= 0; --blk, g = 0)
                f(b, s, blk, g, (a.Hkv - g) * max(tiles(s, blk), 1));
        });
    }
    __device__ __forceinline__ void fill(Piece& p, const Seq& s, int blk, int g) const {
        p.s = s;
        p.g = g;
        p.q0 = blk * per();
        p.nq = min(per(), s.Q - p.q0);
        p.two = p.nq > a.pb;
        p.T = tiles(s, blk);
        p.t0 = 0;
        p.t1 = p.T;
        p.whole = true;
        p.end = false;
    }
    // (the piece that one lane has found, to all of them)
    __device__ __forceinline__ void share(Piece& p, bool mine_) const {
        const int from = __ffs(__ballot_sync(0xffffffffu, mine_)) - 1;
        int* w = reinterpret_cast<int*>(&p);
#pragma unroll
        for (int x = 0; x < (int)sizeof(Piece) / 4; ++x) w[x] = __shfl_sync(0xffffffffu, w[x], from);
    }
    // item j < whole
    __device__ __forceinline__ void item(int j, Piece& p) {
        level(j);
        int n = 0;
        each([&](int, const Seq& s) { n += (blocks_of(s, tau) - blocks_of(s, tau + 1)) * a.Hkv; });
        int r = j - base - scan(n);
        const bool here = r >= 0 && r < n;
        if (here)
            each([&](int, const Seq& s) {
                const int more = blocks_of(s, tau + 1), m = (blocks_of(s, tau) - more) * a.Hkv;
                if (r >= 0 && r < m) fill(p, s, blocks(s) - 1 - more - r / a.Hkv, r % a.Hkv);
                r -= m;
            });
        share(p, here);
    }
    // the rest's unit u, and up to `room` units of its item from there on; the level must be that of `whole`
    __device__ __forceinline__ void unit(int u, int room, Piece& p) const {
        int r = u - before;
        const bool here = r >= 0 && r < mine;
        bool found = false;
        rest([&](int, const Seq& s, int blk, int g, int w) {
            if (here && !found && r < w) {
                found = true;
                fill(p, s, blk, g + r / max(tiles(s, blk), 1));
                p.t0 = r % max(p.T, 1);
                p.t1 = min(p.t0 + room, p.T);
                p.whole = p.t0 == 0 && p.t1 == p.T;
            }
            r -= w;
        });
        share(p, here);
    }
    __device__ __forceinline__ int range(int c) const { return each_cta * c + min(c, longer); }
    // the CTA whose range ends at or behind unit u, the first one
    __device__ __forceinline__ int cta_of_end(int u) const {
        const int head = (each_cta + 1) * longer;
        return (u <= head ? (u + each_cta) / (each_cta + 1) : longer + (u - head + each_cta - 1) / each_cta) - 1;
    }
};

// A CTA's pieces in order: its whole items, then its range of the rest (planned
// only then, behind the whole items' work).
struct Walk {
    int round, u, end;
    int parts;                  // CTAs that share the item that the last piece starts, from this one on (0: none)
    __device__ __forceinline__ void start() { round = parts = 0; }
    __device__ __forceinline__ bool next(Plan& plan, Piece& p) {
        const int grid = plan.grid, c = blockIdx.x;
        if (round >= 0) {
            const int64_t j = (int64_t)round * grid + ((round & 1) ? grid - 1 - c : c);
            ++round;
            if (j >= plan.whole) plan.begin_rest();       // (which may find them better dealt as a whole)
            if (j < plan.whole) {
                plan.item((int)j, p);
                return true;
            }
            round = -1;
            u = end = 0;
            if (c < plan.ctas) {
                u = plan.range(c);
                end = plan.range(c + 1);
            }
        }
        if (u >= end) return false;
        plan.unit(u, end - u, p);
        if (p.t0 == 0 && p.t1 < p.T) {
            parts = plan.cta_of_end(u + p.T) - c + 1;
        }
        u += max(p.t1 - p.t0, 1);
        return true;
    }
};

// ------------------------------------------------------------------ PTX pieces of this kernel

struct Ctl {
    volatile int* abort;
    int* err;
    uint64_t limit;
};
// (inlined: a call would keep ptxas from giving the roles registers of their own)
__device__ __forceinline__ bool wait_spin(uint32_t bar, uint32_t parity, volatile int* abort, int* err, uint64_t limit) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63) == 0) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > limit) {
                raise_error(err, PKV_DEVERR_TIMEOUT);
                *abort = 1;
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const Ctl& c) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_spin(bar, parity, c.abort, c.err, c.limit);
}

// A box of a 3-D tensor (dim, head, token) -> shared memory.
__device__ __forceinline__ void tensor_g2s(uint32_t dst, const CUtensorMap* map, int d, int h, int t, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
            dst),
        "l"(map), "r"(d), "r"(h), "r"(t), "r"(bar)
        : "memory");
}

// Shared-memory matrix descriptor of a 128-byte-swizzled operand.  K-major: sbo = bytes between
// groups of 8 rows (lbo unused).  MN-major: lbo = bytes between 64-element slabs, sbo between groups of 8 k.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// The issuer's operations run in warp-uniform code with one lane's predicate: in code that one lane
// runs alone, every descriptor is moved to a uniform register first, which cost ~107 clocks a MMA
// against the 64 that the tensor core needs for it.
__device__ __forceinline__ void mma_ss(bool lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"((uint32_t)lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(bool lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"((uint32_t)lead)
        : "memory");
}
__device__ __forceinline__ void commit(bool lead, uint32_t bar) {
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
        "r"((uint32_t)lead)
        : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2pack(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void f2unpack(uint64_t r, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t f2fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred P;\nelect.sync _|P, 0xffffffff;\nselp.b32 %0, 1, 0, P;\n}\n" : "=r"(p));
    return p != 0;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
struct Type;
template <>
struct Type<__nv_bfloat16> {
    static constexpr uint32_t INF = 0x7f80u;              // exponent bits of infinities and NaN
    static constexpr float HEADROOM = 4.f;                // octaves of m above the logit it is set by
    // |m| from which its roundings (half of fp32's step at m each, up to three of them) may leave P, l or O
    // their range: 2^29, three times 16 octaves below it
    static constexpr float LIMIT = 0x1p29f;
    // any P of 64 (two a word) at 2 or above: the top exponent bit
    static __device__ __forceinline__ bool high(const uint32_t (&v)[32]) {
        uint32_t any[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int x = 4; x < 32; ++x) any[x & 3] |= v[x];
        return ((any[0] | any[1] | any[2] | any[3]) & 0x40004000u) != 0;
    }
    static constexpr uint32_t id(int M, int N, bool b_mn) { return idesc_bf16_f32(M, N, false, b_mn); }
    static __device__ __forceinline__ float get(const uint8_t* p) { return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p)); }
};
template <>
struct Type<__half> {
    static constexpr uint32_t INF = 0x7c00u;
    static constexpr float HEADROOM = -9.f;               // (P = 2^9 there: 11 bits down to 2^-14)
    static constexpr float LIMIT = 0x1p26f;               // three times 2 octaves below it: P from 2^3 to 2^15
    // at 2^13 or above: the largest bit pattern (P has no sign), whose halves carry into the sign's place
    static __device__ __forceinline__ bool high(const uint32_t (&v)[32]) {
        uint32_t any[2] = {v[0], v[1]};
#pragma unroll
        for (int x = 2; x < 32; x += 4) {
            any[0] = __vimax3_u16x2(any[0], v[x], v[x + 1]);
            if (x + 2 < 32) any[1] = __vimax3_u16x2(any[1], v[x + 2], v[x + 3]);
        }
        return ((__vmaxu2(any[0], any[1]) + 0x10001000u) & 0x80008000u) != 0;
    }
    static constexpr uint32_t id(int M, int N, bool b_mn) { return idesc_f16_f32(M, N, false, b_mn); }
    static __device__ __forceinline__ float get(const uint8_t* p) { return __half2float(*reinterpret_cast<const __half*>(p)); }
};

// ------------------------------------------------------------------ kernel

// (split) where a part of an item goes: the part that starts the item is its CTA's last piece (slot
// 1), any other its CTA's first (slot 0).
template <int D>
__device__ __forceinline__ float* part_slot(const Arg& a, const Piece& p) {
    return a.partials + ((size_t)blockIdx.x * 2 + (p.t0 == 0 ? 1 : 0)) * slot_floats(D);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ Arg a) {
    using K = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];     // (the swizzle needs it; checked below)
    const uint32_t sb = smem_u32(smem);
    // (the warp's number by a shuffle: known to be uniform, and with it the roles' control flow, which the
    // MMA issue needs -- 12 MMAs 926 -> 856 clocks)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    auto bar = [&](int i) -> uint32_t { return sb + K::OFF_BAR + 8 * i; };
    constexpr int NSK = K::NSK, NSV = K::NSV;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + K::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + K::OFF_MISC + 4);
    volatile int* drain_flag = reinterpret_cast<volatile int*>(smem + K::OFF_MISC + 8);   // (drain waits at the end)
    volatile int* nonfinite = reinterpret_cast<volatile int*>(smem + K::OFF_FLAG);
    float* inv_l = reinterpret_cast<float*>(smem + K::OFF_INV);
    const Ctl ctl{abort_flag, a.err, a.wait_limit_ns};

    if (tid == 0) {
        for (int i = 0; i < NSK; ++i) {
            mbar_init(bar(K::KFULL + i), 1);
            mbar_init(bar(K::KEMPTY + i), 2);             // both issuers release every tile
        }
        for (int i = 0; i < NSV; ++i) {
            mbar_init(bar(K::VFULL + i), 1);
            mbar_init(bar(K::VREADY + i), 1);
            mbar_init(bar(K::VEMPTY + i), 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(K::SFULL + i), 1);
            mbar_init(bar(K::PFA + i), 4);                // one arrival a softmax warp
            mbar_init(bar(K::PFB + i), 4);
            mbar_init(bar(K::QFULL + i), 1);
            mbar_init(bar(K::QEMPTY + i), 1);
            mbar_init(bar(K::ODONE + i), 1);
            mbar_init(bar(K::OFREE + i), 4);
            mbar_init(bar(K::LREADY + i), 4);
            mbar_init(bar(K::PVA + i), 1);
            mbar_init(bar(K::TURN + i), 1);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(bar(K::PCFULL + i), 1);
            mbar_init(bar(K::PCEMPTY + i), 15);           // every warp but the guard, which writes them
        }
        mbar_init(bar(K::DRAIN), 2);
        *abort_flag = 0;
        *drain_flag = 0;
        mbar_fence_init();
    }
    if (warp == kProducer && lane < 3)
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(lane == 0 ? &a.q : lane == 1 ? &a.k : &a.v) : "memory");
    if (warp == kGuard) {
        tmem_alloc(smem_u32(tmem_slot), K::TMEM_COLS);
        tmem_relinquish();
    }
    griddep_wait();
    if ((sb & 1023) != 0 && tid == 0) {
        raise_error(a.err, PKV_DEVERR_TIMEOUT);           // (never: the declaration above aligns it)
        *abort_flag = 1;
    }
    tc_fence_before();
    cta_bar_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // The pieces of work, found by the V guard and read here by the other warps: the n-th piece
    // (nullptr: a wait gave up), until its release.  The search costs registers and instruction
    // cache, which 15 warps that each did their own paid for in their loops.
    const Piece* ring = reinterpret_cast<const Piece*>(smem + K::OFF_PIECE);
    auto piece_at = [&](int n) -> const Piece* {
        return __all_sync(0xffffffffu, wait(bar(K::PCFULL + n % kPieces), (n / kPieces) & 1, ctl)) ? ring + n % kPieces
                                                                                                  : nullptr;
    };
    auto release = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(K::PCEMPTY + n % kPieces));
    };

    if (warp < 8) {
        // ------------------------------------------------ softmax of row tile i, thread r = row r
        regs_inc<kRegsSoftmax>();
        const int i = warp >> 2, r = tid & (kRows - 1);
        const int G = a.group, pos = r / G, hl = r - pos * G;
        const uint32_t lbase = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t scol = tmem + lbase + i * kKeys;   // S_i / P_i
        const uint32_t ocol = tmem + lbase + K::COL_O + i * D;
        const float sc = a.scale_log2;
        // every wait and every TMEM access is warp-uniform (tcgen05.ld / st are .aligned)
        auto wait_all = [&](uint32_t bb, uint32_t parity) { return __all_sync(0xffffffffu, wait(bb, parity, ctl)); };
        auto signal = [&](uint32_t bb) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bb);
        };
        bool ok = true;
        int scnt = 0, ocnt = 0;                           // this row tile's S tiles and items
        for (int n = 0; ok; ++n) {
            const Piece* p = piece_at(n);
            if (!p || p->end) break;
            if (i == 1 && !p->two) {
                release(n);
                continue;
            }
            const int t0 = p->t0, t1 = p->t1, q0 = p->q0 + i * a.pb, nq = p->nq - i * a.pb;
            const bool row_ok = pos < a.pb && pos < nq;
            const int shift = p->s.L - p->s.Q + q0;       // the last key that the row tile's first row sees
            // keys 0 .. lim are visible (rows of no query: everything, so that they ask for no mask)
            const int lim = row_ok ? shift + pos : 0x3fffffff;
            const int top_lim = shift + min(nq, a.pb);    // keys that any of its rows sees
            // m: the reference maximum (exp2 units), l: the sum of P
            float m = row_ok ? -INFINITY : 0.f, l = 0.f;
            for (int t = t0; t < t1; ++t, ++scnt) {
                if (!(ok = wait_all(bar(K::SFULL + i), scnt & 1))) break;
                tc_fence_after();
                const int rem = lim - t * kKeys;          // column c is visible iff c <= rem
                const bool masked = !__all_sync(0xffffffffu, rem >= kKeys - 1);
                uint32_t sa[32], sb_[32];
                tmem_ld32_async(scol, sa);
                // O_i *= alpha (exact powers of 2, or 1)
                auto rescale_o = [&](float alpha) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        tmem_ld16(ocol + c, o);
                        uint32_t v[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x) v[x] = __float_as_uint(o[x] * alpha);
                        tmem_st16u(ocol + c, v);
                    }
                    tmem_wait_st();
                };
                tmem_wait_ld_into(sa);
                // the largest visible S of columns [c0, c1)
                auto maximum = [&](int c0, int c1) -> float {
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = c0; c < c1; c += 32) {
                        uint32_t s[32];
                        tmem_ld32_async(scol + c, s);
                        tmem_wait_ld_into(s);
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            mx[x & 3] = fmaxf(mx[x & 3], x <= rem - c ? __uint_as_float(s[x]) : -INFINITY);
                    }
                    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                };
                if (!__all_sync(0xffffffffu, m > -INFINITY)) {
                    // no reference yet (a piece's first tile): the largest of the first 32 keys where all are seen, else
                    // of the tile.  (O and l are 0 so far, or NaN)
                    float top = -INFINITY;
                    if (!masked) {
#pragma unroll
                        for (int x = 0; x < 32; x += 2) top = max3(top, __uint_as_float(sa[x]), __uint_as_float(sa[x + 1]));
                    }
                    if (!__all_sync(0xffffffffu, top > -INFINITY)) top = maximum(0, kKeys);
                    if (m == -INFINITY) m = top * sc + Type<T>::HEADROOM;
                    // (too far below 0 is only seen here: m rises)
                    if (row_ok && m <= -Type<T>::LIMIT && m > -INFINITY) raise_error(a.err, PKV_DEVERR_RANGE);
                }
                // (rare) a P of 64 keys at column c reaches the limit: m rises by a whole number of octaves, and the P
                // written in this tile, O and l are scaled down by as many (exact but for what falls below
                // the type's range, far below the new maximum)
                auto raise_ref = [&](float target, int c) {
                    const float inc = target + Type<T>::HEADROOM > m ? ceilf(target + Type<T>::HEADROOM - m) : 0.f;
                    const int k = (int)fminf(inc, 127.f);
                    const float alpha = k < 127 ? __uint_as_float((uint32_t)(127 - k) << 23) : 0.f;
                    if (c > 0) {                          // the first half's P is being used: it ends in O
                        wait_all(bar(K::PVA + i), scnt & 1);
                        tc_fence_after();
                    }
                    if (t > t0 || c > 0) rescale_o(alpha);
                    l *= alpha;
                    m += inc;
                };
                // P of 32 keys at column c, two per packed fp32 operation (the even key in the low half);
                // adds them to acc.  (Rows with nothing visible so far keep m = -inf: all their P are masked.)
                const uint64_t sc2 = f2pack(__float_as_uint(sc), __float_as_uint(sc));
                auto neg_m = [&] {
                    const float nm = m == -INFINITY ? 0.f : -m;
                    return f2pack(__float_as_uint(nm), __float_as_uint(nm));
                };
                auto emit = [&](const uint32_t (&s)[32], int c, uint32_t* v, uint64_t& acc, uint64_t nm2, auto mask) {
                    uint64_t ca = 0, cb = 0;
#pragma unroll
                    for (int x = 0; x < 32; x += 2) {
                        float x0, x1;
                        f2unpack(f2fma(f2pack(s[x], s[x + 1]), sc2, nm2), x0, x1);
                        float p0 = exp2_fast(x0), p1 = exp2_fast(x1);
                        if constexpr (decltype(mask)::value) {
                            p0 = x <= rem - c ? p0 : 0.f;
                            p1 = x + 1 <= rem - c ? p1 : 0.f;
                        }
                        if ((x >> 1) & 1) cb = f2add(cb, f2pack(__float_as_uint(p0), __float_as_uint(p1)));
                        else ca = f2add(ca, f2pack(__float_as_uint(p0), __float_as_uint(p1)));
                        v[x >> 1] = pack2<T>(p0, p1);
                    }
                    acc = f2add(acc, f2add(ca, cb));
                };
                // The P of 64 keys is written once none is known to reach the limit.  True: written.
                auto write = [&](uint64_t acc, int c, const uint32_t (&v)[32], bool force) -> bool {
                    const bool high = Type<T>::high(v);
                    if (__any_sync(0xffffffffu, row_ok && high) && !force) return false;
                    tmem_st32u(scol + (c >> 1), v);
                    float a0, a1;
                    f2unpack(acc, a0, a1);
                    l += a0 + a1;                         // (behind the store)
                    tmem_wait_st();
                    return true;
                };
                // 64 keys at column c, masked; a second time, with m raised, where the first is too large
                // (NaN logits pass then).  A second half that no row sees is not read by the PV.
                auto careful = [&](int c) {
                    if (c > 0 && c >= top_lim - t * kKeys) return;
                    for (bool force = false;; force = true) {
                        uint32_t v[32];
                        uint64_t acc = 0;
                        const uint64_t nm2 = neg_m();
                        tmem_ld32_async(scol + c, sa);
                        tmem_wait_ld_into(sa);
                        tmem_ld32_async(scol + c + 32, sb_);
                        emit(sa, c, v, acc, nm2, std::true_type{});
                        tmem_wait_ld_into(sb_);
                        emit(sb_, c + 32, v + 16, acc, nm2, std::true_type{});
                        if (write(acc, c, v, force)) break;
                        const float top = maximum(c, c + 64);
                        raise_ref(row_ok ? top * sc : -INFINITY, c);
                    }
                };
                // (one copy of either path: the instruction cache holds little more than a tile's code)
#pragma unroll 1
                for (int c = 0; c < kKeys; c += 64) {
                    bool done = false;
                    if (!masked) {                        // loads in flight behind the arithmetic
                        uint32_t v[32];
                        uint64_t acc = 0;
                        const uint64_t nm2 = neg_m();
                        tmem_ld32_async(scol + c + 32, sb_);
                        emit(sa, c, v, acc, nm2, std::false_type{});
                        tmem_wait_ld_into(sb_);
                        tmem_ld32_async(scol + 64, sa);   // (for the second half; after it, for nothing)
                        emit(sb_, c + 32, v + 16, acc, nm2, std::false_type{});
                        tmem_wait_ld_into(sa);
                        done = write(acc, c, v, false);
                    }
                    if (!done) {
                        careful(c);
                        tmem_ld32_async(scol + 64, sa);
                        tmem_wait_ld_into(sa);
                    }
                    // P of the first 64 keys: their PV may run while the rest is computed
                    signal(bar(K::PFA + i) + (c ? 8 * (K::PFB - K::PFA) : 0));
                }
            }
            if (!ok) break;
            // (a reference so large that fp32 cannot place the weights beside it is reported)
            const float size = fabsf(m);
            if (row_ok && size >= Type<T>::LIMIT && size < INFINITY) raise_error(a.err, PKV_DEVERR_RANGE);
            // this piece's sums go to the epilogue (1 / l) and to memory (lse, or the part's m and l)
            const bool tiles = t1 > t0, sees = lim >= 0;
            // (an item of a single tile gets here before its PV: the epilogue may still hold the last item's)
            if (tiles && ocnt++ > 0 && !(ok = wait_all(bar(K::OFREE + i), ocnt & 1))) break;
            if (p->whole) {
                const int64_t row = p->s.q0 + q0 + pos;
                const int h = p->g * G + hl;
                if (row_ok && a.lse) a.lse[row * a.Hq + h] = sees ? (m + log2f(l)) * 0.693147180559945f : -INFINITY;
                if (tiles) {
                    inv_l[i * kRows + r] = 1.f / l;
                } else if (row_ok) {                      // no keys at all
                    uint8_t* dst = a.out.row(row, h);
                    for (int c = 0; c < D * 2; c += 16) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
                }
            } else {
                float* slot = part_slot<D>(a, *p);
                slot[(size_t)2 * kRows * D + i * kRows + r] = m;
                slot[(size_t)2 * kRows * (D + 1) + i * kRows + r] = l;
            }
            if (tiles) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(K::LREADY + i));
            }
            release(n);
        }
    } else if (warp < kProducer) {
        // ------------------------------------------------ epilogue of both row tiles, thread r = row r
        regs_dec<kRegsEpilogue>();
        const int r = tid & (kRows - 1);
        const int G = a.group, pos = r / G, hl = r - pos * G;
        const uint32_t lbase = (uint32_t)((warp & 3) * 32) << 16;
        auto wait_all = [&](uint32_t bb, uint32_t parity) { return __all_sync(0xffffffffu, wait(bb, parity, ctl)); };
        // (one copy of the code, in loops: it runs once an item, from an instruction cache that holds the
        // softmax's by then; unrolled it took 5 thousand clocks a row tile)
        uint32_t phase = 0;                               // of either row tile's items, as bits
        int item = 0;                                     // the CTA's items with tiles
        bool ok = true;
        for (int n = 0; ok; ++n) {
            const Piece* at = piece_at(n);
            if (!at || at->end) break;
            const Piece p = *at;
            release(n);
            if (p.t1 == p.t0) continue;
            const int it = item++;
#pragma unroll 1
            for (int i = 0; i < (p.two ? 2 : 1); ++i) {
                const uint32_t ocol = tmem + lbase + K::COL_O + i * D;
                const int qi = p.q0 + i * a.pb + pos;
                const bool row_ok = pos < a.pb && qi < p.q0 + p.nq;
                const int lim = p.s.L - p.s.Q + qi;
                if (!(ok = wait_all(bar(K::LREADY + i), (phase >> i) & 1))) break;
                const float inv = lim >= 0 ? inv_l[i * kRows + r] : 0.f;
                if (!(ok = wait_all(bar(K::ODONE + i), (phase >> i) & 1))) break;
                phase ^= 1u << i;
                tc_fence_after();
                // infinities and NaN that the guard took out of V, for the rows that see them
                const bool fix = nonfinite[it & (kFlags - 1)] != 0;
                uint8_t* dst = a.out.row(p.s.q0 + qi, p.g * G + hl);
                float* slot = part_slot<D>(a, p) + (i * kRows + r) * 4;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32(ocol + c, o);
                    if (c + 32 == D) {                    // O_i read: the next item's first PV may overwrite it
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(K::OFREE + i));
                    }
                    if (fix && row_ok) {
                        const int first = max(p.s.L - p.s.Q + p.q0 + 1, p.t0 * kKeys);
                        for (int j = first; j <= min(lim, p.t1 * kKeys - 1); ++j) {
                            const uint8_t* v = a.vrows.row(p.s.k0 + j, p.g) + c * 2;
#pragma unroll
                            for (int x = 0; x < 32; ++x) {
                                const float f = Type<T>::get(v + 2 * x);
                                if (!(fabsf(f) < INFINITY)) o[x] += f;
                            }
                        }
                    }
                    if (!p.whole) {
#pragma unroll
                        for (int x = 0; x < 32; x += 4)
                            *reinterpret_cast<float4*>(slot + (size_t)((c + x) / 4) * 2 * kRows * 4) =
                                make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
                    } else if (row_ok) {
                        uint32_t v[16];
#pragma unroll
                        for (int x = 0; x < 32; x += 2) v[x >> 1] = lim >= 0 ? pack2<T>(o[x] * inv, o[x + 1] * inv) : 0u;
                        if (a.wide) {
                            store32(dst + c * 2, v);
                            store32(dst + c * 2 + 32, v + 8);
                        } else {
#pragma unroll
                            for (int x = 0; x < 16; x += 4)
                                *reinterpret_cast<uint4*>(dst + c * 2 + x * 4) = make_uint4(v[x], v[x + 1], v[x + 2], v[x + 3]);
                        }
                    }
                }
            }
        }
    } else {
        regs_dec<kRegsOther>();
        if (warp == kProducer) {
            // -------------------------------------------- tensor copies: Q tiles, K and V tiles in order
            bool ok = true;
            int nk = 0, nv = 0, nq[2] = {0, 0};           // copies issued: K, V and Q tiles
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
            // one lane: the copies of a piece's tiles
            auto produce = [&](const Piece& p) -> bool {
                if (p.t1 == p.t0) return true;
                for (int i = 0; i < (p.two ? 2 : 1); ++i) {
                    if (nq[i] > 0 && !wait(bar(K::QEMPTY + i), (nq[i] - 1) & 1, ctl)) return false;
                    ++nq[i];
                    mbar_arrive_expect_tx(bar(K::QFULL + i), K::SLABS * a.pb * a.group * 128);
                    for (int s = 0; s < K::SLABS; ++s)
                        tensor_g2s(sb + K::OFF_Q + i * K::TILE + s * K::SLAB, &a.q, s * 64, p.g * a.group,
                                   (int)(p.s.q0 + p.q0 + i * a.pb), bar(K::QFULL + i));
                }
                for (int t = p.t0; t < p.t1; ++t) {
                    const int key = (int)(p.s.k0 + (int64_t)t * kKeys);
                    const int sk = nk % NSK, sv = nv % NSV;
                    if (nk >= NSK && !wait(bar(K::KEMPTY + sk), ((nk - NSK) / NSK) & 1, ctl)) return false;
                    ++nk;
                    mbar_arrive_expect_tx(bar(K::KFULL + sk), K::TILE);
                    for (int s = 0; s < K::SLABS; ++s)
                        tensor_g2s(sb + K::OFF_K + sk * K::TILE + s * K::SLAB, &a.k, s * 64, p.g, key, bar(K::KFULL + sk));
                    if (nv >= NSV && !wait(bar(K::VEMPTY + sv), ((nv - NSV) / NSV) & 1, ctl)) return false;
                    ++nv;
                    mbar_arrive_expect_tx(bar(K::VFULL + sv), K::TILE);
                    for (int s = 0; s < K::SLABS; ++s)
                        tensor_g2s(sb + K::OFF_V + sv * K::TILE + s * K::SLAB, &a.v, s * 64, p.g, key, bar(K::VFULL + sv));
                }
                return true;
            };
            for (int n = 0; __all_sync(0xffffffffu, ok); ++n) {
                const Piece* p = piece_at(n);
                if (!p || p->end) break;
                if (lane == 0) ok = produce(*p);
                release(n);
            }
            if (lane == 0) {
                // drain: every copy in flight lands before the CTA exits
                const Ctl drain{drain_flag, a.err, a.wait_limit_ns};
                for (int t = max(0, nk - NSK); t < nk; ++t) wait(bar(K::KFULL + t % NSK), (t / NSK) & 1, drain);
                for (int t = max(0, nv - NSV); t < nv; ++t) wait(bar(K::VFULL + t % NSV), (t / NSV) & 1, drain);
                for (int i = 0; i < 2; ++i)
                    if (nq[i] > 0) wait(bar(K::QFULL + i), (nq[i] - 1) & 1, drain);
            }
            __syncwarp();
        } else if (warp == kMma || warp == kMma + 1) {
            // -------------------------------------------- MMA issuer of row tile i
            const int i = warp - kMma;
            const bool lead = elect_one();                // (8% faster over all than lane == 0)
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);       // (known to be uniform)
            const uint32_t s_i = tm + __shfl_sync(0xffffffffu, i, 0) * kKeys;
            const uint32_t o_i = tm + K::COL_O + __shfl_sync(0xffffffffu, i, 0) * D;
            const uint32_t qbase = __shfl_sync(0xffffffffu, sb + K::OFF_Q + i * K::TILE, 0);
            auto wait_all = [&](uint32_t bb, uint32_t parity) { return __all_sync(0xffffffffu, wait(bb, parity, ctl)); };
            constexpr uint32_t idS = Type<T>::id(kRows, kKeys, false);
            constexpr uint32_t idPV = Type<T>::id(kRows, D, true);
            int nk = 0, nv = 0;                           // K and V tiles passed (ring slots, phases)
            int pcnt = 0, qcnt = 0, ocnt = 0, turn = 0;   // P tiles, Q tiles, results of this row tile; turns
            bool ok = true;
            auto wait_k = [&] { return wait_all(bar(K::KFULL + nk % NSK), (nk / NSK) & 1); };
            // S_i of the next K tile (waited for); last: the item's last, after which Q_i is free
            auto issue_s = [&](bool last) {
                const int sk = nk++ % NSK;
                const uint32_t kbase = __shfl_sync(0xffffffffu, sb + K::OFF_K + sk * K::TILE, 0);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k / 4) * K::SLAB + (k % 4) * 32;
                    mma_ss(lead, s_i, desc_sw128(qbase + off, 16, 1024), desc_sw128(kbase + off, 16, 1024), idS,
                           k > 0 ? 1u : 0u);
                }
                commit(lead, bar(K::SFULL + i));
                commit(lead, bar(K::KEMPTY + sk));
                if (last) commit(lead, bar(K::QEMPTY + i));
            };
            int n = 0;
            auto next = [&](Piece& x) {                   // the next piece with tiles
                for (;; ++n) {
                    const Piece* at = piece_at(n);
                    if (!at || at->end) return false;
                    x = *at;
                    release(n);
                    if (x.t1 > x.t0) break;
                }
                ++n;
                return true;
            };
            Piece p;
            bool more = next(p), begun = false;           // begun: this piece's first S is issued
            while (more && ok) {
                const int tiles = p.t1 - p.t0;
                if (i == 1 && !p.two) {
                    // no rows here: release this row tile's share of every slot once its tile has landed
                    for (int x = 0; x < tiles && ok; ++x, ++nk, ++nv) {
                        if (!(ok = wait_k())) break;
                        if (lead) mbar_arrive(bar(K::KEMPTY + nk % NSK));
                        if (!(ok = wait_all(bar(K::VREADY + nv % NSV), (nv / NSV) & 1))) break;
                        if (lead) mbar_arrive(bar(K::VEMPTY + nv % NSV));
                    }
                    more = next(p);
                    begun = false;
                    continue;
                }
                if (!begun) {
                    if (!(ok = wait_all(bar(K::QFULL + i), qcnt & 1)) || !(ok = wait_k())) break;
                    ++qcnt;
                    tc_fence_after();
                    issue_s(tiles == 1);
                }
                // keys that any row of this row tile sees, from the piece's first tile on
                const int last = p.s.L - p.s.Q + p.q0 + min(p.nq, (i + 1) * a.pb) - p.t0 * kKeys;
                Piece q;
                bool after = false, follow = false;       // another piece; this row tile has rows in it
                for (int x = 0; x < tiles; ++x, ++nv, ++pcnt) {
                    const bool end = x + 1 == tiles;
                    if (end) {
                        after = next(q);
                        follow = after && (i == 0 || q.two);
                    }
                    const int sv = nv % NSV;
                    const uint32_t vbase = __shfl_sync(0xffffffffu, sb + K::OFF_V + sv * K::TILE, 0);
                    const int steps = min(max((last - x * kKeys + 15) / 16, 1), kKeys / 16);   // 16 keys an MMA
                    auto pv = [&](int k0) {               // 64 keys (unrolled: 12 MMAs issue in 740 clocks, rolled in 1000)
                        if (steps == kKeys / 16) {
#pragma unroll
                            for (int k = k0; k < k0 + 4; ++k)
                                mma_ts(lead, o_i, s_i + k * 8, desc_sw128(vbase + k * 2048, K::SLAB, 1024), idPV,
                                       x > 0 || k > 0 ? 1u : 0u);
                        } else {
#pragma unroll 1
                            for (int k = k0; k < min(k0 + 4, steps); ++k)
                                mma_ts(lead, o_i, s_i + k * 8, desc_sw128(vbase + k * 2048, K::SLAB, 1024), idPV,
                                       x > 0 || k > 0 ? 1u : 0u);
                        }
                    };
                    if (!(ok = wait_all(bar(K::VREADY + sv), (nv / NSV) & 1))) break;
                    // an item's first PV starts O_i afresh: the last one's result has been read
                    if (x == 0 && ocnt > 0 && !(ok = wait_all(bar(K::OFREE + i), (ocnt - 1) & 1))) break;
                    // (what the turn needs is waited for before P, off the path from P to the next S)
                    if (follow && !(ok = wait_all(bar(K::QFULL + i), qcnt & 1))) break;
                    if ((!end || follow) && !(ok = wait_k())) break;
                    if (p.two) {
                        if ((i == 1 || turn > 0) && !(ok = wait_all(bar(K::TURN + i), (i == 1 ? turn : turn - 1) & 1))) break;
                        ++turn;
                    }
                    if (!(ok = wait_all(bar(K::PFA + i), pcnt & 1))) break;
                    tc_fence_after();
                    pv(0);
                    commit(lead, bar(K::PVA + i));
                    if (!(ok = wait_all(bar(K::PFB + i), pcnt & 1))) break;
                    tc_fence_after();
                    pv(4);
                    if (end) commit(lead, bar(K::ODONE + i));
                    commit(lead, bar(K::VEMPTY + sv));
                    if (!end) issue_s(x + 2 == tiles);
                    else if (follow) {
                        ++qcnt;
                        issue_s(q.t1 - q.t0 == 1);
                    }
                    // The turn passes when these MMAs are issued (D = 128: 358 us for 8k rows, 380 passed when they
                    // complete) or, with products half as long, complete (D = 64: 304 us, 315 when issued)
                    if (p.two) {
                        if constexpr (D == 64) commit(lead, bar(K::TURN + 1 - i));
                        else if (lead) mbar_arrive(bar(K::TURN + 1 - i));
                    }
                }
                if (!ok) break;
                ++ocnt;
                more = after;
                begun = follow;
                p = q;
            }
            commit(lead, bar(K::DRAIN));
            // every MMA issued has completed before TMEM is freed
            const Ctl drain{drain_flag, a.err, a.wait_limit_ns};
            wait(bar(K::DRAIN), 0, drain);
            __syncwarp();
        } else if (warp == kGuard) {
            // -------------------------------------------- the plan, and the V guard
            // A piece is planned while the one before it is worked on (planned by the producer between two
            // pieces' copies it held up each item by 3 to 8 thousand clocks).
            Plan plan(a, lane, gridDim.x);
            plan.begin();
            Walk w;
            w.start();
            int n = 0, item = 0, np = 0;                  // V tiles and items seen; pieces published
            auto publish = [&]() -> bool {
                Piece p = {};
                p.end = !w.next(plan, p);                 // (the whole warp; the same in every lane)
                if (np >= kPieces && !__all_sync(0xffffffffu, wait(bar(K::PCEMPTY + np % kPieces), ((np - kPieces) / kPieces) & 1, ctl)))
                    return false;
                if (lane == 0) {
                    const_cast<Piece*>(ring)[np % kPieces] = p;
                    mbar_arrive(bar(K::PCFULL + np % kPieces));
                }
                ++np;
                __syncwarp();
                return true;
            };
            bool ok = publish();
            for (int m = 0; ok; ++m) {
                const Piece& p = ring[m % kPieces];
                if (p.end) break;
                if (p.t1 == p.t0) {
                    ok = publish();
                    continue;
                }
                const int it = item++;
                // keys past `all` are not seen by every row of the item; L and beyond by none
                const int all = p.s.L - p.s.Q + p.q0;
                bool found = false;
                for (int t = p.t0; t < p.t1 && ok; ++t, ++n) {
                    const int sv = n % NSV;
                    if (!(ok = __all_sync(0xffffffffu, wait(bar(K::VFULL + sv), (n / NSV) & 1, ctl)))) break;
                    const int r0 = max(all + 1 - t * kKeys, 0), r1 = min(p.s.L - t * kKeys, kKeys);
                    if (t == p.t0 && lane == 0) nonfinite[it & (kFlags - 1)] = 0;
                    __syncwarp();
                    if (r0 < kKeys) {
                        // A short loop with few branches: code that runs once an item comes from L2, line by line (a
                        // loop with 8 loads in flight took 5 to 8 thousand clocks, single loads tested one by one 8
                        // to 12; a tile's MMAs take 2).  An exponent of all ones carries into the sign's place.
                        uint8_t* base = smem + K::OFF_V + sv * K::TILE;
                        constexpr uint32_t I = Type<T>::INF * 0x10001u, A = 0x80008000u - I;
#pragma unroll 1
                        for (int x = r0 * 8 + lane; x < r1 * 8; x += 2 * 32) {
                            uint32_t bad = 0;
#pragma unroll
                            for (int j = 0; j < 2; ++j)
#pragma unroll
                                for (int s = 0; s < K::SLABS; ++s) {
                                    const uint4 v = *reinterpret_cast<const uint4*>(base + s * K::SLAB + min(x + j * 32, r1 * 8 - 1) * 16);
                                    bad |= ((v.x & I) + A) | ((v.y & I) + A) | ((v.z & I) + A) | ((v.w & I) + A);
                                }
                            if (bad & 0x80008000u) {
                                found = true;
#pragma unroll 1
                                for (int j = 0; j < 2 * K::SLABS; ++j) {
                                    const int y = x + (j / K::SLABS) * 32;
                                    uint32_t* e = reinterpret_cast<uint32_t*>(base + (j % K::SLABS) * K::SLAB + y * 16);
                                    for (int z = 0; z < 4 && y < r1 * 8; ++z) {
                                        const uint32_t hit = ((e[z] & I) + A) & 0x80008000u;
                                        e[z] &= ~((hit >> 15) * 0xffffu);
                                    }
                                }
                            }
                        }
#pragma unroll 1
                        for (int x = r1 * 8 + lane; x < kKeys * 8; x += 32)
                            for (int s = 0; s < K::SLABS; ++s)
                                *reinterpret_cast<uint4*>(base + s * K::SLAB + x * 16) = make_uint4(0, 0, 0, 0);
                        if (__any_sync(0xffffffffu, found) && lane == 0) nonfinite[it & (kFlags - 1)] = 1;
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(K::VREADY + sv));
                    if (t == min(p.t0 + 1, p.t1 - 1)) ok = publish();   // (the copies are up to three tiles ahead)
                }
            }
            if (a.split && lane == 0) {
                Join join = {};
                if (ok && np > 1) {
                    join.p = ring[(np - 2) % kPieces];    // the last piece (the one behind it says `end`)
                    join.parts = w.parts;
                }
                a.joins[blockIdx.x] = join;
            }
        }
    }

    // teardown: every role arrives from its own code path (non-.aligned barrier)
    __syncwarp();
    tc_fence_before();
    cta_bar_sync();
    if (warp == kGuard) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, K::TMEM_COLS);
    }
}

// ------------------------------------------------------------------ join

// Joins the parts of the items that a split launch cut: CTA (c, y) takes the item whose first part
// CTA c left in its slot 1, rows 32 y .. 32 y + 31; a warp's lanes are rows (the slots' layout makes
// its loads contiguous) and warps share the dimensions.  Parts are added in the keys' order.
template <typename T, int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Arg a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x;
    griddep_wait();
    const Join& join = a.joins[c];
    const int parts = join.parts;
    if (parts == 0) return;
    const Piece p = join.p;
    const int R = blockIdx.y * 32 + lane, i = R / kRows, r = R % kRows;
    const int pos = r / a.group, hl = r - pos * a.group, qi = p.q0 + i * a.pb + pos;
    if (!(pos < a.pb && qi < p.q0 + p.nq) || (i == 1 && !p.two)) return;
    const float* slots = a.partials;
    auto slot = [&](int x) { return slots + ((size_t)x * 2 + (x == c ? 1 : 0)) * slot_floats(D); };
    float m = -INFINITY;
    for (int x = c; x < c + parts; ++x) m = fmaxf(m, slot(x)[(size_t)2 * kRows * D + R]);
    const float mref = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float o[D / 8];
#pragma unroll
    for (int d = 0; d < D / 8; ++d) o[d] = 0.f;
    for (int x = c; x < c + parts; ++x) {
        const float* s = slot(x);
        const float mx = s[(size_t)2 * kRows * D + R];
        const float f = mx == -INFINITY ? (s[(size_t)2 * kRows * (D + 1) + R] == 0.f ? 0.f : 1.f) : exp2f(mx - mref);
        l += f * s[(size_t)2 * kRows * (D + 1) + R];
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
            const float4 v = *reinterpret_cast<const float4*>(s + ((size_t)(warp * (D / 32) + d) * 2 * kRows + R) * 4);
            // (a part that saw nothing holds zeros, or non-finite values of V that its rows do see)
            const float g = mx == -INFINITY ? 1.f : f;
            o[4 * d] = fmaf(v.x, g, o[4 * d]);
            o[4 * d + 1] = fmaf(v.y, g, o[4 * d + 1]);
            o[4 * d + 2] = fmaf(v.z, g, o[4 * d + 2]);
            o[4 * d + 3] = fmaf(v.w, g, o[4 * d + 3]);
        }
    }
    const bool sees = p.s.L - p.s.Q + qi >= 0;
    const float inv = sees ? 1.f / l : 0.f;
    const int64_t row = p.s.q0 + qi;
    uint8_t* dst = a.out.row(row, p.g * a.group + hl) + warp * (D / 8) * 2;
#pragma unroll
    for (int d = 0; d < D / 8; d += 8) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = sees ? o[d + e] * inv : 0.f;
        *reinterpret_cast<uint4*>(dst + d * 2) =
            make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
    }
    if (warp == 0 && a.lse) a.lse[row * a.Hq + p.g * a.group + hl] = sees ? (m + log2f(l)) * 0.693147180559945f : -INFINITY;
}

// ------------------------------------------------------------------ host

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder() {
    static const Encode fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult st;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &st) != cudaSuccess ||
            st != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (Encode)p;
    }();
    return fn;
}

// Map of rows [tokens][heads][D] in boxes of 64 dims x `bh` heads x `bt` tokens.
bool make_map(CUtensorMap* m, const pkv_rows* r, const void* fallback, int dtype, int D, int64_t tokens, int bh, int bt) {
    const bool none = tokens < 1;                         // (nothing is ever copied: any valid map)
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)r->num_heads, (cuuint64_t)(none ? 1 : tokens)};
    // strides of dimensions of extent 1 are never used, but are checked
    const cuuint64_t strides[2] = {none || r->num_heads == 1 ? (cuuint64_t)D * 2 : (cuuint64_t)r->head_stride * 2,
                                   none || tokens == 1 ? (cuuint64_t)D * 2 : (cuuint64_t)r->token_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)bh, (cuuint32_t)bt}, one[3] = {1, 1, 1};
    return encoder()(m, dtype == PKV_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                     none ? const_cast<void*>(fallback) : r->data, dims, strides, box, one,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch(const Arg& a, unsigned grid, cudaStream_t st) {
    static std::atomic<uint64_t> set{0};
    cudaError_t e = launch_pdl_bigsmem(set, prompt_kernel<T, D>, dim3(grid), dim3(kThreads), (size_t)Cfg<D>::SMEM, st, a);
    if (e == cudaSuccess && a.split)
        e = launch_pdl(join_kernel<T, D>, dim3(grid, 2 * kRows / 32), dim3(256), (size_t)0, st, a);
    return e;
}

}  // namespace prompt

size_t prompt_workspace_bytes() { return (size_t)prompt::kMaxSplit * (2 * prompt::slot_floats(128) * sizeof(float) + sizeof(prompt::Join)); }

cudaError_t launch_prompt(const pkv_rows* q, const pkv_rows* k, const pkv_rows* v, const pkv_rows* out, float* lse,
                          int dtype, int head_dim, int64_t num_q_rows, int64_t num_kv_rows, const int32_t* q_lens,
                          const int32_t* kv_lens, const int64_t* q_starts, const int64_t* kv_starts, int num_seqs,
                          int max_q_len, float scale, void* workspace, int* err, cudaStream_t st) {
    using namespace prompt;
    const int sms = num_sms_current();
    if (sms <= 0 || !encoder()) return cudaErrorUnknown;
    const int G = q->num_heads / k->num_heads, Hkv = k->num_heads;
    Arg a = {};
    a.pb = kRows / G;
    if (!make_map(&a.q, q, q->data, dtype, head_dim, num_q_rows, G, a.pb)) return cudaErrorInvalidValue;
    if (!make_map(&a.k, k, q->data, dtype, head_dim, num_kv_rows, 1, kKeys)) return cudaErrorInvalidValue;
    if (!make_map(&a.v, v, q->data, dtype, head_dim, num_kv_rows, 1, kKeys)) return cudaErrorInvalidValue;
    auto view = [](const pkv_rows* r) {
        View x = {(uint8_t*)r->data, r->token_stride * 2, r->head_stride * 2, r->num_heads};
        return x;
    };
    a.vrows = view(v);
    a.out = view(out);
    a.lse = lse;
    a.q_lens = q_lens;
    a.kv_lens = kv_lens;
    a.q_starts = q_starts;
    a.kv_starts = kv_starts;
    a.err = err;
    a.joins = (Join*)workspace;                           // then the slots (kMaxSplit records: a multiple of 16 bytes)
    a.partials = (float*)((uint8_t*)workspace + kMaxSplit * sizeof(Join));
    AttnParams dbg = {};
    fill_debug(dbg);
    a.wait_limit_ns = dbg.wait_limit_ns;
    a.hold = dbg.hold;
    a.num_q_rows = num_q_rows;
    a.num_kv_rows = num_kv_rows;
    a.num_seqs = num_seqs;
    a.max_q_len = max_q_len;
    a.Hq = q->num_heads;
    a.Hkv = Hkv;
    a.group = G;
    a.scale_log2 = scale * kLog2e;
    a.wide = rows::wide(a.out);
    // at most this many items (their number depends on the lengths, which the host does not see)
    const int64_t per = 2 * a.pb;
    // (d <= 2^l, M = floor(2^(31 + l) / d) + 1: n M / 2^(31 + l) exceeds n / d by less than 2^-l <= 1 / d)
    a.per_shift = 31;
    while ((1u << (a.per_shift - 31)) < (uint32_t)per) ++a.per_shift;
    a.per_mul = (uint32_t)(((uint64_t)1 << a.per_shift) / per + 1);
    const int64_t items = Hkv * std::min<int64_t>((int64_t)num_seqs * ((max_q_len + per - 1) / per),
                                                  num_q_rows / per + num_seqs);
    if (items > 0x7fffffff) return cudaErrorInvalidValue;
    // Splitting pays (a second launch, parts written and read) where the items do not come out even
    // and some have several tiles; the units of the rest stay below 2^31.
    a.split = workspace != nullptr && num_kv_rows > 4 * kKeys && num_kv_rows < (1 << 30);
    const unsigned grid = (unsigned)(a.split ? std::min(sms, kMaxSplit) : std::min<int64_t>(std::max<int64_t>(items, 1), sms));
    if (dtype == PKV_BF16)
        return head_dim == 128 ? launch<__nv_bfloat16, 128>(a, grid, st) : launch<__nv_bfloat16, 64>(a, grid, st);
    return head_dim == 128 ? launch<__half, 128>(a, grid, st) : launch<__half, 64>(a, grid, st);
}

}  // namespace pkv
