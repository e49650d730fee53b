"""Caches and 64-bit results for the tests of masked attention over the cache (no test functions here)."""

import math

import torch

from paged_kv_decode_14_gb300 import _native as nat


def page_view(pool, heads, dim):
    """[block, kv head, 8-token group, chunk, token, element] of a cache buffer."""
    c = 16 // pool.element_size()
    return pool.view(pool.shape[0], heads, 2, dim // c, 8, c)


class Sequences:
    """Sequences in a cache of which every byte that no query sees is NaN, and every table entry that no query needs
    (whole: only those past the sequence's end) is out of range.  seen[b]: bool [Q, L], what each query sees."""

    def __init__(self, seen, heads, kv_heads, dim, dtype, seed=0, gaps=None, lead=0, plant=(), spread=1.0, whole=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.seen = [s.cuda() for s in seen]
        self.heads, self.kv_heads, self.dim, self.dtype = heads, kv_heads, dim, dtype
        self.q_lens = [s.shape[0] for s in seen]
        self.lens = [s.shape[1] for s in seen]
        starts, at = [], lead
        for b, n in enumerate(self.q_lens):
            starts.append(at)
            at += n + (gaps[b] if gaps else 0)
        self.starts, self.rows = starts, max(at, 1)
        need = [(n + 15) // 16 for n in self.lens]
        blocks = sum(need) + 3
        order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        wide = max(max(need), 1) + 1
        self.table = torch.full((len(need), wide), 1 << 30, dtype=torch.int32, device="cuda")
        fp8 = dtype == "fp8"
        shape = (blocks, kv_heads, 16 * dim)
        pools = []
        for _ in range(2):
            pools.append(torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda") if fp8 else
                         torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda"))
        self.scales = [None, None]
        if fp8:
            self.scales = [0.004 + 0.02 * torch.rand(blocks, kv_heads, generator=g, device="cuda") for _ in range(2)]
        self.values = []                     # per sequence: (K, V) as stored, fp64 [L, Hkv, D]
        at = 0
        for b, n in enumerate(self.lens):
            mine = order[at:at + need[b]]
            at += need[b]
            any_seen = self.seen[b].any(0) if n and self.q_lens[b] else torch.zeros(n, dtype=torch.bool, device="cuda")
            pos = any_seen.nonzero()[:, 0]
            used = torch.full((need[b],), whole, device="cuda")
            used[pos // 16] = True
            self.table[b, :need[b]] = torch.where(used, mine, self.table[b, :need[b]])
            blk = mine[pos // 16].long()
            kv = []
            for i in range(2):
                x = torch.randn(len(pos), kv_heads, dim, generator=g, device="cuda") * (spread if i == 0 else 1.0)
                for what, where, j, h, d, value in plant:
                    if what == b and where == i and any_seen[j]:
                        x[(pos == j).nonzero()[0, 0], h, d] = value
                if fp8:
                    s = self.scales[i][blk][..., None]
                    y = (x / s).clamp(-448, 448).to(torch.float8_e4m3fn)
                    stored, exact = y.view(torch.uint8), y.double() * s.double()
                else:
                    stored = x.bfloat16()
                    exact = stored.double()
                page_view(pools[i], kv_heads, dim)[blk, :, pos % 16 // 8, :, pos % 8, :] = stored.view(
                    len(pos), kv_heads, dim * stored.element_size() // 16, 16 // stored.element_size())
                full = torch.zeros(n, kv_heads, dim, dtype=torch.float64, device="cuda")
                full[pos] = exact
                kv.append(full)
            self.values.append(kv)
        self.cache = nat.PagedKVCache(blocks, kv_heads, dim, dtype, k=pools[0], v=pools[1], k_scales=self.scales[0],
                                      v_scales=self.scales[1])
        self.q = torch.randn(self.rows, heads, dim, generator=g, device="cuda").bfloat16()
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.t_lens, self.t_q = ints(self.lens), ints(self.q_lens)
        self.t_starts = torch.tensor(starts, dtype=torch.int64, device="cuda")
        self.max_q = max(1, max(self.q_lens))
        self.scale = dim ** -0.5
        self.inside = torch.zeros(self.rows, dtype=torch.bool, device="cuda")
        for b, n in enumerate(self.q_lens):
            self.inside[starts[b]:starts[b] + n] = True

    def reference(self):
        """(out, lse, bound on |error| of out, of lse, rows of sequences) in fp64."""
        out = torch.full(self.q.shape, math.nan, dtype=torch.float64, device="cuda")
        lse = torch.full(self.q.shape[:2], math.nan, dtype=torch.float64, device="cuda")
        e_out, e_lse = torch.zeros_like(out), torch.zeros_like(lse)
        grp = self.heads // self.kv_heads
        for b, (n, length) in enumerate(zip(self.q_lens, self.lens)):
            if n == 0:
                continue
            seen, rows = self.seen[b], slice(self.starts[b], self.starts[b] + n)
            for h in range(self.heads):
                k, v = (x[:, h // grp] for x in self.values[b])
                q = self.q[rows, h].double()
                x = (q @ k.t() * self.scale).masked_fill(~seen, -math.inf)
                z = torch.logsumexp(x, -1)
                some = seen.any(1)
                p = torch.where(seen, (x - torch.where(some, z, 0.0)[:, None]).exp(), 0.0)
                fin = torch.isfinite(v)
                o = p @ torch.where(fin, v, 0.0)
                size = p @ torch.where(fin, v, 0.0).abs()
                for j, d in (~fin).nonzero().tolist():
                    o[:, d] += torch.where(seen[:, j], v[j, d], 0.0)
                out[rows, h], lse[rows, h] = o, torch.where(some, z, -math.inf)
                # A logit: a sum of D products in fp32, its scaling, the reference taken off; then the exponential.
                # (fp32's half step is 2^-24; ex2's error 2^-22; a row's largest |q| . |k| bounds what is rounded.)
                most = torch.where(seen, (q.abs() @ torch.nan_to_num(k, 0.0, 0.0, 0.0).abs().t()) * self.scale, 0.0).amax(1) if length else 0.0
                delta = 2.0 ** -24 * (self.dim + 8) * (most + 8) + 2.0 ** -21
                # weights: that, and half a step of bf16; their sum: that, and fp32's rounding of the sum
                total = 2.0 ** -24 * (length + 64)
                e_out[rows, h] = ((2.0 ** -8 + 2 * delta + 2 * total)[:, None] * size * 1.01 + 2.0 ** -8 * o.abs() * 1.01 +
                                  2.0 ** -133)
                e_lse[rows, h] = delta + total + 2.0 ** -22 * (torch.where(some, z, 0.0).abs() + 1)
        return out, lse, e_out, e_lse, self.inside


def check(got, lse, want, fill=None):
    """Against reference(): inside its bounds, NaN and infinities where they belong, rows of no sequence untouched."""
    out, rlse, e_out, e_lse, inside = want
    for x, r, e in ((got, out, e_out), (lse, rlse, e_lse)):
        x = x.double()
        keep = inside.view(-1, *[1] * (x.dim() - 1)).expand_as(x)
        fin = torch.isfinite(r) & keep
        assert torch.equal(torch.isnan(x) & keep, torch.isnan(r) & keep), "NaN in other places"
        inf = torch.isinf(r) & keep
        assert torch.equal(x[inf], r[inf]), "infinities"
        over = ((x - r).abs() - e)[fin]
        if over.numel():
            assert float(over.max()) <= 0, f"off by {float((x - r).abs()[fin].max())}, {float(over.max())} past the bound"
    if fill is not None:
        for x in (got, lse):
            assert (x[~inside] == fill).all(), "rows of no sequence"


def window_mask(length, n, window, sinks):
    p = torch.arange(length - n, length)[:, None]
    j = torch.arange(length)
    return (j <= p) & ((j > p - window) | (j < sinks))


def tree_mask(length, n, bits):
    """bits bool [n, n]."""
    m = torch.ones(n, length, dtype=torch.bool)
    m[:, length - n:] = bits
    return m


def tree_words(bits, rows, starts, words):
    """Rows of mask words int32 [rows, words] from each sequence's bits; bits outside trees are set."""
    m = torch.full((rows, words * 32), True)
    for b, s in zip(bits, starts):
        n = b.shape[0]
        m[s:s + n, :n] = b
    w = (m.view(rows, words, 32).long() << torch.arange(32)).sum(-1)
    return (w << 32 >> 32).to(torch.int32).cuda()
