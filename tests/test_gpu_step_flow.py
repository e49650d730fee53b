"""Masked attention, block tables and accepted paths as a serving loop uses them: together, in graphs, on streams, at
their limits, and with what must be reported."""

import math
import random

import pytest
import torch

from masked_helpers import Sequences, check, page_view, tree_mask, tree_words, window_mask
from paged_kv_decode_14_gb300 import _native as nat

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def windowed(lens, q_lens, window, sinks, **kw):
    return Sequences([window_mask(n, q, window, sinks) for n, q in zip(lens, q_lens)], **kw)


# ------------------------------------------------------------------ together


class Loop:
    """A serving loop whose lengths, tables and pool live on the GPU; the tokens' rows by sequence, in the order that they
    should have in the cache."""

    def __init__(self, seqs, heads, kv_heads, dim, dtype, blocks=400):
        self.heads, self.kv, self.dim, self.dtype, self.seqs = heads, kv_heads, dim, dtype, seqs
        self.g = torch.Generator(device="cuda").manual_seed(3)
        scales = None
        if dtype == "fp8":
            scales = [torch.full((blocks, kv_heads), 0.01, device="cuda") for _ in range(2)]
        self.cache = nat.PagedKVCache(blocks, kv_heads, dim, dtype, k_scales=scales and scales[0],
                                      v_scales=scales and scales[1])
        self.pool = nat.BlockPool(blocks)
        self.table = torch.full((seqs, 64), -1, dtype=torch.int32, device="cuda")
        self.lens = ints([0] * seqs)
        self.ws, self.err = nat.make_masked_workspace(), ints([0])
        self.rows = [[] for _ in range(seqs)]

    def random_rows(self, n, heads):
        return torch.randn(n, heads, self.dim, generator=self.g, device="cuda").bfloat16()

    def grow(self, n):
        """Room for n[b] tokens each, and their K and V in the cache: (granted, starts, k, v)."""
        total = sum(n)
        slots, positions, granted, starts = nat.update_tables(self.pool, self.table, self.lens, ints(n), total,
                                                              device_error=self.err)
        k, v = self.random_rows(total, self.kv), self.random_rows(total, self.kv)
        nat.append(self.cache, k, v, slots, device_error=self.err)
        return granted, starts, k, v

    def values(self, b):
        k, v = (torch.stack([r[i] for r in self.rows[b]]).double() for i in range(2))
        if self.dtype == "fp8":
            k, v = (((x / 0.01).clamp(-448, 448).float().to(torch.float8_e4m3fn)).double() * torch.tensor(0.01).double().item()
                    for x in (k, v))
        return k, v

    def reference(self, q, masks, starts):
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(out)
        for b, m in enumerate(masks):
            k, v = self.values(b)
            m = m.cuda()
            for h in range(self.heads):
                g = h // (self.heads // self.kv)
                rows = slice(starts[b], starts[b] + m.shape[0])
                x = (q[rows, h].double() @ k[:, g].t() * self.dim ** -0.5).masked_fill(~m, -math.inf)
                p = torch.softmax(x, -1)
                out[rows, h], size[rows, h] = p @ v[:, g], p @ v[:, g].abs()
        return out, size

    def check(self, got, q, masks, starts):
        out, size = self.reference(q, masks, starts)
        # (weights and result rounded to bf16, 2^-8 each; the logits' fp32 errors and FP8's scale in fp32 are far below)
        assert ((got.double() - out).abs() <= 2.0 ** -8 * (size + out.abs()) * 1.02 + 1e-4 * size).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_a_speculative_loop(dtype):
    """Prompts, then rounds of drafted trees: grown, attended, their accepted paths kept, the rest dropped; and a windowed
    step over what has become of the cache."""
    rnd = random.Random(5)
    s = Loop(5, 8, 2, 64, dtype)
    n = [40, 1, 17, 100, 64]
    granted, starts, k, v = s.grow(n)
    at = starts.tolist()
    for b in range(5):
        s.rows[b] += [(k[i], v[i]) for i in range(at[b], at[b] + n[b])]
    q = s.random_rows(sum(n), 8)
    out, _ = nat.attention_window(s.cache, q, s.table, s.lens, granted, max(n), 30, 4, 0.125, s.ws, q_starts=starts)
    s.check(out, q, [window_mask(x, x, 30, 4) for x in n], at)
    for turn in range(4):
        t = [rnd.randint(1, 40) for _ in range(5)]
        granted, starts, k, v = s.grow(t)
        at = starts.tolist()
        bits = []
        for x in t:
            m = torch.eye(x, dtype=torch.bool)
            for i in range(1, x):
                m[i] |= m[rnd.randrange(i)]
            bits.append(m)
        q = s.random_rows(sum(t), 8)
        words = tree_words(bits, sum(t), at, 2)
        out, _ = nat.attention_tree(s.cache, q, s.table, s.lens, granted, max(t), words, 0.125, s.ws, q_starts=starts)
        drafted = [[(k[i], v[i]) for i in range(at[b], at[b] + t[b])] for b in range(5)]
        before = [list(r) for r in s.rows]
        for b in range(5):
            s.rows[b] = before[b] + drafted[b]
        s.check(out, q, [tree_mask(len(before[b]) + t[b], t[b], bits[b]) for b in range(5)], at)
        # a branch of each tree is accepted
        paths = [bits[b][rnd.randrange(t[b])].nonzero()[:, 0].tolist() for b in range(5)]
        most = max(map(len, paths))
        keep = ints([len(p) for p in paths])
        nat.keep_path(s.cache, s.table, s.lens, granted, ints([p + [0] * (most - len(p)) for p in paths]), keep,
                      device_error=s.err)
        nat.update_tables(s.pool, s.table, s.lens, keep - granted, 0, device_error=s.err)
        for b in range(5):
            s.rows[b] = before[b] + [drafted[b][j] for j in paths[b]]
        # a decode step with a window
        granted, starts, k, v = s.grow([1] * 5)
        for b in range(5):
            s.rows[b].append((k[b], v[b]))
        q = s.random_rows(5, 8)
        out, _ = nat.attention_window(s.cache, q, s.table, s.lens, granted, 1, 25, 3, 0.125, s.ws)
        s.check(out, q, [window_mask(len(r), 1, 25, 3) for r in s.rows], list(range(5)))
    assert s.lens.tolist() == [len(r) for r in s.rows]
    used = sum(-(-len(r) // 16) for r in s.rows)
    assert s.pool.count.item() == s.pool.num_blocks - used
    nat.update_tables(s.pool, s.table, s.lens, -s.lens, 0, device_error=s.err)
    assert s.pool.count.item() == s.pool.num_blocks and sorted(s.pool.free.tolist()) == list(range(s.pool.num_blocks))
    assert nat.read_device_error(s.err) == 0 and nat.read_device_error(s.ws) == 0


def test_decode_steps_in_a_graph():
    """Table update, append and windowed attention captured once and replayed: lengths grow on the GPU."""
    s = Loop(4, 8, 2, 128, "bf16")
    granted, starts, k, v = s.grow([30, 16, 1, 47])
    base = [30, 16, 1, 47]
    at = starts.tolist()
    for b in range(4):
        s.rows[b] += [(k[i], v[i]) for i in range(at[b], at[b] + base[b])]
    one = ints([1] * 4)
    k1, v1, q1 = s.random_rows(4, 2), s.random_rows(4, 2), s.random_rows(4, 8)
    out = torch.empty_like(q1)

    def step():
        slots, _, granted, _ = nat.update_tables(s.pool, s.table, s.lens, one, 4, device_error=s.err)
        nat.append(s.cache, k1, v1, slots, device_error=s.err)
        return nat.attention_window(s.cache, q1, s.table, s.lens, granted, 1, 20, 2, 128 ** -0.5, s.ws, out=out)

    state = [t.clone() for t in (s.table, s.lens, s.pool.free, s.pool.count)]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    for t, was in zip((s.table, s.lens, s.pool.free, s.pool.count), state):
        t.copy_(was)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(20):
        k1.copy_(s.random_rows(4, 2))
        v1.copy_(s.random_rows(4, 2))
        q1.copy_(s.random_rows(4, 8))
        g.replay()
        for b in range(4):
            s.rows[b].append((k1[b].clone(), v1[b].clone()))
        s.check(out, q1, [window_mask(len(r), 1, 20, 2) for r in s.rows], list(range(4)))
    assert nat.read_device_error(s.err) == 0 and nat.read_device_error(s.ws) == 0


def test_two_streams_with_a_workspace_each():
    a = windowed([4000, 300], [1, 200], 3500, 4, heads=8, kv_heads=2, dim=128, dtype="bf16", seed=1)
    b = windowed([700, 5000], [30, 2], 4800, 0, heads=8, kv_heads=2, dim=64, dtype="fp8", seed=2)
    both = [(a, 3500, 4, torch.cuda.Stream(), nat.make_masked_workspace()), (b, 4800, 0, torch.cuda.Stream(), nat.make_masked_workspace())]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s, w, n, stream, ws in both:
            got.append(nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, w, n, s.scale, ws, stream=stream))
    torch.cuda.synchronize()
    want = [a.reference(), b.reference()]
    for i, (out, lse) in enumerate(got):
        check(out, lse, want[i % 2])


# ------------------------------------------------------------------ limits and reports


@pytest.fixture(scope="module")
def workspace():
    return nat.make_masked_workspace()


def test_offsets_past_32_bits(workspace):
    """A cache of more than 2^32 bytes, its sequences at both ends."""
    blocks, heads, dim = 140000, 8, 128
    s = windowed([100, 40], [3, 1], 64, 4, heads=16, kv_heads=heads, dim=dim, dtype="bf16", seed=4)
    k, v = (torch.empty(blocks, heads, 16 * dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    small = s.cache.k.shape[0]
    move = torch.arange(small, device="cuda")
    move = torch.where(move % 2 == 0, move, blocks - 1 - move)
    k[move], v[move] = s.cache.k, s.cache.v
    ok = s.table < small
    table = torch.where(ok, move[s.table.clamp(max=small - 1).long()].int(), s.table)
    cache = nat.PagedKVCache(blocks, heads, dim, "bf16", k=k, v=v)
    out, lse = nat.attention_window(cache, s.q, table, s.t_lens, s.t_q, s.max_q, 64, 4, s.scale, workspace)
    assert nat.read_device_error(workspace) == 0
    check(out, lse, s.reference())
    err = ints([0])
    at = page_view(k, heads, dim)
    b0, b1 = int(table[0, 5]), int(table[0, 6])                  # positions 80 .. 99; the path is 3 -> 0
    want = at[b1, :, 0, :, 3].clone()                            # position 99 = 16 * 6 + 3
    nat.keep_path(cache, table, ints([100, 40]), ints([20, 1]), ints([[19], [0]]), ints([1, 1]), device_error=err)
    assert torch.equal(at[b0, :, 0, :, 0], want) and nat.read_device_error(err) == 0


def test_bad_lengths_leave_their_rows(workspace):
    s = windowed([40, 30, 20, 16], [3, 2, 4, 1], 1000, 0, heads=4, kv_heads=2, dim=64, dtype="bf16", seed=6, gaps=[1] * 4)
    want = s.reference()
    for lens, q_lens in (([40, 1, 20, 16], [3, 2, 4, 1]), ([40, 30, 1 << 20, 16], [3, 2, 4, 1]), ([40, 30, 20, 16], [3, -1, 4, 1]),
                         ([40, 30, 20, 16], [3, 2, 9, 1])):
        out, lse = torch.full_like(s.q, 7.0), torch.full(s.q.shape[:2], 7.0, device="cuda")
        nat.attention_window(s.cache, s.q, s.table, ints(lens), ints(q_lens), 4, 1000, 0, s.scale, workspace, out=out,
                             lse=lse, q_starts=s.t_starts)
        assert nat.read_device_error(workspace) == nat.DEVERR_LENGTH
        bad = [b for b in range(4) if lens[b] != s.lens[b] or q_lens[b] != s.q_lens[b]]
        inside = s.inside.clone()
        for b in bad:
            inside[s.starts[b]:s.starts[b] + s.q_lens[b]] = False
        check(out, lse, (*want[:4], inside), fill=7.0)
    starts = s.t_starts.clone()
    starts[3] = s.rows                                           # its row lies behind the tensor
    out = torch.full_like(s.q, 7.0)
    nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, 4, 1000, 0, s.scale, workspace, out=out, q_starts=starts)
    assert nat.read_device_error(workspace) == nat.DEVERR_LENGTH
    assert (out[s.starts[3]] == 7.0).all()


@pytest.mark.parametrize("length", [(1 << 31) - 1, (1 << 31) - 512, (1 << 31) - 511])
def test_a_context_near_2_to_31_is_refused(length, workspace):
    """(At most 2^31 - 512 positions; the longest that is taken reads a window's pages at the table's end.)"""
    s = windowed([40, 30], [1, 1], 1000, 0, heads=4, kv_heads=2, dim=64, dtype="bf16", seed=6)
    table = torch.zeros(2, 1 << 27, dtype=torch.int32, device="cuda")
    table[:, :2] = s.table[:, :2]
    table[1, :2] = s.table[0, 0]
    table[1, -40:] = s.table[0, 0]
    out = torch.full_like(s.q, 7.0)
    nat.attention_window(s.cache, s.q, table, ints([16, length]), s.t_q, 1, 16, 0, s.scale, workspace, out=out)
    fits = length <= (1 << 31) - 512
    assert nat.read_device_error(workspace) == (0 if fits else nat.DEVERR_LENGTH)
    assert not (out[0] == 7.0).any() and bool((out[1] == 7.0).all()) != fits
    if fits:                                                     # a window that is one whole page: the same keys as sequence 0's
        one = nat.attention_window(s.cache, s.q[1:], table[:1], ints([16]), ints([1]), 1, 16, 0, s.scale, workspace)[0]
        assert torch.equal(out[1], one[0])


def test_a_bad_block_is_reported(workspace):
    s = windowed([100], [1], 1000, 0, heads=4, kv_heads=2, dim=64, dtype="bf16", seed=6)
    for bad in (-1, s.cache.num_blocks):
        t = s.table.clone()
        t[0, 3] = bad
        nat.attention_window(s.cache, s.q, t, s.t_lens, s.t_q, 1, 1000, 0, s.scale, workspace)
        assert nat.read_device_error(workspace) == nat.DEVERR_BLOCK_ID
    out, lse = nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, 1, 1000, 0, s.scale, workspace)
    check(out, lse, s.reference())


@pytest.mark.parametrize("q_len", [1, 90])
def test_a_wait_that_runs_out(q_len):
    s = windowed([300, 200], [q_len, q_len], 1000, 0, heads=8, kv_heads=2, dim=128, dtype="bf16", seed=6)
    ws = nat.make_masked_workspace()
    flag = ints([0])
    nat.debug_set_wait_limit(20_000_000, flag)
    try:
        nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, 1000, 0, s.scale, ws)
        torch.cuda.synchronize()
    finally:
        nat.debug_set_wait_limit(0, None)
    assert nat.read_device_error(ws) & nat.DEVERR_TIMEOUT
    nat.workspace_init(ws)
    out, lse = nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, 1000, 0, s.scale, ws)
    assert nat.read_device_error(ws) == 0
    check(out, lse, s.reference())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("q_len", [1, 70])
def test_logits_past_the_limit_are_reported(q_len, dtype, workspace):
    s = windowed([200], [q_len], 1000, 0, heads=4, kv_heads=2, dim=64, dtype=dtype, seed=2)
    nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, 1000, 0, 1e10, workspace)
    assert nat.read_device_error(workspace) == nat.DEVERR_RANGE


@pytest.mark.parametrize("q_len", [2, 80])
@pytest.mark.parametrize("place,value", [("v", math.inf), ("v", math.nan), ("k", math.nan), ("v", 0.0), ("v", 1e-30), ("v", 1e4),
                                         ("k", 1e-30), ("k", 0.0)])
def test_scales_of_any_size(place, value, q_len, workspace):
    """One page's scale is infinite, NaN, 0 or far from the others: as its values then are, for the queries that see it."""
    s = windowed([300, 150], [q_len, q_len], 60, 3, heads=8, kv_heads=2, dim=64, dtype="fp8", seed=8)
    i = 0 if place == "k" else 1
    for b, page in ((0, 17), (1, 8)):
        blk = int(s.table[b, page])
        s.scales[i][blk, 1] = value
        pool = (s.cache.k, s.cache.v)[i]
        rows = page_view(pool, 2, 64)[blk, 1].permute(0, 2, 1, 3).reshape(16, 64).view(torch.float8_e4m3fn).double()
        n = min(16, s.lens[b] - 16 * page)
        known = s.values[b][i][16 * page:16 * page + n, 1]
        seen = s.seen[b].any(0)[16 * page:16 * page + n]
        known[seen] = (rows[:n] * float(torch.tensor(value)))[seen]
        known[~seen] = 0.0
    out, lse = nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, 60, 3, s.scale, workspace)
    assert nat.read_device_error(workspace) == 0
    want = s.reference()
    if place == "v" and value == math.inf:                       # infinite times a code of 0, or beside another sign: NaN either way
        r = want[0]
        assert not torch.isfinite(out.double())[~torch.isfinite(r)].any()
        keep = torch.isfinite(r)
        assert ((out.double() - r).abs()[keep] <= want[2][keep]).all()
        return
    check(out, lse, want)


@pytest.mark.parametrize("size", [0.0, 1e-30, 1e-38, 1e30])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_queries_of_any_size(size, dtype, workspace):
    """Rows of queries that are 0, tiny, or huge (with a scale that brings the logits back)."""
    s = windowed([200, 90], [1, 33], 100, 3, heads=8, kv_heads=2, dim=128, dtype=dtype, seed=8)
    s.q = (s.q.double() * size).bfloat16()
    if size > 1:
        s.scale /= size
    out, lse = nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, 100, 3, s.scale, workspace)
    assert nat.read_device_error(workspace) == 0
    check(out, lse, s.reference())


@pytest.mark.parametrize("q_len", [1, 80])
def test_rows_of_zeros_with_a_tiny_scale(q_len, workspace):
    """A scale whose product with an FP8 row's power of two leaves fp32: still the mean of what is visible."""
    s = windowed([200, 90], [q_len, q_len], 50, 3, heads=8, kv_heads=2, dim=64, dtype="fp8", seed=8)
    s.q.zero_()
    s.scale = 1e-30
    out, lse = nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, 50, 3, s.scale, workspace)
    assert nat.read_device_error(workspace) == 0
    check(out, lse, s.reference())


def test_a_wide_window_is_plain_causal_attention(workspace):
    s = windowed([500, 77, 300], [4, 1, 16], 1 << 20, 0, heads=8, kv_heads=2, dim=128, dtype="bf16", seed=5)
    ws = nat.make_workspace(3, 8, 2, 128, 16)
    a = nat.attention(s.cache, s.q, s.table, s.t_lens, s.t_q, 16, s.scale, ws).double()
    b = nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, 16, 1 << 20, 0, s.scale, workspace)[0].double()
    assert ((a - b).abs() <= 2e-3 + 1e-2 * a.abs()).all()


def test_results_as_the_next_attentions_queries(workspace):
    """pkv_paged_attention reads its q while the kernel before it may still run: not before this one's results are there."""
    s = windowed([900] * 24, [1] * 24, 1 << 20, 0, heads=16, kv_heads=4, dim=128, dtype="bf16", seed=5)
    ws = nat.make_workspace(24, 16, 4, 128, 1)
    mid, lse, last = (torch.empty_like(s.q), torch.empty(s.q.shape[:2], device="cuda"), torch.empty_like(s.q))

    def first():
        nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, 1, 1 << 20, 0, s.scale, workspace, out=mid, lse=lse)

    def second():
        nat.attention(s.cache, mid, s.table, s.t_lens, s.t_q, 1, s.scale, ws, out=last)

    first()
    torch.cuda.synchronize()
    second()
    torch.cuda.synchronize()
    want = last.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first()
        second()
    for call in (lambda: (first(), second()), graph.replay):
        for _ in range(20):
            mid.zero_()
            last.zero_()
            call()
            torch.cuda.synchronize()
            assert torch.equal(last, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_thousands_of_sequences(dtype, workspace):
    """A hundred for each of the plan's lanes; with starts given, the same bits."""
    rnd = random.Random(3)
    n, heads, kv, dim, most = 3001, 8, 4, 64, 48
    lens = [rnd.choice((0, 1, 16, 17, rnd.randint(0, most))) for _ in range(n)]
    q_lens = [min(x, rnd.choice((0, 1, 1, 2))) for x in lens]
    blocks = 700
    g = torch.Generator(device="cuda").manual_seed(1)
    if dtype == "fp8":
        pools = [torch.randn(blocks, kv, 16 * dim, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
        scales = [0.5 + torch.rand(blocks, kv, generator=g, device="cuda") for _ in range(2)]
    else:
        pools = [torch.randn(blocks, kv, 16 * dim, generator=g, device="cuda").bfloat16() for _ in range(2)]
        scales = [None, None]
    cache = nat.PagedKVCache(blocks, kv, dim, dtype, k=pools[0], v=pools[1], k_scales=scales[0], v_scales=scales[1])
    table = torch.randint(blocks, (n, 4), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(sum(q_lens), heads, dim, generator=g, device="cuda").bfloat16()
    b, lse = nat.attention_window(cache, q, table, ints(lens), ints(q_lens), 2, 1 << 20, 0, dim ** -0.5, workspace)
    assert nat.read_device_error(workspace) == 0
    # K and V [sequence, kv head, token, dim] in 64 bits, and the rows' sequences and what they see
    k, v = ((page_view(x, kv, dim) if sc is None else page_view(x, kv, dim).view(torch.float8_e4m3fn)).double() *
            (1.0 if sc is None else sc.double()[:, :, None, None, None, None]) for x, sc in zip(pools, scales))
    k, v = (x.permute(0, 1, 2, 4, 3, 5).reshape(blocks, kv, 16, dim)[table.long()].transpose(1, 2).reshape(n, kv, 64, dim)
            for x in (k, v))
    seq = torch.tensor([i for i, x in enumerate(q_lens) for _ in range(x)], device="cuda")
    end = ints([lens[i] - x + 1 + j for i, x in enumerate(q_lens) for j in range(x)])
    hidden = torch.arange(64, device="cuda")[None, None, :] >= end[:, None, None]
    k, v = (x[seq].repeat_interleave(heads // kv, 1) for x in (k, v))
    x = torch.einsum("rhd,rhtd->rht", q.double(), k) * dim ** -0.5
    z = torch.logsumexp(x.masked_fill(hidden, -math.inf), -1)
    w = (x - z[..., None]).exp().masked_fill(hidden, 0.0)
    want, size = torch.einsum("rht,rhtd->rhd", w, v), torch.einsum("rht,rhtd->rhd", w, v.abs())
    # the bound of Sequences.reference, by its arithmetic
    top = (torch.einsum("rhd,rhtd->rht", q.double().abs(), k.abs()) * dim ** -0.5).masked_fill(hidden, 0.0).amax(-1)
    delta, total = 2.0 ** -24 * (dim + 8) * (top + 8) + 2.0 ** -21, 2.0 ** -24 * (64 + 64)
    bound = (2.0 ** -8 + 2 * delta + 2 * total)[..., None] * size * 1.01 + 2.0 ** -8 * want.abs() * 1.01 + 2.0 ** -133
    assert ((b.double() - want).abs() <= bound).all()
    assert ((lse.double() - z).abs() <= delta + total + 2.0 ** -22 * (z.abs() + 1)).all()
    starts = torch.tensor([0] + q_lens[:-1], device="cuda").cumsum(0)
    again = nat.attention_window(cache, q, table, ints(lens), ints(q_lens), 2, 1 << 20, 0, dim ** -0.5, workspace, q_starts=starts)
    assert torch.equal(again[0], b) and torch.equal(again[1], lse)


def test_python_refusals(workspace):
    s = windowed([40], [2], 16, 0, heads=4, kv_heads=2, dim=64, dtype="bf16", seed=6)
    call = lambda **k: nat.attention_window(*[k.get(x, y) for x, y in (  # noqa: E731
        ("cache", s.cache), ("q", s.q), ("table", s.table), ("lens", s.t_lens), ("q_lens", s.t_q))], 2, 16, 0, 0.1, workspace)
    for bad in (dict(q=s.q.float()), dict(q=s.q[:, :, :32]), dict(table=s.table.long()), dict(table=s.table[:, ::2]),
                dict(lens=s.t_lens.cpu()), dict(q_lens=s.t_q.float())):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(ValueError):
        nat.attention_tree(s.cache, s.q, s.table, s.t_lens, s.t_q, 2, ints([[1]]), 0.1, workspace)
    with pytest.raises(nat.PagedKVError):
        nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, 2, 0, 0, 0.1, workspace)
    with pytest.raises(ValueError):
        nat.BlockPool(8, free=ints([0]))
    with pytest.raises(ValueError):
        nat.update_tables(nat.BlockPool(8), s.table, s.t_lens, ints([1, 1]), 2)
