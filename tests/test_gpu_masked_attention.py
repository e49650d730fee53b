"""Attention over the cache with a sliding window and first tokens that stay visible, and of trees of drafted tokens,
against the definition in 64 bits."""

import math
import random

import pytest
import torch

from masked_helpers import Sequences, check, tree_mask, tree_words, window_mask
from paged_kv_decode_14_gb300 import _native as nat

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def workspace():
    return nat.make_masked_workspace()


def run_window(s, window, sinks, workspace, **kw):
    out = nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, window, sinks, s.scale, workspace, **kw)
    assert nat.read_device_error(workspace) == 0
    return out


def windowed(lens, q_lens, window, sinks, **kw):
    return Sequences([window_mask(n, q, window, sinks) for n, q in zip(lens, q_lens)], **kw)


# (lens, q_lens, window, sinks, heads, kv_heads, dim)
WINDOWS = [
    ([1], [1], 1, 0, 1, 1, 64),
    ([7, 1, 40], [1, 1, 1], 8, 2, 4, 2, 128),
    ([300, 129, 16, 17, 500], [1] * 5, 64, 4, 8, 2, 128),            # sinks apart from the window
    ([300, 129, 16, 17, 500], [1] * 5, 64, 0, 8, 8, 64),
    ([200, 64, 33], [1, 1, 1], 1, 0, 6, 2, 64),                      # a query sees itself only
    ([200, 64, 33], [1, 1, 1], 1, 1, 6, 2, 64),
    ([513, 700], [5, 9], 100, 20, 8, 2, 128),                        # verify windows; sinks end inside a page
    ([90, 0, 33, 16], [3, 0, 33, 16], 1000, 4, 5, 1, 128),           # odd groups, an empty sequence, plain causal
    ([350, 260], [350, 200], 90, 3, 8, 2, 64),                       # prompts: two row tiles
    ([700], [600], 130, 16, 4, 4, 128),
    ([400, 190], [100, 190], 1 << 30, 0, 7, 1, 128),                 # no window to speak of, G = 7
    ([400], [260], 17, 200, 2, 2, 64),                               # more sinks than window
    ([150], [150], 40, 1 << 30, 2, 1, 64),                           # all tokens are sinks
    ([300], [20], 50, 5, 128, 1, 64),                                # G = 128: one query a row tile
    ([6000], [1], 5000, 4, 8, 1, 128),                               # one long row group: cut between CTAs
    ([9001, 40], [3, 1], 8000, 10, 6, 2, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("case", range(len(WINDOWS)))
def test_window(case, dtype, workspace):
    lens, q_lens, window, sinks, heads, kv, dim = WINDOWS[case]
    s = windowed(lens, q_lens, window, sinks, heads=heads, kv_heads=kv, dim=dim, dtype=dtype, seed=case)
    out, lse = run_window(s, window, sinks, workspace)
    check(out, lse, s.reference())


def random_bits(n, rnd, general):
    if general:
        return torch.tensor([[rnd.random() < 0.4 for _ in range(n)] for _ in range(n)])
    bits = torch.eye(n, dtype=torch.bool)
    for i in range(1, n):
        p = rnd.randrange(-1, i)
        if p >= 0:
            bits[i] |= bits[p]
    return bits


# (lens, q_lens, heads, kv_heads, dim, general masks)
TREES = [
    ([1], [1], 1, 1, 64, False),
    ([40, 7, 300], [7, 7, 5], 8, 2, 128, False),
    ([33, 129, 16], [33, 40, 16], 4, 1, 128, True),                  # no context, rows that see nothing
    ([500, 77], [64, 70], 8, 2, 64, False),                          # two row tiles, three mask words
    ([700, 0, 260], [64, 0, 33], 7, 1, 128, True),
    ([5000], [6], 4, 1, 64, False),
    ([2100, 4100], [64, 64], 8, 1, 128, False),                      # many rows over a long context
    ([270], [150], 2, 2, 64, True),
]


def treed(lens, q_lens, general, heads, kv_heads, dim, dtype, seed, **kw):
    rnd = random.Random(seed)
    bits = [random_bits(n, rnd, general) for n in q_lens]
    if general:
        for b in bits:
            if len(b) > 2:
                b[2] = False
    s = Sequences([tree_mask(n, q, b) for n, q, b in zip(lens, q_lens, bits)], heads, kv_heads, dim, dtype, seed, whole=True, **kw)
    words = (s.max_q + 31) // 32 + (seed & 1)
    return s, tree_words(bits, s.rows, s.starts, words)


def run_tree(s, words, workspace, **kw):
    out = nat.attention_tree(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, words, s.scale, workspace, **kw)
    assert nat.read_device_error(workspace) == 0
    return out


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree(case, dtype, workspace):
    lens, q_lens, heads, kv, dim, general = TREES[case]
    s, words = treed(lens, q_lens, general, heads, kv, dim, dtype, case)
    out, lse = run_tree(s, words, workspace)
    check(out, lse, s.reference())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("q_lens,ctx,heads", [([120, 77, 1, 64, 65] * 8, 300, 16), ([3, 1, 8, 2] * 20, 600, 16),
                                              ([1] * 300, 90, 32), ([40, 7] * 30, 100, 56)])
def test_many_items_a_cta(q_lens, ctx, heads, dtype, workspace):
    """Several items in a row on every CTA, of one and two row tiles, of one key tile and of many."""
    rnd = random.Random(len(q_lens))
    lens = [q + rnd.randint(0, ctx) for q in q_lens]
    s = windowed(lens, q_lens, 150, 4, heads=heads, kv_heads=8, dim=64, dtype=dtype, seed=3)
    out, lse = run_window(s, 150, 4, workspace)
    check(out, lse, s.reference())
    again = run_window(s, 150, 4, workspace)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


# (sequences, longest query, heads, kv_heads, dim, longest context, kind): more items than CTAs, or much FP8 work, so that several
# kv-heads stay in an item
SHARED = [
    (45, 1, 32, 8, 128, 300, "window"),                              # four: rows of 4 in quarters of the lanes
    (45, 6, 32, 8, 128, 200, "tree"),
    (40, 9, 24, 8, 64, 260, "window"),                               # G = 3
    (45, 11, 20, 4, 128, 150, "window"),                             # two: 55 rows of 64
    (80, 16, 12, 4, 64, 120, "tree"),                                # two: 48 rows
    (45, 2, 28, 4, 128, 200, "window"),                              # four, G = 7: 28 rows of 32
    (5, 3, 16, 8, 128, 12000, "window"),                             # few and long
]


@pytest.mark.parametrize("spread", [1.0, 12.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_items_of_several_heads(case, dtype, spread, workspace):
    """One long sequence among short ones (cut between CTAs), NaN and infinities planted, references that rise."""
    n, most, heads, kv, dim, longest, kind = SHARED[case]
    rnd = random.Random(case)
    q_lens = [most] + [rnd.choice((0, 1, most, rnd.randint(1, most))) for _ in range(n - 1)]
    ctx = [rnd.randint(0, longest) for _ in range(n)]
    ctx[n // 2] = max(3000, longest)
    lens = [q + c for q, c in zip(q_lens, ctx)]
    nan, big = math.nan, math.nan if dtype == "fp8" else math.inf
    plant = [(b, 1, rnd.randrange(lens[b]), rnd.randrange(kv), rnd.randrange(dim), v)
             for b, v in ((0, nan), (n // 2, big), (n - 1, -big), (1, nan)) if lens[b]]
    kw = dict(heads=heads, kv_heads=kv, dim=dim, dtype=dtype, seed=case, plant=plant, spread=spread)
    if kind == "window":
        window = 100 if longest < 5000 else 1 << 30
        s = windowed(lens, q_lens, window, 5, **kw)
        run = lambda: run_window(s, window, 5, workspace)  # noqa: E731
    else:
        s, words = treed(lens, q_lens, True, **kw)
        run = lambda: run_tree(s, words, workspace)  # noqa: E731
    out, lse = run()
    check(out, lse, s.reference())
    again = run()
    assert torch.equal(again[0].view(torch.int16), out.view(torch.int16)) and torch.equal(again[1].view(torch.int32), lse.view(torch.int32))


@pytest.mark.parametrize("seed", range(12))
def test_random(seed, workspace):
    rnd = random.Random(seed)
    kv = rnd.choice((1, 2, 4))
    heads, dim, dtype = kv * rnd.choice((1, 2, 3, 4, 8)), rnd.choice((64, 128)), rnd.choice(("bf16", "fp8"))
    n = rnd.randint(1, 9)
    q_lens = [rnd.choice((0, 1, 1, 2, 17, 90)) for _ in range(n)]
    lens = [q + rnd.choice((0, 0, 5, 100, 1000)) for q in q_lens]
    gaps = [rnd.randint(0, 3) for _ in range(n)]
    window, sinks = rnd.choice((1, 15, 16, 100, 4000)), rnd.choice((0, 1, 16, 50))
    kw = dict(heads=heads, kv_heads=kv, dim=dim, dtype=dtype, seed=seed, gaps=gaps, lead=2)
    if seed % 2:
        s = windowed(lens, q_lens, window, sinks, **kw)
        run = lambda **k: run_window(s, window, sinks, workspace, q_starts=s.t_starts, **k)  # noqa: E731
    else:
        s, words = treed(lens, q_lens, seed % 4 == 0, **kw)
        run = lambda **k: run_tree(s, words, workspace, q_starts=s.t_starts, **k)  # noqa: E731
    out, lse = torch.full_like(s.q, 7.0), torch.full(s.q.shape[:2], 7.0, device="cuda")
    got = run(out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    check(out, lse, s.reference(), fill=7.0)
    again = run()
    assert torch.equal(again[0][s.inside], out[s.inside]) and torch.equal(again[1][s.inside], lse[s.inside])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_nonfinite_values_reach_only_the_rows_that_see_them(dtype, workspace):
    """NaN (bf16: infinities too) in K and V of keys that some of an item's rows see and others do not."""
    nan, inf = math.nan, math.inf
    big = nan if dtype == "fp8" else inf
    lens, q_lens, window, sinks = [200, 330], [70, 5], 40, 3
    plant = [(0, 1, 150, 0, 5, nan), (0, 1, 171, 1, 9, big), (0, 1, 171, 1, 10, -big), (0, 0, 199, 0, 3, nan),
             (1, 1, 2, 0, 0, big), (1, 1, 288, 1, 7, nan), (1, 1, 329, 0, 1, big), (1, 0, 290, 1, 0, nan)]
    s = windowed(lens, q_lens, window, sinks, heads=8, kv_heads=2, dim=64, dtype=dtype, seed=5, plant=plant)
    out, lse = run_window(s, window, sinks, workspace)
    check(out, lse, s.reference())
    rnd = random.Random(2)
    bits = [random_bits(40, rnd, False), random_bits(9, rnd, False)]
    plant = [(0, 1, 260 + 7, 0, 5, nan), (0, 1, 260 + 39, 1, 9, big), (0, 0, 260 + 3, 0, 3, nan), (1, 1, 20, 1, 0, -big)]
    s = Sequences([tree_mask(300, 40, bits[0]), tree_mask(21, 9, bits[1])], 8, 2, 128, dtype, 3, plant=plant,
                  whole=True)
    out, lse = run_tree(s, tree_words(bits, s.rows, s.starts, 2), workspace)
    check(out, lse, s.reference())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("spread", [6.0, 40.0])
def test_large_logits(spread, dtype, workspace):
    """References that rise often: logits of standard deviation `spread`."""
    s = windowed([900, 300, 2500], [1, 130, 4], 700, 4, heads=8, kv_heads=2, dim=128, dtype=dtype, seed=1, spread=spread)
    out, lse = run_window(s, 700, 4, workspace)
    check(out, lse, s.reference())


def test_views_in_place_and_other_strides(workspace):
    """q out of a fused projection, results into a view of heads-major rows, and in place."""
    s = windowed([100, 300], [4, 140], 60, 4, heads=8, kv_heads=2, dim=64, dtype="bf16", seed=8)
    want = s.reference()
    fused = torch.randn(s.rows, 12 * 64, device="cuda").bfloat16()
    q = fused[:, :512].view(s.rows, 8, 64)
    q.copy_(s.q)
    s.q = q
    out = torch.empty(8, s.rows, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    got, lse = run_window(s, 60, 4, workspace, out=out)
    check(got, lse, want)
    odd = torch.empty(s.rows, 8 * 64 + 8, dtype=torch.bfloat16, device="cuda")[:, 8:].view(s.rows, 8, 64)   # 16-byte rows
    got, lse = run_window(s, 60, 4, workspace, out=odd)
    check(got, lse, want)
    got, lse = run_window(s, 60, 4, workspace, out=q)
    assert got is q
    check(got, lse, want)
