"""Items of several kv-heads that are cut between CTAs: which sizes give them follows from the kernel's rules, which are
restated here, so that a test whose sizes no longer do fails."""

import math
import random

import pytest
import torch

from masked_helpers import Sequences, check, tree_mask, tree_words, window_mask
from paged_kv_decode_14_gb300 import _native as nat
from test_gpu_masked_attention import random_bits

pytestmark = pytest.mark.gpu

ROWS, COLS, PAGE, ITEM, CUT, LEAST, FP8_TILES = 128, 128, 16, 4, 8, 4, 16


def plan(lens, q_lens, max_q, heads, kv, fp8, max_blocks, window=None, sinks=0):
    """(kv-heads of an item, whether items are dealt whole, the most parts of an item); window None: a tree."""
    grid = min(torch.cuda.get_device_properties(0).multi_processor_count, 160)
    grp, n = heads // kv, len(lens) * kv
    rows = min(max_q * grp, ROWS)
    hg = 4 if rows <= ROWS // 4 and kv % 4 == 0 else 2 if rows <= ROWS // 2 and kv % 2 == 0 else 1
    keys = min(max_blocks * PAGE, math.inf if window is None else window + sinks + max_q)
    if not (fp8 and n // hg >= 8 and n * keys > grid * FP8_TILES * COLS):
        while hg > 1 and n * 2 // hg <= grid:
            hg //= 2
    pb, pages = ROWS // hg // grp, 8 // hg
    per = 2 * pb if hg == 1 else pb
    items = []                                                           # (key tiles, row tiles)
    for length, q in zip(lens, q_lens):
        for q0 in range(0, q, per):
            nq = min(per, q - q0)
            first = length - q + q0
            many = (length + PAGE - 1) // PAGE
            if window is not None:
                behind = max(0, first - window + 1) // PAGE
                kept = min((min(sinks, length) + PAGE - 1) // PAGE, behind)
                many = (first + nq - 1) // PAGE + 1 - (behind - kept)
            items += [(-(-many // pages), 2 if hg == 1 and nq > pb else 1)] * (kv // hg)
    units = [t * e + ITEM for t, e in items]
    ctas = max(1, min(grid, sum(units) // LEAST))
    flat = len(items) <= grid and max(units) <= sum(units) // ctas + CUT
    share, longer = divmod(sum(units), ctas)
    cta = lambda u: u // (share + 1) if u < (share + 1) * longer else longer + (u - (share + 1) * longer) // share  # noqa: E731
    parts, at = 1, 0
    for (t, e), w in zip(items, units):
        if not flat:
            parts = max(parts, cta(at + ITEM + (t - 1) * e) - cta(at + ITEM) + 1)
        at += w
    return hg, flat, parts


# (sequences, longest query, heads, kv_heads, dim, other contexts, the long one, window (None: a tree), kv-heads an item)
CUT_ITEMS = [
    (90, 1, 32, 8, 128, 300, 9000, 3000, 4),                             # rows of 4 in quarters of the lanes
    (90, 3, 28, 4, 64, 200, 6000, 4000, 4),                              # G = 7, 21 rows of 32
    (160, 4, 28, 4, 128, 60, 5000, 4000, 4),                             # G = 7, 28 rows of 32
    (90, 11, 20, 4, 128, 150, 4000, 2500, 2),                            # 55 rows of 64
    (90, 16, 8, 2, 64, 150, 9000, 1 << 30, 2),                           # 64 rows of 64, no window
    (90, 6, 32, 8, 128, 200, 4000, None, 4),                             # trees
    (90, 13, 16, 4, 64, 100, 5000, None, 2),
    (10, 1, 32, 8, 128, 200, 9000, 7000, (1, 4)),                        # bf16: one; FP8: four (much FP8 work)
]


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("case", range(len(CUT_ITEMS)))
def test_cut_items_of_several_heads(case, dtype):
    """A long context among short ones, NaN and infinities planted over all of it, references that rise."""
    n, most, heads, kv, dim, other, longest, window, want = CUT_ITEMS[case]
    rnd = random.Random(case)
    q_lens = [rnd.choice((1, most, rnd.randint(1, most))) for _ in range(n)]
    q_lens[n // 2] = most
    lens = [q + rnd.randint(0, other) for q in q_lens]
    lens[n // 2] = longest
    nan, big = math.nan, math.nan if dtype == "fp8" else math.inf
    plant = [(b, 1, rnd.randrange(lens[b]), rnd.randrange(kv), rnd.randrange(dim), v)
             for b, v in ((0, nan), (n - 1, -big), (1, nan))]
    # (of the long one in half of the kv-heads only: the others' results are checked)
    plant += [(n // 2, 1, longest - 1 - i * longest // 40, rnd.randrange(max(kv // 2, 1)), rnd.randrange(dim), rnd.choice((nan, big, -big)))
              for i in range(12)]
    kw = dict(heads=heads, kv_heads=kv, dim=dim, dtype=dtype, seed=case, plant=plant,
              spread=(1.0, 12.0)[(case + (dtype == "fp8")) % 2])
    ws = nat.make_masked_workspace()
    if window is None:
        bits = [random_bits(q, rnd, True) for q in q_lens]
        s = Sequences([tree_mask(x, q, b) for x, q, b in zip(lens, q_lens, bits)], whole=True, **kw)
        words = tree_words(bits, s.rows, s.starts, 1)
        run = lambda: nat.attention_tree(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, words, s.scale, ws)  # noqa: E731
    else:
        s = Sequences([window_mask(x, q, window, 5) for x, q in zip(lens, q_lens)], **kw)
        run = lambda: nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, window, 5, s.scale, ws)  # noqa: E731
    hg, flat, parts = plan(lens, q_lens, s.max_q, heads, kv, dtype == "fp8", s.table.shape[1], window, 5)
    want = want if isinstance(want, int) else want[dtype == "fp8"]
    assert hg == want and not flat and parts >= 3, (hg, flat, parts)
    out, lse = run()
    assert nat.read_device_error(ws) == 0
    check(out, lse, s.reference())
    again = run()
    assert torch.equal(again[0].view(torch.int16), out.view(torch.int16)) and torch.equal(again[1].view(torch.int32), lse.view(torch.int32))
