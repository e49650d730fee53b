"""Block tables whose number of rows is only a bound: rows behind the last request's, and captured steps in which requests
stop growing, drop tokens and pass their blocks on."""

import random

import pytest
import torch

from masked_helpers import page_view
from paged_kv_decode_14_gb300 import _native as nat
from test_gpu_step_tables import Model, blocks, ints, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bound", [40, 2048, 2049, 70000])               # (above 2048 rows a cluster of CTAs)
def test_rows_behind_the_last(bound):
    rnd = random.Random(bound)
    m = Model(300, 40, [rnd.randint(0, 90) for _ in range(20)], rnd)
    state = on_gpu(m)
    for grow in ([1, 0, 2, -1] * 5, [0, -1] * 10, [2] * 20, [3] * 20):   # (the last: more rows than 40)
        want = m.update(grow, bound)[0]
        slots, positions, granted, starts = nat.update_tables(*state, ints(grow), bound)
        assert slots.tolist() == [w[0] for w in want] + [-1] * (bound - len(want))
        assert positions.tolist() == [w[1] for w in want] + [0] * (bound - len(want))
        assert state[1].tolist() == m.table and state[2].tolist() == m.lens


def test_rows_of_given_tensors():
    rnd = random.Random(0)
    for pad, rest in ((None, 77), (False, 77), (True, None)):
        m = Model(60, 8, [20, 30], rnd)
        state = on_gpu(m)
        slots = torch.full((9,), 77, dtype=torch.int64, device="cuda")
        positions = torch.full((8,), 77, dtype=torch.int32, device="cuda")
        want = m.update([1, 2], 8)[0]
        nat.update_tables(*state, ints([1, 2]), 8, slots=slots[:8], positions=positions, pad=pad)
        assert slots.tolist() == [w[0] for w in want] + [-1 if rest is None else rest] * 5 + [77]
        assert positions.tolist() == [w[1] for w in want] + [0 if rest is None else rest] * 5


def test_no_requests():
    empty = ints([])
    slots, positions, granted, starts = nat.update_tables(nat.BlockPool(8), torch.empty(0, 4, dtype=torch.int32, device="cuda"),
                                                          empty, empty, 5)
    assert slots.tolist() == [-1] * 5 and positions.tolist() == [0] * 5 and granted.numel() == starts.numel() == 0


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("seqs,bound", [(6, 24), (40, 2100)])
def test_captured_steps_with_a_bound(seqs, bound, given):
    """update, append of all `bound` rows and windowed attention in one graph; the changes are new in each replay.  The
    whole cache is compared after each: nothing but the new tokens' rows may change."""
    rnd = random.Random(seqs + given)
    heads, dim, num = 2, 64, seqs * 6 + 3
    m = Model(num, 12, [0] * seqs, rnd)
    pool, table, lens = on_gpu(m)
    cache = nat.PagedKVCache(num, heads, dim, "bf16", k=torch.zeros(num, heads, 16 * dim, dtype=torch.bfloat16, device="cuda"),
                             v=torch.zeros(num, heads, 16 * dim, dtype=torch.bfloat16, device="cuda"))
    grow, err, ws = ints([0] * seqs), ints([0]), nat.make_masked_workspace()
    k, v = (torch.zeros(bound, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.randn(bound, 2 * heads, dim, device="cuda").bfloat16()
    out = torch.empty_like(q)
    kw = {}
    if given:
        kw = dict(slots=torch.empty(bound, dtype=torch.int64, device="cuda"), pad=True,
                  positions=torch.empty(bound, dtype=torch.int32, device="cuda"))

    def step():
        slots, positions, granted, starts = nat.update_tables(pool, table, lens, grow, bound, device_error=err, **kw)
        nat.append(cache, k, v, slots, device_error=err)
        nat.attention_window(cache, q, table, lens, granted, bound, 40, 2, 0.125, ws, out=out, q_starts=starts)
        return slots

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()                                                           # (no request grows)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        slots = step()
    want_k, want_v = cache.k.clone(), cache.v.clone()
    most = bound // seqs
    for turn in range(25):
        change = [rnd.choice((0, 1, most, rnd.randint(0, most), -rnd.randint(0, m.lens[b]), -m.lens[b])) for b in range(seqs)]
        if turn % 6 == 5:
            change = [min(c, 0) for c in change]                         # nobody grows
        change = [min(c, 190 - m.lens[b]) for b, c in enumerate(change)]
        grow.copy_(ints(change))
        k.copy_(torch.randn(k.shape, device="cuda"))
        v.copy_(torch.randn(v.shape, device="cuda"))
        rows, granted, _, code = m.update(change, bound)
        graph.replay()
        at = torch.tensor([w[0] for w in rows], dtype=torch.int64, device="cuda")
        new = (at >= 0).nonzero()[:, 0]
        for pool_, x in ((want_k, k), (want_v, v)):
            s = at[new]
            page_view(pool_, heads, dim)[s // 16, :, s % 16 // 8, :, s % 8, :] = x[new].view(len(new), heads, dim // 8, 8)
        assert slots.tolist() == at.tolist() + [-1] * (bound - len(rows))
        assert torch.equal(cache.k, want_k) and torch.equal(cache.v, want_v)
        assert lens.tolist() == m.lens and table.tolist() == m.table
        assert nat.read_device_error(err) == code and nat.read_device_error(ws) == 0
        assert len({t for b in range(seqs) for t in m.table[b][:blocks(m.lens[b])]}) == sum(map(blocks, m.lens))
