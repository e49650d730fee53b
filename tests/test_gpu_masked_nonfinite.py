"""Values that are not finite: what they cost a call, where they lie in its pieces of work, and what must not become one."""

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


def time_of(call):
    call()
    times = []
    for _ in range(3):
        a, b = torch.cuda.Event(True), torch.cuda.Event(True)
        torch.cuda.synchronize()
        a.record()
        call()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("heads,seqs", [(8, 64), (2, 8)])                # four kv-heads an item, and one
def test_one_value_does_not_slow_a_call_down(heads, seqs, dtype, workspace):
    length, dim = 4096, 128
    blocks = seqs * length // 16
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(blocks, heads, 16 * dim, generator=g, device="cuda").bfloat16() for _ in range(2))
    scales = [None, None]
    if dtype == "fp8":
        k, v = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
        scales = [torch.ones(blocks, heads, device="cuda") for _ in range(2)]
    cache = nat.PagedKVCache(blocks, heads, dim, dtype, k=k, v=v, k_scales=scales[0], v_scales=scales[1])
    table = torch.randperm(blocks, generator=g, device="cuda").int().view(seqs, -1)
    q = torch.randn(seqs, 4 * heads, dim, generator=g, device="cuda").bfloat16()
    lens, one = (torch.full((seqs,), n, dtype=torch.int32, device="cuda") for n in (length, 1))

    def call():
        return nat.attention_window(cache, q, table, lens, one, 1, 1 << 20, 0, dim ** -0.5, workspace)

    before, clean = call()[0], time_of(call)
    v[table[:, 77].long(), 1, 5] = 0x7f if dtype == "fp8" else math.nan     # a key, a dimension of each sequence's
    after, marked = call()[0], time_of(call)
    assert nat.read_device_error(workspace) == 0
    bad = torch.isnan(after)
    assert bad.sum() == seqs * 4 and bad[:, 4:8].any(-1).all()
    assert torch.equal(after[~bad], before[~bad])
    assert marked < 4 * clean + 0.3, f"{clean} ms, with NaN {marked} ms"
    v[:, :, :] = 0x7f if dtype == "fp8" else math.nan                       # everything
    after, full = call()[0], time_of(call)
    assert nat.read_device_error(workspace) == 0 and torch.isnan(after).all()
    assert full < 100, f"{clean} ms, with NaN alone {full} ms"


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("heads,kv,q_len", [(16, 8, 1), (8, 2, 5), (8, 4, 90), (4, 1, 3)])
def test_values_anywhere_in_long_pieces(heads, kv, q_len, dtype, workspace):
    """Some dozens of values at both ends and in between of contexts whose pieces have more tiles than marks."""
    rnd = random.Random(q_len)
    lens, q_lens = [9000, 300, 3333], [q_len, 1, q_len]
    plant = []
    for b, n in enumerate(lens):
        for j in [0, 1, n - 1, n - 2, n - 17] + [rnd.randrange(n) for _ in range(12)]:
            value = math.nan if dtype == "fp8" else rnd.choice((math.nan, math.inf, -math.inf))
            plant.append((b, 1, j, rnd.randrange(kv), rnd.randrange(64), value))
    kw = dict(heads=heads, kv_heads=kv, dim=64, dtype=dtype, seed=q_len, plant=plant)
    for window, sinks in ((1 << 20, 0), (4000, 3)):
        s = Sequences([window_mask(n, q, window, sinks) for n, q in zip(lens, q_lens)], **kw)
        out, lse = nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, window, sinks, s.scale, workspace)
        assert nat.read_device_error(workspace) == 0
        check(out, lse, s.reference())
    bits = [torch.rand(q, q, generator=torch.Generator().manual_seed(q)) < 0.5 for q in q_lens]
    s = Sequences([tree_mask(n, q, m) for n, q, m in zip(lens, q_lens, bits)], whole=True, **kw)
    words = tree_words(bits, s.rows, s.starts, 3)
    out, lse = nat.attention_tree(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, words, s.scale, workspace)
    assert nat.read_device_error(workspace) == 0
    check(out, lse, s.reference())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("q_len", [1, 80])
def test_logits_of_zero_with_the_largest_scale(q_len, dtype, workspace):
    """scale times log2 e leaves fp32's range: queries of 0 see the mean of their keys' values all the same."""
    s = Sequences([window_mask(n, q_len, 50, 3) for n in (200, 90)], 8, 2, 64, dtype, 8)
    s.q.zero_()
    s.scale = 3.4e38
    out, lse = nat.attention_window(s.cache, s.q, s.table, s.t_lens, s.t_q, s.max_q, 50, 3, s.scale, workspace)
    assert nat.read_device_error(workspace) == 0
    check(out, lse, s.reference())
