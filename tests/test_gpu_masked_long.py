"""Masked attention over very long contexts: pieces of work that take longer than the wait limit, and calls refused by their
size."""

import math

import pytest
import torch

from paged_kv_decode_14_gb300 import _native as nat

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_long_pieces_do_not_run_out_of_time():
    """19 contexts of 2^24 keys, the same 1024 over and over: some 16000 key tiles a CTA, with a wait limit of 2 ms."""
    seqs, length, blocks, dim = 19, 1 << 24, 64, 64
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(blocks, 1, 2, dim // 8, 8, 8, generator=g, device="cuda").bfloat16() for _ in range(2))
    cache = nat.PagedKVCache(blocks, 1, dim, "bf16", k=k.view(blocks, 1, 16 * dim), v=v.view(blocks, 1, 16 * dim))
    table = (torch.arange(length // 16, device="cuda", dtype=torch.int32) % blocks).expand(seqs, -1).contiguous()
    q = torch.randn(seqs, 1, dim, generator=g, device="cuda").bfloat16()
    ws = nat.make_masked_workspace()
    torch.cuda.synchronize()
    nat.debug_set_wait_limit(2_000_000, None)
    try:
        out, lse = nat.attention_window(cache, q, table, ints([length] * seqs), ints([1] * seqs), 1, 1 << 30, 0, 0.125, ws)
        torch.cuda.synchronize()
    finally:
        nat.debug_set_wait_limit(0, None)
    assert nat.read_device_error(ws) == 0
    rows = [x.permute(0, 1, 2, 4, 3, 5).reshape(16 * blocks, dim).double() for x in (k, v)]
    x = q[:, 0].double() @ rows[0].t() * 0.125
    p = torch.softmax(x, -1)
    want, size = p @ rows[1], p @ rows[1].abs()
    # P and out rounded to bf16; the sums: each of a part's up to 2^15 additions in fp32 rounds by 2^-24 of the sum at most
    assert ((out[:, 0].double() - want).abs() <= (2.0 ** -8 + 3 * 2.0 ** -9) * size + 2.0 ** -8 * want.abs()).all()
    z = torch.logsumexp(x, -1) + math.log(length / (16 * blocks))
    assert ((lse[:, 0].double() - z).abs() <= 2 * 2.0 ** -9).all()


@pytest.mark.parametrize("tree", [False, True])
def test_more_work_than_a_call_takes_is_refused(tree):
    """5 sequences of 2^26 keys and 1024 kv-heads, four of them an item: more than 2^31 units.  No table entry is read
    (they are out of range), nothing is written."""
    seqs, length, heads, dim = 5, 1 << 26, 1024, 64
    cache = nat.PagedKVCache(2, heads, dim, "bf16")
    cache.k.zero_()
    cache.v.zero_()
    table = torch.full((seqs, length // 16), 1 << 30, dtype=torch.int32, device="cuda")
    q = torch.ones(seqs, heads, dim, device="cuda").bfloat16()
    ws = nat.make_masked_workspace()
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    args = (cache, q, table, ints([length] * seqs), ints([1] * seqs), 1)
    if tree:
        nat.attention_tree(*args, torch.ones(seqs, 1, dtype=torch.int32, device="cuda"), 0.125, ws, out=out, lse=lse)
    else:
        nat.attention_window(*args, 1 << 30, 0, 0.125, ws, out=out, lse=lse)
    assert nat.read_device_error(ws) == nat.DEVERR_LENGTH
    assert (out == 7.0).all() and (lse == 7.0).all()
    one = nat.attention_window(cache, q[:1], table[:1].zero_(), ints([20]), ints([1]), 1, 1 << 30, 0, 0.125, ws)
    assert nat.read_device_error(ws) == 0 and torch.isfinite(one[1]).all()
