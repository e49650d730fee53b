"""Kernels that read another's outputs right behind it: lengths, tables and slots of pkv_block_tables_update in the append and
in pkv_paged_attention, which begins before the kernels ahead of it have ended."""

import random

import pytest
import torch

from masked_helpers import page_view
from paged_kv_decode_14_gb300 import _native as nat
from test_gpu_step_tables import Model, ints, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype,seqs", [("bf16", 48), ("fp8", 7)])
def test_tables_append_full_attention(dtype, seqs, captured):
    """A layer of full attention in a loop whose tables grow on the GPU.  Between steps every array that the next step's
    kernels read early holds other values than those that it writes."""
    rnd = random.Random(seqs)
    heads, kv, dim = 8, 2, 128
    m = Model(seqs * 14, 12, [rnd.randint(0, 150) for _ in range(seqs)], rnd)
    pool, table, lens = on_gpu(m)
    kvs = dict(k_scales=torch.full((seqs * 14, kv), 0.02, device="cuda"), v_scales=torch.full((seqs * 14, kv), 0.02, device="cuda"))
    cache = nat.PagedKVCache(seqs * 14, kv, dim, dtype, **(kvs if dtype == "fp8" else {}))
    for x in (cache.k, cache.v):
        x.copy_((torch.randn(x.shape, device="cuda") * (30 if dtype == "fp8" else 1)).to(
            torch.float8_e4m3fn if dtype == "fp8" else x.dtype).view(x.dtype))
    grow, err = ints([0] * seqs), ints([0])
    k, v = (torch.randn(seqs, kv, dim, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(seqs, heads, dim, device="cuda").bfloat16()
    ws, out = nat.make_workspace(seqs, heads, kv, dim, 1), torch.empty_like(q)
    slots, positions = (torch.empty(seqs, dtype=t, device="cuda") for t in (torch.int64, torch.int32))
    granted, starts = torch.empty(seqs, dtype=torch.int32, device="cuda"), torch.empty(seqs, dtype=torch.int64, device="cuda")

    def step():
        nat.update_tables(pool, table, lens, grow, seqs, slots=slots, positions=positions, granted=granted, row_starts=starts,
                          pad=True, device_error=err)
        nat.append(cache, k, v, slots, device_error=err)
        nat.attention(cache, q, table, lens, granted, 1, dim ** -0.5, ws, out=out)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    call = step
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        call = graph.replay
    for turn in range(30):
        change = [1 if m.lens[b] < 190 else -150 for b in range(seqs)]
        grow.copy_(ints(change))
        slots.fill_(rnd.randrange(seqs * 14 * 16))                       # (all of them one valid slot)
        granted.fill_(1)
        was_k, was_v = cache.k.clone(), cache.v.clone()
        rows, given, _, code = m.update(change, seqs)
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        assert nat.read_device_error(err) == code == 0 and nat.read_device_error(ws) == 0
        at = torch.tensor([w[0] for w in rows], device="cuda")
        n = len(rows)
        assert slots.tolist() == at.tolist() + [-1] * (seqs - n)
        for was, now, x, sc in ((was_k, cache.k, k, cache.k_scales), (was_v, cache.v, v, cache.v_scales)):
            y = x[:n] if dtype == "bf16" else (x[:n].float() / 0.02).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            c = 16 // y.element_size()
            page_view(was, kv, dim)[at // 16, :, at % 16 // 8, :, at % 8, :] = y.view(n, kv, dim // c, c)
            assert torch.equal(was, now)
        # attention against 64 bits, from the cache as it is (packed rows: requests that grew, in order)
        pages = []
        for x, sc in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
            p = page_view(x, kv, dim)
            p = (p.view(torch.float8_e4m3fn) if dtype == "fp8" else p).double()
            p = p if sc is None else p * sc.double()[:, :, None, None, None, None]
            pages.append(p.permute(0, 2, 4, 1, 3, 5).reshape(-1, 16, kv, dim))
        i = 0
        for b in range(seqs):
            if given[b] == 0:
                continue
            kk, vv = (p[table[b, :(m.lens[b] + 15) // 16].long()].reshape(-1, kv, dim)[:m.lens[b]] for p in pages)
            x = torch.einsum("kgd,tkd->kgt", q[i].double().view(kv, heads // kv, dim), kk) * dim ** -0.5
            want = torch.einsum("kgt,tkd->kgd", torch.softmax(x, -1), vv).reshape(heads, dim)
            assert ((out[i].double() - want).abs() <= 2e-3 + 1e-2 * want.abs()).all()
            i += 1


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kind", ["rope", "rope_scales", "norm_rope", "norm_rope_scales"])
def test_tables_and_appends_that_rotate(kind, captured):
    """Slots and positions of the call before, in the appends that rotate: the cache and q as with slots and positions that
    were there long before."""
    rnd = random.Random(2)
    seqs, heads, kv, dim, bound = 9, 4, 2, 64, 30
    dtype = "fp8" if "scales" in kind else "bf16"
    m = Model(seqs * 14, 12, [rnd.randint(0, 60) for _ in range(seqs)], rnd)
    pool, table, lens = on_gpu(m)
    sc = lambda: dict(k_scales=torch.ones(seqs * 14, kv, device="cuda"), v_scales=torch.ones(seqs * 14, kv, device="cuda"))  # noqa: E731
    caches = [nat.PagedKVCache(seqs * 14, kv, dim, dtype, **(sc() if dtype == "fp8" else {})) for _ in range(2)]
    for c in caches:
        c.k.zero_()
        c.v.zero_()
    k, v = (torch.randn(bound, kv, dim, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(bound, heads, dim, device="cuda").bfloat16()
    grow, rope = ints([0] * seqs), nat.Rope(dim)
    slots, positions = (torch.zeros(bound, dtype=t, device="cuda") for t in (torch.int64, torch.int32))

    def append(cache, slots, positions, q):
        if kind.startswith("norm"):
            return nat.append_norm_rope(cache, q, k, v, slots, positions=positions, rope=rope, fp8_scales_from_values="scales" in kind)
        nat.append_rope(cache, k, v, slots, positions=positions, q=q, fp8_scales_from_values="scales" in kind)
        return q

    inplace = q.clone()

    def step():
        nat.update_tables(pool, table, lens, grow, bound, slots=slots, positions=positions, pad=True)
        return append(caches[0], slots, positions, inplace)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    call = step
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        call = lambda: graph.replay() or got  # noqa: E731
    for turn in range(12):
        change = [rnd.randint(0, 3) if m.lens[b] < 180 else -100 for b in range(seqs)]
        grow.copy_(ints(change))
        rows, _, _, code = m.update(change, bound)
        inplace.copy_(q)
        slots.fill_(rnd.randrange(seqs * 14 * 16))
        positions.fill_(rnd.randrange(1000))
        torch.cuda.synchronize()
        out = call()
        torch.cuda.synchronize()
        n = len(rows)
        want = append(caches[1], torch.tensor([w[0] for w in rows] + [-1] * (bound - n), device="cuda"),
                      ints([w[1] for w in rows] + [0] * (bound - n)), q.clone())
        assert code == 0 and torch.equal(out[:n], want[:n])
        assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
        if dtype == "fp8":
            assert torch.equal(caches[0].k_scales, caches[1].k_scales) and torch.equal(caches[0].v_scales, caches[1].v_scales)
