"""Causal attention of packed prompts over rows, against the definition in 64 bits."""

import math

import numpy as np
import pytest
import torch

from paged_kv_decode_14_gb300 import _native as nat

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def reference(q, k, v, q_lens, kv_lens, scale, q_starts=None, kv_starts=None):
    """(out, lse, sum of weights times |v|) in fp64; rows outside every sequence: nan."""
    Hq, Hkv, D = q.shape[1], k.shape[1], q.shape[2]
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    size = torch.zeros_like(out)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float64, device=q.device)
    q0 = k0 = 0
    for b, (Q, L) in enumerate(zip(q_lens, kv_lens)):
        qs = q_starts[b] if q_starts is not None else q0
        ks = k0 if kv_starts is None else kv_starts[b]
        for h in range(Hq):
            kk, vv = (x[ks:ks + L, h // (Hq // Hkv)].double() for x in (k, v))
            s = q[qs:qs + Q, h].double() @ kk.T * scale
            last = L - Q + torch.arange(Q, device=q.device)
            hid = torch.arange(L, device=q.device)[None] > last[:, None]
            # (hidden values take no part: weights 0 and their values 0)
            for i0 in range(0, Q, 512):
                hi, si = hid[i0:i0 + 512], s[i0:i0 + 512].masked_fill(hid[i0:i0 + 512], -math.inf)
                z = torch.logsumexp(si, -1)
                seen = last[i0:i0 + 512] >= 0
                p = torch.where(hi, 0.0, (si - torch.where(seen, z, 0.0)[:, None]).exp())
                p = torch.where(seen[:, None], p, 0.0)
                n = p.shape[0]
                rows = slice(qs + i0, qs + i0 + n)
                fin = torch.isfinite(vv)
                out[rows, h] = p @ torch.where(fin, vv, 0.0)
                size[rows, h] = p @ torch.where(fin, vv, 0.0).abs()
                lse[rows, h] = torch.where(seen, z, -math.inf)
                for j, d in (~fin).nonzero().tolist():
                    out[qs + i0:qs + i0 + n, h, d] += torch.where(hi[:, j], 0.0, vv[j, d])
        q0, k0 = q0 + Q, k0 + L
    return out, lse, size


def check(got, lse, ref, rlse, size, slack=None):
    """out: the weights are rounded to the inputs' type (half a step of each: HALF * sum w|v|, and as
    much again where the sum that divides them holds unrounded weights), the result once more
    (HALF * |out|).  The logits' fp32 error: a sum of at most 128 products of rounding 2^-24 relative
    to sum |q k| -- for these inputs (|q . k| scale <= ~20, sum |q k| scale <= ~130) below
    128 * 2^-24 * 130 = 2^-10.0 at the very worst and, with the tree of the hardware's sums, a few
    2^-24 * 130 = 2^-15; taken as 2^-13 on each weight and on lse."""
    half = HALF[got.dtype]
    eps = 2.0 ** -13
    own = torch.isnan(rlse)
    g, r = got.double(), ref
    fin = torch.isfinite(r) & ~own[:, :, None]
    tol = half * r.abs() + (half + eps) * size * (1 + half) + 2.0 ** -24
    bad = fin & ~((g - r).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {int(fin.sum())} outputs off, first {bad.nonzero()[0].tolist()}: " \
                          f"{g[bad][0].item()} for {r[bad][0].item()}"
    odd = ~torch.isfinite(r) & ~own[:, :, None]
    assert torch.equal(torch.nan_to_num(g[odd], 7.0, 8.0, 9.0), torch.nan_to_num(r[odd], 7.0, 8.0, 9.0))
    inside = ~own & torch.isfinite(rlse)
    assert ((lse.double() - rlse).abs()[inside] <= eps + 2.0 ** -23 * rlse.abs()[inside]).all()
    empty = ~own & (rlse == -math.inf)
    assert (lse[empty] == -math.inf).all() and (got[empty] == 0).all()


def run(Q, L, Hq, Hkv, D, dtype, seed=0, fused=False, ws="yes", scale=None, edit=None):
    dt = TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn(sum(Q), Hq, D, generator=g, device="cuda").to(dt)
    kv = torch.randn(sum(L), 2 * Hkv, D, generator=g, device="cuda").to(dt)
    k, v = (kv[:, :Hkv], kv[:, Hkv:]) if fused else (kv[:, :Hkv].contiguous(), kv[:, Hkv:].contiguous())
    if edit:
        edit(q, k, v)
    ql, kl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (Q, L))
    scale = D ** -0.5 if scale is None else scale
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = nat.make_prompt_workspace() if ws == "yes" else None
    out, lse = nat.prompt_attention(q, k, v, ql, kl, max(max(Q), 1), scale, workspace=w, device_error=err)
    assert nat.read_device_error(err) == 0
    ref, rlse, size = reference(q, k, v, Q, L, scale)
    check(out, lse, ref, rlse, size)
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (4, 4), (3, 1), (7, 1), (10, 2), (64, 1), (100, 1), (5, 5)])
def test_heads(dtype, D, Hq, Hkv):
    run([33, 1, 130], [33, 1, 130], Hq, Hkv, D, dtype, fused=True)
    run([17, 3], [300, 3], Hq, Hkv, D, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2], [15, 16, 17], [31, 32, 33], [63, 64, 65], [127, 128, 129], [255, 256, 257],
                                  [0, 5, 0, 0, 9, 0], [511, 1, 513], [700]])
def test_lengths(dtype, D, lens):
    run(lens, lens, 8, 2, D, dtype, seed=len(lens))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ws", ["yes", "no"])
@pytest.mark.parametrize("Q,L", [([1], [1000]), ([1, 1, 1], [5, 129, 4000]), ([16], [8192]), ([33, 9], [5001, 127]),
                                 ([64, 1], [64, 3000]), ([200], [2500]), ([5], [12345])])
def test_context_before_the_queries(dtype, ws, Q, L):
    run(Q, L, 8, 2, 128, dtype, ws=ws)
    run(Q, L, 8, 2, 64, dtype, ws=ws, fused=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Q,L", [([10], [0]), ([10], [3]), ([300, 5, 7], [40, 5, 0]), ([0, 6], [9, 6]), ([129], [1])])
def test_rows_that_see_nothing(D, Q, L):
    run(Q, L, 6, 2, D, "bf16")
    run(Q, L, 6, 2, D, "fp16")


def test_many_sequences():
    r = np.random.default_rng(3)
    lens = [int(x) for x in r.integers(0, 40, 150)]
    run(lens, lens, 4, 2, 64, "bf16")
    run(lens, [n + int(c) for n, c in zip(lens, r.integers(0, 200, 150))], 4, 1, 128, "fp16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_growing_and_extreme_logits(dtype):
    """The running maximum rises late, by far, and stays finite."""
    def grow(q, k, v):
        k[:] *= torch.linspace(0, 6, k.shape[0], device="cuda")[:, None, None].to(k.dtype)
        k[-40:] *= 4
    out, lse = run([300], [700], 4, 2, 128, dtype, edit=grow, scale=0.05)

    def low(q, k, v):
        q[:] = 1.0
        k[:] = -8.0
        k[350:] = 2.0
    run([500], [500], 2, 1, 128, dtype, edit=low, scale=0.5)       # logits -512, then 128
    run([500], [500], 2, 1, 64, dtype, edit=low, scale=0.5)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_and_inf_reach_only_rows_that_see_them(dtype, D):
    def edit(q, k, v):
        v[150, 0, 3] = math.nan         # seen by rows 150 ..
        v[40, 1, D - 1] = math.inf
        v[299, 1, 7] = -math.inf        # seen by the last row alone
    run([300], [300], 4, 2, D, dtype, edit=edit)

    def keys(q, k, v):
        k[100, 0] = math.nan
        v[:, :, 0] += 1
    dt = TYPES[dtype]
    q = torch.randn(200, 4, D, device="cuda").to(dt)
    k, v = (torch.randn(200, 2, D, device="cuda").to(dt) for _ in range(2))
    keys(q, k, v)
    lens = torch.tensor([200], dtype=torch.int32, device="cuda")
    out, lse = nat.prompt_attention(q, k, v, lens, lens, 200, 0.1)
    assert torch.isfinite(out[:100]).all() and torch.isnan(out[100:, :2]).all() and torch.isfinite(out[:, 2:]).all()
    assert torch.isnan(lse[100:, :2]).all() and torch.isfinite(lse[:100]).all()


@pytest.mark.parametrize("D", [64, 128])
def test_padded_batches_and_neighbours_full_of_nan(D):
    """Starts place sequences in larger tensors; what lies between them is never read into a result
    nor written."""
    dt = torch.bfloat16
    Q, L = [5, 0, 130, 64], [77, 3, 130, 200]
    qs, ks = [3, 10, 20, 170], [10, 100, 120, 256]
    q = torch.full((240, 4, D), math.nan, dtype=dt, device="cuda")
    k = torch.full((470, 2, D), math.nan, dtype=dt, device="cuda")
    v = torch.full((470, 2, D), math.nan, dtype=dt, device="cuda")
    for a, n in zip(qs, Q):
        q[a:a + n] = torch.randn(n, 4, D, device="cuda").to(dt)
    for a, n in zip(ks, L):
        k[a:a + n], v[a:a + n] = (torch.randn(n, 2, D, device="cuda").to(dt) for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")      # noqa: E731
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device="cuda")      # noqa: E731
    for ws in (None, nat.make_prompt_workspace()):
        out = torch.full((240, 4, D), 7.0, dtype=dt, device="cuda")
        lse = torch.full((240, 4), 7.0, device="cuda")
        nat.prompt_attention(q, k, v, i32(Q), i32(L), 130, 0.1, out=out, lse=lse, q_starts=i64(qs), kv_starts=i64(ks),
                             workspace=ws)
        ref, rlse, size = reference(q, k, v, Q, L, 0.1, qs, ks)
        check(out, lse, ref, rlse, size)
        outside = torch.isnan(rlse)
        assert (out[outside] == 7).all() and (lse[outside] == 7).all()


def test_strided_outputs():
    dt, D = torch.bfloat16, 64
    q = torch.randn(50, 4, D, device="cuda").to(dt)
    k, v = (torch.randn(50, 2, D, device="cuda").to(dt) for _ in range(2))
    lens = torch.tensor([20, 30], dtype=torch.int32, device="cuda")
    want, _ = nat.prompt_attention(q, k, v, lens, lens, 30, 0.1)
    buf = torch.full((50, 9, 2 * D), 3.0, dtype=dt, device="cuda")
    nat.prompt_attention(q, k, v, lens, lens, 30, 0.1, out=buf[:, 2:6, D:])
    assert torch.equal(buf[:, 2:6, D:], want)
    assert (buf[:, :2] == 3).all() and (buf[:, 6:] == 3).all() and (buf[:, :, :D] == 3).all()
    heads_first = torch.empty(4, 50, D, dtype=dt, device="cuda")
    qh = q.transpose(0, 1).contiguous().transpose(0, 1)
    nat.prompt_attention(qh, k, v, lens, lens, 30, 0.1, out=heads_first.transpose(0, 1))
    assert torch.equal(heads_first.transpose(0, 1), want)


def test_bad_lengths_are_reported_and_skipped():
    dt, D = torch.bfloat16, 64
    q = torch.randn(64, 2, D, device="cuda").to(dt)
    k, v = (torch.randn(64, 1, D, device="cuda").to(dt) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")      # noqa: E731
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device="cuda")      # noqa: E731
    ok, _ = nat.prompt_attention(q[:20], k[:20], v[:20], i32([20]), i32([20]), 20, 0.1)
    for ql, kl, qs, ks in (([20, 21], [20, 21], None, None), ([20, -1], [20, 5], None, None), ([20, 5], [20, -4], None, None),
                           ([20, 5], [20, 60], None, None), ([20, 5], [20, 5], [0, 60], [0, 20]),
                           ([20, 5], [20, 5], [0, -3], [0, 20]), ([20, 5], [20, 5], [0, 20], [0, 1 << 40])):
        out = torch.full((64, 2, D), 7.0, dtype=dt, device="cuda")
        nat.prompt_attention(q, k, v, i32(ql), i32(kl), 20, 0.1, out=out, q_starts=None if qs is None else i64(qs),
                             kv_starts=None if ks is None else i64(ks), device_error=err,
                             workspace=nat.make_prompt_workspace())
        assert nat.read_device_error(err) == nat.DEVERR_LENGTH
        assert torch.equal(out[:20], ok) and (out[20:] == 7).all()


def test_deterministic_and_capturable():
    dt = torch.bfloat16
    Q, L = [40, 3], [3000, 900]
    q = torch.randn(sum(Q), 8, 128, device="cuda").to(dt)
    k, v = (torch.randn(sum(L), 2, 128, device="cuda").to(dt) for _ in range(2))
    ql, kl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (Q, L))
    ws = nat.make_prompt_workspace()
    a = nat.prompt_attention(q, k, v, ql, kl, 40, 0.1, workspace=ws)
    out, lse = torch.zeros_like(q), torch.zeros(sum(Q), 8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        nat.prompt_attention(q, k, v, ql, kl, 40, 0.1, out=out, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nat.prompt_attention(q, k, v, ql, kl, 40, 0.1, out=out, lse=lse, workspace=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, a[0]) and torch.equal(lse, a[1])
    # other lengths in the same graph
    ql.copy_(torch.tensor([17, 1], dtype=torch.int32))
    kl.copy_(torch.tensor([2000, 1], dtype=torch.int32))
    g.replay()
    ref, rlse, size = reference(q[:18], k, v, [17, 1], [2000, 1], 0.1)
    check(out[:18], lse[:18], ref, rlse, size)
