"""The row operators used together, and the calls around their edges: a prompt served from projections to
decode, graphs and streams, timeouts, scales at the ends of fp32, addresses past 2^31."""

import math
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

from paged_kv_decode_14_gb300 import _native as nat
from gpu_helpers import ATOL, RTOL
from test_gpu_prompt import check, reference, run
from test_gpu_rows import assert_rows, clone, make, new_cache, page_rows, ref_rows, same_cache

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 6, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_prompt_chunk_decode(dtype, D, Hq, Hkv):
    """Three prompts: the first chunk attends its own rows, the second the context read back from the
    cache, then one decode step attends the cache; each against 64 bits from the rows it was given."""
    first, second, nb = [40, 16, 129], [25, 3, 16], 64
    B, fp8 = len(first), dtype == "fp8"
    per = [-(-(a + b + 1) // 16) for a, b in zip(first, second)]
    ids = np.random.default_rng(D).permutation(nb)
    table = np.zeros((B, max(per)), np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = ids[at:at + n]
        at += n
    slot = lambda b, p: int(table[b, p // 16]) * 16 + p % 16
    c = new_cache(nb, Hkv, D, dtype, seed=D)
    tables = torch.from_numpy(table).cuda()
    rope = nat.Rope(D, 10000.0, False, "bands", 4.0, 64, 1.0, 4.0)
    qw, kw = ((1 + 0.2 * torch.randn(D, device="cuda")).bfloat16() for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws, scale = nat.make_prompt_workspace(), D ** -0.5

    def step(new, have, seed):
        T = sum(new)
        q, k, v = make(T, (Hq, Hkv, Hkv), D, torch.bfloat16, seed)
        pos = i32([have[b] + i for b in range(B) for i in range(new[b])])
        slots = torch.tensor([slot(b, have[b] + i) for b in range(B) for i in range(new[b])], dtype=torch.int64, device="cuda")
        ko = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
        qo = nat.append_norm_rope(c, q, k, v, slots, pos, rope, qw, kw, 1e-6, k_out=ko, fp8_scales_from_values=fp8,
                                  device_error=err)
        assert_rows(qo, *ref_rows(q, qw, 1e-6, pos, rope), "q")
        assert_rows(ko, *ref_rows(k, kw, 1e-6, pos, rope), "k")
        return qo, ko, v

    def context(lens, dt=torch.bfloat16):
        k, v = nat.read_cache(c, tables, i32(lens), sum(lens), dtype=dt, device_error=err)
        # what it reads is what the pages hold
        pk, pv = page_rows(c.k, D, 1 if fp8 else 2), page_rows(c.v, D, 1 if fp8 else 2)
        r = 0
        for b, n in enumerate(lens):
            for p in (0, n // 2, n - 1):
                blk = int(table[b, p // 16])
                for got, page, sc in ((k, pk, c.k_scales), (v, pv, c.v_scales)):
                    want = page[blk, :, p % 16].float() * (sc[blk][:, None] if fp8 else 1.0)
                    assert torch.equal(got[r + p], want.to(dt))
            r += n
        return k, v

    q, k, v = step(first, [0] * B, 1)
    out, lse = nat.prompt_attention(q, k, v, i32(first), i32(first), max(first), scale, workspace=ws, device_error=err)
    check(out, lse, *reference(q, k, v, first, first, scale))

    q, _, _ = step(second, first, 2)
    lens = [a + b for a, b in zip(first, second)]
    k, v = context(lens)
    out, lse = nat.prompt_attention(q, k, v, i32(second), i32(lens), max(second), scale, workspace=ws, device_error=err)
    check(out, lse, *reference(q, k, v, second, lens, scale))

    q, _, _ = step([1] * B, lens, 3)
    lens = [n + 1 for n in lens]
    k, v = context(lens, torch.float32)
    aw = nat.make_workspace(B, Hq, Hkv, D, 1)
    out = nat.attention(c, q, tables, i32(lens), i32([1] * B), 1, scale, aw)
    ref, _, _ = reference(q, k, v, [1] * B, lens, scale)
    assert ((out.double() - ref).abs() <= ATOL + RTOL * ref.abs()).all()
    assert nat.read_device_error(err) == 0


def test_scales_at_the_ends_of_fp32():
    """Continuing a block with any scale a cache may hold gives the IEEE quotient's code, as append does."""
    tiny = [0.0, -0.0, 2.0 ** -149, 2.0 ** -127, 2.0 ** -126, 2.0 ** -101, 2.0 ** -100, 2.0 ** -99, 1e-20, 448.0 ** -1, 1.0,
            2.0 ** 99, 2.0 ** 100, 2.0 ** 101, 2.0 ** 127, math.inf, math.nan, -1.0, -2.0 ** -126]
    nb, Hkv, D = len(tiny), 2, 64
    c = new_cache(nb, Hkv, D, "fp8")
    c.k_scales[:] = torch.tensor(tiny, device="cuda")[:, None]
    c.v_scales[:] = torch.tensor(tiny[::-1], device="cuda")[:, None]
    T = 3 * nb
    slots = torch.tensor([b * 16 + o for b in range(nb) for o in (1, 5, 15)], dtype=torch.int64, device="cuda")
    _, k, v = make(T, (1, Hkv, Hkv), D, torch.bfloat16, 9)
    k, v = k.clone(), v.clone()
    k[::3] *= 2.0 ** -120                      # quotients near 1 for the smallest scales too
    v[::3] *= 2.0 ** -120
    k[1::3] *= 2.0 ** 110
    v[1::3] *= 2.0 ** 110
    k[0, 0, 0], k[1, 0, 1], v[2, 1, 2] = math.inf, math.nan, -math.inf
    a, b = clone(c), clone(c)
    nat.append(a, k, v, slots)
    nat.append_norm_rope(b, None, k, v, slots)
    for x, y in ((a.k, b.k), (a.v, b.v)):
        nan = ((x & 127) == 127) & ((y & 127) == 127)       # (either sign of NaN)
        assert bool(((x == y) | nan).all())


def test_codes_next_to_rounding_boundaries():
    """Values whose quotient by the scale falls on, or one fp32 step beside, the middle between two codes."""
    codes = torch.arange(0, 127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).float()
    mid = ((codes[1:] + codes[:-1]) / 2).double()
    Hkv, D = 1, 64
    nb = 64
    c = new_cache(nb, Hkv, D, "fp8")
    g = torch.Generator(device="cuda").manual_seed(4)
    # for a bf16 value x and a middle m, the scale x / m to fp32, a step up and a step down
    x = torch.randn(nb, generator=g, device="cuda").abs().add(0.5).bfloat16()
    m = mid[torch.randint(0, mid.numel(), (nb,), generator=g, device="cuda")]
    s = (x.double() / m).float()
    s = torch.stack([torch.nextafter(s, torch.zeros_like(s)), s, torch.nextafter(s, torch.full_like(s, 9e9))])[
        torch.arange(nb, device="cuda") % 3, torch.arange(nb, device="cuda")]
    c.k_scales[:, 0] = s
    c.v_scales[:, 0] = s
    slots = torch.arange(nb, device="cuda") * 16 + 3
    k = x[:, None, None].expand(nb, Hkv, D).contiguous()
    a, b = clone(c), clone(c)
    nat.append(a, k, -k, slots)
    nat.append_norm_rope(b, None, k, -k, slots)
    assert same_cache(a, b)


def test_captured_and_on_another_stream():
    """One graph of rows, append, read and attention, replayed with other inputs in the same tensors."""
    D, Hq, Hkv, T = 128, 8, 2, 50
    rope = nat.Rope(D)
    c = new_cache(8, Hkv, D, "fp8")
    q, k, v = (x.clone() for x in make(T, (Hq, Hkv, Hkv), D, torch.bfloat16, 1))
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    slots = torch.arange(T, device="cuda", dtype=torch.int64) + 16
    tables, lens = i32([[1, 2, 3, 4]]), i32([T])
    qo, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(T, Hq, device="cuda")
    kr, vr = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    kn = torch.empty_like(kr)
    ws = nat.make_prompt_workspace()

    def work():
        nat.qk_norm_rope(q, k, pos, rope, eps=1e-5, q_out=qo, k_out=kn)
        nat.append_norm_rope(c, None, kn, v, slots, fp8_scales_from_values=True)
        nat.read_cache(c, tables, lens, T, k_out=kr, v_out=vr)
        nat.prompt_attention(qo, kr, vr, lens, lens, T, 0.1, out=out, lse=lse, workspace=ws)

    work()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            work()
    torch.cuda.current_stream().wait_stream(s)
    for seed in (1, 2, 3):
        for x, y in zip((q, k, v), make(T, (Hq, Hkv, Hkv), D, torch.bfloat16, seed)):
            x.copy_(y)
        for x in (out, lse, kr, vr, kn, qo):
            x.zero_()
        g.replay()
        got = [x.clone() for x in (qo, kn, kr, vr, out, lse)]
        work()
        for x, y in zip(got, (qo, kn, kr, vr, out, lse)):
            assert torch.equal(x, y)
        check(out, lse, *reference(qo, kr, vr, [T], [T], 0.1))
    # a stream given by its handle, while the current one is another
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    a, _ = nat.qk_norm_rope(q, None, pos, rope, eps=1e-5, stream=other)
    other.synchronize()
    assert torch.equal(a, qo)


@pytest.mark.parametrize("L", [300, 5000])
def test_wait_timeout_reports_and_recovers(L):
    """The bounded waits, made to run out by a hold flag that nothing sets; the next call is right.  L = 5000:
    the launch that is split along the keys, with its join."""
    q = torch.randn(300, 4, 128, device="cuda").bfloat16()
    k, v = (torch.randn(L, 2, 128, device="cuda").bfloat16() for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    hold = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = nat.make_prompt_workspace()
    ws.fill_(0xFF)
    ql, kl = i32([300]), i32([L])
    try:
        nat.debug_set_wait_limit(200_000, hold)
        nat.prompt_attention(q, k, v, ql, kl, 300, 0.1, workspace=ws, device_error=err)
        torch.cuda.synchronize()
    finally:
        nat.debug_set_wait_limit(0, None)
    assert nat.read_device_error(err) == nat.DEVERR_TIMEOUT
    out, lse = nat.prompt_attention(q, k, v, ql, kl, 300, 0.1, workspace=ws, device_error=err)
    check(out, lse, *reference(q, k, v, [300], [L], 0.1))
    assert nat.read_device_error(err) == 0


@pytest.mark.parametrize("n", [33, 1500])
def test_more_sequences_than_lanes(n):
    """Ragged batches whose plan takes more than one sequence a lane, whole and cut along the keys."""
    r = np.random.default_rng(n)
    Q = [int(x) for x in r.integers(0, 5, n)]
    L = [q + int(x) for q, x in zip(Q, r.integers(-3, 300, n))]
    L = [max(x, 0) for x in L]
    L[n // 2] += 4000
    run(Q, L, 2, 1, 64, "fp16")
    run(Q, Q, 4, 2, 128, "bf16", ws="no")


def test_large_strides():
    """Head strides of 256 MB (eight heads past 2^31 bytes) and token strides of 512 MB."""
    D, T = 64, 3
    buf = torch.empty(9 << 27, dtype=torch.bfloat16, device="cuda")
    q = buf.as_strided((T, 9, D), (D, 1 << 27, 1))
    src = torch.randn(T, 9, D, device="cuda").bfloat16()
    q.copy_(src)
    pos = i32([5, 70000, 3])
    rope = nat.Rope(D)
    out, _ = nat.qk_norm_rope(q, None, pos, rope, eps=1e-6)
    assert_rows(out, *ref_rows(src, None, 1e-6, pos, rope))
    nat.qk_norm_rope(q, None, pos, rope, eps=1e-6, q_out=q)
    assert torch.equal(q, out)
    kv = buf.as_strided((4, 2, D), (1 << 28, D, 1))
    src = torch.randn(4, 2, D, device="cuda").bfloat16()
    kv.copy_(src)
    qs = torch.randn(4, 4, D, device="cuda").bfloat16()
    a = nat.prompt_attention(qs, kv, kv, i32([4]), i32([4]), 4, 0.1)
    b = nat.prompt_attention(qs, src, src, i32([4]), i32([4]), 4, 0.1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_cache_past_2_31_bytes():
    """Blocks whose pages lie past 2^31 elements of the cache."""
    Hkv, D = 8, 128
    nb = (1 << 31) // (Hkv * 16 * D) + 8
    k, v = (torch.empty(nb, Hkv, 16 * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(nb, Hkv, device="cuda") for _ in range(2))
    c = nat.PagedKVCache(nb, Hkv, D, "fp8", k=k, v=v, k_scales=ks, v_scales=vs)
    blocks = [nb - 1, 0, nb - 8]
    slots = torch.tensor([b * 16 + i for b in blocks for i in range(16)], dtype=torch.int64, device="cuda")
    _, kr, vr = make(48, (1, Hkv, Hkv), D, torch.bfloat16, 2)
    nat.append_norm_rope(c, None, kr, vr, slots, fp8_scales_from_values=True)
    small = new_cache(3, Hkv, D, "fp8")
    nat.append_norm_rope(small, None, kr, vr, torch.arange(48, device="cuda"), fp8_scales_from_values=True)
    a = nat.read_cache(c, i32([blocks]), i32([48]), 48)
    b = nat.read_cache(small, i32([[0, 1, 2]]), i32([48]), 48)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # within half a code of what was written: e4m3's step is at most 2^-3 of the value, or 2^-9 of a scale
    sc = kr.float().abs().view(3, 16, Hkv, D).amax((1, 3)) / 448
    tol = kr.float().abs() * (2.0 ** -4 + 2.0 ** -8) + (sc * 2.0 ** -10).repeat_interleave(16, 0)[:, :, None]
    assert ((a[0].float() - kr.float()).abs() <= tol).all()


def test_two_streams_at_once():
    """Calls in flight on two streams, each with a workspace of its own, as one after the other."""
    Q, L, Hq, Hkv, D = [70, 3], [3000, 700], 8, 2, 128
    sets, want = [], []
    for seed in range(2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        q = torch.randn(sum(Q), Hq, D, generator=g, device="cuda").bfloat16()
        k, v = (torch.randn(sum(L), Hkv, D, generator=g, device="cuda").bfloat16() for _ in range(2))
        out, lse = torch.empty_like(q), torch.empty(sum(Q), Hq, device="cuda")
        sets.append((q, k, v, out, lse, nat.make_prompt_workspace()))
    ql, kl, pos, rope = i32(Q), i32(L), i32(list(range(sum(L)))), nat.Rope(D, interleaved=True)

    def work(s, stream=None):
        q, k, v, out, lse, ws = s
        kr, _ = nat.qk_norm_rope(k, None, pos, rope, eps=1e-6, stream=stream)
        nat.prompt_attention(q, kr, v, ql, kl, max(Q), 0.1, out=out, lse=lse, workspace=ws, stream=stream)
        return kr

    for s in sets:
        work(s)
        want.append((s[3].clone(), s[4].clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        keep = [work(s, st) for _ in range(3) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for s, (out, lse) in zip(sets, want):
            assert torch.equal(s[3], out) and torch.equal(s[4], lse)
        del keep


def test_workspace_is_left_between_calls_of_any_size():
    """One workspace for split and whole calls in turn: nothing of the last call is taken over."""
    ws = nat.make_prompt_workspace()
    g = torch.Generator(device="cuda").manual_seed(3)
    for Q, L in (([40], [5000]), ([3, 3], [3, 3]), ([1] * 9, [1300] * 9), ([600], [700]), ([40], [5000])):
        q = torch.randn(sum(Q), 6, 64, generator=g, device="cuda").half()
        k, v = (torch.randn(sum(L), 3, 64, generator=g, device="cuda").half() for _ in range(2))
        out, lse = nat.prompt_attention(q, k, v, i32(Q), i32(L), max(Q), 0.125, workspace=ws)
        check(out, lse, *reference(q, k, v, Q, L, 0.125))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("octaves", [6, 12, 18])
def test_one_early_key_above_many(dtype, octaves):
    """A first key whose weight is 2^octaves of every other's: the small weights, together far more or less
    than it, keep their bits (they are equal: a rounding that is off is off by as much in the sum)."""
    def edit(q, k, v):
        q[:] = 1.0
        k[:] = 0.0
        k[0] = octaves * math.log(2.0) / 16         # logit 64 x this x scale, rounded to the type
        v[1:] = v[1:].abs()
    run([3, 130], [9000, 1200], 4, 2, 64, dtype, scale=0.25, edit=edit)


def in_a_new_process(code):
    """Runs code where no kernel has been launched before (what a first launch sets lasts as long as the process)."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    head = "import sys, threading, torch\nfrom paged_kv_decode_14_gb300 import _native as nat\n"
    r = subprocess.run([sys.executable, "-c", head + textwrap.dedent(code)], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-2000:] + r.stderr[-2000:]


def test_a_larger_call_captured_after_a_smaller_first_one():
    """One instance of a kernel wants shared memory by the rotation, the head size and whether there are query rows;
    a call that wants more than the first did is captured like any other."""
    in_a_new_process("""
        bf16, dev = torch.bfloat16, "cuda"
        pos = torch.arange(40, device=dev, dtype=torch.int32)
        slots = torch.arange(40, device=dev)
        q, k = torch.randn(40, 8, 128, device=dev).to(bf16), torch.randn(40, 2, 128, device=dev).to(bf16)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        w = torch.randn(40, 2, 256, device=dev).to(bf16)
        wo = torch.empty_like(w)
        zero = lambda: torch.zeros(4, 2, 16 * 128, device=dev, dtype=bf16)
        cache = nat.PagedKVCache(4, 2, 128, "bf16", k=zero(), v=zero())
        rope = nat.Rope(128)
        nat.append_norm_rope(cache, None, k, k, slots, pos, rope, eps=1e-6)             # no query rows
        nat.qk_norm_rope(w[:, :, :136], None, pos, nat.Rope(2))
        def work():
            nat.append_norm_rope(cache, q, k, k, slots, pos, rope, eps=1e-6, q_out=qo, k_out=ko)
            nat.qk_norm_rope(w, None, pos, nat.Rope(250), q_out=wo)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            work()
        g.replay()
        got = [x.clone() for x in (qo, ko, wo)]
        for x in (qo, ko, wo):
            x.zero_()
        work()
        assert all(torch.equal(x, y) for x, y in zip(got, (qo, ko, wo)))
        print("ok")
    """)


def test_first_calls_of_several_sizes_from_host_threads():
    """Four host threads, each with a stream of its own, whose calls of one kernel instance differ in what they want."""
    in_a_new_process("""
        failed = []
        def many(n, wait):
            try:
                stream = torch.cuda.Stream()
                x = torch.randn(16, 2, 256, device="cuda").to(torch.bfloat16)
                pos = torch.arange(16, device="cuda", dtype=torch.int32)
                rope, out = nat.Rope(2 + 84 * n), torch.empty_like(x)
                torch.cuda.synchronize()
                want = None
                wait.wait()
                for _ in range(2000):
                    nat.qk_norm_rope(x, None, pos, rope, q_out=out, stream=stream)
                stream.synchronize()
                want, _ = nat.qk_norm_rope(x, None, pos, rope)
                torch.cuda.synchronize()
                assert torch.equal(want, out)
            except Exception as e:
                failed.append(repr(e))
        wait = threading.Barrier(4)
        threads = [threading.Thread(target=many, args=(n, wait)) for n in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not failed, failed
        print("ok")
    """)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("starts", [None, [3, 15, 0, 31]])
def test_keys_or_values_alone_and_no_lse(dtype, starts):
    """The optional outputs of the C entry points left out: the others are the same bits."""
    lib, bf16, D, Hkv = nat.lib(), torch.bfloat16, 128, 2
    c = new_cache(40, Hkv, D, dtype)
    lens, wide = [33, 1, 160, 17], 12
    tables = torch.randperm(40, device="cuda").to(torch.int32).repeat(2)[:4 * wide].view(4, wide).contiguous()
    ln, st = i32(lens), None if starts is None else i32(starts)
    T = sum(lens)
    want = nat.read_cache(c, tables, ln, T, st)
    ptr = lambda t: None if t is None else t.data_ptr()
    view = lambda t: nat._ROWS.pack(t.data_ptr(), t.stride(0), t.stride(1), t.shape[1])
    stream = torch.cuda.current_stream().cuda_stream
    for one in range(2):
        out = torch.zeros(T, Hkv, D, dtype=bf16, device="cuda")
        rows = [None, None]
        rows[one] = view(out)
        assert lib.pkv_paged_kv_read(nat.ctypes.byref(c.desc()), ptr(tables), wide, ptr(st), ptr(ln), 4, T, *rows, 0, None,
                                     stream) == 0
        assert torch.equal(out, want[one])
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn(40, 6, D, generator=g, device="cuda").to(bf16)
    k, v = (torch.randn(3000, Hkv, D, generator=g, device="cuda").to(bf16) for _ in range(2))
    ws = nat.make_prompt_workspace()
    for w in (None, ws):                                   # whole; split along the keys and joined
        want, _ = nat.prompt_attention(q, k, v, i32([40]), i32([3000]), 40, 0.1, workspace=w)
        out, a, b = torch.zeros_like(q), i32([40]), i32([3000])
        assert lib.pkv_prompt_attention(view(q), view(k), view(v), view(out), None, 0, D, 40, 3000, ptr(a), ptr(b), None,
                                        None, 1, 40, 0.1, ptr(w), 0 if w is None else w.numel(), None, stream) == 0
        assert torch.equal(out, want)


@pytest.mark.parametrize("dtype,top", [("fp16", 25), ("bf16", 28)])
@pytest.mark.parametrize("Q,L", [([300], [300]), ([20, 3], [6000, 500])])
def test_logits_up_to_the_stated_limit(dtype, top, Q, L):
    """Logits of either sign up to 2^top, where a logit's own fp32 step is several octaves: the weights are 0 or
    those of equal keys, late maxima among them."""
    D, Hq, Hkv = 128, 4, 2
    g = torch.Generator(device="cuda").manual_seed(top)
    dt = {"fp16": torch.float16, "bf16": torch.bfloat16}[dtype]
    # q . k / 8 = 128 * 2^(top - 14) k / 8 for |k| <= 2^10: steps of 2^(top - 10)
    q = torch.full((sum(Q), Hq, D), 2.0 ** (top - 14), device="cuda").to(dt)
    k = torch.randint(-256, 257, (sum(L), Hkv, 1), generator=g, device="cuda").float().mul(4).expand(-1, -1, D)
    v = torch.randn(sum(L), Hkv, D, generator=g, device="cuda").to(dt)
    k = k.to(dt).contiguous()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = nat.make_prompt_workspace()
    out, lse = nat.prompt_attention(q, k, v, i32(Q), i32(L), max(Q), 0.125, workspace=ws, device_error=err)
    assert nat.read_device_error(err) == 0
    ref, rlse, size = reference(q, k, v, Q, L, 0.125)
    half = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    # as check(), with weights that are equal but for their rounding
    assert ((out.double() - ref).abs() <= half * ref.abs() + (half + 2.0 ** -13) * size * (1 + half) + 2.0 ** -24).all()
    # scale log2(e), its product with the logit, m + log2(l) and the product with ln 2: four roundings of 2^-24
    assert ((lse.double() - rlse).abs() <= 2.0 ** -22 * rlse.abs() + 2.0 ** -13).all()


@pytest.mark.parametrize("dtype,top", [("fp16", 25), ("bf16", 28)])
@pytest.mark.parametrize("where", ["first", "late", "negative", "negative first"])
def test_logits_past_the_stated_limit_are_reported(dtype, top, where):
    """Twice the limit and more, at a row's first key, at its last, or with the other sign in all of them or the first
    128; in rows of one head only.  Infinite logits are not reported: they have their own results."""
    dt = {"fp16": torch.float16, "bf16": torch.bfloat16}[dtype]
    q = torch.full((200, 4, 128), 2.0 ** (top - 14), device="cuda").to(dt)
    k, v = torch.zeros(200, 2, 128, device="cuda").to(dt), torch.randn(200, 2, 128, device="cuda").to(dt)
    err, n = torch.zeros(1, dtype=torch.int32, device="cuda"), i32([200])
    nat.prompt_attention(q, k, v, n, n, 200, 0.125, device_error=err)
    assert nat.read_device_error(err) == 0
    at = {"first": slice(0, 1), "late": slice(199, 200), "negative": slice(0, 200), "negative first": slice(0, 128)}[where]
    k[at, 1] = -2.0 ** 11 if "negative" in where else 2.0 ** 11
    nat.prompt_attention(q, k, v, n, n, 200, 0.125, device_error=err)
    assert nat.read_device_error(err) == nat.DEVERR_RANGE
    k[at, 1] = -math.inf if "negative" in where else math.inf
    nat.prompt_attention(q, k, v, n, n, 200, 0.125, device_error=err)
    assert nat.read_device_error(err) == 0


def test_attention_in_place_of_its_queries():
    for Q, L, w in (([300, 40], [300, 700], None), ([40, 1], [3000, 2000], nat.make_prompt_workspace())):
        q = torch.randn(sum(Q), 8, 64, device="cuda").half()
        k, v = (torch.randn(sum(L), 2, 64, device="cuda").half() for _ in range(2))
        want, lse = nat.prompt_attention(q, k, v, i32(Q), i32(L), max(Q), 0.125, workspace=w)
        nat.prompt_attention(q, k, v, i32(Q), i32(L), max(Q), 0.125, out=q, workspace=w)
        assert torch.equal(q, want)


def test_calls_from_host_threads():
    """Four host threads, each with a stream, a cache and a workspace of its own, as one after the other."""
    import threading
    D, Hq, Hkv, T = 128, 8, 2, 70
    rope = nat.Rope(D, scaling="bands", factor=4.0, original_len=64)
    lens, tables = i32([T]), i32([[0, 1, 2, 3, 4]])
    pos, slots = torch.arange(T, device="cuda", dtype=torch.int32), torch.arange(T, device="cuda")
    sets = [[x.clone() for x in make(T, (Hq, Hkv, Hkv), D, torch.bfloat16, seed)] for seed in range(4)]
    caches = [[new_cache(5, Hkv, D, "fp8", seed) for _ in range(2)] for seed in range(4)]
    spaces = [nat.make_prompt_workspace() for _ in range(4)]
    failed = []

    def work(n, cache, stream):
        q, k, v = sets[n]
        qo = nat.append_norm_rope(cache, q, k, v, slots, pos, rope, eps=1e-6, fp8_scales_from_values=True, stream=stream)
        kr, vr = nat.read_cache(cache, tables, lens, T, stream=stream)
        return (qo, kr, vr) + nat.prompt_attention(qo, kr, vr, lens, lens, T, 0.1, workspace=spaces[n], stream=stream)

    want = [work(n, caches[n][0], None) for n in range(4)]
    torch.cuda.synchronize()

    def many(n):
        try:
            stream = torch.cuda.Stream()
            for _ in range(100):
                got = work(n, caches[n][1], stream)
            stream.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, want[n]))
        except Exception as e:
            failed.append(repr(e))

    threads = [threading.Thread(target=many, args=(n,)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
