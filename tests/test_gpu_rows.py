"""Norm and rotation of rows, the append that writes them into the cache, and
the cache read back, against the formulas in 64 bits."""

import math

import numpy as np
import pytest
import torch

from paged_kv_decode_14_gb300 import _native as nat

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# half a step of a type, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# The fp32 chain before the rounding: a sum of up to 256 squares (at most 256 / 2 halved by the
# square root = 128 steps of 2^-24 relative), the reciprocal root, two products, cos / sin of an
# angle good to 2^-24 of half a turn (2^-22.3 radians) and one fma: below 2^-16 of |a| + |b|.
CHAIN = 2.0 ** -16


def ref_rows(x, weight, eps, positions, rope, inverse=False):
    """(value, magnitude that the fp32 chain's error is relative to) in fp64."""
    y = x.double()
    if eps is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
        if weight is not None:
            y = y * weight.double()
    size = y.abs().clone()
    if rope is not None:
        rd, n = rope.rotary_dim, rope.rotary_dim // 2
        f = torch.tensor(rope.inv_freq, dtype=torch.float64, device=x.device)
        ang = positions.double()[:, None, None] * f
        c, s = ang.cos() * rope.magnitude, ang.sin() * rope.magnitude * (-1 if inverse else 1)
        ia = torch.arange(n, device=x.device) * 2 if rope.desc.interleaved else torch.arange(n, device=x.device)
        ib = ia + 1 if rope.desc.interleaved else ia + n
        a, b = y[..., ia].clone(), y[..., ib].clone()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * max(1.0, rope.magnitude)
    return y, size


def assert_rows(got, ref, size, what=""):
    half = HALF[got.dtype]
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0         # fp16 subnormals: half of 2^-24
    bad = (got.double() - ref).abs() > half * ref.abs() + CHAIN * size * (1 + half) + tiny
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def make(T, heads, D, dtype, seed, fused=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fused:
        x = torch.randn(T, sum(heads) * D, generator=g, device="cuda").to(dtype)
        return [p.view(T, h, D) for p, h in zip(x.split([h * D for h in heads], 1), heads)]
    return [torch.randn(T, h, D, generator=g, device="cuda").to(dtype) for h in heads]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,rd,inter,scaling", [(128, 128, False, "none"), (128, 64, True, "ramp"), (64, 10, False, "bands"),
                                                (80, 18, False, "linear"), (256, 256, False, "ntk"), (256, 128, False, "none"),
                                                (96, 96, True, "none"), (192, 96, False, "none"), (64, 0, False, "none"),
                                                (16, 6, True, "none")])
@pytest.mark.parametrize("norm", [False, True])
def test_rows(dtype, D, rd, inter, scaling, norm):
    dt = TYPES[dtype]
    T, Hq, Hkv = 37, 7, 3
    q, k, _ = make(T, (Hq, Hkv, Hkv), D, dt, D + rd)
    pos = torch.randint(-5, 1 << 20, (T,), device="cuda", dtype=torch.int32)
    pos[:4] = torch.tensor([0, 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64).to(torch.int32)
    rope = nat.Rope(rd, 500000.0, inter, scaling, 4.0, 4096, 1.0, 8.0) if rd else None
    w = [(1 + 0.3 * torch.randn(D, device="cuda")).to(dt) for _ in range(2)] if norm else [None, None]
    eps = 1e-5 if norm else None
    qo, ko = nat.qk_norm_rope(q, k, pos, rope, w[0], w[1], eps)
    assert_rows(qo, *ref_rows(q, w[0], eps, pos, rope), "q")
    assert_rows(ko, *ref_rows(k, w[1], eps, pos, rope), "k")
    # in place, and without weights / without k
    qi = q.clone()
    nat.qk_norm_rope(qi, None, pos, rope, w[0], None, eps, q_out=qi)
    assert torch.equal(qi, qo)
    if norm:
        qn, _ = nat.qk_norm_rope(q, None, pos, rope, eps=eps)
        assert_rows(qn, *ref_rows(q, None, eps, pos, rope), "unweighted")


@pytest.mark.parametrize("T,Hq", [(1, 1), (1, 64), (2, 48), (300, 5)])
def test_rows_counts(T, Hq):
    q, k, _ = make(T, (Hq, 1, 1), 128, torch.bfloat16, T + Hq)
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 1001
    rope = nat.Rope(128)
    qo, ko = nat.qk_norm_rope(q, k, pos, rope, eps=1e-6)
    assert_rows(qo, *ref_rows(q, None, 1e-6, pos, rope))
    assert_rows(ko, *ref_rows(k, None, 1e-6, pos, rope))
    empty = nat.qk_norm_rope(q[:0], k[:0], pos[:0], rope)
    assert empty[0].shape == (0, Hq, 128)


def test_rows_strided_outputs_leave_the_rest():
    T, D = 21, 64
    q, k, _ = make(T, (4, 2, 2), D, torch.bfloat16, 3)
    buf = torch.full((T, 9, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    rope = nat.Rope(D, interleaved=True)
    head_major = torch.full((2, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    nat.qk_norm_rope(q, k, pos, rope, q_out=buf[:, 1:5, :D], k_out=head_major.transpose(0, 1))
    assert_rows(buf[:, 1:5, :D], *ref_rows(q, None, None, pos, rope))
    assert_rows(head_major.transpose(0, 1), *ref_rows(k, None, None, pos, rope))
    assert (buf[:, 0] == 7).all() and (buf[:, 5:] == 7).all() and (buf[:, 1:5, D:] == 7).all()


def test_inverse_is_the_gradient_and_undoes():
    T, D = 13, 64
    x = torch.randn(T, 2, D, device="cuda")
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 7919
    for inter, scaling in ((False, "none"), (True, "ramp")):
        rope = nat.Rope(32, 10000.0, inter, scaling, 2.0, 128, 1.0, 8.0)
        y, _ = nat.qk_norm_rope(x, None, pos, rope)
        back, _ = nat.qk_norm_rope(y, None, pos, rope, inverse=True)
        m = torch.ones(D, device="cuda", dtype=torch.float64)
        m[:32] = rope.magnitude ** 2
        # two chains, each below CHAIN of the pair's size (at most 2 |x|max magnitude^2)
        assert ((back.double() - x.double() * m).abs() <= 8 * CHAIN * x.abs().max() * rope.magnitude ** 2).all()
        # the gradient of sum(y * g) by differences: the map is linear, so one difference is exact
        g = torch.randn_like(x)
        gx, _ = nat.qk_norm_rope(g, None, pos, rope, inverse=True)
        for t, h, d in ((0, 0, 0), (5, 1, 3), (12, 0, 17), (7, 1, 40)):
            e = torch.zeros_like(x)
            e[t, h, d] = 1.0
            ye, _ = nat.qk_norm_rope(e, None, pos, rope)
            assert abs(float((ye.double() * g.double()).sum()) - float(gx[t, h, d])) <= 8 * CHAIN * float(g.abs().max()) * 2


def test_rows_nan_and_inf_stay_in_their_rows():
    T, D = 9, 128
    q, _, _ = make(T, (4, 1, 1), D, torch.bfloat16, 5)
    q = q.clone()
    q[3, 2, 5], q[6, 0, 127] = float("nan"), float("inf")
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    rope = nat.Rope(64)
    out, _ = nat.qk_norm_rope(q, None, pos, rope)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[3, 2, 5] = want[3, 2, 37] = True       # the pair (5, 5 + 32)
    want[6, 0, 127] = True                      # outside the rotated part
    assert torch.equal(bad, want)
    out, _ = nat.qk_norm_rope(q, None, pos, rope, eps=1e-6)
    assert torch.isfinite(out[:3]).all() and torch.isfinite(out[4:6]).all() and torch.isfinite(out[3, :2]).all()


@pytest.mark.parametrize("first", [1.0, 0.3, 1000.1, 123456.789, 9.9e8, -1.0, -1e-17, -77777.7, 6.283185307179586])
def test_angles_of_far_positions(first):
    """A caller's own frequencies at positions up to the ends of 32 bits, against position * inv_freq modulo a turn in
    60 digits."""
    from decimal import Decimal, localcontext
    pairs, far = 8, [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 2 ** 20, 1, -1, 0]
    rope = nat.Rope(2 * pairs)
    for i in range(pairs):
        rope.desc.inv_freq[i] = first / (1 + 0.7 * i)
    pos = torch.tensor(far, dtype=torch.int64).to(torch.int32).cuda()
    x = torch.zeros(len(far), 1, 16, device="cuda")
    x[..., :pairs] = 1.0                                    # (cos, sin) of every pair
    out, _ = nat.qk_norm_rope(x, None, pos, rope)
    with localcontext() as ctx:
        ctx.prec = 60
        turn = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
        for t, p in enumerate(far):
            for i in range(pairs):
                a = Decimal(p) * Decimal(rope.desc.inv_freq[i])
                a = float(a - (a / turn).to_integral_value() * turn)
                # the angle: 2 pi (2^-31 + 2^-26) = 2^-23.3; cos and sin: an ulp of results up to 1, 2^-24; the two
                # roundings of the rotation: 2^-24.  Together below 2^-22.
                for got, want in ((out[t, 0, i], math.cos(a)), (out[t, 0, pairs + i], math.sin(a))):
                    assert abs(float(got) - want) <= 2.0 ** -22, (p, rope.desc.inv_freq[i], float(got), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 80, 128, 256])
@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-31, 1e-6, 1e37])
def test_norm_of_rows_whose_squares_leave_fp32(dtype, D, eps):
    """Rows from fp32's largest values to its subnormals, side by side in every token (a warp holds several): the
    norm is the formula's, in rows and in the pass that writes the cache."""
    dt, eps = TYPES[dtype], float(np.float32(eps))
    scales = [1.0, 1e20, 2e37, 1e-12, 1e-25, 1e-37, 1e-3]
    T, H = 5, len(scales)
    g = torch.Generator(device="cuda").manual_seed(D)
    # (no element below 2^-7 of a row's unit: a result stays in fp32's normal range or is covered below)
    x = torch.randn(T, H, D, generator=g, device="cuda")
    x = torch.where(x.abs() < 2.0 ** -7, 2.0 ** -7, x)
    x = (x * torch.tensor(scales, device="cuda")[:, None]).to(dt)
    w = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dt)

    def check(got, ref, size):
        # Results below the normal range (fp32's and bf16's alike): half a subnormal step of the type, and in fp32
        # h = 2^-150 for each rounding of the chain there: two before the weight (at most 2.2 here), one after it, and
        # one for either product of the rotation: (2 h 2.2 + h) sqrt(2) + 2 h < 10 h.
        low = HALF[dt] * 2.0 ** -126 + 10 * 2.0 ** -150
        bad = (got.double() - ref).abs() > HALF[dt] * ref.abs() + 2 * CHAIN * size + low
        assert not bad.any(), (bad.nonzero()[0].tolist(), got[bad][0].item(), ref[bad][0].item())

    for weight in (None, w):
        out, _ = nat.qk_norm_rope(x, None, q_weight=weight, eps=eps)
        check(out, *ref_rows(x, weight, eps, None, None))
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 77
    rope = nat.Rope(D // 2)
    out, _ = nat.qk_norm_rope(x, None, pos, rope, w, eps=eps)
    check(out, *ref_rows(x, w, eps, pos, rope))
    if dtype == "bf16" and D in (64, 128):
        c = new_cache(1, H, D, "bf16")
        k_out, slots = torch.empty_like(x), torch.arange(T, device="cuda")
        nat.append_norm_rope(c, None, x, x, slots, pos, rope, None, w, eps, k_out=k_out)
        assert torch.equal(k_out, out) and torch.equal(page_rows(c.k, D, 2)[0, :, :T].transpose(0, 1), out)


def test_norm_of_zero_infinite_and_nan_rows():
    """As the formula has them: 0 / 0 is NaN, finite / infinite is 0, and the rows beside them are untouched."""
    x = torch.randn(3, 8, 128, device="cuda")
    want, _ = nat.qk_norm_rope(x, None, eps=0.0)
    odd = x.clone()
    odd[1, 2] = 0.0
    odd[1, 4, 7] = math.inf
    odd[2, 0, 9] = math.nan
    out, _ = nat.qk_norm_rope(odd, None, eps=0.0)
    assert torch.isnan(out[1, 2]).all() and torch.isnan(out[2, 0]).all()
    assert torch.isnan(out[1, 4, 7]) and (out[1, 4, :7] == 0).all() and (out[1, 4, 8:] == 0).all()
    same = torch.ones(3, 8, dtype=torch.bool, device="cuda")
    same[1, 2] = same[1, 4] = same[2, 0] = False
    assert torch.equal(out[same], want[same])
    out, _ = nat.qk_norm_rope(odd, None, eps=1e-6)
    assert (out[1, 2] == 0).all()


# ------------------------------------------------------------------ append and read


def place(D, E, off, d):
    C = 16 // E
    return ((off // 8) * (D // C) + d // C) * 8 * C + (off % 8) * C + d % C


def page_rows(pool, D, E):
    """[num_blocks, Hkv, 16, D] of a cache buffer, by the header's formula."""
    off, d = np.meshgrid(np.arange(16), np.arange(D), indexing="ij")
    at = torch.from_numpy(place(D, E, off, d)).to(pool.device)
    x = pool if E == 2 else pool.view(torch.float8_e4m3fn).float()
    return x[:, :, at.reshape(-1)].view(pool.shape[0], pool.shape[1], 16, D)


def new_cache(nb, Hkv, D, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if dtype == "bf16":
        kv = [torch.randn(nb, Hkv, 16 * D, generator=g, device="cuda").bfloat16() for _ in range(2)]
        return nat.PagedKVCache(nb, Hkv, D, "bf16", k=kv[0], v=kv[1])
    kv = [torch.randint(0, 127, (nb, Hkv, 16 * D), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
    sc = [0.01 + 0.01 * torch.rand(nb, Hkv, generator=g, device="cuda") for _ in range(2)]
    return nat.PagedKVCache(nb, Hkv, D, "fp8", k=kv[0], v=kv[1], k_scales=sc[0], v_scales=sc[1])


def clone(c):
    return nat.PagedKVCache(c.num_blocks, c.num_kv_heads, c.head_dim, c.kv_dtype, k=c.k.clone(), v=c.v.clone(),
                            k_scales=None if c.k_scales is None else c.k_scales.clone(),
                            v_scales=None if c.v_scales is None else c.v_scales.clone())


def same_cache(a, b):
    return (torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8)) and
            torch.equal(a.v.view(torch.uint8), b.v.view(torch.uint8)) and
            (a.k_scales is None or (torch.equal(a.k_scales, b.k_scales) and torch.equal(a.v_scales, b.v_scales))))


def slots_of(kind, nb, seed):
    """Slot mappings: consecutive prompts, decode steps, shuffled, padded, ragged continuations."""
    r = np.random.default_rng(seed)
    blocks = r.permutation(nb)
    if kind == "prompts":                     # whole prompts of odd lengths, one ending inside a page
        lens, out, at = [33, 1, 48, 15, 16], [], 0
        for n in lens:
            need = -(-n // 16)
            out += [int(blocks[at + i // 16]) * 16 + i % 16 for i in range(n)]
            at += need
        return out
    if kind == "step":                        # one token a sequence, some at a block's start
        return [int(b) * 16 + int(o) for b, o in zip(blocks[:40], r.integers(0, 16, 40))]
    if kind == "chunk":                       # continuing inside pages, then new pages
        out = []
        for s in range(3):
            first = int(r.integers(1, 15))
            out += [int(blocks[4 * s + (first + i) // 16]) * 16 + (first + i) % 16 for i in range(37)]
        return out
    if kind == "shuffled":                    # a started block's tokens anywhere in the call, some missing
        out = [int(b) * 16 + o for b in blocks[:9] for o in range(16) if r.random() < 0.8]
        r.shuffle(out)
        return out
    if kind == "padded":
        out = [int(blocks[0]) * 16 + i for i in range(16)] + [-1] * 5 + [int(blocks[1]) * 16 + i for i in range(7)]
        return out + [-7, int(blocks[2]) * 16]
    raise AssertionError(kind)


KINDS = ["prompts", "step", "chunk", "shuffled", "padded"]


@pytest.mark.parametrize("D,Hkv,G", [(128, 8, 4), (64, 3, 2), (128, 1, 7), (64, 5, 1)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp8", "fp8_values"])
def test_append_plain_equals_append(D, Hkv, G, kind, dtype):
    """Without norm and rotation the new append is the old one, bit for bit."""
    nb = 48
    slots = torch.tensor(slots_of(kind, nb, 7), dtype=torch.int64, device="cuda")
    T = slots.numel()
    q, k, v = make(T, (Hkv * G, Hkv, Hkv), D, torch.bfloat16, T)
    c = new_cache(nb, Hkv, D, dtype[:4] if dtype == "bf16" else "fp8")
    old, new = clone(c), clone(c)
    vals = dtype == "fp8_values"
    nat.append_rope(old, k.contiguous(), v.contiguous(), slots, fp8_scales_from_values=vals)
    k_out = torch.full((T, Hkv, D), 9.0, dtype=torch.bfloat16, device="cuda")
    qo = nat.append_norm_rope(new, q, k, v, slots, k_out=k_out, fp8_scales_from_values=vals)
    assert torch.equal(qo, q) and torch.equal(k_out, k)
    assert same_cache(old, new)


@pytest.mark.parametrize("D,Hkv,G", [(128, 8, 4), (64, 3, 2)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rd,inter,norm", [(64, False, True), (10, False, True), (32, True, False)])
def test_append_norm_rope_bf16(D, Hkv, G, kind, rd, inter, norm):
    nb = 48
    slots = torch.tensor(slots_of(kind, nb, 11), dtype=torch.int64, device="cuda")
    T = slots.numel()
    q, k, v = make(T, (Hkv * G, Hkv, Hkv), D, torch.bfloat16, T)
    pos = torch.randint(0, 1 << 17, (T,), device="cuda", dtype=torch.int32)
    rope = nat.Rope(rd, 10000.0, inter)
    w = [(1 + 0.3 * torch.randn(D, device="cuda")).bfloat16() for _ in range(2)] if norm else [None, None]
    eps = 1e-6 if norm else None
    c = new_cache(nb, Hkv, D, "bf16")
    old = clone(c)
    qo = nat.append_norm_rope(c, q, k, v, slots, pos, rope, w[0], w[1], eps)
    q2, k2 = nat.qk_norm_rope(q, k, pos, rope, w[0], w[1], eps)
    assert torch.equal(qo, q2)
    nat.append(old, k2, v.contiguous(), slots)
    assert same_cache(old, c)
    # key rows in place of their input
    kk = k.clone()
    c3 = clone(old)
    nat.append_norm_rope(c3, None, kk, v, slots, pos, rope, None, w[1], eps, k_out=kk)
    assert torch.equal(kk, k2) and same_cache(old, c3)


@pytest.mark.parametrize("D,Hkv", [(128, 8), (64, 3)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("values", [False, True])
def test_append_norm_rope_fp8(D, Hkv, kind, values):
    nb = 48
    lst = slots_of(kind, nb, 13)
    slots = torch.tensor(lst, dtype=torch.int64, device="cuda")
    T = slots.numel()
    q, k, v = make(T, (Hkv, Hkv, Hkv), D, torch.bfloat16, T + 1)
    pos = torch.randint(0, 1 << 17, (T,), device="cuda", dtype=torch.int32)
    rope = nat.Rope(D, 10000.0)
    w = (1 + 0.3 * torch.randn(D, device="cuda")).bfloat16()
    c = new_cache(nb, Hkv, D, "fp8")
    was = clone(c)
    nat.append_norm_rope(c, q, k, v, slots, pos, rope, w, w, 1e-6, fp8_scales_from_values=values)
    kref, ksize = ref_rows(k, w, 1e-6, pos, rope)
    for ref, size, pool, old, sc, osc in ((kref, ksize, c.k, was.k, c.k_scales, was.k_scales),
                                          (v.double(), 0 * ksize, c.v, was.v, c.v_scales, was.v_scales)):
        want = osc.double().clone()
        if values:
            for b in {s // 16 for s in lst if s >= 0 and s % 16 == 0}:
                m = torch.tensor([s >= 0 and s // 16 == b for s in lst], device="cuda")
                want[b] = ref[m].abs().amax((0, 2)) / 448
        # (fp32: the chain, then one division)
        assert ((sc.double() - want).abs() <= want * (2 * CHAIN * 2 + 2.0 ** -23)).all()
        got, before = page_rows(pool, D, 1), page_rows(old, D, 1)
        written = torch.zeros(nb, 16, dtype=torch.bool, device="cuda")
        for t, s in enumerate(lst):
            if s < 0:
                continue
            b, o = s // 16, s % 16
            written[b, o] = True
            x = got[b, :, o].double() * sc[b].double()[:, None]
            top = 448 * sc[b].double()[:, None]
            r = ref[t].clamp(-top, top)
            # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale among its subnormals
            tol = 2.0 ** -4 * r.abs() + 2.0 ** -10 * sc[b].double()[:, None] + 2 * CHAIN * (size[t] + r.abs())
            assert ((x - r).abs() <= tol).all(), (t, s)
        keep = ~written[:, None, :, None].expand_as(got)
        assert torch.equal(torch.nan_to_num(got[keep], 1e9), torch.nan_to_num(before[keep], 1e9))


@pytest.mark.parametrize("D,Hkv", [(128, 8), (64, 3)])
@pytest.mark.parametrize("order", ["interleaved", "ends", "shuffled", "reversed"])
def test_started_blocks_gathered_from_all_over_the_call(D, Hkv, order):
    """Whole blocks whose tokens are not consecutive, offset 15 among the scattered ones: every block's owner
    finds its last row by the scan, not in its run.  Many calls: every one as the first append's, bit for bit."""
    nb = 96
    blocks = np.random.default_rng(5).permutation(nb).tolist()
    if order == "interleaved":                # token by token through the blocks in turn
        lst = [b * 16 + o for o in range(16) for b in blocks]
    elif order == "ends":                     # runs of 15, all the last rows behind them
        lst = [b * 16 + o for b in blocks for o in range(15)] + [b * 16 + 15 for b in blocks]
    else:
        lst = [b * 16 + o for b in blocks for o in range(16)]
        np.random.default_rng(6).shuffle(lst) if order == "shuffled" else lst.reverse()
    slots = torch.tensor(lst, dtype=torch.int64, device="cuda")
    T = slots.numel()
    _, k, v = make(T, (1, Hkv, Hkv), D, torch.bfloat16, T)
    base = new_cache(nb, Hkv, D, "fp8")
    want = clone(base)
    nat.append_rope(want, k.contiguous(), v.contiguous(), slots, fp8_scales_from_values=True)
    k_out = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    for _ in range(50):
        got = clone(base)
        k_out.fill_(9.0)
        nat.append_norm_rope(got, None, k, v, slots, k_out=k_out, fp8_scales_from_values=True)
        assert same_cache(want, got) and torch.equal(k_out, k)


def test_append_bad_slots_are_reported():
    D, Hkv, nb = 64, 2, 8
    slots = torch.tensor([3, nb * 16, 5, 1 << 40], dtype=torch.int64, device="cuda")
    q, k, v = make(4, (2, Hkv, Hkv), D, torch.bfloat16, 1)
    for dtype, vals in (("bf16", False), ("fp8", False), ("fp8", True)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        c = new_cache(nb, Hkv, D, dtype)
        old = clone(c)
        qo = nat.append_norm_rope(c, q, k, v, slots, fp8_scales_from_values=vals, device_error=err)
        assert nat.read_device_error(err) == nat.DEVERR_SLOT
        assert torch.equal(qo, q)
        good = torch.tensor([0, 2], device="cuda")
        nat.append(old, k[good].contiguous(), v[good].contiguous(), slots[good].contiguous())
        assert same_cache(old, c)


def test_append_fp8_nan_and_zero_blocks():
    D, Hkv, nb = 128, 2, 4
    slots = torch.arange(32, dtype=torch.int64, device="cuda")
    k = torch.zeros(32, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.randn(32, Hkv, D, device="cuda").bfloat16()
    v[3, 0, 5] = float("nan")
    v[20, 1, 7] = float("inf")
    c = new_cache(nb, Hkv, D, "fp8")
    old = clone(c)
    nat.append_norm_rope(c, None, k, v, slots, fp8_scales_from_values=True)
    nat.append_rope(old, k, v, slots, fp8_scales_from_values=True)
    assert (c.k_scales[:2] == 1).all()
    assert same_cache(old, c)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("D,Hkv", [(128, 8), (64, 1), (64, 3)])
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("from_start", [True, False])
def test_read(dtype, D, Hkv, out, from_start):
    nb, dt = 64, TYPES[out]
    c = new_cache(nb, Hkv, D, dtype)
    r = np.random.default_rng(D + Hkv)
    lens = [0, 1, 16, 17, 100, 0, 33, 250]
    starts = [0] * 8 if from_start else [3, 15, 16, 5, 31, 0, 47, 1]
    tables = np.full((8, 17), -1, dtype=np.int32)
    for b in range(8):
        n = -(-(lens[b] + starts[b]) // 16)
        tables[b, :n] = r.integers(0, nb, n)               # (blocks may be shared)
    total = sum(lens)
    buf = torch.full((total + 3, Hkv, 2, D), 5.0, dtype=dt, device="cuda")
    k_out, v_out = buf[:, :, 0], buf[:, :, 1]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    nat.read_cache(c, torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), total + 3,
                   None if from_start else torch.tensor(starts, dtype=torch.int32, device="cuda"), k_out=k_out,
                   v_out=v_out, device_error=err)
    assert nat.read_device_error(err) == 0
    for got, pool, sc in ((k_out, c.k, c.k_scales), (v_out, c.v, c.v_scales)):
        pages = page_rows(pool, D, 2 if dtype == "bf16" else 1).float()
        if sc is not None:
            pages = pages * sc[:, :, None, None]            # (fp32, as defined)
        at = 0
        for b in range(8):
            p = np.arange(starts[b], starts[b] + lens[b])
            want = pages[torch.from_numpy(tables[b][p // 16]).cuda().long(), :, torch.from_numpy(p % 16).cuda()]
            assert torch.equal(got[at:at + lens[b]], want.to(dt)), b
            at += lens[b]
        assert (got[total:] == 5).all()


def test_read_only_one_of_k_and_v_and_bad_input():
    c = new_cache(8, 2, 64, "bf16")
    tb = torch.tensor([[1, 2], [3, 99], [4, 5]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 32, 17], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = nat.read_cache(c, tb, lens, 69, device_error=err)
    assert nat.read_device_error(err) == nat.DEVERR_BLOCK_ID
    pages = page_rows(c.k, 64, 2)
    assert torch.equal(k[:16], pages[1].transpose(0, 1)) and torch.equal(k[52:68], pages[4].transpose(0, 1))
    # a sequence past its table row, a negative length, too few rows
    for bad, n in (([20, 33, 17], 70), ([20, -1, 17], 37), ([20, 16, 17], 40)):
        k2 = torch.full((n, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        nat.read_cache(c, tb, torch.tensor(bad, dtype=torch.int32, device="cuda"), n, k_out=k2, device_error=err)
        assert nat.read_device_error(err) == nat.DEVERR_LENGTH, bad
        assert torch.equal(k2[:16], pages[1].transpose(0, 1))
        if bad[1] == 33:
            assert (k2[20:53] == 3).all()
