"""Host side of the entry points over rows: the rotation's frequencies and the
argument checks, which run before anything is enqueued (no GPU here: the
pointers are never followed)."""

import ctypes
import math
import os
import shutil

import pytest

from paged_kv_decode_14_gb300 import _native as nat

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
PTR = 0x10000


@pytest.fixture(scope="module")
def L():
    from paged_kv_decode_14_gb300 import build as b
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        if not os.path.exists(b.LIB):
            pytest.skip("no nvcc and no prebuilt library")
    else:
        b.build()
    return nat.lib()


def rope(L, rd, theta=10000.0, inter=0, kind=0, factor=1.0, orig=0, low=1.0, high=4.0):
    r = nat.RopeDesc()
    st = L.pkv_rope_init(ctypes.byref(r), rd, inter, theta, kind, factor, orig, low, high)
    return st, r


def test_frequencies_of_every_scaling(L):
    rd, theta, s, orig = 64, 500000.0, 8.0, 8192
    f = [theta ** (-2 * i / rd) for i in range(rd // 2)]

    def of(kind, **k):
        st, r = rope(L, rd, theta, kind=kind, factor=s, orig=orig, **k)
        assert st == OK
        return list(r.inv_freq[:rd // 2]), r.magnitude

    same = dict(rel=1e-14)
    assert of(0)[0] == pytest.approx(f, **same)
    assert of(1)[0] == pytest.approx([x / s for x in f], **same)
    big = theta * s ** (rd / (rd - 2))
    assert of(2)[0] == pytest.approx([big ** (-2 * i / rd) for i in range(rd // 2)], **same)
    got, mag = of(3, low=1.0, high=4.0)
    assert mag == 1.0
    for x, y in zip(f, got):
        turns = orig * x / (2 * math.pi)
        want = x if turns >= 4 else x / s if turns <= 1 else None
        if want is not None:
            assert y == pytest.approx(want, rel=1e-13)
        else:
            assert x / s < y < x
    got, mag = of(4, low=1.0, high=32.0)
    assert mag == pytest.approx(0.1 * math.log(s) + 1, rel=1e-6)     # (a float: half a step is 2^-24)
    assert got[0] == pytest.approx(f[0], rel=1e-13) and got[-1] == pytest.approx(f[-1] / s, rel=1e-13)
    assert all(x / s * (1 - 1e-13) <= y <= x * (1 + 1e-13) for x, y in zip(f, got))


@pytest.mark.parametrize("bad", [dict(rd=0), dict(rd=7), dict(rd=258), dict(theta=1.0), dict(theta=float("nan")),
                                 dict(kind=5), dict(kind=1, factor=0.5), dict(kind=2, rd=2, factor=2.0),
                                 dict(kind=3, factor=2.0, orig=0), dict(kind=4, factor=2.0, orig=64, low=4.0, high=4.0)])
def test_rope_refusals(L, bad):
    a = dict(rd=64)
    a.update(bad)
    assert rope(L, **a)[0] == INVALID


def rows(heads, D=128, ptr=PTR, ts=None, hs=None):
    return nat._ROWS.pack(ptr, heads * D if ts is None else ts, D if hs is None else hs, heads)


def cache(dtype=0, D=128, heads=8):
    return nat.CacheDesc(64, 16, heads, D, dtype, PTR, PTR, PTR if dtype else None, PTR if dtype else None)


def test_qk_norm_rope_refusals(L):
    _, r = rope(L, 128)
    ref = ctypes.addressof(r)

    def call(q=rows(4), qo=rows(4), k=None, ko=None, dt=0, D=128, T=3, pos=PTR, rp=ref, inv=0, qw=None, kw=None, eps=-1.0):
        return L.pkv_qk_norm_rope(q, qo, k, ko, dt, D, T, pos, rp, inv, qw, kw, eps, None)

    assert call(T=0) == OK
    assert call(dt=3) == INVALID
    assert call(D=0) == INVALID
    assert call(D=264) == UNSUPPORTED
    assert call(D=124) == UNSUPPORTED                       # 248 bytes: no whole 16-byte pieces
    assert call(T=-1) == INVALID
    assert call(q=None) == INVALID
    assert call(k=rows(2)) == INVALID                       # k without k_out
    assert call(qo=rows(5)) == INVALID
    assert call(q=rows(4, ptr=PTR + 8)) == INVALID
    assert call(q=rows(4, ts=4 * 128 + 4)) == INVALID       # 8-byte stride
    assert call(qo=rows(4, hs=0)) == INVALID                # an output's rows on top of each other
    assert call(pos=None) == INVALID
    assert call(rp=None, pos=None, eps=float("nan")) == INVALID
    assert call(qw=PTR) == INVALID                          # weight without a norm
    assert call(eps=1e-6, inv=1) == INVALID
    assert call(D=64, q=rows(4, 64), qo=rows(4, 64)) == INVALID   # rotary_dim 128 > 64
    r.inv_freq[3] = float("nan")
    assert call() == INVALID


def test_append_norm_rope_refusals(L):
    def call(c=None, q=rows(32), qo=rows(32), k=rows(8), v=rows(8), ko=None, slots=PTR, T=2, pos=None, rp=None,
             qw=None, kw=None, eps=-1.0, fresh=0):
        c = c or cache()
        return L.pkv_paged_kv_append_norm_rope(ctypes.byref(c), q, qo, k, v, ko, slots, T, pos, rp, qw, kw, eps, fresh,
                                               None, None)

    assert call(T=0) == OK
    assert call(c=cache(D=96)) == UNSUPPORTED
    assert call(slots=None) == INVALID
    assert call(fresh=1) == INVALID                         # a bf16 cache has no scales
    assert call(q=None) == INVALID
    assert call(q=rows(30), qo=rows(30)) == INVALID         # not a multiple of the kv-heads
    assert call(k=rows(4)) == INVALID and call(v=rows(4)) == INVALID and call(ko=rows(4)) == INVALID
    assert call(v=None) == INVALID
    assert call(T=-1) == INVALID


def test_read_refusals(L):
    def call(c=None, bt=PTR, mb=4, st=None, lens=PTR, B=2, n=64, k=rows(8), v=rows(8), dt=0):
        c = c or cache()
        return L.pkv_paged_kv_read(ctypes.byref(c), bt, mb, st, lens, B, n, k, v, dt, None, None)

    assert call(B=0) == OK and call(n=0) == OK and call(k=None, v=None) == OK
    assert call(dt=5) == INVALID
    assert call(bt=None) == INVALID and call(lens=None) == INVALID and call(mb=0) == INVALID
    assert call(k=rows(4)) == INVALID
    assert call(k=rows(8, ptr=PTR + 2)) == INVALID
    assert call(n=-1) == INVALID


def test_prompt_refusals(L):
    def call(q=rows(8), k=rows(2), v=rows(2), o=rows(8), lse=None, dt=0, D=128, nq=9, nk=9, ql=PTR, kl=PTR, B=1, mq=9,
             sc=0.1, ws=None, wn=0):
        return L.pkv_prompt_attention(q, k, v, o, lse, dt, D, nq, nk, ql, kl, None, None, B, mq, sc, ws, wn, None, None)

    assert call(B=0) == OK and call(nq=0) == OK
    assert call(dt=2) == UNSUPPORTED and call(D=96) == UNSUPPORTED
    assert call(nq=1 << 31) == UNSUPPORTED
    assert call(sc=0.0) == INVALID and call(sc=float("inf")) == INVALID and call(sc=float("nan")) == INVALID
    assert call(mq=0) == INVALID and call(ql=None) == INVALID and call(kl=None) == INVALID
    assert call(q=rows(7)) == INVALID                       # heads: not a multiple of the kv-heads
    assert call(o=rows(16)) == INVALID
    assert call(v=rows(1)) == INVALID
    assert call(q=rows(258), o=rows(258), k=rows(1), v=rows(1)) == UNSUPPORTED
    assert call(k=rows(2, ts=0)) == INVALID and call(v=rows(2, hs=-128)) == INVALID
    assert call(ws=PTR, wn=16) == WORKSPACE
    assert call(ws=PTR + 4, wn=1 << 40) == INVALID


def test_bindings_want_gpu_tensors():
    import torch
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nat.qk_norm_rope(x)
    with pytest.raises(ValueError):
        nat.prompt_attention(x, x, x, torch.ones(1, dtype=torch.int32), torch.ones(1, dtype=torch.int32), 2, 0.1)


def test_outputs_whose_rows_share_memory_are_refused(L):
    """Both strides at least a row, yet two (token, head) pairs in one place; either order of nesting is fine."""
    def call(ts, hs, T=4, H=4, D=128):
        return L.pkv_qk_norm_rope(rows(H, D), rows(H, D, ts=ts, hs=hs), None, None, 0, D, T, None, None, 0, None, None,
                                  -2.0, None)

    assert call(128, 128) == INVALID
    assert call(256, 128) == INVALID
    assert call(3 * 128, 128) == INVALID
    assert call(128, 3 * 128) == INVALID
    assert call(-3 * 128, 128) == INVALID
    assert call(64, 4 * 128) == INVALID
    assert call(2 ** 61, 2 ** 61) == INVALID                # (the spans pass 64 bits)
    # (these pass the checks of the rows: what refuses them is the missing device, or that no tokens are given)
    for ts, hs, T, H in ((512, 128, 4, 4), (128, 512, 4, 4), (-512, 128, 4, 4), (128, -512, 4, 4), (0, 128, 1, 4),
                         (128, 0, 4, 1), (0, 0, 1, 1), (640, 128, 4, 4)):
        assert call(ts, hs, T, H) != INVALID
