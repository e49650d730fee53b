"""Host side of the entry points of a step on the GPU: the argument checks, which run before anything is enqueued (no
GPU here: the pointers are never followed)."""

import ctypes
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


def rows(heads=32, D=128, ptr=PTR, ts=None, hs=None):
    return nat._ROWS.pack(ptr, heads * D if ts is None else ts, D if hs is None else hs, heads)


def cache(dtype=0, D=128, heads=8, k=PTR, scales=PTR, block=16):
    return nat._CACHE.pack(64, block, heads, D, dtype, k, PTR, scales if dtype else 0, scales if dtype else 0)


def test_layout_of_the_packed_cache():
    assert nat._CACHE.size == ctypes.sizeof(nat.CacheDesc) and nat._ROWS.size % 8 == 0
    d = nat.CacheDesc.from_buffer_copy(nat._CACHE.pack(5, 16, 3, 64, 1, 0x10, 0x20, 0x30, 0x40))
    assert (d.num_blocks, d.block_size, d.num_kv_heads, d.head_dim, d.kv_dtype) == (5, 16, 3, 64, 1)
    assert (d.k_cache, d.v_cache, d.k_scales, d.v_scales) == (0x10, 0x20, 0x30, 0x40)


@pytest.mark.parametrize("kind", ["window", "tree"])
def test_masked_attention_refusals(L, kind):
    size = L.pkv_masked_workspace_size()
    assert size > 0

    def call(c=cache(), q=rows(), o=rows(), lse=None, n=4, bt=PTR, mb=8, cl=PTR, ql=PTR, qs=None, seqs=2, mq=2, window=16,
             sinks=4, mask=PTR, words=1, scale=0.1, ws=PTR, size=size):
        if kind == "window":
            return L.pkv_paged_attention_window(c, q, o, lse, n, bt, mb, cl, ql, qs, seqs, mq, window, sinks, scale, ws,
                                                size, None)
        return L.pkv_paged_attention_tree(c, q, o, lse, n, bt, mb, cl, ql, qs, seqs, mq, mask, words, scale, ws, size, None)

    assert call(seqs=0) == OK and call(n=0) == OK
    assert call(c=None) == INVALID
    assert call(c=cache(D=96)) == UNSUPPORTED
    assert call(c=cache(block=32)) == UNSUPPORTED
    assert call(c=cache(dtype=1, scales=0)) == INVALID
    assert call(c=cache(k=PTR + 8)) == INVALID
    assert call(q=None) == INVALID and call(o=None) == INVALID
    assert call(bt=None) == INVALID and call(cl=None) == INVALID and call(ql=None) == INVALID
    assert call(mb=0) == INVALID and call(seqs=-1) == INVALID and call(n=-1) == INVALID and call(mq=0) == INVALID
    assert call(q=rows(31), o=rows(31)) == INVALID               # no whole groups
    assert call(o=rows(16)) == INVALID
    assert call(c=cache(heads=1), q=rows(256), o=rows(256)) == UNSUPPORTED     # G = 256
    assert call(q=rows(ptr=PTR + 8)) == INVALID
    assert call(q=rows(ts=32 * 128 + 4)) == INVALID              # 8-byte rows
    assert call(q=rows(ts=-32 * 128)) == INVALID
    assert call(o=rows(hs=0)) == INVALID                         # an output's rows on top of each other
    assert call(o=rows(ts=64)) == INVALID
    assert call(scale=0.0) == INVALID and call(scale=-1.0) == INVALID
    assert call(scale=float("nan")) == INVALID and call(scale=float("inf")) == INVALID
    assert call(ws=None) == WORKSPACE and call(size=size - 1) == WORKSPACE
    assert call(ws=PTR + 8) == INVALID
    assert call(n=1 << 31) == UNSUPPORTED
    if kind == "window":
        assert call(window=0) == INVALID and call(sinks=-1) == INVALID
    else:
        assert call(mask=None) == INVALID
        assert call(mq=33, words=1) == INVALID and call(words=0) == INVALID and call(words=-1) == INVALID


def test_block_tables_update_refusals(L):
    def call(bt=PTR, mb=8, cl=PTR, grow=PTR, seqs=2, free=PTR, count=PTR, blocks=64, slots=PTR, pos=None, granted=None,
             starts=None, n=4):
        return L.pkv_block_tables_update(bt, mb, cl, grow, seqs, free, count, blocks, slots, pos, granted, starts, n, None,
                                         None)

    assert call(seqs=0) == OK
    assert call(seqs=-1) == INVALID and call(n=-1) == INVALID and call(blocks=0) == INVALID and call(mb=0) == INVALID
    for what in ("bt", "cl", "grow", "free", "count", "slots"):
        assert call(**{what: None}) == INVALID
    assert call(seqs=8193) == UNSUPPORTED
    assert call(mb=1 << 27) == UNSUPPORTED
    assert call(blocks=1 << 31) == UNSUPPORTED and call(n=1 << 31) == UNSUPPORTED


def test_keep_path_refusals(L):
    def call(c=cache(), bt=PTR, mb=8, cl=PTR, ql=PTR, path=PTR, most=4, lens=PTR, seqs=2):
        return L.pkv_paged_kv_keep_path(c, bt, mb, cl, ql, path, most, lens, seqs, None, None)

    assert call(seqs=0) == OK
    assert call(c=None) == INVALID and call(c=cache(D=80)) == UNSUPPORTED
    assert call(seqs=-1) == INVALID and call(most=-1) == INVALID and call(mb=0) == INVALID
    for what in ("bt", "cl", "ql", "path", "lens"):
        assert call(**{what: None}) == INVALID
    assert call(seqs=1 << 30) == UNSUPPORTED
    assert call(most=1 << 27) == UNSUPPORTED
