"""Refusals of pkv_block_tables_update_padded, which run before anything is enqueued (no GPU here)."""

from test_step_cpu import INVALID, OK, PTR, UNSUPPORTED, L  # noqa: F401  (L: the library, a fixture)


def test_padded_update_refusals(L):  # noqa: F811
    def call(bt=PTR, mb=8, cl=PTR, grow=PTR, seqs=2, free=PTR, count=PTR, blocks=64, slots=PTR, n=4):
        return L.pkv_block_tables_update_padded(bt, mb, cl, grow, seqs, free, count, blocks, slots, None, None, None, n, None,
                                                None)

    assert call(seqs=0, n=0, slots=None, bt=None) == OK
    assert call(seqs=0, slots=None) == INVALID
    assert call(seqs=-1) == INVALID and call(n=-1) == INVALID and call(blocks=0) == INVALID and call(mb=0) == INVALID
    for what in ("bt", "cl", "grow", "free", "count", "slots"):
        assert call(**{what: None}) == INVALID
    assert call(seqs=8193) == UNSUPPORTED and call(mb=1 << 27) == UNSUPPORTED
    assert call(blocks=1 << 31) == UNSUPPORTED and call(n=1 << 31) == UNSUPPORTED
