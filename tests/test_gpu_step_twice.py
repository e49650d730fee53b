"""Blocks that come back twice: more than the pool has room for."""

import random

import pytest
import torch

from paged_kv_decode_14_gb300 import _native as nat
from test_gpu_step_tables import Model, ints, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [4, 5000])                              # one CTA, and a cluster of eight
@pytest.mark.parametrize("length", [40, 500])                            # dropped blocks by threads, and by warps
def test_drops_past_the_pools_room_are_refused(length, rows):
    """A block of request 0 is free already, and everybody leaves: one more comes back than there is room for."""
    rnd = random.Random(length)
    per = -(-length // 16)
    m = Model(6 * per, 2 * per, [length] * 5 + [0], rnd)                 # (`per` blocks are free)
    m.free[m.count] = m.table[0][0]
    m.count += 1
    pool, table, lens = on_gpu(m)
    before = [t.clone() for t in (pool.free, pool.count, table, lens)]
    err = ints([0])
    slots, _, granted, _ = nat.update_tables(pool, table, lens, ints([-length] * 5 + [0]), rows, device_error=err)
    assert nat.read_device_error(err) == nat.DEVERR_BLOCK_ID
    assert all(torch.equal(x, y) for x, y in zip(before, (pool.free, pool.count, table, lens)))
    assert granted.tolist() == [0] * 6 and slots.tolist() == [-1] * rows
    # beside a request that grows: it does, with blocks that were free before
    slots, _, granted, _ = nat.update_tables(pool, table, lens, ints([-length] * 5 + [3]), rows, device_error=err)
    assert nat.read_device_error(err) == nat.DEVERR_BLOCK_ID
    assert granted.tolist() == [0] * 5 + [3] and lens.tolist() == [length] * 5 + [3]
    top = m.free[m.count - 1]
    assert slots.tolist() == [16 * top + i for i in range(3)] + [-1] * (rows - 3) and pool.count.item() == m.count - 1
    want = [r[:] for r in m.table]
    want[5][0] = top
    assert table.tolist() == want
    # and without it there is room
    nat.update_tables(pool, table, lens, ints([0, 0, 0, 0, -length, -3]), rows, device_error=err)
    assert nat.read_device_error(err) == 0 and lens.tolist() == [length] * 4 + [0, 0]
    assert pool.count.item() == m.count + per
