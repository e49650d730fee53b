"""Block tables from request lengths and accepted paths, against plain Python."""

import random

import pytest
import torch

from masked_helpers import page_view
from paged_kv_decode_14_gb300 import _native as nat

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def blocks(n):
    return -(-n // 16)


class Model:
    """The contract, request by request."""

    def __init__(self, num_blocks, wide, lens, rnd):
        ids = list(range(num_blocks))
        rnd.shuffle(ids)
        self.num_blocks, self.wide, self.lens = num_blocks, wide, list(lens)
        self.table = [[-1] * wide for _ in lens]
        for b, n in enumerate(lens):
            for j in range(blocks(n)):
                self.table[b][j] = ids.pop()
        self.free = ids + [-5] * (num_blocks - len(ids))
        self.count = len(ids)

    def update(self, grow, num_rows):
        err, n = 0, len(self.lens)
        change, rows, at, starts = [], [], 0, []
        ok = 0 <= self.count <= self.num_blocks
        if not ok:
            err |= nat.DEVERR_LENGTH
        for b, g in enumerate(grow):
            bad = self.lens[b] < 0 or self.lens[b] + g < 0 or self.lens[b] + g > 16 * self.wide
            starts.append(at)
            at += max(g, 0)
            if bad or (g > 0 and at > num_rows):
                err |= nat.DEVERR_LENGTH if g else 0
                bad = True
            change.append(0 if bad or not ok else g)
        old = list(self.lens)
        for b in reversed(range(n)):
            if change[b] < 0:
                for j in reversed(range(blocks(old[b] + change[b]), blocks(old[b]))):
                    e = self.table[b][j]
                    self.table[b][j] = -1
                    if 0 <= e < self.num_blocks:
                        self.free[self.count] = e
                        self.count += 1
                    elif e >= self.num_blocks:
                        err |= nat.DEVERR_BLOCK_ID
        need, top = 0, self.count
        slots = []
        for b in range(n):
            c = max(0, blocks(old[b] + change[b]) - blocks(old[b]))
            need += c
            if c and need > top:
                change[b] = 0
                err |= nat.DEVERR_NO_BLOCKS
            elif c:
                for j in range(blocks(old[b]), blocks(old[b]) + c):
                    self.count -= 1
                    self.table[b][j] = self.free[self.count]
            self.lens[b] += change[b]
            for i in range(max(grow[b], 0)):
                p = old[b] + i
                slots.append((self.table[b][p // 16] * 16 + p % 16 if change[b] > 0 else -1, p))
        return slots[:num_rows], [max(c, 0) for c in change], starts, err


def run_both(m, pool, table, lens, grow, num_rows, extra=0, **kw):
    err = ints([0])
    slots = torch.full((num_rows + extra,), 99, dtype=torch.int64, device="cuda")
    pos = torch.full((num_rows + extra,), 99, dtype=torch.int32, device="cuda")
    out = nat.update_tables(pool, table, lens, ints(grow), num_rows, slots=slots[:num_rows], positions=pos[:num_rows],
                            device_error=err, **kw)
    want, granted, starts, code = m.update(grow, num_rows)
    assert slots.tolist()[:len(want)] == [w[0] for w in want]
    assert pos.tolist()[:len(want)] == [w[1] for w in want]
    assert all(x == 99 for x in slots.tolist()[len(want):] + pos.tolist()[len(want):])
    assert out[2].tolist() == granted and out[3].tolist() == starts
    assert table.tolist() == m.table and lens.tolist() == m.lens
    assert pool.count.tolist() == [m.count] and pool.free.tolist()[:m.count] == m.free[:m.count]
    assert nat.read_device_error(err) == code
    return code


def on_gpu(m):
    return (nat.BlockPool(m.num_blocks, free=ints(m.free), count=ints([m.count])), ints(m.table), ints(m.lens))


@pytest.mark.parametrize("n", [1, 3, 40, 1500, 8192])
def test_growth_and_drops(n):
    rnd = random.Random(n)
    top = 200 if n < 100 else 40
    lens = [rnd.choice((0, 1, 15, 16, 17, rnd.randint(0, top))) for _ in range(n)]
    wide = blocks(2 * top + 40)
    m = Model(sum(map(blocks, lens)) + n * 4 + 20, wide, lens, rnd)
    state = on_gpu(m)
    for step in range(4):
        grow = [rnd.choice((0, 1, 1, 2, 17, rnd.randint(0, top // 2), -min(m.lens[b], rnd.randint(0, top)), -m.lens[b]))
                for b in range(n)]
        run_both(m, *state, grow, sum(max(g, 0) for g in grow), extra=3)


def test_the_negated_call_restores_everything():
    rnd = random.Random(4)
    lens = [rnd.randint(0, 90) for _ in range(50)]
    m = Model(900, 12, lens, rnd)
    state = on_gpu(m)
    before = [t.clone() for t in (state[0].free[:m.count], state[0].count, state[1], state[2])]
    grow = [rnd.choice((-lens[b], 5, 40, -min(lens[b], 3), 0)) for b in range(50)]
    for g in (grow, [-x for x in grow]):
        assert run_both(m, *state, g, sum(max(x, 0) for x in g)) == 0
    after = (state[0].free[:m.count], state[0].count, state[1], state[2])
    assert all(torch.equal(x, y) for x, y in zip(before, after))


def test_many_rows():
    """More rows than one CTA takes: a cluster of them."""
    rnd = random.Random(9)
    lens = [rnd.randint(0, 400) for _ in range(30)]
    m = Model(4000, 200, lens, rnd)
    state = on_gpu(m)
    grow = [rnd.choice((rnd.randint(0, 2500), -lens[b], 1, 0)) for b in range(30)]
    run_both(m, *state, grow, sum(max(g, 0) for g in grow))
    run_both(m, *state, [-max(g, 0) for g in grow], 5000)


def test_refusals_of_requests():
    rnd = random.Random(1)
    m = Model(16, 8, [16, 16, 16, 5, 128, 0], rnd)                      # 4 are free
    state = on_gpu(m)
    # the second needs more than are left; the third behind it too; one that needs none is granted
    assert run_both(m, *state, [33, 40, 1, 3, 0, 0], 77) == nat.DEVERR_NO_BLOCKS
    # past the table's row, below 0
    assert run_both(m, *state, [0, 0, 0, -9, 1, 0], 1) == nat.DEVERR_LENGTH
    # rows that do not fit
    assert run_both(m, *state, [1, 2, 0, 1, 0, 0], 3) == nat.DEVERR_LENGTH
    # blocks that come back in the same call are there for it
    assert run_both(m, *state, [0, 0, -16, 0, -128, 100], 100) == 0


def test_bad_ids_and_counts():
    rnd = random.Random(1)
    m = Model(16, 8, [40, 40], rnd)
    m.table[1][0], m.table[1][1], m.table[1][2] = -1, 77, m.table[1][2]   # one given back earlier, one bad
    state = on_gpu(m)
    assert run_both(m, *state, [0, -40], 0) == nat.DEVERR_BLOCK_ID
    m.count = 17
    state = (nat.BlockPool(16, free=state[0].free, count=ints([17])), state[1], state[2])
    assert run_both(m, *state, [1, 1], 2) == nat.DEVERR_LENGTH
    # a bad id in the pool: entry and slots -1
    pool, table, lens, err = nat.BlockPool(8), torch.full((1, 4), -1, dtype=torch.int32, device="cuda"), ints([0]), ints([0])
    pool.free[7] = 8
    slots, pos, granted, _ = nat.update_tables(pool, table, lens, ints([17]), 17, device_error=err)
    assert nat.read_device_error(err) == nat.DEVERR_BLOCK_ID
    assert table.tolist() == [[-1, 1, -1, -1]] and slots.tolist() == [-1] * 16 + [16] and granted.tolist() == [17]


# ------------------------------------------------------------------ accepted paths


def make_cache(dtype, heads, dim, num_blocks, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (num_blocks, heads, 16 * dim)
    if dtype == "bf16":
        k, v = (torch.randn(shape, generator=g, device="cuda").bfloat16() for _ in range(2))
        return nat.PagedKVCache(num_blocks, heads, dim, "bf16", k=k, v=v)
    k, v = (torch.randint(0, 256, shape, generator=g, device="cuda").to(torch.uint8) for _ in range(2))   # every code, NaN too
    s = [torch.exp(torch.randn(num_blocks, heads, generator=g, device="cuda")) for _ in range(2)]
    return nat.PagedKVCache(num_blocks, heads, dim, "fp8", k=k, v=v, k_scales=s[0], v_scales=s[1])


def moved(cache, dtype, table, lens, q_lens, paths):
    got = []
    for pool, scales in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        was, new = (page_view(pool.clone(), cache.num_kv_heads, cache.head_dim) for _ in range(2))
        for b, path in enumerate(paths):
            base = lens[b] - q_lens[b]
            for i, j in enumerate(path):
                src, dst = base + j, base + i
                b0, b1 = int(table[b][src // 16]), int(table[b][dst // 16])
                x = was[b0, :, src % 16 // 8, :, src % 8]
                if scales is not None and b0 != b1:
                    y = x.view(torch.float8_e4m3fn).float() * scales[b0][:, None, None] / scales[b1][:, None, None]
                    x = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                new[b1, :, dst % 16 // 8, :, dst % 8] = x
        got.append(new.reshape(pool.shape))
    return got


def same(x, y):
    if x.dtype == torch.uint8:
        nan = ((x & 0x7f) == 0x7f) & ((y & 0x7f) == 0x7f)
        return bool((nan | (x == y)).all())
    return torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("dim,heads", [(64, 1), (128, 8), (128, 3)])
def test_keep_path(dtype, dim, heads):
    rnd = random.Random(dim + heads)
    lens, q_lens, paths = [], [], []
    for kind in range(14):
        q = rnd.choice((1, 2, 7, 40, 300))
        lens.append(q + rnd.choice((0, 1, 15, 16, 100)))
        q_lens.append(q)
        n = rnd.randint(0, q)
        paths.append(sorted(rnd.sample(range(q), n)) if kind % 3 else list(range(n)))     # (moved rows are read by others)
    need = [blocks(n) for n in lens]
    order = list(range(sum(need) + 2))
    rnd.shuffle(order)
    table = [[order.pop() for _ in range(n)] + [-1] * (max(need) - n) for n in need]
    cache = make_cache(dtype, heads, dim, sum(need) + 2, dim)
    want = moved(cache, dtype, table, lens, q_lens, paths)
    most = max(map(len, paths))
    err = ints([0])
    nat.keep_path(cache, ints(table), ints(lens), ints(q_lens), ints([p + [-1] * (most - len(p)) for p in paths]),
                  ints([len(p) for p in paths]), device_error=err)
    assert nat.read_device_error(err) == 0
    assert same(cache.k, want[0]) and same(cache.v, want[1])


def test_keep_path_leaves_bad_sequences():
    cache = make_cache("bf16", 2, 64, 8, 0)
    before = cache.k.clone(), cache.v.clone()
    table, lens, q_lens = [[0, 1], [2, 3], [4, 9], [5, 6], [7, -1]], [20, 20, 20, 20, 33], [8, 8, 20, 8, 8]
    path = [[0, 2, 2], [1, 8, -1], [17, -1, -1], [1, 2, 3], [1, 2, 3]]
    err = ints([0])
    nat.keep_path(cache, ints(table), ints(lens), ints(q_lens), ints(path), ints([3, 2, 1, 4, 3]), device_error=err)
    assert nat.read_device_error(err) == nat.DEVERR_LENGTH | nat.DEVERR_BLOCK_ID
    assert torch.equal(cache.k, before[0]) and torch.equal(cache.v, before[1])
