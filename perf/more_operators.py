"""Cases of the operators of a serving step that stays on the GPU: attention over the paged cache with a sliding window
and first tokens that stay visible, attention of a tree of drafted tokens, block tables and slots from request lengths,
and the accepted path of a tree moved into place.  Each in a plain form (elementary torch operations) and through the
library's entry points."""

import math
import random

import torch

own = False

NAMES = ("window", "tree", "tables", "keep")


# ------------------------------------------------------------------ cases


def _window(seqs, q_min, q_max, ctx_min, ctx_max, window, sinks, heads, kv_heads, dim, cache, released, mix, **more):
    return dict(more, op="window", seqs=seqs, q_min=q_min, q_max=q_max, ctx_min=ctx_min, ctx_max=ctx_max,
                window=window, sinks=sinks, heads=heads, kv_heads=kv_heads, dim=dim, cache=cache, released=released,
                mix=mix)


def _tree(seqs, q_min, q_max, ctx_min, ctx_max, heads, kv_heads, dim, cache, mix, **more):
    return dict(more, op="tree", seqs=seqs, q_min=q_min, q_max=q_max, ctx_min=ctx_min, ctx_max=ctx_max, heads=heads,
                kv_heads=kv_heads, dim=dim, cache=cache, mix=mix)


def _tables(seqs, new_min, new_max, ctx_min, ctx_max, leave, spare, mix, **more):
    return dict(more, op="tables", seqs=seqs, new_min=new_min, new_max=new_max, ctx_min=ctx_min, ctx_max=ctx_max,
                leave=leave, spare=spare, mix=mix)


def _keep(seqs, q_min, q_max, ctx_min, ctx_max, kv_heads, dim, cache, mix, **more):
    return dict(more, op="keep", seqs=seqs, q_min=q_min, q_max=q_max, ctx_min=ctx_min, ctx_max=ctx_max,
                kv_heads=kv_heads, dim=dim, cache=cache, mix=mix)


def listed():
    return [
        # single tokens of four short conversations of a small model: hardly more than a window each
        _window(4, 1, 1, 1, 192, 64, 4, 8, 2, 64, "bf16", False, 1, name="window_short"),
        # a decode step of 32 sequences, whole contexts resident, of which a layer with a window sees its last 1024
        _window(32, 1, 1, 256, 8192, 1024, 4, 32, 8, 128, "bf16", False, 2, name="window_step"),
        # a decode step of 128 long streams in an FP8 cache, the blocks behind the window given back
        _window(128, 1, 1, 501, 32768, 4096, 16, 32, 8, 128, "fp8", True, 3, name="window_streams_fp8"),
        # four 2k-token prompts of a layer with a window
        _window(4, 2048, 2048, 0, 0, 512, 4, 32, 8, 128, "bf16", False, 4, name="window_prompts"),
        # ragged prompt chunks over contexts that are longer than the window, FP8
        _window(8, 385, 512, 2999, 3584, 2048, 0, 32, 8, 128, "fp8", True, 5, name="window_chunks_fp8"),
        # one request's tree of seven drafted tokens
        _tree(1, 7, 7, 300, 300, 32, 8, 64, "bf16", 6, name="tree_single"),
        # a verify step of 32 requests with trees of up to 24 drafted tokens
        _tree(32, 9, 24, 512, 4072, 32, 8, 128, "bf16", 7, name="tree_step"),
        # trees of 64 drafted tokens over long contexts in an FP8 cache: the most arithmetic
        _tree(16, 64, 64, 8000, 16320, 32, 8, 128, "fp8", 8, name="tree_long_fp8"),
        # 256 decoding requests: a token each, and back
        _tables(256, 1, 1, 1, 2048, 0, 4096, 9, name="tables_step"),
        # requests that bring prompts beside ones that leave, and back
        _tables(96, 1, 1801, 0, 3000, 24, 16384, 10, name="tables_prompts"),
        # the accepted paths of 32 trees
        _keep(32, 9, 24, 512, 4072, 8, 128, "bf16", 11, name="keep_step"),
        # the accepted paths of 256 large trees in an FP8 cache, whose blocks have scales of their own
        _keep(256, 33, 64, 100, 1000, 8, 128, "fp8", 12, name="keep_large_fp8"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("window", "window", "window", "tree", "tree", "tables", "keep"))
    mix = rng.randrange(1 << 20)
    kv = rng.choice((1, 2, 4, 8))
    heads = kv * rng.choice((1, 2, 3, 4, 5, 7, 8))
    dim, cache = rng.choice((64, 128)), rng.choice(("bf16", "fp8"))
    if op == "window":
        kind = rng.choice(("step", "step", "verify", "prompts"))
        window, sinks = _log(rng, 1, 4096), rng.choice((0, 1, 4, 16, 100))
        if kind == "prompts":
            seqs = _log(rng, 1, 8)
            heads = min(heads, 4 * kv)
            hi = _log(rng, 17, int(4096 / math.sqrt(seqs)))
            lo, ctx = (hi + 1) // 2, rng.choice((0, _log(rng, 1, 4096)))
        else:
            seqs = _log(rng, 1, 128)
            lo = hi = 1 if kind == "step" else rng.randint(2, 16)
            ctx = _log(rng, 1, 32768)
        return _window(seqs, lo, hi, ctx // 3, ctx, window, sinks, heads, kv, dim, cache,
                       window + sinks < ctx // 3 and rng.random() < 0.7 or seqs * ctx > 1 << 19, mix)
    if op == "tree":
        seqs, hi = _log(rng, 1, 64), _log(rng, 2, 64)
        ctx = _log(rng, 1, 262144 // seqs)
        while seqs * hi * heads * ctx > 1 << 28:
            ctx //= 2
        return _tree(seqs, (hi + 1) // 2, hi, ctx // 2, ctx, heads, kv, dim, cache, mix)
    if op == "tables":
        seqs = _log(rng, 1, 512)
        hi = _log(rng, 1, max(1, 80000 // seqs))
        return _tables(seqs, rng.randint(0, hi), hi, 0, _log(rng, 1, 4096), rng.randint(0, seqs // 2),
                       _log(rng, 1, 16384), mix)
    seqs, hi = _log(rng, 1, 256), _log(rng, 2, 64)
    return _keep(seqs, (hi + 1) // 2, hi, 0, _log(rng, 1, 1000), kv, dim, cache, mix)


# ------------------------------------------------------------------ what follows from a case alone


def _spread(case, lo, hi, n, salt):
    r = random.Random(case["mix"] * 8 + salt)
    return [r.randint(lo, hi) for _ in range(n)]


def _lens(case):
    """(new tokens, all tokens with them) of each sequence."""
    n = case["seqs"]
    new = _spread(case, case["q_min"], case["q_max"], n, 0)
    return new, [a + b for a, b in zip(new, _spread(case, case["ctx_min"], case["ctx_max"], n, 1))]


def _changes(case):
    """(resident tokens, tokens that come (negative: that leave)) of each request."""
    n = case["seqs"]
    ctx = _spread(case, case["ctx_min"], case["ctx_max"], n, 1)
    new = _spread(case, case["new_min"], case["new_max"], n, 0)
    some = random.Random(case["mix"] * 8 + 2)
    for b in some.sample(range(n), case["leave"]):
        new[b] = -ctx[b] if some.random() < 0.5 else -some.randint(0, ctx[b])
    return ctx, new


def _accepted(case):
    """(path length, leading nodes that lie in place) of each sequence."""
    some = random.Random(case["mix"] * 8 + 3)
    out = []
    for t in _lens(case)[0]:
        n = some.randint(0, min(t, 8))
        stay = some.randint(max(0, 2 * n - t), n)
        out.append((n, stay))
    return out


def _blocks(n):
    return (n + 15) // 16


def _seen(case, q, length):
    """First position of the window part that any of the sequence's queries sees, and the pairs that are seen."""
    w, s = case["window"], case["sinks"]
    pairs = 0
    for p in range(length - q, length):
        lo = max(0, p - w + 1)
        pairs += p + 1 - lo + min(s, lo)
    return max(0, length - q - w + 1), pairs


def work(case):
    op = case["op"]
    if op == "tables":
        ctx, new = _changes(case)
        rows = sum(max(n, 0) for n in new)
        moved = sum(abs(_blocks(c + n) - _blocks(c)) for c, n in zip(ctx, new))
        back = sum(-min(n, 0) for n in new)
        # both ways: lengths and changes; each block's entry and place on the stack; slots and positions
        return {"bytes": 2 * (12 * len(ctx) + 8 * moved) + 12 * (rows + back), "flops": 4 * (rows + back)}
    e, kv, d = 1 if case["cache"] == "fp8" else 2, case["kv_heads"], case["dim"]
    if op == "keep":
        moved = sum(n - stay for n, stay in _accepted(case))
        return {"bytes": 4 * moved * kv * d * e + 4 * sum(n for n, _ in _accepted(case)), "flops": 4 * moved * kv * d}
    new, lens = _lens(case)
    if op == "tree":
        keys = sum(lens)
        # (a tree's rows see few of its own keys: they are left out)
        pairs = sum(q * (n - q) for q, n in zip(new, lens))
    else:
        keys = pairs = 0
        for q, n in zip(new, lens):
            lo, p = _seen(case, q, n)
            keys += n - lo + min(case["sinks"], lo)
            pairs += p
    rows = sum(new)
    scales = keys // 16 * kv * 8 if e == 1 else 0
    return {"bytes": 2 * keys * kv * d * e + scales + 4 * rows * case["heads"] * d + 4 * rows * case["heads"],
            "flops": 4 * d * case["heads"] * pairs}


# ------------------------------------------------------------------ inputs


def _pages(case, g, lens, held):
    """Physical blocks in a seeded order for the blocks of each sequence that `held(b, j)` says are resident:
    (number of blocks, block table)."""
    wide = max(1, max(_blocks(n) for n in lens))
    have = [[j for j in range(_blocks(n)) if held(b, j)] for b, n in enumerate(lens)]
    total = sum(map(len, have)) + 8
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.tensor([b * wide + j for b, row in enumerate(have) for j in row], dtype=torch.long, device="cuda")
    table = torch.full((len(lens) * wide,), -1, dtype=torch.int32, device="cuda")
    table[at] = order[:at.numel()]
    return total, table.view(len(lens), wide)


def _pool(case, g, blocks):
    """A cache as earlier calls left it: (k, v, k_scales, v_scales)."""
    shape = (blocks, case["kv_heads"], 16 * case["dim"])
    if case["cache"] == "bf16":
        k, v = (torch.randn(shape, generator=g, device="cuda").bfloat16() for _ in range(2))
        return k, v, None, None
    pools, scales = [], []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device="cuda")
        s = 0.005 + 0.01 * torch.rand(blocks, case["kv_heads"], generator=g, device="cuda")
        pools.append((x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        scales.append(s)
    return pools[0], pools[1], scales[0], scales[1]


def _trees(g, lens, most):
    """Ancestors and selves of random trees' nodes as bits, int32 [sum of lens, words]: each node hangs on an
    earlier one, or on the context."""
    n, parent = len(lens), []
    up = torch.rand(n, most, generator=g, device="cuda")
    bits = torch.zeros(n, most, dtype=torch.int64, device="cuda")
    for i in range(most):
        parent = (up[:, i] * (i + 1)).long().clamp(max=i) - 1           # -1: the context
        above = bits.gather(1, parent.clamp(min=0)[:, None])[:, 0]
        bits[:, i] = torch.where(parent >= 0, above, torch.zeros_like(above)) | (1 << i if i < 63 else -(1 << 63))
    rows = bits[torch.arange(most, device="cuda")[None] < torch.tensor(lens, device="cuda")[:, None]]
    words = torch.stack((rows << 32 >> 32, rows >> 32), 1).to(torch.int32)
    return words[:, :(most + 31) // 32].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 40) + 29)
    host = random.Random(int(seed) * 7919 + 5)
    s = {"case": case}
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "tables":
        ctx, new = _changes(case)
        need = sum(max(0, _blocks(c + n) - _blocks(c)) for c, n in zip(ctx, new))
        held = sum(_blocks(c) for c in ctx)
        s["num_blocks"] = held + need + case["spare"]
        order = torch.randperm(s["num_blocks"], generator=g, device="cuda").to(torch.int32)
        wide = max(1, max(_blocks(c + max(n, 0)) for c, n in zip(ctx, new)))
        first = torch.tensor([0] + [_blocks(c) for c in ctx], device="cuda").cumsum(0)
        at = torch.arange(wide, device="cuda")
        s["table"] = torch.where(at < (first[1:] - first[:-1])[:, None],
                                 order[(first[:-1, None] + at).clamp(max=s["num_blocks"] - 1)],
                                 torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()
        s["free"] = torch.cat((order[held:], order[:held]))             # (behind the count: whatever lay there)
        s["count"] = ints([s["num_blocks"] - held])
        s["lens"], s["grow"], s["back"] = ints(ctx), ints(new), ints([-n for n in new])
        s["rows"], s["back_rows"] = sum(max(n, 0) for n in new), sum(max(-n, 0) for n in new)
        return s
    new, lens = _lens(case)
    held = lambda b, j: True  # noqa: E731
    if case["op"] == "window" and case["released"]:
        low = [max(0, n - q - case["window"] + 1) // 16 for q, n in zip(new, lens)]
        held = lambda b, j: j >= low[b] or j * 16 < case["sinks"]  # noqa: E731
    blocks, s["table"] = _pages(case, g, lens, held)
    s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"] = _pool(case, g, blocks)
    s["lens"], s["q_lens"], s["max_q"], s["max_len"] = ints(lens), ints(new), max(new), max(lens)
    if case["op"] == "keep":
        paths = []
        for t, (n, stay) in zip(new, _accepted(case)):
            paths.append(list(range(stay)) + sorted(host.sample(range(n, t), n - stay)))
        most = max(1, max(map(len, paths)))
        s["path"] = ints([p + [-1] * (most - len(p)) for p in paths])
        s["path_lens"] = ints([len(p) for p in paths])
        return s
    s["q"] = torch.randn(sum(new), case["heads"], case["dim"], generator=g, device="cuda").bfloat16()
    if case["op"] == "tree":
        s["tree"] = _trees(g, new, s["max_q"])
    return s


# ------------------------------------------------------------------ the plain forms


def _paged(pool, kv_heads, dim):
    """The cache's pages as [block, kv head, 8-token group, 16-byte chunk, token, element]."""
    c = 16 // pool.element_size()
    return pool.view(pool.shape[0], kv_heads, 2, dim // c, 8, c)


def _gather(s, pool, scales, at):
    """The cached rows at positions at [B, K] in 32 bits: [B, Hkv, K, D]."""
    case = s["case"]
    blk = s["table"].gather(1, at // 16).long()
    off = at % 16
    x = _paged(pool, case["kv_heads"], case["dim"])[blk, :, off // 8, :, off % 8, :]
    x = x.reshape(*at.shape, case["kv_heads"], case["dim"])
    if scales is not None:
        x = x.view(torch.float8_e4m3fn).float() * scales[blk][..., None]
    return x.float().transpose(1, 2)


def _rows_of(lens, rows):
    """Sequence and index in it of each packed row."""
    row = torch.arange(rows, device="cuda")
    ends = lens.long().cumsum(0)
    seq = (row[:, None] >= ends).sum(1)
    return seq, row - (ends - lens)[seq]


def _attend(s, at, seen):
    """Attention of the packed queries over positions at [B, K], where seen [B, max_q, K]."""
    case, q = s["case"], s["q"]
    b, hk, d, mq = case["seqs"], case["kv_heads"], case["dim"], s["max_q"]
    grp = case["heads"] // hk
    seq, i = _rows_of(s["q_lens"], q.shape[0])
    first = s["q_lens"].long().cumsum(0) - s["q_lens"]
    qp = q.float()[(first[:, None] + torch.arange(mq, device="cuda")).clamp(max=q.shape[0] - 1)]
    qp = qp.view(b, mq, hk, grp, d).permute(0, 2, 3, 1, 4).reshape(b, hk, grp * mq, d)
    k = _gather(s, s["k_cache"], s["k_scales"], at)
    x = (qp @ k.transpose(-1, -2)).mul_(d ** -0.5).view(b, hk, grp, mq, at.shape[1])
    x.masked_fill_(~seen[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m.isinf(), torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    v = _gather(s, s["v_cache"], s["v_scales"], at)
    o = (p.view(b, hk, grp * mq, -1) @ v).view(b, hk, grp, mq, d) / torch.where(l > 0, l, torch.ones_like(l))
    o, lse = (t.permute(0, 3, 1, 2, 4)[seq, i] for t in (o, m + l.log()))
    return [o.reshape(q.shape).to(q.dtype), lse.reshape(q.shape[:2])]


def _plain_window(s):
    case = s["case"]
    new, lens = _lens(case)
    lo = (s["lens"] - s["q_lens"] - case["window"] + 1).clamp(min=0).long()
    front = lo.clamp(max=case["sinks"])
    most = max(n - max(0, n - q - case["window"] + 1) + min(case["sinks"], max(0, n - q - case["window"] + 1))
               for q, n in zip(new, lens))
    j = torch.arange(most, device="cuda")
    at = torch.where(j < front[:, None], j, j + (lo - front)[:, None])
    here = at < s["lens"][:, None]
    at = at.minimum(s["lens"][:, None] - 1)
    p = (s["lens"] - s["q_lens"])[:, None] + torch.arange(s["max_q"], device="cuda")
    p, key = p[..., None], at[:, None]
    seen = here[:, None] & (key <= p) & ((key > p - case["window"]) | (key < case["sinks"]))
    return _attend(s, at, seen)


def _plain_tree(s):
    at = torch.arange(s["max_len"], device="cuda")[None].expand(s["case"]["seqs"], -1)
    here = at < s["lens"][:, None]
    first = s["q_lens"].long().cumsum(0) - s["q_lens"]
    words = s["tree"].long()[(first[:, None] + torch.arange(s["max_q"], device="cuda")).clamp(max=s["q"].shape[0] - 1)]
    node = at - (s["lens"] - s["q_lens"])[:, None]                       # (negative: the context)
    which = node.clamp(min=0, max=32 * words.shape[2] - 1)
    bits = words.gather(2, (which // 32)[:, None].expand(-1, s["max_q"], -1)) >> (which % 32)[:, None] & 1
    seen = here[:, None] & ((node < 0)[:, None] | (bits != 0))
    return _attend(s, at.minimum(s["lens"][:, None].long() - 1), seen)


def _plain_update(s, grow, rows):
    """Table, lengths, stack and its count updated in place; (slots, positions)."""
    table, lens, free, count = s["table"], s["lens"], s["free"], s["count"]
    old, after = lens.clone(), lens + grow
    j = torch.arange(table.shape[1], device="cuda")
    had, has = ((old + 15) // 16)[:, None], ((after + 15) // 16)[:, None]
    # what leaves goes onto the stack, the last request's last block first
    gone = ((j >= has) & (j < had)).reshape(-1)
    place = gone.flip(0).long().cumsum(0).flip(0) - 1 + count
    stack = torch.cat((free, free.new_zeros(1)))
    stack[torch.where(gone, place, torch.full_like(place, free.numel()))] = table.reshape(-1)
    top = count + gone.sum()
    # what comes is taken from its top, the first request's first block first
    come = ((j >= had) & (j < has)).reshape(-1)
    place = top - come.long().cumsum(0)
    flat = torch.where(come, stack[place.clamp(min=0)], torch.where(gone, -1, table.reshape(-1)))
    table.copy_(flat.view_as(table))
    free.copy_(stack[:-1])
    count.copy_(top - come.sum())
    lens.copy_(after)
    seq, i = _rows_of(grow.clamp(min=0), rows)
    at = old[seq] + i
    return [table[seq, at // 16].long() * 16 + at % 16, at.to(torch.int32)]


def _plain_keep(s):
    case, path = s["case"], s["path"].long()
    i = torch.arange(path.shape[1], device="cuda")
    taken = i < s["path_lens"][:, None]
    base = (s["lens"] - s["q_lens"]).long()[:, None]
    to = torch.where(taken, base + i, torch.zeros_like(path))
    frm = torch.where(taken, base + path, torch.zeros_like(path))
    seq = torch.arange(case["seqs"], device="cuda")[:, None].expand_as(path)
    pick = lambda t: t.masked_select(taken)  # noqa: E731
    seq, to, frm = pick(seq), pick(to), pick(frm)
    b0, b1 = s["table"][seq, frm // 16].long(), s["table"][seq, to // 16].long()
    for pool, scales in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])):
        p = _paged(pool, case["kv_heads"], case["dim"])
        x = p[b0, :, frm % 16 // 8, :, frm % 8, :]
        if scales is not None:
            there = lambda b: scales[b][:, :, None, None]  # noqa: E731
            y = (x.view(torch.float8_e4m3fn).float() * there(b0) / there(b1)).clamp(-448, 448)
            x = torch.where((b0 == b1)[:, None, None, None], x, y.to(torch.float8_e4m3fn).view(torch.uint8))
        p[b1, :, to % 16 // 8, :, to % 8, :] = x
    return _caches(s)


def _caches(s):
    if s["k_scales"] is None:
        return [s["k_cache"], s["v_cache"]]
    return [s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn)]


def _plain(s):
    op = s["case"]["op"]
    if op == "window":
        return _plain_window(s)
    if op == "tree":
        return _plain_tree(s)
    if op == "keep":
        return _plain_keep(s)
    there = _plain_update(s, s["grow"], s["rows"])
    return there + _plain_update(s, s["back"], s["back_rows"]) + [s["table"], s["lens"], s["free"], s["count"]]


# ------------------------------------------------------------------ one pass


def _handles(s, lib):
    """What a program builds once and keeps: the cache handle, the attention's workspace, the pool of blocks."""
    case, h = s["case"], {}
    if case["op"] == "tables":
        h["pool"] = lib.BlockPool(s["num_blocks"], free=s["free"], count=s["count"])
        return h
    h["cache"] = lib.PagedKVCache(s["k_cache"].shape[0], case["kv_heads"], case["dim"], case["cache"], k=s["k_cache"],
                                  v=s["v_cache"], k_scales=s["k_scales"], v_scales=s["v_scales"])
    if case["op"] != "keep":
        h["workspace"] = lib.make_masked_workspace()
    return h


def run(s):
    if not own:
        return _plain(s)
    from paged_kv_decode_14_gb300 import _native as lib

    if "handles" not in s:
        s["handles"] = _handles(s, lib)
    case, h = s["case"], s["handles"]
    if case["op"] == "window":
        return lib.attention_window(h["cache"], s["q"], s["table"], s["lens"], s["q_lens"], s["max_q"], case["window"],
                                    case["sinks"], case["dim"] ** -0.5, h["workspace"])
    if case["op"] == "tree":
        return lib.attention_tree(h["cache"], s["q"], s["table"], s["lens"], s["q_lens"], s["max_q"], s["tree"],
                                  case["dim"] ** -0.5, h["workspace"])
    if case["op"] == "keep":
        lib.keep_path(h["cache"], s["table"], s["lens"], s["q_lens"], s["path"], s["path_lens"])
        return _caches(s)
    there = lib.update_tables(h["pool"], s["table"], s["lens"], s["grow"], s["rows"])
    back = lib.update_tables(h["pool"], s["table"], s["lens"], s["back"], s["back_rows"])
    return [*there[:2], *back[:2], s["table"], s["lens"], s["free"], s["count"]]


# ------------------------------------------------------------------ in 64 bits


def _element(case, off, d):
    """The place of (token `off` of its page, dimension d) in a page."""
    c = 16 if case["cache"] == "fp8" else 8
    return ((off // 8) * (case["dim"] // c) + d // c) * 8 * c + (off % 8) * c + d % c


def _exact_rows(s, b, at):
    """K and V of sequence b at positions `at`, [Hkv, K, D] in 64 bits."""
    case, got = s["case"], []
    blk = s["table"][b].long()[at // 16]
    place = _element(case, (at % 16)[:, None], torch.arange(case["dim"], device="cuda"))
    for pool, scales in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])):
        page = pool if scales is None else pool.view(torch.float8_e4m3fn)
        heads = torch.arange(case["kv_heads"], device="cuda")[:, None, None]
        x = page[blk[None, :, None], heads, place[None]].to(torch.float64)
        got.append(x if scales is None else x * scales[blk].t().to(torch.float64)[..., None])
    return got


def _exact_attention(s):
    case, q = s["case"], s["q"]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    grp, q0 = case["heads"] // case["kv_heads"], 0
    for b, (n, length) in enumerate(zip(s["q_lens"].tolist(), s["lens"].tolist())):
        pos = torch.arange(length, device="cuda")
        i = torch.arange(n, device="cuda")[:, None]
        if case["op"] == "window":
            own_pos = length - n + i
            far = own_pos - pos >= case["window"]
            seen = (pos <= own_pos) & ~(far & (pos >= case["sinks"]))
        else:
            seen = (pos < length - n).expand(n, length).clone()
            words = s["tree"][q0:q0 + n].tolist()
            tree = [[(w[j // 32] >> (j % 32)) & 1 for j in range(n)] for w in words]
            seen[:, length - n:] = torch.tensor(tree, device="cuda") != 0
        at = seen.any(0).nonzero()[:, 0]
        k, v = _exact_rows(s, b, at)
        for r in range(0, n, 1024):
            rows = q[q0 + r:q0 + min(n, r + 1024)].to(torch.float64)
            mask = seen[r:r + 1024][:, at]
            for g in range(case["kv_heads"]):
                for h in range(g * grp, g * grp + grp):
                    x = (rows[:, h] @ k[g].t() * case["dim"] ** -0.5).masked_fill(~mask, -math.inf)
                    z = torch.logsumexp(x, -1)
                    any_ = z > -math.inf
                    p = torch.exp(x - torch.where(any_, z, torch.zeros_like(z))[:, None])
                    out[q0 + r:q0 + r + rows.shape[0], h] = p @ v[g]
                    lse[q0 + r:q0 + r + rows.shape[0], h] = z
        q0 += n
    return [out, lse]


def _exact_tables(s):
    """The stack as a list, request by request; after both calls everything is as it was."""
    case = s["case"]
    stack = s["free"][:int(s["count"])].tolist()
    table, lens = s["table"].tolist(), s["lens"].tolist()
    rest, outs = s["free"].tolist(), []
    for grow in (s["grow"].tolist(), s["back"].tolist()):
        for b in reversed(range(case["seqs"])):
            for j in reversed(range(_blocks(lens[b] + grow[b]), _blocks(lens[b]))):
                stack.append(table[b][j])
                rest[len(stack) - 1] = table[b][j]
                table[b][j] = -1
        slots, positions = [], []
        for b in range(case["seqs"]):
            for j in range(_blocks(lens[b]), _blocks(lens[b] + grow[b])):
                table[b][j] = stack.pop()
            for p in range(lens[b], lens[b] + grow[b]):
                slots.append(table[b][p // 16] * 16 + p % 16)
                positions.append(p)
            lens[b] += grow[b]
        outs += [torch.tensor(slots, dtype=torch.int64), torch.tensor(positions, dtype=torch.int32)]
    return [t.cuda() for t in outs] + [torch.tensor(v, dtype=torch.int32, device="cuda")
                                       for v in (table, lens, rest, [len(stack)])]


def _exact_keep(s):
    case, dims = s["case"], torch.arange(s["case"]["dim"], device="cuda")
    caches = []
    for pool, scales in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])):
        was = (pool if scales is None else pool.view(torch.float8_e4m3fn)).to(torch.float64)
        new = was.clone()
        src, dst = [], []
        for b, n in enumerate(s["path_lens"].tolist()):
            base = int(s["lens"][b] - s["q_lens"][b])
            row, path = s["table"][b].tolist(), s["path"][b].tolist()
            for i in range(n):
                src.append((row[(base + path[i]) // 16], (base + path[i]) % 16))
                dst.append((row[(base + i) // 16], (base + i) % 16))
        if src:
            src, dst = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
            for h in range(case["kv_heads"]):
                x = was[src[:, :1], h, _element(case, src[:, 1:], dims)]
                if scales is not None:
                    r = scales[src[:, 0], h].to(torch.float64) / scales[dst[:, 0], h].to(torch.float64)
                    x = (x * r[:, None]).clamp(-448, 448)
                new[dst[:, :1], h, _element(case, dst[:, 1:], dims)] = x
        caches.append(new)
    return caches


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(s)
    return _exact_keep(s) if case["op"] == "keep" else _exact_attention(s)
