"""Cases of the operators between the projections and the paged KV cache: rotary positions with per-head norms, the
same pass writing the cache (bf16, or e4m3 with page scales), the cache read back into rows, and causal attention of
packed prompts.  Each in a plain form (elementary torch operations) and through the library's entry points."""

import math
import random

import torch

own = False

NAMES = ("norm_rope", "append", "read", "attention")
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases


def _norm_rope(tokens, heads, kv_heads, dim, dtype, rotary, interleaved, scaling, norm, fused, far, **more):
    return dict(more, op="norm_rope", tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
                rotary=rotary, interleaved=interleaved, scaling=scaling, norm=norm, fused=fused, far=far)


def _append(seqs, new_min, new_max, ctx_min, ctx_max, heads, kv_heads, dim, cache, from_values, rotary, interleaved,
            scaling, norm, fused, mix, **more):
    return dict(more, op="append", seqs=seqs, new_min=new_min, new_max=new_max, ctx_min=ctx_min, ctx_max=ctx_max,
                heads=heads, kv_heads=kv_heads, dim=dim, cache=cache, from_values=from_values, rotary=rotary,
                interleaved=interleaved, scaling=scaling, norm=norm, fused=fused, mix=mix)


def _read(seqs, len_min, len_max, kv_heads, dim, cache, dtype, mix, **more):
    return dict(more, op="read", seqs=seqs, len_min=len_min, len_max=len_max, kv_heads=kv_heads, dim=dim, cache=cache,
                dtype=dtype, mix=mix)


def _attention(seqs, q_min, q_max, ctx_min, ctx_max, heads, kv_heads, dim, dtype, fused, mix, **more):
    return dict(more, op="attention", seqs=seqs, q_min=q_min, q_max=q_max, ctx_min=ctx_min, ctx_max=ctx_max,
                heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, fused=fused, mix=mix)


def listed():
    return [
        # the tokens of one decode step of a 32-sequence batch: norms and rotation before anything is cached
        _norm_rope(32, 32, 8, 128, "bf16", 128, False, "none", True, False, 2048, name="norm_rope_step"),
        # a long prompt out of a fused projection, half of each head rotated in the interleaved layout, frequencies
        # scaled for a context that is longer than the one trained on
        _norm_rope(8192, 32, 8, 128, "bf16", 64, True, "ramp", False, True, 131072, name="norm_rope_prompt"),
        # one decode step of a 32-sequence batch into a bf16 cache
        _append(32, 1, 1, 255, 2047, 32, 8, 128, "bf16", False, 128, False, "none", True, False, 1,
                name="append_step"),
        # four whole prompts of about 2k tokens into an FP8 cache whose page scales come from the values
        _append(4, 1801, 2048, 0, 0, 32, 8, 128, "fp8", True, 128, False, "bands", True, True, 2,
                name="append_prompts_fp8"),
        # the windows of a speculative verify step into an FP8 cache that keeps its scales
        _append(32, 5, 5, 512, 4091, 32, 8, 64, "fp8", False, 32, True, "linear", False, False, 3,
                name="append_windows_fp8"),
        # a few short conversations' context brought back as rows
        _read(4, 1, 256, 2, 64, "bf16", "bf16", 4, name="read_short"),
        # the resident context of sixteen long sequences in an FP8 cache, dequantised for their next prompt chunk
        _read(16, 501, 8192, 8, 128, "fp8", "bf16", 5, name="read_context_fp8"),
        # the smallest call: four short prompts of a small model
        _attention(4, 1, 64, 0, 0, 8, 2, 64, "fp16", False, 6, name="attention_short"),
        # four 2k-token prompts
        _attention(4, 2048, 2048, 0, 0, 32, 8, 128, "bf16", False, 7, name="attention_prompts"),
        # one 8k-token prompt out of a fused projection: the largest
        _attention(1, 8192, 8192, 0, 0, 32, 8, 128, "bf16", True, 8, name="attention_prompt_8k"),
        # prompt chunks of ragged lengths over the context that the earlier chunks left
        _attention(8, 385, 512, 2999, 3584, 32, 8, 128, "bf16", False, 9, name="attention_chunks"),
        # the last few tokens of two long prompts: few rows, a long axis
        _attention(2, 9, 33, 32001, 32768, 32, 8, 128, "fp16", False, 10, name="attention_few_rows"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(NAMES)
    kv = rng.choice((1, 2, 4, 8))
    heads = kv * rng.choice((1, 2, 3, 4, 5, 7, 8))
    mix = rng.randrange(1 << 20)
    scaling = rng.choice(("none", "linear", "ntk", "bands", "ramp"))
    inter, norm, fused = (rng.random() < 0.5 for _ in range(3))
    if op == "norm_rope":
        dim = rng.choice((64, 80, 96, 128, 192, 256))
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        most = max(1, (8192 * 40 * 128) // ((heads + kv) * dim * (2 if dtype == "fp32" else 1)))
        return _norm_rope(_log(rng, 1, min(16384, most)), heads, kv, dim, dtype, rng.choice((dim, dim // 2, 18)),
                          inter, scaling, norm, fused, _log(rng, 64, 1 << 20))
    dim = rng.choice((64, 128))
    if op == "append":
        seqs, cache = _log(rng, 1, 64), rng.choice(("bf16", "fp8"))
        heads = min(heads, 40)
        prompts = rng.random() < 0.5
        hi = _log(rng, 1, max(1, 8192 // seqs)) if prompts else rng.choice((1, 1, 2, 5))
        ctx = 0 if prompts and rng.random() < 0.5 else _log(rng, 1, 4096)
        return _append(seqs, (hi + 1) // 2, hi, ctx // 2, ctx, heads, kv, dim, cache, cache == "fp8" and prompts,
                       rng.choice((dim, dim // 2, 10)), inter, scaling, norm, fused, mix)
    if op == "read":
        seqs = _log(rng, 1, 64)
        hi = _log(rng, 1, 65536 // seqs)
        return _read(seqs, (hi + 2) // 3, hi, kv, dim, rng.choice(("bf16", "fp8")),
                     rng.choice(("bf16", "bf16", "fp16", "fp32")), mix)
    seqs = _log(rng, 1, 16)
    heads = min(heads, 32) if heads % kv == 0 and min(heads, 32) % kv == 0 else kv
    hi = _log(rng, 1, int(8192 / math.sqrt(seqs)))
    if rng.random() < 0.4:
        ctx = _log(rng, 16, max(16, min(32768, 8192 * 4096 // (seqs * hi) - hi)))
    else:
        ctx = 0
    return _attention(seqs, (hi + 1) // 2, hi, ctx // 2, ctx, heads, kv, dim, rng.choice(("bf16", "fp16")), fused, mix)


# ------------------------------------------------------------------ what follows from a case alone


def _spread(case, lo, hi, n, salt):
    r = random.Random(case["mix"] * 8 + salt)
    return [r.randint(lo, hi) for _ in range(n)]


def _lens(case):
    """(new tokens or queries, tokens resident before them) of each sequence."""
    n = case["seqs"]
    if case["op"] == "read":
        return [0] * n, _spread(case, case["len_min"], case["len_max"], n, 0)
    lo, hi = ("new_min", "new_max") if case["op"] == "append" else ("q_min", "q_max")
    return _spread(case, case[lo], case[hi], n, 0), _spread(case, case["ctx_min"], case["ctx_max"], n, 1)


THETA, FACTOR, ORIGINAL, LOW, HIGH = 500000.0, 8.0, 8192, 1.0, 4.0


def _frequencies(case):
    """Radians per position of each rotated pair, and the factor of cos and sin, in Python's doubles."""
    rd, kind = case["rotary"], case["scaling"]
    base = THETA * FACTOR ** (rd / (rd - 2)) if kind == "ntk" else THETA
    f = [base ** (-2.0 * i / rd) for i in range(rd // 2)]
    if kind == "linear":
        f = [x / FACTOR for x in f]
    elif kind == "bands":
        t = [min(1.0, max(0.0, (ORIGINAL * x / (2 * math.pi) - LOW) / (HIGH - LOW))) for x in f]
        f = [x * (u + (1 - u) / FACTOR) for x, u in zip(f, t)]
    elif kind == "ramp":
        at = lambda turns: rd * math.log(ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(THETA))  # noqa: E731
        lo, hi = max(0, math.floor(at(32.0))), min(rd - 1, math.ceil(at(1.0)))
        t = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rd // 2)]
        f = [x * ((1 - u) + u / FACTOR) for x, u in zip(f, t)]
    return f, (0.1 * math.log(FACTOR) + 1.0 if kind == "ramp" else 1.0)


def work(case):
    op, d = case["op"], case["dim"]
    if op == "norm_rope":
        e = 4 if case["dtype"] == "fp32" else 2
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * d
        return {"bytes": 2 * n * e + 4 * case["tokens"], "flops": 6 * n}
    new, ctx = _lens(case)
    if op == "append":
        t, e = sum(new), 1 if case["cache"] == "fp8" else 2
        n = t * (case["heads"] + 2 * case["kv_heads"]) * d
        return {"bytes": 2 * n + 2 * t * case["heads"] * d + 2 * t * case["kv_heads"] * d * e + 12 * t, "flops": 6 * n}
    if op == "read":
        t, e = sum(ctx), 1 if case["cache"] == "fp8" else 2
        out = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * t * case["kv_heads"] * d * (e + out), "flops": 2 * t * case["kv_heads"] * d}
    pairs = sum(q * c + q * (q + 1) // 2 for q, c in zip(new, ctx))
    rows, keys = sum(new), sum(new) + sum(ctx)
    return {"bytes": 4 * rows * case["heads"] * d + 4 * rows * case["heads"] + 4 * keys * case["kv_heads"] * d,
            "flops": 4 * d * case["heads"] * pairs}


# ------------------------------------------------------------------ inputs


def _rows(g, tokens, parts, dim, dtype, fused):
    """Random rows of `parts` (numbers of heads): views of one fused projection's output, or tensors of their own."""
    if fused:
        x = torch.randn(tokens, sum(parts) * dim, generator=g, device="cuda").to(dtype)
        return [y.view(tokens, h, dim) for y, h in zip(x.split([h * dim for h in parts], 1), parts)]
    return [torch.randn(tokens, h, dim, generator=g, device="cuda").to(dtype) for h in parts]


def _rope_state(case, g, dtype, s):
    f, s["magnitude"] = _frequencies(case)
    s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    s["eps"] = 1e-6
    s["q_weight"] = s["k_weight"] = None
    if case["norm"]:
        s["q_weight"], s["k_weight"] = (
            (1 + 0.2 * torch.randn(case["dim"], generator=g, device="cuda")).to(dtype) for _ in range(2))


def _pages(case, g, tokens):
    """Physical blocks for sequences of `tokens` tokens, in a seeded order: (number of blocks, block table)."""
    need = [(n + 15) // 16 for n in tokens]
    total = sum(need) + 8
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    wide = max(max(need), 1)
    table = torch.full((len(need), wide), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return total, table


def _pool(case, g, blocks):
    """A cache as earlier calls left it: (k, v, k_scales, v_scales)."""
    shape = (blocks, case["kv_heads"], 16 * case["dim"])
    kv = [torch.randn(shape, generator=g, device="cuda") for _ in range(2)]
    if case["cache"] == "bf16":
        return kv[0].bfloat16(), kv[1].bfloat16(), None, None
    scales = [0.005 + 0.01 * torch.rand(blocks, case["kv_heads"], generator=g, device="cuda") for _ in range(2)]
    codes = [(x / y[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x, y in zip(kv, scales)]
    return codes[0], codes[1], scales[0], scales[1]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2654435761 % (1 << 40) + 17)
    s = {"case": case}
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if case["op"] == "norm_rope":
        dtype, t = TYPES[case["dtype"]], case["tokens"]
        s["q"], s["k"] = _rows(g, t, (case["heads"], case["kv_heads"], case["kv_heads"]), case["dim"], dtype,
                               case["fused"])[:2]
        s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device="cuda", dtype=torch.int32)
        _rope_state(case, g, dtype, s)
        return s
    new, ctx = _lens(case)
    if case["op"] == "attention":
        dtype = TYPES[case["dtype"]]
        keys = [a + b for a, b in zip(new, ctx)]
        if sum(ctx) == 0:
            s["q"], s["k"], s["v"] = _rows(g, sum(new), (case["heads"], case["kv_heads"], case["kv_heads"]),
                                           case["dim"], dtype, case["fused"])
        else:
            s["q"], = _rows(g, sum(new), (case["heads"],), case["dim"], dtype, False)
            s["k"], s["v"] = _rows(g, sum(keys), (case["kv_heads"],) * 2, case["dim"], dtype, case["fused"])
        s["q_lens"], s["kv_lens"] = ints(new), ints(keys)
        s["max_q"], s["max_kv"] = max(new), max(keys)
        return s
    if case["op"] == "read":
        blocks, s["table"] = _pages(case, g, ctx)
        s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"] = _pool(case, g, blocks)
        s["lens"], s["rows"] = ints(ctx), sum(ctx)
        return s
    blocks, table = _pages(case, g, [a + b for a, b in zip(new, ctx)])
    s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"] = _pool(case, g, blocks)
    s["q"], s["k"], s["v"] = _rows(g, sum(new), (case["heads"], case["kv_heads"], case["kv_heads"]), case["dim"],
                                   torch.bfloat16, case["fused"])
    at = torch.cat([torch.arange(c, c + n, device="cuda") for n, c in zip(new, ctx)])
    seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), ints(new).long())
    s["positions"] = at.to(torch.int32)
    s["slots"] = table[seq, at // 16].long() * 16 + at % 16
    _rope_state(case, g, torch.bfloat16, s)
    return s


# ------------------------------------------------------------------ the plain forms


def _norm_rotate(s, x, weight):
    """x [T, H, D] in 32 bits, normed over D where there is a weight, its first `rotary` dimensions rotated."""
    case = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight.float()
    rd = case["rotary"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    c, n = ((t * s["magnitude"]).float()[:, None] for t in (angle.cos(), angle.sin()))
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if case["interleaved"] else (x[..., :rd // 2], x[..., rd // 2:rd])
    y, z = a * c - b * n, b * c + a * n
    r = torch.stack((y, z), -1).flatten(-2) if case["interleaved"] else torch.cat((y, z), -1)
    return torch.cat((r, x[..., rd:]), -1)


def _paged(pool, kv_heads, dim):
    """The cache's pages as [block, kv head, 8-token group, 16-byte chunk, token, element]."""
    c = 16 // pool.element_size()
    return pool.view(pool.shape[0], kv_heads, 2, dim // c, 8, c)


def _store(s, pool, scales, x):
    """Rows x [T, Hkv, D] (32 bits) into the slots; the page scales, replaced for the blocks that the call starts."""
    case = s["case"]
    blk, off = s["slots"] // 16, s["slots"] % 16
    if scales is None:
        x = x.to(torch.bfloat16)
    else:
        if case["from_values"]:
            started = torch.zeros(pool.shape[0], device="cuda").index_put((blk,), (off == 0).float(), accumulate=True)
            most = torch.zeros_like(scales).index_reduce(0, blk, x.abs().amax(-1), "amax")
            fresh = torch.where(most > 0, most / 448.0, torch.ones_like(most))
            scales.copy_(torch.where(started[:, None] > 0, fresh, scales))
        x = (x / scales[blk][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    p = _paged(pool, case["kv_heads"], case["dim"])
    p[blk, :, off // 8, :, off % 8, :] = x.reshape(x.shape[0], case["kv_heads"], p.shape[3], p.shape[5])


def _load(s, pool, scales):
    """The sequences' rows, packed [sum of lens, Hkv, D], in 32 bits."""
    case, row = s["case"], torch.arange(s["rows"], device="cuda")
    ends = s["lens"].long().cumsum(0)
    seq = (row[:, None] >= ends).sum(1)
    at = row - (ends - s["lens"])[seq]
    blk, off = s["table"][seq, at // 16].long(), at % 16
    x = _paged(pool, case["kv_heads"], case["dim"])[blk, :, off // 8, :, off % 8, :]
    x = x.reshape(s["rows"], case["kv_heads"], case["dim"])
    return x.float() if scales is None else x.view(torch.float8_e4m3fn).float() * scales[blk][..., None]


def _padded(x, lens, most):
    """Packed rows [T, H, D] as [B, most, H, D] in 32 bits (past a sequence's end: some other row)."""
    starts = lens.long().cumsum(0) - lens
    at = starts[:, None] + torch.arange(most, device="cuda")
    return x.float()[at.clamp(max=x.shape[0] - 1)]


def _softmax_v(s):
    case, q, k, v = s["case"], s["q"], s["k"], s["v"]
    b, hk, d = case["seqs"], case["kv_heads"], case["dim"]
    grp, mq, mk = case["heads"] // hk, s["max_q"], s["max_kv"]
    qp = _padded(q, s["q_lens"], mq).view(b, mq, hk, grp, d).permute(0, 2, 3, 1, 4).reshape(b, hk, grp * mq, d)
    kp, vp = (_padded(x, s["kv_lens"], mk).permute(0, 2, 1, 3) for x in (k, v))
    x = (qp @ kp.transpose(-1, -2)).mul_(d ** -0.5).view(b, hk, grp, mq, mk)
    i, j = torch.arange(mq, device="cuda")[:, None], torch.arange(mk, device="cuda")
    hidden = j > (s["kv_lens"] - s["q_lens"])[:, None, None] + i
    x.masked_fill_(hidden[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m.isinf(), torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(b, hk, grp * mq, mk) @ vp).view(b, hk, grp, mq, d) / torch.where(l > 0, l, torch.ones_like(l))
    lse = m + l.log()
    # back to the packed rows
    row = torch.arange(q.shape[0], device="cuda")
    ends = s["q_lens"].long().cumsum(0)
    seq = (row[:, None] >= ends).sum(1)
    at = row - (ends - s["q_lens"])[seq]
    o, lse = o.permute(0, 3, 1, 2, 4)[seq, at], lse.permute(0, 3, 1, 2, 4)[seq, at]
    return [o.reshape(q.shape).to(q.dtype), lse.reshape(q.shape[:2])]


def _plain(s):
    case = s["case"]
    if case["op"] == "norm_rope":
        return [_norm_rotate(s, s[x], s[x + "_weight"]).to(s[x].dtype) for x in ("q", "k")]
    if case["op"] == "append":
        _store(s, s["k_cache"], s["k_scales"], _norm_rotate(s, s["k"], s["k_weight"]))
        _store(s, s["v_cache"], s["v_scales"], s["v"].float())
        return _appended(s, _norm_rotate(s, s["q"], s["q_weight"]).to(torch.bfloat16))
    if case["op"] == "read":
        return [_load(s, s[x + "_cache"], s[x + "_scales"]).to(TYPES[case["dtype"]]) for x in ("k", "v")]
    return _softmax_v(s)


def _appended(s, q):
    if s["k_scales"] is None:
        return [q, s["k_cache"], s["v_cache"]]
    return [q, s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn), s["k_scales"],
            s["v_scales"]]


# ------------------------------------------------------------------ one pass


def _handles(s, lib):
    """What a program builds once and keeps: the cache handle, the rotation, the attention's workspace."""
    case = s["case"]
    h = {}
    if "k_cache" in s:
        h["cache"] = lib.PagedKVCache(s["k_cache"].shape[0], case["kv_heads"], case["dim"], case["cache"],
                                      k=s["k_cache"], v=s["v_cache"], k_scales=s["k_scales"], v_scales=s["v_scales"])
    if "inv_freq" in s:
        low, high = (1.0, 32.0) if case["scaling"] == "ramp" else (LOW, HIGH)
        h["rope"] = lib.Rope(case["rotary"], THETA, interleaved=case["interleaved"], scaling=case["scaling"],
                             factor=FACTOR, original_len=ORIGINAL, low=low, high=high)
    if case["op"] == "attention":
        h["workspace"] = lib.make_prompt_workspace()
    return h


def run(s):
    if not own:
        return _plain(s)
    from paged_kv_decode_14_gb300 import _native as lib

    if "handles" not in s:
        s["handles"] = _handles(s, lib)
    case, h = s["case"], s["handles"]
    if case["op"] == "norm_rope":
        return lib.qk_norm_rope(s["q"], s["k"], s["positions"], h["rope"], q_weight=s["q_weight"],
                                k_weight=s["k_weight"], eps=s["eps"] if case["norm"] else None)
    if case["op"] == "append":
        return _appended(s, lib.append_norm_rope(
            h["cache"], s["q"], s["k"], s["v"], s["slots"], s["positions"], h["rope"], q_weight=s["q_weight"],
            k_weight=s["k_weight"], eps=s["eps"] if case["norm"] else None,
            fp8_scales_from_values=case["from_values"]))
    if case["op"] == "read":
        return lib.read_cache(h["cache"], s["table"], s["lens"], s["rows"], dtype=TYPES[case["dtype"]])
    return lib.prompt_attention(s["q"], s["k"], s["v"], s["q_lens"], s["kv_lens"], s["max_q"], case["dim"] ** -0.5,
                                workspace=h["workspace"])


# ------------------------------------------------------------------ in 64 bits


def _exact_row(case, s, x, weight):
    y = x.to(torch.float64)
    if weight is not None:
        y = y / (y.square().sum(-1, keepdim=True) / case["dim"] + s["eps"]).sqrt() * weight.to(torch.float64)
    f, mag = _frequencies(case)
    z, rd = y.clone(), case["rotary"]
    for i, w in enumerate(f):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rd // 2)
        t = s["positions"].to(torch.float64)[:, None] * w
        z[..., a] = mag * (y[..., a] * t.cos() - y[..., b] * t.sin())
        z[..., b] = mag * (y[..., a] * t.sin() + y[..., b] * t.cos())
    return z


def _element(case, off, d):
    """The place of (token `off` of its page, dimension d) in a page."""
    c = 16 if case["cache"] == "fp8" else 8
    return ((off // 8) * (case["dim"] // c) + d // c) * 8 * c + (off % 8) * c + d % c


def _values(pool):
    return (pool if pool.dtype == torch.bfloat16 else pool.view(torch.float8_e4m3fn)).to(torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    dims = torch.arange(case["dim"], device="cuda")
    if case["op"] == "norm_rope":
        return [_exact_row(case, s, s[x], s[x + "_weight"]) for x in ("q", "k")]
    if case["op"] == "append":
        k, v = _exact_row(case, s, s["k"], s["k_weight"]), s["v"].to(torch.float64)
        blk, off = s["slots"] // 16, s["slots"] % 16
        place = _element(case, off[:, None], dims)
        caches, scales = [], []
        for x, pool, given in ((k, s["k_cache"], s["k_scales"]), (v, s["v_cache"], s["v_scales"])):
            out = _values(pool)
            if given is not None:
                sc = given.to(torch.float64)
                if case["from_values"]:
                    first = set(blk[off == 0].tolist())
                    size = x.abs().amax(-1)
                    for at in sorted(first):
                        most = size[blk == at].amax(0) / 448
                        sc[at] = torch.where(most > 0, most, torch.ones_like(most))
                x = (x / sc[blk][..., None]).clamp(-448, 448)
                scales.append(sc)
            for h in range(case["kv_heads"]):
                out[blk[:, None], h, place] = x[:, h]
            caches.append(out)
        return [_exact_row(case, s, s["q"], s["q_weight"])] + caches + scales
    if case["op"] == "read":
        got = []
        for pool, sc in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])):
            parts = []
            for b, n in enumerate(s["lens"].tolist()):
                at = torch.arange(n, device="cuda")
                blk = s["table"][b, at // 16].long()
                place = _element(case, (at % 16)[:, None], dims)
                x = _values(pool.index_select(0, blk)).gather(
                    2, place[:, None].expand(n, case["kv_heads"], case["dim"]))
                parts.append(x if sc is None else x * sc[blk].to(torch.float64)[..., None])
            got.append(torch.cat(parts))
        return got
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    grp, q0, k0 = case["heads"] // case["kv_heads"], 0, 0
    for nq, nk in zip(s["q_lens"].tolist(), s["kv_lens"].tolist()):
        for h in range(case["heads"]):
            k, v = (s[x][k0:k0 + nk, h // grp].to(torch.float64) for x in ("k", "v"))
            for at in range(0, nq, 2048):
                n = min(2048, nq - at)
                x = s["q"][q0 + at:q0 + at + n, h].to(torch.float64) @ k.t() * case["dim"] ** -0.5
                last = nk - nq + at + torch.arange(n, device="cuda")
                x = x.masked_fill(torch.arange(nk, device="cuda") > last[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                seen = last >= 0
                p = torch.where(seen[:, None], (x - torch.where(seen, z, 0 * z)[:, None]).exp(), 0 * x)
                out[q0 + at:q0 + at + n, h] = p @ v
                lse[q0 + at:q0 + at + n, h] = z
        q0, k0 = q0 + nq, k0 + nk
    return [out, lse]
