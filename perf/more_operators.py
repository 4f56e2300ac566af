"""Cases of the attention over prompts, of visible first tokens (sinks) beside a
sliding window, and of the key-value cache held in 4 bits.

`run` computes a case in plain torch operations, or through the library's
entry points where `own` is true.  Shapes are the Beam attention's (48 query
and 8 key-value heads of 128, sliding windows of 512) or generic ones.
"""

import math

import torch

own = False

DEV = "cuda"
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
MOST_SCORES = 48 * 16384 * 16384 // 2   # that the largest listed prompt needs


# ------------------------------------------------------------------ cases

def _prompt(B, new, prefix, cache, hq=48, hkv=8, d=128, window=0, sinks=0, page=64, singles=0, even=False, pad=0):
    return dict(op="prompt", B=B, new=new, prefix=prefix, cache=cache, hq=hq, hkv=hkv, d=d, window=window, sinks=sinks,
                page=page, singles=singles, even=even, pad=pad)


def _decode(B, longest, cache, hq=48, hkv=8, d=128, window=0, sinks=0, page=64, idle=0):
    return dict(op="decode", B=B, longest=longest, cache=cache, hq=hq, hkv=hkv, d=d, window=window, sinks=sinks,
                page=page, idle=idle)


def _append(T, hkv=8, d=128, act="bf16", page=64, prompt=True, idle=0):
    return dict(op="append", T=T, cache="fp4", hkv=hkv, d=d, act=act, page=page, prompt=prompt, idle=idle)


def _read(B, longest, hkv=8, d=128, act="bf16", page=64):
    return dict(op="read", B=B, longest=longest, cache="fp4", hkv=hkv, d=d, act=act, page=page)


def listed():
    return [
        # one short prompt of an odd length
        dict(_prompt(1, 37, 0, "bf16"), name="prompt_bf16_t37"),
        # one ordinary prompt, full attention
        dict(_prompt(1, 2048, 0, "bf16"), name="prompt_bf16_t2048"),
        # one long prompt, full attention
        dict(_prompt(1, 16384, 0, "bf16"), name="prompt_bf16_t16384"),
        # a batch of prompts behind cached prefixes in a sliding-window layer with sinks, 8-bit cache
        dict(_prompt(4, 4096, 8191, "fp8", window=512, sinks=4), name="prompt_window_fp8_b4"),
        # a step that mixes chunks of prompts with single tokens, 4-bit cache, some rows of padding
        dict(_prompt(12, 1000, 4000, "fp4", singles=8, pad=13), name="prompt_mixed_fp4_b12"),
        # eight drafted tokens of four requests verified against long contexts
        dict(_prompt(4, 8, 32768, "bf16", even=True), name="prompt_verify_bf16_b4"),
        # decode of 64 slots (4 idle) in a sliding-window layer with sinks
        dict(_decode(64, 4095, "bf16", window=512, sinks=4, idle=4), name="decode_sinks_bf16_b64"),
        # a small decode batch in a sliding-window layer with sinks, 4-bit cache
        dict(_decode(8, 2048, "fp4", window=512, sinks=64), name="decode_sinks_fp4_b8"),
        # a full serving batch of very different lengths over a 4-bit cache
        dict(_decode(64, 32768, "fp4"), name="decode_ragged_fp4_b64"),
        # one decode step's keys and values stored in 4 bits, and read back
        dict(_append(64, prompt=False, idle=3, page=16), name="append_fp4_t64"),
        # a long prompt's keys and values stored in 4 bits, and read back
        dict(_append(16384), name="append_fp4_t16384"),
        # many 4-bit prefixes read back
        dict(_read(32, 8191), name="read_fp4_b32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv = rng.choice([(48, 8), (48, 8), (32, 8), (8, 8), (16, 1), (40, 4), (64, 2)])
    d = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    act = rng.choice(["bf16", "bf16", "f32"])
    op = rng.choice(["prompt", "prompt", "prompt", "decode", "decode", "append", "read"])
    if op == "append":
        T = _log(rng, 1, max(1, min(16384, 16384 * 8 * 128 * 2 // (hkv * d * BYTES[act]))))
        return _append(T, hkv=hkv, d=d, act=act, page=page, prompt=T > 300,
                       idle=0 if T > 300 or T < 8 else rng.randrange(T // 4))
    if op == "read":
        B = _log(rng, 1, 64)
        longest = _log(rng, 1, max(1, 32 * 8191 * 8 * 128 * 2 // (B * hkv * d * BYTES[act])))
        return _read(B, min(longest, 65536), hkv=hkv, d=d, act=act, page=page)
    window = rng.choice([0, 0, 128, 512, 1000])
    if op == "decode":
        cache = rng.choice(["fp4", "fp4", "fp8", "bf16", "f32"])
        if cache != "fp4":
            window = window or 512
        sinks = rng.choice([1, 4, 64, 200]) if window else 0
        B = _log(rng, 1, 256)
        longest = min(131072, max(1, 64 * 32768 * 8 * 64 // (B * hkv * d * (1 if cache == "fp4" else 4))))
        return _decode(B, _log(rng, 1, longest), cache, hq=hq, hkv=hkv, d=d, window=window, sinks=sinks, page=page,
                       idle=0 if B < 8 else rng.randrange(B // 4))
    cache = rng.choice(["bf16", "bf16", "fp8", "fp4", "f32"])
    sinks = rng.choice([0, 1, 4, 64, 200]) if window else 0
    B = _log(rng, 1, 16)
    most = MOST_SCORES // (B * hq) * 128 // d // (16 if cache == "f32" else 1)   # new tokens times length
    new = _log(rng, 1, min(8192, math.isqrt(most)))
    prefix = rng.choice([0, _log(rng, 1, max(1, min(32768, most // new - new)))])
    singles = rng.randrange(B) if B > 1 and rng.random() < 0.4 else 0
    return _prompt(B, new, prefix, cache, hq=hq, hkv=hkv, d=d, window=window, sinks=sinks, page=page, singles=singles,
                   even=rng.random() < 0.3, pad=rng.choice([0, 0, 5]))


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """New and cached tokens (the new ones among them) of each sequence."""
    B = case["B"]
    if case["op"] == "prompt":
        s = case["singles"]
        step = [1.0 if case["even"] else ((i + 1) / (B - s)) ** 2 for i in range(B - s)]
        new = [1] * s + [max(1, round(case["new"] * x)) for x in step]
        # the longest prefixes with the shortest chunks
        return new, [n + round(case["prefix"] * ((B - i) / B) ** 2) for i, n in enumerate(new)]
    idle = case.get("idle", 0)
    n = B - idle
    lens = [max(1, round(case["longest"] * ((i + 1) / n) ** 2)) for i in range(n)] + [0] * idle
    return [min(x, 1) for x in lens], lens


def _mx_codes(x):
    """E2M1 codes (two a byte) and E8M0 scale bytes of fp32 rows [..., d]: a block's exponent is that of its
    largest magnitude less 2, a code the nearest value, ties to even."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127)
    y = torch.ldexp(b.abs(), -e[..., None]).clamp(max=6.0)
    c = torch.where(y < 2, torch.round(2 * y), torch.where(y < 4, torch.round(y) + 2, torch.round(y / 2) + 4))
    c = c.to(torch.uint8) | (torch.signbit(b).to(torch.uint8) << 3)
    c = c.flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _mx_values(codes, scale):
    """fp32 rows that codes and scale bytes stand for."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = grid[c.int()].unflatten(-1, (-1, 32))
    return torch.ldexp(v, scale.int()[..., None] - 127).flatten(-2)


def _fp8_codes(x):
    s = x.abs().amax(-1) / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (x / s[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s


def _filled(kind, n_pages, hkv, page, d, g):
    """One side (keys or values) of a cache with something in every place, and its scales."""
    shape = (n_pages, hkv, page, d)
    if kind in ACT:
        return torch.randn(shape, generator=g, device=DEV, dtype=ACT[kind]), None
    if kind == "fp8":
        return _fp8_codes(torch.randn(shape, generator=g, device=DEV))
    return _mx_codes(torch.randn(shape, generator=g, device=DEV))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 6271 + 29)
    op, hkv, d, page, kind = case["op"], case["hkv"], case["d"], case["page"], case["cache"]
    act = ACT[case.get("act", "f32" if kind == "f32" else "bf16")]
    s = {"case": case}
    if op == "append":
        T = case["T"]
        kv = torch.randn((T, 2 * hkv * d), generator=g, device=DEV).to(act)      # columns of a merged projection
        s["k"], s["v"] = kv[:, :hkv * d].view(T, hkv, d), kv[:, hkv * d:].view(T, hkv, d)
        n_pages = -(-(T + T // 8 + 1) // page)
        pages = torch.randperm(n_pages, generator=g, device=DEV)
        if case["prompt"]:
            i = torch.arange(T, device=DEV)
            slots = pages[i // page] * page + i % page
            s["page_table"] = pages[None, :].to(torch.int32)
            s["row_offsets"] = torch.tensor([0, T], dtype=torch.int32, device=DEV)
            s["first"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        else:
            # one token of each request; idle requests have no slot, and their rows read back as zeros
            slots = torch.randperm(n_pages * page, generator=g, device=DEV)[:T]
            slots[torch.randperm(T, generator=g, device=DEV)[:case["idle"]]] = -1
            s["page_table"] = torch.where(slots >= 0, slots // page, -1)[:, None].to(torch.int32)
            s["row_offsets"] = torch.arange(T + 1, device=DEV, dtype=torch.int32)
            s["first"] = torch.where(slots >= 0, slots % page, 0).to(torch.int32)
        s["slots"] = slots.to(torch.int32)
        s["rows"] = torch.nonzero(slots >= 0)[:, 0]
        s["k_out"] = torch.empty((T, hkv, d), dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.empty((T, hkv, d), dtype=torch.bfloat16, device=DEV)
    else:
        B = case["B"]
        new, lens = (torch.tensor(x, device=DEV) for x in _lengths(case))
        order = torch.randperm(B, generator=g, device=DEV)
        new, lens = new[order], lens[order]
        longest = max(_lengths(case)[1])
        used = (lens + page - 1) // page
        n_pages = int(used.sum()) + 3
        width = -(-longest // page)
        at = (used.cumsum(0) - used)[:, None] + torch.arange(width, device=DEV)[None, :]
        pages = torch.randperm(n_pages, generator=g, device=DEV)
        own_page = torch.arange(width, device=DEV)[None, :] < used[:, None]
        s["page_table"] = torch.where(own_page, pages[at.clamp(max=n_pages - 1)], -1).to(torch.int32)
        s["lens"] = lens.to(torch.int32)
        off = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    if op == "read":
        off[1:] = lens.cumsum(0)
        s["row_offsets"], n = off, sum(_lengths(case)[1])
        s["k_out"] = torch.empty((n, hkv, d), dtype=act, device=DEV)
        s["v_out"] = torch.empty((n, hkv, d), dtype=act, device=DEV)
    if op in ("prompt", "decode"):
        if op == "prompt":
            off[1:] = new.cumsum(0)
            s["q_offsets"] = off
        T, hq = B if op == "decode" else sum(_lengths(case)[0]) + case["pad"], case["hq"]
        s["q"] = (2.0 * torch.randn((T, hq, d), generator=g, device=DEV)).to(act)
        s["out"] = torch.zeros((T, hq, d), dtype=act, device=DEV)
        s["lse"] = torch.zeros((T, hq), dtype=torch.float32, device=DEV)
    s["ck"], s["ks"] = _filled(kind, n_pages, hkv, page, d, g)
    s["cv"], s["vs"] = _filled(kind, n_pages, hkv, page, d, g)
    if own:
        # the plan and handles that a serving program keeps
        import expert_routed_ffn_amd as beam
        s["cfg"] = beam.AttnCfg(n_heads=case.get("hq", hkv), n_kv_heads=hkv, head_dim=d, rope_dim=0,
                                window=case.get("window", 0), page_size=page, softmax_scale=d ** -0.5,
                                sinks=case.get("sinks", 0))
        s["cache"] = beam.KVCache(s["ck"], s["cv"], s["ks"], s["vs"])
        if op == "decode":
            s["ws"] = beam.attn_workspace(s["cfg"], B, longest)
        if op == "prompt":
            s["ws"] = beam.attn_prompt_workspace(s["cfg"], B, T, longest)
    return s


# ------------------------------------------------------------------ plain forms

def _rows(s, codes, scale, page, off):
    """fp32 [..., hkv, d] rows of one side of the cache."""
    kind = s["case"]["cache"]
    at = page[..., None], torch.arange(s["case"]["hkv"], device=DEV), off[..., None]
    if kind == "fp4":
        return _mx_values(codes[at], scale[at])
    if kind == "fp8":
        return codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scale[at][..., None]
    return codes[at].float()


def _attend(q, k, v, seen, scale):
    """q [B, hkv, n, d] over k, v [B, hkv, L, d], seen [B, n or 1, L] broadcast over the heads of n = G * rows:
    (out, lse); a row that sees nothing gives 0 and -inf."""
    B, hkv, n, d = q.shape
    z = torch.matmul(q, k.transpose(2, 3).contiguous())
    z = z.view(B, hkv, -1, seen.shape[1], seen.shape[2])         # [B, hkv, G, rows, L]
    z.mul_(scale).masked_fill_(~seen[:, None, None], float("-inf"))
    m = z.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    z.sub_(m).exp_()
    total = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(B, hkv, n, -1), v).view(B, hkv, -1, seen.shape[1], d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    return o, (m + total.log())[..., 0]


def _plain_prompt(s):
    case = s["case"]
    B, hq, hkv, d, page = case["B"], case["hq"], case["hkv"], case["d"], case["page"]
    off, lens = s["q_offsets"].long(), s["lens"].long()
    new, length = _lengths(case)
    n, L, total = max(new), max(length), sum(new)
    t = torch.arange(L, device=DEV)
    pages = s["page_table"].long()[:, t // page].clamp(min=0)
    at = (t % page).expand(B, L)
    k = _rows(s, s["ck"], s["ks"], pages, at).transpose(1, 2).contiguous()
    v = _rows(s, s["cv"], s["vs"], pages, at).transpose(1, 2).contiguous()
    # the queries of each sequence padded to the most there are
    i = torch.arange(n, device=DEV)
    count = off[1:] - off[:-1]
    q = s["q"].float()[(off[:-1, None] + i).clamp(max=total - 1)]                    # [B, n, hq, d]
    q = q.view(B, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, d)
    pos = (lens - count)[:, None] + i                                                 # [B, n]
    seen = t <= pos[:, :, None]
    if case["window"]:
        seen &= (t > pos[:, :, None] - case["window"]) | (t < case["sinks"])
    o, lse = _attend(q, k, v, seen, d ** -0.5)
    live = i < count[:, None]
    s["out"][:total] = o.permute(0, 3, 1, 2, 4).reshape(B, n, hq, d)[live].to(s["out"].dtype)
    s["lse"][:total] = lse.permute(0, 3, 1, 2).reshape(B, n, hq)[live]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_decode(s):
    case = s["case"]
    B, hq, hkv, d, page = case["B"], case["hq"], case["hkv"], case["d"], case["page"]
    lens = s["lens"].long()
    span = min(case["window"] or case["longest"], case["longest"])
    start = (lens - span).clamp(min=0)[:, None]
    t = start + torch.arange(span, device=DEV)
    live = t < lens[:, None]
    first = torch.arange(min(case["sinks"], case["longest"]), device=DEV).expand(B, -1)
    t, live = torch.cat([first, t], 1), torch.cat([first < start, live], 1)           # each token once
    t = t.clamp(max=case["longest"] - 1)
    pages = s["page_table"].long().gather(1, t // page).clamp(min=0)
    k = _rows(s, s["ck"], s["ks"], pages, t % page).transpose(1, 2).contiguous()
    v = _rows(s, s["cv"], s["vs"], pages, t % page).transpose(1, 2).contiguous()
    o, lse = _attend(s["q"].float().view(B, hkv, hq // hkv, d), k, v, live[:, None], d ** -0.5)
    return {"out": o.reshape(B, hq, d).to(s["q"].dtype), "lse": lse.reshape(B, hq)}


def _plain_read(s):
    page = s["case"]["page"]
    off = s["row_offsets"].long()
    i = torch.arange(s["k_out"].shape[0], device=DEV)
    b = torch.searchsorted(off, i, right=True) - 1
    t = i - off[b] + (s["first"].long()[b] if "first" in s else 0)
    p = s["page_table"].long()[b, t // page]
    there = (p >= 0)[:, None, None]
    for out, codes, scale in ((s["k_out"], s["ck"], s["ks"]), (s["v_out"], s["cv"], s["vs"])):
        out.copy_(torch.where(there, _rows(s, codes, scale, p.clamp(min=0), t % page), 0.0))
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_append(s):
    case, rows = s["case"], s["rows"]
    slots = s["slots"][rows].long()
    at = (slots // case["page"])[:, None], torch.arange(case["hkv"], device=DEV), (slots % case["page"])[:, None]
    s["ck"][at], s["ks"][at] = _mx_codes(s["k"][rows].float())
    s["cv"][at], s["vs"][at] = _mx_codes(s["v"][rows].float())
    return _plain_read(s)


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import expert_routed_ffn_amd as beam
        cfg = s["cfg"]
        if op == "prompt":
            beam.beam_moe_attn_prompt(cfg, s["q"], s["cache"], s["page_table"], s["q_offsets"], s["lens"],
                                      s["page_table"].shape[1] * cfg.page_size, s["out"], s["ws"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "decode":
            beam.beam_moe_attn_decode(cfg, s["q"], s["cache"], s["page_table"], s["lens"], s["case"]["longest"],
                                      s["out"], s["ws"], lse=s["lse"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "append":
            beam.beam_moe_kv_write(cfg, s["k"], s["v"], s["slots"], s["cache"])
        beam.beam_moe_kv_read(cfg, s["cache"], s["page_table"], s["row_offsets"], s["k_out"], s["v_out"],
                              first=s.get("first"))
        return {"k": s["k_out"], "v": s["v_out"]}
    return {"prompt": _plain_prompt, "decode": _plain_decode, "append": _plain_append, "read": _plain_read}[op](s)


# ------------------------------------------------------------------ work and exact values

def _row_bytes(case):
    d = case["d"]
    return {"fp4": d // 2 + d // 32, "fp8": d + 4, "bf16": 2 * d, "f32": 4 * d}[case["cache"]]


def _up_to(n):
    """1 + 2 + ... + n"""
    return n * (n + 1) // 2 if n > 0 else 0


def _seen(n, length, window, sinks):
    """(query, token) pairs of n new tokens at the end of `length`, and the tokens that any of them sees."""
    if not window:
        return _up_to(length) - _up_to(length - n), length
    p0 = length - n
    in_window = _up_to(min(length, window)) - _up_to(min(p0, window)) + window * (max(length, window) - max(p0, window))
    # sinks behind the window: min(sinks, p + 1 - window) for positions p0 .. length - 1
    def behind(x):
        x -= window
        return _up_to(min(x, sinks)) + sinks * max(0, x - sinks)
    start = max(0, p0 + 1 - window)
    return in_window + behind(length) - behind(p0), length - start + min(sinks, start)


def work(case):
    hkv, d, row, op = case["hkv"], case["d"], _row_bytes(case), case["op"]
    hq = case.get("hq", 0)
    ea = BYTES[case.get("act", "f32" if case["cache"] == "f32" else "bf16")]
    if op == "append":
        live = case["T"] - case["idle"]
        n = 2 * hkv * d
        return {"bytes": live * (n * ea + 2 * 2 * hkv * row) + case["T"] * (2 * n + 12), "flops": 5 * live * n}
    new, lens = _lengths(case)
    if op == "read":
        n = 2 * sum(lens) * hkv
        return {"bytes": n * (row + d * ea) + 4 * sum(-(-x // case["page"]) for x in lens), "flops": n * d}
    seen = [_seen(n, x, case["window"], case["sinks"]) for n, x in zip(new, lens) if n]
    pairs, tokens = sum(a for a, b in seen), sum(b for a, b in seen)
    return {"bytes": 2 * tokens * hkv * row + 2 * sum(new) * hq * d * ea + 4 * sum(new) * hq + 4 * tokens // case["page"],
            "flops": 4 * pairs * hq * d}


def exact(case, seed):
    s = prepare(case, seed)
    op, page, hkv, d, kind = case["op"], case["page"], case["hkv"], case["d"], case["cache"]
    grid = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    grid = torch.tensor(grid + [-x for x in grid], dtype=torch.float64, device=DEV)

    def nearest(x):
        """fp64 values of 4-bit blocks, by distance to every one of the eight magnitudes."""
        x = x.double().unflatten(-1, (-1, 32))
        top = x.abs().max(-1, keepdim=True).values
        step = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top)) - 2), torch.ones_like(top))
        y = (x / step).abs().clamp(max=6.0)
        order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=DEV)        # even codes win ties
        code = order[(y[..., None] - grid[order]).abs().argmin(-1)]
        return (torch.copysign(grid[code], x) * step).flatten(-2)

    def rows(codes, scale, b, tokens):
        """fp64 [h, n, d]: the given tokens of sequence b."""
        p = s["page_table"][b].long()[tokens // page]
        x = codes[p, :, tokens % page]
        if kind == "fp8":
            x = x.double() * scale[p, :, tokens % page].double()[..., None]
        elif kind == "fp4":
            c = torch.stack([x.int() % 16, x.int() // 16], -1).flatten(-2)
            f = torch.exp2(scale[p, :, tokens % page].double() - 127)
            x = grid[c] * f.repeat_interleave(32, -1)
        return x.double().transpose(0, 1).contiguous()

    if op == "append":
        if case["T"] * hkv * d > 1 << 24:      # 64 bytes of distances an element
            return None
        live = (s["slots"] >= 0)[:, None, None]
        return {"k": torch.where(live, nearest(s["k"]), 0.0), "v": torch.where(live, nearest(s["v"]), 0.0)}
    lens = s["lens"].tolist()
    if op == "read":
        every = [torch.arange(n, device=DEV) for n in lens]
        return {"k": torch.cat([rows(s["ck"], s["ks"], b, t).transpose(0, 1) for b, t in enumerate(every)]),
                "v": torch.cat([rows(s["cv"], s["vs"], b, t).transpose(0, 1) for b, t in enumerate(every)])}
    hq = case["hq"]
    G = hq // hkv
    new = (s["q_offsets"][1:] - s["q_offsets"][:-1]).tolist() if op == "prompt" else [min(x, 1) for x in lens]
    first = s["q_offsets"].tolist() if op == "prompt" else list(range(case["B"]))
    if sum(n * x for n, x in zip(new, lens)) * hq * d > 1 << 41:
        return None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, -math.inf if op == "decode" else 0.0, dtype=torch.float64, device=DEV)
    for b, (n, length) in enumerate(zip(new, lens)):
        # a few hundred queries at a time, over what they can see
        for i in range(0, n, 512):
            p = torch.arange(length - n + i, length - n + min(i + 512, n), device=DEV)
            lo = max(0, int(p[0]) + 1 - case["window"]) if case["window"] else 0
            tokens = torch.cat([torch.arange(min(case["sinks"], lo), device=DEV),
                                torch.arange(lo, int(p[-1]) + 1, device=DEV)])
            mask = tokens[None, :] <= p[:, None]
            if case["window"]:
                mask &= (p[:, None] - tokens[None, :] < case["window"]) | (tokens[None, :] < case["sinks"])
            k, v = rows(s["ck"], s["ks"], b, tokens), rows(s["cv"], s["vs"], b, tokens)
            at = slice(first[b] + i, first[b] + i + len(p))
            q = s["q"][at].double().view(len(p), hkv, G, d)
            for h in range(hkv):
                z = q[:, h].reshape(-1, d) @ k[h].T.contiguous() / math.sqrt(d)
                z = z.view(len(p), G, -1).masked_fill(~mask[:, None, :], -math.inf)
                lse[at, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                out[at, h * G:(h + 1) * G] = (torch.softmax(z, -1).view(len(p) * G, -1) @ v[h]).view(len(p), G, d)
    return {"out": out, "lse": lse}
