"""Cases of the attention sublayer's operators: per-head query/key norms with
the position rotation, the paged key-value cache (written, quantised, read
back) and the attention of one new token over it.

`run` computes a case in plain torch operations, or through the library's
entry points where `own` is true.  Shapes are the Beam attention's (48 query
and 8 key-value heads of 128, sliding windows of 512) or generic ones.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
ACT = {"bf16": torch.bfloat16, "f32": torch.float32}
CACHE = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "fp8": 1}


# ------------------------------------------------------------------ cases

def _rope(T, hq=48, hkv=8, d=128, r=128, act="bf16", inter=False, ssmax=0.0, prompt=True, far=0):
    return dict(op="rope", T=T, hq=hq, hkv=hkv, d=d, r=r, act=act, inter=inter, ssmax=ssmax, prompt=prompt, far=far)


def _rope_cache(T, cache, hq=48, hkv=8, d=128, r=128, act="bf16", inter=False, ssmax=0.0, page=64, prompt=True,
                far=0, idle=0):
    return dict(op="rope_cache", T=T, cache=cache, hq=hq, hkv=hkv, d=d, r=r, act=act, inter=inter, ssmax=ssmax,
                page=page, prompt=prompt, far=far, idle=idle)


def _write(T, cache, hkv=8, d=128, act="bf16", page=64, prompt=True, idle=0):
    return dict(op="write", T=T, cache=cache, hkv=hkv, d=d, act=act, page=page, prompt=prompt, idle=idle)


def _read(B, longest, cache, hkv=8, d=128, act="bf16", page=64):
    return dict(op="read", B=B, longest=longest, cache=cache, hkv=hkv, d=d, act=act, page=page)


def _decode(B, longest, cache, hq=48, hkv=8, d=128, window=0, page=64, idle=0):
    return dict(op="decode", B=B, longest=longest, cache=cache, hq=hq, hkv=hkv, d=d, window=window, page=page,
                idle=idle)


def listed():
    return [
        # one decode step of 8 requests, a rotary layer
        dict(_rope(8, prompt=False, far=32768), name="norm_rope_t8"),
        # a prefill chunk in fp32, a partial interleaved rotation, odd token count
        dict(_rope(2047, hq=16, hkv=4, d=64, r=32, act="f32", inter=True, far=1000000), name="norm_rope_f32_t2047"),
        # one decode step of 64 slots (5 idle) of a layer without rotation, queries scaled by position
        dict(_rope_cache(64, "fp8", r=0, ssmax=2048.0, prompt=False, far=100000, idle=5), name="norm_cache_fp8_t64"),
        # a large prefill chunk of a rotary layer into an 8-bit cache
        dict(_rope_cache(16384, "fp8", far=16384), name="norm_cache_fp8_t16384"),
        # keys and values that arrive ready, one decode step
        dict(_write(64, "bf16", prompt=False, idle=3, page=16), name="write_bf16_t64"),
        # a prompt's keys and values quantised into the cache
        dict(_write(16384, "fp8"), name="write_fp8_t16384"),
        # a few cached prefixes read back for a chunked prefill
        dict(_read(5, 997, "bf16", page=16), name="read_bf16_b5"),
        # many 8-bit prefixes read back
        dict(_read(32, 8191, "fp8"), name="read_fp8_b32"),
        # decode of 8 requests, full attention over short contexts
        dict(_decode(8, 2048, "bf16"), name="decode_bf16_b8"),
        # decode of 64 slots (4 idle) in a sliding-window layer
        dict(_decode(64, 4095, "fp8", window=512, idle=4), name="decode_window_fp8_b64"),
        # one request with a very long context
        dict(_decode(1, 131071, "bf16"), name="decode_long_bf16_b1"),
        # a full serving batch of very different lengths over an 8-bit cache
        dict(_decode(64, 32768, "fp8"), name="decode_ragged_fp8_b64"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv = rng.choice([(48, 8), (48, 8), (32, 8), (8, 8), (16, 1), (40, 4), (64, 2)])
    d = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    act = rng.choice(["bf16", "bf16", "f32"])
    cache = rng.choice(["fp8", act])
    op = rng.choice(["rope", "rope_cache", "write", "read", "decode", "decode"])
    most = 16384 * 64 * 128 * 2 // ((hq + 2 * hkv) * d * BYTES[act])   # tokens of the largest listed prefill chunk
    if op in ("rope", "rope_cache"):
        r = rng.choice([0, 32, d // 2, d, d])
        c = dict(hq=hq, hkv=hkv, d=d, r=r, act=act, inter=rng.random() < 0.3,
                 ssmax=rng.choice([2048.0, 4096.0]) if r == 0 else 0.0, far=_log(rng, 4096, 1000000))
        T = _log(rng, 1, min(16384, most))
        if op == "rope":
            return _rope(T, prompt=T > 300, **c)
        return _rope_cache(T, cache, page=page, prompt=T > 300, idle=0 if T > 300 or T < 8 else rng.randrange(T // 4),
                           **c)
    if op == "write":
        T = _log(rng, 1, min(16384, most))
        return _write(T, cache, hkv=hkv, d=d, act=act, page=page, prompt=T > 300,
                      idle=0 if T > 300 or T < 8 else rng.randrange(T // 4))
    if op == "read":
        B = _log(rng, 1, 64)
        longest = _log(rng, 1, max(1, 32 * 8191 * 8 * 128 * 2 // (B * hkv * d * BYTES[act])))
        return _read(B, min(longest, 65536), cache, hkv=hkv, d=d, act=act, page=page)
    cache = rng.choice(["fp8", "bf16", "bf16", "f32"])
    B = _log(rng, 1, 256)
    longest = min(131072, max(1, 64 * 32768 * 8 * 128 // (B * hkv * d * BYTES[cache])))
    return _decode(B, _log(rng, 1, longest), cache, hq=hq, hkv=hkv, d=d,
                   window=rng.choice([0, 0, 128, 512, 1000]), page=page, idle=0 if B < 8 else rng.randrange(B // 4))


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """Cached tokens of each sequence, idle ones last: squares of even steps up to the longest."""
    B, idle = case["B"], case.get("idle", 0)
    n = B - idle
    return [max(1, round(case["longest"] * ((i + 1) / n) ** 2)) for i in range(n)] + [0] * idle


def _quantised(x):
    s = x.abs().amax(-1) / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (x / s[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s


def _filled(kind, n_pages, hkv, page, d, g):
    """One side (keys or values) of a cache with something in every place, and its scales."""
    if kind != "fp8":
        return torch.randn((n_pages, hkv, page, d), generator=g, device=DEV).to(CACHE[kind]), None
    codes = torch.empty((n_pages, hkv, page, d), dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty((n_pages, hkv, page), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 27) // (hkv * page * d))
    for i in range(0, n_pages, step):
        x = torch.randn((min(step, n_pages - i), hkv, page, d), generator=g, device=DEV)
        codes[i:i + step], scale[i:i + step] = _quantised(x)
    return codes, scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 11)
    op, hkv, d, page = case["op"], case["hkv"], case["d"], case.get("page", 64)
    act = ACT[case.get("act", "f32" if case.get("cache") == "f32" else "bf16")]
    s = {"case": case}

    def rows(n, h):
        return torch.randn((n, h, d), generator=g, device=DEV)

    if op in ("rope", "rope_cache", "write"):
        T = case["T"]
        hq = case.get("hq", 0)
        # the rows of a merged projection: queries, keys and values side by side
        qkv = torch.randn((T, (hq + 2 * hkv) * d), generator=g, device=DEV).to(act)
        s["q"] = qkv[:, :hq * d].view(T, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
    if op in ("rope", "rope_cache"):
        far, r = case["far"], case["r"]
        if case["prompt"]:
            first = int(torch.randint(0, max(1, far - T + 1), (1,), generator=g, device=DEV))
            s["positions"] = torch.arange(first, first + T, device=DEV, dtype=torch.int32)
        else:
            s["positions"] = torch.randint(0, far, (T,), generator=g, device=DEV, dtype=torch.int32)
        s["gamma_q"] = (1.5 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(act)
        s["gamma_k"] = (1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(act)
        s["inv_freq"] = None
        if r:
            s["inv_freq"] = (10000.0 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)).float()
        s["q_out"] = torch.empty((T, hq, d), dtype=act, device=DEV)
        s["k_out"] = torch.empty((T, hkv, d), dtype=act, device=DEV)
    if op in ("rope_cache", "write"):
        n_pages = -(-(T + T // 8 + 1) // page)
        pages = torch.randperm(n_pages, generator=g, device=DEV)
        if case["prompt"]:
            i = torch.arange(T, device=DEV)
            slots = pages[i // page] * page + i % page
        else:
            slots = torch.randperm(n_pages * page, generator=g, device=DEV)[:T]
        idle = torch.randperm(T, generator=g, device=DEV)[:case["idle"]]
        slots[idle] = -1                      # rows of idle requests are not cached
        s["slots"] = slots.to(torch.int32)
        s["rows"] = torch.nonzero(slots >= 0)[:, 0]
    if op in ("read", "decode"):
        lens = torch.tensor(_lengths(case), device=DEV)
        lens = lens[torch.randperm(case["B"], generator=g, device=DEV)]
        used = (lens + page - 1) // page
        n_pages = int(used.sum()) + 3
        width = -(-case["longest"] // page)
        at = (used.cumsum(0) - used)[:, None] + torch.arange(width, device=DEV)[None, :]
        pages = torch.randperm(n_pages, generator=g, device=DEV)
        own_page = torch.arange(width, device=DEV)[None, :] < used[:, None]
        s["page_table"] = torch.where(own_page, pages[at.clamp(max=n_pages - 1)], -1).to(torch.int32)
        s["lens"] = lens.to(torch.int32)
    if op == "read":
        off = torch.zeros(case["B"] + 1, dtype=torch.int32, device=DEV)
        off[1:] = lens.cumsum(0)
        s["row_offsets"] = off
        n = sum(_lengths(case))
        s["k_out"] = torch.empty((n, hkv, d), dtype=act, device=DEV)
        s["v_out"] = torch.empty((n, hkv, d), dtype=act, device=DEV)
    if op == "decode":
        B, hq = case["B"], case["hq"]
        s["q"] = (2.0 * rows(B, hq)).to(act)
        s["out"] = torch.empty((B, hq, d), dtype=act, device=DEV)
        s["lse"] = torch.empty((B, hq), dtype=torch.float32, device=DEV)
    if op != "rope":
        s["ck"], s["ks"] = _filled(case["cache"], n_pages, hkv, page, d, g)
        s["cv"], s["vs"] = _filled(case["cache"], n_pages, hkv, page, d, g)
    if own:
        # the plan and handles that a serving program keeps
        import expert_routed_ffn_amd as beam
        s["cfg"] = beam.AttnCfg(n_heads=case.get("hq", hkv), n_kv_heads=hkv, head_dim=d, rope_dim=case.get("r", 0),
                                rope_interleaved=case.get("inter", False), ssmax_len=case.get("ssmax", 0.0),
                                ssmax_exp=0.1, window=case.get("window", 0), page_size=page,
                                softmax_scale=d ** -0.5, rms_eps=EPS)
        if op != "rope":
            s["cache"] = beam.KVCache(s["ck"], s["cv"], s["ks"], s["vs"])
        if op == "decode":
            s["ws"] = beam.attn_workspace(s["cfg"], case["B"], case["longest"])
    return s


# ------------------------------------------------------------------ plain forms

def _norm_rotated(s, x, gamma, scaled):
    case = s["case"]
    r, x = case["r"], x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.float()
    if r:
        a = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
        cos, sin = a.cos().float()[:, None, :], a.sin().float()[:, None, :]
        turned = torch.empty_like(x[..., :r])
        if case["inter"]:
            u, w = x[..., 0:r:2], x[..., 1:r:2]
            turned[..., 0::2] = u * cos - w * sin
            turned[..., 1::2] = w * cos + u * sin
        else:
            u, w = x[..., :r // 2], x[..., r // 2:r]
            turned[..., :r // 2] = u * cos - w * sin
            turned[..., r // 2:] = w * cos + u * sin
        x = torch.cat([turned, x[..., r:]], -1)
    if scaled and case["ssmax"]:
        f = (1.0 + s["positions"].clamp(min=0).float() / case["ssmax"]) ** 0.1
        x = x * f[:, None, None]
    return x


def _put(s, k, v):
    case = s["case"]
    rows = s["rows"]
    slots = s["slots"][rows].long()
    at = (slots // case["page"])[:, None], torch.arange(case["hkv"], device=DEV)[None, :], (slots % case["page"])[:, None]
    for x, codes, scale in ((k, s["ck"], s["ks"]), (v, s["cv"], s["vs"])):
        x = x[rows].float()
        if case["cache"] == "fp8":
            x, scale[at] = _quantised(x)
            codes.view(torch.uint8)[at] = x.view(torch.uint8)
        else:
            codes[at] = x.to(codes.dtype)


def _got(s, codes, scale, page, off):
    """float [..., hkv, d] rows of one side of the cache."""
    h = torch.arange(s["case"]["hkv"], device=DEV)
    at = page[..., None], h, off[..., None]
    if scale is None:
        return codes[at].float()
    return codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scale[at][..., None]


def _plain_read(s):
    case = s["case"]
    off = s["row_offsets"].long()
    i = torch.arange(s["k_out"].shape[0], device=DEV)
    b = torch.searchsorted(off, i, right=True) - 1
    t = i - off[b]
    page = s["page_table"].long()[b, t // case["page"]]
    s["k_out"].copy_(_got(s, s["ck"], s["ks"], page, t % case["page"]))
    s["v_out"].copy_(_got(s, s["cv"], s["vs"], page, t % case["page"]))
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_decode(s):
    case = s["case"]
    B, hq, hkv, d, page = case["B"], case["hq"], case["hkv"], case["d"], case["page"]
    lens = s["lens"].long()
    span = min(case["window"] or case["longest"], case["longest"])
    t = (lens - span).clamp(min=0)[:, None] + torch.arange(span, device=DEV)[None, :]
    live = t < lens[:, None]
    t = t.clamp(max=case["longest"] - 1)
    pages = s["page_table"].long().gather(1, t // page).clamp(min=0)
    k = _got(s, s["ck"], s["ks"], pages, t % page).transpose(1, 2).contiguous()      # [B, hkv, span, d]
    q = s["q"].float().view(B, hkv, hq // hkv, d).transpose(2, 3).contiguous()
    z = torch.matmul(k, q) * d ** -0.5                                               # [B, hkv, span, G]
    del k
    z = z.masked_fill(~live[:, None, :, None], float("-inf"))
    m = z.amax(2, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(z - m)
    total = p.sum(2, keepdim=True)
    v = _got(s, s["cv"], s["vs"], pages, t % page).transpose(1, 2).contiguous()
    o = torch.matmul(p.transpose(2, 3).contiguous(), v)                              # [B, hkv, G, d]
    o = o / torch.where(total > 0, total, torch.ones_like(total)).transpose(2, 3)
    return {"out": o.reshape(B, hq, d).to(s["q"].dtype), "lse": (m + total.log()).reshape(B, hq)}


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        import expert_routed_ffn_amd as beam
        cfg = s["cfg"]
        if op == "rope":
            beam.beam_moe_qk_norm_rope(cfg, s["q"], s["k"], s["positions"], s["q_out"], s["k_out"],
                                       inv_freq=s["inv_freq"], gamma_q=s["gamma_q"], gamma_k=s["gamma_k"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if op == "rope_cache":
            beam.beam_moe_qk_norm_rope_cache(cfg, s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_out"],
                                             s["cache"], inv_freq=s["inv_freq"], gamma_q=s["gamma_q"],
                                             gamma_k=s["gamma_k"])
            return {"q": s["q_out"], "ck": s["ck"], "cv": s["cv"], "ks": s["ks"], "vs": s["vs"]}
        if op == "write":
            beam.beam_moe_kv_write(cfg, s["k"], s["v"], s["slots"], s["cache"])
            return {"ck": s["ck"], "cv": s["cv"], "ks": s["ks"], "vs": s["vs"]}
        if op == "read":
            beam.beam_moe_kv_read(cfg, s["cache"], s["page_table"], s["row_offsets"], s["k_out"], s["v_out"])
            return {"k": s["k_out"], "v": s["v_out"]}
        beam.beam_moe_attn_decode(cfg, s["q"], s["cache"], s["page_table"], s["lens"], s["case"]["longest"],
                                  s["out"], s["ws"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "rope":
        s["q_out"].copy_(_norm_rotated(s, s["q"], s["gamma_q"], True))
        s["k_out"].copy_(_norm_rotated(s, s["k"], s["gamma_k"], False))
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "rope_cache":
        s["q_out"].copy_(_norm_rotated(s, s["q"], s["gamma_q"], True))
        _put(s, _norm_rotated(s, s["k"], s["gamma_k"], False), s["v"])
        return {"q": s["q_out"], "ck": s["ck"], "cv": s["cv"], "ks": s["ks"], "vs": s["vs"]}
    if op == "write":
        _put(s, s["k"], s["v"])
        return {"ck": s["ck"], "cv": s["cv"], "ks": s["ks"], "vs": s["vs"]}
    if op == "read":
        return _plain_read(s)
    return _plain_decode(s)


# ------------------------------------------------------------------ work and exact values

def work(case):
    hkv, d = case["hkv"], case["d"]
    hq, op = case.get("hq", 0), case["op"]
    ea = BYTES[case.get("act", "f32" if case.get("cache") == "f32" else "bf16")]
    row = d * BYTES[case["cache"]] + (4 if case["cache"] == "fp8" else 0) if "cache" in case else 0
    if op == "rope":
        n = case["T"] * (hq + hkv) * d
        return {"bytes": 2 * n * ea + 4 * case["T"], "flops": 10 * n}
    if op == "rope_cache":
        n, live = case["T"] * hq * d, case["T"] - case["idle"]
        return {"bytes": 2 * n * ea + 2 * live * hkv * (d * ea + row) + 8 * case["T"],
                "flops": 10 * (n + live * hkv * d)}
    if op == "write":
        live = case["T"] - case["idle"]
        return {"bytes": 2 * live * hkv * (d * ea + row) + 4 * case["T"], "flops": 4 * live * hkv * d}
    lens = _lengths(case)
    if op == "read":
        n = 2 * sum(lens) * hkv
        return {"bytes": n * (row + d * ea) + 4 * sum(-(-x // case["page"]) for x in lens), "flops": n * d}
    n = sum(min(x, case["window"]) if case["window"] else x for x in lens)
    live = case["B"] - case["idle"]
    return {"bytes": 2 * n * hkv * row + 2 * live * hq * d * ea + 4 * live * hq + 4 * n // case["page"],
            "flops": 4 * n * hq * d}


def _exact_head(x, gamma, pos, inv_freq, r, inter, factor):
    """fp64 rows [T, h, d]: norm, rotation as a product of complex numbers, position factor."""
    x = x.double()
    x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * gamma.double()
    if r:
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           torch.outer(pos.double(), inv_freq.double()))[:, None, :]
        head = x[..., :r]
        pairs = head.unflatten(-1, (r // 2, 2)) if inter else head.unflatten(-1, (2, r // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        x = torch.cat([(z if inter else z.transpose(-1, -2)).flatten(-2), x[..., r:]], -1)
    return x * factor[:, None, None]


def _exact_stored(codes, scale, slots, x, page):
    """The cache side after the rows x [T, h, d] went to their slots, in fp64, and its scales."""
    out = codes.double()
    sc = None if scale is None else scale.double()
    keep = slots >= 0
    x, slots = x[keep], slots[keep].long()
    p, o = torch.div(slots, page, rounding_mode="floor"), slots.remainder(page)
    if sc is not None:
        top = x.abs().max(-1).values
        step = torch.where(top > 0, top / 448, torch.ones_like(top))
        sc[p, :, o] = step
        x = (x / step.unsqueeze(-1)).to(torch.float8_e4m3fn).double()
    out[p, :, o] = x
    return out, sc


def exact(case, seed):
    s = prepare(case, seed)
    op, page = case["op"], case.get("page", 64)
    if op in ("rope", "rope_cache"):
        pos = s["positions"]
        one = torch.ones(case["T"], dtype=torch.float64, device=DEV)
        f = (1 + pos.double().clamp(min=0) / case["ssmax"]) ** 0.1 if case["ssmax"] else one
        q = _exact_head(s["q"], s["gamma_q"], pos, s["inv_freq"], case["r"], case["inter"], f)
        k = _exact_head(s["k"], s["gamma_k"], pos, s["inv_freq"], case["r"], case["inter"], one)
        if op == "rope":
            return {"q": q, "k": k}
        ck, ks = _exact_stored(s["ck"], s["ks"], s["slots"], k, page)
        cv, vs = _exact_stored(s["cv"], s["vs"], s["slots"], s["v"].double(), page)
        return {"q": q, "ck": ck, "cv": cv, "ks": ks, "vs": vs}
    if op == "write":
        ck, ks = _exact_stored(s["ck"], s["ks"], s["slots"], s["k"].double(), page)
        cv, vs = _exact_stored(s["cv"], s["vs"], s["slots"], s["v"].double(), page)
        return {"ck": ck, "cv": cv, "ks": ks, "vs": vs}

    def rows(codes, scale, b, first, n):
        """fp64 [h, n, d]: tokens first..first+n-1 of sequence b."""
        p0, p1 = first // page, -(-(first + n) // page)
        pages = s["page_table"][b, p0:p1].long()
        x = codes[pages].double() if scale is None else codes.view(torch.uint8)[pages].view(
            torch.float8_e4m3fn).double() * scale[pages].double().unsqueeze(-1)
        return x.transpose(0, 1).flatten(1, 2)[:, first - p0 * page:first - p0 * page + n]

    lens = s["lens"].tolist()
    if op == "read":
        k = torch.cat([rows(s["ck"], s["ks"], b, 0, n).transpose(0, 1) for b, n in enumerate(lens)])
        v = torch.cat([rows(s["cv"], s["vs"], b, 0, n).transpose(0, 1) for b, n in enumerate(lens)])
        return {"k": k, "v": v}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.zeros((case["B"], hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((case["B"], hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        w = min(n, case["window"]) if case["window"] else n
        z = torch.bmm(s["q"][b].double().view(hkv, hq // hkv, d),
                      rows(s["ck"], s["ks"], b, n - w, w).transpose(1, 2).contiguous()) / math.sqrt(d)
        lse[b] = torch.logsumexp(z, -1).flatten()
        out[b] = torch.bmm(torch.softmax(z, -1), rows(s["cv"], s["vs"], b, n - w, w).contiguous()).view(hq, d)
    return {"out": out, "lse": lse}
