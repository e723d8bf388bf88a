"""What the operators around the FP8 linear layer are measured on.

Three operators that a decoder layer needs next to the quantized GEMMs:

* "norm": root-mean-square norm with the residual's addition, giving E4M3 codes with one
  scale per token and 128 channels (the input of the FP8 GEMM), BF16, or both;
* "rope": rotary positions of the fused QKV output; rotated queries in BF16, rotated keys
  and the values written to the E4M3 cache;
* "attention": attention of new tokens (one or many per sequence) over the paged E4M3 cache.

``run`` computes them in plain torch (``own`` false) or through this package (``own`` true);
``exact`` is their definition in 64 bits.
"""
import math

import torch

own = False

HIDDEN = 7168


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the norm before a projection when one sequence decodes
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": HIDDEN, "residual": True, "codes": True, "h": False},
        # the same for a prefill chunk of 2048 tokens
        {"name": "norm_chunk", "op": "norm", "rows": 2048, "cols": HIDDEN, "residual": True, "codes": True, "h": False},
        # a first norm (no residual yet) of a ragged batch, BF16 output kept as well, odd number of groups
        {"name": "norm_ragged", "op": "norm", "rows": 333, "cols": 8320, "residual": False, "codes": True, "h": True},
        # the norm before a BF16 head: no codes, every position of a long batch
        {"name": "norm_head", "op": "norm", "rows": 8192, "cols": HIDDEN, "residual": True, "codes": False, "h": True},
        # eight sequences decoding far into a long context
        {"name": "rope_decode", "op": "rope", "tokens": 8, "q_heads": 56, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "scaling": "yarn", "far": 900000},
        # a prefill chunk
        {"name": "rope_chunk", "op": "rope", "tokens": 8192, "q_heads": 56, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "scaling": "none", "far": 32768},
        # the drafter's heads, half of each head rotated, interleaved pairs, an odd number of tokens
        {"name": "rope_partial", "op": "rope", "tokens": 777, "q_heads": 28, "kv_heads": 4, "dim": 128, "rot": 64,
         "interleaved": True, "scaling": "linear", "far": 131072},
        # one sequence decoding over a long context
        {"name": "attn_one_long", "op": "attention", "batch": 1, "q_min": 1, "q_max": 1, "ctx_min": 65001, "ctx_max": 65001,
         "q_heads": 56, "kv_heads": 8, "page": 64, "causal": True},
        # a decode batch of 128 sequences of all lengths, a length of zero among them
        {"name": "attn_decode_batch", "op": "attention", "batch": 128, "q_min": 1, "q_max": 1, "ctx_min": 0, "ctx_max": 4096,
         "q_heads": 56, "kv_heads": 8, "page": 16, "causal": True},
        # the drafter's block of 8 positions, all of them seeing each other
        {"name": "attn_block", "op": "attention", "batch": 16, "q_min": 8, "q_max": 8, "ctx_min": 1000, "ctx_max": 8000,
         "q_heads": 28, "kv_heads": 4, "page": 32, "causal": False},
        # the prefill chunk of 2048 tokens late in a long prompt
        {"name": "attn_chunk_late", "op": "attention", "batch": 1, "q_min": 2048, "q_max": 2048, "ctx_min": 18001, "ctx_max": 18001,
         "q_heads": 56, "kv_heads": 8, "page": 64, "causal": True},
        # prompts of different lengths and single tokens in one batch
        {"name": "attn_mixed", "op": "attention", "batch": 9, "q_min": 1, "q_max": 700, "ctx_min": 0, "ctx_max": 2500,
         "q_heads": 56, "kv_heads": 8, "page": 128, "causal": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "attention", "attention"])
    if op == "norm":
        # groups of 128 columns, odd counts among them
        rows, cols = _log_int(rng, 1, 8192), 128 * _log_int(rng, 1, 64)
        codes = rng.random() < 0.7
        return {"op": op, "rows": rows, "cols": cols, "residual": rng.random() < 0.6, "codes": codes,
                "h": not codes or rng.random() < 0.3}
    heads = rng.choice([(56, 8), (28, 4), (16, 2), (8, 8), (7, 1), (12, 4), (40, 8)])
    if op == "rope":
        dim = rng.choice([64, 128, 128, 256])
        rot = rng.choice([dim, dim, dim // 2, dim // 4, dim - 16])
        return {"op": op, "tokens": _log_int(rng, 1, 4096), "q_heads": heads[0], "kv_heads": heads[1], "dim": dim, "rot": rot,
                "interleaved": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "ntk", "yarn"]),
                "far": _log_int(rng, 64, 1000000)}
    page = rng.choice([8, 16, 32, 64, 128, 256])
    kind = rng.choice(["decode", "block", "chunk", "mixed"])
    if kind == "decode":
        batch = _log_int(rng, 1, 128)
        lo, hi = 0, min(65536, _log_int(rng, 64, 524288 // batch))
        q_min = q_max = 1
    elif kind == "block":
        batch = _log_int(rng, 1, 32)
        q_min = q_max = rng.randint(2, 16)
        lo, hi = 64, min(16384, _log_int(rng, 128, 131072 // batch))
    elif kind == "chunk":
        batch = 1
        q_min = q_max = _log_int(rng, 17, 2048)
        hi = q_max + _log_int(rng, 1, 12000)
        lo = hi
    else:
        batch = rng.randint(2, 12)
        q_min, q_max = 1, _log_int(rng, 2, 700)
        lo, hi = 0, _log_int(rng, 64, 3500)
    return {"op": op, "batch": batch, "q_min": q_min, "q_max": q_max, "ctx_min": lo, "ctx_max": hi, "q_heads": heads[0],
            "kv_heads": heads[1], "page": page, "causal": kind != "block" or rng.random() < 0.5}


# ------------------------------------------------------------------ inputs

ROPE_BASE = 1.2e8


def _rope_table(rot, scaling):
    """(FP32 frequencies of the rotary pairs, factor on cos and sin): base^(-2i/rot), scaled by 8 for
    contexts beyond 32768: "linear" divides every frequency, "ntk" raises the base, "yarn" divides
    the frequencies that turn less than once in the old context and ramps to those that turn often."""
    factor, old, fast, slow = 8.0, 32768, 32.0, 1.0
    base = ROPE_BASE
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2)) if rot > 2 else base
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    m = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        turns = old * f / (2 * math.pi)
        keep = ((turns.log() - math.log(slow)) / (math.log(fast) - math.log(slow))).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        m = 0.1 * math.log(factor) + 1.0
    return f.float(), m


def _lengths(case):
    """Each sequence's number of new tokens and of cache positions (the new tokens among them), from the
    case alone: spread evenly over the ranges, short and long ones mixed."""
    b = case["batch"]
    ctx = [case["ctx_min"] + (case["ctx_max"] - case["ctx_min"]) * i // max(1, b - 1) for i in range(b)]
    q = [case["q_max"] - (case["q_max"] - case["q_min"]) * (i * 5 % b) // max(1, b - 1) for i in range(b)]
    if b == 1:
        ctx = [case["ctx_max"]]
    # a context holds at least the new tokens, but one may be empty (a slot of a padded batch)
    return q, [c if c == 0 else max(c, n) for n, c in zip(q, ctx)]


def _generator(seed, device):
    return torch.Generator(device=device).manual_seed(int(seed))


def _norm_state(case, g, dev):
    m, k = case["rows"], case["cols"]
    x = torch.randn(m, k, generator=g, device=dev).bfloat16()
    # a residual stream has a few channels far larger than the others
    r = torch.randn(m, k, generator=g, device=dev) * 3
    loud = torch.randperm(k, generator=g, device=dev)[: max(1, k // 1000)]
    r[:, loud] *= 30
    w = (1 + 0.2 * torch.randn(k, generator=g, device=dev)).bfloat16()
    return {"x": x, "weight": w, "eps": 1e-5, "residual": r.bfloat16() if case["residual"] else None,
            "residual_out": torch.empty_like(x) if case["residual"] else None,
            "q": torch.empty(m, k, dtype=torch.uint8, device=dev) if case["codes"] else None,
            "s": torch.empty(m, k // 128, device=dev) if case["codes"] else None,
            "h": torch.empty_like(x) if case["h"] else None}


def _rope_state(case, g, dev):
    t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
    qkv = torch.randn(t, (hq + 2 * hk) * d, generator=g, device=dev).bfloat16()
    # runs of consecutive positions from several sequences, up to `far`
    runs = min(t, 4)
    start = torch.randint(0, max(1, case["far"] - t), (runs,), generator=g, device=dev)
    i = torch.arange(t, device=dev)
    pos = start[i * runs // t] + i
    slots = t + t // 4 + 8
    loc = torch.randperm(slots, generator=g, device=dev)[:t]
    freq, m = _rope_table(case["rot"], case["scaling"])
    return {"qkv": qkv, "dim": d, "interleaved": case["interleaved"], "positions": pos, "loc": loc, "inv_freq": freq.to(dev), "mscale": m,
            "k_cache": torch.zeros(slots, hk * d, dtype=torch.uint8, device=dev),
            "v_cache": torch.zeros(slots, hk * d, dtype=torch.uint8, device=dev),
            "q_out": torch.empty(t, hq * d, dtype=torch.bfloat16, device=dev)}


def _attention_state(case, g, dev):
    hq, hk, d, page = case["q_heads"], case["kv_heads"], 128, case["page"]
    q_len, ctx = _lengths(case)
    t, width = sum(q_len), max(1, max(-(-c // page) for c in ctx))
    used = sum(-(-c // page) for c in ctx)
    pages = used + used // 8 + 2
    k = torch.randn(pages * page, hk * d, generator=g, device=dev).to(torch.float8_e4m3fn).view(torch.uint8)
    v = torch.randn(pages * page, hk * d, generator=g, device=dev).to(torch.float8_e4m3fn).view(torch.uint8)
    q = (1.5 * torch.randn(t, hq * d, generator=g, device=dev)).bfloat16()
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    lens = torch.tensor(ctx, device=dev, dtype=torch.int32)
    need = (lens + page - 1) // page
    first = need.cumsum(0) - need
    j = torch.arange(width, device=dev)
    table = torch.where(j < need[:, None], order[(first[:, None] + j).clamp(max=pages - 1)], -1).to(torch.int32)
    # what no sequence has written yet is not a number
    written = torch.zeros(pages, page, dtype=torch.bool, device=dev)
    inside = j[None, :, None] * page + torch.arange(page, device=dev)
    written[table.clamp(min=0).long()[table >= 0]] = (inside < lens[:, None, None])[table >= 0]
    stale = ~written.reshape(-1)
    k[stale] = 0x7F
    v[stale] = 0x7F
    cu = torch.tensor([0] + q_len, device=dev).cumsum(0).to(torch.int32)
    s = {"q": q, "k_cache": k, "v_cache": v, "page_table": table, "seq_lens": lens, "cu_q": cu, "page": page,
         "max_q": case["q_max"], "max_ctx": max(1, max(ctx)), "q_heads": hq, "kv_heads": hk, "causal": case["causal"],
         "out": torch.empty_like(q), "lse": torch.empty(t, hq, device=dev)}
    if own:
        import fp8_block_scaled_09_b200 as fp8bq
        s["workspace"] = fp8bq.new_attention_workspace(t, len(ctx), hq, hk, s["max_q"], dev)
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = _generator(seed, dev)
    make = {"norm": _norm_state, "rope": _rope_state, "attention": _attention_state}[case["op"]]
    return {"op": case["op"], **make(case, g, dev)}


# ------------------------------------------------------------------ one pass

def _e4m3(x):
    """Nearest E4M3 value, saturating."""
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _norm_plain(s):
    x = s["x"].float()
    if s["residual"] is not None:
        r = (x + s["residual"].float()).bfloat16()  # the stream as the next layer reads it
        x = r.float()
    h = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    out = {}
    if s["residual"] is not None:
        out["residual"] = r
    if s["h"] is not None:
        out["h"] = h.bfloat16()
    if s["q"] is not None:
        groups = h.unflatten(-1, (-1, 128))
        top = groups.abs().amax(-1)
        scale = torch.where(top == 0, torch.ones_like(top), top / 448)
        out["codes"] = _e4m3(groups / scale[..., None]).flatten(-2)
        out["scales"] = scale
    return out


def _rope_plain(s):
    t, d = s["qkv"].shape[0], s["k_cache"].shape[1]
    k0 = s["qkv"].shape[1] - 2 * d
    freq = s["inv_freq"]
    rot = 2 * freq.numel()
    # angles of far positions need 64 bits
    angle = s["positions"].double()[:, None] * freq.double()
    cos = (angle.cos() * s["mscale"]).float()[:, None]
    sin = (angle.sin() * s["mscale"]).float()[:, None]
    x = s["qkv"][:, : k0 + d].float().view(t, -1, s["dim"])
    r, rest = x[..., :rot], x[..., rot:]
    if s["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., : rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    y = torch.cat((r, rest), -1).view(t, -1)
    k_cache, v_cache = s["k_cache"], s["v_cache"]
    k_cache[s["loc"]] = _e4m3(y[:, k0:]).view(torch.uint8)
    v_cache[s["loc"]] = _e4m3(s["qkv"][:, k0 + d:].float()).view(torch.uint8)
    return {"q": y[:, :k0].bfloat16(), "k_cache": k_cache.view(torch.float8_e4m3fn), "v_cache": v_cache.view(torch.float8_e4m3fn)}


def _attention_plain(s):
    hq, hk, d = s["q_heads"], s["kv_heads"], 128
    table, lens, cu, page = s["page_table"].long(), s["seq_lens"].long(), s["cu_q"].long(), s["page"]
    b, dev, t = lens.numel(), lens.device, s["q"].shape[0]
    n, c = s["max_q"], s["max_ctx"]
    pos = torch.arange(c, device=dev)
    slot = table[:, pos // page].clamp(min=0) * page + pos % page                        # [b, c]
    live = pos < lens[:, None]
    k = s["k_cache"].view(torch.float8_e4m3fn)[slot].float().view(b, c, hk, d)
    v = s["v_cache"].view(torch.float8_e4m3fn)[slot].float().view(b, c, hk, d)
    v = torch.where(live[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)[:, :, None]      # [b, hk, 1, c, d]
    k = k.permute(0, 2, 3, 1)[:, :, None]                                                # [b, hk, 1, d, c]
    i = torch.arange(n, device=dev)
    q_len = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i).clamp(max=t - 1)
    q = s["q"][row].float().view(b, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4)           # [b, hk, g, n, d]
    score = (q @ k) * d ** -0.5
    seen = live[:, None, :]
    if s["causal"]:
        seen = seen & (pos <= (lens - q_len)[:, None, None] + i[:, None])
    score = score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(total == 0, 1.0, total)
    lse = top + total.log()
    mine = i < q_len[:, None]
    o = o.permute(0, 3, 1, 2, 4).reshape(b, n, hq * d)[mine]
    return {"out": o.bfloat16(), "lse": lse.squeeze(-1).permute(0, 3, 1, 2).reshape(b, n, hq)[mine]}


def _own(s):
    import fp8_block_scaled_09_b200 as fp8bq
    f8 = torch.float8_e4m3fn
    if s["op"] == "norm":
        out = {}
        if s["q"] is not None:
            fp8bq.rms_norm_quantize(s["x"], s["weight"], s["eps"], residual=s["residual"], residual_out=s["residual_out"],
                                    q=s["q"], s=s["s"], h=s["h"])
            out = {"codes": s["q"].view(f8), "scales": s["s"]}
        else:
            fp8bq.rms_norm(s["x"], s["weight"], s["eps"], residual=s["residual"], residual_out=s["residual_out"], h=s["h"])
        if s["h"] is not None:
            out["h"] = s["h"]
        if s["residual"] is not None:
            out["residual"] = s["residual_out"]
        return out
    if s["op"] == "rope":
        fp8bq.rope_kv_write_e4m3(s["qkv"], s["positions"], s["inv_freq"], s["loc"], s["k_cache"], s["v_cache"],
                                 head_dim=s["dim"], interleaved=s["interleaved"], mscale=s["mscale"], q_out=s["q_out"])
        return {"q": s["q_out"], "k_cache": s["k_cache"].view(f8), "v_cache": s["v_cache"].view(f8)}
    fp8bq.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"], s["cu_q"], page_size=s["page"],
                          q_heads=s["q_heads"], kv_heads=s["kv_heads"], max_q_len=s["max_q"], causal=s["causal"],
                          out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm_plain, "rope": _rope_plain, "attention": _attention_plain}[state["op"]](state)


# ------------------------------------------------------------------ the least work

def work(case):
    if case["op"] == "norm":
        m, k = case["rows"], case["cols"]
        per = 2 + (4 if case["residual"] else 0) + (1 + 4 / 128 if case["codes"] else 0) + (2 if case["h"] else 0)
        return {"bytes": m * k * per + 2 * k, "flops": 6 * m * k}
    if case["op"] == "rope":
        t, hq, hk, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        return {"bytes": t * ((hq + 2 * hk) * d * 2 + hq * d * 2 + 2 * hk * d + 16), "flops": t * (hq + hk) * case["rot"] * 3}
    hq, hk, d = case["q_heads"], case["kv_heads"], 128
    q_len, ctx = _lengths(case)
    pairs = 0
    for n, c in zip(q_len, ctx):
        if case["causal"]:
            low = max(0, c - n)  # positions that the first new token has behind it
            m = min(n, c)
            pairs += m * low + m * (m + 1) // 2
        else:
            pairs += n * c
    t = sum(q_len)
    return {"bytes": t * hq * (d * 4 + 4) + sum(ctx) * hk * d * 2, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ the definition in 64 bits

def _e4m3_exact(v):
    """The E4M3 value next to v: steps of an eighth of v's power of two, of 2^-9 below 2^-6."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return ((v / step).round() * step).clamp(-448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        out, m, k = {}, case["rows"], case["cols"]
        x = s["x"].double()
        if case["residual"]:
            out["residual"] = (x + s["residual"].double())
            x = out["residual"].float().bfloat16().double()
        h = s["weight"].double() * x / ((x * x).sum(1, keepdim=True) / k + s["eps"]).sqrt()
        if case["h"]:
            out["h"] = h
        if case["codes"]:
            a = h.reshape(m, k // 128, 128)
            scale = a.abs().max(2).values / 448
            scale[scale == 0] = 1
            out["codes"] = _e4m3_exact(a / scale.unsqueeze(2)).reshape(m, k)
            out["scales"] = scale
        return out
    if case["op"] == "rope":
        t, hq, hk, d, rot = (case[n] for n in ("tokens", "q_heads", "kv_heads", "dim", "rot"))
        x = s["qkv"].double().reshape(t, hq + 2 * hk, d)
        y = x.clone()
        for j in range(rot // 2):
            i0, i1 = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + rot // 2)
            a = s["positions"].double() * s["inv_freq"][j].double()
            c, n = (a.cos() * s["mscale"])[:, None], (a.sin() * s["mscale"])[:, None]
            y[:, : hq + hk, i0] = x[:, : hq + hk, i0] * c - x[:, : hq + hk, i1] * n
            y[:, : hq + hk, i1] = x[:, : hq + hk, i0] * n + x[:, : hq + hk, i1] * c
        kc = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device=x.device)
        vc = torch.zeros_like(kc)
        kc[s["loc"]] = _e4m3_exact(y[:, hq:hq + hk]).reshape(t, -1)
        vc[s["loc"]] = _e4m3_exact(y[:, hq + hk:]).reshape(t, -1)
        return {"q": y[:, :hq].reshape(t, -1), "k_cache": kc, "v_cache": vc}
    hq, hk, d, page = case["q_heads"], case["kv_heads"], 128, case["page"]
    q_len, ctx = _lengths(case)
    out = torch.zeros(sum(q_len), hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(q_len), hq), -math.inf, dtype=torch.float64, device="cuda")
    kc, vc = (s[n].view(torch.float8_e4m3fn).view(-1, page, hk, d) for n in ("k_cache", "v_cache"))
    at = 0
    for b, (n, c) in enumerate(zip(q_len, ctx)):
        pages = s["page_table"][b, : -(-c // page)].long()
        for g in range(hk if c else 0):
            k = kc[pages, :, g].reshape(-1, d)[:c].double()
            v = vc[pages, :, g].reshape(-1, d)[:c].double()
            for h in range(g * (hq // hk), (g + 1) * (hq // hk)):
                z = s["q"][at:at + n, h * d:(h + 1) * d].double() @ k.T / math.sqrt(d)
                if case["causal"]:
                    last = torch.arange(c - n, c, device="cuda")
                    z[torch.arange(c, device="cuda")[None] > last[:, None]] = -math.inf
                lse[at:at + n, h] = z.logsumexp(1)
                p = (z - lse[at:at + n, h][:, None]).exp()
                p[lse[at:at + n, h] == -math.inf] = 0
                out[at:at + n, h] = p @ v
        at += n
    return {"out": out.reshape(-1, hq * d), "lse": lse}
