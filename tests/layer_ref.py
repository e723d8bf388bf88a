"""64-bit references of the decoder-layer operators around the GEMM (norm, rotary
positions, paged attention), written from their definitions, for the GPU tests.
Everything runs on the CPU in float64; nothing here touches the CUDA path."""
import math

import numpy as np
import torch

# half a step, relative to the value (normal numbers)
HALF_BF16 = 2.0 ** -8
HALF_E4M3 = 2.0 ** -4
E4M3_SUB = 2.0 ** -10  # half of E4M3's subnormal step


def e4m3_values(codes: torch.Tensor) -> torch.Tensor:
    return codes.cpu().view(torch.float8_e4m3fn).double()


def rms_norm(x, weight, eps, residual=None):
    """(r BF16 or x, h float64) of the definition."""
    r = x.cpu()
    if residual is not None:
        r = (x.cpu().float() + residual.cpu().float()).bfloat16()
    d = r.double()
    return r, d / torch.sqrt(d.square().mean(-1, keepdim=True) + eps) * weight.cpu().double()


def rope(x, positions, inv_freq, mscale, interleaved):
    """Rotated [T, heads, dim] float64 of BF16 [T, heads, dim], and |a| + |b| of each pair."""
    x = x.cpu().double()
    half = inv_freq.numel()
    u = positions.cpu().double()[:, None] * inv_freq.cpu().double()
    c, s = (u.cos() * mscale)[:, None], (u.sin() * mscale)[:, None]
    y, size = x.clone(), x.abs()
    i0 = torch.arange(half) * 2 if interleaved else torch.arange(half)
    i1 = i0 + (1 if interleaved else half)
    a, b = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = a * c - b * s, b * c + a * s
    size[..., i0] = size[..., i1] = (a.abs() + b.abs()) * abs(mscale)
    return y, size


def attention(q, k_cache, v_cache, table, seq_lens, cu_q, page, q_heads, kv_heads, scale, causal):
    """(out, lse, bound, lse_bound): float64 [T, q_heads, 128], [T, q_heads], and error bounds of both.

    The bound: half a BF16 step of the output, plus what the weights may be off by.  A weight
    is off by 2^-8 of itself (in two E4M3 parts: the first is within 2^-4, the second within 2^-4
    of the rest; in F16 it is 2^-11; an exponential's few FP32 ulps are far below), by 2^-17 of the
    row's largest (the absolute floor of two parts, 2^-10 of 256, and of the sum), and by twice the
    error of its exponent: q may be held in two E4M3 parts (off by 2^-17 of its row's largest
    channel) and 128 products are summed in FP32.

    lse: every exponent is off by that dz at most, so log sum exp(z + e), |e| <= dz, is off by dz at
    most (each term changes by a factor within exp(+-dz)).  dz is relative to the sum of the
    products' sizes, not to the logit, which may cancel.  The weights' sum adds 2^-16 (exponentials
    and additions, a few FP32 ulps each over at most 2^13 positions), the result's own FP32
    arithmetic (maximum + logarithm, changes of base) 2^-21 of it."""
    q = q.cpu().double().view(q.shape[0], q_heads, 128)
    kc, vc = (e4m3_values(c)[:, :kv_heads * 128].view(-1, kv_heads, 128) for c in (k_cache, v_cache))
    table, lens, cu = table.cpu().long(), seq_lens.cpu().tolist(), cu_q.cpu().tolist()
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    lse_bound = torch.zeros(q.shape[:2], dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    for b, n in enumerate(lens):
        rows = range(cu[b], cu[b + 1])
        m = len(rows)
        if n <= 0 or m == 0:
            continue
        c = torch.arange(n)
        slot = table[b, c // page] * page + c % page
        for g in range(kv_heads):
            k, v = kc[slot, g], vc[slot, g]
            for h in range(g * q_heads // kv_heads, (g + 1) * q_heads // kv_heads):
                x = q[cu[b]:cu[b + 1], h]
                z = x @ k.T * scale
                if causal:
                    z = z.masked_fill(c[None] > (n - m + torch.arange(m))[:, None], -math.inf)
                l = torch.logsumexp(z, 1)
                w = (z - l[:, None]).exp()
                w[torch.isinf(l)] = 0
                lse[cu[b]:cu[b + 1], h] = l
                o = w @ v
                dz = scale * (2.0 ** -17 * x.abs().amax(1) * k.abs().sum(1).max() +
                              128 * 2.0 ** -23 * (x.abs() @ k.abs().T).amax(1))
                lse_bound[cu[b]:cu[b + 1], h] = dz + 2.0 ** -16 + 2.0 ** -21 * torch.where(torch.isinf(l), 0.0, l.abs())
                off = (w * (2.0 ** -8 + 2 * dz[:, None])) @ v.abs()
                off += 2.0 ** -17 * w.amax(1, keepdim=True) * ((w > 0).double() @ v.abs())
                out[cu[b]:cu[b + 1], h] = o
                bound[cu[b]:cu[b + 1], h] = HALF_BF16 * o.abs() + off + 1e-30
    return out, lse, bound, lse_bound


def random_batch(q_lens, ctx, q_heads, kv_heads, page, seed, slot_pad=0, spare_pages=3, stale=0x7F):
    """A paged cache with shuffled pages (slots that no sequence has hold `stale` codes), its table
    (unused entries -1), lengths and queries, on the CPU."""
    rng = np.random.default_rng(seed)
    need = [-(-c // page) for c in ctx]
    pages = sum(need) + spare_pages
    width = kv_heads * 128 + slot_pad
    k, v = (torch.full((pages * page, width), stale, dtype=torch.uint8) for _ in range(2))
    table = torch.full((len(ctx), max(1, max(need, default=1))), -1, dtype=torch.int32)
    order = rng.permutation(pages)
    at = 0
    for b, c in enumerate(ctx):
        table[b, :need[b]] = torch.from_numpy(order[at:at + need[b]].astype(np.int32))
        at += need[b]
        pos = torch.arange(c)
        slot = table[b].long()[pos // page] * page + pos % page
        for cache in (k, v):
            vals = torch.from_numpy(rng.standard_normal((c, kv_heads * 128)).astype(np.float32))
            cache[slot, :kv_heads * 128] = vals.to(torch.float8_e4m3fn).view(torch.uint8)
    T = sum(q_lens)
    q = torch.from_numpy(rng.standard_normal((T, q_heads * 128)).astype(np.float32) * 1.5).bfloat16()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32)
    return {"q": q, "k_cache": k, "v_cache": v, "page_table": table,
            "seq_lens": torch.tensor(ctx, dtype=torch.int32), "cu_q": cu}
