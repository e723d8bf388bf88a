"""GPU parity of paged attention against a 64-bit reference on the CPU (layer_ref.attention,
which also derives the tolerance of every output)."""
import math

import numpy as np
import pytest
import torch

import fp8_block_scaled_09_b200 as fp8bq
import layer_ref as ref
from gpu_util import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8bq.lib()
    yield
    assert fp8bq.last_device_status() == 0


def run(c, q_heads, kv_heads, page, causal=True, scale=None, pad_rows=0, ws=None, max_q=None):
    """(out, lse) of one call; checks the guard bands and the padding rows."""
    d = {k: v.cuda() for k, v in c.items()}
    T = c["q"].shape[0]
    q = torch.full((T + pad_rows, q_heads * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[:T] = d["q"]
    out = Guarded((T + pad_rows, q_heads * 128), torch.bfloat16, fill=0x5A)
    lse = Guarded((T + pad_rows, q_heads), torch.float32, fill=0x5A)
    lens = (c["cu_q"][1:] - c["cu_q"][:-1]).tolist()
    fp8bq.paged_attention(q, d["k_cache"], d["v_cache"], d["page_table"], d["seq_lens"], d["cu_q"],
                          page, q_heads, kv_heads, max_q or max(lens), scale=scale, causal=causal,
                          out=out.t, lse=lse.t, workspace=ws)
    torch.cuda.synchronize()
    assert out.guards_intact() and lse.guards_intact()
    assert bool((out.t[T:].view(torch.int16) == 0x5A5A).all()) and bool((lse.t[T:].view(torch.int32) == 0x5A5A5A5A).all())
    return out.t[:T].cpu(), lse.t[:T].cpu()


def check(c, out, lse, q_heads, kv_heads, page, causal=True, scale=None):
    o, l, bound, l_bound = ref.attention(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["seq_lens"],
                                c["cu_q"], page, q_heads, kv_heads, scale or 128 ** -0.5, causal)
    err = (out.double().view(o.shape) - o).abs()
    assert bool(torch.isfinite(out.float()).all())
    assert bool((err <= bound).all()), (float((err / bound.clamp(min=1e-20)).max()), int((err > bound).sum()))
    empty = torch.isinf(l)
    assert bool((lse[empty] == -math.inf).all()) and bool((out.view(o.shape)[empty] == 0).all())
    e = (lse.double() - l).abs()[~empty] - l_bound[~empty]
    assert bool((e <= 0).all()), float(e.max())


HEADS = [(56, 8), (28, 4), (8, 8), (7, 1), (12, 4), (16, 2)]
DECODE_CTX = [[1], [127, 128, 129], [0, 1, 700, 0, 64, 2049], [3000] * 5, [15, 16, 17, 33, 1], [6150],
              # several sequences and chunks for each CTA
              [37 * i % 2900 for i in range(90)],
              # more sequences than CTAs, most of them shorter than a tile, some empty
              [i * 7 % 41 for i in range(700)]]


@pytest.mark.parametrize("page", [8, 16, 64, 128, 512])
@pytest.mark.parametrize("i", range(len(DECODE_CTX)))
def test_decode(i, page):
    hq, hk = HEADS[(i + page) % len(HEADS)]
    ctx = DECODE_CTX[i]
    c = ref.random_batch([1] * len(ctx), ctx, hq, hk, page, 10 * i + page, slot_pad=16 * (i % 2))
    check(c, *run(c, hq, hk, page, pad_rows=i % 3), hq, hk, page)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,ctx,heads,page", [
    ([2, 2], [2, 300], (56, 8), 16),
    ([8] * 4, [8, 9, 1000, 137], (28, 4), 32),            # a drafter's block
    ([8, 3, 0, 8], [700, 3, 50, 0], (56, 8), 64),         # no new tokens; nothing to see
    ([9, 5], [4, 0], (7, 1), 16),                         # more new tokens than positions
    ([5 - i % 4 for i in range(60)], [41 * i % 900 for i in range(60)], (56, 8), 16),
    ([3] * 70, [53 * i % 1500 for i in range(70)], (32, 8), 64),
    ([16], [2500], (32, 8), 128), ([33], [33], (2, 1), 8), ([64, 1], [64, 4000], (4, 4), 256)])
def test_few_tokens(q_lens, ctx, heads, page, causal):
    c = ref.random_batch(q_lens, ctx, *heads, page, 7 + len(ctx))
    check(c, *run(c, *heads, page, causal, pad_rows=2), *heads, page, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,ctx,heads,page", [
    ([128], [128], (7, 1), 64), ([129], [300], (8, 8), 16), ([37], [37], (14, 2), 8),
    ([100, 1, 250], [100, 513, 700], (28, 4), 128), ([19, 0, 65, 40], [3, 0, 65, 0], (56, 8), 32),
    ([257], [1000], (6, 2), 256), ([200], [5000], (8, 1), 64),
    # blocks of up to 64, 128 and 256 rows, whole and split, several for each CTA
    ([5 + i % 15 for i in range(40)], [29 * i % 1200 for i in range(40)], (56, 8), 16),
    ([40 + i % 60 for i in range(24)], [37 * i % 1000 for i in range(24)], (28, 4), 64),
    ([5] * 3, [9000, 3, 4000], (56, 8), 64), ([600] * 2, [600, 0], (8, 8), 128),
    # sequences without positions: first and last, between others, all of them, more than 32
    ([700, 5, 0, 64, 300, 41], [0, 5, 0, 0, 700, 0], (28, 4), 16), ([300, 40], [0, 0], (7, 1), 64),
    ([17 + i % 5 for i in range(90)], [(i % 3) * 31 * i % 500 for i in range(90)], (8, 8), 32)])
def test_chunks(q_lens, ctx, heads, page, causal):
    c = ref.random_batch(q_lens, ctx, *heads, page, 70 + len(ctx))
    check(c, *run(c, *heads, page, causal, pad_rows=1), *heads, page, causal)


@pytest.mark.parametrize("n", [1, 40])
def test_other_scales_and_magnitudes(n):
    """Logits of several hundred (one position takes all the weight), of 1e-3, and a far maximum
    that comes last; also queries with channels of very different size."""
    for k, (mul, scale) in enumerate([(40.0, 1.0), (1e-3, 0.1), (1e-20, 1.0), (2.0 ** 60, 2.0 ** -62)]):
        c = ref.random_batch([n, n], [300, 1500], 7, 1, 16, 50 + k)
        c["q"] = (c["q"].float() * mul).bfloat16()
        c["q"][:, ::5] *= 0.01
        last = c["page_table"][1].long()[torch.arange(1480, 1500) // 16] * 16 + torch.arange(1480, 1500) % 16
        c["k_cache"][last] = 0x70                              # 128
        check(c, *run(c, 7, 1, 16, scale=scale), 7, 1, 16, scale=scale)


def test_extreme_codes():
    """Keys and values at +-448, zeros, and a query of zeros (uniform weights)."""
    c = ref.random_batch([1, 30], [400, 333], 7, 1, 16, 3)
    rng = np.random.default_rng(0)
    live = c["k_cache"] != 0x7F
    big = torch.from_numpy(rng.choice(np.array([0x7E, 0xFE, 0x00, 0x80, 0x01], np.uint8), c["v_cache"].shape))
    c["v_cache"][live] = big[live]
    c["k_cache"][live] = big.flip(1)[live]
    c["q"][5] = 0
    check(c, *run(c, 7, 1, 16), 7, 1, 16)


def test_strided_and_shared_inputs():
    """Queries as columns of a wider tensor, outputs with a row stride, a strided table, the
    same page for two sequences (a shared prefix), and caches as float8 tensors."""
    c = ref.random_batch([1, 1, 3], [200, 200, 90], 14, 2, 32, 4)
    c["page_table"][1] = c["page_table"][0]
    d = {k: v.cuda() for k, v in c.items()}
    wide = torch.randn(5, 14 * 128 + 512, device="cuda").bfloat16()
    wide[:, :14 * 128] = d["q"]
    out = torch.full((5, 14 * 128 + 64), 3.0, dtype=torch.bfloat16, device="cuda")
    table = torch.full((3, d["page_table"].shape[1] + 3), 1 << 30, dtype=torch.int32, device="cuda")
    table[:, :-3] = d["page_table"]
    fp8bq.paged_attention(wide[:, :14 * 128], d["k_cache"].view(torch.float8_e4m3fn), d["v_cache"],
                          table[:, :-3], d["seq_lens"], d["cu_q"], 32, 14, 2, 3, out=out[:, 64:])
    torch.cuda.synchronize()
    assert bool((out[:, :64] == 3).all())
    o, _, bound, _ = ref.attention(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["seq_lens"],
                                c["cu_q"], 32, 14, 2, 128 ** -0.5, True)
    assert bool(((out[:, 64:].cpu().double().view(o.shape) - o).abs() <= bound).all())


@pytest.mark.parametrize("n", [1, 40])
def test_device_side_checks(n):
    """Bad pages read as zeros, bad lengths are clamped, tokens beyond max_q_len are skipped:
    reported, and the other sequences are right."""
    c = ref.random_batch([n, n, n], [100, 200, 300], 7, 1, 16, 5)
    good, good_lse = run(c, 7, 1, 16)
    pages = c["k_cache"].shape[0] // 16
    for bad in (-1, pages, 2 ** 31 - 1, -(2 ** 31)):
        b = {k: v.clone() for k, v in c.items()}
        b["page_table"][1, 3] = bad
        out, lse = run(b, 7, 1, 16)
        assert fp8bq.last_device_status() == 8
        assert torch.equal(out[:n], good[:n]) and torch.equal(out[2 * n:], good[2 * n:])
        # the reference on a cache that has zeros there
        z = {k: v.clone() for k, v in c.items()}
        at = int(z["page_table"][1, 3]) * 16
        z["k_cache"][at:at + 16] = 0
        z["v_cache"][at:at + 16] = 0
        check(z, out, lse, 7, 1, 16)
    for bad, as_if in ((-5, 0), (c["page_table"].shape[1] * 16 + 1, None)):
        b = {k: v.clone() for k, v in c.items()}
        b["seq_lens"][0] = bad
        out, lse = run(b, 7, 1, 16)
        assert fp8bq.last_device_status() == 8
        assert torch.equal(out[n:], good[n:])
        if as_if == 0:
            assert bool((out[:n] == 0).all()) and bool((lse[:n] == -math.inf).all())
    b = {k: v.clone() for k, v in c.items()}
    b["cu_q"] = torch.tensor([0, n, 2 * n, 3 * n + 1], dtype=torch.int32)     # beyond T
    d = {k: v.cuda() for k, v in b.items()}
    out = Guarded((3 * n, 7 * 128), torch.bfloat16)
    fp8bq.paged_attention(d["q"], d["k_cache"], d["v_cache"], d["page_table"], d["seq_lens"], d["cu_q"],
                          16, 7, 1, n + 1, out=out.t)
    assert fp8bq.last_device_status() == 8 and out.guards_intact()
    assert torch.equal(out.t[:2 * n].cpu(), good[:2 * n])


@pytest.mark.parametrize("n", [1, 30])
def test_cache_beyond_4_gib(n):
    """Pages whose bytes lie behind 2^32, written by the rotary call and read by attention."""
    heads, kv, page, ctx = 14, 2, 64, 200
    slots = (1 << 32) // 256 + 64 * page
    kc, vc = (torch.empty(slots, kv * 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(n)
    table = (slots // page - 1 - torch.randperm(8, generator=g)[:4]).int().view(1, 4)
    pos = torch.arange(ctx)
    loc = table[0].long()[pos // page] * page + pos % page
    assert int(loc.min()) * kv * 128 > 1 << 32
    qkv = torch.randn(ctx, (heads + 2 * kv) * 128, generator=g).bfloat16()
    freq = fp8bq.rope_inv_freq(128, 1e4, device="cuda")[0]
    q = fp8bq.rope_kv_write_e4m3(qkv.cuda(), pos.cuda(), freq, loc.cuda(), kc, vc)[-n:]
    out = fp8bq.paged_attention(q, kc, vc, table.cuda(), torch.tensor([ctx], dtype=torch.int32, device="cuda"),
                                torch.tensor([0, n], dtype=torch.int32, device="cuda"), page, heads, kv, n)
    # the same pages as a small cache
    first = slots - 8 * page
    y, size = ref.rope(qkv.view(ctx, -1, 128)[:, :heads + kv], pos, freq, 1.0, False)
    k = ref.e4m3_values(kc[loc.cuda()]).view(ctx, kv, 128)
    assert bool(((k - y[:, heads:]).abs() <= torch.maximum(ref.HALF_E4M3 * y[:, heads:].abs(), torch.tensor(ref.E4M3_SUB))
                 + 2.0 ** -20 * size[:, heads:]).all())
    o, _, bound, _ = ref.attention(q, kc[first:], vc[first:], table - first // page, torch.tensor([ctx]), torch.tensor([0, n]),
                                   page, heads, kv, 128 ** -0.5, True)
    assert bool(((out.cpu().double().view(o.shape) - o).abs() <= bound).all())


@pytest.mark.parametrize("n,heads", [(3, (7, 1)), (60, (7, 1)), (200, (2, 1))])
def test_more_tokens_than_promised(n, heads):
    """Tokens beyond max_q_len are skipped (their rows stay) and reported; those before them stand at
    their positions among all of them.  Offsets that run backwards touch no other row."""
    c = ref.random_batch([n, n], [n + 50, 300], *heads, 16, 8)
    take = 2 if n == 3 else n - 7
    o, _, bound, _ = ref.attention(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["seq_lens"], c["cu_q"], 16, *heads, 128 ** -0.5, True)
    d = {k: v.cuda() for k, v in c.items()}
    call = lambda cu, out, m: fp8bq.paged_attention(d["q"], d["k_cache"], d["v_cache"], d["page_table"], d["seq_lens"], cu,
                                                    16, *heads, m, out=out)
    out = torch.full_like(d["q"], 7.0)
    call(d["cu_q"], out, take)
    assert fp8bq.last_device_status() == 8
    got = out.cpu().double().view(o.shape)
    for b in range(2):
        rows = slice(b * n, b * n + take)
        assert bool(((got[rows] - o[rows]).abs() <= bound[rows]).all())
        assert bool((got[b * n + take:(b + 1) * n] == 7).all())
    for cu in ([0, n, 0], [n, 0, n], [-5, 0, -2 ** 31], [2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]):
        out = Guarded(tuple(c["q"].shape), torch.bfloat16)
        call(torch.tensor(cu, dtype=torch.int32, device="cuda"), out.t, n)
        torch.cuda.synchronize()
        assert out.guards_intact() and fp8bq.last_device_status() == 8


def test_empty_batch_and_cache():
    kc = torch.zeros(0, 128, dtype=torch.uint8, device="cuda")
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    q = torch.ones(2, 256, dtype=torch.bfloat16, device="cuda")
    out = fp8bq.paged_attention(q, kc, kc, z(2, 0), z(2), torch.arange(3, dtype=torch.int32, device="cuda"), 16, 2, 1, 1)
    assert bool((out == 0).all())
    assert fp8bq.paged_attention(q[:0], kc, kc, z(0, 0), z(0), z(1), 16, 2, 1, 0).shape == (0, 256)


def test_runs_repeat_share_a_workspace_and_replay():
    """Two calls with the same inputs give the same bits; one workspace serves decode, chunks and
    a GEMM in turn, on a side stream, and captured graphs that share it replay with new inputs."""
    dec = ref.random_batch([1] * 3, [4000, 10, 900], 56, 8, 16, 1)
    chunk = ref.random_batch([60, 70], [60, 900], 56, 8, 16, 2)
    size = max(fp8bq.attention_workspace_size(3, 3, 56, 8, 1), fp8bq.attention_workspace_size(130, 2, 56, 8, 70),
               fp8bq.workspace_size(fp8bq.OP_GEMM, 8, 256, 1024))
    ws = torch.zeros(max(size, 256), dtype=torch.uint8, device="cuda")
    x = torch.randn(8, 1024, device="cuda").bfloat16()
    qw, sw = fp8bq.quantize_weight(torch.randn(256, 1024, device="cuda").bfloat16())
    y0 = fp8bq.linear(x, qw, sw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = run(dec, 56, 8, 16, ws=ws)
        check(dec, *first, 56, 8, 16)
        many = run(chunk, 56, 8, 16, ws=ws)
        check(chunk, *many, 56, 8, 16)
        qa, sa = fp8bq.quantize_act(x)
        assert torch.equal(fp8bq.gemm(qa, sa, qw, sw, workspace=ws), y0)
        again = run(dec, 56, 8, 16, ws=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    torch.cuda.synchronize()
    graphs = []
    for c, n in ((dec, 1), (chunk, 70)):
        d = {k: v.cuda() for k, v in c.items()}
        out = torch.empty_like(d["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fp8bq.paged_attention(d["q"], d["k_cache"], d["v_cache"], d["page_table"], d["seq_lens"],
                                  d["cu_q"], 16, 56, 8, n, out=out, workspace=ws)
        graphs.append((g, d, out))
    for _ in range(3):
        for g, _, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(graphs[0][2].cpu(), first[0]) and torch.equal(graphs[1][2].cpu(), many[0])
    new = ref.random_batch([1] * 3, [33, 3990, 0], 56, 8, 16, 9)     # other lengths and pages
    for k, v in graphs[0][1].items():
        n = [min(a, b) for a, b in zip(v.shape, new[k].shape)]
        if v.dim() == 2:
            v[:n[0], :n[1]] = new[k][:n[0], :n[1]].cuda()
        else:
            v[:n[0]] = new[k].cuda()
    graphs[0][0].replay()
    got = graphs[0][2].cpu()
    c = {k: v.cpu() for k, v in graphs[0][1].items()}
    o, _, bound, _ = ref.attention(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["seq_lens"], c["cu_q"], 16, 56, 8, 128 ** -0.5, True)
    assert bool(((got.double().view(o.shape) - o).abs() <= bound).all())
