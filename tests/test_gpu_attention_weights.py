"""Paged attention where one position takes most of a row's weight and the others share the rest
(a trained model's first position), over long contexts and with whole heads in one CTA.

The bound of every output comes from the operator, not from the number of positions:
    2^-8 |o|                       the BF16 result
    (2^-8 + 2 dz) sum_c w_c |v_c|  a weight's relative error (two parts of 4 bits) and its exponent's
    1920 * 2^-22 w_max v_max       weights near the largest one: the 1920 positions that are taken
                                   together share a fixed point of steps 2^-21 of their largest
with dz the score's error: queries within 2^-17 of their largest channel, products summed in FP32."""
import math

import pytest
import torch

import fp8_block_scaled_09_b200 as fp8bq
import layer_ref as ref

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8bq.lib()
    yield
    assert fp8bq.last_device_status() == 0


def dominated(positions, gap, at, group, tokens, batch, page, seed, spread=1.0):
    """`batch` sequences over the same pages, one kv head.  Channel 0 of every query is 8 and of every key
    0 but at position `at`, whose logit is `gap` for all rows; the other logits are about N(0, spread^2).
    Values lie around 1, those of position `at` around 0."""
    g = torch.Generator().manual_seed(seed)
    pages = -(-positions // page)
    k = torch.randn(pages * page, 128, generator=g)
    k[:, 0] = 0
    v = 1 + 0.25 * torch.randn(pages * page, 128, generator=g)
    order = torch.randperm(pages, generator=g)
    slot = lambda c: int(order[c // page]) * page + c % page
    k[slot(at)] = 0
    k[slot(at), 0] = gap / (8 * SCALE)
    v[slot(at)] = 0.01 * torch.randn(128, generator=g)
    kc, vc = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
    q = spread * torch.randn(batch * tokens, group, 128, generator=g)
    q[..., 0] = 8
    return {"q": q.bfloat16().view(batch * tokens, -1), "k_cache": kc, "v_cache": vc,
            "page_table": order.int().view(1, -1).expand(batch, -1).contiguous(),
            "seq_lens": torch.full((batch,), positions, dtype=torch.int32),
            "cu_q": torch.arange(batch + 1, dtype=torch.int32) * tokens}


def attend(c, group, tokens, page, rows=slice(None), max_q=None):
    d = {k: v.cuda() for k, v in c.items()}
    lse = torch.empty(c["q"].shape[0], group, device="cuda")
    out = fp8bq.paged_attention(d["q"], d["k_cache"], d["v_cache"], d["page_table"], d["seq_lens"], d["cu_q"], page,
                                group, 1, max_q or tokens, lse=lse)
    return out.cpu().double().view(-1, group, 128), lse.cpu().double()


def check(c, out, lse, group, tokens, sequences):
    table, n = c["page_table"][0].long(), int(c["seq_lens"][0])
    page = c["k_cache"].shape[0] // table.numel()
    slot = (table[:, None] * page + torch.arange(page)).reshape(-1)[:n]
    k, v = (ref.e4m3_values(x)[slot] for x in (c["k_cache"], c["v_cache"]))
    k_sum = k.abs().sum(1).max()
    for b in sequences:
        for i in range(tokens):
            row = b * tokens + i
            x = c["q"][row].double().view(group, 128)
            seen = n - tokens + i + 1
            z = x @ k[:seen].T * SCALE
            l = z.logsumexp(1)
            w = (z - l[:, None]).exp()
            o = w @ v[:seen]
            dz = SCALE * (2.0 ** -17 * x.abs().amax(1) * k_sum + 128 * 2.0 ** -23 * (x.abs() @ k[:seen].abs().T).amax(1))
            bound = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * dz[:, None]) * (w @ v[:seen].abs()) + \
                1920 * 2.0 ** -22 * w.amax(1, keepdim=True) * v.abs().max()
            err = (out[row] - o).abs()
            assert bool((err <= bound).all()), (row, float((err / bound).max()), float((err / o.abs()).max()))
            assert bool(((lse[row] - l).abs() <= dz + 2.0 ** -15).all())


def whole_heads():
    """Sequences that give every CTA two whole heads."""
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("group,tokens", [(7, 1), (16, 1), (7, 2)])
@pytest.mark.parametrize("positions,gap,spread", [
    (32768, 12.0, 1.0), (32768, 13.0, 1.0), (65536, 13.0, 0.3), (131072, 14.0, 1.0), (14001, 13.0, 1.0)])
def test_one_dominant_position_over_a_long_context(positions, gap, spread, group, tokens):
    batch = whole_heads()
    c = dominated(positions, gap, 0, group, tokens, batch, 64, int(gap) + positions + group, spread)
    check(c, *attend(c, group, tokens, 64), group, tokens, (0, 1, batch // 2, batch - 1))


@pytest.mark.parametrize("at", [0, 1919, 1920, 7000, 19998, 19999])
@pytest.mark.parametrize("gap", [8.0, 11.0, 16.0, 30.0, 60.0])
def test_the_dominant_position_anywhere(at, gap):
    """Behind, between and before the positions taken together; so far above the rest that their weights
    leave any fixed point shared with it.  (Of 30 and 60 nothing of the rest shows in BF16 unless it was
    multiplied back by the wrong factor.)"""
    batch = whole_heads()
    c = dominated(20000, gap, at, 7, 1, batch, 16, int(gap) + at)
    check(c, *attend(c, 7, 1, 16), 7, 1, (0, 3, batch - 1))


def test_steps_up_and_down_between_chunks():
    """Logits that fall and rise by up to 200 from one run of positions to the next: the reference that
    weights are held against moves down as well as up."""
    n, page, batch = 16000, 16, whole_heads()
    c = dominated(n, 1.0, 0, 7, 1, batch, page, 5)
    level = torch.tensor([0.0, -90, -200, 40, -90, 40, 3, 2, 0, -60])
    table = c["page_table"][0].long()
    slot = (table[:, None] * page + torch.arange(page)).reshape(-1)
    want = level.repeat_interleave(1600)[:n] / (8 * SCALE)
    c["k_cache"][slot[:n], 0] = want.to(torch.float8_e4m3fn).view(torch.uint8)
    check(c, *attend(c, 7, 1, page), 7, 1, (0, batch - 1))
    one = {k: (v[:1] if k in ("q", "page_table", "seq_lens") else v[:2] if k == "cu_q" else v) for k, v in c.items()}
    check(one, *attend(one, 7, 1, page), 7, 1, (0,))          # the same split over all CTAs


@pytest.mark.parametrize("positions,gap", [(32768, 13.0), (14001, 11.0)])
def test_few_and_many_rows_agree(positions, gap):
    """The last token of a sequence gives the same by itself and as part of a longer block."""
    group, tokens, batch = 7, 40, 4
    c = dominated(positions, gap, 0, group, tokens, batch, 64, 9)
    many, many_lse = attend(c, group, tokens, 64)
    check(c, many, many_lse, group, tokens, (0, batch - 1))
    last = torch.arange(1, batch + 1) * tokens - 1
    one = dict(c, q=c["q"][last], cu_q=torch.arange(batch + 1, dtype=torch.int32))
    few, few_lse = attend(one, group, 1, 64)
    check(one, few, few_lse, group, 1, range(batch))
    # each within the weights' 2^-8, rounded to BF16
    assert bool(((few - many[last]).abs() <= 2.0 ** -6 * many[last].abs() + 1920 * 2.0 ** -22).all())


@pytest.mark.parametrize("tokens", [3, 37])
@pytest.mark.parametrize("gap", [14.0, 18.0, 20.0])
def test_many_rows_under_a_dominant_position_without_a_value(gap, tokens):
    """Here the output is what the far positions leave: weights of 2^-20 to 2^-29 of the largest.  The weights
    of the many-row kernel are F16, 2^7 and more at the largest, so within 2^-11 of themselves or 2^-32 of the
    largest (half of F16's smallest step, 2^-25, over 2^7)."""
    group, n, page, batch = 7, 32768, 64, whole_heads()
    c = dominated(n, gap, 0, group, tokens, batch, page, int(gap))
    first = int(c["page_table"][0, 0]) * page
    c["v_cache"][first] = 0
    out, lse = attend(c, group, tokens, page)
    slot = (c["page_table"][0].long()[:, None] * page + torch.arange(page)).reshape(-1)
    k, v = (ref.e4m3_values(x)[slot] for x in (c["k_cache"], c["v_cache"]))
    for row in (0, tokens - 1, (batch // 2) * tokens, batch * tokens - 1):
        x = c["q"][row].double().view(group, 128)
        seen = n - tokens + row % tokens + 1
        z = x @ k[:seen].T * SCALE
        l = z.logsumexp(1)
        w = (z - l[:, None]).exp()
        o = w @ v[:seen]
        dz = SCALE * (2.0 ** -17 * x.abs().amax(1) * k.abs().sum(1).max() +
                      128 * 2.0 ** -23 * (x.abs() @ k[:seen].abs().T).amax(1))
        bound = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * dz[:, None]) * (w @ v[:seen].abs()) + \
            2.0 ** -32 * w.amax(1, keepdim=True) * v[:seen].abs().sum(0)
        err = (out[row] - o).abs()
        assert bool((err <= bound).all()), (row, float((err / bound).max()), float((err / o.abs()).max()))
        assert bool(((lse[row] - l).abs() <= dz + 2.0 ** -15).all())


@pytest.mark.parametrize("group,tokens", [(7, 1), (16, 1), (8, 2)])
@pytest.mark.parametrize("loud", [1.0, 60.0, 4096.0, 16384.0])
def test_a_loud_query_channel(loud, group, tokens):
    """One channel of every query far above the others, where the keys have nothing: the scores come from the
    quiet ones.  Few-row queries are within 2^-22 of their largest channel (BF16 exact from 2^-14 of it on)."""
    n, page, batch = 700, 16, 3
    g = torch.Generator().manual_seed(int(loud) + group)
    pages = -(-n // page)
    k, v = torch.randn(pages * page, 128, generator=g), torch.randn(pages * page, 128, generator=g)
    k[:, 77] = 0
    q = 1.5 * torch.randn(batch * tokens, group, 128, generator=g)
    q[..., 77] = loud
    c = {"q": q.bfloat16().view(batch * tokens, -1), "k_cache": k.to(torch.float8_e4m3fn).view(torch.uint8),
         "v_cache": v.to(torch.float8_e4m3fn).view(torch.uint8), "page_table": torch.arange(pages).int().expand(batch, -1).contiguous(),
         "seq_lens": torch.full((batch,), n, dtype=torch.int32), "cu_q": torch.arange(batch + 1, dtype=torch.int32) * tokens}
    out, lse = attend(c, group, tokens, page)
    kd, vd = (ref.e4m3_values(c[x])[:n] for x in ("k_cache", "v_cache"))
    for row in range(batch * tokens):
        seen = n - tokens + row % tokens + 1
        x = c["q"][row].double().view(group, 128)
        z = x @ kd[:seen].T * SCALE
        l = z.logsumexp(1)
        w = (z - l[:, None]).exp()
        o = w @ vd[:seen]
        top = x.abs().amax(1, keepdim=True)
        off = (x.abs() < 2.0 ** -14 * top) * 2.0 ** -22 * top
        dz = SCALE * ((off @ kd[:seen].abs().T).amax(1) + 128 * 2.0 ** -23 * (x.abs() @ kd[:seen].abs().T).amax(1))
        bound = 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2 * dz[:, None]) * (w @ vd[:seen].abs()) + \
            n * 2.0 ** -22 * w.amax(1, keepdim=True) * vd.abs().max()
        assert bool(((out[row] - o).abs() <= bound).all()), float(((out[row] - o).abs() / bound).max())
        assert bool(((lse[row] - l).abs() <= dz + 2.0 ** -15).all()), float((lse[row] - l).abs().max())
