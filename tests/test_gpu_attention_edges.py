"""Paged attention at the ends of what its documentation allows: scales that leave FP32's range beside
a row's own power of two, lengths beyond the page table, scores near the documented limit."""
import math

import pytest
import torch

import fp8_block_scaled_09_b200 as fp8bq
import layer_ref as ref
from test_gpu_attention import check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8bq.lib()
    yield
    assert fp8bq.last_device_status() == 0


@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("scale", [2.0 ** -62, 1e-30, 1e-38])
def test_scales_below_the_smallest_float(n, scale):
    """Rows of zeros and of 2^-90 under a small scale: every position that is seen has the same weight."""
    c = ref.random_batch([n, n], [100, 300], 7, 1, 16, 4)
    c["q"].mul_(2.0 ** -90)
    c["q"][::2] = 0
    check(c, *run(c, 7, 1, 16, scale=scale), 7, 1, 16, scale=scale)


@pytest.mark.parametrize("n", [1, 2, 40])
@pytest.mark.parametrize("over", [1, 1 << 20, 2 ** 31 - 1])
def test_a_length_beyond_the_table_is_clamped(n, over):
    """The clamped sequence has max_pages * page_size positions, those of entries that are not in the cache
    zeros, and its tokens stand at the end of those."""
    page = 16
    c = ref.random_batch([n, n, n], [100, 200, 300], 7, 1, page, 5)
    cap = c["page_table"].shape[1] * page
    b = dict(c, seq_lens=c["seq_lens"].clone())
    b["seq_lens"][0] = min(cap + over, 2 ** 31 - 1)
    z = {k: v.clone() for k, v in c.items()}
    slots = z["k_cache"].shape[0]
    for name in ("k_cache", "v_cache"):
        # behind a length a page may hold anything; here those positions count
        at = int(z["page_table"][0, 100 // page]) * page
        z[name][at + 100 % page:at + page] = 0
        z[name] = torch.cat([z[name], torch.zeros(page, 128, dtype=torch.uint8)])
    z["page_table"][0][z["page_table"][0] < 0] = slots // page
    z["seq_lens"][0] = cap
    b["k_cache"], b["v_cache"] = z["k_cache"][:slots], z["v_cache"][:slots]
    out, lse = run(b, 7, 1, page)
    assert fp8bq.last_device_status() == 8
    check(z, out, lse, 7, 1, page)


@pytest.mark.parametrize("n", [1, 2, 40])
def test_scores_near_the_documented_limit(n):
    """Scores up to 2^20: one position has all the weight wherever it leads by more than FP32 can be off by."""
    c = ref.random_batch([n, n], [300, 900], 7, 1, 16, 6)
    scale = 2.0 ** 13
    out, lse = run(c, 7, 1, 16, scale=scale)
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
    q, at, sure = c["q"].double().view(-1, 7, 128), 0, 0
    kd, vd = (ref.e4m3_values(c[x]) for x in ("k_cache", "v_cache"))
    for b, length in enumerate(c["seq_lens"].tolist()):
        pos = torch.arange(length)
        slot = c["page_table"][b].long()[pos // 16] * 16 + pos % 16
        for i in range(n):
            x = q[at]
            z = x @ kd[slot].T * scale
            z[:, length - n + i + 1:] = -math.inf
            assert float(z.abs()[:, :length - n + i + 1].max()) < 2 ** 21
            top, where = z.topk(2, 1)
            dz = scale * (2.0 ** -17 * x.abs().amax(1) * kd[slot].abs().sum(1).max() +
                          128 * 2.0 ** -23 * (x.abs() @ kd[slot].abs().T).amax(1))
            clear = top[:, 0] - top[:, 1] > 2 * dz + 40
            want = vd[slot][where[:, 0]]
            err = (out[at].double().view(7, 128) - want).abs()
            assert bool((err <= 2.0 ** -7 * want.abs() + 2.0 ** -20)[clear].all())
            assert bool(((lse[at].double() - top[:, 0]).abs() <= dz + 2.0 ** -22 * top[:, 0].abs())[clear].all())
            sure, at = sure + int(clear.sum()), at + 1
    assert sure > 7 * n


@pytest.mark.parametrize("n", [1, 40])
def test_the_longest_context(n):
    """2^25 positions over 32 pages that come again and again: the same weights as over each of them once (the last
    tokens' own few positions aside), and a log-sum-exp larger by the log of how often."""
    page, pages, length = 64, 32, 1 << 25
    c = ref.random_batch([n], [pages * page], 7, 1, page, 2, spare_pages=0)
    o, l, bound, l_bound = ref.attention(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["seq_lens"], c["cu_q"],
                                         page, 7, 1, 128 ** -0.5, False)
    times = length // (pages * page)
    long = dict(c, page_table=c["page_table"].repeat(1, times), seq_lens=torch.tensor([length], dtype=torch.int32))
    for causal in (True, False):
        out, lse = run(long, 7, 1, page, causal)
        # 40 masked positions of 2^25 weigh 2^-16 at most (a weight is below 2^4 times the mean here)
        slack = 2.0 ** -16 * c["v_cache"].view(torch.float8_e4m3fn).float().nan_to_num().abs().max() if causal else 0.0
        assert bool(((out.double().view(o.shape) - o).abs() <= bound + slack).all())
        assert bool(((lse.double() - l - math.log(times)).abs() <= l_bound + 2.0 ** -14).all())


@pytest.mark.parametrize("heads,n", [((1024, 1), 1), ((1024, 1024), 1), ((1024, 1024), 3), ((1024, 64), 2), ((1023, 3), 1)])
def test_the_most_heads(heads, n):
    c = ref.random_batch([n, n], [130, 40], *heads, 16, 12)
    check(c, *run(c, *heads, 16), *heads, 16)


@pytest.mark.parametrize("n", [1, 20])
def test_the_most_sequences(n):
    """65536 sequences, every third one empty, over a few shared pages."""
    batch, page, pages = 65536, 8, 4
    g = torch.Generator().manual_seed(n)
    kc, vc = (torch.randn(pages * page, 128, generator=g).to(torch.float8_e4m3fn).view(torch.uint8).cuda() for _ in range(2))
    table = torch.stack([torch.randperm(pages, generator=g)[:3] for _ in range(64)]).int().repeat(batch // 64, 1)
    lens = (torch.arange(batch) % 3 * 11).int()
    q = torch.randn(batch * n, 128, generator=g).bfloat16()
    out = fp8bq.paged_attention(q.cuda(), kc, vc, table.cuda(), lens.cuda(), (torch.arange(batch + 1) * n).int().cuda(),
                                page, 1, 1, n).cpu().double().view(batch, n, 128)
    assert bool((out[::3] == 0).all())
    k, v = ref.e4m3_values(kc.cpu()), ref.e4m3_values(vc.cpu())
    for part in (1, 2):
        b = torch.arange(part, batch, 3)
        pos = torch.arange(11 * part)
        slot = table[b].long()[:, pos // page] * page + pos % page
        z = torch.einsum("bnd,bcd->bnc", q.double().view(batch, n, 128)[b], k[slot]) * 128 ** -0.5
        z = z.masked_fill(pos > (11 * part - n + torch.arange(n))[:, None], -math.inf)
        w = z.softmax(-1).nan_to_num()
        o, size = w @ v[slot], w @ v[slot].abs()
        # BF16, the weights' 2^-8 and an exponent off by 2^-12 (|z| below 16)
        assert bool(((out[b] - o).abs() <= 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -11) * size + 2.0 ** -12).all())
