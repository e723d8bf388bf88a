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
