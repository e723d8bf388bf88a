"""The quantized norm where a group's products r w leave the normal FP32 range beside 448, below and above."""
import pytest
import torch

import fp8_block_scaled_09_b200 as fp8bq
import layer_ref as ref
from test_gpu_norm_rope import _check_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8bq.lib()
    yield
    assert fp8bq.last_device_status() == 0


@pytest.mark.parametrize("K", [128, 1152, 8320, 20480])
@pytest.mark.parametrize("r_log2,w_log2", [(-70, 0), (-70, -10), (-100, 0), (-120, -10), (-126, 0), (-130, 0), (-130, -10),
                                           (-132, -15), (45, 50), (55, 55)])
def test_products_near_the_ends_of_the_range(r_log2, w_log2, K):
    """Rows and groups of this size, zeros among them, in a row by themselves or beside ordinary groups."""
    g = torch.Generator().manual_seed(K + r_log2 - w_log2)
    M = 5
    x = (torch.randn(M, K, generator=g, dtype=torch.float64) * 2.0 ** r_log2).bfloat16()
    w = ((1 + 0.2 * torch.randn(K, generator=g, dtype=torch.float64)) * 2.0 ** w_log2).bfloat16()
    x[:, ::7] = 0
    x[1] = 0
    if K > 128 and r_log2 < 0:
        x[2, 128:256] = torch.randn(128, generator=g).bfloat16()     # the row's sum is ordinary
        x[3, :128] = 0
    h = torch.empty_like(x, device="cuda")
    q, s = fp8bq.rms_norm_quantize(x.cuda(), w.cuda(), 1e-5, h=h)
    _, want = ref.rms_norm(x, w, 1e-5)
    err = (h.cpu().double() - want).abs()
    assert bool((err <= (ref.HALF_BF16 + 2.0 ** -18) * want.abs() + 2.0 ** -133).all())
    _check_codes(q, s, want)
    zero = x.unflatten(-1, (-1, 128)) == 0
    assert bool(((q.cpu().unflatten(-1, (-1, 128)) & 0x7F) == 0)[zero].all())


def test_a_row_of_zeros_without_eps():
    x = torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda")
    x[1] = 1
    q, s = fp8bq.rms_norm_quantize(x, torch.ones(256, dtype=torch.bfloat16, device="cuda"), 0.0)
    assert bool((q[0] == 0).all()) and bool((s[0] == 1).all()) and bool((q[1] == 0x7E).all())
