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
