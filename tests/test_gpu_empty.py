"""Calls with nothing in them: no rows, no tokens, a cache without slots."""
import pytest
import torch

import fp8_block_scaled_09_b200 as fp8bq

pytestmark = pytest.mark.gpu


def bf16(*s):
    return torch.ones(*s, dtype=torch.bfloat16, device="cuda")


def test_no_rows():
    before = fp8bq.launch_count()
    x, w = bf16(4, 256), bf16(256)
    q, s = fp8bq.rms_norm_quantize(x[:0], w, residual=x[:0], residual_out=bf16(0, 256), h=x[:0])
    assert q.shape == (0, 256) and s.shape == (0, 2)
    assert fp8bq.rms_norm(bf16(0, 256), w).shape == (0, 256)
    i = torch.arange(4, device="cuda")
    kc, vc = (torch.full((8, 128), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2))
    freq = fp8bq.rope_inv_freq(128, 1e4, device="cuda")[0]
    assert fp8bq.rope_kv_write_e4m3(bf16(4, 384)[:0], i[:0], freq, i[:0], kc, vc).shape == (0, 128)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    assert fp8bq.paged_attention(bf16(0, 128), kc, vc, z(3, 1), z(3), z(4), 8, 1, 1, 1).shape == (0, 128)
    assert fp8bq.launch_count() == before
    assert bool((kc == 0xA5).all()) and fp8bq.last_device_status() == 0


def test_tokens_without_a_slot_to_go_to():
    """A cache of no slots: padding tokens are skipped, others reported."""
    none = torch.zeros(0, 128, dtype=torch.uint8, device="cuda")
    freq = fp8bq.rope_inv_freq(128, 1e4, device="cuda")[0]
    pos = torch.arange(3, device="cuda")
    out = 7 * bf16(3, 128)
    for loc, status in (([-1, -1, -1], 0), ([-1, 0, -1], 8)):
        fp8bq.rope_kv_write_e4m3(bf16(3, 384), pos, freq, torch.tensor(loc, device="cuda"), none, none, q_out=out)
        assert fp8bq.last_device_status() == status and bool((out == 7).all())
