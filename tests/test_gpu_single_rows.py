"""One token: its row's stride, which nothing uses, may be anything."""
import pytest
import torch

import fp8_block_scaled_09_b200 as fp8bq

pytestmark = pytest.mark.gpu

HEADS, KV = 7, 1


def row_of(values, stride, rows=2):
    """[1, n] with this row stride, as a row of a wider matrix gives it."""
    wide = torch.zeros(rows * stride + values.numel(), dtype=values.dtype, device="cuda")
    t = wide.as_strided((1, values.numel()), (stride, 1))
    t.copy_(values.view(1, -1))
    return t


@pytest.mark.parametrize("extra", [-1152, -1, 0, 1, 4, 8, 12])
def test_single_token(extra):
    g = torch.Generator().manual_seed(1)
    cols, width = (HEADS + 2 * KV) * 128, HEADS * 128
    qkv = torch.randn(1, cols, generator=g).bfloat16().cuda()
    pos, loc = torch.tensor([19], device="cuda"), torch.tensor([3], device="cuda")
    freq = fp8bq.rope_inv_freq(128, 1e4, device="cuda")[0]
    kc, vc = (torch.zeros(32, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    want = fp8bq.rope_kv_write_e4m3(qkv, pos, freq, loc, kc, vc)
    keep = kc.clone(), vc.clone()
    odd = row_of(qkv, cols + extra)
    out = row_of(torch.zeros(width, dtype=torch.bfloat16), max(0, width + extra))
    assert torch.equal(fp8bq.rope_kv_write_e4m3(odd, pos, freq, loc, kc, vc, q_out=out), want)
    assert torch.equal(kc, keep[0]) and torch.equal(vc, keep[1])
    fp8bq.rope_kv_write_e4m3(odd, pos, freq, loc, kc, vc, q_out=odd[:, :width])      # in place
    assert torch.equal(odd[:, :width], want) and torch.equal(odd[:, width:], qkv[:, width:])
    table, lens, cu = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([[0]], [4], [0, 1]))
    a = fp8bq.paged_attention(want, kc, vc, table, lens, cu, 16, HEADS, KV, 1)
    q = row_of(want, max(0, width + extra))
    out = row_of(torch.zeros(width, dtype=torch.bfloat16), max(0, width + extra))
    assert torch.equal(fp8bq.paged_attention(q, kc, vc, table, lens, cu, 16, HEADS, KV, 1, out=out), a)
    assert fp8bq.last_device_status() == 0


def test_rows_of_odd_strides_are_still_refused():
    x = torch.zeros(3, 260, dtype=torch.bfloat16, device="cuda")[:, :256]
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    c = torch.zeros(16, 128, dtype=torch.uint8, device="cuda")
    with pytest.raises(fp8bq.Fp8bqError):
        fp8bq.paged_attention(x, c, c, z(1, 1), z(1), z(2), 16, 2, 1, 3)
