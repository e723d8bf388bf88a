"""GPU parity of the RMS norm with quantized output and of the rotary positions with the
cache write, against 64-bit references on the CPU.

Tolerances, from the definitions: the residual stream is one FP32 addition rounded to BF16,
so it is exact.  h goes through a FP32 sum of squares (in trees of a few hundred terms at
most per thread and lane), one rsqrt and two products: within 2^-19 of itself; scales are
that plus one division.  A code's value times its scale is within half an E4M3 step of h.
Cosine and sine are within 2^-20, queries then round to BF16 and keys to E4M3 once."""
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


def _norm_inputs(M, K, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x, r = torch.randn(M, K, generator=g), 3 * torch.randn(M, K, generator=g)
    r[:, :: max(1, K // 7)] *= 30
    if kind == "zero":       # whole rows and whole groups of zeros
        x[::2], r[::2] = 0, 0
        x[:, :128], r[:, :128] = 0, 0
    elif kind == "large":    # squares near 1e30, still finite in FP32
        x, r = x * 1e15, r * 1e15
    elif kind == "tiny":     # the mean square is far below eps
        x, r = x * 1e-20, r * 1e-20
    w = 1 + 0.2 * torch.randn(K, generator=g)
    return x.bfloat16(), r.bfloat16(), w.bfloat16()


def _check_codes(q, s, h):
    top = h.unflatten(-1, (-1, 128)).abs().amax(-1)
    want = torch.where(top == 0, torch.ones_like(top), top / 448)
    s = s.cpu().double()
    # 2^-149: half a step of a subnormal FP32 scale
    assert bool(((s - want).abs() <= 2.0 ** -18 * want + 2.0 ** -149).all())
    v = ref.e4m3_values(q).unflatten(-1, (-1, 128))
    assert bool((v.abs() <= 448).all())
    got, hg = v * s[..., None], h.unflatten(-1, (-1, 128))
    err = (got - hg).abs()
    ok = err <= torch.maximum(ref.HALF_E4M3 * hg.abs(), ref.E4M3_SUB * s[..., None]) + \
        2.0 ** -17 * hg.abs() + 448 * 2.0 ** -149
    assert bool(ok.all()), float((err / hg.abs().clamp(min=1e-30)).max())


@pytest.mark.parametrize("M,K,residual,kind", [
    (1, 128, True, "normal"), (1, 7168, True, "normal"), (3, 7168, False, "normal"),
    (17, 8320, True, "normal"), (5, 16512, True, "normal"), (2, 32768, True, "normal"),
    (700, 1024, True, "normal"), (5000, 256, False, "normal"), (6, 1152, True, "zero"),
    (6, 1152, False, "large"), (6, 1152, True, "tiny"), (333, 7168, True, "normal"),
    # both sides of the sizes at which rows are held by other numbers of threads
    (148, 8192, True, "normal"), (149, 8192, False, "normal"), (592, 2048, True, "normal"),
    (593, 2048, True, "normal"), (296, 4096, False, "normal"), (149, 4224, True, "normal"),
    (148, 8320, False, "normal"), (149, 8320, True, "normal"), (40, 16384, True, "normal")])
def test_norm_quantize(M, K, residual, kind):
    x, r, w = _norm_inputs(M, K, M + K, kind)
    xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
    q, s = Guarded((M, K), torch.uint8), Guarded((M, K // 128), torch.float32)
    h, ro = Guarded((M, K), torch.bfloat16), Guarded((M, K), torch.bfloat16)
    eps = 1e-5
    fp8bq.rms_norm_quantize(xd, wd, eps, residual=rd if residual else None,
                            residual_out=ro.t if residual else None, q=q.t, s=s.t, h=h.t)
    torch.cuda.synchronize()
    assert all(b.guards_intact() for b in (q, s, h, ro))
    stream, want = ref.rms_norm(x, w, eps, r if residual else None)
    if residual:
        assert torch.equal(ro.t.cpu().view(torch.int16), stream.view(torch.int16))
        assert torch.equal(rd.cpu().view(torch.int16), r.view(torch.int16))  # not in place here
    err = (h.t.cpu().double() - want).abs()
    assert bool((err <= (ref.HALF_BF16 + 2.0 ** -18) * want.abs() + 2.0 ** -133).all())
    _check_codes(q.t, s.t, want)


def test_norm_variants_agree():
    """In place of the residual or of x, codes only, BF16 only: the same bits."""
    x, r, w = _norm_inputs(37, 7168, 5)
    xd, rd, wd = x.cuda(), r.cuda(), w.cuda()
    h, ro = torch.empty_like(xd), torch.empty_like(xd)
    q, s = fp8bq.rms_norm_quantize(xd, wd, residual=rd, residual_out=ro, h=h)
    r2 = rd.clone()
    q2, s2 = fp8bq.rms_norm_quantize(xd, wd, residual=r2)
    x3, h3 = xd.clone(), None
    h3 = fp8bq.rms_norm(x3, wd, residual=rd, residual_out=x3)
    q4, s4 = fp8bq.rms_norm_quantize(ro, wd)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(r2, ro)
    assert torch.equal(h, h3) and torch.equal(x3, ro)
    assert torch.equal(q, q4) and torch.equal(s, s4)


def test_norm_feeds_the_gemm():
    """gemm on the norm's codes, against the 64-bit product of what they stand for."""
    from gpu_util import tolerance_report
    x, r, w = _norm_inputs(9, 1024, 6)
    g = torch.Generator().manual_seed(1)
    qw, sw = fp8bq.quantize_weight((0.02 * torch.randn(384, 1024, generator=g)).bfloat16().cuda())
    q, s = fp8bq.rms_norm_quantize(x.cuda(), w.cuda(), residual=r.cuda())
    y = fp8bq.gemm(q, s, qw, sw)
    a = ref.e4m3_values(q) * s.cpu().double().repeat_interleave(128, 1)
    b = ref.e4m3_values(qw) * sw.cpu().double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    ok, worst, _ = tolerance_report(y.cpu().double().numpy(), (a @ b.T).numpy())
    assert ok, worst


# ------------------------------------------------------------------ rotary positions

@pytest.mark.parametrize("T,hq,hk,dim,rot,inter,scaling,far", [
    (1, 56, 8, 128, 128, False, "yarn", 1000000), (5, 28, 4, 128, 64, True, "linear", 2 ** 31 - 9),
    (33, 7, 1, 64, 64, True, "ntk", 70000), (20, 8, 8, 256, 256, False, "plain", 1 << 20),
    (9, 12, 4, 64, 48, False, "plain", 5), (3, 2, 2, 16, 16, True, "plain", 100),
    (3000, 7, 1, 128, 112, False, "yarn", 300000), (2500, 2, 1, 256, 16, True, "plain", 4096)])
def test_rope(T, hq, hk, dim, rot, inter, scaling, far):
    g = torch.Generator().manual_seed(T + dim)
    cols, pad = (hq + 2 * hk) * dim, 8 * (T % 3)
    qkv = (3 * torch.randn(T, cols + pad, generator=g)).bfloat16()
    qkv[:, ::37] *= 100                                   # beyond 448: saturation
    pos = torch.randint(max(0, far - 5000), far, (T,), generator=g)
    freq, m = fp8bq.rope_inv_freq(rot, 1.2e8, scaling, factor=8.0, old_context=32768)
    slots = T + 5
    loc = torch.randperm(slots, generator=g)[:T]
    if T > 4:
        loc[2], loc[4] = -1, -1                           # padding tokens
    width = hk * dim + 16 * (T % 2)
    kc, vc = (Guarded((slots, width), torch.uint8, fill=0xA5) for _ in range(2))
    qo = Guarded((T, hq * dim), torch.bfloat16, fill=0x5A)
    d = qkv.cuda()
    fp8bq.rope_kv_write_e4m3(d[:, :cols], pos.cuda(), freq.cuda(), loc.cuda(), kc.t, vc.t,
                             head_dim=dim, kv_heads=hk, interleaved=inter, mscale=m, q_out=qo.t)
    torch.cuda.synchronize()
    assert kc.guards_intact() and vc.guards_intact() and qo.guards_intact()
    x = qkv[:, :cols].reshape(T, hq + 2 * hk, dim)
    y, size = ref.rope(x[:, :hq + hk], pos, freq, np.float32(m).item(), inter)
    live = loc >= 0
    q = qo.t.cpu().view(T, hq, dim)
    err = (q.double() - y[:, :hq]).abs()
    assert bool((err <= ref.HALF_BF16 * y[:, :hq].abs() + 2.0 ** -20 * size[:, :hq])[live].all())
    assert bool((q.view(torch.int16)[~live] == 0x5A5A).all())
    assert torch.equal(q[live][..., rot:], x[:, :hq][live][..., rot:])
    k_got = ref.e4m3_values(kc.t)[loc[live], :hk * dim].view(-1, hk, dim)
    k_want, k_size = y[:, hq:][live].clamp(-448, 448), size[:, hq:][live]
    err = (k_got - k_want).abs()
    assert bool((err <= torch.maximum(ref.HALF_E4M3 * k_want.abs(), torch.tensor(ref.E4M3_SUB)) +
                 2.0 ** -20 * k_size).all())
    v_want = x[:, hq + hk:][live].float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(vc.t.cpu()[loc[live], :hk * dim], v_want.reshape(-1, hk * dim))
    # slots no token has, and the bytes behind a slot's heads, stay
    other = torch.ones(slots, dtype=torch.bool)
    other[loc[live]] = False
    for c in (kc, vc):
        assert bool((c.t.cpu()[other] == 0xA5).all()) and bool((c.t.cpu()[:, hk * dim:] == 0xA5).all())


def test_rope_in_place_and_far_positions():
    """In place gives the same queries; position p and p + a whole number of turns agree."""
    T, hq, hk = 6, 4, 2
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(T, (hq + 2 * hk) * 128, generator=g).bfloat16().cuda()
    pos = torch.tensor([0, 1, -1, 999999, 2 ** 31 - 1, 12345]).cuda()
    freq = fp8bq.rope_inv_freq(128, 1e4, device="cuda")[0]
    loc = torch.arange(T).cuda()
    caches = [torch.zeros(T, hk * 128, dtype=torch.uint8, device="cuda") for _ in range(4)]
    q = fp8bq.rope_kv_write_e4m3(qkv, pos, freq, loc, *caches[:2])
    same = qkv.clone()
    fp8bq.rope_kv_write_e4m3(same, pos, freq, loc, *caches[2:], q_out=same[:, :hq * 128])
    assert torch.equal(same[:, :hq * 128], q) and torch.equal(same[:, hq * 128:], qkv[:, hq * 128:])
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    assert torch.equal(q[0], qkv[0, :hq * 128])            # position 0 turns nothing
    # a frequency of 2 pi rounded to FP32 turns by its rounding only, p times
    f = torch.full((64,), 2 * np.pi, dtype=torch.float32)
    p = torch.tensor([1 << 20] * T)
    q = fp8bq.rope_kv_write_e4m3(qkv, p.cuda(), f.cuda(), loc, *caches[:2])
    y, size = ref.rope(qkv.view(T, -1, 128)[:, :hq], p, f, 1.0, False)
    assert bool(((q.cpu().double().view(T, hq, 128) - y).abs() <= ref.HALF_BF16 * y.abs() + 2.0 ** -20 * size).all())


def test_rope_bad_slots_are_skipped_and_reported():
    qkv = torch.ones(4, 3 * 128).bfloat16().cuda()
    kc, vc = (torch.full((4, 128), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2))
    q = torch.full((4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    loc = torch.tensor([4, -2, 1 << 40, 2]).cuda()
    fp8bq.rope_kv_write_e4m3(qkv, torch.arange(4).cuda(), fp8bq.rope_inv_freq(128, 1e4, device="cuda")[0],
                             loc, kc, vc, q_out=q)
    assert fp8bq.last_device_status() == 8
    assert bool((kc[[0, 1, 3]] == 0xA5).all()) and bool((vc[[0, 1, 3]] == 0xA5).all())
    assert bool((vc[2] == 0x38).all()) and bool((q[:3] == 7).all()) and not bool((q[3] == 7).any())
