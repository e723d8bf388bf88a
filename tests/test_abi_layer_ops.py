"""Host-side checks of the norm, rotary and attention entry points (no kernel is launched),
and of the rotary frequency tables against their 64-bit formulas."""
import ctypes
import math

import numpy as np
import pytest
import torch

import fp8_block_scaled_09_b200 as fp8bq
from fp8_block_scaled_09_b200 import build as fp8bq_build

OK, INVALID, SHAPE, MISALIGNED, WORKSPACE = range(5)
P = ctypes.c_void_p
GOOD, ODD = P(0x10000), P(0x10008)   # fake; ODD is not 16-byte aligned
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    fp8bq_build.build()
    return fp8bq.lib()


def test_norm_argument_errors(L):
    def f(x=GOOD, r=GOOD, w=GOOD, eps=1e-5, M=4, K=256, ro=GOOD, q=GOOD, s=GOOD, h=None):
        return L.fp8bq_rms_norm_quantize(x, r, w, eps, M, K, ro, q, s, h, None)
    assert f(K=100) == SHAPE and f(K=0) == SHAPE and f(M=-1) == SHAPE and f(K=32768 + 128) == SHAPE
    assert f(M=1 << 40) == SHAPE
    assert f(eps=-1.0) == INVALID and f(eps=NAN) == INVALID and f(eps=INF) == INVALID
    assert f(q=None) == INVALID and f(s=None) == INVALID            # codes without scales
    assert f(q=None, s=None) == INVALID                              # no output at all
    assert f(ro=None) == INVALID and f(r=None) == INVALID
    assert f(x=None) == INVALID and f(w=None) == INVALID
    for name in ("x", "r", "w", "ro", "q", "s", "h"):
        assert f(**{name: ODD}) == MISALIGNED, name
    assert f(M=0, x=None, w=None) == OK


def test_rope_argument_errors(L):
    def f(x=GOOD, rs=1024, T=4, hq=4, hk=2, d=128, pos=GOOD, fr=GOOD, rot=128, m=1.0, loc=GOOD,
          qo=P(0x20000), qs=512, kc=GOOD, vc=GOOD, slots=8, ss=256):
        return L.fp8bq_rope_kv_write_e4m3(x, rs, T, hq, hk, d, pos, fr, rot, 0, m, loc, qo, qs, kc, vc,
                                          slots, ss, None)
    assert f(T=-1) == INVALID and f(hq=0) == INVALID and f(hk=0) == INVALID and f(slots=-1) == INVALID
    assert f(m=NAN) == INVALID and f(m=INF) == INVALID
    assert f(d=120) == SHAPE and f(d=272) == SHAPE and f(rot=144) == SHAPE and f(rot=24) == SHAPE
    assert f(rot=0) == SHAPE and f(hq=1025, rs=1 << 20, qs=1 << 19) == SHAPE
    assert f(rs=1016) == INVALID and f(qs=504) == INVALID and f(ss=240) == INVALID
    assert f(rs=1028) == SHAPE and f(qs=516) == SHAPE and f(ss=264) == SHAPE
    assert f(slots=1 << 40) == SHAPE
    for name in ("x", "pos", "fr", "loc", "qo", "kc", "vc"):
        assert f(**{name: None}) == INVALID, name
    for name in ("x", "qo", "kc", "vc"):
        assert f(**{name: ODD}) == MISALIGNED, name
    assert f(pos=P(0x10004)) == MISALIGNED and f(loc=P(0x10004)) == MISALIGNED and f(fr=P(0x10002)) == MISALIGNED
    assert f(qo=GOOD) == INVALID                                     # in place with another stride
    assert f(T=0, x=None) == OK


def test_attention_argument_errors(L):
    def f(q=GOOD, qs=512, kc=GOOD, vc=GOOD, slots=64, ss=256, tb=GOOD, ts=4, mp=4, page=16, sl=GOOD,
          cu=GOOD, B=2, T=4, hq=4, hk=2, mq=2, scale=0.1, out=GOOD, os=512, lse=None, ws=GOOD, n=1 << 30):
        return L.fp8bq_paged_attention(q, qs, kc, vc, slots, ss, tb, ts, mp, page, sl, cu, B, T, hq, hk,
                                       mq, scale, 1, out, os, lse, ws, n, None)
    assert f(T=-1) == INVALID and f(B=-1) == INVALID and f(hq=0) == INVALID and f(hk=0) == INVALID
    assert f(mq=0) == INVALID and f(mq=-1) == INVALID and f(slots=-1) == INVALID and f(mp=-1) == INVALID
    assert f(hq=5) == SHAPE and f(hq=2048, hk=2, qs=1 << 18, os=1 << 18) == SHAPE
    assert f(B=65537) == SHAPE and f(T=1 << 21) == SHAPE
    assert f(ts=3) == INVALID
    for s in (0.0, -1.0, NAN, INF):
        assert f(scale=s) == INVALID
    for p in (0, 1, 4, 12, 24, 48, 1 << 21, -16):
        assert f(page=p) == SHAPE, p
    assert f(mp=(1 << 21) + 1, ts=1 << 22) == SHAPE                  # beyond 2^25 positions
    assert f(qs=504) == INVALID and f(os=504) == INVALID and f(ss=240) == INVALID
    assert f(qs=516) == SHAPE and f(os=516) == SHAPE and f(ss=264) == SHAPE
    assert f(slots=1 << 31) == SHAPE
    for name in ("q", "kc", "vc", "tb", "sl", "cu", "out"):
        assert f(**{name: None}) == INVALID, name
    for name in ("q", "kc", "vc", "out"):
        assert f(**{name: ODD}) == MISALIGNED, name
    for name in ("tb", "sl", "cu", "lse"):
        assert f(**{name: P(0x10002)}) == MISALIGNED, name
    assert f(T=0, q=None) == OK and f(B=0, q=None, mq=0) == OK
    need = fp8bq.attention_workspace_size(4, 2, 4, 2, 2)
    assert need % 256 == 0
    if need:
        assert f(ws=None) == WORKSPACE and f(n=need - 1) == WORKSPACE and f(ws=ODD) == MISALIGNED
    assert fp8bq.attention_workspace_size(4, 2, 5, 2, 2) == 0 and fp8bq.attention_workspace_size(0, 2, 4, 2, 2) == 0


def test_rope_inv_freq_tables(L):
    i = np.arange(64)
    plain, m = fp8bq.rope_inv_freq(128, 1.2e8)
    assert m == 1.0 and np.array_equal(plain.numpy(), (1.2e8 ** (-2.0 * i / 128)).astype(np.float32))
    lin, m = fp8bq.rope_inv_freq(128, 1e4, "linear", factor=4.0)
    assert m == 1.0 and np.allclose(lin.numpy(), 1e4 ** (-2.0 * i / 128) / 4, rtol=2 ** -23)
    ntk, m = fp8bq.rope_inv_freq(128, 1e4, "ntk", factor=8.0)
    # the slowest pair is slowed by exactly the factor, the fastest not at all
    assert m == 1.0 and ntk[0] == 1.0 and math.isclose(ntk[-1].item(), 1e4 ** (-126 / 128) / 8, rel_tol=2 ** -22)
    yarn, m = fp8bq.rope_inv_freq(128, 1e4, "yarn", factor=8.0, old_context=4096)
    f = 1e4 ** (-2.0 * i / 128)
    turns = 4096 * f / (2 * math.pi)
    assert math.isclose(m, 0.1 * math.log(8) + 1, rel_tol=2 ** -23)
    assert np.allclose(yarn.numpy()[turns >= 32], f[turns >= 32], rtol=2 ** -23)
    assert np.allclose(yarn.numpy()[turns <= 1], f[turns <= 1] / 8, rtol=2 ** -23)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((yarn.numpy() < f) & (yarn.numpy() > f / 8))[mid].all()
    assert fp8bq.rope_inv_freq(2, 1e4, "ntk", factor=2.0)[0].tolist() == [1.0]


def test_rope_inv_freq_refusals(L):
    ok = dict(rot_dim=128, base=1e4)
    for bad in (dict(rot_dim=0), dict(rot_dim=127), dict(base=1.0), dict(base=NAN), dict(base=INF),
                dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=NAN),
                dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, old_context=NAN),
                dict(scaling="yarn", factor=2.0, old_context=4096, beta_fast=1.0),
                dict(scaling="yarn", factor=2.0, old_context=4096, beta_slow=0.0)):
        with pytest.raises(fp8bq.Fp8bqError):
            fp8bq.rope_inv_freq(**{**ok, **bad})
    with pytest.raises(ValueError):
        fp8bq.rope_inv_freq(128, 1e4, "other")


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    c = torch.zeros(16, 128, dtype=torch.uint8)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fp8bq.rms_norm_quantize(x, w)
    with pytest.raises(ValueError):
        fp8bq.rms_norm(x, w)
    with pytest.raises(ValueError):
        fp8bq.rope_kv_write_e4m3(x, i.long(), w.float(), i.long(), c, c)
    with pytest.raises(ValueError):
        fp8bq.paged_attention(x, c, c, i[:, None], i, torch.zeros(3, dtype=torch.int32), 16, 2, 1, 1)
