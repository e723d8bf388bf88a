"""A decoder layer through the library's own calls, as a serving step uses them: norm (+ residual)
with codes -> QKV GEMM -> rotary positions and cache write -> paged attention -> output
projection -> norm -> gate/up GEMM with the SiLU product -> down projection.  Every stage is checked
against 64 bits on the inputs that it was given; a captured decode step replays bit for bit."""
import numpy as np
import pytest
import torch

import fp8_block_scaled_09_b200 as fp8bq
import layer_ref as ref
from gpu_util import tolerance_report

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, MLP, PAGE = 1024, 7, 1, 512, 16


@pytest.fixture(scope="module", autouse=True)
def _device():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8bq.lib()
    yield
    assert fp8bq.last_device_status() == 0


class Layer:
    def __init__(self, max_tokens, batch, slots):
        g = torch.Generator().manual_seed(1)
        w = lambda n, k: fp8bq.quantize_weight((0.03 * torch.randn(n, k, generator=g)).bfloat16().cuda())
        self.qkv, self.o = w((HEADS + 2 * KV) * 128, HIDDEN), w(HIDDEN, HEADS * 128)
        self.gate_up, self.down = w(2 * MLP, HIDDEN), w(HIDDEN, MLP)
        self.n1, self.n2 = ((1 + 0.1 * torch.randn(HIDDEN, generator=g)).bfloat16().cuda() for _ in range(2))
        self.freq, self.m = fp8bq.rope_inv_freq(128, 1.2e8, "yarn", factor=4.0, old_context=4096, device="cuda")
        self.kc, self.vc = (torch.full((slots, KV * 128), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        sizes = [fp8bq.attention_workspace_size(t, b, HEADS, KV, t) for t, b in ((max_tokens, batch), (batch, batch), (1, 1))]
        for m in (1, batch, max_tokens):
            sizes += [fp8bq.workspace_size(op, m, n, k) for op in (fp8bq.OP_GEMM, fp8bq.OP_LINEAR, fp8bq.OP_GEMM_SILU)
                      for n, k in ((1152, HIDDEN), (HIDDEN, 896), (2 * MLP, HIDDEN), (HIDDEN, MLP))]
        self.ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")   # one for every call

    def step(self, x, residual, pos, loc, table, lens, cu, max_q):
        t = {"x": x, "residual_in": residual.clone()}
        t["q1"], t["s1"] = fp8bq.rms_norm_quantize(x, self.n1, residual=residual)
        t["residual1"] = residual.clone()
        t["qkv"] = fp8bq.gemm(t["q1"], t["s1"], *self.qkv, workspace=self.ws)
        t["q"] = fp8bq.rope_kv_write_e4m3(t["qkv"], pos, self.freq, loc, self.kc, self.vc, mscale=self.m)
        t["attn"] = fp8bq.paged_attention(t["q"], self.kc, self.vc, table, lens, cu, PAGE, HEADS, KV, max_q,
                                          workspace=self.ws)
        t["o"] = fp8bq.linear(t["attn"], *self.o, workspace=self.ws)
        t["q2"], t["s2"] = fp8bq.rms_norm_quantize(t["o"], self.n2, residual=residual)
        t["residual2"] = residual.clone()
        t["q3"], t["s3"] = fp8bq.gemm_silu_mul_quantize(t["q2"], t["s2"], *self.gate_up, workspace=self.ws)
        t["y"] = fp8bq.gemm(t["q3"], t["s3"], *self.down, workspace=self.ws)
        return t

    def check(self, t, pos, loc, table, lens, cu):
        deq_a = lambda q, s: ref.e4m3_values(q) * s.cpu().double().repeat_interleave(128, 1)
        deq_w = lambda w: ref.e4m3_values(w[0]) * w[1].cpu().double().repeat_interleave(128, 0).repeat_interleave(128, 1)

        def product(y, a, w):
            ok, worst, _ = tolerance_report(y.cpu().double().numpy(), (a @ deq_w(w).T).numpy())
            assert ok, worst

        def norm(x, res_in, res_out, q, s, w):
            r, h = ref.rms_norm(x, w, 1e-5, res_in)
            assert torch.equal(r.view(torch.int16), res_out.cpu().view(torch.int16))
            err = (deq_a(q, s) - h).abs().unflatten(-1, (-1, 128))
            top = h.unflatten(-1, (-1, 128)).abs().amax(-1, keepdim=True)
            assert bool((err <= torch.maximum(ref.HALF_E4M3 * h.unflatten(-1, (-1, 128)).abs(), top / 448 * ref.E4M3_SUB)
                         + 2.0 ** -17 * top).all())

        norm(t["x"], t["residual_in"], t["residual1"], t["q1"], t["s1"], self.n1)
        product(t["qkv"], deq_a(t["q1"], t["s1"]), self.qkv)
        n, qkv = t["q"].shape[0], t["qkv"].cpu().view(-1, HEADS + 2 * KV, 128)
        y, size = ref.rope(qkv[:, :HEADS + KV], pos, self.freq.cpu(), np.float32(self.m).item(), False)
        assert bool(((t["q"].cpu().double().view(n, HEADS, 128) - y[:, :HEADS]).abs() <=
                     ref.HALF_BF16 * y[:, :HEADS].abs() + 2.0 ** -20 * size[:, :HEADS]).all())
        k = ref.e4m3_values(self.kc)[loc.cpu()].view(n, KV, 128)
        assert bool(((k - y[:, HEADS:]).abs() <= torch.maximum(ref.HALF_E4M3 * y[:, HEADS:].abs(), torch.tensor(ref.E4M3_SUB))
                     + 2.0 ** -20 * size[:, HEADS:]).all())
        o, _, bound, _ = ref.attention(t["q"], self.kc, self.vc, table, lens, cu, PAGE, HEADS, KV, 128 ** -0.5, True)
        assert bool(((t["attn"].cpu().double().view(o.shape) - o).abs() <= bound).all())
        product(t["o"], deq_a(*fp8bq.quantize_act(t["attn"])), self.o)
        norm(t["o"], t["residual1"], t["residual2"], t["q2"], t["s2"], self.n2)
        q3, s3 = fp8bq.silu_mul_quantize(fp8bq.gemm(t["q2"], t["s2"], *self.gate_up))
        assert torch.equal(q3, t["q3"]) and torch.equal(s3, t["s3"])
        product(t["y"], deq_a(t["q3"], t["s3"]), self.down)


def test_prefill_then_decode():
    lens0 = [37, 150]
    layer = Layer(sum(lens0), 2, 40 * PAGE)
    g = torch.Generator().manual_seed(2)
    table = torch.randperm(40, generator=g)[:26].view(2, 13).int().cuda()
    slot = lambda b, p: table[b].long()[p // PAGE] * PAGE + p % PAGE
    x = torch.randn(sum(lens0), HIDDEN, generator=g).bfloat16().cuda()
    res = (2 * torch.randn(sum(lens0), HIDDEN, generator=g)).bfloat16().cuda()
    pos = torch.cat([torch.arange(n) for n in lens0]).cuda()
    loc = torch.cat([slot(b, torch.arange(n).cuda()) for b, n in enumerate(lens0)])
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    args = (pos, loc, table, i32(lens0), i32([0, lens0[0], sum(lens0)]))
    t = layer.step(x, res, *args, max(lens0))
    layer.check(t, *args)
    # decode: eager, then the same step captured and replayed for the next tokens
    x, res = torch.randn(2, HIDDEN, generator=g).bfloat16().cuda(), torch.randn(2, HIDDEN, generator=g).bfloat16().cuda()
    lens, cu = i32([n + 1 for n in lens0]), i32([0, 1, 2])
    pos = torch.tensor(lens0).cuda()
    loc = torch.stack([slot(b, pos[b]) for b in range(2)])
    first_res = res.clone()
    t = layer.step(x, res, pos, loc, table, lens, cu, 1)
    layer.check(t, pos, loc, table, lens, cu)
    eager = {k: v.clone() for k, v in t.items()}
    res.copy_(first_res)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t = layer.step(x, res, pos, loc, table, lens, cu, 1)
    for _ in range(2):
        res.copy_(first_res)
        graph.replay()
    torch.cuda.synchronize()
    for k in eager:
        assert torch.equal(eager[k].view(torch.uint8), t[k].view(torch.uint8)), k
    for step in range(1, 12):            # over a page's end
        x.copy_(torch.randn(2, HIDDEN, generator=g).bfloat16())
        pos.add_(1)
        lens.add_(1)
        loc.copy_(torch.stack([slot(b, pos[b]) for b in range(2)]))
        graph.replay()
        layer.check(t, pos, loc, table, lens, cu)


def test_two_streams_at_once():
    """Attention on two streams with a workspace each, many times over: the same bits as alone."""
    cases = [(ref.random_batch([1] * 6, [900, 20, 3000, 0, 77, 1500], 56, 8, 16, 1), 1),
             (ref.random_batch([30, 90], [30, 1000], 56, 8, 16, 2), 90)]
    runs = []
    for c, n in cases:
        d = {k: v.cuda() for k, v in c.items()}
        ws = fp8bq.new_attention_workspace(d["q"].shape[0], d["seq_lens"].numel(), 56, 8, n, "cuda")
        call = lambda d=d, n=n, ws=ws: fp8bq.paged_attention(
            d["q"], d["k_cache"], d["v_cache"], d["page_table"], d["seq_lens"], d["cu_q"], 16, 56, 8, n, workspace=ws)
        runs.append((call, call()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    outs = [[], []]
    for _ in range(20):
        for i, (call, _) in enumerate(runs):
            with torch.cuda.stream(streams[i]):
                outs[i].append(call())
    torch.cuda.synchronize()
    for (_, alone), got in zip(runs, outs):
        assert all(torch.equal(alone, o) for o in got)


def test_binding_refuses_wrong_tensors():
    """Types, shapes, layouts and devices that do not fit are refused before anything runs."""
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    x, w = b(4, 256), b(256)
    before = fp8bq.launch_count()
    for bad in (dict(x=x.float()), dict(x=x[0]), dict(x=b(4, 512)[:, ::2]), dict(w=b(128)), dict(w=w.cpu()),
                dict(residual=b(3, 256)), dict(residual_out=x), dict(residual=x, residual_out=b(4, 128)),
                dict(q=torch.zeros(4, 256, device="cuda")), dict(s=torch.zeros(4, 3, device="cuda")), dict(h=b(4, 255))):
        a = {"x": x, "w": w, **bad}
        with pytest.raises((TypeError, ValueError)):
            fp8bq.rms_norm_quantize(a.pop("x"), a.pop("w"), **a)
    i64 = torch.arange(4, device="cuda")
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
    good = dict(qkv=b(4, 3 * 128), positions=i64, inv_freq=torch.ones(64, device="cuda"), loc=i64, k_cache=u8(8, 128), v_cache=u8(8, 128))
    for bad in (dict(qkv=b(4, 100)), dict(qkv=b(4, 2 * 128)), dict(positions=i64.int()), dict(positions=i64[:3]),
                dict(loc=i64.cpu()), dict(inv_freq=torch.ones(2, 32, device="cuda")), dict(v_cache=u8(7, 128)),
                dict(k_cache=u8(8 * 128)), dict(q_out=b(4, 256)), dict(q_out=b(128, 4).T), dict(head_dim=0)):
        with pytest.raises((TypeError, ValueError)):
            fp8bq.rope_kv_write_e4m3(**{**good, **bad})
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    good = dict(q=b(2, 256), k_cache=u8(32, 128), v_cache=u8(32, 128), page_table=i32([0, 1], [1, 0]), seq_lens=i32(5, 6),
                cu_q=i32(0, 1, 2), page_size=16, q_heads=2, kv_heads=1, max_q_len=1)
    for bad in (dict(q=b(2, 128)), dict(q=b(256, 2).T), dict(seq_lens=i32(5)), dict(cu_q=i32(0, 1)), dict(cu_q=torch.arange(3, device="cuda")),
                dict(page_table=i32(0, 1)), dict(page_table=i32([0, 1], [1, 0]).T.contiguous().T), dict(v_cache=u8(16, 128)),
                dict(out=b(2, 255)), dict(lse=b(2, 2)), dict(lse=torch.zeros(2, 1, device="cuda")), dict(workspace=b(1 << 22)),
                dict(page_size=24), dict(q_heads=3, q=b(2, 384), kv_heads=2), dict(max_q_len=0), dict(scale=0.0),
                dict(workspace=u8(256))):
        with pytest.raises((TypeError, ValueError, fp8bq.Fp8bqError)):
            fp8bq.paged_attention(**{**good, **bad})
    assert fp8bq.launch_count() == before
    fp8bq.paged_attention(**good)
    assert fp8bq.launch_count() == before + 1
