"""The first call of a process may stand inside a stream capture: each entry in a process of its own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import sys, torch
sys.path.insert(0, {root!r})
import fp8_block_scaled_09_b200 as fp8bq
b = lambda *s: torch.randn(*s, device="cuda").bfloat16()
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
kc, vc = (torch.zeros(64, 128, dtype=torch.uint8, device="cuda") for _ in range(2))
ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
x, w = b(4, 256), b(256)
qkv, q = b(4, 9 * 128), b(4, 7 * 128)
pos, freq = torch.arange(4, device="cuda"), torch.ones(64, device="cuda")
table, lens, cu1, cu4 = i32([0, 1]), i32(20), i32(0, 1), i32(0, 4)
qw, sw = torch.full((256, 256), 0x30, dtype=torch.uint8, device="cuda"), torch.ones(2, 2, device="cuda")
calls = dict(
    norm=lambda: fp8bq.rms_norm(x, w),
    norm_codes=lambda: fp8bq.rms_norm_quantize(x, w)[0],
    rope=lambda: fp8bq.rope_kv_write_e4m3(qkv, pos, freq, pos, kc, vc),
    attention_few=lambda: fp8bq.paged_attention(q[:1], kc, vc, table.view(1, 2), lens, cu1, 16, 7, 1, 1, workspace=ws),
    attention_many=lambda: fp8bq.paged_attention(q, kc, vc, table.view(1, 2), lens, cu4, 16, 7, 1, 4, workspace=ws),
    attention_own=lambda: fp8bq.paged_attention(q, kc, vc, table.view(1, 2), lens, cu4, 16, 7, 1, 4),
    linear=lambda: fp8bq.linear(x, qw, sw, workspace=ws),
)
call = calls[{name!r}]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = call()
for _ in range(2):
    g.replay()
torch.cuda.synchronize()
assert torch.equal(y.view(torch.uint8), call().view(torch.uint8))
assert fp8bq.last_device_status() == 0
print("same")
"""


@pytest.mark.parametrize("name", ["norm", "norm_codes", "rope", "attention_few", "attention_many", "attention_own", "linear"])
def test_first_call_inside_a_capture(name):
    r = subprocess.run([sys.executable, "-c", SETUP.format(root=ROOT, name=name)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]
