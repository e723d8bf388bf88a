"""The attention's workspace: only its counters are cleared, and nothing else in it is read before it
is written."""
import re
import os

import pytest
import torch

import fp8_block_scaled_09_b200 as fp8bq
from fp8_block_scaled_09_b200 import build as fp8bq_build


@pytest.mark.parametrize("T,B,hq,hk,n", [(1, 1, 7, 1, 1), (16, 8, 56, 8, 2), (300, 2, 56, 8, 200)])
def test_only_the_counters_are_cleared(monkeypatch, T, B, hq, hk, n):
    fp8bq_build.build()
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).fill_(0x5A))
    ws = fp8bq.new_attention_workspace(T, B, hq, hk, n, "cpu")
    assert ws.numel() == fp8bq.attention_workspace_size(T, B, hq, hk, n) > fp8bq.WORKSPACE_HEADER
    assert bool((ws[:fp8bq.WORKSPACE_HEADER] == 0).all()) and bool((ws[fp8bq.WORKSPACE_HEADER:] == 0x5A).all())


def test_the_header_is_the_library_s():
    with open(os.path.join(fp8bq_build.CSRC, "gemm_decode.cuh")) as f:
        counters = int(re.search(r"kMaxCounters = (\d+);", f.read()).group(1))
    assert fp8bq.WORKSPACE_HEADER == 4 * counters


@pytest.mark.gpu
@pytest.mark.parametrize("q_lens,ctx,heads", [([1], [9000], (7, 1)), ([1, 2], [3000, 5000], (8, 1)), ([9], [6000], (7, 1)),
                                              ([200, 1], [5000, 4000], (8, 2)), ([100, 3], [100, 0], (7, 1))])
def test_what_the_memory_held_before_does_not_matter(q_lens, ctx, heads):
    """Calls whose partial results go through a workspace of NaN, and calls that make their own: the bits of a
    call with a workspace of zeros."""
    import layer_ref as ref
    c = {k: v.cuda() for k, v in ref.random_batch(q_lens, ctx, *heads, 16, 3).items()}
    size = fp8bq.attention_workspace_size(sum(q_lens), len(ctx), *heads, max(q_lens))
    call = lambda ws: fp8bq.paged_attention(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["seq_lens"], c["cu_q"],
                                            16, *heads, max(q_lens), workspace=ws)
    want = call(torch.zeros(size, dtype=torch.uint8, device="cuda"))
    dirty = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    dirty[:fp8bq.WORKSPACE_HEADER] = 0
    assert torch.equal(call(dirty), want)
    del dirty
    for _ in range(3):
        torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")       # freed at once: the next one's memory
        assert torch.equal(call(None), want)
    assert fp8bq.last_device_status() == 0
