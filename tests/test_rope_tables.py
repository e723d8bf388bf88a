"""Whole YaRN frequency tables against a restatement of the published recipe (correction range rounded
to whole pairs, linear ramp over the pairs) and of its form without the rounding."""
import math

import numpy as np
import pytest

import fp8_block_scaled_09_b200 as fp8bq
from fp8_block_scaled_09_b200 import build as fp8bq_build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    fp8bq_build.build()


def recipe(dim, base, factor, old, fast, slow, rounded):
    def at(turns):
        return dim * math.log(old / (turns * 2 * math.pi)) / (2 * math.log(base))
    low, high = at(fast), at(slow)
    if rounded:
        low, high = max(math.floor(low), 0), min(math.ceil(high), dim - 1)
        if low == high:
            high += 0.001
    i = np.arange(dim // 2, dtype=np.float64)
    ramp = np.clip((i - low) / (high - low), 0, 1)
    f = 1.0 / base ** (2 * i / dim)
    return f / factor * ramp + f * (1 - ramp)


CASES = [(128, 1e4, 8.0, 4096, 32.0, 1.0), (128, 1.2e8, 8.0, 32768, 32.0, 1.0), (64, 1e4, 4.0, 2048, 32.0, 1.0),
         (256, 1e6, 16.0, 8192, 32.0, 1.0), (128, 5e5, 40.0, 4096, 64.0, 2.0), (16, 1e4, 2.0, 4096, 32.0, 1.0),
         (32, 150.0, 4.0, 8192, 32.0, 1.0),     # the upper end lies behind the last pair
         (64, 1e4, 4.0, 64, 32.0, 1.0),         # the lower end before the first
         (16, 1e9, 4.0, 4096, 2.2, 2.1)]        # both within one pair


@pytest.mark.parametrize("dim,base,factor,old,fast,slow", CASES)
@pytest.mark.parametrize("rounded", [True, False])
def test_yarn_table(dim, base, factor, old, fast, slow, rounded):
    f, m = fp8bq.rope_inv_freq(dim, base, "yarn" if rounded else "yarn_exact", factor=factor, old_context=old,
                               beta_fast=fast, beta_slow=slow)
    want = recipe(dim, base, factor, old, fast, slow, rounded)
    # FP32 storage, half a step, and a few 64-bit roundings
    assert np.all(np.abs(f.numpy() - want) <= (2.0 ** -24 + 2.0 ** -44) * want)
    assert math.isclose(m, 0.1 * math.log(factor) + 1, rel_tol=2.0 ** -23)


def test_the_two_ramps_differ():
    """At 128 channels, base 10^4, factor 8 and an old context of 4096 the ends are pairs 20.94 and 45.03, rounded
    to 20 and 46."""
    a, b = (fp8bq.rope_inv_freq(128, 1e4, s, factor=8.0, old_context=4096)[0].numpy() for s in ("yarn", "yarn_exact"))
    same = a == b
    assert same[:21].all() and same[46:].all() and not same[22:45].any()
    assert 0.2 < np.abs(b / a - 1).max() < 0.21


def test_refusals():
    for scaling in ("yarn", "yarn_exact"):
        for bad in (dict(), dict(old_context=float("inf")), dict(old_context=4096, beta_fast=1.0), dict(old_context=4096, beta_slow=0.0),
                    dict(old_context=4096, factor=0.5)):
            with pytest.raises(fp8bq.Fp8bqError):
                fp8bq.rope_inv_freq(128, 1e4, scaling, **{"factor": 2.0, **bad})
    import ctypes
    f, m = (ctypes.c_float * 64)(), ctypes.c_float()
    for scaling in (-1, 5):
        assert fp8bq.lib().fp8bq_rope_inv_freq(128, 1e4, scaling, 2.0, 4096.0, 32.0, 1.0, f, ctypes.byref(m)) == 1
