"""The row gains of the GPU tests scale the latent values of the rows they name, by
exactly their power of two, for every cache type (CPU)."""
import numpy as np
import pytest

from latent_compressed_attention_mla_b200 import workloads as W
from tests.gpu_harness import OracleProblem


@pytest.mark.parametrize("cache", ["f32", "bf16", "fp8", "fp4"])
def test_gains_scale_the_latent_of_their_rows(cache):
    base = W.TINY_F32 if cache == "f32" else W.V3_FP8_B128_T2.with_(n_heads=2, cache_dtype=cache)
    cfg = base.with_(B=1, T=1, L=(40,), name="gains")

    def gain(b, pos):
        return np.ldexp(1.0, pos % 7 - 3)

    c0, k0 = OracleProblem(cfg).history(0)
    c1, k1 = OracleProblem(cfg, row_gain=gain).history(0)
    assert np.isfinite(c0).all() and np.abs(c0).max() > 0
    assert np.array_equal(c1, c0 * gain(0, np.arange(40))[:, None])
    assert np.array_equal(k1, k0)
