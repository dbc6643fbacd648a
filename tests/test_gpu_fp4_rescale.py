"""Decode over a 4-bit cache at wide logit ranges: the inputs of test_gpu_rescale.py,
where the softmax reference moves after a split's first tile and the output so far is
rescaled, on the tcgen05 kernel (one, and several, query tokens in a group of rows)
and on the few-row kernel.  The gains go to the token scales, so the references of
both kernels move: the scores' maximum, and the few-row kernel's maximum of score and
scale.  Bar: 1e-2 of max|oracle|, the f16 query's 1e-3 to 2e-3 at these ranges
among it.

And two bars that a usual range allows, on the same kernels: the rms error of a step,
which is the bf16 output's own rounding and little else, and the log-sum-exp."""
import numpy as np
import pytest

from latent_compressed_attention_mla_b200 import binding as B
from latent_compressed_attention_mla_b200 import workloads as W
from oracle import mla_oracle as O
from tests.gpu_harness import GpuProblem, OracleProblem, rel_err
from tests.test_gpu_rescale import check_inputs, gain_fn

pytestmark = pytest.mark.gpu


def path_of(heads, T):
    return 2 if heads * T <= 16 else 1


def cfg_of(heads, T, L, seed):
    return W.V3_B1_L4096.with_(name="wide-fp4", cache_dtype="fp4", n_heads=heads, B=len(L), T=T, L=tuple(L), seed=seed)


def cache_of(o, gp, b):
    """History of the oracle, and the step's rows as the device holds them."""
    C0, KR0 = o.history(b)
    idx = gp.seq_idx == b
    c, kr = gp.cache.values(gp.seq_idx[idx].contiguous(), gp.pos[idx].contiguous(), gp.page_table)
    return np.concatenate([C0, c.double().cpu().numpy()]), np.concatenate([KR0, kr.double().cpu().numpy()])


CASES = [(p, h, t, s) for p in ("late-jump", "descending", "spread") for h in (8, 40, 64, 128) for t in (1, 2)
         for s in (1, 3)]


@pytest.mark.parametrize("pattern,heads,T,splits", CASES, ids=[f"{p}-h{h}-t{t}-w{s}" for p, h, t, s in CASES])
def test_wide_logits_match_oracle(pattern, heads, T, splits):
    cfg = cfg_of(heads, T, (1500, 2300), 70 + 7 * splits + T + len(pattern) + heads)
    gain = gain_fn(cfg, splits, pattern)
    o = OracleProblem(cfg, row_gain=gain)
    check_inputs(o, cfg, splits, pattern)
    gp = GpuProblem(cfg, num_splits=splits, row_gain=gain)
    assert B.decode_path(gp.dims, T) == path_of(heads, T)
    out, lse = gp.run()
    assert gp.status() == 0
    for b in range(cfg.B):
        ref, ref_lse = o.expected_absorbed(b, cache=cache_of(o, gp, b))
        assert rel_err(out[b].double().cpu().numpy(), ref) <= 1e-2, b
        assert rel_err(lse[b].double().cpu().numpy(), ref_lse) <= 1e-2, b


# Rounding to bf16 has an rms of 2^-7 / sqrt(12) of the value's power of two, 1.66e-3
# of the value over values of any magnitude.  The rotated query's bf16 adds
# 1.66e-3 x 0.577 (the rms of the scores' rotary part in nats) = 0.96e-3, the f16 of
# q~, P and the partials 0.2e-3 each: 1.95e-3.  With the latent sum rounded to bf16
# before W_uv, or bf16 partials, another 1.66e-3: 2.56e-3.
RMS_BAR = 2.2e-3
# An error of a score, 1.0e-3 nats rms (the two query roundings), enters lse as the
# mean over the keys, at 300 flat ones (effective 70 or so) 1.2e-4, and through the tilt
# of the softmax scale x |q^R| / 8 x 1e-3, as much again; five of both, rounded up,
# is 1.5e-3, where one key more or less in 400 is 2.5e-3.
LSE_BAR = 1.5e-3


@pytest.mark.parametrize("heads,T", [(8, 1), (16, 1), (40, 2), (64, 1), (128, 1), (128, 2)])
def test_error_is_that_of_the_output_rounding(heads, T):
    cfg = cfg_of(heads, T, (300, 330, 360, 390), 5)
    gp = GpuProblem(cfg)
    assert B.decode_path(gp.dims, T) == path_of(heads, T)
    out, lse = gp.run()
    assert gp.status() == 0
    o = OracleProblem(cfg)
    refs = [o.expected_absorbed(b, cache=cache_of(o, gp, b)) for b in range(cfg.B)]
    ref = np.stack([r[0] for r in refs])
    err = out.double().cpu().numpy() - ref
    assert np.sqrt((err ** 2).mean() / (ref ** 2).mean()) <= RMS_BAR
    assert np.abs(lse.double().cpu().numpy() - np.stack([r[1] for r in refs])).max() <= LSE_BAR
