"""Rows of the cache that are not finite.  A query that sees such a row answers
NaN (output and log-sum-exp), whatever the number of splits; every other query's
result is the one without it, bit for bit."""
import numpy as np
import pytest
import torch

from latent_compressed_attention_mla_b200 import binding as B
from latent_compressed_attention_mla_b200 import workloads as W
from tests.gpu_harness import GpuProblem

pytestmark = pytest.mark.gpu

# (cache type, heads, flags); f32: the tiny dims with fp32 activations
DECODES = [("f32", 4, 0), ("bf16", 16, 0), ("bf16", 128, 0), ("fp8", 128, 0), ("fp4", 8, 0), ("fp4", 40, 0),
           ("fp4", 64, 0), ("fp4", 128, 0), ("fp4", 16, B.MLA_FLAG_FORCE_SIMT)]
IDS = [f"{c}-h{h}" + ("-simt" if f else "") for c, h, f in DECODES]


def make(cache, heads, flags, T, L, splits=0):
    base = W.TINY_F32 if cache == "f32" else W.V3_FP8_B128_T2.with_(cache_dtype=cache)
    cfg = base.with_(n_heads=heads, B=len(L), T=T, L=tuple(L), name=f"nonfinite-{cache}-{heads}")
    return cfg, GpuProblem(cfg, flags=flags, num_splits=splits)


def overwrite(gp, b, pos, value, where):
    """Row (b, pos) anew through the append of projected rows, with one element
    of c ("c") or of k^R ("kr") that is not finite."""
    d = gp.dims
    act = B.act_dtype(d)
    c = W.normal(31, 1, d.d_c).view(1, -1).to(act).cuda()
    kr = W.normal(31, 2, d.d_rope).view(1, -1).to(act).cuda()
    (c if where == "c" else kr)[0, 7] = value
    at = torch.tensor([b], dtype=torch.int32, device="cuda"), torch.tensor([pos], dtype=torch.int32, device="cuda")
    gp.cache.append(c, kr, *at, gp.page_table)


@pytest.mark.parametrize("splits", [0, 1, 7])
@pytest.mark.parametrize("cache,heads,flags", DECODES, ids=IDS)
def test_a_visible_row_makes_its_sequence_nan(cache, heads, flags, splits):
    cfg, gp = make(cache, heads, flags, 2, (300, 3000, 65), splits)
    out, lse = gp.run()
    ref, ref_lse = out.clone(), lse.clone()
    overwrite(gp, 1, 1777, float("nan"), "c")
    out, lse = gp.attend_only()
    for b in (0, 2):
        assert torch.equal(out[b], ref[b]) and torch.equal(lse[b], ref_lse[b])
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert torch.isfinite(ref.float()).all() and gp.status() == 0


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
def test_a_visible_row_makes_the_prefill_nan(cache):
    cfg, gp = make(cache, 2, 0, 100, (130,))
    append(gp)
    overwrite(gp, 0, 77, float("nan"), "c")
    out, lse = prefill(cfg, gp)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def append(gp):
    gp.session.append(gp.inputs["h"], gp.seq_idx, gp.pos, gp.weights["W_dkv"], gp.weights["W_kr"], gp.page_table,
                      gp.cache.pool)


def prefill(cfg, gp):
    i = gp.inputs
    out, lse = gp.session.prefill(i["q_nope"], i["q_rope"], gp.weights["W_uk"], gp.weights["W_uv"], gp.cache.pool,
                                  gp.page_table, gp.seq_lens, int(cfg.seq_lens.max()))
    torch.cuda.synchronize()
    return out.clone(), lse.clone()


@pytest.mark.parametrize("where,value", [("c", float("nan")), ("c", float("inf")), ("kr", float("nan"))])
@pytest.mark.parametrize("T", [2, 3])
@pytest.mark.parametrize("cache,heads,flags", DECODES, ids=IDS)
def test_a_hidden_row_does_not_reach_earlier_queries(cache, heads, flags, T, where, value):
    """The last of the new tokens is not finite: the queries before it do not see it
    (it is alone in its page, or in its tile of pages, in some of the sequences)."""
    cfg, gp = make(cache, heads, flags, T, (63 - T, 700, 2, 65 - T, 129 - T, 257 - T))
    out, lse = gp.run()
    ref, ref_lse = out.clone(), lse.clone()
    for b in range(cfg.B):
        overwrite(gp, b, int(cfg.seq_lens[b]) - 1, value, where)
    out, lse = gp.attend_only()
    assert torch.equal(out[:, :-1], ref[:, :-1]) and torch.equal(lse[:, :-1], ref_lse[:, :-1])
    assert torch.isnan(out[:, -1]).all()
    if np.isnan(value) or cache in ("fp8", "fp4"):  # (an infinite score can be the lowest one)
        assert torch.isnan(lse[:, -1]).all()
    assert torch.isfinite(ref.float()).all() and gp.status() == 0


@pytest.mark.parametrize("where", ["c", "kr"])
@pytest.mark.parametrize("L,T,pos", [(0, 200, 150), (70, 129, 70), (70, 129, 198), (300, 1, 300)])
@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
def test_prefill_queries_before_the_row_do_not_see_it(cache, L, T, pos, where):
    cfg, gp = make(cache, 3, 0, T, (L,))
    append(gp)
    overwrite(gp, 0, pos, 1.0, where)
    ref, ref_lse = prefill(cfg, gp)
    overwrite(gp, 0, pos, float("nan"), where)
    out, lse = prefill(cfg, gp)
    n = pos - L  # queries before it
    assert torch.equal(out[:, :n], ref[:, :n]) and torch.equal(lse[:, :n], ref_lse[:, :n])
    assert torch.isnan(out[:, n:]).all() and torch.isnan(lse[:, n:]).all()
    assert torch.isfinite(ref.float()).all() and gp.status() == 0


@pytest.mark.parametrize("cache,heads", [("bf16", 128), ("fp8", 128), ("fp4", 128), ("fp4", 40), ("fp4", 8)])
@pytest.mark.parametrize("batch,T", [(12, 2), (40, 2), (40, 1)])
def test_rows_in_a_large_batch(cache, heads, batch, T):
    """Every block size of the combine: only the sequences with such a row are NaN."""
    cfg, gp = make(cache, heads, 0, T, [60 + 37 * i for i in range(batch)])
    out, lse = gp.run()
    ref, ref_lse = out.clone(), lse.clone()
    bad = [1, 7, batch - 1]
    for b in bad:
        overwrite(gp, b, 20 * b, float("nan"), "kr" if b == 7 else "c")
    out, lse = gp.attend_only()
    for b in range(batch):
        if b in bad:
            assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()
        else:
            assert torch.equal(out[b], ref[b]) and torch.equal(lse[b], ref_lse[b])
    assert torch.isfinite(ref.float()).all() and gp.status() == 0


@pytest.mark.parametrize("heads,T,flags", [(1, 16, 0), (2, 8, 0), (16, 8, 0), (20, 5, 0), (128, 3, 0), (128, 9, 0),
                                           (4, 16, B.MLA_FLAG_FORCE_SIMT)])
@pytest.mark.parametrize("splits", [0, 1])
def test_a_row_among_many_new_tokens(heads, T, flags, splits):
    """One of the new tokens, which may lie in two pages or two tiles, is not finite."""
    cfg, gp = make("fp4", heads, flags, T, (0, 50, 60, 120, 250), splits)
    out, lse = gp.run()
    ref, ref_lse = out.clone(), lse.clone()
    assert torch.isfinite(ref.float()).all()
    for k in (1, T // 2, T - 1):
        gp.run()  # the rows as they were
        for b in range(cfg.B):
            overwrite(gp, b, int(cfg.L[b]) + k, float("nan"), "c")
        out, lse = gp.attend_only()
        assert torch.equal(out[:, :k], ref[:, :k]) and torch.equal(lse[:, :k], ref_lse[:, :k])
        assert torch.isnan(out[:, k:]).all() and torch.isnan(lse[:, k:]).all()
    assert gp.status() == 0
