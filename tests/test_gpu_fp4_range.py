"""Decode over 4-bit rows whose token and block scales differ: the whole range of the
format, mixed within a sequence, against values and the oracle (float64), on every
decode path (0: CUDA cores, 1: tcgen05, 2: few rows)."""
import numpy as np
import pytest
import torch

from latent_compressed_attention_mla_b200 import binding as B
from latent_compressed_attention_mla_b200 import workloads as W
from oracle import mla_oracle as O
from tests.gpu_harness import GpuProblem, OracleProblem, rel_err

pytestmark = pytest.mark.gpu

SIMT = B.MLA_FLAG_FORCE_SIMT
# (heads, query tokens, flags, path)
PATHS = [(8, 1, 0, 2), (16, 1, SIMT, 0), (16, 2, 0, 1), (128, 1, 0, 1)]
IDS = [f"h{h}-t{t}-path{p}" for h, t, _, p in PATHS]


def cfg_of(heads, T, L, **kw):
    return W.V3_FP8_B128_T2.with_(cache_dtype="fp4", n_heads=heads, B=len(L), T=T, L=tuple(L), name="fp4-range", **kw)


def rows_of(n, ts, seed, scales=None):
    """n rows as the cache holds them: random codes, block scales of every kind below
    12 (what the quantiser makes where ts follows the latent) with zeros and
    subnormals among them, token scales ts, k^R of unit variance."""
    r = np.random.default_rng(seed)
    if scales is None:
        scales = r.integers(0, 0x54, size=(n, 32))  # e4m3 0 .. 11
        scales[r.random((n, 32)) < 0.1] = 0
    return {"codes": torch.from_numpy(r.integers(0, 256, size=(n, 256)).astype(np.uint8)),
            "scales": torch.from_numpy(scales.astype(np.uint8)),
            "ts": torch.from_numpy(np.asarray(ts, dtype=np.float32).reshape(n, 1)),
            "kr": torch.from_numpy(r.standard_normal((n, 64)).astype(np.float32)).to(torch.bfloat16)}


def values_of(rows):
    return O.decode_cache_rows({k: v.double().numpy() if k in ("ts", "kr") else v.numpy() for k, v in rows.items()})


def one_hot_w_uv(heads):
    """W_uv[h, v, c] = 1 at c = (4 v + h) mod 512: the outputs are elements of the latent sum."""
    w = np.zeros((heads, 128, 512), np.float32)
    h, v = np.meshgrid(np.arange(heads), np.arange(128), indexing="ij")
    w[h, v, (4 * v + h) % 512] = 1
    return torch.from_numpy(w).to(torch.bfloat16).cuda(), (4 * v + h) % 512


# Range by path (include/mla.h): 0 and 2 take every token scale; 1 holds the latent as
# f16, exact for token scales of 2^-14 and more, to 2^-22 below.
LOW, HIGH = -100, 10  # 2^10 x 64: the largest latents


@pytest.mark.parametrize("heads,T,flags,path", PATHS, ids=IDS)
def test_a_single_key_returns_its_row(heads, T, flags, path):
    """One visible key has the probability 1, so the output is its latent: in six
    significant bits, which no rounding on the way touches."""
    e = np.repeat(np.arange(LOW, HIGH + 1), 2)
    n = len(e)
    ts = np.ldexp(1.0, e)
    rows = rows_of(n, ts, 3)
    if path == 1:  # |c| up to 64512, so s ts up to 10752
        s = O.e4m3_decode(rows["scales"].numpy()) * ts[:, None]
        rows["scales"][torch.from_numpy(s > 10752)] = 0x52  # 10
    cfg = cfg_of(heads, T, [1] * n)
    gp = GpuProblem(cfg, flags=flags)
    assert B.decode_path(gp.dims, T) == path
    for b in range(n):
        gp.cache.write_rows(gp.page_table[b], torch.zeros(1, dtype=torch.long, device="cuda"),
                            {k: v[b:b + 1].cuda() for k, v in rows.items()})
    w_uv, col = one_hot_w_uv(heads)
    i = gp.inputs
    # lens = T: the first query token sees the key at position 0 alone
    lens = torch.full((n,), T, dtype=torch.int32, device="cuda")
    out, lse = gp.session.attend(i["q_nope"], i["q_rope"], gp.weights["W_uk"], w_uv, gp.cache.pool, gp.page_table, lens)
    torch.cuda.synchronize()
    assert gp.status() == 0
    want = values_of(rows)[0][:, col]  # [n, heads, 128]
    got = out[:, 0].double().cpu().numpy()
    err = np.abs(got - want)
    exact = ts >= 2.0 ** -14 if path == 1 else np.ones(n, bool)
    assert err[exact].max() == 0
    if path == 1:
        # 7 x 2^-25 (2^-22.2) in the operand; an f16 value, which the f16 partial keeps and
        # the output rounds to bf16
        assert err[~exact].max() <= 7 * 2.0 ** -25 + 2.0 ** -8 * np.abs(want[~exact]).max(initial=0)
        # (below 2^-17 the f16 values, multiples of 2^-24, have no more bits than bf16)
        small = ts < 2.0 ** -23
        assert err[small].max() <= 2.0 ** -22
    assert torch.isfinite(lse[:, 0]).all()


@pytest.mark.parametrize("heads,T,flags,path", PATHS, ids=IDS)
def test_k_rope_alone_makes_the_token_scale_large(heads, T, flags, path):
    """Rows appended with k^R far above the latent: ts follows k^R and the block scales
    are 0, or the latent's last bits; never 0 times infinity."""
    cfg = cfg_of(heads, T, [40, 40, 40])
    gp = GpuProblem(cfg, flags=flags)
    assert B.decode_path(gp.dims, T) == path
    n = 3 * (40 + T)
    seq = torch.arange(3, dtype=torch.int32, device="cuda").repeat_interleave(40 + T).contiguous()
    pos = torch.arange(40 + T, dtype=torch.int32, device="cuda").repeat(3).contiguous()
    c = W.normal(5, 1, n * 512).view(n, 512).to(torch.bfloat16).cuda() * 6
    # k^R of 2^14, 2^20 and 2^40 times unit variance, and q^R as much smaller
    k_exp = torch.tensor([14, 20, 40], device="cuda").repeat_interleave(40 + T)
    kr = torch.ldexp(W.normal(5, 2, n * 64).view(n, 64).cuda(), k_exp.view(n, 1)).to(torch.bfloat16)
    q_rope = torch.ldexp(gp.inputs["q_rope"].float(), -torch.tensor([14, 20, 40], device="cuda").view(3, 1, 1, 1))
    q_rope = q_rope.to(torch.bfloat16)
    gp.cache.append(c, kr, seq, pos, gp.page_table)
    gc, gk = (x.double().cpu().numpy() for x in gp.cache.values(seq, pos, gp.page_table))
    assert np.isfinite(gc).all() and (gc[:40] != 0).any()
    i = gp.inputs
    out, lse = gp.session.attend(i["q_nope"], q_rope, gp.weights["W_uk"], gp.weights["W_uv"], gp.cache.pool,
                                 gp.page_table, gp.seq_lens)
    torch.cuda.synchronize()
    assert gp.status() == 0
    op = OracleProblem(cfg)
    for b in range(3):
        at = slice(b * (40 + T), (b + 1) * (40 + T))
        o, l, _ = O.decode_absorbed(op.inp["q_nope"][b], q_rope[b].double().cpu().numpy(), gc[at], gk[at], op.w["W_uk"],
                                    op.w["W_uv"], 40 + T, cfg.softmax_scale, cfg.rope_base)
        got = out[b].double().cpu().numpy()
        if np.abs(o).max() == 0:
            assert np.abs(got).max() == 0
        else:
            assert rel_err(got, o) <= 1e-2, b
        assert np.abs(lse[b].double().cpu().numpy() - l).max() <= 1e-2 * max(1.0, np.abs(l).max()), b


def scale_weights(gp, op, factor):
    """W_uk times a power of two on both sides, so that large latents score in the usual range."""
    gp.weights["W_uk"].mul_(factor)
    op.w["W_uk"] = op.w["W_uk"] * factor


def attend_and_check(cfg, gp, op, rows):
    out, lse = gp.attend_only()
    assert gp.status() == 0
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for b in range(cfg.B):
        C, KR = values_of(rows[b])
        o, l, _ = O.decode_absorbed(op.inp["q_nope"][b], op.inp["q_rope"][b], C, KR, op.w["W_uk"], op.w["W_uv"],
                                    int(cfg.seq_lens[b]), cfg.softmax_scale, cfg.rope_base)
        assert rel_err(got[b], o) <= 1e-2, b
        assert np.abs(got_lse[b] - l).max() <= 1e-2 * max(1.0, np.abs(l).max()), b


def fill(gp, cfg, ts_of, seed):
    """Every position of every sequence, the new tokens among them, with rows_of; returns them."""
    rows = []
    for b, n in enumerate(cfg.seq_lens):
        n = int(n)
        ts, scales = ts_of(np.random.default_rng(seed + b), n)
        r = rows_of(n, ts, seed + 100 + b, scales)
        gp.cache.write_rows(gp.page_table[b], torch.arange(n, device="cuda"), {k: v.cuda() for k, v in r.items()})
        rows.append(r)
    return rows


@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("heads,T,flags,path", PATHS + [(40, 3, 0, 1), (4, 4, 0, 2)],
                         ids=IDS + ["h40-t3-path1", "h4-t4-path2"])
def test_token_scales_mixed_in_a_sequence(heads, T, flags, path, splits):
    """Token scales over 2^-14 .. 2^-3 from row to row, and rows of a large scale
    with small block scales (their k^R sets it): a large S + e beside small scores."""
    def ts_of(r, n):
        e = r.integers(-14, -2, size=n).astype(float)
        scales = r.integers(0, 0x54, size=(n, 32))
        scales[r.random((n, 32)) < 0.1] = 0
        big = r.random(n) < 0.125
        e[big] = r.integers(0, 8, size=big.sum())
        scales[big] = r.integers(0, 16, size=(int(big.sum()), 32))  # 0, subnormals, up to 2^-6 x 1.875
        return np.ldexp(1.0, e.astype(int)), scales

    cfg = cfg_of(heads, T, (1, 64, 130, 300, 1500), seed=11 + heads)
    gp = GpuProblem(cfg, flags=flags, num_splits=splits)
    assert B.decode_path(gp.dims, T) == path
    rows = fill(gp, cfg, ts_of, 40)
    attend_and_check(cfg, gp, OracleProblem(cfg), rows)


@pytest.mark.parametrize("heads,T,flags,path", PATHS, ids=IDS)
def test_the_largest_latents(heads, T, flags, path):
    """|c| up to 61440, what the largest latents of the stated range are stored as."""
    def ts_of(r, n):
        scales = r.integers(0x40, 0x53, size=(n, 32))  # 2 .. 10
        scales[:, 0] = 0x52
        return np.full(n, 1024.0), scales

    cfg = cfg_of(heads, T, (1, 70, 600), seed=23)
    gp = GpuProblem(cfg, flags=flags)
    op = OracleProblem(cfg)
    scale_weights(gp, op, 2.0 ** -13)
    rows = fill(gp, cfg, ts_of, 60)
    attend_and_check(cfg, gp, op, rows)
