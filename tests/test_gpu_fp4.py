"""Attention over a 4-bit latent cache against the oracle (float64): every
decode path, prefill, and whole steps (append, then attend).

The stored values are exact on both sides, so the differences are the
attention's own: the bars of the other caches apply (max|gpu - oracle| /
max|oracle| of 1e-5 with fp32 activations, 1e-2 with bf16)."""
import numpy as np
import pytest
import torch

from latent_compressed_attention_mla_b200 import binding as B
from latent_compressed_attention_mla_b200 import workloads as W
from oracle import mla_oracle as O
from tests.gpu_harness import GpuProblem, OracleProblem, rel_err, tolerance

pytestmark = pytest.mark.gpu


class Fp4Oracle(OracleProblem):
    def history(self, b):
        rows = W.history_rows(self.cfg, b, 0, int(self.cfg.L[b]), "cpu")
        return O.decode_cache_rows({k: v.double().numpy() if k in ("ts", "kr") else v.numpy() for k, v in rows.items()})

    def after(self, gp, b):
        """Cache values of sequence b with the step's rows read back from the device cache
        (the append's own rounding is tested apart)."""
        C0, KR0 = self.history(b)
        n = np.nonzero(self.seq_idx == b)[0]
        idx = torch.from_numpy(n)
        c, kr = gp.cache.values(gp.seq_idx[idx.cuda()].contiguous(), gp.pos[idx.cuda()].contiguous(), gp.page_table)
        return np.concatenate([C0, c.double().cpu().numpy()]), np.concatenate([KR0, kr.double().cpu().numpy()])


def fp4_cfg(name="fp4", **kw):
    base = W.V3_FP8_B128_T2.with_(cache_dtype="fp4", name=name)
    return base.with_(**kw)


def check(cfg, flags=0, num_splits=0, step=True, path=None):
    gp = GpuProblem(cfg, flags=flags, num_splits=num_splits)
    if path is not None:
        assert B.decode_path(gp.dims, cfg.T) == path
    gp.session.append(gp.inputs["h"], gp.seq_idx, gp.pos, gp.weights["W_dkv"], gp.weights["W_kr"], gp.page_table,
                      gp.cache.pool)
    out, lse = gp.attend_only()
    assert gp.status() == 0
    op = Fp4Oracle(cfg)
    for b in range(cfg.B):
        o, l, _ = O.decode_absorbed(op.inp["q_nope"][b], op.inp["q_rope"][b], *op.after(gp, b), op.w["W_uk"],
                                    op.w["W_uv"], int(cfg.seq_lens[b]), cfg.softmax_scale, cfg.rope_base)
        assert rel_err(out[b].double().cpu().numpy(), o) <= tolerance(cfg), b
        assert np.abs(lse[b].double().cpu().numpy() - l).max() <= tolerance(cfg) * max(1.0, np.abs(l).max()), b
    return gp, op


@pytest.mark.parametrize("T", [1, 3])
def test_simt_fp32_activations(T):
    cfg = W.TINY_F32.with_(cache_dtype="fp4", T=T, B=2, L=(5, 200), name=f"tiny-fp4-{T}")
    check(cfg)


@pytest.mark.parametrize("page,d_c,d_rope", [(32, 64, 16), (96, 128, 2), (64, 512, 64), (64, 160, 6)])
def test_simt_other_dims(page, d_c, d_rope):
    cfg = W.TINY_F32.with_(cache_dtype="fp4", B=2, L=(1, 90), page_size=page, d_c=d_c, d_rope=d_rope,
                           name=f"tiny-fp4-{d_c}-{d_rope}-{page}")
    check(cfg)


@pytest.mark.parametrize("heads", [4, 16, 128])
def test_simt_bf16_activations(heads):
    cfg = fp4_cfg(n_heads=heads, B=2, T=2, L=(3, 150))
    check(cfg, flags=B.MLA_FLAG_FORCE_SIMT, path=0)


@pytest.mark.parametrize("L,T,heads", [(0, 1, 2), (0, 200, 2), (100, 129, 3), (300, 64, 1)])
def test_prefill(L, T, heads):
    cfg = fp4_cfg(n_heads=heads, B=2, T=T, L=(L, L + 7))
    gp = GpuProblem(cfg)
    i = gp.inputs
    gp.session.append(i["h"], gp.seq_idx, gp.pos, gp.weights["W_dkv"], gp.weights["W_kr"], gp.page_table, gp.cache.pool)
    out, lse = gp.session.prefill(i["q_nope"], i["q_rope"], gp.weights["W_uk"], gp.weights["W_uv"], gp.cache.pool,
                                  gp.page_table, gp.seq_lens, int(cfg.seq_lens.max()))
    torch.cuda.synchronize()
    assert gp.status() == 0
    op = Fp4Oracle(cfg)
    for b in range(cfg.B):
        C, KR = op.after(gp, b)
        o, l = O.decode_explicit(op.inp["q_nope"][b], op.inp["q_rope"][b], C, KR, op.w["W_uk"], op.w["W_uv"],
                                 int(cfg.seq_lens[b]), cfg.softmax_scale, cfg.rope_base)
        assert rel_err(out[b].double().cpu().numpy(), o) <= 1e-2
        assert np.abs(lse[b].double().cpu().numpy() - l).max() <= 1e-2 * max(1.0, np.abs(l).max())


@pytest.mark.parametrize("heads", [16, 128])
def test_step_rows_append_attend_and_read_together(heads):
    """A caller's own projection: rows with a norm into the 4-bit cache, attention
    over them, the rows read back; the same step captured and replayed."""
    cfg = fp4_cfg(n_heads=heads, B=3, T=2, L=(0, 62, 500))
    gp = GpuProblem(cfg)
    n = cfg.B * cfg.T
    kv = (W.normal(9, 1, n * 576).view(n, 576) * 2).to(torch.bfloat16).cuda()
    weights = dict(gp.weights, norm=(W.uniform(9, 2, 512) + 0.5).to(torch.bfloat16).cuda(), norm_eps=1e-5)
    i = gp.inputs

    def step():
        return gp.session.step_rows(kv[:, :512], kv[:, 512:], gp.seq_idx, gp.pos, i["q_nope"], i["q_rope"],
                                    gp.seq_lens, weights, gp.page_table, gp.cache.pool)

    out, _ = step()
    torch.cuda.synchronize()
    first = out.clone()
    op = Fp4Oracle(cfg)
    c = O.rms_norm(kv[:, :512].double().cpu().numpy(), weights["norm"].double().cpu().numpy(), 1e-5)
    kr = O.apply_rope(kv[:, 512:].double().cpu().numpy(), op.pos)
    enc = O.encode_cache_rows(c, kr, "fp4")
    C1, KR1 = O.decode_cache_rows(enc)
    gc, gk = gp.cache.values(gp.seq_idx, gp.pos, gp.page_table)
    assert np.array_equal(gc.double().cpu().numpy(), C1)
    assert np.abs(gk.double().cpu().numpy() - KR1).max() <= 2.0 ** -7 * np.abs(KR1).max()
    for b in range(cfg.B):
        s = op.seq_idx == b
        C0, KR0 = op.history(b)
        o, _, _ = O.decode_absorbed(op.inp["q_nope"][b], op.inp["q_rope"][b], np.concatenate([C0, C1[s]]),
                                    np.concatenate([KR0, KR1[s]]), op.w["W_uk"], op.w["W_uv"], int(cfg.seq_lens[b]),
                                    cfg.softmax_scale, cfg.rope_base)
        assert rel_err(first[b].double().cpu().numpy(), o) <= 1e-2
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
        gp.session.out.zero_()
        g.replay()
    side.synchronize()
    assert torch.equal(gp.session.out, first)
    assert gp.status() == 0


# lengths before the step around pages (64), tiles (256) and splits
RAGGED = (0, 1, 62, 63, 64, 65, 127, 128, 254, 255, 256, 257, 700, 1500)


def tc_path(heads, T):
    """Decode kernel by query rows: warp-level MMA (2) up to 16, tcgen05 (1) above."""
    return 2 if heads * T <= 16 else 1


@pytest.mark.parametrize("heads", [1, 8, 16, 20, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 3, 8])
@pytest.mark.parametrize("num_splits", [0, 1, 7])
def test_tensor_core_ragged(heads, T, num_splits):
    check(fp4_cfg(n_heads=heads, B=len(RAGGED), T=T, L=RAGGED), num_splits=num_splits, path=tc_path(heads, T))


@pytest.mark.parametrize("heads", [16, 33, 128])
def test_tensor_core_long(heads):
    check(fp4_cfg(n_heads=heads, B=1, T=2, L=(9000,)), path=1)
    check(fp4_cfg(n_heads=heads, B=1, T=1, L=(9000,)), path=tc_path(heads, 1))


@pytest.mark.parametrize("heads,T", [(16, 20), (128, 9), (1, 16), (3, 5), (5, 40), (192, 1), (96, 3)])
def test_rows_across_query_tokens(heads, T):
    """Groups of rows that hold several tokens, each with its own causal limit, from empty caches on."""
    check(fp4_cfg(n_heads=heads, B=3, T=T, L=(0, 63, 200)), path=tc_path(heads, T))


@pytest.mark.parametrize("heads", [8, 40, 128])
def test_rows_behind_the_end_do_not_reach_the_output(heads):
    """Everything past a sequence's last key, in its last page and in pages no
    sequence holds, is NaN (codes, scales, token scales and k^R): the outputs are those
    of a clean pool, bit for bit."""
    cfg = fp4_cfg(n_heads=heads, B=5, T=2, L=(0, 5, 62, 300, 1000), spare_pages=3)
    gp = GpuProblem(cfg)
    out, lse = gp.run()
    ref, ref_lse = out.clone(), lse.clone()
    v = gp.cache.views()
    keep = torch.zeros(cfg.num_pages, 64, dtype=torch.bool)
    for b, n in enumerate(cfg.seq_lens):
        pos = np.arange(n)
        keep[gp.pt_host[b, pos // 64], pos % 64] = True
    bad = ~keep.cuda()
    v["scales"][bad] = 0x7F
    v["ts"][bad] = float("nan")
    v["kr"][bad] = float("inf")
    v["codes"][bad] = 0xFF
    out, lse = gp.run()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert gp.status() == 0


@pytest.mark.parametrize("heads", [8, 40, 128])
def test_deterministic_and_page_order_invariant(heads):
    cfg = fp4_cfg(n_heads=heads, B=3, T=2, L=(100, 777, 2000))
    gp = GpuProblem(cfg)
    out, lse = gp.run()
    ref, ref_lse = out.clone(), lse.clone()
    for _ in range(3):
        out, lse = gp.run()
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    other = GpuProblem(cfg, page_table=W.page_table(cfg, seed_offset=5))
    out, lse = other.run()
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)


@pytest.mark.parametrize("heads", [8, 40, 128])
def test_bad_pages_and_short_sequences_are_reported(heads):
    cfg = fp4_cfg(n_heads=heads, B=3, T=2, L=(100, 300, 500))
    gp = GpuProblem(cfg)
    out, _ = gp.run()
    ref = out.clone()
    table = gp.page_table.clone()
    table[1, 2] = cfg.num_pages + 7
    i = gp.inputs
    out, _ = gp.session.attend(i["q_nope"], i["q_rope"], gp.weights["W_uk"], gp.weights["W_uv"], gp.cache.pool, table,
                               gp.seq_lens)
    torch.cuda.synchronize()
    assert gp.status() == B.MLA_ERR_BOUNDS
    assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
    lens = gp.seq_lens.clone()
    lens[1] = 1  # shorter than the two new tokens: no key for this sequence
    out, lse = gp.session.attend(i["q_nope"], i["q_rope"], gp.weights["W_uk"], gp.weights["W_uv"], gp.cache.pool,
                                 gp.page_table, lens)
    torch.cuda.synchronize()
    assert gp.status() == B.MLA_ERR_BOUNDS
    assert (out[1] == 0).all() and torch.isinf(lse[1]).all()
    assert rel_err(out[0].double().cpu().numpy(), ref[0].double().cpu().numpy()) < 1e-2
    assert rel_err(out[2].double().cpu().numpy(), ref[2].double().cpu().numpy()) < 1e-2


@pytest.mark.parametrize("heads", [8, 40, 128])
def test_expired_wait_is_reported_and_the_next_step_is_right(heads):
    """With the self-test flag the load producers issue no load: the bounded waits expire."""
    cfg = fp4_cfg(n_heads=heads, B=2, T=1, L=(100, 300))
    gp = GpuProblem(cfg)
    ref = gp.run()[0].clone()
    gp.session.dims = B.dims_for(cfg, B.MLA_FLAG_SELFTEST_STALL)
    i = gp.inputs
    B.mla_decode(gp.session.dims, i["q_nope"], i["q_rope"], gp.weights["W_uk"], gp.cache.pool, gp.page_table,
                 gp.seq_lens, gp.session.decode_ws)
    assert gp.status() == B.MLA_ERR_TIMEOUT
    gp.session.dims = gp.dims
    assert torch.equal(gp.run()[0], ref)
    assert gp.status() == 0


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("heads", [148, 192])
def test_more_heads_than_multiprocessors(heads, cache):
    """Few tokens and at least as many heads as multiprocessors: the absorption's
    32-token kernel, whatever the head count."""
    cfg = fp4_cfg(n_heads=heads, cache_dtype=cache, B=2, T=1, L=(3, 100))
    gp = GpuProblem(cfg)
    out, _ = gp.run()
    assert gp.status() == 0
    if cache == "fp4":
        op = Fp4Oracle(cfg)
        caches = [op.after(gp, b) for b in range(cfg.B)]
    else:
        op = OracleProblem(cfg)
        caches = [op.cache_values(b) for b in range(cfg.B)]
    for b in range(cfg.B):
        o, _ = op.expected_absorbed(b, cache=caches[b])
        assert rel_err(out[b].double().cpu().numpy(), o) <= 1e-2


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("d_v", [64, 136])
def test_other_value_widths_at_128_heads(cache, d_v):
    """The tensor-core decode's partials are bf16 rows that only the combine of d_v = 128 reads."""
    cfg = fp4_cfg(cache_dtype=cache, B=2, T=1, L=(70, 200), d_v=d_v)
    gp = GpuProblem(cfg)
    assert B.decode_path(gp.dims, 1) == 0
    gp.session.append(gp.inputs["h"], gp.seq_idx, gp.pos, gp.weights["W_dkv"], gp.weights["W_kr"], gp.page_table,
                      gp.cache.pool)
    out, lse = gp.attend_only()
    assert gp.status() == 0
    op = Fp4Oracle(cfg)
    c, kr = gp.cache.values(*every_position(cfg), gp.page_table)
    at = 0
    for b in range(cfg.B):
        n = int(cfg.seq_lens[b])
        o, l, _ = O.decode_absorbed(op.inp["q_nope"][b], op.inp["q_rope"][b], c[at:at + n].double().cpu().numpy(),
                                    kr[at:at + n].double().cpu().numpy(), op.w["W_uk"], op.w["W_uv"], n,
                                    cfg.softmax_scale, cfg.rope_base)
        at += n
        assert rel_err(out[b].double().cpu().numpy(), o) <= tolerance(cfg), b


def every_position(cfg):
    seq = np.concatenate([np.full(int(n), b, np.int32) for b, n in enumerate(cfg.seq_lens)])
    pos = np.concatenate([np.arange(int(n), dtype=np.int32) for n in cfg.seq_lens])
    return torch.from_numpy(seq).cuda(), torch.from_numpy(pos).cuda()


@pytest.mark.parametrize("cache,heads", [("bf16", 128), ("fp8", 128), ("fp4", 128), ("fp4", 8)])
def test_combine_refuses_an_output_that_holds_no_pairs(cache, heads):
    cfg = fp4_cfg(cache_dtype=cache, B=1, T=1, L=(70,), n_heads=heads)
    gp = GpuProblem(cfg)
    assert B.decode_path(gp.dims, 1) >= 1
    out, _ = gp.attend_only()
    odd = torch.zeros(out.numel() + 1, dtype=out.dtype, device="cuda")[1:]
    ws = torch.zeros(B.decode_workspace_bytes(gp.dims, 1, 1, 0), dtype=torch.uint8, device="cuda")
    with pytest.raises(B.MlaError, match="ALIGN"):
        B.mla_combine(gp.dims, gp.weights["W_uv"], 1, 1, ws, odd.view(out.shape))
    assert odd.abs().sum().item() == 0 and gp.status() == 0


@pytest.mark.parametrize("heads", [8, 40, 128])
def test_captured_graphs_replayed_on_two_streams(heads):
    """Two graphs of decode and combine, each with its workspace, replayed side by side with new queries and
    lengths, give what eager calls give."""
    runs = []
    for k in range(2):
        cfg = fp4_cfg(B=3, T=1, L=(5, 700, 131), n_heads=heads, seed=21 + k)
        gp = GpuProblem(cfg)
        gp.session.append(gp.inputs["h"], gp.seq_idx, gp.pos, gp.weights["W_dkv"], gp.weights["W_kr"], gp.page_table,
                          gp.cache.pool)
        ws = torch.empty(B.decode_workspace_bytes(gp.dims, 3, 1), dtype=torch.uint8, device="cuda")
        q_nope, q_rope = gp.inputs["q_nope"].clone(), gp.inputs["q_rope"].clone()
        lens = torch.from_numpy(cfg.seq_lens.astype(np.int32)).cuda()
        out = torch.empty(3, 1, heads, cfg.d_v, dtype=torch.bfloat16, device="cuda")

        def step(gp=gp, ws=ws, q_nope=q_nope, q_rope=q_rope, lens=lens, out=out):
            B.mla_decode(gp.dims, q_nope, q_rope, gp.weights["W_uk"], gp.cache.pool, gp.page_table, lens, ws)
            B.mla_combine(gp.dims, gp.weights["W_uv"], 3, 1, ws, out)

        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        runs.append((g, step, q_nope, lens, out, torch.cuda.Stream()))
    for _ in range(3):
        for _, _, q_nope, lens, _, _ in runs:
            q_nope.mul_(-0.75)
            lens.sub_(1)
        torch.cuda.synchronize()
        for g, _, _, _, _, s in runs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        got = [r[4].clone() for r in runs]
        for r, want in zip(runs, got):
            r[4].zero_()
            r[1]()
            torch.cuda.synchronize()
            assert torch.equal(r[4], want) and want.abs().sum().item() > 0
    assert B.mla_get_status() == 0
