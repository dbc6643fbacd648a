"""mla_append_rows and mla_read_rows against the oracle (float64), on every
cache type, at sizes, strides and values where they can go wrong.

Tolerances.  Quantised rows are compared bit for bit: the kernel's fp32 value of
c is the correctly rounded one (its error before that rounding is far below a
fp32 step), and every later decision is one correctly rounded fp32 division.
Plain rows: the cache type's rounding is off by at most half a step,
finfo.eps / 2 relative (2^-8 bf16, 2^-24 f32), after the fp32 value's own half
step (2^-24).  k^R: the rotation adds the angle's sine and cosine in float
(a few 1e-7) and two fp32 roundings: 1e-6 (|x1| + |x2|) covers them."""
import numpy as np
import pytest
import torch

from latent_compressed_attention_mla_b200 import binding as B
from latent_compressed_attention_mla_b200 import workloads as W
from latent_compressed_attention_mla_b200.paged_cache import PagedLatentCache
from oracle import mla_oracle as O

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp8": 2.0 ** -8, "fp4": 2.0 ** -8}
TYPES = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "fp8"), ("bf16", "fp4"), ("f32", "bf16"), ("f32", "fp8"),
         ("f32", "fp4")]


class Rows:
    """n rows for `batch` sequences; seq/pos a seeded choice of distinct slots."""

    def __init__(self, act, cache, n, d_c=512, d_rope=64, page=64, batch=3, seed=11, scale=0.7, pages_per_seq=None):
        self.act, self.cache_type, self.n = act, cache, n
        self.dims = B.make_dims(8, d_c, d_rope, 128, 128, 512, page_size=page, act=act, cache=cache)
        self.dt = torch.float32 if act == "f32" else torch.bfloat16
        self.kv = (W.normal(seed, 1, n * (d_c + d_rope)).view(n, d_c + d_rope) * scale).to(self.dt)
        self.w = (W.uniform(seed, 2, d_c) + 0.5).to(self.dt)
        per = pages_per_seq or (-(-n // (batch * page)) + 1)
        rng = np.random.default_rng(seed)
        slots = rng.permutation(batch * per * page)[:n]
        self.seq = torch.from_numpy((slots // (per * page)).astype(np.int32))
        self.pos = torch.from_numpy((slots % (per * page)).astype(np.int32))
        self.num_pages = batch * per + 2
        self.table = torch.from_numpy(rng.permutation(self.num_pages)[:batch * per].reshape(batch, per).astype(np.int32))
        self.cache = PagedLatentCache(self.dims, self.num_pages, "cuda", fill=0xA5)
        self.d_c, self.d_rope, self.page = d_c, d_rope, page

    def cuda(self):
        g = lambda t: t.cuda()  # noqa: E731
        kv = g(self.kv)
        return kv[:, :self.d_c], kv[:, self.d_c:], g(self.seq), g(self.pos), g(self.table)

    def append(self, norm=False, eps=1e-6, **kw):
        c, kr, seq, pos, table = self.cuda()
        self.cache.append(c, kr, seq, pos, table, self.w.cuda() if norm else None, eps, **kw)
        torch.cuda.synchronize()

    def stored(self, rows=None):
        """The cache's raw rows at the slots (numpy)."""
        rows = np.arange(self.n) if rows is None else rows
        s, p = self.seq.numpy()[rows], self.pos.numpy()[rows]
        page = torch.from_numpy(self.table.numpy()[s, p // self.page]).long().cuda()
        row = torch.from_numpy(p % self.page).long().cuda()
        out = {k: v[page, row].cpu() for k, v in self.cache.views().items()}
        return {k: (v.float().numpy() if v.dtype == torch.bfloat16 else v.numpy()) for k, v in out.items()}

    def check(self, norm=False, eps=1e-6, rows=None):
        rows = np.arange(self.n) if rows is None else rows
        x = self.kv.double().numpy()[rows]
        c = x[:, :self.d_c]
        if norm:
            c = O.rms_norm(c, self.w.double().numpy(), eps)
        got = self.stored(rows)
        kr = O.apply_rope(x[:, self.d_c:], self.pos.numpy()[rows])
        h = self.d_rope // 2
        pair = np.abs(x[:, self.d_c:self.d_c + h]) + np.abs(x[:, self.d_c + h:])
        # below 2^-126 the step is 2^-133 (bf16) whatever the value: half of it is 2^-134
        tol = (HALF_STEP["f32" if self.cache_type == "f32" else "bf16"] * np.abs(kr) +
               1e-6 * np.concatenate([pair, pair], 1) + 2.0 ** -134)
        over = int((np.abs(got["kr"] - kr) > tol).sum())
        assert over == 0
        if self.cache_type == "fp4":
            codes, s, ts = O.fp4_quantise_latent(c, got["kr"])
            assert np.array_equal(got["ts"].astype(np.float64), ts)
            assert np.array_equal(got["scales"], s)
            # -0 and +0 stand for the same value
            assert np.array_equal(O.e2m1_decode(got["codes"] & 15), O.e2m1_decode(codes & 15))
            assert np.array_equal(O.e2m1_decode(got["codes"] >> 4), O.e2m1_decode(codes >> 4))
        elif self.cache_type == "fp8":
            codes, s = O.fp8_quantise_latent(c)
            assert np.array_equal(got["scales"], s)
            assert np.array_equal(O.e4m3_decode(got["codes"]), O.e4m3_decode(codes))
        else:
            assert np.all(np.abs(got["c"] - c) <= (HALF_STEP[self.cache_type] + 2.0 ** -23) * np.abs(c))

    def values_expected(self, rows=None):
        """What the stored rows stand for, rounded to the activation type."""
        got = self.stored(rows)
        c, kr = O.decode_cache_rows(got)
        rnd = O.to_f32 if self.act == "f32" else O.to_bf16
        return rnd(O.to_f32(c)), rnd(kr)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("act,cache", TYPES)
@pytest.mark.parametrize("n", [1, 7, 300])
def test_append_rows_matches_oracle(act, cache, n, norm):
    r = Rows(act, cache, n)
    before = r.cache.pool.clone()
    r.append(norm)
    r.check(norm)
    assert B.mla_get_status() == 0
    # no byte outside the tokens' rows changed
    for k, v in r.cache.views().items():
        page = torch.from_numpy(r.table.numpy()[r.seq.numpy(), r.pos.numpy() // r.page]).long().cuda()
        row = (r.pos % r.page).long().cuda()
        v[page, row] = torch.full_like(v[page, row].view(torch.uint8), 0xA5).view(v.dtype)
    assert torch.equal(r.cache.pool, before)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
def test_append_rows_many_tokens(cache, norm):
    r = Rows("bf16", cache, 6001, batch=5)  # more than one token per warp
    r.append(norm)
    r.check(norm)


@pytest.mark.parametrize("act,cache", TYPES)
@pytest.mark.parametrize("d_c,d_rope,page", [(64, 16, 16), (16, 0, 1), (80, 6, 7), (512, 200, 3), (1024, 64, 64)])
def test_append_rows_other_dims(act, cache, d_c, d_rope, page):
    if cache == "fp8" and d_c % 128 or act == "f32" and d_c > 512:
        pytest.skip("dims without that cache type")
    r = Rows(act, cache, 37, d_c, d_rope, page)
    r.append(True)
    r.check(True)
    c, kr = r.cache.values(r.seq.cuda(), r.pos.cuda(), r.table.cuda())
    ec, ekr = r.values_expected()
    assert np.array_equal(c.double().cpu().numpy(), ec) and np.array_equal(kr.double().cpu().numpy(), ekr)
    assert B.mla_get_status() == 0


@pytest.mark.parametrize("act,cache", TYPES)
def test_strides_and_alignment_do_not_change_results(act, cache):
    r = Rows(act, cache, 50)
    r.append(True)
    ref = r.cache.pool.clone()
    _, _, seq, pos, table = r.cuda()
    for off, width in ((1, 601), (8, 640), (0, 577)):
        wide = torch.full((50, width + 64), 7.0, dtype=r.dt, device="cuda")
        wide[:, off:off + 512] = r.kv[:, :512].cuda()
        wide[:, width:width + 64] = r.kv[:, 512:].cuda()
        wbuf = torch.zeros(513, dtype=r.dt, device="cuda")
        w = wbuf[off & 1:][:512]
        w.copy_(r.w)
        r.cache.pool.fill_(0xA5)
        r.cache.append(wide[:, off:off + 512], wide[:, width:width + 64], seq, pos, table, w, 1e-6)
        assert torch.equal(r.cache.pool, ref)
    # rows in reverse order (a negative stride is not a torch view): every row twice as far apart
    far = torch.zeros(100, 576, dtype=r.dt, device="cuda")
    far[::2] = r.kv.cuda()
    r.cache.pool.fill_(0xA5)
    r.cache.append(far[::2, :512], far[::2, 512:], seq, pos, table, r.w.cuda(), 1e-6)
    assert torch.equal(r.cache.pool, ref)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
def test_long_positions(cache):
    r = Rows("bf16", cache, 64, page=64, batch=2, pages_per_seq=3000)
    r.append()
    assert int(r.pos.max()) > 100000
    r.check()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_fp4_extreme_values(act):
    r = Rows(act, "fp4", 8)
    kv = r.kv
    kv[0] = 0
    kv[1] *= 2.0 ** 100
    kv[2] *= 2.0 ** -100
    kv[3, :512] = 0          # only k^R sets the token scale
    kv[4, 5:] = 0
    kv[4, 5] = 1e-30         # one tiny element
    kv[5, 16:512] *= 2.0 ** -30  # one block dwarfs the others: their scales round to zero
    kv[6, 512:] *= 2.0 ** 20     # k^R dwarfs c
    kv[7] = torch.finfo(r.dt).tiny
    r.append()
    r.check()
    c, kr = r.cache.values(r.seq.cuda(), r.pos.cuda(), r.table.cuda())
    assert torch.isfinite(c).all() and torch.isfinite(kr).all()
    assert B.mla_get_status() == 0


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_fp4_ties_and_borders(act):
    """Elements on the borders between codes, at several block scales."""
    r = Rows(act, "fp4", 32)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0])
    for i in range(32):
        r.kv[i, :512] = (mids.repeat(32) * (1 + (i % 8) / 8) * 2.0 ** (i // 8 - 2)).to(r.dt)
    r.append()
    r.check()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_fp4_non_finite(act):
    r = Rows(act, "fp4", 6)
    r.kv[0, 17] = float("inf")
    r.kv[1, 500] = float("nan")
    r.kv[2, :512] = float("-inf")
    r.kv[3, 512 + 3] = float("inf")  # k^R: stored as it is
    r.append()
    c, kr = (t.float().cpu() for t in r.cache.values(r.seq.cuda(), r.pos.cuda(), r.table.cuda()))
    bad = torch.zeros(6, 512, dtype=torch.bool)
    bad[0, 16:32] = bad[1, 496:512] = True
    bad[2] = True
    assert torch.equal(torch.isnan(c), bad)
    assert not torch.isfinite(kr[3]).all() and torch.isfinite(kr[[0, 1, 2, 4, 5]]).all()
    r.check(rows=np.array([4, 5]))
    got = r.stored(np.array([0, 1]))
    x = r.kv.double().numpy()[:2, :512]
    codes, s, ts = O.fp4_quantise_latent(x, got["kr"])
    assert np.array_equal(got["scales"], s) and np.array_equal(got["ts"].astype(np.float64), ts)
    assert np.array_equal(got["codes"] & 0x77, codes & 0x77)


@pytest.mark.parametrize("act,cache", TYPES)
def test_read_rows(act, cache):
    r = Rows(act, cache, 211)
    r.append(True)
    order = torch.from_numpy(np.random.default_rng(5).integers(0, 211, 500))  # rows may repeat
    c, kr = r.cache.values(r.seq[order].cuda(), r.pos[order].cuda(), r.table.cuda())
    ec, ekr = r.values_expected(order.numpy())
    assert np.array_equal(c.double().cpu().numpy(), ec)
    assert np.array_equal(kr.double().cpu().numpy(), ekr)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
def test_out_of_range_tokens_are_skipped_and_reported(cache):
    r = Rows("bf16", cache, 9)
    ok = r.cache.pool
    c, kr, seq, pos, table = r.cuda()
    r.append()
    ref = ok.clone()
    per = table.shape[1]
    bad_table = table.clone()
    for what in ("seq_low", "seq_high", "pos_low", "pos_high", "page_low", "page_high"):
        s, p, t = seq.clone(), pos.clone(), table
        if what == "seq_low":
            s[4] = -1
        elif what == "seq_high":
            s[4] = table.shape[0]
        elif what == "pos_low":
            p[4] = -1
        elif what == "pos_high":
            p[4] = per * 64
        else:
            t = bad_table.clone()
            b, pg = int(seq[4]), int(pos[4]) // 64
            t[b, pg] = -1 if what == "page_low" else r.num_pages
        ok.fill_(0xA5)
        r.cache.append(c, kr, s, p, t, None)
        assert B.mla_get_status() == B.MLA_ERR_BOUNDS, what
        hit = [i for i in range(9) if i != 4 and not (what.startswith("page") and int(seq[i]) == int(seq[4])
                                                       and int(pos[i]) // 64 == int(pos[4]) // 64)]
        r.check(rows=np.array(hit))
        row4 = r.stored(np.array([4]))
        assert all((np.ascontiguousarray(v).view(np.uint8) == 0xA5).all() or k in ("kr", "c") for k, v in row4.items())
        # reading: that row's outputs stay as they were
        ok.copy_(ref)
        c_out = torch.full((9, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        k_out = torch.full((9, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        B.mla_read_rows(r.dims, ok, t, s, p, c_out, k_out)
        assert B.mla_get_status() == B.MLA_ERR_BOUNDS, what
        assert (c_out[4] == 3).all() and (k_out[4] == 3).all()
        assert not (c_out[hit] == 3).all(dim=1).any()


def test_no_tokens():
    r = Rows("bf16", "fp4", 4)
    c, kr, seq, pos, table = r.cuda()
    before = r.cache.pool.clone()
    r.cache.append(c[:0], kr[:0], seq[:0], pos[:0], table)
    c0, k0 = r.cache.values(seq[:0], pos[:0], table)
    assert c0.shape == (0, 512) and k0.shape == (0, 64)
    assert torch.equal(r.cache.pool, before)


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
def test_captured_and_replayed_on_a_side_stream(cache):
    r = Rows("bf16", cache, 40)
    c, kr, seq, pos, table = r.cuda()
    kv = torch.zeros(40, 576, dtype=torch.bfloat16, device="cuda")
    w = r.w.cuda()
    c_out = torch.empty(40, 512, dtype=torch.bfloat16, device="cuda")
    k_out = torch.empty(40, 64, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def both():
        r.cache.append(kv[:, :512], kv[:, 512:], seq, pos, table, w)
        B.mla_read_rows(r.dims, r.cache.pool, table, seq, pos, c_out, k_out)

    with torch.cuda.stream(side):
        both()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            both()
        for rep in range(2):
            kv.copy_(r.kv.cuda() * (1 + rep))
            g.replay()
    side.synchronize()
    r.kv *= 2
    r.check(True)
    ec, ekr = r.values_expected()
    assert np.array_equal(c_out.double().cpu().numpy(), ec) and np.array_equal(k_out.double().cpu().numpy(), ekr)


@pytest.mark.parametrize("n", [1, 3, 9, 100, 600])
@pytest.mark.parametrize("entry", ["append_latent", "noalloc"])
def test_append_latent_into_a_4bit_cache(n, entry):
    """The projection's fp32 sums reach the quantiser within 2e-5 of the exact
    ones (a 7,168-term fp32 accumulation), so a stored element is within one
    step (half the widest gap between codes) plus that of the exact latent, and
    a block's scale within one e4m3 step of the exact one's."""
    if entry == "noalloc" and n * 512 > 65536:
        pytest.skip("above the fixed scratch")
    cfg = W.V3_FP8_B128_T2.with_(cache_dtype="fp4", B=n, T=1, L=5, name=f"fp4-append-{n}")
    d = B.dims_for(cfg)
    wts = {k: v.cuda() for k, v in W.weights(cfg, "cpu").items()}
    h = W.step_inputs(cfg, "cpu")["h"]
    seq, pos = (torch.from_numpy(x).cuda() for x in W.new_token_index(cfg))
    table = torch.from_numpy(W.page_table(cfg)).cuda()
    cache = PagedLatentCache(d, cfg.num_pages, "cuda", fill=0xA5)
    if entry == "noalloc":
        B.mla_append_latent_noalloc(d, h.cuda(), seq, pos, wts["W_dkv"], wts["W_kr"], table, cache.pool)
    else:
        ws = torch.empty(B.append_workspace_bytes_fast(d, n), dtype=torch.uint8, device="cuda")
        B.mla_append_latent(d, h.cuda(), seq, pos, wts["W_dkv"], wts["W_kr"], table, cache.pool, ws)
    assert B.mla_get_status() == 0
    some = np.unique(np.linspace(0, n - 1, 20).astype(int))
    c, kr = O.append_latent(h.double().numpy()[some], wts["W_dkv"].double().cpu().numpy(),
                            wts["W_kr"].double().cpu().numpy(), cfg.L[0] + 0 * some)
    got = {k: v for k, v in zip(("c", "kr"), cache.values(seq, pos, table))}
    gc, gk = (got[k].double().cpu().numpy()[some] for k in ("c", "kr"))
    v = cache.views()
    page = table[seq.long(), pos.long() // 64].long()
    raw_s = v["scales"][page, pos.long() % 64].cpu().numpy()[some]
    raw_ts = v["ts"][page, pos.long() % 64].cpu().double().numpy()[some]
    codes, s, ts = O.fp4_quantise_latent(c, gk)
    err = 2e-5 * np.abs(c).max()
    assert np.array_equal(raw_ts, ts)
    assert np.abs(raw_s.astype(int) - s.astype(int)).max() <= 1
    step = np.repeat(O.e4m3_decode(raw_s) * raw_ts, 16, axis=1)
    assert np.all(np.abs(gc - c) <= step * (1 + 1e-6) + err)
    assert (O.fp4_dequantise_latent(codes, s, ts) != gc).mean() < 1e-3  # all but border cases agree exactly
    assert np.all(np.abs(gk - kr) <= 2.0 ** -8 * np.abs(kr) + 4 * err)


MANY = 19_001  # read_rows takes four tokens a warp and append_rows' warps loop


@pytest.mark.parametrize("odd_out", [False, True])
@pytest.mark.parametrize("act,cache", TYPES)
def test_many_rows_in_one_call_are_the_rows_of_many_calls(act, cache, odd_out):
    """Bad slots among them: those write nothing, and their outputs stay as they were."""
    r = Rows(act, cache, MANY, d_c=256, d_rope=64, batch=4)
    bad = np.array([0, 1, 777, 4_000, 4_003, 12_345, MANY - 1])
    r.pos[torch.from_numpy(bad)] = torch.tensor([-1, 10 ** 9, -5, 10 ** 6, -1, 10 ** 8, -1], dtype=torch.int32)
    c, kr, seq, pos, table = r.cuda()
    r.cache.append(c, kr, seq, pos, table, r.w.cuda())
    assert B.mla_get_status() == B.MLA_ERR_BOUNDS
    one = r.cache.pool.clone()
    r.cache.pool.fill_(0xA5)
    for i in range(0, MANY, 3_000):
        j = min(i + 3_000, MANY)
        r.cache.append(c[i:j], kr[i:j], seq[i:j].contiguous(), pos[i:j].contiguous(), table, r.w.cuda())
    assert torch.equal(one, r.cache.pool)

    def out(width):
        flat = torch.full((MANY * width + 1,), 3.0, dtype=r.dt, device="cuda")
        return (flat[1:] if odd_out else flat[:-1]).view(MANY, width)

    co, ko = out(256), out(64)
    B.mla_read_rows(r.dims, r.cache.pool, table, seq, pos, co, ko)
    cs, ks = torch.full_like(co, 3.0), torch.full_like(ko, 3.0)
    for i in range(0, MANY, 3_000):
        j = min(i + 3_000, MANY)
        B.mla_read_rows(r.dims, r.cache.pool, table, seq[i:j].contiguous(), pos[i:j].contiguous(), cs[i:j], ks[i:j])
    torch.cuda.synchronize()
    assert torch.equal(co, cs) and torch.equal(ko, ks)
    assert (co[bad] == 3.0).all() and (ko[bad] == 3.0).all()
    good = np.setdiff1d(np.arange(MANY), bad)
    assert (co[good].float().abs().sum(1) > 0).all()
    assert B.mla_get_status() == B.MLA_ERR_BOUNDS


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
def test_append_and_read_captured_and_replayed_beside_another_stream(cache):
    """One graph of an append and a read, replayed with new inputs while a second stream reads another pool."""
    a, b = Rows("bf16", cache, 300, seed=3), Rows("bf16", cache, 300, seed=4)
    a.append(norm=True)
    b.append(norm=True)
    c, kr, seq, pos, table = a.cuda()
    w = a.w.cuda()
    c, kr = c.contiguous(), kr.contiguous()
    co, ko = torch.empty_like(c), torch.empty_like(kr)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.cache.append(c, kr, seq, pos, table, w)
        B.mla_read_rows(a.dims, a.cache.pool, table, seq, pos, co, ko)
    _, _, seq_b, pos_b, table_b = b.cuda()
    want_b = b.cache.values(seq_b, pos_b, table_b)
    torch.cuda.synchronize()
    for k in range(3):
        c.mul_(-1.5)
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side):
            got_b = b.cache.values(seq_b, pos_b, table_b)
        torch.cuda.synchronize()
        fresh = Rows("bf16", cache, 300, seed=3)
        fresh.cache.append(c, kr, seq, pos, table, w)
        want = fresh.cache.values(seq, pos, table)
        torch.cuda.synchronize()
        assert torch.equal(co, want[0]) and torch.equal(ko, want[1])
        assert torch.equal(got_b[0], want_b[0]) and torch.equal(got_b[1], want_b[1])
