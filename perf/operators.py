"""Cases and plain forms of two operator groups around the paged latent cache.

rows    mla_append_rows (already projected latent rows [c | k^R] of new tokens
        go into the paged cache: optional RMSNorm of c, rotation of k^R at the
        token's position, rounding to the cache type, all in one pass over the
        rows) followed by mla_read_rows (the same rows read back as values).
decode  mla_decode + mla_combine over a 4-bit latent cache, absorbed form.

The 4-bit row.  c is cut into blocks of 16.  A token has a scale ts, a power of
two: with a = max(max|c|, max|k^R| / 64), ts = 2^(floor(log2 a) - 5), not below
2^-100, and 1 where a = 0.  A block has an e4m3 scale s = e4m3(max|block| / (6 ts)),
an element an e2m1 code = e2m1(c / (s ts)) (round to nearest even, saturating;
0 where s = 0), so that c ~ code * s * ts.  The quantisers of this cache and of
the 8-bit one start from the fp32 value of c (after the norm) and round fp32
quotients.  k^R stays bf16.  A page of P tokens
holds [P][d_c/2] code bytes (element 2i in the low half of byte i), [P][d_rope]
bf16, [P][d_c/16] e4m3 scales, [P] fp32 ts, each part on a multiple of 128 bytes.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

# DeepSeek-V3 shapes of this repository's workloads
D_C, D_R, D_NOPE, D_V, D_MODEL, PAGE = 512, 64, 128, 128, 7168, 64
ROPE_BASE = 10000.0
SCALE = 1.0 / math.sqrt(D_NOPE + D_R)
EPS = 1e-6
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
KR_OFF = PAGE * D_C // 2
SC_OFF = KR_OFF + PAGE * D_R * 2
TS_OFF = SC_OFF + PAGE * D_C // 16
FP4_PAGE_BYTES = TS_OFF + PAGE * 4
ROW_BYTES = {"bf16": 2 * (D_C + D_R), "fp8": D_C + 2 * D_R + 4 * (D_C // 128), "fp4": FP4_PAGE_BYTES // PAGE}


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------
def _rows(name, batch, tokens, start, cache, norm):
    """`tokens` new tokens for each of `batch` sequences that hold `start` already."""
    return {"name": name, "op": "rows", "batch": batch, "tokens": tokens, "start": start, "cache": cache, "norm": norm}


def _decode(name, heads, batch, n_q, lo, hi, len_seed):
    """`batch` sequences of lo..hi keys (new tokens included), n_q causal query tokens each."""
    return {"name": name, "op": "decode", "heads": heads, "batch": batch, "n_q": n_q, "lo": lo, "hi": hi,
            "len_seed": len_seed}


def listed():
    return [
        # one stream generating: the new token's row, where only latency counts
        _rows("rows-b1", 1, 1, 4096, "fp4", True),
        # a step of the large batch with two tokens each, today's 8-bit cache
        _rows("rows-b128-t2-fp8", 128, 2, 16384, "fp8", True),
        # a prompt chunk of odd length into the bf16 cache, the projection already normalised
        _rows("rows-chunk-1100-bf16", 1, 1100, 700, "bf16", False),
        # a prefill chunk on top of cached tokens
        _rows("rows-chunk-4096", 1, 4096, 4096, "fp4", True),
        # eight prompts at once, ragged against the pages: the largest
        _rows("rows-b8-t4099", 8, 4099, 33, "fp4", True),
        # one stream, all heads on one GPU
        _decode("decode-h128-b1", 128, 1, 1, 4097, 4097, 1),
        # a ragged serving batch, all heads
        _decode("decode-h128-ragged-b64", 128, 64, 1, 1025, 32769, 2),
        # the large batch with two new tokens each
        _decode("decode-h128-b128-t2", 128, 128, 2, 16386, 16386, 4),
        # one GPU's 16 of the 128 heads where eight GPUs share a layer: the large batch, long contexts, one stream
        _decode("decode-h16-b128", 16, 128, 1, 16385, 16385, 5),
        _decode("decode-h16-l131072", 16, 8, 1, 131073, 131073, 6),
        _decode("decode-h16-b1-t2", 16, 1, 2, 4098, 4098, 7),
        # 64 heads where two GPUs share a layer, ragged
        _decode("decode-h64-ragged-b64", 64, 64, 1, 1025, 32769, 8),
    ]


def draw(rng):
    if rng.random() < 0.4:
        n = int(round(2 ** rng.uniform(0, 15)))  # 1 .. 32768 tokens in all
        batch = max(1, min(n, int(2 ** rng.uniform(0, 7))))
        return {"op": "rows", "batch": batch, "tokens": max(1, n // batch), "start": int(2 ** rng.uniform(0, 17)) - 1,
                "cache": rng.choice(["fp4", "fp4", "fp8", "bf16"]), "norm": rng.random() < 0.7}
    heads = rng.choice([8, 16, 20, 32, 64, 128])
    n_q = rng.choice([1, 1, 2, 3, 4])
    batch = int(round(2 ** rng.uniform(0, 7)))
    most = min(131072.0, 128 * 16386 * 256 / (batch * heads * n_q))  # no more scores than the largest listed case
    most = min(most, 128 * 16386 / batch)
    hi = int(round(2 ** rng.uniform(math.log2(64), math.log2(most))))
    lo = max(n_q, int(hi * rng.uniform(0.02, 1.0)))
    return {"op": "decode", "heads": heads, "batch": batch, "n_q": n_q, "lo": min(lo, hi), "hi": hi,
            "len_seed": rng.randrange(1 << 20)}


def lengths(case):
    r = random.Random(case["len_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]


def work(case):
    if case["op"] == "rows":
        n = case["batch"] * case["tokens"]
        row = ROW_BYTES[case["cache"]]
        # the projected rows in, the cache rows written, read back, and their values out
        return {"bytes": n * (2 * (D_C + D_R) + 2 * row + 2 * (D_C + D_R) + 16) + (2 * D_C if case["norm"] else 0),
                "flops": n * (8 * D_C + 6 * D_R)}
    h, b, t = case["heads"], case["batch"], case["n_q"]
    keys = sum(lengths(case))
    pairs = sum(t * n - t * (t - 1) // 2 for n in lengths(case))  # visible (query token, key) pairs
    weights = h * (D_NOPE + D_V) * D_C * 2
    io = b * t * h * (D_NOPE + D_R + D_V) * 2
    return {"bytes": keys * ROW_BYTES["fp4"] + weights + io,
            "flops": pairs * h * (2 * (D_C + D_R) + 2 * D_C) + 2 * b * t * h * D_C * (D_NOPE + D_V)}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    st = {"case": case}
    b = case["batch"]
    if case["op"] == "rows":
        n, end = b * case["tokens"], case["start"] + case["tokens"]
        # the output of a fused down-projection [c | k^R]: the two parts are strided views
        st["kv"] = (torch.randn(n, D_C + D_R, generator=g, device=dev) * 0.7).to(torch.bfloat16)
        st["weight"] = ((torch.rand(D_C, generator=g, device=dev) + 0.5).to(torch.bfloat16) if case["norm"] else None)
        seq = torch.arange(b, device=dev).repeat_interleave(case["tokens"])
        pos = case["start"] + torch.arange(case["tokens"], device=dev).repeat(b)
        st["seq"], st["pos"] = seq.to(torch.int32), pos.to(torch.int32)
        # the pool holds the pages that the new tokens touch
        first, last = case["start"] // PAGE, (end - 1) // PAGE
        pages = b * (last - first + 1)
        table = torch.full((b, last + 1), -1, dtype=torch.int32, device=dev)
        table[:, first:] = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(b, -1)
        st["table"] = table
        st["pool"] = torch.zeros(pages * PAGE * ROW_BYTES[case["cache"]], dtype=torch.uint8, device=dev)
        st["c_out"] = torch.empty(n, D_C, dtype=torch.bfloat16, device=dev)
        st["kr_out"] = torch.empty(n, D_R, dtype=torch.bfloat16, device=dev)
        return st
    h, t = case["heads"], case["n_q"]
    lens = lengths(case)
    per = [(x + PAGE - 1) // PAGE for x in lens]
    total = sum(per)
    pool = torch.empty(total, FP4_PAGE_BYTES, dtype=torch.uint8, device=dev)
    for p0 in range(0, total, 4096):  # cached tokens: c and the rotated k^R of unit variance
        m = min(4096, total - p0)
        c = torch.randn(m * PAGE, D_C, generator=g, device=dev)
        kr = torch.randn(m * PAGE, D_R, generator=g, device=dev).to(torch.bfloat16)
        codes, s, ts = _quantise_fp4(c, kr.float())
        pool[p0:p0 + m, :KR_OFF] = (codes[:, 0::2] | (codes[:, 1::2] << 4)).view(m, -1)
        pool[p0:p0 + m, KR_OFF:SC_OFF] = kr.view(m, -1).view(torch.uint8)
        pool[p0:p0 + m, SC_OFF:TS_OFF] = s.view(m, -1).view(torch.uint8)
        pool[p0:p0 + m, TS_OFF:] = ts.view(m, -1).view(torch.uint8)
    st["pool"] = pool
    perm = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.full((b, max(per)), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(per):
        table[i, :n] = perm[at:at + n]
        at += n
    st["table"] = table
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)

    def bf(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)

    st["q_nope"], st["q_rope"] = bf(b, t, h, D_NOPE), bf(b, t, h, D_R)
    st["W_uk"], st["W_uv"] = bf(h, D_NOPE, D_C, std=D_C ** -0.5), bf(h, D_V, D_C, std=D_C ** -0.5)
    st["out"] = torch.empty(b, t, h, D_V, dtype=torch.bfloat16, device=dev)
    if own:  # the workspace that a serving program keeps beside its cache
        B, dims = _dims(case)
        st["ws"] = torch.empty(B.decode_workspace_bytes(dims, b, t), dtype=torch.uint8, device=dev)
    return st


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(state):
    if own:
        return _own(state)
    return _plain_rows(state) if state["case"]["op"] == "rows" else _plain_decode(state)


def _dims(case):
    from latent_compressed_attention_mla_b200 import binding as B

    return B, B.make_dims(case.get("heads", 128), D_C, D_R, D_NOPE, D_V, D_MODEL, page_size=PAGE, act="bf16",
                          cache=case.get("cache", "fp4"), softmax_scale=SCALE, rope_base=ROPE_BASE)


def _own(st):
    case = st["case"]
    B, dims = _dims(case)
    if case["op"] == "rows":
        B.mla_append_rows(dims, st["kv"][:, :D_C], st["kv"][:, D_C:], st["seq"], st["pos"], st["table"], st["pool"],
                          norm_weight=st["weight"], norm_eps=EPS)
        B.mla_read_rows(dims, st["pool"], st["table"], st["seq"], st["pos"], st["c_out"], st["kr_out"])
        return st["c_out"], st["kr_out"]
    B.mla_decode(dims, st["q_nope"], st["q_rope"], st["W_uk"], st["pool"], st["table"], st["lens"], st["ws"])
    B.mla_combine(dims, st["W_uv"], case["batch"], case["n_q"], st["ws"], st["out"])
    return st["out"]


def _rotate(x, pos):
    """rotate-half RoPE of x [n, ..., D_R] (float32) at positions pos [n]; angles in 64 bits."""
    half = D_R // 2
    freq = ROPE_BASE ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    ang = pos.double().view(-1, *([1] * (x.dim() - 1))) * freq
    cs, sn = torch.cos(ang).float(), torch.sin(ang).float()
    x1, x2 = x[..., :half], x[..., half:]
    return torch.cat([x1 * cs - x2 * sn, x2 * cs + x1 * sn], dim=-1)


def _quantise_fp4(c, kr):
    """Codes uint8 [n, D_C], e4m3 scales [n, D_C/16], fp32 token scales [n, 1]."""
    blocks = c.view(c.shape[0], -1, 16)
    amax = blocks.abs().amax(-1)
    a = torch.maximum(amax.amax(-1, keepdim=True), kr.to(c.dtype).abs().amax(-1, keepdim=True) / 64)
    e = torch.clamp(torch.frexp(a)[1] - 6, min=-100)
    ts = torch.where(a > 0, torch.ldexp(torch.ones_like(a), e), torch.ones_like(a))
    s = (amax / (6 * ts)).float().to(torch.float8_e4m3fn)
    step = (s.to(c.dtype) * ts).unsqueeze(-1)
    x = torch.where(step > 0, blocks.abs() / step, torch.zeros_like(blocks))
    # borders between the levels; a tie goes to the even code
    code = ((x > 0.25).to(torch.uint8) + (x >= 0.75) + (x > 1.25) + (x >= 1.75) + (x > 2.5) + (x >= 3.5) + (x > 5.0))
    code = code | ((blocks < 0).to(torch.uint8) << 3)
    return code.view(c.shape), s, ts.float()


def _values_fp4(codes, s, ts):
    """What the codes [.., D_C], scales [.., D_C/16] and token scales [.., 1] stand for, in fp32 (exact)."""
    levels = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    v = levels[codes.int()].unflatten(-1, (-1, 16)) * (s.float() * ts).unsqueeze(-1)
    return v.flatten(-2)


def _plain_rows(st):
    case = st["case"]
    kr = _rotate(st["kv"][:, D_C:].float(), st["pos"]).to(torch.bfloat16)
    # values next to a border of the 4- and 8-bit codes need more than 32 bits
    c = st["kv"][:, :D_C].to(torch.float32 if case["cache"] == "bf16" else torch.float64)
    if case["norm"]:
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * st["weight"].to(c.dtype)
    c = c.float()
    if case["cache"] == "fp4":
        c = _values_fp4(*_quantise_fp4(c, kr.float()))
    elif case["cache"] == "fp8":
        t = c.view(c.shape[0], -1, 128)
        amax = t.abs().amax(-1, keepdim=True)
        scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        c = ((t / scale).clamp(-448, 448).to(torch.float8_e4m3fn).float() * scale).view(c.shape)
    return c.to(torch.bfloat16), kr


def _pool_values(st):
    """c [b, L, D_C] and k^R [b, L, D_R] of every table entry's page, in fp32 (L in whole pages)."""
    table = st["table"].clamp(min=0).long()
    pages = st["pool"][table]  # [b, pages, bytes]
    b = table.shape[0]
    by = pages[..., :KR_OFF]
    codes = torch.stack([by & 15, by >> 4], dim=-1).view(b, -1, D_C)
    kr = pages[..., KR_OFF:SC_OFF].contiguous().view(torch.bfloat16).view(b, -1, D_R).float()
    s = pages[..., SC_OFF:TS_OFF].contiguous().view(torch.float8_e4m3fn).view(b, -1, D_C // 16)
    ts = pages[..., TS_OFF:].contiguous().view(torch.float32).view(b, -1, 1)
    return _values_fp4(codes, s, ts), kr


def _plain_decode(st):
    b, t, h = st["q_nope"].shape[:3]
    c, kr = _pool_values(st)
    first = (st["lens"] - t).view(b, 1)
    pos = first + torch.arange(t, device=c.device)  # position of each query token
    qt = torch.einsum("bthd,hdc->bthc", st["q_nope"].float(), st["W_uk"].float()).reshape(b, t * h, D_C)
    qr = _rotate(st["q_rope"].float().view(b * t, h, D_R), pos.reshape(-1)).view(b, t * h, D_R)
    a = torch.matmul(qt, c.transpose(1, 2))
    a += torch.matmul(qr, kr.transpose(1, 2))
    a *= SCALE
    hidden = torch.arange(c.shape[1], device=c.device) > pos.unsqueeze(-1)  # [b, t, L]
    a.view(b, t, h, -1).masked_fill_(hidden.unsqueeze(2), -math.inf)
    a -= a.amax(-1, keepdim=True)
    a.exp_()
    total = a.sum(-1, keepdim=True)
    u = (torch.matmul(a, c) / total).view(b, t, h, D_C)
    return torch.einsum("bthc,hvc->bthv", u, st["W_uv"].float()).to(torch.bfloat16)


# ----------------------------------------------------------------------------
# The definition in 64 bits
# ----------------------------------------------------------------------------
def _turn64(x, pos):
    """RoPE as multiplication of the complex pairs (x_i, x_{i + half}) by exp(i pos freq)."""
    half = D_R // 2
    freq = torch.tensor([ROPE_BASE ** (-i / half) for i in range(half)], dtype=torch.float64, device=x.device)
    z = torch.complex(x[..., :half], x[..., half:])
    z = z * torch.polar(torch.ones_like(freq), pos.double().unsqueeze(-1) * freq)
    return torch.cat([z.real, z.imag], dim=-1)


def _e4m3_64(x):
    """Nonnegative float64 to the nearest e4m3 value, ties to even."""
    e = torch.frexp(x)[1].double() - 1
    q = torch.exp2(torch.clamp(e, min=-6) - 3)
    return torch.clamp(torch.round(x / q) * q, max=448.0)


def _exact_rows(st):
    case = st["case"]
    x = st["kv"].double()
    c = x[:, :D_C]
    kr = _turn64(x[:, D_C:], st["pos"])
    if case["norm"]:
        c = st["weight"].double() * c / torch.sqrt((c * c).sum(-1, keepdim=True) / D_C + EPS)
    if case["cache"] != "bf16":
        c = c.float().double()  # the quantisers start from the fp32 value, and round fp32 quotients
    if case["cache"] == "fp4":
        big = torch.maximum(c.abs().amax(-1), kr.to(torch.bfloat16).double().abs().amax(-1) / 64)
        ts = torch.exp2(torch.clamp(torch.floor(torch.log2(big)) - 5, min=-100))
        ts = torch.where(big > 0, ts, torch.ones_like(ts)).view(-1, 1)
        blk = (c / ts).reshape(c.shape[0], D_C // 16, 16)
        s = _e4m3_64((blk.abs().amax(-1) / 6).float().double()).unsqueeze(-1)
        y = torch.where(s > 0, blk.abs() / s, torch.zeros_like(blk)).float().double()
        mids = torch.tensor([(p + q) / 2 for p, q in zip(LEVELS, LEVELS[1:])], dtype=torch.float64, device=c.device)
        below, above = torch.bucketize(y, mids), torch.bucketize(y, mids, right=True)
        level = torch.where(below % 2 == 0, below, above)  # differ on a tie only
        c = (torch.tensor(LEVELS, dtype=torch.float64, device=c.device)[level] * torch.sign(blk) * s).reshape(c.shape) * ts
    elif case["cache"] == "fp8":
        blk = c.reshape(c.shape[0], D_C // 128, 128)
        top = blk.abs().amax(-1, keepdim=True)
        scale = torch.where(top > 0, top / 448, torch.ones_like(top)).float().double()
        c = (torch.sign(blk) * _e4m3_64((blk.abs() / scale).float().double()) * scale).reshape(c.shape)
    return c, kr


def _exact_decode(st):
    """Keys and values of every head rebuilt from the latent, one sequence at a time."""
    dev = st["pool"].device
    b, t, h = st["q_nope"].shape[:3]
    wk, wv = st["W_uk"].double(), st["W_uv"].double()
    level = np.array(LEVELS + tuple(-v for v in LEVELS))
    pairs = torch.tensor(np.stack([level[np.arange(256) & 15], level[np.arange(256) >> 4]], -1), device=dev)
    outs = []
    for i in range(b):
        n = int(st["lens"][i])
        pg = st["pool"][st["table"][i, :(n + PAGE - 1) // PAGE].long()]
        c = pairs[pg[:, :KR_OFF].long()].reshape(-1, D_C // 16, 16)[:n]
        s = pg[:, SC_OFF:TS_OFF].contiguous().view(torch.float8_e4m3fn).float().double().reshape(-1, D_C // 16, 1)[:n]
        ts = pg[:, TS_OFF:].contiguous().view(torch.float32).double().reshape(-1, 1, 1)[:n]
        c = (c * s * ts).reshape(n, D_C)
        kr = pg[:, KR_OFF:SC_OFF].contiguous().view(torch.bfloat16).double().reshape(-1, D_R)[:n]
        where = torch.arange(n - t, n, device=dev)
        qn = st["q_nope"][i].double()
        qr = _turn64(st["q_rope"][i].double(), where.unsqueeze(-1).expand(t, h))
        rows = []
        for h0 in range(0, h, 32):
            hs = slice(h0, min(h, h0 + 32))
            key = torch.matmul(c, wk[hs].transpose(1, 2))  # [heads, n, d_nope]
            a = torch.matmul(qn[:, hs].transpose(0, 1), key.transpose(1, 2))
            a = SCALE * (a + torch.matmul(qr[:, hs].transpose(0, 1), kr.T))
            a = a.masked_fill(torch.arange(n, device=dev) > where.view(1, t, 1), -math.inf)
            val = torch.matmul(c, wv[hs].transpose(1, 2))
            rows.append(torch.matmul(torch.softmax(a, -1), val).transpose(0, 1))
        outs.append(torch.cat(rows, 1))
    return torch.stack(outs)


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_rows(st) if case["op"] == "rows" else _exact_decode(st)
