"""Pins of the oracle's 4-bit row format and RMSNorm, and the library's host
side for them (page layout, argument checks).  No kernel is launched."""
import ctypes

import numpy as np
import pytest
import torch

from latent_compressed_attention_mla_b200 import binding as B
from latent_compressed_attention_mla_b200 import workloads as W
from latent_compressed_attention_mla_b200.paged_cache import PagedLatentCache
from oracle import mla_oracle as O


def test_e2m1_levels_ties_and_saturation():
    codes = np.arange(16, dtype=np.uint8)
    v = O.e2m1_decode(codes)
    assert list(v[:8]) == [0, .5, 1, 1.5, 2, 3, 4, 6] and np.array_equal(v[8:], -v[:8])
    assert np.array_equal(O.e2m1_encode(v[:8]), codes[:8]) and np.array_equal(O.e2m1_encode(v[9:]), codes[9:])
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert list(O.e2m1_encode(mids)) == [0, 2, 2, 4, 4, 6, 6]  # the even neighbour
    eps = 1e-9
    assert list(O.e2m1_encode(np.array(mids) + eps)) == [1, 2, 3, 4, 5, 6, 7]
    assert list(O.e2m1_encode(np.array(mids) - eps)) == [0, 1, 2, 3, 4, 5, 6]
    assert list(O.e2m1_encode([7.0, 1e9, -7.0])) == [7, 7, 15]


def test_fp4_row_closed_form():
    # one block whose maximum is 6 * 2^k: scale is a power of two and the levels round-trip
    c = np.zeros((1, 32))
    c[0, :16] = np.concatenate([O.E2M1_POS, -O.E2M1_POS]) * 0.25
    codes, s, ts = O.fp4_quantise_latent(c, np.zeros((1, 4)))
    # a = 1.5: ts = 2^(0 - 5); block maximum / (6 ts) = 1.5 / (6 / 32) = 8
    assert ts[0, 0] == 2.0 ** -5 and O.e4m3_decode(s)[0, 0] == 8.0 and O.e4m3_decode(s)[0, 1] == 0.0
    assert np.array_equal(O.fp4_dequantise_latent(codes, s, ts), c)
    assert codes[0, 0] == 0x10 and codes[0, 1] == 0x32  # element 2i in the low half


def test_fp4_token_scale_sees_k_rope_and_edges():
    z = np.zeros((1, 16))
    assert O.fp4_quantise_latent(z, np.zeros((1, 2)))[2] == 1.0
    assert O.fp4_quantise_latent(z, np.full((1, 2), 128.0))[2] == 2.0 ** (1 - 5)
    assert O.fp4_quantise_latent(z + 3e-38, np.zeros((1, 2)))[2] == 2.0 ** -100
    c = z.copy()
    c[0, 3] = np.inf
    codes, s, ts = O.fp4_quantise_latent(np.concatenate([c, z + 1.5], axis=1), np.zeros((1, 2)))
    v = O.fp4_dequantise_latent(codes, s, ts)
    assert np.isnan(v[0, :16]).all() and np.array_equal(v[0, 16:], np.full(16, 1.5))  # scale 8 * 2^-5, code 6


def test_fp4_error_bound_and_scale_invariance():
    c = W.normal(3, 77, 64 * 512).view(64, 512).double().numpy()
    kr = W.normal(3, 78, 64 * 64).view(64, 64).double().numpy()
    codes, s, ts = O.fp4_quantise_latent(c, kr)
    v = O.fp4_dequantise_latent(codes, s, ts)
    step = np.repeat(O.e4m3_decode(s) * ts, 16, axis=1)
    assert np.all(np.abs(v - c) <= step * (1 + 1e-6))  # the widest gap is 2 steps
    c2, s2, ts2 = O.fp4_quantise_latent(c * 2.0 ** 40, kr * 2.0 ** 40)
    assert np.array_equal(c2, codes) and np.array_equal(s2, s) and np.array_equal(ts2, ts * 2.0 ** 40)
    # six significant bits: exact in bf16
    assert np.array_equal(O.to_bf16(v), v)


def test_rms_norm_matches_torch():
    x = W.normal(5, 1, 7 * 48).view(7, 48).double()
    w = W.normal(5, 2, 48).double()
    ref = torch.nn.functional.rms_norm(x, (48,), w, 1e-5)
    assert np.allclose(O.rms_norm(x.numpy(), w.numpy(), 1e-5), ref.numpy(), rtol=1e-13)


def test_fp4_page_layout():
    d = B.dims_for(W.V3_FP8_B128_T2.with_(cache_dtype="fp4"))
    assert B.check_dims(d) == 0
    assert B.cache_page_bytes(d) == PagedLatentCache.layout_page_bytes(d) == 64 * 420
    assert O.cache_bytes_per_token(512, 64, "fp4") == 420
    for kw in (dict(d_c=80, d_rope=6, page_size=7), dict(d_c=16, d_rope=0, page_size=1)):
        d = B.make_dims(4, kw["d_c"], kw["d_rope"], 8, 8, 64, page_size=kw["page_size"], cache="fp4")
        assert B.cache_page_bytes(d) == PagedLatentCache.layout_page_bytes(d) > 0
    # the quantiser's fp32 scratch
    d = B.dims_for(W.V3_FP8_B128_T2.with_(cache_dtype="fp4"))
    assert B.append_workspace_bytes(d, 3) >= 3 * 512 * 4


def test_rows_refusals_before_any_launch():
    L, d = B.lib(), B.dims_for(W.V3_FP8_B128_T2.with_(cache_dtype="fp4"))
    ref = ctypes.byref(d)
    p = lambda x: ctypes.c_void_p(x)  # noqa: E731
    fake = p(0x10000)  # never dereferenced: validation fails first

    def rows(c=fake, cs=512, k=fake, ks=64, w=None, eps=1e-6, n=3, seq=fake, pos=fake, pt=fake, b=1, mp=1, pool=fake,
             pages=1):
        return L.mla_append_rows(ref, c, cs, k, ks, w, eps, n, seq, pos, pt, b, mp, pool, pages, None)

    for kw in (dict(c=None), dict(k=None), dict(cs=511), dict(ks=63), dict(n=-1), dict(seq=None), dict(pos=None),
               dict(pt=None), dict(pool=None), dict(b=0), dict(mp=0), dict(pages=0), dict(w=fake, eps=0.0),
               dict(w=fake, eps=-1.0), dict(w=fake, eps=float("nan")), dict(w=fake, eps=float("inf"))):
        assert rows(**kw) == B.MLA_ERR_INVALID_ARG, kw
    assert rows(pool=p(0x10008)) == B.MLA_ERR_ALIGNMENT
    assert rows(n=0, c=None, k=None, seq=None, pos=None, pt=None, pool=None) == B.MLA_OK

    def read(pool=fake, pages=1, pt=fake, b=1, mp=1, seq=fake, pos=fake, n=3, c=fake, k=fake):
        return L.mla_read_rows(ref, pool, pages, pt, b, mp, seq, pos, n, c, k, None)

    for kw in (dict(pool=None), dict(pages=0), dict(pt=None), dict(b=0), dict(mp=0), dict(seq=None), dict(pos=None),
               dict(n=-1), dict(c=None), dict(k=None)):
        assert read(**kw) == B.MLA_ERR_INVALID_ARG, kw
    assert read(pool=p(0x10008)) == B.MLA_ERR_ALIGNMENT
    assert read(n=0, pool=None, pt=None, seq=None, pos=None, c=None, k=None) == B.MLA_OK
    d.cache_dtype = 4
    assert rows() == B.MLA_ERR_INVALID_ARG and read() == B.MLA_ERR_INVALID_ARG


def test_binding_refuses_wrong_tensors():
    d = B.make_dims(4, 32, 8, 8, 8, 64, cache="fp4")
    x = torch.zeros(3, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on the GPU
        B.mla_append_rows(d, x, x[:, :8], torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                          torch.zeros(1, 1, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8))


@pytest.mark.parametrize("heads", [1, 2, 3, 5])
@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
def test_few_heads_have_a_workspace_size(heads, cache):
    """The automatic split count is defined for head counts below the CUDA-core kernel's group."""
    d = B.make_dims(heads, 512, 64, 128, 128, 7168, cache=cache)
    assert B.auto_splits(d, 1, 1) >= 1
    assert B.decode_workspace_bytes(d, 2, 1, 0) > 0


def test_binding_refuses_another_device_and_other_index_types(monkeypatch):
    class OnDevice:
        def __init__(self, index):
            self.index = index

        def is_contiguous(self):
            return True

        def get_device(self):
            return self.index

    monkeypatch.setattr(B, "_device", lambda: 0)
    B._cuda(OnDevice(0), None)
    with pytest.raises(ValueError, match="cuda:1"):
        B._cuda(OnDevice(0), OnDevice(1))
    i32 = torch.zeros(4, dtype=torch.int32)
    B._index(4, i32.view(2, 2), i32, i32)
    with pytest.raises(ValueError, match="page_table"):
        B._index(4, i32.view(2, 2).long(), i32, i32)
    with pytest.raises(ValueError, match="page_table"):
        B._index(4, i32, i32, i32)
    with pytest.raises(ValueError, match="int32"):
        B._index(4, i32.view(2, 2), i32, i32.long())
