"""mla_append_rows with a norm at the ends of the input type's range: the result, a
latent of the weights' size, is the oracle's bit for bit where it is quantised (the
bars of test_gpu_rows.py)."""
import numpy as np
import pytest
import torch

from latent_compressed_attention_mla_b200 import binding as B
from latent_compressed_attention_mla_b200 import workloads as W
from latent_compressed_attention_mla_b200.paged_cache import PagedLatentCache
from tests.test_gpu_rows import TYPES, Rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size,eps", [(7e37, 1e-6), (1e30, 1e-6), (1e16, 1e-6), (1e-18, 1e-38), (1e-30, 1e-38)])
@pytest.mark.parametrize("d_c,d_rope", [(512, 64), (1024, 16)])
@pytest.mark.parametrize("act,cache", TYPES)
def test_norm_of_very_large_and_small_rows(act, cache, d_c, d_rope, size, eps):
    if act == "f32" and d_c > 512:
        d_c = 384
    r = Rows(act, cache, 200, d_c=d_c, d_rope=d_rope)
    x = W.normal(77, 1, 200 * d_c).view(200, d_c).double() * size
    r.kv[:, :d_c] = x.clamp(-3e38, 3e38).to(r.dt)
    r.append(True, eps)
    r.check(True, float(np.float32(eps)))  # the value that the fp32 argument carries
    assert torch.isfinite(r.kv).all() and B.mla_get_status() == 0


@pytest.mark.parametrize("cache", ["bf16", "fp8", "fp4"])
def test_rows_of_a_page_beyond_32_bits_of_bytes(cache):
    """A page of 2^23 + 64 tokens (one page a sequence): the last rows lie more than
    2^31 bytes into it."""
    size, d_c = (1 << 23) + 64, 512
    pos = torch.tensor([0, 1, size // 2, size - 65, size - 64, size - 2, size - 1], dtype=torch.int32).cuda()
    n = len(pos)
    c = W.normal(78, 1, n * d_c).view(n, d_c).to(torch.bfloat16).cuda()
    kr = W.normal(78, 2, n * 2).view(n, 2).to(torch.bfloat16).cuda()
    seq = torch.zeros(n, dtype=torch.int32).cuda()

    def through(page, at):
        dims = B.make_dims(8, d_c, 2, 128, 128, 512, page_size=page, act="bf16", cache=cache)
        pool = PagedLatentCache(dims, 1, "cuda", fill=0)
        table = torch.zeros(1, 1, dtype=torch.int32).cuda()
        pool.append(c, kr, seq, at, table)
        got = pool.values(seq, at, table)
        return got[0], got[1], pool.views()["kr"][0, at.long()]

    big, small = through(size, pos), through(n, torch.arange(n, dtype=torch.int32).cuda())
    assert torch.equal(big[0], small[0]) and big[0].abs().sum() > 0
    assert torch.equal(big[1], big[2])
    assert B.mla_get_status() == 0
