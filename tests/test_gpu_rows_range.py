"""mla_append_rows with a norm at the ends of the input type's range: the result, a
latent of the weights' size, is the oracle's bit for bit where it is quantised (the
bars of test_gpu_rows.py)."""
import numpy as np
import pytest
import torch

from latent_compressed_attention_mla_b200 import binding as B
from latent_compressed_attention_mla_b200 import workloads as W
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
