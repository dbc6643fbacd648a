"""Decode over a 4-bit cache on the tensor cores with other query widths than 128 (whose
absorption runs on the CUDA cores, into the same operand types), with other RoPE bases
and softmax scales, against the oracle."""
import pytest

from tests.test_gpu_fp4 import check, fp4_cfg, tc_path

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d_nope", [8, 64, 120])
@pytest.mark.parametrize("heads,T", [(8, 1), (5, 3), (40, 2), (128, 1)])
def test_other_query_widths(heads, T, d_nope):
    check(fp4_cfg(n_heads=heads, B=3, T=T, L=(0, 63, 700), d_nope=d_nope), path=tc_path(heads, T))


@pytest.mark.parametrize("heads,T", [(8, 2), (40, 2)])
def test_other_rope_base(heads, T):
    check(fp4_cfg(n_heads=heads, B=2, T=T, L=(5, 700), rope_base=500000.0), path=tc_path(heads, T))


@pytest.mark.parametrize("heads", [8, 40])
def test_many_sequences(heads):
    """More sequences than splits, pages and CTAs: each CTA walks several."""
    check(fp4_cfg(n_heads=heads, B=333, T=1, L=tuple(i % 67 for i in range(333))), path=tc_path(heads, 1))
