"""Sizes and scales at the limits of the 4-bit cache's entry points, refused on
the host before any CUDA call (the pointers are fake)."""

import pytest

from tests.test_abi_cache4_host import attend, b, read, write  # noqa: F401  (b: a fixture)


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("kw", [
    dict(Hkv=1 << 30, Nn=2), dict(Hkv=(1 << 31) - 1, Nn=2), dict(Hkv=1 << 20, Nn=1 << 15),
])
def test_blocks_of_a_sequence_pass_31_bits(b, call, kw):
    """Heads times the blocks of 16 tokens that the rows can touch."""
    assert call(b, B=1, n_pages=1, page=16, max_pages=1, d=16, **kw) == 1


@pytest.mark.parametrize("scale,ks", [(1e-20, 1e-20), (2.0 ** -126, 0.5), (3e38, 1.0), (2.0 ** 100, 2.0 ** 27.9)])
@pytest.mark.parametrize("d", [128, 80])
def test_scales_whose_product_is_no_normal_number(b, scale, ks, d):
    """scale k_scale, and 1 / ln 2 times that, are what scores are multiplied with, in float32."""
    assert attend(b, scale=scale, ks=ks, d=d) == 1
