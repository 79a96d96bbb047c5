"""Pins of the 4-bit cache's oracle: number formats against torch's, rounding
against a search over every value, packing against a layout written out by hand."""

import numpy as np
import pytest

import oracle
from oracle import cache4

torch = pytest.importorskip("torch")


def test_scale_numbers_are_torchs_e4m3():
    codes = torch.arange(127, dtype=torch.uint8)
    assert (codes.view(torch.float8_e4m3fn).double().numpy() == cache4.E4M3).all()


def test_rounding_is_torchs_e4m3():
    x = torch.cat([torch.linspace(0, 460, 5001), torch.rand(5000, generator=torch.Generator().manual_seed(0)) * 0.1,
                   torch.tensor([2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 448.0])]).clamp(max=448.0)
    got = cache4.E4M3[cache4.nearest(x.double().numpy(), cache4.E4M3)]
    assert (got == x.to(torch.float8_e4m3fn).double().numpy()).all()


def test_nearest_code_by_search():
    x = np.concatenate([np.linspace(0, 8, 4001), (cache4.E2M1[1:] + cache4.E2M1[:-1]) / 2])
    d = np.abs(x[:, None] - cache4.E2M1)
    best = d.min(1, keepdims=True)
    for i, got in enumerate(cache4.nearest(x, cache4.E2M1)):
        ties = np.flatnonzero(d[i] == best[i])
        assert got == (ties[0] if len(ties) == 1 else [t for t in ties if t % 2 == 0][0])


@pytest.mark.parametrize("scale", [1.0, 0.03])
def test_error_of_an_entry(scale):
    """Half the widest gap (6 - 4) of what amax / 6 rounds to, and saturation where s is rounded down."""
    x = np.random.default_rng(0).standard_normal((50, 64))
    codes, s = oracle.cache4_quantise(x, scale)
    got = oracle.cache4_values(codes, s, scale)
    amax = np.repeat(np.abs(x.reshape(50, 4, 16)).max(-1), 16, axis=-1)
    assert (np.abs(got - x) <= amax / 6 * (1 + 2.0 ** -4) + scale * 2.0 ** -9).all()
    assert (np.sign(got) * np.sign(x) >= 0).all()


def test_special_groups():
    x = np.zeros((5, 16))
    x[1, 3] = np.nan
    x[2, 5] = -np.inf
    x[3] = 1e-5
    x[4, :2] = 1e9, 3.0
    codes, s = oracle.cache4_quantise(x, 1.0)
    v = oracle.cache4_values(codes, s, 1.0)
    assert (v[0] == 0).all() and np.isnan(v[1]).all() and v[2, 5] == -2688 and (v[2, :5] == 0).all()
    assert (v[3] == 0).all() and v[4, 0] == 2688


def test_layout_of_a_block():
    d = 32
    rng = np.random.default_rng(1)
    kc, vc = rng.integers(0, 16, (16, d)), rng.integers(0, 16, (16, d))
    ks, vs = rng.integers(0, 256, (16, 2)), rng.integers(0, 256, (16, 2))
    block = oracle.cache4_pack(kc, ks, vc, vs)
    assert block.shape == (18 * d,)
    for t in range(16):
        for c in range(d):
            kb = block[c // 16 * 128 + t * 8 + c % 16 // 2]
            assert (kb >> (4 * (c % 2))) & 15 == kc[t, c]
            vb = block[9 * d + c * 8 + t // 2]
            assert (vb >> (4 * (t % 2))) & 15 == vc[t, c]
            assert block[8 * d + t * 2 + c // 16] == ks[t, c // 16]
            assert block[17 * d + c // 16 * 16 + t] == vs[t, c // 16]
    for a, b in zip(oracle.cache4_unpack(block, d), (kc, ks, vc, vs)):
        assert (a == b).all()
