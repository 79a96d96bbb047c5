"""Plain float64 definition of the 4-bit key/value cache's format: groups of 16
entries share one e4m3 scale, entries are e2m1 codes.  Test infrastructure only
(see the package docstring for who may import it)."""

from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# non-negative e4m3 numbers by code; the code past the last one is NaN
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def nearest(x, values):
    """Index of the nearest of ascending ``values`` (saturating), ties to the even index."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    with np.errstate(invalid="ignore"):
        dl, dh = x - values[lo], values[hi] - x
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def cache4_quantise(x, scale: float):
    """``(codes, scales)`` of float64 ``x`` [..., d]: e2m1 codes (0..15) and e4m3 codes [..., d/16]."""
    y = np.asarray(x, dtype=np.float64) / scale
    g = y.reshape(*y.shape[:-1], -1, 16)
    nan = np.isnan(g).any(-1)
    amax = np.max(np.where(np.isnan(g), 0.0, np.abs(g)), axis=-1)
    s = nearest(amax / 6.0, E4M3)
    with np.errstate(invalid="ignore", divide="ignore"):
        m = np.where(s[..., None] == 0, 0, nearest(np.abs(g) / E4M3[s][..., None], E2M1))
    codes = m + 8 * ((g < 0) & (m > 0))
    return codes.reshape(y.shape), np.where(nan, 0x7F, s)


def cache4_values(codes, scales, scale: float):
    """What codes [..., d] and scales [..., d/16] stand for."""
    s = np.concatenate([E4M3, [np.nan], -E4M3, [np.nan]])[scales]
    v = np.concatenate([E2M1, -E2M1])[codes]
    return v * np.repeat(s, 16, axis=-1) * scale


def cache4_pack(k_codes, k_scales, v_codes, v_scales):
    """The 18 d bytes of a block from codes [16, d] and scales [16, d/16] of its 16 tokens."""
    d = k_codes.shape[-1]
    two = lambda c: (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)  # noqa: E731
    k = two(k_codes.reshape(16, d // 16, 16)).transpose(1, 0, 2)
    return np.concatenate([k.ravel(), k_scales.astype(np.uint8).ravel(), two(v_codes.T).ravel(),
                           v_scales.T.astype(np.uint8).ravel()])


def cache4_unpack(block, d: int):
    """``(k_codes, k_scales, v_codes, v_scales)`` of a block's bytes."""
    kc, ks, vc, vs = np.split(np.asarray(block).astype(np.int64), [8 * d, 9 * d, 17 * d])
    each = lambda b: np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)  # noqa: E731
    return (each(kc.reshape(d // 16, 16, 8)).transpose(1, 0, 2).reshape(16, d), ks.reshape(16, d // 16),
            each(vc.reshape(d, 8)).T, vs.reshape(d // 16, 16).T)
