"""Plain float64 definitions of attention with a visibility mask, key and
value widths of their own, and rows that may see nothing.  Test
infrastructure only (see the package docstring for who may import it).

``visible`` is a boolean array broadcastable to ``[..., Nq, Nk]``: True where
a query row sees a key.  A row that sees none has ``O = 0``, ``lse = -inf`` and
no gradient.  Only visible keys enter any sum, so whatever stands at a key
that no row sees (NaN included) has no effect.
"""

from __future__ import annotations

import numpy as np


def _f64(x) -> np.ndarray:
    return np.asarray(x, dtype=np.float64)


def new_token_mask(n_q: int, n_k: int) -> np.ndarray:
    """Rows are the last ``n_q`` of ``n_k`` tokens; each sees the keys up to its own."""
    return np.arange(n_k)[None, :] <= np.arange(n_q)[:, None] + (n_k - n_q)


def masked_probabilities(q, k, scale: float, visible):
    """``P`` (zero where masked) and ``lse``."""
    s = np.matmul(_f64(q), np.swapaxes(_f64(k), -1, -2)) * float(scale)
    visible = np.broadcast_to(visible, s.shape)
    s = np.where(visible, s, -np.inf)
    m = np.max(s, axis=-1, keepdims=True) if s.shape[-1] else np.full(s.shape[:-1] + (1,), -np.inf)
    ref = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(s - ref)
    l = np.sum(e, axis=-1, keepdims=True)
    p = e / np.where(l == 0, 1.0, l)
    with np.errstate(divide="ignore"):
        lse = (ref + np.log(l))[..., 0]
    return p, lse


def masked_forward(q, k, v, scale: float, visible):
    """``O = softmax(S) V`` over the visible keys, and ``lse``."""
    p, lse = masked_probabilities(q, k, scale, visible)
    return np.matmul(p, _f64(v)), lse


def masked_backward(q, k, v, do, scale: float, visible):
    """``(dQ, dK, dV)``: the derivative of ``masked_forward``'s O."""
    q, k, v, do = _f64(q), _f64(k), _f64(v), _f64(do)
    p, _ = masked_probabilities(q, k, scale, visible)
    dv = np.matmul(np.swapaxes(p, -1, -2), do)
    dp = np.matmul(do, np.swapaxes(v, -1, -2))
    ds = p * (dp - np.sum(p * dp, axis=-1, keepdims=True))
    return float(scale) * np.matmul(ds, k), float(scale) * np.matmul(np.swapaxes(ds, -1, -2), q), dv
