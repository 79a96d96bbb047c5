"""Error bounds of the language-model operators against the float64 oracle,
element by element, from the roundings that the kernels make.

Written for a row's exact P_j (normalised), S_j, O, and |.| taken entry-wise:

* a score is a dot product of dk products summed in fp32 in some order: its
  error is at most ``ds = (dk + 8) 2^-22 scale sum_c |q_c k_c|`` (2^-22 a step:
  fp32's half step 2^-24 with a factor for sums that truncate instead of
  rounding);
* exp, the row sum over n keys and the merge of parts add a relative error of
  at most ``(n + 64) 2^-23`` to any P_j (a sum of n terms of one sign);
* so a P_j before its rounding is off by a factor within
  ``e = 2 ds + (n + 64) 2^-23``;
* bf16: P_j is rounded to bf16, half a step u = 2^-8 relative, before it
  multiplies V, and the normaliser may be the sum of the rounded or of the
  unrounded P: each entry of O is off by at most ``(2 u + e) sum_j P_j |v_j|``;
  the fp32 sum over the keys is within the same e; the output's own rounding
  adds u |O|.  float32: u = 0 for P and 2^-24 for the output.
* lse: ``ds + (n + 64) 2^-23`` and fp32's half step of the result.
* backward: D = sum_c dO_c O_c uses the rounded O, so it is off by at most
  ``sum_c |dO_c| tol_O_c`` plus fp32 sums; dP is a dot product of dv products;
  dS = P (dP - D) is rounded to bf16 once (u |dS|), P once for dV; every
  gradient is an fp32 sum of products of those with exact bf16 operands, and
  is rounded to its type once.
"""

import numpy as np

import oracle

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def forward(q, k, v, scale, visible, dtype):
    """(O, lse, tolerance of O, tolerance of lse); all arrays float64 [..., N, d]."""
    u = HALF[dtype] if dtype == "bf16" else 0.0
    p, lse = oracle.masked_probabilities(q, k, scale, visible)
    o = np.matmul(p, v)
    ds, e = _score_errors(q, k, scale, visible)
    tol_o = (2 * u + e) * np.matmul(p, np.abs(v)) + HALF[dtype] * np.abs(o) + 1e-30
    tol_l = e[..., 0] + 2.0 ** -24 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return o, lse, tol_o, tol_l


def _score_errors(q, k, scale, visible):
    """Row-wise (max over the visible keys) ds and e, as [..., N, 1]."""
    a = np.matmul(np.abs(q), np.abs(np.swapaxes(k, -1, -2)))
    a = np.where(np.broadcast_to(visible, a.shape), a, 0.0)
    n = np.sum(np.broadcast_to(visible, a.shape), axis=-1, keepdims=True)
    ds = (q.shape[-1] + 8) * 2.0 ** -22 * scale * (np.max(a, axis=-1, keepdims=True) if a.shape[-1] else 0.0 * n)
    return ds, 2 * ds + (n + 64) * 2.0 ** -23


def backward(q, k, v, do, scale, visible, dtype):
    """((dQ, dK, dV), their tolerances) per head, before any sum over heads and
    without the outputs' own rounding (the caller adds HALF * |gradient|)."""
    u = HALF[dtype] if dtype == "bf16" else 0.0
    p, _ = oracle.masked_probabilities(q, k, scale, visible)
    o, _, tol_o, _ = forward(q, k, v, scale, visible, dtype)
    _, e = _score_errors(q, k, scale, visible)
    grads = oracle.masked_backward(q, k, v, do, scale, visible)
    dp = np.matmul(do, np.swapaxes(v, -1, -2))
    adp = np.matmul(np.abs(do), np.abs(np.swapaxes(v, -1, -2)))
    d = np.sum(p * dp, axis=-1, keepdims=True)
    sums = (v.shape[-1] + 8) * 2.0 ** -22
    err_d = np.sum(np.abs(do) * (tol_o + sums * np.abs(o)), axis=-1, keepdims=True)
    ds = p * (dp - d)
    err_ds = p * (err_d + sums * adp) + (u + 2 * e) * (np.abs(ds) + p * (err_d + sums * adp))
    t = lambda x: np.swapaxes(x, -1, -2)  # noqa: E731
    n_q, n_k = p.shape[-2:]
    sum_k, sum_q = (n_k + 64) * 2.0 ** -22, (n_q + 64) * 2.0 ** -22
    tol_q = scale * (np.matmul(err_ds, np.abs(k)) + sum_k * np.matmul(np.abs(ds), np.abs(k)))
    tol_k = scale * (np.matmul(t(err_ds), np.abs(q)) + sum_q * np.matmul(t(np.abs(ds)), np.abs(q)))
    err_p = (u + 2 * e) * p
    tol_v = np.matmul(t(err_p), np.abs(do)) + sum_q * np.matmul(t(p), np.abs(do))
    return grads, (tol_q, tol_k, tol_v)


def check(name, got, want, tol):
    """Every element within its tolerance; infinities equal, no NaN."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert not np.isnan(got).any(), f"{name}: NaN"
    inf = np.isinf(want)
    assert (got[inf] == want[inf]).all(), f"{name}: infinite entries differ"
    err = np.abs(np.where(inf, 0.0, got) - np.where(inf, 0.0, want))
    worst = np.unravel_index(np.argmax(err / np.broadcast_to(tol, err.shape)), err.shape) if err.size else ()
    assert err.size == 0 or (err <= tol).all(), (
        f"{name}: {(err > tol).sum()} of {err.size} elements out of tolerance, worst at {worst}: "
        f"got {got[worst]}, want {want[worst]}, tolerance {np.broadcast_to(tol, err.shape)[worst]}")


def f64(t):
    return t.detach().double().cpu().numpy()
