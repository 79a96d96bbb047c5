"""Pins of the masked float64 definitions (oracle/sequence.py) against the
dense oracle, closed forms and finite differences."""

import numpy as np

import oracle


def _draw(seed, nq=5, nk=7, dk=4, dv=3):
    r = np.random.default_rng(seed)
    return r.normal(size=(2, nq, dk)), r.normal(size=(2, nk, dk)), r.normal(size=(2, nk, dv)), r.normal(size=(2, nq, dv))


def test_all_visible_is_the_dense_definition():
    q, k, _, _ = _draw(0, 6, 6)
    v = np.random.default_rng(1).normal(size=(2, 6, 4))
    o, lse = oracle.masked_forward(q, k, v, 0.5, True)
    o2, lse2 = oracle.dense_forward(q, k, v, 0.5)
    assert np.allclose(o, o2, atol=1e-14) and np.allclose(lse, lse2, atol=1e-14)
    do = np.random.default_rng(2).normal(size=o.shape)
    for a, b in zip(oracle.masked_backward(q, k, v, do, 0.5, True), oracle.dense_backward(q, k, v, do, 0.5)):
        assert np.allclose(a, b, atol=1e-13)


def test_new_token_mask():
    assert (oracle.new_token_mask(2, 4) == [[1, 1, 1, 0], [1, 1, 1, 1]]).all()
    assert (oracle.new_token_mask(3, 2) == [[0, 0], [1, 0], [1, 1]]).all()  # the first row sees nothing
    assert (oracle.new_token_mask(1, 1) == [[1]]).all()


def test_rows_that_see_nothing():
    q, k, v, do = _draw(3, 4, 2)
    vis = oracle.new_token_mask(4, 2)
    o, lse = oracle.masked_forward(q, k, v, 0.7, vis)
    assert (o[:, :2] == 0).all() and np.isneginf(lse[:, :2]).all()
    assert np.allclose(o[:, 2], v[:, 0])  # one visible key: its value
    assert np.allclose(lse[:, 2], 0.7 * np.sum(q[:, 2] * k[:, 0], -1))
    dq, _, _ = oracle.masked_backward(q, k, v, do, 0.7, vis)
    assert (dq[:, :3] == 0).all()
    o, lse = oracle.masked_forward(q, k[:, :0], v[:, :0], 0.7, True)
    assert (o == 0).all() and np.isneginf(lse).all()


def test_gradients_against_differences():
    q, k, v, do = _draw(4, 6, 5)
    vis = oracle.new_token_mask(6, 5)
    f = lambda: np.sum(oracle.masked_forward(q, k, v, 0.6, vis)[0] * do)  # noqa: E731
    for x, g in zip((q, k, v), oracle.masked_backward(q, k, v, do, 0.6, vis)):
        num = np.zeros_like(x)
        for i in np.ndindex(*x.shape):
            old = x[i]
            x[i] = old + 1e-5
            up = f()
            x[i] = old - 1e-5
            num[i] = (up - f()) / 2e-5
            x[i] = old
        # central differences: truncation ~ 1e-10, cancellation ~ 1e-16 / 1e-5
        assert np.allclose(num, g, atol=1e-8)
