"""Pins of the float64 oracle of the selective state-space scan (CPU): closed forms, the
dense masked product, differences for every gradient."""
import numpy as np
import pytest

import oracle

NAMES = ("k", "v", "q", "logit", "alpha", "beta", "w_r", "H0")


def draw(B, T, N, NQ, K, V, seed):
    r = np.random.Generator(np.random.PCG64(seed))
    return {"k": r.normal(size=(B, T, NQ, K)), "v": r.normal(size=(B, T, N, V)),
            "q": r.normal(size=(B, T, NQ, K)), "logit": r.normal(size=(B, T, N)),
            "alpha": r.uniform(0.1, 2.0, N), "beta": r.uniform(-2.0, 1.0, N),
            "w_r": r.normal(size=(N, V)), "H0": r.normal(size=(B, N, K, V))}


def test_equals_the_dense_masked_product():
    a = draw(2, 9, 4, 2, 3, 5, 1)
    y, HT, _ = oracle.ssm_forward(*(a[n] for n in NAMES))
    d = np.log1p(np.exp(a["logit"] + a["beta"]))
    c = np.cumsum(-a["alpha"] * d, axis=1)
    k, q = np.repeat(a["k"], 2, axis=2), np.repeat(a["q"], 2, axis=2)
    want = a["w_r"] * a["v"] + np.exp(c)[..., None] * np.einsum("btnk,bnkv->btnv", q, a["H0"])
    for t in range(9):
        for s in range(t + 1):
            w = np.exp(c[:, t] - c[:, s]) * d[:, s] * np.sum(q[:, t] * k[:, s], axis=-1)
            want[:, t] += w[..., None] * a["v"][:, s]
    assert np.allclose(y, want, rtol=1e-12, atol=1e-12)


def test_gate_is_the_exp_softplus_gate():
    a = draw(1, 4, 2, 2, 3, 3, 2)
    f = oracle.gates(oracle.GATE_EXP_SOFTPLUS, a["logit"], a["alpha"], a["beta"])
    _, _, st = oracle.ssm_forward(a["k"] * 0, *(a[n] for n in NAMES[1:]))
    for t in range(4):
        assert np.allclose(st[t + 1], f[:, t, :, None, None] * st[t], rtol=1e-13)


def test_masked_tokens_leave_the_state():
    a = draw(1, 5, 2, 1, 3, 4, 3)
    a["logit"][:, 2] = -np.inf
    _, _, st = oracle.ssm_forward(*(a[n] for n in NAMES))
    assert np.array_equal(st[3], st[2])
    g = oracle.ssm_backward(*(a[n] for n in NAMES), dy=np.ones((1, 5, 2, 4)))
    assert np.all(g["dlogit"][:, 2] == 0) and np.all(np.isfinite(g["dH0"]))


def test_pieces_and_steps():
    a = draw(2, 6, 2, 2, 3, 4, 4)
    y, HT, _ = oracle.ssm_forward(*(a[n] for n in NAMES))
    H = a["H0"]
    for t in range(6):
        yt, H = oracle.ssm_step(H, *(a[n][:, t] for n in NAMES[:4]), *(a[n] for n in NAMES[4:7]))
        assert np.allclose(yt, y[:, t], rtol=1e-13, atol=1e-13)
    assert np.allclose(H, HT, rtol=1e-13, atol=1e-13)


@pytest.mark.parametrize("name", NAMES)
def test_gradients_by_differences(name):
    a = draw(2, 5, 4, 2, 3, 2, 5)
    r = np.random.Generator(np.random.PCG64(6))
    dy, dHT = r.normal(size=(2, 5, 4, 2)), r.normal(size=(2, 4, 3, 2))
    g = oracle.ssm_backward(*(a[n] for n in NAMES), dy=dy, dHT=dHT)["d" + name]

    def loss(x):
        y, HT, _ = oracle.ssm_forward(*(x if n == name else a[n] for n in NAMES))
        return np.sum(dy * y) + np.sum(dHT * HT)

    h = 1e-5
    for _ in range(12):
        i = tuple(r.integers(0, s) for s in a[name].shape)
        up, dn = a[name].copy(), a[name].copy()
        up[i] += h
        dn[i] -= h
        # central difference: O(h^2) of third derivatives of order 10, rounding 1e-16 / h
        assert abs((loss(up) - loss(dn)) / (2 * h) - g[i]) <= 1e-7 * max(1.0, abs(g[i])), i
