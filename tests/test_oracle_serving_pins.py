"""Pins of the float64 oracle of the carried convolution and of group norm with a gate (CPU)."""
import numpy as np
import pytest
import torch

import oracle


def rng(s):
    return np.random.Generator(np.random.PCG64(s))


def test_conv_in_pieces_is_the_whole():
    r = rng(1)
    x, w, b = r.normal(size=(2, 11, 3)), r.normal(size=(3, 4)), r.normal(size=3)
    whole = oracle.conv_silu(x, w, b)
    hist, parts = None, []
    for a, e in ((0, 1), (1, 3), (3, 3), (3, 9), (9, 11)):
        o, hist = oracle.conv_carry(x[:, a:e], w, b, hist)
        parts.append(o)
    assert np.allclose(np.concatenate(parts, 1), whole, rtol=1e-14, atol=1e-14)
    assert np.array_equal(hist, x[:, 8:])
    _, h = oracle.conv_carry(x, w, b, None, lens=[1, 5])
    assert np.array_equal(h[0], np.stack([np.zeros(3), np.zeros(3), x[0, 0]]))
    assert np.array_equal(h[1], x[1, 2:5])


@pytest.mark.parametrize("name", ["x", "w", "bias", "hist"])
def test_conv_gradients_by_differences(name):
    r = rng(2)
    a = {"x": r.normal(size=(2, 5, 2)), "w": r.normal(size=(2, 4)), "bias": r.normal(size=2),
         "hist": r.normal(size=(2, 3, 2))}
    dout = r.normal(size=(2, 5, 2))
    dx, dw, db, dh = oracle.conv_carry_backward(a["x"], a["w"], a["bias"], a["hist"], dout)
    g = {"x": dx, "w": dw, "bias": db, "hist": dh}[name]
    h = 1e-6
    for i in np.ndindex(*g.shape):
        v = []
        for s in (h, -h):
            c = {n: t.copy() for n, t in a.items()}
            c[name][i] += s
            v.append(np.sum(dout * oracle.conv_carry(**c)[0]))
        assert abs((v[0] - v[1]) / (2 * h) - g[i]) <= 1e-7 * max(1.0, abs(g[i]))


def test_groupnorm_against_torch():
    r = rng(3)
    rows, G, S = 4, 3, 5
    y, g, dout = (r.normal(size=(rows, G * S)) for _ in range(3))
    ga, be = r.normal(size=G * S), r.normal(size=G * S)
    t = [torch.tensor(v, requires_grad=True) for v in (y, g, ga, be)]
    out = torch.nn.functional.group_norm(t[0], G, t[2], t[3], 1e-5) * torch.nn.functional.silu(t[1])
    assert np.allclose(oracle.groupnorm_gate(y, g, ga, be, G, 1e-5), out.detach().numpy(), atol=1e-13)
    want = torch.autograd.grad(out, t, torch.tensor(dout))
    for got, ref in zip(oracle.groupnorm_gate_backward(y, g, ga, be, G, 1e-5, dout), want):
        assert np.allclose(got, ref.numpy(), rtol=1e-11, atol=1e-11)
