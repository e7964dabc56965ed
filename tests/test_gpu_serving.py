"""GPU parity of the single-token scan, the carried convolution and group norm with a gate against
the float64 oracle, and the layer end to end: a prompt, then tokens, equal to one prompt.

Tolerances (before one rounding of 2^-8 for bf16 results).  SiLU and its derivative are
formed from exp(-|u|) by a base-2 exponential of |u| log2(e) in fp32: relative error
(|u| + 4) 2^-23 in the exponential, at most that in the sigmoid and, times |u|, in SiLU'.
A few roundings of 2^-24 come with each. `act(u)` below is that bound, (4 + |u|)^2 2^-23, relative to
the magnitude of the terms.  Sums of n terms add n 2^-24.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from matrix_state_nonlinear_amd import (m2rnn_conv_carry, m2rnn_conv_carry_bwd, m2rnn_conv_silu,
                                        m2rnn_conv_step, m2rnn_groupnorm_gate,
                                        m2rnn_groupnorm_gate_bwd, m2rnn_ssm_bwd, m2rnn_ssm_fwd,
                                        m2rnn_ssm_step)
from test_gpu_ssm import DEV, DT, NAMES, inputs, magnitude, np_

pytestmark = pytest.mark.gpu


def out_rel(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24


def within(got, ref, bound, dtype, name):
    err = np.abs(np_(got) - ref)
    b = out_rel(dtype) * np.abs(ref) + bound * (1 + out_rel(dtype)) + 1e-30
    assert np.all(np.isfinite(np_(got))), name
    assert np.all(err <= b), (name, float(np.max(err / b)))


def act(u):
    return (4.0 + np.abs(u)) ** 2 * 2.0 ** -23


# ------------------------------------------------------------------ scan, one token

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,N,NQ,K,V", [(1, 1, 1, 1, 1), (3, 2, 1, 5, 7), (2, 4, 2, 64, 64),
                                        (5, 6, 3, 33, 65), (1, 64, 1, 64, 16), (2, 2, 2, 256, 128),
                                        (7, 3, 1, 100, 100), (600, 1, 1, 16, 20), (130, 4, 4, 64, 64)])
def test_step(B, N, NQ, K, V, dtype):
    h, d = inputs(B, 1, N, NQ, K, V, dtype, seed=B + N + K + V)
    if B > 2:
        h["logit"][1] = -np.inf
        d["logit"][1] = -math.inf
    tok = {n: d[n][:, 0].contiguous() if n in ("k", "v", "q", "logit") else d[n] for n in NAMES}
    H = d["H0"].clone()
    y = m2rnn_ssm_step(H, *(tok[n] for n in NAMES))
    ry, rH, _ = oracle.ssm_forward(*(h[n] for n in NAMES), h["H0"])
    a, aH0 = magnitude(h)
    Ay, AH, _ = oracle.ssm_forward(*a, aH0)
    # the state: softplus, one power and two products (64 roundings cover them); y: K more terms
    within(y, ry[:, 0], (K + 70) * 2.0 ** -24 * Ay[:, 0], dtype, "y")
    within(H, rH, 70 * 2.0 ** -24 * AH, "fp32", "H")
    if B > 2:
        assert torch.equal(H[1], d["H0"][1])


def test_step_elements_off_16_byte_addresses():
    h, d = inputs(3, 1, 2, 1, 32, 64, "bf16", seed=2)
    tok = {n: d[n][:, 0].contiguous() if n in ("k", "v", "q", "logit") else d[n] for n in NAMES}

    def shifted(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape)
        s.copy_(t)
        return s

    H, Hs = d["H0"].clone(), shifted(d["H0"])
    y = m2rnn_ssm_step(H, *(tok[n] for n in NAMES))
    ys = m2rnn_ssm_step(Hs, *(shifted(tok[n]) for n in NAMES))
    # the columns' sums run in another order there
    assert torch.equal(H, Hs) and torch.allclose(y.float(), ys.float(), rtol=2.0 ** -7, atol=1e-5)


# ------------------------------------------------------------------ convolution

def conv_inputs(B, T, C, dtype, seed, bias, hist):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dt = DT[dtype]
    t = {"x": r(B, T, C).to(dt), "w": 0.5 * r(C, 4), "bias": 0.1 * r(C) if bias else None,
         "hist": r(B, 3, C).to(dt) if hist else None, "dout": r(B, T, C).to(dt)}
    return ({n: None if v is None else v.double().numpy() for n, v in t.items()},
            {n: None if v is None else v.to(DEV) for n, v in t.items()})


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bias,hist", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("B,T,C", [(1, 1, 1), (2, 1, 8), (3, 2, 7), (2, 3, 64), (1, 4, 520),
                                   (2, 31, 72), (2, 33, 513), (1, 130, 1030), (5, 64, 24)])
def test_conv(B, T, C, bias, hist, dtype):
    h, d = conv_inputs(B, T, C, dtype, B + T + C, bias, hist)
    lens = torch.tensor([(i * 7 + 1) % (T + 2) - (i == 2) for i in range(B)], dtype=torch.int32)
    out, last = m2rnn_conv_carry(d["x"], d["w"], d["bias"], hist=d["hist"], lens=lens.to(DEV))
    plain, last0 = m2rnn_conv_carry(d["x"], d["w"], d["bias"], hist=d["hist"])
    g = m2rnn_conv_carry_bwd(d["x"], d["w"], d["bias"], d["hist"], d["dout"])
    torch.cuda.synchronize()
    assert torch.equal(out, plain)
    ro, rl = oracle.conv_carry(h["x"], h["w"], h["bias"], h["hist"], lens.tolist())
    assert np.array_equal(np_(last), rl)
    assert np.array_equal(np_(last0), oracle.conv_carry(h["x"], h["w"], h["bias"], h["hist"])[1])
    # sizes of u's terms, and of the gradients' with |SiLU'| <= 1.1
    z = np.zeros((B, 3, C)) if h["hist"] is None else h["hist"]
    full = np.abs(np.concatenate([z, h["x"]], 1))
    Au = sum(np.abs(h["w"][:, i]) * full[:, i:i + T] for i in range(4))
    Au = Au + (0 if h["bias"] is None else np.abs(h["bias"]))
    a = act(Au)
    within(out, ro, 2 * a * Au, dtype, "out")
    rdx, rdw, rdb, rdh = oracle.conv_carry_backward(h["x"], h["w"], h["bias"], h["hist"], h["dout"])
    du = 1.1 * np.abs(h["dout"]) * (4 * a + act(Au) * Au)  # error of du
    dA = 1.1 * np.abs(h["dout"])
    e = np.zeros((B, T + 3, C))
    for i in range(4):
        e[:, i:i + T] += np.abs(h["w"][:, i]) * (du + 8 * 2.0 ** -24 * dA)
    within(g["dx"], rdx, e[:, 3:], dtype, "dx")
    n = 32 + 4 + B * math.ceil(T / 32) / 64 + 17
    rel = du + n * 2.0 ** -24 * dA
    within(g["dw"], rdw, np.stack([(rel * full[:, i:i + T]).sum((0, 1)) for i in range(4)], 1),
           "fp32", "dw")
    if bias:
        within(g["dbias"], rdb, rel.sum((0, 1)), "fp32", "dbias")
    else:
        assert g["dbias"] is None
    if hist:
        within(g["dhist"], rdh, e[:, :3], dtype, "dhist")
    else:
        assert g["dhist"] is None
        # without history: m2rnn_conv_silu's definition
        same = m2rnn_conv_silu(d["x"], d["w"], d["bias"])
        within(same, ro, 2 * a * Au, dtype, "conv_silu")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,C", [(1, 1), (3, 8), (512, 64), (2, 1030), (5, 7)])
def test_conv_step_continues_the_prompt(B, C, dtype):
    h, d = conv_inputs(B, 9, C, dtype, B + C, True, True)
    ro, rl = oracle.conv_carry(h["x"], h["w"], h["bias"], h["hist"])
    full = np.abs(np.concatenate([h["hist"], h["x"]], 1))
    Au = sum(np.abs(h["w"][:, i]) * full[:, i:i + 9] for i in range(4)) + np.abs(h["bias"])
    _, hist = m2rnn_conv_carry(d["x"][:, :4].contiguous(), d["w"], d["bias"], hist=d["hist"])
    for t in range(4, 9):
        o = m2rnn_conv_step(hist, d["x"][:, t].contiguous(), d["w"], d["bias"])
        within(o, ro[:, t], (2 * act(Au) * Au)[:, t], dtype, t)
    assert np.array_equal(np_(hist), rl)


def test_conv_empty_calls():
    h, d = conv_inputs(2, 1, 5, "bf16", 1, True, True)
    x0 = d["x"][:, :0].contiguous()
    _, last = m2rnn_conv_carry(x0, d["w"], d["bias"], hist=d["hist"])
    assert torch.equal(last, d["hist"])
    _, last = m2rnn_conv_carry(x0, d["w"], d["bias"])
    assert torch.count_nonzero(last) == 0
    g = m2rnn_conv_carry_bwd(x0, d["w"], d["bias"], d["hist"], d["dout"][:, :0].contiguous())
    assert all(torch.count_nonzero(t) == 0 for t in g.values())


# ------------------------------------------------------------------ group norm

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,G,S", [(1, 1, 1), (3, 1, 16), (5, 16, 64), (70, 3, 24), (4, 7, 23),
                                      (200, 64, 16), (9, 5, 150), (33, 2, 1024), (3, 1, 700),
                                      (17, 1, 4096), (2, 3, 2500), (1000, 1, 8), (300, 70, 1)])
def test_groupnorm(rows, G, S, dtype):
    g = torch.Generator().manual_seed(rows + G + S)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    D, dt, eps = G * S, DT[dtype], 1e-5
    t = {"y": (0.5 * r(rows, D) + 0.3).to(dt), "g": r(rows, D).to(dt), "ga": 1 + 0.2 * r(D),
         "be": 0.1 * r(D), "dout": r(rows, D).to(dt)}
    h = {n: v.double().numpy() for n, v in t.items()}
    d = {n: v.to(DEV) for n, v in t.items()}
    out = m2rnn_groupnorm_gate(d["y"], d["g"], d["ga"], d["be"], G, eps=eps)
    got = m2rnn_groupnorm_gate_bwd(d["y"], d["g"], d["ga"], d["be"], G, d["dout"], eps=eps)
    torch.cuda.synchronize()
    # z: a group's sums have at most 40 serial additions (a lane's 32 elements and 6 exchanges; 4096
    # channels on 256 threads 16 + 8), so the mean is off by 40 2^-24 max|y| =: m, each centred value by
    # m + 2^-24 |y|, the variance by 2 m sd + 40 2^-24 var, 1 / sqrt by half that relatively
    yg = h["y"].reshape(rows, G, S)
    rs = 1 / np.sqrt(yg.var(-1, keepdims=True) + eps)
    z = (yg - yg.mean(-1, keepdims=True)) * rs
    m = 41 * 2.0 ** -24 * np.abs(yg).max(-1, keepdims=True)
    ez = (rs * m * (1 + np.abs(z)) + np.abs(z) * 44 * 2.0 ** -24).reshape(rows, D)
    ers = ((rs * m + 22 * 2.0 ** -24) * np.ones_like(z)).reshape(rows, D)  # relative, of rs
    zf = z.reshape(rows, D)
    a = h["ga"] * zf + h["be"]
    aA = np.abs(h["ga"] * zf) + np.abs(h["be"])
    ea = np.abs(h["ga"]) * ez + 2 * 2.0 ** -24 * aA
    sil = np.abs(oracle.silu(h["g"])) + 1e-30
    ag = act(h["g"])
    within(out, oracle.groupnorm_gate(h["y"], h["g"], h["ga"], h["be"], G, eps),
           ea * sil + aA * ag * np.abs(h["g"]), dtype, "out")
    ref = oracle.groupnorm_gate_backward(h["y"], h["g"], h["ga"], h["be"], G, eps, h["dout"])
    dA = np.abs(h["dout"])
    within(got[1], ref[1], dA * (1.1 * ea + aA * ag * (1 + np.abs(h["g"]))), dtype, "dg_pre")
    da, eda = dA * sil, dA * np.abs(h["g"]) * ag
    n = (40 + 128 + rows / 16) * 2.0 ** -24  # a wave's rows, its exchanges, every sixteenth block
    within(got[2], ref[2], (da * ez + eda * np.abs(zf) + n * da * np.abs(zf)).sum(0), "fp32", "dgamma")
    within(got[3], ref[3], (eda + n * da).sum(0), "fp32", "dbeta")
    dz, edz = np.abs(h["ga"]) * da, np.abs(h["ga"]) * (eda + 2 * 2.0 ** -24 * da)
    mean = lambda v: np.broadcast_to(v.reshape(rows, G, S).mean(-1, keepdims=True), z.shape).reshape(rows, D)  # noqa: E731
    size = dz + mean(dz) + np.abs(zf) * mean(dz * np.abs(zf))
    rsf = (rs * np.ones_like(z)).reshape(rows, D)
    err = rsf * (edz + mean(edz) + np.abs(zf) * mean(edz * np.abs(zf) + dz * ez) + ez * mean(dz * np.abs(zf))
                 + (ers + 44 * 2.0 ** -24) * size)
    within(got[0], ref[0], err, dtype, "dy")


def test_groupnorm_off_16_byte_addresses_and_empty():
    g = torch.Generator().manual_seed(1)
    y, gp, do = (torch.randn(37, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(3))
    ga, be = torch.rand(128, generator=g).to(DEV), torch.rand(128, generator=g).to(DEV)

    def shifted(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape)
        s.copy_(t)
        return s

    want = (m2rnn_groupnorm_gate(y, gp, ga, be, 2),) + m2rnn_groupnorm_gate_bwd(y, gp, ga, be, 2, do)
    s = [shifted(t) for t in (y, gp, ga, be)]
    got = (m2rnn_groupnorm_gate(*s, 2),) + m2rnn_groupnorm_gate_bwd(*s, 2, shifted(do))
    for a, b in zip(want, got):  # another order of the sums
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-4)
    e = y[:0]
    assert m2rnn_groupnorm_gate(e, e, ga, be, 2).shape == (0, 128)
    r = m2rnn_groupnorm_gate_bwd(e, e, ga, be, 2, e)
    assert torch.count_nonzero(r[2]) == 0 and torch.count_nonzero(r[3]) == 0


# ------------------------------------------------------------------ the layer

class Layer:
    """The state-space layer between its projections: q, k, v each through the convolution, the
    scan, the per-head norm with the gate."""

    def __init__(self, N, NQ, K, V, seed):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g).to(DEV)  # noqa: E731
        self.N, self.NQ, self.K, self.V = N, NQ, K, V
        self.C = {"k": NQ * K, "v": N * V, "q": NQ * K}
        self.w = {n: 0.5 * r(c, 4) for n, c in self.C.items()}
        self.b = {n: 0.1 * r(c) for n, c in self.C.items()}
        self.alpha = 1 + 3 * torch.rand(N, generator=g).to(DEV)
        self.beta, self.w_r = r(N) - 2, 1 + 0.1 * r(N, V)
        self.gamma, self.nbeta = 1 + 0.1 * r(N * V), 0.1 * r(N * V)

    def heads(self, n, x):
        return x.view(*x.shape[:-1], self.NQ if n != "v" else self.N, self.V if n == "v" else self.K)

    def prompt(self, x, logit, g, hist=None, H=None, lens=None):
        u, hist2 = {}, {}
        for n in ("k", "v", "q"):
            u[n], hist2[n] = m2rnn_conv_carry(x[n], self.w[n], self.b[n],
                                              hist=None if hist is None else hist[n], lens=lens)
        y, H2 = m2rnn_ssm_fwd(*(self.heads(n, u[n]) for n in ("k", "v", "q")), logit, self.alpha,
                              self.beta, self.w_r, H0=H)
        out = m2rnn_groupnorm_gate(y.flatten(2), g, self.gamma, self.nbeta, self.N)
        return out, hist2, H2

    def token(self, x, logit, g, hist, H):
        u = {n: m2rnn_conv_step(hist[n], x[n], self.w[n], self.b[n]) for n in ("k", "v", "q")}
        y = m2rnn_ssm_step(H, *(self.heads(n, u[n]) for n in ("k", "v", "q")), logit, self.alpha,
                           self.beta, self.w_r)
        return m2rnn_groupnorm_gate(y.flatten(1), g, self.gamma, self.nbeta, self.N)

    def inputs(self, B, T, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        x = {n: torch.randn(B, T, c, generator=g).to(dtype).to(DEV) for n, c in self.C.items()}
        return (x, torch.randn(B, T, self.N, generator=g).to(DEV),
                torch.randn(B, T, self.N * self.V, generator=g).to(dtype).to(DEV))


def test_layer_prompt_then_tokens_is_one_prompt():
    """A padded batch of two prompts, then eight tokens each, against whole prompts; fp32, in
    which the two differ by the order of sums: 1e-4 of outputs of order 1 after a norm."""
    L = Layer(4, 2, 24, 16, seed=1)
    x, logit, g = L.inputs(2, 60, torch.float32, seed=2)
    lens = [45, 52]
    whole = []
    for b in range(2):
        one = lambda t, e: t[b:b + 1, :e].contiguous()  # noqa: E731
        whole.append(L.prompt({n: one(t, lens[b] + 8) for n, t in x.items()},
                              one(logit, lens[b] + 8), one(g, lens[b] + 8)))
    pad = logit[:, :52].clone()
    pad[0, 45:] = -math.inf
    cut = lambda t: t[:, :52].contiguous()  # noqa: E731
    out, hist, H = L.prompt({n: cut(t) for n, t in x.items()}, pad, cut(g),
                            lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    for b in range(2):
        assert torch.allclose(out[b, :lens[b]], whole[b][0][0, :lens[b]], rtol=1e-4, atol=1e-4)
    for i in range(8):
        at = lambda t: torch.stack([t[b, lens[b] + i] for b in range(2)])  # noqa: E731
        o = L.token({n: at(t) for n, t in x.items()}, at(logit), at(g), hist, H)
        for b in range(2):
            assert torch.allclose(o[b], whole[b][0][0, lens[b] + i], rtol=1e-4, atol=1e-4), (b, i)
    for b in range(2):
        assert torch.allclose(H[b], whole[b][2][0], rtol=1e-4, atol=1e-5)
        assert all(torch.equal(hist[n][b], whole[b][1][n][0]) for n in hist)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_layer_training_step_against_autograd_in_64_bits(dtype):
    """Gradients of the layer's inputs and parameters through all backward calls, against torch's
    autograd of the same layer in float64 written token by token."""
    N, NQ, K, V, B, T = 2, 1, 12, 8, 2, 40
    L = Layer(N, NQ, K, V, seed=3)
    x, logit, g = L.inputs(B, T, DT[dtype], seed=4)
    gen = torch.Generator().manual_seed(5)
    dout = torch.randn(B, T, N * V, generator=gen).to(DT[dtype]).to(DEV)
    u = {n: m2rnn_conv_carry(x[n], L.w[n], L.b[n])[0] for n in x}
    kvq = [L.heads(n, u[n]) for n in ("k", "v", "q")]
    y, _ = m2rnn_ssm_fwd(*kvq, logit, L.alpha, L.beta, L.w_r)
    dy, dg, dgamma, dnbeta = m2rnn_groupnorm_gate_bwd(y.flatten(2), g, L.gamma, L.nbeta, N, dout)
    s = m2rnn_ssm_bwd(*kvq, logit, L.alpha, L.beta, L.w_r, None, dy.view(B, T, N, V), want_dh0=False)
    got = {"g": dg, "gamma": dgamma, "nbeta": dnbeta, "logit": s["dlogit"], "alpha": s["dalpha"],
           "beta": s["dbeta"], "w_r": s["dw_r"]}
    for n in ("k", "v", "q"):
        c = m2rnn_conv_carry_bwd(x[n], L.w[n], L.b[n], None, s["d" + n].flatten(2))
        got.update({"x" + n: c["dx"], "w" + n: c["dw"], "b" + n: c["dbias"]})

    leaf = {"g": g, "gamma": L.gamma, "nbeta": L.nbeta, "logit": logit, "alpha": L.alpha,
            "beta": L.beta, "w_r": L.w_r}
    for n in x:
        leaf.update({"x" + n: x[n], "w" + n: L.w[n], "b" + n: L.b[n]})
    leaf = {n: t.double().cpu().requires_grad_(True) for n, t in leaf.items()}
    v = {}
    for n in x:
        f = torch.nn.functional.pad(leaf["x" + n], (0, 0, 3, 0))
        z = sum(leaf["w" + n][:, i] * f[:, i:i + T] for i in range(4)) + leaf["b" + n]
        v[n] = L.heads(n, torch.nn.functional.silu(z))
    d = torch.nn.functional.softplus(leaf["logit"] + leaf["beta"])
    H, ys = torch.zeros(B, N, K, V, dtype=torch.float64), []
    for t in range(T):
        kt, qt = (v[n][:, t].repeat_interleave(N // NQ, 1) for n in ("k", "q"))
        H = (torch.exp(-leaf["alpha"] * d[:, t])[..., None, None] * H
             + (d[:, t][..., None] * kt)[..., None] * v["v"][:, t][:, :, None, :])
        ys.append((H * qt[..., None]).sum(2) + leaf["w_r"] * v["v"][:, t])
    yd = torch.stack(ys, 1).reshape(B * T, N * V)
    out = torch.nn.functional.group_norm(yd, N, leaf["gamma"], leaf["nbeta"], 1e-5)
    out = out.reshape(B, T, N * V) * torch.nn.functional.silu(leaf["g"])
    want = dict(zip(leaf, torch.autograd.grad(out, list(leaf.values()), dout.double().cpu())))
    # bf16: u, y, dy, dk/dv/dq and dx are rounded between the calls, five roundings of 2^-8 with
    # at most a factor 4 from the norm of small groups; fp32: sums of some hundred terms
    tol = 4 * 5 * 2.0 ** -8 if dtype == "bf16" else 1e-4
    for n, r in want.items():
        e = (got[n].double().cpu().reshape(r.shape) - r).norm() / r.norm()
        assert e <= tol, (n, float(e))


def test_layer_captured_and_replayed():
    """A token of the layer and a training window in a graph, replayed with the program's own
    eager work in between: every replay equals the eager calls."""
    L = Layer(4, 1, 32, 16, seed=6)
    x, logit, g = L.inputs(3, 9, torch.bfloat16, seed=7)
    tok = lambda t, i: t[:, i].contiguous()  # noqa: E731
    _, hist0, H0 = L.prompt({n: t[:, :4].contiguous() for n, t in x.items()},
                            logit[:, :4].contiguous(), g[:, :4].contiguous())
    dy = torch.randn(3, 9, 4, 16, device=DEV).to(torch.bfloat16)
    kvq = [L.heads(n, x[n]) for n in ("k", "v", "q")]
    a = (logit, L.alpha, L.beta, L.w_r)
    buf = {n: tok(t, 4) for n, t in x.items()}
    bl, bg = tok(logit, 4), tok(g, 4)
    hist, H = {n: t.clone() for n, t in hist0.items()}, H0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.token(buf, bl, bg, hist, H)
        m2rnn_ssm_bwd(*kvq, *a, None, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = L.token(buf, bl, bg, hist, H)
        grads = m2rnn_ssm_bwd(*kvq, *a, None, dy)
    for n in hist:
        hist[n].copy_(hist0[n])
    H.copy_(H0)
    eh, eH = {n: t.clone() for n, t in hist0.items()}, H0.clone()
    for i in range(4, 9):
        want = L.token({n: tok(t, i) for n, t in x.items()}, tok(logit, i), tok(g, i), eh, eH)
        wg = m2rnn_ssm_bwd(*kvq, *a, None, dy)
        for n in buf:
            buf[n].copy_(tok(x[n], i))
        bl.copy_(tok(logit, i))
        bg.copy_(tok(g, i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(H, eH), i
        assert all(torch.equal(hist[n], eh[n]) for n in hist)
        assert all(torch.equal(grads[n], wg[n]) for n in wg)
