"""Ways to call the scan and the carried convolution that a serving or training loop uses: states
carried in place, graphs that share a workspace, masks of the type's lowest value, no decay."""
import math

import numpy as np
import pytest
import torch

import oracle
from matrix_state_nonlinear_amd import (m2rnn_conv_carry, m2rnn_groupnorm_gate_bwd, m2rnn_ssm_bwd,
                                        m2rnn_ssm_fwd, m2rnn_ssm_step, m2rnn_ssm_workspace_bytes)
from test_gpu_ssm import DEV, NAMES, check, inputs, magnitude, rel_bound
from test_gpu_ssm_bwd import run

pytestmark = pytest.mark.gpu


# one segment per head, several segments, and no tokens
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,N,K,V", [(100, 70, 8, 20, 24), (64, 65, 16, 64, 128), (2, 1000, 2, 72, 100),
                                       (2, 0, 3, 8, 8)])
def test_scan_state_in_place(B, T, N, K, V, dtype):
    _, d = inputs(B, T, N, 1, K, V, dtype, seed=B + T)
    a = [d[n] for n in NAMES]
    y, HT = m2rnn_ssm_fwd(*a, H0=d["H0"])
    H, y2 = d["H0"].clone(), torch.empty_like(y)
    m2rnn_ssm_fwd(*a, H0=H, out=(y2, H))
    assert torch.equal(y, y2) and torch.equal(H, HT)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,C", [(3, 0, 24), (2, 1, 7), (2, 2, 64), (3, 40, 520)])
def test_conv_history_in_place(B, T, C, dtype):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(B, T, C, generator=g).to(dtype).to(DEV)
    h = torch.randn(B, 3, C, generator=g).to(dtype).to(DEV)
    w = torch.randn(C, 4, generator=g).to(DEV)
    lens = torch.tensor([T, T // 2, 0][:B], dtype=torch.int32, device=DEV)
    for n in (None, lens):
        out, last = m2rnn_conv_carry(x, w, hist=h, lens=n)
        h2, out2 = h.clone(), torch.empty_like(out)
        m2rnn_conv_carry(x, w, hist=h2, lens=n, out=(out2, h2))
        assert torch.equal(out, out2) and torch.equal(h2, last)


def test_two_graphs_share_a_workspace():
    """A forward and a backward captured apart with one workspace, replayed in turn."""
    B, T, N, NQ, K, V = 2, 300, 4, 2, 32, 48
    _, d = inputs(B, T, N, NQ, K, V, "bf16", seed=3)
    a = [d[n] for n in NAMES]
    ws = torch.empty(max(m2rnn_ssm_workspace_bytes(b, B, T, N, NQ, K, V) for b in (False, True)),
                     dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for bwd in (False, True):
        f = ((lambda: m2rnn_ssm_bwd(*a, d["H0"], d["dy"], dHT=d["dHT"], workspace=ws)) if bwd else
             (lambda: dict(zip(("y", "HT"), m2rnn_ssm_fwd(*a, H0=d["H0"], workspace=ws)))))
        f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for i in range(3):
        for n in ("k", "v", "q", "dy"):
            d[n].copy_(torch.randn(d[n].shape, generator=torch.Generator().manual_seed(i)).to(DEV) / 4)
        want = [dict(zip(("y", "HT"), m2rnn_ssm_fwd(*a, H0=d["H0"]))),
                m2rnn_ssm_bwd(*a, d["H0"], d["dy"], dHT=d["dHT"])]
        for j in (0, 1, 1, 0):
            graphs[j].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(outs[j][n], want[j][n]) for n in want[j]), (i, j)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sequences_masked_throughout(dtype):
    """Logits of -inf or of the type's lowest value for all tokens: the state goes through as it
    was, and the gradients through the step sizes are zero."""
    B, T, N, NQ, K, V = 2, 150, 2, 1, 24, 40
    _, d = inputs(B, T, N, NQ, K, V, dtype, seed=4)
    d["logit"][0] = -math.inf
    d["logit"][1] = torch.finfo(torch.float32).min
    a = [d[n] for n in NAMES]
    y, HT = m2rnn_ssm_fwd(*a, H0=d["H0"])
    assert torch.equal(HT, d["H0"])
    g = m2rnn_ssm_bwd(*a, d["H0"], d["dy"], dHT=d["dHT"])
    assert all(torch.isfinite(t).all() for t in (y, *g.values()))
    for n in ("dk", "dlogit", "dalpha", "dbeta"):
        assert torch.count_nonzero(g[n]) == 0, n
    H = d["H0"].clone()
    m2rnn_ssm_step(H, *(d[n][:, 0].contiguous() if n in ("k", "v", "q", "logit") else d[n] for n in NAMES))
    assert torch.equal(H, d["H0"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_heads_without_decay(dtype):
    B, T, N, NQ, K, V = 2, 400, 2, 2, 40, 32
    h, d = inputs(B, T, N, NQ, K, V, dtype, seed=6)
    h["alpha"][0] = 0.0
    d["alpha"][0] = 0.0
    y, HT = m2rnn_ssm_fwd(*(d[n] for n in NAMES), H0=d["H0"])
    ry, rH, _ = oracle.ssm_forward(*(h[n] for n in NAMES), h["H0"])
    m, mH0 = magnitude(h)
    Ay, AH, _ = oracle.ssm_forward(*m, mH0)
    check(y, ry, Ay, rel_bound(T, K, dtype, False), 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, "y")
    check(HT, rH, AH, rel_bound(T, K, dtype), 2.0 ** -24, "HT")
    run(h, d, T, K, V, dtype)


def test_norm_backward_of_one_row_twice():
    """The same rows in one call twice give the same gradients, and twice the parameters'."""
    g = torch.Generator().manual_seed(1)
    y, gp, do = (torch.randn(5, 96, generator=g).to(DEV) for _ in range(3))
    ga, be = torch.randn(96, generator=g).to(DEV), torch.randn(96, generator=g).to(DEV)
    one = m2rnn_groupnorm_gate_bwd(y, gp, ga, be, 4, do)
    two = m2rnn_groupnorm_gate_bwd(*(torch.cat([t, t]) for t in (y, gp)), ga, be, 4, torch.cat([do, do]))
    for i in range(2):
        assert torch.equal(two[i][:5], one[i]) and torch.equal(two[i][5:], one[i])
    for i in (2, 3):  # ten terms of order 1, in another order
        assert np.allclose(two[i].cpu(), 2 * one[i].cpu(), rtol=0, atol=2.0 ** -19 * 10)


# one segment per head and several
SPLITS = [(65, 70, 8, 16, 16), (2, 500, 2, 40, 72)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,N,K,V", SPLITS)
@pytest.mark.parametrize("given", ["H0", "dHT"])
def test_backward_with_one_of_the_states(given, B, T, N, K, V, dtype):
    h, d = inputs(B, T, N, 1, K, V, dtype, seed=T)
    other = "dHT" if given == "H0" else "H0"
    h[other] = d[other] = None
    g, _ = run(h, d, T, K, V, dtype)
    less = m2rnn_ssm_bwd(*(d[n] for n in NAMES), d["H0"], d["dy"], dHT=d["dHT"], want_dh0=False)
    assert less["dH0"] is None
    assert all(torch.equal(g[n], less[n]) for n in g if n != "dH0")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,N,K,V", SPLITS + [(100, 70, 8, 40, 72)])
def test_forward_without_the_last_state(B, T, N, K, V, dtype):
    h, d = inputs(B, T, N, 1, K, V, dtype, seed=T + 1)
    y, HT = m2rnn_ssm_fwd(*(d[n] for n in NAMES), H0=d["H0"], want_ht=False)
    assert HT is None
    assert torch.equal(y, m2rnn_ssm_fwd(*(d[n] for n in NAMES), H0=d["H0"])[0])
    ry, _, _ = oracle.ssm_forward(*(h[n] for n in NAMES), h["H0"])
    m, mH0 = magnitude(h)
    Ay, _, _ = oracle.ssm_forward(*m, mH0)
    check(y, ry, Ay, rel_bound(T, K, dtype, False), 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, "y")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,N,NQ,K,V", [(2, 2000, 4, 4, 32, 128), (1, 1500, 8, 1, 64, 16), (2, 1100, 3, 3, 64, 64)])
@pytest.mark.parametrize("carry", [True, False])
def test_decays_gradients_by_their_norms(B, T, N, NQ, K, V, carry, dtype):
    """The decays' gradients over many chunks and segments, closer than by the sums of absolute
    values: roundings of 2^-24 in sums of some 300 terms add at random to 20 2^-24 = 1e-6 of the
    terms, and terms of both signs leave at least a tenth of their norm: 1e-5."""
    h, d = inputs(B, T, N, NQ, K, V, dtype, seed=T + V, carry=carry)
    g = m2rnn_ssm_bwd(*(d[n] for n in NAMES), d["H0"], d["dy"], dHT=d["dHT"])
    ref = oracle.ssm_backward(*(h[n] for n in NAMES), h["H0"], h["dy"], h["dHT"])
    for n in ("dlogit", "dalpha", "dbeta"):
        e = np.linalg.norm(g[n].cpu().double().numpy() - ref[n]) / np.linalg.norm(ref[n])
        print(n, e)
        assert e <= 1e-5, (n, e)
