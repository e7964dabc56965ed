"""GPU parity of the selective state-space scan's backward against the float64 oracle (itself
held to differences on the CPU), and the layer's training step end to end.

Tolerances: as in test_gpu_ssm.py, r A with A the same gradient computed by the oracle from
absolute values.  The decays' gradient is computed from the telescoped sum
    dl_t = sum_{i >= t} (u_i - z_i) + <H_end, R_end>,  u = q . dq, z = k . dk
within a segment, so its A is the same sum of the absolute u and z over all later tokens
(plus <|H_T|, |dHT|>): an upper bound of the segment's, since <H_end, R_end> of absolute
values is at most that sum over the tokens behind the segment.
"""
import numpy as np
import pytest
import torch

import oracle
from matrix_state_nonlinear_amd import m2rnn_ssm_bwd, m2rnn_ssm_fwd
from test_gpu_ssm import DEV, NAMES, check, inputs, magnitude, rel_bound

pytestmark = pytest.mark.gpu


def reference(h):
    """The oracle's gradients and, for each, the A of the bound."""
    ref = oracle.ssm_backward(*(h[n] for n in NAMES), h["H0"], h["dy"], h["dHT"])
    a, aH0 = magnitude(h)
    ady = np.abs(h["dy"])
    adH = None if h["dHT"] is None else np.abs(h["dHT"])
    A = oracle.ssm_backward(*a, aH0, ady, adH)
    B, T, NQ, K = h["k"].shape
    N, V = h["v"].shape[2:]
    G = N // NQ
    # per value head: u and z of absolute values
    rep = lambda x: np.repeat(x, G, axis=2)  # noqa: E731
    per = oracle.ssm_backward(rep(a[0]), a[1], rep(a[2]), *a[3:], aH0, ady, adH)
    u = np.sum(rep(a[2]) * per["dq"], axis=-1)
    z = np.sum(rep(a[0]) * per["dk"], axis=-1)
    later = np.cumsum((u + z)[:, ::-1], axis=1)[:, ::-1]
    if adH is not None:
        _, AH, _ = oracle.ssm_forward(*a, aH0)
        later = later + np.sum(AH * adH, axis=(2, 3))[:, None]
    x = h["logit"] + h["beta"]
    d = np.logaddexp(0.0, x)
    sig = np.exp(-np.logaddexp(0.0, -x))
    with np.errstate(divide="ignore", invalid="ignore"):
        dd = np.where(d > 0, z / d, 0.0)
    A["dlogit"] = sig * (dd + h["alpha"] * later)
    A["dbeta"] = np.sum(A["dlogit"], axis=(0, 1))
    A["dalpha"] = np.sum(d * later, axis=(0, 1))
    return ref, A


def run(h, d, T, K, V, dtype, **kw):
    g = m2rnn_ssm_bwd(*(d[n] for n in NAMES), d["H0"], d["dy"], dHT=d["dHT"], **kw)
    torch.cuda.synchronize()
    ref, A = reference(h)
    share = {}
    for n, r in ref.items():
        io = n in ("dk", "dv", "dq") and dtype == "bf16"
        # sums over the batch and time add at most B T more roundings in double and one in fp32
        share[n] = check(g[n], r, A[n], rel_bound(T, max(K, V), dtype, n == "dH0"),
                         2.0 ** -8 if io else 2.0 ** -22, n)
    return g, share


SIZES = [  # B, T, N, NQ, K, V
    (1, 1, 1, 1, 1, 1), (2, 3, 2, 1, 5, 7), (1, 31, 3, 3, 16, 16), (2, 33, 2, 2, 33, 24),
    (1, 64, 4, 2, 64, 64), (2, 65, 3, 1, 40, 65), (1, 63, 2, 1, 100, 40), (1, 128, 1, 1, 128, 128),
    (1, 129, 2, 2, 200, 100), (1, 130, 2, 1, 256, 128), (1, 700, 2, 1, 64, 20), (3, 257, 2, 2, 72, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("carry", [True, False])
@pytest.mark.parametrize("B,T,N,NQ,K,V", SIZES)
def test_backward(B, T, N, NQ, K, V, carry, dtype):
    h, d = inputs(B, T, N, NQ, K, V, dtype, seed=T * 1000 + K + V + 1, carry=carry)
    g, share = run(h, d, T, K, V, dtype)
    print(f"{(B, T, N, NQ, K, V)} {dtype}: " + " ".join(f"{n} {s:.2f}" for n, s in share.items()))
    again = m2rnn_ssm_bwd(*(d[n] for n in NAMES), d["H0"], d["dy"], dHT=d["dHT"])
    assert all(torch.equal(g[n], again[n]) for n in g)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_many_sequences_one_segment_each(dtype):
    """Enough heads that T is not split: the states start from H0 without a first pass."""
    h, d = inputs(65, 70, 8, 2, 16, 16, dtype, seed=3, carry=False)
    run(h, d, 70, 16, 16, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_strong_decay_and_masked_tokens(dtype):
    B, T, N, NQ, K, V = 2, 300, 2, 1, 48, 32
    h, d = inputs(B, T, N, NQ, K, V, dtype, seed=5, strong=True)
    mask = np.zeros((B, T, N), bool)
    mask[0, 60:70] = True
    mask[1, 200:] = True
    mask[:, 128, 0] = True
    h["logit"][mask] = -np.inf
    h["logit"][0, 100, :] = 300.0
    d["logit"] = torch.from_numpy(h["logit"]).float().to(DEV)
    g, _ = run(h, d, T, K, V, dtype)
    assert torch.all(g["dlogit"].cpu()[torch.from_numpy(mask)] == 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_elements_off_16_byte_addresses(dtype):
    B, T, N, NQ, K, V = 1, 100, 2, 1, 32, 64
    h, d = inputs(B, T, N, NQ, K, V, dtype, seed=9)

    def shifted(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape)
        s.copy_(t)
        return s

    want = m2rnn_ssm_bwd(*(d[n] for n in NAMES), d["H0"], d["dy"], dHT=d["dHT"])
    s = {n: shifted(t) for n, t in d.items()}
    got = m2rnn_ssm_bwd(*(s[n] for n in NAMES), s["H0"], s["dy"], dHT=s["dHT"],
                        out={n: shifted(torch.zeros_like(t)) for n, t in want.items()})
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_backward_matches_differences_of_the_forward():
    """A directional derivative of the GPU forward (fp32) against the GPU gradients."""
    B, T, N, NQ, K, V = 1, 90, 2, 1, 24, 20
    h, d = inputs(B, T, N, NQ, K, V, "fp32", seed=21)
    g = m2rnn_ssm_bwd(*(d[n] for n in NAMES), d["H0"], d["dy"], dHT=d["dHT"])
    gen = torch.Generator().manual_seed(4)
    step = 2.0 ** -7
    for n in NAMES + ("H0",):
        e = torch.randn(d[n].shape, generator=gen).to(DEV)
        loss = []
        for s in (step, -step):
            x = dict(d, **{n: d[n] + s * e})
            y, HT = m2rnn_ssm_fwd(*(x[m] for m in NAMES), H0=x["H0"])
            loss.append((y.double() * d["dy"].double()).sum() + (HT.double() * d["dHT"].double()).sum())
        diff = float((loss[0] - loss[1]) / (2 * step))
        grad = float((g["d" + n].double() * e.double()).sum())
        # the loss is linear in k, v, q, w_r, H0; in the decays the error of the difference is
        # step^2 times third derivatives (alpha up to 16): 1e-2 of the gradient's size.  The
        # forward's fp32 rounding is 2^-24 of sums of some 1e4, over 2 step.
        scale = float((g["d" + n].double() * e.double()).abs().sum())
        assert abs(diff - grad) <= 1e-2 * scale + 1e4 * 2.0 ** -24 / (2 * step), (n, diff, grad)


def test_backward_empty_calls():
    h, d = inputs(2, 1, 3, 3, 8, 8, "fp32", seed=1)
    z = {n: d[n][:, :0].contiguous() if n in ("k", "v", "q", "logit") else d[n] for n in NAMES}
    g = m2rnn_ssm_bwd(*(z[n] for n in NAMES), d["H0"], d["dy"][:, :0].contiguous(), dHT=d["dHT"])
    assert torch.equal(g["dH0"], d["dHT"])
    for n in ("dw_r", "dalpha", "dbeta"):
        assert torch.count_nonzero(g[n]) == 0
