"""GPU parity of the selective state-space scan against the float64 oracle, through the C
ABI: forward, and the run in pieces.

Tolerances, before rounding to the output type.  A is the same quantity computed by the
oracle from absolute values (every term of a sum counts with its size), so an error of r
relative to each term is at most r A.  Per term:
  * the fp32 sums: at most n additions of relative error 2^-24 each, with n <= K (the
    scores) + 3 * 64 (a chunk's inputs, and the state's update) + 4 T / 32 (a product and
    a sum for each chunk, two per rounding, that the state passes);
  * softplus and each power: a few 2^-24, and d's relative error 2^-23 in the exponent
    c = -alpha sum d moves a term by |c| 2^-23, where a term with |c| > 17 is below 2^-24
    of its undecayed size: 64 * 2^-24 covers both;
  * bf16 inputs: the scores and the state enter their products as two bf16 terms, the first
    truncated (below 2^-7), the second rounded to nearest (2^-9 of what is left, 2^-8 of
    it at a power of two): 2^-15 for each of the two.
fp32 inputs are three terms each, exact to 24 bits, with products below 2^-24 left out
(counted three times: 2^-22).  A bf16 result is then rounded once: 2^-8 relative.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from matrix_state_nonlinear_amd import m2rnn_ssm_fwd

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def inputs(B, T, N, NQ, K, V, dtype, seed, carry=True, strong=False):
    """Host float64 arrays (values exact in the device types) and device tensors."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    u = lambda *s: torch.rand(s, generator=g)   # noqa: E731
    dt = DT[dtype]
    d0 = torch.exp(u(N) * math.log(100.0) + math.log(1e-2 if strong else 1e-3))
    t = {"k": (r(B, T, NQ, K) / math.sqrt(K)).to(dt), "v": r(B, T, N, V).to(dt),
         "q": r(B, T, NQ, K).to(dt), "logit": r(B, T, N) * (2.0 if strong else 1.0),
         "alpha": (1.0 + 15.0 * u(N)) * (4.0 if strong else 1.0),
         "beta": d0 + torch.log(-torch.expm1(-d0)), "w_r": 1.0 + 0.1 * r(N, V)}
    t["H0"] = u(B, N, K, V) - 0.5 if carry else None
    t["dy"] = r(B, T, N, V).to(dt)
    t["dHT"] = r(B, N, K, V) if carry else None
    host = {n: None if x is None else x.double().numpy() for n, x in t.items()}
    dev = {n: None if x is None else x.to(DEV) for n, x in t.items()}
    return host, dev


def np_(t):
    return t.detach().cpu().double().numpy()


NAMES = ("k", "v", "q", "logit", "alpha", "beta", "w_r")


def rel_bound(T, K, dtype, states=True):
    n = K + 3 * 64 + 4 * math.ceil(T / 32)
    return (n + 64) * 2.0 ** -24 + (2 * 2.0 ** -15 if dtype == "bf16" and not states
                                    else 2.0 ** -22)


def magnitude(h):
    """The oracle on absolute values (alpha, logit and beta set the decays and stay)."""
    a = {n: np.abs(h[n]) if n not in ("logit", "alpha", "beta") else h[n] for n in NAMES}
    return [a[n] for n in NAMES], None if h["H0"] is None else np.abs(h["H0"])


def check(got, ref, A, rel, out_rel, name):
    err = np.abs(np_(got) - ref)
    bound = out_rel * np.abs(ref) + rel * A * (1 + out_rel) + 1e-30
    assert np.all(np.isfinite(np_(got))), name
    assert np.all(err <= bound), (name, float(np.max(err / bound)))
    return float(np.max(err / bound))


SIZES = [  # B, T, N, NQ, K, V
    (1, 1, 1, 1, 1, 1), (2, 3, 2, 1, 5, 7), (1, 31, 3, 3, 16, 16), (2, 32, 2, 2, 33, 24),
    (1, 33, 4, 2, 64, 64), (1, 63, 2, 1, 100, 40), (1, 64, 1, 1, 128, 128), (2, 65, 3, 1, 40, 65),
    (1, 129, 2, 2, 200, 100), (1, 130, 2, 1, 256, 128), (1, 700, 2, 1, 64, 20),
    (1, 1029, 1, 1, 32, 128), (3, 257, 2, 2, 72, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,N,NQ,K,V", SIZES)
@pytest.mark.parametrize("carry", [True, False])
def test_forward(B, T, N, NQ, K, V, dtype, carry):
    h, d = inputs(B, T, N, NQ, K, V, dtype, seed=T * 1000 + K + V, carry=carry)
    y, HT = m2rnn_ssm_fwd(*(d[n] for n in NAMES), H0=d["H0"])
    torch.cuda.synchronize()
    ry, rH, _ = oracle.ssm_forward(*(h[n] for n in NAMES), h["H0"])
    a, aH0 = magnitude(h)
    Ay, AH, _ = oracle.ssm_forward(*a, aH0)
    e = [check(y, ry, Ay, rel_bound(T, K, dtype, False), 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24,
               "y"),
         check(HT, rH, AH, rel_bound(T, K, dtype), 2.0 ** -24, "HT")]
    print(f"{(B, T, N, NQ, K, V)} {dtype}: share of the bound {e[0]:.2f} {e[1]:.2f}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward_strong_decay_and_masked_tokens(dtype):
    """Decays down to zero within a token, and tokens with logit -inf that leave the state."""
    B, T, N, NQ, K, V = 2, 300, 2, 1, 48, 32
    h, d = inputs(B, T, N, NQ, K, V, dtype, seed=5, strong=True)
    mask = np.zeros((B, T, N), bool)
    mask[0, 60:70] = True
    mask[1, 200:] = True
    mask[:, 128, 0] = True
    h["logit"][mask] = -np.inf
    h["logit"][0, 100, :] = 300.0   # alpha d of hundreds: f = 0
    d["logit"] = torch.from_numpy(h["logit"]).float().to(DEV)
    y, HT = m2rnn_ssm_fwd(*(d[n] for n in NAMES), H0=d["H0"])
    ry, rH, _ = oracle.ssm_forward(*(h[n] for n in NAMES), h["H0"])
    a, aH0 = magnitude(h)
    Ay, AH, _ = oracle.ssm_forward(*a, aH0)
    check(y, ry, Ay, rel_bound(T, K, dtype, False), 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24, "y")
    check(HT, rH, AH, rel_bound(T, K, dtype), 2.0 ** -24, "HT")
    # a padded prompt ends with the state of its last real token
    cut = {n: d[n][1:2, :200].contiguous() if n in ("k", "v", "q", "logit") else d[n] for n in NAMES}
    _, H1 = m2rnn_ssm_fwd(*(cut[n] for n in NAMES), H0=d["H0"][1:2].contiguous())
    check(H1, rH[1:2], AH[1:2], rel_bound(T, K, dtype), 2.0 ** -24, "HT of the padded prompt")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward_elements_off_16_byte_addresses(dtype):
    """Tensors aligned to their element only, with odd widths next to even ones."""
    B, T, N, NQ, K, V = 1, 100, 2, 1, 32, 64
    h, d = inputs(B, T, N, NQ, K, V, dtype, seed=9)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        s = buf[1:].view(t.shape)
        s.copy_(t)
        return s

    want = m2rnn_ssm_fwd(*(d[n] for n in NAMES), H0=d["H0"])
    s = {n: shifted(d[n]) for n in NAMES + ("H0",)}
    out = (shifted(torch.zeros_like(want[0])), shifted(torch.zeros_like(want[1])))
    got = m2rnn_ssm_fwd(*(s[n] for n in NAMES), H0=s["H0"], out=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_forward_in_pieces_and_again():
    """A prompt in pieces, each from the state before, is the prompt; a repeat is bitwise equal."""
    B, T, N, NQ, K, V = 2, 513, 2, 1, 64, 32
    h, d = inputs(B, T, N, NQ, K, V, "fp32", seed=11)
    y, HT = m2rnn_ssm_fwd(*(d[n] for n in NAMES), H0=d["H0"])
    y2, HT2 = m2rnn_ssm_fwd(*(d[n] for n in NAMES), H0=d["H0"])
    assert torch.equal(y, y2) and torch.equal(HT, HT2)
    ry, rH, _ = oracle.ssm_forward(*(h[n] for n in NAMES), h["H0"])
    a, aH0 = magnitude(h)
    Ay, AH, _ = oracle.ssm_forward(*a, aH0)
    H, parts = d["H0"], []
    for t0, t1 in ((0, 1), (1, 65), (65, 200), (200, 513)):
        p = [d[n][:, t0:t1].contiguous() if n in ("k", "v", "q", "logit") else d[n] for n in NAMES]
        yp, H = m2rnn_ssm_fwd(*p, H0=H)
        parts.append(yp)
    check(torch.cat(parts, 1), ry, Ay, rel_bound(T, K, "fp32"), 2.0 ** -24, "y")
    check(H, rH, AH, rel_bound(T, K, "fp32"), 2.0 ** -24, "HT")


def test_forward_empty_calls():
    h, d = inputs(2, 1, 3, 3, 8, 8, "fp32", seed=1)
    z = {n: d[n][:, :0].contiguous() if n in ("k", "v", "q", "logit") else d[n] for n in NAMES}
    y, HT = m2rnn_ssm_fwd(*(z[n] for n in NAMES), H0=d["H0"])
    assert y.shape == (2, 0, 3, 8) and torch.equal(HT, d["H0"])
    _, HT = m2rnn_ssm_fwd(*(z[n] for n in NAMES))
    assert torch.equal(HT, torch.zeros_like(HT))
