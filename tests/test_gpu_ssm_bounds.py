"""Memory behaviour of the scan, the carried convolution and group norm: nothing written outside the
outputs, nothing read that was not written (NaN in workspaces and outputs), offsets beyond 2^31
elements, two calls at once on two streams."""
import pytest
import torch

from matrix_state_nonlinear_amd import (m2rnn_conv_carry, m2rnn_conv_carry_bwd, m2rnn_conv_step,
                                        m2rnn_groupnorm_gate, m2rnn_groupnorm_gate_bwd,
                                        m2rnn_ssm_bwd, m2rnn_ssm_fwd, m2rnn_ssm_step,
                                        m2rnn_ssm_workspace_bytes)
from test_gpu_ssm import DEV, DT, NAMES, inputs

pytestmark = pytest.mark.gpu

PAD = 256  # elements before and behind an output


class Guarded:
    """Outputs of NaN inside larger buffers whose margins hold a mark."""

    def __init__(self):
        self.bufs = []

    def __call__(self, t):
        b = torch.full((t.numel() + 2 * PAD,), 7.0, dtype=t.dtype, device=DEV)
        o = b[PAD:PAD + t.numel()].view(t.shape)
        o.fill_(float("nan"))
        self.bufs.append(b)
        return o

    def check(self):
        for b in self.bufs:
            assert torch.all(b[:PAD] == 7.0) and torch.all(b[-PAD:] == 7.0)


def poisoned(nbytes):
    return torch.full((max(nbytes, 16) // 4,), float("nan"), device=DEV)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,N,NQ,K,V", [(1, 1, 1, 1, 1, 1), (2, 65, 4, 2, 40, 24), (1, 300, 2, 1, 64, 64),
                                          (1, 130, 2, 2, 256, 128), (2, 33, 3, 1, 17, 99),
                                          (1, 200, 4, 4, 32, 128), (1, 97, 8, 1, 64, 16)])
def test_scan_writes_its_outputs_only(B, T, N, NQ, K, V, dtype):
    h, d = inputs(B, T, N, NQ, K, V, dtype, seed=T + K)
    a = [d[n] for n in NAMES]
    want = m2rnn_ssm_fwd(*a, H0=d["H0"])
    g = Guarded()
    ws = poisoned(m2rnn_ssm_workspace_bytes(False, B, T, N, NQ, K, V, DT[dtype]))
    got = m2rnn_ssm_fwd(*a, H0=d["H0"], out=tuple(g(t) for t in want), workspace=ws)
    g.check()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    for dHT in (d["dHT"], None):
        want = m2rnn_ssm_bwd(*a, d["H0"], d["dy"], dHT=dHT)
        g = Guarded()
        ws = poisoned(m2rnn_ssm_workspace_bytes(True, B, T, N, NQ, K, V, DT[dtype]))
        got = m2rnn_ssm_bwd(*a, d["H0"], d["dy"], dHT=dHT, workspace=ws,
                            out={n: g(t) for n, t in want.items()})
        g.check()
        assert all(torch.equal(want[n], got[n]) for n in want)
    tok = [t[:, 0].contiguous() if n in ("k", "v", "q", "logit") else t for n, t in zip(NAMES, a)]
    g = Guarded()
    H = g(d["H0"])
    H.copy_(d["H0"])
    H2 = d["H0"].clone()
    y = m2rnn_ssm_step(H, *tok, out=g(torch.zeros(B, N, V, dtype=DT[dtype])))
    assert torch.equal(y, m2rnn_ssm_step(H2, *tok)) and torch.equal(H, H2)
    g.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,C", [(1, 1, 1), (2, 3, 24), (3, 70, 520), (1, 33, 7)])
def test_conv_writes_its_outputs_only(B, T, C, dtype):
    gen = torch.Generator().manual_seed(T + C)
    x, dout = (torch.randn(B, T, C, generator=gen).to(DT[dtype]).to(DEV) for _ in range(2))
    hist = torch.randn(B, 3, C, generator=gen).to(DT[dtype]).to(DEV)
    w, b = torch.randn(C, 4, generator=gen).to(DEV), torch.randn(C, generator=gen).to(DEV)
    want = m2rnn_conv_carry(x, w, b, hist=hist)
    g = Guarded()
    got = m2rnn_conv_carry(x, w, b, hist=hist, out=tuple(g(t) for t in want))
    g.check()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    want = m2rnn_conv_carry_bwd(x, w, b, hist, dout)
    g = Guarded()
    got = m2rnn_conv_carry_bwd(x, w, b, hist, dout, out={n: g(t) for n, t in want.items()},
                               workspace=poisoned(1 << 22))
    g.check()
    assert all(torch.equal(want[n], got[n]) for n in want)
    g = Guarded()
    h, o = g(hist), g(x[:, 0])
    h.copy_(hist)
    m2rnn_conv_step(h, x[:, 0].contiguous(), w, b, out=o)
    g.check()
    assert torch.all(torch.isfinite(o))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,G,S", [(1, 1, 1), (3, 5, 24), (70, 16, 64), (9, 3, 700), (5, 2, 4100)])
def test_groupnorm_writes_its_outputs_only(rows, G, S, dtype):
    gen = torch.Generator().manual_seed(rows + S)
    y, gp, do = (torch.randn(rows, G * S, generator=gen).to(DT[dtype]).to(DEV) for _ in range(3))
    ga, be = (torch.randn(G * S, generator=gen).to(DEV) for _ in range(2))
    want = m2rnn_groupnorm_gate(y, gp, ga, be, G)
    g = Guarded()
    assert torch.equal(m2rnn_groupnorm_gate(y, gp, ga, be, G, out=g(want)), want)
    g.check()
    want = m2rnn_groupnorm_gate_bwd(y, gp, ga, be, G, do)
    g = Guarded()
    got = m2rnn_groupnorm_gate_bwd(y, gp, ga, be, G, do, out=tuple(g(t) for t in want),
                                   workspace=poisoned(1 << 22))
    g.check()
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_scan_beyond_2_31_elements():
    """v and y of 2.2e9 elements: the tokens behind 2^31 equal the same tokens on their own, from the
    state before them (forward) and in the gradients (the tail's own backward)."""
    B, T, N, NQ, K, V = 1, 266240, 64, 1, 16, 128
    cut = 262144                                  # cut * N * V = 2^31
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    k, v, q = r(B, T, NQ, K) * 0.25, r(B, T, N, V), r(B, T, NQ, K)
    x = torch.randn(B, T, N, generator=g, device=DEV)
    p = (torch.full((N,), 4.0, device=DEV), torch.full((N,), -3.0, device=DEV),
         torch.ones(N, V, device=DEV))
    y, HT = m2rnn_ssm_fwd(k, v, q, x, *p)
    head = [t[:, :cut].contiguous() for t in (k, v, q, x)]
    tail = [t[:, cut:].contiguous() for t in (k, v, q, x)]
    _, H1 = m2rnn_ssm_fwd(*head, *p)
    del head
    y2, HT2 = m2rnn_ssm_fwd(*tail, *p, H0=H1)
    # the same sums in other segments: two bf16 steps of y at most, fp32 rounding of the states
    assert torch.allclose(y[:, cut:].float(), y2.float(), rtol=2.0 ** -6, atol=1e-3)
    assert torch.allclose(HT, HT2, rtol=1e-4, atol=1e-4)
    del y, y2
    dy = r(B, T, N, V)
    got = m2rnn_ssm_bwd(k, v, q, x, *p, None, dy, want_dh0=False)
    want = m2rnn_ssm_bwd(*tail, *p, H1, dy[:, cut:].contiguous())
    for n in ("dk", "dv", "dq", "dlogit"):
        a, b = got[n][:, cut:].float(), want[n].float()
        assert (a - b).norm() <= 2.0 ** -7 * b.norm(), n


def test_conv_and_groupnorm_beyond_2_31_elements():
    T, C = (1 << 20) + 40, 2112
    x = torch.randn(1, T, C, device=DEV, dtype=torch.bfloat16)
    w, b = torch.randn(C, 4, device=DEV), torch.randn(C, device=DEV)
    out, last = m2rnn_conv_carry(x, w, b)
    t0 = T - 30
    o2, l2 = m2rnn_conv_carry(x[:, t0:].contiguous(), w, b, hist=x[:, t0 - 3:t0].contiguous())
    assert torch.equal(out[:, t0:], o2) and torch.equal(last, l2)
    del out
    gb = m2rnn_conv_carry_bwd(x, w, b, None, x)
    g2 = m2rnn_conv_carry_bwd(x[:, t0:].contiguous(), w, b, x[:, t0 - 3:t0].contiguous(),
                              x[:, t0:].contiguous())
    assert torch.equal(gb["dx"][:, t0:], g2["dx"])
    del gb
    y = x.view(T, C)
    ga = torch.randn(C, device=DEV)
    out = m2rnn_groupnorm_gate(y, y, ga, b, 33)
    tail = y[t0:].contiguous()
    assert torch.equal(out[t0:], m2rnn_groupnorm_gate(tail, tail, ga, b, 33))
    del out
    dy, dg, _, _ = m2rnn_groupnorm_gate_bwd(y, y, ga, b, 33, y)
    d2 = m2rnn_groupnorm_gate_bwd(tail, tail, ga, b, 33, tail)
    assert torch.equal(dy[t0:], d2[0]) and torch.equal(dg[t0:], d2[1])


def test_two_streams_at_once():
    """Different calls on two streams, overlapping, give what they give alone."""
    jobs = []
    for i, (B, T, N, NQ, K, V) in enumerate([(4, 700, 8, 2, 64, 32), (2, 1500, 4, 4, 32, 64)]):
        h, d = inputs(B, T, N, NQ, K, V, "bf16", seed=i)
        jobs.append(([d[n] for n in NAMES], d))
    alone = [(m2rnn_ssm_fwd(*a, H0=d["H0"]), m2rnn_ssm_bwd(*a, d["H0"], d["dy"], dHT=d["dHT"]))
             for a, d in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(3):
        for i, (a, d) in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                got[i].append((m2rnn_ssm_fwd(*a, H0=d["H0"]),
                               m2rnn_ssm_bwd(*a, d["H0"], d["dy"], dHT=d["dHT"])))
    torch.cuda.synchronize()
    for i, (f, b) in enumerate(alone):
        for f2, b2 in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(f, f2))
            assert all(torch.equal(b[n], b2[n]) for n in b)
