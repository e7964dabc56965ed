"""Host-side checks of the state-space scan, the carried convolution and group norm with a gate
(no GPU needed, nothing is launched): statuses, workspace sizes, and what the binding refuses."""
import math

import pytest
import torch

import matrix_state_nonlinear_amd as m
from matrix_state_nonlinear_amd import _lib as E

FAKE = 0x1000  # never dereferenced: every call below is rejected on the host


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(E.LIB_PATH):
        from matrix_state_nonlinear_amd import build
        build.build()
    return E.lib()


def sizes(kw, **default):
    a = dict(default, **kw)
    a["NQ"] = a["N"] if a.get("NQ") is None else a["NQ"]
    return a


def fwd(L, **kw):
    a = sizes(kw, B=2, T=8, N=2, NQ=None, K=16, V=16, dt=E.M2RNN_F32, k=FAKE, v=FAKE, q=FAKE, x=FAKE,
              al=FAKE, be=FAKE, w=FAKE, H0=None, y=FAKE, HT=None, ws=FAKE, wsb=1 << 40)
    return L.m2rnn_ssm_fwd(*(a[n] for n in ("B", "T", "N", "NQ", "K", "V", "dt", "k", "v", "q", "x",
                                            "al", "be", "w", "H0", "y", "HT", "ws", "wsb")), None)


def bwd(L, **kw):
    a = sizes(kw, B=2, T=8, N=2, NQ=None, K=16, V=16, dt=E.M2RNN_F32, k=FAKE, v=FAKE, q=FAKE, x=FAKE,
              al=FAKE, be=FAKE, w=FAKE, H0=None, dy=FAKE, dHT=None, dk=FAKE, dv=FAKE, dq=FAKE,
              dx=FAKE, dw=FAKE, da=FAKE, db=FAKE, dH0=None, ws=FAKE, wsb=1 << 40)
    return L.m2rnn_ssm_bwd(*(a[n] for n in ("B", "T", "N", "NQ", "K", "V", "dt", "k", "v", "q", "x",
                                            "al", "be", "w", "H0", "dy", "dHT", "dk", "dv", "dq", "dx",
                                            "dw", "da", "db", "dH0", "ws", "wsb")), None)


def step(L, **kw):
    a = sizes(kw, B=2, N=2, NQ=None, K=16, V=16, dt=E.M2RNN_F32, k=FAKE, v=FAKE, q=FAKE, x=FAKE,
              al=FAKE, be=FAKE, w=FAKE, H=FAKE, y=FAKE)
    return L.m2rnn_ssm_step(*(a[n] for n in ("B", "N", "NQ", "K", "V", "dt", "k", "v", "q", "x", "al",
                                             "be", "w", "H", "y")), None)


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_scan_refuses(L, call):
    bad, uns = E.M2RNN_ERR_INVALID_ARG, E.M2RNN_ERR_UNSUPPORTED
    for kw in ({"B": -1}, {"N": -1}, {"K": 0}, {"V": 0}, {"N": 4, "NQ": 3}, {"N": 4, "NQ": 0},
               {"N": 0, "NQ": 1}, {"dt": 7}, {"dt": -1}):
        assert call(L, **kw) == bad, kw
    for n in ("k", "v", "q", "x", "al", "be", "w"):
        assert call(L, **{n: None}) == bad, n
    for kw in ({"K": 257}, {"V": 129}, {"dt": E.M2RNN_F64}, {"B": 1 << 20, "N": 64}):
        assert call(L, **kw) == uns, kw


def test_scan_refuses_outputs_and_workspaces(L):
    bad = E.M2RNN_ERR_INVALID_ARG
    assert fwd(L, T=-1) == bad and bwd(L, T=-1) == bad
    assert fwd(L, y=None) == bad and step(L, y=None) == bad and step(L, H=None) == bad
    for n in ("dy", "dk", "dv", "dq", "dx", "dw", "da", "db"):
        assert bwd(L, **{n: None}) == bad, n
    assert fwd(L, T=1 << 30) == E.M2RNN_ERR_UNSUPPORTED
    assert bwd(L, B=1 << 10, N=1 << 11, T=1 << 20) == E.M2RNN_ERR_UNSUPPORTED
    # more workgroups than a launch holds, of the pass over 64 tokens x 16 heads
    for call in (fwd, bwd):
        assert call(L, B=1 << 11, T=1 << 19, N=1, K=1, V=1) == E.M2RNN_ERR_UNSUPPORTED
        # and of the sums over heads x 64 columns
        assert call(L, B=1, T=8, N=1 << 21, K=1, V=128) == E.M2RNN_ERR_UNSUPPORTED
    for call, is_bwd in ((fwd, 0), (bwd, 1)):
        need = L.m2rnn_ssm_workspace_bytes(is_bwd, 2, 8, 2, 2, 16, 16, E.M2RNN_F32)
        assert need > 0
        assert call(L, ws=None) == E.M2RNN_ERR_WORKSPACE
        assert call(L, wsb=need - 1) == E.M2RNN_ERR_WORKSPACE
        assert call(L, ws=FAKE + 4) == bad
    # nothing to do: nothing is needed
    assert step(L, B=0, k=None, v=None, q=None, x=None, al=None, be=None, w=None, H=None,
                y=None) == E.M2RNN_OK
    assert fwd(L, B=0, k=None, v=None, q=None, x=None, al=None, be=None, w=None, y=None, ws=None,
               wsb=0) == E.M2RNN_OK


def test_scan_workspace_sizes(L):
    ws = L.m2rnn_ssm_workspace_bytes
    pad = lambda n: (n + 63) // 64 * 64  # noqa: E731
    # many heads: the decays' sums (double) and the step sizes of every token, no segments
    assert ws(0, 64, 100, 16, 16, 64, 64, E.M2RNN_BF16) == 4 * 3 * 64 * 16 * 100
    # one head, 640 tokens: ten segments of states as well
    assert ws(0, 1, 640, 1, 1, 64, 64, E.M2RNN_BF16) == \
        (4 * (2 * 640 + 640 + 10 * 64 * 64 + 64) + 255) // 256 * 256
    # the backward with shared heads keeps per-head dq and dk
    extra = ws(1, 2, 640, 4, 1, 32, 64, E.M2RNN_BF16) - ws(1, 2, 640, 4, 4, 32, 64, E.M2RNN_BF16)
    assert extra == 2 * 4 * pad(2 * 640 * 4 * 32)
    for a in ((0, 2, 0, 2, 2, 16, 16), (0, -1, 5, 2, 2, 16, 16), (1, 2, 5, 2, 2, 300, 16),
              (1, 2, 5, 4, 3, 16, 16)):
        assert ws(*a, E.M2RNN_F32) == 0, a
    assert ws(0, 2, 5, 2, 2, 16, 16, E.M2RNN_F64) == 0


def test_conv_refuses(L):
    bad, uns = E.M2RNN_ERR_INVALID_ARG, E.M2RNN_ERR_UNSUPPORTED

    def carry(**kw):
        a = dict(dict(B=2, T=5, C=8, dt=E.M2RNN_F32, x=FAKE, w=FAKE, b=None, h=None, lens=None, o=FAKE,
                      ho=FAKE), **kw)
        return L.m2rnn_conv_carry(*a.values(), None)

    def back(**kw):
        a = dict(dict(B=2, T=5, C=8, dt=E.M2RNN_F32, x=FAKE, w=FAKE, b=None, h=None, do=FAKE, dx=FAKE,
                      dw=FAKE, db=None, dh=None, ws=FAKE, wsb=1 << 40), **kw)
        return L.m2rnn_conv_carry_bwd(*a.values(), None)

    def one(**kw):
        a = dict(dict(B=2, C=8, dt=E.M2RNN_F32, x=FAKE, w=FAKE, b=None, h=FAKE, o=FAKE), **kw)
        return L.m2rnn_conv_step(*a.values(), None)

    for call in (carry, back, one):
        for kw in ({"B": -1}, {"C": 0}, {"dt": 9}, {"x": None}, {"w": None}):
            assert call(**kw) == bad, (call, kw)
        assert call(dt=E.M2RNN_F64) == uns
        assert call(B=1 << 30, C=1 << 20) == uns
    assert carry(T=-1) == bad and carry(o=None) == bad and carry(lens=FAKE, ho=None) == bad
    assert back(dw=None) == bad and back(dx=None) == bad and back(do=None) == bad
    assert back(b=FAKE) == bad and back(db=FAKE) == bad and back(dh=FAKE) == bad
    assert one(h=None) == bad and one(o=None) == bad
    need = L.m2rnn_conv_carry_workspace_bytes(2, 5, 8)
    assert need == 4 * 5 * 8 // 256 * 256 + 256  # two runs in one group: one row of partials
    assert back(wsb=need - 1) == E.M2RNN_ERR_WORKSPACE and back(ws=None) == E.M2RNN_ERR_WORKSPACE
    assert back(ws=FAKE + 8) == bad
    assert L.m2rnn_conv_carry_workspace_bytes(2, 0, 8) == 0


def test_groupnorm_refuses(L):
    bad, uns = E.M2RNN_ERR_INVALID_ARG, E.M2RNN_ERR_UNSUPPORTED

    def norm(**kw):
        a = dict(dict(rows=3, D=12, G=3, dt=E.M2RNN_F32, eps=1e-5, y=FAKE, g=FAKE, ga=FAKE, be=FAKE,
                      o=FAKE), **kw)
        return L.m2rnn_groupnorm_gate(*a.values(), None)

    def back(**kw):
        a = dict(dict(rows=3, D=12, G=3, dt=E.M2RNN_F32, eps=1e-5, y=FAKE, g=FAKE, ga=FAKE, be=FAKE,
                      do=FAKE, dy=FAKE, dg=FAKE, dga=FAKE, dbe=FAKE, ws=FAKE, wsb=1 << 40), **kw)
        return L.m2rnn_groupnorm_gate_bwd(*a.values(), None)

    for call in (norm, back):
        for kw in ({"rows": -1}, {"D": 0}, {"G": 0}, {"G": 5}, {"dt": 9}, {"eps": -1.0},
                   {"eps": math.nan}, {"eps": math.inf}, {"y": None}, {"g": None}, {"ga": None},
                   {"be": None}):
            assert call(**kw) == bad, (call, kw)
        assert call(dt=E.M2RNN_F64) == uns
        assert call(rows=1 << 40, D=1 << 12, G=1 << 12) == uns
    assert norm(o=None) == bad
    for n in ("do", "dy", "dg", "dga", "dbe"):
        assert back(**{n: None}) == bad, n
    need = L.m2rnn_groupnorm_workspace_bytes(3, 12, 3, E.M2RNN_F32)
    assert need > 0 and back(wsb=need - 1) == E.M2RNN_ERR_WORKSPACE
    assert back(ws=FAKE + 4) == bad
    assert L.m2rnn_groupnorm_workspace_bytes(3, 12, 5, E.M2RNN_F32) == 0


def test_binding_refuses_before_any_launch():
    """Wrong types, shapes, devices and layouts raise ValueError (all tensors here are on the CPU,
    which is itself refused last)."""
    B, T, N, K, V = 1, 4, 2, 8, 8
    k, v = torch.zeros(B, T, N, K), torch.zeros(B, T, N, V)
    x, a, w = torch.zeros(B, T, N), torch.zeros(N), torch.zeros(N, V)
    for bad in ((k.half(), v.half(), k.half(), x, a, a, w), (k, v.bfloat16(), k, x, a, a, w),
                (k, v, k[:, :, :1], x, a, a, w), (k, v, k, x.double(), a, a, w),
                (k, v, k, x, a[:1], a, w), (k, v, k, x, a, a, w.t()[:1])):
        with pytest.raises(ValueError):
            m.m2rnn_ssm_fwd(*bad)
    with pytest.raises(ValueError, match="GPU memory"):
        m.m2rnn_ssm_fwd(k, v, k, x, a, a, w)
    with pytest.raises(ValueError, match="H0"):
        m.m2rnn_ssm_fwd(k, v, k, x, a, a, w, H0=torch.zeros(B, N, K, V + 1))
    with pytest.raises(ValueError, match="dy"):
        m.m2rnn_ssm_bwd(k, v, k, x, a, a, w, None, v[:, 1:])
    with pytest.raises(ValueError, match="dH0"):
        m.m2rnn_ssm_bwd(k, v, k, x, a, a, w, None, v, want_dh0=False,
                        out={"dH0": torch.zeros(B, N, K, V)})
    with pytest.raises(ValueError, match="no outputs.*dK"):
        m.m2rnn_ssm_bwd(k, v, k, x, a, a, w, None, v, out={"dK": k})
    with pytest.raises(ValueError):
        m.m2rnn_ssm_step(torch.zeros(B, N, K, V), k, v, k, x, a, a, w)
    h, wc = torch.zeros(B, 3, 8), torch.zeros(8, 4)
    xc = torch.zeros(B, T, 8)
    for f in (lambda: m.m2rnn_conv_carry(xc.half(), wc), lambda: m.m2rnn_conv_carry(xc, wc.double()),
              lambda: m.m2rnn_conv_carry(xc, wc, hist=h[:, :2]),
              lambda: m.m2rnn_conv_carry(xc, wc, lens=torch.zeros(B, dtype=torch.int64)),
              lambda: m.m2rnn_conv_carry(xc, wc, want_hist=False, lens=torch.zeros(B, dtype=torch.int32)),
              lambda: m.m2rnn_conv_step(h, xc, wc), lambda: m.m2rnn_conv_carry_bwd(xc, wc, None, None, xc[:, 1:]),
              lambda: m.m2rnn_groupnorm_gate(xc, xc, torch.ones(8), torch.ones(8), 3),
              lambda: m.m2rnn_groupnorm_gate(xc, xc.bfloat16(), torch.ones(8), torch.ones(8), 2),
              lambda: m.m2rnn_groupnorm_gate(xc, xc, torch.ones(4), torch.ones(8), 2)):
        with pytest.raises(ValueError):
            f()
