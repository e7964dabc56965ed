"""Python entry points with the C ABI's names: argument marshalling only.

Each function checks that the torch tensors it is given are on one GPU,
contiguous and of the shapes/dtypes the C ABI documents, allocates outputs and
workspace with torch (device memory is the only thing torch provides here),
and calls the library on torch's current stream.  All arithmetic happens in
the HIP kernels.
"""
from __future__ import annotations

import math

import torch

from . import _lib
from ._lib import check

_DT = {torch.float32: _lib.M2RNN_F32, torch.bfloat16: _lib.M2RNN_BF16,
       torch.float64: _lib.M2RNN_F64}


def _ptr(t):
    return None if t is None else ctypes_ptr(t)


def ctypes_ptr(t: torch.Tensor):
    if not t.is_cuda:
        raise ValueError("tensors passed to libm2rnn must live in GPU memory")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libm2rnn must be contiguous")
    return t.data_ptr()


def _stream(device) -> int:
    # torch.cuda.current_stream(device).cuda_stream without the Stream object (4 us of a call)
    return torch._C._cuda_getCurrentRawStream(
        torch.cuda.current_device() if device.index is None else device.index)


def _need(t, shape, dtype, name):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.shape != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _opt(t, shape, dtype, name):
    if t is not None:
        _need(t, shape, dtype, name)


def m2rnn_status_string(status: int) -> str:
    return _lib.status_string(status)


def m2rnn_workspace_bytes(is_bwd: bool, B: int, T: int, n_heads: int, qk_heads: int, K: int,
                          V: int, C: int, state_dtype=torch.float32) -> int:
    return int(_lib.lib().m2rnn_workspace_bytes(int(bool(is_bwd)), B, T, n_heads, qk_heads, K,
                                                V, C, _DT[state_dtype]))


def _heads(k, v):
    """(N, NQ): value heads from v, q/k heads from k (NQ divides N; value head
    n reads q/k head n // (N // NQ))."""
    if k.dim() != 4 or v.dim() != 4:
        raise ValueError("k, q must be [B, T, qk_heads, K] and v [B, T, n_heads, V]")
    N, NQ = v.shape[2], k.shape[2]
    if (NQ < 1 or NQ > N or N % NQ) if N > 0 else NQ != 0:
        raise ValueError(f"qk_heads = {NQ} must divide n_heads = {N}")
    return N, NQ


def _workspace(nbytes: int, device, given=None):
    if nbytes == 0:
        return None, 0
    if given is not None:
        if given.numel() * given.element_size() < nbytes:
            raise ValueError(f"workspace holds {given.numel() * given.element_size()} bytes, "
                             f"{nbytes} needed")
        return given, given.numel() * given.element_size()
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def m2rnn_gates(logit: torch.Tensor, gate_kind: int, alpha=None, beta=None, out=None):
    """f[B, T, N] from the gate logits (sigmoid or exp-softplus form)."""
    if logit.dim() != 3:
        raise ValueError("logit must be [B, T, n_heads]")
    B, T, N = logit.shape
    dt = logit.dtype
    if dt not in (torch.float32, torch.float64):
        raise ValueError("logit must be float32 or float64")
    _opt(alpha, (N,), dt, "alpha")
    _opt(beta, (N,), dt, "beta")
    f = torch.empty_like(logit) if out is None else out
    _need(f, (B, T, N), dt, "out")
    st = _lib.lib().m2rnn_gates(B, T, N, int(gate_kind), _DT[dt], _ptr(logit), _ptr(alpha),
                                _ptr(beta), _ptr(f), _stream(logit.device))
    check(st, "m2rnn_gates")
    return f


def m2rnn_fwd(k, v, q, f, W, w_r, H0=None, C: int = 0, want_ht: bool = True,
              out=None, workspace=None, rc_out=None):
    """Forward recurrence.  Returns (y, HT or None, ckpt or None).

    k, q [B, T, NQ, K] and v [B, T, N, V] in float32 / bfloat16 (float32 state)
    or float64 / bfloat16 (float64 state), where NQ divides N and value head n
    reads q/k head n // (N // NQ); f [B, T, N], W [N, V, V], w_r [N, V],
    H0 [B, N, K, V] in the state dtype (taken from f).  C > 0 also writes the
    checkpoints ckpt[B, N, ceil(T / C), K, V] with ckpt[:, :, c] = H_{cC}.
    ``out`` may hold preallocated (y, HT, ckpt).  ``rc_out`` [B, N, T, K, V] (state
    dtype), when given, receives every step's rc = 1 / (1 + e^{2A}) for m2rnn_bwd.
    """
    N, NQ = _heads(k, v)
    B, T, _, K = k.shape
    V = v.shape[-1]
    sd = f.dtype
    _need(v, (B, T, N, V), k.dtype, "v")
    _need(q, (B, T, NQ, K), k.dtype, "q")
    _need(f, (B, T, N), sd, "f")
    _need(W, (N, V, V), sd, "W")
    _need(w_r, (N, V), sd, "w_r")
    _opt(H0, (B, N, K, V), sd, "H0")
    dev = k.device
    if out is not None:
        y, HT, ckpt = out
    else:
        y = torch.empty((B, T, N, V), dtype=sd, device=dev)
        HT = torch.empty((B, N, K, V), dtype=sd, device=dev) if want_ht else None
        ckpt = (torch.empty((B, N, math.ceil(T / C), K, V), dtype=sd, device=dev)
                if C and C > 0 else None)
    _need(y, (B, T, N, V), sd, "y")
    _opt(HT, (B, N, K, V), sd, "HT")
    if ckpt is not None:
        if not C or C < 1:
            raise ValueError("a checkpoint buffer needs C >= 1")
        _need(ckpt, (B, N, math.ceil(T / C), K, V), sd, "ckpt")
    _opt(rc_out, (B, N, T, K, V), sd, "rc_out")
    ws, wsb = _workspace(m2rnn_workspace_bytes(False, B, T, N, NQ, K, V, max(C, 1), sd), dev,
                         workspace)
    st = _lib.lib().m2rnn_fwd(B, T, N, NQ, K, V, _DT[k.dtype], _DT[sd], _ptr(k), _ptr(v), _ptr(q),
                              _ptr(f), _ptr(W), _ptr(w_r), _ptr(H0), _ptr(y), _ptr(HT),
                              _ptr(ckpt), int(C) if ckpt is not None else 0, _ptr(rc_out),
                              _ptr(ws), wsb, _stream(dev))
    check(st, "m2rnn_fwd")
    return y, HT, ckpt


def _bwd_outputs(k, v, q, gate_kind, logit, alpha, beta, f, W, w_r, H0, ckpt, C, dy, dHT,
                 want_dh0, rc, out):
    """Checks the backward's inputs and returns (B, T, N, NQ, K, V, state dtype,
    output dict) with the given or newly allocated gradient buffers."""
    N, NQ = _heads(k, v)
    B, T, _, K = k.shape
    V = v.shape[-1]
    sd = f.dtype
    _need(v, (B, T, N, V), k.dtype, "v")
    _need(q, (B, T, NQ, K), k.dtype, "q")
    _need(logit, (B, T, N), sd, "logit")
    _need(f, (B, T, N), sd, "f")
    _need(W, (N, V, V), sd, "W")
    _need(w_r, (N, V), sd, "w_r")
    _opt(H0, (B, N, K, V), sd, "H0")
    _need(ckpt, (B, N, math.ceil(T / C), K, V), sd, "ckpt")
    _need(dy, (B, T, N, V), sd, "dy")
    _opt(dHT, (B, N, K, V), sd, "dHT")
    _opt(rc, (B, N, T, K, V), sd, "rc")
    dev = k.device
    exp_gate = gate_kind == _lib.M2RNN_GATE_EXP_SOFTPLUS
    shapes = {"dk": (B, T, NQ, K), "dv": (B, T, N, V), "dq": (B, T, NQ, K), "dlogit": (B, T, N),
              "dW": (N, V, V), "dw_r": (N, V), "dalpha": (N,) if exp_gate else None,
              "dbeta": (N,) if exp_gate else None, "dH0": (B, N, K, V) if want_dh0 else None}
    given = dict(out) if out is not None else {}
    res = {}
    for name, shape in shapes.items():
        if name in given:
            res[name] = given[name]
            if shape is None:
                if res[name] is not None:
                    raise ValueError(f"{name} is not an output of this gate")
            else:
                (_opt if name == "dH0" else _need)(res[name], shape, sd, name)
        else:
            res[name] = None if shape is None else torch.empty(shape, dtype=sd, device=dev)
    return B, T, N, NQ, K, V, sd, res


def _bwd_args(k, v, q, gate_kind, logit, alpha, beta, f, W, w_r, H0, ckpt, C, rc, dy, dHT, o):
    """The pointer arguments shared by m2rnn_bwd and m2rnn_bwd_noalloc, in ABI order
    from k to dH0."""
    return (_ptr(k), _ptr(v), _ptr(q), int(gate_kind), _ptr(logit), _ptr(alpha), _ptr(beta),
            _ptr(f), _ptr(W), _ptr(w_r), _ptr(H0), _ptr(ckpt), int(C), _ptr(rc), _ptr(dy),
            _ptr(dHT), _ptr(o["dk"]), _ptr(o["dv"]), _ptr(o["dq"]), _ptr(o["dlogit"]),
            _ptr(o["dW"]), _ptr(o["dw_r"]), _ptr(o["dalpha"]), _ptr(o["dbeta"]), _ptr(o["dH0"]))


def m2rnn_bwd(k, v, q, gate_kind: int, logit, alpha, beta, f, W, w_r, H0, ckpt, C: int, dy,
              dHT=None, want_dh0: bool = True, workspace=None, rc=None, out=None):
    """Backward of m2rnn_fwd.  Returns a dict with dk, dv, dq, dlogit, dW, dw_r,
    dalpha and dbeta (exp-softplus gate only, else None) and dH0 (or None).
    dk and dq have the shape of k and q: with shared heads (NQ < N) each is
    the sum over the value heads that read it.  ``rc`` (from m2rnn_fwd's rc_out)
    replaces the recomputation of the states; the results are the same.
    ``out`` may hold preallocated gradient buffers under those names (any
    missing one is allocated; dH0 = None there skips it)."""
    B, T, N, NQ, K, V, sd, o = _bwd_outputs(k, v, q, gate_kind, logit, alpha, beta, f, W, w_r,
                                            H0, ckpt, C, dy, dHT, want_dh0, rc, out)
    dev = k.device
    ws, wsb = _workspace(m2rnn_workspace_bytes(True, B, T, N, NQ, K, V, C, sd), dev, workspace)
    st = _lib.lib().m2rnn_bwd(
        B, T, N, NQ, K, V, _DT[k.dtype], _DT[sd],
        *_bwd_args(k, v, q, gate_kind, logit, alpha, beta, f, W, w_r, H0, ckpt, C, rc, dy, dHT, o),
        _ptr(ws), wsb, _stream(dev))
    check(st, "m2rnn_bwd")
    return o


def m2rnn_bwd_noalloc(k, v, q, gate_kind: int, logit, alpha, beta, f, W, w_r, H0, ckpt, C: int,
                      dy, dHT=None, want_dh0: bool = True, rc=None, out=None):
    """m2rnn_bwd without a workspace: the library's static per-device scratch
    (NOALLOC_SCRATCH_BYTES) holds the partial sums.  With every gradient buffer
    given in ``out``, nothing is allocated.  Calls that may overlap on one
    device share the scratch and race."""
    B, T, N, NQ, K, V, sd, o = _bwd_outputs(k, v, q, gate_kind, logit, alpha, beta, f, W, w_r,
                                            H0, ckpt, C, dy, dHT, want_dh0, rc, out)
    st = _lib.lib().m2rnn_bwd_noalloc(
        B, T, N, NQ, K, V, _DT[k.dtype], _DT[sd],
        *_bwd_args(k, v, q, gate_kind, logit, alpha, beta, f, W, w_r, H0, ckpt, C, rc, dy, dHT, o),
        _stream(k.device))
    check(st, "m2rnn_bwd_noalloc")
    return o


def m2rnn_newton_workspace_bytes(B: int, T: int, n_heads: int, K: int, V: int,
                                 states_given: bool) -> int:
    return int(_lib.lib().m2rnn_newton_workspace_bytes(B, T, n_heads, K, V,
                                                       int(bool(states_given))))


def m2rnn_newton_fwd(k, v, q, f, W, w_r, H0=None, iters: int = 3, want_ht: bool = True,
                     want_states: bool = False, want_residual: bool = False, out=None,
                     workspace=None):
    """Parallel-in-time forward by Newton's method (fp32 state, V in 16/32/48/64).

    Arguments as for m2rnn_fwd (k, q, v in float32 or bfloat16; f, W, w_r, H0
    float32).  Returns (y, HT or None, states [B, N, T, K, V] or None,
    residual [iters + 1] or None); ``out`` may hold preallocated
    (y, HT, states, residual).
    """
    N, NQ = _heads(k, v)
    B, T, _, K = k.shape
    V = v.shape[-1]
    sd = torch.float32
    _need(v, (B, T, N, V), k.dtype, "v")
    _need(q, (B, T, NQ, K), k.dtype, "q")
    _need(f, (B, T, N), sd, "f")
    _need(W, (N, V, V), sd, "W")
    _need(w_r, (N, V), sd, "w_r")
    _opt(H0, (B, N, K, V), sd, "H0")
    dev = k.device
    if out is not None:
        y, HT, states, res = out
    else:
        y = torch.empty((B, T, N, V), dtype=sd, device=dev)
        HT = torch.empty((B, N, K, V), dtype=sd, device=dev) if want_ht else None
        states = torch.empty((B, N, T, K, V), dtype=sd, device=dev) if want_states else None
        res = torch.empty((iters + 1,), dtype=sd, device=dev) if want_residual else None
    _need(y, (B, T, N, V), sd, "y")
    _opt(HT, (B, N, K, V), sd, "HT")
    _opt(states, (B, N, T, K, V), sd, "states")
    _opt(res, (iters + 1,), sd, "residual")
    ws, wsb = _workspace(m2rnn_newton_workspace_bytes(B, T, N, K, V, states is not None), dev,
                         workspace)
    st = _lib.lib().m2rnn_newton_fwd(B, T, N, NQ, K, V, _DT[k.dtype], _ptr(k), _ptr(v), _ptr(q),
                                     _ptr(f), _ptr(W), _ptr(w_r), _ptr(H0), int(iters), _ptr(y),
                                     _ptr(HT), _ptr(states), _ptr(res), _ptr(ws), wsb,
                                     _stream(dev))
    check(st, "m2rnn_newton_fwd")
    return y, HT, states, res


def m2rnn_step(H, k, v, q, f, W, w_r, out=None):
    """One token of every sequence (decoding): H [B, N, K, V] (state dtype) is
    updated in place from H_{t-1} to H_t, and y [B, N, V] is returned.  k, q
    [B, NQ, K] and v [B, N, V] in the input dtype, f [B, N], W [N, V, V] and
    w_r [N, V] in the state dtype (taken from H)."""
    if H.dim() != 4 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("H must be [B, N, K, V], k and q [B, qk_heads, K], v [B, n_heads, V]")
    B, N, K, V = H.shape
    NQ = k.shape[1]
    if (NQ < 1 or NQ > N or N % NQ) if N > 0 else NQ != 0:
        raise ValueError(f"qk_heads = {NQ} must divide n_heads = {N}")
    sd = H.dtype
    _need(H, (B, N, K, V), sd, "H")
    _need(k, (B, NQ, K), k.dtype, "k")
    _need(q, (B, NQ, K), k.dtype, "q")
    _need(v, (B, N, V), k.dtype, "v")
    _need(f, (B, N), sd, "f")
    _need(W, (N, V, V), sd, "W")
    _need(w_r, (N, V), sd, "w_r")
    y = torch.empty((B, N, V), dtype=sd, device=H.device) if out is None else out
    _need(y, (B, N, V), sd, "out")
    st = _lib.lib().m2rnn_step(B, N, NQ, K, V, _DT[k.dtype], _DT[sd], _ptr(k), _ptr(v), _ptr(q),
                               _ptr(f), _ptr(W), _ptr(w_r), _ptr(H), _ptr(y), _stream(H.device))
    check(st, "m2rnn_step")
    return y


def _io_param(x, param):
    """(io dtype code, param dtype code) of a block call; param from the parameters."""
    if param.dtype not in (torch.float32, torch.float64):
        raise ValueError("parameters must be float32 or float64")
    return _DT[x.dtype], _DT[param.dtype]


def m2rnn_conv_silu(x, w, bias=None, out=None):
    """Block prologue on one projected tensor x [B, T, C] (float32 / bfloat16, or
    float64 / bfloat16): SiLU of the depthwise causal convolution with w [C, 4]
    (+ bias [C]); returns [B, T, C] in x's dtype."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    B, T, C = x.shape
    io, pd = _io_param(x, w)
    _need(w, (C, 4), w.dtype, "w")
    _opt(bias, (C,), w.dtype, "bias")
    y = torch.empty_like(x) if out is None else out
    _need(y, (B, T, C), x.dtype, "out")
    st = _lib.lib().m2rnn_conv_silu(B, T, C, io, pd, _ptr(x), _ptr(w), _ptr(bias), _ptr(y),
                                    _stream(x.device))
    check(st, "m2rnn_conv_silu")
    return y


def m2rnn_conv_silu_bwd(x, w, bias, dout, workspace=None):
    """Gradients of sum(dout * m2rnn_conv_silu(x, w, bias)): (dx, dw, dbias or None),
    in the parameters' dtype."""
    B, T, C = x.shape
    io, pd = _io_param(x, w)
    _need(w, (C, 4), w.dtype, "w")
    _opt(bias, (C,), w.dtype, "bias")
    _need(dout, (B, T, C), w.dtype, "dout")
    dx = torch.empty((B, T, C), dtype=w.dtype, device=x.device)
    dw = torch.empty((C, 4), dtype=w.dtype, device=x.device)
    dbias = torch.empty((C,), dtype=w.dtype, device=x.device) if bias is not None else None
    nb = int(_lib.lib().m2rnn_block_workspace_bytes(0, B, T, C, pd))
    ws, wsb = _workspace(nb, x.device, workspace)
    st = _lib.lib().m2rnn_conv_silu_bwd(B, T, C, io, pd, _ptr(x), _ptr(w), _ptr(bias),
                                        _ptr(dout), _ptr(dx), _ptr(dw), _ptr(dbias), _ptr(ws),
                                        wsb, _stream(x.device))
    check(st, "m2rnn_conv_silu_bwd")
    return dx, dw, dbias


def m2rnn_gate_rmsnorm(y, g_pre, gamma, eps: float = 1e-6, out=None):
    """Block epilogue: gamma * z / sqrt(mean(z^2) + eps), z = y * SiLU(g_pre), over the
    last dimension D.  y [..., D] and gamma [D] in the state dtype, g_pre [..., D] in the
    input dtype; returns [..., D] in g_pre's dtype."""
    D = y.shape[-1]
    rows = y.numel() // D if D else 0
    io, pd = _io_param(g_pre, y)
    _need(g_pre, tuple(y.shape), g_pre.dtype, "g_pre")
    _need(gamma, (D,), y.dtype, "gamma")
    o = torch.empty(tuple(y.shape), dtype=g_pre.dtype, device=y.device) if out is None else out
    _need(o, tuple(y.shape), g_pre.dtype, "out")
    st = _lib.lib().m2rnn_gate_rmsnorm(rows, D, io, pd, float(eps), _ptr(y), _ptr(g_pre),
                                       _ptr(gamma), _ptr(o), _stream(y.device))
    check(st, "m2rnn_gate_rmsnorm")
    return o


def m2rnn_gate_rmsnorm_bwd(y, g_pre, gamma, dout, eps: float = 1e-6, workspace=None):
    """Gradients of sum(dout * m2rnn_gate_rmsnorm(y, g_pre, gamma, eps)):
    (dy, dg_pre, dgamma) in the state dtype."""
    D = y.shape[-1]
    rows = y.numel() // D if D else 0
    io, pd = _io_param(g_pre, y)
    _need(g_pre, tuple(y.shape), g_pre.dtype, "g_pre")
    _need(gamma, (D,), y.dtype, "gamma")
    _need(dout, tuple(y.shape), y.dtype, "dout")
    dy = torch.empty_like(y)
    dg = torch.empty_like(y)
    dgamma = torch.empty((D,), dtype=y.dtype, device=y.device)
    nb = int(_lib.lib().m2rnn_block_workspace_bytes(1, rows, 1, D, pd))
    ws, wsb = _workspace(nb, y.device, workspace)
    st = _lib.lib().m2rnn_gate_rmsnorm_bwd(rows, D, io, pd, float(eps), _ptr(y), _ptr(g_pre),
                                           _ptr(gamma), _ptr(dout), _ptr(dy), _ptr(dg),
                                           _ptr(dgamma), _ptr(ws), wsb, _stream(y.device))
    check(st, "m2rnn_gate_rmsnorm_bwd")
    return dy, dg, dgamma


def _io_dtype(t, name):
    """The dtype code of a tensor whose type sets a call's (float32 or bfloat16)."""
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"{name} must be float32 or bfloat16")
    return _DT[t.dtype]


def _call(name, dev, *args):
    """Calls the library's function `name` on torch's current stream of the device `dev`, which
    every tensor among the arguments must be on; raises what it returns."""
    vals = []
    for t in args:
        if isinstance(t, torch.Tensor):
            if t.device != dev:
                raise ValueError(f"{name}: tensors on {t.device} and {dev}")
            t = ctypes_ptr(t)
        vals.append(t)
    fn = getattr(_lib.lib(), name)
    index = dev.index
    if torch._C._cuda_getDevice() == index:
        st = fn(*vals, torch._C._cuda_getCurrentRawStream(index))
    else:  # the launches go to the stream's own device
        with torch.cuda.device(dev):
            st = fn(*vals, torch._C._cuda_getCurrentRawStream(index))
    if st != _lib.M2RNN_OK:
        check(st, name)


def _given(spec, out, dev):
    """Output buffers {name: (shape, dtype), or None for one that the call does not have}: those
    given in ``out`` (None there skips dH0 and dhist), the others newly allocated."""
    given = dict(out) if out is not None else {}
    if given.keys() - spec.keys():
        raise ValueError(f"no outputs of this call: {sorted(given.keys() - spec.keys())}")
    o = {}
    for name, sd in spec.items():
        if name in given:
            o[name] = given[name]
            if sd is None:
                if o[name] is not None:
                    raise ValueError(f"{name} is not an output of this call")
            else:
                (_opt if name in ("dH0", "dhist") else _need)(o[name], sd[0], sd[1], name)
        else:
            o[name] = None if sd is None else torch.empty(sd[0], dtype=sd[1], device=dev)
    return o


# ---- the selective state-space scan

def _ssm_sizes(k, v, q, logit, alpha, beta, w_r, H0):
    """Checks the scan's inputs; returns (B, T, N, NQ, K, V, dtype code)."""
    io = _io_dtype(k, "k")
    N, NQ = _heads(k, v)
    B, T, _, K = k.shape
    V = v.shape[-1]
    f32 = torch.float32
    _need(v, (B, T, N, V), k.dtype, "v")
    _need(q, (B, T, NQ, K), k.dtype, "q")
    _need(logit, (B, T, N), f32, "logit")
    _need(alpha, (N,), f32, "alpha")
    _need(beta, (N,), f32, "beta")
    _need(w_r, (N, V), f32, "w_r")
    _opt(H0, (B, N, K, V), f32, "H0")
    return B, T, N, NQ, K, V, io


def m2rnn_ssm_workspace_bytes(is_bwd: bool, B: int, T: int, n_heads: int, qk_heads: int, K: int,
                              V: int, in_dtype=torch.bfloat16) -> int:
    return int(_lib.lib().m2rnn_ssm_workspace_bytes(int(bool(is_bwd)), B, T, n_heads, qk_heads, K,
                                                    V, _DT[in_dtype]))


def m2rnn_ssm_fwd(k, v, q, logit, alpha, beta, w_r, H0=None, want_ht: bool = True, out=None,
                  workspace=None):
    """The selective state-space scan
        d_t = softplus(logit_t + beta),  H_t = exp(-alpha d_t) H_{t-1} + d_t k_t v_t^T,
        y_t = H_t^T q_t + w_r * v_t
    over [B, T] tokens.  k, q [B, T, NQ, K] and v [B, T, N, V] in float32 or bfloat16 (NQ
    divides N as in m2rnn_fwd); logit [B, T, N], alpha, beta [N], w_r [N, V] and H0
    [B, N, K, V] float32.  Returns (y in v's dtype, HT float32 or None); ``out`` may hold
    preallocated (y, HT), where HT may be H0 itself.  logit = -inf makes a token leave the state
    alone."""
    B, T, N, NQ, K, V, io = _ssm_sizes(k, v, q, logit, alpha, beta, w_r, H0)
    dev = k.device
    if out is not None:
        y, HT = out
    else:
        y = torch.empty((B, T, N, V), dtype=v.dtype, device=dev)
        HT = torch.empty((B, N, K, V), dtype=torch.float32, device=dev) if want_ht else None
    _need(y, (B, T, N, V), v.dtype, "y")
    _opt(HT, (B, N, K, V), torch.float32, "HT")
    ws, wsb = _workspace(m2rnn_ssm_workspace_bytes(False, B, T, N, NQ, K, V, k.dtype), dev,
                         workspace)
    _call("m2rnn_ssm_fwd", dev, B, T, N, NQ, K, V, io, k, v, q, logit, alpha, beta, w_r, H0, y, HT,
          ws, wsb)
    return y, HT


def m2rnn_ssm_bwd(k, v, q, logit, alpha, beta, w_r, H0, dy, dHT=None, want_dh0: bool = True,
                  workspace=None, out=None):
    """Backward of m2rnn_ssm_fwd: a dict with dk, dv, dq (k's dtype), dlogit, dw_r, dalpha,
    dbeta and dH0 (or None) in float32.  dy [B, T, N, V] in v's dtype, dHT [B, N, K, V] float32
    or None.  ``out`` may hold preallocated buffers under those names (any missing one is
    allocated; dH0 = None there skips it)."""
    B, T, N, NQ, K, V, io = _ssm_sizes(k, v, q, logit, alpha, beta, w_r, H0)
    f32 = torch.float32
    _need(dy, (B, T, N, V), v.dtype, "dy")
    _opt(dHT, (B, N, K, V), f32, "dHT")
    dev = k.device
    spec = {"dk": ((B, T, NQ, K), k.dtype), "dv": ((B, T, N, V), k.dtype),
            "dq": ((B, T, NQ, K), k.dtype), "dlogit": ((B, T, N), f32), "dw_r": ((N, V), f32),
            "dalpha": ((N,), f32), "dbeta": ((N,), f32),
            "dH0": ((B, N, K, V), f32) if want_dh0 else None}
    o = _given(spec, out, dev)
    ws, wsb = _workspace(m2rnn_ssm_workspace_bytes(True, B, T, N, NQ, K, V, k.dtype), dev,
                         workspace)
    _call("m2rnn_ssm_bwd", dev, B, T, N, NQ, K, V, io, k, v, q, logit, alpha, beta, w_r, H0, dy,
          dHT, o["dk"], o["dv"], o["dq"], o["dlogit"], o["dw_r"], o["dalpha"], o["dbeta"], o["dH0"],
          ws, wsb)
    return o


def m2rnn_ssm_step(H, k, v, q, logit, alpha, beta, w_r, out=None):
    """One token of every sequence through the scan (decoding): H [B, N, K, V] float32 is updated
    in place from H_{t-1} to H_t, and y [B, N, V] in v's dtype is returned.  k, q [B, NQ, K] and v
    [B, N, V] in float32 or bfloat16; logit [B, N], alpha, beta [N], w_r [N, V] float32."""
    if H.dim() != 4 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("H must be [B, N, K, V], k and q [B, qk_heads, K], v [B, n_heads, V]")
    B, N, K, V = H.shape
    NQ = k.shape[1]
    if (NQ < 1 or NQ > N or N % NQ) if N > 0 else NQ != 0:
        raise ValueError(f"qk_heads = {NQ} must divide n_heads = {N}")
    f32 = torch.float32
    io = _io_dtype(k, "k")
    _need(H, (B, N, K, V), f32, "H")
    _need(k, (B, NQ, K), k.dtype, "k")
    _need(q, (B, NQ, K), k.dtype, "q")
    _need(v, (B, N, V), k.dtype, "v")
    _need(logit, (B, N), f32, "logit")
    _need(alpha, (N,), f32, "alpha")
    _need(beta, (N,), f32, "beta")
    _need(w_r, (N, V), f32, "w_r")
    if out is None:
        y = torch.empty_like(v)
    else:
        y = out
        _need(y, (B, N, V), v.dtype, "out")
    _call("m2rnn_ssm_step", H.device, B, N, NQ, K, V, io, k, v, q, logit, alpha, beta, w_r, H, y)
    return y


# ---- the convolution with a carried history

def m2rnn_conv_carry(x, w, bias=None, hist=None, want_hist: bool = True, lens=None, out=None):
    """m2rnn_conv_silu with the three inputs before x: x [B, T, C] and hist [B, 3, C] (oldest
    first, None = zero) in float32 or bfloat16, w [C, 4] and bias [C] float32.  Returns (out
    [B, T, C], the history after x [B, 3, C] or None); ``lens`` [B] int32 says how many of each
    sequence's inputs count for it (a padded batch).  ``out`` may hold preallocated (out, hist),
    where the second may be ``hist`` itself."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    io = _io_dtype(x, "x")
    B, T, C = x.shape
    _need(w, (C, 4), torch.float32, "w")
    _opt(bias, (C,), torch.float32, "bias")
    _opt(hist, (B, 3, C), x.dtype, "hist")
    _opt(lens, (B,), torch.int32, "lens")
    if out is not None:
        o, ho = out
    else:
        o = torch.empty_like(x)
        ho = torch.empty((B, 3, C), dtype=x.dtype, device=x.device) if want_hist else None
    _need(o, (B, T, C), x.dtype, "out")
    _opt(ho, (B, 3, C), x.dtype, "hist_out")
    if lens is not None and ho is None:
        raise ValueError("lens sets the history that is returned: want_hist=False leaves it no use")
    _call("m2rnn_conv_carry", x.device, B, T, C, io, x, w, bias, hist, lens, o, ho)
    return o, ho


def m2rnn_conv_carry_bwd(x, w, bias, hist, dout, workspace=None, out=None):
    """Gradients of sum(dout * m2rnn_conv_carry(x, w, bias, hist)[0]): a dict with dx, dhist (x's
    dtype; None without hist), dw and dbias (float32; None without bias).  dout in x's dtype;
    ``out`` may hold preallocated buffers under those names."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    io = _io_dtype(x, "x")
    B, T, C = x.shape
    f32 = torch.float32
    _need(w, (C, 4), f32, "w")
    _opt(bias, (C,), f32, "bias")
    _opt(hist, (B, 3, C), x.dtype, "hist")
    _need(dout, (B, T, C), x.dtype, "dout")
    spec = {"dx": ((B, T, C), x.dtype), "dw": ((C, 4), f32),
            "dbias": ((C,), f32) if bias is not None else None,
            "dhist": ((B, 3, C), x.dtype) if hist is not None else None}
    o = _given(spec, out, x.device)
    ws, wsb = _workspace(int(_lib.lib().m2rnn_conv_carry_workspace_bytes(B, T, C)), x.device,
                         workspace)
    _call("m2rnn_conv_carry_bwd", x.device, B, T, C, io, x, w, bias, hist, dout, o["dx"], o["dw"],
          o["dbias"], o["dhist"], ws, wsb)
    return o


def m2rnn_conv_step(hist, x, w, bias=None, out=None):
    """One token of every sequence through the convolution: hist [B, 3, C] is shifted by x
    [B, C] in place, and SiLU of the convolution [B, C] is returned (all in x's dtype; w [C, 4]
    and bias [C] float32)."""
    if x.dim() != 2:
        raise ValueError("x must be [B, C]")
    io = _io_dtype(x, "x")
    B, C = x.shape
    _need(hist, (B, 3, C), x.dtype, "hist")
    _need(w, (C, 4), torch.float32, "w")
    _opt(bias, (C,), torch.float32, "bias")
    if out is None:
        o = torch.empty_like(x)
    else:
        o = out
        _need(o, (B, C), x.dtype, "out")
    _call("m2rnn_conv_step", x.device, B, C, io, x, w, bias, hist, o)
    return o


# ---- group norm with a gate

def _groupnorm_sizes(y, g_pre, gamma, beta, groups):
    shape = y.shape
    D = shape[-1]
    if groups < 1 or D < 1 or D % groups:
        raise ValueError(f"groups = {groups} must divide D = {D}")
    _need(g_pre, shape, y.dtype, "g_pre")
    _need(gamma, (D,), torch.float32, "gamma")
    _need(beta, (D,), torch.float32, "beta")
    return y.numel() // D, D, _io_dtype(y, "y")


def m2rnn_groupnorm_gate(y, g_pre, gamma, beta, groups: int, eps: float = 1e-5, out=None):
    """(gamma * z + beta) * SiLU(g_pre), z = y normalised (mean and variance) over each of the
    ``groups`` runs of D / groups consecutive channels of the last dimension D.  y and g_pre
    [..., D] in float32 or bfloat16, gamma and beta [D] float32; returns [..., D] in y's dtype."""
    rows, D, io = _groupnorm_sizes(y, g_pre, gamma, beta, groups)
    if out is None:
        o = torch.empty_like(y)
    else:
        o = out
        _need(o, y.shape, y.dtype, "out")
    _call("m2rnn_groupnorm_gate", y.device, rows, D, int(groups), io, float(eps), y, g_pre, gamma,
          beta, o)
    return o


def m2rnn_groupnorm_gate_bwd(y, g_pre, gamma, beta, groups: int, dout, eps: float = 1e-5,
                             workspace=None, out=None):
    """Gradients of sum(dout * m2rnn_groupnorm_gate(...)): (dy, dg_pre) in y's dtype and (dgamma,
    dbeta) in float32; ``out`` may hold those four preallocated."""
    rows, D, io = _groupnorm_sizes(y, g_pre, gamma, beta, groups)
    _need(dout, tuple(y.shape), y.dtype, "dout")
    if out is not None:
        dy, dg, dgamma, dbeta = out
    else:
        dy, dg = torch.empty_like(y), torch.empty_like(y)
        dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(beta)
    _need(dy, tuple(y.shape), y.dtype, "dy")
    _need(dg, tuple(y.shape), y.dtype, "dg_pre")
    _need(dgamma, (D,), torch.float32, "dgamma")
    _need(dbeta, (D,), torch.float32, "dbeta")
    nb = int(_lib.lib().m2rnn_groupnorm_workspace_bytes(rows, D, int(groups), io))
    ws, wsb = _workspace(nb, y.device, workspace)
    _call("m2rnn_groupnorm_gate_bwd", y.device, rows, D, int(groups), io, float(eps), y, g_pre,
          gamma, beta, dout, dy, dg, dgamma, dbeta, ws, wsb)
    return dy, dg, dgamma, dbeta
