"""The state-space layer's operators as a user calls them, next to their plain forms.

Operators (include/m2rnn.h has their contracts):

* the selective state-space scan (m2rnn_ssm_fwd, m2rnn_ssm_bwd, m2rnn_ssm_step):
      d_t = softplus(logit_t + beta),  f_t = exp(-alpha d_t),
      H_t = f_t H_{t-1} + d_t k_t v_t^T,  y_t = H_t^T q_t + w_r (.) v_t;
* the short causal convolution with a carried history (m2rnn_conv_carry,
  m2rnn_conv_carry_bwd, m2rnn_conv_step): out = SiLU(bias + 4 taps), the three inputs before
  the sequence given and the three last ones returned;
* the per-head group norm with a SiLU gate (m2rnn_groupnorm_gate, m2rnn_groupnorm_gate_bwd):
      out = (gamma (.) (y - mean) / sqrt(var + eps) + beta) (.) SiLU(g_pre).

`own` chooses between the plain forms (elementary torch operations in 32 bits, decays in 64)
and the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda:0"
CHUNK = 256          # plain form of the scan: tokens per block of its quadratic part
EPS = 1e-5


# --------------------------------------------------------------------------- cases

def _ssm(name, kind, B, T, N, NQ, K, V, dtype, carry):
    return {"name": name, "kind": kind, "B": B, "T": T, "N": N, "NQ": NQ, "K": K, "V": V,
            "dtype": dtype, "carry": carry}


def _conv(name, kind, B, T, C, dtype, bias, carry):
    return {"name": name, "kind": kind, "B": B, "T": T, "C": C, "dtype": dtype, "bias": bias,
            "carry": carry}


def _norm(name, kind, rows, D, groups, dtype):
    return {"name": name, "kind": kind, "rows": rows, "D": D, "groups": groups, "dtype": dtype}


def listed():
    return [
        # prompts: four long ones at the library's long-context size
        _ssm("prompt_t16k_k64", "ssm_prompt", 4, 16384, 16, 16, 64, 64, "bf16", True),
        # one long prompt through a layer with the largest state (128 x 128 a head)
        _ssm("prompt_big_state", "ssm_prompt", 1, 16384, 32, 32, 128, 128, "bf16", True),
        # three prompts of an odd length, shared q/k, odd head sizes, in fp32
        _ssm("prompt_ragged_fp32", "ssm_prompt", 3, 1021, 6, 2, 40, 24, "fp32", True),
        # training at the library's forward + backward size
        _ssm("train_k32_v128", "ssm_train", 16, 4096, 16, 16, 32, 128, "bf16", False),
        # training with one q and k for all value heads (the multi-value layout)
        _ssm("train_multi_value", "ssm_train", 2, 4096, 64, 1, 64, 16, "bf16", False),
        # fp32 training on a window whose state comes in and goes on (truncated backward)
        _ssm("train_window_fp32", "ssm_train", 8, 2048, 8, 8, 64, 64, "fp32", True),
        # decoding: one token of each of 512 sequences
        _ssm("step_512", "ssm_step", 512, 1, 16, 16, 64, 64, "bf16", True),
        # decoding one sequence, shared q/k: the call's latency
        _ssm("step_1_multi_value", "ssm_step", 1, 1, 64, 1, 64, 16, "bf16", True),
        # training through the convolution of one projected tensor (16 heads x 64 channels)
        _conv("conv_train_t16k", "conv_train", 4, 16384, 1024, "bf16", True, True),
        # its single-token form for 512 sequences
        _conv("conv_step_512", "conv_step", 512, 1, 1024, "bf16", True, True),
        # training through the layer's epilogue, one group per head
        _norm("norm_train_64k", "norm_train", 65536, 1024, 16, "bf16"),
        # the epilogue of a decoding step: 512 tokens of 64 heads x 16 channels
        _norm("norm_fwd_512", "norm_fwd", 512, 1024, 64, "bf16"),
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))

    kind = rng.choice(["ssm_prompt", "ssm_prompt", "ssm_train", "ssm_train", "ssm_step",
                       "conv_prompt", "conv_train", "conv_step", "norm_fwd", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind.startswith("ssm"):
        NQ = rng.choice([1, 1, 2, 4, 8])
        N = NQ * rng.choice([1, 1, 2, 3, 8])
        K = rng.choice([16, 32, 64, 64, 128, 256, rng.randint(1, 256)])
        V = rng.choice([16, 32, 64, 64, 128, rng.randint(1, 128)])
        if kind == "ssm_step":
            B, T = log_int(1, 600), 1
            B = max(1, min(B, int(3.0e8 / (N * K * V))))
        else:
            T = log_int(1, 16384)
            B = rng.randint(1, 8)
            while B > 1 and B * T * N > 400000:
                B -= 1
            T = max(1, min(T, int(1.2e9 / (B * N * K * V)), 400000 // (B * N)))
        return {"kind": kind, "B": B, "T": T, "N": N, "NQ": NQ, "K": K, "V": V, "dtype": dtype,
                "carry": True if kind != "ssm_train" else rng.random() < 0.5}
    if kind.startswith("conv"):
        C = rng.choice([64, 256, 1024, 2048, rng.randint(1, 2100)])
        B = log_int(1, 600) if kind == "conv_step" else rng.randint(1, 8)
        T = 1 if kind == "conv_step" else max(1, min(log_int(1, 16384), 40000000 // (B * C)))
        return {"kind": kind, "B": B, "T": T, "C": C, "dtype": dtype, "bias": rng.random() < 0.7,
                "carry": kind != "conv_train" or rng.random() < 0.5}
    groups = rng.choice([1, 4, 16, 64, rng.randint(1, 70)])
    size = rng.choice([16, 64, 128, rng.randint(1, 150)])
    rows = max(1, min(log_int(1, 65536), 40000000 // (groups * size)))
    return {"kind": kind, "rows": rows, "D": groups * size, "groups": groups, "dtype": dtype}


# --------------------------------------------------------------------------- inputs

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    dt = _dtype(case)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    kind = case["kind"]
    s = {"kind": kind}
    if kind.startswith("ssm"):
        B, T, N, NQ, K, V = (case[x] for x in ("B", "T", "N", "NQ", "K", "V"))
        s["k"] = (randn(B, T, NQ, K) / math.sqrt(K)).to(dt)
        s["v"] = randn(B, T, N, V).to(dt)
        s["q"] = randn(B, T, NQ, K).to(dt)
        s["logit"] = randn(B, T, N)
        # step sizes around 1e-3 .. 1e-1 at logit 0 and decay rates 1 .. 16, the usual
        # initialisation of such layers
        d0 = torch.exp(rand(N) * math.log(100.0) + math.log(1e-3))
        s["beta"] = d0 + torch.log(-torch.expm1(-d0))
        s["alpha"] = 1.0 + 15.0 * rand(N)
        s["w_r"] = 1.0 + 0.1 * randn(N, V)
        s["H0"] = (rand(B, N, K, V) - 0.5) if case["carry"] else None
        if kind == "ssm_train":
            s["dy"] = randn(B, T, N, V).to(dt)
            s["dHT"] = randn(B, N, K, V) if case["carry"] else None
        if kind == "ssm_step":
            for n in ("k", "v", "q", "logit"):
                s[n] = s[n][:, 0].contiguous()
    elif kind.startswith("conv"):
        B, T, C = case["B"], case["T"], case["C"]
        s["x"] = randn(B, T, C).to(dt)
        s["w"] = 0.5 * randn(C, 4)
        s["bias"] = 0.1 * randn(C) if case["bias"] else None
        s["hist"] = randn(B, 3, C).to(dt) if case["carry"] else None
        if kind == "conv_train":
            s["dout"] = randn(B, T, C).to(dt)
        if kind == "conv_step":
            s["x"] = s["x"][:, 0].contiguous()
    else:
        rows, D = case["rows"], case["D"]
        s["groups"] = case["groups"]
        s["y"] = (0.5 * randn(rows, D)).to(dt)
        s["g_pre"] = randn(rows, D).to(dt)
        s["gamma"] = 0.5 + rand(D)
        s["beta"] = 0.1 * randn(D)
        if kind == "norm_train":
            s["dout"] = randn(rows, D).to(dt)
    return s


# --------------------------------------------------------------------------- plain forms

def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _plain_ssm(k, v, q, logit, alpha, beta, w_r, H0):
    """The scan in blocks: within a block the masked, decayed product of q and k; between
    blocks the decayed sum of the blocks' updates.  k, v, q, alpha, beta, logit in fp32."""
    B, T, NQ, K = k.shape
    N, V = v.shape[2], v.shape[3]
    G = N // NQ
    L = min(CHUNK, T)
    C = -(-T // L)

    def blocks(x):  # [B, T, h, n] -> [B, h, C, L, n], zeros behind the end
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, C * L - T))
        return x.reshape(B, C, L, x.shape[2], x.shape[3]).permute(0, 3, 1, 2, 4)

    d = _softplus(logit.double() + beta.double())                        # [B, T, N]
    rate = blocks((-alpha.double() * d)[..., None])[..., 0]              # log f
    d = blocks(d.float()[..., None])[..., 0]                             # [B, N, C, L]
    cum = rate.cumsum(-1)
    kb, qb, vb = blocks(k), blocks(q), blocks(v)
    mask = torch.ones(L, L, dtype=torch.bool, device=k.device).tril()
    decay = (cum[..., :, None] - cum[..., None, :]).masked_fill(~mask, -math.inf).exp().float()
    s = torch.matmul(qb, kb.transpose(-1, -2).contiguous())              # [B, NQ, C, L, L]
    p = s.repeat_interleave(G, dim=1) * decay * d[..., None, :]
    y = torch.matmul(p, vb)
    kh, qh = kb.repeat_interleave(G, dim=1), qb.repeat_interleave(G, dim=1)
    out_w = (cum[..., -1:] - cum).exp().float() * d
    upd = torch.matmul((kh * out_w[..., None]).transpose(-1, -2).contiguous(), vb)
    first = H0 if H0 is not None else torch.zeros_like(upd[:, :, 0])
    upd = torch.cat([first[:, :, None], upd], dim=2).reshape(B, N, C + 1, K * V)
    ct = torch.nn.functional.pad(cum[..., -1].cumsum(-1), (1, 0))        # [B, N, C + 1]
    mask = torch.ones(C + 1, C + 1, dtype=torch.bool, device=k.device).tril()
    between = (ct[..., :, None] - ct[..., None, :]).masked_fill(~mask, -math.inf).exp().float()
    start = torch.matmul(between, upd).reshape(B, N, C + 1, K, V)
    y = y + torch.matmul(qh * cum.exp().float()[..., None], start[:, :, :C])
    y = y.permute(0, 2, 3, 1, 4).reshape(B, C * L, N, V)[:, :T]
    return y + w_r * v, start[:, :, C]


def _plain_conv(x, w, bias, hist):
    B, T, C = x.shape
    past = hist if hist is not None else torch.zeros(B, 3, C, device=x.device, dtype=x.dtype)
    full = torch.cat([past, x], dim=1)
    u = (full[:, 0:T] * w[:, 0] + full[:, 1:T + 1] * w[:, 1]
         + full[:, 2:T + 2] * w[:, 2] + full[:, 3:T + 3] * w[:, 3])
    if bias is not None:
        u = u + bias
    return u / (1.0 + torch.exp(-u)), full[:, T:]


def _plain_norm(y, g_pre, gamma, beta, groups):
    rows, D = y.shape
    yg = y.reshape(rows, groups, D // groups)
    c = yg - yg.mean(-1, keepdim=True)
    z = (c / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS)).reshape(rows, D)
    return (gamma * z + beta) * (g_pre / (1.0 + torch.exp(-g_pre)))


def _leaf(x):
    return None if x is None else x.float().detach().requires_grad_(True)


def _run_plain(s):
    kind = s["kind"]
    if kind == "ssm_prompt":
        y, HT = _plain_ssm(s["k"].float(), s["v"].float(), s["q"].float(), s["logit"], s["alpha"],
                           s["beta"], s["w_r"], s["H0"])
        return {"y": y.to(s["v"].dtype), "HT": HT}
    if kind == "ssm_train":
        names = ["k", "v", "q", "logit", "w_r", "alpha", "beta"] + ["H0"] * (s["H0"] is not None)
        x = {n: _leaf(s[n]) for n in names}
        y, HT = _plain_ssm(x["k"], x["v"], x["q"], x["logit"], x["alpha"], x["beta"], x["w_r"],
                           x.get("H0"))
        outs, grads = [y], [s["dy"].float()]
        if s["dHT"] is not None:
            outs, grads = outs + [HT], grads + [s["dHT"]]
        g = dict(zip(names, torch.autograd.grad(outs, [x[n] for n in names], grads)))
        io = s["v"].dtype
        res = {"y": y.detach().to(io), "HT": HT.detach()}
        for n in names:
            res["d" + n] = g[n].to(io) if n in ("k", "v", "q") else g[n]
        return res
    if kind == "ssm_step":
        d = _softplus(s["logit"].double() + s["beta"].double())
        f = torch.exp(-s["alpha"].double() * d).float()[..., None, None]
        G = s["v"].shape[1] // s["k"].shape[1]
        k, q = (s[n].float().repeat_interleave(G, dim=1) for n in ("k", "q"))
        v, H = s["v"].float(), s["H0"]
        H.mul_(f).add_((k * d.float()[..., None])[..., :, None] * v[..., None, :])
        y = torch.matmul(q[..., None, :], H)[..., 0, :] + s["w_r"] * v
        return {"y": y.to(s["v"].dtype), "H": H}
    if kind == "conv_prompt":
        hist = None if s["hist"] is None else s["hist"].float()
        out, last = _plain_conv(s["x"].float(), s["w"], s["bias"], hist)
        return {"out": out.to(s["x"].dtype), "hist": last.to(s["x"].dtype)}
    if kind == "conv_train":
        names = ["x", "w"] + [n for n in ("bias", "hist") if s[n] is not None]
        x = {n: _leaf(s[n]) for n in names}
        out, last = _plain_conv(x["x"], x["w"], x.get("bias"), x.get("hist"))
        g = dict(zip(names, torch.autograd.grad(out, [x[n] for n in names], s["dout"].float())))
        io = s["x"].dtype
        res = {"out": out.detach().to(io), "hist": last.detach().to(io)}
        for n in names:
            res["d" + n] = g[n].to(io) if n in ("x", "hist") else g[n]
        return res
    if kind == "conv_step":
        out, last = _plain_conv(s["x"].float()[:, None], s["w"], s["bias"], s["hist"].float())
        s["hist"].copy_(last)
        return {"out": out[:, 0].to(s["x"].dtype), "hist": s["hist"]}
    if kind == "norm_fwd":
        out = _plain_norm(s["y"].float(), s["g_pre"].float(), s["gamma"], s["beta"], s["groups"])
        return {"out": out.to(s["y"].dtype)}
    names = ["y", "g_pre", "gamma", "beta"]
    x = {n: _leaf(s[n]) for n in names}
    out = _plain_norm(*(x[n] for n in names), s["groups"])
    g = dict(zip(names, torch.autograd.grad(out, [x[n] for n in names], s["dout"].float())))
    io = s["y"].dtype
    return {"out": out.detach().to(io), "dy": g["y"].to(io), "dg_pre": g["g_pre"].to(io),
            "dgamma": g["gamma"], "dbeta": g["beta"]}


# --------------------------------------------------------------------------- the library

def _run_own(s):
    import matrix_state_nonlinear_amd as m

    kind = s["kind"]
    if kind.startswith("ssm"):
        a = tuple(s[n] for n in ("k", "v", "q", "logit", "alpha", "beta", "w_r"))
        if kind == "ssm_step":
            return {"y": m.m2rnn_ssm_step(s["H0"], *a), "H": s["H0"]}
        y, HT = m.m2rnn_ssm_fwd(*a, H0=s["H0"])
        if kind == "ssm_prompt":
            return {"y": y, "HT": HT}
        g = m.m2rnn_ssm_bwd(*a, s["H0"], s["dy"], dHT=s["dHT"], want_dh0=s["H0"] is not None)
        return {"y": y, "HT": HT, **{n: t for n, t in g.items() if t is not None}}
    if kind == "conv_step":
        return {"out": m.m2rnn_conv_step(s["hist"], s["x"], s["w"], s["bias"]), "hist": s["hist"]}
    if kind.startswith("conv"):
        out, last = m.m2rnn_conv_carry(s["x"], s["w"], s["bias"], hist=s["hist"])
        if kind == "conv_prompt":
            return {"out": out, "hist": last}
        g = m.m2rnn_conv_carry_bwd(s["x"], s["w"], s["bias"], s["hist"], s["dout"])
        return {"out": out, "hist": last, **{n: t for n, t in g.items() if t is not None}}
    a = tuple(s[n] for n in ("y", "g_pre", "gamma", "beta", "groups"))
    out = m.m2rnn_groupnorm_gate(*a, eps=EPS)
    if kind == "norm_fwd":
        return {"out": out}
    dy, dg, dgamma, dbeta = m.m2rnn_groupnorm_gate_bwd(*a, s["dout"], eps=EPS)
    return {"out": out, "dy": dy, "dg_pre": dg, "dgamma": dgamma, "dbeta": dbeta}


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# --------------------------------------------------------------------------- work

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    kind = case["kind"]
    if kind.startswith("ssm"):
        B, T, N, NQ, K, V = (case[x] for x in ("B", "T", "N", "NQ", "K", "V"))
        tok, state = B * T, 4 * B * N * K * V
        io = e * tok * (2 * NQ * K + N * V) + 4 * tok * N   # k, q, v, logit
        par = 4 * N * (V + 2)
        if kind == "ssm_train":
            # in: k, q, v, logit, dy; out: y, dk, dq, dv, dlogit; H0, dHT in, HT, dH0 out
            return {"bytes": 2 * io + 2 * e * tok * N * V + 2 * par
                    + state * (4 if case["carry"] else 1),
                    "flops": 14.0 * tok * N * K * V}
        # the rank-1 write (2 K V) and the readout (2 K V) of each token and head
        return {"bytes": io + e * tok * N * V + par + 2 * state, "flops": 4.0 * tok * N * K * V}
    if kind.startswith("conv"):
        n = case["B"] * case["T"] * case["C"]
        hist = e * 3 * case["B"] * case["C"] * (1 + case["carry"])
        par = 4 * case["C"] * (5 if case["bias"] else 4)
        if kind == "conv_train":   # x, dout in; out, dx out; dhist out
            return {"bytes": 4 * e * n + 2 * hist + 2 * par, "flops": 40.0 * n}
        return {"bytes": 2 * e * n + hist + par, "flops": 12.0 * n}
    n = case["rows"] * case["D"]
    if kind == "norm_train":       # y, g_pre, dout in; out, dy, dg_pre out
        return {"bytes": 6 * e * n + 16 * case["D"], "flops": 45.0 * n}
    return {"bytes": 3 * e * n + 8 * case["D"], "flops": 15.0 * n}


# --------------------------------------------------------------------------- 64-bit values

def _sig(x):
    return torch.special.expit(x)


def _exact_ssm(s, train):
    """Token by token from the recurrence, and its chain rule in reverse."""
    f8 = torch.float64
    k, v, q = (s[n].to(f8) for n in ("k", "v", "q"))
    B, T, NQ, K = k.shape
    N, V = v.shape[2:]
    G = N // NQ
    x = s["logit"].to(f8) + s["beta"].to(f8)
    alpha, w_r = s["alpha"].to(f8), s["w_r"].to(f8)
    d = torch.logaddexp(x, torch.zeros_like(x))
    f = torch.exp(-alpha * d)
    head = torch.arange(N, device=DEV) // G
    y = torch.empty(B, T, N, V, dtype=f8, device=DEV)
    HT = torch.empty(B, N, K, V, dtype=f8, device=DEV)
    res = {"y": y, "HT": HT}
    if train:
        dkh = torch.empty(B, T, N, K, dtype=f8, device=DEV)
        dqh = torch.empty_like(dkh)
        dv, dd, df = torch.empty_like(v), torch.empty_like(x), torch.empty_like(x)
        dH0 = torch.empty_like(HT)
    per = max(1, int(2e9 // (T * N * K * V))) if train else B   # sequences at a time
    for b0 in range(0, B, per):
        r = slice(b0, min(B, b0 + per))
        n = r.stop - r.start
        H = (s["H0"][r].to(f8).clone() if s["H0"] is not None
             else torch.zeros(n, N, K, V, dtype=f8, device=DEV))
        kd = (k[r][:, :, head] * d[r][..., None]).transpose(0, 1).contiguous()
        qh = q[r][:, :, head].transpose(0, 1).contiguous()
        vt, ft = v[r].transpose(0, 1).contiguous(), f[r].transpose(0, 1).contiguous()
        kept = torch.empty(T + 1, n, N, K, V, dtype=f8, device=DEV) if train else None
        if train:
            kept[0] = H
        for t in range(T):
            H.mul_(ft[t][..., None, None]).addcmul_(kd[t][..., :, None], vt[t][..., None, :])
            if train:
                kept[t + 1] = H
            else:
                y[r, t] = torch.matmul(qh[t][..., None, :], H)[..., 0, :]
        HT[r] = H
        if not train:
            continue
        y[r] = torch.matmul(qh[..., None, :], kept[1:])[..., 0, :].transpose(0, 1)
        dyt = s["dy"][r].to(f8).transpose(0, 1).contiguous()
        kh = k[r][:, :, head].transpose(0, 1).contiguous()
        R = (s["dHT"][r].to(f8).clone() if s["dHT"] is not None
             else torch.zeros(n, N, K, V, dtype=f8, device=DEV))
        for t in range(T - 1, -1, -1):
            R.addcmul_(qh[t][..., :, None], dyt[t][..., None, :])
            dqh[r, t] = torch.matmul(kept[t + 1], dyt[t][..., :, None])[..., 0]
            rv = torch.matmul(R, vt[t][..., :, None])[..., 0]
            dkh[r, t] = rv * d[r, t][..., None]
            dd[r, t] = (rv * kh[t]).sum(-1)
            dv[r, t] = torch.matmul(kd[t][..., None, :], R)[..., 0, :]
            df[r, t] = (R * kept[t]).sum((-1, -2))
            R.mul_(ft[t][..., None, None])
        dH0[r] = R
    y += w_r * v
    if train:
        dy = s["dy"].to(f8)
        dl = df * f                      # with respect to log f
        through = _sig(x) * (dd - alpha * dl)
        res.update({"dk": dkh.reshape(B, T, NQ, G, K).sum(3), "dq": dqh.reshape(B, T, NQ, G, K).sum(3),
                    "dv": dv + w_r * dy, "dlogit": through, "dw_r": (dy * v).sum((0, 1)),
                    "dalpha": (-d * dl).sum((0, 1)), "dbeta": through.sum((0, 1))})
        if s["H0"] is not None:
            res["dH0"] = dH0
    return res


def _exact_conv(s, kind):
    f8 = torch.float64
    x = s["x"].to(f8)
    x = x[:, None] if kind == "conv_step" else x
    B, T, C = x.shape
    w = s["w"].to(f8)
    full = torch.zeros(B, T + 3, C, dtype=f8, device=DEV)
    full[:, 3:] = x
    if s["hist"] is not None:
        full[:, :3] = s["hist"].to(f8)
    u = sum(w[:, i] * full[:, i:i + T] for i in range(4))
    u = u if s["bias"] is None else u + s["bias"].to(f8)
    sg = _sig(u)
    if kind == "conv_step":
        return {"out": (u * sg)[:, 0], "hist": full[:, T:]}
    res = {"out": u * sg, "hist": full[:, T:]}
    if kind == "conv_train":
        du = s["dout"].to(f8) * (sg + u * sg * (1 - sg))
        dfull = torch.zeros_like(full)
        for i in range(4):
            dfull[:, i:i + T] += w[:, i] * du
        res["dx"] = dfull[:, 3:]
        res["dw"] = torch.stack([(du * full[:, i:i + T]).sum((0, 1)) for i in range(4)], dim=1)
        if s["bias"] is not None:
            res["dbias"] = du.sum((0, 1))
        if s["hist"] is not None:
            res["dhist"] = dfull[:, :3]
    return res


def _exact_norm(s, train):
    f8 = torch.float64
    y, g, gamma, beta = (s[n].to(f8) for n in ("y", "g_pre", "gamma", "beta"))
    rows, D = y.shape
    shape = (rows, s["groups"], D // s["groups"])
    var, mean = torch.var_mean(y.reshape(shape), dim=-1, correction=0, keepdim=True)
    inv = (var + EPS).rsqrt()
    z = ((y.reshape(shape) - mean) * inv).reshape(rows, D)
    sg = _sig(g)
    a = gamma * z + beta
    res = {"out": a * g * sg}
    if train:
        dout = s["dout"].to(f8)
        da = dout * g * sg
        dz = (da * gamma).reshape(shape)
        zg = z.reshape(shape)
        dy = inv * (dz - dz.mean(-1, keepdim=True) - zg * (dz * zg).mean(-1, keepdim=True))
        res.update({"dy": dy.reshape(rows, D), "dg_pre": dout * a * (sg + g * sg * (1 - sg)),
                    "dgamma": (da * z).sum(0), "dbeta": da.sum(0)})
    return res


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "ssm_step":
        for n in ("k", "v", "q", "logit"):
            s[n] = s[n][:, None]
        r = _exact_ssm(s, False)
        return {"y": r["y"][:, 0], "H": r["HT"]}
    if kind.startswith("ssm"):
        return _exact_ssm(s, kind == "ssm_train")
    if kind.startswith("conv"):
        return _exact_conv(s, kind)
    return _exact_norm(s, kind == "norm_train")
