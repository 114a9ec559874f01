"""Cases of the gated delta rule and of the row norms, their plain forms and their definitions in 64 bits.

The delta rule keeps a fast weight S [dk, dv] per head.  With a_i = exp(g_i):
  r_i = v_i - a_i S_{i-1}^T k_i,  S_i = a_i S_{i-1} + k_i (beta_i r_i)^T,  out_i = S_i^T q_i.
The row norms are layer norm and RMS norm over the last axis, with the gradients of weight and bias.
"""
import math

import torch

own = False

CHUNK = 64
GATE_FLOOR = -128.0        # exp(-128) is 0 in 32 bits: a gate below this (-inf: a new document) forgets all
NORM_EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # training step's forward of a 16-head layer at the head size of the causal workload
        dict(name="delta_fwd_train_d128", op="delta_fwd", B=4, H=16, N=4096, dk=128, dv=128, dtype="bf16", gate="soft", state="none"),
        # prefill of long prompts that hands its state on to single-token steps
        dict(name="delta_fwd_prefill_long", op="delta_fwd", B=2, H=16, N=16384, dk=128, dv=128, dtype="bf16", gate="soft", state="final"),
        # packed documents of odd lengths continued from an earlier state, small heads
        dict(name="delta_fwd_packed_d64", op="delta_fwd", B=2, H=8, N=4093, dk=64, dv=64, dtype="bf16", gate="reset", state="carry"),
        # 32-bit check run of a small model
        dict(name="delta_fwd_f32_small", op="delta_fwd", B=1, H=4, N=256, dk=32, dv=32, dtype="f32", gate="soft", state="final"),
        # training step's backward at the same heads
        dict(name="delta_bwd_train_d128", op="delta_bwd", B=4, H=16, N=2048, dk=128, dv=128, dtype="bf16", gate="soft", state=False),
        # backward of one segment of a longer sequence: state and its gradient pass through, odd length
        dict(name="delta_bwd_f32_carry", op="delta_bwd", B=2, H=4, N=1001, dk=64, dv=32, dtype="f32", gate="soft", state=True),
        # serving: one token for a large batch, and for one sequence
        dict(name="delta_step_batch", op="delta_step", B=256, H=32, dk=128, dv=128, dtype="bf16", gate="soft"),
        dict(name="delta_step_one", op="delta_step", B=1, H=8, dk=64, dv=64, dtype="bf16", gate="soft"),
        # layer norm of every head's read-out; RMS norm of a model's rows in 32 bits, odd width
        dict(name="norm_fwd_heads", op="norm_fwd", rows=1048576, d=128, kind="layer", dtype="bf16", weight=True, bias=True),
        dict(name="norm_fwd_rms_f32_odd", op="norm_fwd", rows=777, d=2049, kind="rms", dtype="f32", weight=True, bias=False),
        # their backward: every head's read-out, and a model's rows
        dict(name="norm_bwd_heads", op="norm_bwd", rows=524288, d=128, kind="layer", dtype="bf16", weight=True, bias=True),
        dict(name="norm_bwd_model", op="norm_bwd", rows=8192, d=2048, kind="layer", dtype="bf16", weight=True, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta_fwd", "delta_fwd", "delta_bwd", "delta_bwd", "delta_step", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("norm"):
        d = _log(rng, 8, 8192)
        rows = _log(rng, 1, max(1, min(1 << 19, (1 << 26) // d)))
        weight = rng.random() < 0.8
        return dict(op=op, rows=rows, d=d, kind=rng.choice(["layer", "rms"]), dtype=dtype,
                    weight=weight, bias=weight and rng.random() < 0.5)
    dims = [16, 32, 64, 128]
    big = rng.random() < 0.5
    c = dict(op=op, dk=128 if big else rng.choice(dims), dv=128 if big else rng.choice(dims), dtype=dtype,
             gate=rng.choice(["none", "soft", "soft", "reset"]))
    if op == "delta_step":
        return dict(c, B=_log(rng, 1, 256), H=rng.randint(1, 32), gate=rng.choice(["none", "soft"]))
    top = 16384 if op == "delta_fwd" else 2048
    N = _log(rng, 1, top)
    H = rng.randint(1, 16)
    room = ((1 << 19) if op == "delta_fwd" else (1 << 17)) // (N * H)
    B = _log(rng, 1, max(1, min(8, room)))
    state = rng.choice(["none", "final", "carry"]) if op == "delta_fwd" else rng.random() < 0.4
    return dict(c, B=B, H=H, N=N, state=state)


# ------------------------------------------------------------------ inputs
def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-6)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float32)
    rand = lambda *s: torch.rand(s, generator=gen, device="cuda", dtype=torch.float32)
    t, op = DTYPES[case["dtype"]], case["op"]
    s = {"case": dict(case)}
    if op.startswith("norm"):
        rows, d = case["rows"], case["d"]
        s["x"] = (randn(rows, d) * (0.5 + rand(rows, 1)) + 0.5 * randn(rows, 1)).to(t)
        s["w"] = 1.0 + 0.2 * randn(d) if case["weight"] else None
        s["b"] = 0.2 * randn(d) if case["bias"] else None
        if op == "norm_bwd":
            s["dy"] = randn(rows, d).to(t)
        return s
    lead = (case["B"], case["H"]) if op == "delta_step" else (case["B"], case["H"], case["N"])
    dk, dv = case["dk"], case["dv"]
    # unit keys with a part in common, as trained ones have; the 1/sqrt(dk) of the scores sits in q
    common = randn(case["B"], case["H"], *([1] * (len(lead) - 2)), dk)
    s["q"] = (_unit(randn(*lead, dk)) * dk ** -0.5).to(t)
    s["k"] = _unit(randn(*lead, dk) + 0.3 * common).to(t)
    s["v"] = randn(*lead, dv).to(t)
    s["beta"] = torch.sigmoid(randn(*lead))
    s["g"] = None
    if case["gate"] != "none":
        # decays from a few tokens to a few thousand, by head and token
        s["g"] = -torch.exp(1.5 * randn(*lead) + 2.0 * randn(case["B"], case["H"], *([1] * (len(lead) - 2))) - 5.0)
        if case["gate"] == "reset":
            s["g"] = torch.where(rand(*lead) < 1.0 / 300, torch.full_like(s["g"], -math.inf), s["g"])
    state = lambda: 0.1 * randn(case["B"], case["H"], dk, dv)
    if op == "delta_step":
        s["S"] = state()
    else:
        s["S0"] = state() if case["state"] in ("carry", True) else None
    if op == "delta_bwd":
        s["dout"] = randn(*lead, dv).to(t)
        s["dS"] = state() if case["state"] else None
    return s


# ------------------------------------------------------------------ plain forms
def _chunks(x, C):
    """[B, H, N, ...] as [B, H, chunks, C, ...], with zeros behind the last token."""
    B, H, N = x.shape[:3]
    n = -(-N // C)
    pad = x.new_zeros((B, H, n * C - N) + tuple(x.shape[3:]))
    return torch.cat([x, pad], 2).reshape((B, H, n, C) + tuple(x.shape[3:]))


def _delta_plain(q, k, v, g, beta, S):
    """out and the last state in 32 bits; gates, their exponents and the solve inside a chunk in 64."""
    N, C = q.shape[2], min(CHUNK, q.shape[2])
    q, k, v, beta = _chunks(q, C), _chunks(k, C), _chunks(v, C), _chunks(beta, C)
    n = q.shape[2]
    gam = torch.zeros_like(beta, dtype=torch.float64) if g is None else _chunks(g, C).double().clamp_min(GATE_FLOOR).cumsum(-1)
    low = torch.ones(C, C, device=q.device, dtype=torch.bool).tril()
    Gam = torch.exp((gam[..., :, None] - gam[..., None, :]).masked_fill(~low, -math.inf))
    kt = k.transpose(-1, -2)
    P = (Gam * (q @ kt)).float()
    A = (Gam * (k @ kt)).tril(-1) * beta[..., None, :].double()
    # (I + A)^-1 of a strictly lower A: (I - A)(I + A^2)(I + A^4)...
    eye = torch.eye(C, device=q.device, dtype=torch.float64)
    T, W = eye - A, A @ A
    for _ in range(max(0, (C - 1).bit_length() - 1)):
        T, W = T + T @ W, W @ W
    T = T.float()
    eg = torch.exp(gam)[..., None].float()
    el = torch.exp(gam[..., -1:] - gam)[..., None].float()
    out = []
    for c in range(n):
        r = T[:, :, c] @ (v[:, :, c] - eg[:, :, c] * (k[:, :, c] @ S))
        u = beta[:, :, c, :, None] * r
        out.append(eg[:, :, c] * (q[:, :, c] @ S) + P[:, :, c] @ u)
        S = eg[:, :, c, -1:] * S + kt[:, :, c] @ (el[:, :, c] * u)
    return torch.cat(out, 2)[:, :, :N], S


def _zero_state(s):
    c = s["case"]
    return torch.zeros(c["B"], c["H"], c["dk"], c["dv"], device=s["q"].device)


def _norm_parts(s):
    c, x = s["case"], s["x"].float()
    if c["kind"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + NORM_EPS)
    return x * rstd, rstd


def _plain(s):
    c = s["case"]
    t, op = DTYPES[c["dtype"]], c["op"]
    if op == "delta_fwd":
        out, S = _delta_plain(s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["beta"],
                              _zero_state(s) if s["S0"] is None else s["S0"])
        return {"out": out.to(t)} if c["state"] == "none" else {"out": out.to(t), "S": S}
    if op == "delta_bwd":
        leaf = {n: s[n].float().detach().requires_grad_(True) for n in ("q", "k", "v", "beta")}
        leaf["g"] = None if s["g"] is None else s["g"].detach().requires_grad_(True)
        leaf["S0"] = (_zero_state(s) if s["S0"] is None else s["S0"]).detach().requires_grad_(True)
        out, S = _delta_plain(leaf["q"], leaf["k"], leaf["v"], leaf["g"], leaf["beta"], leaf["S0"])
        loss = (out * s["dout"].float()).sum()
        if s["dS"] is not None:
            loss = loss + (S * s["dS"]).sum()
        names = [n for n in leaf if leaf[n] is not None and (n != "S0" or c["state"])]
        grads = dict(zip(names, torch.autograd.grad(loss, [leaf[n] for n in names])))
        return {"d" + n: x.to(t) if n in ("q", "k", "v") else x for n, x in grads.items()}
    if op == "delta_step":
        q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
        a = 1.0 if s["g"] is None else torch.exp(s["g"])[..., None, None]
        S = a * s["S"]
        r = v - (S * k[..., None]).sum(-2)
        S = S + k[..., None] * (s["beta"][..., None] * r)[..., None, :]
        s["S"].copy_(S)
        return {"out": (S * q[..., None]).sum(-2).to(t), "S": s["S"]}
    xh, rstd = _norm_parts(s)
    if op == "norm_fwd":
        y = xh if s["w"] is None else xh * s["w"]
        return {"out": (y if s["b"] is None else y + s["b"]).to(t)}
    dy = s["dy"].float()
    wdy = dy if s["w"] is None else dy * s["w"]
    dx = wdy - xh * (wdy * xh).mean(-1, keepdim=True)
    if c["kind"] == "layer":
        dx = dx - wdy.mean(-1, keepdim=True)
    got = {"dx": (rstd * dx).to(t)}
    if s["w"] is not None:
        got["dw"] = (dy * xh).sum(0)
    if s["b"] is not None:
        got["db"] = dy.sum(0)
    return got


def _own(s):
    from weight_state_recurrence_b200 import linattn
    c = s["case"]
    if c["op"] == "delta_fwd":
        out, S = linattn.delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S0"], want_state=c["state"] != "none")
        return {"out": out} if S is None else {"out": out, "S": S}
    if c["op"] == "delta_bwd":
        dq, dk, dv, dg, dbeta, dS0 = linattn.delta_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["dout"],
                                                       s["S0"], s["dS"], want_dS_init=c["state"])
        got = {"dq": dq, "dk": dk, "dv": dv, "dbeta": dbeta, "dg": dg, "dS0": dS0}
        return {n: x for n, x in got.items() if x is not None}
    if c["op"] == "delta_step":
        out = linattn.delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"])
        return {"out": out, "S": s["S"]}
    kind = linattn.LINATTN_NORM_LAYER if c["kind"] == "layer" else linattn.LINATTN_NORM_RMS
    if c["op"] == "norm_fwd":
        return {"out": linattn.norm_fwd(s["x"], s["w"], s["b"], NORM_EPS, kind)}
    dx, dw, db = linattn.norm_bwd(s["x"], s["w"], s["dy"], NORM_EPS, kind, want_dweight=s["w"] is not None,
                                  want_dbias=s["b"] is not None)
    got = {"dx": dx, "dw": dw, "db": db}
    return {n: x for n, x in got.items() if x is not None}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"].startswith("norm"):
        n = c["rows"] * c["d"]
        vec = 4 * c["d"] * (c["weight"] + c["bias"])
        if c["op"] == "norm_fwd":
            return {"bytes": 2 * e * n + vec, "flops": 8 * n}
        return {"bytes": 3 * e * n + vec + 4 * c["d"] * c["weight"], "flops": 14 * n}
    dk, dv = c["dk"], c["dv"]
    heads = c["B"] * c["H"]
    tok = heads * c.get("N", 1)
    gate = 4 * (1 + (c["gate"] != "none"))
    S = 4 * heads * dk * dv
    if c["op"] == "delta_fwd":
        states = {"none": 0, "final": 1, "carry": 2}[c["state"]]
        return {"bytes": tok * (2 * e * (dk + dv) + gate) + states * S, "flops": 6 * tok * dk * dv}
    if c["op"] == "delta_bwd":
        return {"bytes": tok * (e * (4 * dk + 3 * dv) + 2 * gate) + 3 * bool(c["state"]) * S, "flops": 16 * tok * dk * dv}
    return {"bytes": tok * (2 * e * (dk + dv) + gate) + 2 * S, "flops": 6 * tok * dk * dv}


# ------------------------------------------------------------------ the definitions in 64 bits
def _walk(q, k, v, a, beta, S, keep):
    """The recurrence token by token; `keep`: the state before each token of the first ones kept, and each r."""
    outs, rs, before = [], [], []
    for i in range(q.shape[2]):
        if keep:
            before.append(S)
        S = S * a[:, :, i, None, None]
        r = v[:, :, i] - torch.einsum("bhkv,bhk->bhv", S, k[:, :, i])
        S = S + torch.einsum("bhk,bhv->bhkv", k[:, :, i], beta[:, :, i, None] * r)
        outs.append(torch.einsum("bhkv,bhk->bhv", S, q[:, :, i]))
        rs.append(r)
    return outs, rs, before, S


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"].startswith("norm"):
        return _exact_norm(s)
    d64 = lambda n: s[n].double()
    q, k, v, beta = d64("q"), d64("k"), d64("v"), d64("beta")
    a = torch.ones_like(beta) if s["g"] is None else torch.exp(d64("g"))
    if c["op"] == "delta_step":
        one = lambda x: x.unsqueeze(2)
        outs, _, _, S = _walk(one(q), one(k), one(v), one(a), one(beta), d64("S"), False)
        return {"out": outs[0], "S": S}
    S = _zero_state(s).double() if s["S0"] is None else d64("S0")
    if c["op"] == "delta_fwd":
        outs, _, _, S = _walk(q, k, v, a, beta, S, False)
        out = torch.stack(outs, 2)
        return {"out": out} if c["state"] == "none" else {"out": out, "S": S}
    # backward: states at every 64th token, then block by block from the end
    N, starts = q.shape[2], [S]
    cut = lambda x, i: x[:, :, i:i + 64]
    for i in range(0, N, 64):
        S = _walk(cut(q, i), cut(k, i), cut(v, i), cut(a, i), cut(beta, i), S, False)[3]
        starts.append(S)
    do = d64("dout")
    D = torch.zeros_like(S) if s["dS"] is None else d64("dS")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    da, db = torch.zeros_like(a), torch.zeros_like(beta)
    for blk in range(len(starts) - 2, -1, -1):
        i0 = 64 * blk
        _, rs, before, after = _walk(cut(q, i0), cut(k, i0), cut(v, i0), cut(a, i0), cut(beta, i0), starts[blk], True)
        for j in range(len(rs) - 1, -1, -1):
            i = i0 + j
            Si = before[j + 1] if j + 1 < len(rs) else after
            dq[:, :, i] = torch.einsum("bhkv,bhv->bhk", Si, do[:, :, i])
            D = D + torch.einsum("bhk,bhv->bhkv", q[:, :, i], do[:, :, i])
            bi, ai = beta[:, :, i, None], a[:, :, i, None]
            du = torch.einsum("bhkv,bhk->bhv", D, k[:, :, i])
            db[:, :, i] = (du * rs[j]).sum(-1)
            dr = bi * du
            dv[:, :, i] = dr
            dk[:, :, i] = torch.einsum("bhkv,bhv->bhk", D, bi * rs[j]) - ai * torch.einsum("bhkv,bhv->bhk", before[j], dr)
            Dd = D - torch.einsum("bhk,bhv->bhkv", k[:, :, i], dr)
            da[:, :, i] = (Dd * before[j]).sum((-1, -2))
            D = ai[..., None] * Dd
    got = {"dq": dq, "dk": dk, "dv": dv, "dbeta": db}
    if s["g"] is not None:
        got["dg"] = da * a
    if c["state"]:
        got["dS0"] = D
    return got


def _exact_norm(s):
    c, x = s["case"], s["x"].double()
    n = x.shape[1]
    m = x.sum(1, keepdim=True) / n if c["kind"] == "layer" else torch.zeros_like(x[:, :1])
    var = ((x - m) ** 2).sum(1, keepdim=True) / n
    sd = (var + NORM_EPS).sqrt()
    xh = (x - m) / sd
    w = torch.ones(n, dtype=x.dtype, device=x.device) if s["w"] is None else s["w"].double()
    if c["op"] == "norm_fwd":
        return {"out": xh * w + (0.0 if s["b"] is None else s["b"].double())}
    dy = s["dy"].double()
    dxh = dy * w
    dvar = (dxh * (x - m)).sum(1, keepdim=True) * -0.5 / sd ** 3
    dx = dxh / sd + dvar * 2.0 * (x - m) / n
    if c["kind"] == "layer":
        dx = dx - (dxh / sd).sum(1, keepdim=True) / n
    got = {"dx": dx}
    if s["w"] is not None:
        got["dw"] = (dy * xh).sum(0)
    if s["b"] is not None:
        got["db"] = dy.sum(0)
    return got
