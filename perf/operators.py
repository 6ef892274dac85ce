"""The trainable sequence block's operators as they are timed: layer normalisation, the gated
feed-forward branch and linear attention with a decay for each head, each in its directions.

`own` false runs the plain form (elementary torch operations in 32 bits, rounded once at the
end); `own` true makes the calls a user makes of this repository's kernels.  `listed()` holds
the fixed cases, `draw(rng)` gives more of the same ranges, `exact(case, seed)` the definition
in 64 bits, written apart from the plain form.

Definitions (x_t a token's row):
  layer norm   y = (x - mean) rstd gamma + beta, rstd = 1 / sqrt(var + eps)
  feed-forward y = (act(x Wg^T) * (x Wu^T)) Wd^T + res, act = SiLU or GELU (v Phi(v))
  linear attention, per head with decay g:  S_t = g S_{t-1} + k_t v_t^T,  o_t = S_t^T q_t
"""
import math

import torch

own = False

F32, BF16 = "f32", "bf16"
EPS = 1e-6


def _dt(name):
    return torch.bfloat16 if name == BF16 else torch.float32


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one 14 x 14 feature map of the plain backbone (384 channels): the smallest call
        {"name": "ln_fwd_196x384", "op": "ln_fwd", "rows": 196, "dim": 384, "dtype": BF16},
        # the 56 x 56 stride-4 maps of a batch of 32 (64 channels)
        {"name": "ln_fwd_100352x64", "op": "ln_fwd", "rows": 100352, "dim": 64, "dtype": BF16},
        # the plain backbone's batch of 128 maps in training, the residual's gradient joined in
        {"name": "ln_bwd_25088x384", "op": "ln_bwd", "rows": 25088, "dim": 384, "dtype": BF16, "dres": True},
        # a wide fp32 layer with an odd number of rows
        {"name": "ln_bwd_8209x2560_f32", "op": "ln_bwd", "rows": 8209, "dim": 2560, "dtype": F32, "dres": False},
        # one new token of each of four sequences: the weights' bytes are all there is
        {"name": "ffn_fwd_4x2048x5632", "op": "ffn_fwd", "rows": 4, "dim": 2048, "hidden": 5632, "act": "silu",
         "save": False, "res": True},
        # the stride-16 maps (14 x 14, 256 channels, batch 64) in training: pre-activations kept
        {"name": "ffn_fwd_12544x256x1024", "op": "ffn_fwd", "rows": 12544, "dim": 256, "hidden": 1024, "act": "gelu",
         "save": True, "res": True},
        # a prompt of 8192 tokens through a wide layer
        {"name": "ffn_fwd_8192x2048x5632", "op": "ffn_fwd", "rows": 8192, "dim": 2048, "hidden": 5632, "act": "silu",
         "save": False, "res": True},
        # the same layer's backward pass: the largest case
        {"name": "ffn_bwd_8192x2048x5632", "op": "ffn_bwd", "rows": 8192, "dim": 2048, "hidden": 5632, "act": "silu"},
        # rows and widths that end inside a tile
        {"name": "ffn_bwd_1531x520x1384", "op": "ffn_bwd", "rows": 1531, "dim": 520, "hidden": 1384, "act": "gelu"},
        # a long prompt of one sequence, q, k and v slices of one projection's rows, the state kept
        {"name": "lattn_fwd_1x16384_16x128", "op": "lattn_fwd", "B": 1, "T": 16384, "heads": 16, "d": 128,
         "packed": True, "lengths": False, "state": True},
        # a training batch of padded sequences
        {"name": "lattn_bwd_8x2048_16x64", "op": "lattn_bwd", "B": 8, "T": 2048, "heads": 16, "d": 64,
         "packed": False, "lengths": True, "state": False},
        # one new token of each of 64 sequences
        {"name": "lattn_step_64_16x64", "op": "lattn_step", "B": 64, "heads": 16, "d": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "ffn_fwd", "ffn_fwd", "ffn_bwd", "lattn_fwd", "lattn_bwd", "lattn_step"])
    if op in ("ln_fwd", "ln_bwd"):
        dim = _log(rng, 16, 8192)
        if rng.random() < 0.6:
            dim = max(8, dim // 8 * 8)
        rows = _log(rng, 1, max(1, min(131072, (1 << 26) // dim)))
        c = {"op": op, "rows": rows, "dim": dim, "dtype": rng.choice([F32, BF16])}
        if op == "ln_bwd":
            c["dres"] = rng.random() < 0.5
        return c
    if op in ("ffn_fwd", "ffn_bwd"):
        dim = max(8, _log(rng, 64, 4096) // 8 * 8)
        hidden = max(8, int(dim * rng.uniform(1.3, 4.5)) // 8 * 8)
        most = 8192 * 2048 * 5632 // (dim * hidden)
        rows = _log(rng, 1, max(1, min(65536, most)))
        c = {"op": op, "rows": rows, "dim": dim, "hidden": hidden, "act": rng.choice(["silu", "gelu"])}
        if op == "ffn_fwd":
            c["save"] = rng.random() < 0.5
            c["res"] = rng.random() < 0.5
        return c
    d = rng.choice([32, 64, 128])
    heads = _log(rng, 1, 32)
    if op == "lattn_step":
        return {"op": op, "B": _log(rng, 1, max(1, (1 << 24) // (heads * d * d))), "heads": heads, "d": d}
    T = _log(rng, 1, 32768)
    B = _log(rng, 1, max(1, min(64, (1 << 25) // (T * heads * d))))
    return {"op": op, "B": B, "T": T, "heads": heads, "d": d, "packed": rng.random() < 0.5,
            "lengths": rng.random() < 0.5, "state": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _decays(heads):
    """Retentions spread as 1 - 2^-(2 .. 10) over the heads: memories of 4 to 1024 tokens."""
    e = [2.0 + 8.0 * i / max(1, heads - 1) for i in range(heads)]
    return torch.tensor([1.0 - 2.0 ** -x for x in e], dtype=torch.float32)


def _inputs(case, seed):
    """The tensors of one pass, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)

    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        M, D, dt = case["rows"], case["dim"], _dt(case["dtype"])
        s = {}
        # a residual stream: a common offset, and channels of unlike size
        width = torch.exp(0.5 * torch.randn(D, device="cuda", generator=g))
        s["x"] = (torch.randn(M, D, device="cuda", generator=g) * width + 0.3).to(dt)
        s["gamma"] = 1.0 + normal(D, scale=0.2, dtype=torch.float32)
        s["beta"] = normal(D, scale=0.2, dtype=torch.float32)
        if op == "ln_bwd":
            s["dy"] = normal(M, D, dtype=dt)
            s["dres"] = normal(M, D, dtype=dt) if case["dres"] else None
            x = s["x"].double()
            mean = x.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = (((x - mean[:, None]) ** 2).mean(1) + EPS).rsqrt().float()
        return s
    if op in ("ffn_fwd", "ffn_bwd"):
        M, D, F = case["rows"], case["dim"], case["hidden"]
        s = {"x": normal(M, D), "W_gate": normal(F, D, scale=D ** -0.5), "W_up": normal(F, D, scale=D ** -0.5),
             "W_down": normal(D, F, scale=F ** -0.5)}
        if op == "ffn_fwd":
            s["res"] = normal(M, D) if case["res"] else None
        else:
            # what the forward kept: the two pre-activations, in bf16
            s["gate"] = (s["x"].float() @ s["W_gate"].float().t()).to(torch.bfloat16)
            s["up"] = (s["x"].float() @ s["W_up"].float().t()).to(torch.bfloat16)
            s["dy"] = normal(M, D)
        return s
    B, H, d = case["B"], case["heads"], case["d"]
    if op == "lattn_step":
        D = H * d
        return {"q": normal(B, D, scale=d ** -0.5), "k": normal(B, D), "v": normal(B, D),
                "state": normal(B, H, d, d, dtype=torch.float32), "decay": _decays(H)}
    T, D = case["T"], H * d
    s = {"decay": _decays(H), "lengths": None, "state_in": None, "dstate_out": None}
    qkv = torch.randn(B, T, 3, D, device="cuda", generator=g)
    qkv[:, :, 0] *= d ** -0.5
    qkv = qkv.to(torch.bfloat16)
    if case["packed"]:
        s["q"], s["k"], s["v"] = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    else:
        s["q"], s["k"], s["v"] = (qkv[:, :, i].contiguous() for i in range(3))
    if case["lengths"]:
        s["lengths"] = torch.randint(0, T + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
        s["lengths"][0] = T
    if case["state"]:
        s["state_in"] = normal(B, H, d, d, dtype=torch.float32)
    if op == "lattn_bwd":
        s["do"] = normal(B, T, D)
        if case["state"]:
            s["dstate_out"] = normal(B, H, d, d, dtype=torch.float32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    op = case["op"]
    # the output buffers that a program keeps
    if op == "ln_fwd":
        s["y"] = torch.empty_like(s["x"])
        s["mean"] = torch.empty(case["rows"], device="cuda")
        s["rstd"] = torch.empty(case["rows"], device="cuda")
    elif op == "ln_bwd":
        s["dx"] = torch.empty_like(s["x"])
        s["dgamma"] = torch.empty(case["dim"], device="cuda")
        s["dbeta"] = torch.empty(case["dim"], device="cuda")
    elif op == "ffn_fwd":
        s["y"] = torch.empty_like(s["x"])
        if case["save"]:
            s["gate"] = torch.empty(case["rows"], case["hidden"], device="cuda", dtype=torch.bfloat16)
            s["up"] = torch.empty_like(s["gate"])
    elif op == "ffn_bwd":
        s["dx"] = torch.empty_like(s["x"])
        s["grads"] = {k: torch.empty_like(s[k]) for k in ("W_gate", "W_up", "W_down")}
    elif op == "lattn_step":
        s["o"] = torch.empty_like(s["q"])
    else:
        B, T, H, d = case["B"], case["T"], case["heads"], case["d"]
        # rows past a sequence's length stay as they were
        if op == "lattn_fwd":
            s["o"] = torch.zeros(B, T, H * d, device="cuda", dtype=torch.bfloat16)
            s["state_out"] = torch.empty(B, H, d, d, device="cuda") if case["state"] else None
        else:
            if case["packed"]:
                dqkv = torch.zeros(B, T, 3, H * d, device="cuda", dtype=torch.bfloat16)
                s["dq"], s["dk"], s["dv"] = dqkv[:, :, 0], dqkv[:, :, 1], dqkv[:, :, 2]
            else:
                s["dq"], s["dk"], s["dv"] = (torch.zeros(B, T, H * d, device="cuda", dtype=torch.bfloat16)
                                             for _ in range(3))
            s["dstate_in"] = torch.empty(B, H, d, d, device="cuda") if case["state"] else None
    if own:
        import self_referential_nested_b200 as S
        s["S"] = S
        if op in ("ln_fwd", "ln_bwd"):
            s["h"] = S.srnl_ln_create(dict(dim=case["dim"], eps=EPS, act_dtype=case["dtype"]))
        elif op in ("ffn_fwd", "ffn_bwd"):
            s["h"] = S.srnl_ffn_create(dict(dim=case["dim"], hidden=case["hidden"], max_rows=case["rows"],
                                            activation=case["act"], training=op == "ffn_bwd"))
            s["params"] = {k: s[k] for k in ("W_gate", "W_up", "W_down")}
        else:
            D = case["heads"] * case["d"]
            s["h"] = S.srnl_lattn_create(dict(B=case["B"], T=case.get("T", 1), heads=case["heads"], d=case["d"],
                                              ld=3 * D if case.get("packed") else 0), s["decay"].numpy())
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    return _run_own(op, s) if own else _PLAIN[op](s)


def _run_own(op, s):
    S, h = s["S"], s["h"]
    if op == "ln_fwd":
        S.srnl_ln_forward(h, s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "ln_bwd":
        S.srnl_ln_backward(h, s["x"], s["dy"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"],
                           dres=s["dres"])
        return {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "ffn_fwd":
        S.srnl_ffn_forward(h, s["x"], s["params"], s["y"], res=s["res"], gate=s.get("gate"), up=s.get("up"))
        return {k: s[k] for k in ("y", "gate", "up") if k in s}
    if op == "ffn_bwd":
        S.srnl_ffn_backward(h, s["x"], s["gate"], s["up"], s["dy"], s["params"], s["dx"], s["grads"])
        return {"dx": s["dx"], "grads": s["grads"]}
    if op == "lattn_step":
        S.srnl_lattn_step(h, s["q"], s["k"], s["v"], s["o"], s["state"])
        return {"o": s["o"], "state": s["state"]}
    if op == "lattn_fwd":
        S.srnl_lattn_forward(h, s["q"], s["k"], s["v"], s["o"], lengths=s["lengths"], state_in=s["state_in"],
                             state_out=s["state_out"])
        return {k: s[k] for k in ("o", "state_out") if s[k] is not None}
    S.srnl_lattn_backward(h, s["q"], s["k"], s["v"], s["do"], s["dq"], s["dk"], s["dv"], lengths=s["lengths"],
                          state_in=s["state_in"], dstate_out=s["dstate_out"], dstate_in=s["dstate_in"])
    return {k: s[k] for k in ("dq", "dk", "dv", "dstate_in") if s[k] is not None}


def _plain_ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = ((c * c).mean(1) + EPS).rsqrt()
    y = c * rstd[:, None] * s["gamma"] + s["beta"]
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_ln_bwd(s):
    dy = s["dy"].float()
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    w = dy * s["gamma"]
    dx = (w - w.mean(1, keepdim=True) - xhat * (w * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0)}


def _act(v, kind):
    """The activation and its derivative."""
    if kind == "silu":
        p = torch.sigmoid(v)
        return v * p, p * (1 + v * (1 - p))
    p = 0.5 * (1 + torch.erf(v * 0.5 ** 0.5))
    return v * p, p + v * torch.exp(-0.5 * v * v) * (2 * math.pi) ** -0.5


def _plain_ffn_fwd(s):
    x = s["x"].float()
    gate, up = x @ s["W_gate"].float().t(), x @ s["W_up"].float().t()
    y = (_act(gate, s["case"]["act"])[0] * up) @ s["W_down"].float().t()
    if s["res"] is not None:
        y = y + s["res"].float()
    out = {"y": y.to(torch.bfloat16)}
    if s["case"]["save"]:
        out["gate"], out["up"] = gate.to(torch.bfloat16), up.to(torch.bfloat16)
    return out


def _plain_ffn_bwd(s):
    x, dy, up = s["x"].float(), s["dy"].float(), s["up"].float()
    a, da = _act(s["gate"].float(), s["case"]["act"])
    dh = dy @ s["W_down"].float()
    dgate, dup = dh * up * da, dh * a
    dx = dgate @ s["W_gate"].float() + dup @ s["W_up"].float()
    grads = {"W_gate": dgate.t() @ x, "W_up": dup.t() @ x, "W_down": dy.t() @ (a * up)}
    return {"dx": dx.to(torch.bfloat16), "grads": {k: v.to(torch.bfloat16) for k, v in grads.items()}}


def _plain_lattn_step(s):
    B, H, d, _ = s["state"].shape
    q, k, v = (s[n].float().view(B, H, d) for n in "qkv")
    s["state"].mul_(s["decay"].cuda()[:, None, None]).add_(k[..., :, None] * v[..., None, :])
    o = (q[..., :, None] * s["state"]).sum(2)
    return {"o": o.reshape(B, H * d).to(torch.bfloat16), "state": s["state"]}


def _heads(t, d):
    """[B, T, H d] -> fp32 [B, H, T, d]."""
    B, T, D = t.shape
    return t.float().view(B, T, D // d, d).transpose(1, 2)


def _rows(t):
    """fp32 [B, H, T, d] -> bf16 [B, T, H d]."""
    B, H, T, d = t.shape
    return t.transpose(1, 2).reshape(B, T, H * d).to(torch.bfloat16)


def _decayed(a, b, c, lg, chunk=64):
    """sum_{j <= t} g^(t - j) (a_t . b_j) c_j over [B, H, T, d]; lg [H]: log g in 64 bits."""
    B, H, T, d = a.shape
    n = -(-T // chunk)
    a, b, c = (torch.nn.functional.pad(t, (0, 0, 0, n * chunk - T)).view(B, H, n, chunk, d) for t in (a, b, c))
    i = torch.arange(chunk, device=a.device, dtype=torch.float64)
    m = torch.arange(n, device=a.device, dtype=torch.float64)

    def power(e):   # g^e where e >= 0, else 0
        return torch.where(e >= 0, torch.exp(lg[:, None, None] * e.clamp_min(0)), 0.0).float()

    inside = ((a @ b.transpose(-1, -2)) * power(i[:, None] - i)[:, None]) @ c
    kv = (b * power(chunk - 1 - i[None])[:, 0, :, None][:, None]).transpose(-1, -2) @ c
    before = power(chunk * (m[:, None] - 1 - m)) @ kv.reshape(B, H, n, d * d)   # state at each chunk's start
    across = (a * power(i[None] + 1)[:, 0, :, None][:, None]) @ before.view(B, H, n, d, d)
    return (inside + across).reshape(B, H, n * chunk, d)[:, :, :T]


def _lattn_setup(s):
    """Head layouts with the rows past each length zeroed, and g^(t + 1), g^(len - 1 - t), g^len."""
    c = s["case"]
    T = c["T"]
    lg = s["decay"].cuda().double().log()
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((c["B"],), T, device="cuda")
    t = torch.arange(T, device="cuda")
    live = (t < n[:, None])[:, None, :, None]
    fore = torch.exp(lg[:, None] * (t + 1))[None, :, :, None].float()
    back = torch.exp(lg[None, :, None] * (n[:, None, None] - 1 - t).clamp_min(0))[..., None].float()
    whole = torch.exp(lg * n[:, None])[..., None, None].float()
    return lg, live, fore, back, whole


def _plain_lattn_fwd(s):
    d = s["case"]["d"]
    lg, live, fore, back, whole = _lattn_setup(s)
    q, k, v = (_heads(s[n], d) * live for n in "qkv")
    o = _decayed(q, k, v, lg)
    if s["state_in"] is not None:
        o = o + (q * fore) @ s["state_in"]
    out = {"o": _rows(o * live)}
    if s["state_out"] is not None:
        out["state_out"] = (k * back).transpose(-1, -2) @ v
        if s["state_in"] is not None:
            out["state_out"] = out["state_out"] + whole * s["state_in"]
    return out


def _plain_lattn_bwd(s):
    d = s["case"]["d"]
    lg, live, fore, back, whole = _lattn_setup(s)
    q, k, v, do = (_heads(s[n], d) * live for n in ("q", "k", "v", "do"))
    dq = _decayed(do, v, k, lg)
    dk = _decayed(v.flip(2), do.flip(2), q.flip(2), lg).flip(2)
    dv = _decayed(k.flip(2), q.flip(2), do.flip(2), lg).flip(2)
    if s["state_in"] is not None:
        dq = dq + (do * fore) @ s["state_in"].transpose(-1, -2)
    if s["dstate_out"] is not None:
        dk = dk + (v * back) @ s["dstate_out"].transpose(-1, -2)
        dv = dv + (k * back) @ s["dstate_out"]
    out = {"dq": _rows(dq * live), "dk": _rows(dk * live), "dv": _rows(dv * live)}
    if s["dstate_in"] is not None:
        out["dstate_in"] = (q * fore).transpose(-1, -2) @ do
        if s["dstate_out"] is not None:
            out["dstate_in"] = out["dstate_in"] + whole * s["dstate_out"]
    return out


_PLAIN = {"ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd, "ffn_fwd": _plain_ffn_fwd, "ffn_bwd": _plain_ffn_bwd,
          "lattn_step": _plain_lattn_step, "lattn_fwd": _plain_lattn_fwd, "lattn_bwd": _plain_lattn_bwd}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        M, D, e = case["rows"], case["dim"], 2 if case["dtype"] == BF16 else 4
        if op == "ln_fwd":
            return {"bytes": 2 * M * D * e + 8 * M + 8 * D, "flops": 8 * M * D}
        return {"bytes": (4 if case["dres"] else 3) * M * D * e + 8 * M + 12 * D, "flops": 14 * M * D}
    if op == "ffn_fwd":
        M, D, F = case["rows"], case["dim"], case["hidden"]
        rows = 2 + (1 if case["res"] else 0)
        return {"bytes": 2 * (3 * D * F + rows * M * D + (2 * M * F if case["save"] else 0)), "flops": 6 * M * D * F}
    if op == "ffn_bwd":
        M, D, F = case["rows"], case["dim"], case["hidden"]
        return {"bytes": 2 * (6 * D * F + 3 * M * D + 2 * M * F), "flops": 12 * M * D * F}
    B, H, d = case["B"], case["heads"], case["d"]
    if op == "lattn_step":
        return {"bytes": B * H * (8 * d * d + 8 * d), "flops": 5 * B * H * d * d}
    n = B * case["T"] * H * d
    state = B * H * d * d * 4 if case["state"] else 0
    if op == "lattn_fwd":
        return {"bytes": 8 * n + 2 * state, "flops": 4 * n * d}
    return {"bytes": 14 * n + 3 * state, "flops": 10 * n * d}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    f = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point() and v.is_cuda}
    op = case["op"]
    if op == "ln_fwd":
        var, mean = torch.var_mean(f["x"], 1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        return {"y": torch.addcmul(f["beta"], (f["x"] - mean[:, None]) * rstd[:, None], f["gamma"]), "mean": mean,
                "rstd": rstd}
    if op == "ln_bwd":
        # the Jacobian of a row applied to its cotangent: (I - 1 1^T / D - xhat xhat^T / D) / sigma
        D = case["dim"]
        xhat = torch.addcmul(-f["mean"][:, None] * f["rstd"][:, None], f["x"], f["rstd"][:, None])
        w = f["dy"] * f["gamma"]
        proj = (w.sum(1, keepdim=True) + xhat * torch.einsum("md,md->m", w, xhat)[:, None]) / D
        dx = f["rstd"][:, None] * (w - proj)
        return {"dx": dx if s["dres"] is None else dx + f["dres"], "dgamma": torch.einsum("md,md->d", f["dy"], xhat),
                "dbeta": torch.einsum("md->d", f["dy"])}
    if op == "ffn_fwd":
        gate, up = torch.einsum("md,fd->mf", f["x"], f["W_gate"]), torch.einsum("md,fd->mf", f["x"], f["W_up"])
        act = gate / (1 + torch.exp(-gate)) if case["act"] == "silu" else gate * 0.5 * torch.erfc(-gate / math.sqrt(2))
        y = torch.einsum("mf,df->md", act * up, f["W_down"])
        y = y if s["res"] is None else y + f["res"]
        return {"y": y, "gate": gate, "up": up} if case["save"] else {"y": y}
    if op == "ffn_bwd":
        gate, up = f["gate"], f["up"]
        if case["act"] == "silu":
            p = 1 / (1 + torch.exp(-gate))
            slope = p + gate * p * (1 - p)
        else:
            p = 0.5 * torch.erfc(-gate / math.sqrt(2))
            slope = p + gate * torch.exp(-gate * gate / 2) / math.sqrt(2 * math.pi)
        dh = torch.einsum("md,df->mf", f["dy"], f["W_down"])
        dgate, dup = dh * up * slope, dh * gate * p
        return {"dx": torch.einsum("mf,fd->md", dgate, f["W_gate"]) + torch.einsum("mf,fd->md", dup, f["W_up"]),
                "grads": {"W_gate": torch.einsum("mf,md->fd", dgate, f["x"]),
                          "W_up": torch.einsum("mf,md->fd", dup, f["x"]),
                          "W_down": torch.einsum("md,mf->df", f["dy"], gate * p * up)}}
    B, H, d = case["B"], case["heads"], case["d"]
    g = s["decay"].double().cuda()[:, None, None]
    if op == "lattn_step":
        q, k, v = (f[n].view(B, H, d) for n in "qkv")
        state = g * f["state"] + torch.einsum("bhi,bhj->bhij", k, v)
        return {"o": torch.einsum("bhi,bhij->bhj", q, state).reshape(B, H * d), "state": state}
    # the recurrence itself, token by token
    T = case["T"]
    n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    if T * B * H * d * d > 1 << 36:   # minutes of 64-bit state traffic
        return None
    end = torch.tensor(n, device="cuda")[:, None, None, None]

    def tokens(name):
        return f[name].reshape(B, T, H, d).transpose(0, 1).contiguous()

    q, k, v = tokens("q"), tokens("k"), tokens("v")
    zero = torch.zeros(B, H, d, d, device="cuda", dtype=torch.float64)
    S = f["state_in"].clone() if s["state_in"] is not None else zero
    if op == "lattn_fwd":
        o = torch.zeros(T, B, H, d, device="cuda", dtype=torch.float64)
        for t in range(T):
            S = torch.where(end > t, torch.addcmul(g * S, k[t][..., :, None], v[t][..., None, :]), S)
            o[t] = torch.where(end[..., 0] > t, torch.matmul(q[t][..., None, :], S)[..., 0, :], 0.0)
        out = {"o": o.transpose(0, 1).reshape(B, T, H * d)}
        if case["state"]:
            out["state_out"] = S
        return out
    do = tokens("do")
    dq, dk, dv = (torch.zeros(T, B, H, d, device="cuda", dtype=torch.float64) for _ in range(3))
    for t in range(T):
        S = torch.where(end > t, torch.addcmul(g * S, k[t][..., :, None], v[t][..., None, :]), S)
        dq[t] = torch.where(end[..., 0] > t, torch.matmul(S, do[t][..., :, None])[..., 0], 0.0)
    R = f["dstate_out"].clone() if s["dstate_out"] is not None else zero   # dL/dS_t carried back
    for t in range(T - 1, -1, -1):
        A = torch.addcmul(R, q[t][..., :, None], do[t][..., None, :])
        dk[t] = torch.where(end[..., 0] > t, torch.matmul(A, v[t][..., :, None])[..., 0], 0.0)
        dv[t] = torch.where(end[..., 0] > t, torch.matmul(k[t][..., None, :], A)[..., 0, :], 0.0)
        R = torch.where(end > t, g * A, R)
    out = {m: x.transpose(0, 1).reshape(B, T, H * d) for m, x in (("dq", dq), ("dk", dk), ("dv", dv))}
    if case["state"]:
        out["dstate_in"] = R
    return out
