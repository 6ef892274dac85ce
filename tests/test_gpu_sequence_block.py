"""A pre-norm residual block of a sequence model, run with the operators together:

    n1 = LN(x), o = mixer(n1), x1 = x + o, n2 = LN(x1), y = FFN(n2) + x1

with linear attention or the SRNL sequence layer as the mixer; forward and backward, a prompt
followed by single tokens, and both captured into graphs.

Tolerance with linear attention.  The block is evaluated in 64 bits twice, once as it is defined
and once with every tensor that passes from one operator to the next, or is rounded inside one,
rounded to bf16 in both directions.  The norm of their difference is what those roundings
amount to.  The kernels round at the same points and at one more, the masked products of q and
k, which weighs no more than the rounding of o; two sums of independent roundings of which one
has at most as many again differ in norm by a factor of sqrt(2).  2 is allowed.
"""
import numpy as np
import pytest
import torch

import self_referential_nested_b200 as S
from srnl_inputs import make_seq_inputs

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_referential_nested_b200 import build
    build.build()
    torch.cuda.set_device(0)


class Rounded(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, on):
        ctx.on = on
        return x.to(BF).double() if on else x.clone()

    @staticmethod
    def backward(ctx, g):
        return (g.to(BF).double() if ctx.on else g), None


def make(B, T, H, d, hidden, seed=0):
    g = torch.Generator().manual_seed(seed)
    D = H * d

    def n(*s, scale=1.0, dt=BF):
        return (torch.randn(*s, generator=g) * scale).to(dt).cuda()

    return {"x": n(B, T, D), "dy": n(B, T, D), "W_qkv": n(3 * D, D, scale=D ** -0.5),
            "W_gate": n(hidden, D, scale=D ** -0.5), "W_up": n(hidden, D, scale=D ** -0.5),
            "W_down": n(D, hidden, scale=hidden ** -0.5),
            "g1": 1 + n(D, scale=0.1, dt=torch.float32), "b1": n(D, scale=0.1, dt=torch.float32),
            "g2": 1 + n(D, scale=0.1, dt=torch.float32), "b2": n(D, scale=0.1, dt=torch.float32),
            "decay": np.array([1 - 2.0 ** -(2 + i) for i in range(H)], dtype=np.float32)}


def block64(t, H, d, rounded):
    """y and the gradients of every leaf, in 64 bits."""
    leaves = {k: t[k].double().requires_grad_() for k in ("x", "W_qkv", "W_gate", "W_up", "W_down", "g1", "b1", "g2", "b2")}
    L = leaves
    D = H * d

    def r(v):
        return Rounded.apply(v, rounded)

    def norm(x, g, b):
        c = x - x.mean(-1, keepdim=True)
        return c / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS) * g + b

    B, T, _ = t["x"].shape
    qkv = r(r(norm(L["x"], L["g1"], L["b1"])) @ L["W_qkv"].t())
    q, k, v = (qkv[..., i * D:(i + 1) * D].view(B, T, H, d).transpose(1, 2) for i in range(3))
    i = torch.arange(T, device="cuda")
    e = (i[:, None] - i).double()
    lg = torch.tensor(t["decay"], device="cuda", dtype=torch.float64).log()[:, None, None]
    w = torch.where(e >= 0, torch.exp(lg * e.clamp_min(0)), 0.0)
    o = r((((q @ k.transpose(-1, -2)) * w) @ v).transpose(1, 2).reshape(B, T, D))
    x1 = r(L["x"] + o)
    n2 = r(norm(x1, L["g2"], L["b2"]))
    gate, up = r(n2 @ L["W_gate"].t()), r(n2 @ L["W_up"].t())
    y = r(r(torch.nn.functional.silu(gate) * up) @ L["W_down"].t() + x1)
    y.backward(t["dy"].double())
    return {"y": y.detach(), **{"d" + k: p.grad for k, p in leaves.items()}}


def round_out(name, v):
    return v.to(BF).double() if name not in ("dg1", "db1", "dg2", "db2") else v


class Block:
    """The block with its handles and buffers, as a user's program would keep them."""

    def __init__(self, t, B, T, H, d, hidden, training):
        D = H * d
        self.t, self.D, self.training = t, D, training
        self.ln = S.srnl_ln_create(dict(dim=D, eps=EPS, act_dtype="bf16"))
        self.la = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d, ld=3 * D), t["decay"])
        self.ff = S.srnl_ffn_create(dict(dim=D, hidden=hidden, max_rows=B * T, training=training))
        new = lambda *s, dt=BF: torch.empty(*s, device="cuda", dtype=dt)
        self.n1, self.o, self.x1, self.n2, self.y = (new(B, T, D) for _ in range(5))
        self.qkv = new(B, T, 3 * D)
        self.state = new(B, H, d, d, dt=torch.float32)
        if training:
            self.stat = [new(B * T, dt=torch.float32) for _ in range(4)]
            self.gate, self.up = new(B * T, hidden), new(B * T, hidden)
            self.dn, self.dx1, self.dx = (new(B, T, D) for _ in range(3))
            self.dqkv = new(B, T, 3 * D)
            self.dW = {k: torch.empty_like(t[k]) for k in S.FFN_KEYS}
            self.dW_qkv = torch.empty_like(t["W_qkv"])
            self.dgb = {k: torch.empty_like(t[k]) for k in ("g1", "b1", "g2", "b2")}

    def close(self):
        for h in (self.ln, self.la, self.ff):
            h.close()

    def parts(self, qkv):
        return (qkv[..., i * self.D:(i + 1) * self.D] for i in range(3))

    def forward(self, x):
        t = self.t
        m = self.stat if self.training else [None] * 4
        S.srnl_ln_forward(self.ln, x, t["g1"], t["b1"], self.n1, m[0], m[1])
        torch.matmul(self.n1, t["W_qkv"].t(), out=self.qkv)
        S.srnl_lattn_forward(self.la, *self.parts(self.qkv), self.o, state_out=self.state)
        torch.add(x, self.o, out=self.x1)
        S.srnl_ln_forward(self.ln, self.x1, t["g2"], t["b2"], self.n2, m[2], m[3])
        S.srnl_ffn_forward(self.ff, self.n2, t, self.y, res=self.x1, gate=self.gate if self.training else None,
                           up=self.up if self.training else None)
        return self.y

    def backward(self, x, dy):
        t, g = self.t, self.dgb
        S.srnl_ffn_backward(self.ff, self.n2, self.gate, self.up, dy, t, self.dn, self.dW)
        S.srnl_ln_backward(self.ln, self.x1, self.dn, t["g2"], self.stat[2], self.stat[3], self.dx1, g["g2"], g["b2"], dres=dy)
        S.srnl_lattn_backward(self.la, *self.parts(self.qkv), self.dx1, *self.parts(self.dqkv))
        torch.matmul(self.dqkv, t["W_qkv"], out=self.dn)
        torch.matmul(self.dqkv.flatten(0, 1).t(), self.n1.flatten(0, 1), out=self.dW_qkv)
        S.srnl_ln_backward(self.ln, x, self.dn, t["g1"], self.stat[0], self.stat[1], self.dx, g["g1"], g["b1"], dres=self.dx1)

    def step(self, x, y):
        """One token of each sequence, [B, 1, D]: the buffers' first rows serve."""
        t = self.t
        S.srnl_ln_forward(self.ln, x, t["g1"], t["b1"], self.n1)
        torch.matmul(self.n1, t["W_qkv"].t(), out=self.qkv)
        q, k, v = (p[:, 0] for p in self.parts(self.qkv))
        S.srnl_lattn_step(self.la, q, k, v, self.o, self.state)
        torch.add(x, self.o, out=self.x1)
        S.srnl_ln_forward(self.ln, self.x1, t["g2"], t["b2"], self.n2)
        S.srnl_ffn_forward(self.ff, self.n2, t, y, res=self.x1)

    def results(self):
        return {"y": self.y, "dx": self.dx, "dW_qkv": self.dW_qkv, **{"d" + k: v for k, v in self.dW.items()},
                **{"d" + k: v for k, v in self.dgb.items()}}


def within(name, got, exact, rounded):
    assert bool(torch.isfinite(got).all()), name
    err, room = float((got.double() - exact).norm()), float((round_out(name, rounded) - exact).norm())
    assert err <= 2 * room, (name, err, room)


SHAPES = [(6, 1, 4, 32, 40), (2, 37, 3, 64, 520), (3, 130, 2, 128, 648), (2, 700, 4, 32, 264)]


@pytest.mark.parametrize("B,T,H,d,hidden", SHAPES)
def test_forward_and_backward(B, T, H, d, hidden):
    t = make(B, T, H, d, hidden, seed=T)
    b = Block(t, B, T, H, d, hidden, True)
    try:
        b.forward(t["x"])
        b.backward(t["x"], t["dy"])
        torch.cuda.synchronize()
        S.srnl_lattn_device_status(b.la)
        S.srnl_ffn_device_status(b.ff)
        exact, rounded = block64(t, H, d, False), block64(t, H, d, True)
        for name, got in b.results().items():
            within(name, got, exact[name], rounded[name])
    finally:
        b.close()


@pytest.mark.parametrize("B,P,N,H,d,hidden", [(5, 1, 3, 4, 32, 40), (5, 150, 6, 2, 64, 520), (40, 20, 4, 2, 128, 264)])
def test_a_prompt_then_tokens(B, P, N, H, d, hidden):
    t = make(B, P + N, H, d, hidden, seed=B)
    prompt, token = Block(t, B, P, H, d, hidden, False), Block(t, B, 1, H, d, hidden, False)
    try:
        ys = [prompt.forward(t["x"][:, :P].contiguous()).clone()]
        token.state.copy_(prompt.state)
        y = torch.empty(B, 1, H * d, device="cuda", dtype=BF)
        for i in range(P, P + N):
            token.step(t["x"][:, i:i + 1].contiguous(), y)
            ys.append(y.clone())
        got = torch.cat(ys, 1)
        exact, rounded = block64(t, H, d, False)["y"], block64(t, H, d, True)["y"]
        within("y", got[:, :P], exact[:, :P], rounded[:, :P])
        within("y", got[:, P:], exact[:, P:], rounded[:, P:])
    finally:
        prompt.close()
        token.close()


def test_graphs_give_equal_bits():
    """A training step and a token's step captured, replayed on new inputs, while the eager runs go
    on in between on buffers of their own."""
    B, T, H, d, hidden = 2, 300, 2, 64, 520
    t = make(B, T, H, d, hidden, seed=1)
    eager, kept = Block(t, B, T, H, d, hidden, True), Block(t, B, T, H, d, hidden, True)
    tok_e, tok_g = Block(t, B, 1, H, d, hidden, False), Block(t, B, 1, H, d, hidden, False)
    train = token = None
    try:
        x, dy = t["x"].clone(), t["dy"].clone()
        x1 = t["x"][:, :1].contiguous()
        ye, yg = torch.empty_like(x1), torch.empty_like(x1)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):   # the library products' first calls are not captured
            kept.forward(x)
            kept.backward(x, dy)
            tok_g.state.zero_()
            tok_g.step(x1, yg)
        side.synchronize()
        train, token = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(train):
            kept.forward(x)
            kept.backward(x, dy)
        with torch.cuda.graph(token):
            tok_g.step(x1, yg)
        tok_e.state.zero_()
        tok_g.state.zero_()
        for seed in (3, 4):
            new = make(B, T, H, d, hidden, seed=seed)
            x.copy_(new["x"])
            dy.copy_(new["dy"])
            x1.copy_(new["x"][:, 5:6])
            train.replay()
            eager.forward(new["x"])
            eager.backward(new["x"], new["dy"])
            token.replay()
            tok_e.step(x1, ye)
            torch.cuda.synchronize()
            for (n, a), c in zip(kept.results().items(), eager.results().values()):
                assert torch.equal(a, c), n
            assert torch.equal(ye, yg) and torch.equal(tok_e.state, tok_g.state)
    finally:
        del train, token
        for b in (eager, kept, tok_e, tok_g):
            b.close()


def test_around_the_sequence_layer():
    """The SRNL sequence layer as the mixer: its own results are compared elsewhere; here what
    surrounds it, forward and backward, given what it returned.  Each operator's output is one
    rounding (2^-8 of the value) from its formula in 64 bits, but for fp32 sums, for which the same
    again is allowed."""
    inp = make_seq_inputs(2, 257, 64, 2, "bf16", seed=3)
    B, T, D, hidden = inp.B, inp.T, inp.D, 2 * inp.D
    t = make(B, T, inp.heads, D // inp.heads, hidden, seed=2)
    x = torch.from_numpy(inp.x_bits.view(np.int16)).cuda().view(BF)
    seq = S.srnl_seq_create(dict(B=B, T=T, D=D, heads=inp.heads, d=32, alpha=0.95, eps=1e-6, chunk=64, act_dtype="bf16",
                                 gen_dtype="f32"), inp.params())
    ln = S.srnl_ln_create(dict(dim=D, eps=EPS, act_dtype="bf16"))
    ff = S.srnl_ffn_create(dict(dim=D, hidden=hidden, max_rows=B * T, training=True))
    try:
        new = lambda *s, dt=BF: torch.empty(*s, device="cuda", dtype=dt)
        n1, o, n2, y, dn, dx1, dn1, dx = (new(B, T, D) for _ in range(8))
        m1, r1, m2, r2 = (new(B * T, dt=torch.float32) for _ in range(4))
        gate, up = new(B * T, hidden), new(B * T, hidden)
        S.srnl_ln_forward(ln, x, t["g1"], t["b1"], n1, m1, r1)
        S.srnl_seq_forward(seq, n1, o)
        x1 = x + o
        S.srnl_ln_forward(ln, x1, t["g2"], t["b2"], n2, m2, r2)
        S.srnl_ffn_forward(ff, n2, t, y, res=x1, gate=gate, up=up)
        dy = t["dy"]
        S.srnl_ffn_backward(ff, n2, gate, up, dy, t, dn)
        S.srnl_ln_backward(ln, x1, dn, t["g2"], m2, r2, dx1, dres=dy)
        S.srnl_seq_backward(seq, n1, dx1, dn1)
        S.srnl_ln_backward(ln, x, dn1, t["g1"], m1, r1, dx, dres=dx1)
        torch.cuda.synchronize()
        S.srnl_seq_device_status(seq)

        def norm64(v, g, b, up=None, res=None):
            v = v.double().requires_grad_()
            c = v - v.mean(-1, keepdim=True)
            out = c / torch.sqrt((c * c).mean(-1, keepdim=True) + EPS) * g.double() + b.double()
            if up is None:
                return out.detach()
            out.backward(up.double())
            return v.grad + res.double()

        for name, got, ref in (("n1", n1, norm64(x, t["g1"], t["b1"])), ("n2", n2, norm64(x1, t["g2"], t["b2"])),
                               ("dx1", dx1, norm64(x1, t["g2"], t["b2"], dn, dy)), ("dx", dx, norm64(x, t["g1"], t["b1"], dn1, dx1))):
            assert float((got.double() - ref).abs().max()) <= 2 * 2.0 ** -8 * float(ref.abs().max()), name
            assert float((got.double() - ref).norm()) <= 2.0 ** -8 * float(ref.norm()), name
        assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(dn1).all())
    finally:
        for h in (seq, ln, ff):
            h.close()


def test_around_the_sequence_layer_value_by_value():
    """The same chain: the feed-forward branch's pre-activations, output and gradients against its formulas in 64 bits, given
    what the norms returned, to the branch's own tolerances; the sequence layer's output and gradient against its
    oracle, to the bars of its own tests for bf16 outputs (1e-2 of the norm)."""
    from oracle import srnl_grad as GR
    from oracle import srnl_oracle as O
    from test_gpu_ffn import act64
    from test_gpu_ffn import within as ffn_within

    inp = make_seq_inputs(2, 150, 64, 2, "bf16", seed=5)
    B, T, D, hidden = inp.B, inp.T, inp.D, 3 * inp.D
    t = make(B, T, inp.heads, D // inp.heads, hidden, seed=6)
    x = torch.from_numpy(inp.x_bits.view(np.int16)).cuda().view(BF)
    params = inp.params()
    seq = S.srnl_seq_create(dict(B=B, T=T, D=D, heads=inp.heads, d=32, alpha=0.95, eps=1e-6, chunk=64, act_dtype="bf16",
                                 gen_dtype="f32"), params)
    ln = S.srnl_ln_create(dict(dim=D, eps=EPS, act_dtype="bf16"))
    ff = S.srnl_ffn_create(dict(dim=D, hidden=hidden, max_rows=B * T, training=True))
    try:
        new = lambda *s, dt=BF: torch.empty(*s, device="cuda", dtype=dt)
        n1, o, n2, y, dn, dx1, dn1 = (new(B, T, D) for _ in range(7))
        m2, r2 = (new(B * T, dt=torch.float32) for _ in range(2))
        gate, up, dW = new(B * T, hidden), new(B * T, hidden), {k: torch.empty_like(t[k]) for k in S.FFN_KEYS}
        S.srnl_ln_forward(ln, x, t["g1"], t["b1"], n1)
        S.srnl_seq_forward(seq, n1, o)
        x1 = x + o
        S.srnl_ln_forward(ln, x1, t["g2"], t["b2"], n2, m2, r2)
        S.srnl_ffn_forward(ff, n2, t, y, res=x1, gate=gate, up=up)
        S.srnl_ffn_backward(ff, n2, gate, up, t["dy"], t, dn, dW)
        S.srnl_ln_backward(ln, x1, dn, t["g2"], m2, r2, dx1, dres=t["dy"])
        S.srnl_seq_backward(seq, n1, dx1, dn1)
        torch.cuda.synchronize()
        S.srnl_seq_device_status(seq)
        S.srnl_ffn_device_status(ff)
    finally:
        for h in (seq, ln, ff):
            h.close()
    rows = lambda v: v.reshape(B * T, -1).double()
    v, dy, (Wg, Wu, Wd) = rows(n2), rows(t["dy"]), (t[k].double() for k in S.FFN_KEYS)
    zero = torch.zeros((), device="cuda", dtype=torch.float64)
    g64, u64 = v @ Wg.t(), v @ Wu.t()
    ffn_within(gate, g64, v.abs() @ Wg.abs().t(), zero, D)
    ffn_within(up, u64, v.abs() @ Wu.abs().t(), zero, D)
    hid = act64(g64, "silu")[0] * u64
    ffn_within(rows(y), hid @ Wd.t() + rows(x1), hid.abs() @ Wd.abs().t(), (hid ** 2) @ (Wd ** 2).t(), hidden)
    g, u = gate.double(), up.double()
    a, da = act64(g, "silu")
    dh = dy @ Wd
    dg, du, hid = dh * u * da, dh * a, a * u
    ffn_within(rows(dn), dg @ Wg + du @ Wu, dg.abs() @ Wg.abs() + du.abs() @ Wu.abs(), (dg ** 2) @ (Wg ** 2) + (du ** 2) @ (Wu ** 2),
               2 * hidden + D)
    ffn_within(dW["W_gate"], dg.t() @ v, dg.abs().t() @ v.abs(), (dg ** 2).t() @ (v ** 2), B * T + D)
    ffn_within(dW["W_up"], du.t() @ v, du.abs().t() @ v.abs(), (du ** 2).t() @ (v ** 2), B * T + D)
    ffn_within(dW["W_down"], dy.t() @ hid, dy.abs().t() @ hid.abs(), (dy ** 2).t() @ (hid ** 2), B * T)
    host = lambda v: v.float().cpu().numpy()
    ref = O.sequence_forward(host(n1), params, alpha_max=0.95, chunk=64, heads=inp.heads)
    ref = ref[0] if isinstance(ref, tuple) else ref
    assert O.rel_fro(host(o), ref) <= 1e-2
    ref = GR.sequence_backward(host(n1), params, host(dx1), alpha_max=0.95, chunk=64, heads=inp.heads)
    assert O.rel_fro(host(dn1), ref["x"]) <= 1e-2
