"""Linear attention with a decay for each head (srnl_lattn_*): prompts, gradients and single
tokens against the definition in 64 bits, written out as a sum over all pairs of tokens.

Tolerances.  half = 2^-8 bounds a bf16 rounding relative to the value.  An output is rounded
once.  The masked a b^T of a chunk (at most the 127 tokens before and the token itself) is
rounded: errors of zero mean and a standard deviation of at most half / sqrt(3) each, seven
standard deviations of their sum.  The state as an operand and the rows of its update are split
into two bf16 parts: 2^-16 of the magnitude each; fp32 sums and powers are counted as another
half of that pair.  States are fp32: the split of the update's rows and the fp32 sums alone.
"""
import math

import numpy as np
import pytest
import torch

import self_referential_nested_b200 as S

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_referential_nested_b200 import build
    build.build()
    torch.cuda.set_device(0)


def make(B, T, H, d, seed=0, packed=False):
    g = torch.Generator().manual_seed(seed)
    D = H * d
    x = torch.randn(B, T, 4, D, generator=g)
    x[:, :, 0] *= d ** -0.5
    x = x.to(BF).cuda()
    t = {n: (x[:, :, i] if packed and n != "do" else x[:, :, i].contiguous()) for i, n in enumerate(("q", "k", "v", "do"))}
    t["s0"] = torch.randn(B, H, d, d, generator=g).cuda()
    t["ds"] = torch.randn(B, H, d, d, generator=g).cuda()
    t["ld"] = 4 * D if packed else 0
    return t


def heads(x, d):
    B, T, D = x.shape
    return x.double().view(B, T, D // d, d).transpose(1, 2)


def pair_sum(a, b, c, w, near):
    """sum_j w_tj (a_t . b_j) c_j, its magnitude, and the spread of the rounded near pairs."""
    p = (a @ b.transpose(-1, -2)) * w
    return p @ c, ((a.abs() @ b.abs().transpose(-1, -2)) * w) @ c.abs(), ((p * near) ** 2) @ (c ** 2)


def reference(t, decay, lens, with_s0, with_ds):
    """{name: (value, magnitude, spread)} of o, dq, dk, dv and the states."""
    d = t["s0"].shape[-1]
    q, k, v, do = (heads(t[n], d) for n in ("q", "k", "v", "do"))
    B, H, T, _ = q.shape
    lg = torch.tensor(decay, device="cuda", dtype=torch.float64).log()
    n = torch.tensor(lens, device="cuda")
    i = torch.arange(T, device="cuda")
    live = (i < n[:, None])[:, None, :, None].double()
    q, k, v, do = (x * live for x in (q, k, v, do))
    e = (i[:, None] - i).double()
    w = torch.where(e >= 0, torch.exp(lg[:, None, None] * e.clamp_min(0)), 0.0)[None]
    near = ((e >= 0) & (e < 128)).double()
    s0 = t["s0"].double() * with_s0
    ds = t["ds"].double() * with_ds
    fore = torch.exp(lg[None, :, None] * (i + 1.0))[..., None]
    back = torch.exp(lg[None, :, None] * (n[:, None, None] - 1 - i).clamp_min(0).double())[..., None]
    whole = torch.exp(lg * n[:, None])[..., None, None]
    wt, nt = w.transpose(-1, -2), near.t()

    def plus(x, a, f, z):
        return x[0] + (a * f) @ z, x[1] + (a.abs() * f) @ z.abs(), x[2]

    out = {"o": plus(pair_sum(q, k, v, w, near), q, fore, s0),
           "dq": plus(pair_sum(do, v, k, w, near), do, fore, s0.transpose(-1, -2)),
           "dk": plus(pair_sum(v, do, q, wt, nt), v, back, ds.transpose(-1, -2)),
           "dv": plus(pair_sum(k, q, do, wt, nt), k, back, ds)}
    out = {m: tuple((y * live).transpose(1, 2).reshape(B, T, H * d) for y in x) for m, x in out.items()}
    st = (k * back).transpose(-1, -2), (q * fore).transpose(-1, -2)
    out["state"] = st[0] @ v + whole * s0, st[0].abs() @ v.abs() + whole * s0.abs()
    out["dstate"] = st[1] @ do + whole * ds, st[1].abs() @ do.abs() + whole * ds.abs()
    return out


def within(got, ref, magnitude, spread=None):
    assert bool(torch.isfinite(got).all())
    tol = 1.5 * 2.0 ** -16 * magnitude if spread is None else \
        HALF * ref.abs() + 7 * HALF / math.sqrt(3) * spread.sqrt() + 1.5 * 2.0 ** -15 * magnitude
    worst = ((got.double() - ref).abs() / (tol + 1e-30)).max()
    assert float(worst) <= 1, float(worst)


CASES = [  # B, T, heads, d, lengths, packed
    (1, 1, 1, 32, None, False), (2, 5, 3, 64, None, True), (1, 7, 2, 128, None, False),
    (3, 64, 2, 32, [64, 0, 1], False), (3, 65, 2, 64, [65, 63, 64], True), (2, 128, 1, 128, None, True),
    (3, 129, 2, 128, [129, 0, 128], False), (2, 300, 5, 64, [300, 299], False), (4, 333, 3, 32, [1, 333, 200, 64], True),
    (1, 2100, 2, 64, None, False), (2, 1500, 1, 128, [1500, 700], False), (2, 1200, 2, 32, [900, 1200], True),
    (40, 70, 4, 64, None, False),
    # a few tokens, on both sides of what the kernel for them takes
    (2, 16, 2, 128, [16, 3], False), (3, 12, 3, 32, None, True), (2, 17, 2, 64, [17, 0], True), (4, 16, 1, 64, None, False),
    (3, 8, 2, 32, [8, 0, 3], True), (2, 9, 3, 64, [9, 1], False), (2, 31, 1, 128, [31, 8], True), (5, 32, 3, 32, None, False),
    (3, 32, 2, 128, [32, 17, 0], False), (2, 33, 2, 64, [33, 32], False),
    # more CTAs than run at once, lengths in no order, several equal: the longest go first
    (60, 260, 3, 64, [(97 * i) % 261 for i in range(30)] * 2, False), (50, 200, 3, 128, [200 - (i * i) % 190 for i in range(50)], False),
]


@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("B,T,H,d,lens,packed", CASES)
def test_forward_and_backward(B, T, H, d, lens, packed, state):
    t = make(B, T, H, d, seed=T + d, packed=packed)
    decay = np.array([[1.0, 0.5, 0.97, 0.999, 1e-6][i % 5] for i in range(H)], dtype=np.float32)
    n = torch.tensor(lens, device="cuda", dtype=torch.int32) if lens else None
    D = H * d
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d, ld=t["ld"]), decay)
    try:
        o = torch.full((B, T, D), 7.0, device="cuda", dtype=BF)
        so, dsi = torch.full_like(t["s0"], 7.0), torch.full_like(t["s0"], 7.0)
        S.srnl_lattn_forward(h, t["q"], t["k"], t["v"], o, lengths=n, state_in=t["s0"] if state else None,
                             state_out=so if state else None)
        g = torch.full((B, T, 4, D), 7.0, device="cuda", dtype=BF)
        dq, dk, dv = ((g[:, :, i] if packed else torch.full((B, T, D), 7.0, device="cuda", dtype=BF)) for i in range(3))
        S.srnl_lattn_backward(h, t["q"], t["k"], t["v"], t["do"], dq, dk, dv, lengths=n,
                              state_in=t["s0"] if state else None, dstate_out=t["ds"] if state else None,
                              dstate_in=dsi if state else None)
        torch.cuda.synchronize()
        S.srnl_lattn_device_status(h)
    finally:
        h.close()
    ln = lens or [T] * B
    ref = reference(t, decay, ln, state, state)
    for name, got in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        for b in range(B):
            assert bool((got[b, ln[b]:] == 7).all()), name   # rows behind a sequence stay
            if ln[b]:
                within(got[b, :ln[b]], *(x[b, :ln[b]] for x in ref[name]))
    if packed:
        assert bool((g[:, :, 3] == 7).all())
    if state:
        within(so, *ref["state"])
        within(dsi, *ref["dstate"])


@pytest.mark.parametrize("d", [32, 64, 128])
def test_gradients_against_differences(d):
    """The loss is bilinear in each input, so a difference over a step of one is its gradient."""
    B, T, H = 2, 150, 2
    t = make(B, T, H, d, seed=1)
    decay = np.array([0.9, 0.995], dtype=np.float32)
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), decay)
    try:
        g = {n: torch.empty_like(t["q"]) for n in "qkv"}
        g["s0"] = torch.empty_like(t["s0"])
        S.srnl_lattn_backward(h, t["q"], t["k"], t["v"], t["do"], g["q"], g["k"], g["v"], state_in=t["s0"],
                              dstate_out=t["ds"], dstate_in=g["s0"])
        torch.cuda.synchronize()
    finally:
        h.close()
    gen = torch.Generator().manual_seed(7)
    for name, grad in g.items():
        v = torch.randn(grad.shape, generator=gen).cuda().double()

        def loss(s):
            u = dict(t)
            u[name] = t[name].double() + s * v
            r = reference(u, decay, [T] * B, True, True)
            return float((r["o"][0] * t["do"].double()).sum() + (r["state"][0] * t["ds"].double()).sum())

        num = loss(0.5) - loss(-0.5)
        # n independent roundings, two a value (its own, and its pairs'): seven standard deviations
        rms = float((grad.double() * v).square().sum().sqrt())
        rel = 7 * HALF / math.sqrt(3) * math.sqrt(2) if grad.dtype is BF else 7 * 1.5 * 2.0 ** -16
        assert abs(num - float((grad.double() * v).sum())) <= rel * rms + 2.0 ** -15 * float((grad.double() * v).abs().sum())


@pytest.mark.parametrize("B,H,d", [(1, 1, 32), (3, 2, 64), (2, 3, 128), (70, 4, 64)])
def test_a_prompt_then_tokens(B, H, d):
    """A prompt's state carried on token by token gives the longer prompt's outputs and state."""
    T, more = 90, 5
    t = make(B, T + more, H, d, seed=d)
    decay = np.linspace(0.8, 1.0, H).astype(np.float32)
    cut = {n: t[n][:, :T].contiguous() for n in "qkv"}
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), decay)
    try:
        o, st = torch.empty(B, T, H * d, device="cuda", dtype=BF), torch.empty_like(t["s0"])
        S.srnl_lattn_forward(h, cut["q"], cut["k"], cut["v"], o, state_in=t["s0"], state_out=st)
        steps = []
        for i in range(T, T + more):
            one = torch.empty(B, H * d, device="cuda", dtype=BF)
            S.srnl_lattn_step(h, *(t[n][:, i].contiguous() for n in "qkv"), one, st)
            steps.append(one)
        torch.cuda.synchronize()
    finally:
        h.close()
    ref = reference(t, decay, [T + more] * B, True, False)
    within(torch.cat([o, torch.stack(steps, 1)], 1), *ref["o"])
    within(st, *ref["state"])


def test_step_rows_of_a_joint_projection():
    B, H, d = 5, 2, 64
    D = H * d
    x = torch.randn(B, 3, D, generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    s0 = torch.randn(B, H, d, d, generator=torch.Generator().manual_seed(4)).cuda()
    h = S.srnl_lattn_create(dict(B=B, T=1, heads=H, d=d, ld=3 * D), np.array([0.5, 1.0], np.float32))
    try:
        o, st = torch.empty(B, D, device="cuda", dtype=BF), s0.clone()
        S.srnl_lattn_step(h, x[:, 0], x[:, 1], x[:, 2], o, st)
        torch.cuda.synchronize()
    finally:
        h.close()
    q, k, v = (x[:, i].double().view(B, H, d) for i in range(3))
    ref = torch.tensor([0.5, 1.0], device="cuda", dtype=torch.float64)[:, None, None] * s0.double() + k[..., None] * v[..., None, :]
    # a product and a sum; d products and sums
    assert bool(((st.double() - ref).abs() <= 2.0 ** -23 * (s0.double().abs() + (k[..., None] * v[..., None, :]).abs())).all())
    out = (q[..., None] * ref).sum(2)
    mag = (q.abs()[..., None] * ref.abs()).sum(2)
    assert bool(((o.double().view(B, H, d) - out).abs() <= HALF * out.abs() + 2.0 ** -17 * mag).all())


@pytest.mark.parametrize("d", [32, 64, 128])
def test_a_sequence_touches_no_other(d):
    B, T, H = 3, 200, 2
    t = make(B, T, H, d, seed=11)
    n = torch.tensor([200, 100, 150], device="cuda", dtype=torch.int32)
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), np.array([0.9, 0.99], np.float32))
    try:
        def both():
            o, g = torch.zeros_like(t["q"]), [torch.zeros_like(t["q"]) for _ in range(3)]
            st = torch.empty_like(t["s0"])
            S.srnl_lattn_forward(h, t["q"], t["k"], t["v"], o, lengths=n, state_out=st)
            S.srnl_lattn_backward(h, t["q"], t["k"], t["v"], t["do"], *g, lengths=n)
            torch.cuda.synchronize()
            return [o, *g, st]

        before = both()
        for x in "qkv":   # behind the lengths, and one head of sequence 0
            t[x][1, 100:] = float("nan")
            t[x][2, 150:] = float("inf")
            t[x][0, 50, d:] = float("nan")
        t["do"][1, 100:] = float("nan")
        after = both()
    finally:
        h.close()
    for a, b in zip(before, after):
        assert torch.equal(a[1:], b[1:])
        if a.dim() == 3:
            assert torch.equal(a[0, :, :d], b[0, :, :d]) and bool(torch.isnan(b[0, 50:, d:]).any())


def test_lengths_outside_the_range_are_clamped():
    B, T, H, d = 2, 70, 1, 64
    t = make(B, T, H, d, seed=2)
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), np.array([0.9], np.float32))
    try:
        def go(lens):
            o, st = torch.zeros_like(t["q"]), torch.empty_like(t["s0"])
            S.srnl_lattn_forward(h, t["q"], t["k"], t["v"], o, lengths=torch.tensor(lens, device="cuda", dtype=torch.int32),
                                 state_in=t["s0"], state_out=st)
            torch.cuda.synchronize()
            return o, st

        a, b = go([1 << 30, -5]), go([T, 0])
    finally:
        h.close()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(a[1][1], t["s0"][1]) and not a[0][1].any()


def test_a_decay_next_to_one_over_a_long_sequence():
    """g = 1 - 2^-20 over 2^18 tokens of ones: the state is a geometric sum, 2^20 (1 - g^n)."""
    T, d = 1 << 18, 32
    g = np.float32(1 - 2.0 ** -20)
    one = torch.ones(1, T, d, device="cuda", dtype=BF)
    h = S.srnl_lattn_create(dict(B=1, T=T, heads=1, d=d), np.array([g]))
    try:
        o, st = torch.empty_like(one), torch.empty(1, 1, d, d, device="cuda")
        S.srnl_lattn_forward(h, one, one, one, o, state_out=st)
        torch.cuda.synchronize()
    finally:
        h.close()
    G = float(g)
    want = (1 - math.exp(T * math.log(G))) / (1 - G)
    assert float((st.double() - want).abs().max()) <= 1.5 * 2.0 ** -16 * want


def test_rows_beyond_32_bits():
    """A row pitch that puts the last tokens past 2^31 elements; a short memory makes the last
    outputs a sum over few tokens."""
    T, d, ld = 70000, 32, 32768
    buf = torch.zeros(1, T, ld, device="cuda", dtype=BF)
    gen = torch.Generator(device="cuda").manual_seed(5)
    sl = [buf[:, :, i * d:(i + 1) * d] for i in range(3)]
    for x in sl:
        x.copy_(torch.randn(1, T, d, device="cuda", generator=gen))
    h = S.srnl_lattn_create(dict(B=1, T=T, heads=1, d=d, ld=ld), np.array([0.5], np.float32))
    try:
        o = torch.empty(1, T, d, device="cuda", dtype=BF)
        S.srnl_lattn_forward(h, *sl, o)
        dq, dk, dv = (buf[:, :, (i + 3) * d:(i + 4) * d] for i in range(3))
        S.srnl_lattn_backward(h, *sl, o, dq, dk, dv)
        torch.cuda.synchronize()
    finally:
        h.close()
    n = 300
    for lo in (0, T - n):
        t = {m: x[:, lo:lo + n] for m, x in zip("qkv", sl)}
        t["do"] = o[:, lo:lo + n]
        t["s0"] = t["ds"] = torch.zeros(1, 1, d, d, device="cuda")
        ref = reference(t, [0.5], [n], False, False)
        a, b = (0, n - 100) if lo == 0 else (100, n)   # 100 tokens away the rest is worth 2^-100
        for name, got in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
            within(got[:, lo + a:lo + b], *(x[:, a:b] for x in ref[name]))


@pytest.mark.parametrize("B,T,H,d", [(1, 1000, 1, 64), (2, 200, 3, 128)])
def test_two_calls_a_stream_and_a_graph_give_equal_bits(B, T, H, d):
    t = make(B, T, H, d, seed=9)
    decay = np.full(H, 0.98, np.float32)
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), decay)
    h2 = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), decay)
    try:
        def step(h, stream=None):
            outs = [torch.empty_like(t["q"]) for _ in range(4)] + [torch.empty_like(t["s0"]) for _ in range(2)]

            def go():
                S.srnl_lattn_forward(h, t["q"], t["k"], t["v"], outs[0], state_in=t["s0"], state_out=outs[4], stream=stream)
                S.srnl_lattn_backward(h, t["q"], t["k"], t["v"], t["do"], *outs[1:4], state_in=t["s0"],
                                      dstate_out=t["ds"], dstate_in=outs[5], stream=stream)

            return go, outs

        go0, o0 = step(h)
        go0()
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        go1, o1 = step(h, s1)
        go2, o2 = step(h2, s2)
        go1()
        go2()
        torch.cuda.synchronize()
        go3, o3 = step(h)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go3()
        graph.replay()
        torch.cuda.synchronize()
        for o in (o1, o2, o3):
            assert all(torch.equal(a, b) for a, b in zip(o, o0))
        del graph
    finally:
        h.close()
        h2.close()


def test_refusals():
    B, T, H, d = 2, 9, 2, 32
    t = make(B, T, H, d)
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), np.array([0.9, 0.9], np.float32))
    try:
        o = torch.empty_like(t["q"])

        def refused(text, call, *a, **kw):
            with pytest.raises(S.SrnlError) as e:
                call(h, *a, **kw)
            assert e.value.status == S.SRNL_E_INVAL and text in str(e.value), str(e.value)

        q, k, v = t["q"], t["k"], t["v"]
        refused("q must be", S.srnl_lattn_forward, q[:, :5], k, v, o)
        refused("k must be", S.srnl_lattn_forward, q, k.float(), v, o)
        refused("v must be", S.srnl_lattn_forward, q, k, make(B, T, H, d, packed=True)["v"], o)
        refused("o must be", S.srnl_lattn_forward, q, k, v, o[:1])
        refused("lengths must be", S.srnl_lattn_forward, q, k, v, o, lengths=torch.tensor([1, 2], device="cuda"))
        refused("state_in must be", S.srnl_lattn_forward, q, k, v, o, state_in=t["s0"][:1])
        refused("NULL", S.srnl_lattn_forward, q, None, v, o)
        refused("o overlaps q", S.srnl_lattn_forward, q, k, v, q)
        refused("state_out overlaps state_in", S.srnl_lattn_forward, q, k, v, o, state_in=t["s0"], state_out=t["s0"])
        refused("dv overlaps dq", S.srnl_lattn_backward, q, k, v, t["do"], o, torch.empty_like(o), o)
        refused("dk overlaps do", S.srnl_lattn_backward, q, k, v, t["do"], o, t["do"], torch.empty_like(o))
        refused("q must be", S.srnl_lattn_step, q, k, v, o, t["s0"])
        one = [x[:, 0].contiguous() for x in (q, k, v)]
        refused("o overlaps q", S.srnl_lattn_step, *one, one[0], t["s0"])
        refused("NULL", S.srnl_lattn_step, *one, torch.empty_like(one[0]), None)
        # slices of one row do not overlap, slices that share columns do
        x = torch.zeros(B, T, 4 * H * d, device="cuda", dtype=BF)
        hp = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d, ld=4 * H * d), np.array([0.9, 0.9], np.float32))
        try:
            sl = [x[:, :, i * 16:i * 16 + H * d] for i in range(4)]
            with pytest.raises(S.SrnlError) as e:
                S.srnl_lattn_backward(hp, q_ := sl[0], q_, q_, t["do"], sl[1], x[:, :, 128:192], x[:, :, 192:256])
            assert "dq overlaps q" in str(e.value)
            S.srnl_lattn_backward(hp, q_, q_, q_, t["do"], *(x[:, :, i * 64:i * 64 + 64] for i in (1, 2, 3)))
            torch.cuda.synchronize()
        finally:
            hp.close()
    finally:
        h.close()


@pytest.mark.parametrize("lo", [1, 129])
def test_padding_of_a_short_last_chunk_stays_out_of_the_state(lo):
    """128-wide heads whose last chunk is shorter than half: what lies behind the last token (NaN, infinities) reaches
    neither the state nor the outputs, whichever of the CTA's warps clears it.  Many CTAs, several calls."""
    B, H, d = 63, 4, 128
    T = lo + 190
    t = make(B, T, H, d, seed=lo)
    lens = [lo + i for i in range(B)]   # 1 to 63 tokens in the last chunk
    n = torch.tensor(lens, device="cuda", dtype=torch.int32)
    decay = np.array([1.0, 0.9, 0.99, 0.5], np.float32)
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), decay)
    try:
        def go():
            o, st = torch.zeros(B, T, H * d, device="cuda", dtype=BF), torch.empty_like(t["s0"])
            g, dsi = [torch.zeros_like(t["q"]) for _ in range(3)], torch.empty_like(t["s0"])
            S.srnl_lattn_forward(h, t["q"], t["k"], t["v"], o, lengths=n, state_in=t["s0"], state_out=st)
            S.srnl_lattn_backward(h, t["q"], t["k"], t["v"], t["do"], *g, lengths=n, state_in=t["s0"], dstate_out=t["ds"],
                                  dstate_in=dsi)
            torch.cuda.synchronize()
            return [o, st, *g, dsi]

        clean = go()
        for x in ("q", "k", "v", "do"):
            for b in range(B):
                t[x][b, lens[b]:] = (float("nan"), float("inf"), -float("inf"))[b % 3]
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(go(), clean))
        S.srnl_lattn_device_status(h)
    finally:
        h.close()


def long_sum(a, b, w, H, d):
    """sum_t w[h, t] a_t b_t^T in 64 bits, a piece at a time: [B, H, d, d]."""
    B, T, _ = a.shape
    out = torch.zeros(B, H, d, d, device="cuda", dtype=torch.float64)
    for x in range(B):
        for t in range(0, T, 8192):
            p, r = (y[x, t:t + 8192].double().view(-1, H, d).transpose(0, 1) for y in (a, b))
            out[x] += (p * w[:, t:t + 8192, None]).transpose(-1, -2) @ r
    return out


@pytest.mark.parametrize("B,T,H,d", [(4, 32768, 32, 64), (1, 16384, 16, 128), (2, 8192, 37, 64), (1, 65536, 3, 32), (3, 300, 6, 128),
                                     (2, 500, 6, 64), (1, 600, 6, 32)])
def test_states_of_long_memories(B, T, H, d):
    """The returned state and its gradient, head by head, to 2e-6 of their norm with memories that never fade.

    A chunk's products are summed in steps of 16 tokens, three parts each: 24 steps, which cut off half of a unit (2^-24 of
    the sum so far, itself half of the whole on average): 0.7e-6.  The chunks' sums, 256 of them at most, add 2^-25 each at
    random, 0.5e-6; weights and factors 4 u = 0.25e-6."""
    gen = torch.Generator(device="cuda").manual_seed(T + d)
    q, k, v = (torch.randn(B, T, H * d, device="cuda", generator=gen).to(BF) for _ in range(3))
    decay = np.array([[1.0, 1 - 2.0 ** -20, 0.999][i % 3] for i in range(H)], dtype=np.float32)
    st, ds = torch.empty(B, H, d, d, device="cuda"), torch.empty(B, H, d, d, device="cuda")
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), decay)
    try:
        o = torch.empty_like(q)
        S.srnl_lattn_forward(h, q, k, v, o, state_out=st)
        g = [torch.empty_like(q) for _ in range(3)]
        S.srnl_lattn_backward(h, q, k, v, v, *g, dstate_in=ds)
        torch.cuda.synchronize()
        S.srnl_lattn_device_status(h)
    finally:
        h.close()
    lg = torch.tensor(decay, device="cuda", dtype=torch.float64).log()[:, None]
    i = torch.arange(T, device="cuda")
    for got, a, e in ((st, k, T - 1 - i), (ds, q, i + 1)):
        ref = long_sum(a, v, torch.exp(lg * e), H, d)
        off = (got.double() - ref).flatten(2).norm(dim=2) / ref.flatten(2).norm(dim=2)
        assert float(off.max()) <= 2e-6, off


@pytest.mark.parametrize("T,at,g", [(300, 270, 0.97), (300, 100, 0.99), (1000, 200, 0.999), (1000, 990, 0.97)])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_one_token_in_the_state(d, T, at, g):
    """All tokens but one are zeros: its trace in the returned state holds g^m k v^T to 32 u (u = 2^-24), where two bf16 parts
    of g^m k would leave up to 64 u.  Roundings: the power 4 u and its argument 4 u, the factor it is split into and the
    product with k 2 u, three cut sums 6 u, two chunks' or three segments' factors 3 u each."""
    H = 8
    gen = torch.Generator(device="cuda").manual_seed(d + at)
    k, v = torch.zeros(1, T, H * d, device="cuda", dtype=BF), torch.zeros(1, T, H * d, device="cuda", dtype=BF)
    k[:, at], v[:, at] = (torch.randn(1, H * d, device="cuda", generator=gen).to(BF) for _ in range(2))
    st, o = torch.empty(1, H, d, d, device="cuda"), torch.empty_like(k)
    h = S.srnl_lattn_create(dict(B=1, T=T, heads=H, d=d), np.full(H, g, np.float32))
    try:
        S.srnl_lattn_forward(h, k, k, v, o, state_out=st)
        torch.cuda.synchronize()
    finally:
        h.close()
    x = k[0, at].double().view(H, d) * float(np.float32(g)) ** (T - 1 - at)
    y = v[0, at].double().view(H, d)
    ref = x[:, :, None] * y[:, None, :]
    assert bool(((st[0].double() - ref).abs() <= 32 * 2.0 ** -24 * ref.abs()).all())
    # the inputs do tell two parts from three, whichever power the kernel splits: the chunk's own
    w = k[0, at].float() * np.float32(g) ** np.float32(127 - at % 128 if T - at > 128 else T - 1 - at)
    hi = w.to(BF).float()
    two = hi.double() + (w - hi).to(BF).double()
    assert float(((two - w.double()).abs() / w.abs()).max()) > 34 * 2.0 ** -24


def test_other_orders_of_the_axes_are_refused():
    B, T, H, d = 2, 9, 3, 32
    t = make(B, T, H, d)
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), np.full(H, 0.9, np.float32))
    try:
        q, k, v, o = t["q"], t["k"], t["v"], torch.empty_like(t["q"])
        flip = lambda x: x.transpose(0, 1).contiguous()
        one = [x[:, 0].contiguous() for x in (q, k, v)]
        g = [torch.empty_like(q) for _ in range(3)]
        calls = [("o", lambda: S.srnl_lattn_forward(h, q, k, v, flip(o))), ("o", lambda: S.srnl_lattn_step(h, *one, flip(one[0]), t["s0"])),
                 ("state_in", lambda: S.srnl_lattn_forward(h, q, k, v, o, state_in=flip(t["s0"]))),
                 ("state_out", lambda: S.srnl_lattn_forward(h, q, k, v, o, state_out=flip(t["s0"]))),
                 ("do", lambda: S.srnl_lattn_backward(h, q, k, v, flip(o), *g)),
                 ("dstate_out", lambda: S.srnl_lattn_backward(h, q, k, v, o, *g, dstate_out=flip(t["s0"]))),
                 ("state", lambda: S.srnl_lattn_step(h, *one, o[:, 0].contiguous(), flip(t["s0"])))]
        for name, call in calls:
            with pytest.raises(S.SrnlError) as e:
                call()
            assert e.value.status == S.SRNL_E_INVAL and f"{name} must be" in str(e.value)
        S.srnl_lattn_forward(h, q, k, v, o.view(B, T, H, d), state_in=t["s0"].view(B * H, d, d))   # the same layout, told otherwise
        torch.cuda.synchronize()
    finally:
        h.close()


def test_a_new_handle_is_ready_for_any_stream():
    """Creation copies the decays on the default stream: behind work of that stream's own, the handle is not returned before
    they are there, and a call on a stream that waits for nothing finds them."""
    B, T, H, d = 2, 40, 3, 64
    t = make(B, T, H, d, seed=4)
    busy = torch.randn(8192, 8192, device="cuda", dtype=BF)
    side = torch.cuda.Stream()
    outs = []
    for i in range(3):
        torch.cuda.synchronize()
        for _ in range(10):
            busy @ busy
        h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), np.full(H, 0.9, np.float32))
        assert torch.cuda.default_stream().query()
        try:
            o, st = torch.full_like(t["q"], float("nan")), torch.empty_like(t["s0"])
            torch.cuda.synchronize()
            S.srnl_lattn_forward(h, t["q"], t["k"], t["v"], o, state_in=t["s0"], state_out=st, stream=side)
            torch.cuda.synchronize()
            outs.append((o, st))
        finally:
            h.close()
    assert all(torch.equal(a, b) for x in outs for a, b in zip(x, outs[0]))
    within(outs[0][0], *reference(t, [0.9] * H, [T] * B, True, False)["o"])


@pytest.mark.parametrize("B,T,H,d,lens", [(2, 12, 3, 32, None), (2, 16, 2, 128, [16, 9]), (3, 300, 3, 64, [300, 150, 260]),
                                          (2, 290, 2, 128, [290, 201]), (2, 200, 3, 32, None), (1, 1000, 2, 64, None), (1, 900, 1, 128, [899]),
                                          (40, 260, 3, 128, [260 - 3 * i for i in range(40)])])
def test_what_is_not_finite_reaches_no_earlier_token(B, T, H, d, lens):
    """One value of one token NaN or infinite: forward nothing before that token changes by a bit, backward nothing behind
    it but where the definition has it; nor any other head, sequence, or channel that it does not enter.  From the
    token on its channel is not finite."""
    decay = np.linspace(0.9, 1.0, H).astype(np.float32)
    t = make(B, T, H, d, seed=d + T)
    n = torch.tensor(lens, device="cuda", dtype=torch.int32) if lens else None
    D = H * d
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), decay)

    def run(t):
        o, st, dsi = torch.zeros(B, T, D, device="cuda", dtype=BF), torch.empty_like(t["s0"]), torch.empty_like(t["s0"])
        g = [torch.zeros_like(o) for _ in range(3)]
        S.srnl_lattn_forward(h, t["q"], t["k"], t["v"], o, lengths=n, state_in=t["s0"], state_out=st)
        S.srnl_lattn_backward(h, t["q"], t["k"], t["v"], t["do"], *g, lengths=n, state_in=t["s0"], dstate_out=t["ds"], dstate_in=dsi)
        torch.cuda.synchronize()
        return {"o": o, "dq": g[0], "dk": g[1], "dv": g[2], "state": st, "dstate": dsi}

    try:
        clean = run(t)
        b, head, ch = B - 1, H - 1, d - 3
        last = (lens[b] if lens else T) - 1
        col = head * d + ch
        for at in sorted({0, 1, last // 3, last // 2 + 1, last}):
            for name in ("q", "k", "v", "do"):
                for value in (float("nan"), float("inf")):
                    u = dict(t)
                    u[name] = t[name].clone()
                    u[name][b, at, col] = value
                    # a second token further on, which adds nothing to what the first one spoils
                    if at + 5 <= last and name in ("k", "v"):
                        u[name][b, at + 5, col] = -value
                    got = run(u)
                    from_, upto, own = slice(at, last + 1), slice(0, at + 1), slice(at, at + 1)
                    whole, one = slice(head * d, (head + 1) * d), slice(col, col + 1)
                    # rows and columns that may change: {output: (rows, columns)}, and those that have to be spoilt
                    may = {"q": {"o": (own, whole), "dk": (upto, one), "dv": (upto, whole)},
                           "k": {"o": (from_, whole), "dq": (from_, one), "dv": (None, whole)},
                           "v": {"o": (from_, one), "dq": (from_, whole), "dk": (None, whole)},
                           "do": {"dq": (own, whole), "dk": (upto, whole), "dv": (upto, one)}}[name]
                    for out in ("o", "dq", "dk", "dv"):
                        a, c = got[out].clone(), clean[out].clone()
                        rows, cols = may.get(out, (slice(0, 0), whole))
                        hit = [at] + ([at + 5] if at + 5 <= last and name in ("k", "v") else [])
                        for r in ([rows] if rows is not None else [slice(x, x + 1) for x in hit]):
                            if out in may and r.stop > r.start:
                                assert not bool(torch.isfinite(a[b, r, cols]).any()), (name, value, at, out)
                            a[b, r, cols] = c[b, r, cols] = 0
                        assert torch.equal(a, c), (name, value, at, out)
                    a, c = got["state"].clone(), clean["state"].clone()
                    if name in ("k", "v"):
                        part = a[b, head, ch] if name == "k" else a[b, head, :, ch]
                        assert not bool(torch.isfinite(part).any())
                        part.zero_()
                        (c[b, head, ch] if name == "k" else c[b, head, :, ch]).zero_()
                    assert torch.equal(a, c), (name, value, at, "state")
                    a, c = got["dstate"].clone(), clean["dstate"].clone()
                    if name in ("q", "do"):
                        part = a[b, head, ch] if name == "q" else a[b, head, :, ch]
                        assert not bool(torch.isfinite(part).any())
                        part.zero_()
                        (c[b, head, ch] if name == "q" else c[b, head, :, ch]).zero_()
                    assert torch.equal(a, c), (name, value, at, "dstate")
        S.srnl_lattn_device_status(h)
    finally:
        h.close()


@pytest.mark.parametrize("B,T,H,d", [(2, 16, 2, 64), (2, 300, 3, 64), (3, 400, 2, 128), (1, 1000, 2, 32)])
def test_values_beyond_half_the_exponents(B, T, H, d):
    """Values of 2^80: finite, whatever the watch for what is not makes of them.  Every result is linear in v, and in do: a power
    of two times them is that power times the results, bit by bit."""
    t = make(B, T, H, d, seed=T)
    lens = torch.tensor([T - 7 * i for i in range(B)], device="cuda", dtype=torch.int32)
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), np.linspace(0.9, 1.0, H).astype(np.float32))
    try:
        def run(v, do, s0):
            o, st, g, dsi = torch.zeros_like(t["q"]), torch.empty_like(s0), [torch.zeros_like(t["q"]) for _ in range(3)], torch.empty_like(s0)
            S.srnl_lattn_forward(h, t["q"], t["k"], v, o, lengths=lens, state_in=s0, state_out=st)
            S.srnl_lattn_backward(h, t["q"], t["k"], t["v"], do, *g, lengths=lens, dstate_in=dsi)
            torch.cuda.synchronize()
            return [o, st, *g, dsi]

        big = 2.0 ** 80
        small, large = run(t["v"], t["do"], t["s0"]), run(t["v"] * big, t["do"] * big, t["s0"] * big)
        for a, b in zip(small, large):
            assert bool(torch.isfinite(b).all()) and torch.equal(a.double() * big, b.double())
        S.srnl_lattn_device_status(h)
    finally:
        h.close()


def test_outputs_over_the_lengths_are_refused():
    B, T, H, d = 4, 40, 2, 32
    t = make(B, T, H, d)
    h = S.srnl_lattn_create(dict(B=B, T=T, heads=H, d=d), np.full(H, 0.9, np.float32))
    try:
        o, st = torch.empty_like(t["q"]), torch.empty_like(t["s0"])
        g = [torch.empty_like(o) for _ in range(3)]
        calls = [("o", o, lambda n: S.srnl_lattn_forward(h, t["q"], t["k"], t["v"], o, lengths=n)),
                 ("state_out", st, lambda n: S.srnl_lattn_forward(h, t["q"], t["k"], t["v"], o, lengths=n, state_out=st)),
                 ("dv", g[2], lambda n: S.srnl_lattn_backward(h, t["q"], t["k"], t["v"], t["do"], *g, lengths=n)),
                 ("dstate_in", st, lambda n: S.srnl_lattn_backward(h, t["q"], t["k"], t["v"], t["do"], *g, lengths=n, dstate_in=st))]
        for name, out, call in calls:
            n = out.view(torch.int32).flatten()[20:20 + B]
            n.copy_(torch.tensor([40, 0, 7, 33]))
            with pytest.raises(S.SrnlError) as e:
                call(n)
            assert e.value.status == S.SRNL_E_INVAL and f"{name} overlaps lengths" in str(e.value)
            call(n.clone())
        torch.cuda.synchronize()
    finally:
        h.close()
