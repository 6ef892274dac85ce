"""The gated feed-forward branch (srnl_ffn_*), forward and backward, against its definition in
64 bits.

Tolerances.  half = 2^-8 bounds a bf16 rounding relative to the value.  An output is rounded once:
half of its value.  A product over K values that were each rounded on the way (h, dgate, dup)
adds K errors, each at most half of its value and of zero mean, that is of standard deviation at
most half / sqrt(3): seven standard deviations of their sum cover every one of the few million
values compared here (2.6e-12 each).  Sums in fp32 add 2 u (K / 16 + 16) of the magnitudes
(u = 2^-24; 16 products a step), the activations 2^-18 of the hidden value.
"""
import math

import numpy as np
import pytest
import torch

import self_referential_nested_b200 as S

pytestmark = pytest.mark.gpu

HALF, U = 2.0 ** -8, 2.0 ** -24
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_referential_nested_b200 import build
    build.build()
    torch.cuda.set_device(0)


def make(rows, dim, hidden, seed=0):
    g = torch.Generator().manual_seed(seed)

    def n(*s, scale=1.0):
        return (torch.randn(*s, generator=g) * scale).to(BF).cuda()

    return {"x": n(rows, dim), "res": n(rows, dim), "dy": n(rows, dim),
            "p": {"W_gate": n(hidden, dim, scale=dim ** -0.5), "W_up": n(hidden, dim, scale=dim ** -0.5),
                  "W_down": n(dim, hidden, scale=hidden ** -0.5)}}


def act64(v, kind):
    if kind == "silu":
        p = torch.sigmoid(v)
        return v * p, p * (1 + v * (1 - p))
    p = 0.5 * torch.special.erfc(-v / math.sqrt(2))
    return v * p, p + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)


def within(got, ref, magnitude, spread2, K, slack=0.0):
    """|got - ref| <= half |ref| + 7 half / sqrt(3) sqrt(spread2) + fp32 sums (+ slack)."""
    assert bool(torch.isfinite(got).all())
    tol = HALF * ref.abs() + 7 * HALF / math.sqrt(3) * spread2.sqrt() + (2 * U * (K / 16 + 16) + 2.0 ** -18) * magnitude + slack
    worst = ((got.double() - ref).abs() / tol.clamp_min(1e-300)).max()
    assert float(worst) <= 1, float(worst)


SHAPES = [(1, 8, 8), (3, 64, 128), (7, 72, 136), (16, 128, 256), (33, 264, 520), (64, 256, 1024), (128, 512, 648),
          (129, 136, 1384), (256, 256, 256), (300, 520, 1384), (777, 1024, 2056), (2050, 264, 264),
          # long sums over few tiles: K goes to the CTAs in parts
          (40, 72, 2056), (65, 264, 4104), (301, 136, 4104), (300, 136, 4104), (34, 1096, 3000),
          (3000, 72, 136), (5001, 136, 264)]   # and of many rows the weights' gradients


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,dim,hidden", SHAPES)
def test_forward_and_backward(rows, dim, hidden, act):
    t = make(rows, dim, hidden, seed=rows)
    h = S.srnl_ffn_create(dict(dim=dim, hidden=hidden, max_rows=rows + 5, activation=act, training=True))
    keep = rows % 2 == 1 or rows >= 256
    try:
        y = torch.full((rows + 3, dim), 7.0, device="cuda", dtype=BF)   # rows behind the last stay
        gate, up = (torch.full((rows + 3, hidden), 7.0, device="cuda", dtype=BF) for _ in range(2))
        S.srnl_ffn_forward(h, t["x"], t["p"], y[:rows], res=t["res"] if keep else None, gate=gate[:rows], up=up[:rows])
        y2 = torch.empty(rows, dim, device="cuda", dtype=BF)
        S.srnl_ffn_forward(h, t["x"], t["p"], y2, res=t["res"] if keep else None)   # nothing kept: the same y
        dx = torch.full((rows + 3, dim), 7.0, device="cuda", dtype=BF)
        grads = {k: torch.full_like(v, float("nan")) for k, v in t["p"].items()}
        S.srnl_ffn_backward(h, t["x"], gate[:rows], up[:rows], t["dy"], t["p"], dx[:rows], grads)
        torch.cuda.synchronize()
        S.srnl_ffn_device_status(h)
    finally:
        h.close()
    for b in (y, gate, up, dx):
        assert bool((b[rows:] == 7).all())
    assert torch.equal(y[:rows], y2)
    y, gate, up, dx = y[:rows], gate[:rows], up[:rows], dx[:rows]
    x, dy = t["x"].double(), t["dy"].double()
    Wg, Wu, Wd = (t["p"][k].double() for k in S.FFN_KEYS)
    g64, u64 = x @ Wg.t(), x @ Wu.t()
    zero = torch.zeros((), device="cuda", dtype=torch.float64)
    within(gate, g64, x.abs() @ Wg.abs().t(), zero, dim)
    within(up, u64, x.abs() @ Wu.abs().t(), zero, dim)
    hid = act64(g64, act)[0] * u64
    ref = hid @ Wd.t()
    ref = ref + t["res"].double() if keep else ref
    within(y, ref, hid.abs() @ Wd.abs().t(), (hid ** 2) @ (Wd ** 2).t(), hidden)

    g, u = gate.double(), up.double()
    a, da = act64(g, act)
    dh = dy @ Wd
    dg, du, hid = dh * u * da, dh * a, a * u
    within(dx, dg @ Wg + du @ Wu, dg.abs() @ Wg.abs() + du.abs() @ Wu.abs(), (dg ** 2) @ (Wg ** 2) + (du ** 2) @ (Wu ** 2),
           2 * hidden + dim)
    within(grads["W_gate"], dg.t() @ x, dg.abs().t() @ x.abs(), (dg ** 2).t() @ (x ** 2), rows + dim)
    within(grads["W_up"], du.t() @ x, du.abs().t() @ x.abs(), (du ** 2).t() @ (x ** 2), rows + dim)
    within(grads["W_down"], dy.t() @ hid, dy.abs().t() @ hid.abs(), (dy ** 2).t() @ (hid ** 2), rows)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_against_differences(act):
    """Central differences of sum(dy * y) in 64 bits against the returned gradients, along random
    directions: a sum of n gradients, each off by its tolerance at most, divided as n roundings
    of zero mean divide: a standard deviation of half / sqrt(3) |g| sqrt(2) each (its own rounding
    and that of the products' factors), seven of them."""
    rows, dim, hidden = 40, 72, 136
    t = make(rows, dim, hidden, seed=4)
    h = S.srnl_ffn_create(dict(dim=dim, hidden=hidden, max_rows=rows, activation=act, training=True))
    try:
        y, gate, up = (torch.empty(rows, n, device="cuda", dtype=BF) for n in (dim, hidden, hidden))
        S.srnl_ffn_forward(h, t["x"], t["p"], y, gate=gate, up=up)
        grads = {k: torch.empty_like(v) for k, v in t["p"].items()}
        grads["x"] = torch.empty_like(y)
        S.srnl_ffn_backward(h, t["x"], gate, up, t["dy"], t["p"], grads["x"], {k: grads[k] for k in S.FFN_KEYS})
        torch.cuda.synchronize()
    finally:
        h.close()
    base = {k: v.double() for k, v in t["p"].items()}
    base["x"] = t["x"].double()
    gen = torch.Generator().manual_seed(2)
    for name, grad in grads.items():
        v = torch.randn(grad.shape, generator=gen).cuda().double()

        def loss(s):
            q = dict(base)
            q[name] = q[name] + s * v
            hid = act64(q["x"] @ q["W_gate"].t(), act)[0] * (q["x"] @ q["W_up"].t())
            return float((t["dy"].double() * (hid @ q["W_down"].t())).sum())

        num = (loss(1e-5) - loss(-1e-5)) / 2e-5
        # gate and up are rounded too, which moves every gradient of a row together: counted as
        # four roundings in place of two
        rms = float((grad.double() * v).square().sum().sqrt())
        assert abs(num - float((grad.double() * v).sum())) <= 7 * HALF / math.sqrt(3) * 2 * rms * math.sqrt(2) + 1e-5


def test_gradients_that_are_not_asked_for():
    rows, dim, hidden = 200, 128, 264
    t = make(rows, dim, hidden, seed=6)
    h = S.srnl_ffn_create(dict(dim=dim, hidden=hidden, max_rows=rows, training=True))
    try:
        y, gate, up = (torch.empty(rows, n, device="cuda", dtype=BF) for n in (dim, hidden, hidden))
        S.srnl_ffn_forward(h, t["x"], t["p"], y, gate=gate, up=up)

        def back(keys, with_dx=True):
            dx = torch.empty_like(y) if with_dx else None
            g = {k: torch.empty_like(t["p"][k]) for k in keys}
            S.srnl_ffn_backward(h, t["x"], gate, up, t["dy"], t["p"], dx, g)
            torch.cuda.synchronize()
            return dx, g

        dx, full = back(S.FFN_KEYS)
        for keys in (("W_gate",), ("W_up",), ("W_down",), ("W_up", "W_down"), ()):
            d, g = back(keys)
            assert torch.equal(d, dx) and all(torch.equal(g[k], full[k]) for k in keys)
        _, g = back(S.FFN_KEYS, with_dx=False)
        assert all(torch.equal(g[k], full[k]) for k in S.FFN_KEYS)
        back((), with_dx=False)
    finally:
        h.close()


@pytest.mark.parametrize("rows", [5, 300])
def test_a_row_touches_no_other(rows):
    dim, hidden = 128, 256
    t = make(rows, dim, hidden, seed=7)
    h = S.srnl_ffn_create(dict(dim=dim, hidden=hidden, max_rows=rows))
    try:
        y0, y1 = torch.empty(rows, dim, device="cuda", dtype=BF), torch.empty(rows, dim, device="cuda", dtype=BF)
        S.srnl_ffn_forward(h, t["x"], t["p"], y0)
        t["x"][2, 5] = float("nan")
        S.srnl_ffn_forward(h, t["x"], t["p"], y1)
        torch.cuda.synchronize()
    finally:
        h.close()
    keep = [i for i in range(rows) if i != 2]
    assert torch.equal(y0[keep], y1[keep]) and bool(torch.isnan(y1[2]).all())


def test_saturated_activations():
    """Pre-activations of +-200: SiLU and GELU are v or 0 there, with slopes 1 and 0."""
    dim = hidden = 64
    eye = torch.eye(64, device="cuda", dtype=BF)
    x = torch.full((4, 64), 200.0, device="cuda", dtype=BF)
    x[1], x[3] = -200.0, -200.0
    one = torch.ones(4, 64, device="cuda", dtype=BF)
    for act in ("silu", "gelu"):
        h = S.srnl_ffn_create(dict(dim=dim, hidden=hidden, max_rows=4, activation=act, training=True))
        try:
            y, gate, up, dx = (torch.empty(4, 64, device="cuda", dtype=BF) for _ in range(4))
            p = {"W_gate": eye, "W_up": eye, "W_down": eye}
            S.srnl_ffn_forward(h, x, p, y, gate=gate, up=up)
            S.srnl_ffn_backward(h, x, gate, up, one, p, dx)
            torch.cuda.synchronize()
        finally:
            h.close()
        # v^2 = 40000 rounds to 39936; d(v act(v)) = act + v act' = 400
        assert bool((y[0::2].float() == 39936).all()) and bool((y[1::2] == 0).all())
        assert bool((dx[0::2] == 400).all()) and bool((dx[1::2] == 0).all())


@pytest.mark.parametrize("rows,dim,hidden", [(3, 264, 520), (200, 264, 520), (200, 264, 4104)])   # the last: K in parts
def test_two_calls_a_stream_and_a_graph_give_equal_bits(rows, dim, hidden):
    t = make(rows, dim, hidden, seed=9)
    h = S.srnl_ffn_create(dict(dim=dim, hidden=hidden, max_rows=rows, training=True))
    h2 = S.srnl_ffn_create(dict(dim=dim, hidden=hidden, max_rows=rows, training=True))
    try:
        def step(h, stream=None):
            y, gate, up = (torch.empty(rows, n, device="cuda", dtype=BF) for n in (dim, hidden, hidden))
            dx, g = torch.empty_like(y), {k: torch.empty_like(v) for k, v in t["p"].items()}

            def go():
                S.srnl_ffn_forward(h, t["x"], t["p"], y, res=t["res"], gate=gate, up=up, stream=stream)
                S.srnl_ffn_backward(h, t["x"], gate, up, t["dy"], t["p"], dx, g, stream=stream)

            return go, [y, gate, up, dx, *g.values()]

        go0, o0 = step(h)
        go0()
        torch.cuda.synchronize()
        # two handles on two streams at once
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
        S.srnl_ffn_device_status(h)
        S.srnl_ffn_device_status(h2)
    finally:
        h.close()
        h2.close()


def test_no_rows_and_refusals():
    dim, hidden = 64, 128
    t = make(4, dim, hidden)
    h = S.srnl_ffn_create(dict(dim=dim, hidden=hidden, max_rows=4, training=True))
    try:
        e, f = torch.empty(0, dim, device="cuda", dtype=BF), torch.empty(0, hidden, device="cuda", dtype=BF)
        S.srnl_ffn_forward(h, e, t["p"], torch.empty_like(e))
        g = {k: torch.full_like(v, 3.0) for k, v in t["p"].items()}
        S.srnl_ffn_backward(h, e, f, f, e, t["p"], torch.empty_like(e), g)
        torch.cuda.synchronize()
        assert not any(bool(v.any()) for v in g.values())
        y, gate = torch.empty_like(t["x"]), torch.empty(4, hidden, device="cuda", dtype=BF)

        def refused(text, call, *a, **kw):
            with pytest.raises(S.SrnlError) as err:
                call(h, *a, **kw)
            assert err.value.status == S.SRNL_E_INVAL and text in str(err.value)

        big = torch.zeros(5, dim, device="cuda", dtype=BF)
        refused("max_rows", S.srnl_ffn_forward, big, t["p"], torch.empty_like(big))
        refused("together", S.srnl_ffn_forward, t["x"], t["p"], y, gate=gate)
        refused("overlaps", S.srnl_ffn_forward, t["x"], t["p"], t["x"])
        refused("overlaps", S.srnl_ffn_forward, t["x"], t["p"], y, res=y)
        refused("up overlaps gate", S.srnl_ffn_forward, t["x"], t["p"], y, gate=gate, up=gate)
        refused("x must be", S.srnl_ffn_forward, t["x"].float(), t["p"], y)
        refused("W_up must be", S.srnl_ffn_forward, t["x"], dict(t["p"], W_up=t["p"]["W_up"].float()), y)
        refused("NULL", S.srnl_ffn_forward, t["x"], {k: v for k, v in t["p"].items() if k != "W_up"}, y)
        buf = torch.zeros(4 * dim + 8, device="cuda", dtype=BF)
        refused("aligned", S.srnl_ffn_forward, buf[1:257].view(4, dim), t["p"], y)
        refused("NULL", S.srnl_ffn_backward, t["x"], gate, None, t["dy"], t["p"], y)
        S.srnl_ffn_device_status(h)
    finally:
        h.close()
    h = S.srnl_ffn_create(dict(dim=dim, hidden=hidden, max_rows=4))
    try:
        refused("training", S.srnl_ffn_backward, t["x"], gate, gate.clone(), t["dy"], t["p"], y)
    finally:
        h.close()


@pytest.mark.parametrize("rows", [8, 300])   # few rows, and tiles
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_over_their_range(act, rows):
    """act(v) and its slope for every v on a grid from far below zero, where they are small beside v, to above: identity
    weights make y act(v), and the gradients act(v) and act'(v), each after one or two roundings.

    Relative to the magnitude of its terms each is off by at most 2^-14: the exponential's argument by two roundings and
    its own, 2.5 u |v|^2 / 2 ln 2 / ln 2 = 210 u at -13 (SiLU: 2 u |v| = 174 u at -87), the exponential and the reciprocal
    by 4 u each, the rest of the formula by 2^-18; 2^-14 is 1024 u.  Beside that only what lies below fp32's smallest
    normal number is lost."""
    n = 64
    eye, zero = torch.eye(n, device="cuda", dtype=BF), torch.zeros(n, n, device="cuda", dtype=BF)
    lowest = -12.75 if act == "gelu" else -80.0
    v = torch.linspace(lowest, 6, rows * n, device="cuda").to(BF).view(rows, n)
    one = torch.ones(rows, n, device="cuda", dtype=BF)
    x, dy = torch.cat([v, one], 1), torch.cat([one, 0 * one], 1)
    p = {"W_gate": torch.cat([eye, zero], 1), "W_up": torch.cat([zero, eye], 1), "W_down": torch.cat([eye, zero], 0)}
    h = S.srnl_ffn_create(dict(dim=2 * n, hidden=n, max_rows=rows, activation=act, training=True))
    try:
        y, dx = torch.empty_like(x), torch.empty_like(x)
        gate, up = torch.empty_like(v), torch.empty_like(v)
        S.srnl_ffn_forward(h, x, p, y, gate=gate, up=up)
        S.srnl_ffn_backward(h, x, gate, up, dy, p, dx)
        torch.cuda.synchronize()
        S.srnl_ffn_device_status(h)
    finally:
        h.close()
    assert torch.equal(gate, v) and torch.equal(up, one) and not bool(y[:, n:].any())
    u = v.double()
    f, df = act64(u, act)
    if act == "silu":
        s = torch.sigmoid(u)
        terms = s + u.abs() * s * torch.sigmoid(-u)
        df = s + u * s * torch.sigmoid(-u)   # 1 - s without cancellation
    else:
        terms = 0.5 * torch.special.erfc(-u / math.sqrt(2)) + u.abs() * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    for name, got, ref, size in (("y", y[:, :n], f, f.abs()), ("act", dx[:, n:], f, f.abs()), ("slope", dx[:, :n], df, terms)):
        # rounded to bf16 once; the second time it is a bf16 number already
        off = (got.double() - ref).abs() / (HALF * ref.abs() + 2.0 ** -14 * size + 2.0 ** -120)
        assert float(off.max()) <= 1, (name, float(off.max()), float(u.flatten()[off.argmax()]))


def test_transposed_weights_and_rows_are_refused():
    dim, hidden = 64, 128
    t = make(4, dim, hidden)
    h = S.srnl_ffn_create(dict(dim=dim, hidden=hidden, max_rows=4, training=True))
    try:
        y, gate, up = (torch.empty(4, n, device="cuda", dtype=BF) for n in (dim, hidden, hidden))
        g = {k: torch.empty_like(v) for k, v in t["p"].items()}
        flip = lambda v: v.t().contiguous()
        calls = [(k, lambda k=k: S.srnl_ffn_forward(h, t["x"], dict(t["p"], **{k: flip(t["p"][k])}), y)) for k in S.FFN_KEYS]
        calls += [(k, lambda k=k: S.srnl_ffn_backward(h, t["x"], gate, up, t["dy"], t["p"], y, dict(g, **{k: flip(g[k])})))
                  for k in S.FFN_KEYS]
        calls += [("x", lambda: S.srnl_ffn_forward(h, flip(t["x"]), t["p"], y)), ("res", lambda: S.srnl_ffn_forward(h, t["x"], t["p"], y, res=flip(y))),
                  ("gate", lambda: S.srnl_ffn_forward(h, t["x"], t["p"], y, gate=flip(gate), up=up)),
                  ("dy", lambda: S.srnl_ffn_backward(h, t["x"], gate, up, flip(t["dy"]), t["p"], y))]
        for name, call in calls:
            with pytest.raises(S.SrnlError) as e:
                call()
            assert e.value.status == S.SRNL_E_INVAL and f"{name} must be" in str(e.value)
    finally:
        h.close()


def test_a_new_handle_is_ready_for_any_stream():
    """Creation clears the counters that products in parts rely on, on the default stream: behind work of that stream's own,
    the handle is not returned before they are clear, and a call on a stream that waits for nothing finds them so."""
    rows, dim, hidden = 300, 136, 4104
    t = make(rows, dim, hidden, seed=3)
    busy = torch.randn(8192, 8192, device="cuda", dtype=BF)
    side = torch.cuda.Stream()
    ys = []
    for i in range(3):
        torch.cuda.synchronize()
        for _ in range(10):
            busy @ busy
        h = S.srnl_ffn_create(dict(dim=dim, hidden=hidden, max_rows=rows))
        assert torch.cuda.default_stream().query()
        try:
            y = torch.full((rows, dim), float("nan"), device="cuda", dtype=BF)
            torch.cuda.synchronize()
            S.srnl_ffn_forward(h, t["x"], t["p"], y, stream=side)
            torch.cuda.synchronize()
            S.srnl_ffn_device_status(h)
            ys.append(y)
        finally:
            h.close()
    assert bool(torch.isfinite(ys[0]).all()) and all(torch.equal(y, ys[0]) for y in ys)


# More tiles than pairs of CTAs (74), so that a pair takes a second and a third one, in either tile width (columns, tiles):
MANY_TILES = [
    (5000, 1032, 1544),    # projections 256, 260; output 256, 100; hidden gradients 256, 140; gradients 256, 205
    (20000, 264, 520),     # 256, 395; 256, 158; 256, 237; gradients in parts, 256, 230
    (9473, 264, 264),      # output 128, 114; hidden gradients 128, 114
    (4943, 64, 888),       # hidden gradients 128, 140
    (3721, 8, 552),        # projections 128, 135
    (257, 1032, 9000),     # output in parts, 128, 72; gradients in parts, 256, 600
    (34, 3136, 7296),      # output in parts, 256, 52
    (37, 1424, 832),       # gradients 128, 150
    (157, 16, 8744),       # gradients in parts, 128, 151
    (8885, 1392, 8),       # output 256, 210
]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,dim,hidden", MANY_TILES)
def test_forward_and_backward_of_many_tiles(rows, dim, hidden, act):
    test_forward_and_backward(rows, dim, hidden, act)
