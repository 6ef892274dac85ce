"""Layer normalisation forward and backward (srnl_ln_*) against its definition in 64 bits.

Tolerances.  u = 2^-24 is half an fp32 step.  A row's sum is at most 32 additions in a lane and
10 across lanes, so a sum is off by at most 42 u times the sum of magnitudes; a product or a
difference adds u each, rsqrtf 2 u.  An output rounded to its type adds eps / 2 of its value.  A
column's sum over rows is at most rows / 148 + 8 + 4 + 37 + 32 additions (a block's rows, its groups and
warps, 1184 partials over 32 warps), under 200 for the rows used here.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import self_referential_nested_b200 as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from self_referential_nested_b200 import build
    build.build()
    torch.cuda.set_device(0)


def make(rows, dim, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    t = {"x": (torch.randn(rows, dim, generator=g) * torch.exp(0.5 * torch.randn(dim, generator=g)) + 0.5).to(dt),
         "dy": torch.randn(rows, dim, generator=g).to(dt), "dres": torch.randn(rows, dim, generator=g).to(dt),
         "gamma": 1 + 0.3 * torch.randn(dim, generator=g), "beta": 0.3 * torch.randn(dim, generator=g)}
    return {k: v.cuda() for k, v in t.items()}


def forward(h, t, extra=0):
    rows, dim = t["x"].shape
    # rows behind the last one keep what they hold
    buf = torch.full((rows + extra, dim), 7.0, device="cuda", dtype=t["x"].dtype)
    mean, rstd = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
    S.srnl_ln_forward(h, t["x"], t["gamma"], t["beta"], buf[:rows], mean, rstd)
    torch.cuda.synchronize()
    assert bool((buf[rows:] == 7).all())
    return buf[:rows], mean, rstd


def reference(t, eps):
    x, g, b = t["x"].double(), t["gamma"].double(), t["beta"].double()
    mean = x.mean(1, keepdim=True)
    rstd = (((x - mean) ** 2).mean(1, keepdim=True) + eps).rsqrt()
    return (x - mean) * rstd * g + b, mean, rstd


SHAPES = [(1, 1), (5, 3), (1, 8), (7, 33), (3, 64), (1000, 64), (37, 100), (65, 128), (9, 129), (130, 256), (21, 257),
          (196, 384), (11, 512), (13, 513), (50, 1000), (600, 1024), (5, 1025), (17, 2048), (301, 2560), (9, 4096),
          (3, 8191), (4, 8192), (5000, 96), (4001, 7), (3003, 2051), (2500, 1023), (700, 4096), (1, 8192),
          (2000, 8), (999, 2044)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_forward_and_backward(rows, dim, dtype):
    eps = 1e-5
    t = make(rows, dim, dtype, seed=rows + dim)
    half = torch.finfo(DT[dtype]).eps / 2 if dtype == "bf16" else U
    h = S.srnl_ln_create(dict(dim=dim, eps=eps, act_dtype=dtype))
    try:
        y, mean, rstd = forward(h, t, extra=2)
        eps64 = float(np.float32(eps))
        ref, m, r = reference(t, eps64)
        size = t["x"].double().abs().mean(1, keepdim=True)
        g, b = t["gamma"].double().abs(), t["beta"].double().abs()
        xhat = (ref - t["beta"].double()) / t["gamma"].double()
        xh = (t["x"].double() - m) * r
        # of a value: its own roundings and rstd's (half of 45 u, 2 u), the mean's 42 u, beta's
        tol = half * ref.abs() + U * (30 * xh.abs() * g + 46 * size * r * g + 2 * b)
        assert bool(((y.double() - ref).abs() <= tol).all())
        assert bool(((mean.double() - m[:, 0]).abs() <= 44 * U * size[:, 0]).all())
        # the mean's error squared enters the variance: below u where |mean| is of the spread's order
        assert bool(((rstd.double() / r[:, 0] - 1).abs() <= 30 * U + (46 * U * size * r)[:, 0] ** 2).all())

        dres = t["dres"] if rows % 2 else None
        dx = torch.full_like(t["x"], float("nan"))
        dg, db = torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
        S.srnl_ln_backward(h, t["x"], t["dy"], t["gamma"], mean, rstd, dx, dg, db, dres=dres)
        torch.cuda.synchronize()
    finally:
        h.close()
    # the statistics are inputs of the backward pass
    r64, dy = rstd.double()[:, None], t["dy"].double()
    xh = (t["x"].double() - mean.double()[:, None]) * r64
    w = dy * t["gamma"].double()
    ref = r64 * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    if dres is not None:
        ref = ref + dres.double()
    # three terms: w's own, the two sums (42 additions, and the factors' roundings)
    big = r64 * (6 * w.abs() + 50 * w.abs().mean(1, keepdim=True) + 56 * xh.abs() * (w * xh).abs().mean(1, keepdim=True))
    tol = half * ref.abs() + U * (big + 4 * ref.abs())
    assert bool(((dx.double() - ref).abs() <= tol).all())
    assert bool(((dg.double() - (dy * xh).sum(0)).abs() <= 200 * U * (dy * xh).abs().sum(0)).all())
    assert bool(((db.double() - dy.sum(0)).abs() <= 200 * U * dy.abs().sum(0)).all())


@pytest.mark.parametrize("rows,dim", [(6, 24), (3, 129), (2, 2052)])
def test_gradients_against_differences(rows, dim):
    """Central differences of sum(dy * y) in 64 bits along random directions of x, gamma, beta."""
    eps = 1e-5
    t = make(rows, dim, "f32", seed=3)
    h = S.srnl_ln_create(dict(dim=dim, eps=eps, act_dtype="f32"))
    try:
        _, mean, rstd = forward(h, t)
        dx, dg, db = torch.empty_like(t["x"]), torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
        S.srnl_ln_backward(h, t["x"], t["dy"], t["gamma"], mean, rstd, dx, dg, db)
        torch.cuda.synchronize()
    finally:
        h.close()
    gen = torch.Generator().manual_seed(9)
    step = 1e-5
    for name, grad in (("x", dx), ("gamma", dg), ("beta", db)):
        v = torch.randn(grad.shape, generator=gen).cuda().double()

        def loss(s):
            p = {k: a.double() for k, a in t.items()}
            p[name] = p[name] + s * v
            return float((p["dy"] * reference(p, float(np.float32(eps)))[0]).sum())

        num = (loss(step) - loss(-step)) / (2 * step)
        # fp32 gradients: 60 u of the magnitudes; differences: step^2 and 1e-16 / step
        assert abs(num - float((grad.double() * v).sum())) <= 100 * U * float((grad.double() * v).abs().sum()) + 1e-6


def test_no_rows():
    h = S.srnl_ln_create(dict(dim=40, act_dtype="bf16"))
    try:
        x = torch.empty(0, 40, device="cuda", dtype=torch.bfloat16)
        g, b, e = torch.ones(40, device="cuda"), torch.ones(40, device="cuda"), torch.empty(0, device="cuda")
        S.srnl_ln_forward(h, x, g, b, torch.empty_like(x), e, torch.empty_like(e))
        dg, db = torch.full_like(g, 3.0), torch.full_like(g, 3.0)
        S.srnl_ln_backward(h, x, torch.empty_like(x), g, e, e, torch.empty_like(x), dg, db)
        torch.cuda.synchronize()
        assert not dg.any() and not db.any()
    finally:
        h.close()


@pytest.mark.parametrize("dim", [64, 100, 2048])
def test_a_row_touches_no_other(dim):
    """A row of NaN or infinity changes its own outputs alone; a constant row gives beta."""
    t = make(40, dim, "f32", seed=5)
    h = S.srnl_ln_create(dict(dim=dim, act_dtype="f32"))
    try:
        y0, m0, r0 = forward(h, t)
        t["x"][3, 1], t["x"][17], t["x"][21, 0] = float("nan"), float("inf"), float("-inf")
        t["x"][30] = 2.5
        y1, m1, r1 = forward(h, t)
    finally:
        h.close()
    keep = [i for i in range(40) if i not in (3, 17, 21, 30)]
    assert torch.equal(y0[keep], y1[keep]) and torch.equal(m0[keep], m1[keep]) and torch.equal(r0[keep], r1[keep])
    assert bool(torch.isnan(y1[[3, 17, 21]]).all())
    # 2.5 dim / dim is exact or off by half a step of 2.5, which 1 / sqrt(eps) = 1000 enlarges
    assert float((y1[30] - t["beta"]).abs().max()) <= 43 * U * 2.5 * 1000 * float(t["gamma"].abs().max())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [9, 33, 301, 509, 1533, 4097, 8191])
def test_an_odd_row_keeps_its_neighbours_out(dim, dtype):
    """Rows share 16-byte units with their neighbours where the row's length is odd: rows of NaN and
    infinity in x, dy and dres change no bit of the rows beside them, forward or backward."""
    t = make(37, dim, dtype, seed=6)
    h = S.srnl_ln_create(dict(dim=dim, act_dtype=dtype))
    bad = [0, 2, 17, 35]
    keep = [i for i in range(37) if i not in bad]
    try:
        outs = []
        for spoil in (False, True):
            if spoil:
                t["x"][bad], t["dy"][bad], t["dres"][bad] = float("nan"), float("inf"), float("nan")
            y, mean, rstd = forward(h, t)
            dx = torch.empty_like(t["x"])
            S.srnl_ln_backward(h, t["x"], t["dy"], t["gamma"], mean, rstd, dx, dres=t["dres"])
            outs.append((y[keep], mean[keep], rstd[keep], dx[keep]))
        for a, b in zip(*outs):
            assert torch.equal(a, b) and bool(torch.isfinite(a).all())
    finally:
        h.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_handles_of_long_odd_rows_side_by_side(dtype):
    """A later handle of shorter rows leaves an earlier one's calls as they are."""
    ts = [make(9, dim, dtype, seed=dim) for dim in (8191, 6205, 7001)]
    hs = [S.srnl_ln_create(dict(dim=t["gamma"].numel(), act_dtype=dtype)) for t in ts]
    try:
        for h, t in list(zip(hs, ts)) + list(zip(hs, ts))[::-1]:
            y, _, _ = forward(h, t)
            ref = reference(t, float(np.float32(1e-6)))[0]
            # a rounding of the output, and fp32 sums and products a hundred steps long
            assert float((y.double() - ref).norm()) <= (torch.finfo(DT[dtype]).eps / 2 + 100 * U) * float(ref.norm())
    finally:
        for h in hs:
            h.close()


def test_large_offset_keeps_the_spread():
    """The variance is taken from the centred values: an offset of 4096 spreads leaves it right."""
    x = torch.randn(64, 512, generator=torch.Generator().manual_seed(1)).cuda() + 4096.0
    t = {"x": x, "gamma": torch.ones(512, device="cuda"), "beta": torch.zeros(512, device="cuda")}
    h = S.srnl_ln_create(dict(dim=512, act_dtype="f32"))
    try:
        y, _, rstd = forward(h, t)
    finally:
        h.close()
    ref, m, r = reference(t, float(np.float32(1e-6)))
    bound = 46 * U * 4100   # the mean's error, against a spread of one
    assert float((y.double() - ref).abs().max()) <= bound
    assert float((rstd.double() / r[:, 0] - 1).abs().max()) <= 30 * U + bound ** 2


@pytest.mark.parametrize("dim", [64, 1000, 2560])
def test_two_calls_a_stream_and_a_graph_give_equal_bits(dim):
    t = make(2000, dim, "bf16", seed=8)
    h = S.srnl_ln_create(dict(dim=dim, act_dtype="bf16"))
    try:
        y, mean, rstd = forward(h, t)
        outs = [(torch.empty_like(y), torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")) for _ in range(3)]

        def back(o, stream=None):
            S.srnl_ln_backward(h, t["x"], t["dy"], t["gamma"], mean, rstd, o[0], o[1], o[2], dres=t["dres"], stream=stream)

        back(outs[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        back(outs[1], side)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.srnl_ln_forward(h, t["x"], t["gamma"], t["beta"], y, mean, rstd)
            back(outs[2])
        y_eager = y.clone()
        for o in outs[2]:
            o.zero_()
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), y_eager.view(torch.int16))
        for o in outs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
        del g
    finally:
        h.close()


def test_refusals():
    h = S.srnl_ln_create(dict(dim=64, act_dtype="bf16"))
    try:
        x = torch.zeros(5, 64, device="cuda", dtype=torch.bfloat16)
        y, g = torch.empty_like(x), torch.ones(64, device="cuda")

        def refused(text, **kw):
            a = dict(x=x, gamma=g, beta=g, y=y, mean=None, rstd=None)
            a.update(kw)
            with pytest.raises(S.SrnlError) as e:
                S.srnl_ln_forward(h, **a)
            assert e.value.status == S.SRNL_E_INVAL and text in str(e.value)

        refused("y must be", y=torch.empty(4, 64, device="cuda", dtype=torch.bfloat16))
        refused("x must be", x=x.float())
        refused("gamma must be", gamma=g.double())
        refused("x must be", x=torch.zeros(5, 128, device="cuda", dtype=torch.bfloat16)[:, ::2])
        refused("beta must be", beta=torch.ones(64))
        refused("overlaps", y=x)
        buf = torch.zeros(5 * 64 + 8, device="cuda", dtype=torch.bfloat16)
        refused("aligned", x=buf[1:321].view(5, 64))
        refused("aligned", gamma=torch.ones(65, device="cuda")[1:])
        refused("overlap", mean=torch.zeros(5, device="cuda"), rstd=y.view(torch.float32).view(-1)[:5])
        st = torch.zeros(5, device="cuda")
        with pytest.raises(S.SrnlError) as e:
            S.srnl_ln_backward(h, x, x, g, st, st, x)
        assert e.value.status == S.SRNL_E_INVAL and "overlaps" in str(e.value)
        h.close()
        with pytest.raises(RuntimeError):
            S.srnl_ln_forward(h, x, g, g, y)
    finally:
        h.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_odd_rows_whose_weights_just_fill_a_block(dtype):
    """Odd rows keep gamma and beta in shared memory: 48 KB and a little less or more of them, in a process of its own,
    so that no handle of longer rows has raised the kernels' limit before."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = f"""
import numpy as np, torch, sys
sys.path[:0] = [{here!r}, {os.path.dirname(here)!r}]
import self_referential_nested_b200 as S
from test_gpu_norm import DT, U, forward, make, reference
for dim in (6091, 6095, 6097, 6101, 6113, 6121, 6127, 6129, 6135):
    t = make(5, dim, {dtype!r}, seed=dim)
    h = S.srnl_ln_create(dict(dim=dim, act_dtype={dtype!r}))
    y, mean, rstd = forward(h, t)
    ref = reference(t, float(np.float32(1e-6)))[0]
    # a rounding of the output, and fp32 sums and products a hundred steps long
    assert float((y.double() - ref).norm()) <= (torch.finfo(DT[{dtype!r}]).eps / 2 + 100 * U) * float(ref.norm()), dim
    dx = torch.full_like(y, float("nan"))
    S.srnl_ln_backward(h, t["x"], t["dy"], t["gamma"], mean, rstd, dx)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(dx).all())
    h.close()
"""
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [3, 20, 33, 100, 301, 1000, 1533, 2052, 2500, 8191])
def test_backward_of_a_row_far_from_zero(dim, dtype):
    """A constant row of 1e36 with 1 / sqrt(eps) as its rstd: x - mean is zero, mean rstd beyond fp32.  No column outside
    the row, on a lane with nothing to do or in a unit shared with a neighbour, enters its sums."""
    t = make(6, dim, dtype, seed=dim)
    t["x"][2] = 1e36
    mean, rstd = t["x"].double().mean(1).float(), torch.ones(6, device="cuda")
    mean[2], rstd[2] = t["x"][2, 0].float(), 1000.0
    h = S.srnl_ln_create(dict(dim=dim, act_dtype=dtype))
    try:
        dx = torch.full_like(t["x"], float("nan"))
        dg, db = torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
        S.srnl_ln_backward(h, t["x"], t["dy"], t["gamma"], mean, rstd, dx, dg, db)
        torch.cuda.synchronize()
    finally:
        h.close()
    r64, dy = rstd.double()[:, None], t["dy"].double()
    xh = (t["x"].double() - mean.double()[:, None]) * r64
    w = dy * t["gamma"].double()
    ref = r64 * (w - w.mean(1, keepdim=True) - xh * (w * xh).mean(1, keepdim=True))
    half = torch.finfo(DT[dtype]).eps / 2
    # as for the shapes above
    big = r64 * (6 * w.abs() + 50 * w.abs().mean(1, keepdim=True) + 56 * xh.abs() * (w * xh).abs().mean(1, keepdim=True))
    assert bool(((dx.double() - ref).abs() <= half * ref.abs() + U * (big + 4 * ref.abs())).all())
    assert bool(((dg.double() - (dy * xh).sum(0)).abs() <= 200 * U * (dy * xh).abs().sum(0)).all())
    assert bool(((db.double() - dy.sum(0)).abs() <= 200 * U * dy.abs().sum(0)).all())


def test_transposed_rows_are_refused():
    h = S.srnl_ln_create(dict(dim=64, act_dtype="bf16"))
    try:
        x, g = torch.zeros(5, 64, device="cuda", dtype=torch.bfloat16), torch.ones(64, device="cuda")
        y, m = torch.empty_like(x), torch.zeros(5, device="cuda")
        other = torch.zeros(64, 5, device="cuda", dtype=torch.bfloat16)
        calls = [("x", lambda: S.srnl_ln_forward(h, other, g, g, y)), ("y", lambda: S.srnl_ln_forward(h, x, g, g, other)),
                 ("dy", lambda: S.srnl_ln_backward(h, x, other, g, m, m, y)), ("dx", lambda: S.srnl_ln_backward(h, x, x, g, m, m, other)),
                 ("dres", lambda: S.srnl_ln_backward(h, x, x, g, m, m, y, dres=other))]
        for name, call in calls:
            with pytest.raises(S.SrnlError) as e:
                call()
            assert e.value.status == S.SRNL_E_INVAL and f"{name} must be" in str(e.value)
        S.srnl_ln_forward(h, x.view(5, 1, 64), g, g, y.view(5, 8, 8))   # the same rows, told otherwise
        torch.cuda.synchronize()
    finally:
        h.close()
