"""moe_norm and moe_norm_backward against the fp64 oracle."""
import math

import pytest
import torch

import sparse_moe_layer_renormalised_b200 as moe
from ops_util import DT, HALF, TINY, Guarded, within, workspace
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu

# A row sum runs over at most 64 values in a thread, 5 steps in a warp and 5 over the warps, each step 2^-24 of
# the sum of magnitudes; with the products' own roundings under 100 steps.
A = 100 * 2.0 ** -24
SHAPES = [(1, 1), (3, 2), (2, 7), (5, 31), (4, 32), (9, 33), (7, 64), (130, 128), (3, 129), (2, 200), (33, 256), (6, 257),
          (5, 1000), (4, 1024), (3, 1025), (3, 1032), (64, 2048), (3, 3001), (2, 4100), (9, 5001), (300, 7168), (2, 8193),
          (3, 8200), (2, 16383), (5, 16384)]


def _data(T, H, dtype, seed, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H, generator=g) * 1.7 + offset).to(DT[dtype])
    gamma = 1.0 + 0.2 * torch.randn(H, generator=g)
    beta = 0.3 * torch.randn(H, generator=g)
    dy = torch.randn(T, H, generator=g).to(DT[dtype])
    return x, gamma, beta, dy


def _check(x, gamma, beta, dtype, kind, eps=1e-6, stats=True, inplace=False):
    T, H = x.shape
    g = Guarded()
    xd = g.new((T, H), DT[dtype], x)
    gd = None if gamma is None else g.new((H,), torch.float32, gamma)
    bd = None if beta is None else g.new((H,), torch.float32, beta)
    y = xd if inplace else g.new((T, H), DT[dtype])
    mean = g.new((T,), torch.float32) if stats and kind == "layer" else None
    rstd = g.new((T,), torch.float32) if stats else None
    assert moe.moe_norm(moe.norm_desc(T, H, kind, eps, dtype), xd, gd, bd, y, mean, rstd) == moe.MOE_OK
    g.check()
    want, m, r = oo.norm(x, gamma, beta, eps, kind)
    size = x.double().abs().mean(1, keepdim=True)  # what a mean's error is relative to
    off = A * size * r[:, None]                    # of a normalised value, by the mean
    xh = (x.double() - m[:, None]) * r[:, None]
    gm = 1.0 if gamma is None else gamma.double().abs()
    tol = gm * (A * xh.abs() + off + (x.double().abs() * r[:, None]) * 2.0 ** -23) + want.abs() * (HALF[dtype] + 2.0 ** -22) + TINY[dtype]
    if beta is not None:
        tol = tol + beta.double().abs() * 2.0 ** -23
    within(y, want, tol, f"y {kind} {T}x{H}")
    if stats:
        if kind == "layer":
            within(mean, m, A * size[:, 0] + 1e-37, "mean")
        within(rstd, r, r * (A + off[:, 0] ** 2 + 2.0 ** -22), "rstd")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm(dtype, kind, T, H):
    x, gamma, beta, _ = _data(T, H, dtype, T + H)
    if H <= 2 and kind == "layer":
        x = x * 3  # (values apart)
    eps = 1e-6 if H > 8 else 1e-2  # short rows of nearly equal values: no blow-up of their rounding
    _check(x, gamma, beta if kind == "layer" else None, dtype, kind, eps)
    _check(x, None, None, dtype, kind, eps, stats=False, inplace=True)


def test_norm_beta_without_gamma_and_large_offset():
    """A mean far above the spread: the variance is that of the centred values."""
    x, gamma, beta, _ = _data(8, 1024, "f32", 3, offset=1000.0)
    _check(x, None, beta, "f32", "layer")
    _check(x, gamma, beta, "f32", "rms")


def test_norm_constant_and_zero_rows():
    x = torch.zeros(3, 96)
    x[1] = 5.0
    x[2, 0] = 1.0
    for kind in ("layer", "rms"):
        _check(x, torch.ones(96), None, "f32", kind, 1e-6)


def test_norm_non_finite_rows_stay_alone():
    x, gamma, beta, _ = _data(4, 520, "bf16", 5)
    x[1, 7] = math.inf
    x[2, 9] = math.nan
    y = torch.empty_like(x, device="cuda")
    assert moe.moe_norm(moe.norm_desc(4, 520, "layer"), x.cuda(), gamma.cuda(), beta.cuda(), y) == moe.MOE_OK
    want, _, _ = oo.norm(x[[0, 3]], gamma, beta, 1e-6)
    within(y[[0, 3]], want, want.abs() * 2.0 ** -8 + 1e-4)
    assert bool(torch.isnan(y[1]).any()) and bool(torch.isnan(y[2]).all())


def _check_backward(x, dy, gamma, dtype, kind, eps=1e-6, need=(True, True), alias=None):
    T, H = x.shape
    _, m, r = oo.norm(x, None, None, eps, kind)
    m, r = m.float(), r.float()
    g = Guarded()
    xd, dyd = g.new((T, H), DT[dtype], x), g.new((T, H), DT[dtype], dy)
    gd = None if gamma is None else g.new((H,), torch.float32, gamma)
    md, rd = g.new((T,), torch.float32, m), g.new((T,), torch.float32, r)
    dx = {None: None, "x": xd, "dy": dyd}[alias]
    dx = g.new((T, H), DT[dtype]) if dx is None else dx
    dgamma = g.new((H,), torch.float32) if need[0] else None
    dbeta = g.new((H,), torch.float32) if need[1] else None
    d = moe.norm_desc(T, H, kind, eps, dtype)
    ws = workspace(moe.moe_norm_backward_workspace_size(d))
    st = moe.moe_norm_backward(d, dyd, xd, gd, md if kind == "layer" else None, rd, dx, dgamma, dbeta, ws)
    assert st == moe.MOE_OK
    g.check()
    wdx, wdg, wdb = oo.norm_backward(dy, x, gamma, m, r, kind)
    r64 = r.double()[:, None]
    m64 = m.double()[:, None] if kind == "layer" else torch.zeros(T, 1, dtype=torch.float64)
    xh = ((x.double() - m64) * r64).abs()
    gg = (dy.double() * (1.0 if gamma is None else gamma.double())).abs()
    dxh = 2.0 ** -23 * ((x.double().abs() + m64.abs()) * r64 + xh)  # a normalised value's error
    s1, s2 = gg.mean(1, keepdim=True), (gg * xh).mean(1, keepdim=True)
    e2 = A * s2 + (gg * dxh).mean(1, keepdim=True)
    tol = r64 * (2.0 ** -22 * (gg + s1 + xh * s2) + A * s1 + xh * e2 + dxh * s2) + wdx.abs() * HALF[dtype] + TINY[dtype]
    within(dx, wdx, tol, f"dx {kind} {T}x{H}")
    # the rows of a block in a row, then the blocks' parts
    steps = (T / 148 + 64) * 2.0 ** -24
    if need[0]:
        within(dgamma, wdg, (dy.double().abs() * (steps * xh + dxh)).sum(0) + 1e-37, "dgamma")
    if need[1]:
        within(dbeta, wdb, steps * dy.double().abs().sum(0) + 1e-37, "dbeta")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T,H", SHAPES + [(1000, 96), (5000, 64), (777, 2056)])
def test_norm_backward(dtype, kind, T, H):
    x, gamma, _, dy = _data(T, H, dtype, 2 * T + H)
    _check_backward(x, dy, gamma, dtype, kind, 1e-6 if H > 8 else 1e-2)


@pytest.mark.parametrize("need", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("alias", ["x", "dy"])
def test_norm_backward_optional_outputs_and_in_place(need, alias):
    for H in (64, 2048, 3001):
        x, gamma, _, dy = _data(50, H, "bf16", H)
        _check_backward(x, dy, gamma if need[0] else None, "bf16", "layer", need=need, alias=alias)


def test_norm_backward_of_no_rows_writes_zeros():
    d = moe.norm_desc(0, 77)
    ws = workspace(moe.moe_norm_backward_workspace_size(d))
    dg, db = torch.full((77,), math.nan, device="cuda"), torch.full((77,), math.nan, device="cuda")
    assert moe.moe_norm_backward(d, None, None, None, None, None, None, dg, db, ws) == moe.MOE_OK
    assert bool((dg == 0).all()) and bool((db == 0).all())


def test_norm_backward_deterministic():
    x, gamma, _, dy = _data(700, 1536, "bf16", 4)
    d = moe.norm_desc(700, 1536, "rms")
    _, _, r = oo.norm(x, None, None, 1e-6, "rms")
    args = [t.cuda() for t in (dy, x, gamma, r.float())]
    res = []
    for _ in range(3):
        ws = workspace(moe.moe_norm_backward_workspace_size(d))
        dx, dg, db = torch.empty_like(args[1]), torch.empty(1536, device="cuda"), torch.empty(1536, device="cuda")
        assert moe.moe_norm_backward(d, args[0], args[1], args[2], None, args[3], dx, dg, db, ws) == moe.MOE_OK
        res.append((dx.cpu(), dg.cpu(), db.cpu()))
    for a in res[1:]:
        assert all(torch.equal(p, q) for p, q in zip(a, res[0]))


@pytest.mark.parametrize("offset", [10.0, 100.0, 1000.0])
@pytest.mark.parametrize("T,H", [(3, 96), (40, 1024), (700, 1536), (5, 1001), (700, 515)])
def test_norm_backward_of_rows_far_from_zero(T, H, offset):
    """fp32 rows whose mean is far above their spread: the mean is subtracted first, and no error grows with it."""
    x, gamma, _, dy = _data(T, H, "f32", H, offset)
    _, m, r = oo.norm(x, None, None, 1e-6, "layer")
    m, r = m.float(), r.float()
    r64 = r.double()[:, None]
    xh = (x.double() - m.double()[:, None]) * r64
    dy = (dy.double() * 0.3 + xh).float()  # along the rows: the sum of g xh counts in dx
    d = moe.norm_desc(T, H, "layer", 1e-6, "f32")
    dx, dgamma, dbeta = torch.empty(T, H, device="cuda"), torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    ws = workspace(moe.moe_norm_backward_workspace_size(d))
    args = [t.cuda() for t in (dy, x, gamma, m, r)]
    assert moe.moe_norm_backward(d, *args, dx, dgamma, dbeta, ws) == moe.MOE_OK
    assert moe.moe_device_error() == (moe.MOE_OK, 0)
    wdx, wdg, wdb = oo.norm_backward(dy, x, gamma, m, r, "layer")
    # from the given mean and rstd: a difference, a product, each off by 2^-24 of itself (twice that allowed)
    xh = xh.abs()
    dxh = 2.0 ** -22 * xh
    gg = (dy.double() * gamma.double()).abs()
    s1, s2 = gg.mean(1, keepdim=True), (gg * xh).mean(1, keepdim=True)
    e2 = A * s2 + (gg * dxh).mean(1, keepdim=True)
    tol = r64 * (2.0 ** -22 * (gg + s1 + xh * s2) + A * s1 + xh * e2 + dxh * s2) + wdx.abs() * HALF["f32"] + TINY["f32"]
    within(dx, wdx, tol, f"dx {T}x{H}")
    steps = (T / 148 + 64) * 2.0 ** -24
    within(dgamma, wdg, (dy.double().abs() * (steps * xh + dxh)).sum(0) + 1e-37, "dgamma")
    within(dbeta, wdb, steps * dy.double().abs().sum(0) + 1e-37, "dbeta")


# Many rows a group: rings that wrap, several groups a block, block counts cut to whole windows, parameters in
# shared memory; odd rows, whole windows and the longest ones.
MANY = [(4097, 5001), (3001, 257), (5000, 33), (149, 1031), (296, 4100), (700, 8193), (700, 16383), (5000, 64), (1200, 2048),
        (1500, 7168), (450, 16384)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T,H", MANY)
def test_norm_many_rows(dtype, kind, T, H):
    x, gamma, beta, _ = _data(T, H, dtype, T + 3 * H)
    _check(x, gamma, beta if kind == "layer" else None, dtype, kind)
    _check(x, gamma, None, dtype, kind, inplace=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T,H", MANY)
def test_norm_backward_many_rows(dtype, kind, T, H):
    x, gamma, _, dy = _data(T, H, dtype, 5 * T + H)
    _check_backward(x, dy, gamma, dtype, kind)
    _check_backward(x, dy, gamma, dtype, kind, need=(True, False), alias="x" if kind == "layer" else "dy")


def test_norm_offsets_past_32_bits():
    T, H = 160_000, 16384  # 5.2 GB of bf16
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda").normal_(0.1, 1.0)
    d = moe.norm_desc(T, H, "layer", 1e-6, "bf16")
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    y = torch.empty_like(x)
    assert moe.moe_norm(d, x, None, None, y, mean, rstd) == moe.MOE_OK
    tail = slice(T - 3, T)
    want, m, r = oo.norm(x[tail].cpu(), None, None, 1e-6)
    within(y[tail], want, want.abs() * 2.0 ** -8 + 1e-4)
    ws = workspace(moe.moe_norm_backward_workspace_size(d))
    dx = torch.empty_like(x)
    assert moe.moe_norm_backward(d, y, x, None, mean, rstd, dx, None, None, ws) == moe.MOE_OK
    wdx, _, _ = oo.norm_backward(y[tail].cpu(), x[tail].cpu(), None, m, r)
    within(dx[tail], wdx, wdx.abs() * 2.0 ** -7 + 1e-4)
