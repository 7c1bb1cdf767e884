"""moe_linear and moe_linear_backward against the fp64 oracle."""
import math

import pytest
import torch

import sparse_moe_layer_renormalised_b200 as moe
from ops_util import DT, HALF, TINY, Guarded, within, workspace
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
# the smallest, one tile and its ragged edges, few rows with a split sum, and large enough for the wide tiles
SHAPES = [(1, 8, 8), (3, 16, 40), (5, 72, 136), (16, 128, 64), (17, 256, 200), (1, 1000, 3584), (4, 7168, 512), (33, 136, 1000),
          (64, 512, 512), (65, 384, 72), (128, 1032, 264), (129, 640, 264), (200, 1000, 328), (256, 2048, 512),
          (1111, 2048, 1024), (2049, 2312, 520), (4100, 3592, 136), (300, 8200, 1032), (520, 2304, 2112), (2048, 7168, 640), (2304, 8456, 1096)]


def _accumulation(R):
    """Error of an fp32 sum of R exact products in steps of 16, each step cut at 2^-23 of the terms' magnitudes."""
    return (R / 16 + 32) * 2.0 ** -23


def _data(M, N, K, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return r(M, K).to(DT[dtype]), (r(N, K) * K ** -0.5).to(DT[dtype]), r(N) * 0.2, r(M, N)


def _linear(d, *args):
    return moe.moe_linear(d, *args, workspace(moe.moe_linear_workspace_size(d)))


def _check(M, N, K, dtype, act, y_out=None, bias=True, residual=True, pre=True, inplace=False):
    y_out = y_out or dtype
    x, w, b, res = _data(M, N, K, dtype, M + 3 * N + K)
    g = Guarded()
    xd, wd = g.new((M, K), DT[dtype], x), g.new((N, K), DT[dtype], w)
    bd = g.new((N,), torch.float32, b) if bias else None
    res = res.to(DT[y_out])
    rd = g.new((M, N), DT[y_out], res) if residual else None
    pd = g.new((M, N), DT[dtype]) if pre else None
    y = rd if inplace else g.new((M, N), DT[y_out])
    d = moe.linear_desc(M, N, K, act, dtype, y_out)
    assert _linear(d, xd, wd, bd, rd, pd, y) == moe.MOE_OK
    g.check()
    want_pre, want = oo.linear(x, w, b if bias else None, res if residual else None, act)
    size = x.double().abs() @ w.double().abs().T
    err = _accumulation(K) * size + 2.0 ** -23 * want_pre.abs()
    what = f"{act} {M}x{N}x{K} {dtype}"
    if pre:
        within(pd, want_pre.cpu(), (err + want_pre.abs() * HALF[dtype] + TINY[dtype]).cpu(), "pre " + what)
    # no activation is steeper than 1.13; its evaluation: 2^-19 of the argument for |a| to about 10
    tol = 1.13 * err + (0.0 if act in ("none", "relu") else 2.0 ** -19 * (want_pre.abs() + 1.0))
    tol = tol + want.abs() * (HALF[y_out] + 2.0 ** -23) + TINY[y_out] + (res.double().abs() * 2.0 ** -23 if residual else 0.0)
    within(y, want.cpu(), tol.cpu(), "y " + what)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(dtype, M, N, K):
    _check(M, N, K, dtype, ACTS[(M + N + K) % 5])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(7, 264, 128), (1200, 2048, 192)])
def test_activations_types_and_options(act, M, N, K):
    for dtype in ("bf16", "f16"):
        _check(M, N, K, dtype, act, y_out="f32", pre=False)
        _check(M, N, K, dtype, act, bias=False, residual=False)
        _check(M, N, K, dtype, act, residual=True, inplace=True, pre=False)


def test_f32_outputs_keep_fp32_accuracy():
    """Router logits: fp32 out of bf16 operands."""
    for M in (64, 2048):
        _check(M, 896, 7168, "bf16", "none", y_out="f32", bias=False, residual=False, pre=False)


def test_non_finite_rows_stay_alone():
    M, N, K = 40, 256, 512
    x, w, b, _ = _data(M, N, K, "bf16", 1)
    x[3, 100] = math.inf
    x[9, 5] = math.nan
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    assert _linear(moe.linear_desc(M, N, K), x, w, None, None, None, y) == moe.MOE_OK
    bad = ~torch.isfinite(y).all(1).cpu()
    assert bad.nonzero().view(-1).tolist() == [3, 9]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ACTS)
def test_activations_far_out(act, dtype):
    """Pre-activations from 0 to the type's largest, and the slopes there."""
    big = 6e4 if dtype == "f16" else 1e30
    v = torch.tensor([0.0, 1e-4, 0.5, 3.0, 8.0, 12.0, 20.0, 88.0, 89.0, 100.0, 104.0, 1000.0, big, -0.0, -1e-4, -0.5, -3.0,
                      -8.0, -12.0, -20.0, -88.0, -89.0, -100.0, -104.0, -1000.0, -big]).to(DT[dtype])
    n, N = v.numel(), 64
    x, eye = torch.zeros(n, N, dtype=DT[dtype]), torch.eye(N).to(DT[dtype])
    x[torch.arange(n), torch.arange(n)] = v
    for rows in (n, 2600):  # a few rows, and enough for the wide tiles (of a wider product)
        cols = N if rows == n else 1024
        w = torch.zeros(cols, N, dtype=DT[dtype])
        w[:N] = eye
        xx = x.repeat(-(-rows // n), 1)[:rows].contiguous()
        y = torch.empty(rows, cols, dtype=DT[dtype], device="cuda")
        pre = torch.empty_like(y)
        assert _linear(moe.linear_desc(rows, cols, N, act, dtype), xx.cuda(), w.cuda(), None, None, pre, y) == moe.MOE_OK
        at = torch.arange(rows), torch.arange(rows) % n
        want = oo.act(xx[at].double(), act)
        tol = want.abs() * (HALF[dtype] + 2.0 ** -18) + 2.0 ** -19 * xx[at].double().abs().clamp_max(30.0) + TINY[dtype]
        within(y[at], want, tol, act)
        # the slope: dW of a product with one row of ones is dp itself
    dy = torch.ones(1, n, dtype=DT[dtype])
    d = moe.linear_desc(1, -(-n // 8) * 8, 8, act, dtype)
    pad = d.N - n
    p1 = torch.cat([v, torch.zeros(pad, dtype=DT[dtype])]).view(1, -1)
    dy = torch.ones(1, d.N, dtype=DT[dtype])
    db = torch.empty(d.N, device="cuda")
    ws = workspace(moe.moe_linear_backward_workspace_size(d))
    assert moe.moe_linear_backward(d, dy.cuda(), p1.cuda(), None, None, None, None, db, ws) == moe.MOE_OK
    want = oo.act_grad(p1[0].double().clamp(-1e3, 1e3), act) if act != "none" else torch.ones(d.N, dtype=torch.float64)
    within(db, want, 2.0 ** -18 * torch.ones_like(want) * (1.0 + p1[0].double().abs().clamp_max(10.0)), act + "'")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_keep_small_values(act, dtype):
    """fp32 outputs of activations far on the negative side, where they are small: relative errors."""
    v = torch.cat([torch.linspace(-9, 9, 577), torch.linspace(-12.5, -9, 63)]).to(DT[dtype])
    v = v[v != 0]
    for rows, cols in ((32, 64), (2600, 1024)):  # a few rows, and enough for the wide tiles
        g = torch.Generator().manual_seed(rows)
        x = torch.zeros(rows, 64, dtype=DT[dtype])
        at = torch.randint(0, v.numel(), (rows, 64), generator=g)
        x[:] = v[at]
        w = torch.zeros(cols, 64, dtype=DT[dtype])
        w[:64] = torch.eye(64).to(DT[dtype])
        y = torch.empty(rows, cols, device="cuda")
        assert _linear(moe.linear_desc(rows, cols, 64, act, dtype, "f32"), x.cuda(), w.cuda(), None, None, None, y) == moe.MOE_OK
        a = x.double()
        want = {"silu": lambda: a * torch.sigmoid(a), "gelu": lambda: 0.5 * a * torch.erfc(-a / math.sqrt(2.0)),
                "gelu_tanh": lambda: a * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))}[act]()
        arg = {"silu": a.abs(), "gelu": a * a / 2, "gelu_tanh": 2 * math.sqrt(2 / math.pi) * (a.abs() + 0.044715 * a.abs() ** 3)}[act]
        # a sigmoid or an exponential below 2^-126 is 0: the value a sigmoid(.), or at most |a| e^(-a^2 / 2) / 2, then
        # loses up to |a| 2^-126
        within(y[:, :64], want, want.abs() * (2.0 ** -19 + 2.0 ** -21 * arg) + a.abs() * 2.0 ** -126, act)


def _check_backward(M, N, K, dtype, act, need=(True, True, True)):
    x, w, b, dy = _data(M, N, K, dtype, M + N + 7 * K)
    dy = dy.to(DT[dtype])
    pre = oo.linear(x, w, b, None, act)[0].to(DT[dtype])
    g = Guarded()
    xd, wd = g.new((M, K), DT[dtype], x), g.new((N, K), DT[dtype], w)
    pd, dyd = g.new((M, N), DT[dtype], pre), g.new((M, N), DT[dtype], dy)
    dx = g.new((M, K), DT[dtype]) if need[0] else None
    dw = g.new((N, K), DT[dtype]) if need[1] else None
    db = g.new((N,), torch.float32) if need[2] else None
    d = moe.linear_desc(M, N, K, act, dtype)
    ws = workspace(moe.moe_linear_backward_workspace_size(d))
    st = moe.moe_linear_backward(d, dyd, pd if act != "none" else None, xd if need[1] else None, wd if need[0] else None,
                                 dx, dw, db, ws)
    assert st == moe.MOE_OK
    g.check()
    dp, wdx, wdw, wdb = oo.linear_backward(dy, pre, x, w, act)
    # dp: its evaluation, and one rounding as the products' operand (none without an activation)
    ev = 0.0 * dp if act in ("none", "relu") else 2.0 ** -19 * dy.double().abs() * (1.0 + pre.double().abs())
    edp = ev + (0.0 if act == "none" else dp.abs() * HALF[dtype] + TINY[dtype])
    what = f"{act} {M}x{N}x{K} {dtype}"
    for got, want, other, R, name in ((dx, wdx, lambda e: e @ w.double().abs(), N, "dx"),
                                      (dw, wdw, lambda e: e.T @ x.double().abs(), M, "dweight")):
        if got is None:
            continue
        tol = other(edp) + _accumulation(R) * other(dp.abs()) + want.abs() * HALF[dtype] + TINY[dtype]
        within(got, want.cpu(), tol.cpu(), f"{name} {what}")
        # two independent roundings of rms at most HALF / sqrt 3 each: 0.82 HALF of the result
        # (f16 with subnormal outputs or operands aside)
        if dtype == "bf16" and want.numel() > 1000:
            rel = float((got.double() - want).norm() / want.norm())
            assert rel <= HALF[dtype], f"{name} {what}: {rel:.3g}"
    if db is not None:
        steps = (M / 148 + 64) * 2.0 ** -24
        within(db, wdb.cpu(), (steps * dp.abs().sum(0) + (0.0 if act == "none" else ev.sum(0)) + 1e-37).cpu(), "dbias " + what)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_backward(dtype, M, N, K):
    _check_backward(M, N, K, dtype, ACTS[(M + N + K + 1) % 5])


@pytest.mark.parametrize("act", ACTS)
def test_backward_activations_and_optional_outputs(act):
    for need in ((True, True, True), (True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        _check_backward(77, 264, 136, "bf16", act, need)
    _check_backward(2500, 2304, 2056, "bf16", act)


def test_backward_of_no_rows_writes_zeros():
    d = moe.linear_desc(0, 64, 128, "silu")
    ws = workspace(moe.moe_linear_backward_workspace_size(d))
    dw, db = torch.full((64, 128), math.nan, dtype=torch.bfloat16, device="cuda"), torch.full((64,), math.nan, device="cuda")
    assert moe.moe_linear_backward(d, None, None, None, None, None, dw, db, ws) == moe.MOE_OK
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_gradients_against_differences():
    """The library's own forward pass, perturbed: d loss / d x and d W along random directions."""
    M, N, K = 48, 256, 128
    g = torch.Generator().manual_seed(12)
    # values on a coarse grid and steps that bf16 holds exactly; fp32 outputs
    x = (torch.randint(-8, 9, (M, K), generator=g) / 8).bfloat16().cuda()
    w = (torch.randint(-8, 9, (N, K), generator=g) / 32).bfloat16().cuda()
    dy = (torch.randint(-4, 5, (M, N), generator=g) / 4).bfloat16().cuda()
    d32 = moe.linear_desc(M, N, K, "silu", "bf16", "f32")

    def loss(x, w):
        y = torch.empty(M, N, device="cuda")
        assert _linear(d32, x, w, None, None, None, y) == moe.MOE_OK
        return float((y.double() * dy.double()).sum())

    pre = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    y = torch.empty(M, N, device="cuda")
    assert _linear(d32, x, w, None, None, pre, y) == moe.MOE_OK
    d = moe.linear_desc(M, N, K, "silu")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = workspace(moe.moe_linear_backward_workspace_size(d))
    assert moe.moe_linear_backward(d, dy, pre, x, w, dx, dw, None, ws) == moe.MOE_OK
    h = 2.0 ** -6
    for t, grad, f in ((x, dx, lambda v: loss(v, w)), (w, dw, lambda v: loss(x, v))):
        step = (torch.randint(0, 2, t.shape, generator=g) * 2 - 1).bfloat16().cuda() * h
        up, down = (t.float() + step.float()).bfloat16(), (t.float() - step.float()).bfloat16()
        diff = (f(up) - f(down)) / 2
        want = float((grad.double() * step.double()).sum())
        # bf16 roundings of pre (2^-8 of about 1 into act'), dp and the gradient: each at most 2^-8 of every term,
        # independent: their sum over n terms grows as sqrt n; a third derivative below 1 leaves a cubic term
        scale = float((grad.double() * step.double()).norm())
        cubic = float((dy.double().abs().sum())) * (h * K ** 0.5) ** 3 / 6
        assert abs(diff - want) <= 5 * scale * 3 * 2.0 ** -8 + cubic, (diff, want, scale, cubic)


def test_deterministic():
    for M in (5, 3000):
        x, w, b, res = _data(M, 2048, 2048, "bf16", 3)
        res = res.bfloat16()
        outs = []
        for _ in range(3):
            y = torch.empty(M, 2048, dtype=torch.bfloat16, device="cuda")
            assert _linear(moe.linear_desc(M, 2048, 2048, "gelu"), x, w, b, res, None, y) == moe.MOE_OK
            outs.append(y.cpu())
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_offsets_past_32_bits():
    """More than 2^32 elements of y, pre, dy and dp: the last rows and columns come out as the formulas give them."""
    M, N, K = 66000, 66048, 64
    x, w, b, _ = _data(M, 64, K, "bf16", 1)
    w = (torch.randn(N, K, device="cuda") * K ** -0.5).bfloat16()
    b = torch.randn(N, device="cuda") * 0.2
    d = moe.linear_desc(M, N, K, "silu")
    y, pre = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert _linear(d, x, w, b, None, pre, y) == moe.MOE_OK
    rows, cols = slice(M - 5, M), slice(N - 72, N)
    want_pre, want = oo.linear(x[rows], w[cols], b[cols], None, "silu")
    err = _accumulation(K) * (x[rows].double().abs() @ w[cols].double().abs().T) + 2.0 ** -23 * want_pre.abs()
    within(pre[rows, cols], want_pre.cpu(), (err + want_pre.abs() * HALF["bf16"] + TINY["bf16"]).cpu(), "pre")
    tol = 1.13 * err + 2.0 ** -19 * (want_pre.abs() + 1.0) + want.abs() * (HALF["bf16"] + 2.0 ** -23) + TINY["bf16"]
    within(y[rows, cols], want.cpu(), tol.cpu(), "y")
    # gradients: dy is y; the last row of dx, and the last rows of dW by all of dp
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = workspace(moe.moe_linear_backward_workspace_size(d))
    assert moe.moe_linear_backward(d, y, pre, x, w, dx, dw, db, ws) == moe.MOE_OK
    assert moe.moe_device_error() == (moe.MOE_OK, 0)
    last = slice(M - 1, M)
    _, wdx, _, _ = oo.linear_backward(y[last], pre[last], x[last], w, "silu")
    dp = (y[last].double() * oo.act_grad(pre[last], "silu")).abs()
    edp = 2.0 ** -19 * y[last].double().abs() * (1.0 + pre[last].double().abs()) + dp * HALF["bf16"] + TINY["bf16"]
    tol = (edp + _accumulation(N) * dp) @ w.double().abs() + wdx.abs() * HALF["bf16"] + TINY["bf16"]
    within(dx[last], wdx.cpu(), tol.cpu(), "dx")
    _, _, wdw, wdb = oo.linear_backward(y[:, cols].contiguous(), pre[:, cols].contiguous(), x, w[cols], "silu")
    dp = (y[:, cols].double() * oo.act_grad(pre[:, cols], "silu")).abs()
    ev = 2.0 ** -19 * y[:, cols].double().abs() * (1.0 + pre[:, cols].double().abs())
    tol = (ev + dp * HALF["bf16"] + TINY["bf16"] + _accumulation(M) * dp).T @ x.double().abs() + wdw.abs() * HALF["bf16"] + TINY["bf16"]
    within(dw[cols], wdw.cpu(), tol.cpu(), "dweight")
    within(db[cols], wdb.cpu(), ((M / 148 + 64) * 2.0 ** -24 * dp.sum(0) + ev.sum(0) + 1e-37).cpu(), "dbias")
