"""The operators of include/moe_ops.h without a GPU: the library exports what the
header declares, bad arguments are refused before any launch, and the fp64
oracle's gradients agree with differences and with automatic differentiation."""
import ctypes
import math
import os
import re

import pytest
import torch

import sparse_moe_layer_renormalised_b200 as moe
from conftest import ROOT
from oracle import ops_oracle as oo

FAKE = 1 << 20  # an aligned address; never dereferenced because validation fails first
BAD, UNSUP = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
F64 = torch.float64


def test_library_exports_every_operator():
    src = open(os.path.join(ROOT, "include", "moe_ops.h")).read()
    names = re.findall(r"MOE_API\s+[\w\s\*]+?\b(moe_\w+)\s*\(", src)
    lib = ctypes.CDLL(moe.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    assert set(names) == set(moe.EXPORTED_OPS) and len(names) == len(set(names))


# ------------------------------------------------------------------------------ refusals
ROUTE = dict(T=4, E=64, k=8)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=1025), dict(k=0), dict(k=33, E=64), dict(k=9, E=8),
    dict(groups=0), dict(groups=3), dict(groups=64), dict(groups=8, keep_groups=0), dict(groups=8, keep_groups=9),
    dict(groups=16, keep_groups=1), dict(group_top=0), dict(group_top=3), dict(groups=32, E=32, k=4, group_top=2),
    dict(scale=math.inf), dict(scale=math.nan)])
def test_route_refuses_bad_descriptors(kw):
    d = moe.route_desc(**{**ROUTE, **kw})
    assert moe.moe_route(d, FAKE, FAKE, FAKE, FAKE, 0) == BAD
    assert moe.moe_route_backward(d, FAKE, FAKE, FAKE, FAKE, 0) == BAD


def test_route_refuses_bad_types_and_pointers():
    d = moe.route_desc(**ROUTE)
    d.dtype = 2  # MOE_MXFP4
    assert moe.moe_route(d, FAKE, None, FAKE, FAKE, 0) == BAD
    d = moe.route_desc(**ROUTE)
    d.score = 2
    assert moe.moe_route(d, FAKE, None, FAKE, FAKE, 0) == BAD
    d = moe.route_desc(**ROUTE)
    for i, args in enumerate([(None, None, FAKE, FAKE), (FAKE + 8, None, FAKE, FAKE), (FAKE, FAKE + 4, FAKE, FAKE),
                              (FAKE, None, None, FAKE), (FAKE, None, FAKE, FAKE + 4)]):
        assert moe.moe_route(d, *args, 0) == BAD, i
    for i, args in enumerate([(None, FAKE, FAKE, FAKE), (FAKE, None, FAKE, FAKE), (FAKE, FAKE, FAKE + 4, FAKE),
                              (FAKE, FAKE, FAKE, None)]):
        assert moe.moe_route_backward(d, *args, 0) == BAD, i
    empty = moe.route_desc(**{**ROUTE, "T": 0})
    assert moe.moe_route(empty, None, None, None, None, 0) == moe.MOE_OK
    assert moe.moe_route_backward(empty, None, None, None, None, 0) == moe.MOE_OK


def test_norm_refuses():
    ok = dict(T=4, H=64)
    for kw in (dict(T=-1), dict(H=0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(T=1 << 31)):
        d = moe.norm_desc(**{**ok, **kw})
        assert moe.moe_norm(d, FAKE, None, None, FAKE, None, None, 0) == BAD, kw
        assert moe.moe_norm_backward_workspace_size(d) == 0
        assert moe.moe_norm_backward(d, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, 0) == BAD
    d = moe.norm_desc(4, 16385)
    assert moe.moe_norm(d, FAKE, None, None, FAKE, None, None, 0) == UNSUP
    assert moe.moe_norm_backward(d, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, 0) == UNSUP
    d = moe.norm_desc(4, 64)
    assert moe.moe_norm(d, None, None, None, FAKE, None, None, 0) == BAD
    assert moe.moe_norm(d, FAKE, FAKE + 4, None, FAKE, None, None, 0) == BAD
    assert moe.moe_norm(d, FAKE, None, None, FAKE + 2, None, None, 0) == BAD
    rms = moe.norm_desc(4, 64, kind="rms")
    assert moe.moe_norm(rms, FAKE, None, None, FAKE, FAKE, FAKE, 0) == BAD  # no mean to give
    n = moe.moe_norm_backward_workspace_size(d)
    assert n > 0
    good = [FAKE] * 8
    for i in (0, 1, 3, 4, 5):  # dy, x, mean, rstd, dx
        args = list(good)
        args[i] = None
        assert moe.moe_norm_backward(d, *args, FAKE, n, 0) == BAD, i
    assert moe.moe_norm_backward(d, *good, FAKE, n - 1, 0) == BAD
    assert moe.moe_norm_backward(d, *good, FAKE + 16, n, 0) == BAD
    assert moe.moe_norm_backward(d, *good, None, n, 0) == BAD
    assert moe.moe_norm_backward(rms, *good, FAKE, n, 0) == BAD  # a mean with RMS norm
    assert moe.moe_norm(moe.norm_desc(0, 64), None, None, None, None, None, None, 0) == moe.MOE_OK


def test_linear_refuses():
    ok = dict(M=4, N=64, K=64)
    ptrs = [FAKE, FAKE, None, None, None, FAKE]
    for kw, st in ((dict(M=-1), BAD), (dict(N=0), BAD), (dict(K=0), BAD), (dict(M=1 << 31), BAD), (dict(N=63), UNSUP),
                   (dict(K=12), UNSUP), (dict(dtype="f32"), UNSUP), (dict(dtype="bf16", y_out="f16"), BAD)):
        d = moe.linear_desc(**{**ok, **kw})
        assert moe.moe_linear(d, *ptrs, None, None, 0) == st, kw
        assert moe.moe_linear_backward_workspace_size(d) == 0, kw
        assert moe.moe_linear_backward(d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, 0) == st, kw
    d = moe.linear_desc(**ok)
    for act in (-1, 5):
        d.act = act
        assert moe.moe_linear(d, *ptrs, None, None, 0) == BAD
    d = moe.linear_desc(**ok, act="silu")
    for i, v in ((0, None), (1, None), (5, None), (0, FAKE + 8), (2, FAKE + 4), (3, FAKE + 2), (4, FAKE + 8)):
        bad = list(ptrs)
        bad[i] = v
        assert moe.moe_linear(d, *bad, None, None, 0) == BAD, (i, v)
    n = moe.moe_linear_backward_workspace_size(d)
    good = [FAKE] * 7
    for i in (0, 1, 2, 3):  # dy, pre, x, weight
        bad = list(good)
        bad[i] = None
        assert moe.moe_linear_backward(d, *bad, FAKE, n, 0) == BAD, i
    assert moe.moe_linear_backward(d, *good, FAKE, n - 1, 0) == BAD
    assert moe.moe_linear_backward(d, *good, FAKE + 16, n, 0) == BAD
    assert moe.moe_linear_backward(d, *good, None, n, 0) == BAD
    big = moe.linear_desc(4096, 4096, 64)
    n = moe.moe_linear_workspace_size(big)
    assert n > 0 and moe.moe_linear_workspace_size(d) == 0
    for ws, size in ((None, n), (FAKE, n - 1), (FAKE + 16, n)):
        assert moe.moe_linear(big, *ptrs, ws, size, 0) == BAD
    assert moe.moe_linear(moe.linear_desc(0, 64, 64), None, None, None, None, None, None, None, None, 0) == moe.MOE_OK


def test_clip_refuses():
    t = [torch.zeros(5), torch.zeros(3, dtype=torch.bfloat16)]
    lst = moe.tensor_list(t)
    n = moe.moe_clip_grads_workspace_size(lst)
    assert n > 0
    for bad in (-1.0, math.inf, math.nan):
        assert moe.moe_clip_grads(lst, "l2", bad, FAKE, FAKE, n, 0) == BAD
    assert moe.moe_clip_grads(lst, "l2", 1.0, None, FAKE, n, 0) == BAD
    assert moe.moe_clip_grads(lst, "l2", 1.0, FAKE + 2, FAKE, n, 0) == BAD
    assert moe.moe_clip_grads(lst, "l2", 1.0, FAKE, FAKE, n - 1, 0) == BAD
    assert moe.moe_clip_grads(lst, "l2", 1.0, FAKE, FAKE + 8, n, 0) == BAD
    for field, value in (("in_", 0), ("out", 0), ("n", -1), ("dtype", 3), ("in_", FAKE + 2), ("out", FAKE + 1)):
        lst = moe.tensor_list(t)
        setattr(lst.array[0], field, value)
        assert moe.moe_clip_grads(lst, "l2", 1.0, FAKE, FAKE, n, 0) == BAD, field
        assert moe.moe_clip_grads_workspace_size(lst) == 0
    with pytest.raises(ValueError):
        moe.tensor_list([torch.zeros(3)], [torch.zeros(4)])
    with pytest.raises(ValueError):
        moe.tensor_list([torch.zeros(3)], [torch.zeros(3, dtype=torch.float16)])
    with pytest.raises(ValueError):
        moe.tensor_list([torch.zeros(3, dtype=torch.int32)])
    with pytest.raises(ValueError):
        moe.tensor_list([torch.zeros(4, 4).t()])


# ------------------------------------------------------------------------------ the oracle itself
def _differences(f, x, h=1e-6):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        a, b = x.clone(), x.clone()
        a.view(-1)[i] += h
        b.view(-1)[i] -= h
        g.view(-1)[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_oracle_route_gradient_against_differences(score, renorm):
    g = torch.Generator().manual_seed(3)
    l = torch.randn(3, 7, generator=g, dtype=F64)
    idx, w = oo.route(l, None, 3, score=score, renorm=renorm, scale=1.7)
    dw = torch.randn(3, 3, generator=g, dtype=F64)
    assert torch.allclose(w, oo.route_weights(l, idx, score, renorm, 1.7))
    want = _differences(lambda x: (oo.route_weights(x, idx, score, renorm, 1.7) * dw).sum(), l)
    got = oo.route_backward(l, idx, dw, score, renorm, 1.7)
    assert (got - want).abs().max() < 1e-8
    x = l.clone().requires_grad_(True)
    auto, = torch.autograd.grad((oo.route_weights(x, idx, score, renorm, 1.7) * dw).sum(), x)
    assert (got - auto).abs().max() < 1e-13


def test_oracle_route_by_hand():
    l = torch.tensor([[1.0, 3.0, 2.0, 3.0, -math.inf, math.nan, 0.0, 0.5]])
    idx, w = oo.route(l, None, 8, score="softmax")
    assert idx.tolist() == [[1, 3, 2, 0, 7, 6, 4, 5]]
    assert w[0, 6] == 0 and w[0, 7] == 0 and abs(float(w.sum()) - 1) < 1e-12
    # two groups of four: sums of the best two are 6 and 0.5 + 0 (masked ones do not count)
    idx, _ = oo.route(l, None, 2, groups=2, keep=1, group_top=2, score="sigmoid")
    assert idx.tolist() == [[1, 3]]
    idx, w = oo.route(torch.full((1, 4), -math.inf), None, 2, score="softmax")
    assert idx.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_oracle_norm_gradients(kind):
    g = torch.Generator().manual_seed(5)
    x, dy = torch.randn(4, 9, generator=g, dtype=F64), torch.randn(4, 9, generator=g, dtype=F64)
    gamma, beta = torch.randn(9, generator=g, dtype=F64), torch.randn(9, generator=g, dtype=F64)
    y, mean, rstd = oo.norm(x, gamma, beta, 1e-5, kind)
    dx, dgamma, dbeta = oo.norm_backward(dy, x, gamma, mean, rstd, kind)
    assert (dx - _differences(lambda v: (oo.norm(v, gamma, beta, 1e-5, kind)[0] * dy).sum(), x)).abs().max() < 1e-7
    assert (dgamma - _differences(lambda v: (oo.norm(x, v, beta, 1e-5, kind)[0] * dy).sum(), gamma)).abs().max() < 1e-7
    assert (dbeta - _differences(lambda v: (oo.norm(x, gamma, v, 1e-5, kind)[0] * dy).sum(), beta)).abs().max() < 1e-7
    if kind == "layer":
        ref = torch.nn.functional.layer_norm(x, (9,), gamma, beta, 1e-5)
        assert (y - ref).abs().max() < 1e-12


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_oracle_linear_gradients(kind):
    g = torch.Generator().manual_seed(6)
    x, w = torch.randn(4, 6, generator=g, dtype=F64), torch.randn(5, 6, generator=g, dtype=F64)
    b, dy = torch.randn(5, generator=g, dtype=F64), torch.randn(4, 5, generator=g, dtype=F64)
    pre, _ = oo.linear(x, w, b, None, kind)
    _, dx, dw, db = oo.linear_backward(dy, pre, x, w, kind)
    loss = lambda x, w, b: (oo.linear(x, w, b, None, kind)[1] * dy).sum()  # noqa: E731
    assert (dx - _differences(lambda v: loss(v, w, b), x)).abs().max() < 1e-7
    assert (dw - _differences(lambda v: loss(x, v, b), w)).abs().max() < 1e-7
    assert (db - _differences(lambda v: loss(x, w, v), b)).abs().max() < 1e-7


def test_oracle_clip():
    norm, out = oo.clip([torch.tensor([3.0, 0.0]), torch.tensor([4.0])], 1.0)
    assert norm == 5.0 and abs(float(out[1][0]) - 0.8) < 1e-6
    norm, out = oo.clip([torch.tensor([3.0]), torch.tensor([math.inf])], 1.0)
    assert norm == math.inf and float(out[0][0]) == 3.0
    assert oo.clip([torch.tensor([3.0, -7.0])], 100.0, "max")[0] == 7.0
