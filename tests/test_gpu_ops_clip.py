"""moe_clip_grads against the fp64 oracle."""
import math

import pytest
import torch

import sparse_moe_layer_renormalised_b200 as moe
from ops_util import DT, HALF, TINY, workspace, within
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
NAMES = {v: k for k, v in DT.items()}


def _run(grads, out, max_norm, kind="l2"):
    lst = moe.tensor_list(grads, out)
    norm = torch.full((1,), math.nan, device="cuda")
    ws = workspace(moe.moe_clip_grads_workspace_size(lst))
    assert moe.moe_clip_grads(lst, kind, max_norm, norm, ws) == moe.MOE_OK
    torch.cuda.synchronize()
    assert moe.moe_device_error() == (moe.MOE_OK, 0)
    return float(norm)


def _check(grads, max_norm, kind="l2"):
    """Out of place (the gradients stay) and in place."""
    host = [g.cpu() for g in grads]
    want_norm, want = oo.clip(host, max_norm, kind)
    out = [torch.full_like(g, 7.0) for g in grads]
    norm = _run(grads, out, max_norm, kind)
    # squares of a vector in fp32: at most 8 roundings of 2^-24, halved by the root; then one of the result
    rel = 8 * 2.0 ** -24
    if math.isfinite(want_norm):
        assert abs(norm - want_norm) <= rel * want_norm + 1e-45
    else:
        assert norm == want_norm or (math.isnan(norm) and math.isnan(want_norm))
    for g, h, o, w in zip(grads, host, out, want):
        assert torch.equal(g.cpu().view(torch.uint8), h.view(torch.uint8)) if g.numel() else True
        n = NAMES[g.dtype]
        within(o.view(-1), w, w.abs() * (HALF[n] + 2 * rel) + TINY[n], "clipped")
    inp = [g.clone() for g in grads]
    assert _run(inp, None, max_norm, kind) == norm or math.isnan(norm)
    for a, b in zip(inp, out):
        assert torch.equal(a.view(-1).view(torch.uint8), b.view(-1).view(torch.uint8))


def _grads(sizes, dtypes, seed, std=0.1):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(DT[dtypes[i % len(dtypes)]]).cuda() for i, n in enumerate(sizes)]


@pytest.mark.parametrize("dtypes", [["f32"], ["bf16"], ["f16"], ["f32", "bf16", "f16"]])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e6])
@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("sizes", [[1], [7], [4096], [0, 5, 0, 1], [4097, 3, 100_000, 64], [1, 2, 3, 4, 5, 6, 7, 8, 9],
                                   [1_000_003, 17]])
def test_clip(dtypes, max_norm, kind, sizes):
    _check(_grads(sizes, dtypes, sum(sizes)), max_norm, kind)


def test_no_tensors():
    assert _run([], [], 1.0) == 0.0
    assert _run([torch.empty(0, device="cuda")] * 3, None, 1.0, "max") == 0.0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_views_at_every_alignment(dtype):
    """Gradients as views of one flat buffer: input and output at different alignments, neighbours left alone."""
    for off_in in range(0, 9):
        for off_out in (0, 1, 5, 8):
            sizes = [33, 1, 5000, 8]
            flat = (torch.randn(6000, generator=torch.Generator().manual_seed(off_in)) * 0.3).to(DT[dtype]).cuda()
            out = torch.full((6000,), 7.0, dtype=DT[dtype], device="cuda")
            a = list(flat[off_in:off_in + sum(sizes)].split(sizes))
            b = list(out[off_out:off_out + sum(sizes)].split(sizes))
            norm = _run(a, b, 1.0)
            want_norm, want = oo.clip([t.cpu() for t in a], 1.0)
            assert abs(norm - want_norm) <= 1e-6 * want_norm
            for o, w in zip(b, want):
                within(o, w, w.abs() * (HALF[dtype] + 2.0 ** -20) + TINY[dtype])
            assert bool((out[:off_out] == 7).all()) and bool((out[off_out + sum(sizes):] == 7).all())


@pytest.mark.parametrize("count", [63, 64, 65, 1024, 1025, 2500])
def test_many_tensors(count):
    sizes = [(i * 37) % 101 for i in range(count)]
    _check(_grads(sizes, ["f32", "bf16"], count), 0.7)


def test_the_most_tensors():
    buf = torch.randn(65536 * 5, generator=torch.Generator().manual_seed(2)).cuda()
    want_norm, (want,) = oo.clip([buf.cpu()], 1.0)
    norm = _run(list(buf.split(5)), None, 1.0)
    assert abs(norm - want_norm) <= 1e-6 * want_norm
    within(buf, want, want.abs() * 2.0 ** -20)


@pytest.mark.parametrize("value", [1e30, 1e-30, 3e38, 1e-38])
def test_squares_beyond_fp32(value):
    """Squares that overflow or vanish in fp32 (and in bf16's range) are added up in fp64."""
    for dtype in ("f32", "bf16"):
        g = [torch.full((1000,), value, dtype=DT[dtype], device="cuda"), torch.zeros(50, dtype=DT[dtype], device="cuda")]
        host = [t.cpu() for t in g]
        want, _ = oo.clip(host, 1.0)
        norm = _run([t.clone() for t in g], None, 1.0)
        if want > torch.finfo(torch.float32).max:
            assert norm == math.inf  # the norm itself is past fp32
        else:
            assert abs(norm - want) <= 1e-6 * want + 1e-45
        _check(g, 1.0, "max")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [1e30, 1e-30, 3e38, 1e-38])
@pytest.mark.parametrize("max_norm", [1.0, 1e-3, 0.0])
def test_factors_of_any_size(value, max_norm, dtype):
    """Factors below the smallest normal fp32 number lose nothing; a norm past the largest one is not finite."""
    for count in (1, 1000):
        g = [torch.full((count,), value, dtype=DT[dtype], device="cuda"), torch.zeros(50, dtype=DT[dtype], device="cuda")]
        for kind in ("l2", "max"):
            _check([t.clone() for t in g], max_norm, kind)


def test_a_norm_past_fp32_leaves_the_gradients():
    """Finite gradients whose norm fp32 does not hold: norm_out is not finite, so nothing is scaled."""
    g = [torch.full((1000,), 3e38, device="cuda"), torch.full((7,), 2.0, dtype=torch.bfloat16, device="cuda")]
    keep = [t.clone() for t in g]
    assert _run(g, None, 1.0) == math.inf
    for a, b in zip(g, keep):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    out = [torch.zeros_like(t) for t in g]
    assert _run(g, out, 1.0) == math.inf
    for a, b in zip(out, keep):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("kind", ["l2", "max"])
def test_non_finite_gradients_are_reported_and_left(bad, kind):
    for dtype in ("f32", "bf16", "f16"):
        g = _grads([100, 5000, 3], [dtype], 3, std=10.0)
        g[1][4321] = bad
        keep = [t.clone() for t in g]
        norm = _run(g, None, 1.0, kind)
        assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
        for a, b in zip(g, keep):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_large_tensor_past_32_bits():
    n = (1 << 32) // 2 + 12345  # elements whose bytes pass 2^32
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-3:] = 2.0
    g[12] = 1.0
    assert abs(_run([g], None, 1.0) - math.sqrt(13.0)) < 1e-5
    got = g[-3:].float().cpu()
    assert bool(((got - 2.0 / math.sqrt(13.0)).abs() < 2.0 ** -8).all()) and float(g[5]) == 0.0


def test_deterministic():
    g = _grads([3_000_001, 70_000, 5], ["f32"], 1)
    norms = {_run(g, [torch.empty_like(t) for t in g], 1.0) for _ in range(5)}
    assert len(norms) == 1
