"""moe_route and moe_route_backward against the fp64 oracle: indices exactly,
weights and gradients to the rounding of their arithmetic."""
import math

import pytest
import torch

import sparse_moe_layer_renormalised_b200 as moe
from ops_util import DT, HALF, TINY, Guarded, within
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
INF = math.inf


def _spread(logits):
    """[T, 1]: how far the unmasked logits of a row lie from its largest (or from 0)."""
    l = logits.cpu().to(torch.float64)
    l = torch.where(torch.isfinite(l), l, torch.zeros_like(l))
    return (l.max(1, keepdim=True).values - l.min(1, keepdim=True).values).clamp_min(0) + l.abs().max(1, keepdim=True).values


def _rel(logits):
    """Relative error of a score: the exponentials (fast ones: 2 + 1.173 |x| steps of 2^-23 at argument x, in
    the softmax's sum), the rounding of l - max (|l - max| 2^-24), a sum of up to 32 lanes' sums of 32
    (10 tree steps and 32 in a row, 2^-24 each), a reciprocal, products: (24 + 3 spread) steps of 2^-23."""
    return (24.0 + 3.0 * _spread(logits)) * 2.0 ** -23


def _run(logits, bias, k, dtype, **kw):
    T, E = logits.shape
    g = Guarded()
    l = g.new((T, E), DT[dtype], logits)
    b = None if bias is None else g.new((E,), torch.float32, bias)
    idx, w = g.new((T, k), torch.int32), g.new((T, k), torch.float32)
    d = moe.route_desc(T, E, k, dtype=dtype, **kw)
    assert moe.moe_route(d, l, b, idx, w) == moe.MOE_OK
    g.check()
    return l.cpu(), idx.cpu().to(torch.int64), w


def _check(logits, bias, k, dtype, **kw):
    l, idx, w = _run(logits, bias, k, dtype, **kw)
    okw = {("keep" if n == "keep_groups" else n): v for n, v in kw.items()}
    want_idx, want_w = oo.route(l, bias, k, **okw)
    assert torch.equal(idx, want_idx), "indices differ in rows %s" % (idx != want_idx).any(1).nonzero().view(-1)[:8].tolist()
    within(w, want_w, want_w.abs() * _rel(l) + 1e-37, "weights")


def _logits(T, E, seed, std=1.5):
    return torch.randn(T, E, generator=torch.Generator().manual_seed(seed)) * std


def _bias(E, seed, std=0.05):
    return torch.randn(E, generator=torch.Generator().manual_seed(seed)) * std


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 1), (5, 8, 8), (3, 33, 5), (7, 60, 4), (64, 64, 6), (33, 129, 32),
                                   (9, 160, 8), (40, 256, 8), (17, 384, 7), (5, 512, 32), (3, 777, 31), (50, 896, 16),
                                   (6, 1000, 9), (8, 1023, 12), (11, 1024, 32)])
def test_route(dtype, score, T, E, k):
    for i, bias in enumerate((None, _bias(E, E + k), torch.zeros(E))):
        _check(_logits(T, E, T + E + i), bias, k, dtype, score=score, renorm=i != 1, scale=1.0 if i else 2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("E,k,groups,keep", [(64, 4, 4, 1), (256, 8, 8, 4), (160, 6, 8, 3), (96, 8, 32, 9), (99, 10, 11, 7),
                                             (72, 3, 3, 2), (1024, 32, 16, 5), (64, 32, 32, 16), (64, 8, 8, 8)])
def test_groups(score, group_top, E, k, groups, keep):
    for dtype in ("f32", "bf16"):
        for bias in (None, _bias(E, 7)):
            _check(_logits(20, E, E + k), bias, k, dtype, score=score, groups=groups, keep_groups=keep,
                   group_top=group_top)


def test_groups_of_one_expert():
    _check(_logits(20, 32, 1), _bias(32, 2), 8, "f32", groups=32, keep_groups=8, group_top=1)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
def test_masks(score, biased, groups, keep):
    """Rows with nothing left, with fewer than k left, one group left, NaN and infinities in masked places."""
    E, k = 96, 12
    l = _logits(24, E, 11)
    l[0] = -INF
    l[1] = math.nan
    l[2, ::2] = -INF
    l[3, 5:] = -INF            # five left, k = 12
    l[4] = -INF
    l[4, 77] = 0.3             # one left
    l[5, :72] = math.nan       # the last group alone
    l[6] = torch.finfo(torch.float32).min
    l[7, 10:] = torch.finfo(torch.float32).min
    l[8, ::3] = math.nan
    l[9, 20] = INF
    l[10, 20] = INF
    l[10, 3] = INF
    l[11] = 0.0
    l[12] = -0.0
    l[12, ::2] = 0.0
    l[13] = 80.0               # saturated scores
    l[14] = -80.0
    l[15] = -200.0
    for dtype in ("f32", "bf16"):
        for renorm in (True, False):
            _check(l, _bias(E, 3) if biased else None, k, dtype, score=score, groups=groups, keep_groups=keep,
                   group_top=2 if groups > 1 else 1, renorm=renorm)


def test_bias_infinities_and_nan():
    E = 64
    b = _bias(E, 5)
    b[3] = -INF
    b[4] = math.nan
    b[7] = INF
    b[9] = INF
    l = _logits(10, E, 6)
    l[4, 8:] = -INF
    for score in ("sigmoid", "softmax"):
        l_, idx, w = _run(l, b, 8, "f32", score=score)
        want_idx, want_w = oo.route(l_, b, 8, score=score)
        assert torch.equal(idx, want_idx)
        within(w, want_w, want_w * _rel(l_) + 1e-37)


@pytest.mark.parametrize("E,k", [(64, 8), (896, 16), (896, 32), (1000, 5)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_keys_fp32_cannot_tell_apart(E, k, score):
    """Biases that bring every key of a row within 2^-24 of one value: the order
    is that of the real numbers, which fp32 keys lose."""
    for seed in range(4):
        l = _logits(1, E, seed + E)
        s = oo.scores(l, score)[0]
        b = (0.75 - s).to(torch.float32)
        _check(l.expand(3, E).contiguous(), b, k, "f32", score=score)
        _check(l.expand(3, E).contiguous(), b, min(k, 8), "f32", score=score, groups=4, keep_groups=2, group_top=2)


@pytest.mark.parametrize("E,k", [(64, 8), (896, 16), (1024, 32)])
def test_ties_go_to_the_lower_index(E, k):
    g = torch.Generator().manual_seed(E)
    few = torch.randint(0, 3, (16, E), generator=g).float()  # three values only
    for bias in (None, torch.zeros(E), torch.full((E,), 0.25)):
        for score in ("sigmoid", "softmax"):
            _check(few, bias, k, "bf16", score=score)
            _check(few, bias, k, "f32", score=score, groups=8, keep_groups=5, group_top=2)


def _many_reference(l, b, k, groups, keep, group_top, score):
    """idx of many rows on the GPU in fp64 by stable sorts (finite logits)."""
    l = l.double()
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    key = l if b is None else s + b.double()
    if groups > 1:
        T, E = l.shape
        val = s if b is None else key
        best = val.view(T, groups, -1).sort(dim=2, descending=True).values[:, :, :group_top].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :keep]
        out = torch.ones(T, groups, dtype=torch.bool, device=l.device).scatter_(1, kept, False)
        key = key.masked_fill(out.repeat_interleave(E // groups, 1), -INF)
    return key.sort(dim=1, descending=True, stable=True).indices[:, :k]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,groups,keep,group_top", [(896, 16, 1, 1, 1), (896, 32, 1, 1, 1), (1000, 32, 1, 1, 1),
                                                       (128, 8, 1, 1, 1), (256, 8, 8, 4, 2), (512, 24, 16, 7, 2)])
def test_many_rows(score, E, k, groups, keep, group_top):
    """Enough rows that every path of the selection is taken, the rare near ties among them."""
    T = 16384
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        std = (1.5, 0.01, 6.0, 1.5)[seed]  # usual, nearly equal, saturated, and half-precision logits
        l = torch.randn(T, E, generator=g, device="cuda") * std
        dtype = "bf16" if seed == 3 else "f32"
        l = l.to(DT[dtype])
        b = torch.randn(E, generator=g, device="cuda") * 0.05
        for bias in (b, None):
            idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
            d = moe.route_desc(T, E, k, groups=groups, keep_groups=keep, group_top=group_top, score=score, dtype=dtype)
            assert moe.moe_route(d, l, bias, idx, w) == moe.MOE_OK
            assert moe.moe_device_error() == (moe.MOE_OK, 0)
            want = _many_reference(l, bias, k, groups, keep, group_top, score)
            assert int((idx.long() != want).any(1).sum()) == 0, (seed, bias is None)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size,spread", [(30.0, 1e-5), (100.0, 1e-4), (3.0, 1e-6)])
@pytest.mark.parametrize("T,E,k,groups,keep", [(3000, 16, 4, 8, 4), (12000, 16, 4, 8, 4), (2000, 256, 8, 8, 4),
                                               (12000, 128, 8, 16, 5)])
def test_group_scores_whose_keys_cancel(score, size, spread, T, E, k, groups, keep):
    """A group's two best keys near +size and -size: their sum is far smaller than what their roundings are
    relative to, and the groups differ by less than those."""
    g = torch.Generator().manual_seed(E + T)
    l = torch.randn(T, E, generator=g) * spread
    gsize = E // groups
    b = torch.full((groups, gsize), -size)
    b[:, 0] = size
    b = b.reshape(E).contiguous()
    # the groups' scores in fp64: far enough apart that fp64 itself orders them (keys of `size` are rounded by
    # 2^-53 size each, sums by less)
    key = oo.scores(l, score) + b.double()
    rank = key.view(T, groups, gsize).sort(dim=2, descending=True).values[:, :, :2].sum(2)
    rank = rank.sort(dim=1, descending=True).values
    clear = rank[:, keep - 1] - rank[:, keep] > 16 * size * 2.0 ** -53
    assert int(clear.sum()) > 0.99 * T
    _, idx, _ = _run(l, b, k, "f32", score=score, groups=groups, keep_groups=keep, group_top=2)
    want = _many_reference(l, b, k, groups, keep, 2, score)
    # which groups; the order of the experts in them has tests of its own
    got_groups, want_groups = ((i // gsize).sort(1).values for i in (idx, want))
    wrong = (got_groups != want_groups).any(1) & clear
    assert int(wrong.sum()) == 0, f"{int(wrong.sum())} rows with a wrong set of groups"


def _special_rows(E, seed):
    """Rows with nothing left, little left, NaN, infinities, ties, saturated and usual logits."""
    l = _logits(26, E, seed)
    l[0] = -INF
    l[1] = math.nan
    l[2, ::2] = -INF
    l[3, E // 20:] = -INF
    l[4] = -INF
    l[4, E - 1] = 0.3
    l[5, :E * 3 // 4] = math.nan
    l[6] = torch.finfo(torch.float32).min
    l[7, E // 9:] = torch.finfo(torch.float32).min
    l[8, ::3] = math.nan
    l[9, E // 3] = INF
    l[10, E // 3] = INF
    l[10, E // 30] = INF
    l[11] = 0.0
    l[12] = -0.0
    l[12, ::2] = 0.0
    l[13] = 80.0
    l[14] = -80.0
    l[15] = -200.0
    l[16] = torch.randint(0, 3, (E,), generator=torch.Generator().manual_seed(seed)).float()
    return l


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,k,groups,keep,group_top", [
    (128, 8, 1, 1, 1), (127, 5, 1, 1, 1), (64, 6, 1, 1, 1), (61, 8, 1, 1, 1), (96, 12, 1, 1, 1), (125, 16, 1, 1, 1),
    (96, 12, 4, 2, 2), (128, 8, 8, 4, 2), (128, 16, 32, 9, 2), (66, 7, 11, 5, 1), (60, 10, 3, 2, 2), (32, 8, 32, 8, 1),
    (8, 8, 1, 1, 1), (3, 2, 1, 1, 1), (1, 1, 1, 1, 1)])
def test_many_short_rows(score, dtype, E, k, groups, keep, group_top):
    """More rows than the GPU holds warps: several tokens a warp, usual and special ones side by side, and a last
    warp with a part of them."""
    warps = 32 * torch.cuda.get_device_properties(0).multi_processor_count
    b = _bias(E, E)
    odd = b.clone()
    odd[0] = -INF
    odd[E // 2] = math.nan
    odd[E - 1] = INF
    for i, bias in enumerate((None, b, torch.zeros(E), odd, 0.75)):
        l = _special_rows(E, E + k)
        if isinstance(bias, float):  # keys within 2^-24 of one value in the last row
            bias = (bias - oo.scores(l[25:], score)[0]).to(torch.float32)
        n, T = l.shape[0], warps + 5
        at = torch.arange(T) * 7 % n
        kw = dict(score=score, groups=groups, group_top=group_top, renorm=i != 1, scale=1.0 if i else 2.5)
        l_, idx, w = _run(l[at], bias, k, dtype, keep_groups=keep, **kw)
        want_idx, want_w = oo.route(l.to(DT[dtype]), bias, k, keep=keep, **kw)
        want_idx, want_w = want_idx[at], want_w[at]
        assert torch.equal(idx, want_idx), (i, (idx != want_idx).any(1).nonzero().view(-1)[:8].tolist())
        within(w, want_w, want_w.abs() * _rel(l_) + 1e-37, "weights")
    assert moe.moe_device_error() == (moe.MOE_OK, 0)


def test_deterministic_and_rows_independent():
    l = _logits(300, 896, 1)
    b = _bias(896, 2)
    _, i1, w1 = _run(l, b, 16, "f32")
    _, i2, w2 = _run(l, b, 16, "f32")
    assert torch.equal(i1, i2) and torch.equal(w1, w2)
    _, i3, w3 = _run(l[17:18].contiguous(), b, 16, "f32")
    assert torch.equal(i3[0], i1[17]) and torch.equal(w3[0], w1[17])


# ------------------------------------------------------------------------------ gradients
def _check_backward(l, idx, dw, dtype, score, renorm, scale=1.5):
    T, E = l.shape
    k = idx.shape[1]
    g = Guarded()
    ld = g.new((T, E), DT[dtype], l)
    i_d, dw_d = g.new((T, k), torch.int32, idx), g.new((T, k), torch.float32, dw)
    out = g.new((T, E), DT[dtype])
    d = moe.route_desc(T, E, k, score=score, renorm=renorm, scale=scale, dtype=dtype)
    assert moe.moe_route_backward(d, ld, i_d, dw_d, out) == moe.MOE_OK
    g.check()
    want = oo.route_backward(ld.cpu(), idx, dw, score, renorm, scale)
    s = oo.scores(ld.cpu(), score)
    if renorm and score == "softmax":
        chosen = torch.zeros_like(s).scatter(1, idx, s.gather(1, idx))
        total = chosen.sum(1, keepdim=True)
        s = torch.where(total > 0, chosen / torch.where(total > 0, total, 1.0), 0.0)
    if renorm and score == "sigmoid":
        total = s.gather(1, idx).sum(1, keepdim=True)
        s = torch.where(total > 0, s / torch.where(total > 0, total, 1.0), 0.0)
    # each dl is a score (or share) times a difference of terms of at most scale * max|dw|
    dmax = (dw.to(torch.float64).abs() * torch.isfinite(dw)).nan_to_num(0, 0, 0).max(1, keepdim=True).values * scale
    # (64 * 2^-53 of it: the oracle's own sum over up to 32 chosen ones, whose true value is 0 with renorm)
    tol = 2.0 * s * dmax * (_rel(ld) + 40 * 2.0 ** -24) + want.abs() * HALF[dtype] + TINY[dtype] + 64 * 2.0 ** -53 * dmax
    within(out, want, tol, "dlogits")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 2), (3, 33, 5), (64, 64, 6), (9, 160, 8), (5, 777, 31), (40, 896, 16),
                                   (3, 1024, 32), (2, 1023, 1)])
def test_backward(dtype, score, renorm, T, E, k):
    g = torch.Generator().manual_seed(T + E + k)
    l = _logits(T, E, T * 3 + E)
    idx = torch.argsort(torch.rand(T, E, generator=g), 1)[:, :k].contiguous()
    dw = torch.randn(T, k, generator=g)
    _check_backward(l, idx, dw, dtype, score, renorm)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_masks(score, renorm):
    T, E, k = 8, 40, 6
    l = _logits(T, E, 4)
    l[0] = -INF
    l[1] = math.nan
    l[2, ::2] = -INF
    l[3, 3:] = math.nan
    l[4] = 0.0
    l[5] = -100.0
    idx, _ = oo.route(l, None, k, score=score)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(9))
    dw[0] = math.nan   # all masked: not used
    dw[3, 3:] = INF    # masked ones
    for dtype in ("f32", "bf16"):
        _check_backward(l, idx, dw, dtype, score, renorm)


def test_backward_reports_bad_indices():
    """Out of range and repeated indices: recorded, skipped, the rest of the row as without them."""
    T, E, k = 2, 64, 4
    l = _logits(T, E, 8).cuda()
    dw = torch.ones(T, k, device="cuda")
    out = torch.full((T, E), math.nan, device="cuda")
    for bad, code in (([3, 64, 5, 6], 11), ([3, -1, 5, 6], 11), ([3, 5, 5, 6], 12)):
        idx = torch.tensor([bad, [0, 1, 2, 3]], dtype=torch.int32, device="cuda")
        for score in ("sigmoid", "softmax"):
            d = moe.route_desc(T, E, k, score=score, renorm=False)
            assert moe.moe_route_backward(d, l, idx, dw, out) == moe.MOE_OK
            assert moe.moe_device_error() == (moe.MOE_ERR_DEVICE, code)
            good = sorted({b for b in bad if 0 <= b < E})
            want = oo.route_backward(l[:1].cpu(), torch.tensor([good]), torch.ones(1, len(good)), score, False, 1.0)
            within(out[:1], want, 1e-5)
    assert moe.moe_device_error() == (moe.MOE_OK, 0)


def test_offsets_past_32_bits():
    """More than 2^32 bytes of logits: rows at the far end come out as they do alone."""
    T, E, k = 1_300_000, 1024, 8
    l = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_(0.0, 1.5)
    d = moe.route_desc(T, E, k, score="softmax", dtype="bf16", renorm=False)
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    assert moe.moe_route(d, l, None, idx, w) == moe.MOE_OK
    tail = slice(T - 5, T)
    want_idx, want_w = oo.route(l[tail].cpu(), None, k, score="softmax", renorm=False)
    assert torch.equal(idx[tail].cpu().long(), want_idx)
    within(w[tail], want_w, want_w * 1e-5)
    dl = torch.empty_like(l)
    assert moe.moe_route_backward(d, l, idx, torch.ones_like(w), dl) == moe.MOE_OK
    want = oo.route_backward(l[tail].cpu(), want_idx, torch.ones(5, k), "softmax", False, 1.0)
    within(dl[tail], want, want.abs() * (HALF["bf16"] + 1e-4) + 1e-6)
    assert moe.moe_device_error() == (moe.MOE_OK, 0)
