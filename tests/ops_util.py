"""Helpers of the GPU tests of the operators around the layer."""
from __future__ import annotations

import torch

import sparse_moe_layer_renormalised_b200 as moe

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# half a step of the type, relative to the value; and half the step of its smallest numbers
HALF = {k: torch.finfo(v).eps / 2 for k, v in DT.items()}
TINY = {k: torch.finfo(v).tiny * torch.finfo(v).eps / 2 for k, v in DT.items()}
GUARD = 256


class Guarded:
    """Device buffers with a guard behind each: check() fails where a call wrote past an end."""

    def __init__(self):
        self.flats = []

    def new(self, shape, dtype, fill=None):
        n = 1
        for s in shape:
            n *= s
        flat = torch.full((n + GUARD,), -77.0 if dtype.is_floating_point else -77, dtype=dtype, device="cuda")
        view = flat[:n].view(shape)
        if fill is not None:
            view.copy_(fill)
        self.flats.append((flat, n))
        return view

    def check(self):
        torch.cuda.synchronize()
        for flat, n in self.flats:
            assert bool((flat[n:] == -77).all()), "a call wrote past the end of a buffer"
        assert moe.moe_device_error() == (moe.MOE_OK, 0)


def within(got, want, tol, what=""):
    """|got - want| <= tol elementwise; where want is not finite, got is the same."""
    got, want = got.cpu().to(torch.float64), want.to(torch.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert bool((torch.isnan(got) == torch.isnan(want)).all()), what
    inf = torch.isinf(want)
    assert bool((got[inf] == want[inf]).all()), what
    tol = torch.as_tensor(tol, dtype=torch.float64).expand(want.shape)
    over = (got - want).abs()[fine] / tol[fine].clamp_min(1e-300)
    if over.numel():
        assert float(over.max()) <= 1.0, f"{what}: {float(over.max()):.3g} times the tolerance"


def workspace(nbytes):
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda").fill_(0xA5)
