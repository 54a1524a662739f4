"""A NaN in the silu gate's inputs stays visible: in every output that it enters
and in no other."""

import pytest
import torch

from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV

pytestmark = pytest.mark.gpu

NAN = float("nan")


def is_nan_byte(q):
    return (q & 0x7F) == 0x7F


def inputs(dtype, tiny):
    """Rows whose other tiles are ordinary, or (tiny) whose scales take the steps of
    tiny ones: a row next to a NaN's may have them."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    u = torch.randn((128, 512), generator=gen, device=DEV)
    da = torch.randn((128, 256), generator=gen, device=DEV)
    if tiny:
        u[1::2] = 0.0
        da[1::2] = 0.0
    return u.to(dtype), da.to(dtype)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("tiny", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_in_either_half(dtype, tiny, pow2):
    u, da = inputs(dtype, tiny)
    clean = T.swiglu_quantize(u, pow2=pow2)
    where = torch.zeros((128, 256), dtype=torch.bool, device=DEV)
    u = u.clone()
    for row, col in ((0, 3), (2, 130), (64, 255)):      # the gate
        u[row, col], where[row, col] = NAN, True
    for row, col in ((4, 77), (100, 128)):              # the linear half
        u[row, 256 + col], where[row, col] = NAN, True
    q, s, uq, us = T.swiglu_quantize(u, pow2=pow2)
    assert torch.equal(is_nan_byte(q), where) and torch.equal(is_nan_byte(uq), torch.isnan(u))
    rows = torch.tensor([r for r in range(128) if r not in (0, 2, 4, 64, 100)], device=DEV)
    assert all(torch.equal(a[rows], b[rows]) for a, b in zip((q, s, uq, us), clean))
    # back from the checkpoint that holds them
    dq, ds, du, a = T.swiglu_backward(da, uq, us, want_du=True, want_a=True, pow2=pow2)
    assert torch.equal(torch.isnan(a), where)
    gate = torch.isnan(u[:, :256])
    nan_du = torch.cat([where, gate], dim=1)  # dg by either half, dl by the gate
    assert torch.equal(torch.isnan(du), nan_du) and torch.equal(is_nan_byte(dq), nan_du)
    tq = T.swiglu_backward_128x1(da, uq, us, pow2=pow2)
    assert torch.equal(tq[0], dq) and torch.equal(tq[1], ds)
    assert torch.equal(is_nan_byte(tq[2]), nan_du.t()) and torch.equal(is_nan_byte(tq[4]), where.t())


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("tiny", [False, True])
def test_nan_in_the_gradient(tiny, pow2):
    u, da = inputs(torch.float32, tiny)
    _, _, uq, us = T.swiglu_quantize(u, pow2=pow2)
    where = torch.zeros((128, 256), dtype=torch.bool, device=DEV)
    da = da.clone()
    for row, col in ((0, 0), (6, 201), (127, 255)):
        da[row, col], where[row, col] = NAN, True
    both = torch.cat([where, where], dim=1)
    dq, _, du, a = T.swiglu_backward(da, uq, us, want_du=True, want_a=True, pow2=pow2)
    assert torch.equal(torch.isnan(du), both) and torch.equal(is_nan_byte(dq), both) and not bool(torch.isnan(a).any())
    tq = T.swiglu_backward_128x1(da, uq, us, pow2=pow2)
    assert torch.equal(is_nan_byte(tq[2]), both.t()) and not bool(is_nan_byte(tq[4]).any())
