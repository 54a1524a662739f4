"""The silu gate's transposed 128x1 tiles where a column's scale is not an
ordinary one, and values that leave fp32's range.

Expected bytes and scales are the oracle quantizer's of the fp32 values that the
other form of the gradient stores (they are formed by the same steps), bit for
bit."""

import numpy as np
import pytest
import torch

import oracle
from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

RULES = {False: oracle.SCALE_AMAX, True: oracle.SCALE_POW2}


def checkpoint(g, l):
    """The checkpoint of the rows' gate and linear halves."""
    q, s = oracle.quantize_1x128(np.concatenate([g, l], axis=1).astype(np.float32), oracle.SCALE_AMAX)
    return torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)


def both(da, uq, us, pow2):
    wide = T.swiglu_backward(da, uq, us, want_du=True, want_a=True, pow2=pow2)
    return T.swiglu_backward_128x1(da, uq, us, pow2=pow2), wide


@pytest.mark.parametrize("pow2", [False, True])
def test_finite_inputs_whose_products_overflow(pow2):
    """da l = 1e30 * 1e30 (and a = g l = 1e38 * 100) in some columns and rows: the power-of-two
    rule's scale of an infinite maximum is 2^120 in both tilings, an infinite value 448 of the
    steps and the others their nearest; the amax rule's scale is infinite."""
    rng = np.random.default_rng(1)
    rows = inner = 256
    g, l = (rng.uniform(0.5, 2, (rows, inner)).astype(np.float32) for _ in range(2))
    da = rng.standard_normal((rows, inner)).astype(np.float32)
    # whole tiles of the checkpoint share a scale: rows 3 and 130 have far linear halves
    l[[3, 130]] *= np.float32(1e30)
    da[[3, 130], 5] = [1e30, -1e30]
    g[200], l[200] = 1e37 * rng.uniform(1, 2, inner), 1e3
    da = torch.from_numpy(da).to(DEV)
    uq, us = checkpoint(g, l)
    (dq, ds, dqt, dst, aqt, ast), (wq, ws, du, a) = both(da, uq, us, pow2)
    assert torch.equal(dq, wq) and torch.equal(ds, ws)
    assert bool(torch.isinf(du).any()) and bool(torch.isinf(a).any()) and not bool(torch.isnan(du).any() | torch.isnan(a).any())
    for q, s, v in ((dqt, dst, du), (aqt, ast, a)):
        v = v.t().contiguous()
        tile = v.view(v.shape[0], -1, 128)
        far = torch.isinf(tile).any(2)
        assert bool(far.any()) and not bool(far.all())
        if not pow2:
            assert torch.equal(torch.isinf(s), far)
            continue
        assert torch.all(s[far] == 2.0 ** 120)
        # the quotients by a power of two are exact: E4M3 of them, saturated
        want = torch.clamp(tile / s[:, :, None], -448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).view(v.shape)
        assert torch.equal(q, want)
    if pow2:
        tile = du.view(rows, -1, 128)
        want = torch.clamp(tile / ds[:, :, None], -448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8).view(du.shape)
        assert torch.equal(dq, want)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["zero block", "zero columns", "tiny columns", "signs of zero", "all of them"])
def test_columns_without_an_ordinary_scale(kind, dtype, pow2):
    """Blocks and columns of zeros (padding, rows without a gradient), maxima around the
    borders of the fast form (2^-55), of the lifted quotients (2^-64 448) and of the floored
    scales (2^-126 448), beside ordinary columns."""
    say("128x1 %s %s pow2 %d" % (kind, dtype, pow2))
    rng = np.random.default_rng(2)
    rows, inner = 384, 256
    g, l = (rng.standard_normal((rows, inner)).astype(np.float32) for _ in range(2))
    da = rng.standard_normal((rows, inner)).astype(np.float32) * np.float32(0.01)
    if kind in ("zero block", "all of them"):
        da[128:256] = 0.0
    if kind in ("zero columns", "all of them"):
        da[:, 3::7] = 0.0
    if kind in ("tiny columns", "all of them"):
        for c, e in enumerate((-40, -50, -54, -55, -56, -57, -62, -64, -66, -70, -100, -115, -117, -119, -121, -125, -126, -127, -130)):
            da[:, 10 + 11 * c] *= np.float32(2.0) ** e
    if kind in ("signs of zero", "all of them"):
        da[::2, 5] = -0.0
        da[1::2, 5] = 0.0
        g[:, 6] = np.where(np.arange(rows) % 2, 0.0, -0.0)
        l[:, 130] = 0.0
    if kind == "all of them":
        g[256:], l[256:] = 0.0, 0.0     # rows that hold nothing: a is 0 too
    da = torch.from_numpy(da).to(DEV).to(dtype)
    uq, us = checkpoint(g, l)
    (dq, ds, dqt, dst, aqt, ast), _ = both(da, uq, us, pow2)
    _, _, du, a = T.swiglu_backward(da.float(), uq, us, want_du=True, want_a=True, pow2=pow2)
    for q, s, v in ((dq.t(), ds.t(), du.t()), (dqt, dst, du), (aqt, ast, a)):
        v = np.ascontiguousarray(v.cpu().numpy().T)
        if q is not dqt and q is not aqt:
            q, s = q.t(), s.t()
        qo, so = oracle.quantize_1x128(v, RULES[pow2])
        assert np.array_equal(s.cpu().numpy(), so)
        assert np.array_equal(q.cpu().numpy(), qo), np.argwhere(q.cpu().numpy() != qo)[:5]
