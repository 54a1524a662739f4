"""The norms around a block where a workgroup takes row after row, the next one
loaded while this one is worked on: at least three to each and a rest, against the
64-bit oracle (tolerances as in test_gpu_block_norm.py, whose shapes give every
workgroup one row), and long calls against calls of so few rows, bit for bit."""

import numpy as np
import pytest
import torch

from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say
from oracle import moe
from test_gpu_block_norm import check_forward, check_gradient, dev, draw, gate_of, gradient_inputs

pytestmark = pytest.mark.gpu

CUS = 256


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["none", "cols", "rows"])
@pytest.mark.parametrize("rows,cols", [(3 * CUS + 5, 4224), (3 * 14 * CUS + 9, 128), (3 * 4 * CUS + 100, 1024), (3 * CUS + 1, 8192)])
def test_forward(rows, cols, gate, dtype):
    say("block norm rows %d x %d gate %s %s" % (rows, cols, gate, dtype))
    rng = np.random.default_rng(rows + cols)
    # eps 0, and rows whose squares leave fp32's range, of z, of the sum, or of both, in the
    # middle of a workgroup's run and at its ends
    for pow2, gtype, want_y, rs, bs, eps in ((False, "f32", True, 0.9, 0.25, 0.0), (True, "bf16", False, 1.0, -1.0, 1e-6)):
        z, r = draw(rng, (rows, cols), dtype, 3.0), draw(rng, (rows, cols), dtype, 2.0)
        far = rng.choice(rows, 12, replace=False)
        z[far[:4]] *= np.float32(2.0 ** 100)
        z[far[4:8]] *= np.float32(2.0 ** -90)
        r[far[2:6]] *= np.float32(2.0 ** 90)
        z[far[8:10]] *= np.float32(2.0 ** 100)
        r[far[10:]] *= np.float32(2.0 ** 100)
        gp, gm = (moe.round_to(1 + 0.2 * rng.standard_normal(cols), gtype == "bf16") for _ in range(2))
        g, gd = gate_of(rng, gate, rows, cols, dtype, gtype)
        out = T.rmsnorm_block_quantize(dev(z, dtype), dev(r, dtype), dev(gp, gtype), dev(gm, gtype), gate=gd, residual_scale=rs,
                                       block_scale=bs, eps=eps, pow2=pow2, want_y=want_y)
        check_forward(z, r, gp, gm, g, rs, bs, eps, dtype, pow2, out)


@pytest.mark.parametrize("pow2,want_y", [(False, True), (True, False)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["none", "cols", "rows"])
# (inputs past the caches, where loads and stores are others, and within them)
@pytest.mark.parametrize("rows,cols", [(20011, 2048), (9001, 7168), (7001, 1152)])
def test_a_long_call_is_its_rows(rows, cols, gate, dtype, pow2, want_y):
    say("block norm rows %d x %d gate %s %s" % (rows, cols, gate, dtype))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(rows)
    z, r = (torch.randn((rows, cols), generator=gen, device=DEV).to(dtype) for _ in range(2))
    z[rows // 3] *= 2.0 ** 100
    r[rows // 2] *= 2.0 ** 100
    gp, gm = (1 + 0.2 * torch.randn(cols, generator=gen, device=DEV) for _ in range(2))
    g = {"none": None, "cols": gp * 0.5, "rows": z.flip(0).contiguous()}[gate]
    kw = dict(residual_scale=0.9, block_scale=0.25, pow2=pow2)
    long = T.rmsnorm_block_quantize(z, r, gp, gm, gate=g, want_y=want_y, **kw)
    some = list(range(0, rows - 256, 1783)) + [rows // 3 - 100, rows // 2 - 100, rows - 256]
    for a in some:
        part = T.rmsnorm_block_quantize(z[a:a + 256], r[a:a + 256], gp, gm, gate=g[a:a + 256] if gate == "rows" else g, want_y=want_y, **kw)
        for x, y in zip(long, part):
            assert (x is None) == (y is None)
            assert x is None or torch.equal(x[a:a + 256], y), a


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["none", "cols", "rows"])
@pytest.mark.parametrize("rows,cols", [(1030, 4224), (4 * 1024 + 3, 136), (1700, 2048)])
def test_gradient(rows, cols, gate, dtype):
    say("block norm gradient rows %d x %d gate %s %s" % (rows, cols, gate, dtype))
    rng = np.random.default_rng(rows * 3 + cols)
    dy, z, h, gp, gm, post, rstd, g, gd, dh = gradient_inputs(rng, rows, cols, dtype, "f32", gate, True)
    out = T.rmsnorm_block_backward(dev(dy, dtype), dev(z, dtype), dev(h, dtype), dev(gp, "f32"), dev(gm, "f32"), dev(post, "f32"),
                                   dev(rstd, "f32"), gate=gd, residual_scale=0.9, block_scale=0.25, dh=dev(dh, dtype))
    check_gradient(dy, z, h, gp, gm, post, rstd, g, 0.9, 0.25, dh, dtype, gate, out)
