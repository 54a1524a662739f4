"""The forms of the norm, of combine and of their gradients for inputs past
the caches (over 128 MiB) against the ordinary ones: rows and tokens are
independent, so a large call's rows are, bit for bit, what a small call gives
on them, in every type and at widths of every workgroup shape."""

import pytest
import torch

from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

LIMIT = 128 << 20
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def rows_past(cols, dtype, inputs):
    return LIMIT // (cols * (2 if dtype == "bf16" else 4) * inputs) + 7


def randn(rows, cols, dtype, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return torch.randn((rows, cols), generator=gen, device=DEV).to(TYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [128, 1024, 4224, 7168, 8320, 16512, 32768])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(cols, dtype, residual):
    rows = rows_past(cols, dtype, 2 if residual else 1)
    say("norm past the caches: %d x %d %s" % (rows, cols, dtype))
    x, g = randn(rows, cols, dtype, 1), torch.rand(cols, device=DEV) + 0.5
    r = randn(rows, cols, dtype, 2) if residual else None
    for want_y in (False, True):
        big = T.rmsnorm_quantize(x, g, r, want_y=want_y)
        for at in (0, rows // 2, rows - 6):
            j = slice(at, at + 6)
            small = T.rmsnorm_quantize(x[j], g, None if r is None else r[j], want_y=want_y)
            for a, b in zip(big, small):
                assert (a is None and b is None) or torch.equal(a[j], b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [128, 1024, 4232, 7168, 8320, 16512, 32768])
@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_gradient(cols, dtype, with_dh):
    rows = rows_past(cols, dtype, 3 if with_dh else 2)
    say("norm gradient past the caches: %d x %d %s" % (rows, cols, dtype))
    dy, h, g = randn(rows, cols, dtype, 1), randn(rows, cols, dtype, 2), torch.rand(cols, device=DEV) + 0.5
    dh = randn(rows, cols, dtype, 3) if with_dh else None
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dx, dgamma = T.rmsnorm_backward(dy, h, g, rstd, dh=dh)
    for at in (0, rows // 2, rows - 6):
        j = slice(at, at + 6)
        assert torch.equal(dx[j], T.rmsnorm_backward(dy[j], h[j], g, rstd[j], dh=None if dh is None else dh[j])[0])
    # dgamma: fp32 sums of products (bound as in the parity tests)
    total, size = (torch.zeros(cols, dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(0, rows, 4096):
        p = dy[i:i + 4096].double() * (h[i:i + 4096].double() * rstd[i:i + 4096, None].double())
        total += p.sum(0)
        size += p.abs().sum(0)
    assert torch.all((dgamma.double() - total).abs() <= (rows / 256 + 96) * 2.0 ** -24 * size)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols,k", [(136, 8), (1024, 3), (4096, 8), (7168, 2), (16512, 9)])
def test_combine_and_gradient(cols, k, dtype):
    tokens = rows_past(cols * k, dtype, 1)
    say("combine past the caches: %d x %d of %d %s" % (tokens, k, cols, dtype))
    z, base, dy = randn(tokens * k, cols, dtype, 1), randn(tokens, cols, dtype, 2), randn(tokens, cols, dtype, 3)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    pos = torch.randperm(tokens * k, generator=gen, device=DEV).to(torch.int32).view(tokens, k)
    pos[2] = -2 - pos[2]                                  # a token whose entries were dropped
    w = torch.rand((tokens, k), generator=gen, device=DEV)
    for weights, b in ((w, base), (None, None)):
        out = T.combine(z, pos, weights, base=b)
        for at in (0, tokens // 2, tokens - 5):
            j = slice(at, at + 5)
            small = T.combine(z, pos[j].contiguous(), None if weights is None else weights[j], base=None if b is None else b[j])
            assert torch.equal(out[j], small)
    dz, dw = T.combine_backward(dy, z, pos, w)
    for at in (0, tokens // 2, tokens - 5):
        j = slice(at, at + 5)
        p = pos[j].reshape(-1).long()
        near = z[torch.where(p >= 0, p, -2 - p)]
        places = torch.arange(5 * k, dtype=torch.int32, device=DEV)
        places = torch.where(p >= 0, places, -2 - places).view(5, k)
        sz, sw = T.combine_backward(dy[j], near, places, w[j])
        assert torch.equal(dw[j], sw) and torch.equal(dz[torch.where(p >= 0, p, -2 - p)], sz)
