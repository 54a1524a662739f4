"""GPU parity of the norm with 8-bit output and of its gradient against the
64-bit oracle.

Tolerances, derived (u = 2^-24, an fp32 rounding; b = 2^-8, a bf16 one (8 significant bits)):
  * rstd: a sum of positive squares in which no term passes more than 64
    additions, then the mean, the root and the quotient: 32 u + 4 u relative
    (the root halves the sum's error).
  * y: rstd's error, two products: RSTD + 2 u relative, then the type's
    rounding.
  * q: the quantizers' bytes of an fp32 y, so with a stored fp32 y bytes and
    scales are the oracle quantizer's exactly.  With bf16 the decoded value
    is within half an E4M3 step of y / s, both perturbed by Y.
  * dx: dx = rstd (a - xh m): each product some roundings, m a mean whose
    terms pass at most 64 additions.  |err| <= 80 u (rstd (|a| + |xh| mean|a xh|) + |dh|).
  * dgamma: terms pass rows / strips additions of a strip, at most 64 of a
    thread, 16 of a workgroup: (rows / 256 + 96) u sum |dy xh|."""

import numpy as np
import pytest
import torch

import oracle
from oracle import moe
from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

U, UB = 2.0 ** -24, 2.0 ** -8
RSTD = 36 * U
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV).to(dtype)


def host(t):
    return t.float().cpu().numpy()


def draw(rng, shape, dtype, std=1.0, outliers=True):
    x = rng.standard_normal(shape).astype(np.float32) * np.float32(std)
    if outliers and x.size:
        x.flat[rng.choice(x.size, max(1, x.size // 500))] *= np.float32(60)
    return moe.round_to(x, dtype == "bf16")


def check_forward(x, r, gamma, dtype, out, eps, pow2, xdev):
    q, s, h, y, rstd = out
    ho, rstd_o, yo = moe.rmsnorm(x, gamma, eps, r, dtype == "bf16")
    assert np.array_equal(host(h), ho)
    if r is None:
        assert h.data_ptr() == xdev.data_ptr()
    assert np.max(np.abs(host(rstd) / rstd_o - 1)) <= RSTD
    tol = RSTD + 2 * U
    ty = tol + (UB if dtype == "bf16" else U)
    yg = host(y).astype(np.float64)
    assert np.all(np.abs(yg - yo) <= ty * np.abs(yo) + 1e-40)
    rule = oracle.SCALE_POW2 if pow2 else oracle.SCALE_AMAX
    if dtype == "f32":
        qo, so = oracle.quantize_1x128(host(y), rule)
        assert np.array_equal(s.cpu().numpy(), so)
        assert np.array_equal(q.cpu().numpy(), qo)
        return
    sg = s.cpu().numpy().astype(np.float64)
    amax = np.abs(yo).reshape(yo.shape[0], -1, 128).max(axis=2)
    ideal = np.maximum(amax / 448.0, 2.0 ** -126)
    if pow2:
        m, _ = np.frexp(sg)
        assert np.all(m == 0.5)
        assert np.all(sg >= ideal * (1 - tol)) and np.all((sg < 2 * ideal * (1 + tol)) | (sg == 2.0 ** -126))
    else:
        assert np.all(np.abs(sg - ideal) <= (tol + 2 * U) * ideal)
    v = yo / np.repeat(sg, 128, axis=1)
    got = oracle.decode(q.cpu().numpy())
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    assert np.all(np.abs(got - v) <= 0.5 * step * (1 + 1e-6) + 2 * (tol + 2 * U) * np.abs(v))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 128), (1, 7168), (2, 384), (77, 1024), (5, 4096), (3, 4224), (300, 640),
                                       (9, 5120), (6, 7168), (4, 8192), (3, 8320), (2, 16512), (2, 32768)])
def test_forward_shapes(rows, cols, dtype):
    say("norm %d x %d %s" % (rows, cols, dtype))
    rng = np.random.default_rng(rows * 7 + cols)
    for residual, pow2, gtype in ((True, False, "bf16"), (False, True, "f32")):
        x = draw(rng, (rows, cols), dtype)
        r = draw(rng, (rows, cols), dtype, 2.0) if residual else None
        gamma = moe.round_to(1 + 0.2 * rng.standard_normal(cols), gtype == "bf16")
        xd = dev(x, TYPES[dtype])
        out = T.rmsnorm_quantize(xd, dev(gamma, TYPES[gtype]), None if r is None else dev(r, TYPES[dtype]), eps=1e-6,
                                 pow2=pow2, want_y=True)
        check_forward(x, r, gamma, dtype, out, 1e-6, pow2, xd)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_strides_layouts_and_missing_outputs(dtype):
    rng = np.random.default_rng(11)
    rows, cols = 37, 896
    wide = draw(rng, (rows, 2 * cols + 64), dtype)
    gamma = moe.round_to(1 + 0.2 * rng.standard_normal(cols), False)
    wd = dev(wide, TYPES[dtype])
    xd, rd = wd[:, :cols], wd[:, cols + 64:]
    g = dev(gamma, torch.float32)
    a = T.rmsnorm_quantize(xd, g, rd, want_y=True)
    check_forward(wide[:, :cols], wide[:, cols + 64:], gamma, dtype, a, 1e-6, False, xd)
    b = T.rmsnorm_quantize(xd, g, rd, scale_layout="row_major")
    assert b[1].is_contiguous() and b[3] is None
    for i in (0, 1, 2, 4):
        assert torch.equal(a[i], b[i])
    # rows do not depend on their number or place
    for n in (1, 5):
        c = T.rmsnorm_quantize(xd[8:8 + n], g, rd[8:8 + n])
        assert torch.equal(c[0], a[0][8:8 + n]) and torch.equal(c[1], a[1][8:8 + n]) and torch.equal(c[2], a[2][8:8 + n])


def test_forward_zero_rows_and_values():
    g = torch.ones(256, device=DEV)
    q, s, h, y, rstd = T.rmsnorm_quantize(torch.empty((0, 256), device=DEV), g)
    assert q.shape == (0, 256) and s.shape == (0, 2) and rstd.shape == (0,)
    x = torch.zeros((3, 256), device=DEV)
    x[1, :128] = -2.0
    q, s, h, y, rstd = T.rmsnorm_quantize(x, g, eps=0.25, want_y=True)
    assert torch.all(rstd[[0, 2]] == 2.0) and torch.all(q[0] == 0) and torch.all(s[[0, 2]] == 2.0 ** -126)
    assert float(rstd[1]) == np.float32(1 / np.sqrt(np.float32(2.25)))
    assert torch.all(q[1, :128] == 0xFE) and torch.all(y[1, 128:] == 0) and float(s[1, 1]) == 2.0 ** -126


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 7168), (2, 136), (77, 1024), (1100, 264), (5, 4104), (2500, 128),
                                       (9, 5120), (3, 8320), (2, 32768)])
def test_gradient(rows, cols, dtype):
    say("norm gradient %d x %d %s" % (rows, cols, dtype))
    rng = np.random.default_rng(rows + cols)
    for with_dh, gtype in ((True, "f32"), (False, "bf16")):
        h, dy = draw(rng, (rows, cols), dtype, 2.0), draw(rng, (rows, cols), dtype, 0.1, False)
        dh = draw(rng, (rows, cols), dtype, 0.2, False) if with_dh else None
        gamma = moe.round_to(1 + 0.2 * rng.standard_normal(cols), gtype == "bf16")
        rstd = (1 / np.sqrt(np.mean(h.astype(np.float64) ** 2, axis=1) + 1e-6)).astype(np.float32)
        dt = TYPES[dtype]
        args = (dev(dy, dt), dev(h, dt), dev(gamma, TYPES[gtype]), dev(rstd, torch.float32))
        dx, dgamma = T.rmsnorm_backward(*args, dh=None if dh is None else dev(dh, dt))
        dxo, dgo = moe.rmsnorm_grad(dy, h, gamma, rstd, dh)
        xh, a = h.astype(np.float64) * rstd[:, None].astype(np.float64), dy.astype(np.float64) * gamma
        size = rstd[:, None] * (np.abs(a) + np.abs(xh) * np.mean(np.abs(a * xh), axis=1, keepdims=True))
        size += 0 if dh is None else np.abs(dh)
        tol = 80 * U * size + (UB * np.abs(dxo) if dtype == "bf16" else 0)
        assert np.all(np.abs(host(dx) - dxo) <= tol)
        assert np.all(np.abs(host(dgamma) - dgo) <= (rows / 256 + 96) * U * np.sum(np.abs(dy * xh), axis=0))
        again = T.rmsnorm_backward(*args, dh=None if dh is None else dev(dh, dt))
        assert torch.equal(dx, again[0]) and torch.equal(dgamma, again[1])


def test_gradient_strides():
    rng = np.random.default_rng(3)
    rows, cols = 19, 264
    wide = dev(draw(rng, (rows, 3 * cols + 16), "bf16"), torch.bfloat16)
    dy, h, dh = wide[:, :cols], wide[:, cols:2 * cols], wide[:, 2 * cols + 16:]
    g, rstd = torch.rand(cols, device=DEV), torch.rand(rows, device=DEV)
    a = T.rmsnorm_backward(dy, h, g, rstd, dh=dh)
    b = T.rmsnorm_backward(dy.contiguous(), h.contiguous(), g, rstd, dh=dh.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_gradient_of_no_rows_is_zero():
    e = torch.empty((0, 264), device=DEV)
    dx, dgamma = T.rmsnorm_backward(e, e, torch.ones(264, device=DEV), torch.empty(0, device=DEV))
    assert dx.shape == (0, 264) and torch.all(dgamma == 0)


def test_gradient_against_differences_of_the_kernel():
    # loss = sum dy * y + sum dh * h in 64 bits of the kernel's own fp32
    # outputs.  A central difference with step d is off by its truncation,
    # which the step 2 d has four times of, and by the outputs' rounding.
    rng = np.random.default_rng(8)
    rows, cols = 3, 256
    x, dy, dh = (rng.standard_normal((rows, cols)).astype(np.float32) for _ in range(3))
    gamma = (1 + 0.3 * rng.standard_normal(cols)).astype(np.float32)

    def forward(a, g):
        _, _, _, y, rstd = T.rmsnorm_quantize(dev(a, torch.float32), dev(g, torch.float32), eps=1e-6, want_y=True)
        return host(y).astype(np.float64), rstd

    def loss(a, g):
        return np.sum(dy * forward(a, g)[0]) + np.sum(dh.astype(np.float64) * a)

    y, rstd = forward(x, gamma)
    dx, dgamma = T.rmsnorm_backward(dev(dy, torch.float32), dev(x, torch.float32), dev(gamma, torch.float32), rstd,
                                    dh=dev(dh, torch.float32))
    noise = 2.0 ** -18 * np.sum(np.abs(dy * y))
    for _ in range(4):
        v = rng.standard_normal((rows, cols)).astype(np.float32)
        u = rng.standard_normal(cols).astype(np.float32)
        for which, grad in (("x", np.sum(host(dx).astype(np.float64) * v)),
                            ("gamma", np.sum(host(dgamma).astype(np.float64) * u))):
            diff = []
            for d in (2.0 ** -5, 2.0 ** -6):
                if which == "x":
                    diff.append((loss(x + d * v, gamma) - loss(x - d * v, gamma)) / (2 * d))
                else:
                    diff.append((loss(x, gamma + d * u) - loss(x, gamma - d * u)) / (2 * d))
            assert abs(diff[1] - grad) <= abs(diff[0] - diff[1]) + noise / 2.0 ** -5, (which, diff, grad)


FLT_MAX = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [256, 7168, 16512])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_every_magnitude(cols, dtype, eps):
    # squares that overflow fp32 or vanish in it, rows of zeros, one large
    # element among tiny ones, ordinary rows between them
    say("norm of every magnitude: %d %s eps %g" % (cols, dtype, eps))
    rng = np.random.default_rng(cols)
    mags = [1e-44, 1e-38, 1e-30, 1e-20, 1e-16, 1e-15, 1.0, 1e10, 1e17, 2.2e17, 1e19, 1e25, 5e37, 0.0]
    x = rng.standard_normal((len(mags) + 2, cols))
    x /= np.abs(x).max(axis=1, keepdims=True)
    x[:len(mags)] *= 2.0 * np.array(mags)[:, None]
    x[-2] = 1e-30 * np.sign(x[-2])
    x[-2, 3] = 3e38
    x[-1] = np.sign(x[-1]) * 3.3e38
    x = moe.round_to(x, dtype == "bf16")
    gamma = moe.round_to(1 + 0.2 * rng.uniform(-1, 1, cols), False)
    xd, gd = dev(x, TYPES[dtype]), dev(gamma, torch.float32)
    for residual in (None, np.zeros_like(x)):
        q, s, h, y, rstd = T.rmsnorm_quantize(xd, gd, None if residual is None else dev(residual, TYPES[dtype]), eps=eps,
                                              want_y=True)
        ho, ro, yo = moe.rmsnorm(x, gamma, eps, residual, dtype == "bf16")
        assert np.array_equal(host(h), ho)
        # half a subnormal step where rstd is that small, and what it makes of y
        assert np.all(np.abs(host(rstd) - ro) <= RSTD * ro + 2.0 ** -150)
        ty = RSTD + 2 * U + (UB if dtype == "bf16" else U)
        lost = 2.0 ** -150 * np.abs(ho).astype(np.float64) * np.abs(gamma)
        assert np.all(np.abs(host(y) - yo) <= ty * np.abs(yo) + lost * (1 + ty) + 1e-40)
        zero = ~np.any(x, axis=1)
        assert np.any(zero) and np.all(host(rstd)[zero] == (0.0 if eps == 0 else np.float32(1 / np.sqrt(np.float32(eps)))))
        z = torch.from_numpy(zero).to(DEV)
        assert torch.all((q[z] & 0x7F) == 0) and torch.all(s[z] == 2.0 ** -126)  # (-0 keeps its sign)
        if dtype == "f32":
            qo, so = oracle.quantize_1x128(host(y))
            assert np.array_equal(s.cpu().numpy(), so) and np.array_equal(q.cpu().numpy(), qo)
    # a row's result is its own
    alone = T.rmsnorm_quantize(xd[9:10], gd, eps=eps, want_y=True)
    assert torch.equal(alone[0], q[9:10]) and torch.equal(alone[3], y[9:10]) and torch.equal(alone[4], rstd[9:10])

    # the gradient, where rstd keeps it inside fp32
    dy, dh = (moe.round_to(0.1 * rng.standard_normal(x.shape), dtype == "bf16") for _ in range(2))
    r = host(rstd)
    keep = (r < 1e30) & np.isfinite(r)
    at = torch.from_numpy(np.flatnonzero(keep)).to(DEV)
    dt = TYPES[dtype]
    dx, dgamma = T.rmsnorm_backward(dev(dy[keep], dt), xd[at], gd, rstd[at], dh=dev(dh[keep], dt))
    dxo, dgo = moe.rmsnorm_grad(dy[keep], x[keep], gamma, r[keep], dh[keep])
    xh, a = x[keep].astype(np.float64) * r[keep, None].astype(np.float64), dy[keep].astype(np.float64) * gamma
    size = r[keep, None] * (np.abs(a) + np.abs(xh) * np.mean(np.abs(a * xh), axis=1, keepdims=True)) + np.abs(dh[keep])
    assert np.all(np.abs(host(dx) - dxo) <= 80 * U * size + (UB * np.abs(dxo) if dtype == "bf16" else 0))
    assert np.all(np.abs(host(dgamma) - dgo) <= 97 * U * np.sum(np.abs(dy[keep] * xh), axis=0))
    if eps == 0:
        z = np.flatnonzero(zero[keep])
        assert np.array_equal(host(dx)[z], dh[keep][z])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [16392, 20480, 24584, 32768])
def test_gradient_of_the_widest_rows(cols, dtype):
    # one workgroup of 1024 threads to a row, the last units part of them only
    say("norm gradient, %d columns %s" % (cols, dtype))
    rng = np.random.default_rng(cols)
    rows = 70
    h, dy, dh = draw(rng, (rows, cols), dtype, 2.0), draw(rng, (rows, cols), dtype, 0.1, False), draw(rng, (rows, cols), dtype, 0.2)
    gamma = moe.round_to(1 + 0.2 * rng.standard_normal(cols), False)
    rstd = (1 / np.sqrt(np.mean(h.astype(np.float64) ** 2, axis=1) + 1e-6)).astype(np.float32)
    dt = TYPES[dtype]
    dx, dgamma = T.rmsnorm_backward(dev(dy, dt), dev(h, dt), dev(gamma, torch.float32), dev(rstd, torch.float32), dh=dev(dh, dt))
    dxo, dgo = moe.rmsnorm_grad(dy, h, gamma, rstd, dh)
    xh, a = h.astype(np.float64) * rstd[:, None].astype(np.float64), dy.astype(np.float64) * gamma
    size = rstd[:, None] * (np.abs(a) + np.abs(xh) * np.mean(np.abs(a * xh), axis=1, keepdims=True)) + np.abs(dh)
    assert np.all(np.abs(host(dx) - dxo) <= 80 * U * size + (UB * np.abs(dxo) if dtype == "bf16" else 0))
    assert np.all(np.abs(host(dgamma) - dgo) <= (rows / 256 + 96) * U * np.sum(np.abs(dy * xh), axis=0))
