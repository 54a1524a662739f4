"""GPU parity of the norms after and before a block, with gate and scaled
residual addition, and of their gradient, against the 64-bit oracle.

Tolerances, derived (u = 2^-24, an fp32 rounding; b = 2^-8, a bf16 one):
  * rstd_post and rstd: a sum of positive squares in which no term passes more
    than 64 additions, the mean (a product by 1 / cols: 2 u, and eps), the root
    (which halves those errors) and its Newton step (2 u): 36 u relative.
  * h: t = z rstd_post gamma_post gate block_scale passes 36 u + 4 u, the
    residual's product and the sum u each: 41 u |t| + u |residual_scale r| + u |h|,
    then the type's rounding.
  * rstd, y, q, s are of the h that was stored: the norm's tolerances, with
    y = 36 u + 2 u and its rounding, bytes and scales of a stored fp32 y the
    oracle quantizer's exactly.
  * dH as the norm's dx: E = 80 u (rstd (|a| + |xh| mean|a xh|) + |dh|);
    dr = residual_scale dH: |residual_scale| (E + u |dH|).
  * w = block_scale dH gate gamma_post: F = |block_scale gate gamma_post| (E + 3 u
    |dH|); dz = rstd_post (w - zh m), m = mean(w zh): rstd_post (F + 4 u |w| + |zh|
    (mean(F |zh|) + 80 u mean|w zh|) + 4 u |zh m|).
  * sums over rows: (rows / 256 + 96) u of the terms' magnitudes, plus the terms'
    own errors: 2 u relative for dgamma, F-like ones for the others."""

import numpy as np
import pytest
import torch

import oracle
from oracle import block, moe
from fp8_fine_grained_x1_amd import binding as B
from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

U, UB = 2.0 ** -24, 2.0 ** -8
RSTD = 36 * U
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(x, dtype):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV).to(TYPES[dtype])


def host(t):
    return t.float().cpu().numpy()


def draw(rng, shape, dtype, std=1.0):
    x = rng.standard_normal(shape).astype(np.float32) * np.float32(std)
    if x.size:
        x.flat[rng.choice(x.size, max(1, x.size // 500))] *= np.float32(60)
    return moe.round_to(x, dtype == "bf16")


def gate_of(rng, kind, rows, cols, dtype, gtype):
    if kind == "none":
        return None, None
    if kind == "cols":
        g = moe.round_to(rng.standard_normal(cols), gtype == "bf16")
        return g, dev(g, gtype)
    g = moe.round_to(rng.standard_normal((rows, cols)), dtype == "bf16")
    return g, dev(g, dtype)


def check_forward(z, r, gp, gm, gate, rs, bs, eps, dtype, pow2, out):
    q, s, h, y, post, rstd = out
    ho, post_o = block.block_sum(z, r, gp, gate, np.float32(rs), np.float32(bs), eps)
    assert np.max(np.abs(host(post) / post_o - 1), initial=0) <= RSTD
    t = np.abs(ho - np.float64(np.float32(rs)) * r)
    err = 41 * U * t + U * np.abs(rs * r.astype(np.float64)) + U * np.abs(ho)
    err = err + (UB * (np.abs(ho) + err) if dtype == "bf16" else 0)
    hg = host(h)
    assert np.all(np.abs(hg - ho) <= err)
    # the next norm, of the stored h
    _, rstd_o, yo = moe.rmsnorm(hg, gm, eps)
    assert np.max(np.abs(host(rstd) / rstd_o - 1), initial=0) <= RSTD
    tol = RSTD + 2 * U
    if y is not None:
        assert np.all(np.abs(host(y) - yo) <= (tol + (UB if dtype == "bf16" else U)) * np.abs(yo) + 1e-40)
    rule = oracle.SCALE_POW2 if pow2 else oracle.SCALE_AMAX
    if dtype == "f32" and y is not None:
        qo, so = oracle.quantize_1x128(host(y), rule)
        assert np.array_equal(s.cpu().numpy(), so) and np.array_equal(q.cpu().numpy(), qo)
    check_bytes(q, s, yo, tol, pow2)


def check_bytes(q, s, yo, tol, pow2):
    """Bytes and 1x128 scales of values that are within tol (relative) of yo."""
    sg = s.cpu().numpy().astype(np.float64)
    ideal = np.maximum(np.abs(yo).reshape(yo.shape[0], -1, 128).max(axis=2) / 448.0, 2.0 ** -126)
    if pow2:
        m, _ = np.frexp(sg)
        assert np.all(m == 0.5)
        assert np.all(sg >= ideal * (1 - tol)) and np.all((sg < 2 * ideal * (1 + tol)) | (sg == 2.0 ** -126))
    else:
        assert np.all(np.abs(sg - ideal) <= (tol + 2 * U) * ideal)
    v = yo / np.repeat(sg, 128, axis=1)
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
    assert np.all(np.abs(oracle.decode(q.cpu().numpy()) - v) <= 0.5 * step * (1 + 1e-6) + 2 * (tol + 2 * U) * np.abs(v))


SHAPES = [(1, 128), (1, 7168), (2, 384), (77, 1024), (5, 4096), (3, 4224), (300, 640), (9, 5120), (4, 8192), (3, 8320), (2, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["none", "cols", "rows"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, gate, dtype):
    say("block norm %d x %d gate %s %s" % (rows, cols, gate, dtype))
    rng = np.random.default_rng(rows * 7 + cols)
    for pow2, gtype, want_y, rs, bs in ((False, "bf16", True, 0.9, 0.25), (True, "f32", False, 1.0, -1.0)):
        z, r = draw(rng, (rows, cols), dtype, 3.0), draw(rng, (rows, cols), dtype, 2.0)
        gp, gm = (moe.round_to(1 + 0.2 * rng.standard_normal(cols), gtype == "bf16") for _ in range(2))
        g, gd = gate_of(rng, gate, rows, cols, dtype, gtype)
        out = T.rmsnorm_block_quantize(dev(z, dtype), dev(r, dtype), dev(gp, gtype), dev(gm, gtype), gate=gd, residual_scale=rs,
                                       block_scale=bs, pow2=pow2, want_y=want_y)
        assert (out[3] is None) == (not want_y)
        check_forward(z, r, gp, gm, g, rs, bs, 1e-6, dtype, pow2, out)


def gradient_inputs(rng, rows, cols, dtype, gtype, gate, dh=True):
    z, h, dy = (draw(rng, (rows, cols), dtype, s) for s in (3.0, 2.0, 0.5))
    gp, gm = (moe.round_to(1 + 0.2 * rng.standard_normal(cols), gtype == "bf16") for _ in range(2))
    g, gd = gate_of(rng, gate, rows, cols, dtype, gtype)
    post, rstd = (np.float32(1 / np.sqrt(np.mean(v.astype(np.float64) ** 2, axis=1) + 1e-6)) for v in (z, h))
    return dy, z, h, gp, gm, post, rstd, g, gd, draw(rng, (rows, cols), dtype, 0.3) if dh else None


def check_gradient(dy, z, h, gp, gm, post, rstd, g, rs, bs, dh, dtype, gate, out):
    dz, dr, dgp, dgm, dgate = out
    rs, bs = np.float64(np.float32(rs)), np.float64(np.float32(bs))
    rows = z.shape[0]
    dzo, dro, dgpo, dgmo, dgo = block.block_norm_grad(dy, z, h, gp, gm, post, rstd, g, rs, bs, dh)
    gv = np.ones(z.shape) if g is None else np.broadcast_to(np.asarray(g, np.float64), z.shape)
    i2, i1 = rstd.astype(np.float64)[:, None], post.astype(np.float64)[:, None]
    xh, zh = h * i2, z * i1
    a = dy.astype(np.float64) * gm
    dH = dro / rs
    E = 80 * U * (i2 * (np.abs(a) + np.abs(xh) * np.mean(np.abs(a * xh), axis=1, keepdims=True)) + (0 if dh is None else np.abs(dh)))
    round_ = (lambda v, e: UB * (np.abs(v) + e)) if dtype == "bf16" else (lambda v, e: U * np.abs(v))
    e_dr = np.abs(rs) * (E + U * np.abs(dH))
    assert np.all(np.abs(host(dr) - dro) <= e_dr + round_(dro, e_dr))
    k = np.abs(bs * gv * gp)
    w, F = k * np.abs(dH), k * (E + 3 * U * np.abs(dH))
    mean = lambda v: np.mean(v, axis=1, keepdims=True)  # noqa: E731
    m = np.abs(mean(bs * gv * gp * dH * zh))
    e_dz = i1 * (F + 4 * U * w + np.abs(zh) * (mean(F * np.abs(zh)) + 80 * U * mean(w * np.abs(zh))) + 4 * U * np.abs(zh) * m)
    assert np.all(np.abs(host(dz) - dzo) <= e_dz + round_(dzo, e_dz))
    n = rows / 256 + 96
    t = np.abs(dy * xh)
    assert np.all(np.abs(host(dgm) - dgmo) <= (n + 2) * U * t.sum(axis=0) + 1e-40)
    e = np.abs(bs * zh) * (E + 3 * U * np.abs(dH))
    t = np.abs(bs * zh * dH)
    assert np.all(np.abs(host(dgp) - dgpo) <= ((n + 4) * U * t * np.abs(gv) + e * np.abs(gv)).sum(axis=0) + 1e-40)
    if gate == "none":
        assert dgate is None
    elif gate == "cols":
        assert dgate.dtype == torch.float32
        assert np.all(np.abs(host(dgate) - dgo.sum(axis=0)) <= (((n + 4) * U * t + e) * np.abs(gp)).sum(axis=0) + 1e-40)
    else:
        e_dg = (e + 4 * U * t) * np.abs(gp)
        assert dgate.dtype == dz.dtype and np.all(np.abs(host(dgate) - dgo) <= e_dg + round_(dgo, e_dg))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["none", "cols", "rows"])
@pytest.mark.parametrize("rows,cols", SHAPES + [(3, 8), (70, 136), (1100, 256), (2, 5128), (2, 12296)])
def test_gradient(rows, cols, gate, dtype):
    say("block norm gradient %d x %d gate %s %s" % (rows, cols, gate, dtype))
    rng = np.random.default_rng(rows * 5 + cols)
    for gtype, with_dh, rs, bs in (("bf16", True, 0.9, 0.25), ("f32", False, 1.0, -1.0)):
        dy, z, h, gp, gm, post, rstd, g, gd, dh = gradient_inputs(rng, rows, cols, dtype, gtype, gate, with_dh)
        out = T.rmsnorm_block_backward(dev(dy, dtype), dev(z, dtype), dev(h, dtype), dev(gp, gtype), dev(gm, gtype),
                                       dev(post, "f32"), dev(rstd, "f32"), gate=gd, residual_scale=rs, block_scale=bs, dh=dev(dh, dtype))
        check_gradient(dy, z, h, gp, gm, post, rstd, g, rs, bs, dh, dtype, gate, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_layouts_and_outputs_left_out(dtype):
    rng = np.random.default_rng(11)
    rows, cols = 37, 896
    wide = dev(draw(rng, (rows, 7 * cols + 64), dtype), dtype)
    part = [wide[:, i * cols + (64 if i > 2 else 0):][:, :cols] for i in range(7)]
    z, r, gate, dy, h, dh, _ = part
    gp, gm = (dev(1 + 0.2 * rng.standard_normal(cols), "f32") for _ in range(2))
    a = T.rmsnorm_block_quantize(z, r, gp, gm, gate=gate, want_y=True)
    b = T.rmsnorm_block_quantize(z.contiguous(), r.contiguous(), gp, gm, gate=gate.contiguous(), scale_layout="row_major")
    assert b[1].is_contiguous() and b[3] is None
    assert all(torch.equal(a[i], b[i]) for i in (0, 1, 2, 4, 5))
    for n in (1, 5):
        c = T.rmsnorm_block_quantize(z[8:8 + n], r[8:8 + n], gp, gm, gate=gate[8:8 + n], want_y=True)
        assert all(torch.equal(x, y[8:8 + n]) for x, y in zip(c, a))
    ga = T.rmsnorm_block_backward(dy, z, h, gp, gm, a[4], a[5], gate=gate, dh=dh)
    gb = T.rmsnorm_block_backward(*(t.contiguous() for t in (dy, z, h)), gp, gm, a[4], a[5], gate=gate.contiguous(), dh=dh.contiguous())
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))
    # outputs between guard bands and left out, through the C interface
    t = B.FP8FG_BF16 if dtype == "bf16" else B.FP8FG_F32
    o = torch.full((rows, cols + 32), 7.0, dtype=TYPES[dtype], device=DEV)
    B.fp8_rmsnorm_block_quantize(z, t, rows, cols, z.stride(0), r, r.stride(0), gp, gm, 1, gate, gate.stride(0), 1.0, 1.0, 1e-6, 0,
                                 o[:, 16:], o.stride(0), None, 0, None, 0, None, 0, 0, None, None)
    assert torch.equal(o[:, 16:16 + cols], a[2]) and torch.all(o[:, :16] == 7) and torch.all(o[:, 16 + cols:] == 7)
    y = torch.empty((rows, cols), dtype=TYPES[dtype], device=DEV)
    B.fp8_rmsnorm_block_quantize(z, t, rows, cols, z.stride(0), r, r.stride(0), gp, gm, 1, gate, gate.stride(0), 1.0, 1.0, 1e-6, 0,
                                 o[:, 16:], o.stride(0), y, cols, None, 0, None, 0, 0, None, None)
    assert torch.equal(y, a[3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_beyond_fp32s_range_and_zero_rows(dtype):
    cols = 256
    z = torch.zeros((5, cols), device=DEV)
    z[0], z[1], z[2], z[3, 3] = 2.0 ** 100, 2.0 ** -100, 3.0, 2.0 ** -120
    z = z.to(TYPES[dtype])
    r = torch.zeros_like(z)
    r[4] = 1.0
    g = torch.ones(cols, device=DEV)
    q, s, h, y, post, rstd = T.rmsnorm_block_quantize(z, r, g, g, eps=0.0, want_y=True)
    zd = z.double()
    m = zd.square().mean(1)
    want = torch.where(m > 0, m.rsqrt(), torch.zeros_like(m)).clamp(max=float(torch.finfo(torch.float32).max))
    assert torch.all((post.double() - want).abs() <= RSTD * want)
    assert float(post[4]) == 0 and torch.all(h[4] == 1) and torch.all(q[4] == 0x7E)
    assert torch.all((h[:3].double() - 1).abs() <= UB)
    dz, dr, dgp, dgm, _ = T.rmsnorm_block_backward(h, z, h, g, g, post, rstd)
    assert torch.all(dz[4] == 0) and all(torch.isfinite(t.float()).all() for t in (dz, dr, dgp, dgm))


def test_no_rows():
    for gate in (None, torch.full((256,), 2.0, device=DEV), torch.empty((0, 256), device=DEV)):
        e, g, n = torch.empty((0, 256), device=DEV), torch.ones(256, device=DEV), torch.empty(0, device=DEV)
        out = T.rmsnorm_block_quantize(e, e, g, g, gate=gate, want_y=True)
        assert out[0].shape == (0, 256) and out[1].shape == (0, 2) and out[2].shape == (0, 256)
        dz, dr, dgp, dgm, dg = T.rmsnorm_block_backward(e, e, e, g, g, n, n, gate=gate)
        assert dz.shape == (0, 256) and torch.all(dgp == 0) and torch.all(dgm == 0)
        assert dg is None if gate is None else torch.all(dg == 0)


def test_gradient_against_differences():
    """Of sum(dy y) + sum(dh h) in fp32 at 64-bit sums with step 2^-6: y and h are off
    by 80 u |y| each, 2^-18 of terms up to 4: over 2 x 128 of them and a step of
    2^-5 below 256 * 4 * 80 u / 2^-5 * 2^-3 (independent signs, 1 / sqrt(256)
    rounded up) < 2e-2 of the largest derivatives (above 0.5), d^2 f''' / 6 below
    1e-3."""
    rng = np.random.default_rng(12)
    rows, cols, d = 1, 128, 2.0 ** -6
    z, r, dy, dh = (rng.standard_normal((rows, cols)).astype(np.float32) for _ in range(4))
    gp, gm, g = (np.float32(1 + 0.3 * rng.standard_normal(cols)) for _ in range(3))
    kw = dict(residual_scale=0.8, block_scale=0.6)

    def f(z, r, gp, gm, g):
        _, _, h, y, post, rstd = T.rmsnorm_block_quantize(dev(z, "f32"), dev(r, "f32"), dev(gp, "f32"), dev(gm, "f32"), gate=dev(g, "f32"),
                                                          want_y=True, **kw)
        return float((y.double().cpu().numpy() * dy).sum() + (h.double().cpu().numpy() * dh).sum()), h, post, rstd

    a = [z, r, gp, gm, g]
    _, h, post, rstd = f(*a)
    dz, dr, dgp, dgm, dg = T.rmsnorm_block_backward(dev(dy, "f32"), dev(z, "f32"), h, dev(gp, "f32"), dev(gm, "f32"), post, rstd,
                                                    gate=dev(g, "f32"), dh=dev(dh, "f32"), **kw)
    for i, got in enumerate((dz, dr, dgp, dgm, dg)):
        got = host(got).ravel()
        for c in (int(np.argmax(np.abs(got))), 3):
            hi, lo = (v.copy() for v in (a[i], a[i]))
            hi.flat[c] += d
            lo.flat[c] -= d
            diff = (f(*[hi if j == i else a[j] for j in range(5)])[0] - f(*[lo if j == i else a[j] for j in range(5)])[0]) / (2 * d)
            assert abs(diff - got[c]) < 2.1e-2, (i, c, diff, got[c])


def test_results_repeat():
    x = torch.randn((700, 1024), device=DEV).to(torch.bfloat16)
    g = torch.ones(1024, device=DEV)
    q, s, h, y, post, rstd = T.rmsnorm_block_quantize(x, x, g, g)
    a = T.rmsnorm_block_backward(x, x, h, g, g, post, rstd, gate=g)
    for _ in range(3):
        assert all(torch.equal(u, v) for u, v in zip(a, T.rmsnorm_block_backward(x, x, h, g, g, post, rstd, gate=g)))


def test_helpers_refuse():
    x, g, n = torch.zeros((4, 256), device=DEV), torch.ones(256, device=DEV), torch.ones(4, device=DEV)
    b = g.to(torch.bfloat16)
    for call in (lambda: T.rmsnorm_block_quantize(x.double(), x, g, g), lambda: T.rmsnorm_block_quantize(x, x[:2], g, g),
                 lambda: T.rmsnorm_block_quantize(x, x, g, b), lambda: T.rmsnorm_block_quantize(x, x, g[:128], g),
                 lambda: T.rmsnorm_block_quantize(x, x, g, g, gate=b), lambda: T.rmsnorm_block_quantize(x, x, g, g, gate=x[:, :128]),
                 lambda: T.rmsnorm_block_quantize(x, x, g, g, gate=x.to(torch.bfloat16)), lambda: T.rmsnorm_block_quantize(x, x.cpu(), g, g),
                 lambda: T.rmsnorm_block_quantize(x, None, g, g), lambda: T.rmsnorm_block_backward(x, x, x, g, g, n[:2], n),
                 lambda: T.rmsnorm_block_backward(x, x[:, :128], x, g, g, n, n), lambda: T.rmsnorm_block_backward(x, x, x, g, g, n, n.double()),
                 lambda: T.rmsnorm_block_backward(x, x, x, g, g, n, n, gate=n), lambda: T.rmsnorm_block_backward(x.t(), x, x, g, g, n, n)):
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: T.rmsnorm_block_quantize(x, x, g, g, block_scale=float("inf")), B.FP8FG_EINVAL),
                         (lambda: T.rmsnorm_block_quantize(x, x, g, g, eps=-1.0), B.FP8FG_EINVAL),
                         (lambda: T.rmsnorm_block_quantize(x[:, :64].contiguous(), x[:, :64].contiguous(), g[:64], g[:64]), B.FP8FG_ESHAPE)):
        with pytest.raises(B.Fp8fgError) as e:
            call()
        assert e.value.status == status
