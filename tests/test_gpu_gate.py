"""GPU parity of the silu gate with 8-bit outputs and checkpoints, and of its
gradient, against the 64-bit oracle.

Tolerances, derived (u = 2^-24, an fp32 rounding; b = 2^-8, a bf16 one):
  * sigmoid and 1 - sigmoid: exp within 2 ulp (4 u), 1 + t and its quotient 4 u,
    a product u: 10 u relative, above an absolute 2^-125 (where exp ends).
  * a = (g s) l: two products more, 12 u.
  * dl = da (g s): 12 u.  dg = ((da l) s) (1 + g r): the bracket is off by 11 u
    |g r| + u |1 + g r|, the products by 13 u: 14 u |da l s (1 + g r)| + 11 u |da
    l s g r|.
  * each plus the type's rounding where it is stored.
  * bytes and scales of an fp32 tensor that is stored too are the oracle
    quantizer's exactly; otherwise a decoded value is within half an E4M3
    step of v / s, both perturbed by the value's error.
The checkpoint's bytes and scales are the oracle quantizer's of u exactly."""

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
TINY = 2.0 ** -125
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
RULES = {False: oracle.SCALE_AMAX, True: oracle.SCALE_POW2}


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV).to(TYPES[dtype])


def host(t):
    return t.float().cpu().numpy()


def draw(rng, shape, dtype, std=1.5):
    x = rng.standard_normal(shape).astype(np.float32) * np.float32(std)
    if x.size:
        x.flat[rng.choice(x.size, max(1, x.size // 300))] *= np.float32(25)
    return moe.round_to(x, dtype == "bf16")


def check_bytes(q, s, v, err, pow2, what):
    """E4M3 bytes and 1x128 scales of values v, each known to within err."""
    q, sg = q.cpu().numpy(), s.cpu().numpy().astype(np.float64)
    amax = np.abs(v).reshape(v.shape[0], -1, 128).max(axis=2)
    off = err.reshape(v.shape[0], -1, 128).max(axis=2) / 448.0
    ideal = np.maximum(amax / 448.0, 2.0 ** -126)
    if pow2:
        m, _ = np.frexp(sg)
        assert np.all(m == 0.5), what
        assert np.all(sg >= (ideal - off) * (1 - 2 * U)) and np.all((sg < 2 * (ideal + off) * (1 + 2 * U)) | (sg == 2.0 ** -126)), what
    else:
        assert np.all(np.abs(sg - ideal) <= off + 2 * U * ideal), what
    sw = np.repeat(sg, 128, axis=1)
    w = v / sw
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(w), 2.0 ** -6))) - 3)
    assert np.all(np.abs(oracle.decode(q) - np.clip(w, -448, 448)) <= 0.5 * step * (1 + 1e-6) + 2 * err / sw + 4 * U * np.abs(w)), what


def grad_errors(da, u):
    """([dg | dl], a) and the errors allowed of them before any rounding."""
    du, a = block.swiglu_grad(da, u)
    g, l = np.split(np.asarray(u, np.float64), 2, axis=1)
    s, r = block.sigmoid(g)
    d = np.asarray(da, np.float64)
    floor = TINY * (np.abs(d * l) * (1 + np.abs(g)))
    e_dg = 14 * U * np.abs(du[:, :g.shape[1]]) + 11 * U * np.abs(d * l * s * g * r) + floor + TINY
    e_dl = 12 * U * np.abs(du[:, g.shape[1]:]) + TINY * np.abs(d * g) + TINY
    return du, a, np.concatenate([e_dg, e_dl], axis=1), 12 * U * np.abs(a) + TINY * np.abs(g * l) + TINY


SHAPES = [(1, 128), (8, 2048), (3, 384), (16, 256), (17, 128), (33, 640), (130, 1408), (257, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,inner", SHAPES)
def test_forward(rows, inner, dtype):
    say("gate %d x %d %s" % (rows, inner, dtype))
    rng = np.random.default_rng(rows * 3 + inner)
    for pow2, layout in ((False, "group_major"), (True, "row_major")):
        u = draw(rng, (rows, 2 * inner), dtype)
        q, s, uq, us = T.swiglu_quantize(dev(u, dtype), pow2=pow2, scale_layout=layout)
        assert s.stride() == ((1, rows) if layout == "group_major" else (inner // 128, 1))
        qo, so = oracle.quantize_1x128(u, RULES[pow2])
        assert np.array_equal(uq.cpu().numpy(), qo) and np.array_equal(us.cpu().numpy(), so)
        a = block.swiglu(u)
        g, l = np.split(u.astype(np.float64), 2, axis=1)
        check_bytes(q, s, a, 12 * U * np.abs(a) + TINY * np.abs(g * l) + TINY, pow2, (rows, inner))
        # serving: nothing is kept, the rest is the same
        q2, s2, none, none2 = T.swiglu_quantize(dev(u, dtype), pow2=pow2, scale_layout=layout, keep=False)
        assert none is None and none2 is None and torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,inner", SHAPES)
def test_gradient(rows, inner, dtype):
    say("gate gradient %d x %d %s" % (rows, inner, dtype))
    rng = np.random.default_rng(rows * 5 + inner)
    for pow2, layout in ((False, "group_major"), (True, "row_major")):
        uq, us = oracle.quantize_1x128(draw(rng, (rows, 2 * inner), "f32"), RULES[pow2])
        da = draw(rng, (rows, inner), dtype, 0.01)
        u = block.kept(uq, us)
        args = (dev(da, dtype), torch.from_numpy(uq).to(DEV), torch.from_numpy(us).to(DEV))
        dq, ds, du, a = T.swiglu_backward(*args, want_du=True, want_a=True, pow2=pow2, scale_layout=layout)
        duo, ao, e_du, e_a = grad_errors(da, u)
        b = UB if dtype == "bf16" else 0.0
        assert np.all(np.abs(host(du) - duo) <= e_du + b * (np.abs(duo) + e_du))
        assert np.all(np.abs(host(a) - ao) <= e_a + b * (np.abs(ao) + e_a))
        if dtype == "f32":
            qo, so = oracle.quantize_1x128(host(du), RULES[pow2])
            assert np.array_equal(dq.cpu().numpy(), qo) and np.array_equal(ds.cpu().numpy(), so)
        check_bytes(dq, ds, duo, e_du, pow2, (rows, inner))
        for du_, a_ in ((False, False), (True, False), (False, True)):
            got = T.swiglu_backward(*args, want_du=du_, want_a=a_, pow2=pow2, scale_layout=layout)
            assert torch.equal(got[0], dq) and torch.equal(got[1], ds)
            assert torch.equal(got[2], du) if du_ else got[2] is None
            assert torch.equal(got[3], a) if a_ else got[3] is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,inner", [(128, 128), (256, 384), (384, 1408), (1024, 256)])
def test_gradient_128x1(rows, inner, dtype):
    say("gate gradient 128x1 %d x %d %s" % (rows, inner, dtype))
    rng = np.random.default_rng(rows * 7 + inner)
    for pow2, layout in ((False, "group_major"), (True, "row_major")):
        uq, us = oracle.quantize_1x128(draw(rng, (rows, 2 * inner), "f32"), RULES[pow2])
        da = dev(draw(rng, (rows, inner), dtype, 0.01), dtype)
        args = (torch.from_numpy(uq).to(DEV), torch.from_numpy(us).to(DEV))
        dq, ds, dqt, dst, aqt, ast = T.swiglu_backward_128x1(da, *args, pow2=pow2, scale_layout=layout)
        # the fp32 values, stored: bytes and scales are the oracle quantizers' of them
        want = T.swiglu_backward(da.float(), *args, want_du=True, want_a=True, pow2=pow2, scale_layout=layout)
        assert torch.equal(dq, want[0]) and torch.equal(ds, want[1]) and ds.stride() == want[1].stride()
        for q, s, v in ((dqt, dst, want[2]), (aqt, ast, want[3])):
            qo, so = oracle.quantize_1x128(np.ascontiguousarray(host(v).T), RULES[pow2])
            assert np.array_equal(q.cpu().numpy(), qo) and np.array_equal(s.cpu().numpy(), so)


def test_gradient_against_differences():
    """Of sum(da a) by u, in fp64 from the device's a: with step d the
    difference is off by d^2 |a'''| / 6 < d^2 |l| and the fp32 a by 13 u |a| / d
    each: at d = 2^-6, |l| <= 3, |a| <= 12 below 2e-3 of values up to 10."""
    rng = np.random.default_rng(4)
    d = 2.0 ** -6
    u = np.round(rng.uniform(-3, 3, (1, 256)) * 64) / 64
    uq = torch.zeros((1, 256), dtype=torch.uint8, device=DEV)

    def a_of(v):
        # a checkpoint that holds one value exactly: E4M3 1.0 with the value as its scale, column by column
        out = np.zeros(128)
        for c in (0, 5, 77):
            q = np.zeros((1, 256), np.uint8)
            q[0, c] = q[0, 128 + c] = 0x38
            s = np.array([[v[0, c], v[0, 128 + c]]], np.float32)
            got = T.swiglu_backward(torch.ones((1, 128), device=DEV), torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV),
                                    want_du=True, want_a=True)
            out[c] = host(got[3])[0, c]
            grads[c] = host(got[2])[0, [c, 128 + c]]
        return out

    grads = {}
    a_of(u)
    at = dict(grads)
    for half in (0, 1):
        lo, hi = u.copy(), u.copy()
        lo[0, half * 128:half * 128 + 128] -= d
        hi[0, half * 128:half * 128 + 128] += d
        diff = (a_of(hi) - a_of(lo)) / (2 * d)
        for c in (0, 5, 77):
            assert abs(diff[c] - at[c][half]) < 2e-3, (half, c)
    assert uq.sum() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_guard_bands(dtype):
    rng = np.random.default_rng(9)
    rows, inner = 37, 256
    wide = dev(draw(rng, (rows, 4 * inner + 64), dtype), dtype)
    u, da = wide[:, 64:64 + 2 * inner], wide[:, 64 + 2 * inner:64 + 3 * inner]
    a = T.swiglu_quantize(u)
    b = T.swiglu_quantize(u.contiguous())
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    kept = torch.zeros((rows, 2 * inner + 48), dtype=torch.uint8, device=DEV)
    kept[:, 16:16 + 2 * inner] = a[2]
    g = T.swiglu_backward(da, kept[:, 16:16 + 2 * inner], a[3].contiguous(), want_du=True, want_a=True)
    h = T.swiglu_backward(da.contiguous(), a[2], a[3], want_du=True, want_a=True)
    assert all(torch.equal(x, y) for x, y in zip(g, h))
    # a row does not depend on the others
    for n in (1, 5):
        c = T.swiglu_quantize(u[7:7 + n])
        assert all(torch.equal(x, y[7:7 + n]) for x, y in zip(c, a))
        c = T.swiglu_backward(da[7:7 + n], a[2][7:7 + n], a[3][7:7 + n], want_du=True, want_a=True)
        assert all(torch.equal(x, y[7:7 + n]) for x, y in zip(c, h))
    # outputs between guard bands, with any scale strides, through the C interface
    xt = B.FP8FG_BF16 if dtype == "bf16" else B.FP8FG_F32
    q = torch.full((rows, inner + 32), 0x55, dtype=torch.uint8, device=DEV)
    k = torch.full((rows, 2 * inner + 32), 0x55, dtype=torch.uint8, device=DEV)
    s, ks = torch.full((rows, 8), -1.0, device=DEV), torch.full((rows, 16), -1.0, device=DEV)
    B.fp8_swiglu_quantize(u, xt, rows, inner, u.stride(0), None, 0, q[:, 16:], q.stride(0), s[:, 1:], 8, 3, k[:, 16:], k.stride(0),
                          ks[:, 1:], 16, 4)
    assert torch.equal(q[:, 16:16 + inner], a[0]) and torch.all(q[:, :16] == 0x55) and torch.all(q[:, 16 + inner:] == 0x55)
    assert torch.equal(k[:, 16:16 + 2 * inner], a[2]) and torch.all(k[:, :16] == 0x55) and torch.all(k[:, 16 + 2 * inner:] == 0x55)
    assert torch.equal(s[:, 1:5:3], a[1]) and torch.all(s[:, [0, 2, 3, 5, 6, 7]] == -1)
    assert torch.equal(ks[:, 1:14:4], a[3])


@pytest.mark.parametrize("count", [0, 1, 15, 16, 17, 40, 41, 1000, -3])
def test_rows_behind_the_used_ones_are_left_alone(count):
    rows, inner = 41, 256
    n = min(max(count, 0), rows)
    u = torch.randn((rows, 2 * inner), device=DEV).to(torch.bfloat16)
    u[n:] = float("nan")
    da = torch.randn((rows, inner), device=DEV).to(torch.bfloat16)
    used = torch.tensor([5, count], dtype=torch.int32, device=DEV)[1:]
    q, k = (torch.full((rows, w * inner), 0x55, dtype=torch.uint8, device=DEV) for w in (1, 2))
    s, ks = (torch.full((w * inner // 128, rows), -1.0, device=DEV).t() for w in (1, 2))
    B.fp8_swiglu_quantize(u, 0, rows, inner, 2 * inner, used, 0, q, inner, s, 1, rows, k, 2 * inner, ks, 1, rows)
    want = T.swiglu_quantize(u[:n].contiguous())
    for got, w in zip((q, s, k, ks), want):
        assert torch.equal(got[:n], w) and torch.all(got[n:] == (0x55 if got.dtype == torch.uint8 else -1))
    k[n:], ks[n:] = 0x7F, float("nan")
    dq = torch.full((rows, 2 * inner), 0x55, dtype=torch.uint8, device=DEV)
    ds = torch.full((2 * inner // 128, rows), -1.0, device=DEV).t()
    du, a = torch.full((rows, 2 * inner), 7.0, device=DEV).to(torch.bfloat16), torch.full((rows, inner), 7.0, device=DEV).to(torch.bfloat16)
    B.fp8_swiglu_backward(da, 0, rows, inner, inner, k, 2 * inner, ks, 1, rows, used, 0, dq, 2 * inner, ds, 1, rows, du, 2 * inner, a, inner)
    want = T.swiglu_backward(da[:n].contiguous(), k[:n], ks[:n], want_du=True, want_a=True)
    for got, w, left in zip((dq, ds, du, a), want, (0x55, -1, 7, 7)):
        assert torch.equal(got[:n], w) and torch.all(got[n:] == left)
    # the helper takes it too
    got = T.swiglu_quantize(u, used=used)
    assert torch.equal(got[0][:n], q[:n]) and torch.equal(got[2][:n], k[:n])


def test_outputs_left_out():
    rows, inner = 5, 128
    uq, us = (torch.randint(0, 0x70, (rows, 2 * inner), dtype=torch.uint8, device=DEV), torch.rand((rows, 2), device=DEV))
    da = torch.randn((rows, inner), device=DEV)
    want = T.swiglu_backward(da, uq, us, want_du=True, want_a=True)
    du, a = torch.empty_like(want[2]), torch.empty_like(want[3])
    B.fp8_swiglu_backward(da, 1, rows, inner, inner, uq, 2 * inner, us, 2, 1, None, 0, None, 0, None, 0, 0, du, 2 * inner, None, 0)
    B.fp8_swiglu_backward(da, 1, rows, inner, inner, uq, 2 * inner, us, 2, 1, None, 0, None, 0, None, 0, 0, None, 0, a, inner)
    assert torch.equal(du, want[2]) and torch.equal(a, want[3])


def test_extreme_values():
    """Gates far out, zeros of both signs, tiles whose scales are tiny or floored."""
    g = np.array([0.0, -0.0, 88.0, -88.0, 1e4, -1e4, 3e38, -3e38, 1e-40, -87.0, 20.0, -20.0, 1e-3, -1e-3, -104.0, 60.0], np.float32)
    u = np.zeros((4, 256), np.float32)
    u[:, :128] = np.tile(g, 8)
    u[0, 128:], u[1, 128:], u[2, 128:], u[3, 128:] = 1.0, -2.0, 2.0 ** -100, 0.0
    q, s, uq, us = T.swiglu_quantize(dev(u, "f32"))
    a = block.swiglu(u)
    # row 1: |3e38 * -2| = 6e38 passes fp32's largest number 3.4e38, so the fp32 product is infinite and the scale with it
    assert np.abs(a[1]).max() > np.finfo(np.float32).max and torch.isinf(s[1, 0])
    rows = [0, 2, 3]
    check_bytes(q[rows], s[rows], a[rows], 12 * U * np.abs(a[rows]) + 1e-30, False, "far gates")
    u[:, :128] = np.clip(u[:, :128], -104, 60)
    q, s, uq, us = T.swiglu_quantize(dev(u, "f32"))
    a = block.swiglu(u)
    check_bytes(q, s, a, 12 * U * np.abs(a) + TINY * 110 * np.abs(u[:, 128:]) + TINY, False, "gates")
    da = np.ones((4, 128), np.float32)
    kq, ks = oracle.quantize_1x128(u, oracle.SCALE_AMAX)
    got = T.swiglu_backward(dev(da, "f32"), torch.from_numpy(kq).to(DEV), torch.from_numpy(ks).to(DEV), want_du=True, want_a=True)
    duo, ao, e_du, e_a = grad_errors(da, block.kept(kq, ks))
    assert np.all(np.isfinite(host(got[2]))) and np.all(np.abs(host(got[2]) - duo) <= e_du) and np.all(np.abs(host(got[3]) - ao) <= e_a)


def test_empty():
    e = torch.empty((0, 512), device=DEV)
    q, s, uq, us = T.swiglu_quantize(e)
    assert q.shape == (0, 256) and s.shape == (0, 2) and uq.shape == (0, 512) and us.shape == (0, 4)
    out = T.swiglu_backward(torch.empty((0, 256), device=DEV), uq, us, want_du=True, want_a=True)
    assert out[0].shape == (0, 512) and out[2].shape == (0, 512) and out[3].shape == (0, 256)
    out = T.swiglu_backward_128x1(torch.empty((0, 256), device=DEV), uq, us)
    assert out[2].shape == (512, 0) and out[4].shape == (256, 0)


def test_helpers_refuse():
    u = torch.zeros((4, 512), device=DEV)
    uq, us = torch.zeros((4, 512), dtype=torch.uint8, device=DEV), torch.ones((4, 4), device=DEV)
    da = torch.zeros((4, 256), device=DEV)
    one = torch.zeros(1, dtype=torch.int32, device=DEV)
    for call in (lambda: T.swiglu_quantize(u.half()), lambda: T.swiglu_quantize(u.t()), lambda: T.swiglu_quantize(u[:, :511]),
                 lambda: T.swiglu_quantize(u, used=one.long()), lambda: T.swiglu_quantize(u, used=torch.zeros(2, dtype=torch.int32, device=DEV)),
                 lambda: T.swiglu_quantize(u, used=one.cpu()), lambda: T.swiglu_backward(da, uq[:, :256], us),
                 lambda: T.swiglu_backward(da, uq.float(), us), lambda: T.swiglu_backward(da, uq, us[:, :2]),
                 lambda: T.swiglu_backward(da, uq, us.double()), lambda: T.swiglu_backward(da[:2], uq, us),
                 lambda: T.swiglu_backward(da.double(), uq, us), lambda: T.swiglu_backward_128x1(da, uq, us.cpu())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: T.swiglu_quantize(u[:, :200].contiguous()), lambda: T.swiglu_backward_128x1(da, uq, us)):
        with pytest.raises(B.Fp8fgError) as e:
            call()
        assert e.value.status == B.FP8FG_ESHAPE
