"""GPU parity of the row movement (dispatch, combine and its gradient)
against the oracle.  Places, rows and scales are exact.  A combined value
sums k + 1 products in fp32: |err| <= (k + 2) u sum |w z|; a dot product over
C columns adds at most C / 512 + 16 terms on any path: (C / 512 + 20) u sum |dy z|
(u = 2^-24, plus bf16's rounding 2^-8 of the result)."""

import numpy as np
import pytest
import torch

from oracle import moe
from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

U, UB = 2.0 ** -24, 2.0 ** -8
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(x, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV).to(dtype)


def draw_idx(rng, M, k, E, drops):
    idx = rng.integers(0, E, size=(M, k)).astype(np.int32)
    if drops and M:
        idx[rng.random((M, k)) < 0.2] = -1
        idx.flat[0] = E + 5
        idx[-1] = -1
    return idx


def check_places(idx, E, got):
    offsets, pos, token = (t.cpu().numpy() for t in got)
    oo, po, to = moe.dispatch(idx, E)
    assert np.array_equal(offsets, oo)
    assert np.array_equal(pos, po)
    assert np.array_equal(token, to)
    return po, to


SHAPES = [(1, 1, 1, 128), (1, 8, 16, 7168), (3, 2, 5, 256), (64, 8, 16, 1152), (61, 8, 256, 384), (130, 1, 8, 128),
          (257, 3, 1024, 128), (500, 8, 60, 256), (1200, 2, 8, 128), (2049, 4, 160, 128), (6000, 8, 256, 128),
          (40000, 8, 300, 128), (1, 64, 1, 128)]


@pytest.mark.parametrize("M,k,E,C", SHAPES)
@pytest.mark.parametrize("drops", [False, True])
def test_dispatch_e4m3(M, k, E, C, drops):
    say("dispatch %d x %d over %d experts, %d columns" % (M, k, E, C))
    rng = np.random.default_rng(M + E)
    idx = draw_idx(rng, M, k, E, drops)
    x = rng.integers(0, 255, size=(M, C)).astype(np.uint8)
    s = rng.random((M, C // 128)).astype(np.float32)
    for layout in ("group_major", "row_major"):
        sd = torch.from_numpy(s).to(DEV)
        if layout == "group_major":
            sd = sd.t().contiguous().t()
        q, qs, *places = T.dispatch(torch.from_numpy(idx).to(DEV), E, torch.from_numpy(x).to(DEV), sd,
                                    scale_layout=layout)
        po, to = check_places(idx, E, places)
        assert np.array_equal(q.cpu().numpy(), np.where(to[:, None] >= 0, x[to], 0))
        assert np.array_equal(qs.cpu().numpy(), np.where(to[:, None] >= 0, s[to], np.float32(2.0 ** -126)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,k,E,C", [(1, 2, 4, 8), (70, 8, 16, 264), (900, 6, 64, 1032)])
def test_dispatch_other_types_and_strides(M, k, E, C, dtype):
    rng = np.random.default_rng(M)
    idx = draw_idx(rng, M, k, E, True)
    x = moe.round_to(rng.standard_normal((M, C + 24)), dtype == "bf16")
    wide = np.zeros((M, k + 3), np.int32)
    wide[:, 2:2 + k] = idx
    out, none, *places = T.dispatch(torch.from_numpy(wide).to(DEV)[:, 2:2 + k], E, dev(x, TYPES[dtype])[:, 8:8 + C])
    assert none is None
    po, to = check_places(idx, E, places)
    assert np.array_equal(out.float().cpu().numpy(), np.where(to[:, None] >= 0, x[to, 8:8 + C], 0))


def test_dispatch_one_expert_and_none():
    for e in (0, 3, -1):
        idx = np.full((3000, 3), e, np.int32)
        x = np.arange(3000 * 128, dtype=np.int64).astype(np.uint8).reshape(3000, 128)
        s = np.ones((3000, 1), np.float32)
        q, qs, *places = T.dispatch(torch.from_numpy(idx).to(DEV), 4, torch.from_numpy(x).to(DEV), torch.from_numpy(s).to(DEV))
        po, to = check_places(idx, 4, places)
        assert np.array_equal(q.cpu().numpy(), np.where(to[:, None] >= 0, x[to], 0))


def test_dispatch_of_no_tokens():
    idx = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    x = torch.empty((0, 256), dtype=torch.uint8, device=DEV)
    q, s, offsets, pos, token = T.dispatch(idx, 7, x, torch.empty((0, 2), device=DEV))
    assert q.shape == (0, 256) and torch.all(offsets == 0) and offsets.shape == (8,) and token.numel() == 0


CSHAPES = [(1, 1, 8), (1, 8, 7168), (5, 3, 264), (61, 8, 1152), (300, 6, 2048), (700, 2, 2056), (9, 64, 520),
           (3, 4, 16392)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,k,C", CSHAPES)
def test_combine(M, k, C, dtype):
    say("combine %d x %d, %d columns, %s" % (M, k, C, dtype))
    rng = np.random.default_rng(M + C)
    b16 = dtype == "bf16"
    for drops, weighted, with_base in ((False, True, True), (True, True, False), (True, False, True)):
        _, pos, token = moe.dispatch(draw_idx(rng, M, k, 16, drops), 16)
        z = moe.round_to(rng.standard_normal((M * k, C)), b16)
        w = rng.standard_normal((M, k)).astype(np.float32) if weighted else None
        base = moe.round_to(rng.standard_normal((M, C)), b16) if with_base else None
        zd = dev(z, TYPES[dtype])
        zd[torch.from_numpy(token).to(DEV) < 0] = float("nan")        # rows of dropped entries are not read
        y = T.combine(zd, torch.from_numpy(pos).to(DEV), None if w is None else dev(w),
                      base=None if base is None else dev(base, TYPES[dtype])).float().cpu().numpy()
        ref = moe.combine(z, pos, w, base)
        size = moe.combine(np.abs(z), pos, None if w is None else np.abs(w), None if base is None else np.abs(base))
        assert np.all(np.abs(y - ref) <= (k + 2) * U * size + (UB * np.abs(ref) if b16 else 0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,k,C", CSHAPES)
def test_combine_gradient(M, k, C, dtype):
    say("combine gradient %d x %d, %d columns, %s" % (M, k, C, dtype))
    rng = np.random.default_rng(M + C + 1)
    b16 = dtype == "bf16"
    for drops, weighted in ((False, True), (True, True), (True, False)):
        _, pos, token = moe.dispatch(draw_idx(rng, M, k, 16, drops), 16)
        z, dy = moe.round_to(rng.standard_normal((M * k, C)), b16), moe.round_to(rng.standard_normal((M, C)), b16)
        w = rng.standard_normal((M, k)).astype(np.float32) if weighted else None
        zd = dev(z, TYPES[dtype])
        zd[torch.from_numpy(token).to(DEV) < 0] = float("nan")
        torch.full((M * k, C), float("nan"), dtype=TYPES[dtype], device=DEV)   # what fresh memory may hold
        args = (dev(dy, TYPES[dtype]), zd, torch.from_numpy(pos).to(DEV), None if w is None else dev(w))
        dz, dw = T.combine_backward(*args)
        dzo, dwo = moe.combine_grad(dy, z, pos, w)
        assert np.all(np.abs(dz.float().cpu().numpy() - dzo) <= (UB if b16 else U) * np.abs(dzo))
        size = moe.combine_grad(np.abs(dy), np.abs(z), pos)[1]
        assert np.all(np.abs(dw.cpu().numpy() - dwo) <= (C / 512 + 20) * U * size)
        again = T.combine_backward(*args)
        assert torch.equal(dz, again[0]) and torch.equal(dw, again[1])


def test_combine_strides_and_places_out_of_range():
    rng = np.random.default_rng(2)
    z = dev(rng.standard_normal((40, 264 + 16)))[:, 8:8 + 264]
    base = dev(rng.standard_normal((10, 300)))[:, 4:4 + 264]
    w = dev(rng.standard_normal((10, 9)))[:, 3:7]
    pos = torch.from_numpy(rng.permutation(40).reshape(10, 4).astype(np.int32)).to(DEV)
    a = T.combine(z, pos, w, base=base)
    assert torch.equal(a, T.combine(z.contiguous(), pos, w.contiguous(), base=base.contiguous()))
    far = pos.clone()
    far[0, 1], far[1, 2], far[2, 3] = 40, 2 ** 31 - 1, -2 ** 31
    w0 = w.clone()
    w0[0, 1] = w0[1, 2] = w0[2, 3] = 0
    assert torch.equal(T.combine(z, far, w, base=base), T.combine(z, pos, w0, base=base))
    dy = dev(rng.standard_normal((10, 300)))[:, 4:4 + 264]
    b, c = T.combine_backward(dy, z, pos, w), T.combine_backward(dy.contiguous(), z.contiguous(), pos, w.contiguous())
    assert torch.equal(b[0], c[0]) and torch.equal(b[1], c[1])
    assert torch.all(T.combine_backward(dy, z, far, w)[1][[0, 1, 2], [1, 2, 3]] == 0)


def test_combine_without_tokens_or_rows():
    z = torch.empty((0, 64), device=DEV)
    pos = torch.empty((0, 3), dtype=torch.int32, device=DEV)
    assert T.combine(z, pos).shape == (0, 64)
    assert T.combine_backward(z, z, pos, None)[1].shape == (0, 3)
    base = torch.rand((5, 64), device=DEV)
    assert torch.equal(T.combine(z, torch.full((5, 2), -1, dtype=torch.int32, device=DEV), base=base), base)


def test_dispatch_gradient_is_combine_without_weights():
    # <dispatch(x), g> = <x, combine(g)> for every x and g
    rng = np.random.default_rng(4)
    idx = draw_idx(rng, 50, 4, 6, True)
    x, g = rng.standard_normal((50, 64)).astype(np.float32), rng.standard_normal((200, 64)).astype(np.float32)
    out, _, _, pos, _ = T.dispatch(torch.from_numpy(idx).to(DEV), 6, dev(x))
    back = T.combine(dev(g), pos)
    a = np.sum(out.cpu().numpy().astype(np.float64) * g)
    b = np.sum(x.astype(np.float64) * back.cpu().numpy())
    assert abs(a - b) <= 16 * U * np.sum(np.abs(out.cpu().numpy() * g))


def test_combine_gradient_against_differences_of_the_kernel():
    # combine is linear in z and in w, so a difference with any step is the
    # derivative, up to the rounding of both sides' fp32 results
    rng = np.random.default_rng(12)
    _, pos, _ = moe.dispatch(draw_idx(rng, 20, 3, 7, True), 7)
    p = torch.from_numpy(pos).to(DEV)
    z, dz_dir = (rng.standard_normal((60, 136)).astype(np.float32) for _ in range(2))
    w, dw_dir = (rng.standard_normal((20, 3)).astype(np.float32) for _ in range(2))
    dy = rng.standard_normal((20, 136)).astype(np.float32)
    dz, dw = (t.cpu().numpy().astype(np.float64) for t in T.combine_backward(dev(dy), dev(z), p, dev(w)))

    def loss(a, b):
        return np.sum(dy * T.combine(dev(a), p, dev(b)).cpu().numpy().astype(np.float64))

    for a, b, grad in (((z + dz_dir, w), (z - dz_dir, w), np.sum(dz * dz_dir)), ((z, w + dw_dir), (z, w - dw_dir), np.sum(dw * dw_dir))):
        size = sum(np.sum(np.abs(dy) * moe.combine(np.abs(x), pos, np.abs(y))) for x, y in (a, b))
        assert abs((loss(*a) - loss(*b)) / 2 - grad) <= 32 * U * size


@pytest.mark.parametrize("M,k,E", [(1549, 1, 40), (1550, 1, 40), (1095, 2, 9), (1096, 2, 9), (750, 4, 64), (751, 4, 64),
                                   (375, 8, 256), (376, 8, 256), (187, 16, 60), (188, 16, 60), (100, 17, 60)])
def test_dispatch_on_both_sides_of_one_launch(M, k, E):
    # sizes around the border between the one-launch and the three-launch form
    say("dispatch border %d x %d" % (M, k))
    rng = np.random.default_rng(M + k)
    idx = draw_idx(rng, M, k, E, True)
    x = rng.integers(0, 255, size=(M, 256)).astype(np.uint8)
    s = rng.random((M, 2)).astype(np.float32)
    q, qs, *places = T.dispatch(torch.from_numpy(idx).to(DEV), E, torch.from_numpy(x).to(DEV), torch.from_numpy(s).to(DEV))
    po, to = check_places(idx, E, places)
    assert np.array_equal(q.cpu().numpy(), np.where(to[:, None] >= 0, x[to], 0))
    assert np.array_equal(qs.cpu().numpy(), np.where(to[:, None] >= 0, s[to], np.float32(2.0 ** -126)))
