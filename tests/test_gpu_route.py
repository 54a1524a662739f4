"""GPU parity of the router and its gradient against the 64-bit oracle.

The indexes have to be the oracle's exactly: scores are rounded once to
fp32, choices are one fp32 addition, ties go to the lower index.

Tolerances (u = 2^-24): weights: k <= 64 additions of positive scores, their
own rounding, a quotient and a product: 70 u relative.  Gradient: with the
fp32 exponential within 2 ulp and at most 1024 / 64 + 6 additions on any
term, |err| <= 64 u (|v_e| + sum_i |v_i| s_i) s_e (scores normalised as in the
formula), then the type's rounding."""

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


def check(l, k, dtype="f32", **kw):
    l = moe.round_to(l, dtype == "bf16")
    bias = kw.pop("bias", None)
    idx, w = T.route(dev(l, TYPES[dtype]), k, bias=None if bias is None else dev(bias), **kw)
    io, wo = moe.route(l, k, bias=bias, **kw)
    got = idx.cpu().numpy()
    bad = np.flatnonzero(np.any(got != io, axis=1))
    assert bad.size == 0, (bad[:4], got[bad[:2]], io[bad[:2]])
    assert np.all(np.abs(w.cpu().numpy() - wo) <= 70 * U * np.abs(wo) + 1e-37)
    return l, io


# experts, k, groups, top_groups, group_top
SHAPES = [(1, 1, 1, 1, 2), (2, 2, 2, 1, 1), (8, 2, 1, 1, 2), (16, 8, 1, 1, 2), (60, 4, 1, 1, 2), (64, 6, 8, 3, 1),
          (65, 5, 5, 2, 2), (72, 8, 8, 4, 2), (128, 8, 4, 4, 2), (160, 6, 8, 3, 1), (192, 8, 6, 2, 2),
          (252, 7, 6, 3, 2), (256, 8, 8, 4, 2), (256, 1, 64, 5, 2), (257, 64, 1, 1, 2), (300, 8, 100, 9, 2),
          (384, 8, 1, 1, 2), (512, 10, 16, 4, 2), (1000, 33, 8, 7, 2), (1024, 64, 1024, 100, 2), (1024, 8, 2, 1, 1)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "E%d_k%d_g%d_%d_%d" % s)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route(shape, score):
    E, k, groups, top_groups, group_top = shape
    say("route %s %s" % (shape, score))
    rng = np.random.default_rng(E + k)
    for rows, dtype, with_bias, renorm in ((1, "f32", True, True), (67, "bf16", False, True), (130, "f32", True, False)):
        l = rng.standard_normal((rows, E)) * 2
        bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if with_bias else None
        check(l, k, dtype, bias=bias, score=score, groups=groups, top_groups=top_groups, group_top=group_top,
              renorm=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (8, 3)])
def test_ties_go_to_the_lower_index(score, groups, top_groups):
    rng = np.random.default_rng(5)
    l = np.round(rng.standard_normal((64, 96)))
    l[0] = 0.0
    check(l, 12, score=score, groups=groups, top_groups=top_groups)
    check(l, 12, score=score, groups=groups, top_groups=top_groups, bias=np.zeros(96, np.float32) - np.float32(0))
    check(l, 12, score=score, groups=groups, top_groups=top_groups, group_top=1,
          bias=(np.round(rng.standard_normal(96)) / 4).astype(np.float32))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,top_groups", [(40, 1, 1), (40, 8, 3), (160, 4, 2), (320, 8, 2)])
def test_masks_and_extreme_logits(score, E, groups, top_groups):
    rng = np.random.default_rng(E)
    low = float(np.finfo(np.float32).min)
    rows = []
    base = rng.standard_normal((12, E))
    rows.append(np.full(E, -np.inf))                      # nothing left
    rows.append(np.full(E, np.nan))
    rows.append(np.full(E, low))                          # numbers all the same
    rows.append(np.full(E, np.inf))
    for i, v in enumerate((-np.inf, np.nan, low, np.inf)):
        a = base[i].copy()
        a[rng.permutation(E)[: E - 3]] = v                # three ordinary ones
        rows.append(a)
        a = base[i + 4].copy()
        a[rng.permutation(E)[:2]] = v
        rows.append(a)
    a = np.full(E, -np.inf)
    a[E - 1] = 0.5                                        # one candidate, in the last group
    rows.append(a)
    a = base[9] * 200                                     # scores that underflow
    rows.append(a)
    a = np.full(E, -np.inf)
    a[: E // max(groups, 2)] = base[10][: E // max(groups, 2)]  # whole groups masked
    rows.append(a)
    l = np.stack(rows)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    with np.errstate(all="ignore"):
        for renorm in (False, True):
            for b in (None, bias):
                check(l, 6, score=score, groups=groups, top_groups=top_groups, renorm=renorm, bias=b)
    nb = bias.copy()
    nb[3], nb[7], nb[9] = np.nan, -np.inf, np.inf
    check(base, 6, score=score, groups=groups, top_groups=top_groups, bias=nb)


def test_near_scores_are_told_apart():
    # choices one fp32 step apart, reached through the score's rounding: the
    # bias undoes all but the last bits of the score
    rng = np.random.default_rng(6)
    l = (rng.standard_normal((400, 64))).astype(np.float32)
    for row in range(0, 400, 8):
        s = moe.scores(l[row], "sigmoid").astype(np.float32)
        check(l[row:row + 8], 8, score="sigmoid", bias=(np.float32(1.0) - s))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_rows(dtype):
    rng = np.random.default_rng(7)
    wide = moe.round_to(rng.standard_normal((33, 200)), dtype == "bf16")
    d = dev(wide, TYPES[dtype])
    for E, at in ((100, 3), (64, 1), (129, 7)):
        idx, w = T.route(d[:, at:at + E], 5)
        io, wo = moe.route(wide[:, at:at + E], 5)
        assert np.array_equal(idx.cpu().numpy(), io)
        dl = T.route_backward(torch.ones_like(w), d[:, at:at + E], idx, renorm=False)
        dc = T.route_backward(torch.ones_like(w), d[:, at:at + E].contiguous(), idx, renorm=False)
        assert torch.equal(dl, dc)
    idx, w = T.route(d[:0], 5)
    assert idx.shape == (0, 5) and w.shape == (0, 5)
    assert T.route_backward(w, d[:0], idx).shape == (0, 200)


@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (60, 4), (64, 64), (65, 5), (160, 6), (256, 8), (257, 33), (1000, 8),
                                 (1024, 64)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient(E, k, score, renorm, dtype):
    rng = np.random.default_rng(E + k)
    rows = 29
    l = moe.round_to(rng.standard_normal((rows, E)) * 2, dtype == "bf16")
    idx = np.stack([rng.permutation(E)[:k] for _ in range(rows)]).astype(np.int32)
    idx[3, k // 2:] = -1
    idx[4, :] = -1
    idx[5, 0] = E
    if E > 4:
        l[6, rng.permutation(E)[: E // 2]] = -np.inf
        l[7, 2] = np.nan
        l[8, 1] = np.inf
        l[9] = -np.inf
        l[10] = np.finfo(np.float32).min if dtype == "f32" else -3.0e38
    l = moe.round_to(l, dtype == "bf16")
    dw = rng.standard_normal((rows, k)).astype(np.float32)
    got = T.route_backward(dev(dw), dev(l, TYPES[dtype]), torch.from_numpy(idx).to(DEV), score=score, renorm=renorm,
                           scale=1.5).float().cpu().numpy()
    with np.errstate(all="ignore"):
        ref = moe.route_grad(dw, l, idx, score=score, renorm=renorm, scale=1.5)
    size = np.zeros((rows, E))
    for t in range(rows):
        keep = [j for j in range(k) if 0 <= idx[t, j] < E]
        at = idx[t, keep]
        v = np.zeros(E)
        v[at] = np.abs(dw[t, keep]) * 1.5
        if renorm:
            s = np.zeros(E)
            if score == "softmax":
                s[at] = moe.scores(l[t, at], "softmax")
            else:
                s[at] = moe.scores(l[t], score)[at]
                s = s / max(s.sum(), 1e-300)
            size[t, at] = (s * (v + np.sum(v * s)))[at]
        else:
            s = moe.scores(l[t], score)
            size[t] = s * (v + (np.sum(v * s) if score == "softmax" else 0))
    tol = 64 * U * size + (UB * np.abs(ref) if dtype == "bf16" else 0) + 1e-37
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    assert bad.size == 0, [(int(t), int(e), got[t, e], ref[t, e]) for t, e in bad[:5]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences_of_the_kernel(score, renorm):
    # loss = sum of w dw over the kernel's own weights; a wide gap around the
    # k-th expert keeps the choice constant
    rng = np.random.default_rng(9)
    rows, E, k = 6, 24, 4
    l = rng.standard_normal((rows, E)).astype(np.float32) * 0.5
    for t in range(rows):
        l[t, rng.permutation(E)[:k]] += 2.5
    dw = rng.standard_normal((rows, k))
    idx, w = T.route(dev(l), k, score=score, renorm=renorm, scale=1.3)

    def loss(a):
        i, v = T.route(dev(a), k, score=score, renorm=renorm, scale=1.3)
        v = v.cpu().numpy().astype(np.float64)
        order = np.argsort(i.cpu().numpy(), axis=1)
        assert np.array_equal(np.take_along_axis(i.cpu().numpy(), order, 1), np.sort(idx.cpu().numpy(), axis=1))
        first = np.argsort(idx.cpu().numpy(), axis=1)
        return np.sum(np.take_along_axis(v, order, 1) * np.take_along_axis(dw, first, 1))

    dl = T.route_backward(dev(dw), dev(l), idx, score=score, renorm=renorm, scale=1.3).cpu().numpy().astype(np.float64)
    noise = 2.0 ** -20 * np.sum(np.abs(dw) * w.cpu().numpy())
    for _ in range(4):
        v = rng.uniform(-1, 1, (rows, E))
        diff = [(loss(l + d * v) - loss(l - d * v)) / (2 * d) for d in (2.0 ** -4, 2.0 ** -5)]
        assert abs(diff[1] - np.sum(dl * v)) <= abs(diff[0] - diff[1]) + noise / 2.0 ** -5 + 2.0 ** -20


@pytest.mark.parametrize("E,k,groups,top_groups,group_top", [
    (8, 2, 1, 1, 2), (64, 6, 8, 3, 1), (100, 16, 1, 1, 2), (160, 6, 8, 3, 1), (240, 8, 6, 2, 2), (252, 7, 6, 3, 2),
    (256, 8, 8, 4, 2), (256, 8, 4, 1, 2), (256, 17, 1, 1, 2), (256, 8, 16, 5, 2), (256, 8, 32, 5, 2), (257, 8, 1, 1, 2),
    (30, 3, 15, 4, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_many_rows_match_few(E, k, groups, top_groups, group_top, score):
    # long calls run several tokens to a wave: the same experts as short
    # calls choose, and the oracle's on a sample with ties, masks and extremes
    say("route of many rows: %d experts" % E)
    rng = np.random.default_rng(E + groups)
    rows = 4099
    l = (rng.standard_normal((rows, E)) * 2).astype(np.float32)
    l[::7] = np.round(l[::7])
    l[5::50, : E // 2] = -np.inf
    l[6::50] = -np.inf
    l[8::50, E - 1] = np.nan
    l[9::50, 0] = np.inf
    l[10::50] *= 100
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32)
    kw = dict(score=score, groups=groups, top_groups=top_groups, group_top=group_top, scale=1.5)
    d, b = dev(l), dev(bias)
    idx, w = T.route(d, k, bias=b, **kw)
    few = [T.route(d[i:i + 1000], k, bias=b, **kw) for i in range(0, rows, 1000)]
    assert torch.equal(idx, torch.cat([f[0] for f in few]))
    assert torch.all((w - torch.cat([f[1] for f in few])).abs() <= 140 * U * w.abs())
    at = np.concatenate([np.arange(0, 70), np.arange(rows - 9, rows)])
    with np.errstate(all="ignore"):
        io, wo = moe.route(l[at], k, bias=bias, **kw)
    assert np.array_equal(idx.cpu().numpy()[at], io)
    assert np.all(np.abs(w.cpu().numpy()[at] - wo) <= 70 * U * np.abs(wo) + 1e-37)


@pytest.mark.parametrize("E,groups,top_groups,rows", [(4, 1, 1, 3), (96, 8, 3, 5), (256, 1, 1, 7), (256, 8, 4, 2600),
                                                      (300, 100, 9, 5), (1024, 4, 2, 3)])
@pytest.mark.parametrize("gap", [5.0, 100.0, 200.0, 1e4])
def test_renormalised_softmax_of_experts_far_below_the_top(E, groups, top_groups, rows, gap):
    # the bias keeps the first expert out, whose logit is `gap` above the
    # rest: the others' scores underflow, their shares do not.  The choice is
    # the bias's, so the differences of the kernel's weights are its gradient.
    say("route below the top: %d experts, gap %g" % (E, gap))
    rng = np.random.default_rng(E + rows)
    k = min(3, E - 1)
    l = rng.uniform(-1, 1, (rows, E)).astype(np.float32)
    l[:, 0] = gap
    bias = np.zeros(E, np.float32)
    size = E // groups
    picked = rng.permutation(np.arange(1, size))[:k] if size > k else np.arange(1, 1 + k)
    bias[picked] = 4 + 2.0 * np.arange(picked.size)
    bias[0] = -4.0
    kw = dict(groups=groups, top_groups=top_groups, scale=1.5)
    idx, w = T.route(dev(l), k, bias=dev(bias), **kw)
    got = idx.cpu().numpy()
    with np.errstate(all="ignore"):
        io, wo = moe.route(l[:8], k, bias=bias, **kw)
    assert np.array_equal(got[:8], io) and np.all(got > 0)
    e = np.exp(np.take_along_axis(l, got, 1).astype(np.float64))
    share = 1.5 * e / e.sum(1, keepdims=True)
    assert np.all(np.abs(w.cpu().numpy() - share) <= 70 * U * share)
    assert np.all(np.abs(w.cpu().numpy()[:8] - wo) <= 70 * U * np.abs(wo) + 1e-37)

    dw = rng.standard_normal((rows, k)).astype(np.float32)
    dl = T.route_backward(dev(dw), dev(l), idx, scale=1.5).cpu().numpy().astype(np.float64)

    def loss(a):
        i, v = T.route(dev(a), k, bias=dev(bias), **kw)
        assert torch.equal(i, idx)
        return np.sum(v.cpu().numpy().astype(np.float64) * dw, axis=1)

    # a central difference is off by its truncation, which twice the step has
    # four times of, by the weights' rounding (2^-20 of their size, over the
    # step) and the gradient's own (128 u of it), 2^-15 of it together
    v = rng.uniform(-1, 1, (rows, E))
    diff = [(loss(l + d * v) - loss(l - d * v)) / (2 * d) for d in (2.0 ** -3, 2.0 ** -4)]
    bound = np.abs(diff[0] - diff[1]) + 2.0 ** -15 * np.sum(np.abs(dw * w.cpu().numpy()), axis=1)
    assert np.all(np.abs(diff[1] - np.sum(dl * v, axis=1)) <= bound)


# Rows of 96 float32 logits (bytes in hex) with a score so near the middle of
# two fp32 numbers that the order of the softmax's fp64 sum decides it.
NEAR = [
    ("234471c0f0d279bfd16625c0663cfebe0fdb93bd453b59c0b87280bfe59b57c09ae35f404cf70fc0823438bfac64bbbf72e506c0a06f933f"
     "86650bbf3f77573ed59e39402fb1974066e74f3cf741be3ed98922bebadf2940dc94da3f88cf304088e5a0bf719e4f40c3d82a3f0dad263f"
     "18430ec04efc11c099cd774096eff23e8a0cbebdce7f96401bdf4ec0431cfcbebc9f22bf8d2aa93fa077034000c3dcbf24445bc0991492be"
     "04fbe13fac161e4088142240b4e7b7bf01c337bf7cce99c0123f983f06af9a3ffd385fc0d8c3b23fa561fcbf61cd06401a9e823ee33433c0"
     "7d5f373f0a3e2c401bb0573e6fdb1940b7df1e404cdbaf3ff88012c07d3f7c404a62be3fbff7833f5b25ce3fd101ff3fcf75a43f2202cabf"
     "819cdcbf2eb7f6befa62f43eb8f05140869f983eb3dd543dbc6850bf228ab23fc919a2be92b4b9bf1dcb05bf2da264bf5d98503e330e78be"
     "ec9c98c08efb1b406f9be9bf1719c93f9e0723bec6b31e401ae81dc02abbcb3fdc0d23406f568cbeed1b833fc29d3f40"),
    ("cb9cf43f0e569e3f6ab7c23e0b14d33fbff18e3f343303c0f8a20bc088d307c0b969bfbfe9840940eb3d9e3fa0a061c0e1bf25bf804bccbf"
     "ebc50e3fc16e58c0d7b1f6be55092fbb4787e1bf95bbd1beb452cabfe64005bfef52693fca9f3240146f96bf4596d73fce0a3ac022cc6340"
     "46ed1cbf252b08c0794eefbf318c14be50631440e68af3bfde738440364c9f3fe250963f62f76cbd3d6c923ed05b3040da04ba3f366d9abf"
     "0a049d40dca6d43fdf63543f5630a7bf886e053f0479174009dd1440164a22bfa9b0483f6aac133fc4b2ce3fea4ccd3ee8a4c83e4a7e3bc0"
     "0beccb3f5d05c13ff9275340ef79bebfa19794c02b0f0040ff84554061059bbf9533aebff4c53dc00d4ca73f51a28ebf37071840dfc7843f"
     "ee2c05c0dbffc53ebce41e40457d173e3755a3bc1fafc9bff4cc7740b6dbd63edd1d903f35bc39c081316f3d77cb8e3fd80cc2bff7160bbf"
     "06341ebececbde3e6a64c4bf0dd954bfe0bf6bc0f3657dc0938d6a40816f663f9d3d32bedadb34c04d0614c0063bddbe"),
]


@pytest.mark.parametrize("row", NEAR, ids=["a", "b"])
def test_a_tokens_weights_do_not_depend_on_the_number_of_tokens(row):
    l = torch.from_numpy(np.frombuffer(bytes.fromhex(row), np.float32).copy()).to(DEV).expand(2700, -1).contiguous()
    idx, w = T.route(l, 32, renorm=False)
    one = T.route(l[:1], 32, renorm=False)
    assert torch.equal(idx, one[0].expand_as(idx)) and torch.equal(w, one[1].expand_as(w))
    s = moe.scores(l[0].cpu().numpy(), "softmax")[one[0][0].cpu().numpy()]
    assert np.all(np.abs(one[1][0].cpu().numpy() - s) <= 1.001 * U * s)


@pytest.mark.parametrize("E,k,groups,top_groups", [(96, 32, 1, 1), (100, 16, 1, 1), (240, 8, 6, 2), (256, 8, 8, 4), (256, 32, 1, 1)])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_long_and_short_calls_agree_bit_for_bit(E, k, groups, top_groups, renorm, score):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(E + k)
    l = torch.randn((16384, E), generator=gen, device=DEV) * 2
    kw = dict(groups=groups, top_groups=top_groups, renorm=renorm, score=score, scale=1.5)
    idx, w = T.route(l, k, **kw)
    few = [T.route(l[i:i + 2048], k, **kw) for i in range(0, 16384, 2048)]
    assert torch.equal(idx, torch.cat([f[0] for f in few])) and torch.equal(w, torch.cat([f[1] for f in few]))


@pytest.mark.parametrize("E,k,groups,top_groups", [(64, 6, 8, 3), (128, 8, 4, 2), (256, 8, 1, 1), (256, 8, 8, 4), (200, 8, 1, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [2600, 77])
def test_rows_by_16_bytes_and_by_elements(E, k, groups, top_groups, score, dtype, rows):
    # aligned rows are read 16 bytes at a time; rows that start elsewhere, or
    # a bias that does, element by element: the same results, the oracle's
    say("route by 16 bytes and elements: %d x %d %s" % (rows, E, dtype))
    rng = np.random.default_rng(E + rows)
    l = moe.round_to(rng.standard_normal((rows, E)) * 2, dtype == "bf16")
    l[::9] = np.round(l[::9])
    l[4::40, : E // 2] = -np.inf
    l[6::40, 1] = np.nan
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32)
    d, b = dev(l, TYPES[dtype]), dev(bias)
    kw = dict(score=score, groups=groups, top_groups=top_groups, scale=1.5)
    idx, w = T.route(d, k, bias=b, **kw)
    at = np.r_[0:48, rows - 20:rows]
    with np.errstate(all="ignore"):
        io, wo = moe.route(l[at], k, bias=bias, **kw)
    assert np.array_equal(idx.cpu().numpy()[at], io)
    assert np.all(np.abs(w.cpu().numpy()[at] - wo) <= 70 * U * np.abs(wo) + 1e-37)
    wide = torch.zeros((rows, E + 9), dtype=d.dtype, device=DEV)
    far = torch.zeros(E + 1, device=DEV)
    far[1:] = b
    for start in (0, 1, 8):       # an odd pitch; and an odd start; an aligned start of rows at an odd pitch
        wide[:, start:start + E] = d
        for bb in (b, far[1:]):
            i2, w2 = T.route(wide[:, start:start + E], k, bias=bb, **kw)
            assert torch.equal(idx, i2) and torch.equal(w, w2)
    i2, w2 = T.route(d, k, bias=far[1:], **kw)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
