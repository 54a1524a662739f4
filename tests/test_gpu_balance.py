"""GPU parity of the router's balance loss and its gradient against the 64-bit
oracle.

Tolerances, derived (u = 2^-24; D the largest |l - max l| of a token, at most
100 since exp of less is 0 in fp32 sums):
  * a share: exp of a rounded difference (4 + D) u, of a sigmoid also its
    quotient 6 u; the sum's terms pass at most 16 + 6 additions with the same
    errors weighted: share (2 D + 50) u relative.
  * counts are exact; slope is one rounding of an fp64 value: 2 u.
  * loss: a chunk's tokens are added in fp32, at most one per wave and lane group
    at a time: (tokens / 8 + 16) u, chunks of at most tokens / 256 + 39, then
    fp64: (2 D + 50 + chunk / 8 + 16 + 4) u relative.
  * gradient: share (c - m), m = sum c share over at most 22 additions:
    (2 (2 D + 50) + 40) u share (|c| + sum |c| share), of a sigmoid 12 u more,
    then base's addition and the type's rounding.  The exponential is 0 below
    2^-126, so a share is off by up to 2^-126 too, and the gradient by 2^-126
    (|c| + sum |c| share), whose own product may be another 2^-126 below the
    normal numbers: 2^-125 (|c| + sum |c| share + 1)."""

import numpy as np
import pytest
import torch

from oracle import block, moe
from fp8_fine_grained_x1_amd import binding as B
from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

U, UB = 2.0 ** -24, 2.0 ** -8
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(x, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(DEV).to(TYPES[dtype])


def ints(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def spread(l):
    l = np.asarray(l, np.float64)
    with np.errstate(invalid="ignore"):
        d = np.where(np.isfinite(l), l, np.nan)
    ok = np.isfinite(d).any(axis=1)
    if not ok.any():
        return 0.0
    d = d[ok]
    return float(min(100.0, np.nanmax(np.nanmax(d, axis=1, keepdims=True) - d)))


def draw(rng, T_, E, k, dtype, masks=True):
    l = rng.standard_normal((T_, E)) * 1.5 + rng.standard_normal(E)
    l = moe.round_to(l, dtype == "bf16")
    idx = np.argsort(-(l + 0.5 * rng.standard_normal((T_, E))), axis=1)[:, :k].astype(np.int32)
    if masks and T_ > 2:
        l[rng.random((T_, E)) < 0.1] = -np.inf
        l[T_ // 3, 0] = np.nan
        pad = rng.random(T_) < 0.15
        pad[T_ // 2] = True
        l[pad] = -np.inf
        idx[pad] = -1
        idx[rng.random((T_, k)) < 0.05] = E + 3
    return l, idx


def offsets_of(rng, T_, S, inside=True):
    if S == 0:
        return np.zeros(1, np.int32)
    cuts = np.sort(rng.integers(0, T_ + 1, S + 1))
    if inside:
        cuts[0], cuts[-1] = 0, T_
    return cuts.astype(np.int32)


def check(l, idx, off, score, dtype, scale=1.0, dloss=None, base=None):
    ld, od = dev(l, dtype), None if off is None else ints(off)
    loss, counts, slope = T.balance_loss(ld, ints(idx), od, score=score, scale=scale)
    lo, co, so = block.balance(l, idx, off, score, np.float32(scale))
    assert np.array_equal(counts.cpu().numpy(), co)
    assert np.all(np.abs(slope.cpu().numpy() - so) <= 2 * U * np.abs(so))
    D = spread(l)
    chunk = l.shape[0] / 256 + 39
    assert np.all(np.abs(loss.cpu().numpy() - lo) <= (2 * D + 70 + chunk / 8) * U * np.abs(lo) + 1e-40), (loss, lo)
    sl = slope.cpu().numpy()
    got = T.balance_loss_backward(None if dloss is None else dev(dloss), ld, slope, od, score=score,
                                  base=None if base is None else dev(base, dtype)).float().cpu().numpy()
    want = block.balance_grad(dloss, l, sl, off, score, base)
    share, _ = block.shares(l, score)
    c = np.zeros(l.shape)
    for s, (a, b) in enumerate(block._bounds(off, l.shape[0])):
        c[a:b] = np.abs(sl[s].astype(np.float64) * (1.0 if dloss is None else dloss[s]))
    cc = c + (c * share).sum(axis=1, keepdims=True)
    err = (2 * (2 * D + 50) + 40 + 12) * U * share * cc + 2.0 ** -125 * (cc + 1)
    err = err + (UB if dtype == "bf16" else U) * np.abs(want) + (U * np.abs(base) if base is not None else 0)
    assert np.all(np.abs(got - want) <= err), float(np.max(np.abs(got - want) / err))
    return loss, counts, slope, got


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,experts,k,seqs", [(1, 4, 1, 1), (3, 1, 1, 2), (61, 16, 8, 3), (5, 7, 3, 9), (200, 64, 6, 1), (333, 160, 6, 5),
                                                 (512, 256, 8, 4), (513, 256, 8, 4), (700, 100, 4, 300), (1500, 256, 8, 1),
                                                 (2111, 63, 5, 17), (900, 257, 8, 3), (640, 512, 8, 2), (600, 1024, 64, 3), (999, 1001, 2, 2)])
def test_against_the_oracle(rows, experts, k, seqs, dtype, score):
    say("balance %d x %d k %d seqs %d %s %s" % (rows, experts, k, seqs, dtype, score))
    rng = np.random.default_rng(rows + experts + seqs)
    l, idx = draw(rng, rows, experts, k, dtype)
    off = offsets_of(rng, rows, seqs)
    check(l, idx, off, score, dtype, 0.01, rng.uniform(-1, 1, seqs).astype(np.float32),
          moe.round_to(rng.standard_normal((rows, experts)) * 1e-3, dtype == "bf16"))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_sequence_and_defaults(score):
    rng = np.random.default_rng(0)
    for rows in (40, 3000):
        l, idx = draw(rng, rows, 32, 4, "f32")
        a = check(l, idx, None, score, "f32")
        b = check(l, idx, np.array([0, rows]), score, "f32")
        assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3])) and np.array_equal(a[3], b[3])


@pytest.mark.parametrize("rows", [50, 2000])
def test_tokens_in_no_sequence_and_empty_sequences(rows):
    rng = np.random.default_rng(1)
    l, idx = draw(rng, rows, 24, 2, "f32")
    off = np.array([7, 7, 7, rows // 2, rows // 2, rows - 9, rows - 9], np.int32)
    base = rng.standard_normal((rows, 24)).astype(np.float32)
    l2 = l.copy()
    l2[:7], l2[rows - 9:] = np.nan, np.inf     # (not of any sequence)
    _, counts, slope, got = check(l, idx, off, "softmax", "f32", base=base)
    assert np.array_equal(got[:7], base[:7]) and np.array_equal(got[rows - 9:], base[rows - 9:])
    for s in (0, 1, 3, 5):
        assert int(counts[s].sum()) == 0 and float(slope[s].sum()) == 0
    a = T.balance_loss(dev(l), ints(idx), ints(off))
    b = T.balance_loss(dev(l2), ints(idx), ints(off))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_that_leave_the_rows():
    # held within the rows, whatever they are
    rng = np.random.default_rng(2)
    for rows in (60, 1100):
        l, idx = draw(rng, rows, 8, 2, "f32")
        check(l, idx, np.array([-5, 20, rows + 100], np.int32), "sigmoid", "f32")
        out = T.balance_loss(dev(l), ints(idx), ints([30, 10, 2 ** 31 - 1, -2 ** 31, 50]))
        g = T.balance_loss_backward(None, dev(l), out[2], ints([30, 10, 2 ** 31 - 1, -2 ** 31, 50]))
        assert out[0].shape == (4,) and g.shape == (rows, 8)
    torch.cuda.synchronize()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_logits(score):
    # scores that underflow keep their ratios; nothing overflows
    l = np.array([[-200.0, -201.0, -202.0, -250.0], [90.0, -90.0, 0.0, 1.0], [-3e38, -3e38, -3e38, -3e38], [3e38, 3e38, -3e38, 0.0],
                  [-120.0, 5.0, -np.inf, np.nan], [-np.inf] * 4, [1e-40, 0.0, -0.0, -1e-40]], np.float32)
    idx = np.array([[0, 1], [0, 3], [2, 3], [0, 1], [1, 0], [-1, -1], [3, 0]], np.int32)
    check(l, idx, None, score, "f32")


@pytest.mark.parametrize("rows", [9, 900])
def test_masked_tokens_do_not_count(rows):
    rng = np.random.default_rng(5)
    l, idx = draw(rng, rows, 16, 2, "f32", masks=False)
    keep = rng.random(rows) < 0.6
    keep[0] = True
    padded, pidx = l.copy(), idx.copy()
    padded[~keep], pidx[~keep] = -np.inf, -1
    a = T.balance_loss(dev(padded), ints(pidx))
    b = T.balance_loss(dev(l[keep]), ints(idx[keep]))
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert abs(float(a[0]) - float(b[0])) <= 200 * U * float(b[0])
    g = T.balance_loss_backward(None, dev(padded), a[2])
    assert torch.all(g[torch.from_numpy(~keep).to(DEV)] == 0)
    everything = T.balance_loss(torch.full((rows, 16), float("-inf"), device=DEV), torch.full((rows, 2), -1, dtype=torch.int32, device=DEV))
    assert all(float(t.abs().sum()) == 0 for t in everything)


def test_same_expert_twice_counts_twice():
    idx = ints([[3, 3], [3, 1]])
    _, counts, _ = T.balance_loss(torch.zeros((2, 4), device=DEV), idx)
    assert counts.tolist() == [[0, 1, 0, 3]]


@pytest.mark.parametrize("experts", [16, 18])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides(experts, dtype):
    # rows of another pitch and start: the same within the sums' order (rows of 4 elements at a time, or single ones)
    rng = np.random.default_rng(6)
    for rows in (70, 800):
        l, idx = draw(rng, rows, experts, 2, dtype, masks=False)
        a = T.balance_loss(dev(l, dtype), ints(idx))
        base = dev(rng.standard_normal((rows, experts)), dtype)
        ga = T.balance_loss_backward(None, dev(l, dtype), a[2], base=base).float()
        for pad in (1, 4, 8):
            wide = torch.zeros((rows, 2 * experts + pad), dtype=TYPES[dtype], device=DEV)
            wide[:, pad:pad + experts] = dev(l, dtype)
            wi = torch.zeros((rows, 7), dtype=torch.int32, device=DEV)
            wi[:, 3:5] = ints(idx)
            v = wide[:, pad:pad + experts]
            b = T.balance_loss(v, wi[:, 3:5])
            assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
            assert abs(float(a[0]) - float(b[0])) <= 200 * U * float(a[0])
            wb = torch.zeros((rows, 3 * experts + pad), dtype=TYPES[dtype], device=DEV)
            wb[:, pad:pad + experts] = base
            gb = T.balance_loss_backward(None, v, a[2], base=wb[:, pad:pad + experts]).float()
            assert torch.all((ga - gb).abs() <= (2 * UB if dtype == "bf16" else 2 * U) * ga.abs() + 200 * U * float(a[2].max()))
            # outputs between guard bands, through the C interface
            out = torch.full((rows, 2 * experts + pad), 7.0, dtype=TYPES[dtype], device=DEV)
            t = B.FP8FG_BF16 if dtype == "bf16" else B.FP8FG_F32
            B.fp8_balance_loss_backward(None, v, t, rows, experts, v.stride(0), a[2], None, 1, 0, wb[:, pad:], wb.stride(0),
                                        out[:, pad:], out.stride(0))
            assert torch.equal(out[:, pad:pad + experts].float(), gb)
            assert torch.all(out[:, :pad] == 7) and torch.all(out[:, pad + experts:] == 7)


def test_gradient_against_differences():
    """Of the fp32 loss (about 1, off by 90 u = 6e-6) with step 2^-3: each
    difference is off by 2 * 6e-6 / 2^-2 and by (2^-3)^2 / 6 |f'''| with |f'''| <=
    the slope (below 0.2): together below 6e-4."""
    rng = np.random.default_rng(7)
    l, idx = draw(rng, 12, 6, 2, "f32", masks=False)
    d = 2.0 ** -3
    for score in ("softmax", "sigmoid"):
        loss, _, slope = T.balance_loss(dev(l), ints(idx), score=score)
        assert float(slope.max()) < 0.2
        g = T.balance_loss_backward(None, dev(l), slope, score=score).cpu().numpy()
        for t, e in ((0, 0), (3, 5), (11, 2)):
            hi, lo = l.copy(), l.copy()
            hi[t, e] += d
            lo[t, e] -= d
            diff = (float(T.balance_loss(dev(hi), ints(idx), score=score)[0]) - float(T.balance_loss(dev(lo), ints(idx), score=score)[0])) / (2 * d)
            assert abs(diff - g[t, e]) < 6e-4


def test_empty():
    l, i = torch.empty((0, 8), device=DEV), torch.empty((0, 2), dtype=torch.int32, device=DEV)
    loss, counts, slope = T.balance_loss(l, i, ints([0, 0, 0]))
    assert loss.tolist() == [0, 0] and counts.shape == (2, 8) and int(counts.sum()) == 0 and float(slope.sum()) == 0
    assert T.balance_loss_backward(None, l, slope, ints([0, 0, 0])).shape == (0, 8)
    l, i = torch.zeros((3, 8), device=DEV), torch.zeros((3, 2), dtype=torch.int32, device=DEV)
    loss, counts, slope = T.balance_loss(l, i, ints([0]))
    assert loss.shape == (0,) and counts.shape == (0, 8)
    base = torch.randn((3, 8), device=DEV)
    assert torch.equal(T.balance_loss_backward(None, l, slope, ints([0]), base=base), base)


def test_results_repeat():
    rng = np.random.default_rng(8)
    l, idx = draw(rng, 5000, 256, 8, "f32")
    off = ints(offsets_of(rng, 5000, 7))
    a = T.balance_loss(dev(l), ints(idx), off)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, T.balance_loss(dev(l), ints(idx), off)))


def test_helpers_refuse():
    l, i, off = torch.zeros((4, 8), device=DEV), torch.zeros((4, 2), dtype=torch.int32, device=DEV), ints([0, 4])
    s = torch.zeros((1, 8), device=DEV)
    for call in (lambda: T.balance_loss(l.double(), i), lambda: T.balance_loss(l, i.long()), lambda: T.balance_loss(l, i[:3]),
                 lambda: T.balance_loss(l, i, off.long()), lambda: T.balance_loss(l, i, off[:0]), lambda: T.balance_loss(l, i, off.cpu()),
                 lambda: T.balance_loss_backward(None, l, s[:, :4]), lambda: T.balance_loss_backward(None, l, s, ints([0, 1, 2])),
                 lambda: T.balance_loss_backward(s[0, :2], l, s), lambda: T.balance_loss_backward(None, l, s, base=l[:2]),
                 lambda: T.balance_loss_backward(None, l, s, base=l.to(torch.bfloat16)), lambda: T.balance_loss_backward(None, l, s.double())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(B.Fp8fgError) as e:
        T.balance_loss(torch.zeros((4, 1025), device=DEV), i)
    assert e.value.status == B.FP8FG_EUNSUPPORTED
