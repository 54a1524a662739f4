"""The balance loss of logits that lie far from 0: a softmax does not know a
common offset, a sigmoid's small scores keep their relative accuracy.

Of sequences of one token with 16 experts the loss is the sum of k shares by
exact counts, so that its error is the shares' own.  Bounds, derived (u =
2^-24; D the largest logit less the smallest of a token):
  * exp within 2 ulp: 4 u; where it is formed below the largest logit that
    difference's rounding too, D u.
  * a softmax's score (4 + D) u; of a sigmoid also 1 + t (u, and t's error), the
    hardware's reciprocal (2 u) and a product: (4 + D) + 4 + 1 + 2 + 1 u.
  * a share: its score and their sum (the same error weighted, and 3 + 4
    additions), a reciprocal with a correction step 2 u, a product u.
  * the k shares are added in fp64 and the loss rounded once: u.
Together (2 (4 + D) + 11) u of a softmax, (2 (12 + D) + 11) u of a sigmoid.  In
sequences of n tokens a share's sum over the tokens passes at most n more
additions."""

import numpy as np
import pytest
import torch

from oracle import block, moe
from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
E, K = 16, 2


def dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(DEV).to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def run(l, idx, off, score, dtype):
    loss, counts, slope = T.balance_loss(dev(l, dtype), torch.from_numpy(idx).to(DEV), torch.from_numpy(off).to(DEV), score=score)
    want, co, _ = block.balance(l, idx, off, score, 1.0)
    assert np.array_equal(counts.cpu().numpy(), co)
    return loss.cpu().numpy().astype(np.float64), want, slope


def bound(l, score, n):
    D = np.max(l.max(axis=1) - l.min(axis=1))
    return (2 * ((4 if score == "softmax" else 12) + D) + 11 + n) * U


# (700 tokens of 16 experts are one launch, 1500 two)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,n", [(300, 1), (1500, 1), (300, 3), (1500, 50), (1500, 1500)])
@pytest.mark.parametrize("offset", [-80.0, -8.0, 0.0, 8.0, 20.0, 40.0, 60.0, 80.0])
def test_common_offset(offset, tokens, n, dtype):
    say("balance offset %g tokens %d of %d %s" % (offset, tokens, n, dtype))
    rng = np.random.default_rng(int(offset) % 97 + tokens + n)
    l = moe.round_to(rng.uniform(-1.5, 1.5, (tokens, E)) + offset, dtype == "bf16")
    idx = np.argsort(rng.random((tokens, E)), axis=1)[:, :K].astype(np.int32)
    off = np.minimum(np.arange(0, tokens + n, n), tokens).astype(np.int32)
    for score in ("softmax", "sigmoid"):
        loss, want, slope = run(l, idx, off, score, dtype)
        err = np.max(np.abs(loss / want - 1))
        assert err <= bound(l, score, 0 if n == 1 else n), (score, err / U)
        # the gradient too: its terms share (c - m) cancel, so by their magnitudes
        got = T.balance_loss_backward(None, dev(l, "f32"), slope, torch.from_numpy(off).to(DEV), score=score).cpu().numpy()
        sl = slope.cpu().numpy().astype(np.float64)
        c = np.concatenate([np.repeat(sl[s:s + 1], b - a, axis=0) for s, (a, b) in enumerate(zip(off, off[1:]))])
        share, _ = block.shares(l, score)
        size = share * (c + (c * share).sum(axis=1, keepdims=True))
        assert np.all(np.abs(got - block.balance_grad(None, l, sl, off, score)) <= (2 * bound(l, score, 0) + 24 * U) * size + 2.0 ** -125)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("far", [10.0, 30.0, 50.0, 65.0])
def test_small_shares_beside_a_large_one(far, score):
    """The chosen experts' logits lie far below another's, which keeps the sum of the
    scores ordinary: the differences need no rounding there, so D is no part of the
    bound (their scores are formed directly)."""
    rng = np.random.default_rng(int(far))
    tokens = 500
    l = (-far + rng.uniform(-1.5, 1.5, (tokens, E))).astype(np.float32)
    l[:, 0] = 0.75
    idx = np.stack([1 + rng.integers(0, 7, tokens), 8 + rng.integers(0, 8, tokens)], axis=1).astype(np.int32)
    off = np.arange(tokens + 1, dtype=np.int32)
    loss, want, _ = run(l, idx, off, score, "f32")
    err = np.max(np.abs(loss / want - 1))
    assert err <= (2 * (4 if score == "softmax" else 12) + 11) * U, err / U
