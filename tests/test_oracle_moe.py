"""Pins of oracle/moe.py: gradients against central differences of the
forward functions in 64 bits, the router against an exhaustive search, the
row movement against the properties that define it."""

import itertools

import numpy as np
import pytest

from oracle import moe

D = 1e-6          # difference step: truncation ~ D^2, cancellation ~ 1e-16 / D
TOL = 1e-7        # both far below it for values of order one


def norm64(x, gamma, eps):
    return x / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps) * gamma


@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.5])
def test_norm_gradient_against_differences(eps):
    rng = np.random.default_rng(1)
    h, dy, dh = (rng.standard_normal((3, 16)) for _ in range(3))
    gamma = rng.standard_normal(16)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    dx, dgamma = moe.rmsnorm_grad(dy, h, gamma, rstd, dh)
    loss = lambda a, g: np.sum(dy * norm64(a, g, eps)) + np.sum(dh * a)  # noqa: E731
    for _ in range(6):
        v, u = rng.standard_normal(h.shape), rng.standard_normal(16)
        num = (loss(h + D * v, gamma) - loss(h - D * v, gamma)) / (2 * D)
        assert abs(num - np.sum(dx * v)) < TOL * 100
        num = (loss(h, gamma + D * u) - loss(h, gamma - D * u)) / (2 * D)
        assert abs(num - np.sum(dgamma * u)) < TOL * 100


def test_norm_forward():
    rng = np.random.default_rng(2)
    x, r = (rng.standard_normal((4, 256)).astype(np.float32) for _ in range(2))
    g = rng.standard_normal(256).astype(np.float32)
    h, rstd, y = moe.rmsnorm(x, g, 1e-6, r)
    assert np.array_equal(h, x + r)
    assert np.allclose(np.mean((h * rstd[:, None]) ** 2, axis=1), 1.0, atol=1e-5)
    assert np.allclose(y, norm64(h.astype(np.float64), g.astype(np.float64), 1e-6), rtol=1e-14)
    hb, _, _ = moe.rmsnorm(x, g, 1e-6, r, bf16=True)
    assert np.all((hb.view(np.uint32) & 0xFFFF) == 0)
    assert np.max(np.abs(hb - h) / np.abs(h)) <= 2.0 ** -8


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    T, E, k = 4, 10, 3
    l = rng.standard_normal((T, E)).astype(np.float32)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[1, 2] = -1
    dw = rng.standard_normal((T, k))
    got = moe.route_grad(dw, l, idx, score=score, renorm=renorm, scale=1.7)

    def loss(a):
        total = 0.0
        for t in range(T):
            s = 1 / (1 + np.exp(-a[t])) if score == "sigmoid" else np.exp(a[t]) / np.sum(np.exp(a[t]))
            keep = idx[t] >= 0
            w = s[idx[t][keep]]
            w = w / w.sum() if renorm else w
            total += 1.7 * np.sum(dw[t][keep] * w)
        return total

    a = l.astype(np.float64)
    for t, e in itertools.product(range(T), range(E)):
        v = np.zeros_like(a)
        v[t, e] = D
        assert abs((loss(a + v) - loss(a - v)) / (2 * D) - got[t, e]) < TOL


@pytest.mark.parametrize("seed", range(20))
def test_route_is_the_best_set(seed):
    # the chosen experts have the largest sum of choices over every set of k
    # experts from every allowed set of groups, the groups being the best ones
    rng = np.random.default_rng(seed)
    groups, size, k = 3, 3, 3
    E = groups * size
    l = np.round(rng.standard_normal(E) * 2).astype(np.float32) / 2      # ties happen
    if seed % 4 == 0:
        l[rng.integers(0, E)] = -np.inf
    bias = (np.round(rng.standard_normal(E)) / 8).astype(np.float32)
    top_groups, group_top = 1 + seed % 2, 1 + seed % 2
    idx, w = moe.route_token(l, k, bias=bias, score="sigmoid", groups=groups, top_groups=top_groups,
                             group_top=group_top, renorm=False)
    s = np.where(l == -np.inf, 0, 1 / (1 + np.exp(-l.astype(np.float64)))).astype(np.float32)
    c = np.where(l == -np.inf, -np.inf, s + bias).astype(np.float32)
    live = [e for e in idx if e >= 0]
    assert len(set(live)) == len(live)
    assert np.allclose(w[:len(live)], s[live])
    assert list(c[live]) == sorted(c[live], reverse=True)
    value = [np.sum(np.sort(c[g * size:(g + 1) * size])[::-1][:group_top][np.isfinite(np.sort(
        c[g * size:(g + 1) * size])[::-1][:group_top])], dtype=np.float32) for g in range(groups)]
    used = {e // size for e in live}
    assert len(used) <= top_groups
    kept = max(itertools.combinations(range(groups), top_groups), key=lambda gs: (sum(value[g] for g in gs),
                                                                                 tuple(-g for g in gs)))
    assert used <= set(kept)
    pool = [e for g in kept for e in range(g * size, (g + 1) * size) if np.isfinite(c[e])]
    n = min(k, len(pool))
    assert len(live) == n
    best = max(itertools.combinations(pool, n), key=lambda es: (sum(float(c[e]) for e in es), tuple(-e for e in es)))
    assert set(live) == set(best)


def test_route_masks():
    nan, inf = np.nan, np.inf
    low = float(np.finfo(np.float32).min)
    idx, w = moe.route_token([-inf, nan, -inf], 2)
    assert list(idx) == [-1, -1] and list(w) == [0, 0]
    idx, w = moe.route_token([-inf, 1.0, nan], 2, renorm=True, scale=2.0)
    assert list(idx) == [1, -1] and list(w) == [2, 0]
    idx, w = moe.route_token([low, low, low], 2, renorm=False)        # numbers, not masks
    assert list(idx) == [0, 1] and np.allclose(w, 1 / 3)
    idx, w = moe.route_token([0.0, inf, inf], 2, renorm=False)
    assert list(idx) == [1, 2] and list(w) == [0.5, 0.5]
    idx, w = moe.route_token([low, low], 1, score="sigmoid", renorm=True)
    assert list(idx) == [0] and list(w) == [0]


@pytest.mark.parametrize("M,k,E", [(0, 2, 3), (1, 1, 1), (7, 3, 5), (20, 2, 4)])
def test_dispatch_properties(M, k, E):
    rng = np.random.default_rng(M)
    idx = rng.integers(-1, E + 1, size=(M, k)).astype(np.int32)
    offsets, pos, token = moe.dispatch(idx, E)
    assert offsets[0] == 0 and np.all(np.diff(offsets) >= 0)
    rows = np.where(pos >= 0, pos, -2 - pos).reshape(-1)
    assert sorted(rows) == list(range(M * k))
    for e in range(E):
        assert offsets[e + 1] - offsets[e] == np.sum(idx == e)
        where = [(t, j) for t in range(M) for j in range(k) if idx[t, j] == e]
        assert [pos[t, j] for t, j in where] == list(range(offsets[e], offsets[e + 1]))
        assert [token[pos[t, j]] for t, j in where] == [t for t, _ in where]
    assert np.all(token[offsets[E]:] == -1) and np.sum(pos < 0) == M * k - offsets[E]


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(5)
    idx = np.array([[0, 1], [2, -1], [1, 0]], np.int32)
    _, pos, _ = moe.dispatch(idx, 3)
    z, w, dy = rng.standard_normal((6, 4)), rng.standard_normal((3, 2)), rng.standard_normal((3, 4))
    dz, dw = moe.combine_grad(dy, z, pos, w)
    loss = lambda a, b: np.sum(dy * moe.combine(a, pos, b))  # noqa: E731
    for _ in range(4):
        u, v = rng.standard_normal(z.shape), rng.standard_normal(w.shape)
        assert abs((loss(z + D * u, w) - loss(z - D * u, w)) / (2 * D) - np.sum(dz * u)) < TOL * 10
        assert abs((loss(z, w + D * v) - loss(z, w - D * v)) / (2 * D) - np.sum(dw * v)) < TOL * 10
    assert np.all(dz[5] == 0) and dw[1, 1] == 0


@pytest.mark.parametrize("gap", [5.0, 100.0, 200.0, 1e4])
def test_weights_of_experts_far_below_the_top(gap):
    # the bias keeps the largest logit out: the weights are the others' shares, and the gradient is theirs
    l = np.array([gap, 0.0, 1.0, -1.0], np.float32)
    bias = np.array([-2.0, 0.5, 0.75, 0.0], np.float32)  # experts 2, 1 by it at every gap
    idx, w = moe.route_token(l, 2, bias=bias, scale=1.5)
    e = np.exp(1.0)
    assert list(idx) == [2, 1] and np.allclose(w, [1.5 * e / (1 + e), 1.5 / (1 + e)], rtol=1e-12)
    dw = np.array([1.0, -0.5])
    got = moe.route_grad(dw[None], l[None], idx[None], scale=1.5)[0]
    for n in range(4):
        v = np.zeros(4, np.float32)
        v[n] = 2.0 ** -6
        diff = (np.sum(dw * moe.route_token(l + v, 2, bias=bias, scale=1.5)[1]) -
                np.sum(dw * moe.route_token(l - v, 2, bias=bias, scale=1.5)[1])) / 2.0 ** -5
        assert abs(diff - got[n]) < 2.0 ** -12
