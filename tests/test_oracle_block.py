"""Pins of the oracle of the silu gate, the balance loss and the norms around a
block: gradients against central differences of the forward functions, the
loss against its definition.

A central difference with step d has an error of about d^2 |f'''| / 6 + 2^-52
|f| / d: with d = 1e-5 below 1e-8 of values near 1."""

import numpy as np
import pytest

from oracle import block, moe

D = 1e-5


def differences(f, x):
    out = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += D
        b[i] -= D
        out[i] = (f(a) - f(b)) / (2 * D)
    return out


def test_gate_and_its_gradient():
    rng = np.random.default_rng(0)
    u, da = rng.standard_normal((3, 8)) * 3, rng.standard_normal((3, 4))
    u[0, 0], u[0, 1], u[1, 0] = 0.0, 40.0, -40.0
    want = u[:, :4] / (1 + np.exp(-u[:, :4])) * u[:, 4:]
    assert np.allclose(block.swiglu(u), want, rtol=1e-14, atol=0)
    du, a = block.swiglu_grad(da, u)
    assert np.allclose(a, want, rtol=1e-14, atol=0)
    assert np.allclose(du, differences(lambda v: (block.swiglu(v) * da).sum(), u), atol=2e-8)


def test_checkpoint_values():
    q = np.zeros((1, 256), np.uint8)
    q[0, :3], q[0, 128] = (0x7E, 0x38, 0xB8), 0x01       # 448, 1, -1; 2^-9
    v = block.kept(q, np.array([[0.5, 2.0 ** 20]], np.float32))
    assert list(v[0, :4]) == [224.0, 0.5, -0.5, 0.0] and v[0, 128] == 2.0 ** 11


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_shares(score):
    l = np.array([[0.5, -1.0, 2.0, 0.0], [-300.0, -301.0, -np.inf, np.nan], [-np.inf] * 4, [800.0, -800.0, 3.0, 3.0]], np.float32)
    p, live = block.shares(l, score)
    assert list(live) == [True, True, False, True] and np.all(p[2] == 0) and np.all(p[1, 2:] == 0)
    s = np.exp(l[0].astype(float)) if score == "softmax" else 1 / (1 + np.exp(-l[0].astype(float)))
    assert np.allclose(p[0], s / s.sum(), rtol=1e-14)
    assert np.allclose(p[1, :2], np.array([1, np.exp(-1)]) / (1 + np.exp(-1)), rtol=1e-12)
    assert np.allclose(p[[0, 1, 3]].sum(axis=1), 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_by_its_definition(score):
    rng = np.random.default_rng(1)
    T, E, k = 11, 5, 2
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[3] = -np.inf
    l[5, 2] = np.nan
    idx = np.array([rng.choice(E, k, replace=False) for _ in range(T)])
    idx[3] = -1
    idx[6, 1] = 7
    off = [1, 4, 4, 10]
    loss, counts, slope = block.balance(l, idx, off, score, 0.3)
    share, live = block.shares(l, score)
    for s in range(3):
        tokens = [t for t in range(off[s], off[s + 1]) if live[t]]
        n, total = len(tokens), 0.0
        for e in range(E):
            c = sum(int(i == e) for t in tokens for i in idx[t])
            assert counts[s, e] == c
            if n:
                total += 0.3 * (E / (k * n) * c) * (sum(share[t, e] for t in tokens) / n)
        assert abs(loss[s] - total) < 1e-14
    assert np.all(slope[1] == 0) and loss[1] == 0
    # an even load and even shares give the scale
    even, _, _ = block.balance(np.zeros((4, 4), np.float32), np.arange(8).reshape(4, 2) % 4, None, score, 0.7)
    assert abs(even[0] - 0.7) < 1e-12


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient(score):
    rng = np.random.default_rng(2)
    l = rng.standard_normal((6, 4))
    idx = rng.integers(0, 4, (6, 2))
    off, d = [0, 2, 5], np.array([0.7, -1.3])
    _, _, slope = block.balance(l, idx, off, score)
    base = rng.standard_normal(l.shape)
    got = block.balance_grad(d, l, slope, off, score, base)
    assert np.array_equal(got[5], base[5])
    want = differences(lambda v: float((block.balance(v, idx, off, score)[0] * d).sum()), l)
    # (the loss counts tokens: its differences are those of fp64 logits)
    assert np.allclose(got - base, want, atol=1e-8)
    l[1, 2] = -np.inf
    assert np.isfinite(block.balance_grad(None, l, slope, off, score)).all()
    assert block.balance_grad(None, l, slope, off, score)[1, 2] == 0


@pytest.mark.parametrize("gate", ["none", "cols", "rows"])
def test_block_norm_and_its_gradient(gate):
    rng = np.random.default_rng(3)
    M, C = 3, 6
    z, r, dy, dh = (rng.standard_normal((M, C)) for _ in range(4))
    gp, gm = 1 + 0.3 * rng.standard_normal(C), 1 + 0.3 * rng.standard_normal(C)
    g = {"none": np.ones(C), "cols": rng.standard_normal(C), "rows": rng.standard_normal((M, C))}[gate]
    rs, bs, eps = 0.8, 0.3, 1e-3

    def forward(z, r, gp, gm, g):  # in float64 throughout: no rounding of h
        t = z / np.sqrt((z * z).mean(axis=1, keepdims=True) + eps) * gp * g
        h = rs * r + bs * t
        return h, h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * gm

    def loss(*a):
        h, y = forward(*a)
        return float((y * dy).sum() + (h * dh).sum())

    a = [z, r, gp, gm, g]
    h, y = forward(*a)
    post = 1 / np.sqrt((z * z).mean(axis=1) + eps)
    rstd = 1 / np.sqrt((h * h).mean(axis=1) + eps)
    dz, dr, dgp, dgm, dg = block.block_norm_grad(dy, z, h, gp, gm, post, rstd, None if gate == "none" else g, rs, bs, dh)
    for i, got in ((0, dz), (1, dr), (2, dgp), (3, dgm), (4, dg if gate == "rows" else dg.sum(axis=0))):
        want = differences(lambda v: loss(*[v if j == i else a[j] for j in range(5)]), a[i])
        assert np.allclose(got, want, atol=5e-8), i
    # the forward oracle on inputs that fp32 holds
    z32, r32 = z.astype(np.float32), r.astype(np.float32)
    ho, yo, po, ro = block.block_norm(z32, r32, gp, gm, g, rs, bs, eps)
    h2, y2 = forward(z32.astype(float), r32.astype(float), gp, gm, g)
    assert np.max(np.abs(ho - h2)) < 2.0 ** -23 and np.max(np.abs(yo - y2)) < 2.0 ** -21
    assert np.allclose(po, post, rtol=1e-6) and np.allclose(ro, rstd, rtol=1e-6)
    assert np.array_equal(block.block_norm(z32, r32, gp, gm, g, rs, bs, eps, bf16=True)[0], moe.round_to(h2, True))
