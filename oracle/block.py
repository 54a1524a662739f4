"""Oracle of the silu gate, the router's balance loss and the norms around a
block (test infrastructure only), in 64-bit NumPy.

The arithmetic is float64 throughout; what the operators define as fp32 or as
the tensors' type is rounded there and nowhere else: a checkpoint's value (the
fp32 product of an E4M3 value and its scale) and h (the residual sum in the
tensors' type).

Parity: pinned by tests/test_oracle_block.py -- gradients against central
differences of the forward functions, the balance loss against its definition
token by token.
"""

import numpy as np

from .e4m3 import decode
from .moe import rmsnorm, rmsnorm_grad, round_to


def sigmoid(x):
    """(sigmoid, 1 - sigmoid), neither by cancellation."""
    t = np.exp(-np.abs(x))
    big, small = 1.0 / (1.0 + t), t / (1.0 + t)
    return np.where(x >= 0, big, small), np.where(x >= 0, small, big)


def swiglu(u):
    """silu(gate) * lin of u = [gate | lin], float64."""
    u = np.asarray(u, np.float64)
    g, l = np.split(u, 2, axis=1)
    return g * sigmoid(g)[0] * l


def kept(uq, us):
    """The values of an E4M3 checkpoint with 1x128 scales, fp32."""
    v = decode(uq).astype(np.float32)
    return v * np.repeat(np.asarray(us, np.float32), 128, axis=1)


def swiglu_grad(da, u):
    """([dgate | dlin], a) in float64 at the (checkpoint's) u."""
    u, da = np.asarray(u, np.float64), np.asarray(da, np.float64)
    g, l = np.split(u, 2, axis=1)
    s, r = sigmoid(g)
    return np.concatenate([da * l * s * (1 + g * r), da * g * s], axis=1), g * s * l


def shares(logits, score):
    """(share float64 [T][E], live [T]) of float32-held logits."""
    l = np.asarray(logits, np.float64)
    masked = np.isnan(l) | (l == -np.inf)
    out = np.zeros(l.shape)
    for t in range(l.shape[0]):
        ok = ~masked[t]
        if not ok.any():
            continue
        v = l[t, ok]
        # ratios of exp(l), or of the sigmoids also where they underflow
        logs = v if score == "softmax" else -np.logaddexp(0.0, -v)
        e = np.exp(logs - logs.max())
        out[t, ok] = e / e.sum()
    return out, ~masked.all(axis=1)


def _bounds(offsets, rows):
    off = [0, rows] if offsets is None else [min(max(int(o), 0), rows) for o in offsets]
    return list(zip(off, off[1:]))


def balance(logits, idx, offsets=None, score="softmax", scale=1.0):
    """(loss [S], counts int [S][E], slope [S][E]) in float64."""
    E, k = logits.shape[1], idx.shape[1]
    share, live = shares(logits, score)
    loss, counts, slopes = [], [], []
    for lo, hi in _bounds(offsets, logits.shape[0]):
        n = int(live[lo:hi].sum())
        flat = idx[lo:hi].ravel()
        c = np.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
        slope = scale * E / (k * float(n) ** 2) * c if n else np.zeros(E)
        counts.append(c)
        slopes.append(slope)
        loss.append(float((slope * share[lo:hi].sum(axis=0)).sum()))
    S = len(loss)
    return np.array(loss), np.array(counts).reshape(S, E), np.array(slopes).reshape(S, E)


def balance_grad(dloss, logits, slope, offsets=None, score="softmax", base=None):
    l = np.asarray(logits, np.float64)
    share, _ = shares(logits, score)
    out = np.zeros(l.shape) if base is None else np.asarray(base, np.float64).copy()
    for s, (lo, hi) in enumerate(_bounds(offsets, l.shape[0])):
        c = np.asarray(slope[s], np.float64) * (1.0 if dloss is None else float(dloss[s]))
        p = share[lo:hi]
        d = p * (c - (p @ c)[:, None])
        if score == "sigmoid":
            with np.errstate(invalid="ignore"):
                d = d * np.where(p > 0, sigmoid(np.where(p > 0, l[lo:hi], 0.0))[1], 0.0)
        out[lo:hi] += d
    return out


def block_sum(z, r, gamma_post, gate=None, residual_scale=1.0, block_scale=1.0, eps=1e-6):
    """(residual_scale r + block_scale gate norm(z) float64 before its rounding, rstd_post)."""
    _, post, t = rmsnorm(z, gamma_post, eps)
    if gate is not None:
        t = t * np.asarray(gate, np.float64)
    return np.float64(residual_scale) * np.asarray(r, np.float64) + np.float64(block_scale) * t, post


def block_norm(z, r, gamma_post, gamma, gate=None, residual_scale=1.0, block_scale=1.0, eps=1e-6, bf16=False):
    """(h float32, y float64, rstd_post, rstd)."""
    h, post = block_sum(z, r, gamma_post, gate, residual_scale, block_scale, eps)
    h = round_to(h, bf16)
    _, rstd, y = rmsnorm(h, gamma, eps)
    return h, y, post, rstd


def block_norm_grad(dy, z, h, gamma_post, gamma, rstd_post, rstd, gate=None, residual_scale=1.0, block_scale=1.0, dh=None):
    """(dz, dr, dgamma_post, dgamma, dgate by element) in float64."""
    dH, dgamma = rmsnorm_grad(dy, h, gamma, rstd, dh)
    g = 1.0 if gate is None else np.asarray(gate, np.float64)
    t = np.float64(block_scale) * dH
    dz, dgamma_post = rmsnorm_grad(t * g, z, gamma_post, rstd_post)
    zh = np.asarray(z, np.float64) * np.asarray(rstd_post, np.float64)[:, None]
    return dz, np.float64(residual_scale) * dH, dgamma_post, dgamma, t * zh * np.asarray(gamma_post, np.float64)
