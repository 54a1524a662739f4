"""Oracle of the operators around the GEMMs of a mixture-of-experts layer
(test infrastructure only): the norm that produces the quantized activations,
the router, the row movement, and their gradients, in 64-bit NumPy.

The arithmetic is float64 throughout; what the operators define as fp32 or
as the tensors' type is rounded there and nowhere else: h = RN(x + r) in the
type of x, the router's scores (rounded once to fp32) and choices (one fp32
addition), because the order of the experts hangs on them.

Parity: pinned by tests/test_oracle_moe.py -- gradients against central
differences of the forward functions, the router against an exhaustive
search over subsets, the row movement by its defining properties.
"""

import itertools

import numpy as np

from .gemm import bf16_rne_bits
from .quant import bf16_bits_to_f32


def round_to(v, bf16):
    """float64/float32 values rounded to the tensor type, as float32."""
    v = np.asarray(v)
    if bf16:
        return bf16_bits_to_f32(bf16_rne_bits(v.astype(np.float32)))
    return v.astype(np.float32)


def rmsnorm(x, gamma, eps, residual=None, bf16=False):
    """(h float32, rstd float64, y float64) of fp32-held inputs; rstd is at
    most the largest fp32 number and 0 where the mean square and eps are."""
    x = np.asarray(x, np.float32)
    h = x if residual is None else round_to(x + np.asarray(residual, np.float32), bf16)
    d = h.astype(np.float64)
    m = np.mean(d * d, axis=1) + eps
    rstd = np.where(m > 0, np.minimum(1.0 / np.sqrt(np.where(m > 0, m, 1.0)), np.finfo(np.float32).max), 0.0)
    return h, rstd, d * rstd[:, None] * np.asarray(gamma, np.float64)


def rmsnorm_grad(dy, h, gamma, rstd, dh=None):
    """(dx, dgamma) in float64, rstd given."""
    dy, h, gamma = (np.asarray(v, np.float64) for v in (dy, h, gamma))
    xh = h * np.asarray(rstd, np.float64)[:, None]
    a = dy * gamma
    dx = np.asarray(rstd, np.float64)[:, None] * (a - xh * np.mean(a * xh, axis=1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, np.sum(dy * xh, axis=0)


def scores(logits, kind):
    """float64 scores of one token's float32 logits; -inf and NaN give 0."""
    l = np.asarray(logits, np.float32).astype(np.float64)
    masked = np.isnan(l) | (l == -np.inf)
    out = np.zeros(l.shape)
    live = l[~masked]
    if live.size == 0:
        return out
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            out[~masked] = 1.0 / (1.0 + np.exp(-live))
        else:
            top = live.max()
            e = np.where(live == top, 1.0, np.exp(np.where(live == top, 0.0, live - top)))
            out[~masked] = e / e.sum()
    return out


def _best(values, n):
    """Indexes of the n largest, lower index first on equal values."""
    return sorted(values, key=lambda e: (-values[e], e))[:n]


def route_token(logits, k, bias=None, score="softmax", groups=1, top_groups=1, group_top=2, renorm=True, scale=1.0):
    l = np.asarray(logits, np.float32)
    E = l.size
    s = scores(l, score).astype(np.float32)
    c = s if bias is None else (s + np.asarray(bias, np.float32)).astype(np.float32)
    open_ = [e for e in range(E) if not (np.isnan(l[e]) or l[e] == -np.inf or np.isnan(c[e]) or c[e] == -np.inf)]
    if top_groups < groups:
        size = E // groups
        value = {}
        for g in range(groups):
            best = sorted((c[e] for e in open_ if e // size == g), reverse=True)[:group_top]
            if best:
                value[g] = np.float32(best[0] + best[1]) if len(best) == 2 else best[0]
        kept = set(_best(value, top_groups))
        open_ = [e for e in open_ if e // size in kept]
    chosen = _best({e: c[e] for e in open_}, k)
    idx = np.full(k, -1, np.int32)
    w = np.zeros(k)
    idx[:len(chosen)] = chosen
    if chosen and renorm and score == "softmax":
        # the shares of the chosen in the softmax over all experts are the
        # softmax over the chosen alone, also where those scores underflow
        w[:len(chosen)] = scores(l[chosen], score)
    elif chosen:
        w[:len(chosen)] = s[chosen].astype(np.float64)
    total = w.sum()
    if renorm:
        w = w / total if total > 0 else np.zeros(k)
    return idx, w * scale


def route(logits, k, **kw):
    """(idx int32 [M][k], w float64 [M][k])."""
    rows = [route_token(row, k, **kw) for row in np.asarray(logits, np.float32)]
    if not rows:
        return np.zeros((0, k), np.int32), np.zeros((0, k))
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


def route_grad(dw, logits, idx, score="softmax", renorm=True, scale=1.0):
    """d(sum w dw) / d(logits) in float64, by the chain rule through the
    scores: first dL/ds, then the scores' Jacobian."""
    logits = np.asarray(logits, np.float32)
    out = np.zeros(logits.shape)
    for t in range(logits.shape[0]):
        E = logits.shape[1]
        keep = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        at = idx[t, keep]
        g = np.asarray(dw, np.float64)[t, keep] * scale
        if renorm and score == "softmax":
            # the weights are the softmax over the chosen logits alone
            p = scores(logits[t, at], "softmax")
            out[t, at] = p * (g - np.sum(p * g))
            continue
        s = scores(logits[t], score)
        ds = np.zeros(E)
        if renorm:
            total = s[at].sum()
            if total > 0:
                ds[at] = (g - np.sum(g * s[at]) / total) / total
        else:
            ds[at] = g
        out[t] = ds * s * (1.0 - s) if score == "sigmoid" else s * (ds - np.sum(ds * s))
    return out


def dispatch(idx, experts):
    """(offsets, pos, token) of fp8_dispatch, by listing the entries."""
    idx = np.asarray(idx)
    M, k = idx.shape
    buckets = [[] for _ in range(experts + 1)]
    for t in range(M):
        for j in range(k):
            e = idx[t, j]
            buckets[e if 0 <= e < experts else experts].append((t, j))
    pos = np.zeros((M, k), np.int32)
    token = np.zeros(M * k, np.int32)
    offsets = np.zeros(experts + 1, np.int32)
    for r, (e, (t, j)) in enumerate(itertools.chain.from_iterable(((e, x) for x in b) for e, b in enumerate(buckets))):
        pos[t, j] = r if e < experts else -2 - r
        token[r] = t if e < experts else -1
    offsets[1:] = np.cumsum([len(b) for b in buckets[:experts]])
    return offsets, pos, token


def combine(z, pos, w=None, base=None):
    z = np.asarray(z, np.float64)
    M, k = pos.shape
    out = np.zeros((M, z.shape[1])) if base is None else np.array(base, np.float64)
    for t in range(M):
        for j in range(k):
            if 0 <= pos[t, j] < z.shape[0]:
                out[t] += z[pos[t, j]] * (1.0 if w is None else float(w[t, j]))
    return out


def combine_grad(dy, z, pos, w=None):
    """(dz, dw); rows that no place names stay zero."""
    dy, z = np.asarray(dy, np.float64), np.asarray(z, np.float64)
    dz, dw = np.zeros(z.shape), np.zeros(pos.shape)
    for t in range(pos.shape[0]):
        for j in range(pos.shape[1]):
            r = pos[t, j]
            if 0 <= r < z.shape[0]:
                dz[r] = dy[t] * (1.0 if w is None else float(w[t, j]))
                dw[t, j] = np.dot(dy[t], z[r])
    return dz, dw
