"""Measured cases of a block's other operators: the silu gate between the
experts' products with 8-bit checkpoints, the router's balance loss, and the
norms after and before a block with its gate and residual scale.

  gate      silu(gate) * lin of the up product, quantized to E4M3 with 1x128 scales, and the E4M3
            checkpoint of its input; its gradient from that checkpoint, as the 1x128 operand of the
            data gradient and, transposed, the 128x1 operands of the weight gradients
  balance   per-sequence balance loss of a router, experts' counts; its gradient
  block     norm of a block's output, gate, scaled residual addition and the next norm, quantized;
            its gradient

With ``own`` false ``run`` computes them with elementary torch operations in
32 bits; with ``own`` true it calls the library.  ``exact`` holds the same
definitions in 64 bits, written apart from both.
"""

import math

import torch

own = False

DEV = "cuda:0"
E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -126
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def _balance(name, op, rows, experts, k, seqs, score, dtype, pad, base=False):
    return dict(name=name, op=op, rows=rows, experts=experts, k=k, seqs=seqs, score=score, dtype=dtype, pad=pad, base=base)


def _block(name, op, rows, cols, dtype, gate, want_y=False, dh=True):
    return dict(name=name, op=op, rows=rows, cols=cols, dtype=dtype, gate=gate, want_y=want_y, dh=dh)


def listed():
    return [
        # one token being served by 8 experts: nothing is kept for a backward pass; latency
        dict(name="gate_8x2048_bf16", op="gate", rows=8, inner=2048, dtype="bf16", keep=False),
        # a ragged batch in f32
        dict(name="gate_1111x1408_f32", op="gate", rows=1111, inner=1408, dtype="f32", keep=True),
        # a training batch of the grouped workloads' rows and down-projection width
        dict(name="gate_16384x4096_bf16", op="gate", rows=16384, inner=4096, dtype="bf16", keep=True),
        # gradient of an odd number of experts' rows, with the bf16 tensors that weight
        # gradients outside the FP8 path read
        dict(name="gate_grad_5003x2048_bf16", op="gate_grad", rows=5003, inner=2048, dtype="bf16", wide=True),
        # gradient of the training batch, 8-bit operand of the data gradient only
        dict(name="gate_grad_16384x4096_bf16", op="gate_grad", rows=16384, inner=4096, dtype="bf16", wide=False),
        # the backward workload's token count through a dense expert: operands of the data
        # gradient and, over 128 tokens at a time, of both weight gradients
        dict(name="gate_grad_t_8192x4096_bf16", op="gate_grad_t", rows=8192, inner=4096, dtype="bf16"),
        # a few short sequences over the decode workload's experts
        _balance("balance_61x16_softmax_f32", "balance", 61, 16, 8, 3, "softmax", "f32", False),
        # packed sequences of a training batch, 8 of 256 experts, some tokens padding
        _balance("balance_16384x256_sigmoid_f32", "balance", 16384, 256, 8, 8, "sigmoid", "f32", True),
        # its gradient, added to the gradient of the router's weights
        _balance("balance_grad_16384x256_sigmoid_f32", "balance_grad", 16384, 256, 8, 8, "sigmoid", "f32", True, True),
        # one token being served, learned gate per channel, both outputs of the next norm; latency
        _block("block_1x7168_bf16", "block", 1, 7168, "bf16", "cols", want_y=True),
        # a training batch at the hidden size
        _block("block_8192x7168_bf16", "block", 8192, 7168, "bf16", "cols", want_y=True),
        # its gradient, with the residual stream's own gradient joining in
        _block("block_grad_8192x7168_bf16", "block_grad", 8192, 7168, "bf16", "cols"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "gate", "gate_grad", "gate_grad_t", "balance", "balance", "balance_grad", "block", "block",
                     "block_grad"])
    dtype = rng.choice(["bf16", "f32"])
    if op in ("balance", "balance_grad"):
        rows = _log_int(rng, 1, 16384)
        experts = rng.randint(4, 256)
        c = _balance("", op, rows, experts, rng.randint(1, min(8, experts)), _log_int(rng, 1, min(64, rows)),
                     rng.choice(["softmax", "sigmoid"]), dtype, rng.random() < 0.5, rng.random() < 0.7)
    elif op in ("block", "block_grad"):
        rows = _log_int(rng, 1, 8192)
        gate = rng.choice(["none", "cols", "rows"])
        if dtype == "f32" or gate == "rows":
            rows = -(-rows // 2)
        c = _block("", op, rows, 128 * rng.randint(1, 56), dtype, gate, rng.random() < 0.5, rng.random() < 0.7)
    else:
        rows = _log_int(rng, 1, 16384)
        if dtype == "f32":
            rows = -(-rows // 2)
        c = dict(op=op, rows=rows, inner=128 * rng.randint(1, 32), dtype=dtype)
        if op == "gate":
            c.update(keep=rng.random() < 0.7)
        elif op == "gate_grad":
            c.update(wide=rng.random() < 0.5)
            if c["wide"]:
                c["rows"] = -(-rows // 2)
        else:
            c["rows"] = 128 * max(1, rows // 256)
    c.pop("name", None)
    return c


def work(case):
    """Bytes read once and written once, and operations, of one pass."""
    op, T = case["op"], case["rows"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op in ("gate", "gate_grad", "gate_grad_t"):
        n, tiles = T * case["inner"], T * case["inner"] // 128
        if op == "gate":  # both halves in, the product out and, kept, both halves again in 8 bits
            kept = 2 * case["keep"]
            return {"bytes": n * (2 * e + 1 + kept) + 4 * tiles * (1 + kept), "flops": (12 + 3 * kept) * n}
        if op == "gate_grad":  # the product's gradient and the checkpoint in, 8 bits (and the wide tensors) out
            return {"bytes": n * (e + 4 + 3 * e * case["wide"]) + 4 * tiles * 4, "flops": 26 * n}
        return {"bytes": n * (e + 7) + 4 * tiles * 7, "flops": 36 * n}
    if op in ("balance", "balance_grad"):
        E, S = case["experts"], case["seqs"]
        if op == "balance":  # logits and choices in; loss, counts and slopes out
            return {"bytes": T * E * e + 4 * T * case["k"] + 4 * (2 * S + 1) + 8 * S * E, "flops": 6 * T * E}
        return {"bytes": T * E * e * (2 + case["base"]) + 4 * (2 * S + 1) + 4 * S * E, "flops": 10 * T * E}
    n, C = T * case["cols"], case["cols"]
    rows_gate, cols_gate = case["gate"] == "rows", case["gate"] == "cols"
    if op == "block":  # z, r (and gate) in; their sum, 8-bit rows and scales (and the norm itself) out
        per = e * (3 + rows_gate + case["want_y"]) + 1
        return {"bytes": n * per + n // 128 * 4 + 8 * T + 2 * C * (2 + cols_gate), "flops": 14 * n}
    per = e * (5 + case["dh"] + 2 * rows_gate)  # dy, h, z (and dh, gate) in; dz, dr (and the gate's) out
    return {"bytes": n * per + 8 * T + C * (2 * (2 + cols_gate) + 4 * (2 + cols_gate)), "flops": 24 * n}


# ------------------------------------------------------------------ inputs

def _hidden(shape, dtype, gen, std=1.0, outliers=0.001, mult=100.0):
    """Activations as the workloads draw them: normal, a few of them large."""
    x = torch.randn(shape, generator=gen, device=DEV) * std
    if outliers:
        x = torch.where(torch.rand(shape, generator=gen, device=DEV) < outliers, x * mult, x)
    return x.to(dtype)


def _offsets(rows, seqs, gen):
    """Bounds of sequences of uneven lengths that fill the rows."""
    cuts = torch.rand(seqs + 1, generator=gen, device=DEV) + 0.1
    ends = torch.cumsum(cuts[1:], 0) / cuts[1:].sum() * rows
    off = torch.zeros(seqs + 1, dtype=torch.int32, device=DEV)
    off[1:] = ends.round().to(torch.int32).clamp_(0, rows)
    off[-1] = rows
    return off


def _group_major(s):
    return s.t().contiguous().t()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 6007 + 29)
    st = {"case": dict(case)}
    op, T, dt = case["op"], case["rows"], TYPES[case["dtype"]]
    if op in ("gate", "gate_grad", "gate_grad_t"):
        I = case["inner"]
        u = _hidden((T, 2 * I), dt, gen, std=1.5, mult=20.0)
        if op == "gate":
            st["u"] = u
        else:
            # the forward pass kept the quantizers' bytes and their group-major scales
            q, s = _q1x128(u.float())
            st["uq"], st["us"] = q.view(torch.uint8), _group_major(s)
            st["da"] = _hidden((T, I), dt, gen, std=0.01, outliers=0.0)
    elif op in ("balance", "balance_grad"):
        E, k = case["experts"], case["k"]
        logits = torch.randn((T, E), generator=gen, device=DEV) * 1.5 + torch.randn(E, generator=gen, device=DEV) * 0.5
        bias = torch.randn(E, generator=gen, device=DEV) * 0.05
        idx = torch.topk(torch.sigmoid(logits) + bias, k, dim=1).indices.to(torch.int32)
        if case["pad"]:  # padding tokens: every expert masked, none chosen
            pad = torch.rand(T, generator=gen, device=DEV) < 0.1
            logits[pad] = float("-inf")
            idx[pad] = -1
        st["logits"], st["idx"], st["offsets"] = logits.to(dt), idx, _offsets(T, case["seqs"], gen)
        if op == "balance_grad":
            st["slope"] = _plain_balance(st)["slope"]
            st["dloss"] = torch.rand(case["seqs"], generator=gen, device=DEV) + 0.5
            st["base"] = _hidden((T, E), dt, gen, std=1e-4, outliers=0.0) if case["base"] else None
    else:
        C = case["cols"]
        vec = lambda mean: (mean + 0.1 * torch.randn(C, generator=gen, device=DEV)).to(torch.bfloat16)  # noqa: E731
        st["gamma_post"], st["gamma"] = vec(1.0), vec(1.0)
        st["gate"] = None
        if case["gate"] == "cols":
            st["gate"] = vec(0.5)
        elif case["gate"] == "rows":
            st["gate"] = torch.sigmoid(torch.randn((T, C), generator=gen, device=DEV)).to(dt)
        st["z"] = _hidden((T, C), dt, gen, std=3.0)
        # the residual stream after some layers; depth-scaled additions
        st["scales"] = (0.9, 0.25)
        r = _hidden((T, C), dt, gen, std=2.0)
        if op == "block":
            st["r"] = r
        else:
            st["h"] = r
            st["dy"] = _hidden((T, C), dt, gen, std=0.01, outliers=0.0)
            st["dh"] = _hidden((T, C), dt, gen, std=0.02, outliers=0.0) if case["dh"] else None
            st["rstd_post"] = torch.rsqrt(st["z"].float().square().mean(1) + EPS)
            st["rstd"] = torch.rsqrt(r.float().square().mean(1) + EPS)
    return st


# ------------------------------------------------------------- plain forms

def _q1x128(v):
    """E4M3 values and scales of 1x128 tiles of 32-bit rows."""
    t = v.view(v.shape[0], -1, 128)
    m = t.abs().amax(2)
    s = (m / torch.full_like(m, E4M3_MAX)).clamp_min(SCALE_FLOOR)  # (a number would be multiplied by its reciprocal)
    return (t / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(v.shape), s


def _q128x1(v):
    return _q1x128(v.t().contiguous())


def _plain_gate(st):
    u = st["u"].float()
    g, l = u.chunk(2, dim=1)
    q, s = _q1x128(g * torch.sigmoid(g) * l)
    uq, us = _q1x128(u) if st["case"]["keep"] else (None, None)
    return {"q": q, "s": s, "uq": uq, "us": us}


def _plain_gate_parts(st):
    c = st["case"]
    u = st["uq"].view(torch.float8_e4m3fn).float().view(c["rows"], -1, 128) * st["us"][:, :, None]
    g, l = u.view(c["rows"], -1).chunk(2, dim=1)
    sg = torch.sigmoid(g)
    da = st["da"].float()
    return torch.cat([da * l * sg * (1 + g * (1 - sg)), da * g * sg], dim=1), g * sg * l


def _plain_gate_grad(st):
    du, a = _plain_gate_parts(st)
    dq, ds = _q1x128(du)
    if not st["case"]["wide"]:
        return {"dq": dq, "ds": ds, "du": None, "a": None}
    return {"dq": dq, "ds": ds, "du": du.to(st["da"].dtype), "a": a.to(st["da"].dtype)}


def _plain_gate_grad_t(st):
    du, a = _plain_gate_parts(st)
    dq, ds = _q1x128(du)
    dqt, dst = _q128x1(du)
    aqt, ast = _q128x1(a)
    return {"dq": dq, "ds": ds, "dqt": dqt, "dst": dst, "aqt": aqt, "ast": ast}


def _plain_shares(st):
    """Each token's shares of the experts and, of a sigmoid, 1 - its scores;
    masked tokens have none."""
    l = st["logits"].float()
    live = (l > float("-inf")).any(1)
    l = torch.where(live[:, None], l, torch.zeros_like(l))
    if st["case"]["score"] == "softmax":
        share, rest = torch.softmax(l, 1), None
    else:
        s = torch.sigmoid(l)
        share, rest = s / s.sum(1, keepdim=True), torch.sigmoid(-l)
    return torch.where(live[:, None], share, torch.zeros_like(share)), rest, live


def _sequence(st):
    t = torch.arange(st["case"]["rows"], dtype=torch.int32, device=DEV)
    return torch.searchsorted(st["offsets"][1:], t, right=True)


def _plain_balance(st):
    c = st["case"]
    E, S, k = c["experts"], c["seqs"], c["k"]
    share, _, live = _plain_shares(st)
    idx = st["idx"].long()
    hits = torch.zeros((c["rows"], E + 1), dtype=torch.float32, device=DEV).scatter_(1, torch.where(idx >= 0, idx, E), 1.0)
    # sums over a sequence as products with its members' indicator (whole numbers below 2^24
    # are exact in 32 bits; sums of shares are long)
    member = (_sequence(st) == torch.arange(S, device=DEV)[:, None]).float()
    tokens = (member * live.float()).sum(1)
    counts = member @ hits[:, :E]
    slope = counts * (E / k) / tokens.clamp_min(1.0).square()[:, None]
    total = member.double() @ share.double()
    return {"loss": (slope.double() * total).sum(1).float(), "counts": counts.to(torch.int32), "slope": slope}


def _plain_balance_grad(st):
    share, rest, _ = _plain_shares(st)
    c = (st["dloss"][:, None] * st["slope"])[_sequence(st)]
    dl = share * (c - (c * share).sum(1, keepdim=True))
    if rest is not None:
        dl = dl * rest
    if st["base"] is not None:
        dl = dl + st["base"].float()
    return {"dlogits": dl.to(st["logits"].dtype)}


def _plain_block(st):
    c, (rs, bs) = st["case"], st["scales"]
    z = st["z"].float()
    rstd_post = torch.rsqrt(z.square().mean(1) + EPS)
    t = z * rstd_post[:, None] * st["gamma_post"].float()
    if st["gate"] is not None:
        t = t * st["gate"].float()
    h = (rs * st["r"].float() + bs * t).to(st["z"].dtype)
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(1) + EPS)
    y = f * rstd[:, None] * st["gamma"].float()
    q, s = _q1x128(y)
    return {"q": q, "s": s, "h": h, "y": y.to(h.dtype) if c["want_y"] else None, "rstd_post": rstd_post, "rstd": rstd}


def _plain_block_grad(st):
    c, (rs, bs), dt = st["case"], st["scales"], st["z"].dtype
    g, rstd = st["dy"].float(), st["rstd"][:, None]
    xh = st["h"].float() * rstd
    a = g * st["gamma"].float()
    dh = rstd * (a - xh * (a * xh).mean(1, keepdim=True))
    if st["dh"] is not None:
        dh = dh + st["dh"].float()
    zh = st["z"].float() * st["rstd_post"][:, None]
    gp = st["gamma_post"].float()
    b = bs * dh
    dgate = None
    if st["gate"] is not None:
        dgate = b * gp * zh
        dgate = dgate.to(dt) if c["gate"] == "rows" else dgate.sum(0)
        b = b * st["gate"].float()
    bg = b * gp
    dz = st["rstd_post"][:, None] * (bg - zh * (bg * zh).mean(1, keepdim=True))
    return {"dz": dz.to(dt), "dr": (rs * dh).to(dt), "dgamma_post": (b * zh).sum(0), "dgamma": (g * xh).sum(0),
            "dgate": dgate}


# ----------------------------------------------------- the library's calls

def _own(st):
    from fp8_fine_grained_x1_amd import tensors as T
    c = st["case"]
    op = c["op"]
    f8 = torch.float8_e4m3fn
    if op == "gate":
        q, s, uq, us = T.swiglu_quantize(st["u"], keep=c["keep"])
        return {"q": q.view(f8), "s": s, "uq": uq.view(f8) if c["keep"] else None, "us": us}
    if op == "gate_grad":
        dq, ds, du, a = T.swiglu_backward(st["da"], st["uq"], st["us"], want_du=c["wide"], want_a=c["wide"])
        return {"dq": dq.view(f8), "ds": ds, "du": du, "a": a}
    if op == "gate_grad_t":
        dq, ds, dqt, dst, aqt, ast = T.swiglu_backward_128x1(st["da"], st["uq"], st["us"])
        return {"dq": dq.view(f8), "ds": ds, "dqt": dqt.view(f8), "dst": dst, "aqt": aqt.view(f8), "ast": ast}
    if op == "balance":
        loss, counts, slope = T.balance_loss(st["logits"], st["idx"], st["offsets"], score=c["score"])
        return {"loss": loss, "counts": counts, "slope": slope}
    if op == "balance_grad":
        return {"dlogits": T.balance_loss_backward(st["dloss"], st["logits"], st["slope"], st["offsets"], score=c["score"],
                                                   base=st["base"])}
    rs, bs = st["scales"]
    if op == "block":
        q, s, h, y, rstd_post, rstd = T.rmsnorm_block_quantize(
            st["z"], st["r"], st["gamma_post"], st["gamma"], gate=st["gate"], residual_scale=rs, block_scale=bs, eps=EPS,
            want_y=c["want_y"])
        return {"q": q.view(f8), "s": s, "h": h, "y": y, "rstd_post": rstd_post, "rstd": rstd}
    dz, dr, dgamma_post, dgamma, dgate = T.rmsnorm_block_backward(
        st["dy"], st["z"], st["h"], st["gamma_post"], st["gamma"], st["rstd_post"], st["rstd"], gate=st["gate"],
        residual_scale=rs, block_scale=bs, dh=st["dh"])
    return {"dz": dz, "dr": dr, "dgamma_post": dgamma_post, "dgamma": dgamma, "dgate": dgate}


_PLAIN = {"gate": _plain_gate, "gate_grad": _plain_gate_grad, "gate_grad_t": _plain_gate_grad_t, "balance": _plain_balance,
          "balance_grad": _plain_balance_grad, "block": _plain_block, "block_grad": _plain_block_grad}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact

def _e4m3(v):
    """The nearest E4M3 value, ties to the even one, of 64-bit values."""
    v = v.clamp(-E4M3_MAX, E4M3_MAX)
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _tiles(v, dim):
    """E4M3 values and scales of 64-bit values in tiles of 128 along dim (0 or
    1); along 0 the result is laid out transposed."""
    v = v if dim == 1 else v.t()
    tile = v.unflatten(1, (-1, 128))
    s = torch.maximum(tile.max(2).values, -tile.min(2).values) / E4M3_MAX
    s = torch.where(s < SCALE_FLOOR, SCALE_FLOOR, s)
    # (the definition's quotient is by the stored scale and rounded to 32 bits)
    return _e4m3((tile / s.float().double().unsqueeze(2)).float().double()).flatten(1), s


def _logistic(a):
    return 1.0 / (1.0 + torch.exp(-a))


def _exact_gate(case, st):
    op, I = case["op"], case["inner"]
    if op == "gate":
        u = st["u"].double()
        q, s = _tiles(u[:, I:] * u[:, :I] * _logistic(u[:, :I]), 1)
        uq, us = _tiles(u, 1) if case["keep"] else (None, None)
        return {"q": q, "s": s, "uq": uq, "us": us}
    u = st["uq"].view(torch.float8_e4m3fn).double() * st["us"].double().repeat_interleave(128, dim=1)
    u = u.float().double()  # (the checkpoint's value is the fp32 product)
    gate, lin, da = u[:, :I], u[:, I:], st["da"].double()
    sig = _logistic(gate)
    a = gate * sig * lin
    # d silu(x) / dx = sig + x sig (1 - sig)
    du = torch.cat([da * lin * (sig + gate * sig / (1.0 + torch.exp(gate))), da * gate * sig], 1)
    dq, ds = _tiles(du, 1)
    if op == "gate_grad":
        return {"dq": dq, "ds": ds, "du": du if case["wide"] else None, "a": a if case["wide"] else None}
    dqt, dst = _tiles(du, 0)
    aqt, ast = _tiles(a, 0)
    return {"dq": dq, "ds": ds, "dqt": dqt, "dst": dst, "aqt": aqt, "ast": ast}


def _exact_balance(case, st):
    E, k = case["experts"], case["k"]
    bounds = st["offsets"].tolist()
    loss, slopes, grads = [], [], []
    for s, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        l = st["logits"][lo:hi].double()
        live = ~torch.isneginf(l).all(1)
        masked = torch.where(live[:, None], l, 0.0)
        score = torch.exp(masked - torch.logsumexp(masked, 1, keepdim=True)) if case["score"] == "softmax" else _logistic(masked)
        share = torch.where(live[:, None], score / score.sum(1, keepdim=True), 0.0)
        if case["op"] == "balance":
            n = int(live.sum())
            hits = torch.nn.functional.one_hot(st["idx"][lo:hi].long().flatten() + 1, E + 1).sum(0)[1:].double()
            f = hits * E / (k * max(n, 1))
            p = share.sum(0) / max(n, 1)
            loss.append((f * p).sum())
            slopes.append(f / max(n, 1))
        else:
            c = st["slope"][s].double() * st["dloss"][s].double()
            # of L = sum_i c_i share_i: d share_i / d log s_j = share_i ([i = j] - share_j)
            d = c * share - share * (share @ c)[:, None]
            if case["score"] == "sigmoid":
                d = d * _logistic(-masked)   # d log s / dl
            grads.append(d)
    if case["op"] == "balance":
        return {"loss": torch.stack(loss), "counts": None, "slope": torch.stack(slopes)}
    d = torch.cat(grads, 0)
    return {"dlogits": d if st["base"] is None else d + st["base"].double()}


def _exact_block(case, st):
    C, (rs, bs), dt = case["cols"], st["scales"], st["z"].dtype
    gate = 1.0 if st["gate"] is None else st["gate"].double()
    gp, gm, z = st["gamma_post"].double(), st["gamma"].double(), st["z"].double()
    if case["op"] == "block":
        n1 = torch.sqrt((z * z).sum(1) / C + EPS)
        # (the next norm is of the stored sum)
        sum_ = st["r"].double() * rs + z / n1[:, None] * (gp * gate) * bs
        h = sum_.to(dt).double()
        n2 = torch.sqrt((h * h).sum(1) / C + EPS)
        y = h / n2[:, None] * gm
        q, s = _tiles(y, 1)
        return {"q": q, "s": s, "h": sum_, "y": y if case["want_y"] else None, "rstd_post": 1.0 / n1, "rstd": 1.0 / n2}
    h, dy = st["h"].double(), st["dy"].double()
    i1, i2 = st["rstd_post"].double()[:, None], st["rstd"].double()[:, None]
    # L = <dy, gm h / n2> + <dh, h>, h = rs r + bs gate gp z / n1, both 1/n given
    v = dy * gm
    total = v * i2 - h * (v * h).sum(1, keepdim=True) * i2.pow(3) / C
    if st["dh"] is not None:
        total = total + st["dh"].double()
    w = total * bs * gate * gp
    dz = w * i1 - z * (w * z).sum(1, keepdim=True) * i1.pow(3) / C
    per = total * bs * z * i1
    dgate = None if st["gate"] is None else per * gp
    return {"dz": dz, "dr": total * rs, "dgamma_post": (per * gate).sum(0), "dgamma": (dy * h * i2).sum(0),
            "dgate": dgate if case["gate"] != "cols" else dgate.sum(0)}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op.startswith("gate"):
        return _exact_gate(case, st)
    return _exact_balance(case, st) if op.startswith("balance") else _exact_block(case, st)
