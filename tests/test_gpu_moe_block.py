"""The silu gate with checkpoints, the balance loss and the norms around a block
together, as examples/moe_block.py runs them: against a plain block in 32 bits
through autograd, with masked experts and padding, in a graph, on other streams.

The block's tolerances: E4M3 rounds to 4 significant bits, about 2.6% rms of a
value.  Every FP8 product has two such operands (3.7% of its result), the
forward chains two (5.2%); the backward four, and its gate's input is the 8-bit
checkpoint (2.6% of each half, 3.7% together): 8.3%, bf16 roundings below 0.4%
each, and the norm after the block, which keeps relative errors.  15% in the
forward's block part, 20% in the backward's; the balance loss and the gate's
and gammas' sums over tokens average those errors."""

import os
import sys

import pytest
import torch

from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_block  # noqa: E402

pytestmark = pytest.mark.gpu

HIDDEN, INNER, E, K = 512, 256, 8, 3
RS, BS, BAL, SCALE = 0.9, 0.5, 0.02, 1.5


def make(score="sigmoid"):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    n = lambda *s, std: torch.randn(s, generator=gen, device=DEV) * std  # noqa: E731
    w = (n(HIDDEN, E, std=2 * HIDDEN ** -0.5), n(E, HIDDEN, 2 * INNER, std=HIDDEN ** -0.5).to(torch.bfloat16),
         n(E, INNER, HIDDEN, std=INNER ** -0.5).to(torch.bfloat16), 1 + n(HIDDEN, std=0.1), 1 + n(HIDDEN, std=0.1),
         0.5 + n(HIDDEN, std=0.2))
    return moe_block.MoEBlock(*w, K, bias=n(E, std=0.01), score=score, scale=SCALE, balance=BAL, residual_scale=RS, block_scale=BS), w


def rel(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


def inputs(tokens, seed=2):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return [torch.randn((tokens, HIDDEN), generator=gen, device=DEV).to(torch.bfloat16) for _ in range(3)]


def plain(w, idx, y, h, mask, seqs, score):
    """(next y, next h, loss of each sequence, block part) in 32 bits with the given choice."""
    wr, up, down, gp, gm, gate = w
    logits = y @ wr + (0 if mask is None else mask)
    live = (idx >= 0).any(dim=1)
    l = torch.where(live[:, None], logits, torch.zeros_like(logits))
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, dim=1)
    s = s * live[:, None]
    c = torch.gather(s, 1, idx.clamp_min(0).long()) * (idx >= 0)
    wts = c / c.sum(1, keepdim=True).clamp_min(1e-30) * SCALE
    o = torch.zeros_like(h)
    for e in range(E):
        g, lin = (y @ up[e].float()).chunk(2, dim=1)
        o = o + ((torch.nn.functional.silu(g) * lin) @ down[e].float()) * ((idx == e) * wts).sum(1, keepdim=True)
    part = BS * gate * o * torch.rsqrt(o.square().mean(1, keepdim=True) + 1e-6) * gp
    h2 = RS * h + part
    y2 = h2 * torch.rsqrt(h2.square().mean(1, keepdim=True) + 1e-6) * gm
    share = s / s.sum(1, keepdim=True).clamp_min(1e-30)
    loss = []
    for a, b in zip(seqs, seqs[1:]):
        n = live[a:b].sum().clamp_min(1)
        f = torch.stack([(idx[a:b] == e).sum() for e in range(E)]).float() * E / (K * n)
        loss.append(BAL * (f * share[a:b].sum(0) / n).sum())
    return y2, h2, torch.stack(loss), part


@pytest.mark.parametrize("tokens,bounds", [(1, (0, 1)), (37, (0, 10, 10, 37)), (300, (0, 128, 300)), (700, (0, 700))])
@pytest.mark.parametrize("score,masked", [("sigmoid", False), ("sigmoid", True), ("softmax", False)])
def test_block_against_a_plain_one(tokens, bounds, score, masked):
    say("block of %d tokens" % tokens)
    block, w = make(score)
    x, gy, gh = inputs(tokens)
    q, s, h, y, _ = T.rmsnorm_quantize(x, torch.ones(HIDDEN, device=DEV), want_y=True)
    seqs = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    mask = None
    if masked:
        mask = torch.zeros((tokens, E), device=DEV)
        mask[::4] = float("-inf")         # padding
        if tokens == 1:
            mask[0, 1:] = 0.0
    (q2, s2, y2, h2), loss, counts, saved = block.forward(q, s, y, h, seqs, mask)
    idx = saved[2]
    if masked and tokens > 1:
        assert torch.all(idx[::4] == -1)
        assert torch.equal(h2[::4], (RS * h[::4].float()).to(h.dtype))   # nothing joins the stream
    dloss = torch.linspace(0.5, 1.5, len(bounds) - 1, device=DEV)
    got = block.backward(gy, gh, dloss, saved)
    yf, hf = y.float().requires_grad_(), h.float().requires_grad_()
    p = [w[0].clone().requires_grad_(), w[1], w[2], *(v.clone().requires_grad_() for v in w[3:])]
    y2p, h2p, lossp, part = plain(p, idx, yf, hf, mask, bounds, score)
    assert rel(h2.float() - RS * h.float(), part) < 0.15
    assert rel(y2, y2p) < 0.15
    assert torch.allclose(loss, lossp, rtol=2e-3, atol=1e-7)
    assert int(counts.sum()) == int((idx >= 0).sum())
    ((y2p * gy.float()).sum() + (h2p * gh.float()).sum() + (lossp * dloss).sum()).backward()
    want = (yf.grad, hf.grad, p[0].grad, p[3].grad, p[4].grad, p[5].grad)
    for name, a, b in zip(("dy", "dh", "dw_route", "dgamma_post", "dgamma", "dgate"), got, want):
        assert torch.isfinite(a.float()).all(), name
        assert rel(a, b) < 0.20, (name, rel(a, b))
    if masked and tokens > 1:
        assert torch.all(got[0][::4] == 0)      # no gradient reaches a padding token's norm


def step(block, q, s, y, h, seqs, gy, gh):
    out, loss, counts, saved = block.forward(q, s, y, h, seqs)
    return (*out, loss, counts, *block.backward(gy, gh, None, saved))


@pytest.mark.parametrize("tokens", [1, 70, 1300])
def test_forward_and_backward_replay_in_a_graph(tokens):
    # (the stream's gradient products are torch's; they are checked with the rest against the eager call)
    block, _ = make()
    x, gy, gh = inputs(tokens)
    ones = torch.ones(HIDDEN, device=DEV)
    q, s, h, y, _ = T.rmsnorm_quantize(x, ones, want_y=True)
    seqs = torch.tensor([0, tokens // 3, tokens], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(block, q, s, y, h, seqs, gy, gh)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(block, q, s, y, h, seqs, gy, gh)
    for rep in range(3):
        new = inputs(tokens, 20 + rep)
        q1, s1, h1, y1, _ = T.rmsnorm_quantize(new[0], ones, want_y=True)
        for dst, src in ((q, q1), (s, s1), (h, h1), (y, y1), (gy, new[1]), (gh, new[2])):
            dst.copy_(src)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(held, step(block, q, s, y, h, seqs, gy, gh))):
            assert torch.equal(a, b), (rep, i)
        torch.cuda.synchronize()


def operators(tokens, E=64, k=4, inner=256, **kw):
    """Every operator once (long and short forms by the tokens), outputs in a list."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(tokens)
    n = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    u, da = n(tokens, 2 * inner).to(torch.bfloat16), n(tokens, inner).to(torch.bfloat16)
    l = n(tokens, E)
    idx = torch.topk(l, k, dim=1).indices.to(torch.int32)
    off = torch.tensor([0, tokens // 2, tokens], dtype=torch.int32, device=DEV)
    z, r = n(tokens, 2 * inner).to(torch.bfloat16), n(tokens, 2 * inner).to(torch.bfloat16)
    g = 1 + 0.1 * n(2 * inner)

    def run(**kw):
        q, s, uq, us = T.swiglu_quantize(u, **kw)
        out = [q, s, uq, us, *T.swiglu_backward(da, uq, us, want_du=True, want_a=True, **kw)]
        if tokens % 128 == 0:
            out += T.swiglu_backward_128x1(da, uq, us, **kw)
        loss, counts, slope = T.balance_loss(l, idx, off, score="sigmoid", **kw)
        out += [loss, counts, slope, T.balance_loss_backward(loss, l, slope, off, score="sigmoid", base=l, **kw)]
        for gate in (None, g, r):
            f = T.rmsnorm_block_quantize(z, r, g, g, gate=gate, want_y=True, **kw)
            b = T.rmsnorm_block_backward(f[3], z, f[2], g, g, f[4], f[5], gate=gate, dh=r, **kw)
            out += [*f, *(t for t in b if t is not None)]
        return out
    return run


@pytest.mark.parametrize("tokens", [1, 128, 1500])
def test_operators_on_another_stream(tokens):
    run = operators(tokens)
    want = run()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        got = run(stream=stream)
        torch.cuda.synchronize()
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(want, got))


def test_operators_on_two_streams_at_once():
    # workspaces of calls in flight together are their own
    runs = [operators(n) for n in (1500, 1408)]
    want = [r() for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(runs[i]())
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(want[i], g))


def test_two_graphs_of_the_operators():
    # captured calls keep workspaces of their own: graphs replayed one after the other and again
    runs = [operators(n) for n in (1500, 1408)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for r in runs:
            r()
    torch.cuda.current_stream().wait_stream(side)
    graphs, held = [], []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(r())
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(want[i], held[i])), order
        eager = runs[0]()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[0], eager))


def test_no_autograd_graph_on_outputs():
    u = torch.randn((4, 256), device=DEV, requires_grad=True)
    assert not any(t.requires_grad for t in T.swiglu_quantize(u))
    g = torch.ones(256, device=DEV, requires_grad=True)
    assert not any(t.requires_grad for t in T.rmsnorm_block_quantize(u, u, g, g, want_y=True))


def test_example_runs():
    block = moe_block.random_block(256, 128, 4, 2, scale=2.5)
    x, g, gh = (torch.randn((64, 256), device=DEV).to(torch.bfloat16) for _ in range(3))
    q, s, h, y, _ = T.rmsnorm_quantize(x, torch.ones(256, device=DEV), want_y=True)
    out, loss, counts, saved = block.forward(q, s, y, h)
    assert loss.shape == (1,) and counts.shape == (1, 4) and all(torch.isfinite(t.float()).all() for t in (out[2], out[3], loss))
    assert all(torch.isfinite(t.float()).all() for t in block.backward(g, gh, None, saved))
