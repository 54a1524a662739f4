"""The operators together, as examples/moe_layer.py runs them: against a plain
layer in 32 bits, with masked experts, in a graph, on another stream; and what
the tensor helpers refuse.

The layer's tolerance: E4M3 rounds to 4 significant bits, an error of at most
2^-4 and about 2.6% rms of a value.  Every FP8 product has two such operands
(3.7% of its result, the errors being independent), the forward chains two,
the backward four: 5.2% and 7.4%, plus bf16 roundings below 0.4% each.  The
expert part alone is compared (the residual would hide it): 10% and 15%."""

import os
import sys

import numpy as np
import pytest
import torch

from fp8_fine_grained_x1_amd import binding as B
from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402

pytestmark = pytest.mark.gpu

HIDDEN, INNER, E, K = 512, 256, 8, 3


def make(**kw):
    """The layer and its bf16 weights."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    n = lambda *s, std: torch.randn(s, generator=gen, device=DEV) * std  # noqa: E731
    w = (1.0 + n(HIDDEN, std=0.1), n(HIDDEN, E, std=2 * HIDDEN ** -0.5),
         n(E, HIDDEN, 2 * INNER, std=HIDDEN ** -0.5).to(torch.bfloat16), n(E, INNER, HIDDEN, std=INNER ** -0.5).to(torch.bfloat16))
    return moe_layer.MoELayer(*w, K, bias=n(E, std=0.01), score="sigmoid", scale=1.5, **kw), w


def rel(a, b):
    a, b = a.double(), b.double()
    return float((a - b).norm() / b.norm())


def plain(w, idx, x, r):
    """The layer in 32 bits with the given choice, through autograd."""
    gamma, wr, up, down = w
    h = x + r
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * gamma
    s = torch.gather(torch.sigmoid(y @ wr), 1, idx.clamp_min(0).long()) * (idx >= 0)
    wts = s / s.sum(1, keepdim=True).clamp_min(1e-30) * 1.5
    out = torch.zeros_like(h)
    for e in range(E):
        gate, lin = (y @ up[e].float()).chunk(2, dim=1)
        f = (torch.nn.functional.silu(gate) * lin) @ down[e].float()
        out = out + f * ((idx == e) * wts).sum(1, keepdim=True)
    return h, out


def inputs(tokens, seed=2):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    return [(torch.randn((tokens, HIDDEN), generator=gen, device=DEV)).to(torch.bfloat16) for _ in range(3)]


@pytest.mark.parametrize("tokens", [1, 37, 300])
@pytest.mark.parametrize("masked", [False, True])
def test_layer_against_a_plain_one(tokens, masked):
    say("layer of %d tokens" % tokens)
    layer, w = make()
    x, r, g = inputs(tokens)
    mask = None
    if masked:
        # some experts barred, some tokens with fewer than k left, one with none
        mask = torch.zeros((tokens, E), device=DEV)
        mask[:, 1] = float("-inf")
        mask[::5, 2:] = float("-inf")
        mask[tokens // 2] = float("-inf")
    out, saved = layer.forward(x, r, mask)
    idx = saved[4]
    if masked:
        assert not torch.any(idx == 1) and torch.all(idx[tokens // 2] == -1)
        assert torch.equal(out[tokens // 2], saved[0][tokens // 2])
    xf, rf = x.float().requires_grad_(), r.float().requires_grad_()
    gamma, wr = w[0].clone().requires_grad_(), w[1].clone().requires_grad_()
    h, experts = plain((gamma, wr) + w[2:], idx, xf, rf)
    if tokens > 1 or not masked:
        assert rel(out.float() - saved[0].float(), experts) < 0.10
    dx, dgamma, dwr = layer.backward(g, saved)
    (h + experts).backward(g.float())
    if tokens > 1 or not masked:
        assert rel(dx.float() - g.float(), xf.grad - g.float()) < 0.15
        assert rel(dgamma, gamma.grad) < 0.15
        assert rel(dwr, wr.grad) < 0.15
    assert torch.isfinite(dx.float()).all() and torch.isfinite(dgamma).all() and torch.isfinite(dwr).all()
    if masked:
        assert torch.equal(dx[tokens // 2], g[tokens // 2])     # nothing but the residual's gradient


@pytest.mark.parametrize("tokens", [1, 70, 700])
def test_layer_replays_in_a_graph(tokens):
    layer, _ = make()
    x, r, g = inputs(tokens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(x, r)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out_g, saved_g = layer.forward(x, r)
    for rep in range(3):
        a, b, _ = inputs(tokens, 10 + rep)
        x.copy_(a)
        r.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        out, saved = layer.forward(x, r)
        torch.cuda.synchronize()
        assert torch.equal(out, out_g), rep
        for i in (3, 4, 5, 6, 7):
            assert torch.equal(saved[i], saved_g[i]), (rep, i)


def test_operators_replay_in_a_graph():
    # the long forms of dispatch and route, and the gradients
    tokens, k = 4300, 4
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    x = torch.randn((tokens, 256), generator=gen, device=DEV).to(torch.bfloat16)
    l = torch.randn((tokens, 64), generator=gen, device=DEV)
    gamma = torch.ones(256, device=DEV)

    def step():
        q, s, h, y, rstd = T.rmsnorm_quantize(x, gamma, residual=x, want_y=True)
        idx, w = T.route(l, k, score="sigmoid", groups=8, top_groups=3)
        d = T.dispatch(idx, 64, q, s)
        z = torch.repeat_interleave(y, k, dim=0)
        out = T.combine(z, d[3], w, base=h)
        dz, dw = T.combine_backward(out, z, d[3], w)
        dl = T.route_backward(dw, l, idx, score="sigmoid")
        return (*d, out, dz, dw, dl, *T.rmsnorm_backward(out, h, gamma, rstd))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for rep in range(3):
        x.copy_(torch.randn((tokens, 256), generator=gen, device=DEV))
        l.copy_(torch.randn((tokens, 64), generator=gen, device=DEV))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b), rep
        torch.cuda.synchronize()


def test_another_stream():
    tokens, k = 1500, 4
    x = torch.randn((tokens, 256), device=DEV).to(torch.bfloat16)
    l = torch.randn((tokens, 64), device=DEV)
    gamma = torch.ones(256, device=DEV)

    def step(**kw):
        q, s, h, y, rstd = T.rmsnorm_quantize(x, gamma, residual=x, want_y=True, **kw)
        idx, w = T.route(l, k, **kw)
        d = T.dispatch(idx, 64, q, s, **kw)
        out = T.combine(torch.empty((0, 256), dtype=torch.bfloat16, device=DEV), torch.full_like(idx, -1), w, base=h, **kw)
        return (*d, idx, w, out, *T.rmsnorm_backward(y, h, gamma, rstd, **kw), T.route_backward(w, l, idx, **kw))

    want = step()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        got = step(stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_on_another_stream_are_that_streams_memory(raw):
    # a block that the current stream has freed may have work pending there: the other stream must not write it
    x = torch.randn((2048, 1024), device=DEV)
    pos = torch.zeros((2048, 1), dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = torch.empty_like(x)
    at = freed.data_ptr()
    del freed
    out = T.combine(x, pos, stream=side.cuda_stream if raw else side)
    again = torch.empty_like(x)  # the current stream's: the freed block
    torch.cuda.synchronize()
    assert again.data_ptr() == at and out.data_ptr() != at
    assert torch.equal(out, x[:1].expand_as(x))


def test_the_default_stream_by_its_null_handle():
    x = torch.randn((5, 256), device=DEV)
    pos = torch.tensor([[3], [-1], [0]], dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    out = T.combine(x, pos, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, torch.stack([x[3], torch.zeros_like(x[0]), x[0]]))


def test_grouped_gemm_leaves_rows_past_the_experts_alone():
    # dispatch puts dropped entries behind offsets[E]: the grouped GEMM's every tile shape leaves those rows of c as they are
    rng = np.random.default_rng(0)
    rows, valid = 700, 450
    x = torch.randn((rows, 256), device=DEV).to(torch.bfloat16)
    qa, sa = T.quantize_1x128(x)
    wq, ws = zip(*[T.quantize_block(torch.randn((256, 256), device=DEV).to(torch.bfloat16)) for _ in range(4)])
    qb, sb = torch.stack(wq), torch.stack(ws)
    cuts = np.sort(rng.integers(0, valid, 3))
    for end in (valid, 0):
        off = torch.tensor([0, *(np.minimum(cuts, end)), end], dtype=torch.int32, device=DEV)
        for kw in (dict(), dict(tiles="wide"), dict(tiles="narrow"), dict(flags=B.FP8FG_GEMM_FP8_MFMA),
                   dict(flags=B.FP8FG_GEMM_E8M0_SCALES)):
            c = torch.full((rows, 256), 7.0, device=DEV)
            T.grouped_gemm(qa, sa, off, qb, sb, out=c, **kw)
            assert torch.all(c[end:] == 7.0)
            assert end == 0 or not torch.any(torch.all(c[:end] == 7.0, dim=1))


def test_refusals_on_the_gpu():
    f = torch.zeros((4, 256), device=DEV)
    b = f.to(torch.bfloat16)
    g = torch.ones(256, device=DEV)
    i = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    u8, s = torch.zeros((4, 256), dtype=torch.uint8, device=DEV), torch.ones((4, 2), device=DEV)
    r1 = torch.ones(4, device=DEV)
    w = torch.ones((4, 2), device=DEV)
    bad = [
        lambda: T.rmsnorm_quantize(f.half(), g), lambda: T.rmsnorm_quantize(f, g[:128]), lambda: T.rmsnorm_quantize(f, g.cpu()),
        lambda: T.rmsnorm_quantize(f, g, residual=b), lambda: T.rmsnorm_quantize(f, g, residual=f[:3]),
        lambda: T.rmsnorm_quantize(f.t(), g), lambda: T.rmsnorm_quantize(f[0], g), lambda: T.rmsnorm_quantize(f, g, scale_layout="x"),
        lambda: T.rmsnorm_quantize(f, "g"),
        lambda: T.rmsnorm_backward(b, f, g, r1), lambda: T.rmsnorm_backward(f, f, g, r1[:3]), lambda: T.rmsnorm_backward(f, f, g, r1.half()),
        lambda: T.rmsnorm_backward(f, f, g, r1, dh=f[:, :128]),
        lambda: T.route(f, 2, bias=g[:5]), lambda: T.route(f, 2, bias=g.half()), lambda: T.route(f, 2, score="relu"), lambda: T.route(f, -1),
        lambda: T.route_backward(w, f, i.long()), lambda: T.route_backward(w[:3], f, i), lambda: T.route_backward(w, f, i[:3]),
        lambda: T.dispatch(i.long(), 8, f), lambda: T.dispatch(i[:3], 8, f), lambda: T.dispatch(i, 8, u8), lambda: T.dispatch(i, 8, f, s),
        lambda: T.dispatch(i, 8, u8, s[:, :1]), lambda: T.dispatch(i, 8, u8, s.half()), lambda: T.dispatch(i, -2, f), lambda: T.dispatch(i, 8, f.half()),
        lambda: T.combine(f, i.long()), lambda: T.combine(f, i, w[:, :1]), lambda: T.combine(f, i, w, base=f[:3]), lambda: T.combine(f, i, w, base=b),
        lambda: T.combine(f.half(), i), lambda: T.combine(f, i.t()),
        lambda: T.combine_backward(f, f, i, w), lambda: T.combine_backward(b, torch.zeros((8, 256), device=DEV), i, w),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            say("refusal %d was not raised" % n)
    with pytest.raises(B.Fp8fgError) as e:
        T.route(f, 300)
    assert e.value.status == B.FP8FG_ESHAPE
    with pytest.raises(B.Fp8fgError) as e:
        T.rmsnorm_quantize(f[:, :200], g[:200])
    assert e.value.status == B.FP8FG_ESHAPE
    with pytest.raises(B.Fp8fgError) as e:
        T.dispatch(i, 5000, f)
    assert e.value.status == B.FP8FG_EUNSUPPORTED
    with pytest.raises(TypeError):
        T.route(f, "k")


@pytest.mark.parametrize("call,status", [
    (lambda f, i: T.route(f, 1 << 31), B.FP8FG_ESHAPE), (lambda f, i: T.route(f, 1 << 45), B.FP8FG_ESHAPE),
    (lambda f, i: T.route(f, (1 << 63) - 1), B.FP8FG_ESHAPE), (lambda f, i: T.route(f, 0), B.FP8FG_EINVAL),
    (lambda f, i: T.route(f, 2, group_top=(1 << 32) + 1), B.FP8FG_EINVAL), (lambda f, i: T.route(f, 2, groups=1 << 40), B.FP8FG_ESHAPE),
    (lambda f, i: T.dispatch(i, 1 << 40, f), B.FP8FG_EUNSUPPORTED), (lambda f, i: T.dispatch(i, (1 << 63) - 1, f), B.FP8FG_EUNSUPPORTED),
    (lambda f, i: T.dispatch(i, 0, f), B.FP8FG_EINVAL), (lambda f, i: T.dispatch(i[:, :0], 8, f), B.FP8FG_EINVAL),
])
def test_sizes_are_refused_before_anything_is_allocated(call, status):
    f, i = torch.zeros((4, 256), device=DEV), torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    with pytest.raises(B.Fp8fgError) as e:
        call(f, i)
    assert e.value.status == status
    assert torch.cuda.max_memory_allocated() - held <= 1 << 16


def test_a_stream_of_another_device_is_refused():
    class Other:
        cuda_stream, device = 1, torch.device("cuda", 1)

    x = torch.randn((5, 256), device=DEV)
    with pytest.raises(ValueError):
        T.route(x, 2, stream=Other())
