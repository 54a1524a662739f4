"""The mixture-of-experts operators on tensors past 4 GiB and 2^31 elements:
byte and element offsets beyond 32 bits.  Rows (tokens) are independent, so
what a large call gives for its last rows has to be, bit for bit, what a small
call gives on them alone; copies are compared in full."""

import pytest
import torch

from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

C = 7168


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def bits(rows, cols, dtype):
    """Normal values, made in pieces."""
    out = torch.empty((rows, cols), dtype=dtype, device=DEV)
    for i in range(0, rows, 1 << 15):
        out[i:i + (1 << 15)].normal_()
    return out


def test_norm_and_gradient():
    rows = 310_000                                    # 2.2e9 elements
    say("norm of %d x %d" % (rows, C))
    x = bits(rows, C, torch.bfloat16)
    g = torch.rand(C, device=DEV)
    q, s, h, y, rstd = T.rmsnorm_quantize(x, g, residual=x, want_y=True)
    for at in (0, rows // 2, rows - 5):
        a = T.rmsnorm_quantize(x[at:at + 5], g, residual=x[at:at + 5], want_y=True)
        for big, small in zip((q, s, h, y, rstd), a):
            assert torch.equal(big[at:at + 5], small)
    del q, s, y
    dx, dgamma = T.rmsnorm_backward(x, h, g, rstd, dh=x)
    at = rows - 5
    assert torch.equal(dx[at:], T.rmsnorm_backward(x[at:], h[at:], g, rstd[at:], dh=x[at:])[0])
    # dgamma: the sum of the pieces' (each adds up to 2^16 rows in fp32; bound as in the parity tests)
    total, size = torch.zeros(C, dtype=torch.float64, device=DEV), torch.zeros(C, dtype=torch.float64, device=DEV)
    for i in range(0, rows, 1 << 14):
        j = slice(i, i + (1 << 14))
        p = x[j].double() * (h[j].double() * rstd[j, None].double())
        total += p.sum(0)
        size += p.abs().sum(0)
    assert torch.all((dgamma.double() - total).abs() <= (rows / 256 + 96) * 2.0 ** -24 * size)


def test_dispatch_and_combine():
    tokens, k, experts = 80_000, 8, 256               # 640000 rows of 7168 bytes
    say("dispatch of %d x %d" % (tokens, k))
    q = torch.randint(0, 255, (tokens, C), dtype=torch.uint8, device=DEV)
    s = torch.rand((C // 128, tokens), device=DEV).t()
    idx = torch.rand((tokens, experts), device=DEV).topk(k, dim=1).indices.to(torch.int32)
    idx[-1, 2] = -1
    out, os, offsets, pos, token = T.dispatch(idx, experts, q, s)
    valid = tokens * k - 1
    assert int(offsets[-1]) == valid and int(token[-1]) == -1 and int(pos[-1, 2]) == -2 - valid
    order = torch.sort(torch.where(idx < 0, experts, idx).reshape(-1), stable=True).indices
    assert torch.equal(token[:valid].long(), (order // k)[:valid])
    flat = pos.reshape(-1).long()
    assert torch.equal(torch.where(flat >= 0, flat, -2 - flat)[order], torch.arange(tokens * k, device=DEV))
    for i in range(0, valid, 1 << 16):
        j = slice(i, min(i + (1 << 16), valid))
        assert torch.equal(out[j], q[token[j].long()]) and torch.equal(os[j], s[token[j].long()])
    assert torch.all(out[valid:] == 0) and torch.all(os[valid:] == 2.0 ** -126)
    del out, os, q
    few = 42_000
    z = bits(few * k, C, torch.bfloat16)               # 4.8 GB
    pos = T.dispatch(idx[:few].contiguous(), experts, torch.zeros((few, 8), device=DEV))[3]
    w = torch.rand((few, k), device=DEV)
    y = T.combine(z, pos, w)
    at = few - 9
    assert torch.equal(y[at:], T.combine(z, pos[at:].contiguous(), w[at:]))
    far = T.combine(z[pos[at:].reshape(-1).long()], torch.arange(9 * k, dtype=torch.int32, device=DEV).view(9, k), w[at:])
    assert torch.equal(y[at:], far)
    dz, dw = T.combine_backward(y, z, pos, w)
    for t in (0, few // 2, few - 1):
        assert torch.equal(dz[pos[t].long()], (w[t, :, None] * y[t].float()).to(torch.bfloat16))
        ref = (z[pos[t].long()].double() * y[t].double()).sum(1)
        size = (z[pos[t].long()].double() * y[t].double()).abs().sum(1)
        assert torch.all((dw[t].double() - ref).abs() <= (C / 512 + 20) * 2.0 ** -24 * size)


def test_route_and_gradient():
    rows, experts, k = 9_000_000, 256, 8               # 2.3e9 logits
    say("route of %d tokens" % rows)
    l = torch.empty((rows, experts), device=DEV)
    for i in range(0, rows, 1 << 20):
        l[i:i + (1 << 20)].normal_()
    kw = dict(score="sigmoid", groups=8, top_groups=4)
    idx, w = T.route(l, k, **kw)
    for at in (0, rows // 2, rows - 5000):
        a, b = T.route(l[at:at + 5000], k, **kw)
        assert torch.equal(a, idx[at:at + 5000]) and torch.equal(b, w[at:at + 5000])
    dl = T.route_backward(w, l, idx, score="sigmoid")
    for at in (0, rows // 2, rows - 5000):
        j = slice(at, at + 5000)
        assert torch.equal(dl[j], T.route_backward(w[j], l[j], idx[j], score="sigmoid"))
