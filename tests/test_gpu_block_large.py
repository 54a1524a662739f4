"""The silu gate, the balance loss and the norms around a block on tensors past 4
GiB and 2^31 elements: the last rows of a long call against a call on those rows
alone (a row does not depend on the others), and sums against sums of parts."""

import pytest
import torch

from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

ROWS, COLS = 262144 + 128, 8192          # 2^31 + 2^20 elements, 4 GiB + 2 MiB in bf16


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def filled(rows, cols, seed):
    """Normal bf16 rows, made a part at a time."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    out = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    for part in out.split(1 << 15):
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV))
    return out


def test_gate_past_4_gib():
    say("gate of %d x %d" % (ROWS, COLS // 2))
    u = filled(ROWS, COLS, 1)
    q, s, uq, us = T.swiglu_quantize(u)
    for rows in (slice(0, 128), slice(131072 - 64, 131072 + 64), slice(ROWS - 128, ROWS)):
        for got, want in zip((q, s, uq, us), T.swiglu_quantize(u[rows].contiguous())):
            assert torch.equal(got[rows], want)
    del u, q, s
    da = filled(ROWS, COLS // 2, 2)
    last = slice(ROWS - 128, ROWS)
    dq, ds, du, a = T.swiglu_backward(da, uq, us, want_du=True, want_a=True)
    want = T.swiglu_backward(da[last], uq[last], us[last], want_du=True, want_a=True)
    for got, w in zip((dq, ds, du, a), want):
        assert torch.equal(got[last], w)
    del du, a
    dq2, ds2, dqt, dst, aqt, ast = T.swiglu_backward_128x1(da, uq, us)
    assert torch.equal(dq, dq2) and torch.equal(ds, ds2)
    want = T.swiglu_backward_128x1(da[last], uq[last], us[last])
    assert torch.equal(dqt[:, last], want[2]) and torch.equal(dst[:, -1:], want[3])
    assert torch.equal(aqt[:, last], want[4]) and torch.equal(ast[:, -1:], want[5])


def test_block_norm_past_4_gib():
    say("block norm of %d x %d" % (ROWS, COLS))
    z, r = filled(ROWS, COLS, 3), filled(ROWS, COLS, 4)
    g = 1 + 0.1 * torch.randn(COLS, device=DEV)
    out = T.rmsnorm_block_quantize(z, r, g, g, gate=g)
    last = slice(ROWS - 100, ROWS)
    for got, want in zip(out, T.rmsnorm_block_quantize(z[last], r[last], g, g, gate=g)):
        assert want is None or torch.equal(got[last], want)
    h, post, rstd = out[2], out[4], out[5]
    del out
    full = T.rmsnorm_block_backward(r, z, h, g, g, post, rstd, gate=g, dh=z)
    part = T.rmsnorm_block_backward(r[last], z[last], h[last], g, g, post[last], rstd[last], gate=g, dh=z[last])
    assert torch.equal(full[0][last], part[0]) and torch.equal(full[1][last], part[1])
    # the sums over rows: those of 8 parts, within (rows / strips + 96) 2^-24 of the terms' magnitudes each way
    parts = [T.rmsnorm_block_backward(r[i], z[i], h[i], g, g, post[i], rstd[i], gate=g, dh=z[i])
             for i in (slice(k * ROWS // 8, (k + 1) * ROWS // 8) for k in range(8))]
    xh_dy = 0.0
    for k in range(8):
        i = slice(k * ROWS // 8, (k + 1) * ROWS // 8)
        for a in range(i.start, i.stop, 1 << 15):
            b = slice(a, min(a + (1 << 15), i.stop))
            xh_dy = xh_dy + (r[b].float() * h[b].float() * rstd[b, None]).abs().sum(0)
    want = sum(p[3].double() for p in parts)
    assert torch.all((full[3].double() - want).abs() <= 2 * (ROWS / 256 + 96) * 2.0 ** -24 * xh_dy.double())
    for j in (2, 4):
        want = sum(p[j].double() for p in parts)
        assert float((full[j].double() - want).norm()) <= 1e-4 * float(want.norm()) + 1e-2


def test_balance_past_4_gib():
    rows, experts, k = (1 << 22) + 77, 256, 2
    say("balance of %d x %d" % (rows, experts))
    l = torch.empty((rows, experts), device=DEV)
    for part in l.split(1 << 18):
        part.normal_()
    idx = torch.randint(0, experts, (rows, k), dtype=torch.int32, device=DEV)
    loss, counts, slope = T.balance_loss(l, idx, score="sigmoid")
    assert torch.equal(counts[0].long(), torch.bincount(idx.flatten().long(), minlength=experts))
    total = torch.zeros(experts, dtype=torch.float64, device=DEV)
    for part in l.split(1 << 18):
        p = torch.sigmoid(part.double())
        total += (p / p.sum(1, keepdim=True)).sum(0)
    want = float((slope[0].double() * total).sum())
    # a share within 100 u, a chunk's 4096 tokens over 16 waves added in fp32
    assert abs(float(loss) - want) <= (100 + 4096 / 16 + 20) * 2.0 ** -24 * want
    g = T.balance_loss_backward(None, l, slope, score="sigmoid")
    last = slice(rows - 100, rows)
    assert torch.equal(g[last], T.balance_loss_backward(None, l[last], slope, score="sigmoid"))
