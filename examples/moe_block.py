"""A mixture-of-experts block in FP8 for training, forward and backward, on one
GPU, with norms before and after it, 8-bit activation checkpoints and a balance
loss.

    python examples/moe_block.py [--tokens 1024] [--hidden 7168] [--inner 2048] [--experts 16] [--k 8] [--seqs 4]

Between two blocks the residual stream h and its norm (y, and in E4M3 q with s)
are passed on.  A block takes every token to k experts, keeps in 8 bits what its
silu gate needs again, sums the experts' rows by their weights, and adds
gate * norm(sum) to the scaled stream; the next norm follows in the same
call.  The balance loss is per sequence.  The experts' weights are frozen
here; the gradients go to y, the stream, the router, both gammas and the
gate.  Nothing synchronizes with the host, so that both passes can be captured
in a graph.
"""

import argparse
import os
import sys
import time

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp8_fine_grained_x1_amd import tensors as T  # noqa: E402


def _experts(w, transpose):
    """Block-quantized weights of every expert of w [E][K][N]: bytes [E][N][K]
    (or [E][K][N]) and scales [E][K/128][N/128]."""
    pairs = [T.quantize_block(e, transpose=transpose) for e in w]
    return torch.stack([p[0] for p in pairs]), torch.stack([p[1] for p in pairs])


class MoEBlock:
    """w_up [E][hidden][2 inner] and w_down [E][inner][hidden] in bf16 are
    quantized once, in the forward's and in the backward's layout; w_route
    [hidden][E] f32, the balance bias [E], gamma_post and the next norm's gamma
    and the block's gate ([hidden], one type) are kept."""

    def __init__(self, w_route, w_up, w_down, gamma_post, gamma, gate, k, bias=None, score="sigmoid", scale=1.0,
                 balance=1e-3, residual_scale=1.0, block_scale=1.0, eps=1e-6):
        self.w_route, self.bias, self.k, self.experts = w_route, bias, k, w_up.shape[0]
        self.score, self.scale, self.balance = score, scale, balance
        self.gamma_post, self.gamma, self.gate = gamma_post, gamma, gate
        self.scales, self.eps = dict(residual_scale=residual_scale, block_scale=block_scale), eps
        self.up, self.up_s = _experts(w_up, True)
        self.down, self.down_s = _experts(w_down, True)
        self.up_t, s = _experts(w_up, False)
        self.up_ts = s.transpose(1, 2)          # the gradient's K runs over the forward's N
        self.down_t, s = _experts(w_down, False)
        self.down_ts = s.transpose(1, 2)

    def forward(self, q, s, y, h, seqs=None, mask=None):
        """q, s, y: the norm of the stream h as the last block (or
        rmsnorm_quantize) left them; seqs: bounds of the sequences; mask [tokens][E]:
        added to the router's logits (-inf bars an expert, a row of -inf is
        padding).  Returns ((q, s, y, h) of the next block, the balance loss of each
        sequence, the experts' counts, what the backward needs)."""
        logits = y.float() @ self.w_route
        if mask is not None:
            logits = logits + mask
        idx, w = T.route(logits, self.k, bias=self.bias, score=self.score, scale=self.scale)
        loss, counts, slope = T.balance_loss(logits, idx, seqs, score=self.score, scale=self.balance)
        xq, xs, offsets, pos, _ = T.dispatch(idx, self.experts, q, s)
        u = T.grouped_gemm(xq, xs, offsets, self.up, self.up_s)
        aq, a_s, uq, us = T.swiglu_quantize(u, used=offsets[-1:])
        z = T.grouped_gemm(aq, a_s, offsets, self.down, self.down_s)
        o = T.combine(z, pos, w)
        q2, s2, h2, y2, rstd_post, rstd = T.rmsnorm_block_quantize(
            o, h, self.gamma_post, self.gamma, gate=self.gate, eps=self.eps, want_y=True, **self.scales)
        return (q2, s2, y2, h2), loss, counts, (y, logits, idx, w, offsets, pos, slope, seqs, uq, us, z, o, h2, rstd_post, rstd)

    def backward(self, dy, dh, dloss, saved):
        """dy, dh: gradients of the next y and h; dloss: of each sequence's
        balance loss (None: ones).  Returns (dy, dh) of this block's inputs and the
        gradients of w_route, gamma_post, gamma and the gate."""
        y, logits, idx, w, offsets, pos, slope, seqs, uq, us, z, o, h2, rstd_post, rstd = saved
        do, dstream, dgamma_post, dgamma, dgate = T.rmsnorm_block_backward(
            dy, o, h2, self.gamma_post, self.gamma, rstd_post, rstd, gate=self.gate, dh=dh, **self.scales)
        dz, dw = T.combine_backward(do, z, pos, w)
        dq, ds = T.quantize_1x128(dz)
        da = T.grouped_gemm(dq, ds, offsets, self.down_t, self.down_ts)
        duq, dus, _, _ = T.swiglu_backward(da, uq, us, used=offsets[-1:])
        dxe = T.grouped_gemm(duq, dus, offsets, self.up_t, self.up_ts)
        dlogits = T.route_backward(dw, logits, idx, score=self.score, scale=self.scale)
        dlogits = T.balance_loss_backward(dloss, logits, slope, seqs, score=self.score, base=dlogits)
        dy_in = (T.combine(dxe, pos).float() + dlogits @ self.w_route.t()).to(y.dtype)
        return dy_in, dstream, y.float().t() @ dlogits, dgamma_post, dgamma, dgate


def random_block(hidden, inner, experts, k, device="cuda:0", seed=0, **kw):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)

    def normal(*shape, std, mean=0.0):
        return mean + torch.randn(shape, generator=gen, device=device) * std

    return MoEBlock(normal(hidden, experts, std=hidden ** -0.5),
                    normal(experts, hidden, 2 * inner, std=hidden ** -0.5).to(torch.bfloat16),
                    normal(experts, inner, hidden, std=inner ** -0.5).to(torch.bfloat16), normal(hidden, std=0.1, mean=1.0),
                    normal(hidden, std=0.1, mean=1.0), normal(hidden, std=0.1, mean=0.5), k, bias=normal(experts, std=0.01), **kw)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--k", type=int, default=8)
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    block = random_block(a.hidden, a.inner, a.experts, a.k, scale=2.5)
    x, g, gh = (torch.randn((a.tokens, a.hidden), device="cuda:0").to(torch.bfloat16) for _ in range(3))
    seqs = torch.arange(0, a.seqs + 1, device="cuda:0", dtype=torch.int32) * (a.tokens // a.seqs)
    q, s, h, y, _ = T.rmsnorm_quantize(x, torch.ones(a.hidden, device="cuda:0"), want_y=True)
    for name, step in (("forward", lambda: block.forward(q, s, y, h, seqs)),
                       ("forward and backward", lambda: block.backward(g, gh, None, block.forward(q, s, y, h, seqs)[3]))):
        for _ in range(3):
            step()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(a.steps):
            step()
        torch.cuda.synchronize()
        print("%s of %d tokens: %.3f ms" % (name, a.tokens, (time.perf_counter() - t0) / a.steps * 1e3))
    print("balance loss of each sequence:", block.forward(q, s, y, h, seqs)[1].tolist())


if __name__ == "__main__":
    main()
