"""A mixture-of-experts layer in FP8, forward and backward, on one GPU.

    python examples/moe_layer.py [--tokens 64] [--hidden 7168] [--inner 2048] [--experts 16] [--k 8]

h = x + residual; y = norm(h); every token goes to k experts (silu-gated, both
products in block-scaled FP8); out = h + sum of its experts' rows by their
weights.  The operators of ``fp8_fine_grained_x1_amd.tensors`` run in order:
rmsnorm_quantize -> route -> dispatch -> grouped_gemm -> (silu gate) ->
quantize_1x128 -> grouped_gemm -> combine, and their gradients back to x and
the residual, to gamma and to the router.  The experts' weights are frozen
here.  Nothing synchronizes with the host, so that ``forward`` can be captured
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


class MoELayer:
    """w_up [E][hidden][2 inner] and w_down [E][inner][hidden] in bf16 are
    quantized once, in the forward's and in the backward's layout; gamma
    [hidden], w_route [hidden][E] f32 and the balance bias [E] are kept."""

    def __init__(self, gamma, w_route, w_up, w_down, k, bias=None, score="sigmoid", groups=1, top_groups=1, scale=1.0,
                 eps=1e-6):
        self.gamma, self.w_route, self.bias, self.eps = gamma, w_route, bias, eps
        self.k, self.experts = k, w_up.shape[0]
        self.routing = dict(score=score, groups=groups, top_groups=top_groups, scale=scale)
        self.up, self.up_s = _experts(w_up, True)
        self.down, self.down_s = _experts(w_down, True)
        self.up_t, s = _experts(w_up, False)
        self.up_ts = s.transpose(1, 2)          # the gradient's K runs over the forward's N
        self.down_t, s = _experts(w_down, False)
        self.down_ts = s.transpose(1, 2)

    def forward(self, x, residual, mask=None):
        """mask: [tokens][E] added to the router's logits (-inf bars an expert).
        Returns (out, what the backward needs)."""
        q, s, h, y, rstd = T.rmsnorm_quantize(x, self.gamma, residual=residual, eps=self.eps, want_y=True)
        logits = y.float() @ self.w_route
        if mask is not None:
            logits = logits + mask
        idx, w = T.route(logits, self.k, bias=self.bias, **self.routing)
        xq, xs, offsets, pos, _ = T.dispatch(idx, self.experts, q, s)
        u = T.grouped_gemm(xq, xs, offsets, self.up, self.up_s)
        gate, lin = u.float().chunk(2, dim=1)
        aq, a_s = T.quantize_1x128((torch.nn.functional.silu(gate) * lin).to(torch.bfloat16))
        z = T.grouped_gemm(aq, a_s, offsets, self.down, self.down_s)
        out = T.combine(z, pos, w, base=h)
        return out, (h, y, rstd, logits, idx, w, offsets, pos, u, z)

    def backward(self, dout, saved):
        """Gradients (dx, dgamma, dw_route); dx is the residual's too."""
        h, y, rstd, logits, idx, w, offsets, pos, u, z = saved
        dz, dw = T.combine_backward(dout, z, pos, w)
        dq, ds = T.quantize_1x128(dz)
        da = T.grouped_gemm(dq, ds, offsets, self.down_t, self.down_ts).float()
        gate, lin = u.float().chunk(2, dim=1)
        sg = torch.sigmoid(gate)
        du = torch.cat([da * lin * sg * (1 + gate * (1 - sg)), da * gate * sg], dim=1).to(torch.bfloat16)
        dq, ds = T.quantize_1x128(du)
        dxe = T.grouped_gemm(dq, ds, offsets, self.up_t, self.up_ts)
        dlogits = T.route_backward(dw, logits, idx, score=self.routing["score"], scale=self.routing["scale"])
        dy = T.combine(dxe, pos).float() + dlogits @ self.w_route.t()
        dx, dgamma = T.rmsnorm_backward(dy.to(h.dtype), h, self.gamma, rstd, dh=dout)
        return dx, dgamma, y.float().t() @ dlogits


def random_layer(hidden, inner, experts, k, device="cuda:0", seed=0, **kw):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)

    def normal(*shape, std):
        return torch.randn(shape, generator=gen, device=device) * std

    return MoELayer(1.0 + normal(hidden, std=0.1), normal(hidden, experts, std=hidden ** -0.5),
                    normal(experts, hidden, 2 * inner, std=hidden ** -0.5).to(torch.bfloat16),
                    normal(experts, inner, hidden, std=inner ** -0.5).to(torch.bfloat16), k,
                    bias=normal(experts, std=0.01), **kw)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--k", type=int, default=8)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    layer = random_layer(a.hidden, a.inner, a.experts, a.k, scale=2.5)
    x, r, g = (torch.randn((a.tokens, a.hidden), device="cuda:0").to(torch.bfloat16) for _ in range(3))
    for name, step in (("forward", lambda: layer.forward(x, r)),
                       ("forward and backward", lambda: layer.backward(g, layer.forward(x, r)[1]))):
        for _ in range(3):
            step()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(a.steps):
            out = step()
        torch.cuda.synchronize()
        ms = (time.perf_counter() - t0) / a.steps * 1e3
        print("%s of %d tokens: %.3f ms, |out| %.3f" % (name, a.tokens, ms, float(out[0].float().square().mean().sqrt())))


if __name__ == "__main__":
    main()
