"""The silu gate's fp32 values are no less exact than the composition of
elementary fp32 operations that they replace: their root mean square error
against 64 bits, over a million values, is at most the composition's.  (No
tolerance: both errors are of the same inputs.  They are taken relative to the
value, of dg to its two terms da l sg and da l sg g (1 - sg), which cancel around
g = -1.28.)"""

import pytest
import torch

from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def rms(v, exact, size):
    ok = size > 1e-20
    return float(((v.double() - exact)[ok] / size[ok]).square().mean().sqrt()) * 2 ** 24


@pytest.mark.parametrize("std", [0.5, 1.5, 4.0])
def test_gradient_and_result_against_the_composition(std):
    rows, inner = 1024, 1024
    gen = torch.Generator(device=DEV)
    gen.manual_seed(7)
    _, _, uq, us = T.swiglu_quantize(torch.randn((rows, 2 * inner), generator=gen, device=DEV) * std)
    da = torch.randn((rows, inner), generator=gen, device=DEV)
    _, _, du, a = T.swiglu_backward(da, uq, us, want_du=True, want_a=True)
    u = uq.view(torch.float8_e4m3fn).float() * us.repeat_interleave(128, dim=1)
    g, l = u.chunk(2, dim=1)
    s = torch.sigmoid(g)
    parts = ("dg", du[:, :inner], da * l * s * (1 + g * (1 - s))), ("dl", du[:, inner:], da * g * s), ("a", a, g * s * l)
    G, L, D = g.double(), l.double(), da.double()
    S = torch.sigmoid(G)
    R = torch.sigmoid(-G)
    exact = {"dg": D * L * S * (1 + G * R), "dl": D * G * S, "a": G * S * L}
    size = {k: v.abs() for k, v in exact.items()}
    size["dg"] = (D * L * S).abs() * (1 + (G * R).abs())
    for name, own, plain in parts:
        e, p = rms(own, exact[name], size[name]), rms(plain, exact[name], size[name])
        say("std %g %s: rms error %.3f roundings, the composition's %.3f" % (std, name, e, p))
        assert e <= p, (name, e, p)
