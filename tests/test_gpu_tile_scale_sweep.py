"""The tile scales and quotients of the silu gate's checkpoint (the form that it
shares with the norms around a block) for every significand of a tile's
maximum: scale RN32(m / 448), bytes of RN32(x / scale), against 64-bit
arithmetic on the same card.

A quotient of two fp32 numbers that is formed in 64 bits and rounded to 32 is
the correctly rounded one (53 >= 2 * 24 + 2 bits).  The maxima are all 2^23
of a binade, of ordinary size and on both sides of the borders at which the
fast form ends (2^-55; the largest numbers).  Beside its maximum a tile holds
values around the borders between two E4M3 values, where a quotient that is
off in its last bit shows in the byte, and others of any size below it."""

import pytest
import torch

from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

TILES = 1 << 18


def borders():
    """The midpoints between neighbouring positive E4M3 values."""
    v = torch.arange(0, 0x7F, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
    return (v[1:] + v[:-1]) / 2


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("exponent", [0, -56, -55, -54, 126, 127])
def test_every_significand(exponent, pow2):
    say("tile scales, 2^%d, pow2 %d" % (exponent, pow2))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(exponent + 200)
    mid = borders()
    for first in range(0, 1 << 23, TILES):
        bits = torch.arange(first, first + TILES, dtype=torch.int32, device=DEV) | ((exponent + 127) << 23)
        m = bits.view(torch.float32)
        if pow2:
            mant, e = torch.frexp(m.double() / 448)
            s = torch.where(mant == 0.5, e - 1, e).double().exp2()   # the least power of two at or above m / 448
        else:
            s = (m.double() / 448).float().double()
        at = mid[torch.randint(0, mid.numel(), (TILES, 64), generator=gen, device=DEV)] * s[:, None]
        at = torch.minimum(at, m[:, None].double() * (1 - 2.0 ** -20))    # (within fp32, with the steps below)
        near = (at.float().view(torch.int32) + torch.randint(-2, 3, at.shape, generator=gen, device=DEV, dtype=torch.int32)).view(torch.float32)
        rest = torch.rand((TILES, 64), generator=gen, device=DEV) * m[:, None]
        x = torch.cat([near, rest], 1)
        x = torch.minimum(x, m[:, None])
        x = torch.where(torch.rand(x.shape, generator=gen, device=DEV) < 0.5, x, -x)
        x[:, 7] = torch.where(bits % 2 == 0, m, -m)
        _, _, q, got = T.swiglu_quantize(x.view(TILES // 2, 256), pow2=pow2, scale_layout="row_major")
        assert torch.equal(got.view(-1).double(), s), "scales from %d" % first
        want = (x.double() / s[:, None]).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(q.view(TILES, 128), want), "bytes from %d" % first
