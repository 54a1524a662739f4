"""The silu gate on more tiles than its largest grid takes at once (2^25), whose
last workgroups go round their loop again: the last rows against a call on those
rows alone."""

import pytest
import torch

from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

ROWS = (1 << 25) + 4099


def filled(cols, gen):
    out = torch.empty((ROWS, cols), dtype=torch.bfloat16, device=DEV)
    for part in out.split(1 << 22):
        part.normal_(generator=gen)
    return out


@pytest.mark.parametrize("layout", ["group_major", "row_major"])
def test_more_tiles_than_the_grid(layout):
    say("gate of %d tiles" % ROWS)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    u = filled(256, gen)
    out = T.swiglu_quantize(u, scale_layout=layout)
    parts = (slice(0, 64), slice((1 << 25) - 64, (1 << 25) + 64), slice(ROWS - 4099, ROWS))
    for p in parts:
        assert all(torch.equal(a[p], b) for a, b in zip(out, T.swiglu_quantize(u[p], scale_layout=layout)))
    _, _, uq, us = out
    del u, out
    da = filled(128, gen)
    out = T.swiglu_backward(da, uq, us, scale_layout=layout)
    for p in parts:
        want = T.swiglu_backward(da[p], uq[p], us[p], scale_layout=layout)
        assert torch.equal(out[0][p], want[0]) and torch.equal(out[1][p], want[1])
    del da, uq, us, out
    torch.cuda.empty_cache()
