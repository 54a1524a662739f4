"""A gate of rows that is one row, expanded: its pitch of 0 means a gate per
column to the library, of the gammas' type, which an expanded row of x's type
need not hold.  It is refused; the vector is the way to pass it."""

import pytest
import torch

from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gtype", [torch.bfloat16, torch.float32])
def test_expanded_rows_are_refused(dtype, gtype):
    x = torch.randn((6, 256), device=DEV).to(dtype)
    g = torch.ones(256, dtype=gtype, device=DEV)
    n = torch.ones(6, device=DEV)
    for gate in (x[:1].expand(6, 256), x[0].expand(6, 256)):
        with pytest.raises(ValueError, match="gate"):
            T.rmsnorm_block_quantize(x, x, g, g, gate=gate)
        with pytest.raises(ValueError, match="gate"):
            T.rmsnorm_block_backward(x, x, x, g, g, n, n, gate=gate)
    # rows of their own, a single row, and none are taken
    out = T.rmsnorm_block_quantize(x, x, g, g, gate=x[:1].expand(6, 256).contiguous())
    one = T.rmsnorm_block_quantize(x[:1], x[:1], g, g, gate=x[:1].expand(1, 256))
    assert torch.equal(one[2], out[2][:1])
    grads = T.rmsnorm_block_backward(x[:1], x[:1], one[2], g, g, one[4], one[5], gate=x[:1].expand(1, 256))
    assert grads[4].shape == (1, 256) and grads[4].dtype == dtype
    assert T.rmsnorm_block_quantize(x[:0], x[:0], g, g, gate=x[:0])[2].shape == (0, 256)
