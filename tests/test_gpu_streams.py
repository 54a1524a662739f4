"""The quantizer and GEMM helpers with stream=: what they give is the current
stream's result bit for bit, outputs are the other stream's memory, and what
they read is not handed out again while that stream may still read it."""

import pytest
import torch

from fp8_fine_grained_x1_amd import tensors as T
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

M, K, N = 512, 1024, 768


def inputs():
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    x = torch.randn((M, K), generator=gen, device=DEV).to(torch.bfloat16)
    w = torch.randn((K, N), generator=gen, device=DEV).to(torch.bfloat16)
    qa, sa = T.quantize_1x128(x)
    qb, sb = T.quantize_block(w)
    off = torch.tensor([0, 100, 100, M], dtype=torch.int32, device=DEV)
    return dict(x=x, w=w, qa=qa, sa=sa, qb=qb, sb=sb, off=off, qg=torch.stack([qb] * 3), sg=torch.stack([sb] * 3))


# name -> (the call, the input that is its own)
CALLS = {
    "quantize_1x128": (lambda d, **k: T.quantize_1x128(d["x"], **k), "x"),
    "quantize_128x1": (lambda d, **k: T.quantize_128x1(d["x"], **k), "x"),
    "requantize_128x1": (lambda d, **k: T.requantize_128x1(d["qa"], d["sa"], **k), "qa"),
    "quantize_block": (lambda d, **k: T.quantize_block(d["w"], **k), "w"),
    "gemm": (lambda d, **k: (T.gemm(d["qa"], d["sa"], d["qb"], d["sb"], **k),), "qb"),
    "grouped_gemm": (lambda d, **k: (T.grouped_gemm(d["qa"], d["sa"], d["off"], d["qg"], d["sg"], **k),), "qg"),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("raw", [False, True])
def test_outputs_and_inputs_on_another_stream(name, raw):
    say("%s on another stream" % name)
    call, own = CALLS[name]
    d = inputs()
    want = call(d)
    side = torch.cuda.Stream()
    big = torch.randn((4096, 4096), device=DEV)
    torch.cuda.synchronize()
    # what the current stream frees is not where the other's outputs go
    freed = [torch.empty_like(t) for t in want]
    at = {t.data_ptr() for t in freed}
    del freed
    with torch.cuda.stream(side):
        for _ in range(20):
            big = big @ big.clamp(-1e-3, 1e-3)       # the call below waits behind these
    got = call(d, stream=side.cuda_stream if raw else side)
    assert not any(t.data_ptr() in at for t in got)
    # the input is given back while the other stream has yet to read it
    shape, dtype, was = d[own].shape, d[own].dtype, d[own].data_ptr()
    del d[own]
    again = torch.empty(shape, dtype=dtype, device=DEV)
    busy = not side.query()
    again.zero_()
    torch.cuda.synchronize()
    assert not busy or again.data_ptr() != was
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_out_given_and_the_null_handle():
    d = inputs()
    want = T.gemm(d["qa"], d["sa"], d["qb"], d["sb"])
    torch.cuda.synchronize()
    c = torch.zeros_like(want)
    torch.cuda.synchronize()
    for stream in (0, torch.cuda.Stream()):
        assert T.gemm(d["qa"], d["sa"], d["qb"], d["sb"], out=c, stream=stream) is c
        torch.cuda.synchronize()
        assert torch.equal(c, want)
        c.zero_()
        torch.cuda.synchronize()
