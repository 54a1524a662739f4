"""The C-ABI boundary of the silu gate, the balance loss and the norms around a
block on the CPU: every invalid call is refused with the documented status
before any HIP call, empty calls are no-ops, workspace sizes are what the calls
take.  Also the tensor helpers' own refusals."""

import os
import subprocess
import sys

import pytest
import torch

from fp8_fine_grained_x1_amd import binding as B
from fp8_fine_grained_x1_amd import build
from fp8_fine_grained_x1_amd import tensors as T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20       # a fake, aligned device address
BIG = 1 << 30
INVAL, SHAPE, ALIGN, UNSUP, OK = B.FP8FG_EINVAL, B.FP8FG_ESHAPE, B.FP8FG_EALIGN, B.FP8FG_EUNSUPPORTED, B.FP8FG_OK
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.LIB_PATH):
        build.build(verbose=False)
    return B.lib()


def gate(**kw):
    a = dict(u=P, u_type=B.FP8FG_BF16, rows=4, inner=256, ldu=512, used=P, scale_rule=0, q=P, ldq=256, s=P, s_rs=1, s_ts=4,
             uq=P, lduq=512, us=P, us_rs=1, us_ts=4, stream=0, check=False)
    a.update(kw)
    return B.fp8_swiglu_quantize(**a)


def gate_grad(**kw):
    a = dict(da=P, type=B.FP8FG_BF16, rows=4, inner=256, ldda=256, uq=P, lduq=512, us=P, us_rs=1, us_ts=4, used=P, scale_rule=0,
             dq=P, lddq=512, ds=P, ds_rs=1, ds_ts=4, du=P, lddu=512, a=P, lda=256, stream=0, check=False)
    a.update(kw)
    return B.fp8_swiglu_backward(**a)


def gate_grad_t(**kw):
    a = dict(da=P, type=B.FP8FG_BF16, rows=128, inner=256, ldda=256, uq=P, lduq=512, us=P, us_rs=1, us_ts=128, scale_rule=0, dq=P,
             lddq=512, ds=P, ds_rs=1, ds_ts=128, dqt=P, lddqt=128, dst=P, dst_rs=1, dst_ts=512, aqt=P, ldaqt=128, ast=P, ast_rs=1,
             ast_ts=256, stream=0, check=False)
    a.update(kw)
    return B.fp8_swiglu_backward_128x1(**a)


def balance(**kw):
    a = dict(logits=P, l_type=B.FP8FG_F32, rows=4, experts=64, ldl=64, idx=P, ld_idx=6, k=6, offsets=P, seqs=3, score=1, scale=1.0,
             loss=P, counts=P, slope=P, workspace=P, workspace_bytes=BIG, stream=0, check=False)
    a.update(kw)
    return B.fp8_balance_loss(**a)


def balance_grad(**kw):
    a = dict(dloss=P, logits=P, l_type=B.FP8FG_F32, rows=4, experts=64, ldl=64, slope=P, offsets=P, seqs=3, score=1, base=P,
             ldb=64, dlogits=P, lddl=64, stream=0, check=False)
    a.update(kw)
    return B.fp8_balance_loss_backward(**a)


def block(**kw):
    a = dict(z=P, x_type=B.FP8FG_BF16, rows=4, cols=256, ldz=256, r=P, ldr=256, gamma_post=P, gamma=P, g_type=B.FP8FG_F32, gate=P,
             ldg=256, residual_scale=1.0, block_scale=1.0, eps=1e-6, scale_rule=0, h=P, ldh=256, y=P, ldy=256, q=P, ldq=256, s=P,
             s_rs=1, s_ts=4, rstd_post=P, rstd=P, stream=0, check=False)
    a.update(kw)
    return B.fp8_rmsnorm_block_quantize(**a)


def block_grad(**kw):
    a = dict(dy=P, x_type=B.FP8FG_BF16, rows=4, cols=256, lddy=256, dh=P, lddh=256, z=P, ldz=256, h=P, ldh=256, gamma_post=P,
             gamma=P, g_type=B.FP8FG_F32, gate=P, ldg=256, rstd_post=P, rstd=P, residual_scale=1.0, block_scale=1.0, dz=P, lddz=256,
             dr=P, lddr=256, dgamma_post=P, dgamma=P, dgate=P, lddg=256, workspace=P, workspace_bytes=BIG, stream=0, check=False)
    a.update(kw)
    return B.fp8_rmsnorm_block_backward(**a)


GATE_ALL = [
    (dict(scale_rule=2), INVAL), (dict(rows=-1), INVAL), (dict(inner=-128), INVAL), (dict(us_rs=-1), INVAL), (dict(inner=200), SHAPE),
    (dict(lduq=384), SHAPE), (dict(uq=P + 8), ALIGN), (dict(us=P + 2), ALIGN), (dict(us=None), INVAL), (dict(lduq=520), ALIGN),
    (dict(us_ts=1 << 31), UNSUP), (dict(us_rs=1 << 30), UNSUP), (dict(rows=0), OK), (dict(inner=0), OK),
]


@pytest.mark.parametrize("kw,status", GATE_ALL + [
    (dict(u_type=B.FP8FG_E4M3), INVAL), (dict(u=None), INVAL), (dict(q=None), INVAL), (dict(s=None), INVAL), (dict(ldu=256), SHAPE),
    (dict(ldq=128), SHAPE), (dict(u=P + 8), ALIGN), (dict(q=P + 4), ALIGN), (dict(s=P + 1), ALIGN), (dict(used=P + 2), ALIGN),
    (dict(ldu=516), ALIGN), (dict(rows=1 << 31), UNSUP), (dict(rows=(1 << 31) - 1, inner=256), UNSUP), (dict(ldu=1 << 30), UNSUP),
    (dict(inner=1 << 28, ldu=1 << 29, ldq=1 << 28, lduq=1 << 29, rows=1), UNSUP), (dict(inner=1 << 62), UNSUP),
    (dict(rows=0, u=None, s=None), OK),
])
def test_gate_refusals(kw, status):
    assert gate(**kw) == status


@pytest.mark.parametrize("kw,status", GATE_ALL + [
    (dict(type=B.FP8FG_E4M3), INVAL), (dict(da=None), INVAL), (dict(uq=None), INVAL), (dict(ds=None), INVAL),
    (dict(dq=None, du=None, a=None), INVAL), (dict(ldda=128), SHAPE), (dict(lddq=256), SHAPE), (dict(lddu=256), SHAPE),
    (dict(lda=128), SHAPE), (dict(da=P + 8), ALIGN), (dict(dq=P + 8), ALIGN), (dict(du=P + 8), ALIGN), (dict(a=P + 2), ALIGN),
    (dict(ds=P + 2), ALIGN), (dict(used=P + 1), ALIGN), (dict(lddq=520), ALIGN), (dict(rows=1 << 31), UNSUP), (dict(lda=1 << 30), UNSUP),
    (dict(ds_ts=1 << 31), UNSUP),
])
def test_gate_gradient_refusals(kw, status):
    assert gate_grad(**kw) == status


@pytest.mark.parametrize("kw,status", GATE_ALL + [
    (dict(type=3), INVAL), (dict(da=None), INVAL), (dict(uq=None), INVAL), (dict(dq=None), INVAL), (dict(dqt=None), INVAL),
    (dict(aqt=None), INVAL), (dict(ds=None), INVAL), (dict(dst=None), INVAL), (dict(ast=None), INVAL), (dict(rows=100), SHAPE),
    (dict(rows=256), SHAPE), (dict(ldda=128), SHAPE), (dict(lddq=256), SHAPE), (dict(lddqt=64), SHAPE), (dict(ldaqt=64), SHAPE),
    (dict(dqt=P + 8), ALIGN), (dict(aqt=P + 8), ALIGN), (dict(dst=P + 2), ALIGN), (dict(ast=P + 2), ALIGN), (dict(lddqt=136), ALIGN),
    (dict(rows=128 * 65536, lddqt=1 << 24, ldaqt=1 << 24), UNSUP), (dict(dst_ts=1 << 31), UNSUP), (dict(ast_rs=1 << 30), UNSUP),
])
def test_gate_gradient_128x1_refusals(kw, status):
    assert gate_grad_t(**kw) == status


BALANCE_BOTH = [
    (dict(l_type=2), INVAL), (dict(score=2), INVAL), (dict(rows=-1), INVAL), (dict(experts=0), INVAL), (dict(seqs=-1), INVAL),
    (dict(offsets=None), INVAL), (dict(logits=None), INVAL), (dict(slope=None), INVAL), (dict(ldl=32), SHAPE), (dict(logits=P + 2), ALIGN),
    (dict(offsets=P + 2), ALIGN), (dict(slope=P + 2), ALIGN), (dict(rows=1 << 31), UNSUP), (dict(ldl=1 << 30), UNSUP),
    (dict(seqs=1 << 31), UNSUP),
]


@pytest.mark.parametrize("kw,status", BALANCE_BOTH + [
    (dict(k=0), INVAL), (dict(scale=NAN), INVAL), (dict(scale=INF), INVAL), (dict(idx=None), INVAL), (dict(loss=None), INVAL),
    (dict(counts=None), INVAL), (dict(workspace=None), INVAL), (dict(workspace_bytes=-1), INVAL), (dict(ld_idx=5), SHAPE),
    (dict(k=65, ld_idx=65), SHAPE), (dict(workspace_bytes=15), SHAPE), (dict(idx=P + 2), ALIGN), (dict(loss=P + 2), ALIGN),
    (dict(counts=P + 2), ALIGN), (dict(workspace=P + 8), ALIGN), (dict(experts=1025, ldl=1025), UNSUP),
    (dict(experts=128, ldl=128, k=65, ld_idx=65), UNSUP), (dict(rows=1 << 28, k=8, ld_idx=8), UNSUP),
    (dict(seqs=0), OK), (dict(seqs=0, logits=None, loss=None), OK),
    (dict(rows=0, loss=None), INVAL),
])
def test_balance_refusals(kw, status):
    assert balance(**kw) == status


@pytest.mark.parametrize("kw,status", BALANCE_BOTH + [
    (dict(dlogits=None), INVAL), (dict(ldb=-1), INVAL), (dict(ldb=63), SHAPE), (dict(lddl=63), SHAPE), (dict(base=P + 2), ALIGN),
    (dict(dlogits=P + 1), ALIGN), (dict(dloss=P + 2), ALIGN), (dict(experts=1025, ldl=1025, ldb=1025, lddl=1025), UNSUP),
    (dict(lddl=1 << 30), UNSUP), (dict(rows=0), OK), (dict(rows=0, logits=None, dlogits=None), OK),
])
def test_balance_gradient_refusals(kw, status):
    assert balance_grad(**kw) == status


WIDE = dict(cols=16384 + 128, ldz=1 << 16, ldg=1 << 16, ldh=1 << 16)
BLOCK_BOTH = [
    (dict(x_type=2), INVAL), (dict(g_type=2), INVAL), (dict(rows=-1), INVAL), (dict(ldg=-1), INVAL), (dict(residual_scale=NAN), INVAL),
    (dict(block_scale=INF), INVAL), (dict(z=None), INVAL), (dict(h=None), INVAL), (dict(gamma=None), None), (dict(gamma_post=None), None),
    (dict(ldz=128), SHAPE), (dict(ldh=128), SHAPE), (dict(ldg=128), SHAPE), (dict(z=P + 8), ALIGN), (dict(h=P + 8), ALIGN),
    (dict(gate=P + 8), ALIGN), (dict(gamma=P + 8), ALIGN), (dict(gamma_post=P + 4), ALIGN), (dict(rstd=P + 2), ALIGN),
    (dict(rstd_post=P + 2), ALIGN), (dict(ldz=260), ALIGN), (dict(rows=1 << 31), UNSUP), (dict(ldg=1 << 30), UNSUP), (dict(cols=0), OK),
]
BLOCK_BOTH = [(kw, INVAL if st is None else st) for kw, st in BLOCK_BOTH]


@pytest.mark.parametrize("kw,status", BLOCK_BOTH + [
    (dict(scale_rule=2), INVAL), (dict(eps=-1.0), INVAL), (dict(eps=NAN), INVAL), (dict(r=None), INVAL), (dict(s=None), INVAL),
    (dict(cols=200), SHAPE), (dict(ldr=128), SHAPE), (dict(ldy=128), SHAPE), (dict(ldq=128), SHAPE), (dict(r=P + 8), ALIGN),
    (dict(y=P + 8), ALIGN), (dict(q=P + 8), ALIGN), (dict(s=P + 2), ALIGN), (dict(ldq=264), ALIGN), (dict(s_ts=1 << 31), UNSUP),
    (dict(WIDE, ldr=1 << 16, ldy=1 << 16, ldq=1 << 16), UNSUP), (dict(rows=0), OK), (dict(rows=0, z=None, gamma=None), OK),
])
def test_block_refusals(kw, status):
    assert block(**kw) == status


@pytest.mark.parametrize("kw,status", BLOCK_BOTH + [
    (dict(dy=None), INVAL), (dict(dz=None), INVAL), (dict(dr=None), INVAL), (dict(dgamma=None), INVAL), (dict(dgamma_post=None), INVAL),
    (dict(dgate=None), INVAL), (dict(ldg=0, dgate=None), INVAL), (dict(rows=0, ldg=0, dgate=None), INVAL), (dict(rstd=None), INVAL),
    (dict(rstd_post=None), INVAL), (dict(workspace=None), INVAL), (dict(workspace_bytes=-1), INVAL), (dict(rows=0, dgamma=None), INVAL),
    (dict(rows=0, ldg=0, gamma_post=None), INVAL),
    (dict(cols=252), SHAPE), (dict(lddy=128), SHAPE), (dict(lddh=128), SHAPE), (dict(lddz=128), SHAPE), (dict(lddr=128), SHAPE),
    (dict(lddg=128), SHAPE), (dict(workspace_bytes=15), SHAPE), (dict(dy=P + 8), ALIGN), (dict(dh=P + 8), ALIGN), (dict(dz=P + 8), ALIGN),
    (dict(dr=P + 8), ALIGN), (dict(dgate=P + 8), ALIGN), (dict(ldg=0, dgate=P + 2), ALIGN), (dict(dgamma=P + 2), ALIGN),
    (dict(dgamma_post=P + 2), ALIGN), (dict(workspace=P + 8), ALIGN),
    (dict(WIDE, lddy=1 << 16, lddh=1 << 16, lddz=1 << 16, lddr=1 << 16, lddg=1 << 16), UNSUP), (dict(lddz=1 << 30), UNSUP),
])
def test_block_gradient_refusals(kw, status):
    assert block_grad(**kw) == status


def test_workspace_sizes():
    for rows, cols in ((1, 8), (100, 256), (10 ** 6, 16384)):
        n = B.fp8_rmsnorm_block_backward_workspace(rows, cols)
        assert cols * 8 <= n <= 2048 * cols * 4 and n % (cols * 8) == 0
        ld = dict(rows=rows, cols=cols, **{k: cols for k in ("lddy", "lddh", "ldz", "ldh", "ldg", "lddz", "lddr", "lddg")})
        assert block_grad(workspace_bytes=n - 1, **ld) == SHAPE
    for bad in ((-1, 256), (4, -8), (4, 252), (4, 16392), (1 << 31, 256)):
        assert B.fp8_rmsnorm_block_backward_workspace(*bad) == 0
    for rows, experts, seqs in ((0, 1, 1), (5, 256, 3), (10 ** 6, 1024, 77), ((1 << 31) - 1, 8, 1)):
        n = B.fp8_balance_loss_workspace(rows, experts, seqs)
        assert n > 0
        assert balance(rows=rows, experts=experts, ldl=experts, k=1, ld_idx=1, seqs=seqs, workspace_bytes=n - 1) == SHAPE
    for bad in ((-1, 8, 1), (1, 0, 1), (1, 1025, 1), (1, 8, -1), (1 << 31, 8, 1), (1, 8, 1 << 31)):
        assert B.fp8_balance_loss_workspace(*bad) == 0


def calls(x, v, i):
    """The helpers on x [4][256], v [256] or [4], i int32 [4][2]."""
    u8 = torch.zeros((4, 512), dtype=torch.uint8)
    return [lambda **k: T.swiglu_quantize(x, **k), lambda **k: T.swiglu_backward(x, u8, torch.zeros(4, 4), **k),
            lambda **k: T.swiglu_backward_128x1(x, u8, torch.zeros(4, 4), **k), lambda **k: T.balance_loss(x, i, **k),
            lambda **k: T.balance_loss_backward(None, x, torch.zeros(1, 256), **k),
            lambda **k: T.rmsnorm_block_quantize(x, x, v, v, **k),
            lambda **k: T.rmsnorm_block_backward(x, x, x, v, v, torch.ones(4), torch.ones(4), **k)]


def test_tensor_helpers_refuse_host_memory():
    for call in calls(torch.zeros(4, 256), torch.ones(256), torch.zeros((4, 2), dtype=torch.int32)):
        with pytest.raises(ValueError):
            call()


def test_tensor_helpers_refuse_what_is_no_tensor():
    for bad in (None, 3, [[1.0]], "x"):
        for call in calls(bad, bad, bad):
            for kw in (dict(), dict(stream=0)):
                with pytest.raises(ValueError):
                    call(**kw)


def test_tensor_helpers_refuse_unknown_names():
    x = torch.zeros(4, 256)
    for call in (lambda: T.swiglu_quantize(x, scale_layout="rows"), lambda: T.balance_loss(x, x, score="relu"),
                 lambda: T.rmsnorm_block_quantize(x, x, x, x, scale_layout="columns")):
        with pytest.raises(ValueError):
            call()


def test_under_host_sanitizers():
    # this file's argument matrix against a host-sanitized build
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    if os.environ.get("FP8FG_SANITIZED_CHILD"):
        pytest.skip("already under the sanitizers")
    path, _ = build.build_host_sanitized()
    env = dict(os.environ, LD_PRELOAD=build.asan_runtime(), FP8FG_SANITIZED_CHILD="1",
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    code = ("import sys; sys.path.insert(0, %r); from fp8_fine_grained_x1_amd import binding as B; B.LIB_PATH = %r; "
            "import pytest; sys.exit(pytest.main(['-q', '-p', 'no:cacheprovider', %r]))"
            % (ROOT, path, os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    text = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in text and "runtime error:" not in text, text[-4000:]
    assert r.returncode == 0, text[-4000:]
    assert " passed" in text and "failed" not in text
