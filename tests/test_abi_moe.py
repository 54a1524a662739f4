"""The C-ABI boundary of the norm, router and row-movement entry points on
the CPU: every invalid call is refused with the documented status before any
HIP call, empty calls are no-ops, workspace sizes are what the calls take.
Also the tensor helpers' own refusals."""

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


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(B.LIB_PATH):
        build.build(verbose=False)
    return B.lib()


def norm(**kw):
    a = dict(x=P, x_type=B.FP8FG_BF16, rows=4, cols=256, ldx=256, r=P, ldr=256, gamma=P, g_type=B.FP8FG_F32, eps=1e-6,
             scale_rule=0, h=P, ldh=256, y=P, ldy=256, q=P, ldq=256, s=P, s_rs=1, s_ts=4, rstd=P, stream=0, check=False)
    a.update(kw)
    return B.fp8_rmsnorm_quantize(**a)


def norm_grad(**kw):
    a = dict(dy=P, x_type=B.FP8FG_BF16, rows=4, cols=256, lddy=256, dh=P, lddh=256, h=P, ldh=256, gamma=P,
             g_type=B.FP8FG_F32, rstd=P, dx=P, lddx=256, dgamma=P, workspace=P, workspace_bytes=BIG, stream=0, check=False)
    a.update(kw)
    return B.fp8_rmsnorm_backward(**a)


def route(**kw):
    a = dict(logits=P, l_type=B.FP8FG_F32, rows=4, experts=64, ldl=64, bias=P, score=1, groups=8, top_groups=4, group_top=2,
             k=6, renorm=1, scale=1.0, idx=P, ld_idx=6, w=P, ldw=6, stream=0, check=False)
    a.update(kw)
    return B.fp8_route(**a)


def route_grad(**kw):
    a = dict(logits=P, l_type=B.FP8FG_F32, rows=4, experts=64, ldl=64, score=1, k=6, renorm=1, scale=1.0, idx=P, ld_idx=6,
             dw=P, lddw=6, dlogits=P, lddl=64, stream=0, check=False)
    a.update(kw)
    return B.fp8_route_backward(**a)


def dispatch(**kw):
    a = dict(idx=P, ld_idx=2, tokens=4, k=2, experts=8, x=P, x_type=B.FP8FG_E4M3, cols=256, ldx=256, xs=P, xs_rs=1, xs_ts=4,
             offsets=P, pos=P, token=P, out=P, ldo=256, os=P, os_rs=1, os_ts=8, workspace=P, workspace_bytes=BIG, stream=0,
             check=False)
    a.update(kw)
    return B.fp8_dispatch(**a)


def combine(**kw):
    a = dict(z=P, type=B.FP8FG_BF16, z_rows=8, tokens=4, k=2, cols=264, ldz=264, pos=P, w=P, ldw=2, base=P, ldb=264, out=P,
             ldo=264, stream=0, check=False)
    a.update(kw)
    return B.fp8_combine(**a)


def combine_grad(**kw):
    a = dict(dy=P, type=B.FP8FG_BF16, z_rows=8, tokens=4, k=2, cols=264, lddy=264, z=P, ldz=264, pos=P, w=P, ldw=2, dz=P,
             lddz=264, dw=P, lddw=2, stream=0, check=False)
    a.update(kw)
    return B.fp8_combine_backward(**a)


INVAL, SHAPE, ALIGN, UNSUP, OK = B.FP8FG_EINVAL, B.FP8FG_ESHAPE, B.FP8FG_EALIGN, B.FP8FG_EUNSUPPORTED, B.FP8FG_OK
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [
    (dict(x_type=B.FP8FG_E4M3), INVAL), (dict(g_type=2), INVAL), (dict(scale_rule=2), INVAL), (dict(rows=-1), INVAL),
    (dict(ldr=-1), INVAL), (dict(s_ts=-1), INVAL), (dict(eps=-1e-9), INVAL), (dict(eps=NAN), INVAL), (dict(eps=INF), INVAL),
    (dict(x=None), INVAL), (dict(gamma=None), INVAL), (dict(s=None), INVAL),
    (dict(cols=200), SHAPE), (dict(ldx=128), SHAPE), (dict(ldr=128), SHAPE), (dict(ldh=128), SHAPE), (dict(ldy=128), SHAPE),
    (dict(ldq=128), SHAPE),
    (dict(x=P + 8), ALIGN), (dict(r=P + 2), ALIGN), (dict(gamma=P + 4), ALIGN), (dict(h=P + 8), ALIGN), (dict(y=P + 8), ALIGN),
    (dict(q=P + 8), ALIGN), (dict(s=P + 2), ALIGN), (dict(rstd=P + 1), ALIGN), (dict(ldx=260), ALIGN), (dict(ldq=264), ALIGN),
    (dict(cols=32768 + 128, ldx=1 << 16, ldr=1 << 16, ldh=1 << 16, ldy=1 << 16, ldq=1 << 16), UNSUP),
    (dict(rows=1 << 31), UNSUP), (dict(ldx=1 << 30), UNSUP), (dict(s_ts=1 << 31), UNSUP),
    (dict(rows=0), OK), (dict(cols=0), OK), (dict(rows=0, x=None, gamma=None), OK),
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x_type=2), INVAL), (dict(g_type=7), INVAL), (dict(rows=-1), INVAL), (dict(workspace_bytes=-1), INVAL),
    (dict(dy=None), INVAL), (dict(h=None), INVAL), (dict(dx=None), INVAL), (dict(gamma=None), INVAL), (dict(rstd=None), INVAL),
    (dict(dgamma=None), INVAL), (dict(workspace=None), INVAL), (dict(rows=0, dgamma=None), INVAL),
    (dict(cols=252), SHAPE), (dict(lddy=128), SHAPE), (dict(lddh=128), SHAPE), (dict(ldh=128), SHAPE), (dict(lddx=128), SHAPE),
    (dict(workspace_bytes=15), SHAPE),
    (dict(dy=P + 8), ALIGN), (dict(h=P + 8), ALIGN), (dict(dh=P + 8), ALIGN), (dict(dx=P + 8), ALIGN), (dict(gamma=P + 8), ALIGN),
    (dict(rstd=P + 2), ALIGN), (dict(dgamma=P + 2), ALIGN), (dict(workspace=P + 4), ALIGN), (dict(ldh=260), ALIGN),
    (dict(cols=32776, lddy=1 << 16, lddh=1 << 16, ldh=1 << 16, lddx=1 << 16), UNSUP), (dict(rows=1 << 31), UNSUP),
    (dict(cols=0), OK),
])
def test_norm_gradient_refusals(kw, status):
    assert norm_grad(**kw) == status


ROUTE_BOTH = [
    (dict(l_type=2), INVAL), (dict(score=2), INVAL), (dict(renorm=2), INVAL), (dict(rows=-1), INVAL), (dict(experts=0), INVAL),
    (dict(k=0), INVAL), (dict(scale=NAN), INVAL), (dict(scale=INF), INVAL), (dict(logits=None), INVAL), (dict(idx=None), INVAL),
    (dict(ld_idx=-1), INVAL), (dict(ldl=32), SHAPE), (dict(ld_idx=5), SHAPE), (dict(logits=P + 2), ALIGN), (dict(idx=P + 2), ALIGN),
    (dict(rows=1 << 31), UNSUP), (dict(ldl=1 << 30), UNSUP), (dict(rows=0), OK), (dict(rows=0, logits=None, idx=None), OK),
]


@pytest.mark.parametrize("kw,status", ROUTE_BOTH + [
    (dict(groups=0), INVAL), (dict(top_groups=0), INVAL), (dict(group_top=3), INVAL), (dict(w=None), INVAL), (dict(groups=7), SHAPE),
    (dict(top_groups=9), SHAPE), (dict(k=65, ld_idx=65, ldw=65), SHAPE), (dict(ldw=5), SHAPE), (dict(bias=P + 2), ALIGN),
    (dict(w=P + 1), ALIGN), (dict(experts=1032, ldl=1032), UNSUP), (dict(experts=128, ldl=128, k=65, ld_idx=65, ldw=65), UNSUP),
])
def test_route_refusals(kw, status):
    assert route(**kw) == status


@pytest.mark.parametrize("kw,status", ROUTE_BOTH + [
    (dict(dw=None), INVAL), (dict(dlogits=None), INVAL), (dict(lddw=5), SHAPE), (dict(lddl=63), SHAPE), (dict(dw=P + 2), ALIGN),
    (dict(dlogits=P + 2), ALIGN), (dict(experts=1025, ldl=1025, lddl=1025), UNSUP),
])
def test_route_gradient_refusals(kw, status):
    assert route_grad(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x_type=3), INVAL), (dict(tokens=-1), INVAL), (dict(k=0), INVAL), (dict(experts=0), INVAL), (dict(os_ts=-1), INVAL),
    (dict(idx=None), INVAL), (dict(xs=None), INVAL), (dict(os=None), INVAL), (dict(out=None), INVAL), (dict(offsets=None), INVAL),
    (dict(pos=None), INVAL), (dict(token=None), INVAL), (dict(workspace=None), INVAL),
    (dict(cols=200), SHAPE), (dict(ld_idx=1), SHAPE), (dict(ldx=128), SHAPE), (dict(ldo=128), SHAPE), (dict(workspace_bytes=3), SHAPE),
    (dict(x_type=B.FP8FG_BF16, cols=252), SHAPE),
    (dict(x=P + 8), ALIGN), (dict(out=P + 8), ALIGN), (dict(ldx=264), ALIGN), (dict(idx=P + 2), ALIGN), (dict(xs=P + 2), ALIGN),
    (dict(os=P + 2), ALIGN), (dict(pos=P + 2), ALIGN), (dict(token=P + 2), ALIGN), (dict(offsets=P + 2), ALIGN),
    (dict(workspace=P + 2), ALIGN),
    (dict(tokens=1 << 30), UNSUP), (dict(experts=1025), UNSUP), (dict(tokens=1 << 31, k=1 << 31, ld_idx=1 << 31), UNSUP),
    (dict(ldx=1 << 30), UNSUP), (dict(tokens=0, offsets=None), INVAL),
])
def test_dispatch_refusals(kw, status):
    assert dispatch(**kw) == status


COMBINE_BOTH = [
    (dict(type=2), INVAL), (dict(tokens=-1), INVAL), (dict(z_rows=-1), INVAL), (dict(k=0), INVAL), (dict(z=None), INVAL),
    (dict(pos=None), INVAL), (dict(cols=260), SHAPE), (dict(ldz=256), SHAPE), (dict(ldw=1), SHAPE), (dict(z=P + 8), ALIGN),
    (dict(pos=P + 2), ALIGN), (dict(w=P + 2), ALIGN), (dict(ldz=268), ALIGN), (dict(z_rows=1 << 31), UNSUP),
    (dict(tokens=1 << 31), UNSUP), (dict(ldz=1 << 30), UNSUP), (dict(tokens=0), OK),
]


@pytest.mark.parametrize("kw,status", COMBINE_BOTH + [
    (dict(out=None), INVAL), (dict(ldb=256), SHAPE), (dict(ldo=256), SHAPE), (dict(base=P + 8), ALIGN), (dict(out=P + 8), ALIGN),
    (dict(cols=0), OK),
])
def test_combine_refusals(kw, status):
    assert combine(**kw) == status


@pytest.mark.parametrize("kw,status", COMBINE_BOTH + [
    (dict(dy=None), INVAL), (dict(dz=None), INVAL), (dict(lddy=256), SHAPE), (dict(lddz=256), SHAPE), (dict(lddw=1), SHAPE),
    (dict(dy=P + 8), ALIGN), (dict(dz=P + 8), ALIGN), (dict(dw=P + 2), ALIGN),
])
def test_combine_gradient_refusals(kw, status):
    assert combine_grad(**kw) == status


def test_workspace_sizes():
    assert B.fp8_rmsnorm_backward_workspace(0, 256) == 0
    for rows, cols in ((1, 8), (100, 256), (10 ** 6, 32768)):
        n = B.fp8_rmsnorm_backward_workspace(rows, cols)
        assert cols * 4 <= n <= 1024 * cols * 4 and n % (cols * 4) == 0
        ld = dict(rows=rows, cols=cols, lddy=cols, lddh=cols, ldh=cols, lddx=cols)
        assert norm_grad(workspace_bytes=n - 1, **ld) == SHAPE
    for bad in ((-1, 256), (4, -8), (4, 40000)):
        assert B.fp8_rmsnorm_backward_workspace(*bad) == 0
    for tokens, k, experts in ((0, 1, 1), (5, 8, 256), (1 << 20, 8, 1024)):
        n = B.fp8_dispatch_workspace(tokens, k, experts)
        assert n >= (experts + 1) * 4
        if tokens:
            assert dispatch(tokens=tokens, k=k, ld_idx=k, experts=experts, workspace_bytes=n - 1) == SHAPE
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 1025), (1 << 30, 8, 8)):
        assert B.fp8_dispatch_workspace(*bad) == 0


def test_tensor_helpers_refuse_what_the_library_cannot_see():
    # host memory, and (on the meta device, which has none) types and shapes
    cpu = torch.zeros(4, 256)
    g = torch.ones(256)
    i = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: T.rmsnorm_quantize(cpu, g), lambda: T.rmsnorm_backward(cpu, cpu, g, torch.ones(4)),
                 lambda: T.route(cpu, 2), lambda: T.route_backward(cpu[:, :2], cpu, i),
                 lambda: T.dispatch(i, 8, cpu), lambda: T.combine(cpu, i), lambda: T.combine_backward(cpu, cpu, i, None)):
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


@pytest.mark.parametrize("rows,cols", [(4, 252), (4, 4), (1 << 31, 256), (1 << 40, 8), (4, 32776)])
def test_no_workspace_for_a_refused_norm_gradient(rows, cols):
    assert B.fp8_rmsnorm_backward_workspace(rows, cols) == 0
    ld = max(cols, 8)
    assert norm_grad(rows=rows, cols=cols, lddy=ld, lddh=ld, ldh=ld, lddx=ld) in (SHAPE, ALIGN, UNSUP)


@pytest.mark.parametrize("k", [(1 << 31) - 15, (1 << 31) - 1, 1 << 31, 1 << 40])
def test_combine_refuses_places_past_its_steps(k):
    # (the kernels count the places in int32, 8 at a time)
    assert combine(tokens=1, k=k, w=None) == UNSUP
    assert combine_grad(tokens=1, k=k, w=None, dw=None, z=None) == UNSUP


def test_tensor_helpers_refuse_what_is_no_tensor():
    i = torch.zeros((4, 2), dtype=torch.int32)
    for bad in (None, 3, [[1.0]], "x"):
        for call in (lambda **k: T.rmsnorm_quantize(bad, bad, **k), lambda **k: T.rmsnorm_backward(bad, bad, bad, bad, **k),
                     lambda **k: T.route(bad, 2, **k), lambda **k: T.route_backward(bad, bad, i, **k),
                     lambda **k: T.dispatch(i, 8, bad, **k), lambda **k: T.combine(bad, i, **k),
                     lambda **k: T.combine_backward(bad, bad, i, None, **k)):
            for kw in (dict(), dict(stream=0)):
                with pytest.raises(ValueError):
                    call(**kw)
