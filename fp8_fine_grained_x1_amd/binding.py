"""ctypes binding of libfp8fg.so -- argument marshalling only.

Each function has the name and the parameter list of the C entry point in
``include/fp8fg.h``.  Pointer parameters accept a torch tensor (its
``data_ptr()`` is passed), a raw integer address, or None (NULL).  ``stream``
accepts a ``torch.cuda.Stream``, a raw ``hipStream_t`` integer, or None: the
current torch stream of the tensors' device, or NULL when no CUDA tensor is
involved.  The call runs with the tensors' device made current.

A nonzero status raises ``Fp8fgError`` unless ``check=False`` (then the
status is returned).  All computation happens in the library's HIP kernels;
there is no fallback: if the library is missing, the import of its handle
raises.
"""

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8fg.so")

# mirrors of the header's enums
FP8FG_OK, FP8FG_EINVAL, FP8FG_ESHAPE, FP8FG_EALIGN, FP8FG_EUNSUPPORTED, FP8FG_ELAUNCH = range(6)
FP8FG_BF16, FP8FG_F32, FP8FG_E4M3 = 0, 1, 2
FP8FG_TILE_1x128, FP8FG_TILE_128x1 = 0, 1
FP8FG_SCALE_AMAX, FP8FG_SCALE_POW2 = 0, 1
FP8FG_BSCALE_BLOCK128, FP8FG_BSCALE_COL = 0, 1
FP8FG_GEMM_DEFAULT, FP8FG_GEMM_NO_PROMOTION, FP8FG_GEMM_FP8_MFMA, FP8FG_GEMM_E8M0_SCALES = 0, 1, 2, 4
FP8FG_GEMM_TILES_WIDE, FP8FG_GEMM_TILES_NARROW = 8, 16
FP8FG_SCORE_SOFTMAX, FP8FG_SCORE_SIGMOID = 0, 1

EXPORTED = ("fp8_quantize_rowtile", "fp8_quantize_block", "fp8_gemm_blockscaled",
            "fp8_grouped_gemm_blockscaled", "fp8_rmsnorm_quantize",
            "fp8_rmsnorm_backward_workspace", "fp8_rmsnorm_backward", "fp8_route",
            "fp8_route_backward", "fp8_dispatch_workspace", "fp8_dispatch", "fp8_combine",
            "fp8_combine_backward", "fp8fg_status_string")


class Fp8fgError(RuntimeError):
    def __init__(self, status, func):
        self.status = status
        super().__init__("%s failed: status %d (%s)" % (func, status, status_string(status)))


_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_F = ctypes.c_float

_SIGS = {
    "fp8_quantize_rowtile": [_P, _I, _L, _L, _L, _P, _L, _L, _I, _I, _P, _L, _P, _L, _L, _P],
    "fp8_quantize_block": [_P, _I, _L, _L, _L, _I, _I, _P, _L, _P, _L, _L, _P],
    "fp8_gemm_blockscaled": [_L, _L, _L, _P, _L, _P, _L, _L, _P, _L, _P, _L, _L, _I, _P, _I, _L,
                             _I, _P],
    "fp8_grouped_gemm_blockscaled": [_L, _P, _L, _L, _L, _P, _L, _P, _L, _L, _P, _L, _L, _P, _L,
                                     _L, _L, _P, _I, _L, _I, _P],
    "fp8_rmsnorm_quantize": [_P, _I, _L, _L, _L, _P, _L, _P, _I, _F, _I, _P, _L, _P, _L, _P, _L,
                             _P, _L, _L, _P, _P],
    "fp8_rmsnorm_backward": [_P, _I, _L, _L, _L, _P, _L, _P, _L, _P, _I, _P, _P, _L, _P, _P, _L,
                             _P],
    "fp8_route": [_P, _I, _L, _L, _L, _P, _I, _L, _L, _I, _L, _I, _F, _P, _L, _P, _L, _P],
    "fp8_route_backward": [_P, _I, _L, _L, _L, _I, _L, _I, _F, _P, _L, _P, _L, _P, _L, _P],
    "fp8_dispatch": [_P, _L, _L, _L, _L, _P, _I, _L, _L, _P, _L, _L, _P, _P, _P, _P, _L, _P, _L,
                     _L, _P, _L, _P],
    "fp8_combine": [_P, _I, _L, _L, _L, _L, _L, _P, _P, _L, _P, _L, _P, _L, _P],
    "fp8_combine_backward": [_P, _I, _L, _L, _L, _L, _L, _P, _L, _P, _P, _L, _P, _L, _P, _L, _P],
}

# functions that return a size in bytes instead of a status
_SIZES = {
    "fp8_rmsnorm_backward_workspace": [_L, _L],
    "fp8_dispatch_workspace": [_L, _L, _L],
}


def lib():
    """The loaded library (loaded once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libfp8fg.so is not built; run `python -m fp8_fine_grained_x1_amd.build`")
        l = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        for name, args in _SIZES.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = ctypes.c_int64
        l.fp8fg_status_string.argtypes = [ctypes.c_int]
        l.fp8fg_status_string.restype = ctypes.c_char_p
        _lib = l
    return _lib


def status_string(status):
    return lib().fp8fg_status_string(int(status)).decode()


def _ptr(x):
    if x is None or type(x) is int:
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return int(x)


def _cuda_device(args):
    for a in args:
        if getattr(a, "is_cuda", False):
            return a.device
    return None


def _stream(stream, device):
    if stream is None:
        if device is None:
            return None
        import torch
        return torch._C._cuda_getCurrentRawStream(device.index)
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


def _call(name, check, ptr_args, build):
    # A call costs a few microseconds of host time, which is what the calls
    # on few rows take altogether: the device is made current only where it
    # is not already.
    dev = _cuda_device(ptr_args)
    fn = getattr(_lib or lib(), name)
    if dev is None:
        rc = fn(*build(None))
    else:
        import torch
        if torch.cuda.current_device() == dev.index:
            rc = fn(*build(dev))
        else:
            with torch.cuda.device(dev):
                rc = fn(*build(dev))
    if check and rc != FP8FG_OK:
        raise Fp8fgError(rc, name)
    return rc


def fp8_quantize_rowtile(x, x_type, rows, cols, ldx, x_scale, xs_rs, xs_ts, tile, scale_rule,
                         q, ldq, s, s_rs, s_ts, stream=None, check=True):
    return _call("fp8_quantize_rowtile", check, (x, x_scale, q, s), lambda dev: (
        _ptr(x), x_type, rows, cols, ldx, _ptr(x_scale), xs_rs, xs_ts, tile, scale_rule,
        _ptr(q), ldq, _ptr(s), s_rs, s_ts, _stream(stream, dev)))


def fp8_quantize_block(w, w_type, rows, cols, ldw, scale_rule, transpose_out, q, ldq, s, s_rs,
                       s_cs, stream=None, check=True):
    return _call("fp8_quantize_block", check, (w, q, s), lambda dev: (
        _ptr(w), w_type, rows, cols, ldw, scale_rule, transpose_out, _ptr(q), ldq, _ptr(s),
        s_rs, s_cs, _stream(stream, dev)))


def fp8_gemm_blockscaled(M, N, K, a, lda, sa, sa_ms, sa_ks, b, ldb, sb, sb_ns, sb_ks,
                         b_scale_mode, c, c_type, ldc, flags, stream=None, check=True):
    return _call("fp8_gemm_blockscaled", check, (a, sa, b, sb, c), lambda dev: (
        M, N, K, _ptr(a), lda, _ptr(sa), sa_ms, sa_ks, _ptr(b), ldb, _ptr(sb), sb_ns, sb_ks,
        b_scale_mode, _ptr(c), c_type, ldc, flags, _stream(stream, dev)))


def fp8_grouped_gemm_blockscaled(G, offsets, M_total, N, K, a, lda, sa, sa_ms, sa_ks, b, ldb,
                                 b_gs, sb, sb_ns, sb_ks, sb_gs, c, c_type, ldc, flags,
                                 stream=None, check=True):
    return _call("fp8_grouped_gemm_blockscaled", check, (offsets, a, sa, b, sb, c), lambda dev: (
        G, _ptr(offsets), M_total, N, K, _ptr(a), lda, _ptr(sa), sa_ms, sa_ks, _ptr(b), ldb,
        b_gs, _ptr(sb), sb_ns, sb_ks, sb_gs, _ptr(c), c_type, ldc, flags,
        _stream(stream, dev)))


def fp8_rmsnorm_quantize(x, x_type, rows, cols, ldx, r, ldr, gamma, g_type, eps, scale_rule, h, ldh,
                         y, ldy, q, ldq, s, s_rs, s_ts, rstd, stream=None, check=True):
    return _call("fp8_rmsnorm_quantize", check, (x, r, gamma, h, y, q, s, rstd), lambda dev: (
        _ptr(x), x_type, rows, cols, ldx, _ptr(r), ldr, _ptr(gamma), g_type, eps, scale_rule,
        _ptr(h), ldh, _ptr(y), ldy, _ptr(q), ldq, _ptr(s), s_rs, s_ts, _ptr(rstd),
        _stream(stream, dev)))


def fp8_rmsnorm_backward_workspace(rows, cols):
    return lib().fp8_rmsnorm_backward_workspace(rows, cols)


def fp8_rmsnorm_backward(dy, x_type, rows, cols, lddy, dh, lddh, h, ldh, gamma, g_type, rstd, dx,
                         lddx, dgamma, workspace, workspace_bytes, stream=None, check=True):
    return _call("fp8_rmsnorm_backward", check, (dy, dh, h, gamma, rstd, dx, dgamma, workspace), lambda dev: (
        _ptr(dy), x_type, rows, cols, lddy, _ptr(dh), lddh, _ptr(h), ldh, _ptr(gamma), g_type,
        _ptr(rstd), _ptr(dx), lddx, _ptr(dgamma), _ptr(workspace), workspace_bytes,
        _stream(stream, dev)))


def fp8_route(logits, l_type, rows, experts, ldl, bias, score, groups, top_groups, group_top, k,
              renorm, scale, idx, ld_idx, w, ldw, stream=None, check=True):
    return _call("fp8_route", check, (logits, bias, idx, w), lambda dev: (
        _ptr(logits), l_type, rows, experts, ldl, _ptr(bias), score, groups, top_groups, group_top,
        k, renorm, scale, _ptr(idx), ld_idx, _ptr(w), ldw, _stream(stream, dev)))


def fp8_route_backward(logits, l_type, rows, experts, ldl, score, k, renorm, scale, idx, ld_idx, dw,
                       lddw, dlogits, lddl, stream=None, check=True):
    return _call("fp8_route_backward", check, (logits, idx, dw, dlogits), lambda dev: (
        _ptr(logits), l_type, rows, experts, ldl, score, k, renorm, scale, _ptr(idx), ld_idx,
        _ptr(dw), lddw, _ptr(dlogits), lddl, _stream(stream, dev)))


def fp8_dispatch_workspace(tokens, k, experts):
    return lib().fp8_dispatch_workspace(tokens, k, experts)


def fp8_dispatch(idx, ld_idx, tokens, k, experts, x, x_type, cols, ldx, xs, xs_rs, xs_ts, offsets,
                 pos, token, out, ldo, os, os_rs, os_ts, workspace, workspace_bytes, stream=None,
                 check=True):
    return _call("fp8_dispatch", check, (idx, x, xs, offsets, pos, token, out, os, workspace), lambda dev: (
        _ptr(idx), ld_idx, tokens, k, experts, _ptr(x), x_type, cols, ldx, _ptr(xs), xs_rs, xs_ts,
        _ptr(offsets), _ptr(pos), _ptr(token), _ptr(out), ldo, _ptr(os), os_rs, os_ts,
        _ptr(workspace), workspace_bytes, _stream(stream, dev)))


def fp8_combine(z, type, z_rows, tokens, k, cols, ldz, pos, w, ldw, base, ldb, out, ldo, stream=None,
                check=True):
    return _call("fp8_combine", check, (z, pos, w, base, out), lambda dev: (
        _ptr(z), type, z_rows, tokens, k, cols, ldz, _ptr(pos), _ptr(w), ldw, _ptr(base), ldb,
        _ptr(out), ldo, _stream(stream, dev)))


def fp8_combine_backward(dy, type, z_rows, tokens, k, cols, lddy, z, ldz, pos, w, ldw, dz, lddz, dw,
                         lddw, stream=None, check=True):
    return _call("fp8_combine_backward", check, (dy, z, pos, w, dz, dw), lambda dev: (
        _ptr(dy), type, z_rows, tokens, k, cols, lddy, _ptr(z), ldz, _ptr(pos), _ptr(w), ldw,
        _ptr(dz), lddz, _ptr(dw), lddw, _stream(stream, dev)))
