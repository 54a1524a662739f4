"""Tensor-level helpers over the C ABI: allocate outputs with torch on the
inputs' device and call the binding.  No arithmetic happens here.

Layouts (row-major, last index contiguous):
  quantize_1x128(x [M][K])            -> q u8 [M][K],  s f32 [M][K/128]
  quantize_128x1(x [T][F])            -> qT u8 [F][T], sT f32 [F][T/128]
  requantize_128x1(q [T][F], s [T][F/128]) -> same as quantize_128x1
  Per-row tile scales are indexed s[row][group] in every case; by default
  they are stored group-major (the returned tensor is a transposed view of
  a [groups][rows] buffer, strides (1, rows)), so that the GEMM's per-group
  load of consecutive rows' scales is one contiguous read.
  scale_layout="row_major" stores them [rows][groups] instead.
  quantize_block(w [K][N], transpose) -> q u8 [N][K] (transpose) or [K][N],
                                         s f32 [K/128][N/128]
  gemm(qa [M][K], sa [M][K/128], qb [N][K], sb)  -> c [M][N]
       sb [K/128][N/128] (block scales) or [N][K/128] (per-column scales)
  grouped_gemm(qa, sa, offsets i32 [G+1], qb [G][N][K], sb [G][K/128][N/128])

A mixture-of-experts layer around them:
  rmsnorm_quantize(x [M][C], gamma [C], residual) -> q, s, h [M][C], y, rstd [M]
  rmsnorm_backward(dy, h, gamma, rstd, dh)        -> dx [M][C], dgamma [C]
  route(logits [M][E], k)          -> idx i32 [M][k], w f32 [M][k]
  route_backward(dw, logits, idx)  -> dlogits [M][E]
  dispatch(idx, E, x [M][C], s)    -> x' [M k][C], s', offsets i32 [E+1],
                                      pos i32 [M][k], token i32 [M k]
  combine(z [R][C], pos, w, base)  -> [M][C]
  combine_backward(dy, z, pos, w)  -> dz [R][C], dw [M][k]
These check the shapes, types, devices and row layouts that the C interface
cannot see and raise ValueError.

With ``stream`` every function here allocates and runs on that one (the caller
orders it after the producers of the inputs, and the current stream after it
before the outputs are used); the inputs are marked as in use there, the
outputs as in use on the current stream too.  Outputs carry no autograd graph,
also where inputs require gradients: the backward functions are called.
"""

import torch

from . import binding as B

_XTYPE = {torch.bfloat16: B.FP8FG_BF16, torch.float32: B.FP8FG_F32}
_CTYPE = {torch.bfloat16: B.FP8FG_BF16, torch.float32: B.FP8FG_F32}


def _on_stream(f, stream, x, inputs):
    """f() with `stream` (a torch stream or a raw handle) as the current one of
    x's device.

    On another stream than the current one the outputs and workspaces come
    from that stream's memory: a block that the current stream has freed may
    still be in use there.  The inputs are marked as in use on it, the outputs
    as in use on the current one."""
    if not hasattr(stream, "cuda_stream"):
        stream = (torch.cuda.ExternalStream(int(stream), device=x.device) if int(stream) else
                  torch.cuda.default_stream(x.device))
    if stream.device != x.device:
        raise ValueError("stream must be one of the inputs' device")
    current = torch.cuda.current_stream(x.device)
    with torch.cuda.stream(stream):
        out = f()
    for t in inputs:
        if t is not None:
            t.record_stream(stream)
    for t in (out if isinstance(out, tuple) else (out,)):
        if t is not None:
            t.record_stream(current)
    return out


def _rule(pow2):
    return B.FP8FG_SCALE_POW2 if pow2 else B.FP8FG_SCALE_AMAX


def _scales(rows, groups, layout, device):
    """Scale tensor indexed [row][group]."""
    if layout == "group_major":
        return torch.empty_strided((rows, groups), (1, rows), dtype=torch.float32, device=device)
    if layout == "row_major":
        return torch.empty((rows, groups), dtype=torch.float32, device=device)
    raise ValueError("scale_layout must be 'group_major' or 'row_major'")


def quantize_1x128(x, pow2=False, scale_layout="group_major", stream=None):
    if stream is not None and x.is_cuda:
        return _on_stream(lambda: quantize_1x128(x, pow2, scale_layout), stream, x, (x,))
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    s = _scales(M, K // 128, scale_layout, x.device)
    B.fp8_quantize_rowtile(x, _XTYPE[x.dtype], M, K, x.stride(0), None, 0, 0,
                           B.FP8FG_TILE_1x128, _rule(pow2), q, q.stride(0), s, s.stride(0),
                           s.stride(1), stream)
    return q, s


def quantize_128x1(x, pow2=False, scale_layout="group_major", stream=None):
    if stream is not None and x.is_cuda:
        return _on_stream(lambda: quantize_128x1(x, pow2, scale_layout), stream, x, (x,))
    T, F = x.shape
    qt = torch.empty((F, T), dtype=torch.uint8, device=x.device)
    st = _scales(F, T // 128, scale_layout, x.device)
    B.fp8_quantize_rowtile(x, _XTYPE[x.dtype], T, F, x.stride(0), None, 0, 0,
                           B.FP8FG_TILE_128x1, _rule(pow2), qt, qt.stride(0), st, st.stride(0),
                           st.stride(1), stream)
    return qt, st


def requantize_128x1(q, s, pow2=False, scale_layout="group_major", stream=None):
    if stream is not None and q.is_cuda:
        return _on_stream(lambda: requantize_128x1(q, s, pow2, scale_layout), stream, q, (q, s))
    T, F = q.shape
    qt = torch.empty((F, T), dtype=torch.uint8, device=q.device)
    st = _scales(F, T // 128, scale_layout, q.device)
    B.fp8_quantize_rowtile(q, B.FP8FG_E4M3, T, F, q.stride(0), s, s.stride(0), s.stride(1),
                           B.FP8FG_TILE_128x1, _rule(pow2), qt, qt.stride(0), st, st.stride(0),
                           st.stride(1), stream)
    return qt, st


def quantize_block(w, pow2=False, transpose=True, stream=None):
    if stream is not None and w.is_cuda:
        return _on_stream(lambda: quantize_block(w, pow2, transpose), stream, w, (w,))
    K, N = w.shape
    shape = (N, K) if transpose else (K, N)
    q = torch.empty(shape, dtype=torch.uint8, device=w.device)
    s = torch.empty((K // 128, N // 128), dtype=torch.float32, device=w.device)
    B.fp8_quantize_block(w, _XTYPE[w.dtype], K, N, w.stride(0), _rule(pow2), int(transpose), q,
                         q.stride(0), s, s.stride(0), s.stride(1), stream)
    return q, s


def tile_flags(tiles):
    """None (chosen from the shape), 'wide' (256-row tiles) or 'narrow'
    (64x128 tiles) -> the GEMM flag bits that fix the default path's tiles."""
    return {None: 0, "wide": B.FP8FG_GEMM_TILES_WIDE, "narrow": B.FP8FG_GEMM_TILES_NARROW}[tiles]


def gemm(qa, sa, qb, sb, out_dtype=torch.bfloat16, col_scales=False, no_promotion=False,
         fp8_mfma=False, e8m0_scales=False, out=None, stream=None, tiles=None):
    """col_scales=False: sb [K/128][N/128] block scales; True: sb [N][K/128].
    no_promotion: per-tensor scales (sa, sb hold one value each), whole-K
    FP8 matrix-core accumulation.  fp8_mfma: K-group partial sums from the
    FP8 MFMA instead of the exact default path.  e8m0_scales: the FP8 MFMA
    applies the scales' powers of two as its E8M0 operand scales.  tiles:
    see tile_flags (default path only)."""
    if stream is not None and qa.is_cuda:
        return _on_stream(lambda: gemm(qa, sa, qb, sb, out_dtype, col_scales, no_promotion, fp8_mfma, e8m0_scales, out,
                                       tiles=tiles), stream, qa, (qa, sa, qb, sb, out))
    M, K = qa.shape
    N = qb.shape[0]
    c = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=qa.device)
    mode = B.FP8FG_BSCALE_COL if col_scales else B.FP8FG_BSCALE_BLOCK128
    if no_promotion:
        # per-tensor scales broadcast with zero strides
        sa_ms, sa_ks, sb_ns, sb_ks = 0, 0, 0, 0
    else:
        sa_ms, sa_ks = sa.stride(0), sa.stride(1)
        if col_scales:
            sb_ns, sb_ks = sb.stride(0), sb.stride(1)
        else:
            sb_ns, sb_ks = sb.stride(1), sb.stride(0)
    flags = ((B.FP8FG_GEMM_NO_PROMOTION if no_promotion else 0) | (B.FP8FG_GEMM_FP8_MFMA if fp8_mfma else 0) |
             (B.FP8FG_GEMM_E8M0_SCALES if e8m0_scales else 0) | tile_flags(tiles))
    B.fp8_gemm_blockscaled(M, N, K, qa, qa.stride(0), sa, sa_ms, sa_ks, qb, qb.stride(0), sb,
                           sb_ns, sb_ks, mode, c, _CTYPE[c.dtype], c.stride(0), flags, stream)
    return c


def grouped_gemm(qa, sa, offsets, qb, sb, out_dtype=torch.bfloat16, out=None, stream=None,
                 flags=B.FP8FG_GEMM_DEFAULT, tiles=None):
    if stream is not None and qa.is_cuda:
        return _on_stream(lambda: grouped_gemm(qa, sa, offsets, qb, sb, out_dtype, out, flags=flags, tiles=tiles), stream, qa,
                          (qa, sa, offsets, qb, sb, out))
    M, K = qa.shape
    G, N, _ = qb.shape
    c = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=qa.device)
    B.fp8_grouped_gemm_blockscaled(G, offsets, M, N, K, qa, qa.stride(0), sa, sa.stride(0),
                                   sa.stride(1), qb, qb.stride(1), qb.stride(0), sb, sb.stride(2),
                                   sb.stride(1), sb.stride(0), c, _CTYPE[c.dtype], c.stride(0),
                                   flags | tile_flags(tiles), stream)
    return c


_native_module = None


def _native():
    """The native helpers (checks, allocation, call) of the functions below."""
    global _native_module
    if _native_module is None:
        try:
            from . import _native as m
        except ImportError as e:
            raise RuntimeError("the _native module is not built; run `python -m fp8_fine_grained_x1_amd.build`") from e
        m.set_error(B.Fp8fgError)
        _native_module = m
    return _native_module


def _call(name, stream, x, inputs, args):
    """The native helper `name` with `args` and a stream's handle, on `stream`
    (see _on_stream) or the current one of x's device."""
    f = getattr(_native(), name)
    d = x.get_device() if isinstance(x, torch.Tensor) else -1
    if d < 0:
        return f(*args, 0)  # refuses
    if stream is not None:
        return _on_stream(lambda: _call(name, None, x, inputs, args), stream, x, inputs)
    return f(*args, torch._C._cuda_getCurrentRawStream(d))


_LAYOUT = {"group_major": True, "row_major": False}
_SCORE = {"softmax": B.FP8FG_SCORE_SOFTMAX, "sigmoid": B.FP8FG_SCORE_SIGMOID}


def _of(table, key, name):
    if key not in table:
        raise ValueError("%s must be one of %s" % (name, sorted(table)))
    return table[key]


def rmsnorm_quantize(x, gamma, residual=None, eps=1e-6, pow2=False, scale_layout="group_major",
                     want_y=False, stream=None):
    """h = x + residual (x where there is none), y = h * rstd * gamma, and
    y in E4M3 with 1x128 scales.  Returns (q, s, h, y, rstd); y is None
    unless want_y."""
    return _call("rmsnorm_quantize", stream, x, (x, gamma, residual),
                 (x, gamma, residual, eps, _rule(pow2), _of(_LAYOUT, scale_layout, "scale_layout"), want_y))


def rmsnorm_backward(dy, h, gamma, rstd, dh=None, stream=None):
    """Gradients of rmsnorm_quantize's y (through the quantizer as it is) and,
    with dh, of its h.  Returns (dx, dgamma); dx is residual's gradient too."""
    args = (dy, h, gamma, rstd, dh)
    return _call("rmsnorm_backward", stream, h, args, args)[:2]


def route(logits, k, bias=None, score="softmax", groups=1, top_groups=1, group_top=2, renorm=True,
          scale=1.0, stream=None):
    """The k experts of each token and their weights; see fp8_route in
    include/fp8fg.h for the choice, masks and ties."""
    return _call("route", stream, logits, (logits, bias),
                 (logits, k, bias, _of(_SCORE, score, "score"), groups, top_groups, group_top, renorm, scale))


def route_backward(dw, logits, idx, score="softmax", renorm=True, scale=1.0, stream=None):
    """Gradient of route's weights with respect to the logits."""
    return _call("route_backward", stream, logits, (dw, logits, idx),
                 (dw, logits, idx, _of(_SCORE, score, "score"), renorm, scale))[0]


def dispatch(idx, experts, x, s=None, scale_layout="group_major", stream=None):
    """Rows of x (E4M3 bytes with their 1x128 scales s, or bf16 / f32) copied
    into the order of their experts.  Returns (x', s', offsets, pos, token);
    s' is None for bf16 / f32.  Entries of idx outside [0, experts) come last
    with zero rows."""
    return _call("dispatch", stream, x, (idx, x, s),
                 (idx, experts, x, s, _of(_LAYOUT, scale_layout, "scale_layout")))[:5]


def combine(z, pos, w=None, base=None, stream=None):
    """base + sum_j w[:, j] * z[pos[:, j]] (w None: ones, the gradient of
    dispatch; base None: nothing added)."""
    args = (z, pos, w, base)
    return _call("combine", stream, z, args, args)[0]


def combine_backward(dy, z, pos, w, stream=None):
    """Gradients of combine's z and w for the places of one dispatch (every
    row of z in one place)."""
    args = (dy, z, pos, w)
    return _call("combine_backward", stream, z, args, args)
