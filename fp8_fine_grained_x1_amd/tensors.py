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
cannot see and raise ValueError.  They allocate on the current stream; with
``stream`` they run on that one (the caller orders it after the producers of
the inputs) and mark what they allocated as in use there.
"""

import torch

from . import binding as B

_XTYPE = {torch.bfloat16: B.FP8FG_BF16, torch.float32: B.FP8FG_F32}
_CTYPE = {torch.bfloat16: B.FP8FG_BF16, torch.float32: B.FP8FG_F32}


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
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    s = _scales(M, K // 128, scale_layout, x.device)
    B.fp8_quantize_rowtile(x, _XTYPE[x.dtype], M, K, x.stride(0), None, 0, 0,
                           B.FP8FG_TILE_1x128, _rule(pow2), q, q.stride(0), s, s.stride(0),
                           s.stride(1), stream)
    return q, s


def quantize_128x1(x, pow2=False, scale_layout="group_major", stream=None):
    T, F = x.shape
    qt = torch.empty((F, T), dtype=torch.uint8, device=x.device)
    st = _scales(F, T // 128, scale_layout, x.device)
    B.fp8_quantize_rowtile(x, _XTYPE[x.dtype], T, F, x.stride(0), None, 0, 0,
                           B.FP8FG_TILE_128x1, _rule(pow2), qt, qt.stride(0), st, st.stride(0),
                           st.stride(1), stream)
    return qt, st


def requantize_128x1(q, s, pow2=False, scale_layout="group_major", stream=None):
    T, F = q.shape
    qt = torch.empty((F, T), dtype=torch.uint8, device=q.device)
    st = _scales(F, T // 128, scale_layout, q.device)
    B.fp8_quantize_rowtile(q, B.FP8FG_E4M3, T, F, q.stride(0), s, s.stride(0), s.stride(1),
                           B.FP8FG_TILE_128x1, _rule(pow2), qt, qt.stride(0), st, st.stride(0),
                           st.stride(1), stream)
    return qt, st


def quantize_block(w, pow2=False, transpose=True, stream=None):
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
    M, K = qa.shape
    G, N, _ = qb.shape
    c = out if out is not None else torch.empty((M, N), dtype=out_dtype, device=qa.device)
    B.fp8_grouped_gemm_blockscaled(G, offsets, M, N, K, qa, qa.stride(0), sa, sa.stride(0),
                                   sa.stride(1), qb, qb.stride(1), qb.stride(0), sb, sb.stride(2),
                                   sb.stride(1), sb.stride(0), c, _CTYPE[c.dtype], c.stride(0),
                                   flags | tile_flags(tiles), stream)
    return c


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _alloc(rows, cols, dtype, device):
    # empty_strided is the cheapest of torch's allocating calls
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _alloc1(n, dtype, device):
    return torch.empty_strided((n,), (1,), dtype=dtype, device=device)


def _rows2d(name, x, like=None, dtypes=None):
    """x is a 2-d GPU tensor with contiguous rows, where `like` is given of
    its shape, type and device."""
    _need(x.is_cuda, "%s must be on the GPU" % name)
    _need(x.dim() == 2 and (x.stride(1) == 1 or x.shape[1] <= 1), "%s must be 2-d with contiguous rows" % name)
    if dtypes is not None:
        _need(x.dtype in dtypes, "%s has type %s" % (name, x.dtype))
    if like is not None:
        _need(x.shape == like.shape and x.dtype == like.dtype and x.device == like.device,
              "%s does not match in shape, type or device" % name)


def _pitch(x):
    """Row pitch of a 2-d tensor; a single row's stride carries no meaning."""
    return x.stride(0) if x.shape[0] > 1 else max(x.shape[1], 1)


def _on_stream(stream, *tensors):
    """Tells torch's allocator that tensors of the current stream are in use
    on `stream` (a torch stream or a raw handle)."""
    if stream is None:
        return
    for t in tensors:
        if t is not None and t.is_cuda:
            st = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=t.device)
            t.record_stream(st)


def rmsnorm_quantize(x, gamma, residual=None, eps=1e-6, pow2=False, scale_layout="group_major",
                     want_y=False, stream=None):
    """h = x + residual (x where there is none), y = h * rstd * gamma, and
    y in E4M3 with 1x128 scales.  Returns (q, s, h, y, rstd); y is None
    unless want_y."""
    _rows2d("x", x, dtypes=_XTYPE)
    M, C = x.shape
    _need(gamma.dim() == 1 and gamma.shape[0] == C and gamma.is_contiguous() and gamma.dtype in _XTYPE and
          gamma.device == x.device, "gamma must be a contiguous vector of the columns")
    if residual is not None:
        _rows2d("residual", residual, like=x)
    dev = x.device
    q = _alloc(M, C, torch.uint8, dev)
    s = _scales(M, C // 128, scale_layout, dev)
    h = x if residual is None else _alloc(M, C, x.dtype, dev)
    y = _alloc(M, C, x.dtype, dev) if want_y else None
    rstd = _alloc1(M, torch.float32, dev)
    B.fp8_rmsnorm_quantize(x, _XTYPE[x.dtype], M, C, _pitch(x), residual,
                           0 if residual is None else _pitch(residual), gamma, _XTYPE[gamma.dtype],
                           eps, _rule(pow2), None if residual is None else h, C, y, C, q, C, s,
                           s.stride(0), s.stride(1), rstd, stream)
    _on_stream(stream, q, s, h, y, rstd)
    return q, s, h, y, rstd


def rmsnorm_backward(dy, h, gamma, rstd, dh=None, stream=None):
    """Gradients of rmsnorm_quantize's y (through the quantizer as it is) and,
    with dh, of its h.  Returns (dx, dgamma); dx is residual's gradient too."""
    _rows2d("h", h, dtypes=_XTYPE)
    _rows2d("dy", dy, like=h)
    if dh is not None:
        _rows2d("dh", dh, like=h)
    M, C = h.shape
    _need(gamma.dim() == 1 and gamma.shape[0] == C and gamma.is_contiguous() and gamma.dtype in _XTYPE and
          gamma.device == h.device, "gamma must be a contiguous vector of the columns")
    _need(rstd.shape == (M,) and rstd.dtype == torch.float32 and rstd.is_contiguous() and rstd.device == h.device,
          "rstd must be a contiguous f32 vector of the rows")
    dx = _alloc(M, C, h.dtype, h.device)
    dgamma = _alloc1(C, torch.float32, h.device)
    n = B.fp8_rmsnorm_backward_workspace(M, C)
    ws = _alloc1(max(n, 16), torch.uint8, h.device)
    B.fp8_rmsnorm_backward(dy, _XTYPE[h.dtype], M, C, _pitch(dy), dh, 0 if dh is None else _pitch(dh), h,
                           _pitch(h), gamma, _XTYPE[gamma.dtype], rstd, dx, C, dgamma, ws, n, stream)
    _on_stream(stream, dx, dgamma, ws)
    return dx, dgamma


_SCORE = {"softmax": B.FP8FG_SCORE_SOFTMAX, "sigmoid": B.FP8FG_SCORE_SIGMOID}


def route(logits, k, bias=None, score="softmax", groups=1, top_groups=1, group_top=2, renorm=True,
          scale=1.0, stream=None):
    """The k experts of each token and their weights; see fp8_route in
    include/fp8fg.h for the choice, masks and ties."""
    _rows2d("logits", logits, dtypes=_XTYPE)
    _need(score in _SCORE, "score must be 'softmax' or 'sigmoid'")
    M, E = logits.shape
    if bias is not None:
        _need(bias.shape == (E,) and bias.dtype == torch.float32 and bias.is_contiguous() and
              bias.device == logits.device, "bias must be a contiguous f32 vector of the experts")
    idx = _alloc(M, k, torch.int32, logits.device)
    w = _alloc(M, k, torch.float32, logits.device)
    B.fp8_route(logits, _XTYPE[logits.dtype], M, E, _pitch(logits), bias, _SCORE[score], groups,
                top_groups, group_top, k, int(renorm), scale, idx, k, w, k, stream)
    _on_stream(stream, idx, w)
    return idx, w


def route_backward(dw, logits, idx, score="softmax", renorm=True, scale=1.0, stream=None):
    """Gradient of route's weights with respect to the logits."""
    _rows2d("logits", logits, dtypes=_XTYPE)
    _need(score in _SCORE, "score must be 'softmax' or 'sigmoid'")
    M, E = logits.shape
    _rows2d("idx", idx, dtypes=(torch.int32,))
    _rows2d("dw", dw, dtypes=(torch.float32,))
    k = idx.shape[1]
    _need(idx.shape == (M, k) and dw.shape == (M, k) and idx.device == logits.device and dw.device == logits.device,
          "idx and dw must be [tokens][k] on the logits' device")
    dl = _alloc(M, E, logits.dtype, logits.device)
    B.fp8_route_backward(logits, _XTYPE[logits.dtype], M, E, _pitch(logits), _SCORE[score], k, int(renorm),
                         scale, idx, _pitch(idx), dw, _pitch(dw), dl, E, stream)
    _on_stream(stream, dl)
    return dl


_MOVE = {torch.uint8: B.FP8FG_E4M3, torch.bfloat16: B.FP8FG_BF16, torch.float32: B.FP8FG_F32}


def dispatch(idx, experts, x, s=None, scale_layout="group_major", stream=None):
    """Rows of x (E4M3 bytes with their 1x128 scales s, or bf16 / f32) copied
    into the order of their experts.  Returns (x', s', offsets, pos, token);
    s' is None for bf16 / f32.  Entries of idx outside [0, experts) come last
    with zero rows."""
    _rows2d("idx", idx, dtypes=(torch.int32,))
    _rows2d("x", x, dtypes=_MOVE)
    M, k = idx.shape
    C = x.shape[1]
    dev = x.device
    _need(x.shape[0] == M and idx.device == dev, "idx must be [tokens][k] on x's device")
    e4m3 = x.dtype == torch.uint8
    _need((s is not None) == e4m3, "E4M3 rows need their scales, others have none")
    out_s = None
    if e4m3:
        _need(s.shape == (M, C // 128) and s.dtype == torch.float32 and s.device == dev,
              "s must be the f32 [tokens][columns / 128] scales of x")
        out_s = _scales(M * k, C // 128, scale_layout, dev)
    out = _alloc(M * k, C, x.dtype, dev)
    offsets = _alloc1(experts + 1, torch.int32, dev)
    pos = _alloc(M, k, torch.int32, dev)
    token = _alloc1(M * k, torch.int32, dev)
    n = B.fp8_dispatch_workspace(M, k, experts)
    ws = _alloc1(max(n, 16), torch.uint8, dev)
    st = (s.stride(0), s.stride(1), out_s.stride(0), out_s.stride(1)) if e4m3 else (0, 0, 0, 0)
    B.fp8_dispatch(idx, _pitch(idx), M, k, experts, x, _MOVE[x.dtype], C, _pitch(x), s, st[0], st[1],
                   offsets, pos, token, out, C, out_s, st[2], st[3], ws, n, stream)
    _on_stream(stream, out, out_s, offsets, pos, token, ws)
    return out, out_s, offsets, pos, token


def _check_places(pos, w, like):
    _need(pos.dim() == 2 and pos.dtype == torch.int32 and pos.is_contiguous() and pos.device == like.device,
          "pos must be contiguous int32 [tokens][k] on the rows' device")
    if w is not None:
        _rows2d("w", w, dtypes=(torch.float32,))
        _need(w.shape == pos.shape and w.device == like.device, "w must be f32 [tokens][k] on the rows' device")


def combine(z, pos, w=None, base=None, stream=None):
    """base + sum_j w[:, j] * z[pos[:, j]] (w None: ones, the gradient of
    dispatch; base None: nothing added)."""
    _rows2d("z", z, dtypes=_XTYPE)
    _check_places(pos, w, z)
    M, k = pos.shape
    R, C = z.shape
    out = _alloc(M, C, z.dtype, z.device)
    if base is not None:
        _rows2d("base", base, like=out)
    B.fp8_combine(z, _XTYPE[z.dtype], R, M, k, C, _pitch(z), pos, w, 0 if w is None else _pitch(w),
                  base, 0 if base is None else _pitch(base), out, C, stream)
    _on_stream(stream, out)
    return out


def combine_backward(dy, z, pos, w, stream=None):
    """Gradients of combine's z and w for the places of one dispatch (every
    row of z in one place)."""
    _rows2d("z", z, dtypes=_XTYPE)
    _rows2d("dy", dy, dtypes=_XTYPE)
    _check_places(pos, w, z)
    M, k = pos.shape
    R, C = z.shape
    _need(dy.shape == (M, C) and dy.dtype == z.dtype and dy.device == z.device,
          "dy must be [tokens][columns] of z's type and device")
    _need(R == M * k, "z must have tokens * k rows")
    dz = _alloc(R, C, z.dtype, z.device)
    dw = _alloc(M, k, torch.float32, z.device)
    B.fp8_combine_backward(dy, _XTYPE[z.dtype], R, M, k, C, _pitch(dy), z, _pitch(z), pos, w,
                           0 if w is None else _pitch(w), dz, C, dw, k, stream)
    _on_stream(stream, dz, dw)
    return dz, dw
