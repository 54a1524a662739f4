// C ABI of libfp8fg.so: argument validation, then kernel launch.
//
// Every check here runs on the host before any HIP call, so invalid calls
// return an error without touching a device (and can be exercised on a
// machine without a GPU).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cmath>
#include <initializer_list>

#include "fp8fg.h"
#include "launch.h"

namespace fp8fg {

namespace {
constexpr int kMaxDevices = 64;
std::atomic<int> g_cu_count[kMaxDevices];
}  // namespace

int device_cu_count() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;
  if (dev < kMaxDevices) {
    const int cached = g_cu_count[dev].load(std::memory_order_relaxed);
    if (cached > 0) return cached;
  }
  int n = 0;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
    n = 256;
  if (dev < kMaxDevices) g_cu_count[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace fp8fg

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int elem_size(int t) { return t == FP8FG_F32 ? 4 : (t == FP8FG_BF16 ? 2 : 1); }

int launched(hipError_t e) { return e == hipSuccess ? FP8FG_OK : FP8FG_ELAUNCH; }

// grids of the 128x128-block quantizers: one 256-thread workgroup per block
constexpr int64_t kMaxGridY = 65535;
constexpr int64_t kMaxGridX = 0xFFFFFFFFll / 256;

}  // namespace

namespace {

constexpr int64_t kMaxPitchA = (int64_t)1 << 23;          // bytes per row of A
constexpr int64_t kMaxPitchB = (int64_t)1 << 24;          // bytes per row of B
constexpr int64_t kMaxScaleRowStride = (int64_t)1 << 21;  // elements
constexpr int64_t kMaxScaleKSpan = (int64_t)1 << 29;      // elements

int check_gemm_common(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda,
                      const float* sa, int64_t sa_ms, int64_t sa_ks, const uint8_t* b,
                      int64_t ldb, const float* sb, int64_t sb_ns, int64_t sb_ks,
                      int b_scale_mode, void* c, int c_type, int64_t ldc, int flags) {
  if (b_scale_mode != FP8FG_BSCALE_BLOCK128 && b_scale_mode != FP8FG_BSCALE_COL) return FP8FG_EINVAL;
  if (c_type != FP8FG_BF16 && c_type != FP8FG_F32) return FP8FG_EINVAL;
  constexpr int kFp8Flags = FP8FG_GEMM_NO_PROMOTION | FP8FG_GEMM_FP8_MFMA | FP8FG_GEMM_E8M0_SCALES;
  constexpr int kTileFlags = FP8FG_GEMM_TILES_WIDE | FP8FG_GEMM_TILES_NARROW;
  if (flags & ~(kFp8Flags | kTileFlags)) return FP8FG_EINVAL;
  if ((flags & FP8FG_GEMM_E8M0_SCALES) && (flags & FP8FG_GEMM_NO_PROMOTION)) return FP8FG_EINVAL;
  // a tile choice exists only on the default path with block scales
  if ((flags & kTileFlags) == kTileFlags) return FP8FG_EINVAL;
  if ((flags & kTileFlags) && ((flags & kFp8Flags) || b_scale_mode != FP8FG_BSCALE_BLOCK128))
    return FP8FG_EINVAL;
  if (M < 0 || N < 0 || K < 0 || lda < 0 || ldb < 0 || ldc < 0) return FP8FG_EINVAL;
  if (sa_ms < 0 || sa_ks < 0 || sb_ns < 0 || sb_ks < 0) return FP8FG_EINVAL;
  if ((flags & FP8FG_GEMM_NO_PROMOTION) && (sa_ks != 0 || sb_ks != 0)) return FP8FG_EINVAL;
  if (K % 128 || N % 128) return FP8FG_ESHAPE;
  if (M == 0 || N == 0) return FP8FG_OK;
  if (!c || !sa || !sb || (K > 0 && (!a || !b))) return FP8FG_EINVAL;
  if (lda < K || ldb < K || ldc < N) return FP8FG_ESHAPE;
  if (!aligned(a, 16) || !aligned(b, 16) || lda % 16 || ldb % 16 ||
      !aligned(c, c_type == FP8FG_F32 ? 4 : 2) || !aligned(sa, 4) || !aligned(sb, 4))
    return FP8FG_EALIGN;
  // The kernels address a tile's operands and scales with 32-bit buffer
  // offsets (row pitch times tile rows, K offsets, scale strides).
  const int64_t nkb = K / 128;
  if (lda >= kMaxPitchA || ldb >= kMaxPitchB || K >= ((int64_t)1 << 31)) return FP8FG_EUNSUPPORTED;
  if (!(flags & FP8FG_GEMM_NO_PROMOTION)) {
    const int64_t kspan = kMaxScaleKSpan / (nkb > 0 ? nkb : 1);
    if (sa_ms >= kMaxScaleRowStride || sa_ks >= kspan || sb_ks >= kspan)
      return FP8FG_EUNSUPPORTED;
    if (b_scale_mode == FP8FG_BSCALE_COL && sb_ns >= kMaxScaleRowStride) return FP8FG_EUNSUPPORTED;
  }
  return FP8FG_OK;
}

bool is_xtype(int t) { return t == FP8FG_BF16 || t == FP8FG_F32; }

// A [rows][cols] operand whose rows are read and written 16 bytes at a time:
// its status (a null one passes unless it is needed).
int check_rows(const void* p, bool needed, int64_t ld, int64_t cols, int size) {
  if (!p) return needed ? FP8FG_EINVAL : FP8FG_OK;
  if (ld < cols) return FP8FG_ESHAPE;
  if (!aligned(p, 16) || (ld % 16 * size) % 16) return FP8FG_EALIGN;
  return FP8FG_OK;
}

// The first status that is not FP8FG_OK.
template <typename... S>
int first_of(S... st) {
  int rc = FP8FG_OK;
  ((rc = rc != FP8FG_OK ? rc : st), ...);
  return rc;
}

bool negative(std::initializer_list<int64_t> v) {
  for (const int64_t x : v)
    if (x < 0) return true;
  return false;
}

bool beyond(int64_t limit, std::initializer_list<int64_t> v) {
  for (const int64_t x : v)
    if (x > limit) return true;
  return false;
}

// Row pitches whose byte offsets stay in 64 bits for every int32 row.
constexpr int64_t kMaxPitch = (int64_t)1 << 29;
constexpr int64_t kMaxI32 = 0x7FFFFFFF;
// Columns whose 16-byte vectors a 32-bit index counts.
constexpr int64_t kMaxMoveCols = (int64_t)1 << 28;

int check_route(int l_type, int64_t rows, int64_t experts, int64_t ldl, int score, int64_t k,
                int renorm, float scale) {
  if (!is_xtype(l_type)) return FP8FG_EINVAL;
  if (score != FP8FG_SCORE_SOFTMAX && score != FP8FG_SCORE_SIGMOID) return FP8FG_EINVAL;
  if (renorm != 0 && renorm != 1) return FP8FG_EINVAL;
  if (negative({rows, ldl}) || experts < 1 || k < 1 || !std::isfinite(scale)) return FP8FG_EINVAL;
  if (k > experts || ldl < experts) return FP8FG_ESHAPE;
  return FP8FG_OK;
}

// Sizes of the silu gate's calls: the status of their common arguments.
int check_gate(int type, int64_t rows, int64_t inner, int scale_rule) {
  if (!is_xtype(type)) return FP8FG_EINVAL;
  if (scale_rule != FP8FG_SCALE_AMAX && scale_rule != FP8FG_SCALE_POW2) return FP8FG_EINVAL;
  if (rows < 0 || inner < 0) return FP8FG_EINVAL;
  return inner % 128 ? FP8FG_ESHAPE : FP8FG_OK;
}
bool gate_fits(int64_t rows, int64_t inner) {
  return rows <= kMaxI32 && inner <= ((int64_t)1 << 27) && rows * (inner / 128) <= (int64_t)1 << 31;
}

// The last row's code, -2 - (tokens * k - 1), has to fit an int32 too.
bool dispatch_fits(int64_t tokens, int64_t k, int64_t experts) {
  return k <= kMaxI32 && tokens <= (kMaxI32 - 2) / k && experts <= fp8fg::kRouteMaxExperts;
}

// HIP takes at most 2^32 - 1 work-items along a grid dimension.
constexpr int64_t kMaxGridItems = 0xFFFFFFFFll;

// Every launch the plan makes fits the grid limit for its workgroup size.
bool grid_fits(const fp8fg::GemmPlan& pl) {
  for (const fp8fg::GemmLaunch& l : pl.launch)
    if (l.nblocks > kMaxGridItems / pl.threads) return false;
  return true;
}

}  // namespace

extern "C" {

const char* fp8fg_status_string(int status) {
  switch (status) {
    case FP8FG_OK: return "ok";
    case FP8FG_EINVAL: return "invalid argument (null pointer, negative size or stride, bad enum)";
    case FP8FG_ESHAPE: return "bad shape (size not a required multiple, or leading dimension or workspace too small)";
    case FP8FG_EALIGN: return "misaligned pointer or row pitch (16-byte alignment required)";
    case FP8FG_EUNSUPPORTED: return "valid but unsupported combination";
    case FP8FG_ELAUNCH: return "HIP kernel launch failed";
    default: return "unknown status";
  }
}

int fp8_quantize_rowtile(const void* x, int x_type, int64_t rows, int64_t cols, int64_t ldx,
                         const float* x_scale, int64_t xs_rs, int64_t xs_ts, int tile,
                         int scale_rule, uint8_t* q, int64_t ldq, float* s, int64_t s_rs,
                         int64_t s_ts, void* stream) {
  if (x_type != FP8FG_BF16 && x_type != FP8FG_F32 && x_type != FP8FG_E4M3) return FP8FG_EINVAL;
  if (tile != FP8FG_TILE_1x128 && tile != FP8FG_TILE_128x1) return FP8FG_EINVAL;
  if (scale_rule != FP8FG_SCALE_AMAX && scale_rule != FP8FG_SCALE_POW2) return FP8FG_EINVAL;
  if (rows < 0 || cols < 0 || ldx < 0 || ldq < 0 || s_rs < 0 || s_ts < 0) return FP8FG_EINVAL;
  if (x_type == FP8FG_E4M3 && (xs_rs < 0 || xs_ts < 0)) return FP8FG_EINVAL;
  if (x_type == FP8FG_E4M3 && tile != FP8FG_TILE_128x1) return FP8FG_EUNSUPPORTED;
  if (tile == FP8FG_TILE_1x128) {
    if (cols % 128) return FP8FG_ESHAPE;
  } else {
    if (rows % 128 || cols % 128) return FP8FG_ESHAPE;
  }
  if (rows == 0 || cols == 0) return FP8FG_OK;
  if (!x || !q || !s) return FP8FG_EINVAL;
  if (x_type == FP8FG_E4M3 && !x_scale) return FP8FG_EINVAL;
  if (ldx < cols) return FP8FG_ESHAPE;
  if (ldq < (tile == FP8FG_TILE_1x128 ? cols : rows)) return FP8FG_ESHAPE;
  if (!aligned(x, 16) || (ldx * elem_size(x_type)) % 16 || !aligned(q, 16) || ldq % 16 ||
      !aligned(s, 4) || (x_scale && !aligned(x_scale, 4)))
    return FP8FG_EALIGN;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (tile == FP8FG_TILE_1x128) {
    if (rows * (cols / 128) > (int64_t)1 << 31) return FP8FG_EUNSUPPORTED;
    fp8fg::RowtileArgs a{x, x_type, rows, cols, ldx, scale_rule, q, ldq, s, s_rs, s_ts};
    return launched(fp8fg::launch_quant_1x128(a, st));
  }
  if (rows / 128 > kMaxGridY || cols / 128 > kMaxGridX) return FP8FG_EUNSUPPORTED;
  fp8fg::Tile128Args a{x,     x_type, rows, cols, ldx, x_scale, xs_rs, xs_ts, scale_rule,
                       /*per_column=*/true, /*transpose=*/true, q, ldq, s, s_rs, s_ts};
  return launched(fp8fg::launch_quant_tile128(a, st));
}

int fp8_quantize_block(const void* w, int w_type, int64_t rows, int64_t cols, int64_t ldw,
                       int scale_rule, int transpose_out, uint8_t* q, int64_t ldq, float* s,
                       int64_t s_rs, int64_t s_cs, void* stream) {
  if (w_type != FP8FG_BF16 && w_type != FP8FG_F32) return FP8FG_EINVAL;
  if (scale_rule != FP8FG_SCALE_AMAX && scale_rule != FP8FG_SCALE_POW2) return FP8FG_EINVAL;
  if (transpose_out != 0 && transpose_out != 1) return FP8FG_EINVAL;
  if (rows < 0 || cols < 0 || ldw < 0 || ldq < 0 || s_rs < 0 || s_cs < 0) return FP8FG_EINVAL;
  if (rows % 128 || cols % 128) return FP8FG_ESHAPE;
  if (rows == 0 || cols == 0) return FP8FG_OK;
  if (!w || !q || !s) return FP8FG_EINVAL;
  if (ldw < cols || ldq < (transpose_out ? rows : cols)) return FP8FG_ESHAPE;
  if (!aligned(w, 16) || (ldw * elem_size(w_type)) % 16 || !aligned(q, 16) || ldq % 16 ||
      !aligned(s, 4))
    return FP8FG_EALIGN;
  if (rows / 128 > kMaxGridY || cols / 128 > kMaxGridX) return FP8FG_EUNSUPPORTED;
  fp8fg::Tile128Args a{w,       w_type, rows, cols,       ldw,
                       nullptr, 0,      0,    scale_rule, /*per_column=*/false,
                       transpose_out != 0, q, ldq, s, s_rs, s_cs};
  return launched(fp8fg::launch_quant_tile128(a, reinterpret_cast<hipStream_t>(stream)));
}


int fp8_gemm_blockscaled(int64_t M, int64_t N, int64_t K, const uint8_t* a, int64_t lda,
                         const float* sa, int64_t sa_ms, int64_t sa_ks, const uint8_t* b,
                         int64_t ldb, const float* sb, int64_t sb_ns, int64_t sb_ks,
                         int b_scale_mode, void* c, int c_type, int64_t ldc, int flags,
                         void* stream) {
  const int rc = check_gemm_common(M, N, K, a, lda, sa, sa_ms, sa_ks, b, ldb, sb, sb_ns, sb_ks,
                                   b_scale_mode, c, c_type, ldc, flags);
  if (rc != FP8FG_OK || M == 0 || N == 0) return rc;
  fp8fg::GemmArgs g{M,  N,  K,  a,      lda,    sa, sa_ms,
                    sa_ks, b, ldb, sb, sb_ns, sb_ks, b_scale_mode,
                    c,  c_type, ldc, flags,
                    0,  nullptr, 0,  0};
  const fp8fg::GemmPlan plan = fp8fg::plan_gemm(g, fp8fg::device_cu_count());
  if (!grid_fits(plan)) return FP8FG_EUNSUPPORTED;
  return launched(fp8fg::launch_gemm(g, plan, reinterpret_cast<hipStream_t>(stream)));
}

int fp8_grouped_gemm_blockscaled(int64_t G, const int32_t* offsets, int64_t M_total, int64_t N,
                                 int64_t K, const uint8_t* a, int64_t lda, const float* sa,
                                 int64_t sa_ms, int64_t sa_ks, const uint8_t* b, int64_t ldb,
                                 int64_t b_gs, const float* sb, int64_t sb_ns, int64_t sb_ks,
                                 int64_t sb_gs, void* c, int c_type, int64_t ldc, int flags,
                                 void* stream) {
  if (G < 0 || M_total < 0 || b_gs < 0 || sb_gs < 0) return FP8FG_EINVAL;
  if (G == 0) return M_total == 0 ? FP8FG_OK : FP8FG_EINVAL;
  // the expert offsets are int32, so every row index must be one
  if (G > 0x7FFFFFFF || M_total > 0x7FFFFFFF) return FP8FG_EUNSUPPORTED;
  const int rc = check_gemm_common(M_total, N, K, a, lda, sa, sa_ms, sa_ks, b, ldb, sb, sb_ns,
                                   sb_ks, FP8FG_BSCALE_BLOCK128, c, c_type, ldc, flags);
  if (rc != FP8FG_OK || M_total == 0 || N == 0) return rc;
  if (!offsets) return FP8FG_EINVAL;
  if (!aligned(offsets, 4)) return FP8FG_EALIGN;
  if (b_gs % 16) return FP8FG_EALIGN;
  fp8fg::GemmArgs g{M_total, N,  K,  a,      lda,    sa, sa_ms,
                    sa_ks,   b,  ldb, sb, sb_ns, sb_ks, FP8FG_BSCALE_BLOCK128,
                    c,       c_type, ldc, flags,
                    G,       offsets, b_gs, sb_gs};
  const fp8fg::GemmPlan plan = fp8fg::plan_gemm(g, fp8fg::device_cu_count());
  if (!grid_fits(plan)) return FP8FG_EUNSUPPORTED;
  return launched(fp8fg::launch_gemm(g, plan, reinterpret_cast<hipStream_t>(stream)));
}

int fp8_rmsnorm_quantize(const void* x, int x_type, int64_t rows, int64_t cols, int64_t ldx,
                         const void* r, int64_t ldr, const void* gamma, int g_type, float eps,
                         int scale_rule, void* h, int64_t ldh, void* y, int64_t ldy, uint8_t* q,
                         int64_t ldq, float* s, int64_t s_rs, int64_t s_ts, float* rstd,
                         void* stream) {
  if (!is_xtype(x_type) || !is_xtype(g_type)) return FP8FG_EINVAL;
  if (scale_rule != FP8FG_SCALE_AMAX && scale_rule != FP8FG_SCALE_POW2) return FP8FG_EINVAL;
  if (negative({rows, cols, ldx, ldr, ldh, ldy, ldq, s_rs, s_ts})) return FP8FG_EINVAL;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return FP8FG_EINVAL;
  if (cols % 128) return FP8FG_ESHAPE;
  if (rows == 0 || cols == 0) return FP8FG_OK;
  if (!gamma || (q && !s)) return FP8FG_EINVAL;
  const int size = elem_size(x_type);
  const int rc = first_of(check_rows(x, true, ldx, cols, size), check_rows(r, false, ldr, cols, size),
                          check_rows(h, false, ldh, cols, size), check_rows(y, false, ldy, cols, size),
                          check_rows(q, false, ldq, cols, 1));
  if (rc != FP8FG_OK) return rc;
  if (!aligned(gamma, 16) || !aligned(s, 4) || !aligned(rstd, 4)) return FP8FG_EALIGN;
  if (cols > fp8fg::kNormMaxCols || rows > kMaxI32 || beyond(kMaxPitch, {ldx, ldr, ldh, ldy, ldq, s_rs}) ||
      s_ts > kMaxI32)
    return FP8FG_EUNSUPPORTED;
  const fp8fg::NormArgs a{x, x_type, rows, cols, ldx, r,   ldr, gamma, g_type, eps, scale_rule,
                          h, ldh,    y,    ldy,  q,   ldq, s,   s_rs,  s_ts,   rstd};
  return launched(fp8fg::launch_norm(a, reinterpret_cast<hipStream_t>(stream)));
}

int64_t fp8_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > kMaxI32 || cols < 0 || cols % 8 || cols > fp8fg::kNormMaxCols) return 0;
  return fp8fg::norm_grad_strips(rows, cols) * cols * (int64_t)sizeof(float);
}

int fp8_rmsnorm_backward(const void* dy, int x_type, int64_t rows, int64_t cols, int64_t lddy,
                         const void* dh, int64_t lddh, const void* h, int64_t ldh,
                         const void* gamma, int g_type, const float* rstd, void* dx, int64_t lddx,
                         float* dgamma, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!is_xtype(x_type) || !is_xtype(g_type)) return FP8FG_EINVAL;
  if (negative({rows, cols, lddy, lddh, ldh, lddx, workspace_bytes})) return FP8FG_EINVAL;
  if (cols % 8) return FP8FG_ESHAPE;
  if (cols == 0) return FP8FG_OK;
  if (!dgamma) return FP8FG_EINVAL;
  if (!aligned(dgamma, 4)) return FP8FG_EALIGN;
  if (rows > 0) {
    if (!gamma || !rstd || !workspace) return FP8FG_EINVAL;
    const int size = elem_size(x_type);
    const int rc = first_of(check_rows(dy, true, lddy, cols, size), check_rows(dh, false, lddh, cols, size),
                            check_rows(h, true, ldh, cols, size), check_rows(dx, true, lddx, cols, size));
    if (rc != FP8FG_OK) return rc;
    if (!aligned(gamma, 16) || !aligned(rstd, 4) || !aligned(workspace, 16)) return FP8FG_EALIGN;
  }
  if (cols > fp8fg::kNormMaxCols || rows > kMaxI32 || beyond(kMaxPitch, {lddy, lddh, ldh, lddx}))
    return FP8FG_EUNSUPPORTED;
  if (workspace_bytes < fp8_rmsnorm_backward_workspace(rows, cols)) return FP8FG_ESHAPE;
  const fp8fg::NormGradArgs a{dy,    x_type, rows, cols, lddy, dh,     lddh,  h,
                              ldh,   gamma,  g_type, rstd, dx, lddx, dgamma,
                              reinterpret_cast<float*>(workspace)};
  return launched(fp8fg::launch_norm_grad(a, reinterpret_cast<hipStream_t>(stream)));
}

int fp8_route(const void* logits, int l_type, int64_t rows, int64_t experts, int64_t ldl,
              const float* bias, int score, int64_t groups, int64_t top_groups, int group_top,
              int64_t k, int renorm, float scale, int32_t* idx, int64_t ld_idx, float* w,
              int64_t ldw, void* stream) {
  const int rc = check_route(l_type, rows, experts, ldl, score, k, renorm, scale);
  if (rc != FP8FG_OK) return rc;
  if (groups < 1 || top_groups < 1 || (group_top != 1 && group_top != 2)) return FP8FG_EINVAL;
  if (ld_idx < 0 || ldw < 0) return FP8FG_EINVAL;
  if (experts % groups || top_groups > groups || ld_idx < k || ldw < k) return FP8FG_ESHAPE;
  if (rows == 0) return FP8FG_OK;
  if (!logits || !idx || !w) return FP8FG_EINVAL;
  if (!aligned(logits, elem_size(l_type)) || !aligned(bias, 4) || !aligned(idx, 4) || !aligned(w, 4))
    return FP8FG_EALIGN;
  if (experts > fp8fg::kRouteMaxExperts || k > fp8fg::kRouteMaxK || rows > kMaxI32 ||
      beyond(kMaxPitch, {ldl, ld_idx, ldw}))
    return FP8FG_EUNSUPPORTED;
  const fp8fg::RouteArgs a{logits, l_type, rows, (int)experts, ldl, bias, score, (int)groups, (int)top_groups,
                           group_top, (int)k, renorm, scale, idx, ld_idx, w, ldw};
  return launched(fp8fg::launch_route(a, reinterpret_cast<hipStream_t>(stream)));
}

int fp8_route_backward(const void* logits, int l_type, int64_t rows, int64_t experts, int64_t ldl,
                       int score, int64_t k, int renorm, float scale, const int32_t* idx,
                       int64_t ld_idx, const float* dw, int64_t lddw, void* dlogits,
                       int64_t lddl, void* stream) {
  const int rc = check_route(l_type, rows, experts, ldl, score, k, renorm, scale);
  if (rc != FP8FG_OK) return rc;
  if (negative({ld_idx, lddw, lddl})) return FP8FG_EINVAL;
  if (ld_idx < k || lddw < k || lddl < experts) return FP8FG_ESHAPE;
  if (rows == 0) return FP8FG_OK;
  if (!logits || !idx || !dw || !dlogits) return FP8FG_EINVAL;
  const int size = elem_size(l_type);
  if (!aligned(logits, size) || !aligned(dlogits, size) || !aligned(idx, 4) || !aligned(dw, 4))
    return FP8FG_EALIGN;
  if (experts > fp8fg::kRouteMaxExperts || k > fp8fg::kRouteMaxK || rows > kMaxI32 ||
      beyond(kMaxPitch, {ldl, ld_idx, lddw, lddl}))
    return FP8FG_EUNSUPPORTED;
  const fp8fg::RouteGradArgs a{logits, l_type, rows, (int)experts, ldl, score, (int)k, renorm, scale,
                               idx, ld_idx, dw, lddw, dlogits, lddl};
  return launched(fp8fg::launch_route_grad(a, reinterpret_cast<hipStream_t>(stream)));
}

int64_t fp8_dispatch_workspace(int64_t tokens, int64_t k, int64_t experts) {
  if (tokens < 0 || k < 1 || experts < 1 || !dispatch_fits(tokens, k, experts)) return 0;
  return fp8fg::dispatch_counts(tokens * k, experts) * (int64_t)sizeof(int32_t);
}

int fp8_dispatch(const int32_t* idx, int64_t ld_idx, int64_t tokens, int64_t k, int64_t experts,
                 const void* x, int x_type, int64_t cols, int64_t ldx, const float* xs,
                 int64_t xs_rs, int64_t xs_ts, int32_t* offsets, int32_t* pos, int32_t* token,
                 void* out, int64_t ldo, float* os, int64_t os_rs, int64_t os_ts, void* workspace,
                 int64_t workspace_bytes, void* stream) {
  if (!is_xtype(x_type) && x_type != FP8FG_E4M3) return FP8FG_EINVAL;
  if (negative({ld_idx, tokens, cols, ldx, xs_rs, xs_ts, ldo, os_rs, os_ts, workspace_bytes}) || k < 1 || experts < 1)
    return FP8FG_EINVAL;
  const bool e4m3 = x_type == FP8FG_E4M3;
  if (x && cols % (e4m3 ? 128 : 8)) return FP8FG_ESHAPE;
  if (ld_idx < k) return FP8FG_ESHAPE;
  if (!offsets || !workspace) return FP8FG_EINVAL;
  if (!aligned(offsets, 4) || !aligned(workspace, 16)) return FP8FG_EALIGN;
  const bool rows = x && cols > 0 && tokens > 0;
  if (tokens > 0) {
    if (!idx || !pos || !token) return FP8FG_EINVAL;
    if (!aligned(idx, 4) || !aligned(pos, 4) || !aligned(token, 4)) return FP8FG_EALIGN;
  }
  if (rows) {
    if (e4m3 && (!xs || !os)) return FP8FG_EINVAL;
    const int size = elem_size(x_type);
    const int rc = first_of(check_rows(x, true, ldx, cols, size), check_rows(out, true, ldo, cols, size));
    if (rc != FP8FG_OK) return rc;
    if (e4m3 && (!aligned(xs, 4) || !aligned(os, 4))) return FP8FG_EALIGN;
  }
  if (!dispatch_fits(tokens, k, experts) || beyond(kMaxPitch, {ld_idx, ldx, xs_rs, ldo, os_rs}) ||
      beyond(kMaxI32, {xs_ts, os_ts}) || (x && cols > kMaxMoveCols))
    return FP8FG_EUNSUPPORTED;
  if (workspace_bytes < fp8_dispatch_workspace(tokens, k, experts)) return FP8FG_ESHAPE;
  const fp8fg::DispatchArgs a{idx, ld_idx, tokens, (int)k, (int)experts, rows ? x : nullptr, x_type, cols,
                              ldx, xs, xs_rs, xs_ts, offsets, pos, token, out, ldo, os, os_rs, os_ts,
                              reinterpret_cast<int32_t*>(workspace)};
  return launched(fp8fg::launch_dispatch(a, reinterpret_cast<hipStream_t>(stream)));
}

int fp8_combine(const void* z, int type, int64_t z_rows, int64_t tokens, int64_t k, int64_t cols,
                int64_t ldz, const int32_t* pos, const float* w, int64_t ldw, const void* base,
                int64_t ldb, void* out, int64_t ldo, void* stream) {
  if (!is_xtype(type)) return FP8FG_EINVAL;
  if (negative({z_rows, tokens, cols, ldz, ldw, ldb, ldo}) || k < 1) return FP8FG_EINVAL;
  if (cols % 8) return FP8FG_ESHAPE;
  if (tokens == 0 || cols == 0) return FP8FG_OK;
  if (!pos) return FP8FG_EINVAL;
  if (w && ldw < k) return FP8FG_ESHAPE;
  const int size = elem_size(type);
  const int rc = first_of(check_rows(z, z_rows > 0, ldz, cols, size), check_rows(base, false, ldb, cols, size),
                          check_rows(out, true, ldo, cols, size));
  if (rc != FP8FG_OK) return rc;
  if (!aligned(pos, 4) || !aligned(w, 4)) return FP8FG_EALIGN;
  if (beyond(kMaxI32, {z_rows, tokens}) || k > fp8fg::kCombineMaxK || cols > kMaxMoveCols || beyond(kMaxPitch, {ldz, ldw, ldb, ldo}))
    return FP8FG_EUNSUPPORTED;
  const fp8fg::CombineArgs a{z, type, z_rows, tokens, (int)k, cols, ldz, pos, w, ldw, base, ldb, out, ldo};
  return launched(fp8fg::launch_combine(a, reinterpret_cast<hipStream_t>(stream)));
}

int fp8_combine_backward(const void* dy, int type, int64_t z_rows, int64_t tokens, int64_t k,
                         int64_t cols, int64_t lddy, const void* z, int64_t ldz,
                         const int32_t* pos, const float* w, int64_t ldw, void* dz, int64_t lddz,
                         float* dw, int64_t lddw, void* stream) {
  if (!is_xtype(type)) return FP8FG_EINVAL;
  if (negative({z_rows, tokens, cols, lddy, ldz, ldw, lddz, lddw}) || k < 1) return FP8FG_EINVAL;
  if (cols % 8) return FP8FG_ESHAPE;
  if (tokens == 0) return FP8FG_OK;
  if (!pos) return FP8FG_EINVAL;
  if ((w && ldw < k) || (dw && lddw < k)) return FP8FG_ESHAPE;
  const int size = elem_size(type);
  const int rc = first_of(check_rows(dy, cols > 0, lddy, cols, size),
                          check_rows(z, dw && z_rows > 0 && cols > 0, ldz, cols, size),
                          check_rows(dz, z_rows > 0 && cols > 0, lddz, cols, size));
  if (rc != FP8FG_OK) return rc;
  if (!aligned(pos, 4) || !aligned(w, 4) || !aligned(dw, 4)) return FP8FG_EALIGN;
  if (beyond(kMaxI32, {z_rows, tokens}) || k > fp8fg::kCombineMaxK || cols > kMaxMoveCols ||
      beyond(kMaxPitch, {lddy, ldz, ldw, lddz, lddw}))
    return FP8FG_EUNSUPPORTED;
  const fp8fg::CombineGradArgs a{dy, type, z_rows, tokens, (int)k, cols, lddy, z, ldz, pos, w, ldw, dz, lddz, dw, lddw};
  return launched(fp8fg::launch_combine_grad(a, reinterpret_cast<hipStream_t>(stream)));
}

int fp8_swiglu_quantize(const void* u, int u_type, int64_t rows, int64_t inner, int64_t ldu,
                        const int32_t* used, int scale_rule, uint8_t* q, int64_t ldq, float* s,
                        int64_t s_rs, int64_t s_ts, uint8_t* uq, int64_t lduq, float* us,
                        int64_t us_rs, int64_t us_ts, void* stream) {
  const int sizes = check_gate(u_type, rows, inner, scale_rule);
  if (sizes != FP8FG_OK) return sizes;
  if (negative({ldu, ldq, s_rs, s_ts, lduq, us_rs, us_ts})) return FP8FG_EINVAL;
  if (rows == 0 || inner == 0) return FP8FG_OK;
  if (!s || (uq && !us)) return FP8FG_EINVAL;
  if (inner > kMaxPitch) return FP8FG_EUNSUPPORTED;
  const int rc = first_of(check_rows(u, true, ldu, 2 * inner, elem_size(u_type)), check_rows(q, true, ldq, inner, 1),
                          check_rows(uq, false, lduq, 2 * inner, 1));
  if (rc != FP8FG_OK) return rc;
  if (!aligned(s, 4) || !aligned(us, 4) || !aligned(used, 4)) return FP8FG_EALIGN;
  if (!gate_fits(rows, inner) || beyond(kMaxPitch, {ldu, ldq, s_rs, lduq, us_rs}) || beyond(kMaxI32, {s_ts, us_ts}))
    return FP8FG_EUNSUPPORTED;
  const fp8fg::GateArgs a{u, u_type, rows, inner, ldu, used, scale_rule, q, ldq, s, s_rs, s_ts, uq, lduq, us, us_rs, us_ts};
  return launched(fp8fg::launch_gate(a, reinterpret_cast<hipStream_t>(stream)));
}

int fp8_swiglu_backward(const void* da, int type, int64_t rows, int64_t inner, int64_t ldda,
                        const uint8_t* uq, int64_t lduq, const float* us, int64_t us_rs,
                        int64_t us_ts, const int32_t* used, int scale_rule, uint8_t* dq,
                        int64_t lddq, float* ds, int64_t ds_rs, int64_t ds_ts, void* du,
                        int64_t lddu, void* a, int64_t lda, void* stream) {
  const int sizes = check_gate(type, rows, inner, scale_rule);
  if (sizes != FP8FG_OK) return sizes;
  if (negative({ldda, lduq, us_rs, us_ts, lddq, ds_rs, ds_ts, lddu, lda})) return FP8FG_EINVAL;
  if (rows == 0 || inner == 0) return FP8FG_OK;
  if (!us || (dq && !ds) || (!dq && !du && !a)) return FP8FG_EINVAL;
  if (inner > kMaxPitch) return FP8FG_EUNSUPPORTED;
  const int size = elem_size(type);
  const int rc = first_of(check_rows(da, true, ldda, inner, size), check_rows(uq, true, lduq, 2 * inner, 1),
                          check_rows(dq, false, lddq, 2 * inner, 1), check_rows(du, false, lddu, 2 * inner, size),
                          check_rows(a, false, lda, inner, size));
  if (rc != FP8FG_OK) return rc;
  if (!aligned(us, 4) || !aligned(ds, 4) || !aligned(used, 4)) return FP8FG_EALIGN;
  if (!gate_fits(rows, inner) || beyond(kMaxPitch, {ldda, lduq, us_rs, lddq, ds_rs, lddu, lda}) ||
      beyond(kMaxI32, {us_ts, ds_ts}))
    return FP8FG_EUNSUPPORTED;
  const fp8fg::GateGradArgs g{da, type, rows, inner, ldda, uq, lduq, us, us_rs, us_ts, used, scale_rule,
                              dq, lddq, ds, ds_rs, ds_ts, du, lddu, a, lda};
  return launched(fp8fg::launch_gate_grad(g, reinterpret_cast<hipStream_t>(stream)));
}

int fp8_swiglu_backward_128x1(const void* da, int type, int64_t rows, int64_t inner, int64_t ldda,
                              const uint8_t* uq, int64_t lduq, const float* us, int64_t us_rs,
                              int64_t us_ts, int scale_rule, uint8_t* dq, int64_t lddq, float* ds,
                              int64_t ds_rs, int64_t ds_ts, uint8_t* dqt, int64_t lddqt, float* dst,
                              int64_t dst_rs, int64_t dst_ts, uint8_t* aqt, int64_t ldaqt, float* ast,
                              int64_t ast_rs, int64_t ast_ts, void* stream) {
  const int sizes = check_gate(type, rows, inner, scale_rule);
  if (sizes != FP8FG_OK) return sizes;
  if (negative({ldda, lduq, us_rs, us_ts, lddq, ds_rs, ds_ts, lddqt, dst_rs, dst_ts, ldaqt, ast_rs, ast_ts}))
    return FP8FG_EINVAL;
  if (rows % 128) return FP8FG_ESHAPE;
  if (rows == 0 || inner == 0) return FP8FG_OK;
  if (!us || !ds || !dst || !ast) return FP8FG_EINVAL;
  if (inner > kMaxPitch) return FP8FG_EUNSUPPORTED;
  const int rc = first_of(check_rows(da, true, ldda, inner, elem_size(type)), check_rows(uq, true, lduq, 2 * inner, 1),
                          check_rows(dq, true, lddq, 2 * inner, 1), check_rows(dqt, true, lddqt, rows, 1),
                          check_rows(aqt, true, ldaqt, rows, 1));
  if (rc != FP8FG_OK) return rc;
  if (!aligned(us, 4) || !aligned(ds, 4) || !aligned(dst, 4) || !aligned(ast, 4)) return FP8FG_EALIGN;
  if (!gate_fits(rows, inner) || rows / 128 > kMaxGridY ||
      beyond(kMaxPitch, {ldda, lduq, us_rs, lddq, ds_rs, lddqt, dst_rs, ldaqt, ast_rs}) ||
      beyond(kMaxI32, {us_ts, ds_ts, dst_ts, ast_ts}))
    return FP8FG_EUNSUPPORTED;
  const fp8fg::GateGradTileArgs g{da, type, rows, inner, ldda, uq, lduq, us, us_rs, us_ts, scale_rule, dq, lddq, ds,
                                  ds_rs, ds_ts, dqt, lddqt, dst, dst_rs, dst_ts, aqt, ldaqt, ast, ast_rs, ast_ts};
  return launched(fp8fg::launch_gate_grad_tile(g, reinterpret_cast<hipStream_t>(stream)));
}

int64_t fp8_balance_loss_workspace(int64_t rows, int64_t experts, int64_t seqs) {
  if (rows < 0 || rows > kMaxI32 || experts < 1 || experts > fp8fg::kRouteMaxExperts || seqs < 0 || seqs > kMaxI32) return 0;
  return fp8fg::balance_workspace(rows, experts, seqs);
}

int fp8_balance_loss(const void* logits, int l_type, int64_t rows, int64_t experts, int64_t ldl,
                     const int32_t* idx, int64_t ld_idx, int64_t k, const int32_t* offsets,
                     int64_t seqs, int score, float scale, float* loss, int32_t* counts,
                     float* slope, void* workspace, int64_t workspace_bytes, void* stream) {
  const int rc = check_route(l_type, rows, experts, ldl, score, k, 0, scale);
  if (rc != FP8FG_OK) return rc;
  if (negative({ld_idx, seqs, workspace_bytes}) || (!offsets && seqs != 1)) return FP8FG_EINVAL;
  if (ld_idx < k) return FP8FG_ESHAPE;
  if (seqs == 0) return FP8FG_OK;
  if (!loss || !counts || !slope || !workspace || (rows > 0 && (!logits || !idx))) return FP8FG_EINVAL;
  if (!aligned(logits, elem_size(l_type)) || !aligned(idx, 4) || !aligned(offsets, 4) || !aligned(loss, 4) ||
      !aligned(counts, 4) || !aligned(slope, 4) || !aligned(workspace, 16))
    return FP8FG_EALIGN;
  if (experts > fp8fg::kRouteMaxExperts || k > fp8fg::kRouteMaxK || beyond(kMaxI32, {rows, seqs}) || rows * k > kMaxI32 ||
      beyond(kMaxPitch, {ldl, ld_idx}))
    return FP8FG_EUNSUPPORTED;
  if (workspace_bytes < fp8_balance_loss_workspace(rows, experts, seqs)) return FP8FG_ESHAPE;
  const fp8fg::BalanceArgs a{logits, l_type, rows, (int)experts, ldl, idx, ld_idx, (int)k, offsets, seqs, score, scale,
                             loss, counts, slope, workspace};
  return launched(fp8fg::launch_balance(a, reinterpret_cast<hipStream_t>(stream)));
}

int fp8_balance_loss_backward(const float* dloss, const void* logits, int l_type, int64_t rows,
                              int64_t experts, int64_t ldl, const float* slope, const int32_t* offsets,
                              int64_t seqs, int score, const void* base, int64_t ldb, void* dlogits,
                              int64_t lddl, void* stream) {
  const int rc = check_route(l_type, rows, experts, ldl, score, 1, 0, 1.0f);
  if (rc != FP8FG_OK) return rc;
  if (negative({seqs, ldb, lddl}) || (!offsets && seqs != 1)) return FP8FG_EINVAL;
  if (lddl < experts || (base && ldb < experts)) return FP8FG_ESHAPE;
  if (rows == 0) return FP8FG_OK;
  if (!logits || !dlogits || (seqs > 0 && !slope)) return FP8FG_EINVAL;
  const int size = elem_size(l_type);
  if (!aligned(logits, size) || !aligned(base, size) || !aligned(dlogits, size) || !aligned(dloss, 4) ||
      !aligned(slope, 4) || !aligned(offsets, 4))
    return FP8FG_EALIGN;
  if (experts > fp8fg::kRouteMaxExperts || beyond(kMaxI32, {rows, seqs}) || beyond(kMaxPitch, {ldl, ldb, lddl}))
    return FP8FG_EUNSUPPORTED;
  const fp8fg::BalanceGradArgs a{dloss, logits, l_type, rows, (int)experts, ldl, slope, offsets, seqs, score,
                                 base, ldb, dlogits, lddl};
  return launched(fp8fg::launch_balance_grad(a, reinterpret_cast<hipStream_t>(stream)));
}

int fp8_rmsnorm_block_quantize(const void* z, int x_type, int64_t rows, int64_t cols, int64_t ldz,
                               const void* r, int64_t ldr, const void* gamma_post, const void* gamma,
                               int g_type, const void* gate, int64_t ldg, float residual_scale,
                               float block_scale, float eps, int scale_rule, void* h, int64_t ldh,
                               void* y, int64_t ldy, uint8_t* q, int64_t ldq, float* s, int64_t s_rs,
                               int64_t s_ts, float* rstd_post, float* rstd, void* stream) {
  if (!is_xtype(x_type) || !is_xtype(g_type)) return FP8FG_EINVAL;
  if (scale_rule != FP8FG_SCALE_AMAX && scale_rule != FP8FG_SCALE_POW2) return FP8FG_EINVAL;
  if (negative({rows, cols, ldz, ldr, ldg, ldh, ldy, ldq, s_rs, s_ts})) return FP8FG_EINVAL;
  if (!(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(residual_scale) || !std::isfinite(block_scale))
    return FP8FG_EINVAL;
  if (cols % 128) return FP8FG_ESHAPE;
  if (rows == 0 || cols == 0) return FP8FG_OK;
  if (!gamma_post || !gamma || (q && !s)) return FP8FG_EINVAL;
  const int size = elem_size(x_type);
  const bool row_gate = gate && ldg > 0;
  const int rc = first_of(check_rows(z, true, ldz, cols, size), check_rows(r, true, ldr, cols, size),
                          check_rows(row_gate ? gate : nullptr, false, ldg, cols, size),
                          check_rows(h, true, ldh, cols, size), check_rows(y, false, ldy, cols, size),
                          check_rows(q, false, ldq, cols, 1));
  if (rc != FP8FG_OK) return rc;
  if (!aligned(gamma_post, 16) || !aligned(gamma, 16) || !aligned(gate, 16) || !aligned(s, 4) || !aligned(rstd_post, 4) ||
      !aligned(rstd, 4))
    return FP8FG_EALIGN;
  if (cols > fp8fg::kBlockNormMaxCols || rows > kMaxI32 || beyond(kMaxPitch, {ldz, ldr, ldg, ldh, ldy, ldq, s_rs}) ||
      s_ts > kMaxI32)
    return FP8FG_EUNSUPPORTED;
  const fp8fg::BlockNormArgs a{z, x_type, rows, cols, ldz, r, ldr, gamma_post, gamma, g_type, gate, ldg,
                               residual_scale, block_scale, eps, scale_rule, h, ldh, y, ldy, q, ldq, s, s_rs, s_ts,
                               rstd_post, rstd};
  return launched(fp8fg::launch_block_norm(a, reinterpret_cast<hipStream_t>(stream)));
}

int64_t fp8_rmsnorm_block_backward_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > kMaxI32 || cols < 0 || cols % 8 || cols > fp8fg::kBlockNormMaxCols) return 0;
  return 2 * fp8fg::block_norm_strips(rows, cols) * cols * (int64_t)sizeof(float);
}

int fp8_rmsnorm_block_backward(const void* dy, int x_type, int64_t rows, int64_t cols, int64_t lddy,
                               const void* dh, int64_t lddh, const void* z, int64_t ldz, const void* h,
                               int64_t ldh, const void* gamma_post, const void* gamma, int g_type,
                               const void* gate, int64_t ldg, const float* rstd_post, const float* rstd,
                               float residual_scale, float block_scale, void* dz, int64_t lddz, void* dr,
                               int64_t lddr, float* dgamma_post, float* dgamma, void* dgate, int64_t lddg,
                               void* workspace, int64_t workspace_bytes, void* stream) {
  if (!is_xtype(x_type) || !is_xtype(g_type)) return FP8FG_EINVAL;
  if (negative({rows, cols, lddy, lddh, ldz, ldh, ldg, lddz, lddr, lddg, workspace_bytes})) return FP8FG_EINVAL;
  if (!std::isfinite(residual_scale) || !std::isfinite(block_scale)) return FP8FG_EINVAL;
  if (cols % 8) return FP8FG_ESHAPE;
  if (cols == 0) return FP8FG_OK;
  const bool col_gate = gate && ldg == 0, row_gate = gate && ldg > 0;
  if (!dgamma_post || !dgamma || (col_gate && !dgate) || (row_gate && rows > 0 && !dgate)) return FP8FG_EINVAL;
  if (!aligned(dgamma_post, 4) || !aligned(dgamma, 4) || (col_gate && !aligned(dgate, 4))) return FP8FG_EALIGN;
  if (rows > 0) {
    if (!rstd_post || !rstd || !workspace) return FP8FG_EINVAL;
    const int size = elem_size(x_type);
    const int rc = first_of(check_rows(dy, true, lddy, cols, size), check_rows(dh, false, lddh, cols, size),
                            check_rows(z, true, ldz, cols, size), check_rows(h, true, ldh, cols, size),
                            check_rows(row_gate ? gate : nullptr, false, ldg, cols, size),
                            check_rows(dz, true, lddz, cols, size), check_rows(dr, true, lddr, cols, size),
                            check_rows(row_gate ? dgate : nullptr, false, lddg, cols, size));
    if (rc != FP8FG_OK) return rc;
    if (!aligned(rstd_post, 4) || !aligned(rstd, 4) || !aligned(workspace, 16)) return FP8FG_EALIGN;
  }
  // (read also for rows == 0 where a column gate's gradient is formed)
  if ((rows > 0 || col_gate) && (!gamma_post || !gamma)) return FP8FG_EINVAL;
  if (!aligned(gamma_post, 16) || !aligned(gamma, 16) || !aligned(gate, 16)) return FP8FG_EALIGN;
  if (cols > fp8fg::kBlockNormMaxCols || rows > kMaxI32 ||
      beyond(kMaxPitch, {lddy, lddh, ldz, ldh, ldg, lddz, lddr, lddg}))
    return FP8FG_EUNSUPPORTED;
  if (workspace_bytes < fp8_rmsnorm_block_backward_workspace(rows, cols)) return FP8FG_ESHAPE;
  const fp8fg::BlockNormGradArgs a{dy, x_type, rows, cols, lddy, dh, lddh, z, ldz, h, ldh, gamma_post, gamma, g_type,
                                   gate, ldg, rstd_post, rstd, residual_scale, block_scale, dz, lddz, dr, lddr,
                                   dgamma_post, dgamma, dgate, lddg, reinterpret_cast<float*>(workspace)};
  return launched(fp8fg::launch_block_norm_grad(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
