// Internal interface between the C ABI (abi.cpp) and the kernel files.
// Arguments reaching these launchers have already been validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8fg {

// Compute units of the current device (cached per device).
int device_cu_count();

struct RowtileArgs {
  const void* x;
  int x_type;          // 0 bf16, 1 f32
  int64_t rows, cols, ldx;
  int rule;            // 0 amax, 1 pow2
  uint8_t* q;
  int64_t ldq;
  float* s;
  int64_t s_rs, s_ts;
};
hipError_t launch_quant_1x128(const RowtileArgs& a, hipStream_t st);

// 128 x 128 work blocks: the 128x1 (per-column) and the 128x128 (per-block)
// quantizers, with or without a transposed byte layout.
struct Tile128Args {
  const void* x;
  int x_type;          // 0 bf16, 1 f32, 2 e4m3 (requantization)
  int64_t rows, cols, ldx;
  const float* xs;     // input 1x128 scales (e4m3 input only)
  int64_t xs_rs, xs_ts;
  int rule;
  bool per_column;     // true: 128x1 tiles; false: 128x128 blocks
  bool transpose;      // write q[c * ldq + r]
  uint8_t* q;
  int64_t ldq;
  float* s;
  int64_t s_a, s_b;    // per_column: s[c * s_a + (r/128) * s_b]; block: s[(r/128) * s_a + (c/128) * s_b]
};
hipError_t launch_quant_tile128(const Tile128Args& a, hipStream_t st);

struct GemmArgs {
  int64_t M, N, K;
  const uint8_t* a;
  int64_t lda;
  const float* sa;
  int64_t sa_ms, sa_ks;
  const uint8_t* b;
  int64_t ldb;
  const float* sb;
  int64_t sb_ns, sb_ks;
  int b_scale_mode;    // 0 block128, 1 per column
  void* c;
  int c_type;          // 0 bf16, 1 f32
  int64_t ldc;
  int flags;           // FP8FG_GEMM_* bit set
  // grouped
  int64_t G;           // 0 = dense
  const int32_t* offsets;
  int64_t b_gs, sb_gs;
};
// Which GEMM kernel runs, and its launches (at most two: the default path's
// 256- and 192-column tiles).  Computed on the host from the arguments alone
// (and the CU count), before anything is enqueued, so that the caller can
// check the grid sizes of exactly the launches that will be made.
enum class GemmKernel { kNone, kMx, kStream, kRescale, kBlockscaled };
struct GemmLaunch {
  int64_t tiles_n;   // column tiles of this launch
  int64_t n_base;    // first output column of this launch's tiles
  int64_t nblocks;   // workgroups (0: no launch)
};
struct GemmPlan {
  GemmKernel kernel;
  int mode;          // arithmetic of gemm_blockscaled_kernel (exact / FP8 flags)
  int threads;       // per workgroup
  GemmLaunch launch[2];
};
GemmPlan plan_gemm(const GemmArgs& g, int cus);
hipError_t launch_gemm(const GemmArgs& g, const GemmPlan& plan, hipStream_t st);
// Split of N into column tiles of 256 and 192 for the default GEMM path
// (both zero: the path does not apply).  cus = 0 asks for 256-column tiles
// only (grouped GEMM).
struct ColumnPlan {
  int64_t n256, n192;
};
ColumnPlan plan_columns(int64_t tiles_m, int64_t N, int cus);

// Inputs of more bytes than this are read past the caches: less of them is
// likely to lie in the 256 MB Infinity Cache, where their producer left them.
constexpr int64_t kStreamBytes = (int64_t)128 << 20;

// Whether `rows * per * cols` elements of `size` bytes are more than that.
// The combine's product passes 64 bits at sizes that it takes (rows read
// again and again): compared in fp64.
inline bool past_caches(int64_t rows, int64_t per, int64_t cols, int size) {
  return (double)rows * (double)per * (double)cols * size > (double)kStreamBytes;
}

// ------------------------------------------------- norm (norm.hip)
struct NormArgs {
  const void* x;
  int x_type;          // 0 bf16, 1 f32 (also r, h, y)
  int64_t rows, cols, ldx;
  const void* r;       // added to x; null: none
  int64_t ldr;
  const void* gamma;
  int g_type;          // 0 bf16, 1 f32
  float eps;
  int rule;            // 0 amax, 1 pow2
  void* h;             // x + r; null: not stored
  int64_t ldh;
  void* y;             // the norm itself; null: not stored
  int64_t ldy;
  uint8_t* q;          // null: no quantized output
  int64_t ldq;
  float* s;
  int64_t s_rs, s_ts;
  float* rstd;         // null: not stored
};
hipError_t launch_norm(const NormArgs& a, hipStream_t st);

struct NormGradArgs {
  const void* dy;
  int x_type;          // of dy, dh, h, dx
  int64_t rows, cols, lddy;
  const void* dh;      // added to dx; null: none
  int64_t lddh;
  const void* h;
  int64_t ldh;
  const void* gamma;
  int g_type;
  const float* rstd;
  void* dx;
  int64_t lddx;
  float* dgamma;
  float* partial;      // [norm_grad_strips(rows, cols)][cols]
};
// Row strips of the gradient kernel, each with its own partial sum of
// dgamma; a function of the sizes alone.
int64_t norm_grad_strips(int64_t rows, int64_t cols);
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t st);
// Widest row a workgroup holds in registers.
constexpr int64_t kNormMaxCols = 32768;

// ------------------------------------------------- router (route.hip)
struct RouteArgs {
  const void* logits;
  int l_type;          // 0 bf16, 1 f32
  int64_t rows;
  int experts;
  int64_t ldl;
  const float* bias;   // null: none
  int score;           // 0 softmax, 1 sigmoid
  int groups, top_groups, group_top;
  int k;
  int renorm;
  float scale;
  int32_t* idx;
  int64_t ld_idx;
  float* w;
  int64_t ldw;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t st);

struct RouteGradArgs {
  const void* logits;
  int l_type;          // of logits and dlogits
  int64_t rows;
  int experts;
  int64_t ldl;
  int score;
  int k;
  int renorm;
  float scale;
  const int32_t* idx;
  int64_t ld_idx;
  const float* dw;
  int64_t lddw;
  void* dl;
  int64_t lddl;
};
hipError_t launch_route_grad(const RouteGradArgs& a, hipStream_t st);
constexpr int64_t kRouteMaxExperts = 1024;
constexpr int64_t kRouteMaxK = 64;

// ------------------------------------------------- dispatch and combine (dispatch.hip)
struct DispatchArgs {
  const int32_t* idx;
  int64_t ld_idx, tokens;
  int k, experts;
  const void* x;       // null: places only
  int x_type;          // 0 bf16, 1 f32, 2 e4m3
  int64_t cols, ldx;
  const float* xs;     // 1x128 scales of e4m3 rows
  int64_t xs_rs, xs_ts;
  int32_t* offsets;
  int32_t* pos;        // [tokens][k]
  int32_t* token;      // [tokens * k]
  void* out;
  int64_t ldo;
  float* os;
  int64_t os_rs, os_ts;
  int32_t* counts;     // dispatch_counts(tokens * k, experts) of them
};
// Counts of entries per expert and chunk of the (token, choice) list.
int64_t dispatch_counts(int64_t entries, int64_t experts);
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t st);

struct CombineArgs {
  const void* z;
  int type;            // 0 bf16, 1 f32: z, base, out
  int64_t z_rows, tokens;
  int k;
  int64_t cols, ldz;
  const int32_t* pos;  // [tokens][k]
  const float* w;      // null: ones
  int64_t ldw;
  const void* base;    // null: none
  int64_t ldb;
  void* out;
  int64_t ldo;
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t st);
// The kernels step through the places in int32, 8 at a time, and past the
// last ones.
constexpr int64_t kCombineMaxK = 0x7FFFFFFF - 15;

struct CombineGradArgs {
  const void* dy;
  int type;            // dy, z, dz
  int64_t z_rows, tokens;
  int k;
  int64_t cols, lddy;
  const void* z;       // null with dw: not needed
  int64_t ldz;
  const int32_t* pos;
  const float* w;      // null: ones
  int64_t ldw;
  void* dz;
  int64_t lddz;
  float* dw;           // null: not wanted
  int64_t lddw;
};
hipError_t launch_combine_grad(const CombineGradArgs& a, hipStream_t st);

// ------------------------------------------------- silu gate (gate.hip)
struct GateArgs {
  const void* u;
  int u_type;          // 0 bf16, 1 f32
  int64_t rows, inner, ldu;
  const int32_t* used; // rows in use; null: all
  int rule;            // 0 amax, 1 pow2
  uint8_t* q;
  int64_t ldq;
  float* s;
  int64_t s_rs, s_ts;
  uint8_t* uq;         // checkpoint of u; null: not kept
  int64_t lduq;
  float* us;
  int64_t us_rs, us_ts;
};
hipError_t launch_gate(const GateArgs& a, hipStream_t st);

struct GateGradArgs {
  const void* da;
  int type;            // 0 bf16, 1 f32 (da, du, a)
  int64_t rows, inner, ldda;
  const uint8_t* uq;
  int64_t lduq;
  const float* us;
  int64_t us_rs, us_ts;
  const int32_t* used; // null: all
  int rule;
  uint8_t* q;          // of [dg | dl]; null: not wanted
  int64_t ldq;
  float* s;
  int64_t s_rs, s_ts;
  void* du;            // null: not wanted
  int64_t lddu;
  void* a;             // null: not wanted
  int64_t lda;
};
hipError_t launch_gate_grad(const GateGradArgs& a, hipStream_t st);

struct GateGradTileArgs {
  const void* da;
  int type;
  int64_t rows, inner, ldda;
  const uint8_t* uq;
  int64_t lduq;
  const float* us;
  int64_t us_rs, us_ts;
  int rule;
  uint8_t* q;          // 1x128 tiles of [dg | dl]
  int64_t ldq;
  float* s;
  int64_t s_rs, s_ts;
  uint8_t* qt;         // 128x1 tiles of it, transposed
  int64_t ldqt;
  float* st;
  int64_t st_rs, st_ts;
  uint8_t* aq;         // 128x1 tiles of a, transposed
  int64_t ldaq;
  float* as;
  int64_t as_rs, as_ts;
};
hipError_t launch_gate_grad_tile(const GateGradTileArgs& a, hipStream_t st);

// ------------------------------------------------- balance loss (balance.hip)
struct BalanceArgs {
  const void* logits;
  int l_type;          // 0 bf16, 1 f32
  int64_t rows;
  int experts;
  int64_t ldl;
  const int32_t* idx;
  int64_t ld_idx;
  int k;
  const int32_t* offsets;  // [seqs + 1]; null: one sequence of all rows
  int64_t seqs;
  int score;           // 0 softmax, 1 sigmoid
  float scale;
  float* loss;         // [seqs]
  int32_t* counts;     // [seqs][experts]
  float* slope;        // [seqs][experts]
  void* workspace;     // balance_workspace(...) bytes
};
// Bytes of partial sums; a function of the sizes alone.
int64_t balance_workspace(int64_t rows, int64_t experts, int64_t seqs);
hipError_t launch_balance(const BalanceArgs& a, hipStream_t st);

struct BalanceGradArgs {
  const float* dloss;  // [seqs]; null: ones
  const void* logits;
  int l_type;          // of logits, base and dl
  int64_t rows;
  int experts;
  int64_t ldl;
  const float* slope;
  const int32_t* offsets;
  int64_t seqs;
  int score;
  const void* base;    // added; null: none
  int64_t ldb;
  void* dl;
  int64_t lddl;
};
hipError_t launch_balance_grad(const BalanceGradArgs& a, hipStream_t st);

// ------------------------------------------------- norms after and before a block (block_norm.hip)
struct BlockNormArgs {
  const void* z;
  int x_type;          // 0 bf16, 1 f32: z, r, h, y and a gate of rows
  int64_t rows, cols, ldz;
  const void* r;
  int64_t ldr;
  const void* gamma_post;
  const void* gamma;
  int g_type;          // 0 bf16, 1 f32: the gammas and a gate of columns
  const void* gate;    // null: none
  int64_t ldg;         // 0: one per column; otherwise the pitch of a gate of rows
  float residual_scale, block_scale, eps;
  int rule;
  void* h;
  int64_t ldh;
  void* y;             // null: not stored
  int64_t ldy;
  uint8_t* q;          // null: no quantized output
  int64_t ldq;
  float* s;
  int64_t s_rs, s_ts;
  float* rstd_post;    // null: not stored
  float* rstd;         // null: not stored
};
hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t st);

struct BlockNormGradArgs {
  const void* dy;
  int x_type;          // dy, dh, z, h, dz, dr, and gate and dgate of rows
  int64_t rows, cols, lddy;
  const void* dh;      // null: none
  int64_t lddh;
  const void* z;
  int64_t ldz;
  const void* h;
  int64_t ldh;
  const void* gamma_post;
  const void* gamma;
  int g_type;
  const void* gate;
  int64_t ldg;
  const float* rstd_post;
  const float* rstd;
  float residual_scale, block_scale;
  void* dz;
  int64_t lddz;
  void* dr;
  int64_t lddr;
  float* dgamma_post;
  float* dgamma;
  void* dgate;         // f32 [cols], or rows of x_type; null without a gate
  int64_t lddg;
  float* partial;      // [2][block_norm_strips(rows, cols)][cols]
};
int64_t block_norm_strips(int64_t rows, int64_t cols);
hipError_t launch_block_norm_grad(const BlockNormGradArgs& a, hipStream_t st);
// Widest row a workgroup of 1024 threads holds, 16 elements to each.
constexpr int64_t kBlockNormMaxCols = 16384;

}  // namespace fp8fg
