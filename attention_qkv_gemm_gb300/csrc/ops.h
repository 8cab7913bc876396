// ops.h -- argument blocks and host launchers of the operators that stand on their own beside
// the forward and its attention: the root-mean-square norm (rmsnorm.cu), layer norm (layernorm.cu),
// the gated feed-forward (glu.cu) and the linear layer (linear.cu).
#pragma once
#include "kernels.h"
#include "tfl.h"

namespace tfl {

// Root-mean-square norm (rmsnorm.cu).  Types are TFL_F32 / TFL_F16 / TFL_BF16 / TFL_E4M3.
struct RmsArgs {
  int64_t rows = 0;
  int D = 0;
  int tpr = 0;                   // threads that hold one row (a power of two), set by the launcher
  int64_t ahead = 0;             // rows between a row and the one prefetched beside it, likewise
  float inv_d = 0.f, eps = 0.f;
  int x_type = 0, res_type = 0, y_type = 0;
  const void* x = nullptr;       // [rows, D]
  const void* res = nullptr;     // [rows, D] or null
  const float* gamma = nullptr;  // [D]
  void* res_out = nullptr;       // [rows, D] of res_type, or null
  void* y = nullptr;             // [rows, D]
  float* y_scale = nullptr;      // [rows], e4m3 only
};
struct RmsGradArgs {
  int64_t rows = 0;
  int D = 0;
  int tpr = 0;
  float inv_d = 0.f, eps = 0.f;
  int x_type = 0, res_type = 0;
  const void* sum = nullptr;     // [rows, D] of res_type
  const float* gamma = nullptr;  // [D]
  const void* dy = nullptr;      // [rows, D] of x_type
  const void* dres = nullptr;    // [rows, D] of res_type, or null
  void* dx = nullptr;            // [rows, D] of x_type, or null
  void* dsum = nullptr;          // [rows, D] of res_type, or null
  float* dgamma = nullptr;       // [D]
  float* partial = nullptr;      // [blocks, D] partial sums of dgamma
  int blocks = 0;
};
constexpr int kRmsMaxRegisterRow = 32768;  // widest row the forward holds in registers (the backward: half)
cudaError_t launch_rms_forward(const RmsArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_rms_backward(const RmsGradArgs& a, int num_sms, cudaStream_t s);

// Layer norm (layernorm.cu).
struct LnArgs {
  int64_t rows = 0;
  int D = 0;
  int tpr = 0;                   // threads that hold one row (a power of two up to 32, or whole warps), set by the launcher
  int64_t ahead = 0;             // rows between a row and the one prefetched beside it, likewise
  float inv_d = 0.f, eps = 0.f;
  int x_type = 0, res_type = 0, y_type = 0;
  const void* x = nullptr;       // [rows, D]
  const void* res = nullptr;     // [rows, D] or null
  const float* gamma = nullptr;  // [D]
  const float* beta = nullptr;   // [D] or null
  void* res_out = nullptr;       // [rows, D] of res_type, or null
  void* y = nullptr;             // [rows, D]
  float* y_scale = nullptr;      // [rows], e4m3 only
  float2* stats = nullptr;       // [rows] mean and 1 / sqrt(var + eps), or null
};
struct LnGradArgs {
  int64_t rows = 0;
  int D = 0;
  int tpr = 0;                    // as above
  float inv_d = 0.f;
  int x_type = 0, res_type = 0;
  const void* sum = nullptr;      // [rows, D] of res_type
  const float2* stats = nullptr;  // [rows]
  const float* gamma = nullptr;   // [D]
  const void* dy = nullptr;       // [rows, D] of x_type
  const void* dres = nullptr;     // [rows, D] of res_type, or null
  void* dx = nullptr;             // [rows, D] of x_type, or null
  void* dsum = nullptr;           // [rows, D] of res_type, or null
  float* dgamma = nullptr;        // [D]
  float* dbeta = nullptr;         // [D] or null
  float* partial = nullptr;       // [blocks, 2 D] partial sums of dgamma and dbeta
  int blocks = 0;
  // where a block's rows of partial sums go, set by the launcher
  float *part_gamma = nullptr, *part_beta = nullptr;
  size_t part_stride = 0;
};
// Which kernel a call takes: TFL_LN_FORM_*, and for the forms in vectors the threads of a block (at most) and a
// thread's vectors of a row.  lines: the buffers of rows begin on 16 bytes; params: gamma and beta do.
struct LnPlan {
  int form = 0, threads = 0, vectors = 0;
};
LnPlan ln_forward_plan(int D, int64_t rows, bool res_f32, bool lines, bool params, int num_sms);
LnPlan ln_backward_plan(int D, int64_t rows, bool lines, bool params, int num_sms);
cudaError_t launch_ln_forward(const LnArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_ln_backward(const LnGradArgs& a, int num_sms, cudaStream_t s);

// Matrix products of the gated feed-forward (glu.cu) and the linear layer (linear.cu), tile by tile
// (tile_gemm.cuh).
enum TileMode : int {
  GLU_FORWARD = 0,  // out[M, N] = act(A B0^T) * (A B1^T)
  GLU_SLOPES = 1,   // out[M, N] = dh u act'(g), out2[M, N] = dh act(g), g = A B0^T, u = A B1^T
  GRAD_DX = 2,      // out[M, N] = A0 B0 + A1 B1, the second sum empty for the linear layer
  GRAD_DW = 3,      // out[M, N] = A0^T B0, out2[M, N] = A1^T B0, the second for the feed-forward only
  LIN_FORWARD = 4,  // z[M, N] = A B0^T + bias, out[M, N] = act(z) + res
};
// A divisor of tile numbers, with what stands in for the division (tile_gemm.cuh).
struct Divisor {
  int d = 1, shift = -1;
  uint32_t factor = 0;
};
// The order of tiles: planes of tiles, groups of `rows` row blocks in them.
struct TileOrder {
  int num_m = 0;
  Divisor plane, group, rows, last_rows;
};
struct TileArgs {
  int M = 0, N = 0;              // rows and columns of the output
  int num_k = 0;                 // k-blocks of a tile
  int k_half = 0;                // DX: k-blocks of the first product
  int planes = 2;                // DW: outputs, or shares of the tokens
  int group_m = 8;               // row blocks of a group of tiles
  TileOrder order;               // set by the launcher
  int bno = 0, split = 1, stages = 0, stage_bytes = 0, a_bytes = 0;  // set by the launcher from the plan
  int act = 0;
  int bf16_operands = 0;         // 16-bit operands: bf16, else fp16
  int bf16_out = 0;              // 16-bit outputs (and dh): bf16, else fp16
  int ldo = 0;                   // row pitch of out and out2 (LIN_FORWARD: of the residual)
  const uint16_t* dh = nullptr;  // SLOPES: [M, N]
  uint16_t* out = nullptr;
  uint16_t* out2 = nullptr;
  const float *x_scale = nullptr, *g_scale = nullptr, *u_scale = nullptr;  // e4m3: [M], [N], [N]
  const float* bias = nullptr;   // LIN_FORWARD: [N] or null
  const void* res = nullptr;     // LIN_FORWARD: [M, N] of the output's type, or null
  int z = 0;                     // LIN_FORWARD: z is stored
  int out_f32 = 0;               // LIN_FORWARD: y (and res) fp32
  int* status = nullptr;
  int64_t timeout_ns = 2000000000LL;
};
constexpr int kTileRows = 128;  // rows of A a CTA takes
struct TileMaps {
  CUtensorMap a0, a1, b0, b1;  // LIN_FORWARD: a1 is y, b1 z, in boxes of 64 bytes by 32 rows
  CUtensorMap r;               // LIN_FORWARD: the residual, in the same boxes
};
// How a call is cut: CTAs of a pair (2) or lone ones (1), lone CTAs that share a tile's k-blocks,
// output columns of a tile, tiles that run at once,
// rows of A a CTA loads for a tile, tiles in all.
struct TilePlan {
  int cg = 0, split = 1, bno = 0, units = 0, a_rows = 0;
  int64_t tiles = 0;
  double cost = 0;  // the estimate it was chosen by, in cycles
};
// What runs at once on a device: lone CTAs, CTA pairs, and clusters of 2, 4 and 8 lone CTAs.
struct TileUnits {
  int sms = 0, pairs = 0, splits[3] = {};
};
// whole_lines: the rows of x and the weights begin on 128-byte lines.  planes: GRAD_DW's outputs; shares: of the
// tokens, of num_k k-blocks each (no tile is then shared by a cluster).
TilePlan tile_plan(int mode, bool whole_lines, int64_t M, int64_t N, int64_t num_k, const TileUnits& u, int planes = 2,
                   int shares = 1);
int tile_form(const TilePlan& p, int mode);  // TFL_GLU_FORM_* of the kernel it runs in
// Kernel attributes, and all of *u but sms for the current device.
cudaError_t prepare_tile_kernels(TileUnits* u);
cudaError_t prepare_linear_kernels();
// All modes but LIN_FORWARD, and that one.
cudaError_t launch_tiles(const TilePlan& p, int mode, bool f8, const TileMaps& mp, const TileArgs& a, cudaStream_t s);
cudaError_t launch_linear(const TilePlan& p, bool f8, const TileMaps& mp, const TileArgs& a, cudaStream_t s);
// GRAD_DW over shares of the tokens into fp32 partial sums [planes, M, N], and their sum in 16 bits.
cudaError_t prepare_linear_shares();
cudaError_t launch_linear_shares(const TilePlan& p, const TileMaps& mp, const TileArgs& a, cudaStream_t s);
cudaError_t launch_share_sums(const float* parts, int shares, int64_t values, bool bf16, uint16_t* out, cudaStream_t s);
#define TFL_DECLARE_LINEAR_FORM(NAME)   \
  cudaError_t prepare_linear_##NAME();  \
  cudaError_t launch_linear_##NAME(const TilePlan& p, bool f8, const TileMaps& mp, const TileArgs& a, cudaStream_t s);
TFL_DECLARE_LINEAR_FORM(wide)
TFL_DECLARE_LINEAR_FORM(pair)
TFL_DECLARE_LINEAR_FORM(lone)
TFL_DECLARE_LINEAR_FORM(shared)
#undef TFL_DECLARE_LINEAR_FORM

// The gated feed-forward's forward for at most kGluFewTokens tokens (glu_few.cu).
constexpr int kGluFewTokens = 16;
struct GluFewArgs {
  int tokens = 0, d_ff = 0;
  int row_bytes = 0;             // of x, Wg and Wu: d_model elements
  int act = 0, bf16_out = 0;
  const uint8_t *x = nullptr, *wg = nullptr, *wu = nullptr;
  const float *x_scale = nullptr, *g_scale = nullptr, *u_scale = nullptr;  // e4m3
  uint16_t* out = nullptr;
};
bool glu_few_fits(int64_t tokens, int64_t row_bytes);  // whether this kernel is the faster one
cudaError_t launch_glu_few(int type, const GluFewArgs& a, int num_sms, cudaStream_t s);

// The linear layer's forward for at most kLinFewTokens tokens (linear_few.cu).
constexpr int kLinFewTokens = 16;
struct LinFewArgs {
  int tokens = 0, d_out = 0;
  int row_bytes = 0;             // of x and W: d_in elements
  int act = 0, bf16 = 0;         // 16-bit outputs and z: bf16, else fp16
  int out_f32 = 0;
  const uint8_t *x = nullptr, *w = nullptr;
  const float *x_scale = nullptr, *w_scale = nullptr;  // e4m3
  const float* bias = nullptr;
  const void* res = nullptr;
  uint16_t* z = nullptr;
  void* out = nullptr;
};
// Whether this kernel is the faster one.
bool lin_few_fits(int64_t tokens, int64_t row_bytes, int64_t d_out, bool f8, int num_sms);
cudaError_t launch_lin_few(int type, const LinFewArgs& a, int num_sms, cudaStream_t s);

// The linear layer's dz = dy act'(z) and the sums of its columns (linear.cu).
struct LinSlopeArgs {
  int64_t rows = 0;
  int cols = 0, pitch = 0;       // of dy and z; row pitch of dz
  int tx = 0;                    // threads across 8 columns each, set by the launcher
  int dy_type = 0, type = 0, act = 0;
  const void* dy = nullptr;
  const uint16_t* z = nullptr;   // unused without an activation
  uint16_t* dz = nullptr;        // or null
  float* db = nullptr;           // [cols] or null
  float* partial = nullptr;      // [blocks, cols]
  int blocks = 0;                // rows of partial sums there is room for
};
// *parts: the rows of partial sums that launch_lin_db has yet to add up (0: db is done).
cudaError_t launch_lin_slopes(const LinSlopeArgs& a, int num_sms, cudaStream_t s, int* parts);
cudaError_t launch_lin_db(const LinSlopeArgs& a, int parts, cudaStream_t s);

}  // namespace tfl
