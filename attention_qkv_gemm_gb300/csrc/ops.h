// ops.h -- argument blocks and host launchers of the operators that stand on their own beside
// the forward and its attention: the root-mean-square norm (rmsnorm.cu) and the gated
// feed-forward (glu.cu).
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

// Gated feed-forward (glu.cu).
enum GluMode : int {
  GLU_FORWARD = 0,  // out[M, N] = act(A B0^T) * (A B1^T)
  GLU_SLOPES = 1,   // out[M, N] = dh u act'(g), out2[M, N] = dh act(g), g = A B0^T, u = A B1^T
  GLU_DX = 2,       // out[M, N] = A0 B0 + A1 B1
  GLU_DW = 3,       // out[M, N] = A0^T B0, out2[M, N] = A1^T B0
};
struct GluArgs {
  int M = 0, N = 0;              // rows and columns of the output
  int num_k = 0;                 // k-blocks of a tile
  int k_half = 0;                // DX: k-blocks of the first product
  int bno = 0, split = 1, stages = 0, stage_bytes = 0, a_bytes = 0;  // set by the launcher from the plan
  int act = 0;
  int bf16_operands = 0;         // 16-bit operands: bf16, else fp16
  int bf16_out = 0;              // 16-bit outputs (and dh): bf16, else fp16
  int ldo = 0;                   // row pitch of out and out2
  const uint16_t* dh = nullptr;  // SLOPES: [M, N]
  uint16_t* out = nullptr;
  uint16_t* out2 = nullptr;
  const float *x_scale = nullptr, *g_scale = nullptr, *u_scale = nullptr;  // e4m3: [M], [N], [N]
  int* status = nullptr;
  int64_t timeout_ns = 2000000000LL;
};
constexpr int kGluRows = 128;  // rows of A a CTA takes
struct GluMaps {
  CUtensorMap a0, a1, b0, b1;
};
// How a call is cut: CTAs of a pair (2) or lone ones (1), lone CTAs that share a tile's k-blocks,
// output columns of a tile, tiles that run at once,
// rows of A a CTA loads for a tile, tiles in all.
struct GluPlan {
  int cg = 0, split = 1, bno = 0, units = 0, a_rows = 0;
  int64_t tiles = 0;
};
// What runs at once on a device: lone CTAs, CTA pairs, and clusters of 2, 4 and 8 lone CTAs.
struct GluUnits {
  int sms = 0, pairs = 0, splits[3] = {};
};
// whole_lines: the rows of x and the weights begin on 128-byte lines.
GluPlan glu_plan(int mode, bool whole_lines, int64_t M, int64_t N, int64_t num_k, const GluUnits& u);
int glu_form(const GluPlan& p, int mode);  // TFL_GLU_FORM_* of the kernel it runs in
// Kernel attributes, and all of *u but sms for the current device.
cudaError_t prepare_glu_kernels(GluUnits* u);
cudaError_t launch_glu(const GluPlan& p, int mode, bool f8, const GluMaps& mp, const GluArgs& a, cudaStream_t s);

// The forward for at most kGluFewTokens tokens (glu_few.cu).
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

}  // namespace tfl
