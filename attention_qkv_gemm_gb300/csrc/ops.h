// ops.h -- argument blocks and host launchers of the operators that stand on their own beside
// the forward and its attention: the root-mean-square norm (rmsnorm.cu).
#pragma once
#include "kernels.h"
#include "tfl.h"

namespace tfl {

// Root-mean-square norm (rmsnorm.cu).  Types are TFL_F32 / TFL_F16 / TFL_BF16 / TFL_E4M3.
struct RmsArgs {
  int64_t rows = 0;
  int D = 0;
  int tpr = 0;                   // threads that hold one row (a power of two), set by the launcher
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
cudaError_t launch_rms_backward(const RmsGradArgs& a, cudaStream_t s);

}  // namespace tfl
