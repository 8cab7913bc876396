// linear_form.cuh -- the linear layer's kernels of one form of tiles: every epilogue for 16-bit operands, those
// without z for e4m3 (which have no backward).  One translation unit a form, so that they compile side by side.
#pragma once
#include "tile_gemm.cuh"

#define TFL_LIN_EPILOGUES(X, CG, FORM)                                                                  \
  X(CG, false, FORM, 0) X(CG, false, FORM, 1) X(CG, false, FORM, 2) X(CG, false, FORM, 3)               \
  X(CG, false, FORM, 4) X(CG, false, FORM, 5) X(CG, false, FORM, 6) X(CG, false, FORM, 7)               \
  X(CG, true, FORM, 0) X(CG, true, FORM, 1) X(CG, true, FORM, 4) X(CG, true, FORM, 5)
#define TFL_LIN_PREPARE(CG, F8, FORM, EPI) \
  if (e == cudaSuccess) e = prepare_one<CG, LIN_FORWARD, F8, FORM, EPI>();
#define TFL_LIN_LAUNCH(CG, F8, FORM, EPI) \
  if (f8 == F8 && epi == EPI) return launch_one<CG, LIN_FORWARD, F8, FORM, EPI>(mp, a, p, s);
#define TFL_LINEAR_FORM(NAME, CG, FORM)                                                                 \
  cudaError_t prepare_linear_##NAME() {                                                                 \
    cudaError_t e = cudaSuccess;                                                                        \
    TFL_LIN_EPILOGUES(TFL_LIN_PREPARE, CG, FORM)                                                        \
    return e;                                                                                           \
  }                                                                                                     \
  cudaError_t launch_linear_##NAME(const TilePlan& p, bool f8, const TileMaps& mp, const TileArgs& a,   \
                                   cudaStream_t s) {                                                    \
    const int epi = (a.out_f32 ? kEpiF32 : 0) | (a.z ? kEpiZ : 0) | (a.res ? kEpiRes : 0);              \
    TFL_LIN_EPILOGUES(TFL_LIN_LAUNCH, CG, FORM)                                                         \
    return cudaErrorInvalidValue;                                                                       \
  }
