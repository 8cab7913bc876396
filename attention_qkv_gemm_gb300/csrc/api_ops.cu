// api_ops.cu -- the C ABI of the operators that stand on their own (include/tfl.h): the
// root-mean-square norm.
#include <cmath>
#include <new>

#include "host.h"
#include "ops.h"

using namespace tfl;

namespace {

bool type_16bit(int t) { return t == TFL_F16 || t == TFL_BF16; }
size_t type_size(int t) { return t == TFL_F32 ? 4 : t == TFL_E4M3 ? 1 : 2; }
bool misaligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

// A buffer of a call: its bytes, and the type of its elements.
struct Span {
  const void* p;
  size_t bytes;
  int type;
};

// Two buffers may be one (same start, same type) where every element is read by the thread
// that later writes it; any other common byte is an error.
bool overlap(const Span& a, const Span& b, bool may_be_same) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  if (may_be_same && a.p == b.p && a.type == b.type) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// The current device, which has to be one this library's kernels run on.
int usable_device(int* dev, int* num_sms) {
  TFL_CUDA(cudaGetDevice(dev), "cudaGetDevice");
  int major = 0, minor = 0;
  TFL_CUDA(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev), "cudaDeviceGetAttribute");
  TFL_CUDA(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev), "cudaDeviceGetAttribute");
  TFL_CUDA(cudaDeviceGetAttribute(num_sms, cudaDevAttrMultiProcessorCount, *dev), "cudaDeviceGetAttribute");
  if (!(major == 10 && minor == 3))
    return fail(TFL_ERR_UNSUPPORTED, "device is sm_" + std::to_string(major) + std::to_string(minor) +
                                         "; this library is built for sm_103a (GB300)");
  return TFL_OK;
}

int same_device(int device) {
  int dev = 0;
  TFL_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev != device)
    return fail(TFL_ERR_INVALID_ARG, "the current device is not the one the handle was created on");
  return TFL_OK;
}

}  // namespace

// ---------------------------------------------------------------------------
// Root-mean-square norm.
struct tfl_rmsnorm {
  int D = 0, x_type = 0, res_type = 0, y_type = 0;
  float eps = 0.f;
  int device = 0, num_sms = 0;
  float* partial = nullptr;  // [blocks, D], the backward's partial sums of dgamma
  int blocks = 0;
};

extern "C" {

int tfl_rmsnorm_create(int32_t d_model, int32_t x_type, int32_t res_type, int32_t y_type, float eps,
                       tfl_rmsnorm** out) {
  g_err.clear();
  if (!out) return fail(TFL_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (d_model < 1 || d_model > (1 << 24)) return fail(TFL_ERR_INVALID_ARG, "d_model must be in 1 .. 2^24");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(TFL_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (x_type != TFL_F32 && !type_16bit(x_type)) return fail(TFL_ERR_UNSUPPORTED, "x must be fp32, fp16 or bf16");
  if (res_type != TFL_F32 && res_type != x_type)
    return fail(TFL_ERR_UNSUPPORTED, "the residual must be fp32 or of x's type");
  if (!(y_type == x_type || y_type == TFL_E4M3 || (x_type == TFL_F32 && type_16bit(y_type))))
    return fail(TFL_ERR_UNSUPPORTED, "y must be of x's type or e4m3, or fp16 or bf16 for an fp32 x");
  int dev = 0, sms = 0;
  if (int rc = usable_device(&dev, &sms)) return rc;
  tfl_rmsnorm* n = new (std::nothrow) tfl_rmsnorm();
  if (!n) return fail(TFL_ERR_OOM, "handle allocation failed");
  n->D = d_model;
  n->x_type = x_type;
  n->res_type = res_type;
  n->y_type = y_type;
  n->eps = eps;
  n->device = dev;
  n->num_sms = sms;
  if (y_type == x_type) {
    // one row of partial sums a block of the backward: as many blocks as fill the GPU, but
    // no more rows than 64 MiB hold
    const int64_t fit = ((int64_t)64 << 20) / ((int64_t)d_model * 4);
    const int64_t want = (int64_t)sms * 4;
    n->blocks = (int)(fit < 1 ? 1 : fit < want ? fit : want);
    if (cudaMalloc(&n->partial, (size_t)n->blocks * d_model * sizeof(float)) != cudaSuccess) {
      cudaGetLastError();
      delete n;
      return fail(TFL_ERR_OOM, "scratch allocation for the norm's backward failed");
    }
  }
  *out = n;
  return TFL_OK;
}

int tfl_rmsnorm_forward(tfl_rmsnorm* n, int64_t rows, const void* x, const void* res, const float* gamma,
                        void* res_out, void* y, float* y_scale, tfl_stream stream) {
  g_err.clear();
  if (!n) return fail(TFL_ERR_INVALID_ARG, "handle is NULL");
  if (rows < 0 || rows >= ((int64_t)1 << 31)) return fail(TFL_ERR_INVALID_ARG, "rows must be in 0 .. 2^31 - 1");
  if (rows == 0) return TFL_OK;
  if (!x || !gamma || !y) return fail(TFL_ERR_INVALID_ARG, "x, gamma and y must be non-NULL device pointers");
  if ((n->y_type == TFL_E4M3) != (y_scale != nullptr))
    return fail(TFL_ERR_INVALID_ARG, "y_scale goes with an e4m3 y, and only with one");
  const size_t xs = type_size(n->x_type), rs = type_size(n->res_type), ys = type_size(n->y_type);
  if (misaligned(x, xs) || misaligned(res, rs) || misaligned(res_out, rs) || misaligned(y, ys) ||
      misaligned(gamma, 4) || misaligned(y_scale, 4))
    return fail(TFL_ERR_INVALID_ARG, "a buffer is not aligned to its elements");
  const size_t count = (size_t)rows * n->D;
  const Span sx{x, count * xs, n->x_type}, sr{res, count * rs, n->res_type}, sg{gamma, (size_t)n->D * 4, TFL_F32};
  const Span so{res_out, count * rs, n->res_type}, sy{y, count * ys, n->y_type};
  const Span sc{y_scale, (size_t)rows * 4, TFL_F32};
  if (overlap(so, sr, true) || overlap(so, sx, true) || overlap(so, sg, false) || overlap(sy, sx, true) ||
      overlap(sy, sr, false) || overlap(sy, sg, false) || overlap(sy, so, false) || overlap(sc, sx, false) ||
      overlap(sc, sr, false) || overlap(sc, sg, false) || overlap(sc, so, false) || overlap(sc, sy, false))
    return fail(TFL_ERR_INVALID_ARG, "an output overlaps another buffer");
  if (int rc = same_device(n->device)) return rc;
  RmsArgs a;
  a.rows = rows;
  a.D = n->D;
  a.inv_d = 1.0f / (float)n->D;
  a.eps = n->eps;
  a.x_type = n->x_type;
  a.res_type = n->res_type;
  a.y_type = n->y_type;
  a.x = x;
  a.res = res;
  a.gamma = gamma;
  a.res_out = res_out;
  a.y = y;
  a.y_scale = y_scale;
  TFL_CUDA(launch_rms_forward(a, n->num_sms, static_cast<cudaStream_t>(stream)), "norm forward");
  return TFL_OK;
}

int tfl_rmsnorm_backward(tfl_rmsnorm* n, int64_t rows, const void* sum, const float* gamma, const void* dy,
                         const void* dres, void* dx, void* dsum, float* dgamma, tfl_stream stream) {
  g_err.clear();
  if (!n) return fail(TFL_ERR_INVALID_ARG, "handle is NULL");
  if (n->y_type != n->x_type) return fail(TFL_ERR_UNSUPPORTED, "the backward needs a norm whose y is of x's type");
  if (rows < 0 || rows >= ((int64_t)1 << 31)) return fail(TFL_ERR_INVALID_ARG, "rows must be in 0 .. 2^31 - 1");
  if (!dgamma || misaligned(dgamma, 4)) return fail(TFL_ERR_INVALID_ARG, "dgamma must be a 4-byte aligned device pointer");
  if (int rc = same_device(n->device)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    TFL_CUDA(cudaMemsetAsync(dgamma, 0, (size_t)n->D * 4, st), "dgamma clear");
    return TFL_OK;
  }
  if (!sum || !gamma || !dy) return fail(TFL_ERR_INVALID_ARG, "sum, gamma and dy must be non-NULL device pointers");
  if (!dx && !dsum) return fail(TFL_ERR_INVALID_ARG, "dx or dsum must be given");
  const size_t xs = type_size(n->x_type), rs = type_size(n->res_type);
  if (misaligned(sum, rs) || misaligned(gamma, 4) || misaligned(dy, xs) || misaligned(dres, rs) ||
      misaligned(dx, xs) || misaligned(dsum, rs))
    return fail(TFL_ERR_INVALID_ARG, "a buffer is not aligned to its elements");
  const size_t count = (size_t)rows * n->D;
  const Span ins[3] = {{sum, count * rs, n->res_type}, {dy, count * xs, n->x_type}, {dres, count * rs, n->res_type}};
  const Span outs[2] = {{dx, count * xs, n->x_type}, {dsum, count * rs, n->res_type}};
  const Span sg{gamma, (size_t)n->D * 4, TFL_F32}, sd{dgamma, (size_t)n->D * 4, TFL_F32};
  bool bad = overlap(outs[0], outs[1], false) || overlap(sd, sg, false);
  for (const Span& o : outs) {
    for (const Span& i : ins) bad = bad || overlap(o, i, true);
    bad = bad || overlap(o, sg, false) || overlap(o, sd, false);
  }
  for (const Span& i : ins) bad = bad || overlap(sd, i, false);
  if (bad) return fail(TFL_ERR_INVALID_ARG, "an output overlaps another buffer");
  RmsGradArgs a;
  a.rows = rows;
  a.D = n->D;
  a.inv_d = 1.0f / (float)n->D;
  a.eps = n->eps;
  a.x_type = n->x_type;
  a.res_type = n->res_type;
  a.sum = sum;
  a.gamma = gamma;
  a.dy = dy;
  a.dres = dres;
  a.dx = dx;
  a.dsum = dsum;
  a.dgamma = dgamma;
  a.partial = n->partial;
  a.blocks = n->blocks;
  TFL_CUDA(launch_rms_backward(a, st), "norm backward");
  return TFL_OK;
}

void tfl_rmsnorm_destroy(tfl_rmsnorm* n) {
  if (!n) return;
  cudaDeviceSynchronize();
  if (n->partial) cudaFree(n->partial);
  delete n;
}

}  // extern "C"
