// api_ops.cu -- the C ABI of the operators that stand on their own (include/tfl.h): the
// root-mean-square norm, layer norm, the gated feed-forward and the linear layer.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>
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

// Frees a handle's memory with its device current, after what still runs there.
void release(int device, void* p) {
  int dev = device;
  cudaGetDevice(&dev);
  if (dev != device) cudaSetDevice(device);
  cudaDeviceSynchronize();
  if (p) cudaFree(p);
  if (dev != device) cudaSetDevice(dev);
}

int same_device(int device) {
  int dev = 0;
  TFL_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev != device)
    return fail(TFL_ERR_INVALID_ARG, "the current device is not the one the handle was created on");
  return TFL_OK;
}

// What the two norms are created with.
int check_norm(int32_t d_model, int32_t x_type, int32_t res_type, int32_t y_type, float eps) {
  if (d_model < 1 || d_model > (1 << 24)) return fail(TFL_ERR_INVALID_ARG, "d_model must be in 1 .. 2^24");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(TFL_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (x_type != TFL_F32 && !type_16bit(x_type)) return fail(TFL_ERR_UNSUPPORTED, "x must be fp32, fp16 or bf16");
  if (res_type != TFL_F32 && res_type != x_type)
    return fail(TFL_ERR_UNSUPPORTED, "the residual must be fp32 or of x's type");
  if (!(y_type == x_type || y_type == TFL_E4M3 || (x_type == TFL_F32 && type_16bit(y_type))))
    return fail(TFL_ERR_UNSUPPORTED, "y must be of x's type or e4m3, or fp16 or bf16 for an fp32 x");
  return TFL_OK;
}

// Rows of partial sums of a backward, one a block: as many blocks as fill the GPU, but no more rows of
// `values` floats than 64 MiB hold.
int partial_rows(int64_t values, int sms) {
  const int64_t fit = ((int64_t)64 << 20) / (values * 4);
  const int64_t want = (int64_t)sms * 4;
  return (int)(fit < 1 ? 1 : fit < want ? fit : want);
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
  if (int rc = check_norm(d_model, x_type, res_type, y_type, eps)) return rc;
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
    n->blocks = partial_rows(d_model, sms);
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
  TFL_CUDA(launch_rms_backward(a, n->num_sms, st), "norm backward");
  return TFL_OK;
}

void tfl_rmsnorm_destroy(tfl_rmsnorm* n) {
  if (!n) return;
  release(n->device, n->partial);
  delete n;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Layer norm.
struct tfl_layernorm {
  int D = 0, x_type = 0, res_type = 0, y_type = 0;
  float eps = 0.f;
  int device = 0, num_sms = 0;
  float* partial = nullptr;  // [blocks, 2 D], the backward's partial sums of dgamma and dbeta
  int blocks = 0;
};

extern "C" {

int tfl_layernorm_create(int32_t d_model, int32_t x_type, int32_t res_type, int32_t y_type, float eps,
                         tfl_layernorm** out) {
  g_err.clear();
  if (!out) return fail(TFL_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (int rc = check_norm(d_model, x_type, res_type, y_type, eps)) return rc;
  int dev = 0, sms = 0;
  if (int rc = usable_device(&dev, &sms)) return rc;
  tfl_layernorm* n = new (std::nothrow) tfl_layernorm();
  if (!n) return fail(TFL_ERR_OOM, "handle allocation failed");
  n->D = d_model;
  n->x_type = x_type;
  n->res_type = res_type;
  n->y_type = y_type;
  n->eps = eps;
  n->device = dev;
  n->num_sms = sms;
  if (y_type == x_type) {
    n->blocks = partial_rows((int64_t)d_model * 2, sms);
    if (cudaMalloc(&n->partial, (size_t)n->blocks * d_model * 2 * sizeof(float)) != cudaSuccess) {
      cudaGetLastError();
      delete n;
      return fail(TFL_ERR_OOM, "scratch allocation for the norm's backward failed");
    }
  }
  *out = n;
  return TFL_OK;
}

int tfl_layernorm_forward(tfl_layernorm* n, int64_t rows, const void* x, const void* res, const float* gamma,
                          const float* beta, void* res_out, void* y, float* y_scale, float* stats, tfl_stream stream) {
  g_err.clear();
  if (!n) return fail(TFL_ERR_INVALID_ARG, "handle is NULL");
  if (rows < 0 || rows >= ((int64_t)1 << 31)) return fail(TFL_ERR_INVALID_ARG, "rows must be in 0 .. 2^31 - 1");
  if (rows == 0) return TFL_OK;
  if (!x || !gamma || !y) return fail(TFL_ERR_INVALID_ARG, "x, gamma and y must be non-NULL device pointers");
  if ((n->y_type == TFL_E4M3) != (y_scale != nullptr))
    return fail(TFL_ERR_INVALID_ARG, "y_scale goes with an e4m3 y, and only with one");
  const size_t xs = type_size(n->x_type), rs = type_size(n->res_type), ys = type_size(n->y_type);
  if (misaligned(x, xs) || misaligned(res, rs) || misaligned(res_out, rs) || misaligned(y, ys) ||
      misaligned(gamma, 4) || misaligned(beta, 4) || misaligned(y_scale, 4))
    return fail(TFL_ERR_INVALID_ARG, "a buffer is not aligned to its elements");
  if (misaligned(stats, 8)) return fail(TFL_ERR_INVALID_ARG, "stats must be 8-byte aligned");
  const size_t count = (size_t)rows * n->D, D = n->D;
  const Span ins[4] = {{x, count * xs, n->x_type}, {res, count * rs, n->res_type}, {gamma, D * 4, TFL_F32}, {beta, D * 4, TFL_F32}};
  const Span outs[4] = {{res_out, count * rs, n->res_type},
                        {y, count * ys, n->y_type},
                        {y_scale, (size_t)rows * 4, TFL_F32},
                        {stats, (size_t)rows * 8, TFL_F32}};
  bool bad = false;
  for (int o = 0; o < 4; ++o) {
    // res_out may be res or x, y may be x
    for (int i = 0; i < 4; ++i) bad = bad || overlap(outs[o], ins[i], (o == 0 && i < 2) || (o == 1 && i == 0));
    for (int k = 0; k < o; ++k) bad = bad || overlap(outs[o], outs[k], false);
  }
  if (bad) return fail(TFL_ERR_INVALID_ARG, "an output overlaps another buffer");
  if (int rc = same_device(n->device)) return rc;
  LnArgs a;
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
  a.beta = beta;
  a.res_out = res_out;
  a.y = y;
  a.y_scale = y_scale;
  a.stats = reinterpret_cast<float2*>(stats);
  TFL_CUDA(launch_ln_forward(a, n->num_sms, static_cast<cudaStream_t>(stream)), "layer norm forward");
  return TFL_OK;
}

int tfl_layernorm_backward(tfl_layernorm* n, int64_t rows, const void* sum, const float* stats, const float* gamma,
                           const void* dy, const void* dres, void* dx, void* dsum, float* dgamma, float* dbeta,
                           tfl_stream stream) {
  g_err.clear();
  if (!n) return fail(TFL_ERR_INVALID_ARG, "handle is NULL");
  if (n->y_type != n->x_type) return fail(TFL_ERR_UNSUPPORTED, "the backward needs a norm whose y is of x's type");
  if (rows < 0 || rows >= ((int64_t)1 << 31)) return fail(TFL_ERR_INVALID_ARG, "rows must be in 0 .. 2^31 - 1");
  if (!dgamma || misaligned(dgamma, 4)) return fail(TFL_ERR_INVALID_ARG, "dgamma must be a 4-byte aligned device pointer");
  if (misaligned(dbeta, 4)) return fail(TFL_ERR_INVALID_ARG, "dbeta must be 4-byte aligned");
  const size_t D = n->D;
  const Span sd[2] = {{dgamma, D * 4, TFL_F32}, {dbeta, D * 4, TFL_F32}};
  if (overlap(sd[0], sd[1], false)) return fail(TFL_ERR_INVALID_ARG, "an output overlaps another buffer");
  if (int rc = same_device(n->device)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    TFL_CUDA(cudaMemsetAsync(dgamma, 0, D * 4, st), "dgamma clear");
    if (dbeta) TFL_CUDA(cudaMemsetAsync(dbeta, 0, D * 4, st), "dbeta clear");
    return TFL_OK;
  }
  if (!sum || !stats || !gamma || !dy)
    return fail(TFL_ERR_INVALID_ARG, "sum, stats, gamma and dy must be non-NULL device pointers");
  if (!dx && !dsum) return fail(TFL_ERR_INVALID_ARG, "dx or dsum must be given");
  const size_t xs = type_size(n->x_type), rs = type_size(n->res_type);
  if (misaligned(sum, rs) || misaligned(gamma, 4) || misaligned(dy, xs) || misaligned(dres, rs) ||
      misaligned(dx, xs) || misaligned(dsum, rs))
    return fail(TFL_ERR_INVALID_ARG, "a buffer is not aligned to its elements");
  if (misaligned(stats, 8)) return fail(TFL_ERR_INVALID_ARG, "stats must be 8-byte aligned");
  const size_t count = (size_t)rows * D;
  const Span ins[3] = {{sum, count * rs, n->res_type}, {dy, count * xs, n->x_type}, {dres, count * rs, n->res_type}};
  const Span outs[2] = {{dx, count * xs, n->x_type}, {dsum, count * rs, n->res_type}};
  const Span sg{gamma, D * 4, TFL_F32}, ss{stats, (size_t)rows * 8, TFL_F32};
  bool bad = overlap(outs[0], outs[1], false);
  for (const Span& o : outs) {
    for (const Span& i : ins) bad = bad || overlap(o, i, true);
    bad = bad || overlap(o, sg, false) || overlap(o, ss, false) || overlap(o, sd[0], false) || overlap(o, sd[1], false);
  }
  for (const Span& d : sd) {
    for (const Span& i : ins) bad = bad || overlap(d, i, false);
    bad = bad || overlap(d, sg, false) || overlap(d, ss, false);
  }
  if (bad) return fail(TFL_ERR_INVALID_ARG, "an output overlaps another buffer");
  LnGradArgs a;
  a.rows = rows;
  a.D = n->D;
  a.inv_d = 1.0f / (float)n->D;
  a.x_type = n->x_type;
  a.res_type = n->res_type;
  a.sum = sum;
  a.stats = reinterpret_cast<const float2*>(stats);
  a.gamma = gamma;
  a.dy = dy;
  a.dres = dres;
  a.dx = dx;
  a.dsum = dsum;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.partial = n->partial;
  a.blocks = n->blocks;
  TFL_CUDA(launch_ln_backward(a, n->num_sms, st), "layer norm backward");
  return TFL_OK;
}

void tfl_layernorm_destroy(tfl_layernorm* n) {
  if (!n) return;
  release(n->device, n->partial);
  delete n;
}

int tfl_selftest_layernorm_plan(int32_t d_model, int32_t res_type, int32_t part, int64_t rows, int32_t aligned,
                                int32_t sms, int32_t* out) {
  g_err.clear();
  if (!out || d_model < 1 || d_model > (1 << 24) || (res_type != TFL_F32 && !type_16bit(res_type)) || part < 0 || part > 1 ||
      rows < 1 || rows >= ((int64_t)1 << 31) || sms < 0)
    return fail(TFL_ERR_INVALID_ARG, "no such launch");
  int dev = 0, units = sms;
  if (!sms)
    if (int rc = usable_device(&dev, &units)) return rc;
  const bool on16 = aligned != 0;
  const LnPlan p = part ? ln_backward_plan(d_model, rows, on16, on16, units)
                        : ln_forward_plan(d_model, rows, res_type == TFL_F32, on16, on16, units);
  out[0] = p.form;
  out[1] = p.threads;
  out[2] = p.vectors;
  return TFL_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Gated feed-forward.
struct tfl_glu {
  int D = 0, F = 0, in_type = 0, out_type = 0, act = 0;
  int64_t max_grad_tokens = 0;
  int device = 0;
  TileUnits units;
  int* status = nullptr;                          // status word (256 bytes), then dg and du
  uint16_t *dg = nullptr, *du = nullptr;          // [max_grad_tokens, F] in rows of `pitch`
  int pitch = 0;                                  // F to the next 128 bytes: a copied box row is then one line
};

namespace {

// A row-major [rows, cols] matrix in boxes of 128 bytes of columns by box_rows, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int elem, uint32_t box_rows,
              int64_t pitch = 0) {
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)((pitch ? pitch : cols) * elem)};
  cuuint32_t box[2] = {(cuuint32_t)(128 / elem), box_rows};
  cuuint32_t es[2] = {1, 1};
  return get_encode()(m, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
                      const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A row-major [rows, cols] output or residual in boxes of 64 bytes by 32 rows, 64-byte swizzle.
bool make_io_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int elem) {
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(cols * elem)};
  cuuint32_t box[2] = {(cuuint32_t)(64 / elem), 32};
  cuuint32_t es[2] = {1, 1};
  return get_encode()(m, elem == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
                      const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Kernel attributes and what runs at once on a device: the same for every handle, asked once.
int tile_units(int dev, int sms, TileUnits* u) {
  constexpr int kDevices = 64;
  static std::mutex lock;
  static TileUnits known[kDevices];
  std::lock_guard<std::mutex> hold(lock);
  if (dev < kDevices && known[dev].sms) {
    *u = known[dev];
    return TFL_OK;
  }
  TFL_CUDA(prepare_tile_kernels(u), "feed-forward kernel attributes");
  TFL_CUDA(prepare_linear_kernels(), "linear layer kernel attributes");
  u->sms = sms;
  if (dev < kDevices) known[dev] = *u;
  return TFL_OK;
}

// How the forward and the three launches of the backward are cut.
TilePlan glu_call_plan(int D, int F, bool f8, int mode, int64_t tokens, const TileUnits& u) {
  const int ke = f8 ? 128 : 64;
  const bool lines = D * (f8 ? 1 : 2) % 128 == 0;
  if (mode == GRAD_DX) return tile_plan(mode, lines, tokens, D, 2 * ((F + ke - 1) / ke), u);
  if (mode == GRAD_DW) return tile_plan(mode, lines, F, D, (tokens + ke - 1) / ke, u);
  return tile_plan(mode, lines, tokens, F, (D + ke - 1) / ke, u);
}

constexpr int kMnBox = 64;  // MN-major operands come in boxes of 64 k rows

int check_tokens(const tfl_glu* g, int64_t tokens) {
  if (tokens < 0 || tokens > INT32_MAX - 512) return fail(TFL_ERR_INVALID_ARG, "tokens must be in 0 .. 2^31 - 513");
  if ((tokens + 127) / 128 * ((g->F + 15) / 16) > INT32_MAX || (tokens + 127) / 128 * ((g->D + 31) / 32) > INT32_MAX)
    return fail(TFL_ERR_UNSUPPORTED, "too many tokens for this width");
  return TFL_OK;
}

// What a plan self-test is asked about: the given units, or the current device's.
int selftest_units(const int32_t* units, TileUnits* u) {
  if (units) {
    u->sms = units[0];
    u->pairs = units[1];
    for (int i = 0; i < 3; ++i) u->splits[i] = units[2 + i];
    if (u->sms < 1 || u->pairs < 1) return fail(TFL_ERR_INVALID_ARG, "a device runs lone CTAs and pairs");
    return TFL_OK;
  }
  int dev = 0, sms = 0;
  if (int rc = usable_device(&dev, &sms)) return rc;
  return tile_units(dev, sms, u);
}

void tell_plan(const TilePlan& p, int mode, int32_t* out) {
  out[0] = tile_form(p, mode);
  out[1] = p.bno;
  out[2] = (int32_t)(p.tiles > INT32_MAX ? INT32_MAX : p.tiles);
  out[3] = p.units;
}

int read_status(int* status, cudaStream_t stream) {
  TFL_CUDA(cudaStreamSynchronize(stream), "cudaStreamSynchronize");
  int v = 0;
  TFL_CUDA(cudaMemcpy(&v, status, sizeof(int), cudaMemcpyDeviceToHost), "status read");
  if (v) TFL_CUDA(cudaMemset(status, 0, sizeof(int)), "status clear");
  if (v & TFL_DEV_TIMEOUT) return fail(TFL_ERR_DEVICE_TIMEOUT, "a device-side wait ran out of time");
  return TFL_OK;
}

TileArgs glu_args(const tfl_glu* g) {
  TileArgs a;
  a.act = g->act;
  a.bf16_operands = g->in_type == TFL_BF16;
  a.bf16_out = g->out_type == TFL_BF16;
  a.status = g->status;
  return a;
}

}  // namespace

extern "C" {

int tfl_glu_create(int32_t d_model, int32_t d_ff, int32_t in_type, int32_t out_type, int32_t act,
                   int64_t max_grad_tokens, tfl_glu** out) {
  g_err.clear();
  if (!out) return fail(TFL_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (d_model < 1 || d_ff < 1) return fail(TFL_ERR_INVALID_ARG, "d_model and d_ff must be >= 1");
  if (act != TFL_ACT_SILU && act != TFL_ACT_GELU) return fail(TFL_ERR_INVALID_ARG, "no such activation");
  if (max_grad_tokens < 0 || max_grad_tokens > INT32_MAX - 512)
    return fail(TFL_ERR_INVALID_ARG, "max_grad_tokens must be in 0 .. 2^31 - 513");
  if (!type_16bit(out_type) || !(in_type == out_type || in_type == TFL_E4M3))
    return fail(TFL_ERR_UNSUPPORTED, "the output must be fp16 or bf16, the operands of its type or e4m3");
  if (in_type == TFL_E4M3 && max_grad_tokens) return fail(TFL_ERR_UNSUPPORTED, "e4m3 operands have no backward");
  const int step = in_type == TFL_E4M3 ? 16 : 8;
  if (d_model % step || d_ff % step || d_model > (1 << 24) || d_ff > (1 << 24))
    return fail(TFL_ERR_UNSUPPORTED,
                "d_model and d_ff must be multiples of 8 (16 for e4m3 operands), at most 2^24");
  int dev = 0, sms = 0;
  if (int rc = usable_device(&dev, &sms)) return rc;
  if (!get_encode()) return fail(TFL_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  TileUnits units;
  if (int rc = tile_units(dev, sms, &units)) return rc;
  if (units.pairs < 1) return fail(TFL_ERR_UNSUPPORTED, "the device runs no CTA pairs");
  tfl_glu* g = new (std::nothrow) tfl_glu();
  if (!g) return fail(TFL_ERR_OOM, "handle allocation failed");
  g->D = d_model;
  g->F = d_ff;
  g->in_type = in_type;
  g->out_type = out_type;
  g->act = act;
  g->max_grad_tokens = max_grad_tokens;
  g->device = dev;
  g->units = units;
  g->pitch = (d_ff + 63) / 64 * 64;
  const size_t each = ((size_t)max_grad_tokens * g->pitch * 2 + 255) / 256 * 256;
  if (cudaMalloc(&g->status, 256 + 2 * each) != cudaSuccess) {
    cudaGetLastError();
    delete g;
    return fail(TFL_ERR_OOM, "scratch allocation for the feed-forward failed");
  }
  g->dg = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(g->status) + 256);
  g->du = g->dg + each / 2;
  if (cudaMemset(g->status, 0, 256) != cudaSuccess) {
    cudaFree(g->status);
    delete g;
    return fail(TFL_ERR_CUDA, "status word clear failed");
  }
  *out = g;
  return TFL_OK;
}

int tfl_glu_forward(tfl_glu* g, int64_t tokens, const void* x, const float* x_scale, const void* wg,
                    const float* wg_scale, const void* wu, const float* wu_scale, void* h, tfl_stream stream) {
  g_err.clear();
  if (!g) return fail(TFL_ERR_INVALID_ARG, "handle is NULL");
  if (int rc = check_tokens(g, tokens)) return rc;
  if (tokens == 0) return TFL_OK;
  if (!x || !wg || !wu || !h) return fail(TFL_ERR_INVALID_ARG, "x, wg, wu and h must be non-NULL device pointers");
  const bool f8 = g->in_type == TFL_E4M3;
  if (f8 ? !(x_scale && wg_scale && wu_scale) : (x_scale || wg_scale || wu_scale))
    return fail(TFL_ERR_INVALID_ARG, "scales go with e4m3 operands, and only with them");
  if (misaligned(x, 16) || misaligned(wg, 16) || misaligned(wu, 16) || misaligned(h, 16) ||
      misaligned(x_scale, 4) || misaligned(wg_scale, 16) || misaligned(wu_scale, 16))
    return fail(TFL_ERR_INVALID_ARG, "x, wg, wu, h and the weights' scales must be 16-byte aligned");
  const size_t es = f8 ? 1 : 2, T = (size_t)tokens, D = g->D, F = g->F;
  const Span sh{h, T * F * 2, g->out_type};
  const Span in[6] = {{x, T * D * es, 0},      {wg, F * D * es, 0},    {wu, F * D * es, 0},
                      {x_scale, T * 4, 0}, {wg_scale, F * 4, 0}, {wu_scale, F * 4, 0}};
  for (const Span& i : in)
    if (overlap(sh, i, false)) return fail(TFL_ERR_INVALID_ARG, "h overlaps another buffer");
  if (int rc = same_device(g->device)) return rc;
  if (glu_few_fits(tokens, (int64_t)g->D * (int64_t)es)) {
    GluFewArgs a;
    a.tokens = (int)tokens;
    a.d_ff = g->F;
    a.row_bytes = g->D * (int)es;
    a.act = g->act;
    a.bf16_out = g->out_type == TFL_BF16;
    a.x = static_cast<const uint8_t*>(x);
    a.wg = static_cast<const uint8_t*>(wg);
    a.wu = static_cast<const uint8_t*>(wu);
    a.x_scale = x_scale;
    a.g_scale = wg_scale;
    a.u_scale = wu_scale;
    a.out = static_cast<uint16_t*>(h);
    TFL_CUDA(launch_glu_few(g->in_type, a, g->units.sms, static_cast<cudaStream_t>(stream)), "feed-forward");
    return TFL_OK;
  }
  const TilePlan p = glu_call_plan(g->D, g->F, f8, GLU_FORWARD, tokens, g->units);
  TileMaps mp;
  if (!make_map(&mp.a0, x, tokens, g->D, (int)es, p.a_rows) || !make_map(&mp.b0, wg, g->F, g->D, (int)es, p.bno) ||
      !make_map(&mp.b1, wu, g->F, g->D, (int)es, p.bno))
    return fail(TFL_ERR_CUDA, "feed-forward tensor map encoding failed");
  mp.a1 = mp.a0;
  TileArgs a = glu_args(g);
  a.M = (int)tokens;
  a.N = g->F;
  a.num_k = (g->D + (f8 ? 127 : 63)) / (f8 ? 128 : 64);
  a.x_scale = x_scale;
  a.g_scale = wg_scale;
  a.u_scale = wu_scale;
  a.ldo = g->F;
  a.out = static_cast<uint16_t*>(h);
  TFL_CUDA(launch_tiles(p, GLU_FORWARD, f8, mp, a, static_cast<cudaStream_t>(stream)), "feed-forward");
  return TFL_OK;
}

int tfl_glu_backward(tfl_glu* g, int64_t tokens, const void* x, const void* wg, const void* wu, const void* dh,
                     void* dx, void* dwg, void* dwu, tfl_stream stream) {
  g_err.clear();
  if (!g) return fail(TFL_ERR_INVALID_ARG, "handle is NULL");
  if (int rc = check_tokens(g, tokens)) return rc;
  if (g->in_type == TFL_E4M3) return fail(TFL_ERR_UNSUPPORTED, "e4m3 operands have no backward");
  if (tokens > g->max_grad_tokens)
    return fail(TFL_ERR_INVALID_ARG, "more tokens than the max_grad_tokens the handle was created with");
  if (!dwg || !dwu) return fail(TFL_ERR_INVALID_ARG, "dwg and dwu must be non-NULL device pointers");
  const size_t T = (size_t)tokens, D = g->D, F = g->F;
  if (misaligned(dwg, 16) || misaligned(dwu, 16)) return fail(TFL_ERR_INVALID_ARG, "every buffer must be 16-byte aligned");
  const Span outs[3] = {{dx, T * D * 2, 0}, {dwg, F * D * 2, 0}, {dwu, F * D * 2, 0}};
  if (overlap(outs[1], outs[2], false)) return fail(TFL_ERR_INVALID_ARG, "an output overlaps another buffer");
  if (int rc = same_device(g->device)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    TFL_CUDA(cudaMemsetAsync(dwg, 0, F * D * 2, st), "dwg clear");
    TFL_CUDA(cudaMemsetAsync(dwu, 0, F * D * 2, st), "dwu clear");
    return TFL_OK;
  }
  if (!x || !wg || !wu || !dh || !dx)
    return fail(TFL_ERR_INVALID_ARG, "x, wg, wu, dh and dx must be non-NULL device pointers");
  if (misaligned(x, 16) || misaligned(wg, 16) || misaligned(wu, 16) || misaligned(dh, 16) || misaligned(dx, 16))
    return fail(TFL_ERR_INVALID_ARG, "every buffer must be 16-byte aligned");
  const Span ins[4] = {{x, T * D * 2, 0}, {wg, F * D * 2, 0}, {wu, F * D * 2, 0}, {dh, T * F * 2, 0}};
  bool bad = overlap(outs[0], outs[1], false) || overlap(outs[0], outs[2], false);
  for (const Span& o : outs)
    for (const Span& i : ins) bad = bad || overlap(o, i, false);
  if (bad) return fail(TFL_ERR_INVALID_ARG, "an output overlaps another buffer");

  const int Di = g->D, Fi = g->F, Ti = (int)tokens;
  const int kd = (Di + 63) / 64, kf = (Fi + 63) / 64, kt = (Ti + 63) / 64;
  const TilePlan p1 = glu_call_plan(Di, Fi, false, GLU_SLOPES, tokens, g->units);
  const TilePlan p2 = glu_call_plan(Di, Fi, false, GRAD_DX, tokens, g->units);
  const TilePlan p3 = glu_call_plan(Di, Fi, false, GRAD_DW, tokens, g->units);
  TileMaps m1, m2, m3;
  bool ok = make_map(&m1.a0, x, tokens, Di, 2, p1.a_rows) && make_map(&m1.b0, wg, Fi, Di, 2, p1.bno) &&
            make_map(&m1.b1, wu, Fi, Di, 2, p1.bno);
  m1.a1 = m1.a0;
  ok = ok && make_map(&m2.a0, g->dg, tokens, Fi, 2, p2.a_rows, g->pitch) &&
       make_map(&m2.a1, g->du, tokens, Fi, 2, p2.a_rows, g->pitch) &&
       make_map(&m2.b0, wg, Fi, Di, 2, kMnBox) && make_map(&m2.b1, wu, Fi, Di, 2, kMnBox);
  ok = ok && make_map(&m3.a0, g->dg, tokens, Fi, 2, kMnBox, g->pitch) &&
       make_map(&m3.a1, g->du, tokens, Fi, 2, kMnBox, g->pitch) &&
       make_map(&m3.b0, x, tokens, Di, 2, kMnBox);
  m3.b1 = m3.b0;
  if (!ok) return fail(TFL_ERR_CUDA, "feed-forward tensor map encoding failed");

  TileArgs a = glu_args(g);
  a.M = Ti;
  a.N = Fi;
  a.num_k = kd;
  a.dh = static_cast<const uint16_t*>(dh);
  a.ldo = g->pitch;
  a.out = g->dg;
  a.out2 = g->du;
  TFL_CUDA(launch_tiles(p1, GLU_SLOPES, false, m1, a, st), "feed-forward slopes");
  a = glu_args(g);
  a.M = Ti;
  a.N = Di;
  a.k_half = kf;
  a.num_k = 2 * kf;
  a.ldo = Di;
  a.out = static_cast<uint16_t*>(dx);
  TFL_CUDA(launch_tiles(p2, GRAD_DX, false, m2, a, st), "feed-forward dx");
  a = glu_args(g);
  a.M = Fi;
  a.N = Di;
  a.num_k = kt;
  a.ldo = Di;
  a.out = static_cast<uint16_t*>(dwg);
  a.out2 = static_cast<uint16_t*>(dwu);
  TFL_CUDA(launch_tiles(p3, GRAD_DW, false, m3, a, st), "feed-forward weight gradients");
  return TFL_OK;
}

int tfl_selftest_glu_plan(int32_t d_model, int32_t d_ff, int32_t in_type, int32_t part, int64_t tokens,
                          const int32_t* units, int32_t* out) {
  g_err.clear();
  const bool f8 = in_type == TFL_E4M3;
  if (!out || d_model < 1 || d_model > (1 << 24) || d_ff < 1 || d_ff > (1 << 24) || tokens < 1 ||
      tokens > INT32_MAX - 512 || part < GLU_FORWARD || part > GRAD_DW ||
      !(f8 ? part == GLU_FORWARD : type_16bit(in_type)))
    return fail(TFL_ERR_INVALID_ARG, "no such launch");
  TileUnits u;
  if (int rc = selftest_units(units, &u)) return rc;
  for (int i = 0; i < 4; ++i) out[i] = 0;
  if (part == GLU_FORWARD && glu_few_fits(tokens, (int64_t)d_model * (f8 ? 1 : 2))) return TFL_OK;
  tell_plan(glu_call_plan(d_model, d_ff, f8, part, tokens, u), part, out);
  return TFL_OK;
}

int tfl_glu_status(tfl_glu* g, tfl_stream stream) {
  g_err.clear();
  if (!g) return fail(TFL_ERR_INVALID_ARG, "handle is NULL");
  return read_status(g->status, static_cast<cudaStream_t>(stream));
}

void tfl_glu_destroy(tfl_glu* g) {
  if (!g) return;
  release(g->device, g->status);
  delete g;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Linear layer.
struct tfl_linear {
  int K = 0, N = 0, in_type = 0, out_type = 0, act = 0, dy_type = 0;
  int64_t max_grad_tokens = 0;
  int device = 0;
  TileUnits units;
  int* status = nullptr;       // status word (256 bytes), then partial sums of db, then dz
  float* partial = nullptr;    // [blocks, N]
  int blocks = 0;
  float* parts = nullptr;      // dw's partial sums over shares of the tokens
  uint16_t* dz = nullptr;      // [max_grad_tokens, N] in rows of `pitch`; null where dy serves
  int pitch = 0;               // N to the next 128 bytes: a copied box row is then one line
};

namespace {

enum LinPart : int { LIN_PART_FORWARD = 0, LIN_PART_DX = 1, LIN_PART_DW = 2 };

// How dw is cut: over shares of the tokens, by the sizes of the call alone, so that any handle gives the same bits.
// Their partial sums cost their bytes (written and read, about 4000 a cycle) and one more launch (4500 cycles).
struct DwPlan {
  TilePlan p;
  int shares = 1;
};
constexpr int64_t kMostShareBytes = 24 << 20;
constexpr int kShares[] = {2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
bool shares_fit(int shares, int K, int N, int64_t tokens) {
  return (int64_t)shares * K * N * 4 <= kMostShareBytes && (tokens + 63) / 64 >= 4 * shares;
}
// The most that any call of up to this many tokens takes.
int most_shares(int K, int N, int64_t tokens) {
  int most = 1;
  for (int shares : kShares)
    if (shares_fit(shares, K, N, tokens)) most = shares;
  return most;
}
DwPlan linear_dw_plan(int K, int N, int64_t tokens, const TileUnits& u) {
  const bool lines = K * 2 % 128 == 0;
  const int64_t num_k = (tokens + 63) / 64;
  DwPlan best;
  best.p = tile_plan(GRAD_DW, lines, N, K, num_k, u, 1);
  double cost = best.p.cost;
  for (int shares : kShares) {
    if (!shares_fit(shares, K, N, tokens)) break;
    const TilePlan p = tile_plan(GRAD_DW, lines, N, K, (num_k + shares - 1) / shares, u, 1, shares);
    const double with = p.cost + 4500.0 + 8.0 * shares * K * N / 4000.0;
    if (p.cg && with < cost * 0.97) {
      cost = with;
      best.p = p;
      best.shares = shares;
    }
  }
  return best;
}

TilePlan linear_call_plan(int K, int N, bool f8, int part, int64_t tokens, const TileUnits& u) {
  const int ke = f8 ? 128 : 64;
  const bool lines = K * (f8 ? 1 : 2) % 128 == 0;
  if (part == LIN_PART_DX) return tile_plan(GRAD_DX, lines, tokens, K, (N + ke - 1) / ke, u, 1);
  if (part == LIN_PART_DW) return linear_dw_plan(K, N, tokens, u).p;
  return tile_plan(LIN_FORWARD, lines, tokens, N, (K + ke - 1) / ke, u);
}

int check_tokens(const tfl_linear* l, int64_t tokens) {
  if (tokens < 0 || tokens > INT32_MAX - 512) return fail(TFL_ERR_INVALID_ARG, "tokens must be in 0 .. 2^31 - 513");
  if ((tokens + 127) / 128 * ((l->N + 31) / 32) > INT32_MAX || (tokens + 127) / 128 * ((l->K + 31) / 32) > INT32_MAX)
    return fail(TFL_ERR_UNSUPPORTED, "too many tokens for this width");
  return TFL_OK;
}

// Row blocks of a group of tiles: a wave of 76 tiles of 256 x 256 touches the fewest operands as 8 or 9 of each;
// where all columns of the output are fewer tiles than that they go first, so that no row block is left to
// another wave (100000 x 4096 x 1024 bf16 read 1.8 GB instead of 1.3).
int tile_group(const TilePlan& p, int64_t cols) { return (cols + p.bno - 1) / p.bno <= 8 ? 1 : 8; }

TileArgs linear_args(const tfl_linear* l) {
  TileArgs a;
  a.act = l->act;
  a.bf16_operands = l->in_type == TFL_BF16;
  a.bf16_out = l->out_type == TFL_BF16;
  a.out_f32 = l->out_type == TFL_F32;
  a.status = l->status;
  return a;
}

}  // namespace

extern "C" {

int tfl_linear_create(int32_t d_in, int32_t d_out, int32_t in_type, int32_t out_type, int32_t act, int32_t dy_type,
                      int64_t max_grad_tokens, tfl_linear** out) {
  g_err.clear();
  if (!out) return fail(TFL_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (d_in < 1 || d_out < 1) return fail(TFL_ERR_INVALID_ARG, "d_in and d_out must be >= 1");
  if (act != TFL_ACT_SILU && act != TFL_ACT_GELU && act != TFL_ACT_NONE)
    return fail(TFL_ERR_INVALID_ARG, "no such activation");
  if (max_grad_tokens < 0 || max_grad_tokens > INT32_MAX - 512)
    return fail(TFL_ERR_INVALID_ARG, "max_grad_tokens must be in 0 .. 2^31 - 513");
  const bool f8 = in_type == TFL_E4M3;
  if (!type_16bit(in_type) && !f8) return fail(TFL_ERR_UNSUPPORTED, "the operands must be fp16, bf16 or e4m3");
  if (out_type != TFL_F32 && !(type_16bit(out_type) && (f8 || out_type == in_type)))
    return fail(TFL_ERR_UNSUPPORTED, "the output must be fp32 or of the operands' 16-bit type (e4m3: fp16 or bf16)");
  if (f8 && max_grad_tokens) return fail(TFL_ERR_UNSUPPORTED, "e4m3 operands have no backward");
  if (max_grad_tokens && dy_type != TFL_F32 && dy_type != in_type)
    return fail(TFL_ERR_UNSUPPORTED, "dy must be fp32 or of the operands' type");
  const int step = f8 ? 16 : 8;
  if (d_in % step || d_out % step || d_in > (1 << 24) || d_out > (1 << 24))
    return fail(TFL_ERR_UNSUPPORTED, "d_in and d_out must be multiples of 8 (16 for e4m3 operands), at most 2^24");
  int dev = 0, sms = 0;
  if (int rc = usable_device(&dev, &sms)) return rc;
  if (!get_encode()) return fail(TFL_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  TileUnits units;
  if (int rc = tile_units(dev, sms, &units)) return rc;
  if (units.pairs < 1) return fail(TFL_ERR_UNSUPPORTED, "the device runs no CTA pairs");
  tfl_linear* l = new (std::nothrow) tfl_linear();
  if (!l) return fail(TFL_ERR_OOM, "handle allocation failed");
  l->K = d_in;
  l->N = d_out;
  l->in_type = in_type;
  l->out_type = out_type;
  l->act = act;
  l->dy_type = dy_type;
  l->max_grad_tokens = max_grad_tokens;
  l->device = dev;
  l->units = units;
  l->pitch = (d_out + 63) / 64 * 64;
  size_t sums = 0, slopes = 0, parts = 0;
  if (max_grad_tokens) {
    const int shares = most_shares(d_in, d_out, max_grad_tokens);
    if (shares > 1) parts = ((size_t)shares * d_in * d_out * 4 + 255) / 256 * 256;
    l->blocks = partial_rows(d_out, sms * 2);
    sums = ((size_t)l->blocks * d_out * 4 + 255) / 256 * 256;
    if (act != TFL_ACT_NONE || dy_type == TFL_F32) slopes = (size_t)max_grad_tokens * l->pitch * 2;
  }
  if (cudaMalloc(&l->status, 256 + sums + parts + slopes) != cudaSuccess) {
    cudaGetLastError();
    delete l;
    return fail(TFL_ERR_OOM, "scratch allocation for the linear layer failed");
  }
  uint8_t* base = reinterpret_cast<uint8_t*>(l->status);
  if (sums) l->partial = reinterpret_cast<float*>(base + 256);
  if (parts) l->parts = reinterpret_cast<float*>(base + 256 + sums);
  if (slopes) l->dz = reinterpret_cast<uint16_t*>(base + 256 + sums + parts);
  if (cudaMemset(l->status, 0, 256) != cudaSuccess) {
    cudaFree(l->status);
    delete l;
    return fail(TFL_ERR_CUDA, "status word clear failed");
  }
  *out = l;
  return TFL_OK;
}

int tfl_linear_forward(tfl_linear* l, int64_t tokens, const void* x, const float* x_scale, const void* w,
                       const float* w_scale, const float* bias, const void* res, void* z, void* y, tfl_stream stream) {
  g_err.clear();
  if (!l) return fail(TFL_ERR_INVALID_ARG, "handle is NULL");
  if (int rc = check_tokens(l, tokens)) return rc;
  if (tokens == 0) return TFL_OK;
  if (!x || !w || !y) return fail(TFL_ERR_INVALID_ARG, "x, w and y must be non-NULL device pointers");
  const bool f8 = l->in_type == TFL_E4M3;
  if (f8 ? !(x_scale && w_scale) : (x_scale || w_scale))
    return fail(TFL_ERR_INVALID_ARG, "scales go with e4m3 operands, and only with them");
  if (z && (f8 || l->act == TFL_ACT_NONE))
    return fail(TFL_ERR_INVALID_ARG, "z goes with 16-bit operands and an activation, and only with them");
  if (misaligned(x, 16) || misaligned(w, 16) || misaligned(y, 16) || misaligned(z, 16) || misaligned(res, 16) ||
      misaligned(bias, 16) || misaligned(w_scale, 16) || misaligned(x_scale, 4))
    return fail(TFL_ERR_INVALID_ARG, "every buffer but x's scales must be 16-byte aligned");
  const size_t es = f8 ? 1 : 2, os = type_size(l->out_type), T = (size_t)tokens, K = l->K, N = l->N;
  const Span sy{y, T * N * os, l->out_type}, sz{z, T * N * 2, l->in_type}, sr{res, T * N * os, l->out_type};
  const Span in[5] = {{x, T * K * es, 0}, {w, N * K * es, 0}, {x_scale, T * 4, 0}, {w_scale, N * 4, 0}, {bias, N * 4, 0}};
  bool bad = overlap(sy, sz, false) || overlap(sy, sr, true) || overlap(sz, sr, false);
  for (const Span& i : in) bad = bad || overlap(sy, i, false) || overlap(sz, i, false);
  if (bad) return fail(TFL_ERR_INVALID_ARG, "an output overlaps another buffer");
  if (int rc = same_device(l->device)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (lin_few_fits(tokens, (int64_t)l->K * (int64_t)es, l->N, f8, l->units.sms)) {
    LinFewArgs a;
    a.tokens = (int)tokens;
    a.d_out = l->N;
    a.row_bytes = l->K * (int)es;
    a.act = l->act;
    a.bf16 = f8 ? l->out_type == TFL_BF16 : l->in_type == TFL_BF16;
    a.out_f32 = l->out_type == TFL_F32;
    a.x = static_cast<const uint8_t*>(x);
    a.w = static_cast<const uint8_t*>(w);
    a.x_scale = x_scale;
    a.w_scale = w_scale;
    a.bias = bias;
    a.res = res;
    a.z = static_cast<uint16_t*>(z);
    a.out = y;
    TFL_CUDA(launch_lin_few(l->in_type, a, l->units.sms, st), "linear layer");
    return TFL_OK;
  }
  const TilePlan p = linear_call_plan(l->K, l->N, f8, LIN_PART_FORWARD, tokens, l->units);
  TileMaps mp;
  if (!make_map(&mp.a0, x, tokens, l->K, (int)es, p.a_rows) || !make_map(&mp.b0, w, l->N, l->K, (int)es, p.bno / p.cg) ||
      !make_io_map(&mp.a1, y, tokens, l->N, (int)os) || !make_io_map(&mp.b1, z ? z : y, tokens, l->N, z ? 2 : (int)os) ||
      !make_io_map(&mp.r, res ? res : y, tokens, l->N, (int)os))
    return fail(TFL_ERR_CUDA, "linear layer tensor map encoding failed");
  TileArgs a = linear_args(l);
  a.M = (int)tokens;
  a.N = l->N;
  a.num_k = (l->K + (f8 ? 127 : 63)) / (f8 ? 128 : 64);
  a.x_scale = x_scale;
  a.g_scale = w_scale;
  a.bias = bias;
  a.res = res;
  a.z = z != nullptr;
  a.group_m = tile_group(p, l->N);
  a.ldo = l->N;
  TFL_CUDA(launch_linear(p, f8, mp, a, st), "linear layer");
  return TFL_OK;
}

int tfl_linear_backward(tfl_linear* l, int64_t tokens, const void* x, const void* w, const void* z, const void* dy,
                        void* dx, void* dw, float* db, tfl_stream stream) {
  g_err.clear();
  if (!l) return fail(TFL_ERR_INVALID_ARG, "handle is NULL");
  if (int rc = check_tokens(l, tokens)) return rc;
  if (l->in_type == TFL_E4M3) return fail(TFL_ERR_UNSUPPORTED, "e4m3 operands have no backward");
  if (tokens > l->max_grad_tokens)
    return fail(TFL_ERR_INVALID_ARG, "more tokens than the max_grad_tokens the handle was created with");
  if (!dx && !dw && !db) return fail(TFL_ERR_INVALID_ARG, "one of dx, dw and db must be given");
  if (misaligned(x, 16) || misaligned(w, 16) || misaligned(z, 16) || misaligned(dy, 16) || misaligned(dx, 16) ||
      misaligned(dw, 16) || misaligned(db, 16))
    return fail(TFL_ERR_INVALID_ARG, "every buffer must be 16-byte aligned");
  const size_t T = (size_t)tokens, K = l->K, N = l->N;
  const Span outs[3] = {{dx, T * K * 2, 0}, {dw, N * K * 2, 0}, {db, N * 4, 0}};
  const Span ins[4] = {{x, T * K * 2, 0}, {w, N * K * 2, 0}, {z, T * N * 2, 0}, {dy, T * N * type_size(l->dy_type), 0}};
  bool bad = overlap(outs[0], outs[1], false) || overlap(outs[0], outs[2], false) || overlap(outs[1], outs[2], false);
  for (const Span& o : outs)
    for (const Span& i : ins) bad = bad || overlap(o, i, false);
  if (bad) return fail(TFL_ERR_INVALID_ARG, "an output overlaps another buffer");
  if (tokens && (!dy || (dx && !w) || (dw && !x)))
    return fail(TFL_ERR_INVALID_ARG, "dy, w for dx and x for dw must be non-NULL device pointers");
  const bool act = l->act != TFL_ACT_NONE;
  if (tokens && act != (z != nullptr))
    return fail(TFL_ERR_INVALID_ARG, "z goes with an activation, and only with one");
  if (int rc = same_device(l->device)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    if (dw) TFL_CUDA(cudaMemsetAsync(dw, 0, N * K * 2, st), "dw clear");
    if (db) TFL_CUDA(cudaMemsetAsync(db, 0, N * 4, st), "db clear");
    return TFL_OK;
  }
  const int Ki = l->K, Ni = l->N, Ti = (int)tokens;
  const int kn = (Ni + 63) / 64, kt = (Ti + 63) / 64;
  const bool slopes = l->dz && (dx || dw);
  const void* dz = slopes ? l->dz : dy;
  const int pitch = slopes ? l->pitch : Ni;
  const TilePlan p1 = linear_call_plan(Ki, Ni, false, LIN_PART_DX, tokens, l->units);
  const DwPlan dwp = linear_dw_plan(Ki, Ni, tokens, l->units);
  const TilePlan& p2 = dwp.p;
  TileMaps m1, m2;
  if (dx && !(make_map(&m1.a0, dz, tokens, Ni, 2, p1.a_rows, pitch) && make_map(&m1.b0, w, Ni, Ki, 2, kMnBox)))
    return fail(TFL_ERR_CUDA, "linear layer tensor map encoding failed");
  if (dw && !(make_map(&m2.a0, dz, tokens, Ni, 2, kMnBox, pitch) && make_map(&m2.b0, x, tokens, Ki, 2, kMnBox)))
    return fail(TFL_ERR_CUDA, "linear layer tensor map encoding failed");
  m1.a1 = m1.a0;
  m1.b1 = m1.b0;
  m2.a1 = m2.a0;
  m2.b1 = m2.b0;
  LinSlopeArgs sa;
  int parts = 0;
  if (slopes || db) {
    sa.rows = tokens;
    sa.cols = Ni;
    sa.pitch = l->pitch;
    sa.dy_type = l->dy_type;
    sa.type = l->in_type;
    sa.act = l->act;
    sa.dy = dy;
    sa.z = static_cast<const uint16_t*>(z);
    sa.dz = slopes ? l->dz : nullptr;
    sa.db = db;
    sa.partial = l->partial;
    sa.blocks = l->blocks;
    TFL_CUDA(launch_lin_slopes(sa, l->units.sms, st, &parts), "linear layer slopes");
  }
  // dx, dw and db's sum read the slopes and nothing of one another's, but each waits for the launch in front of it:
  // only griddepcontrol.wait makes an earlier kernel's writes visible to a kernel that started early, and it waits for
  // all of that kernel.
  TileArgs a = linear_args(l);
  a.bf16_out = a.bf16_operands;
  if (dx) {
    a.M = Ti;
    a.N = Ki;
    a.num_k = a.k_half = kn;
    a.group_m = tile_group(p1, Ki);
    a.ldo = Ki;
    a.out = static_cast<uint16_t*>(dx);
    TFL_CUDA(launch_tiles(p1, GRAD_DX, false, m1, a, st), "linear layer dx");
  }
  if (dw) {
    a.M = Ni;
    a.N = Ki;
    a.num_k = kt;
    a.planes = dwp.shares;
    a.group_m = tile_group(p2, Ki);
    a.ldo = Ki;
    a.out = static_cast<uint16_t*>(dw);
    if (dwp.shares > 1) {
      a.out = reinterpret_cast<uint16_t*>(l->parts);
      TFL_CUDA(launch_linear_shares(p2, m2, a, st), "linear layer weight gradient");
      TFL_CUDA(launch_share_sums(l->parts, dwp.shares, (int64_t)Ni * Ki, a.bf16_operands, static_cast<uint16_t*>(dw), st),
               "linear layer weight gradient's sum");
    } else {
      TFL_CUDA(launch_tiles(p2, GRAD_DW, false, m2, a, st), "linear layer weight gradient");
    }
  }
  if (parts) TFL_CUDA(launch_lin_db(sa, parts, st), "linear layer db");
  return TFL_OK;
}

int tfl_selftest_linear_plan(int32_t d_in, int32_t d_out, int32_t in_type, int32_t part, int64_t tokens,
                             const int32_t* units, int32_t* out) {
  g_err.clear();
  const bool f8 = in_type == TFL_E4M3;
  if (!out || d_in < 1 || d_in > (1 << 24) || d_out < 1 || d_out > (1 << 24) || tokens < 1 || tokens > INT32_MAX - 512 ||
      part < LIN_PART_FORWARD || part > LIN_PART_DW || !(f8 ? part == LIN_PART_FORWARD : type_16bit(in_type)))
    return fail(TFL_ERR_INVALID_ARG, "no such launch");
  TileUnits u;
  if (int rc = selftest_units(units, &u)) return rc;
  for (int i = 0; i < 4; ++i) out[i] = 0;
  if (part == LIN_PART_FORWARD && lin_few_fits(tokens, (int64_t)d_in * (f8 ? 1 : 2), d_out, f8, u.sms)) return TFL_OK;
  const int mode = part == LIN_PART_FORWARD ? LIN_FORWARD : part == LIN_PART_DX ? GRAD_DX : GRAD_DW;
  tell_plan(linear_call_plan(d_in, d_out, f8, part, tokens, u), mode, out);
  return TFL_OK;
}

int tfl_linear_status(tfl_linear* l, tfl_stream stream) {
  g_err.clear();
  if (!l) return fail(TFL_ERR_INVALID_ARG, "handle is NULL");
  return read_status(l->status, static_cast<cudaStream_t>(stream));
}

void tfl_linear_destroy(tfl_linear* l) {
  if (!l) return;
  release(l->device, l->status);
  delete l;
}

}  // extern "C"
