// api_ops.cu -- the C ABI of the operators that stand on their own (include/tfl.h): the
// root-mean-square norm and the gated feed-forward.
#include <cudaTypedefs.h>

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
// Gated feed-forward.
struct tfl_glu {
  int D = 0, F = 0, in_type = 0, out_type = 0, act = 0;
  int64_t max_grad_tokens = 0;
  int device = 0;
  GluUnits units;
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

// Kernel attributes and what runs at once on a device: the same for every handle, asked once.
int glu_units(int dev, int sms, GluUnits* u) {
  constexpr int kDevices = 64;
  static std::mutex lock;
  static GluUnits known[kDevices];
  std::lock_guard<std::mutex> hold(lock);
  if (dev < kDevices && known[dev].sms) {
    *u = known[dev];
    return TFL_OK;
  }
  TFL_CUDA(prepare_glu_kernels(u), "feed-forward kernel attributes");
  u->sms = sms;
  if (dev < kDevices) known[dev] = *u;
  return TFL_OK;
}

// How the forward and the three launches of the backward are cut.
GluPlan glu_call_plan(int D, int F, bool f8, int mode, int64_t tokens, const GluUnits& u) {
  const int ke = f8 ? 128 : 64;
  const bool lines = D * (f8 ? 1 : 2) % 128 == 0;
  if (mode == GLU_DX) return glu_plan(mode, lines, tokens, D, 2 * ((F + ke - 1) / ke), u);
  if (mode == GLU_DW) return glu_plan(mode, lines, F, D, (tokens + ke - 1) / ke, u);
  return glu_plan(mode, lines, tokens, F, (D + ke - 1) / ke, u);
}

constexpr int kMnBox = 64;  // MN-major operands come in boxes of 64 k rows

int check_tokens(const tfl_glu* g, int64_t tokens) {
  if (tokens < 0 || tokens > INT32_MAX - 512) return fail(TFL_ERR_INVALID_ARG, "tokens must be in 0 .. 2^31 - 513");
  if ((tokens + 127) / 128 * ((g->F + 15) / 16) > INT32_MAX || (tokens + 127) / 128 * ((g->D + 31) / 32) > INT32_MAX)
    return fail(TFL_ERR_UNSUPPORTED, "too many tokens for this width");
  return TFL_OK;
}

GluArgs glu_args(const tfl_glu* g) {
  GluArgs a;
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
  GluUnits units;
  if (int rc = glu_units(dev, sms, &units)) return rc;
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
  const GluPlan p = glu_call_plan(g->D, g->F, f8, GLU_FORWARD, tokens, g->units);
  GluMaps mp;
  if (!make_map(&mp.a0, x, tokens, g->D, (int)es, p.a_rows) || !make_map(&mp.b0, wg, g->F, g->D, (int)es, p.bno) ||
      !make_map(&mp.b1, wu, g->F, g->D, (int)es, p.bno))
    return fail(TFL_ERR_CUDA, "feed-forward tensor map encoding failed");
  mp.a1 = mp.a0;
  GluArgs a = glu_args(g);
  a.M = (int)tokens;
  a.N = g->F;
  a.num_k = (g->D + (f8 ? 127 : 63)) / (f8 ? 128 : 64);
  a.x_scale = x_scale;
  a.g_scale = wg_scale;
  a.u_scale = wu_scale;
  a.ldo = g->F;
  a.out = static_cast<uint16_t*>(h);
  TFL_CUDA(launch_glu(p, GLU_FORWARD, f8, mp, a, static_cast<cudaStream_t>(stream)), "feed-forward");
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
  const GluPlan p1 = glu_call_plan(Di, Fi, false, GLU_SLOPES, tokens, g->units);
  const GluPlan p2 = glu_call_plan(Di, Fi, false, GLU_DX, tokens, g->units);
  const GluPlan p3 = glu_call_plan(Di, Fi, false, GLU_DW, tokens, g->units);
  GluMaps m1, m2, m3;
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

  GluArgs a = glu_args(g);
  a.M = Ti;
  a.N = Fi;
  a.num_k = kd;
  a.dh = static_cast<const uint16_t*>(dh);
  a.ldo = g->pitch;
  a.out = g->dg;
  a.out2 = g->du;
  TFL_CUDA(launch_glu(p1, GLU_SLOPES, false, m1, a, st), "feed-forward slopes");
  a = glu_args(g);
  a.M = Ti;
  a.N = Di;
  a.k_half = kf;
  a.num_k = 2 * kf;
  a.ldo = Di;
  a.out = static_cast<uint16_t*>(dx);
  TFL_CUDA(launch_glu(p2, GLU_DX, false, m2, a, st), "feed-forward dx");
  a = glu_args(g);
  a.M = Fi;
  a.N = Di;
  a.num_k = kt;
  a.ldo = Di;
  a.out = static_cast<uint16_t*>(dwg);
  a.out2 = static_cast<uint16_t*>(dwu);
  TFL_CUDA(launch_glu(p3, GLU_DW, false, m3, a, st), "feed-forward weight gradients");
  return TFL_OK;
}

int tfl_selftest_glu_plan(int32_t d_model, int32_t d_ff, int32_t in_type, int32_t part, int64_t tokens,
                          const int32_t* units, int32_t* out) {
  g_err.clear();
  const bool f8 = in_type == TFL_E4M3;
  if (!out || d_model < 1 || d_model > (1 << 24) || d_ff < 1 || d_ff > (1 << 24) || tokens < 1 ||
      tokens > INT32_MAX - 512 || part < GLU_FORWARD || part > GLU_DW ||
      !(f8 ? part == GLU_FORWARD : type_16bit(in_type)))
    return fail(TFL_ERR_INVALID_ARG, "no such launch");
  GluUnits u;
  if (units) {
    u.sms = units[0];
    u.pairs = units[1];
    for (int i = 0; i < 3; ++i) u.splits[i] = units[2 + i];
    if (u.sms < 1 || u.pairs < 1) return fail(TFL_ERR_INVALID_ARG, "a device runs lone CTAs and pairs");
  } else {
    int dev = 0, sms = 0;
    if (int rc = usable_device(&dev, &sms)) return rc;
    if (int rc = glu_units(dev, sms, &u)) return rc;
  }
  for (int i = 0; i < 4; ++i) out[i] = 0;
  if (part == GLU_FORWARD && glu_few_fits(tokens, (int64_t)d_model * (f8 ? 1 : 2))) return TFL_OK;
  const GluPlan p = glu_call_plan(d_model, d_ff, f8, part, tokens, u);
  out[0] = glu_form(p, part);
  out[1] = p.bno;
  out[2] = (int32_t)(p.tiles > INT32_MAX ? INT32_MAX : p.tiles);
  out[3] = p.units;
  return TFL_OK;
}

int tfl_glu_status(tfl_glu* g, tfl_stream stream) {
  g_err.clear();
  if (!g) return fail(TFL_ERR_INVALID_ARG, "handle is NULL");
  TFL_CUDA(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)), "cudaStreamSynchronize");
  int v = 0;
  TFL_CUDA(cudaMemcpy(&v, g->status, sizeof(int), cudaMemcpyDeviceToHost), "status read");
  if (v) TFL_CUDA(cudaMemset(g->status, 0, sizeof(int)), "status clear");
  if (v & TFL_DEV_TIMEOUT) return fail(TFL_ERR_DEVICE_TIMEOUT, "a device-side wait ran out of time");
  return TFL_OK;
}

void tfl_glu_destroy(tfl_glu* g) {
  if (!g) return;
  release(g->device, g->status);
  delete g;
}

}  // extern "C"
