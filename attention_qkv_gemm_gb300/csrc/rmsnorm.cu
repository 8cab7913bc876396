// rmsnorm.cu -- root-mean-square norm with the residual's addition, forward and backward.
//
//   s = x + res,  r = 1 / sqrt(mean(s^2) + eps),  y = s r gamma
// and, with a = dy gamma, the gradient of s and gamma:
//   ds = dres + r a - s r^3 mean(a s),   dgamma = sum over rows of dy s r.
//
// Every value is read once and written once: bandwidth bounds it, so a row lives in the
// registers of TPR threads between its loads and its stores, TPR the smallest power of two
// that holds it at NV vectors of 8 a thread (one warp a row up to 8 * 32 * NV values, so the
// common widths need no block barrier).  Sums are fp32: a thread's own elements in order, then
// a butterfly, so a row's result does not depend on the other rows.
//
// The e4m3 form divides a row by its scale = max|y| / 448 (448 is e4m3's largest value) and
// rounds once; max|y| = r max|s gamma| comes from the same pass as the sum of squares.
//
// Widths that 8 does not divide, unaligned buffers and rows too long for registers take the
// element-wise kernels at the end: two passes over a row, the second from L1 / L2.
#include "ops.h"
#include "ptx.cuh"
#include "xpose.cuh"

namespace tfl {

namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kMinAmax = 7.888609052210118e-31f;  // 2^-100: the least row maximum a scale is taken from

struct E4m3 {
  uint8_t v;
};

// Maximum that keeps a NaN (fmaxf drops it): a row holding one gets a NaN scale.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// ---- 8 consecutive values <-> fp32
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const __half* p, float* v) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* v) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__half* p, const float* v) {
  uint4 o;
  pack_f16<8>(v, &o, false);
  *reinterpret_cast<uint4*>(p) = o;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  uint4 o;
  pack_bf16<8>(v, &o);
  *reinterpret_cast<uint4*>(p) = o;
}
__device__ __forceinline__ void store8(E4m3* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
}

// Sum (or maximum) over the `tpr` threads of this thread's row group; `red` holds one float a
// warp and value.  Groups of up to a warp stay inside it.
template <int N>
__device__ __forceinline__ void group_reduce(float* v, int tpr, bool last_is_max, float* red) {
  const int lanes = tpr < 32 ? tpr : 32;
#pragma unroll 1
  for (int o = lanes >> 1; o; o >>= 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float t = __shfl_xor_sync(0xffffffffu, v[k], o);
      v[k] = (last_is_max && k == N - 1) ? max_nan(v[k], t) : v[k] + t;
    }
  }
  if (tpr <= 32) return;
  const int warp = threadIdx.x >> 5, nw = tpr >> 5, w0 = warp & ~(nw - 1);
  __syncthreads();  // the previous row's values have been read
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) red[k * 32 + warp] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = red[k * 32 + w0];
  for (int w = 1; w < nw; ++w) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float t = red[k * 32 + w0 + w];
      v[k] = (last_is_max && k == N - 1) ? max_nan(v[k], t) : v[k] + t;
    }
  }
}

template <class X, class R, class Y, int NV>
__global__ void __launch_bounds__(1024) rms_forward_kernel(const RmsArgs a) {
  constexpr bool Q = sizeof(Y) == 1;
  __shared__ float red[64];
  grid_launch_dependents();
  grid_wait_prior();
  const int tpr = a.tpr, t = threadIdx.x & (tpr - 1);
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < a.rows;  // the whole block meets at group_reduce's barriers
  const int nvec = a.D >> 3;
  const size_t base = (size_t)row * a.D;
  float s[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = t + j * tpr;
    if (live && c < nvec) {
      load8(static_cast<const X*>(a.x) + base + c * 8, s[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[j][i] = 0.f;
    }
  }
  if (a.res) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = t + j * tpr;
      if (live && c < nvec) {
        float r[8];
        load8(static_cast<const R*>(a.res) + base + c * 8, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j][i] += r[i];
      }
    }
  }
  float v[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[0] = fmaf(s[j][i], s[j][i], v[0]);
  }
  if (a.res_out) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = t + j * tpr;
      if (live && c < nvec) store8(static_cast<R*>(a.res_out) + base + c * 8, s[j]);
    }
  }
  // gamma goes into the row now: y = r (s gamma), and max|y| needs the product
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = t + j * tpr;
    if (live && c < nvec) {
      float g[8];
      load8(a.gamma + c * 8, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[j][i] *= g[i];
        if (Q) v[1] = max_nan(v[1], fabsf(s[j][i]));
      }
    }
  }
  group_reduce<Q ? 2 : 1>(v, tpr, Q, red);
  float r = rsqrtf(v[0] * a.inv_d + a.eps);
  if constexpr (Q) {
    const float amax = max_nan(v[1] * r, kMinAmax);
    if (live && t == 0) a.y_scale[row] = amax / kE4m3Max;
    r *= kE4m3Max / amax;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = t + j * tpr;
    if (live && c < nvec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[j][i] *= r;
      store8(static_cast<Y*>(a.y) + base + c * 8, s[j]);
    }
  }
}

// Backward.  A block keeps its row groups over all their rows (grid-stride), so each thread
// sums dgamma of its own columns in registers; the groups of a block are joined in shared
// memory and every block writes one row of partial sums, which rms_dgamma_kernel adds in
// block order: the result depends on the sizes and the SM count only, not on timing.
template <class X, class R, int NV>
__global__ void __launch_bounds__(512) rms_backward_kernel(const RmsGradArgs a) {
  __shared__ float red[64];
  extern __shared__ float part[];  // [groups][D] when the block has more than one group
  grid_launch_dependents();
  grid_wait_prior();
  const int tpr = a.tpr, t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = blockDim.x / tpr;
  const int nvec = a.D >> 3;
  float dg[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[j][i] = 0.f;
  for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < a.rows; row0 += (int64_t)gridDim.x * groups) {
    const int64_t row = row0 + group;
    const bool live = row < a.rows;
    const size_t base = (size_t)row * a.D;
    float s[NV][8], dy[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = t + j * tpr;
      if (live && c < nvec) {
        load8(static_cast<const R*>(a.sum) + base + c * 8, s[j]);
        load8(static_cast<const X*>(a.dy) + base + c * 8, dy[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j][i] = dy[j][i] = 0.f;
      }
    }
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = t + j * tpr;
      if (c < nvec) {
        float g[8];
        load8(a.gamma + c * 8, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[0] = fmaf(s[j][i], s[j][i], v[0]);
          v[1] = fmaf(dy[j][i] * g[i], s[j][i], v[1]);
        }
      }
    }
    group_reduce<2>(v, tpr, false, red);
    const float r = rsqrtf(v[0] * a.inv_d + a.eps);
    const float k = r * r * r * (v[1] * a.inv_d);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = t + j * tpr;
      if (live && c < nvec) {
        float g[8], o[8];
        load8(a.gamma + c * 8, g);
        if (a.dres) {
          load8(static_cast<const R*>(a.dres) + base + c * 8, o);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dg[j][i] = fmaf(dy[j][i] * r, s[j][i], dg[j][i]);
          o[i] += fmaf(r * g[i], dy[j][i], -s[j][i] * k);
        }
        if (a.dsum) store8(static_cast<R*>(a.dsum) + base + c * 8, o);
        if (a.dx) store8(static_cast<X*>(a.dx) + base + c * 8, o);
      }
    }
  }
  float* out = a.partial + (size_t)blockIdx.x * a.D;
  if (groups == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = t + j * tpr;
      if (c < nvec) store8(out + c * 8, dg[j]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = t + j * tpr;
    if (c < nvec) store8(part + (size_t)group * a.D + c * 8, dg[j]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
    float v = 0.f;
    for (int g = 0; g < groups; ++g) v += part[(size_t)g * a.D + c];
    out[c] = v;
  }
}

// dgamma[c] = sum over the blocks' partial rows: 32 columns a block, 32 threads a column.
__global__ void __launch_bounds__(1024) rms_dgamma_kernel(const float* partial, int n, int D, float* dgamma) {
  __shared__ float red[32][33];
  grid_launch_dependents();
  grid_wait_prior();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (c < D)
    for (int i = threadIdx.y; i < n; i += 32) v += partial[(size_t)i * D + c];
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = red[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int col = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && col < D) dgamma[col] = v;
}

// ---- element-wise form: any width and element-aligned buffers, one block a row
__device__ __forceinline__ float load1(const void* p, int type, size_t i) {
  if (type == TFL_F32) return static_cast<const float*>(p)[i];
  if (type == TFL_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store1(void* p, int type, size_t i, float v) {
  if (type == TFL_F32)
    static_cast<float*>(p)[i] = v;
  else if (type == TFL_F16)
    static_cast<__half*>(p)[i] = __float2half_rn(v);
  else if (type == TFL_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<uint8_t*>(p)[i] = (uint8_t)e4m3x2(v, 0.f);
}

__global__ void __launch_bounds__(256) rms_forward_any_kernel(const RmsArgs a) {
  __shared__ float red[64];
  grid_launch_dependents();
  grid_wait_prior();
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const size_t base = (size_t)row * a.D;
    float v[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < a.D; c += 256) {
      float s = load1(a.x, a.x_type, base + c);
      if (a.res) s += load1(a.res, a.res_type, base + c);
      v[0] = fmaf(s, s, v[0]);
      v[1] = max_nan(v[1], fabsf(s * a.gamma[c]));
    }
    group_reduce<2>(v, 256, true, red);
    float r = rsqrtf(v[0] * a.inv_d + a.eps);
    if (a.y_type == TFL_E4M3) {
      const float amax = max_nan(v[1] * r, kMinAmax);
      if (threadIdx.x == 0) a.y_scale[row] = amax / kE4m3Max;
      r *= kE4m3Max / amax;
    }
    for (int c = threadIdx.x; c < a.D; c += 256) {
      float s = load1(a.x, a.x_type, base + c);
      if (a.res) s += load1(a.res, a.res_type, base + c);
      if (a.res_out) store1(a.res_out, a.res_type, base + c, s);
      store1(a.y, a.y_type, base + c, s * a.gamma[c] * r);
    }
  }
}

// The thread that owns column c in every row of the block also adds up its dgamma, in the
// block's row of partial sums.
__global__ void __launch_bounds__(256) rms_backward_any_kernel(const RmsGradArgs a) {
  __shared__ float red[64];
  grid_launch_dependents();
  grid_wait_prior();
  float* part = a.partial + (size_t)blockIdx.x * a.D;
  for (int c = threadIdx.x; c < a.D; c += 256) part[c] = 0.f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const size_t base = (size_t)row * a.D;
    float v[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < a.D; c += 256) {
      const float s = load1(a.sum, a.res_type, base + c);
      v[0] = fmaf(s, s, v[0]);
      v[1] = fmaf(load1(a.dy, a.x_type, base + c) * a.gamma[c], s, v[1]);
    }
    group_reduce<2>(v, 256, false, red);
    const float r = rsqrtf(v[0] * a.inv_d + a.eps);
    const float k = r * r * r * (v[1] * a.inv_d);
    for (int c = threadIdx.x; c < a.D; c += 256) {
      const float s = load1(a.sum, a.res_type, base + c), dy = load1(a.dy, a.x_type, base + c);
      float o = a.dres ? load1(a.dres, a.res_type, base + c) : 0.f;
      o += fmaf(r * a.gamma[c], dy, -s * k);
      part[c] = fmaf(dy * r, s, part[c]);
      if (a.dsum) store1(a.dsum, a.res_type, base + c, o);
      if (a.dx) store1(a.dx, a.x_type, base + c, o);
    }
  }
}

int pow2_at_least(int v) {
  int p = 1;
  while (p < v) p <<= 1;
  return p;
}

template <class X, class R, class Y>
cudaError_t forward_vec(RmsArgs a, cudaStream_t s) {
  const int nvec = a.D / 8;
  const int nv = nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4;
  a.tpr = pow2_at_least((nvec + nv - 1) / nv);
  const int threads = a.tpr > 256 ? a.tpr : 256;
  const int64_t per = threads / a.tpr;
  const dim3 grid((unsigned)((a.rows + per - 1) / per));
  if (nv == 1) return launch_dependent(rms_forward_kernel<X, R, Y, 1>, grid, threads, 0, s, a);
  if (nv == 2) return launch_dependent(rms_forward_kernel<X, R, Y, 2>, grid, threads, 0, s, a);
  return launch_dependent(rms_forward_kernel<X, R, Y, 4>, grid, threads, 0, s, a);
}

template <class X, class R>
cudaError_t forward_y(const RmsArgs& a, cudaStream_t s) {
  if (a.y_type == TFL_E4M3) return forward_vec<X, R, E4m3>(a, s);
  if constexpr (sizeof(X) == 4) {
    if (a.y_type == TFL_F16) return forward_vec<X, R, __half>(a, s);
    if (a.y_type == TFL_BF16) return forward_vec<X, R, __nv_bfloat16>(a, s);
  }
  return forward_vec<X, R, X>(a, s);
}

template <class X, class R>
cudaError_t backward_vec(RmsGradArgs a, cudaStream_t s) {
  const int nvec = a.D / 8;
  const int nv = nvec <= 32 ? 1 : nvec <= 1024 ? 2 : 4;
  a.tpr = pow2_at_least((nvec + nv - 1) / nv);
  const int threads = a.tpr > 256 ? a.tpr : 256, groups = threads / a.tpr;
  const int64_t need = (a.rows + groups - 1) / groups;
  const int grid = (int)(need < a.blocks ? need : a.blocks);
  const size_t smem = groups > 1 ? (size_t)groups * a.D * sizeof(float) : 0;  // at most 16 KB
  cudaError_t e;
  if (nv == 1)
    e = launch_dependent(rms_backward_kernel<X, R, 1>, grid, threads, smem, s, a);
  else if (nv == 2)
    e = launch_dependent(rms_backward_kernel<X, R, 2>, grid, threads, smem, s, a);
  else
    e = launch_dependent(rms_backward_kernel<X, R, 4>, grid, threads, smem, s, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(rms_dgamma_kernel, (a.D + 31) / 32, dim3(32, 32), 0, s, (const float*)a.partial, grid, a.D,
                          a.dgamma);
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

cudaError_t launch_rms_forward(const RmsArgs& a, int num_sms, cudaStream_t s) {
  const bool vec = a.D % 8 == 0 && a.D <= kRmsMaxRegisterRow && aligned(a.x, 16) && aligned(a.res, 16) &&
                   aligned(a.gamma, 16) && aligned(a.res_out, 16) && aligned(a.y, a.y_type == TFL_E4M3 ? 8 : 16);
  if (!vec) {
    const int64_t most = (int64_t)num_sms * 8;
    return launch_dependent(rms_forward_any_kernel, (unsigned)(a.rows < most ? a.rows : most), 256, 0, s, a);
  }
  if (a.x_type == TFL_F32) return forward_y<float, float>(a, s);
  if (a.x_type == TFL_F16)
    return a.res_type == TFL_F32 ? forward_y<__half, float>(a, s) : forward_y<__half, __half>(a, s);
  return a.res_type == TFL_F32 ? forward_y<__nv_bfloat16, float>(a, s)
                               : forward_y<__nv_bfloat16, __nv_bfloat16>(a, s);
}

cudaError_t launch_rms_backward(const RmsGradArgs& a, cudaStream_t s) {
  const bool vec = a.D % 8 == 0 && a.D <= kRmsMaxRegisterRow / 2 && aligned(a.sum, 16) && aligned(a.gamma, 16) &&
                   aligned(a.dy, 16) && aligned(a.dres, 16) && aligned(a.dx, 16) && aligned(a.dsum, 16);
  if (!vec) {
    const int grid = (int)(a.rows < a.blocks ? a.rows : a.blocks);
    cudaError_t e = launch_dependent(rms_backward_any_kernel, grid, 256, 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_dependent(rms_dgamma_kernel, (a.D + 31) / 32, dim3(32, 32), 0, s, (const float*)a.partial, grid,
                            a.D, a.dgamma);
  }
  if (a.x_type == TFL_F32) return backward_vec<float, float>(a, s);
  if (a.x_type == TFL_F16)
    return a.res_type == TFL_F32 ? backward_vec<__half, float>(a, s)
                                 : backward_vec<__half, __half>(a, s);
  return a.res_type == TFL_F32 ? backward_vec<__nv_bfloat16, float>(a, s)
                               : backward_vec<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // namespace tfl
