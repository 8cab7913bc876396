// rowops.cuh -- what the row norms share (rmsnorm.cu, layernorm.cu): eight values of a row a thread at a
// time, sums over the threads that hold a row, columns' partial sums of the backward passes.
#pragma once
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

// ---- 8 consecutive values as loaded, and as fp32
template <class T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
template <class T>
__device__ __forceinline__ void load_raw(const T* p, Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4*>(p)[i];
}
template <class T>
__device__ __forceinline__ void zero_raw(Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.w[i] = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void widen(const Raw8<float>& r, float* v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[4 * i] = __uint_as_float(r.w[i].x), v[4 * i + 1] = __uint_as_float(r.w[i].y);
    v[4 * i + 2] = __uint_as_float(r.w[i].z), v[4 * i + 3] = __uint_as_float(r.w[i].w);
  }
}
__device__ __forceinline__ void widen(const Raw8<__half>& r, float* v) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void widen(const Raw8<__nv_bfloat16>& r, float* v) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <class T>
__device__ __forceinline__ void load8(const T* p, float* v) {
  Raw8<T> r;
  load_raw(p, r);
  widen(r, v);
}
// The same as four packed pairs.
template <class T>
__device__ __forceinline__ void widen2(const Raw8<T>& r, uint64_t* v) {
  float f[8];
  widen(r, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2_pack(f[2 * i], f[2 * i + 1]);
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

// Brings `bytes` from p on into L2, one 128-byte line a thread and turn (the last line only if a
// multiple of 128 bytes from p lies in it).
__device__ __forceinline__ void lines_to_l2(const void* p, int bytes, int t, int threads) {
  for (int o = t * 128; o < bytes; o += threads * 128) prefetch_l2(static_cast<const uint8_t*>(p) + o);
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

// Both sums of a row, for a group that loops over its rows on its own: groups wider than a warp
// meet at a named barrier of their own, once a row (the buffers alternate).  Inside a warp the two
// sums are folded into one first: half of the lanes go on with each.
template <int WARPS = 16>  // of the widest group
__device__ __forceinline__ void row_sums(float& a, float& b, int tpr, int group, int parity, float2 (*red)[32]) {
  const int lane = threadIdx.x & 31;
  const int lanes = tpr < 32 ? tpr : 32;
  if (lanes > 1) {
    const int h = lanes >> 1;
    const bool upper = (lane & h) != 0;
    float v = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, h);
#pragma unroll
    for (int o = 8; o; o >>= 1)
      if (o < h) v += __shfl_xor_sync(0xffffffffu, v, o);
    const float w = __shfl_xor_sync(0xffffffffu, v, h);
    a = upper ? w : v;
    b = upper ? v : w;
  }
  if (tpr <= 32) return;
  const int warp = threadIdx.x >> 5, nw = tpr >> 5;
  if (lane == 0) red[parity][warp] = make_float2(a, b);
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
  const float2 p = red[parity][group * nw + (lane & (nw - 1))];
  a = p.x;
  b = p.y;
#pragma unroll
  for (int o = WARPS / 2; o; o >>= 1) {
    if (o < nw) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
  }
}

// ---- single values of any type
__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(__half v) { return __half2float(v); }
__device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void assign(float& d, float v) { d = v; }
__device__ __forceinline__ void assign(__half& d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void assign(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
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

// out[c] = sum over n partial rows (`pitch` values apart) of column c < cols; columns from D on go to out2.
// C columns a block, Y threads a column with two loads at once, joined in a fixed order.  8 x 128 for the
// partial rows of a whole GPU (enough blocks for it at the common widths), 32 x 8 for those of a few blocks.
template <int C, int Y>
__global__ void __launch_bounds__(C * Y) column_sums_kernel(const float* partial, int n, int pitch, int cols, int D,
                                                            float* out, float* out2) {
  __shared__ float red[Y][C + 1];
  grid_launch_dependents();
  grid_wait_prior();
  const int x = threadIdx.x % C, y = threadIdx.x / C, c = blockIdx.x * C + x;
  auto put = [&](int col, float sum) {
    if (col < D)
      out[col] = sum;
    else
      out2[col - D] = sum;
  };
  float v = 0.f;
  if (c < cols) {
#pragma unroll 2
    for (int i = y; i < n; i += Y) v += partial[(size_t)i * pitch + c];
  }
  red[y][x] = v;
  __syncthreads();
  if constexpr (Y >= 32) {  // warp w < C adds up column w
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (w >= C) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < Y / 32; ++i) v += red[lane + 32 * i][w];
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && blockIdx.x * C + w < cols) put(blockIdx.x * C + w, v);
  } else if (y == 0 && c < cols) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < Y; ++i) v += red[i][x];
    put(c, v);
  }
}

inline cudaError_t launch_column_sums(const float* partial, int n, int pitch, int cols, int D, float* out, float* out2,
                                      cudaStream_t s) {
  if (n <= 64)
    return launch_dependent(column_sums_kernel<32, 8>, (cols + 31) / 32, 256, 0, s, partial, n, pitch, cols, D, out, out2);
  return launch_dependent(column_sums_kernel<8, 128>, (cols + 7) / 8, 1024, 0, s, partial, n, pitch, cols, D, out, out2);
}

inline int pow2_at_least(int v) {
  int p = 1;
  while (p < v) p <<= 1;
  return p;
}

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// f(X(), R()) for the C++ types of a call's x and residual.
template <class F>
cudaError_t with_types(int x_type, int res_type, F f) {
  if (x_type == TFL_F32) return f(float(), float());
  if (x_type == TFL_F16) return res_type == TFL_F32 ? f(__half(), float()) : f(__half(), __half());
  return res_type == TFL_F32 ? f(__nv_bfloat16(), float()) : f(__nv_bfloat16(), __nv_bfloat16());
}

}  // namespace

}  // namespace tfl
