// rmsnorm.cu -- root-mean-square norm with the residual's addition, forward and backward.
//
//   s = x + res,  r = 1 / sqrt(mean(s^2) + eps),  y = s r gamma
// and, with a = dy gamma, the gradient of s and gamma:
//   ds = dres + r a - s r^3 mean(a s),   dgamma = sum over rows of dy s r
// with t = s r as dres + r a - t (r (r mean(a s))) and the sum of dy t: t is at most sqrt(d) and
// r mean(a s) of the size of a, where r^3 alone overflows from r = 7e12 on (rows of size 1e-13, eps 0).
//
// Every value is read once and written once: bandwidth bounds it, so a row lives in the
// registers of TPR threads between its loads and its stores, TPR the smallest power of two
// that holds it at NV vectors of 8 a thread (one warp a row up to 8 * 32 * NV values, so the
// common widths need no block barrier).  Sums are fp32: a thread's own elements in order, then
// a butterfly, so a row's result does not depend on the other rows.
//
// Measured: 100000 x 1024 bf16 to e4m3 106 us (the copy bandwidth), 8192 x 1024 fp16 with an fp32
// residual 18.3 us (0.81 of it), one row 2.7 us in a graph; backward 20011 x 4096 fp16 110 us (0.88),
// 8192 x 1024 bf16 / fp32 24.9 us (0.80, 3.5 us of it the second launch for dgamma).
//
// The e4m3 form divides a row by its scale = max|y| / 448 (448 is e4m3's largest value) and
// rounds once; max|y| = r max|s gamma| comes from the same pass as the sum of squares.  y is formed
// before 448 / max|y| is applied: their product alone overflows for a row of zeros with a small eps
// (r = 1e6 times 448 2^100).
//
// Widths that 8 does not divide, unaligned buffers and rows too long for registers take the
// element-wise kernels at the end.
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
__device__ __forceinline__ void load_gamma(const float* p, float* v) {  // read by every row: from L1
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void gamma2(const float* p, uint64_t* v) {
  float f[8];
  load_gamma(p, f);
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
  // While this row is reduced, the rows of the block that will take this one's place start on
  // their way to L2 (100000 x 1024 bf16 to e4m3: 130 -> 106 us).
  const int64_t later = row + a.ahead;
  if (later < a.rows) {
    lines_to_l2(static_cast<const X*>(a.x) + (size_t)later * a.D, a.D * (int)sizeof(X), t, tpr);
    if (a.res) lines_to_l2(static_cast<const R*>(a.res) + (size_t)later * a.D, a.D * (int)sizeof(R), t, tpr);
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
      load_gamma(a.gamma + c * 8, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[j][i] *= g[i];
        if (Q) v[1] = max_nan(v[1], fabsf(s[j][i]));
      }
    }
  }
  group_reduce<Q ? 2 : 1>(v, tpr, Q, red);
  const float r = rsqrtf(v[0] * a.inv_d + a.eps);
  float to8 = 1.0f;
  if constexpr (Q) {
    const float amax = max_nan(v[1] * r, kMinAmax);
    if (live && t == 0) a.y_scale[row] = amax / kE4m3Max;
    to8 = kE4m3Max / amax;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = t + j * tpr;
    if (live && c < nvec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[j][i] = Q ? s[j][i] * r * to8 : s[j][i] * r;
      store8(static_cast<Y*>(a.y) + base + c * 8, s[j]);
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

// Backward.  A row group keeps its columns over all its rows, so each thread holds gamma and sums
// dgamma of its own columns in registers; the groups of a block are joined in shared memory and
// every block writes one row of partial sums, which rms_dgamma_kernel adds in block order: the
// result depends on the sizes and the SM count only, not on timing.
//
// Three streams in and one or two out bound it, so loads have to stay in flight while a row is
// reduced and written: the next row is loaded, as stored, before the current one is worked on
// (20011 x 4096 fp16 229 -> 150 us).  Instructions come next: packed fp32 pairs, the two sums folded
// into one butterfly, pointers carried along (150 -> 110 us).  A ring of rows in shared memory filled
// by cp.async holds more bytes in flight but was slower: 161 us where this form took 150, and 39
// against 28 us at 8192 x 1024.
template <class X, class R, int NV, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) rms_backward_kernel(const RmsGradArgs a) {
  constexpr bool AHEAD = NV == 1 || (NV == 2 && sizeof(R) == 2);  // room for the next row
  constexpr bool KEEP = NV == 1;                                  // room for gamma
  __shared__ float2 red[2][32];
  extern __shared__ float part[];  // [groups][D + 4] when the block has more than one group
  grid_launch_dependents();
  grid_wait_prior();
  const int tpr = a.tpr, t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = THREADS / tpr;
  const int nvec = a.D >> 3, rows = (int)a.rows;
  const int stride = gridDim.x * groups, first = blockIdx.x * groups + group;
  bool in[NV];  // vectors of this thread that exist
  uint64_t dg[NV][4], gk[KEEP ? NV : 1][4];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    in[j] = t + j * tpr < nvec;
#pragma unroll
    for (int i = 0; i < 4; ++i) dg[j][i] = 0;  // two zeros
    if constexpr (KEEP) {
      if (in[j]) {
        gamma2(a.gamma + (t + j * tpr) * 8, gk[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) gk[j][i] = 0;
      }
    }
  }
  // this thread's first vector of the row to load next and of the row to write next
  const size_t step = (size_t)stride * a.D, begin = (size_t)first * a.D + t * 8;
  const R* sp = static_cast<const R*>(a.sum) + begin;
  const X* yp = static_cast<const X*>(a.dy) + begin;
  const R* ep = a.dres ? static_cast<const R*>(a.dres) + begin : nullptr;
  const R* ep_late = ep;
  R* dsum = a.dsum ? static_cast<R*>(a.dsum) + begin : nullptr;
  X* dx = a.dx ? static_cast<X*>(a.dx) + begin : nullptr;
  const int jump = tpr * 8;  // from one vector of a thread to its next
  Raw8<R> s1[NV], e1[NV], e[NV];
  Raw8<X> y1[NV];
  auto fetch = [&](bool live) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (live && in[j]) {
        load_raw(sp + j * jump, s1[j]);
        load_raw(yp + j * jump, y1[j]);
        if (AHEAD && ep) load_raw(ep + j * jump, e1[j]);
      } else {
        zero_raw(s1[j]);
        zero_raw(y1[j]);
      }
    }
    sp += step;
    yp += step;
    if (AHEAD && ep) ep += step;
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) zero_raw(e1[j]);
  int parity = 0;
  if (AHEAD) fetch(first < rows);
  // groups that share a warp go through the same number of rows (its shuffles need all lanes)
  const int lead = tpr < 32 ? first / (32 / tpr) * (32 / tpr) : first;  // of the warp's groups
  int64_t next = first;
  for (int64_t at = lead; at < rows; at += stride) {
    const bool live = next < rows;
    next += stride;
    if (!AHEAD) fetch(live);
    uint64_t s[NV][4], y[NV][4];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      widen2(s1[j], s[j]);
      widen2(y1[j], y[j]);
      e[j] = e1[j];
    }
    if (AHEAD) fetch(next < rows);
    uint64_t ss = 0, as = 0;  // two zeros each
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint64_t g[4] = {0, 0, 0, 0};
      if (!KEEP && in[j]) gamma2(a.gamma + (t + j * tpr) * 8, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ss = f2_fma(s[j][i], s[j][i], ss);
        as = f2_fma(f2_mul(y[j][i], KEEP ? gk[KEEP ? j : 0][i] : g[i]), s[j][i], as);
      }
    }
    float v0, v1, hi;
    f2_unpack(ss, v0, hi);
    v0 += hi;
    f2_unpack(as, v1, hi);
    v1 += hi;
    row_sums(v0, v1, tpr, group, parity, red);
    parity ^= 1;
    const float r = rsqrtf(v0 * a.inv_d + a.eps);
    const uint64_t r2 = f2_splat(r), k2 = f2_splat(-(r * (r * (v1 * a.inv_d))));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (live && in[j]) {
        uint64_t g[4], o[4];
        if constexpr (!KEEP) gamma2(a.gamma + (t + j * tpr) * 8, g);
        if (!AHEAD && ep_late) load_raw(ep_late + j * jump, e[j]);
        widen2(e[j], o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t t2 = f2_mul(s[j][i], r2);
          dg[j][i] = f2_fma(y[j][i], t2, dg[j][i]);
          o[i] = f2_fma(y[j][i], f2_mul(KEEP ? gk[KEEP ? j : 0][i] : g[i], r2), f2_fma(t2, k2, o[i]));
        }
        float of[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_unpack(o[i], of[2 * i], of[2 * i + 1]);
        if (dsum) store8(dsum + j * jump, of);
        if (dx) store8(dx + j * jump, of);
      }
    }
    if (dsum) dsum += step;
    if (dx) dx += step;
    if (!AHEAD && ep_late) ep_late += step;
  }
  float dgf[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(dg[j][i], dgf[j][2 * i], dgf[j][2 * i + 1]);
  float* out = a.partial + (size_t)blockIdx.x * a.D;
  if (groups == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = t + j * tpr;
      if (c < nvec) store8(out + c * 8, dgf[j]);
    }
    return;
  }
  const int pitch = a.D + 4;  // columns of 8 rows in a row lie in different banks
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = t + j * tpr;
    if (c < nvec) store8(part + group * pitch + c * 8, dgf[j]);
  }
  __syncthreads();
  if (groups > 32) {  // short rows: a warp a column (in turn, 768 rows would be a long chain of additions)
    for (int c = threadIdx.x >> 5; c < a.D; c += THREADS / 32) {
      float v = 0.f;
      for (int g = threadIdx.x & 31; g < groups; g += 32) v += part[g * pitch + c];
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if ((threadIdx.x & 31) == 0) out[c] = v;
    }
    return;
  }
  for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
    float v = 0.f;
    for (int g = 0; g < groups; ++g) v += part[g * pitch + c];
    out[c] = v;
  }
}

// dgamma[c] = sum over the blocks' partial rows: C columns a block, Y threads a column with two
// loads at once, joined in a fixed order.  8 x 128 for the partial rows of a whole GPU (enough blocks
// for it at the common widths), 32 x 8 for those of a few blocks.
template <int C, int Y>
__global__ void __launch_bounds__(C * Y) rms_dgamma_kernel(const float* partial, int n, int D, float* dgamma) {
  __shared__ float red[Y][C + 1];
  grid_launch_dependents();
  grid_wait_prior();
  const int x = threadIdx.x % C, y = threadIdx.x / C, c = blockIdx.x * C + x;
  float v = 0.f;
  if (c < D) {
#pragma unroll 2
    for (int i = y; i < n; i += Y) v += partial[(size_t)i * D + c];
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
    if (lane == 0 && blockIdx.x * C + w < D) dgamma[blockIdx.x * C + w] = v;
  } else if (y == 0 && c < D) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < Y; ++i) v += red[i][x];
    dgamma[c] = v;
  }
}

// ---- element-wise forms: any width and element-aligned buffers, one block a row
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

// Rows of up to T NE values: T threads with NE each in registers, all loads at once (1531 x 1001 fp32
// 5.2 us; the two passes below take 8.5 us).
template <class X, class R, int T, int NE>
__global__ void __launch_bounds__(T) rms_forward_values_kernel(const RmsArgs a) {
  __shared__ float red[64];
  grid_launch_dependents();
  grid_wait_prior();
  const size_t base = (size_t)blockIdx.x * a.D + threadIdx.x;
  const X* x = static_cast<const X*>(a.x) + base;
  const R* res = a.res ? static_cast<const R*>(a.res) + base : nullptr;
  float s[NE], v[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < NE; ++j) s[j] = (int)threadIdx.x + j * T < a.D ? value(x[j * T]) : 0.f;
  if (res) {
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if ((int)threadIdx.x + j * T < a.D) s[j] += value(res[j * T]);
  }
  const int64_t later = blockIdx.x + a.ahead;  // as in rms_forward_kernel
  if (later < a.rows) {
    lines_to_l2(static_cast<const X*>(a.x) + (size_t)later * a.D, a.D * (int)sizeof(X), threadIdx.x, T);
    if (a.res) lines_to_l2(static_cast<const R*>(a.res) + (size_t)later * a.D, a.D * (int)sizeof(R), threadIdx.x, T);
  }
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int c = threadIdx.x + j * T;
    v[0] = fmaf(s[j], s[j], v[0]);
    if (c < a.D) {
      if (a.res_out) assign(static_cast<R*>(a.res_out)[base + j * T], s[j]);
      s[j] *= __ldg(a.gamma + c);
      v[1] = max_nan(v[1], fabsf(s[j]));
    }
  }
  group_reduce<2>(v, T, true, red);
  const float r = rsqrtf(v[0] * a.inv_d + a.eps);
  float to8 = 1.0f;
  if (a.y_type == TFL_E4M3) {
    const float amax = max_nan(v[1] * r, kMinAmax);
    if (threadIdx.x == 0) a.y_scale[blockIdx.x] = amax / kE4m3Max;
    to8 = kE4m3Max / amax;
  }
#pragma unroll
  for (int j = 0; j < NE; ++j)
    if ((int)threadIdx.x + j * T < a.D) store1(a.y, a.y_type, base + j * T, s[j] * r * to8);
}

// Groups of G threads take rows of up to G NE values, all groups of a block together T threads.  The
// next row is on its way while one is worked on, without its residual gradient where registers are
// short (NE = 8), and gamma then comes from L1.  Loads of single values bound it: 9807 x 103 fp16 takes
// 7.3 us (24.5 with a whole block a row), 3000 x 3333 bf16 30 us (floor 12), 1115 x 8190 fp32 44 us (22).
template <class X, class R, int T, int G, int NE>
__global__ void __launch_bounds__(T, 1024 / T) rms_backward_values_kernel(const RmsGradArgs a) {
  constexpr bool ROOM = NE <= 4, ROOM_E = NE <= 6;
  constexpr int GROUPS = T / G;
  __shared__ float2 red[2][32];
  __shared__ float part[GROUPS > 1 ? T * NE : 1];
  grid_launch_dependents();
  grid_wait_prior();
  const int t = threadIdx.x % G, group = threadIdx.x / G, D = a.D;
  const int64_t stride = (int64_t)gridDim.x * GROUPS;
  float dg[NE], gk[ROOM ? NE : 1];
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    dg[j] = 0.f;
    if constexpr (ROOM) gk[j] = t + j * G < D ? __ldg(a.gamma + t + j * G) : 0.f;
  }
  auto gamma = [&](int j) { return ROOM ? gk[ROOM ? j : 0] : __ldg(a.gamma + t + j * G); };
  R s1[NE], e1[NE];
  X y1[NE];
  auto fetch_res = [&](int64_t row) {
    const R* p = static_cast<const R*>(a.dres) + (size_t)row * D + t;
#pragma unroll
    for (int j = 0; j < NE; ++j) e1[j] = a.dres && row < a.rows && t + j * G < D ? p[j * G] : R(0.f);
  };
  auto fetch = [&](int64_t row) {
    const R* p = static_cast<const R*>(a.sum) + (size_t)row * D + t;
    const X* q = static_cast<const X*>(a.dy) + (size_t)row * D + t;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const bool in = row < a.rows && t + j * G < D;
      s1[j] = in ? p[j * G] : R(0.f);
      y1[j] = in ? q[j * G] : X(0.f);
    }
    if (ROOM_E) fetch_res(row);
  };
  int parity = 0;
  int64_t row = (int64_t)blockIdx.x * GROUPS + group;
  fetch(row);
  for (; row < a.rows; row += stride) {
    float s[NE], y[NE], e[NE];
    if (!ROOM_E) fetch_res(row);
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      s[j] = value(s1[j]);
      y[j] = value(y1[j]);
      if (ROOM_E) e[j] = value(e1[j]);
    }
    fetch(row + stride);
    float v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      v0 = fmaf(s[j], s[j], v0);
      if (t + j * G < D) v1 = fmaf(y[j] * gamma(j), s[j], v1);
    }
    row_sums<32>(v0, v1, G, group, parity, red);
    parity ^= 1;
    const float r = rsqrtf(v0 * a.inv_d + a.eps);
    const float k = r * (r * (v1 * a.inv_d));
    const size_t base = (size_t)row * D + t;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      if (t + j * G < D) {
        if (!ROOM_E) e[j] = value(e1[j]);
        const float sr = s[j] * r;
        dg[j] = fmaf(y[j], sr, dg[j]);
        const float o = fmaf(y[j], r * gamma(j), fmaf(-sr, k, e[j]));
        if (a.dsum) assign(static_cast<R*>(a.dsum)[base + j * G], o);
        if (a.dx) assign(static_cast<X*>(a.dx)[base + j * G], o);
      }
    }
  }
  float* out = a.partial + (size_t)blockIdx.x * D;
  if constexpr (GROUPS == 1) {
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if (t + j * G < D) out[t + j * G] = dg[j];
  } else {
#pragma unroll
    for (int j = 0; j < NE; ++j) part[(group * NE + j) * G + t] = dg[j];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += T) {
      float v = 0.f;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) v += part[g * NE * G + c];
      out[c] = v;
    }
  }
}

// Wider rows: two passes, the second from L1 / L2.
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
    const float r = rsqrtf(v[0] * a.inv_d + a.eps);
    float to8 = 1.0f;
    if (a.y_type == TFL_E4M3) {
      const float amax = max_nan(v[1] * r, kMinAmax);
      if (threadIdx.x == 0) a.y_scale[row] = amax / kE4m3Max;
      to8 = kE4m3Max / amax;
    }
    for (int c = threadIdx.x; c < a.D; c += 256) {
      float s = load1(a.x, a.x_type, base + c);
      if (a.res) s += load1(a.res, a.res_type, base + c);
      if (a.res_out) store1(a.res_out, a.res_type, base + c, s);
      store1(a.y, a.y_type, base + c, s * a.gamma[c] * r * to8);
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
    const float k = r * (r * (v[1] * a.inv_d));
    for (int c = threadIdx.x; c < a.D; c += 256) {
      const float s = load1(a.sum, a.res_type, base + c), dy = load1(a.dy, a.x_type, base + c);
      const float sr = s * r;
      const float o = fmaf(dy, r * a.gamma[c], fmaf(-sr, k, a.dres ? load1(a.dres, a.res_type, base + c) : 0.f));
      part[c] = fmaf(dy, sr, part[c]);
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
cudaError_t forward(RmsArgs a, int num_sms, cudaStream_t s) {
  const int nvec = a.D / 8;
  const int nv = nvec <= 32 ? 1 : nvec <= 64 ? 2 : 4;
  a.tpr = pow2_at_least((nvec + nv - 1) / nv);
  const int threads = a.tpr > 256 ? a.tpr : 256;
  const int64_t per = threads / a.tpr;
  const unsigned grid = (unsigned)((a.rows + per - 1) / per);
  a.ahead = per * num_sms * (1024 / threads);  // 64 registers a thread: 1024 threads an SM
  if (nv == 1) return launch_dependent(rms_forward_kernel<X, R, Y, 1>, grid, threads, 0, s, a);
  if (nv == 2) return launch_dependent(rms_forward_kernel<X, R, Y, 2>, grid, threads, 0, s, a);
  return launch_dependent(rms_forward_kernel<X, R, Y, 4>, grid, threads, 0, s, a);
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Blocks of a backward over groups of rows: what the GPU holds at once, and one alone for so few that
// a second launch would cost more than their turns; a lone block writes dgamma itself, where that takes
// the 16-byte stores of the partial rows.
int backward_blocks(RmsGradArgs& a, int64_t groups_of_rows, int at_once) {
  int64_t n = at_once < a.blocks ? at_once : a.blocks;
  if (groups_of_rows < n) n = groups_of_rows <= 3 ? 1 : groups_of_rows;
  if (n == 1 && aligned(a.dgamma, 16)) a.partial = a.dgamma;
  return (int)n;
}

cudaError_t add_partials(const RmsGradArgs& a, int n, cudaStream_t s) {
  if (a.partial == a.dgamma) return cudaSuccess;
  const float* p = a.partial;
  if (n <= 64) return launch_dependent(rms_dgamma_kernel<32, 8>, (a.D + 31) / 32, 256, 0, s, p, n, a.D, a.dgamma);
  return launch_dependent(rms_dgamma_kernel<8, 128>, (a.D + 7) / 8, 1024, 0, s, p, n, a.D, a.dgamma);
}

template <class X, class R, int NV, int THREADS, int BLOCKS>
cudaError_t backward_with(RmsGradArgs a, int num_sms, cudaStream_t s) {
  a.tpr = pow2_at_least((a.D / 8 + NV - 1) / NV);
  const int groups = THREADS / a.tpr;
  const int grid = backward_blocks(a, (a.rows + groups - 1) / groups, num_sms * BLOCKS);
  const size_t smem = groups > 1 ? (size_t)groups * (a.D + 4) * sizeof(float) : 0;  // at most 36 KB
  const cudaError_t e = launch_dependent(rms_backward_kernel<X, R, NV, THREADS, BLOCKS>, grid, THREADS, smem, s, a);
  return e == cudaSuccess ? add_partials(a, grid, s) : e;
}

template <class X, class R, int T, int G, int NE>
cudaError_t backward_values(RmsGradArgs a, int num_sms, cudaStream_t s) {
  const int grid = backward_blocks(a, (a.rows + T / G - 1) / (T / G), num_sms * (1024 / T));
  const cudaError_t e = launch_dependent(rms_backward_values_kernel<X, R, T, G, NE>, grid, T, 0, s, a);
  return e == cudaSuccess ? add_partials(a, grid, s) : e;
}

template <class X, class R>
cudaError_t backward(const RmsGradArgs& a, int num_sms, cudaStream_t s) {
  constexpr int WIDE = sizeof(R) == 4;  // fp32 rows take more registers, and carry more bytes a thread
  // one wide block an SM where the rows give each of them work (fewer partial rows to add: 8192 x 1024
  // fp16 18.0 -> 16.1 us then, 16.6 now), narrower ones to spread fewer rows over all SMs (500 x 2048: 6.5, wide 6.9)
  if (a.D <= 2048 && a.rows * pow2_at_least(a.D / 8) >= (int64_t)num_sms * 768)
    return backward_with<X, R, 1, WIDE ? 512 : 768, 1>(a, num_sms, s);
  if (a.D <= 2048) return backward_with<X, R, 1, 256, WIDE ? 2 : 3>(a, num_sms, s);
  if (a.D <= 4096) return WIDE ? backward_with<X, R, 1, 512, 1>(a, num_sms, s) : backward_with<X, R, 2, 256, 2>(a, num_sms, s);
  if (a.D <= 8192) return backward_with<X, R, 2, 512, 1>(a, num_sms, s);
  return backward_with<X, R, 4, 512, 1>(a, num_sms, s);
}

constexpr int kRmsMaxValues = 8192;  // widest row the element-wise kernels hold in registers

// f(X(), R()) for the C++ types of a call's x and residual.
template <class F>
cudaError_t with_types(int x_type, int res_type, F f) {
  if (x_type == TFL_F32) return f(float(), float());
  if (x_type == TFL_F16) return res_type == TFL_F32 ? f(__half(), float()) : f(__half(), __half());
  return res_type == TFL_F32 ? f(__nv_bfloat16(), float()) : f(__nv_bfloat16(), __nv_bfloat16());
}

}  // namespace

cudaError_t launch_rms_forward(const RmsArgs& a, int num_sms, cudaStream_t s) {
  const bool vec = a.D % 8 == 0 && a.D <= kRmsMaxRegisterRow && aligned(a.x, 16) && aligned(a.res, 16) &&
                   aligned(a.gamma, 16) && aligned(a.res_out, 16) && aligned(a.y, a.y_type == TFL_E4M3 ? 8 : 16);
  if (!vec && a.D <= kRmsMaxValues) {
    return with_types(a.x_type, a.res_type, [&](auto x, auto r) {
      using X = decltype(x);
      using R = decltype(r);
      const unsigned n = (unsigned)a.rows;
      RmsArgs b = a;
      b.ahead = a.D <= 4096 ? (int64_t)num_sms * 8 : a.rows;  // none for the widest: 9000 x 6001 139 us without, 180 with
      if (a.D <= 1024) return launch_dependent(rms_forward_values_kernel<X, R, 256, 4>, n, 256, 0, s, b);
      if (a.D <= 4096) return launch_dependent(rms_forward_values_kernel<X, R, 256, 16>, n, 256, 0, s, b);
      return launch_dependent(rms_forward_values_kernel<X, R, 1024, 8>, n, 1024, 0, s, b);
    });
  }
  if (!vec) {
    const int64_t most = (int64_t)num_sms * 8;
    return launch_dependent(rms_forward_any_kernel, (unsigned)(a.rows < most ? a.rows : most), 256, 0, s, a);
  }
  return with_types(a.x_type, a.res_type, [&](auto x, auto r) {
    using X = decltype(x);
    using R = decltype(r);
    if (a.y_type == TFL_E4M3) return forward<X, R, E4m3>(a, num_sms, s);
    if constexpr (sizeof(X) == 4) {
      if (a.y_type == TFL_F16) return forward<X, R, __half>(a, num_sms, s);
      if (a.y_type == TFL_BF16) return forward<X, R, __nv_bfloat16>(a, num_sms, s);
    }
    return forward<X, R, X>(a, num_sms, s);
  });
}

cudaError_t launch_rms_backward(const RmsGradArgs& args, int num_sms, cudaStream_t s) {
  RmsGradArgs a = args;
  const bool vec = a.D % 8 == 0 && a.D <= kRmsMaxRegisterRow / 2 && aligned(a.sum, 16) && aligned(a.gamma, 16) && aligned(a.dy, 16) &&
                   aligned(a.dres, 16) && aligned(a.dx, 16) && aligned(a.dsum, 16);
  if (!vec) {
    if (a.D > kRmsMaxValues) {
      const int grid = backward_blocks(a, a.rows, num_sms * 4);
      const cudaError_t e = launch_dependent(rms_backward_any_kernel, grid, 256, 0, s, a);
      return e == cudaSuccess ? add_partials(a, grid, s) : e;
    }
    return with_types(a.x_type, a.res_type, [&](auto x, auto r) {
      using X = decltype(x);
      using R = decltype(r);
      if (a.D <= 128) return backward_values<X, R, 256, 32, 4>(a, num_sms, s);
      if (a.D <= 256) return backward_values<X, R, 256, 64, 4>(a, num_sms, s);
      if (a.D <= 512) return backward_values<X, R, 256, 128, 4>(a, num_sms, s);
      if (a.D <= 1024) return backward_values<X, R, 256, 256, 4>(a, num_sms, s);
      if (a.D <= 2048) return backward_values<X, R, 512, 512, 4>(a, num_sms, s);
      if (a.D <= 4096) return backward_values<X, R, 1024, 1024, 4>(a, num_sms, s);
      if (a.D <= 5120) return backward_values<X, R, 1024, 1024, 5>(a, num_sms, s);
      if (a.D <= 6144) return backward_values<X, R, 1024, 1024, 6>(a, num_sms, s);
      return backward_values<X, R, 1024, 1024, 8>(a, num_sms, s);
    });
  }
  return with_types(a.x_type, a.res_type, [&](auto x, auto r) {
    return backward<decltype(x), decltype(r)>(a, num_sms, s);
  });
}

}  // namespace tfl
