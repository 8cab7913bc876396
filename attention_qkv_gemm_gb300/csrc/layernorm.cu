// layernorm.cu -- layer norm with the residual's addition, forward and backward.
//
//   s = x + res,  m = mean(s),  r = 1 / sqrt(mean((s - m)^2) + eps),  t = (s - m) r,  y = t gamma + beta
// and, with a = dy gamma, the gradients of s, gamma and beta:
//   ds = dres + r (a - mean(a) - t mean(a t)),   dgamma = sum over rows of dy t,   dbeta = sum of dy
//
// Every value is read once and written once: bandwidth bounds it.  As in rmsnorm.cu a row lives in the
// registers of TPR threads between its loads and its stores.  The variance is taken from the centred
// values of the row in registers, never as mean(s^2) - m^2, which loses everything where the mean is
// large.  The mean itself is off by the rounding of a sum of D terms; the centred values' own mean d
// repairs it (m + d, and (s - m)^2 less d^2), which costs one more sum in the same butterfly.
//
// 8192 x 1024 fp16 with an fp32 residual: 18.5 us, 5.4 TB/s, 0.80 of the copy rate (three waves of blocks, start and
// tail); 100000 x 1024 bf16 to e4m3 110 us, 0.96.  Backward 8192 x 1024 bf16 / fp32 25.0 us, 0.79 (21.5 and
// 3.5 for the second kernel).
//
// The backward takes m and r from the forward (8 bytes a row): from s alone it would need two more
// sums a row that wait for each other before the two that the gradient needs.
//
// Unaligned buffers, rows too long for registers and few rows of widths that 8 does not divide take the
// element-wise kernels.
#include "rowops.cuh"

namespace tfl {

namespace {

// gamma and beta: read by every row, from L1
__device__ __forceinline__ void load_params2(const float* p, uint64_t* v) {
  float f[8];
  load8(p, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = f2_pack(f[2 * i], f[2 * i + 1]);
}

// From the sums over a row's centred values c = s - m0: sum c and sum c^2, the row's mean and 1 / sqrt(var + eps).
__device__ __forceinline__ void finish_stats(float m0, float sum, float square, const LnArgs& a, float& shift, float& mean,
                                             float& rstd) {
  shift = sum * a.inv_d;  // a NaN stays one
  mean = m0 + shift;
  rstd = rsqrtf(max_nan(square * a.inv_d - shift * shift, 0.f) + a.eps);
}

// Sum (or maximum) over the threads of this thread's row: up to a warp's own, or the block's whole warps.  `red`
// holds one float a warp and value.
template <int N>
__device__ __forceinline__ void row_reduce(float* v, int tpr, bool last_is_max, float* red) {
  const int lanes = tpr < 32 ? tpr : 32;
  auto join = [&](float x, float y, int k) { return last_is_max && k == N - 1 ? max_nan(x, y) : x + y; };
#pragma unroll 1
  for (int o = lanes >> 1; o; o >>= 1) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = join(v[k], __shfl_xor_sync(0xffffffffu, v[k], o), k);
  }
  if (tpr <= 32) return;
  __syncthreads();  // the values before have been read
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) red[k * 32 + (threadIdx.x >> 5)] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = red[k * 32];
  for (int w = 1; w < tpr >> 5; ++w) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = join(v[k], red[k * 32 + w], k);
  }
}

template <class X, class R, class Y, int NV>
__global__ void __launch_bounds__(1024) ln_forward_kernel(const LnArgs a) {
  constexpr bool Q = sizeof(Y) == 1;
  __shared__ float red[64];
  grid_launch_dependents();
  grid_wait_prior();
  // a row's threads: a power of two up to a warp's 32, with other rows in the block, or whole warps that are the
  // block
  const int tpr = a.tpr, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + group;
  const bool live = row < a.rows;  // the whole block meets at row_reduce's barriers
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
  // their way to L2.
  const int64_t later = row + a.ahead;
  if (later < a.rows) {
    lines_to_l2(static_cast<const X*>(a.x) + (size_t)later * a.D, a.D * (int)sizeof(X), t, tpr);
    if (a.res) lines_to_l2(static_cast<const R*>(a.res) + (size_t)later * a.D, a.D * (int)sizeof(R), t, tpr);
  }
  float v[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[0] += s[j][i];
  }
  if (a.res_out) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = t + j * tpr;
      if (live && c < nvec) store8(static_cast<R*>(a.res_out) + base + c * 8, s[j]);
    }
  }
  row_reduce<1>(v, tpr, false, red);
  const float m0 = v[0] * a.inv_d;
  v[0] = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (t + j * tpr < nvec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[j][i] -= m0;
        v[0] += s[j][i];
        v[1] = fmaf(s[j][i], s[j][i], v[1]);
      }
    }
  }
  row_reduce<2>(v, tpr, false, red);
  float shift, mean, r;
  finish_stats(m0, v[0], v[1], a, shift, mean, r);
  if (a.stats && live && t == 0) a.stats[row] = make_float2(mean, r);
  v[0] = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = t + j * tpr;
    if (live && c < nvec) {
      float g[8], b[8];
      load8(a.gamma + c * 8, g);
      if (a.beta) {
        load8(a.beta + c * 8, b);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[j][i] = fmaf((s[j][i] - shift) * r, g[i], b[i]);
        if (Q) v[0] = max_nan(v[0], fabsf(s[j][i]));
      }
      if (!Q) store8(static_cast<Y*>(a.y) + base + c * 8, s[j]);
    }
  }
  if constexpr (Q) {
    row_reduce<1>(v, tpr, true, red);
    const float amax = max_nan(v[0], kMinAmax);
    if (live && t == 0) a.y_scale[row] = amax / kE4m3Max;
    const float to8 = kE4m3Max / amax;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = t + j * tpr;
      if (live && c < nvec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j][i] *= to8;
        store8(static_cast<Y*>(a.y) + base + c * 8, s[j]);
      }
    }
  }
}

// Both sums of a row, as row_sums in rowops.cuh, but over any number of whole warps (16 at most).
template <int WARPS = 16>
__device__ __forceinline__ void row_pair(float& a, float& b, int tpr, int group, int parity, float2 (*red)[32]) {
  const int lane = threadIdx.x & 31;
  if (tpr <= 32) {
    row_sums(a, b, tpr, group, parity, red);
    return;
  }
  row_sums(a, b, 32, group, parity, red);
  const int nw = tpr >> 5;
  if (lane == 0) red[parity][threadIdx.x >> 5] = make_float2(a, b);
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
  const int w = lane & (WARPS - 1);
  const float2 p = w < nw ? red[parity][group * nw + w] : make_float2(0.f, 0.f);
  a = p.x;
  b = p.y;
#pragma unroll
  for (int o = WARPS / 2; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
}

__device__ __forceinline__ void assign(E4m3& d, float v) { d.v = (uint8_t)e4m3x2(v, 0.f); }

// Part of a vector: its first n values, zeros behind.
template <class T>
__device__ __forceinline__ void load_first(const T* p, int n, Raw8<T>& r) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = i < n ? value(p[i]) : 0.f;
  store8(reinterpret_cast<T*>(&r), f);
}

// Which of a vector's columns col .. col + 7 a row of D values has: 16 bits each, all set or none.
__device__ __forceinline__ void own_columns(int col, int D, bool in, uint32_t* own) {
  auto has = [&](int i) { return in && col + i >= 0 && col + i < D; };
#pragma unroll
  for (int i = 0; i < 4; ++i) own[i] = (has(2 * i) ? 0xffffu : 0u) | (has(2 * i + 1) ? 0xffff0000u : 0u);
}
__device__ __forceinline__ bool has_column(const uint32_t* own, int i) {
  return own[i / 2] & (i & 1 ? 0xffff0000u : 0xffffu);
}
// The others' values, whatever they are, become zeros.
template <class T>
__device__ __forceinline__ void drop_others(Raw8<T>& r, const uint32_t* own) {
  if constexpr (sizeof(T) == 2) {
    r.w[0].x &= own[0], r.w[0].y &= own[1], r.w[0].z &= own[2], r.w[0].w &= own[3];
  } else {
    uint32_t* w = &r.w[0].x;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = has_column(own, i) ? w[i] : 0u;
  }
}
template <class T>
__device__ __forceinline__ void store_own(T* p, const float* v, const uint32_t* own) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (has_column(own, i)) assign(p[i], v[i]);
}

// The largest of a row's values, likewise.
template <int WARPS = 16>
__device__ __forceinline__ float row_largest(float v, int tpr, int group, int parity, float2 (*red)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int o = (tpr < 32 ? tpr : 32) >> 1; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (tpr <= 32) return v;
  const int nw = tpr >> 5;
  if (lane == 0) red[parity][threadIdx.x >> 5].x = v;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(tpr) : "memory");
  const int w = lane & (WARPS - 1);
  v = w < nw ? red[parity][group * nw + w].x : 0.f;
#pragma unroll
  for (int o = WARPS / 2; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Forward of widths that 8 does not divide, in vectors: row groups that loop over rows which begin alike, with
// gamma and beta in registers, as the backward below does it (100000 x 103 bf16 / fp32 to e4m3 31 us; a value at a
// time, a block a row, 224).
template <class X, class R, class Y, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) ln_forward_straddle_kernel(const LnArgs a) {
  constexpr bool Q = sizeof(Y) == 1;
  constexpr int WARPS = THREADS > 512 ? 32 : 16;  // of the widest group
  __shared__ float2 red[2][32];
  grid_launch_dependents();
  grid_wait_prior();
  const int tpr = a.tpr, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr, groups = THREADS / tpr;
  const int rows = (int)a.rows, D = a.D;
  const int stride = gridDim.x * groups, first = blockIdx.x * groups + group;
  const int shift = (int)(((int64_t)first * D) & 7), col = t * 8 - shift;
  const bool in = t < (shift + D + 7) >> 3, edge = col < 0 || col + 8 > D;
  uint32_t own[4];
  own_columns(col, D, in, own);
  auto mine = [&](int i) { return has_column(own, i); };
  float g[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    g[i] = mine(i) ? a.gamma[col + i] : 0.f;
    b[i] = mine(i) && a.beta ? a.beta[col + i] : 0.f;
  }
  const size_t step = (size_t)stride * D;
  size_t at = (size_t)first * D + t * 8 - shift;  // of the row to load next
  Raw8<X> x1;
  Raw8<R> r1;
  zero_raw(r1);
  auto fetch = [&](int64_t row) {
    if (row < rows && in) {
      const X* x = static_cast<const X*>(a.x) + at;
      const R* r = a.res ? static_cast<const R*>(a.res) + at : nullptr;
      if (row == rows - 1 && col + 8 > D) {  // behind the last row there is nothing to read
        load_first(x, D - col, x1);
        if (r) load_first(r, D - col, r1);
      } else {
        load_raw(x, x1);
        if (r) load_raw(r, r1);
      }
    } else {
      zero_raw(x1);
      zero_raw(r1);
    }
    at += step;
  };
  int parity = 0;
  fetch(first);
  const int lead = tpr < 32 ? first / (32 / tpr) * (32 / tpr) : first;  // groups that share a warp go together
  int64_t row = first;
  size_t to = at - step;
  for (int64_t turn = lead; turn < rows; turn += stride, row += stride, to += step) {
    const bool live = row < rows && in;
    float s[8], r[8];
    widen(x1, s);
    widen(r1, r);
    fetch(row + stride);
    float v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = !edge || mine(i) ? s[i] + r[i] : 0.f;
      v0 += s[i];
    }
    auto store = [&](auto* p, const float* v) {
      if (!live) return;
      if (edge) {
        store_own(p + to, v, own);
      } else {
        store8(p + to, v);
      }
    };
    if (a.res_out) store(static_cast<R*>(a.res_out), s);
    row_pair<WARPS>(v0, v1, tpr, group, parity, red);
    parity ^= 1;
    const float m0 = v0 * a.inv_d;
    v0 = v1 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = !edge || mine(i) ? s[i] - m0 : 0.f;
      v0 += s[i];
      v1 = fmaf(s[i], s[i], v1);
    }
    row_pair<WARPS>(v0, v1, tpr, group, parity, red);
    parity ^= 1;
    float off, mean, rstd;
    finish_stats(m0, v0, v1, a, off, mean, rstd);
    if (a.stats && live && t == 0) a.stats[row] = make_float2(mean, rstd);
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = fmaf((s[i] - off) * rstd, g[i], b[i]);
      if (Q && (!edge || mine(i))) most = max_nan(most, fabsf(s[i]));
    }
    if constexpr (Q) {
      if (!in) most = 0.f;
      most = max_nan(row_largest<WARPS>(most, tpr, group, parity, red), kMinAmax);
      parity ^= 1;
      if (live && t == 0) a.y_scale[row] = most / kE4m3Max;
      const float to8 = kE4m3Max / most;
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] *= to8;
    }
    store(static_cast<Y*>(a.y), s);
  }
}

// Backward.  As in rms_backward_kernel: a row group keeps its columns over all its rows, so each thread
// holds gamma and sums dgamma and dbeta of its own columns in registers; the groups of a block are joined
// in shared memory and every block writes one row of partial sums, which column_sums_kernel adds in block
// order: the result depends on the sizes and the SM count only.  The next row is loaded, as stored, before
// the current one is worked on.
//
// STRADDLE: widths that 8 does not divide, in 16-byte vectors all the same.  A row then begins `shift`
// values into a vector, (row D) mod 8; a group takes rows a multiple of 8 / gcd(D, 8) apart, so its shift
// and its threads' columns stay.  A row's first and last vectors hold values of its neighbours, which count
// as nothing and are not written (6011 x 1001 fp16 16.6 us, 25.2 a value at a time; without the prefetch that
// wide rows' loads need, 5000 x 7001 128 instead of 108 us).
template <class X, class R, int NV, int THREADS, int BLOCKS, bool STRADDLE>
__global__ void __launch_bounds__(THREADS, BLOCKS) ln_backward_kernel(const LnGradArgs a) {
  constexpr bool AHEAD = NV == 1;                // room for the next row, its residual's gradient and gamma
  constexpr bool EARLY = AHEAD || THREADS < 512;  // room for the next row
  __shared__ float2 red[2][32];
  // [groups][D + 4] when the block has more than one group; gamma as this block's rows lie, if it has to be shifted
  // and there are no registers for it (then it has one)
  extern __shared__ float part[];
  grid_launch_dependents();
  grid_wait_prior();
  const int tpr = a.tpr, group = threadIdx.x / tpr, t = threadIdx.x - group * tpr, groups = THREADS / tpr;
  const int rows = (int)a.rows, D = a.D;
  const bool spare = group >= groups;  // warps that make no whole group
  const int stride = gridDim.x * groups, first = spare ? rows : blockIdx.x * groups + group;
  const int shift = STRADDLE ? (int)(((int64_t)first * D) & 7) : 0;
  const int nvec = (shift + D + 7) >> 3;
  auto col = [&](int j) { return (t + j * tpr) * 8 - shift; };  // this thread's columns: from here on
  bool in[NV];                                                  // vectors of this thread that exist
  uint64_t dg[NV][4], db[NV][4], gk[AHEAD ? NV : 1][4];
  uint32_t own[NV][4];  // STRADDLE
  auto gamma_of = [&](int j) { return STRADDLE ? part + (t + j * tpr) * 8 : a.gamma + col(j); };  // not AHEAD
  auto edge = [&](int j) { return STRADDLE && (col(j) < 0 || col(j) + 8 > D); };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    in[j] = !spare && t + j * tpr < nvec;
#pragma unroll
    for (int i = 0; i < 4; ++i) dg[j][i] = db[j][i] = 0;  // two zeros
    if constexpr (STRADDLE) {
      own_columns(col(j), D, in[j], own[j]);
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = in[j] && col(j) + i >= 0 && col(j) + i < D ? a.gamma[col(j) + i] : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (AHEAD) gk[j][i] = f2_pack(f[2 * i], f[2 * i + 1]);
      }
      if constexpr (!AHEAD) {
        if (!spare) store8(part + (t + j * tpr) * 8, f);  // each thread its own
      }
    } else if constexpr (AHEAD) {
      if (in[j]) {
        load_params2(a.gamma + col(j), gk[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) gk[j][i] = 0;
      }
    }
  }
  // this thread's first vector of the row to load next and of the row to write next
  const size_t step = (size_t)stride * D, begin = (size_t)first * D + t * 8 - shift;
  const R* sp = static_cast<const R*>(a.sum) + begin;
  const X* yp = static_cast<const X*>(a.dy) + begin;
  const R* ep = a.dres ? static_cast<const R*>(a.dres) + begin : nullptr;
  const R* ep_late = ep;
  const float2* stat = a.stats + first;
  R* dsum = a.dsum ? static_cast<R*>(a.dsum) + begin : nullptr;
  X* dx = a.dx ? static_cast<X*>(a.dx) + begin : nullptr;
  const int jump = tpr * 8;  // from one vector of a thread to its next
  Raw8<R> s1[NV], e1[NV], e[NV];
  Raw8<X> y1[NV];
  float2 st1 = make_float2(0.f, 0.f);
  auto fetch = [&](int64_t row) {
    const bool live = row < rows;
    if (live) st1 = *stat;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (live && in[j]) {
        if (STRADDLE && row == rows - 1 && col(j) + 8 > D) {  // behind the last row there is nothing to read
          load_first(sp + j * jump, D - col(j), s1[j]);
          load_first(yp + j * jump, D - col(j), y1[j]);
          if (AHEAD && ep) load_first(ep + j * jump, D - col(j), e1[j]);
        } else {
          load_raw(sp + j * jump, s1[j]);
          load_raw(yp + j * jump, y1[j]);
          if (AHEAD && ep) load_raw(ep + j * jump, e1[j]);
        }
      } else {
        zero_raw(s1[j]);
        zero_raw(y1[j]);
      }
    }
    stat += stride;
    sp += step;
    yp += step;
    if (ep) ep += step;
    // the row behind that one to L2: with one row in registers the bytes in flight are what bounds the rate
    if (!(STRADDLE && AHEAD) && row + stride < rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!in[j]) continue;
        const int o = j * jump;
        if (t % (16 / sizeof(R)) == 0) prefetch_l2(sp + o);
        if (t % (16 / sizeof(X)) == 0) prefetch_l2(yp + o);
        if (t % (16 / sizeof(R)) == 0 && ep) prefetch_l2(ep + o);
      }
    }
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) zero_raw(e1[j]);
  int parity = 0;
  if (EARLY) fetch(first);
  // groups that share a warp go through the same number of rows (its shuffles need all lanes)
  const int lead = tpr < 32 ? first / (32 / tpr) * (32 / tpr) : first;  // of the warp's groups
  int64_t next = first;
  for (int64_t at = lead; at < rows; at += stride) {
    const bool live = next < rows;
    if (!EARLY) fetch(next);
    next += stride;
    uint64_t s[NV][4], y[NV][4];
    const float2 st = st1;
    const uint64_t mean2 = f2_splat(st.x), r2 = f2_splat(st.y);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (STRADDLE) drop_others(y1[j], own[j]);  // a neighbour's values count as nothing
      widen2(s1[j], s[j]);
      widen2(y1[j], y[j]);
      e[j] = e1[j];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[j][i] = f2_mul(f2_sub(s[j][i], mean2), r2);  // t
      if (edge(j)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float t0, t1;
          f2_unpack(s[j][i], t0, t1);
          s[j][i] = f2_pack(has_column(own[j], 2 * i) ? t0 : 0.f, has_column(own[j], 2 * i + 1) ? t1 : 0.f);
        }
      }
    }
    if (EARLY) fetch(next);
    uint64_t sa = 0, at2 = 0;  // two zeros each
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      uint64_t g[4] = {0, 0, 0, 0};
      if (!AHEAD && in[j]) load_params2(gamma_of(j), g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t w = f2_mul(y[j][i], AHEAD ? gk[AHEAD ? j : 0][i] : g[i]);
        sa = f2_add(sa, w);
        at2 = f2_fma(w, s[j][i], at2);
      }
    }
    float v0, v1, hi;
    f2_unpack(sa, v0, hi);
    v0 += hi;
    f2_unpack(at2, v1, hi);
    v1 += hi;
    row_pair(v0, v1, tpr, group, parity, red);
    parity ^= 1;
    const uint64_t k0 = f2_splat(-(v0 * a.inv_d)), k1 = f2_splat(-(v1 * a.inv_d));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (live && in[j]) {
        uint64_t g[4], o[4];
        if constexpr (!AHEAD) load_params2(gamma_of(j), g);
        if (!AHEAD && ep_late) {
          if (STRADDLE && next - stride == rows - 1 && col(j) + 8 > D)
            load_first(ep_late + j * jump, D - col(j), e[j]);
          else
            load_raw(ep_late + j * jump, e[j]);
        }
        widen2(e[j], o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dg[j][i] = f2_fma(y[j][i], s[j][i], dg[j][i]);
          db[j][i] = f2_add(y[j][i], db[j][i]);
          const uint64_t d = f2_fma(s[j][i], k1, f2_fma(y[j][i], AHEAD ? gk[AHEAD ? j : 0][i] : g[i], k0));
          o[i] = f2_fma(d, r2, o[i]);
        }
        float of[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_unpack(o[i], of[2 * i], of[2 * i + 1]);
        if (edge(j)) {
          if (dsum) store_own(dsum + j * jump, of, own[j]);
          if (dx) store_own(dx + j * jump, of, own[j]);
        } else {
          if (dsum) store8(dsum + j * jump, of);
          if (dx) store8(dx + j * jump, of);
        }
      }
    }
    if (dsum) dsum += step;
    if (dx) dx += step;
    if (!AHEAD && ep_late) ep_late += step;
  }
  const int pitch = D + 4;  // columns of 8 rows in a row lie in different banks
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    float* out = (which ? a.part_beta : a.part_gamma);
    if (!out) break;  // no dbeta
    out += (size_t)blockIdx.x * a.part_stride;
    if (which) __syncthreads();  // dgamma's sums have been read
    float* to = groups == 1 ? out : part + group * pitch;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!in[j]) continue;
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) f2_unpack(which ? db[j][i] : dg[j][i], f[2 * i], f[2 * i + 1]);
      if constexpr (STRADDLE) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col(j) + i >= 0 && col(j) + i < D) to[col(j) + i] = f[i];
      } else {
        store8(to + col(j), f);
      }
    }
    if (groups == 1) continue;
    __syncthreads();
    if (groups > 32) {  // short rows: a warp a column (in turn, 512 rows would be a long chain of additions)
      for (int c = threadIdx.x >> 5; c < D; c += THREADS / 32) {
        float v = 0.f;
        for (int g = threadIdx.x & 31; g < groups; g += 32) v += part[g * pitch + c];
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if ((threadIdx.x & 31) == 0) out[c] = v;
      }
    } else {
      for (int c = threadIdx.x; c < D; c += blockDim.x) {
        float v = 0.f;
        for (int g = 0; g < groups; ++g) v += part[g * pitch + c];
        out[c] = v;
      }
    }
  }
}

// ---- element-wise forms: any width and element-aligned buffers
// Rows of up to T NE values, one block a row: T threads with NE each in registers, all loads at once.
template <class X, class R, int T, int NE>
__global__ void __launch_bounds__(T) ln_forward_values_kernel(const LnArgs a) {
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
  const int64_t later = blockIdx.x + a.ahead;  // as in ln_forward_kernel
  if (later < a.rows) {
    lines_to_l2(static_cast<const X*>(a.x) + (size_t)later * a.D, a.D * (int)sizeof(X), threadIdx.x, T);
    if (a.res) lines_to_l2(static_cast<const R*>(a.res) + (size_t)later * a.D, a.D * (int)sizeof(R), threadIdx.x, T);
  }
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    v[0] += s[j];
    if ((int)threadIdx.x + j * T < a.D && a.res_out) assign(static_cast<R*>(a.res_out)[base + j * T], s[j]);
  }
  group_reduce<1>(v, T, false, red);
  const float m0 = v[0] * a.inv_d;
  v[0] = 0.f;
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    if ((int)threadIdx.x + j * T < a.D) {
      s[j] -= m0;
      v[0] += s[j];
      v[1] = fmaf(s[j], s[j], v[1]);
    }
  }
  group_reduce<2>(v, T, false, red);
  float shift, mean, r;
  finish_stats(m0, v[0], v[1], a, shift, mean, r);
  if (a.stats && threadIdx.x == 0) a.stats[blockIdx.x] = make_float2(mean, r);
  v[0] = 0.f;
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    const int c = threadIdx.x + j * T;
    if (c < a.D) {
      s[j] = fmaf((s[j] - shift) * r, a.gamma[c], a.beta ? a.beta[c] : 0.f);
      v[0] = max_nan(v[0], fabsf(s[j]));
    }
  }
  float to8 = 1.0f;
  if (a.y_type == TFL_E4M3) {
    group_reduce<1>(v, T, true, red);
    const float amax = max_nan(v[0], kMinAmax);
    if (threadIdx.x == 0) a.y_scale[blockIdx.x] = amax / kE4m3Max;
    to8 = kE4m3Max / amax;
  }
#pragma unroll
  for (int j = 0; j < NE; ++j)
    if ((int)threadIdx.x + j * T < a.D) store1(a.y, a.y_type, base + j * T, s[j] * to8);
}

// Groups of G threads take rows of up to G NE values, all groups of a block together T threads.  The
// next row is on its way while one is worked on, without its residual gradient where registers are
// short (NE > 4), and gamma then comes from L1.
template <class X, class R, int T, int G, int NE>
__global__ void __launch_bounds__(T, 1024 / T) ln_backward_values_kernel(const LnGradArgs a) {
  constexpr bool ROOM = NE <= 4;
  constexpr int GROUPS = T / G;
  __shared__ float2 red[2][32];
  __shared__ float part[GROUPS > 1 ? T * NE : 1];
  grid_launch_dependents();
  grid_wait_prior();
  const int t = threadIdx.x % G, group = threadIdx.x / G, D = a.D;
  const int64_t stride = (int64_t)gridDim.x * GROUPS;
  float dg[NE], db[NE], gk[ROOM ? NE : 1];
#pragma unroll
  for (int j = 0; j < NE; ++j) {
    dg[j] = db[j] = 0.f;
    if (ROOM || j == 0) gk[ROOM ? j : 0] = t + j * G < D ? a.gamma[t + j * G] : 0.f;
  }
  auto gamma = [&](int j) { return ROOM ? gk[ROOM ? j : 0] : a.gamma[t + j * G]; };
  R s1[NE], e1[NE];
  X y1[NE];
  float2 st1 = make_float2(0.f, 0.f);
  auto fetch_res = [&](int64_t row) {
    const R* p = static_cast<const R*>(a.dres) + (size_t)row * D + t;
#pragma unroll
    for (int j = 0; j < NE; ++j) e1[j] = a.dres && row < a.rows && t + j * G < D ? p[j * G] : R(0.f);
  };
  auto fetch = [&](int64_t row) {
    const R* p = static_cast<const R*>(a.sum) + (size_t)row * D + t;
    const X* q = static_cast<const X*>(a.dy) + (size_t)row * D + t;
    if (row < a.rows) st1 = a.stats[row];
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const bool in = row < a.rows && t + j * G < D;
      s1[j] = in ? p[j * G] : R(0.f);
      y1[j] = in ? q[j * G] : X(0.f);
    }
    if (ROOM) fetch_res(row);
  };
  int parity = 0;
  int64_t row = (int64_t)blockIdx.x * GROUPS + group;
  fetch(row);
  for (; row < a.rows; row += stride) {
    float s[NE], y[NE], e[NE];
    const float2 st = st1;
    if (!ROOM) fetch_res(row);
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      s[j] = (value(s1[j]) - st.x) * st.y;  // t
      y[j] = value(y1[j]);
      if (ROOM) e[j] = value(e1[j]);
    }
    fetch(row + stride);
    float v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      if (t + j * G < D) {
        const float w = y[j] * gamma(j);
        v0 += w;
        v1 = fmaf(w, s[j], v1);
      }
    }
    row_sums<32>(v0, v1, G, group, parity, red);
    parity ^= 1;
    const float k0 = -(v0 * a.inv_d), k1 = -(v1 * a.inv_d);
    const size_t base = (size_t)row * D + t;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      if (t + j * G < D) {
        if (!ROOM) e[j] = value(e1[j]);
        dg[j] = fmaf(y[j], s[j], dg[j]);
        db[j] += y[j];
        const float o = fmaf(fmaf(s[j], k1, fmaf(y[j], gamma(j), k0)), st.y, e[j]);
        if (a.dsum) assign(static_cast<R*>(a.dsum)[base + j * G], o);
        if (a.dx) assign(static_cast<X*>(a.dx)[base + j * G], o);
      }
    }
  }
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    float* out = (which ? a.part_beta : a.part_gamma);
    if (!out) break;
    out += (size_t)blockIdx.x * a.part_stride;
    if constexpr (GROUPS == 1) {
#pragma unroll
      for (int j = 0; j < NE; ++j)
        if (t + j * G < D) out[t + j * G] = which ? db[j] : dg[j];
    } else {
      if (which) __syncthreads();  // dgamma's sums have been read
#pragma unroll
      for (int j = 0; j < NE; ++j) part[(group * NE + j) * G + t] = which ? db[j] : dg[j];
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += T) {
        float v = 0.f;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) v += part[g * NE * G + c];
        out[c] = v;
      }
    }
  }
}

// Wider rows: three passes, the later ones from L1 / L2.
__global__ void __launch_bounds__(256) ln_forward_any_kernel(const LnArgs a) {
  __shared__ float red[64];
  grid_launch_dependents();
  grid_wait_prior();
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const size_t base = (size_t)row * a.D;
    auto sum = [&](int c) {
      const float s = load1(a.x, a.x_type, base + c);
      return a.res ? s + load1(a.res, a.res_type, base + c) : s;
    };
    auto norm = [&](float t, int c) { return fmaf(t, a.gamma[c], a.beta ? a.beta[c] : 0.f); };
    float v[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < a.D; c += 256) v[0] += sum(c);
    group_reduce<1>(v, 256, false, red);
    const float m0 = v[0] * a.inv_d;
    v[0] = 0.f;
    for (int c = threadIdx.x; c < a.D; c += 256) {
      const float d = sum(c) - m0;
      v[0] += d;
      v[1] = fmaf(d, d, v[1]);
    }
    group_reduce<2>(v, 256, false, red);
    float shift, mean, r;
    finish_stats(m0, v[0], v[1], a, shift, mean, r);
    if (a.stats && threadIdx.x == 0) a.stats[row] = make_float2(mean, r);
    float to8 = 1.0f;
    if (a.y_type == TFL_E4M3) {
      v[0] = 0.f;
      for (int c = threadIdx.x; c < a.D; c += 256)
        v[0] = max_nan(v[0], fabsf(norm((sum(c) - m0 - shift) * r, c)));
      group_reduce<1>(v, 256, true, red);
      const float amax = max_nan(v[0], kMinAmax);
      if (threadIdx.x == 0) a.y_scale[row] = amax / kE4m3Max;
      to8 = kE4m3Max / amax;
    }
    for (int c = threadIdx.x; c < a.D; c += 256) {
      const float s = sum(c);
      if (a.res_out) store1(a.res_out, a.res_type, base + c, s);
      store1(a.y, a.y_type, base + c, norm((s - m0 - shift) * r, c) * to8);
    }
  }
}

// The thread that owns column c in every row of the block also adds up its dgamma and dbeta, in the
// block's row of partial sums.
__global__ void __launch_bounds__(256) ln_backward_any_kernel(const LnGradArgs a) {
  __shared__ float red[64];
  grid_launch_dependents();
  grid_wait_prior();
  float* pg = a.part_gamma + (size_t)blockIdx.x * a.part_stride;
  float* pb = a.part_beta ? a.part_beta + (size_t)blockIdx.x * a.part_stride : nullptr;
  for (int c = threadIdx.x; c < a.D; c += 256) {
    pg[c] = 0.f;
    if (pb) pb[c] = 0.f;
  }
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const size_t base = (size_t)row * a.D;
    const float2 st = a.stats[row];
    float v[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < a.D; c += 256) {
      const float w = load1(a.dy, a.x_type, base + c) * a.gamma[c];
      v[0] += w;
      v[1] = fmaf(w, (load1(a.sum, a.res_type, base + c) - st.x) * st.y, v[1]);
    }
    group_reduce<2>(v, 256, false, red);
    const float k0 = -(v[0] * a.inv_d), k1 = -(v[1] * a.inv_d);
    for (int c = threadIdx.x; c < a.D; c += 256) {
      const float t = (load1(a.sum, a.res_type, base + c) - st.x) * st.y, dy = load1(a.dy, a.x_type, base + c);
      const float d = fmaf(t, k1, fmaf(dy, a.gamma[c], k0));
      const float o = fmaf(d, st.y, a.dres ? load1(a.dres, a.res_type, base + c) : 0.f);
      pg[c] = fmaf(dy, t, pg[c]);
      if (pb) pb[c] += dy;
      if (a.dsum) store1(a.dsum, a.res_type, base + c, o);
      if (a.dx) store1(a.dx, a.x_type, base + c, o);
    }
  }
}

// Threads that hold a row of `nvec` vectors, n each.
int row_threads(int nvec, int n) {
  const int t = (nvec + n - 1) / n;
  return t <= 32 ? pow2_at_least(t) : (t + 31) / 32 * 32;
}

// Four vectors a thread, where an fp32 residual doubles their bytes two: the rows in flight are what counts,
// and more, smaller blocks leave less of a last round (8192 x 1024 fp16 / fp32 in blocks of 256 threads 20.5
// with four and 19.7 us with two, in blocks of 64 20.1 and 18.3; 16384 x 2048 bf16 46.4, 54.5, 42.8 and 47.8).
// Other numbers where they leave fewer lanes without a vector (12275 x 2168 fp16 to e4m3 49.9 us with four, 41.6
// with three; two 16-bit vectors only where they spare a fifth: 5274 x 3336 fp16 30.9 us, with four 28.2).
int row_vectors(int nvec, bool res_f32) {
  if (nvec <= 32) return 1;
  int nv = 1, slots = 1 << 30;
  const int order[2][3] = {{4, 3, 2}, {2, 3, 4}};
  for (int n : order[res_f32]) {
    if (row_threads(nvec, n) > 1024 || (nvec <= 64 && n != 2)) continue;
    const int cost = row_threads(nvec, n) * n * (!res_f32 && n == 2 ? 6 : 5);
    if (cost < slots) {
      nv = n;
      slots = cost;
    }
  }
  return nv;
}
// Short rows share a block (65536 x 128 fp16 / fp32: 16.8 us in blocks of 256 threads, 17.9 of 64).
int block_threads(int nv, int tpr) { return tpr > 32 ? tpr : nv == 1 ? 256 : 64; }

template <class X, class R, class Y>
cudaError_t forward(LnArgs a, const LnPlan& p, int num_sms, cudaStream_t s) {
  a.tpr = row_threads(a.D / 8, p.vectors);
  const int64_t per = p.threads / a.tpr;
  const unsigned grid = (unsigned)((a.rows + per - 1) / per);
  a.ahead = per * num_sms * (1024 / p.threads);  // 64 registers a thread: 1024 threads an SM
  if (p.vectors == 1) return launch_dependent(ln_forward_kernel<X, R, Y, 1>, grid, p.threads, 0, s, a);
  if (p.vectors == 2) return launch_dependent(ln_forward_kernel<X, R, Y, 2>, grid, p.threads, 0, s, a);
  if (p.vectors == 3) return launch_dependent(ln_forward_kernel<X, R, Y, 3>, grid, p.threads, 0, s, a);
  return launch_dependent(ln_forward_kernel<X, R, Y, 4>, grid, p.threads, 0, s, a);
}

// Rows of a group are a multiple of the period apart after which a row begins at the same place in a vector: the
// least number of blocks whose groups are one.
int even_blocks(int D, int groups) {
  const int period = D % 4 == 0 ? 2 : D % 2 == 0 ? 4 : 8;
  int n = 1;
  while (n * groups % period) ++n;
  return n;
}

template <class X, class R, class Y, int THREADS, int BLOCKS>
cudaError_t forward_straddle(LnArgs a, int num_sms, cudaStream_t s) {
  const int least = (a.D + 14) / 8;  // vectors that a row may reach into
  a.tpr = least <= 32 ? pow2_at_least(least) : (least + 31) / 32 * 32;
  const int groups = THREADS / a.tpr;
  const int threads = groups * a.tpr;
  int64_t n = (int64_t)num_sms * (BLOCKS * THREADS / threads);
  const int64_t all = (a.rows + groups - 1) / groups;
  n = all <= n ? all : n - n % even_blocks(a.D, groups);
  return launch_dependent(ln_forward_straddle_kernel<X, R, Y, THREADS, BLOCKS>, (unsigned)n, threads, 0, s, a);
}

// Blocks of a backward over groups of rows: what the GPU holds at once, and one alone for so few that
// a second launch would cost more than their turns; `even`: a multiple of it, where a block has several
// turns.  A lone block writes dgamma and dbeta itself, where they take the 16-byte stores of the partial rows.
int backward_blocks(LnGradArgs& a, int64_t groups_of_rows, int at_once, int even = 1) {
  int64_t n = at_once < a.blocks ? at_once : a.blocks;
  if (groups_of_rows <= n)
    n = groups_of_rows <= 3 && even == 1 ? 1 : groups_of_rows;
  else
    n -= n % even;
  const bool lone = n == 1 && aligned(a.dgamma, 16) && aligned(a.dbeta, 16);
  a.part_stride = 2 * (size_t)a.D;
  a.part_gamma = lone ? a.dgamma : a.partial;
  a.part_beta = !a.dbeta ? nullptr : lone ? a.dbeta : a.partial + a.D;
  return (int)n;
}

cudaError_t add_partials(const LnGradArgs& a, int n, cudaStream_t s) {
  if (a.part_gamma == a.dgamma) return cudaSuccess;
  return launch_column_sums(a.partial, n, 2 * a.D, a.dbeta ? 2 * a.D : a.D, a.D, a.dgamma, a.dbeta, s);
}

template <class X, class R, int NV, int THREADS, int BLOCKS, bool STRADDLE = false>
cudaError_t backward_with(LnGradArgs a, int num_sms, cudaStream_t s) {
  // (a row that begins inside a vector reaches into up to D / 8 + 2 of them)
  const int least = ((STRADDLE ? (a.D + 14) / 8 : a.D / 8) + NV - 1) / NV;
  a.tpr = least <= 32 ? pow2_at_least(least) : (least + 31) / 32 * 32;
  constexpr bool SHIFTED = STRADDLE && NV > 1;  // gamma in shared memory: one group a block
  if (SHIFTED && a.tpr <= THREADS / 2) a.tpr = THREADS / 2 + 32;
  const int groups = THREADS / a.tpr;
  const int even = STRADDLE ? even_blocks(a.D, groups) : 1;
  const int grid = backward_blocks(a, (a.rows + groups - 1) / groups, num_sms * BLOCKS, even);
  const size_t smem = SHIFTED      ? (size_t)a.tpr * NV * 8 * sizeof(float)  // 32 KB
                      : groups > 1 ? (size_t)groups * (a.D + 4) * sizeof(float)  // at most 36 KB
                                   : 0;
  const cudaError_t e = launch_dependent(ln_backward_kernel<X, R, NV, THREADS, BLOCKS, STRADDLE>, grid, THREADS, smem, s, a);
  return e == cudaSuccess ? add_partials(a, grid, s) : e;
}

template <class X, class R, int T, int G, int NE>
cudaError_t backward_values(LnGradArgs a, int num_sms, cudaStream_t s) {
  const int grid = backward_blocks(a, (a.rows + T / G - 1) / (T / G), num_sms * (1024 / T));
  const cudaError_t e = launch_dependent(ln_backward_values_kernel<X, R, T, G, NE>, grid, T, 0, s, a);
  return e == cudaSuccess ? add_partials(a, grid, s) : e;
}

// widest row whose vectors, wherever it begins, 512 and 1024 threads hold (the backward: 512 of two vectors)
constexpr int kLnMaxStraddle = 4082, kLnMaxStraddleWide = 8178;

template <class X, class R, bool STRADDLE>
cudaError_t backward(const LnGradArgs& a, const LnPlan& p, int num_sms, cudaStream_t s) {
  if constexpr (!STRADDLE) {
    if (p.threads == 256) return backward_with<X, R, 1, 256, 2>(a, num_sms, s);
    if (p.vectors == 4) return backward_with<X, R, 4, 512, 1>(a, num_sms, s);
  }
  if (p.vectors == 1) return backward_with<X, R, 1, 512, 1, STRADDLE>(a, num_sms, s);
  return p.threads == 512 ? backward_with<X, R, 2, 512, 1, STRADDLE>(a, num_sms, s)
                          : backward_with<X, R, 2, 384, 1, STRADDLE>(a, num_sms, s);
}

constexpr int kLnMaxValues = 8192;        // widest row the element-wise kernels hold in registers
constexpr int kLnMaxRegisterRow = 32768;  // widest the vector kernels do (the backward: half)

}  // namespace

LnPlan ln_forward_plan(int D, int64_t rows, bool res_f32, bool lines, bool params, int num_sms) {
  LnPlan p;
  if (lines && params && D % 8 == 0 && D <= kLnMaxRegisterRow) {
    p.form = TFL_LN_FORM_VECTORS;
    p.vectors = row_vectors(D / 8, res_f32);
    p.threads = block_threads(p.vectors, row_threads(D / 8, p.vectors));
    return p;
  }
  // (few rows are done as soon a value at a time, a block each: 1000 x 1001 fp16 / fp32 4.4 us, 6.0 in vectors;
  // 6011 x 1001 17.3 and 15.7, 1000 x 3333 bf16 15.2 and 10.9, 5000 x 7001 fp16 168 and 67)
  if (lines && D % 8 != 0 && D >= 8 && D <= kLnMaxStraddleWide && rows >= (D > 2034 ? 1 : 16) * (int64_t)num_sms) {
    p.form = TFL_LN_FORM_STRADDLE;
    p.vectors = 1;
    p.threads = D <= 2034 ? 256 : D <= kLnMaxStraddle ? 512 : 1024;
    return p;
  }
  p.form = D <= kLnMaxValues ? TFL_LN_FORM_VALUES : TFL_LN_FORM_ANY;
  return p;
}

LnPlan ln_backward_plan(int D, int64_t rows, bool lines, bool params, int num_sms) {
  LnPlan p;
  // (few rows are done as soon a value at a time: 9807 x 103 fp16 7.8 us, 8.9 in vectors; 20000 x 203 20.9 and
  // 14.4; 500 x 4099 18.9 and 21.4, 2000 x 4099 47.5 and 39.5, 5000 x 7001 211 and 108)
  const bool straddle = lines && D % 8 != 0 && D >= 8 && D <= kLnMaxStraddleWide && rows * D >= (D > kLnMaxStraddle ? 8000000 : 2000000);
  const bool vec = lines && params && D % 8 == 0 && D <= kLnMaxRegisterRow / 2;
  if (!straddle && !vec) {
    p.form = D <= kLnMaxValues ? TFL_LN_FORM_VALUES : TFL_LN_FORM_ANY;
    return p;
  }
  p.form = straddle ? TFL_LN_FORM_STRADDLE : TFL_LN_FORM_VECTORS;
  // (with 384 threads the registers hold the next row too: 5000 x 5120 bf16 64.9 -> 58.3 us, 4000 x 6003 fp32 103 -> 84;
  // 512 would spill: 4000 x 8192 fp16 68 -> 78)
  const int over = straddle ? 14 : 0;  // a row that begins inside a vector may reach into two more
  p.vectors = D + over <= 4096 ? 1 : straddle || D <= 8192 ? 2 : 4;
  p.threads = p.vectors == 2 && D + over <= 6144 ? 384 : 512;
  // one wide block an SM where the rows give each of them work (fewer partial rows to add), narrower
  // ones to spread fewer rows over all SMs (rows that begin inside a vector are many enough)
  if (!straddle && D <= 2048 && rows * pow2_at_least(D / 8) < (int64_t)num_sms * 512) p.threads = 256;
  return p;
}

cudaError_t launch_ln_forward(const LnArgs& a, int num_sms, cudaStream_t s) {
  const bool lines = aligned(a.x, 16) && aligned(a.res, 16) && aligned(a.res_out, 16) && aligned(a.y, a.y_type == TFL_E4M3 ? 8 : 16);
  const bool params = aligned(a.gamma, 16) && aligned(a.beta, 16);
  const LnPlan p = ln_forward_plan(a.D, a.rows, a.res_type == TFL_F32, lines, params, num_sms);
  if (p.form == TFL_LN_FORM_ANY) {
    const int64_t most = (int64_t)num_sms * 8;
    return launch_dependent(ln_forward_any_kernel, (unsigned)(a.rows < most ? a.rows : most), 256, 0, s, a);
  }
  return with_types(a.x_type, a.res_type, [&](auto x, auto r) {
    using X = decltype(x);
    using R = decltype(r);
    if (p.form == TFL_LN_FORM_VALUES) {
      const unsigned n = (unsigned)a.rows;
      LnArgs b = a;
      b.ahead = a.D <= 4096 ? (int64_t)num_sms * 8 : a.rows;  // none for the widest
      if (a.D <= 1024) return launch_dependent(ln_forward_values_kernel<X, R, 256, 4>, n, 256, 0, s, b);
      if (a.D <= 4096) return launch_dependent(ln_forward_values_kernel<X, R, 256, 16>, n, 256, 0, s, b);
      return launch_dependent(ln_forward_values_kernel<X, R, 1024, 8>, n, 1024, 0, s, b);
    }
    auto go = [&](auto y) {
      using Y = decltype(y);
      if (p.form == TFL_LN_FORM_VECTORS) return forward<X, R, Y>(a, p, num_sms, s);
      return p.threads == 256   ? forward_straddle<X, R, Y, 256, 3>(a, num_sms, s)
             : p.threads == 512 ? forward_straddle<X, R, Y, 512, 1>(a, num_sms, s)
                                : forward_straddle<X, R, Y, 1024, 1>(a, num_sms, s);
    };
    if (a.y_type == TFL_E4M3) return go(E4m3());
    if constexpr (sizeof(X) == 4) {
      if (a.y_type == TFL_F16) return go(__half());
      if (a.y_type == TFL_BF16) return go(__nv_bfloat16());
    }
    return go(X());
  });
}

cudaError_t launch_ln_backward(const LnGradArgs& args, int num_sms, cudaStream_t s) {
  LnGradArgs a = args;
  const bool lines = aligned(a.sum, 16) && aligned(a.dy, 16) && aligned(a.dres, 16) && aligned(a.dx, 16) && aligned(a.dsum, 16);
  const LnPlan p = ln_backward_plan(a.D, a.rows, lines, aligned(a.gamma, 16), num_sms);
  if (p.form == TFL_LN_FORM_ANY) {
    const int grid = backward_blocks(a, a.rows, num_sms * 4);
    const cudaError_t e = launch_dependent(ln_backward_any_kernel, grid, 256, 0, s, a);
    return e == cudaSuccess ? add_partials(a, grid, s) : e;
  }
  return with_types(a.x_type, a.res_type, [&](auto x, auto r) {
    using X = decltype(x);
    using R = decltype(r);
    if (p.form == TFL_LN_FORM_STRADDLE) return backward<X, R, true>(a, p, num_sms, s);
    if (p.form == TFL_LN_FORM_VECTORS) return backward<X, R, false>(a, p, num_sms, s);
    if (a.D <= 128) return backward_values<X, R, 256, 32, 4>(a, num_sms, s);
    if (a.D <= 256) return backward_values<X, R, 256, 64, 4>(a, num_sms, s);
    if (a.D <= 512) return backward_values<X, R, 256, 128, 4>(a, num_sms, s);
    if (a.D <= 1024) return backward_values<X, R, 256, 256, 4>(a, num_sms, s);
    if (a.D <= 2048) return backward_values<X, R, 512, 512, 4>(a, num_sms, s);
    if (a.D <= 4096) return backward_values<X, R, 1024, 1024, 4>(a, num_sms, s);
    if (a.D <= 6144) return backward_values<X, R, 1024, 1024, 6>(a, num_sms, s);
    return backward_values<X, R, 1024, 1024, 8>(a, num_sms, s);
  });
}

}  // namespace tfl
