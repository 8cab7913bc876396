// linear_few.cu -- the linear layer's forward for a few tokens (at most 16).
//
// The weights are read once for a handful of rows: d_out d_in elements bound it, so what counts is loads
// in flight, an even share for every SM and a short start.  As in glu_few.cu there is no shared-memory
// ring, tensor memory or TMA, and a lane's fragment words come from 16 consecutive bytes of its row
// (the order of k is free as long as both operands agree).  Here the tokens are the 16 rows of an m16n8
// MMA's A operand and 8 rows of W its B operand, so that a warp needs only 8 output columns: one matrix
// has half the rows of the feed-forward's two, and d_out may be no more than a few per SM.  The warps of
// a block split k and are joined in shared memory, in warp order.
#include <type_traits>

#include "mathfn.cuh"
#include "ops.h"

namespace tfl {

namespace {

template <int TYPE>
__device__ __forceinline__ void mma_step(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
#define TFL_MMA(SHAPE_TYPES)                                                                               \
  asm("mma.sync.aligned." SHAPE_TYPES " {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"             \
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                                     \
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if constexpr (TYPE == TFL_F16) TFL_MMA("m16n8k16.row.col.f32.f16.f16.f32");
  if constexpr (TYPE == TFL_BF16) TFL_MMA("m16n8k16.row.col.f32.bf16.bf16.f32");
  if constexpr (TYPE == TFL_E4M3) TFL_MMA("m16n8k32.row.col.f32.e4m3.e4m3.f32");
#undef TFL_MMA
}

// Weights are read once by one warp: no place in L1.
__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// TYPE: of the operands; NT: token groups of 8; G: column groups of 8 a warp; U: 64-byte steps of a row in
// flight a warp, 512 G bytes of weights each; LINES: 128-byte lines of them, a row and warp, that are
// prefetched.
template <int TYPE, int NT, int G, int U, int LINES>
__global__ void __launch_bounds__(256) lin_few_kernel(const LinFewArgs a) {
  __shared__ float red[8][G * 4][32];
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int f0 = blockIdx.x * (8 * G);
  const int row_bytes = a.row_bytes;
  float acc[G][4];
#pragma unroll
  for (int n = 0; n < G; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  // This lane's token of each group (past the last: the last again, not stored).  x and its scales may
  // still be written while this kernel starts: plain loads, behind the wait.
  const uint8_t* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xr[n] = a.x + (size_t)min(n * 8 + r, a.tokens - 1) * row_bytes + c * 16;
  const uint8_t* w[G];  // (past the last column: the last group again, not stored)
#pragma unroll
  for (int n = 0; n < G; ++n) w[n] = a.w + (size_t)min(f0 + n * 8 + r, a.d_out - 8 + r) * row_bytes + c * 16;
  auto steps = [&](int base, auto whole) {  // U steps, all of them inside the row or not
    uint4 wv[U][G], x[U][NT];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int off = base + j * 64;
      const bool in = decltype(whole)::value || off + c * 16 < row_bytes;  // rows are 16-byte pieces
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int n = 0; n < G; ++n) wv[j][n] = in ? load_once(w[n] + off) : zero;
#pragma unroll
      for (int n = 0; n < NT; ++n) x[j][n] = in ? *reinterpret_cast<const uint4*>(xr[n] + off) : zero;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint4 x0 = x[j][0], x1 = NT == 2 ? x[j][NT - 1] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int n = 0; n < G; ++n) {
        mma_step<TYPE>(acc[n], x0.x, x1.x, x0.y, x1.y, wv[j][n].x, wv[j][n].y);
        mma_step<TYPE>(acc[n], x0.z, x1.z, x0.w, x1.w, wv[j][n].z, wv[j][n].w);
      }
    }
  };
  int base = warp * (U * 64);
  // The weights of the first steps set out for L2 while the kernels before this one still run (what
  // they write is only read after the wait).
#pragma unroll
  for (int i = 0; i < LINES * G; i += 4) {
    const int at = i + (lane >> 3), row = f0 + (at % G) * 8 + (lane & 7), off = base + at / G * 128;
    if (at < LINES * G && row < a.d_out && off < row_bytes) prefetch_l2(a.w + (size_t)row * row_bytes + off);
  }
  grid_wait_prior();
  for (; base + U * 64 <= row_bytes; base += warps * (U * 64)) steps(base, std::true_type());
  if (base < row_bytes) steps(base, std::false_type());
#pragma unroll
  for (int n = 0; n < G; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp][n * 4 + i][lane] = acc[n][i];
  __syncthreads();
  // accumulator word i of a lane: token lane / 4 (+ 8 for i >= 2), column 2 (lane % 4) + i % 2
  for (int i = threadIdx.x; i < NT * G * 64; i += blockDim.x) {
    const int f8 = i & 7, n = (i >> 3) % G, t = i / (8 * G);  // column of a group, group, token
    const int f = f0 + n * 8 + f8, word = n * 4 + (t >> 3) * 2 + (f8 & 1), l = (t & 7) * 4 + (f8 >> 1);
    if (t >= a.tokens || f >= a.d_out) continue;
    float z = 0.f;
    for (int k = 0; k < warps; ++k) z += red[k][word][l];
    if constexpr (TYPE == TFL_E4M3) z *= a.x_scale[t] * a.w_scale[f];
    if (a.bias) z += a.bias[f];
    const size_t at = (size_t)t * a.d_out + f;
    auto round16 = [&](float v) {
      return a.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
    };
    if (a.z) a.z[at] = round16(z);
    float y = a.act == TFL_ACT_SILU   ? z * rcp_approx(1.0f + ex2(z * -1.4426950408889634f))
              : a.act == TFL_ACT_GELU ? gelu_as7126(z)
                                      : z;
    if (a.out_f32) {
      if (a.res) y += static_cast<const float*>(a.res)[at];
      static_cast<float*>(a.out)[at] = y;
    } else {
      if (a.res) {
        const uint16_t v = static_cast<const uint16_t*>(a.res)[at];
        y += a.bf16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
      }
      static_cast<uint16_t*>(a.out)[at] = round16(y);
    }
  }
}

// Warps a block (they split k): as few as still give every SM 24 warps, no more than a row feeds.
int few_warps(const LinFewArgs& a, int g, int u, int num_sms) {
  int warps = 2;
  while (warps < 8 && warps * u * 64 < a.row_bytes && (int64_t)(a.d_out / (8 * g)) * warps < (int64_t)num_sms * 24) warps *= 2;
  return warps;
}

template <int TYPE, int NT, int G, int U, int LINES>
cudaError_t launch_form(const LinFewArgs& a, int num_sms, cudaStream_t s) {
  return launch_dependent(lin_few_kernel<TYPE, NT, G, U, LINES>, (a.d_out + 8 * G - 1) / (8 * G),
                          few_warps(a, G, U, num_sms) * 32, 0, s, a);
}

template <int TYPE>
cudaError_t launch_type(const LinFewArgs& a, int num_sms, cudaStream_t s) {
  if (a.tokens > 8) return launch_form<TYPE, 2, 1, 4, 2>(a, num_sms, s);
  return launch_form<TYPE, 1, 1, 8, 4>(a, num_sms, s);
}

}  // namespace

bool lin_few_fits(int64_t tokens, int64_t row_bytes) {
  return (tokens <= 8 && row_bytes <= 16 * 1024) || (tokens <= kLinFewTokens && tokens * row_bytes <= 32 * 1024);
}

cudaError_t launch_lin_few(int type, const LinFewArgs& a, int num_sms, cudaStream_t s) {
  if (type == TFL_F16) return launch_type<TFL_F16>(a, num_sms, s);
  if (type == TFL_BF16) return launch_type<TFL_BF16>(a, num_sms, s);
  return launch_type<TFL_E4M3>(a, num_sms, s);
}

}  // namespace tfl
