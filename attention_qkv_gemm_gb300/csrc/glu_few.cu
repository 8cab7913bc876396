// glu_few.cu -- the gated feed-forward forward for a few tokens (at most 16).
//
// The weights are read once for a handful of rows: 2 d_ff d_model elements bound it, so what
// counts is loads in flight, an even share for every SM and a short start.  No shared-memory
// ring, tensor memory or TMA: a warp takes 8 output columns, with their 8 gate rows and 8 up rows
// as the 16 rows of an m16n8 MMA's A operand, read straight from global memory into the
// fragment's registers.  The MMA sums over k, whose order is free as long as both operands agree:
// each lane's fragment words are taken from 16 consecutive bytes of its row, so that four lanes
// read 64 bytes of a row and one 16-byte load serves two MMAs.  Gate and up of a column and token
// land in the same thread.  The warps of a block split k and are joined in shared memory, in warp
// order.
// One token x 1024 x 4096 bf16 takes 3.8 us (16.8 MB; 5.9 us in the tiled kernel), 8 tokens x 4096 x
// 10240 27 us in bf16 (168 MB, 0.92 of the copy bandwidth) and 15 us in e4m3.
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

// TYPE: of the operands; NT: token tiles of 8; U: 64-byte steps of a row in flight a warp, 1 KB of weights
// each; LINES: 128-byte lines of them, a row and warp, that are prefetched.
template <int TYPE, int NT, int U, int LINES>
__global__ void __launch_bounds__(256) glu_few_kernel(const GluFewArgs a) {
  __shared__ float red[8][NT * 4][32];
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int f0 = blockIdx.x * 8;
  const int row_bytes = a.row_bytes;
  const size_t row0 = (size_t)(f0 + r) * row_bytes + c * 16;
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  // This lane's token of each tile (past the last: the last again, not stored).  x and its scales may
  // still be written while this kernel starts: plain loads, behind the wait.
  const uint8_t* xr[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) xr[n] = a.x + (size_t)min(n * 8 + r, a.tokens - 1) * row_bytes + c * 16;
  const uint8_t *wg = a.wg + row0, *wu = a.wu + row0;
  auto steps = [&](int base, auto whole) {  // U steps, all of them inside the row or not
    uint4 g[U], u[U], x[U][NT];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int off = base + j * 64;
      const bool in = decltype(whole)::value || off + c * 16 < row_bytes;  // rows are 16-byte pieces
      const uint4 zero = make_uint4(0, 0, 0, 0);
      g[j] = in ? load_once(wg + off) : zero;
      u[j] = in ? load_once(wu + off) : zero;
#pragma unroll
      for (int n = 0; n < NT; ++n) x[j][n] = in ? *reinterpret_cast<const uint4*>(xr[n] + off) : zero;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_step<TYPE>(acc[n], g[j].x, u[j].x, g[j].y, u[j].y, x[j][n].x, x[j][n].y);
        mma_step<TYPE>(acc[n], g[j].z, u[j].z, g[j].w, u[j].w, x[j][n].z, x[j][n].w);
      }
    }
  };
  int base = warp * (U * 64);
  // The weights of the first steps set out for L2 while the kernels before this one still run (what
  // they write is only read after the wait).
#pragma unroll
  for (int i = 0; i < LINES / 2; ++i) {
    const int row = f0 + (lane & 7), off = base + (i * 2 + (lane >> 4)) * 128;
    if (off < row_bytes) prefetch_l2((lane & 8 ? a.wu : a.wg) + (size_t)row * row_bytes + off);
  }
  grid_wait_prior();
  for (; base + U * 64 <= row_bytes; base += warps * (U * 64)) steps(base, std::true_type());
  if (base < row_bytes) steps(base, std::false_type());
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp][n * 4 + i][lane] = acc[n][i];
  __syncthreads();
  // accumulator word i of a lane: i < 2 gate, else up; column lane / 4; token 2 (lane % 4) + i % 2
  for (int i = threadIdx.x; i < NT * 64; i += blockDim.x) {
    const int l = i & 31, odd = (i >> 5) & 1, n = i >> 6;
    const int t = n * 8 + (l & 3) * 2 + odd, f = f0 + (l >> 2);
    if (t >= a.tokens) continue;
    float g = 0.f, u = 0.f;
    for (int w = 0; w < warps; ++w) {
      g += red[w][n * 4 + odd][l];
      u += red[w][n * 4 + 2 + odd][l];
    }
    if constexpr (TYPE == TFL_E4M3) {
      const float sx = a.x_scale[t];
      g *= sx * __ldg(a.g_scale + f);
      u *= sx * __ldg(a.u_scale + f);
    }
    const float act = a.act == TFL_ACT_SILU ? g * rcp_approx(1.0f + ex2(g * -1.4426950408889634f)) : gelu_as7126(g);
    const size_t at = (size_t)t * a.d_ff + f;
    if (a.bf16_out)
      reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(act * u);
    else
      reinterpret_cast<__half*>(a.out)[at] = __float2half_rn(act * u);
  }
}

// Warps a block (they split k): as few as still give every SM 24 warps, no more than a row feeds.
int few_warps(const GluFewArgs& a, int u, int num_sms) {
  int warps = 2;
  while (warps < 8 && warps * u * 64 < a.row_bytes && (int64_t)(a.d_ff / 8) * warps < (int64_t)num_sms * 24) warps *= 2;
  return warps;
}

// Eight steps in flight a warp for 16-bit rows that feed as many warps with them and leave the last
// round of a row's steps (warps x U x 64 bytes each) nearly full: 8 tokens x 2048 x 8192 bf16 11.7 us,
// 14.2 with four, but 1024 x 4096 5.6 against 4.1 us, 2600 x 1200 9.0 against 6.9, 8192 x 4096 e4m3 12.9
// against 12.2.  A row of one round is prefetched whole (1280 x 5120 5.1 us, 8.2 with two lines of
// four); of more rounds two lines are enough (2048 x 8192 11.5 us, whole 12.7).
template <int TYPE>
cudaError_t launch_type(const GluFewArgs& a, int num_sms, cudaStream_t s) {
  const int groups = a.d_ff / 8, w8 = few_warps(a, 8, num_sms), w4 = few_warps(a, 4, num_sms);
  if (a.tokens > 8) return launch_dependent(glu_few_kernel<TYPE, 2, 4, 2>, groups, w4 * 32, 0, s, a);
  if constexpr (TYPE != TFL_E4M3) {
    const int round = w8 * 8 * 64, rounds = (a.row_bytes + round - 1) / round;
    if (a.row_bytes > 2048 && rounds == 1) return launch_dependent(glu_few_kernel<TYPE, 1, 8, 4>, groups, w8 * 32, 0, s, a);
    if (rounds > 1 && a.row_bytes * 8 >= rounds * round * 7)
      return launch_dependent(glu_few_kernel<TYPE, 1, 8, 2>, groups, w8 * 32, 0, s, a);
  }
  return launch_dependent(glu_few_kernel<TYPE, 1, 4, 2>, groups, w4 * 32, 0, s, a);
}

}  // namespace

// Every block reads all of x, from its SM's L1 as long as the rows fit there beside one another:
// 16 tokens of 2 KB (1024 x 4096 bf16) take 4.2 us here and 5.9 us in the tiled kernel, 16 tokens
// of 8 KB (4096 x 10240) 42 us here and 28 us there.  Up to 8 tokens, rows of up to 16 KB, this kernel
// starts sooner behind the norm before it (together: one token x 2048 x 8192 bf16 14.0 us, 16.6 with the
// tiled kernel, 8 x 8192 x 4096 e4m3 16.8 against 20.3) and is faster alone (11.5 against 13.0); blocks
// that between them walk thousands of longer rows get less from memory (16384 x 8192 bf16: 159 us
// against 87 us).
bool glu_few_fits(int64_t tokens, int64_t row_bytes) {
  return (tokens <= 8 && row_bytes <= 16 * 1024) || (tokens <= kGluFewTokens && tokens * row_bytes <= 32 * 1024);
}

cudaError_t launch_glu_few(int type, const GluFewArgs& a, int num_sms, cudaStream_t s) {
  if (type == TFL_F16) return launch_type<TFL_F16>(a, num_sms, s);
  if (type == TFL_BF16) return launch_type<TFL_BF16>(a, num_sms, s);
  return launch_type<TFL_E4M3>(a, num_sms, s);
}

}  // namespace tfl
