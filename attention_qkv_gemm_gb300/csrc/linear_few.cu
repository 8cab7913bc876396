// linear_few.cu -- the linear layer's forward for a few tokens (at most 16).
//
// The weights are read once for a handful of rows: d_out d_in elements bound it, so what counts is loads
// in flight, an even share for every SM and a short start.  As in glu_few.cu there is no shared-memory
// ring, tensor memory or TMA, and a lane's fragment words come from 16 consecutive bytes of its row
// (the order of k is free as long as both operands agree).  Here the tokens are the 16 rows of an m16n8
// MMA's A operand and 8 rows of W its B operand, so that a warp needs only 8 output columns: one matrix
// has half the rows of the feed-forward's two, and d_out may be no more than a few per SM.  The warps of
// a block split k and are joined in shared memory, in warp order.
//
// 1 x 1024 x 4096 bf16 3.4 us in a graph (2.5 TB/s of weights; a launch and a round trip to memory), 3.7 by calls;
// 16 x 4096 x 4096 8.1 us, 4.1 TB/s.
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
__global__ void __launch_bounds__(512) lin_few_kernel(const LinFewArgs a) {
  __shared__ float red[16][G * 4][32];
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

// A warp loads all its steps, then multiplies: so a row in one turn of a block's warps (up to sixteen, four
// steps each; two turns of 8 KB rows), 8 columns a block where the GPU holds all blocks at once and 16 where
// it does not: a second wave of blocks costs more than their loads (one token x 2048 x 8192 bf16, 1024 blocks of
// sixteen warps 11.5 us, 512 of them 7.0).
struct FewForm {
  int g = 0, warps = 0;  // column groups of a block; 0: none fits
};
FewForm few_form(int64_t row_bytes, int64_t d_out, int num_sms) {
  int w = 1;
  while (w < 16 && w * 256 < row_bytes) w *= 2;
  // columns the GPU holds at once: `regs` registers a thread
  auto wave = [&](int g, int warps, int regs) {
    const int by_registers = 65536 / (regs * warps * 32), by_warps = 64 / warps, most = by_registers < by_warps ? by_registers : by_warps;
    return (int64_t)num_sms * (most < 32 ? most : 32) * 8 * g;
  };
  if (d_out <= wave(1, w, 40)) return {1, w};
  if (d_out <= wave(2, w, 60)) return {2, w};
  if (w > 1 && d_out <= wave(2, w / 2, 60)) return {2, w / 2};
  return {};
}

template <int TYPE, int NT>
cudaError_t launch_tokens(const LinFewArgs& a, int num_sms, cudaStream_t s) {
  const FewForm f = few_form(a.row_bytes, a.d_out, num_sms);
  if (f.g == 1) return launch_dependent(lin_few_kernel<TYPE, NT, 1, 4, 2>, a.d_out / 8, f.warps * 32, 0, s, a);
  return launch_dependent(lin_few_kernel<TYPE, NT, 2, 4, 2>, (a.d_out + 15) / 16, f.warps * 32, 0, s, a);
}

template <int TYPE>
cudaError_t launch_type(const LinFewArgs& a, int num_sms, cudaStream_t s) {
  return a.tokens > 8 ? launch_tokens<TYPE, 2>(a, num_sms, s) : launch_tokens<TYPE, 1>(a, num_sms, s);
}

}  // namespace

// Against the tiled kernel (in graphs): 8 tokens x 1024 x 4096 bf16 3.6 against 6.2 us, 16 x 4096 x 4096 8.1
// against 9.8, but rows of 16 KB or weights that take a second wave of blocks are the tiled kernel's (8 x 8192 x
// 512 8.5 against 7.8, 8 x 4096 x 16384 27.7 against 23.1), and e4m3 weights past 16 MB with two groups of tokens
// (16 x 8192 x 4096 12.3 against 10.0).  The limit on the row goes by its bytes alone: at 4096 columns of 16 KB rows this
// kernel would still be ahead (4 to 16 tokens 13.2 to 13.6 us against 14.5 to 14.7).
bool lin_few_fits(int64_t tokens, int64_t row_bytes, int64_t d_out, bool f8, int num_sms) {
  if (tokens > kLinFewTokens || row_bytes > 8192 || (f8 && tokens > 8 && row_bytes * d_out > (16 << 20))) return false;
  return few_form(row_bytes, d_out, num_sms).g != 0;
}

cudaError_t launch_lin_few(int type, const LinFewArgs& a, int num_sms, cudaStream_t s) {
  if (type == TFL_F16) return launch_type<TFL_F16>(a, num_sms, s);
  if (type == TFL_BF16) return launch_type<TFL_BF16>(a, num_sms, s);
  return launch_type<TFL_E4M3>(a, num_sms, s);
}

}  // namespace tfl
