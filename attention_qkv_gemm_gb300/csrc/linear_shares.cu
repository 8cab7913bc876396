// linear_shares.cu -- the linear layer's weight gradient (linear.cu) over shares of the tokens.
//
// dW = dz^T x has d_out d_in outputs and a sum over all tokens.  Where the outputs are few tiles and the tokens
// many, tiles alone leave most SMs idle (a cluster shares a tile eight ways at most), so the tokens are dealt out
// too: each share has fp32 partial sums of its own, which one more pass adds in order and rounds once.
// 41798 x 120 x 224 bf16: dW 11.5 us and 3.4 for the sum, the whole backward 50.0 -> 37 us; 65536 x 128 x 384
// fp16 50.1 -> 46.7.
#include "tile_gemm.cuh"

namespace tfl {

#define TFL_SHARE_VARIANTS(X) X(2, kWide) X(2, kNarrow) X(1, kNarrow)

cudaError_t prepare_linear_shares() {
  cudaError_t e = cudaSuccess;
#define TFL_PREP(CG, FORM) \
  if (e == cudaSuccess) e = prepare_one<CG, GRAD_DW, false, FORM, kEpiF32>();
  TFL_SHARE_VARIANTS(TFL_PREP)
#undef TFL_PREP
  return e;
}

cudaError_t launch_linear_shares(const TilePlan& p, const TileMaps& mp, const TileArgs& a, cudaStream_t s) {
  const int form = tile_form(p, GRAD_DW) == TFL_GLU_FORM_WIDE ? kWide : kNarrow;
#define TFL_LAUNCH(CG, FORM) \
  if (p.cg == CG && form == FORM) return launch_one<CG, GRAD_DW, false, FORM, kEpiF32>(mp, a, p, s);
  TFL_SHARE_VARIANTS(TFL_LAUNCH)
#undef TFL_LAUNCH
  return cudaErrorInvalidValue;
}

namespace {

// out = the sum of `shares` planes of `values`: four values a lane, the shares dealt out to the eight warps of a
// block and joined in warp order.
template <bool BF16>
__global__ void __launch_bounds__(256) share_sums_kernel(const float* parts, int shares, int64_t values, uint16_t* out) {
  __shared__ float4 red[8][32];
  grid_launch_dependents();
  grid_wait_prior();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t at = ((int64_t)blockIdx.x * 32 + lane) * 4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (at < values) {
#pragma unroll 4
    for (int k = warp; k < shares; k += 8) {
      const float4 a = *reinterpret_cast<const float4*>(parts + (size_t)k * values + at);
      v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
    }
  }
  red[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || at >= values) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) {
    const float4 a = red[k][lane];
    v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
  }
  const float f[8] = {v.x, v.y, v.z, v.w, 0.f, 0.f, 0.f, 0.f};
  uint4 o;
  pack16<8>(f, &o, BF16);
  *reinterpret_cast<uint2*>(out + at) = make_uint2(o.x, o.y);
}

}  // namespace

cudaError_t launch_share_sums(const float* parts, int shares, int64_t values, bool bf16, uint16_t* out, cudaStream_t s) {
  const unsigned grid = (unsigned)((values / 4 + 31) / 32);
  return bf16 ? launch_dependent(share_sums_kernel<true>, grid, 256, 0, s, parts, shares, values, out)
              : launch_dependent(share_sums_kernel<false>, grid, 256, 0, s, parts, shares, values, out);
}

}  // namespace tfl
