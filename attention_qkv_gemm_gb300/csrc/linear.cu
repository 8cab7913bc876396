// linear.cu -- the linear layer with its epilogue, y = act(x W^T + b) + res, forward and backward.
//
// Forward: the tiled tcgen05 kernel (tile_gemm.cuh) in mode LIN_FORWARD (a translation unit for each form of
// it: linear_wide.cu, linear_pair.cu, linear_lone.cu, linear_shared.cu).  Bias, activation and residual are
// applied to the fp32 accumulators, so only y is rounded, once; for training z = x W^T + b is stored too,
// rounded to the operands' type, since the backward would need the whole product again for act'(z)
// (half as much work as both gradients) where reading z costs 2 bytes a value.
//
// Backward, with dz = dy act'(z):
//   dx = dz W       GRAD_DX of the same kernel, W read as [k, n] (MN-major)
//   dW = dz^T x     GRAD_DW, a sum over the tokens, both operands MN-major; where the outputs are few tiles, over
//                   shares of the tokens (linear_shares.cu)
//   db = sum dz     and dz itself, in one pass over dy and z; fp32 sums of the unrounded dz
// dz is rounded to the operands' type, which the tensor cores take.  Without an activation and with dy of
// that type it is dy, and the pass only adds up its columns.
//
// What bounds it: with many tokens and long rows the tensor cores and the power cap (100000 x 4096 x 1024 bf16 with an
// fp32 residual and output 507 us in a burst, 1.65 PFLOP/s, 581 in a long run; 439 with 16-bit output alone;
// the backward of 16384 x 2048 x 8192 with GELU 790 us, 120 of them dz); with short rows the epilogue and memory
// (65536 x 128 x 384 fp16 14.4 us, 4.6 TB/s; 8192 x 1024 x 4096 fp16 GELU 44.7 us and 52.7 with z).
//
// Sums over d_in are the tensor cores' fp32 accumulation, which need not round to nearest: an fp32 y of 4096
// products is off by 2e-6 of its size where sums rounded to nearest are off by 3e-7 (a 16-bit y's own rounding: 4e-3
// in bf16, 5e-4 in fp16).
#include "tile_gemm.cuh"

#include "rowops.cuh"

namespace tfl {

cudaError_t prepare_linear_kernels() {
  cudaError_t e = prepare_linear_wide();
  if (e == cudaSuccess) e = prepare_linear_pair();
  if (e == cudaSuccess) e = prepare_linear_lone();
  if (e == cudaSuccess) e = prepare_linear_shares();
  return e == cudaSuccess ? prepare_linear_shared() : e;
}

cudaError_t launch_linear(const TilePlan& p, bool f8, const TileMaps& mp, const TileArgs& a, cudaStream_t s) {
  switch (tile_form(p, LIN_FORWARD)) {
    case TFL_GLU_FORM_WIDE: return launch_linear_wide(p, f8, mp, a, s);
    case TFL_GLU_FORM_PAIR: return launch_linear_pair(p, f8, mp, a, s);
    case TFL_GLU_FORM_SHARED: return launch_linear_shared(p, f8, mp, a, s);
  }
  return launch_linear_lone(p, f8, mp, a, s);
}

namespace {

// z within +-1e4, where the slopes are 0 and 1 to the last bit: at infinity their products are no numbers.
__device__ __forceinline__ float bounded(float z) { return fabsf(z) > 1e4f ? copysignf(1e4f, z) : z; }

// dz = dy act'(z) and this block's sums of its columns: TX threads across 8 columns each, 256 / TX rows at
// a time, the rows of a column slab shared out to gridDim.y blocks.  Every value is read once: bandwidth
// bounds it (2979 x 2856 fp32 to fp16, 51 MB: 11.4 us from cold caches, 4.5 TB/s).
template <class DY, class T, int ACT>
__global__ void __launch_bounds__(256, ACT == TFL_ACT_NONE ? 5 : 4) lin_slopes_kernel(const LinSlopeArgs a) {
  constexpr int AT_ONCE = sizeof(DY) == 4 ? 2 : 4;  // rows in flight a thread
  __shared__ float part[256 * 8];
  grid_launch_dependents();
  grid_wait_prior();
  const int tx = a.tx, x = threadIdx.x & (tx - 1), y = threadIdx.x / tx, ys = 256 / tx;
  const int c = (blockIdx.x * tx + x) * 8;
  const bool in = c < a.cols;
  // whole turns of the block's rows
  const int64_t turns = (a.rows + ys - 1) / ys, t0 = turns * blockIdx.y / gridDim.y, t1 = turns * (blockIdx.y + 1) / gridDim.y;
  const int64_t end = t1 * ys < a.rows ? t1 * ys : a.rows;
  const DY* dy = static_cast<const DY*>(a.dy) + c;
  const T* z = reinterpret_cast<const T*>(a.z) + c;
  T* dz = reinterpret_cast<T*>(a.dz) + c;
  uint64_t sum[4] = {0, 0, 0, 0};  // two zeros each
  for (int64_t row = t0 * ys + y; row < end; row += AT_ONCE * ys) {
    Raw8<DY> d1[AT_ONCE];
    Raw8<T> z1[AT_ONCE];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      const int64_t r = row + (int64_t)j * ys;
      if (in && r < end) {
        load_raw(dy + (size_t)r * a.cols, d1[j]);
        if (ACT != TFL_ACT_NONE) load_raw(z + (size_t)r * a.cols, z1[j]);
      } else {
        zero_raw(d1[j]);
        zero_raw(z1[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      const int64_t r = row + (int64_t)j * ys;
      uint64_t d[4];
      widen2(d1[j], d);
      if constexpr (ACT != TFL_ACT_NONE) {
        float f[8];
        widen(z1[j], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // an infinite z (fp16 overflows past 65504) has the slope of a large one; a NaN stays one
          uint64_t unused, slope;
          act2<ACT, true>(f2_pack(bounded(f[2 * i]), bounded(f[2 * i + 1])), unused, slope);
          d[i] = f2_mul(d[i], slope);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = f2_add(sum[i], d[i]);
      if (a.dz && in && r < end) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_unpack(d[i], o[2 * i], o[2 * i + 1]);
        store8(dz + (size_t)r * a.pitch, o);
      }
    }
  }
  if (!a.db) return;
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(sum[i], f[2 * i], f[2 * i + 1]);
  store8(part + threadIdx.x * 8, f);
  __syncthreads();
  for (int i = threadIdx.x; i < tx * 8; i += 256) {
    const int col = blockIdx.x * tx * 8 + i;
    float v = 0.f;
    for (int k = 0; k < ys; ++k) v += part[k * tx * 8 + i];
    if (col < a.cols) a.partial[(size_t)blockIdx.y * a.cols + col] = v;
  }
}

template <class DY, class T>
cudaError_t slopes(LinSlopeArgs a, int num_sms, cudaStream_t s, int* parts) {
  a.tx = pow2_at_least(a.cols / 8);
  if (a.tx > 32) a.tx = 32;
  const int64_t slabs = (a.cols / 8 + a.tx - 1) / a.tx, ys = 256 / a.tx, turns = (a.rows + ys - 1) / ys;
  // Blocks of a slab: four an SM, with rows for a few turns each (2957 x 672 fp16 GELU in 1110 blocks of one turn
  // 12.9 us, in 279 6.3), but no fewer than two an SM that have rows at all (204 x 336 in 84 blocks 6.2, in 324 4.8).
  int64_t n = ((int64_t)num_sms * 4 + slabs - 1) / slabs;
  const int64_t few = (turns + 3) / 4, fill = ((int64_t)num_sms * 2 + slabs - 1) / slabs;
  if (n > few) n = few > fill ? few : fill < turns ? fill : turns;
  if (n > a.blocks) n = a.blocks;
  if (n > 65535) n = 65535;
  const bool lone = n == 1;
  if (lone) a.partial = a.db;
  const dim3 grid((unsigned)slabs, (unsigned)n);
  *parts = a.db && !lone ? (int)n : 0;
  return a.act == TFL_ACT_SILU   ? launch_dependent(lin_slopes_kernel<DY, T, TFL_ACT_SILU>, grid, 256, 0, s, a)
         : a.act == TFL_ACT_GELU ? launch_dependent(lin_slopes_kernel<DY, T, TFL_ACT_GELU>, grid, 256, 0, s, a)
                                 : launch_dependent(lin_slopes_kernel<DY, T, TFL_ACT_NONE>, grid, 256, 0, s, a);
}

}  // namespace

cudaError_t launch_lin_slopes(const LinSlopeArgs& a, int num_sms, cudaStream_t s, int* parts) {
  if (a.type == TFL_F16)
    return a.dy_type == TFL_F32 ? slopes<float, __half>(a, num_sms, s, parts) : slopes<__half, __half>(a, num_sms, s, parts);
  return a.dy_type == TFL_F32 ? slopes<float, __nv_bfloat16>(a, num_sms, s, parts)
                              : slopes<__nv_bfloat16, __nv_bfloat16>(a, num_sms, s, parts);
}

cudaError_t launch_lin_db(const LinSlopeArgs& a, int parts, cudaStream_t s) {
  return launch_column_sums(a.partial, parts, a.cols, a.cols, a.cols, a.db, nullptr, s);
}

}  // namespace tfl
