// tile_gemm.cuh -- the persistent tcgen05 matrix-product kernel behind the gated feed-forward (glu.cu)
// and the linear layer (linear.cu), fp32 accumulation in tensor memory.
//
// Structure: warp 0 feeds a ring of k-blocks (128 bytes of k a row, 128-byte swizzle) by TMA,
// warp 1 issues the MMAs, the others are the epilogue (two or four per tensor-memory lane quarter), two
// accumulators so that a tile's epilogue runs under the next tile's MMAs.
//
// Ragged sizes: TMA fills what lies outside a matrix with zeros (zero rows and zero k add
// nothing), and the epilogue stores only rows and columns that exist.
#pragma once
#include "cluster.cuh"
#include "mathfn.cuh"
#include "ops.h"
#include "xpose.cuh"

namespace tfl {

namespace {

constexpr int kKBytes = 128;       // bytes of k a row and stage
constexpr int kMnChunk = 64 * 128; // MN-major operands: 64 k rows of 64 values

constexpr int kMaxBN = 256;        // accumulator columns of a tile, at most
constexpr int kMaxStages = 12;
// Shared memory: ring, one 32-row transpose stage an epilogue warp, barriers.
constexpr int kBarrierBytes = 256;
__host__ __device__ constexpr int xpose_bytes(bool sixteen) { return sixteen ? 32768 : 16384; }
constexpr int kTileSmem = 232448;
// lin: two stages a warp that TMA swizzles (on 512 bytes), and a barrier for each.
constexpr int kLinStage = 2048, kLinRing = 161 * 1024;
constexpr int kLinResBar = 31;  // the first of those barriers, behind the others
__host__ __device__ constexpr int ring_bytes(bool wide, bool lin = false) {
  return lin ? kLinRing : kTileSmem - 1024 - xpose_bytes(wide) - kBarrierBytes;
}
static_assert(1024 + kLinRing + 32 * kLinStage + (kLinResBar + 32) * 8 <= kTileSmem, "shared memory");

// The activation of a packed pair of fp32 values (FMA-pipe work runs two lanes an instruction;
// the busy epilogue warps otherwise take issue slots from the thread that issues the MMAs):
// a = act(g) and, when wanted, slope = act'(g).
//   SiLU  p = 1 / (1 + e^-g);  a = g p,  slope = p + p (g - a)
//   GELU  exact erf form, erf from Abramowitz & Stegun 7.1.26 as in gelu_as7126 (its packed form takes
//         max(g, 0) - |g| erfc / 2, which is no number at +infinity):
//         a = g Phi(g),  slope = Phi(g) + g phi(g)
template <int ACT, bool SLOPE>
__device__ __forceinline__ void act2(uint64_t g, uint64_t& a, uint64_t& slope) {
  if constexpr (ACT == TFL_ACT_SILU) {
    float e0, e1;
    f2_unpack(f2_mul(g, f2_splat(-1.4426950408889634f)), e0, e1);
    f2_unpack(f2_add(f2_pack(ex2(e0), ex2(e1)), f2_splat(1.0f)), e0, e1);
    const uint64_t p = f2_pack(rcp_approx(e0), rcp_approx(e1));
    a = f2_mul(g, p);
    if constexpr (SLOPE) slope = f2_fma(p, f2_sub(g, a), p);
  } else {
    constexpr float p_s = 0.3275911f * 0.7071067811865476f;
    constexpr float h1 = 0.5f * 0.254829592f, h2 = 0.5f * -0.284496736f, h3 = 0.5f * 1.421413741f,
                    h4 = 0.5f * -1.453152027f, h5 = 0.5f * 1.061405429f;
    float x0, x1, d0, d1;
    f2_unpack(g, x0, x1);
    f2_unpack(f2_fma(f2_pack(fabsf(x0), fabsf(x1)), f2_splat(p_s), f2_splat(1.0f)), d0, d1);
    const uint64_t t = f2_pack(rcp_approx(d0), rcp_approx(d1));
    uint64_t poly = f2_fma(f2_splat(h5), t, f2_splat(h4));
    poly = f2_fma(poly, t, f2_splat(h3));
    poly = f2_fma(poly, t, f2_splat(h2));
    poly = f2_fma(poly, t, f2_splat(h1));
    f2_unpack(f2_mul(f2_mul(g, g), f2_splat(-0.7213475204444817f)), d0, d1);
    const uint64_t e = f2_pack(ex2(d0), ex2(d1));
    f2_unpack(f2_mul(f2_mul(t, poly), e), d0, d1);  // erfc(|g| / sqrt 2) / 2
    const uint64_t cdf = f2_pack(x0 >= 0.f ? 1.0f - d0 : d0, x1 >= 0.f ? 1.0f - d1 : d1);
    a = f2_mul(g, cdf);
    if constexpr (SLOPE) slope = f2_fma(f2_mul(g, f2_splat(0.3989422804014327f)), e, cdf);
  }
}
// N outputs of a row: g <- act(g) u.
template <int ACT, int N>
__device__ __forceinline__ void forward_values(float* g, const float* u) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    uint64_t a, unused;
    act2<ACT, false>(f2_pack(g[i], g[i + 1]), a, unused);
    f2_unpack(f2_mul(a, f2_pack(u[i], u[i + 1])), g[i], g[i + 1]);
  }
}
// g <- act(g).  GELU as gelu2_as7126 folds it, max(g, 0) - |g| erfc / 2, with a positive g's |g| held below 1e4 so
// that +infinity's product with erfc = 0 is 0 (-infinity's stays no number, as in the other kernels and in SiLU; a
// NaN reaches erfc): two instructions a value fewer than act2's.
template <int ACT, int N>
__device__ __forceinline__ void activate(float* g) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint64_t x = f2_pack(g[i], g[i + 1]);
    if constexpr (ACT == TFL_ACT_GELU) {
      constexpr float p_s = 0.3275911f * 0.7071067811865476f;
      constexpr float h1 = 0.5f * 0.254829592f, h2 = 0.5f * -0.284496736f, h3 = 0.5f * 1.421413741f,
                      h4 = 0.5f * -1.453152027f, h5 = 0.5f * 1.061405429f;
      const uint64_t size = f2_pack(fabsf(fminf(g[i], 1e4f)), fabsf(fminf(g[i + 1], 1e4f)));
      float d0, d1;
      f2_unpack(f2_fma(size, f2_splat(p_s), f2_splat(1.0f)), d0, d1);
      const uint64_t t = f2_pack(rcp_approx(d0), rcp_approx(d1));
      // minus the polynomial, so that the last product is an addition
      uint64_t poly = f2_fma(f2_splat(-h5), t, f2_splat(-h4));
      poly = f2_fma(poly, t, f2_splat(-h3));
      poly = f2_fma(poly, t, f2_splat(-h2));
      poly = f2_fma(poly, t, f2_splat(-h1));
      f2_unpack(f2_mul(f2_mul(x, x), f2_splat(-0.7213475204444817f)), d0, d1);
      const uint64_t erfc = f2_mul(f2_mul(t, poly), f2_pack(ex2(d0), ex2(d1)));
      f2_unpack(f2_fma(size, erfc, f2_pack(fmaxf(g[i], 0.f), fmaxf(g[i + 1], 0.f))), g[i], g[i + 1]);
    } else {
      uint64_t a, unused;
      act2<ACT, false>(x, a, unused);
      f2_unpack(a, g[i], g[i + 1]);
    }
  }
}
// g <- dh u act'(g), u <- dh act(g).
template <int ACT, int N>
__device__ __forceinline__ void slope_values(float* g, float* u, const float* dh) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    uint64_t a, slope;
    act2<ACT, true>(f2_pack(g[i], g[i + 1]), a, slope);
    const uint64_t d = f2_pack(dh[i], dh[i + 1]);
    f2_unpack(f2_mul(f2_mul(d, f2_pack(u[i], u[i + 1])), slope), g[i], g[i + 1]);
    f2_unpack(f2_mul(d, a), u[i], u[i + 1]);
  }
}

template <int N>
__device__ __forceinline__ void pack16(const float* v, uint4* o, int bf16) {
  if (bf16)
    pack_bf16<N>(v, o);
  else
    pack_f16<N>(v, o, false);
}
__device__ __forceinline__ void unpack16(const uint4& w, float* v, int bf16) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// W 16-bit columns of the warp's 32 rows through the stage to global memory; rows by mask,
// columns (8 a chunk) below `cols`.
template <int W>
__device__ __forceinline__ void store_cols(uint8_t* st, int lane, const uint4* v, uint16_t* row0, size_t pitch,
                                           uint32_t rows, int cols) {
  using X = XStage<W * 2>;
  X::put_row(st, lane, v);
  __syncwarp();
  uint4 o[X::CPR];
#pragma unroll
  for (int k = 0; k < X::CPR; ++k)
    o[k] = *reinterpret_cast<const uint4*>(st + X::off(X::RPI * k + lane / X::CPR, lane % X::CPR));
  const int q = lane % X::CPR;
#pragma unroll
  for (int k = 0; k < X::CPR; ++k) {
    const int i = X::RPI * k + lane / X::CPR;
    if (((rows >> i) & 1u) && q * 8 < cols) *reinterpret_cast<uint4*>(row0 + (size_t)i * pitch + q * 8) = o[k];
  }
  __syncwarp();
}
// The same for 16 fp32 columns (32 rows of 64 bytes: a warp's whole stage).
__device__ __forceinline__ void store_cols_f32(uint8_t* st, int lane, const float* v, float* row0, size_t pitch,
                                               uint32_t rows, int cols) {
  using X = XStage<64>;
  uint4 w[4];
  pack_f32x16(v, w);
  X::put_row(st, lane, w);
  __syncwarp();
  const int q = lane % X::CPR;
  uint4 o[X::CPR];
#pragma unroll
  for (int k = 0; k < X::CPR; ++k) o[k] = *reinterpret_cast<const uint4*>(st + X::off(X::RPI * k + lane / X::CPR, q));
#pragma unroll
  for (int k = 0; k < X::CPR; ++k) {
    const int i = X::RPI * k + lane / X::CPR;
    if (((rows >> i) & 1u) && q * 4 < cols) *reinterpret_cast<uint4*>(row0 + (size_t)i * pitch + q * 4) = o[k];
  }
  __syncwarp();
}
// The 16-bit columns the same way back: this thread's row of W 16-bit columns (zeros outside).
template <int W>
__device__ __forceinline__ void load_cols(uint8_t* st, int lane, uint4* v, const uint16_t* row0, size_t pitch,
                                          uint32_t rows, int cols) {
  using X = XStage<W * 2>;
  const int q = lane % X::CPR;
  uint4 f[X::CPR];
#pragma unroll
  for (int k = 0; k < X::CPR; ++k) {
    const int i = X::RPI * k + lane / X::CPR;
    f[k] = ((rows >> i) & 1u) && q * 8 < cols
               ? *reinterpret_cast<const uint4*>(row0 + (size_t)i * pitch + q * 8)
               : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int k = 0; k < X::CPR; ++k)
    *reinterpret_cast<uint4*>(st + X::off(X::RPI * k + lane / X::CPR, q)) = f[k];
  __syncwarp();
#pragma unroll
  for (int k = 0; k < X::CPR; ++k) v[k] = *reinterpret_cast<const uint4*>(st + X::off(lane, k));
  __syncwarp();
}

// Until at most N of the warp's last tile stores still read shared memory.
template <int N>
__device__ __forceinline__ void stores_read() {
  if ((threadIdx.x & 31) == 0) bulk_wait_read<N>();
  __syncwarp();
}

// The feed-forward's e4m3 scales of output column n, gate's and up's (glu.cu).
template <int MODE>
__device__ __forceinline__ float2 column_scales(const TileArgs& args, int n);

struct Tile {
  int m, n, z;
};

// n / d for n < 2^31 by a multiplication with ceil(2^(31 + s) / d), s = ceil(log2 d) (the round-up method of
// Granlund and Montgomery): every warp finds every tile, and three divisions a tile cost it some 400 cycles.
__device__ __forceinline__ int over(int n, const Divisor& d) {
  return d.shift < 0 ? n : (int)(__umulhi((uint32_t)n, d.factor) >> d.shift);
}
// Tiles in groups of row blocks, column by column inside a group, so that the tiles in flight share
// operands through L2.  DW: plane by plane, first all of dWg, then all of dWu, or one share of the tokens
// after the other.
__device__ __forceinline__ Tile tile_at(int t, const TileOrder& o) {
  Tile r;
  r.z = over(t, o.plane);
  t -= r.z * o.plane.d;
  const int g = over(t, o.group), first = g * o.rows.d;
  t -= g * o.group.d;
  const bool whole = o.num_m - first >= o.rows.d;  // the last group of a plane may have fewer row blocks
  r.n = over(t, whole ? o.rows : o.last_rows);
  r.m = first + t - r.n * (whole ? o.rows.d : o.last_rows.d);
  return r;
}

// kWide: tiles of kMaxBN accumulator columns and 128 loaded rows of A, all sizes constants.
// kNarrow: the plan's widths.
// kSplit: the same, with the k-blocks of a tile shared out to a cluster of lone CTAs (few tiles:
// the whole GPU works on them); each CTA finishes some of the tile's 32-column pieces, and the
// others send it their sums through its shared memory, added in CTA order.  One tile a CTA.
enum TileForm : int { kWide = 0, kNarrow = 1, kSplit = 2 };
// Epilogue warps: sixteen for the wide tiles, 32 columns each, which a short k needs (8192 x 1024 x 4096
// e4m3 47.5 -> 45.4 us; the eight before computed 32 columns at a time and stored 64, these 16 and 32,
// and have the registers for it).  Eight for the narrow tiles, most of which have one or two chunks; the linear
// layer always sixteen (its tiles may have as few as one k-block).
__host__ __device__ constexpr int epi_warps(int form, bool lin) { return form == kWide || lin ? 16 : 8; }
__host__ __device__ constexpr int tile_threads(int form, int mode) { return 64 + 32 * epi_warps(form, mode == LIN_FORWARD); }
// EPI: what the linear layer's epilogue does besides bias and activation, each a kernel of its own (one for all
// spilled 600 to 1800 bytes).  GRAD_DW with kEpiF32: the planes are
// shares of the tokens, each with fp32 sums of its own.
enum EpiBits : int { kEpiF32 = 1, kEpiZ = 2, kEpiRes = 4 };  // y (and the residual) fp32; z stored; residual added
template <int CG, int MODE, bool F8, int FORM, int EPI>
__global__ void __launch_bounds__(tile_threads(FORM, MODE), 1)
    tile_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
               const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1,
                const __grid_constant__ CUtensorMap tmR, const TileArgs args) {
  constexpr bool WIDE = FORM == kWide, SPLIT = FORM == kSplit;
  static_assert(!SPLIT || CG == 1, "lone CTAs share a tile's k-blocks");
  constexpr bool TWO = MODE == GLU_FORWARD || MODE == GLU_SLOPES;  // two products side by side
  constexpr bool LIN = MODE == LIN_FORWARD;
  constexpr bool A_MN = MODE == GRAD_DW, B_MN = MODE == GRAD_DX || MODE == GRAD_DW;
  constexpr int KE = F8 ? 128 : 64;                                // k elements a stage
  extern __shared__ uint8_t smem_raw[];
  grid_launch_dependents();
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* xpose = smem + ring_bytes(WIDE, LIN);
  uint64_t* full = reinterpret_cast<uint64_t*>(xpose + (LIN ? 32 * kLinStage : xpose_bytes(WIDE)));
  uint64_t* empty = full + kMaxStages;
  uint64_t* accf = empty + kMaxStages;
  uint64_t* acce = accf + 2;
  uint64_t* drain = acce + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  uint64_t* res_bar = full + kLinResBar;  // LIN_FORWARD: two an epilogue warp
  int* never_flag = abort_flag + 1;  // stays 0: lets the drain waits ignore abort_flag

  constexpr int kWideStage = (kTileRows + kMaxBN / CG) * kKBytes;
  const int bno = WIDE ? (TWO ? kMaxBN / 2 : kMaxBN) : args.bno;  // output columns of a tile
  const int bn = TWO ? 2 * bno : bno;                             // accumulator columns
  const int stages = WIDE ? ring_bytes(true, LIN) / kWideStage : args.stages;
  const int stage_bytes = WIDE ? kWideStage : args.stage_bytes;
  const int a_bytes = WIDE ? kTileRows * kKBytes : args.a_bytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)cluster_rank() : 0;             // of the pair
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&accf[a], 1);
      mbar_init(&acce[a], CG * epi_warps(FORM, LIN));
    }
    mbar_init(drain, 1);
    if constexpr (LIN) {
      for (int w = 0; w < 2 * epi_warps(FORM, LIN); ++w) mbar_init(&res_bar[w], 1);
    }
    *abort_flag = 0;
    *never_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA0);
    tma_prefetch_desc(&tmB0);
  }
  // The first weights of a lone CTA set out for L2 while earlier kernels still run (a prefetch returns
  // nothing that a later write could make stale): behind a norm, 128 tokens x 4096 x 10240 bf16 take
  // 38.9 instead of 39.9 us, 17 x 8192 x 4096 alone 24.8 instead of 25.8.  In the backward and the pairs'
  // forms, which are not bound by memory, it cost 1 to 4 %.
  if constexpr ((MODE == GLU_FORWARD || LIN) && CG == 1) {
    if (threadIdx.x == 64) {
      const int n = SPLIT ? args.split : 1, part = SPLIT ? (int)cluster_rank() : 0;
      const Tile tl = tile_at(blockIdx.x / n, args.order);
      const int kb = args.num_k * part / n, end = min(kb + stages, args.num_k * (part + 1) / n);
      for (int k = kb; k < end; ++k) {
        tma_prefetch_2d(&tmB0, k * KE, tl.n * bno);
        if constexpr (TWO) tma_prefetch_2d(&tmB1, k * KE, tl.n * bno);
      }
    }
  }
  if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, 2 * kMaxBN);
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the peer's barriers exist before anything reaches them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl wc{args.status, abort_flag, args.timeout_ns};
  grid_wait_prior();  // everything below reads or writes what earlier kernels use

  const int total = args.order.plane.d * (MODE == GRAD_DW ? args.planes : 1);
  const int split = SPLIT ? args.split : 1, part = SPLIT ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / (CG * split), units = gridDim.x / (CG * split);
  // This CTA's k-blocks of a tile: all, its share of a shared tile, or a plane's share of the tokens.
  constexpr bool CHUNKS = MODE == GRAD_DW && (EPI & kEpiF32);
  auto k_begin = [&](const Tile& tl) {
    return CHUNKS ? (int)((int64_t)args.num_k * tl.z / args.planes) : args.num_k * part / split;
  };
  auto k_end = [&](const Tile& tl) {
    return CHUNKS ? (int)((int64_t)args.num_k * (tl.z + 1) / args.planes) : args.num_k * (part + 1) / split;
  };

  uint32_t issued_mask = 0, issued_par = 0;  // stages with loads in flight (abort path)
  bool mma_issued = false;

  if (warp == 0) {
    if (elect_one()) {
      const int mn_chunks = (bn / CG + 63) / 64;  // MN-major B: 64-column boxes of this CTA
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        const Tile tl = tile_at(t, args.order);
        const int m0 = (tl.m * CG + rank) * kTileRows, kb1 = k_end(tl);
        for (int kb = k_begin(tl); kb < kb1; ++kb) {
          if (!wait_bounded(&empty[stage], phase ^ 1u, wc)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + (size_t)stage * stage_bytes;
          uint8_t* sb = sa + a_bytes;
          uint64_t* bar = &full[stage];
          // both CTAs' loads complete on the leader's barrier, which expects the pair's bytes
          if (rank == 0) mbar_arrive_expect_tx(bar, CG * stage_bytes);
          const uint32_t pair_bar = CG == 2 ? map_rank(bar, 0) : 0;
          auto load = [&](uint8_t* dst, const CUtensorMap* m, int c0, int c1) {
            if constexpr (CG == 2)
              tma_load_2d_pair(dst, m, pair_bar, c0, c1);
            else
              tma_load_2d(dst, m, bar, c0, c1);
          };
          if constexpr (TWO) {
            const int k = kb * KE, n0 = tl.n * bno;
            load(sa, &tmA0, k, m0);
            if constexpr (CG == 2) {  // CTA 0 brings the gate's rows, CTA 1 the other projection's
              load(sb, rank == 0 ? &tmB0 : &tmB1, k, n0);
            } else {
              load(sb, &tmB0, k, n0);
              load(sb + bno * kKBytes, &tmB1, k, n0);
            }
          } else if constexpr (LIN) {
            load(sa, &tmA0, kb * KE, m0);
            load(sb, &tmB0, kb * KE, tl.n * bno + rank * (bn / CG));
          } else if constexpr (MODE == GRAD_DX) {
            const bool second = kb >= args.k_half;
            const int k = (second ? kb - args.k_half : kb) * KE, n0 = tl.n * bno + rank * (bn / CG);
            load(sa, second ? &tmA1 : &tmA0, k, m0);
            for (int c = 0; c < mn_chunks; ++c) load(sb + c * kMnChunk, second ? &tmB1 : &tmB0, n0 + c * 64, k);
          } else {
            const int k = kb * KE, n0 = tl.n * bno + rank * (bn / CG);
#pragma unroll
            for (int c = 0; c < kTileRows / 64; ++c) load(sa + c * kMnChunk, tl.z && !CHUNKS ? &tmA1 : &tmA0, m0 + c * 64, k);
            for (int c = 0; c < mn_chunks; ++c) load(sb + c * kMnChunk, &tmB0, n0 + c * 64, k);
          }
          issued_mask |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    if constexpr (SPLIT) {  // the two meetings of the epilogue below
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = (1u << 4) | (args.bf16_operands ? (1u << 7) | (1u << 10) : 0u) |
                             ((uint32_t)A_MN << 15) | ((uint32_t)B_MN << 16) | ((uint32_t)(bn >> 3) << 17) |
                             ((uint32_t)((kTileRows * CG) >> 4) << 24);
      // K-major: 8-row groups 1024 bytes apart, a k-step 32 bytes on; MN-major: chunks of 64
      // values kMnChunk apart, 8-k groups 1024 bytes apart, a k-step 16 rows of 128 bytes on
      const uint32_t s0 = smem_u32(smem);
      const uint64_t ad0 = sdesc(s0, A_MN ? kMnChunk : 16, 1024, kSw128);
      const uint64_t bd0 = sdesc(s0 + a_bytes, B_MN ? kMnChunk : 16, 1024, kSw128);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        if (!wait_bounded(&acce[acc], acc_phase ^ 1u, wc)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(acc * kMaxBN);
        const Tile tl = CHUNKS ? tile_at(t, args.order) : Tile{0, 0, 0};
        const int kb0 = k_begin(tl), kb1 = k_end(tl);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_bounded(&full[stage], phase, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = (uint32_t)(stage * (stage_bytes >> 4));
          const uint64_t ad = ad0 + at, bd = bd0 + at;
          umma_cg<CG, F8>(d, ad, bd, idesc, kb != kb0);
#pragma unroll
          for (int k = 1; k < 4; ++k)
            umma_cg<CG, F8>(d, ad + (uint32_t)(k * (A_MN ? 2048 : 32) >> 4), bd + (uint32_t)(k * (B_MN ? 2048 : 32) >> 4),
                            idesc, 1u);
          mma_issued = true;
          umma_commit_cg<CG>(&empty[stage]);
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_cg<CG>(&accf[acc]);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
    }
    if constexpr (SPLIT) {
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    constexpr int H = epi_warps(FORM, LIN) / 4;  // warps of a lane quarter, which take the chunks in turn
    constexpr int W = 32;                   // columns stored at a time
    constexpr int LD = H == 4 ? 16 : 32;    // columns computed at a time
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* st = xpose + (warp - 2) * (LIN ? 2 * kLinStage : 32 * 2 * W);
    int acc = 0;
    uint32_t acc_phase = 0;
    // The linear layer's two stages a warp.  Pieces go out in turn, so that with one store still reading its
    // stage the other stage is free.  A residual's piece that does not exist (no row or column of it) takes no
    // copy: what is added there is not stored.
    uint64_t* res_in = res_bar + (warp - 2) * 2;
    const int swizzle = ((lane >> 1) & 3) << 4;  // TMA's 64-byte swizzle: the piece of 16 bytes by bits of the row
    uint32_t res_phase = 0, res_flying = 0;      // a bit a stage
    int turn = 0;
    bool dead = false;
    float warm[F8 ? 4 : 2] = {};
    auto load_res = [&](int stage, int n, int m0) {
      res_flying |= 1u << stage;
      if (lane == 0) {
        const bool exists = n < args.N && m0 < args.M;
        mbar_arrive_expect_tx(&res_in[stage], exists ? kLinStage : 0);
        if (exists) tma_load_2d(st + stage * kLinStage, &tmR, &res_in[stage], n, m0);
      }
    };
    auto store_stage = [&](const CUtensorMap* map, int stage, int n, int m0, bool exists) {
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (exists) tma_store_2d(map, st + stage * kLinStage, n, m0);
        bulk_commit();  // (an empty group where nothing is stored: the waits count groups)
      }
    };
    const uint32_t acce_addr[2] = {CG == 2 ? map_rank(&acce[0], 0) : 0, CG == 2 ? map_rank(&acce[1], 0) : 0};
    for (int t = unit; t < total; t += units) {
      const Tile tl = tile_at(t, args.order);
      const int m0 = (tl.m * CG + rank) * kTileRows + q * 32, m = m0 + lane;
      const uint32_t rows = __ballot_sync(0xffffffffu, m < args.M);
      const int n_tile = tl.n * bno;  // first output column of the tile
      // e4m3: the row's scale and this lane's share of the first chunk's column scales, on their
      // way while the products finish; columns past the last read the last one's (not stored)
      float sx = 1.0f, sg = 0.f, su = 0.f;
      auto fetch_scales = [&](int c) {
        if constexpr (F8 && !LIN) {
          const float2 s = column_scales<MODE>(args, min(n_tile + c * W + lane, args.N - 1));
          sg = s.x;
          su = s.y;
        }
      };
      if constexpr (F8) {
        sx = m < args.M ? args.x_scale[m] : 0.f;  // written by the kernel before this one: a plain load
        fetch_scales(part + split * half);
      }
      // The lines of the next tile's bias and scales into L1 (from L2 they came some 700 cycles late, twice a
      // tile); the loads' results are taken, for nothing, a tile later, when they have long arrived.
      if constexpr (LIN) {
#pragma unroll
        for (float& v : warm) asm volatile("" ::"f"(v));
        const int n = t + units < total ? tile_at(t + units, args.order).n * bno + lane : args.N;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = n + (part + split * (half + i * H)) * W;
          if (col < args.N) {
            if (args.bias) warm[i] = args.bias[col];
            if constexpr (F8) warm[2 + i] = args.g_scale[col];
          }
        }
      }
      // the first piece's residual sets out while the products finish, and the other chunks' for L2
      if constexpr (LIN) {
        int c = part + split * half;
        if ((EPI & kEpiRes) && c * W < bno) {
          if (EPI & kEpiZ) turn = 0;
          stores_read<1>();
          load_res(turn, n_tile + c * W, m0);
          const int size = EPI & kEpiF32 ? 4 : 2;
          const uint8_t* r = static_cast<const uint8_t*>(args.res) + (size_t)min(m, args.M - 1) * args.ldo * size;
          while ((c += H * split) * W < bno)
            if (n_tile + c * W < args.N) prefetch_l2(r + (n_tile + c * W) * size);
        }
      }
      const bool ok = wait_bounded(&accf[acc], acc_phase, wc);
      // (a split tile's CTAs meet all the same: its outputs are invalid then, as the status says)
      if (!__all_sync(0xffffffffu, ok) && !SPLIT) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kMaxBN);
      const int chunks = (bno + W - 1) / W;
      const int last = chunks - 1 - ((chunks - 1 - half) & (H - 1));  // this warp's last chunk (< half: it has none)
      auto hand_back = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2)
            mbar_arrive_cluster_relaxed(acce_addr[acc]);
          else
            mbar_arrive(&acce[acc]);
        }
      };
      if (!SPLIT && half > last) hand_back();
      // kSplit: piece c is finished by CTA c % split.  Its sums from another CTA lie in the ring of
      // that CTA, idle by now: [other CTAs][pieces][8, or 2 x 8, parts of a row][128 rows][4 floats], so
      // that a warp's stores and loads are of whole lines.
      constexpr int kPart = kTileRows * 16, kPiece = (TWO ? 16 : 8) * kPart;
      const int pieces = SPLIT ? (chunks + split - 1) / split : 0;
      if constexpr (SPLIT) {
        cluster_sync();  // every CTA of the tile has its sums, and an idle ring
        tc_fence_after();
        for (int c = 0, i = 0; c < chunks; ++c) {
          const int owner = c % split;
          if (owner == part || (i++ & (H - 1)) != half) continue;
          float g[W], u[W];
          tmem_ld32(tb + c * W, g);
          if constexpr (TWO) tmem_ld32(tb + bno + c * W, u);
          tmem_wait_ld();
          const int slot = part < owner ? part : part - 1;
          const uint32_t to =
              map_rank(smem, owner) + (uint32_t)((slot * pieces + c / split) * kPiece + (q * 32 + lane) * 16);
          if (m < args.M) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              store_cluster(to + k * kPart, g[4 * k], g[4 * k + 1], g[4 * k + 2], g[4 * k + 3]);
              if constexpr (TWO)
                store_cluster(to + (8 + k) * kPart, u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
            }
          }
        }
        __syncwarp();
        cluster_sync();  // the sums have arrived
      }
      // The linear layer's 32 columns from c on, in halves of 16 (there are 96 registers): y's piece (32 columns
      // of 16 bits or 16 of fp32) is put into a stage and stored by TMA; the residual's piece comes into that
      // stage by TMA before, and each lane adds it to its row in place.  Without z the two stages take turns, and
      // the next piece's residual sets out before this one is worked on; with z, held packed, y has the first
      // stage and z the second.  False: a wait ran out.
      [[maybe_unused]] auto lin_chunk = [&](int c) -> bool {
        constexpr bool RES = EPI & kEpiRes, Z = EPI & kEpiZ, OUT32 = EPI & kEpiF32;
        const int n0 = n_tile + c * W;
        const bool exists = n0 < args.N && m0 < args.M;
        uint4 z[Z ? 4 : 1];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int n = n0 + b * 16;
          float g[16];
          tmem_ld16(tb + c * W + b * 16, g);
          float4 bias[4];
          [[maybe_unused]] float4 ws[4];  // the same for all lanes, from L1
          auto fetch = [&](const float* p, float4* v) {
            if (n + 16 <= args.N) {
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float4*>(p + n + i * 4);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                v[i] = n + i * 4 < args.N ? *reinterpret_cast<const float4*>(p + n + i * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
          };
          if (args.bias) fetch(args.bias, bias);
          if constexpr (F8) fetch(args.g_scale, ws);
          tmem_wait_ld();
          if (!SPLIT && b == 1 && c == last) hand_back();
          if constexpr (SPLIT) {
            for (int k = 0; k < split - 1; ++k) {
              const uint8_t* from = smem + (k * pieces + c / split) * kPiece + (q * 32 + lane) * 16 + b * 4 * kPart;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 a = *reinterpret_cast<const float4*>(from + i * kPart);
                g[4 * i] += a.x, g[4 * i + 1] += a.y, g[4 * i + 2] += a.z, g[4 * i + 3] += a.w;
              }
            }
          }
          auto each2 = [&](const float4* v, auto f) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              f2_unpack(f(f2_pack(g[4 * i], g[4 * i + 1]), f2_pack(v[i].x, v[i].y)), g[4 * i], g[4 * i + 1]);
              f2_unpack(f(f2_pack(g[4 * i + 2], g[4 * i + 3]), f2_pack(v[i].z, v[i].w)), g[4 * i + 2], g[4 * i + 3]);
            }
          };
          if constexpr (F8) {
            const uint64_t sx2 = f2_splat(sx);
            each2(ws, [&](uint64_t v, uint64_t s) { return f2_mul(v, f2_mul(sx2, s)); });
          }
          if (args.bias) each2(bias, [](uint64_t v, uint64_t s) { return f2_add(v, s); });
          if constexpr (Z) pack16<16>(g, z + b * 2, args.bf16_operands);
          if (args.act == TFL_ACT_SILU)
            activate<TFL_ACT_SILU, 16>(g);
          else if (args.act == TFL_ACT_GELU)
            activate<TFL_ACT_GELU, 16>(g);
          const int stage = Z ? 0 : turn;
          const int next = OUT32 && b == 0 ? n + 16 : c + H * split < chunks ? n0 + H * split * W : -1;
          if (b == 0 || OUT32) {  // a piece begins: its stage
            if constexpr (RES) {
              if (!Z && next >= 0) {  // the other stage's store was the last
                stores_read<0>();
                load_res(stage ^ 1, next, m0);
              }
              if (!__all_sync(0xffffffffu, wait_bounded(&res_in[stage], (res_phase >> stage) & 1u, wc))) return false;
              res_flying &= ~(1u << stage);
              res_phase ^= 1u << stage;
            } else if (Z && b == 1) {  // the last store was from this stage, in any other case from the other one
              stores_read<0>();
            } else {
              stores_read<1>();
            }
          }
          uint8_t* own = st + stage * kLinStage + lane * 64;
          auto at = [&](int i) { return reinterpret_cast<uint4*>(own + ((i << 4) ^ swizzle)); };
          if constexpr (OUT32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4* s = at(i);
              if constexpr (RES) {
                const uint4 r = *s;
                g[4 * i] += __uint_as_float(r.x), g[4 * i + 1] += __uint_as_float(r.y);
                g[4 * i + 2] += __uint_as_float(r.z), g[4 * i + 3] += __uint_as_float(r.w);
              }
              *s = make_uint4(__float_as_uint(g[4 * i]), __float_as_uint(g[4 * i + 1]), __float_as_uint(g[4 * i + 2]),
                              __float_as_uint(g[4 * i + 3]));
            }
          } else {
            if constexpr (RES) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float r[8];
                unpack16(*at(b * 2 + i), r, args.bf16_out);
#pragma unroll
                for (int k = 0; k < 8; ++k) g[8 * i + k] += r[k];
              }
            }
            uint4 w[2];
            pack16<16>(g, w, args.bf16_out);
#pragma unroll
            for (int i = 0; i < 2; ++i) *at(b * 2 + i) = w[i];
            if (b == 0) continue;
          }
          store_stage(&tmA1, stage, OUT32 ? n : n0, m0, exists && (!OUT32 || n < args.N));
          turn ^= 1;
          if constexpr (Z) {
            if (b == 1) {
              stores_read<1>();
              own = st + kLinStage + lane * 64;
#pragma unroll
              for (int i = 0; i < 4; ++i) *at(i) = z[i];
              store_stage(&tmB1, 1, n0, m0, exists);
            }
            if (RES && next >= 0) {
              stores_read<0>();
              load_res(0, next, m0);
            }
          }
        }
        return true;
      };
#pragma unroll 1
      for (int c = part + split * half; c < chunks; c += H * split) {
        const int n0 = n_tile + c * W;                       // first output column
        const int cols = min(args.N - n0, bno - c * W);      // columns of this chunk that exist
        if constexpr (LIN) {
          if (!lin_chunk(c)) {
            dead = true;
            break;
          }
        } else {
          uint4 o[W / 8], o2[W / 8];
          if constexpr (MODE == GLU_SLOPES)
            load_cols<W>(st, lane, o2, args.dh + (size_t)m0 * args.N + n0, args.N, rows, cols);
          if constexpr (F8) {  // the chunk's scales to every lane, through the stage
            float* sc = reinterpret_cast<float*>(st);
            sc[lane] = sg;
            sc[W + lane] = su;
            __syncwarp();
            if (c + H * split < chunks) fetch_scales(c + H * split);
          }
#pragma unroll
          for (int b = 0; b < W / LD; ++b) {
            const int col = c * W + b * LD;
            float g[LD], u[LD];
            if constexpr (LD == 16) {
              tmem_ld16(tb + col, g);
              if constexpr (TWO) tmem_ld16(tb + bno + col, u);
            } else {
              tmem_ld32(tb + col, g);
              if constexpr (TWO) tmem_ld32(tb + bno + col, u);
            }
            tmem_wait_ld();
            // once the accumulator is in registers it is handed back, before arithmetic and stores
            if (!SPLIT && b == W / LD - 1 && c == last) hand_back();
            if constexpr (SPLIT) {
              for (int k = 0; k < split - 1; ++k) {
                const uint8_t* from = smem + (k * pieces + c / split) * kPiece + (q * 32 + lane) * 16;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float4 a = *reinterpret_cast<const float4*>(from + i * kPart);
                  g[4 * i] += a.x, g[4 * i + 1] += a.y, g[4 * i + 2] += a.z, g[4 * i + 3] += a.w;
                  if constexpr (TWO) {
                    const float4 e = *reinterpret_cast<const float4*>(from + (8 + i) * kPart);
                    u[4 * i] += e.x, u[4 * i + 1] += e.y, u[4 * i + 2] += e.z, u[4 * i + 3] += e.w;
                  }
                }
              }
            }
            if constexpr (F8) {
              const float* sc = reinterpret_cast<const float*>(st) + b * LD;
#pragma unroll
              for (int i = 0; i < LD; i += 4) {
                const float4 a = *reinterpret_cast<const float4*>(sc + i);
                const float4 e = *reinterpret_cast<const float4*>(sc + W + i);
                auto scale2 = [&](float* v, float s0, float s1) {
                  f2_unpack(f2_mul(f2_pack(v[0], v[1]), f2_mul(f2_splat(sx), f2_pack(s0, s1))), v[0], v[1]);
                };
                scale2(g + i, a.x, a.y), scale2(g + i + 2, a.z, a.w);
                scale2(u + i, e.x, e.y), scale2(u + i + 2, e.z, e.w);
              }
              if (b == W / LD - 1) __syncwarp();  // the stage is free for the rows
            }
            if constexpr (MODE == GLU_FORWARD) {
              // the activation is chosen once for all values: a branch at each would keep the
              // compiler from interleaving their chains
              if (args.act == TFL_ACT_SILU)
                forward_values<TFL_ACT_SILU, LD>(g, u);
              else
                forward_values<TFL_ACT_GELU, LD>(g, u);
            } else if constexpr (MODE == GLU_SLOPES) {
              float dh[LD];
#pragma unroll
              for (int i = 0; i < LD / 8; ++i) unpack16(o2[b * (LD / 8) + i], dh + 8 * i, args.bf16_out);
              if (args.act == TFL_ACT_SILU)
                slope_values<TFL_ACT_SILU, LD>(g, u, dh);
              else
                slope_values<TFL_ACT_GELU, LD>(g, u, dh);
              pack16<LD>(u, o2 + b * (LD / 8), args.bf16_out);
            }
            if constexpr (CHUNKS) {
#pragma unroll
              for (int k = 0; k < LD; k += 16)
                store_cols_f32(st, lane, g + k,
                               reinterpret_cast<float*>(args.out) + ((size_t)tl.z * args.M + m0) * args.ldo + n0 + b * LD + k,
                               args.ldo, rows, cols - b * LD - k);
            } else {
              pack16<LD>(g, o + b * (LD / 8), args.bf16_out);
            }
          }
          const size_t to = (size_t)m0 * args.ldo + n0;
          if constexpr (!CHUNKS)
            store_cols<W>(st, lane, o, (MODE == GRAD_DW && tl.z ? args.out2 : args.out) + to, args.ldo, rows, cols);
          if constexpr (MODE == GLU_SLOPES) store_cols<W>(st, lane, o2, args.out2 + to, args.ldo, rows, cols);
        }
      }
      if (dead) break;
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if constexpr (LIN) {
      // nothing may land in or be read from this CTA's shared memory once it is gone
      const WaitCtl dc{args.status, never_flag, 100000000LL};
      for (int s = 0; s < 2; ++s)
        if (res_flying & (1u << s)) wait_bounded(&res_in[s], (res_phase >> s) & 1u, dc);
      stores_read<0>();
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // Abort path: let the copies and MMAs in flight land before the shared and tensor memory
    // are released (bounded as well).  A pair's copies complete on the leader's barriers.
    const WaitCtl dc{args.status, never_flag, 100000000LL};
    if (warp == 0 && rank == 0 && elect_one()) {
      for (int s = 0; s < stages; ++s)
        if (issued_mask & (1u << s)) wait_bounded(&full[s], (issued_par >> s) & 1u, dc);
    }
    if (warp == 1 && elect_one() && mma_issued) {
      umma_commit_cg<CG>(drain);
      wait_bounded(drain, 0, dc);
    }
    __syncthreads();
  }
  if constexpr (CG == 2) cluster_sync();  // nothing of the peer reaches this CTA any more (a split tile's CTAs met after the last)
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<CG>(tmem_base, 2 * kMaxBN);
  }
}

Divisor divisor(int d) {
  Divisor r;
  r.d = d;
  if (d == 1) return r;  // shift -1
  int s = 0;
  while ((1ll << s) < d) ++s;
  r.factor = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
  r.shift = s - 1;
  return r;
}

template <int CG, int MODE, bool F8, int FORM, int EPI = 0>
cudaError_t launch_one(const TileMaps& mp, TileArgs a, const TilePlan& p, cudaStream_t s) {
  a.bno = p.bno;
  a.split = p.split;
  const int num_m = (a.M + kTileRows * CG - 1) / (kTileRows * CG), num_n = (a.N + p.bno - 1) / p.bno;
  const int group = a.group_m < num_m ? a.group_m : num_m;
  a.order.num_m = num_m;
  a.order.plane = divisor(num_m * num_n);
  a.order.group = divisor(group * num_n);
  a.order.rows = divisor(group);
  a.order.last_rows = divisor(num_m % group ? num_m % group : group);
  const int bn = (MODE == GLU_FORWARD || MODE == GLU_SLOPES) ? 2 * p.bno : p.bno;
  const bool b_mn = MODE == GRAD_DX || MODE == GRAD_DW;
  a.a_bytes = p.a_rows * kKBytes;
  a.stage_bytes = a.a_bytes + (b_mn ? (bn / CG + 63) / 64 * kMnChunk : bn / CG * kKBytes);
  a.stages = ring_bytes(FORM == kWide, MODE == LIN_FORWARD) / a.stage_bytes;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  const int cluster = CG * p.split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.tiles < p.units ? p.tiles : p.units) * cluster);
  cfg.blockDim = dim3(tile_threads(FORM, MODE));
  cfg.dynamicSmemBytes = kTileSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, tile_kernel<CG, MODE, F8, FORM, EPI>, mp.a0, mp.a1, mp.b0, mp.b1, mp.r, a);
}

template <int CG, int MODE, bool F8, int FORM, int EPI = 0>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(tile_kernel<CG, MODE, F8, FORM, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem);
}

// Clusters of `size` CTAs that the GPU holds at once, one CTA an SM (a cluster stays within a GPU
// processing cluster, so fewer than SMs / size may fit).
template <int CG, int FORM>
cudaError_t clusters_at_once(int size, int* n) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(tile_threads(FORM, GLU_FORWARD));
  cfg.dynamicSmemBytes = kTileSmem;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = size;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(n, tile_kernel<CG, GLU_FORWARD, false, FORM, 0>, &cfg);
}

}  // namespace

}  // namespace tfl
