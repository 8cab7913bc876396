// glu.cu -- the gated feed-forward block h = act(x Wg^T) * (x Wu^T), forward and backward.
//
// One persistent tcgen05 GEMM kernel in four modes, fp32 accumulation in tensor memory:
//   GLU_FORWARD   both projections of a tile at once: the accumulator's first half of columns
//                 is x Wg^T, its second half x Wu^T of the same output columns, so the
//                 activation and the product run in the epilogue and only h is written.
//                 16-bit operands, or e4m3 with one scale a row of x, Wg and Wu (the scales
//                 factor out of the sums, so the epilogue applies them).
//   GLU_SLOPES    the same two products; with dh the epilogue forms dg = dh u act'(g) and
//                 du = dh act(g) from the fp32 accumulators.  Nothing of the forward is kept:
//                 reading back 16-bit g and u would cost 4 bytes a value of memory and round
//                 them once more, where recomputing rounds only dg and du (once, to the
//                 operand type the tensor cores take).
//   GLU_DX        dx = dg Wg + du Wu: one sum over 2 d_ff, W read as [k, n] (MN-major).
//   GLU_DW        dWg = dg^T x and dWu = du^T x: sums over the tokens, both operands MN-major.
//
// Structure: warp 0 feeds a ring of k-blocks (128 bytes of k a row, 128-byte swizzle) by TMA,
// warp 1 issues the MMAs, the others are the epilogue (two or four per tensor-memory lane quarter), two
// accumulators so that a tile's epilogue runs under the next tile's MMAs.
//
// What bounds it: with many tokens the tensor cores, and in long runs the power cap (8192 x 1024 x 4096
// fp16 forward 78 us in a burst, 1.76 PFLOP/s, 0.94 of the measured burst rate, 92 us in a long run;
// 16384 x 2048 x 8192 bf16 backward 1.71 ms and 2.01 ms; 74 us and 1.76 ms on another GPU); with few
// tokens the weights' bytes (40 x 4096 x 10240 e4m3: 16.4 us for 85 MB, 5.2 TB/s).  A pair's 256 x 256
// tile took the first two from 107 to 101 us and from 2.26 to 2.06 ms against a lone CTA's 128 x 256, a
// thread that the compiler knows to be alone for the issue of MMAs from 82 to 74 us and from 1.95 to
// 1.76 ms (bursts, one GPU).  The epilogue's arithmetic is not free even where it hides under the MMAs:
// its warps take issue slots from that thread, hence packed pairs and the short issue loop.
//
// Ragged sizes: TMA fills what lies outside a matrix with zeros (zero rows and zero k add
// nothing), and the epilogue stores only rows and columns that exist.
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
__host__ __device__ constexpr int xpose_bytes(bool wide) { return wide ? 32768 : 16384; }
constexpr int kGluSmem = 232448;
__host__ __device__ constexpr int ring_bytes(bool wide) { return kGluSmem - 1024 - xpose_bytes(wide) - kBarrierBytes; }

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
// The same way back: this thread's row of W 16-bit columns (zeros outside).
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

struct Tile {
  int m, n, z;
};

// Tiles in groups of kGroupM row blocks, column by column inside a group, so that the tiles in
// flight share operands through L2.  DW: first all of dWg, then all of dWu.
constexpr int kGroupM = 8;
__device__ __forceinline__ Tile tile_at(int t, int num_m, int num_n, int group_m) {
  Tile r;
  const int per = num_m * num_n;
  r.z = t / per;
  t -= r.z * per;
  const int g = t / (group_m * num_n), first = g * group_m;
  const int gm = min(num_m - first, group_m);
  t -= g * group_m * num_n;
  r.n = t / gm;
  r.m = first + t - r.n * gm;
  return r;
}

// kWide: tiles of kMaxBN accumulator columns and 128 loaded rows of A, all sizes constants.
// kNarrow: the plan's widths.
// kSplit: the same, with the k-blocks of a tile shared out to a cluster of lone CTAs (few tiles:
// the whole GPU works on them); each CTA finishes some of the tile's 32-column pieces, and the
// others send it their sums through its shared memory, added in CTA order.  One tile a CTA.
enum GluForm : int { kWide = 0, kNarrow = 1, kSplit = 2 };
// Epilogue warps: sixteen for the wide tiles, 32 columns each, which a short k needs (8192 x 1024 x 4096
// e4m3 47.5 -> 45.4 us; the eight before computed 32 columns at a time and stored 64, these 16 and 32,
// and have the registers for it).  Eight for the narrow tiles, most of which have one or two chunks.
__host__ __device__ constexpr int epi_warps(int form) { return form == kWide ? 16 : 8; }
__host__ __device__ constexpr int glu_threads(int form) { return 64 + 32 * epi_warps(form); }
template <int CG, int MODE, bool F8, int FORM>
__global__ void __launch_bounds__(glu_threads(FORM), 1)
    glu_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
               const __grid_constant__ CUtensorMap tmB0, const __grid_constant__ CUtensorMap tmB1, const GluArgs args) {
  constexpr bool WIDE = FORM == kWide, SPLIT = FORM == kSplit;
  static_assert(!SPLIT || CG == 1, "lone CTAs share a tile's k-blocks");
  constexpr bool TWO = MODE == GLU_FORWARD || MODE == GLU_SLOPES;  // two products side by side
  constexpr bool A_MN = MODE == GLU_DW, B_MN = MODE == GLU_DX || MODE == GLU_DW;
  constexpr int KE = F8 ? 128 : 64;                                // k elements a stage
  extern __shared__ uint8_t smem_raw[];
  grid_launch_dependents();
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* xpose = smem + ring_bytes(WIDE);
  uint64_t* full = reinterpret_cast<uint64_t*>(xpose + xpose_bytes(WIDE));
  uint64_t* empty = full + kMaxStages;
  uint64_t* accf = empty + kMaxStages;
  uint64_t* acce = accf + 2;
  uint64_t* drain = acce + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* never_flag = abort_flag + 1;  // stays 0: lets the drain waits ignore abort_flag

  constexpr int kWideStage = (kGluRows + kMaxBN / CG) * kKBytes;
  const int bno = WIDE ? (TWO ? kMaxBN / 2 : kMaxBN) : args.bno;  // output columns of a tile
  const int bn = TWO ? 2 * bno : bno;                             // accumulator columns
  const int stages = WIDE ? ring_bytes(true) / kWideStage : args.stages;
  const int stage_bytes = WIDE ? kWideStage : args.stage_bytes;
  const int a_bytes = WIDE ? kGluRows * kKBytes : args.a_bytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)cluster_rank() : 0;             // of the pair
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&accf[a], 1);
      mbar_init(&acce[a], CG * epi_warps(FORM));
    }
    mbar_init(drain, 1);
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
  if constexpr (MODE == GLU_FORWARD && CG == 1) {
    if (threadIdx.x == 64) {
      const int n = SPLIT ? args.split : 1, part = SPLIT ? (int)cluster_rank() : 0;
      const Tile tl = tile_at(blockIdx.x / n, (args.M + kGluRows - 1) / kGluRows, (args.N + bno - 1) / bno, kGroupM);
      const int kb = args.num_k * part / n, end = min(kb + stages, args.num_k * (part + 1) / n);
      for (int k = kb; k < end; ++k) {
        tma_prefetch_2d(&tmB0, k * KE, tl.n * bno);
        tma_prefetch_2d(&tmB1, k * KE, tl.n * bno);
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

  const int num_m = (args.M + kGluRows * CG - 1) / (kGluRows * CG), num_n = (args.N + bno - 1) / bno;
  const int total = num_m * num_n * (MODE == GLU_DW ? 2 : 1);
  const int split = SPLIT ? args.split : 1, part = SPLIT ? (int)cluster_rank() : 0;
  const int unit = blockIdx.x / (CG * split), units = gridDim.x / (CG * split);
  const int kb0 = args.num_k * part / split, kb1 = args.num_k * (part + 1) / split;  // this CTA's k-blocks

  uint32_t issued_mask = 0, issued_par = 0;  // stages with loads in flight (abort path)
  bool mma_issued = false;

  if (warp == 0) {
    if (elect_one()) {
      const int mn_chunks = (bn / CG + 63) / 64;  // MN-major B: 64-column boxes of this CTA
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        const Tile tl = tile_at(t, num_m, num_n, kGroupM);
        const int m0 = (tl.m * CG + rank) * kGluRows;
        for (int kb = kb0; kb < kb1; ++kb) {
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
          } else if constexpr (MODE == GLU_DX) {
            const bool second = kb >= args.k_half;
            const int k = (second ? kb - args.k_half : kb) * KE, n0 = tl.n * bno + rank * (bn / CG);
            load(sa, second ? &tmA1 : &tmA0, k, m0);
            for (int c = 0; c < mn_chunks; ++c) load(sb + c * kMnChunk, second ? &tmB1 : &tmB0, n0 + c * 64, k);
          } else {
            const int k = kb * KE, n0 = tl.n * bno + rank * (bn / CG);
#pragma unroll
            for (int c = 0; c < kGluRows / 64; ++c) load(sa + c * kMnChunk, tl.z ? &tmA1 : &tmA0, m0 + c * 64, k);
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
                             ((uint32_t)((kGluRows * CG) >> 4) << 24);
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
    constexpr int H = epi_warps(FORM) / 4;  // warps of a lane quarter, which take the chunks in turn
    constexpr int W = 32;                   // columns stored at a time
    constexpr int LD = H == 4 ? 16 : 32;    // columns computed at a time
    const int q = warp & 3, half = (warp - 2) >> 2;
    uint8_t* st = xpose + (warp - 2) * (32 * 2 * W);
    int acc = 0;
    uint32_t acc_phase = 0;
    const uint32_t acce_addr[2] = {CG == 2 ? map_rank(&acce[0], 0) : 0, CG == 2 ? map_rank(&acce[1], 0) : 0};
    for (int t = unit; t < total; t += units) {
      const Tile tl = tile_at(t, num_m, num_n, kGroupM);
      const int m0 = (tl.m * CG + rank) * kGluRows + q * 32, m = m0 + lane;
      const uint32_t rows = __ballot_sync(0xffffffffu, m < args.M);
      const int n_tile = tl.n * bno;  // first output column of the tile
      // e4m3: the row's scale and this lane's share of the first chunk's column scales, on their
      // way while the products finish; columns past the last read the last one's (not stored)
      float sx = 1.0f, sg = 0.f, su = 0.f;
      auto fetch_scales = [&](int c) {
        const int n = min(n_tile + c * W + lane, args.N - 1);
        sg = __ldg(args.g_scale + n);
        su = __ldg(args.u_scale + n);
      };
      if constexpr (F8) {
        sx = m < args.M ? args.x_scale[m] : 0.f;  // written by the kernel before this one: a plain load
        fetch_scales(part + split * half);
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
      constexpr int kPart = kGluRows * 16, kPiece = (TWO ? 16 : 8) * kPart;
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
#pragma unroll 1
      for (int c = part + split * half; c < chunks; c += H * split) {
        const int n0 = n_tile + c * W;                       // first output column
        const int cols = min(args.N - n0, bno - c * W);      // columns of this chunk that exist
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
          pack16<LD>(g, o + b * (LD / 8), args.bf16_out);
        }
        const size_t to = (size_t)m0 * args.ldo + n0;
        store_cols<W>(st, lane, o, (MODE == GLU_DW && tl.z ? args.out2 : args.out) + to, args.ldo, rows, cols);
        if constexpr (MODE == GLU_SLOPES) store_cols<W>(st, lane, o2, args.out2 + to, args.ldo, rows, cols);
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
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

template <int CG, int MODE, bool F8, int FORM>
cudaError_t launch_one(const GluMaps& mp, GluArgs a, const GluPlan& p, cudaStream_t s) {
  a.bno = p.bno;
  a.split = p.split;
  const int bn = (MODE == GLU_FORWARD || MODE == GLU_SLOPES) ? 2 * p.bno : p.bno;
  const bool b_mn = MODE == GLU_DX || MODE == GLU_DW;
  a.a_bytes = p.a_rows * kKBytes;
  a.stage_bytes = a.a_bytes + (b_mn ? (bn / CG + 63) / 64 * kMnChunk : bn / CG * kKBytes);
  a.stages = ring_bytes(FORM == kWide) / a.stage_bytes;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  const int cluster = CG * p.split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.tiles < p.units ? p.tiles : p.units) * cluster);
  cfg.blockDim = dim3(glu_threads(FORM));
  cfg.dynamicSmemBytes = kGluSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, glu_kernel<CG, MODE, F8, FORM>, mp.a0, mp.a1, mp.b0, mp.b1, a);
}

template <int CG, int MODE, bool F8, int FORM>
cudaError_t prepare_one() {
  return cudaFuncSetAttribute(glu_kernel<CG, MODE, F8, FORM>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGluSmem);
}

// Clusters of `size` CTAs that the GPU holds at once, one CTA an SM (a cluster stays within a GPU
// processing cluster, so fewer than SMs / size may fit).
template <int CG, int FORM>
cudaError_t clusters_at_once(int size, int* n) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(glu_threads(FORM));
  cfg.dynamicSmemBytes = kGluSmem;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = size;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(n, glu_kernel<CG, GLU_FORWARD, false, FORM>, &cfg);
}

}  // namespace

// Every (mode, operand form) in every (CTAs of a tile, form).
#define TFL_GLU_MODES(X, CG, FORM)                                                                  \
  X(CG, GLU_FORWARD, false, FORM) X(CG, GLU_FORWARD, true, FORM) X(CG, GLU_SLOPES, false, FORM)     \
  X(CG, GLU_DX, false, FORM) X(CG, GLU_DW, false, FORM)
#define TFL_GLU_VARIANTS(X) \
  TFL_GLU_MODES(X, 2, kWide) TFL_GLU_MODES(X, 2, kNarrow) TFL_GLU_MODES(X, 1, kNarrow) TFL_GLU_MODES(X, 1, kSplit)

cudaError_t prepare_glu_kernels(GluUnits* u) {
  cudaError_t e = cudaSuccess;
#define TFL_PREP(CG, MODE, F8, FORM) \
  if (e == cudaSuccess) e = prepare_one<CG, MODE, F8, FORM>();
  TFL_GLU_VARIANTS(TFL_PREP)
#undef TFL_PREP
  if (e == cudaSuccess) e = clusters_at_once<2, kWide>(2, &u->pairs);
  for (int i = 0; i < 3 && e == cudaSuccess; ++i) e = clusters_at_once<1, kSplit>(2 << i, &u->splits[i]);
  return e;
}

// CTA pairs take tiles of 256 rows: each CTA stages half of B, so a k-block of a 256 x 256 tile
// costs 32 KB of shared-memory writes and L2 reads a CTA where a lone CTA's 128 x 256 tile costs
// 48 KB for the same products.
//
// Fewer than 128 rows of A: only those (to the next 8) are loaded and given room in the ring; the
// MMA still reads 128, the others being whatever lies behind, and their results are not stored.
//
// The cut goes by an estimate of the cycles a launch takes.  Its constants were fitted to the times of
// all cuts of 192 launches (12 to 3000 tokens, weights of 520 x 5696 to 4096 x 10240, all modes) before the
// wide tiles had sixteen epilogue warps; with them, the cut that it takes is still 1 % slower than the
// fastest on average, 19 % at worst (100 x 1024 x 4096 bf16, 7.0 us where tiles of 32 columns take 5.9).
//   A k-block costs its products (a 256-column accumulator: 555, narrower ones 8 % more a column; e4m3's
//   have twice the k), its operand stream from L2 (74 bytes a cycle and SM, 44 where rows do not begin
//   on a 128-byte line and a box row takes two) or issuing its four MMAs and commit (240, a pair 350),
//   whichever is longest.
//   A round of tiles costs its k-blocks or its share of what has to come from memory (3800 bytes a
//   cycle, which fewer than about 112 SMs do not draw), whichever is longer, and 0.44 of the other; at
//   least its epilogues, 450 for each turn of two warps of a lane quarter (the wide tiles' four are
//   charged the same).
//   The last tile's epilogue is not hidden: 1200 a turn.
//   Pairs start later and end later (1950).  Sharing a tile's k-blocks out to a cluster costs two
//   meetings (1100) and the exchange of the sums (11 bytes a cycle and CTA); the pieces have to fit in
//   the ring.
// So wide tiles where there are rounds of them, narrower ones where that fills a last round or
// spreads the weights of a few rows over all SMs, and shared k-blocks where the tiles are few and
// the rows long (60 tokens x 2048 x 8192 backward: 110 -> 55 us, most of it dx).
GluPlan glu_plan(int mode, bool whole_lines, int64_t M, int64_t N, int64_t num_k, const GluUnits& u) {
  const bool two = mode == GLU_FORWARD || mode == GLU_SLOPES;
  const int64_t twice = mode == GLU_DW ? 2 : 1;
  const double memory = (double)(M * twice + (two ? 2 : 1) * N) * num_k * kKBytes / 3800.0;
  GluPlan best;
  double best_cost = 0;
  for (int form = 0; form < 5; ++form) {  // pairs; lone CTAs; clusters of 2, 4, 8 lone CTAs
    const int cg = form == 0 ? 2 : 1, split = form < 2 ? 1 : 1 << (form - 1);
    if ((cg == 2 && M <= kGluRows) || (split > 1 && num_k < 2 * split)) continue;
    const int64_t units = form == 0 ? u.pairs : form == 1 ? u.sms : u.splits[form - 2];
    if (units < 1) continue;
    const int64_t tile_rows = kGluRows * cg, num_m = (M + tile_rows - 1) / tile_rows;
    const int64_t rows = M < kGluRows ? M : kGluRows;  // rows of A outside the matrix cost no reads
    // tcgen05.mma takes N in steps of 16, a pair's in steps of 32
    for (int bn = kMaxBN; bn >= 32; bn -= 16 * cg) {
      const int bno = two ? bn / 2 : bn, chunks = (bno + 31) / 32;
      const int64_t tiles = num_m * ((N + bno - 1) / bno) * twice;
      const int64_t rounds = (tiles + units - 1) / units, last = tiles - (rounds - 1) * units;
      const int pieces = (chunks + split - 1) / split;
      if (split > 1 && (rounds > 1 || (split - 1) * pieces * kGluRows * (two ? 256 : 128) > ring_bytes(false))) continue;
      double block = (bn == kMaxBN ? 555.0 : 600.0) * bn / kMaxBN;
      const double stream = (double)(rows + bn / cg) * kKBytes / (whole_lines ? 74.0 : 44.0);
      if (block < stream) block = stream;
      const double issue = cg == 2 ? 350.0 : 240.0;
      if (block < issue) block = issue;
      const double products = (double)((num_k + split - 1) / split) * block;
      auto round = [&](int64_t n) {  // n tiles at once
        const double active = (double)n * cg * split;
        const double read = memory * n / tiles * (active < 112.0 ? 112.0 / active : 1.0);
        return products > read ? products + 0.44 * read : read + 0.44 * products;
      };
      const int turns = (pieces + 1) / 2;
      const double full = round(units) > 450.0 * turns ? round(units) : 450.0 * turns;
      double cost = (rounds - 1) * (full + 600.0) + round(last) + 600.0 + 1200.0 * turns;
      if (cg == 2) cost += 1950.0;
      if (split > 1) cost += 1100.0 + (double)rows * bn * 4 * (split - 1) / split / 11.0;
      if (!best.cg || cost < best_cost * 0.98) {
        best.cg = cg;
        best.split = split;
        best.a_rows = M < kGluRows && mode != GLU_DW ? (int)((M + 7) / 8 * 8) : kGluRows;
        best.bno = bno;
        best.units = (int)units;
        best.tiles = tiles;
        best_cost = cost;
      }
    }
  }
  return best;
}

int glu_form(const GluPlan& p, int mode) {
  const bool wide = p.bno == (mode == GLU_FORWARD || mode == GLU_SLOPES ? kMaxBN / 2 : kMaxBN);
  if (p.cg == 2) return wide ? TFL_GLU_FORM_WIDE : TFL_GLU_FORM_PAIR;
  return p.split > 1 ? TFL_GLU_FORM_SHARED : TFL_GLU_FORM_LONE;
}

cudaError_t launch_glu(const GluPlan& p, int mode, bool f8, const GluMaps& mp, const GluArgs& a, cudaStream_t s) {
  const int is = glu_form(p, mode);
  const int form = is == TFL_GLU_FORM_SHARED ? kSplit : is == TFL_GLU_FORM_WIDE ? kWide : kNarrow;
#define TFL_LAUNCH(CG, MODE, F8, FORM) \
  if (p.cg == CG && form == FORM && mode == MODE && f8 == F8) return launch_one<CG, MODE, F8, FORM>(mp, a, p, s);
  TFL_GLU_VARIANTS(TFL_LAUNCH)
#undef TFL_LAUNCH
  return cudaErrorInvalidValue;
}

}  // namespace tfl
