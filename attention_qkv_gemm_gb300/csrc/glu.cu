// glu.cu -- the gated feed-forward block h = act(x Wg^T) * (x Wu^T), forward and backward.
//
// One persistent tcgen05 GEMM kernel (tile_gemm.cuh) in four modes:
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
//   GRAD_DX       dx = dg Wg + du Wu: one sum over 2 d_ff, W read as [k, n] (MN-major).
//   GRAD_DW       dWg = dg^T x and dWu = du^T x: sums over the tokens, both operands MN-major.
//
// What bounds it: with many tokens the tensor cores, and in long runs the power cap (8192 x 1024 x 4096
// fp16 forward 78 us in a burst, 1.76 PFLOP/s, 0.94 of the measured burst rate, 92 us in a long run;
// 16384 x 2048 x 8192 bf16 backward 1.71 ms and 2.01 ms; 74 us and 1.76 ms on another GPU); with few
// tokens the weights' bytes (40 x 4096 x 10240 e4m3: 16.4 us for 85 MB, 5.2 TB/s).  A pair's 256 x 256
// tile took the first two from 107 to 101 us and from 2.26 to 2.06 ms against a lone CTA's 128 x 256, a
// thread that the compiler knows to be alone for the issue of MMAs from 82 to 74 us and from 1.95 to
// 1.76 ms (bursts, one GPU).  The epilogue's arithmetic is not free even where it hides under the MMAs:
// its warps take issue slots from that thread, hence packed pairs and the short issue loop.
#include "tile_gemm.cuh"

namespace tfl {

namespace {

template <int MODE>
__device__ __forceinline__ float2 column_scales(const TileArgs& args, int n) {
  return make_float2(__ldg(args.g_scale + n), __ldg(args.u_scale + n));
}

}  // namespace

// Every (mode, operand form) in every (CTAs of a tile, form).
#define TFL_GLU_MODES(X, CG, FORM)                                                                  \
  X(CG, GLU_FORWARD, false, FORM) X(CG, GLU_FORWARD, true, FORM) X(CG, GLU_SLOPES, false, FORM)     \
  X(CG, GRAD_DX, false, FORM) X(CG, GRAD_DW, false, FORM)
#define TFL_GLU_VARIANTS(X) \
  TFL_GLU_MODES(X, 2, kWide) TFL_GLU_MODES(X, 2, kNarrow) TFL_GLU_MODES(X, 1, kNarrow) TFL_GLU_MODES(X, 1, kSplit)

cudaError_t prepare_tile_kernels(TileUnits* u) {
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
TilePlan tile_plan(int mode, bool whole_lines, int64_t M, int64_t N, int64_t num_k, const TileUnits& u, int planes,
                   int shares) {
  const bool two = mode == GLU_FORWARD || mode == GLU_SLOPES;
  const int64_t twice = mode == GRAD_DW ? planes * shares : 1;
  const double memory = (double)(M * twice + (two ? 2 : 1) * shares * N) * num_k * kKBytes / 3800.0;
  TilePlan best;
  for (int form = 0; form < (shares > 1 ? 2 : 5); ++form) {  // pairs; lone CTAs; clusters of 2, 4, 8 lone CTAs
    const int cg = form == 0 ? 2 : 1, split = form < 2 ? 1 : 1 << (form - 1);
    if ((cg == 2 && M <= kTileRows) || (split > 1 && num_k < 2 * split)) continue;
    const int64_t units = form == 0 ? u.pairs : form == 1 ? u.sms : u.splits[form - 2];
    if (units < 1) continue;
    const int64_t tile_rows = kTileRows * cg, num_m = (M + tile_rows - 1) / tile_rows;
    const int64_t rows = M < kTileRows ? M : kTileRows;  // rows of A outside the matrix cost no reads
    // tcgen05.mma takes N in steps of 16, a pair's in steps of 32; the linear layer stores 32 columns at a time
    for (int bn = kMaxBN; bn >= 32; bn -= mode == LIN_FORWARD ? 32 : 16 * cg) {
      const int bno = two ? bn / 2 : bn, chunks = (bno + 31) / 32;
      const int64_t tiles = num_m * ((N + bno - 1) / bno) * twice;
      const int64_t rounds = (tiles + units - 1) / units, last = tiles - (rounds - 1) * units;
      const int pieces = (chunks + split - 1) / split;
      if (split > 1 && (rounds > 1 || (split - 1) * pieces * kTileRows * (two ? 256 : 128) > ring_bytes(false, mode == LIN_FORWARD))) continue;
      double block = (bn == kMaxBN ? 555.0 : 600.0) * bn / kMaxBN;
      // (MN-major B comes in boxes of 64 columns; the feed-forward's constants were fitted without that)
      const int loaded = planes == 1 && (mode == GRAD_DX || mode == GRAD_DW) ? (bn / cg + 63) / 64 * 64 : bn / cg;
      const double stream = (double)(rows + loaded) * kKBytes / (whole_lines ? 74.0 : 44.0);
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
      if (!best.cg || cost < best.cost * 0.98) {
        best.cg = cg;
        best.split = split;
        best.a_rows = M < kTileRows && mode != GRAD_DW ? (int)((M + 7) / 8 * 8) : kTileRows;
        best.bno = bno;
        best.units = (int)units;
        best.tiles = tiles;
        best.cost = cost;
      }
    }
  }
  return best;
}

int tile_form(const TilePlan& p, int mode) {
  const bool wide = p.bno == (mode == GLU_FORWARD || mode == GLU_SLOPES ? kMaxBN / 2 : kMaxBN);
  if (p.cg == 2) return wide ? TFL_GLU_FORM_WIDE : TFL_GLU_FORM_PAIR;
  return p.split > 1 ? TFL_GLU_FORM_SHARED : TFL_GLU_FORM_LONE;
}

cudaError_t launch_tiles(const TilePlan& p, int mode, bool f8, const TileMaps& mp, const TileArgs& a, cudaStream_t s) {
  const int is = tile_form(p, mode);
  const int form = is == TFL_GLU_FORM_SHARED ? kSplit : is == TFL_GLU_FORM_WIDE ? kWide : kNarrow;
#define TFL_LAUNCH(CG, MODE, F8, FORM) \
  if (p.cg == CG && form == FORM && mode == MODE && f8 == F8) return launch_one<CG, MODE, F8, FORM>(mp, a, p, s);
  TFL_GLU_VARIANTS(TFL_LAUNCH)
#undef TFL_LAUNCH
  return cudaErrorInvalidValue;
}

}  // namespace tfl
