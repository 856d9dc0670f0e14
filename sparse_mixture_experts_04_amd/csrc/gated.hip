// Kernel of a product of the gated block.
#include <algorithm>
#include <cmath>

#include "blocks.h"
#include "gated.h"

namespace moe {

static bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Forward: blocks of 32 rows (blocks.hip) for rows of 16 bytes.  In fp32 they are
// bound by the same instruction as tiles of 64 and 128 and start and end sooner; in
// bf16 they are taken for few rows a group, and where their estimated time is below
// that of the tiles.  Measured (us, bf16, blocks / tiles; fp32, blocks / tiles of 64):
//   M=333 d=520 F=264       5.0 / 13.7     8.4 / 24
//   M=64 d=2048 F=768       5.9 / 13.3     15.6 / 38
//   M=256, 512, 1000        9.6 / 17.4, 14.4 / 19.5, 26.0 / 27.4     (1000 rows) 72 / 110
//   M=2000 d=1024 F=512     21.8 / 18.3    53 / 62 (M=2048)
//   M=300 d=7168 F=2048     62.7 / 36.5
//   d=2048 F=768, 256 groups   384 rows 205 / 226, 1000 rows 285 / 291
//                              1000 rows 525 / 637, 4000 rows 657 / 1109
static bool in_blocks(int M, int d, int F, int E, bool bf16, GatedPart part) {
  if (part != GatedPart::kForward) return false;
  return !bf16 || (E == 1 ? M <= 16 : M / E < 3) ||
         blocks_time(M, F, 2LL * d, E, true) < gated_tiles_time(M, d, F, E, part);
}

// Gradients of few results: blocks of 32 x 32 whose K the waves of a workgroup share, K
// in chunks of 64 for each; as the forward pass of rows that do not start on 16 bytes.
// On the fp32 matrix cores: while tiles of 64 would leave compute units without one.
// Measured (us, tiles of 64 / blocks): fp32 M=333 d=520 F=264 dx 32 / 10.5, dW 19 / 10.
// bf16 in rows of 16 bytes has tiles on its own matrix instruction, so that only chunks
// few and short win (us, its tiles / blocks, dx and dW):
//   M=40 d=64 F=32   14 / 5.1      700 rows, 7 groups, d=256 F=96    20.9 / 14.7
//   M=333 d=520 F=264  24.4 / 18.6     2000 rows, 64 groups          20.2 / 29
//   M=64 d=2048 F=768  21.9 / 44
struct SmallWork {
  double blocks, chunks;
};
static SmallWork small_work(int M, int d, int F, int E, GatedPart part) {
  const double entries = std::ceil(M / 32.0) + (E > 1 ? std::min(M, E) : 0);
  if (part == GatedPart::kDx) return {entries * std::ceil(d / 32.0), std::ceil(F / 32.0)};
  return {std::ceil(2.0 * F / 32) * E * std::ceil(d / 32.0), std::ceil(M / 64.0 / E)};
}
static bool is_small(int M, int d, int F, int E, bool big, GatedPart part) {
  if (big) {
    if (part == GatedPart::kForward) return false;
    const SmallWork w = small_work(M, d, F, E, part);
    return w.chunks <= 10 && w.blocks <= 512 && w.blocks * w.chunks <= 2048;
  }
  const double cols = part == GatedPart::kForward ? 2.0 * F : d;
  const double rows = part == GatedPart::kDw ? 2.0 * F * E : M;
  return std::ceil(rows / 64) * std::ceil(cols / 64) < 256;
}

static bool rows_of_8(int d, int F, bool bf16) { return bf16 && d % 8 == 0 && F % 8 == 0; }

size_t gated_part_floats(int M, int d, int F, int E, bool bf16, GatedPart part) {
  if (!rows_of_8(d, F, bf16) || M == 0 || in_blocks(M, d, F, E, bf16, part) ||
      is_small(M, d, F, E, true, part))
    return 0;
  const int s = gated_splits(M, d, F, E, part);
  if (s == 1) return 0;
  const size_t rows = part == GatedPart::kDw ? 2 * static_cast<size_t>(F) : M;
  return s * rows * (part == GatedPart::kForward ? 2 * static_cast<size_t>(F) : d);
}

// Rows of x and of the matrices that start on 16 bytes.
static bool wide_rows(const GatedArgs& a) {
  return static_cast<long long>(a.d) * (a.bf16 ? 2 : 4) % 16 == 0 && on16(a.x) && on16(a.w_gate) &&
         on16(a.w_up);
}
// Whether the tiles on the bf16 matrix instruction take a product.
static bool big_tiles(const GatedArgs& a, GatedPart part) {
  const bool out16 = part == GatedPart::kForward ? on16(a.h) && on16(a.pre)
                     : part == GatedPart::kDx    ? on16(a.dx)
                                                 : on16(a.dw_gate) && on16(a.dw_up);
  return rows_of_8(a.d, a.F, a.bf16) && wide_rows(a) && out16;
}

hipError_t launch_gated(const GatedArgs& a, GatedPart part, hipStream_t st) {
  const bool big = big_tiles(a, part);
  if (part == GatedPart::kForward && wide_rows(a) &&
      (!big || in_blocks(a.M, a.d, a.F, a.E, a.bf16, part))) {
    BlockArgs b{};
    b.a = a.x;
    b.w0 = a.w_gate;
    b.w1 = a.w_up;
    b.offsets = a.offsets;
    b.out = a.h;
    b.pre = a.pre;
    b.M = a.M;
    b.N = a.F;
    b.K = a.d;
    b.E = a.E;
    return launch_blocks(b, a.bf16 ? BlockKind::kGatedBf16 : BlockKind::kGatedF32, st);
  }
  if (is_small(a.M, a.d, a.F, a.E, big, part)) return launch_gated_small(a, part, st);
  if (big) {
    GatedArgs b = a;
    b.splits = gated_part_floats(a.M, a.d, a.F, a.E, true, part) > 0
                   ? gated_splits(a.M, a.d, a.F, a.E, part)
                   : 1;
    return launch_gated_big(b, part, st);
  }
  return launch_gated_tile(a, part, st);
}

// Small gradients take one launch together; with few and short chunks da and du are
// made where they are used, which saves the launch before it (us, a launch for each /
// one after da and du / one alone): fp32 M=333 d=520 F=264 22.8 / 16 / 21.5, M=40 d=256
// F=64 10.1 / 6.9 / 6.3, 300 rows, 7 groups, d=256 F=96 15.4 / 10.5 / 10.1, M=1000 d=256
// F=128 22.2 / 19.2 / 30.
hipError_t launch_gated_gradients(const GatedArgs& a, hipStream_t st) {
  bool small = true;
  double blocks = 0, chunks = 0;
  for (GatedPart part : {GatedPart::kDx, GatedPart::kDw}) {
    if (!(part == GatedPart::kDx ? a.dx : a.dw_gate)) continue;
    small = small && is_small(a.M, a.d, a.F, a.E, big_tiles(a, part), part);
    const SmallWork w = small_work(a.M, a.d, a.F, a.E, part);
    blocks += w.blocks;
    chunks = std::max(chunks, w.chunks);
  }
  if (blocks == 0) return hipSuccess;  // nothing is wanted
  const bool from_pre = small && chunks <= 4 && blocks <= 512;
  hipError_t e = from_pre ? hipSuccess : launch_gated_dau(a, st);
  if (e != hipSuccess) return e;
  if (small) return launch_gated_small_grads(a, from_pre, st);
  if (a.dx) e = launch_gated(a, GatedPart::kDx, st);
  if (e == hipSuccess && a.dw_gate) e = launch_gated(a, GatedPart::kDw, st);
  return e;
}

}  // namespace moe
