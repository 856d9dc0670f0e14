// Kernel of a product of the gated block.
#include "gated.h"
#include "stream.h"

namespace moe {

static bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Few rows a group: the stream of the weights instead of tiles.  Measured (us, stream
// / tiles, the forward pass):
//   d=2048 F=768    bf16  1 row 9 / 13, 16 rows 12 / 12, 64 rows 15 / 13.5
//                   fp32  1 row 11 / 18, 32 rows 15.5 / 18, 64 rows 22 / 19
//   d=7168 F=2048   bf16  8 rows 18 / 20, 32 rows 28 / 22    fp32  32 rows 48 / 69
//   d=512 F=2048    fp32  16 rows 12 / 8
//   d=2048 F=768, 256 groups   bf16  384 rows 217 / 226, 1000 rows 316 / 273
//                              fp32  1000 rows 668 / 1086, 4000 rows 1047 / 1833
static bool streams(int M, int d, int E, bool bf16, GatedPart part) {
  if (part != GatedPart::kForward) return false;
  if (bf16) return E == 1 ? M <= 16 : M / E < 3;
  return d >= 1024 && (E == 1 ? M <= 32 : M / E < 24);
}

size_t gated_part_floats(int M, int d, int F, int E, bool bf16, GatedPart part) {
  if (!bf16 || d % 8 != 0 || F % 8 != 0 || M == 0 || streams(M, d, E, bf16, part)) return 0;
  const int s = gated_splits(M, d, F, E, part);
  if (s == 1) return 0;
  const size_t rows = part == GatedPart::kDw ? 2 * static_cast<size_t>(F) : M;
  return s * rows * (part == GatedPart::kForward ? 2 * static_cast<size_t>(F) : d);
}

hipError_t launch_gated(const GatedArgs& a, GatedPart part, hipStream_t st) {
  // rows of x and of the matrices that start on 16 bytes
  const bool wide = static_cast<long long>(a.d) * (a.bf16 ? 2 : 4) % 16 == 0 && on16(a.x) &&
                    on16(a.w_gate) && on16(a.w_up);
  if (streams(a.M, a.d, a.E, a.bf16, part) && wide) {
    StreamArgs s{};
    s.a = a.x;
    s.w0 = a.w_gate;
    s.w1 = a.w_up;
    s.offsets = a.offsets;
    s.out = a.h;
    s.pre = a.pre;
    s.M = a.M;
    s.N = a.F;
    s.K = a.d;
    s.E = a.E;
    return launch_stream(s, a.bf16 ? StreamKind::kGatedBf16 : StreamKind::kGatedF32, st);
  }
  const bool out16 = part == GatedPart::kForward ? on16(a.h) && on16(a.pre)
                     : part == GatedPart::kDx    ? on16(a.dx)
                                                 : on16(a.dw_gate) && on16(a.dw_up);
  if (a.bf16 && wide && a.F % 8 == 0 && out16) {
    GatedArgs b = a;
    b.splits = gated_part_floats(a.M, a.d, a.F, a.E, true, part) > 0
                   ? gated_splits(a.M, a.d, a.F, a.E, part)
                   : 1;
    return launch_gated_big(b, part, st);
  }
  return launch_gated_tile(a, part, st);
}

}  // namespace moe
