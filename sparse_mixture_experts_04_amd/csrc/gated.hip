// Kernel of a product of the gated block.
#include "gated.h"
#include "stream.h"

namespace moe {

static bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

hipError_t launch_gated(const GatedArgs& a, GatedPart part, hipStream_t st) {
  // rows of x and of the matrices that start on 16 bytes
  const bool wide = static_cast<long long>(a.d) * (a.bf16 ? 2 : 4) % 16 == 0 && on16(a.x) &&
                    on16(a.w_gate) && on16(a.w_up);
  if (part == GatedPart::kForward && wide && a.M / a.E < 24) {
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
    const long long mean = part == GatedPart::kDw ? a.F : a.M / a.E;
    return launch_gated_big(a, part, mean > 160 ? 256 : 128, st);
  }
  return launch_gated_tile(a, part, st);
}

}  // namespace moe
