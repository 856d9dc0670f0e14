// C ABI of the gated feed-forward block: host-side validation, workspace layout
// and the order of launches (include/moe.h has the meaning of every argument).
#include <initializer_list>

#include "../../include/moe.h"
#include "api.h"
#include "gated.h"

using namespace moe;

namespace {

constexpr long long kGatedMaxRows = (1LL << 31) - 1024;  // rounded up to a tile: 32 bits
constexpr int kGatedMaxWidth = 131072;

moe_status check_gated(const moe_gated_ff_desc* d) {
  if (!d) return MOE_ERR_NULL;
  if (d->M < 0 || d->d <= 0 || d->F <= 0 || d->E <= 0) return MOE_ERR_SHAPE;
  if (d->act != MOE_F32 && d->act != MOE_BF16) return MOE_ERR_DTYPE;
  if (d->d > kGatedMaxWidth || d->F > kGatedMaxWidth || d->E > kMaxGroups ||
      d->M > kGatedMaxRows)
    return MOE_ERR_UNSUPPORTED;
  const long long lim = 1LL << 40, wide = d->d > 2 * d->F ? d->d : 2 * d->F;
  if (d->M >= lim / wide || static_cast<long long>(d->E) * d->F >= lim / d->d)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

GatedArgs gated_args(const moe_gated_ff_desc* d, const void* x, const void* w_gate,
                     const void* w_up, const int32_t* offsets) {
  GatedArgs a{};
  a.x = x;
  a.w_gate = w_gate;
  a.w_up = w_up;
  a.offsets = offsets;
  a.M = d->M;
  a.d = d->d;
  a.F = d->F;
  a.E = d->E;
  a.bf16 = d->act == MOE_BF16;
  return a;
}

// Whether p starts on a value of the block's type.
bool on_value(const void* p, const GatedArgs& a) {
  return reinterpret_cast<uintptr_t>(p) % (a.bf16 ? 2 : 4) == 0;
}
bool on4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

// Carves the workspace into a: dau of the backward pass, the products where they are
// not saved, and the sums of the slices of one product after another.
void carve_gated(Carver& c, GatedArgs& a, bool backward, bool saved) {
  if (backward) {
    const size_t cols = static_cast<size_t>(a.M) * 2 * a.F;
    a.dau = a.bf16 ? static_cast<void*>(c.take<bf16_t>(cols)) : c.take<float>(cols);
    if (!saved) a.pre = c.take<float>(cols);
  }
  size_t part = 0;
  for (GatedPart k : {GatedPart::kForward, GatedPart::kDx, GatedPart::kDw}) {
    if (!backward && k != GatedPart::kForward) continue;
    const size_t n = gated_part_floats(a.M, a.d, a.F, a.E, a.bf16, k);
    part = n > part ? n : part;
  }
  a.part = c.take<float>(part);
}

}  // namespace

extern "C" {

moe_status moe_gated_ff_workspace_size(const moe_gated_ff_desc* desc, int32_t backward,
                                       int32_t saved, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const moe_status st = check_gated(desc);
  if (st != MOE_OK) return st;
  GatedArgs a = gated_args(desc, nullptr, nullptr, nullptr, nullptr);
  Carver c{nullptr};
  carve_gated(c, a, backward != 0, saved != 0);
  *bytes = c.used;
  return MOE_OK;
}

moe_status moe_gated_ff(const moe_gated_ff_desc* desc, const void* x, const void* w_gate,
                        const void* w_up, const int32_t* offsets, void* h, float* pre, void* ws,
                        size_t ws_bytes, hipStream_t stream) {
  moe_status st = check_gated(desc);
  if (st != MOE_OK) return st;
  if (desc->M == 0) return MOE_OK;
  if (!x || !w_gate || !w_up || !h || (!offsets && desc->E != 1)) return MOE_ERR_NULL;
  GatedArgs a = gated_args(desc, x, w_gate, w_up, offsets);
  if (!on_value(x, a) || !on_value(w_gate, a) || !on_value(w_up, a) || !on_value(h, a) ||
      !on4(offsets) || !on4(pre))
    return MOE_ERR_UNSUPPORTED;
  size_t need = 0;
  st = moe_gated_ff_workspace_size(desc, 0, 1, &need);
  if (st != MOE_OK) return st;
  if (need > 0 && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) % 16 != 0) return MOE_ERR_UNSUPPORTED;
  Carver c{static_cast<char*>(ws)};
  carve_gated(c, a, false, true);
  a.h = h;
  a.pre = pre;
  return hip_status(launch_gated(a, GatedPart::kForward, stream));
}

moe_status moe_gated_ff_backward(const moe_gated_ff_desc* desc, const void* x, const void* w_gate,
                                 const void* w_up, const int32_t* offsets, const void* dh,
                                 const float* pre, void* dx, void* dw_gate, void* dw_up, void* ws,
                                 size_t ws_bytes, hipStream_t stream) {
  size_t need = 0;
  moe_status st = moe_gated_ff_workspace_size(desc, 1, pre != nullptr, &need);
  if (st != MOE_OK) return st;
  if ((dw_gate == nullptr) != (dw_up == nullptr)) return MOE_ERR_NULL;
  if (!offsets && desc->E != 1) return MOE_ERR_NULL;
  // without rows the gradients of the weights are zeros all the same
  const bool rows = desc->M > 0;
  if (rows && (!x || !w_gate || !w_up || !dh)) return MOE_ERR_NULL;
  GatedArgs a = gated_args(desc, x, w_gate, w_up, offsets);
  for (const void* p : {x, w_gate, w_up, dh, const_cast<const void*>(dx),
                        const_cast<const void*>(dw_gate), const_cast<const void*>(dw_up)})
    if (!on_value(p, a)) return MOE_ERR_UNSUPPORTED;
  if (!on4(offsets) || !on4(pre)) return MOE_ERR_UNSUPPORTED;
  if (need > 0 && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) % 16 != 0) return MOE_ERR_UNSUPPORTED;
  Carver c{static_cast<char*>(ws)};
  carve_gated(c, a, true, pre != nullptr);
  a.dh = dh;
  a.dx = dx;
  a.dw_gate = dw_gate;
  a.dw_up = dw_up;
  hipError_t e = hipSuccess;
  if (rows) {
    if (pre) {
      a.pre = const_cast<float*>(pre);
    } else {
      // h is not wanted: the product runs again for a and u alone
      e = launch_gated(a, GatedPart::kForward, stream);
    }
    if (e == hipSuccess) e = launch_gated_gradients(a, stream);
  } else if (dw_gate) {
    e = launch_gated(a, GatedPart::kDw, stream);
  }
  return hip_status(e);
}

}  // extern "C"
