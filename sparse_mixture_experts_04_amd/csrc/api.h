// Host-side helpers of the C ABI: descriptor checks and workspace carving.
#pragma once

#include <cmath>

#include "../../include/moe.h"
#include "common.h"

namespace moe {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline moe_status check_desc(const moe_desc* d) {
  if (!d) return MOE_ERR_NULL;
  if (d->T < 0 || d->d <= 0 || d->F <= 0 || d->E <= 0 || d->S < 0 || d->k <= 0)
    return MOE_ERR_SHAPE;
  if (d->act != MOE_F32 && d->act != MOE_BF16) return MOE_ERR_DTYPE;
  const bool fp4 = d->act == MOE_BF16 && d->weight == MOE_MXFP4;
  if (d->weight != d->act && !fp4) return MOE_ERR_DTYPE;
  if (d->gate_norm != MOE_GATE_RATIO && d->gate_norm != MOE_GATE_LOGSUMEXP) return MOE_ERR_SHAPE;
  if (!(d->gate_scale > 0.0f) || !(d->gate_scale < INFINITY)) return MOE_ERR_SHAPE;
  if (!(d->capacity_factor >= 0.0f) || !(d->capacity_factor < INFINITY)) return MOE_ERR_SHAPE;
  if ((d->E != 64 && d->E != 128 && d->E != 256) || d->S > 2 || d->k != 6)
    return MOE_ERR_UNSUPPORTED;
  if (d->d % 32 != 0) return MOE_ERR_UNSUPPORTED;
  const long long T = d->T;
  if (T * d->k >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  const long long wide = d->d > d->F ? d->d : d->F;
  if (T * (d->k + d->S) * wide >= (1LL << 40)) return MOE_ERR_UNSUPPORTED;
  // FP4 routed weights: decode batches (the 32-row GEMM path) only
  if (fp4 && T * d->k >= 48LL * d->E) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The expert GEMMs' tiles need d % 256 == 0 and F % 128 == 0 (the router,
// dispatch, combine and bias update only d % 32 == 0).
inline moe_status check_ffn_desc(const moe_desc* d) {
  const moe_status st = check_desc(d);
  if (st != MOE_OK) return st;
  if (d->d % 256 != 0 || d->F % 128 != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

inline Shape to_shape(const moe_desc* d) {
  Shape s;
  s.T = d->T;
  s.d = d->d;
  s.F = d->F;
  s.E = d->E;
  s.S = d->S;
  s.k = d->k;
  s.bf16 = d->act == MOE_BF16;
  s.w_fp4 = d->weight == MOE_MXFP4;
  s.gate_logsumexp = d->gate_norm == MOE_GATE_LOGSUMEXP;
  s.gate_scale = d->gate_scale;
  s.capacity = INT32_MAX;
  if (d->capacity_factor > 0.0f) {
    const double c = std::ceil(static_cast<double>(d->capacity_factor) *
                               static_cast<double>(static_cast<long long>(d->k) * d->T) /
                               static_cast<double>(d->E));
    s.capacity = c < static_cast<double>(INT32_MAX) ? static_cast<int>(c) : INT32_MAX;
  }
  return s;
}

// Workspace carving: a bump allocator over the caller's buffer.
struct Carver {
  char* base;
  size_t used = 0;
  template <typename T> T* take(size_t count) {
    T* p = reinterpret_cast<T*>(base ? base + used : nullptr);
    used = align_up(used + count * sizeof(T));
    return p;
  }
};

inline moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

inline bool weights_ok(const moe_weights* w, const Shape& s) {
  if (!(w && w->w_gate && w->w_up && w->w_down)) return false;
  if (s.S > 0 && !(w->ws_gate && w->ws_up && w->ws_down)) return false;
  return !s.w_fp4 || (w->sc_gate && w->sc_up && w->sc_down);
}

}  // namespace moe
