// Rows of the groups of an 8-bit product.
#pragma once

#include "groups.h"
#include "int8.h"

namespace moe {

static_assert(kInt8MaxGroups <= kMaxGroups, "groups of a plan");

// Row of a that row r of a group is (first row lo of the group's rows).
template <bool GATED>
__device__ __forceinline__ long long source_row(const Int8Args& p, bool routed, int ge, int lo,
                                                int r) {
  if (!routed) return GATED ? r : static_cast<long long>(p.M) + static_cast<long long>(ge) * p.T + r;
  return GATED ? clampi(p.sorted_pair[lo + r] / p.k, 0, p.T - 1) : lo + r;
}

hipError_t launch_gemm_int8_tiles(const Int8Args& a, bool gated, hipStream_t st);

}  // namespace moe
