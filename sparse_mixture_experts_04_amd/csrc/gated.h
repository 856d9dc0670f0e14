// Internal declarations of the gated feed-forward block and its gradients.
#pragma once

#include "common.h"
#include "groups.h"

namespace moe {

// h = silu(a) * u with a = x Wg^T, u = x Wu^T, for the rows of E groups (see
// group_rows in groups.h; S = T = 0), and from dh the gradients
//   da = dh u s (1 + a (1 - s)),  du = dh a s,  s = 1 / (1 + exp(-a))
//   dx = da Wg + du Wu,  dWg = da^T x,  dWu = du^T x
// da and du lie side by side in dau [M, 2F], a and u in pre [M, 2F].
struct GatedArgs {
  const void* x;          // [M, d]
  const void* w_gate;     // [E, F, d]
  const void* w_up;
  const int32_t* offsets;
  void* h;                // [M, F], null: not wanted
  float* pre;             // [M, 2F], null: not kept
  const void* dh;         // [M, F]
  void* dau;              // [M, 2F]
  void* dx;               // [M, d], null: not wanted
  void* dw_gate;          // [E, F, d], null: not wanted
  void* dw_up;
  float* part;            // sums of slices of K
  int M, d, F, E;
  static constexpr int S = 0, T = 0;
  int splits;             // slices of K (gated_splits; set by launch_gated)
  bool bf16;
};

// Which of the block's products a launch computes.
enum class GatedPart { kForward, kDx, kDw };

__device__ __forceinline__ float sigmoid(float a) { return 1.0f / (1.0f + expf(-a)); }

// The kernel of one of the block's products.
hipError_t launch_gated(const GatedArgs& a, GatedPart part, hipStream_t st);
// The gradients that are wanted, from pre and dh.
hipError_t launch_gated_gradients(const GatedArgs& a, hipStream_t st);
// Any sizes, either type, on the fp32 matrix cores (gated_tile.hip): in tiles; in blocks
// of 32 x 32 whose K the waves share; all gradients in one launch of such blocks
// (from_pre: da and du made where they are used, otherwise they lie in dau).
hipError_t launch_gated_tile(const GatedArgs& a, GatedPart part, hipStream_t st);
hipError_t launch_gated_small(const GatedArgs& a, GatedPart part, hipStream_t st);
hipError_t launch_gated_small_grads(const GatedArgs& a, bool from_pre, hipStream_t st);
// bf16 rows of 16-byte pieces, in tiles of 128 or 256 rows (gated_big.hip).
hipError_t launch_gated_big(const GatedArgs& a, GatedPart part, hipStream_t st);
int gated_splits(int M, int d, int F, int E, GatedPart part);
// Estimated time of the 128-row tiles (us).
double gated_tiles_time(int M, int d, int F, int E, GatedPart part);
// Floats of GatedArgs::part that a product may need (0: none).
size_t gated_part_floats(int M, int d, int F, int E, bool bf16, GatedPart part);
// pre, dh -> dau.
hipError_t launch_gated_dau(const GatedArgs& a, hipStream_t st);

}  // namespace moe
