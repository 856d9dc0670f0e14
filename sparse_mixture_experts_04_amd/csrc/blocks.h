// Internal declarations of the products in blocks of 32 rows (blocks.hip).
#pragma once

#include "common.h"
#include "groups.h"

namespace moe {

enum class BlockKind { kFp8, kGatedBf16, kGatedF32 };

struct BlockArgs {
  const void* a;          // activations [M, K]
  const void* w0;         // weights [E, N, K]; gated: Wg and Wu
  const void* w1;
  const float* a_scale;   // kFp8: [M, K / 128]
  const float* w_scale;   // kFp8: [E, ceil(N / 128), K / 128]
  const int32_t* offsets;
  void* out;              // [M, N], null: not wanted (gated)
  float* pre;             // gated: [M, 2N], null: not kept
  int M, N, K, E;
  static constexpr int S = 0, T = 0;
  bool out_bf16;          // kFp8
};

// Rows of a and of the weights start on 16 bytes and are a multiple of it long.
hipError_t launch_blocks(const BlockArgs& a, BlockKind kind, hipStream_t st);

// Estimated time of it (us): two workgroups a compute unit at a time, and for each block
// a start, an end and a step for every 128 bytes of a row.
double blocks_time(int M, int N, long long row_bytes, int E, bool gated);

}  // namespace moe
