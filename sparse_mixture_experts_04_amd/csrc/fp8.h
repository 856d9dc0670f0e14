// Internal declarations of the products of 8-bit floating point (e4m3).
#pragma once

#include "common.h"
#include "groups.h"

namespace moe {

// A scale covers kFp8Block values of a row of activations, and kFp8Block x
// kFp8Block of a weight matrix; rows of codes are padded with zeros to a multiple.
constexpr int kFp8Block = 128;
constexpr float kFp8Max = 448.0f;   // largest e4m3 value
inline long long fp8_row(long long K) { return (K + kFp8Block - 1) / kFp8Block * kFp8Block; }

hipError_t launch_quantize_fp8(long long rows, int K, bool bf16, const void* x, uint8_t* codes,
                               float* scales, hipStream_t st);
hipError_t launch_quantize_fp8_weights(int E, int N, int K, bool bf16, const void* w,
                                       uint8_t* codes, float* scales, hipStream_t st);

// out[r, n] = sum_b a_scale[r, b] w_scale[g, n / 128, b] sum_{k in b} a[r, k] w[g, n, k]
// for the rows r of group g (group_rows in groups.h).
struct Fp8Args {
  const uint8_t* a;       // [M, Kp]
  const float* a_scale;   // [M, Kp / 128]
  const uint8_t* w;       // [E, N, Kp]
  const float* w_scale;   // [E, ceil(N / 128), Kp / 128]
  const int32_t* offsets;
  void* out;              // [M, N]
  float* part;            // [splits, M, N]
  int M, N, Kp, E;
  static constexpr int S = 0, T = 0;
  int splits;             // slices of K (fp8_splits)
  bool out_bf16;
};
// Whether a product goes in blocks of 32 rows (blocks.hip).
bool fp8_blocks(int M, int N, int Kp, int E);
int fp8_splits(int M, int N, int Kp, int E);
// Estimated time of the 128-row tiles (us).
double fp8_tiles_time(int M, int N, int Kp, int E);
hipError_t launch_gemm_fp8(const Fp8Args& a, hipStream_t st);
hipError_t launch_gemm_fp8_big(const Fp8Args& a, hipStream_t st);

}  // namespace moe
