// Internal declarations of the 8-bit integer products.
#pragma once

#include "common.h"

namespace moe {

// Rows of codes are padded with zeros to a multiple of kCodeRow values.
constexpr int kCodeRow = 128;
inline long long code_row(long long K) { return (K + kCodeRow - 1) / kCodeRow * kCodeRow; }

// A sum of K products of codes of magnitude up to 127 fits 32 bits:
// 127^2 * 131072 < 2^31.
constexpr int kInt8MaxK = 131072;
constexpr int kInt8MaxGroups = 256;
// Rows and columns of a product, at most: rounded up to a tile they stay in 32 bits.
constexpr long long kInt8MaxRows = (1LL << 31) - 1024;

// Rows of fp32 or bf16 values to codes [rows, code_row(K)] and scales [rows].
hipError_t launch_quantize_int8(long long rows, int K, bool bf16, const void* x, int8_t* codes,
                                float* scales, hipStream_t st);

// One or two grouped products of 8-bit rows.  Groups 0..E-1 own the rows
// offsets[g]..offsets[g+1] (clamped to [0, M]; without offsets group 0 owns all
// M rows); groups E..E+S-1 are the shared experts with T rows each.
// Plain: out[r, n] = s_r t_n sum_k a[r, k] w0[g, n, k]; the rows of shared
// expert s are M + s T + t.  GATED: h[r, n] = silu(gate) * up, gate and up the
// products with w0 and w1, in fp32; row r of a routed group is row
// sorted_pair[r] / k of a, row t of a shared group is row t of a.
struct Int8Args {
  const int8_t* a;
  const float* a_scale;
  const int8_t* w0;       // routed [E, N, Kp]
  const int8_t* w1;       // GATED: the up weights
  const float* t0;        // [E, N]
  const float* t1;
  const int8_t* ws0;      // shared [S, N, Kp]
  const int8_t* ws1;
  const float* ts0;
  const float* ts1;
  const int32_t* offsets;
  const int32_t* sorted_pair;
  void* out;              // routed rows
  void* out_shared;       // shared rows s T + t
  int M, N, Kp, E, S, T, k;
  bool out_bf16;          // plain: bf16 or fp32 output (GATED: fp32)
};
// counters: gemm_int8_counter_ints() of workspace, for up to two products in turn.
// cleared: whether a call before this one has cleared them; set when this one has.
hipError_t launch_gemm_int8(const Int8Args& a, bool gated, int32_t* counters, bool& cleared,
                            hipStream_t st);
size_t gemm_int8_counter_ints();

}  // namespace moe
