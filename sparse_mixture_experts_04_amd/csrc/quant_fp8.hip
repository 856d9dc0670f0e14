// Quantisers of the e4m3 products.
//
// A block of values (128 of a row, or 128 x 128 of a weight matrix) becomes
// s = max|x| / 448, rounded to fp32 and at least 2^-126, and for each value the
// e4m3 number nearest to the exact quotient x / s, ties to the even code.  A block
// of zeros has scale 0 and codes 0, one that holds a NaN or an infinity scale NaN
// and codes 0.
//
// The conversion instruction rounds fp32 to the nearest e4m3 number, but the fp32
// product x (1 / s) is up to 3 units in the last place off the quotient.  Where two
// values 2^-21 on either side of it round alike, so does the quotient.  Elsewhere
// (one value in some 10^5) the two candidates' midpoint m decides: m has 5
// significant bits, and x - m s in one fused multiply-add has the exact sign.
#include <cmath>
#include <type_traits>

#include "fp8.h"
#include "int8_quant.h"

namespace moe {

namespace {

__device__ __forceinline__ float fp8_value(uint32_t code) {
  return __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(code), 0);
}
// The code of x / s out of the two on either side, lo and hi in order of magnitude.
__device__ __forceinline__ uint32_t fp8_near(float x, float s, uint32_t lo, uint32_t hi) {
  const float a = fp8_value(lo & 0x7f), b = fp8_value(hi & 0x7f);
  // the smallest scales moved up by a power of two, where the difference is a normal number
  const float up60 = s < 0x1p-60f ? 0x1p60f : 1.0f;
  const float r = fmaf(-0.5f * (a + b), s * up60, fabsf(x) * up60);
  const bool up = r > 0.0f || (r == 0.0f && (hi & 1) == 0);
  return up ? hi : lo;
}

// The codes of x0 / s and x1 / s in the low 16 bits (inv = 1 / s).
__device__ __forceinline__ uint32_t fp8_pair(float x0, float x1, float s, float inv) {
  constexpr float kLo = 1.0f - 0x1p-21f, kHi = 1.0f + 0x1p-21f;
  const float q0 = x0 * inv, q1 = x1 * inv;
  uint32_t lo = __builtin_amdgcn_cvt_pk_fp8_f32(q0 * kLo, q1 * kLo, 0, false) & 0xffffu;
  const uint32_t hi = __builtin_amdgcn_cvt_pk_fp8_f32(q0 * kHi, q1 * kHi, 0, false) & 0xffffu;
  if (lo != hi)
    lo = fp8_near(x0, s, lo & 0xff, hi & 0xff) | fp8_near(x1, s, lo >> 8, hi >> 8) << 8;
  return lo;
}

__device__ __forceinline__ uint2 fp8_pack(const float (&v)[8], float s, float inv) {
  return make_uint2(fp8_pair(v[0], v[1], s, inv) | fp8_pair(v[2], v[3], s, inv) << 16,
                    fp8_pair(v[4], v[5], s, inv) | fp8_pair(v[6], v[7], s, inv) << 16);
}

// Scale of a block whose largest magnitude has these bits; `live` where its codes
// are not all 0.  A positive scale is at least 2^-126, so that its reciprocal is
// finite.
__device__ __forceinline__ float fp8_scale(uint32_t top, bool& live) {
  const bool finite = top < kNotFinite;
  live = finite && top > 0;
  const float s = fmaxf(__uint_as_float(top) / kFp8Max, 0x1p-126f);
  return live ? s : finite ? 0.0f : NAN;
}

// Largest over the 8 lanes around a lane, without the LDS that a shuffle takes.
__device__ __forceinline__ uint32_t max8(uint32_t v) {
  auto step = [&](auto ctrl) {
    const uint32_t u = __builtin_amdgcn_update_dpp(0u, v, decltype(ctrl)::value, 0xf, 0xf, true);
    v = u > v ? u : v;
  };
  step(std::integral_constant<int, 0xb1>{});   // lanes 1 apart
  step(std::integral_constant<int, 0x4e>{});   // 2
  step(std::integral_constant<int, 0x141>{});  // 4 (mirrored eights)
  return v;
}

// 8 lanes hold a block of a row, 16 values each: 16 bytes of codes a store.
// WHOLE: K is a multiple of 128, the blocks of all rows follow each other, and no
// thread has to find its row by a division.
// Bound by memory: bf16 [16384, 7168] takes 72 us (352 MB, 4.9 TB/s; with a division
// a block and shuffles through LDS 101), [24576, 2048] 31.5.
template <typename T, bool VEC, bool WHOLE>
__global__ __launch_bounds__(256) void quantize_fp8_kernel(const T* __restrict__ x, long long rows,
                                                           int K, int blocks,
                                                           uint8_t* __restrict__ codes,
                                                           float* __restrict__ scales) {
  const long long total = rows * blocks;
  const int in = threadIdx.x & 7;
  // every lane of a wave takes part in the exchange, also past the end
  for (long long b0 = static_cast<long long>(blockIdx.x) * 32; b0 < total;
       b0 += static_cast<long long>(gridDim.x) * 32) {
    const long long b = b0 + (threadIdx.x >> 3);
    const bool mine = b < total;
    const long long row = WHOLE || !mine ? 0 : b / blocks;
    const int k = WHOLE ? in * 16 : static_cast<int>(mine ? b - row * blocks : 0) * kFp8Block + in * 16;
    const T* from = x + (WHOLE ? b * kFp8Block : row * K) + k;
    float v[2][8] = {};
    uint32_t top = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (mine && (WHOLE || k + 8 * h < K)) {
        uint4 w[sizeof(T) / 2];
        hold8<T, VEC>(from + 8 * h, WHOLE ? 8 : K - k - 8 * h, w);
        values(w, v[h]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) top = max_bits(v[h], top);
    top = max8(top);
    bool live;
    const float s = fp8_scale(top, live);
    if (!mine) continue;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (live) {
      const float inv = 1.0f / s;
      const uint2 a = fp8_pack(v[0], s, inv), c = fp8_pack(v[1], s, inv);
      w = make_uint4(a.x, a.y, c.x, c.y);
    }
    *reinterpret_cast<uint4*>(codes + b * kFp8Block + in * 16) = w;
    if (in == 0) scales[b] = s;
  }
}

// A 128 x 128 block of a weight matrix by a workgroup: 16 threads a row, 16 rows
// at a time, every value in registers between the maximum and the rounding.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void quantize_fp8_weights_kernel(
    const T* __restrict__ w, int N, int K, int kblocks, uint8_t* __restrict__ codes,
    float* __restrict__ scales) {
  const int kb = blockIdx.x, nblocks = (N + kFp8Block - 1) / kFp8Block;
  const long long Kp = static_cast<long long>(kblocks) * kFp8Block;
  const int k = kb * kFp8Block + (threadIdx.x & 15) * 8;
  const int nb = blockIdx.y;
  const long long e = blockIdx.z;
  uint4 h[8][sizeof(T) / 2];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = nb * kFp8Block + i * 16 + (threadIdx.x >> 4);
    float v[8] = {};
    __builtin_memset(h[i], 0, sizeof(h[i]));
    if (n < N && k < K) {
      hold8<T, VEC>(w + (e * N + n) * K + k, K - k, h[i]);
      values(h[i], v);
    }
    top = max_bits(v, top);
  }
  top = row_max<256>(top);
  bool live;
  const float s = fp8_scale(top, live);
  const float inv = 1.0f / s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int n = nb * kFp8Block + i * 16 + (threadIdx.x >> 4);
    if (n >= N) continue;
    float v[8];
    values(h[i], v);
    *reinterpret_cast<uint2*>(codes + (e * N + n) * Kp + k) =
        live ? fp8_pack(v, s, inv) : make_uint2(0u, 0u);
  }
  if (threadIdx.x == 0) scales[(e * nblocks + nb) * kblocks + kb] = s;
}

template <typename T>
hipError_t run_rows(long long rows, int K, const T* x, uint8_t* codes, float* scales,
                    hipStream_t st) {
  const bool vec = K % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
  const int blocks = static_cast<int>(fp8_row(K) / kFp8Block);
  const long long want = (rows * blocks + 31) / 32;
  const unsigned grid = static_cast<unsigned>(want < (1 << 20) ? want : (1 << 20));
  auto go = [&](auto kernel) { kernel<<<grid, 256, 0, st>>>(x, rows, K, blocks, codes, scales); };
  if (vec) K % kFp8Block == 0 ? go(quantize_fp8_kernel<T, true, true>) : go(quantize_fp8_kernel<T, true, false>);
  else K % kFp8Block == 0 ? go(quantize_fp8_kernel<T, false, true>) : go(quantize_fp8_kernel<T, false, false>);
  return hipGetLastError();
}

template <typename T>
hipError_t run_weights(int E, int N, int K, const T* w, uint8_t* codes, float* scales,
                       hipStream_t st) {
  const bool vec = K % 8 == 0 && reinterpret_cast<uintptr_t>(w) % 16 == 0;
  const int blocks = static_cast<int>(fp8_row(K) / kFp8Block);
  const dim3 grid(blocks, (N + kFp8Block - 1) / kFp8Block, E);
  if (vec) quantize_fp8_weights_kernel<T, true><<<grid, 256, 0, st>>>(w, N, K, blocks, codes, scales);
  else quantize_fp8_weights_kernel<T, false><<<grid, 256, 0, st>>>(w, N, K, blocks, codes, scales);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_fp8(long long rows, int K, bool bf16, const void* x, uint8_t* codes,
                               float* scales, hipStream_t st) {
  return bf16 ? run_rows(rows, K, static_cast<const bf16_t*>(x), codes, scales, st)
              : run_rows(rows, K, static_cast<const float*>(x), codes, scales, st);
}

hipError_t launch_quantize_fp8_weights(int E, int N, int K, bool bf16, const void* w,
                                       uint8_t* codes, float* scales, hipStream_t st) {
  return bf16 ? run_weights(E, N, K, static_cast<const bf16_t*>(w), codes, scales, st)
              : run_weights(E, N, K, static_cast<const float*>(w), codes, scales, st);
}

}  // namespace moe
