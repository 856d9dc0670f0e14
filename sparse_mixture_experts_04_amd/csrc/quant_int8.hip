// Rows of values to 8-bit integers with one scale per row.
//
//   s = max |x| / 127          q_k = round(127 x_k / max |x|), ties to even
//
// used per token for activations and per output channel for weights.  The
// codes are those of exact arithmetic: a fp32 quotient decides unless it lies
// within 1e-4 of a rounding border (its error is below 2e-5 for |q| <= 127);
// there the quotient is taken in fp64, whose error (2^-53 of it) is smaller
// than the distance of any quotient of two fp32 values to a border it is not
// on.  A row of zeros gets scale 0; a row holding a NaN or an infinity gets
// codes 0 and scale NaN, so that only its own products become NaN.
//
// Bound by memory: 131072 x 2048 fp32 in 240 us (5.6 TB/s), 16384 x 7168 bf16 in 78
// (4.5 TB/s), where the rounding's 6 or so instructions a value keep the vector
// units as busy; one row of 2048 2.4 us, latency.  Rows that do not start on 16
// bytes are read by 16-byte loads all the same (4291 x 1449 fp32 8.7 us, value by
// value 17.2).
#include "int8_quant.h"

namespace moe {

// A row of up to 512 NC values by a wave, four rows a workgroup: every chunk of 8
// values a lane has is loaded before the first is used and stays in registers,
// so the row is read once.
template <typename T, int NC, bool VEC>
__global__ __launch_bounds__(256) void quantize_int8_wave_kernel(const T* __restrict__ x,
                                                                 long long rows, int K, int Kp,
                                                                 int8_t* __restrict__ codes,
                                                                 float* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;  // whole waves leave
  const T* xr = x + row * K;
  const int chunks = (K + 7) / 8;
  uint4 held[NC][sizeof(T) / 2];  // as they were read
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = lane + 64 * j;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) held[j][i] = make_uint4(0u, 0u, 0u, 0u);
    if (c < chunks) hold8<T, VEC>(xr + c * 8, K - c * 8, held[j]);
  }
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    float v[8];
    values(held[j], v);
    top = max_bits(v, top);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t u = __shfl_xor(top, o);
    top = u > top ? u : top;
  }
  const float m = __uint_as_float(top);
  const bool finite = top < kNotFinite;
  const bool live = finite && top > 0;
  const float inv = 127.0f / m;
  int8_t* cr = codes + row * Kp;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = lane + 64 * j;
    if (c >= Kp / 8) continue;
    float v[8];
    values(held[j], v);
    *reinterpret_cast<uint2*>(cr + c * 8) = live ? pack_codes(v, m, inv) : make_uint2(0u, 0u);
  }
  if (lane == 0) scales[row] = finite ? m / 127.0f : NAN;
}

// A row by a workgroup, read twice, the second time from the cache: few rows,
// where one row's latency counts, and rows too long for the kernel above.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void quantize_int8_kernel(const T* __restrict__ x, int K, int Kp,
                                                            int8_t* __restrict__ codes,
                                                            float* __restrict__ scales) {
  const long long row = blockIdx.x;
  const float s = quantize_row<T, VEC, 256>(x + row * K, K, Kp, codes + row * Kp);
  if (threadIdx.x == 0) scales[row] = s;
}

template <typename T, int NC>
static void run_wave(long long rows, int K, bool vec, const T* x, int8_t* codes, float* scales,
                     hipStream_t st) {
  const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
  const int Kp = static_cast<int>(code_row(K));
  if (vec) quantize_int8_wave_kernel<T, NC, true><<<grid, 256, 0, st>>>(x, rows, K, Kp, codes, scales);
  else quantize_int8_wave_kernel<T, NC, false><<<grid, 256, 0, st>>>(x, rows, K, Kp, codes, scales);
}

template <typename T>
static hipError_t run_quantize(long long rows, int K, const T* x, int8_t* codes, float* scales,
                               hipStream_t st) {
  const bool vec = K % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
  const int Kp = static_cast<int>(code_row(K));
  if (rows <= 1024 || Kp > 8192) {
    const unsigned grid = static_cast<unsigned>(rows);
    if (vec) quantize_int8_kernel<T, true><<<grid, 256, 0, st>>>(x, K, Kp, codes, scales);
    else quantize_int8_kernel<T, false><<<grid, 256, 0, st>>>(x, K, Kp, codes, scales);
  } else if (Kp <= 1024) {
    run_wave<T, 2>(rows, K, vec, x, codes, scales, st);
  } else if (Kp <= 2048) {
    run_wave<T, 4>(rows, K, vec, x, codes, scales, st);
  } else if (Kp <= 4096) {
    run_wave<T, 8>(rows, K, vec, x, codes, scales, st);
  } else {
    run_wave<T, 16>(rows, K, vec, x, codes, scales, st);
  }
  return hipGetLastError();
}

hipError_t launch_quantize_int8(long long rows, int K, bool bf16, const void* x, int8_t* codes,
                                float* scales, hipStream_t st) {
  // a launch takes fewer than 2^32 threads, and a row up to 256 of them
  constexpr long long kRowsPerLaunch = 1LL << 23;
  const long long Kp = code_row(K);
  for (long long r = 0; r < rows; r += kRowsPerLaunch) {
    const long long n = rows - r < kRowsPerLaunch ? rows - r : kRowsPerLaunch;
    const hipError_t e =
        bf16 ? run_quantize(n, K, static_cast<const bf16_t*>(x) + r * K, codes + r * Kp,
                            scales + r, st)
             : run_quantize(n, K, static_cast<const float*>(x) + r * K, codes + r * Kp,
                            scales + r, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
