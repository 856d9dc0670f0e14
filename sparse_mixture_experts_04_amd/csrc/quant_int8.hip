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
#include "int8_quant.h"

namespace moe {

// A row in chunks of 8 values, by a workgroup (TPR 256) or a wave (TPR 64);
// it is read twice, the second time from the cache.
template <typename T, int TPR, bool VEC>
__global__ __launch_bounds__(256) void quantize_int8_kernel(const T* __restrict__ x,
                                                            long long rows, int K, int Kp,
                                                            int8_t* __restrict__ codes,
                                                            float* __restrict__ scales) {
  if constexpr (TPR == 256) {
    const long long row = blockIdx.x;
    const float s = quantize_row<T, VEC, 256>(x + row * K, K, Kp, codes + row * Kp);
    if (threadIdx.x == 0) scales[row] = s;
  } else {
    const int i0 = threadIdx.x & 63;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (row >= rows) return;  // whole waves leave
    const T* xr = x + row * K;
    float m = 0.0f;
    bool bad = false;
    const int chunks = (K + 7) / 8;
    for (int c = i0; c < chunks; c += 64) {
      float v[8];
      load8<T, VEC>(xr + c * 8, K - c * 8, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m = fmaxf(m, fabsf(v[i]));
        bad = bad || !(fabsf(v[i]) < INFINITY);
      }
    }
    if (bad) m = INFINITY;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    const bool finite = m < INFINITY;
    const bool live = finite && m > 0.0f;
    const float inv = 127.0f / m;
    int8_t* cr = codes + row * Kp;
    for (int c = i0; c < Kp / 8; c += 64) {
      uint2 w = make_uint2(0u, 0u);
      if (live && c < chunks) {
        float v[8];
        load8<T, VEC>(xr + c * 8, K - c * 8, v);
        w = make_uint2(pack_codes(v, m, inv), pack_codes(v + 4, m, inv));
      }
      *reinterpret_cast<uint2*>(cr + c * 8) = w;
    }
    if (i0 == 0) scales[row] = finite ? m / 127.0f : NAN;
  }
}

template <typename T>
static hipError_t run_quantize(long long rows, int K, const T* x, int8_t* codes, float* scales,
                               hipStream_t st) {
  const int Kp = static_cast<int>(code_row(K));
  const bool vec = K % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0;
  if (rows <= 1024) {  // one workgroup per row: a row's latency counts
    const unsigned grid = static_cast<unsigned>(rows);
    if (vec) quantize_int8_kernel<T, 256, true><<<grid, 256, 0, st>>>(x, rows, K, Kp, codes, scales);
    else quantize_int8_kernel<T, 256, false><<<grid, 256, 0, st>>>(x, rows, K, Kp, codes, scales);
  } else {
    const unsigned grid = static_cast<unsigned>((rows + 3) / 4);
    if (vec) quantize_int8_kernel<T, 64, true><<<grid, 256, 0, st>>>(x, rows, K, Kp, codes, scales);
    else quantize_int8_kernel<T, 64, false><<<grid, 256, 0, st>>>(x, rows, K, Kp, codes, scales);
  }
  return hipGetLastError();
}

hipError_t launch_quantize_int8(long long rows, int K, bool bf16, const void* x, int8_t* codes,
                                float* scales, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  return bf16 ? run_quantize(rows, K, static_cast<const bf16_t*>(x), codes, scales, st)
              : run_quantize(rows, K, static_cast<const float*>(x), codes, scales, st);
}

}  // namespace moe
