// Rounding of values to 8-bit codes (see quant_int8.hip for the rule).
#pragma once

#include "int8.h"

namespace moe {

// Codes of 8 values, 4 to a word.  x * inv + 1.5 * 2^23 rounds the quotient to
// the nearest integer, ties to even, and leaves it in the sum's low bits; the
// remainder tells whether it lay near a border.
__device__ __forceinline__ uint2 pack_codes(const float (&v)[8], float amax, float inv) {
  constexpr float kMagic = 12582912.0f;
  uint32_t bits[8];
  float near = inv < INFINITY ? 0.0f : 1.0f;  // inv overflows for amax below 127 / FLT_MAX
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = fmaf(v[i], inv, kMagic);
    near = fmaxf(near, fabsf(fmaf(v[i], inv, kMagic - f)));
    bits[i] = __float_as_uint(f);
  }
  if (near >= 0.4999f) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      bits[i] = static_cast<uint32_t>(static_cast<int>(
          rint(127.0 * static_cast<double>(v[i]) / static_cast<double>(amax))));
  }
  // the low bytes of four words
  auto four = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u),
                                 __builtin_amdgcn_perm(b, a, 0x0c0c0400u), 0x05040100u);
  };
  return make_uint2(four(bits[0], bits[1], bits[2], bits[3]),
                    four(bits[4], bits[5], bits[6], bits[7]));
}

// Largest magnitude of 8 values as bits: an infinity or a NaN counts as more than
// every finite value (0x7f800000 on).
__device__ __forceinline__ uint32_t max_bits(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
    m = u > m ? u : m;
  }
  return m;
}
constexpr uint32_t kNotFinite = 0x7f800000u;

// 8 values from p as they lie in memory, `n` of them in the row (VEC: all, and p is
// 16-byte aligned; otherwise aligned to a value, which a wide load takes too).
template <typename T, bool VEC>
__device__ __forceinline__ void hold8(const T* p, int n, uint4 (&h)[sizeof(T) / 2]) {
  if (VEC) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) h[i] = reinterpret_cast<const uint4*>(p)[i];
  } else if (n >= 8) {
    __builtin_memcpy(h, p, sizeof(h));
  } else {
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : T{0};
    __builtin_memcpy(h, v, sizeof(h));
  }
}
__device__ __forceinline__ void values(const uint4 (&h)[1], float (&v)[8]) {
  const uint32_t w[4] = {h[0].x, h[0].y, h[0].z, h[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void values(const uint4 (&h)[2], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {h[i].x, h[i].y, h[i].z, h[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * i + j] = __uint_as_float(w[j]);
  }
}

// Largest of the maxima that the NT threads of a workgroup hold.
template <int NT>
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
  __shared__ uint32_t sm[NT / 64];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t u = __shfl_xor(m, o);
    m = u > m ? u : m;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
  __syncthreads();
  m = sm[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) m = sm[w] > m ? sm[w] : m;
  return m;
}

// One row of K values by the NT threads of a workgroup, in chunks of 8: load(c,
// n, v) gives chunk c (n of its values exist), store(c, w) takes its codes.
// Returns the scale.
template <int NT, class Load, class Store>
__device__ __forceinline__ float quantize_row(int K, int Kp, Load load, Store store) {
  const int chunks = (K + 7) / 8;
  uint32_t top = 0;
  for (int c = threadIdx.x; c < chunks; c += NT) {
    float v[8];
    load(c, K - c * 8, v);
    top = max_bits(v, top);
  }
  top = row_max<NT>(top);
  const float m = __uint_as_float(top);
  const bool finite = top < kNotFinite;
  const bool live = finite && top > 0;
  const float inv = 127.0f / m;
  for (int c = threadIdx.x; c < Kp / 8; c += NT) {
    uint2 w = make_uint2(0u, 0u);
    if (live && c < chunks) {
      float v[8];
      load(c, K - c * 8, v);
      w = pack_codes(v, m, inv);
    }
    store(c, w);
  }
  return finite ? m / 127.0f : NAN;
}

// A row in memory.
template <typename T, bool VEC, int NT>
__device__ __forceinline__ float quantize_row(const T* xr, int K, int Kp, int8_t* cr) {
  return quantize_row<NT>(
      K, Kp,
      [&](int c, int n, float (&v)[8]) {
        uint4 h[sizeof(T) / 2];
        hold8<T, VEC>(xr + c * 8, n, h);
        values(h, v);
      },
      [&](int c, uint2 w) { *reinterpret_cast<uint2*>(cr + c * 8) = w; });
}

}  // namespace moe
