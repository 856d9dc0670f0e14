// Rounding of values to 8-bit codes (see quant_int8.hip for the rule).
#pragma once

#include "int8.h"

namespace moe {

__device__ __forceinline__ int quant_code(float x, float amax, float inv) {
  const float t = x * inv;
  float r = rintf(t);
  // !(..) also catches an inv that overflowed (amax below 127 / FLT_MAX)
  if (!(fabsf(t - r) < 0.4999f))
    r = static_cast<float>(rint(127.0 * static_cast<double>(x) / static_cast<double>(amax)));
  return static_cast<int>(r);
}

__device__ __forceinline__ uint32_t pack_codes(const float* v, float amax, float inv) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= (static_cast<uint32_t>(quant_code(v[i], amax, inv)) & 0xffu) << (8 * i);
  return w;
}

// 8 values from p; `n` of them exist (VEC: all, and p is 16-byte aligned).
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
  if constexpr (VEC && sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else if constexpr (VEC) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? ActTraits<T>::load(p + i) : 0.0f;
  }
}

// max |x| of a row held by the NT threads of a workgroup as their own maxima
// (`bad`: a value was not finite): the maximum, or infinity.
template <int NT>
__device__ __forceinline__ float row_amax(float m, bool bad) {
  __shared__ float sm[NT / 64];
  if (bad) m = INFINITY;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
  __syncthreads();
  m = sm[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) m = fmaxf(m, sm[w]);
  return m;
}

// One row of K values by the NT threads of a workgroup, in chunks of 8: load(c,
// n, v) gives chunk c (n of its values exist), store(c, w) takes its codes.
// Returns the scale.
template <int NT, class Load, class Store>
__device__ __forceinline__ float quantize_row(int K, int Kp, Load load, Store store) {
  const int chunks = (K + 7) / 8;
  float m = 0.0f;
  bool bad = false;
  for (int c = threadIdx.x; c < chunks; c += NT) {
    float v[8];
    load(c, K - c * 8, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m = fmaxf(m, fabsf(v[i]));
      bad = bad || !(fabsf(v[i]) < INFINITY);
    }
  }
  m = row_amax<NT>(m, bad);
  const bool finite = m < INFINITY;
  const bool live = finite && m > 0.0f;
  const float inv = 127.0f / m;
  for (int c = threadIdx.x; c < Kp / 8; c += NT) {
    uint2 w = make_uint2(0u, 0u);
    if (live && c < chunks) {
      float v[8];
      load(c, K - c * 8, v);
      w = make_uint2(pack_codes(v, m, inv), pack_codes(v + 4, m, inv));
    }
    store(c, w);
  }
  return finite ? m / 127.0f : NAN;
}

// A row in memory.
template <typename T, bool VEC, int NT>
__device__ __forceinline__ float quantize_row(const T* xr, int K, int Kp, int8_t* cr) {
  return quantize_row<NT>(
      K, Kp, [&](int c, int n, float (&v)[8]) { load8<T, VEC>(xr + c * 8, n, v); },
      [&](int c, uint2 w) { *reinterpret_cast<uint2*>(cr + c * 8) = w; });
}

}  // namespace moe
