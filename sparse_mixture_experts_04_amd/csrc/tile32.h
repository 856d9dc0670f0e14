// Tile of a matrix product on the fp32 matrix cores, for operands in any type,
// order, size and alignment.
//
// C[m, n] = sum_k A(m, k) B(n, k) for a tile of 64 R x 64 R by 256 threads: wave
// (wm, wn) owns 32 R x 32 R of it as R x R blocks of v_mfma_f32_32x32x2_f32, whose
// operand is one value a lane (row lane % 32, k = lane / 32).  Steps of 16 values
// of K go through LDS as [k][row], so an operand that is contiguous along K is
// turned round on its way and one that is contiguous along its rows is copied; the
// next step's values are in registers while this one is multiplied.  A wave's two
// LDS reads feed an instruction of 64 cycles, so the matrix units are the bound
// (153 TFLOP/s for a large fp32 product of the library on this card).
#pragma once

#include "common.h"

namespace moe {

constexpr int kT32Threads = 256;
constexpr int kT32K = 16;    // K step
constexpr int kT32Pad = 4;   // floats between LDS rows: the turned writes touch every bank

template <int R>
struct Tile32 {
  static constexpr int N = 64 * R;
  static constexpr int LD = N + kT32Pad;
  static constexpr int PER = N * kT32K / kT32Threads / 4;  // groups of 4 values a thread loads
  struct Lds {
    float a[2][kT32K][LD], b[2][kT32K][LD];
  };
};

// Four consecutive values from p, of which the first n exist (VEC-aligned ones in
// one load).
template <typename T>
__device__ __forceinline__ void load4(const T* p, int n, bool vec, float (&v)[4]) {
  if (vec && n >= 4) {
    if constexpr (sizeof(T) == 4) {
      const float4 f = *reinterpret_cast<const float4*>(p);
      v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      v[0] = __uint_as_float(w.x << 16);
      v[1] = __uint_as_float(w.x & 0xffff0000u);
      v[2] = __uint_as_float(w.y << 16);
      v[3] = __uint_as_float(w.y & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? ActTraits<T>::load(p + i) : 0.0f;
  }
}

// An operand: load(r, k, v) gives 4 values of it, zero where they lie outside.
// ALONG_K: rows r, K values k..k+3; otherwise rows r..r+3 at K value k.
// The product over K values [0, K) is added to acc: lane l's register 4q + e of
// block (i, j) is row 32 (R wm + i) + l % 32, column 32 (R wn + j) + 8q + 4 (l / 32) + e.
template <int R, bool A_ALONG_K, bool B_ALONG_K, class LoadA, class LoadB>
__device__ __forceinline__ void tile32_product(typename Tile32<R>::Lds& lds, int K, LoadA la,
                                               LoadB lb, f32x16_t (&acc)[R][R]) {
  using C = Tile32<R>;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  float ra[C::PER][4], rb[C::PER][4];
  auto fetch = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < C::PER; ++q) {
      if (A_ALONG_K) la(tid / 4 + 64 * q, k0 + tid % 4 * 4, ra[q]);
      else la((tid + 256 * q) % (C::N / 4) * 4, k0 + (tid + 256 * q) / (C::N / 4), ra[q]);
      if (B_ALONG_K) lb(tid / 4 + 64 * q, k0 + tid % 4 * 4, rb[q]);
      else lb((tid + 256 * q) % (C::N / 4) * 4, k0 + (tid + 256 * q) / (C::N / 4), rb[q]);
    }
  };
  auto put = [&](float (&s)[kT32K][C::LD], bool along_k, float (&r)[C::PER][4])
      __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < C::PER; ++q) {
      if (along_k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[tid % 4 * 4 + i][tid / 4 + 64 * q] = r[q][i];
      } else {
        const int at = tid + 256 * q;
        *reinterpret_cast<float4*>(&s[at / (C::N / 4)][at % (C::N / 4) * 4]) =
            make_float4(r[q][0], r[q][1], r[q][2], r[q][3]);
      }
    }
  };
  if (K <= 0) return;
  __syncthreads();  // the tile before is done with the LDS
  fetch(0);
  put(lds.a[0], A_ALONG_K, ra);
  put(lds.b[0], B_ALONG_K, rb);
  __syncthreads();
  for (int k0 = 0, s = 0; k0 < K; k0 += kT32K, s ^= 1) {
    const bool more = k0 + kT32K < K;
    if (more) fetch(k0 + kT32K);
#pragma unroll
    for (int kk = 0; kk < kT32K; kk += 2) {
      float a[R], b[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        a[i] = lds.a[s][kk + (lane >> 5)][32 * (R * wm + i) + (lane & 31)];
        b[i] = lds.b[s][kk + (lane >> 5)][32 * (R * wn + i) + (lane & 31)];
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(b[j], a[i], acc[i][j], 0, 0, 0);
    }
    if (more) {
      put(lds.a[s ^ 1], A_ALONG_K, ra);
      put(lds.b[s ^ 1], B_ALONG_K, rb);
    }
    __syncthreads();
  }
}

}  // namespace moe
