// e4m3 products of few results.
//
// A workgroup's 8 waves share K of one 32 x 32 block of y, a block of the scales (128
// codes) at a time: each wave loads its rows' codes from global memory straight into
// registers (a lane 16 bytes of row lane % 32, two blocks in flight), multiplies them
// as bf16 (exact, sums in fp32) and joins the block by s_row s_column; the waves' sums
// are added through LDS, in order.  No step waits for another wave, and K needs no
// sums in memory and no second launch: what bounds it is one wave's share of K, then
// the operands' way from the L2, each read once for every 32 rows of the other.  M=333
// K=1111 N=770 takes 7.3 us (16 waves: 8.9; 128-row tiles 16.7), M=8 K=2048 N=7168 5.9.
#include "fp8.h"

namespace moe {

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8, kThreads = 64 * kWaves;


// Eight codes as bf16, which holds every e4m3 value.
__device__ __forceinline__ bf16x8_t wide8(uint32_t lo, uint32_t hi) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  union {
    bf16x2_t pair[4];
    bf16x8_t all;
  } u;
  u.pair[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  u.pair[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  u.pair[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  u.pair[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return u.all;
}

// A lane's codes of a block of both operands, and the block's scale.
struct Block {
  u32x4_t a[4], w[4];
  float sa, sw;
};

__global__ __launch_bounds__(kThreads, 4) void gemm_fp8_small_kernel(Fp8Args p) {
  __shared__ float red[kWaves][16][65];
  __shared__ EntryPlan plan;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r32 = lane & 31, half = lane >> 5;
  make_entries<kThreads, 32, kMaxGroups>(p, plan);
  const int nb = p.Kp / kFp8Block, nw = (p.N + kFp8Block - 1) / kFp8Block;
  const int n_tiles = (p.N + 31) / 32;
  const long long total = static_cast<long long>(plan.start[p.E]) * n_tiles;
  const int b0 = nb * wave / kWaves, b1 = nb * (wave + 1) / kWaves;

  for (long long it = blockIdx.x; it < total; it += gridDim.x) {
    const int ent = static_cast<int>(it / n_tiles), n0 = static_cast<int>(it % n_tiles) * 32;
    const int g = entry_group(plan, p.E, ent);
    const int m0 = (ent - plan.start[g]) * 32, rows = min(plan.rows[g] - m0, 32);
    const long long row0 = static_cast<long long>(plan.lo[g]) + m0;
    const long long row = row0 + min(r32, rows - 1);
    const uint8_t* a = p.a + row * p.Kp + 16 * half;
    const uint8_t* w =
        p.w + (static_cast<long long>(g) * p.N + min(n0 + r32, p.N - 1)) * p.Kp + 16 * half;
    const float* as = p.a_scale + row * nb;
    const float* ws = p.w_scale + (static_cast<long long>(g) * nw + n0 / kFp8Block) * nb;
    auto load = [&](int b, Block& k) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        k.a[j] = *reinterpret_cast<const u32x4_t*>(a + b * kFp8Block + 32 * j);
        k.w[j] = *reinterpret_cast<const u32x4_t*>(w + b * kFp8Block + 32 * j);
      }
      k.sa = as[b];
      k.sw = ws[b];
    };
    f32x16_t acc = {};
    auto multiply = [&](const Block& k) __attribute__((always_inline)) {
      f32x16_t s = {};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wide8(k.w[j][2 * q], k.w[j][2 * q + 1]),
                                                      wide8(k.a[j][2 * q], k.a[j][2 * q + 1]), s,
                                                      0, 0, 0);
      const float f = k.sa * k.sw;
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[r] = fmaf(s[r], f, acc[r]);
    };
    int b = b0;
    for (; b + 1 < b1; b += 2) {
      Block k[2];
      load(b, k[0]);
      load(b + 1, k[1]);
      multiply(k[0]);
      multiply(k[1]);
    }
    if (b < b1) {
      Block k;
      load(b, k);
      multiply(k);
    }
    __syncthreads();  // the item before is done with red
#pragma unroll
    for (int r = 0; r < 16; ++r) red[wave][r][lane] = acc[r];
    __syncthreads();
    // register 4 q + e of lane l: row l % 32, column 8 q + 4 (l / 32) + e
    const int c = tid & 31, reg = 4 * (c >> 3) + (c & 3), from = (c & 4) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (tid >> 5) + 16 * i;
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) v += red[k][reg][from + r];
      if (r < rows && n0 + c < p.N) {
        const size_t at = static_cast<size_t>(row0 + r) * p.N + n0 + c;
        if (p.out_bf16) static_cast<bf16_t*>(p.out)[at] = f32_to_bf16(v);
        else static_cast<float*>(p.out)[at] = v;
      }
    }
  }
}

}  // namespace

hipError_t launch_gemm_fp8_small(const Fp8Args& a, hipStream_t st) {
  gemm_fp8_small_kernel<<<1024, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
