// e4m3 products of few results.
//
// A workgroup's 8 waves share K of one 32 x 32 block of y, a block of the scales (128
// codes) at a time: each wave copies its rows' codes into LDS of its own (whole lines of
// 128 bytes by direct loads), reads them as fragments, starts the next block's copy,
// multiplies (codes as bf16: exact, sums in fp32) and joins the block by s_row
// s_column; the waves' sums are added through LDS, in order.  No step waits for another
// wave, and K needs no sums in memory and no second launch: what bounds it is one
// wave's share of K, then the operands' way from the L2, each read once for every 32
// rows of the other.
// (Fragments straight from global memory, 16 bytes of 32 rows a load, come at 16 bytes a
// cycle and compute unit.)  Measured (us, straight from memory / through LDS): 1 x 7168
// by 2048 10.9 / 6.8, 64 x 7168 by 2048 16 / 8.6, 333 x 1111 by 770 7.2 / 5.6, 8 x 2048
// by 7168 5.9 / 4.7; 4000 x 200 by 100, of two steps a wave at most, 4.7 / 5.2.
#include "fp8.h"
#include "tile_kt.h"

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

constexpr int kPiece = 32 * kFp8Block;  // bytes of a block of 32 rows

// Bytes from a row block's first row of this lane's source of load q (8 rows a load,
// 16 bytes a lane; the last row there is stands in for the ones behind it).  Chunk c of
// row r lies in slot c ^ (r % 8), so that 8 rows' reads meet 8 different ones.
__device__ __forceinline__ uint32_t source(int q, int lane, int last, int ld) {
  const int r = q * 8 + (lane >> 3);
  return static_cast<uint32_t>(min(r, last)) * ld + (((lane & 7) ^ (lane >> 3)) << 4);
}

__global__ __launch_bounds__(kThreads, 4) void gemm_fp8_small_kernel(Fp8Args p) {
  union Lds {
    uint8_t stage[kWaves][2][kPiece];  // each wave's rows of a, of w
    float red[kWaves][16][65];
  };
  __shared__ __attribute__((aligned(1024))) Lds lds;
  __shared__ EntryPlan plan;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r32 = lane & 31, half = lane >> 5;
  make_entries<kThreads, 32, kMaxGroups>(p, plan);
  const int nb = p.Kp / kFp8Block, nw = (p.N + kFp8Block - 1) / kFp8Block;
  const int n_tiles = (p.N + 31) / 32;
  const long long total = static_cast<long long>(plan.start[p.E]) * n_tiles;
  const int b0 = nb * wave / kWaves, b1 = nb * (wave + 1) / kWaves;
  const uint32_t at_a = lds_address(lds.stage[wave][0]), at_w = at_a + kPiece;
  typedef const u32x4_t __attribute__((address_space(3)))* lds_piece;

  for (long long it = blockIdx.x; it < total; it += gridDim.x) {
    const int ent = static_cast<int>(it / n_tiles), n0 = static_cast<int>(it % n_tiles) * 32;
    const int g = __builtin_amdgcn_readfirstlane(entry_group(plan, p.E, ent));
    const int m0 = __builtin_amdgcn_readfirstlane((ent - plan.start[g]) * 32);
    const int rows = __builtin_amdgcn_readfirstlane(min(plan.rows[g] - m0, 32));
    const long long row0 = static_cast<long long>(__builtin_amdgcn_readfirstlane(plan.lo[g])) + m0;
    const int cols = min(p.N - n0, 32);
    const uint8_t* a = p.a + row0 * p.Kp;
    const uint8_t* w = p.w + (static_cast<long long>(g) * p.N + n0) * p.Kp;
    const float* as = p.a_scale + (row0 + min(r32, rows - 1)) * nb;
    const float* ws = p.w_scale + (static_cast<long long>(g) * nw + n0 / kFp8Block) * nb;
    uint32_t from_a[4], from_w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      from_a[q] = source(q, lane, rows - 1, p.Kp);
      from_w[q] = source(q, lane, cols - 1, p.Kp);
    }
    float sa = 0.0f, sw = 0.0f;
    // rows of which a load would copy none are left out: no result reads them
    auto copy = [&](int b) __attribute__((always_inline)) {
      sa = as[b];
      sw = ws[b];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (8 * q < rows)
          dma16_at(reinterpret_cast<const bf16_t*>(a + b * kFp8Block), from_a[q], at_a + q * 1024);
        if (8 * q < cols)
          dma16_at(reinterpret_cast<const bf16_t*>(w + b * kFp8Block), from_w[q], at_w + q * 1024);
      }
    };
    __syncthreads();  // the item before is done with red
    f32x16_t acc = {};
    if (b0 < b1) copy(b0);
    for (int b = b0; b < b1; ++b) {
      const float f = sa * sw;
      u32x4_t ka[4], kw[4];
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the copy is there
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t o = r32 * kFp8Block + (((2 * j + half) ^ (r32 & 7)) << 4);
        ka[j] = *(lds_piece)(at_a + o);
        kw[j] = *(lds_piece)(at_w + o);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next copy lands
      __builtin_amdgcn_sched_barrier(0);
      if (b + 1 < b1) copy(b + 1);
      f32x16_t s = {};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wide8(kw[j][2 * q], kw[j][2 * q + 1]),
                                                      wide8(ka[j][2 * q], ka[j][2 * q + 1]), s, 0,
                                                      0, 0);
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[r] = fmaf(s[r], f, acc[r]);
    }
    __syncthreads();  // red lies where the rows were
#pragma unroll
    for (int r = 0; r < 16; ++r) lds.red[wave][r][lane] = acc[r];
    __syncthreads();
    // register 4 q + e of lane l: row l % 32, column 8 q + 4 (l / 32) + e
    const int c = tid & 31, reg = 4 * (c >> 3) + (c & 3), from = (c & 4) * 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (tid >> 5) + 16 * i;
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k) v += lds.red[k][reg][from + r];
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
