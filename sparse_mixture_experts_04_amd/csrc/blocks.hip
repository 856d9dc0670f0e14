// Products in blocks of 32 rows: e4m3 with block scales and the gated block in bf16, for
// few results or few rows a group, and the gated block in fp32.
//
// A workgroup's 8 waves share K of one block of 32 rows x 32 weight rows (gated: 16 of Wg
// and the same 16 of Wu), a step of 128 bytes of a row at a time: each wave copies its
// rows' step into LDS of its own (whole lines by direct loads), reads it as fragments,
// starts the next step's copy and multiplies; the waves' sums are added through LDS, in
// order.  No step waits for another wave, and K needs no sums in memory and no second
// launch: what bounds it is one wave's share of K, then the operands' way from the L2,
// each read once for every 32 rows of the other.
// e4m3 codes are multiplied as bf16 (exact, sums in fp32); a step is one block of the
// scales and joins the sums by s_row s_column.
// (Fragments straight from global memory, 16 bytes of 32 rows a load, come at 16 bytes a
// cycle and compute unit.)  Measured (us, e4m3, straight from memory / through LDS): 1 x
// 7168 by 2048 10.9 / 6.8, 64 x 7168 by 2048 16 / 8.6, 333 x 1111 by 770 7.2 / 5.6, 8 x
// 2048 by 7168 5.9 / 4.7; 4000 x 200 by 100, of two steps a wave at most, 4.7 / 5.2.
// Few rows of many weights read them at 5 to 6.6 TB/s: 8 x 4096 by 65536 in e4m3 41 us,
// gated, 384 rows over 256 groups of d=2048 F=768, bf16 205 us.  fp32 is bound by its
// matrix instruction from some 500 rows on (M=2048 d=2048 F=768 134 us, 96 TFLOP/s).
#include <algorithm>
#include <cmath>

#include "blocks.h"
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

constexpr int kStep = 128;          // bytes of a row per step
constexpr int kPiece = 32 * kStep;  // of 32 rows

// Chunk of 16 bytes of a step that this lane copies (of row lane / 8 of each load's 8).
// Chunk c of row r lies in slot c ^ (r % 8), so that 8 rows' reads meet 8 different ones.
__device__ __forceinline__ int my_chunk(int lane) { return (lane & 7) ^ (lane >> 3); }

template <BlockKind KIND>
__global__ __launch_bounds__(kThreads, 4) void blocks_kernel(BlockArgs p) {
  constexpr bool GATED = KIND != BlockKind::kFp8;
  constexpr int SIZE = KIND == BlockKind::kFp8 ? 1 : KIND == BlockKind::kGatedBf16 ? 2 : 4;
  constexpr int NOUT = GATED ? 16 : 32;
  union Lds {
    uint8_t stage[kWaves][2][kPiece];  // each wave's rows of a, of the weights
    float red[kWaves][16][65];
  };
  __shared__ __attribute__((aligned(1024))) Lds lds;
  __shared__ EntryPlan plan;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r32 = lane & 31, half = lane >> 5, r16 = lane & 15, quad = lane >> 4;
  make_entries<kThreads, 32, kMaxGroups>(p, plan);
  const int ld = p.K * SIZE;  // bytes of a row
  const int nk = (ld + kStep - 1) / kStep, nw = (p.N + 127) / 128;
  const int n_tiles = (p.N + NOUT - 1) / NOUT;
  const long long total = static_cast<long long>(plan.start[p.E]) * n_tiles;
  const int b0 = static_cast<int>(static_cast<long long>(nk) * wave / kWaves);
  const int b1 = static_cast<int>(static_cast<long long>(nk) * (wave + 1) / kWaves);
  const uint32_t at_a = lds_address(lds.stage[wave][0]), at_w = at_a + kPiece;
  typedef const u32x4_t __attribute__((address_space(3)))* lds_piece;
  const int chunk = my_chunk(lane);

  for (long long it = blockIdx.x; it < total; it += gridDim.x) {
    const int ent = static_cast<int>(it / n_tiles), n0 = static_cast<int>(it % n_tiles) * NOUT;
    const int g = __builtin_amdgcn_readfirstlane(entry_group(plan, p.E, ent));
    const int m0 = __builtin_amdgcn_readfirstlane((ent - plan.start[g]) * 32);
    const int rows = __builtin_amdgcn_readfirstlane(min(plan.rows[g] - m0, 32));
    const long long row0 = static_cast<long long>(__builtin_amdgcn_readfirstlane(plan.lo[g])) + m0;
    const int cols = min(p.N - n0, NOUT);
    const char* a = static_cast<const char*>(p.a) + row0 * ld;
    const long long wat = (static_cast<long long>(g) * p.N + n0) * ld;
    const float* as = GATED ? nullptr : p.a_scale + (row0 + min(r32, rows - 1)) * nk;
    const float* ws = GATED ? nullptr : p.w_scale + (static_cast<long long>(g) * nw + n0 / 128) * nk;
    // bytes from the first row of this lane's source of load q; the last row there is
    // stands in for the ones behind it
    uint32_t from_a[4], from_w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = q * 8 + (lane >> 3), rw = GATED ? r & 15 : r;
      from_a[q] = static_cast<uint32_t>(min(r, rows - 1)) * ld + chunk * 16;
      from_w[q] = static_cast<uint32_t>(min(rw, cols - 1)) * ld + chunk * 16;
    }
    float sa = 0.0f, sw = 0.0f;
    // rows of which a load would copy none are left out: no result reads them
    auto copy = [&](int b) __attribute__((always_inline)) {
      if constexpr (!GATED) {
        sa = as[b];
        sw = ws[b];
      }
      // what lies behind the end of a row is another row's, or nobody's: zeros
      const bool whole = !GATED || (b + 1) * kStep <= ld, in = b * kStep + chunk * 16 < ld;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const char* w = static_cast<const char*>(GATED && q >= 2 ? p.w1 : p.w0) + wat;
        auto one = [&](const char* from, uint32_t off, uint32_t to) __attribute__((always_inline)) {
          from += b * kStep;
          if (whole) dma16_at(reinterpret_cast<const bf16_t*>(from), off, to + q * 1024);
          else dma16_to(in ? reinterpret_cast<const bf16_t*>(from + off)
                           : reinterpret_cast<const bf16_t*>(&kTileZeros), to + q * 1024);
        };
        if (8 * q < rows) one(a, from_a[q], at_a);
        if (8 * (GATED ? q & 1 : q) < cols) one(w, from_w[q], at_w);
      }
    };
    __syncthreads();  // the item before is done with red
    f32x16_t acc = {};
    // fp32, up to 16 rows: instructions of 16 x 16 do in half the time
    const bool few = KIND == BlockKind::kGatedF32 && rows <= 16;
    f32x4_t acc16[2] = {};
    if (b0 < b1) copy(b0);
    for (int b = b0; b < b1; ++b) {
      const float f = sa * sw;
      u32x4_t ka[4], kw[4];
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the copy is there
      __builtin_amdgcn_sched_barrier(0);
      if (few) {  // lane: row lane % 16 of a, of Wg and of Wu, chunks lane / 16 and 4 on
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t o = r16 * kStep + (((4 * j + quad) ^ (r16 & 7)) << 4);
          ka[j] = *(lds_piece)(at_a + o);
          kw[j] = *(lds_piece)(at_w + o);
          kw[2 + j] = *(lds_piece)(at_w + 16 * kStep + o);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t o = r32 * kStep + (((2 * j + half) ^ (r32 & 7)) << 4);
          ka[j] = *(lds_piece)(at_a + o);
          kw[j] = *(lds_piece)(at_w + o);
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next copy lands
      __builtin_amdgcn_sched_barrier(0);
      if (b + 1 < b1) copy(b + 1);
      if constexpr (KIND == BlockKind::kFp8) {
        f32x16_t s = {};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wide8(kw[j][2 * q], kw[j][2 * q + 1]),
                                                        wide8(ka[j][2 * q], ka[j][2 * q + 1]), s,
                                                        0, 0, 0);
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[r] = fmaf(s[r], f, acc[r]);
      } else if (few) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int t = 0; t < 2; ++t)
              acc16[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(kw[2 * t + j][e]),
                                                              __uint_as_float(ka[j][e]), acc16[t],
                                                              0, 0, 0);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (SIZE == 2) {
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, kw[j]),
                                                          __builtin_bit_cast(bf16x8_t, ka[j]),
                                                          acc, 0, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(kw[j][e]),
                                                         __uint_as_float(ka[j][e]), acc, 0, 0, 0);
          }
        }
      }
    }
    __syncthreads();  // red lies where the rows were
    if (few) {  // register e of lane l, tile t: row l % 16, weight row 16 t + 4 (l / 16) + e
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          lds.red[wave][4 * (2 * t + (quad >> 1)) + e][(quad & 1) * 32 + r16] = acc16[t][e];
    } else {
#pragma unroll
      for (int r = 0; r < 16; ++r) lds.red[wave][r][lane] = acc[r];
    }
    __syncthreads();
    // register 4 q + e of lane l: row l % 32, weight row 8 q + 4 (l / 32) + e
    auto sum = [&](int row, int c) __attribute__((always_inline)) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < kWaves; ++k)
        v += lds.red[k][4 * (c >> 3) + (c & 3)][(c & 4) * 8 + row];
      return v;
    };
    constexpr int kSpan = kThreads / NOUT;  // rows a turn
#pragma unroll
    for (int i = 0; i < 32 / kSpan; ++i) {
      const int r = tid / NOUT + kSpan * i, c = tid % NOUT;
      const float v = sum(r, c), u = GATED ? sum(r, c + 16) : 0.0f;
      if (r >= rows || c >= cols) continue;
      const size_t row = static_cast<size_t>(row0 + r);
      const float y = GATED ? v * (1.0f / (1.0f + expf(-v))) * u : v;
      if (!GATED || p.out) {
        if (GATED ? SIZE == 2 : p.out_bf16) static_cast<bf16_t*>(p.out)[row * p.N + n0 + c] = f32_to_bf16(y);
        else static_cast<float*>(p.out)[row * p.N + n0 + c] = y;
      }
      if (GATED && p.pre) {
        p.pre[row * 2 * p.N + n0 + c] = v;
        p.pre[row * 2 * p.N + p.N + n0 + c] = u;
      }
    }
  }
}

}  // namespace

// Blocks there may be: an entry for each 32 rows of a group, one at least for each group
// with rows.
static double most_blocks(int M, int N, int E, bool gated) {
  return (std::ceil(M / 32.0) + (E > 1 ? std::min(M, E) : 0)) * std::ceil(N / (gated ? 16.0 : 32.0));
}

double blocks_time(int M, int N, long long row_bytes, int E, bool gated) {
  return 3.0 + std::max(0.5, most_blocks(M, N, E, gated) / 512) *
                   (2.3 + 0.18 * std::ceil(row_bytes / 128.0));
}

hipError_t launch_blocks(const BlockArgs& a, BlockKind kind, hipStream_t st) {
  const unsigned grid =
      static_cast<unsigned>(std::min(1024.0, most_blocks(a.M, a.N, a.E, kind != BlockKind::kFp8)));
  if (kind == BlockKind::kFp8) blocks_kernel<BlockKind::kFp8><<<grid, kThreads, 0, st>>>(a);
  else if (kind == BlockKind::kGatedBf16) blocks_kernel<BlockKind::kGatedBf16><<<grid, kThreads, 0, st>>>(a);
  else blocks_kernel<BlockKind::kGatedF32><<<grid, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
