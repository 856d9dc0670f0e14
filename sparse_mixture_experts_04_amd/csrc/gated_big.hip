// Gated block and its gradients for large batches in bf16: tiles of 128 or 256 rows x
// 256 columns on the bf16 matrix cores (big_tile.h, tile_kt.h).
//
// Forward: 256 weight rows of a tile are, per 64, 32 rows of Wg and the same 32 of
// Wu; silu and the product are taken from the sums in registers.  dx: dau's rows, K
// over its 2F columns; the weights are contiguous along their rows d.  dW: rows are
// columns of dau (F of dWg, then of dWu), K the rows of the group, both operands
// contiguous along their rows.
// Rows of x, the matrices, dau and the results start on 16 bytes (d and F are
// multiples of 8).
#include <algorithm>
#include <cmath>

#include "gated.h"
#include "tile_kt.h"

namespace moe {

namespace {

using Big = BigShape<256, 32, 3, 6>;
using Mid = BigShape<128, 64, 3, 3>;

// Whether a gradient's product takes 256-row tiles: they use what they load twice as
// often, and need as many of them as there are compute units to keep busy.  (The
// forward pass is faster in 128-row tiles at every size measured, M=8192 d=7168
// F=2048 393 against 406 us, 24576 rows over 128 experts 244 against 274.)
// Measured (us, 256 / 128 rows):
//   dx  M=8192 d=7168 F=2048  424 / 451   dW  383 / 479
//       1024                   70 / 56         63 / 80
//       24576 rows, 128 experts, d=2048 F=768  243 / 255   dW  366 / 424
//       M=4096 d=2048 F=768    35 / 30         64 / 48
bool large_tiles(const GatedArgs& a, GatedPart part) {
  const double rows = part == GatedPart::kDw ? 2.0 * a.F * a.E : a.M;
  const long long mean = part == GatedPart::kDw ? a.F : a.M / a.E;
  return mean >= 160 && rows * a.d / 65536.0 >= 224.0;
}

// SPLIT: K is cut into p.splits slices, each an item of its own, whose fp32 sums go to
// slice s of p.part [splits, rows, columns] (forward [M, 2F], dx [M, d], dW [2F, d]).
template <class C, GatedPart PART, bool SPLIT = false>
__global__ __launch_bounds__(512, 1) void gated_big_kernel(GatedArgs p) {
  constexpr bool FWD = PART == GatedPart::kForward, DW = PART == GatedPart::kDw;
  constexpr bool TA = DW, TB = !FWD;
  constexpr int NOUT = FWD ? C::NB / 2 : C::NB;
  __shared__ __attribute__((aligned(1024))) bf16_t lds[C::LDS_ELEMS];
  __shared__ EntryPlan plan;
  bf16_t* sA[C::NSA];
  bf16_t* sB[C::NSB];
#pragma unroll
  for (int i = 0; i < C::NSA; ++i) sA[i] = lds + i * C::A_STAGE;
#pragma unroll
  for (int i = 0; i < C::NSB; ++i) sB[i] = lds + C::NSA * C::A_STAGE + i * C::B_STAGE;
  static_assert(C::MT * NOUT <= C::LDS_ELEMS, "output tile");
  static_assert(!SPLIT || C::MT * C::NB * 2 <= C::LDS_ELEMS, "fp32 tile");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  make_entries<C::THREADS, C::MT, kMaxGroups>(p, plan);
  const int d = p.d, F = p.F, F2 = 2 * F;
  const int ncols = FWD ? F : d;  // columns of the result
  const int n_tiles = (ncols + NOUT - 1) / NOUT;
  const int m_tiles = (F + C::MT - 1) / C::MT;  // kDw: row tiles of a matrix
  const int splits = SPLIT ? p.splits : 1;
  const long long total = (DW ? static_cast<long long>(p.E) * 2 * m_tiles
                              : static_cast<long long>(plan.start[p.E])) * n_tiles * splits;
  const int xcd = blockIdx.x % kXcds;
  const bf16_t* x = static_cast<const bf16_t*>(p.x);
  const bf16_t* dau = static_cast<const bf16_t*>(p.dau);
  const int lrow = lane / C::CPR;

  const long long chunk = (total + kXcds - 1) / kXcds;
  for (long long mine = blockIdx.x / kXcds;; mine += gridDim.x / kXcds) {
    const long long turn = xcd * chunk + mine;
    if (mine >= chunk || turn >= total) break;
    __syncthreads();  // the item before is done with the LDS
    const long long it = SPLIT ? turn / splits : turn;
    const int slice = SPLIT ? static_cast<int>(turn % splits) : 0;
    int g, m0, rows, nt;
    bool half = false;
    if constexpr (DW) {
      // column tiles outer, row tiles (of dWg, then dWu) inner
      const int per = 2 * m_tiles * n_tiles, at = static_cast<int>(it % per);
      g = static_cast<int>(it / per);
      nt = at / (2 * m_tiles);
      half = at % (2 * m_tiles) >= m_tiles;
      m0 = (at % (2 * m_tiles) - (half ? m_tiles : 0)) * C::MT;
      rows = min(F - m0, C::MT);
    } else {
      g = entry_group(plan, p.E, static_cast<int>(it / n_tiles));
      const Item item = place_item(it, plan.start, g, n_tiles, C::MT, plan.rows[g], true);
      m0 = item.m0;
      rows = item.rows;
      nt = item.n;
    }
    // (uniform, but read from LDS: tell the compiler)
    auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    g = uni(g);
    m0 = uni(m0);
    rows = uni(rows);
    const long long row0 = uni(plan.lo[g]);
    const int n0 = uni(nt) * NOUT;
    const size_t wat = static_cast<size_t>(g) * F * d;
    const bf16_t* wg = static_cast<const bf16_t*>(p.w_gate) + wat;
    const bf16_t* wu = static_cast<const bf16_t*>(p.w_up) + wat;
    const int kend = FWD ? d : DW ? uni(plan.rows[g]) : F;
    const int nseg = (kend + C::BK - 1) / C::BK;
    const int steps = PART == GatedPart::kDx ? 2 * nseg : nseg;
    const int first = SPLIT ? static_cast<int>(static_cast<long long>(steps) * slice / splits) : 0;
    const int nk = SPLIT ? static_cast<int>(static_cast<long long>(steps) * (slice + 1) / splits) - first
                         : steps;

    KtLoads<C::LPW_MAX> t;
    t.kend = kend;
    t.nseg = nseg;
    t.first = first;
    t.jump = 0;
    // offsets inside a tile stay below 2^32: 256 rows of up to 2 * 131072 values
    if (wm == 1) {
      t.kstride = TA ? F2 : 1;
      if (PART == GatedPart::kDx) t.jump = F;
      t.base = FWD ? x + (row0 + m0) * d : dau + (row0 + (DW ? 0 : m0)) * F2 + (half ? F : 0);
#pragma unroll
      for (int q = 0; q < C::LPW_A; ++q) {
        const int j = wn * C::LPW_A + q;
        int k;
        if constexpr (TA) {
          int col;
          lines_place<C::MT>(lane, j, k, col);
          t.off[q] = 2u * (static_cast<uint32_t>(k) * F2 + min(m0 + col, F - 8));
        } else {
          const int r = j * C::RPL + lrow;
          k = src_chunk<C>(lane, j);
          t.off[q] = 2u * (static_cast<uint32_t>(r < rows ? r : rows - 1) * (FWD ? d : F2) + k);
        }
        if (q == 0) t.kpos = k;
      }
    } else {
      t.kstride = TB ? d : 1;
      if (PART == GatedPart::kDx) t.jump = wu - wg;
      t.base = DW ? x + row0 * d : FWD ? wg + static_cast<size_t>(n0) * d : wg;
      t.upper = wu - wg;
#pragma unroll
      for (int q = 0; q < C::LPW_B; ++q) {
        const int j = wn * C::LPW_B + q;
        int k;
        if constexpr (TB) {
          int col;
          lines_place<C::NB>(lane, j, k, col);
          t.off[q] = 2u * (static_cast<uint32_t>(k) * d + min(n0 + col, d - 8));
        } else {
          // of 64 LDS rows, which a wave loads, 32 are rows of Wg and 32 of Wu
          const int R = j * C::RPL + lrow;
          const int col = min(n0 + (R >> 6) * 32 + (R & 31), F - 1);
          k = src_chunk<C>(lane, j);
          t.off[q] = 2u * (static_cast<uint32_t>(col - n0) * d + k);
        }
        if (q == 0) t.kpos = k;
      }
    }
    f32x16_t acc[C::BM][C::BN];
#pragma unroll
    for (int i = 0; i < C::BM; ++i)
#pragma unroll
      for (int j = 0; j < C::BN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    if ((!DW && !SPLIT) || nk > 0) {  // a group without rows: zeros
      const int nblk = (rows + 31) >> 5;
      const int nv = min((nblk - wm + 1) >> 1, C::BM);
      if (wm == 0) kt_kloop_nv<C, TA, TB, 0, C::BM>(t, nk, sA, sB, wave, lane, nv, acc);
      else kt_kloop_nv<C, TA, TB, 1, C::BM>(t, nk, sA, sB, wave, lane, nv, acc);
      wait_vm<0>();
      __syncthreads();
    }

    // ---- epilogue: block (i, j) holds the transposed product: lane l -> tile
    // row (2i + wm) * 32 + l % 32, registers 4q..4q+3 -> columns 8q + 4 (l / 32) +
    // 0..3 of column block j (forward: block 0 a, 1 u).  Through an LDS tile, 16-byte
    // chunk c of row r in slot c ^ (r % CPR), to coalesced stores.
    if constexpr (SPLIT) {
      // the columns of dx or dW, or forward a and u of a row [2F]
      const size_t ld = FWD ? F2 : d;
      float* to = p.part + (static_cast<size_t>(slice) * (DW ? F2 : p.M) +
                            (DW ? (half ? F : 0) : row0) + m0) * ld;
      constexpr int CPR = C::NB / 4;
      float* tile = reinterpret_cast<float*>(lds);
#pragma unroll
      for (int i = 0; i < C::BM; ++i) {
        const int row = (2 * i + wm) * 32 + (lane & 31);
#pragma unroll
        for (int j = 0; j < C::BN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int ch = wn * 16 + j * 8 + 2 * q + (lane >> 5);
            *reinterpret_cast<float4*>(tile + (row * CPR + (ch ^ (row & (CPR - 1)))) * 4) =
                make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                            acc[i][j][4 * q + 3]);
          }
      }
      __syncthreads();
      for (int c = tid; c < rows * CPR; c += C::THREADS) {
        const int row = c / CPR, ch = c % CPR;
        // forward: of 64 columns of the tile, 32 are a's and 32 u's
        const int col = n0 + (FWD ? ch / 16 * 32 + ch % 8 * 4 : ch * 4);
        if (col < ncols)
          *reinterpret_cast<float4*>(to + row * ld + (FWD && (ch & 8) ? F : 0) + col) =
              *reinterpret_cast<const float4*>(tile + (row * CPR + (ch ^ (row & (CPR - 1)))) * 4);
      }
      continue;
    }
    if (FWD && !p.h && !p.pre) continue;
    constexpr int CPR = NOUT / 8;
    bf16_t* tile = lds;
#pragma unroll
    for (int i = 0; i < C::BM; ++i) {
      const int row = (2 * i + wm) * 32 + (lane & 31);
      bf16_t* trow = tile + row * NOUT + 4 * (lane >> 5);
      const int sw = row & (CPR - 1);
#pragma unroll
      for (int j = 0; j < (FWD ? 1 : C::BN); ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = acc[i][j][4 * q + e];
            if (FWD) v[e] = v[e] * sigmoid(v[e]) * acc[i][1][4 * q + e];
          }
          // (a and u straight from the registers, 32 bytes of a row at a time; through
          // an LDS tile the forward pass of 24576 rows over 128 experts took 313 us
          // against 275)
          const int c = n0 + wn * 32 + 8 * q + 4 * (lane >> 5);
          if (FWD && p.pre && row < rows && c < F) {
            float* o = p.pre + (row0 + m0 + row) * F2 + c;
            *reinterpret_cast<float4*>(o) = make_float4(acc[i][0][4 * q], acc[i][0][4 * q + 1],
                                                        acc[i][0][4 * q + 2], acc[i][0][4 * q + 3]);
            *reinterpret_cast<float4*>(o + F) = make_float4(acc[i][1][4 * q], acc[i][1][4 * q + 1],
                                                            acc[i][1][4 * q + 2], acc[i][1][4 * q + 3]);
          }
          const uint32_t w0 = f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16);
          const uint32_t w1 = f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16);
          const int ch = FWD ? wn * 4 + q : wn * 8 + j * 4 + q;
          *reinterpret_cast<uint2*>(trow + ((ch ^ sw) << 3)) = make_uint2(w0, w1);
        }
    }
    bf16_t* out = FWD ? static_cast<bf16_t*>(p.h) + (row0 + m0) * F
                  : DW ? static_cast<bf16_t*>(half ? p.dw_up : p.dw_gate) + wat +
                             static_cast<size_t>(m0) * d
                       : static_cast<bf16_t*>(p.dx) + (row0 + m0) * d;
    if (FWD && !p.h) continue;
    __syncthreads();
    for (int c = tid; c < rows * CPR; c += C::THREADS) {
      const int row = c / CPR, ch = c % CPR;
      if (n0 + ch * 8 < ncols)
        *reinterpret_cast<uint4*>(out + static_cast<size_t>(row) * ncols + n0 + ch * 8) =
            *reinterpret_cast<const uint4*>(tile + row * NOUT + ((ch ^ (row & (CPR - 1))) << 3));
    }
  }
}

// The result from the slices' sums, in order, 4 values of a row a thread.  Forward:
// h from a and u, and pre.  Rows outside the one group keep what they held.
template <GatedPart PART>
__global__ __launch_bounds__(256) void gated_reduce_kernel(GatedArgs p) {
  constexpr bool FWD = PART == GatedPart::kForward, DW = PART == GatedPart::kDw;
  long long first = 0, last = DW ? 2 * p.F : p.M;
  if (!DW && p.offsets) {
    first = clampi(p.offsets[0], 0, p.M);
    last = clampi(p.offsets[1], 0, p.M);
  }
  const int cols = FWD ? p.F : p.d, ld = FWD ? 2 * p.F : p.d, quads = cols / 4;
  const size_t slice = static_cast<size_t>(DW ? 2 * p.F : p.M) * ld;
  for (long long i = first * quads + static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
       i < last * quads; i += static_cast<long long>(gridDim.x) * 256) {
    const long long row = i / quads;
    const int c = static_cast<int>(i - row * quads) * 4;
    const float* from = p.part + row * ld + c;
    f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f}, u = v;
    for (int s = 0; s < p.splits; ++s) {
      v += *reinterpret_cast<const f32x4_t*>(from + s * slice);
      if (FWD) u += *reinterpret_cast<const f32x4_t*>(from + s * slice + p.F);
    }
    if (FWD && p.pre) {
      *reinterpret_cast<f32x4_t*>(p.pre + row * ld + c) = v;
      *reinterpret_cast<f32x4_t*>(p.pre + row * ld + p.F + c) = u;
    }
    if (FWD && !p.h) continue;
    if (FWD)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] * sigmoid(v[e]) * u[e];
    bf16_t* out = FWD ? static_cast<bf16_t*>(p.h) + row * p.F
                  : DW ? (row < p.F ? static_cast<bf16_t*>(p.dw_gate) + row * p.d
                                    : static_cast<bf16_t*>(p.dw_up) + (row - p.F) * p.d)
                       : static_cast<bf16_t*>(p.dx) + row * p.d;
    *reinterpret_cast<uint2*>(out + c) =
        make_uint2(f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16),
                   f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16));
  }
}

template <GatedPart PART>
hipError_t run(const GatedArgs& a, hipStream_t st) {
  const int grid = (device_cus_big() + kXcds - 1) / kXcds * kXcds;
  auto go = [&](auto kernel) { kernel<<<grid, Mid::THREADS, 0, st>>>(a); };
  if (a.splits > 1) {
    go(gated_big_kernel<Mid, PART, true>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long long rows = PART == GatedPart::kDw ? 2LL * a.F : a.M;
    const long long blocks = (rows * (PART == GatedPart::kForward ? a.F : a.d) / 4 + 255) / 256;
    gated_reduce_kernel<PART><<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256, 0, st>>>(a);
  } else if constexpr (PART == GatedPart::kForward) {
    go(gated_big_kernel<Mid, PART>);
  } else {
    if (large_tiles(a, PART)) go(gated_big_kernel<Big, PART>);
    else go(gated_big_kernel<Mid, PART>);
  }
  return hipGetLastError();
}

}  // namespace

// Slices of K of a product of one group on 128-row tiles: where there are few tiles a
// workgroup walks all of K alone (a step of 64 takes 0.6 us of it), while others have
// none.  Estimated (us): the walk, and for slices 6 and their sums written and read
// at 4 TB/s.  Measured (us, one walk / slices, d=7168 F=2048): 256 rows forward 68 /
// 31, dx 39 / 27, dW 31 / 24; 1024 rows forward 72 / 62; 64 rows of d=2048 F=768
// forward 21.5 / 13.6, dx 12.6 / 7.2.
static int splits_of(int M, int d, int F, int E, GatedPart part, double& time) {
  const bool fwd = part == GatedPart::kForward, dw = part == GatedPart::kDw;
  const double rows = dw ? 2.0 * F : M, cols = fwd ? 2.0 * F : d;
  const double entries = std::ceil(rows / 128.0) * (dw ? E : 1) + (!dw && E > 1 ? std::min(M, E) : 0);
  const double items = entries * std::ceil(cols / 256.0);
  const double nk = fwd  ? std::ceil(d / 64.0)
                    : dw ? std::ceil(M / 64.0 / E)
                         : 2.0 * std::ceil(F / 64.0);
  int best = 1;
  time = nk * 0.6 * std::ceil(items / 256.0);
  for (int s = 2; E == 1 && s <= 16 && s * 2 <= nk; ++s) {
    const double t = 6.0 + std::ceil(nk / s) * 0.6 * std::ceil(items * s / 256.0) +
                     8.0 * s * rows * cols / 4e6;
    if (t < 0.9 * time) {
      time = t;
      best = s;
    }
  }
  return best;
}

int gated_splits(int M, int d, int F, int E, GatedPart part) {
  double time;
  return splits_of(M, d, F, E, part, time);
}

double gated_tiles_time(int M, int d, int F, int E, GatedPart part) {
  double time;
  splits_of(M, d, F, E, part, time);
  return 7.0 + time;
}

hipError_t launch_gated_big(const GatedArgs& a, GatedPart part, hipStream_t st) {
  switch (part) {
    case GatedPart::kForward: return run<GatedPart::kForward>(a, st);
    case GatedPart::kDx: return run<GatedPart::kDx>(a, st);
    default: return run<GatedPart::kDw>(a, st);
  }
}

}  // namespace moe
