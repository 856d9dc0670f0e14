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
#include "gated.h"
#include "tile_kt.h"

namespace moe {

namespace {

using Big = BigShape<256, 32, 3, 6>;
using Mid = BigShape<128, 64, 3, 3>;

template <class C, GatedPart PART>
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

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  make_entries<C::THREADS, C::MT, kMaxGroups>(p, plan);
  const int d = p.d, F = p.F, F2 = 2 * F;
  const int ncols = FWD ? F : d;  // columns of the result
  const int n_tiles = (ncols + NOUT - 1) / NOUT;
  const int m_tiles = (F + C::MT - 1) / C::MT;  // kDw: row tiles of a matrix
  const long long total = (DW ? static_cast<long long>(p.E) * 2 * m_tiles
                              : static_cast<long long>(plan.start[p.E])) * n_tiles;
  const int xcd = blockIdx.x % kXcds;
  const bf16_t* x = static_cast<const bf16_t*>(p.x);
  const bf16_t* dau = static_cast<const bf16_t*>(p.dau);
  const int lrow = lane / C::CPR;

  const long long chunk = (total + kXcds - 1) / kXcds;
  for (long long mine = blockIdx.x / kXcds;; mine += gridDim.x / kXcds) {
    const long long it = xcd * chunk + mine;
    if (mine >= chunk || it >= total) break;
    __syncthreads();  // the item before is done with the LDS
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
    const int nk = PART == GatedPart::kDx ? 2 * nseg : nseg;

    KtLoads<C::LPW_MAX> t;
    t.kend = kend;
    t.nseg = nseg;
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
    if (!DW || nk > 0) {  // a group without rows: zeros
      const int nblk = (rows + 31) >> 5;
      const int nv = min((nblk - wm + 1) >> 1, C::BM);
      if (wm == 0) kt_kloop_nv<C, TA, TB, 0, C::BM>(t, nk, sA, sB, wave, lane, nv, acc);
      else kt_kloop_nv<C, TA, TB, 1, C::BM>(t, nk, sA, sB, wave, lane, nv, acc);
      wait_vm<0>();
      __syncthreads();
    }

    // ---- epilogue: block (i, j) holds the transposed product: lane l -> tile
    // row (2i + wm) * 32 + l % 32, registers 4q..4q+3 -> columns 8q + 4 (l / 32) +
    // 0..3 of column block j (forward: block 0 a, 1 u).  Through the LDS tile, 16-byte
    // chunk c of row r in slot c ^ (r % CPR), to coalesced stores.
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
          if (FWD && p.pre && row < rows) {
            const int c = n0 + wn * 32 + 8 * q + 4 * (lane >> 5);
            if (c < F) {
              float* o = p.pre + (row0 + m0 + row) * F2 + c;
              *reinterpret_cast<float4*>(o) = make_float4(acc[i][0][4 * q], acc[i][0][4 * q + 1],
                                                          acc[i][0][4 * q + 2], acc[i][0][4 * q + 3]);
              *reinterpret_cast<float4*>(o + F) =
                  make_float4(acc[i][1][4 * q], acc[i][1][4 * q + 1], acc[i][1][4 * q + 2],
                              acc[i][1][4 * q + 3]);
            }
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

template <class C>
hipError_t run(const GatedArgs& a, GatedPart part, hipStream_t st) {
  const int grid = (device_cus_big() + kXcds - 1) / kXcds * kXcds;
  if (part == GatedPart::kForward)
    gated_big_kernel<C, GatedPart::kForward><<<grid, C::THREADS, 0, st>>>(a);
  else if (part == GatedPart::kDx)
    gated_big_kernel<C, GatedPart::kDx><<<grid, C::THREADS, 0, st>>>(a);
  else
    gated_big_kernel<C, GatedPart::kDw><<<grid, C::THREADS, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_big(const GatedArgs& a, GatedPart part, int rows, hipStream_t st) {
  return rows == Big::MT ? run<Big>(a, part, st) : run<Mid>(a, part, st);
}

}  // namespace moe
