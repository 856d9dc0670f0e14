// Grouped products of 8-bit integer rows: y = s_r t_n (q . w), and the SwiGLU
// pair of them for the experts' gate/up half.
//
// The sums are exact in int32 (K <= 131072), so the only rounding is the
// scaling in fp32 and the store.
#include <cmath>

#include "big_tile.h"
#include "int8_rows.h"

namespace moe {

// ------------------------------------------------------------ large batches
//
// The bf16 experts' tile and K loop (big_tile.h) on 8-bit operands: the same
// bytes per step hold twice the K, and the int8 matrix instruction does twice
// the products in the same cycles.  Row tiles of up to 256 rows (or 128 where
// groups hold few) x 256 weight rows; each XCD's workgroups share a contiguous
// run of the items, evenly or by a counter (by_counters).
//
// Large products run at the rate of the matrix instructions' own library product
// (8192^3 2.09 POP/s here): 16384x2048x7168 takes 218 to 241 us, 2.0 to 2.2 POP/s,
// the matrix units busy in 56% of the cycles of a clock that the load pulls down
// to 1.8 GHz (of 2.4), memory at 1.8 TB/s.  The experts of a large batch (d=7168,
// F=2048, 131072 rows in ragged groups) run at 1.9 POP/s gate/up (52% busy) and
// 1.6 down (42%), where K is short and the epilogue (scales, bf16, the staged
// tile) a seventh of a tile's time.  With few rows a group it streams the
// weights: T=64 there reads 2.71 + 1.36 GB in 500 + 298 us, 5.4 and 4.6 TB/s.
// The 256-row forms use all 256 registers; the gated and the bf16 one keep one or
// two more in scratch memory, stored before the K loop and read after it.
using BigI8 = BigShape<256, 32, 3, 6, MmaI8>;
using MidI8 = BigShape<128, 64, 3, 3, MmaI8>;
static_assert(BigI8::LDS_ELEMS * 2 <= 147456 && MidI8::LDS_ELEMS * 2 <= 147456, "LDS");

// Work counters in the workspace: a set of kXcds for each of up to two products.
constexpr int kCounters = 2 * kXcds;

__global__ void int8_counters_kernel(int32_t* counters) {
  if (threadIdx.x < kCounters) counters[threadIdx.x] = 0;
}

// 4 consecutive values of a scale row of n values, from column c on (0 past its
// end).
__device__ __forceinline__ void scale4(const float* t, int c, int n, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = c + i < n ? t[c + i] : 0.0f;
}

template <class C, bool GATED, bool OUT_BF16>
__global__ __launch_bounds__(512, 1) void gemm_int8_big_kernel(Int8Args p,
                                                               int32_t* counters) {
  __shared__ __attribute__((aligned(1024))) bf16_t lds[C::LDS_ELEMS];
  __shared__ EntryPlan plan;
  __shared__ long long s_item;
  bf16_t* sA[C::NSA];
  bf16_t* sB[C::NSB];
#pragma unroll
  for (int i = 0; i < C::NSA; ++i) sA[i] = lds + i * C::A_STAGE;
#pragma unroll
  for (int i = 0; i < C::NSB; ++i) sB[i] = lds + C::NSA * C::A_STAGE + i * C::B_STAGE;
  constexpr int NOUT = GATED ? C::NB / 2 : C::NB;   // output columns of a tile
  constexpr int OB = OUT_BF16 ? 2 : 4;              // bytes of an output value
  // the staged output tile; fp32 outputs of a whole tile do not fit and go
  // straight from the registers
  constexpr bool STAGED = C::MT * NOUT * OB <= C::LDS_ELEMS * 2;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int G = p.E + p.S;
  make_entries<C::THREADS, C::MT>(p, plan);
  const int n_tiles = (p.N + NOUT - 1) / NOUT;
  const long long total = static_cast<long long>(plan.start[G]) * n_tiles;
  const int xcd = blockIdx.x % kXcds;
  const int kld = p.Kp / 2;  // row length in 16-bit units
  const int nk = kld / C::BK;
  const size_t wstride = static_cast<size_t>(p.N) * kld;
  const int lrow = lane / C::CPR;
  const bf16_t* A = reinterpret_cast<const bf16_t*>(p.a);

  const long long chunk = (total + kXcds - 1) / kXcds;
  for (long long mine = blockIdx.x / kXcds;; mine += gridDim.x / kXcds) {
    long long gitem = xcd * chunk + mine;
    if (counters) {
      if (tid == 0) s_item = claim_item(counters, xcd, total);
      __syncthreads();
      gitem = s_item;
      if (gitem < 0) break;
    } else {
      if (mine >= chunk || gitem >= total) break;
      __syncthreads();  // the item before is done with the LDS
    }
    const int g = entry_group(plan, G, static_cast<int>(gitem / n_tiles));
    const Item item = place_item(gitem, plan.start, g, n_tiles, C::MT, plan.rows[g], true);
    const bool routed = g < p.E;
    const int ge = routed ? g : g - p.E;
    const int row0 = routed ? plan.lo[g] : 0;
    // row of a and of its scale for tile row r
    auto source = [&](int r) -> long long {
      return source_row<GATED>(p, routed, ge, row0,
                               item.m0 + (r < item.rows ? r : item.rows - 1));
    };
    BigCtx<C> t;
    if (wm == 1) {
#pragma unroll
      for (int q = 0; q < C::LPW_A; ++q) {
        const int j = wn * C::LPW_A + q;
        t.src[q] = A + source(j * C::RPL + lrow) * kld + src_chunk<C>(lane, j);
      }
    } else {
#pragma unroll
      for (int q = 0; q < C::LPW_B; ++q) {
        const int j = wn * C::LPW_B + q;
        const int R = j * C::RPL + lrow;  // LDS B row
        const int cg = R >> 6, rl = R & 63;
        const bool up = GATED && rl >= 32;
        const int8_t* base = up ? (routed ? p.w1 : p.ws1) : (routed ? p.w0 : p.ws0);
        int col = GATED ? item.n * NOUT + cg * 32 + (rl & 31) : item.n * NOUT + R;
        col = col < p.N ? col : p.N - 1;
        t.src[q] = reinterpret_cast<const bf16_t*>(base) + ge * wstride +
                   static_cast<size_t>(col) * kld + src_chunk<C>(lane, j);
      }
    }
    typename C::Acc acc[C::BM][C::BN];
#pragma unroll
    for (int i = 0; i < C::BM; ++i)
#pragma unroll
      for (int j = 0; j < C::BN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    const int nblk = (item.rows + 31) >> 5;
    const int nv = min((nblk - wm + 1) >> 1, C::BM);
    if (wm == 0) big_kloop_nv<C, GATED, 0, C::BM>(t, nk, sA, sB, wave, lane, nv, acc);
    else big_kloop_nv<C, GATED, 1, C::BM>(t, nk, sA, sB, wave, lane, nv, acc);
    wait_vm<0>();
    __syncthreads();

    // ---- epilogue: block (i, j) holds the transposed product: lane l -> tile
    // row (2i + wm) * 32 + l % 32, registers 4q..4q+3 -> output columns
    // 8q + 4 (l / 32) + 0..3 of column block j (GATED: block 0 gate, 1 up).
    // Staged: 16-byte chunk c of row r in slot c ^ (r % CPR) of the LDS tile.
    const float* t0 = (routed ? p.t0 : p.ts0) + static_cast<size_t>(ge) * p.N;
    const float* t1 = GATED ? (routed ? p.t1 : p.ts1) + static_cast<size_t>(ge) * p.N : nullptr;
    char* out = static_cast<char*>(routed ? p.out : p.out_shared);
    const size_t orow0 = routed ? static_cast<size_t>(row0) + item.m0
                                : static_cast<size_t>(ge) * p.T + item.m0;
    constexpr int CPR = NOUT * OB / 16;
    char* tile = reinterpret_cast<char*>(lds);
    float sr[C::BM];
#pragma unroll
    for (int i = 0; i < C::BM; ++i) sr[i] = p.a_scale[source((2 * i + wm) * 32 + (lane & 31))];
    constexpr int JN = GATED ? 1 : C::BN;
#pragma unroll
    for (int j = 0; j < JN; ++j) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = (GATED ? wn * 32 : wn * 64 + j * 32) + 8 * q + 4 * (lane >> 5);
        const int col = item.n * NOUT + c;
        float s0[4], s1[4];
        scale4(t0, col, p.N, s0);
        if (GATED) scale4(t1, col, p.N, s1);
#pragma unroll
        for (int i = 0; i < C::BM; ++i) {
          const int row = (2 * i + wm) * 32 + (lane & 31);
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = static_cast<float>(acc[i][j][4 * q + e]) * (sr[i] * s0[e]);
            if (GATED) {
              const float up = static_cast<float>(acc[i][1][4 * q + e]) * (sr[i] * s1[e]);
              v[e] = v[e] / (1.0f + expf(-v[e])) * up;
            }
          }
          if constexpr (STAGED && OUT_BF16) {
            const uint32_t w0 = f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16);
            const uint32_t w1 = f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16);
            *reinterpret_cast<uint2*>(tile + row * NOUT * OB +
                                      (((c >> 3) ^ (row & (CPR - 1))) << 4) + (c & 4) * 2) =
                make_uint2(w0, w1);
          } else if constexpr (STAGED) {
            *reinterpret_cast<float4*>(tile + row * NOUT * OB +
                                       (((c >> 2) ^ (row & (CPR - 1))) << 4)) =
                make_float4(v[0], v[1], v[2], v[3]);
          } else if (row < item.rows) {
            float* o = reinterpret_cast<float*>(out) + (orow0 + row) * p.N + col;
            if (p.N % 4 == 0 && col + 4 <= p.N) {
              *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (col + e < p.N) o[e] = v[e];
            }
          }
        }
      }
    }
    if constexpr (STAGED) {
      __syncthreads();
      constexpr int PER = 16 / OB;  // values of a chunk
      const int col0 = item.n * NOUT;
      const bool whole = p.N % PER == 0;  // rows of y start on 16 bytes
      for (int c = tid; c < item.rows * CPR; c += C::THREADS) {
        const int row = c / CPR, ch = c % CPR;
        const uint4 v = *reinterpret_cast<const uint4*>(tile + row * NOUT * OB +
                                                        ((ch ^ (row & (CPR - 1))) << 4));
        const int col = col0 + ch * PER;
        char* o = out + ((orow0 + row) * p.N + col) * OB;
        if (whole) {
          if (col < p.N) *reinterpret_cast<uint4*>(o) = v;
        } else {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            if (col + e >= p.N) break;
            if (OUT_BF16) reinterpret_cast<bf16_t*>(o)[e] = static_cast<bf16_t>(w[e / 2] >> (16 * (e & 1)));
            else reinterpret_cast<uint32_t*>(o)[e] = w[e % 4];
          }
        }
      }
    }
  }
}

template <class C>
static hipError_t run_big(const Int8Args& a, bool gated, int32_t* ctr, hipStream_t st) {
  const int grid = (device_cus_big() + kXcds - 1) / kXcds * kXcds;
  if (gated) gemm_int8_big_kernel<C, true, false><<<grid, C::THREADS, 0, st>>>(a, ctr);
  else if (a.out_bf16) gemm_int8_big_kernel<C, false, true><<<grid, C::THREADS, 0, st>>>(a, ctr);
  else gemm_int8_big_kernel<C, false, false><<<grid, C::THREADS, 0, st>>>(a, ctr);
  return hipGetLastError();
}

// ------------------------------------------------------------------ host

size_t gemm_int8_counter_ints() { return kCounters; }

// Kernel of a product, by estimates of their times (us) fitted to measured ones.
// They agree to the bit, so the choice is one of speed alone.  M is the rows, mu
// the mean rows of a group, G the groups expected to have any:
//   tiles  7 + the weights read once per 16 rows of a group, at 9 TB/s while
//          they stay in the caches and 5.3 from memory, + 3 for each turn of the
//          256 workgroups to stage 16 rows
//   128    11 + the slower of the weights read once at 5.3 TB/s and the rounds of
//          256 tiles: a full one 7.6 per 1000 of K, one of few tiles 5, and 5 more
//          for each round after the first
//   256    13.7 + the same with 14.2 and 8.4
// Measured (us; N x K, groups):
//   rows              1     64    256   1024   4096   12000   16384   4 a group  96 a group
//   tiles 2048x7168  15     16     34    110    402    1183    1587      194        1474
//   128              35     35     46     48     67     177     241      205         261
//   256              55     55     73     75     82     188     218      241         300
//   (the last two columns 2048x2048, 256 groups)
enum class Path { kTiles, kMid, kBig };
static Path path(const Int8Args& a, bool gated) {
  const double n = gated ? 2.0 * a.N : a.N, k = a.Kp, mu = static_cast<double>(a.M) / a.E;
  const double full = a.E == 1 ? 1.0 : a.E * (1.0 - std::exp(-mu));
  const double weights = (full + a.S) * n * k * 1e-6;  // megabytes
  // row tiles of MT rows: at least one a group with rows, half a tile wasted
  auto row_tiles = [&](double mt) {
    const double r = a.E == 1 ? std::ceil(a.M / mt) : full * std::fmax(1.0, mu / mt + 0.5);
    return r + a.S * std::ceil(a.T / mt);
  };
  const double r16 = row_tiles(16);
  const double tiles = 7.0 + r16 * n * k * 1e-6 / (weights < 200.0 ? 9.0 : 5.3) + r16 * 3.0 / 256.0;
  const double cols = std::ceil(n / 256.0), stream = weights / 5.3;
  auto large = [&](double mt, double fixed, double few, double all) {
    const double t = row_tiles(mt) * cols / 256.0, before = std::ceil(t) - 1.0;
    return fixed + std::fmax(stream, 5.0 * before + k * 1e-3 * (before * all + few +
                                                                (all - few) * (t - before)));
  };
  const double mid = large(128, 11.0, 5.0, 7.6), big = large(256, 13.7, 8.4, 14.2);
  if (tiles <= mid && tiles <= big) return Path::kTiles;
  return mid <= big ? Path::kMid : Path::kBig;
}

// Whether the workgroups of the large tiles take their items from counters: it
// evens out groups that end in a part of a tile, and costs a launch that clears
// the counters (5 us) and 5 to 10 us of atomics at both ends of the kernel.  From
// about 16 items a workgroup on, where there are groups.  Measured (us; counters
// with their launch / fixed shares):
//   items a workgroup   1 (3655x3920x1393)       58 / 36
//                       2 (16384x2048x7168)     263 / 235
//                       3 (24576x768x2048, 256 groups)   134 / 120
//                       7 (prefill experts' gate/up, K 2048)   255 / 256
//                       40 (large experts' gate/up, K 7168)    4128 / 4353
static bool by_counters(const Int8Args& a, bool gated, int mt) {
  if (a.E == 1 && a.S == 0) return false;
  const long long rows = a.M + static_cast<long long>(a.S) * a.T;
  const long long cols = (a.N + (gated ? 127 : 255)) / (gated ? 128 : 256);
  return rows / mt * cols >= 16LL * device_cus_big();
}

hipError_t launch_gemm_int8(const Int8Args& a, bool gated, int32_t* counters, bool& cleared,
                            hipStream_t st) {
  if (a.M == 0 && (a.S == 0 || a.T == 0)) return hipSuccess;
  const Path way = path(a, gated);
  if (way == Path::kTiles) return launch_gemm_int8_tiles(a, gated, st);
  int32_t* ctr = nullptr;
  if (by_counters(a, gated, way == Path::kMid ? MidI8::MT : BigI8::MT)) {
    ctr = counters + (cleared ? kXcds : 0);
    if (!cleared) {
      int8_counters_kernel<<<1, 64, 0, st>>>(counters);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      cleared = true;
    }
  }
  return way == Path::kMid ? run_big<MidI8>(a, gated, ctr, st) : run_big<BigI8>(a, gated, ctr, st);
}

}  // namespace moe
