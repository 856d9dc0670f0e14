// Gated block and its gradients on the fp32 matrix cores: any sizes, either type.
//
// Three products (gated.h).  Forward: rows of x against 32-row blocks of 16 rows of
// Wg and the same 16 rows of Wu, so that a lane ends with a and u of the same
// columns.  dx: rows of dau, whose 2F values of K meet the rows of Wg, then of Wu.
// dW: columns of dau (rows of the result: F of dWg, then F of dWu) and of x, K the
// rows of the group; a group without rows writes zeros.
#include "gated.h"
#include "tile32.h"

namespace moe {

namespace {

template <int R, typename T, GatedPart PART>
__global__ __launch_bounds__(kT32Threads) void gated_tile_kernel(GatedArgs p) {
  using C = Tile32<R>;
  __shared__ __attribute__((aligned(16))) typename C::Lds lds;
  __shared__ EntryPlan plan;
  constexpr bool FWD = PART == GatedPart::kForward, DW = PART == GatedPart::kDw;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1, half = lane >> 5;
  make_entries<kT32Threads, C::N, kMaxGroups>(p, plan);
  const int d = p.d, F = p.F, F2 = 2 * F;
  constexpr int NOUT = FWD ? C::N / 2 : C::N;   // columns of the result in a tile
  const int n_tiles = ((FWD ? F : d) + NOUT - 1) / NOUT;
  const int m_tiles = (F2 + C::N - 1) / C::N;   // kDw: row tiles of a group's result
  const long long total = (DW ? static_cast<long long>(p.E) * m_tiles
                              : static_cast<long long>(plan.start[p.E])) * n_tiles;
  const T* x = static_cast<const T*>(p.x);
  const T* dau = static_cast<const T*>(p.dau);
  // rows that start on 4 values
  auto quads = [](const void* b, int ld) {
    return ld % 4 == 0 && reinterpret_cast<uintptr_t>(b) % (4 * sizeof(T)) == 0;
  };
  const bool vx = quads(x, d), vw = quads(p.w_gate, d) && quads(p.w_up, d), vd = F % 2 == 0;

  for (long long it = blockIdx.x; it < total; it += gridDim.x) {
    const int ent = static_cast<int>(it / n_tiles), nt = static_cast<int>(it % n_tiles);
    const int g = DW ? ent / m_tiles : entry_group(plan, p.E, ent);
    const int m0 = (DW ? ent % m_tiles : ent - plan.start[g]) * C::N;
    const int rows = DW ? min(F2 - m0, C::N) : min(plan.rows[g] - m0, C::N);
    const long long row0 = plan.lo[g];
    const int n0 = nt * NOUT;
    const size_t wat = static_cast<size_t>(g) * F * d;
    const T* wg = static_cast<const T*>(p.w_gate) + wat;
    const T* wu = static_cast<const T*>(p.w_up) + wat;
    f32x16_t acc[R][R];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    if constexpr (FWD) {
      auto la = [&](int r, int k, float (&v)[4]) {
        load4(x + (row0 + m0 + min(r, rows - 1)) * d + k, d - k, vx, v);
      };
      auto lb = [&](int r, int k, float (&v)[4]) {
        const int c = min(n0 + r / 32 * 16 + r % 16, F - 1);
        load4((r & 16 ? wu : wg) + static_cast<size_t>(c) * d + k, d - k, vw, v);
      };
      tile32_product<R, true, true>(lds, d, la, lb, acc);
    } else if constexpr (PART == GatedPart::kDx) {
      auto la = [&](int r, int k, float (&v)[4]) {
        load4(dau + (row0 + m0 + min(r, rows - 1)) * F2 + k, F2 - k, vd, v);
      };
      auto lb = [&](int r, int k, float (&v)[4]) {
        const T* w = k < F ? wg + static_cast<size_t>(k) * d : wu + static_cast<size_t>(k - F) * d;
        load4(w + n0 + r, k < F2 ? d - n0 - r : 0, vw, v);
      };
      tile32_product<R, true, false>(lds, F2, la, lb, acc);
    } else {
      const int K = plan.rows[g];
      auto la = [&](int r, int k, float (&v)[4]) {
        load4(dau + (row0 + k) * F2 + m0 + r, k < K ? F2 - m0 - r : 0, vd, v);
      };
      auto lb = [&](int r, int k, float (&v)[4]) {
        load4(x + (row0 + k) * d + n0 + r, k < K ? d - n0 - r : 0, vx, v);
      };
      tile32_product<R, false, false>(lds, K, la, lb, acc);
    }

#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = 32 * (R * wm + i) + (lane & 31);
      if (r >= rows) continue;
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int q = 0; q < (FWD ? 2 : 4); ++q) {
          const int c = n0 + (FWD ? 16 : 32) * (R * wn + j) + 8 * q + 4 * half;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (FWD) {
              if (c + e >= F) continue;
              const float a = acc[i][j][4 * q + e], u = acc[i][j][8 + 4 * q + e];
              const size_t row = static_cast<size_t>(row0 + m0 + r);
              if (p.h) ActTraits<T>::store(static_cast<T*>(p.h) + row * F + c + e, a * sigmoid(a) * u);
              if (p.pre) {
                p.pre[row * F2 + c + e] = a;
                p.pre[row * F2 + F + c + e] = u;
              }
            } else {
              if (c + e >= d) continue;
              T* out;
              if (!DW) {
                out = static_cast<T*>(p.dx) + static_cast<size_t>(row0 + m0 + r) * d;
              } else {
                const int n = m0 + r;
                out = (n < F ? static_cast<T*>(p.dw_gate) + wat + static_cast<size_t>(n) * d
                             : static_cast<T*>(p.dw_up) + wat + static_cast<size_t>(n - F) * d);
              }
              ActTraits<T>::store(out + c + e, acc[i][j][4 * q + e]);
            }
          }
        }
    }
  }
}

// dau from pre and dh, in fp32, rounded once to T (the products that read dau take
// T).  A thread per 4 columns of a row.
template <typename T>
__global__ __launch_bounds__(256) void gated_dau_kernel(GatedArgs p, int quads) {
  const int F = p.F;
  const long long total = static_cast<long long>(p.M) * quads;
  const bool vec = F % 4 == 0 && reinterpret_cast<uintptr_t>(p.dh) % (4 * sizeof(T)) == 0 &&
                   reinterpret_cast<uintptr_t>(p.pre) % 16 == 0;
  const T* dh = static_cast<const T*>(p.dh);
  T* dau = static_cast<T*>(p.dau);
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * 256) {
    const long long row = i / quads;
    const int c = static_cast<int>(i - row * quads) * 4, n = F - c;
    float a[4], u[4], g[4], da[4], du[4];
    load4(p.pre + row * 2 * F + c, n, vec, a);
    load4(p.pre + row * 2 * F + F + c, n, vec, u);
    load4(dh + row * F + c, n, vec, g);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float s = sigmoid(a[e]);
      da[e] = g[e] * u[e] * s * (1.0f + a[e] * (1.0f - s));
      du[e] = g[e] * a[e] * s;
    }
    T* o = dau + row * 2 * F + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e >= n) break;
      ActTraits<T>::store(o + e, da[e]);
      ActTraits<T>::store(o + F + e, du[e]);
    }
  }
}

template <int R, typename T>
void run(const GatedArgs& a, GatedPart part, int grid, hipStream_t st) {
  if (part == GatedPart::kForward)
    gated_tile_kernel<R, T, GatedPart::kForward><<<grid, kT32Threads, 0, st>>>(a);
  else if (part == GatedPart::kDx)
    gated_tile_kernel<R, T, GatedPart::kDx><<<grid, kT32Threads, 0, st>>>(a);
  else
    gated_tile_kernel<R, T, GatedPart::kDw><<<grid, kT32Threads, 0, st>>>(a);
}

}  // namespace

hipError_t launch_gated_tile(const GatedArgs& a, GatedPart part, hipStream_t st) {
  // tiles of 64 while 128 would leave compute units without one
  const int cols = part == GatedPart::kForward ? 2 * a.F : a.d;
  const long long rows = part == GatedPart::kDw ? 2LL * a.F * a.E : a.M;
  const long long large = (rows + 127) / 128 * ((cols + 127) / 128);
  const int grid = 1024;
  if (large >= 256) {
    if (a.bf16) run<2, bf16_t>(a, part, grid, st);
    else run<2, float>(a, part, grid, st);
  } else {
    if (a.bf16) run<1, bf16_t>(a, part, grid, st);
    else run<1, float>(a, part, grid, st);
  }
  return hipGetLastError();
}

hipError_t launch_gated_dau(const GatedArgs& a, hipStream_t st) {
  const int quads = (a.F + 3) / 4;
  const long long blocks = (static_cast<long long>(a.M) * quads + 255) / 256;
  const unsigned grid = static_cast<unsigned>(blocks < 8192 ? blocks : 8192);
  if (a.bf16) gated_dau_kernel<bf16_t><<<grid, 256, 0, st>>>(a, quads);
  else gated_dau_kernel<float><<<grid, 256, 0, st>>>(a, quads);
  return hipGetLastError();
}

}  // namespace moe
