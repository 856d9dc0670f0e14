// Grouped products of e4m3 rows with block scales.
#include "fp8.h"
#include "tile32.h"

namespace moe {

namespace {

template <int R>
__global__ __launch_bounds__(kT32Threads) void gemm_fp8_tile_kernel(Fp8Args p) {
  using C = Tile32<R>;
  __shared__ __attribute__((aligned(16))) typename C::Lds lds;
  __shared__ EntryPlan plan;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1, half = lane >> 5;
  make_entries<kT32Threads, C::N, kMaxGroups>(p, plan);
  const int n_tiles = (p.N + C::N - 1) / C::N, kb = p.Kp / kFp8Block;
  const int nb = (p.N + kFp8Block - 1) / kFp8Block;
  const long long total = static_cast<long long>(plan.start[p.E]) * n_tiles;
  auto four = [](const uint8_t* c, float s, float (&v)[4]) {
    const int w = *reinterpret_cast<const int*>(c);
    v[0] = s * __builtin_amdgcn_cvt_f32_fp8(w, 0);
    v[1] = s * __builtin_amdgcn_cvt_f32_fp8(w, 1);
    v[2] = s * __builtin_amdgcn_cvt_f32_fp8(w, 2);
    v[3] = s * __builtin_amdgcn_cvt_f32_fp8(w, 3);
  };
  for (long long it = blockIdx.x; it < total; it += gridDim.x) {
    const int ent = static_cast<int>(it / n_tiles), n0 = static_cast<int>(it % n_tiles) * C::N;
    const int g = entry_group(plan, p.E, ent);
    const int m0 = (ent - plan.start[g]) * C::N, rows = min(plan.rows[g] - m0, C::N);
    const long long row0 = static_cast<long long>(plan.lo[g]) + m0;
    f32x16_t acc[R][R];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    auto la = [&](int r, int k, float (&v)[4]) {
      const long long row = row0 + min(r, rows - 1);
      four(p.a + row * p.Kp + k, p.a_scale[row * kb + k / kFp8Block], v);
    };
    auto lb = [&](int r, int k, float (&v)[4]) {
      const int n = min(n0 + r, p.N - 1);
      four(p.w + (static_cast<long long>(g) * p.N + n) * p.Kp + k,
           p.w_scale[(static_cast<long long>(g) * nb + n / kFp8Block) * kb + k / kFp8Block], v);
    };
    tile32_product<R, true, true>(lds, p.Kp, la, lb, acc);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = 32 * (R * wm + i) + (lane & 31);
      if (r >= rows) continue;
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int c = n0 + 32 * (R * wn + j) + 8 * (q / 4) + 4 * half + q % 4;
          if (c >= p.N) continue;
          const size_t at = static_cast<size_t>(row0 + r) * p.N + c;
          if (p.out_bf16) static_cast<bf16_t*>(p.out)[at] = f32_to_bf16(acc[i][j][q]);
          else static_cast<float*>(p.out)[at] = acc[i][j][q];
        }
    }
  }
}

}  // namespace

hipError_t launch_gemm_fp8(const Fp8Args& a, hipStream_t st) {
  if (a.M >= 64) return launch_gemm_fp8_big(a, st);
  gemm_fp8_tile_kernel<2><<<1024, kT32Threads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
