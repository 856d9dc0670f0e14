// Gated block and its gradients on the fp32 matrix cores: any sizes, either type.
//
// Three products (gated.h).  Forward: rows of x against 32-row blocks of 16 rows of
// Wg and the same 16 rows of Wu, so that a lane ends with a and u of the same
// columns.  dx: rows of dau, whose 2F values of K meet the rows of Wg, then of Wu.
// dW: columns of dau (rows of the result: F of dWg, then F of dWu) and of x, K the
// rows of the group; a group without rows writes zeros.
#include <algorithm>
#include <cmath>

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

// da and du of a value of a, u and dh, rounded to T: the bf16 matrix instruction takes
// bf16, and two bf16 parts of each (which would hold 16 bits) twice the products of dx
// and dW, 2/3 of a training step's.  Half a step of bf16 on each (2^-8 at most, 0.0017 in
// the mean) beside the same of the result: the gradients' error is 0.0023 on random
// values, 0.0017 without.
template <typename T>
__device__ __forceinline__ void gate_grad(float a, float u, float g, float& da, float& du) {
  const float s = sigmoid(a);
  da = g * u * s * (1.0f + a * (1.0f - s));
  du = g * a * s;
  if constexpr (sizeof(T) == 2) {
    da = __uint_as_float(static_cast<uint32_t>(f32_to_bf16(da)) << 16);
    du = __uint_as_float(static_cast<uint32_t>(f32_to_bf16(du)) << 16);
  }
}

// The same for results of few tiles, where one step after another of a large tile is
// waiting for memory: a workgroup's 8 waves share K of one 32 x 32 block (forward: 32
// rows x 16 columns), each from global memory straight into registers, and add their
// sums through LDS in order.  An instruction's two k are 4 apart (lane / 32), so that
// an operand contiguous along K is read 4 values a lane.
// FROM_PRE: dau is not there, its values are made of pre's and dh's where they are
// used.
constexpr int kSmallWaves = 8;
typedef float SmallSums[kSmallWaves][16][64];

template <GatedPart PART>
__device__ __forceinline__ long long small_items(const GatedArgs& p, const EntryPlan& plan) {
  constexpr int NOUT = PART == GatedPart::kForward ? 16 : 32;
  const int n_tiles = ((PART == GatedPart::kForward ? p.F : p.d) + NOUT - 1) / NOUT;
  return (PART == GatedPart::kDw ? static_cast<long long>(p.E) * ((2 * p.F + 31) / 32)
                                 : static_cast<long long>(plan.start[p.E])) * n_tiles;
}

template <typename T, GatedPart PART, bool FROM_PRE>
__device__ __forceinline__ void small_item(const GatedArgs& p, const EntryPlan& plan, long long it,
                                           SmallSums& red) {
  constexpr bool FWD = PART == GatedPart::kForward, DW = PART == GatedPart::kDw;
  constexpr int NOUT = FWD ? 16 : 32;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r32 = lane & 31, half = lane >> 5;
  const int d = p.d, F = p.F, F2 = 2 * F;
  const int n_tiles = ((FWD ? F : d) + NOUT - 1) / NOUT, m_tiles = (F2 + 31) / 32;
  const T* x = static_cast<const T*>(p.x);
  const T* dau = static_cast<const T*>(p.dau);
  const T* dh = static_cast<const T*>(p.dh);
  auto on4 = [](const void* b) { return reinterpret_cast<uintptr_t>(b) % (4 * sizeof(T)) == 0; };
  const bool vx = d % 4 == 0 && on4(x), vw = d % 4 == 0 && on4(p.w_gate) && on4(p.w_up);
  const bool vd = F % 2 == 0;
  const bool vp = F % 4 == 0 && on4(dh) && reinterpret_cast<uintptr_t>(p.pre) % 16 == 0;

  const int ent = static_cast<int>(it / n_tiles), n0 = static_cast<int>(it % n_tiles) * NOUT;
  const int g = DW ? ent / m_tiles : entry_group(plan, p.E, ent);
  const int m0 = (DW ? ent % m_tiles : ent - plan.start[g]) * 32;
  const int rows = DW ? min(F2 - m0, 32) : min(plan.rows[g] - m0, 32);
  const long long row0 = plan.lo[g];
  const size_t wat = static_cast<size_t>(g) * F * d;
  const T* wg = static_cast<const T*>(p.w_gate) + wat;
  const T* wu = static_cast<const T*>(p.w_up) + wat;
  const int K = FWD ? d : DW ? plan.rows[g] : F2;
  const int chunks = (K + 7) / 8;
  const int c0 = chunks * wave / kSmallWaves, c1 = chunks * (wave + 1) / kSmallWaves;
  // this lane's row and column of the operands
  const long long row = row0 + m0 + min(r32, rows - 1);
  const T* xr = x + row * d;
  const T* wr = (r32 & 16 ? wu : wg) + static_cast<size_t>(min(n0 + (r32 & 15), F - 1)) * d;
  const int mc = min(m0 + r32, F2 - 1), nc = min(n0 + r32, d - 1);
  // value f of [da | du] of a row
  auto grad = [&](long long r, int f) __attribute__((always_inline)) {
    const int c = f < F ? f : f - F;
    float da, du;
    gate_grad<T>(p.pre[r * F2 + c], p.pre[r * F2 + F + c], ActTraits<T>::load(dh + r * F + c), da, du);
    return f < F ? da : du;
  };
  f32x16_t acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
#pragma unroll 4
  for (int c = c0; c < c1; ++c) {
    const int k = c * 8 + 4 * half;
    float a[4], b[4];
    if constexpr (FWD) {
      load4(xr + k, d - k, vx, a);
      load4(wr + k, d - k, vw, b);
    } else if constexpr (!DW) {
      if constexpr (!FROM_PRE) {
        load4(dau + row * F2 + k, F2 - k, vd, a);
      } else if (vp) {
        const int at = k < F ? k : k - F;
        float ga[4], gu[4], gh[4];
        load4(p.pre + row * F2 + at, F - at, true, ga);
        load4(p.pre + row * F2 + F + at, F - at, true, gu);
        load4(dh + row * F + at, F - at, true, gh);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float da, du;
          gate_grad<T>(ga[e], gu[e], gh[e], da, du);
          a[e] = k < F ? da : du;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = k + e < F2 ? grad(row, k + e) : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int f = k + e;
        const T* w = f < F ? wg + static_cast<size_t>(f) * d : wu + static_cast<size_t>(f - F) * d;
        b[e] = f < F2 ? ActTraits<T>::load(w + nc) : 0.0f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = k + e >= K ? 0.0f
               : FROM_PRE ? grad(row0 + k + e, mc)
                          : ActTraits<T>::load(dau + (row0 + k + e) * F2 + mc);
        b[e] = k + e < K ? ActTraits<T>::load(x + (row0 + k + e) * d + nc) : 0.0f;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(b[e], a[e], acc, 0, 0, 0);
  }
  __syncthreads();  // the block before is done with red
#pragma unroll
  for (int r = 0; r < 16; ++r) red[wave][r][lane] = acc[r];
  __syncthreads();
  // thread: lane l's registers r and r + 8 of all waves
  const int r = wave;
  float v[2] = {0.0f, 0.0f};
#pragma unroll
  for (int w = 0; w < kSmallWaves; ++w) {
    v[0] += red[w][r][lane];
    v[1] += red[w][r + 8][lane];
  }
  if (r32 >= rows) return;
  if constexpr (FWD) {
    const int c = n0 + 8 * (r / 4) + 4 * half + r % 4;
    if (c >= F) return;
    const size_t at = static_cast<size_t>(row0 + m0 + r32);
    if (p.h) ActTraits<T>::store(static_cast<T*>(p.h) + at * F + c, v[0] * sigmoid(v[0]) * v[1]);
    if (p.pre) {
      p.pre[at * F2 + c] = v[0];
      p.pre[at * F2 + F + c] = v[1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = n0 + 8 * (r / 4 + 2 * i) + 4 * half + r % 4;
      if (c >= d) continue;
      const int n = m0 + r32;
      T* out = !DW ? static_cast<T*>(p.dx) + static_cast<size_t>(row0 + m0 + r32) * d
               : n < F ? static_cast<T*>(p.dw_gate) + wat + static_cast<size_t>(n) * d
                       : static_cast<T*>(p.dw_up) + wat + static_cast<size_t>(n - F) * d;
      ActTraits<T>::store(out + c, v[i]);
    }
  }
}

template <typename T, GatedPart PART>
__global__ __launch_bounds__(64 * kSmallWaves) void gated_small_kernel(GatedArgs p) {
  __shared__ SmallSums red;
  __shared__ EntryPlan plan;
  make_entries<64 * kSmallWaves, 32, kMaxGroups>(p, plan);
  const long long total = small_items<PART>(p, plan);
  for (long long it = blockIdx.x; it < total; it += gridDim.x)
    small_item<T, PART, false>(p, plan, it, red);
}

// All gradients in one launch.
template <typename T, bool FROM_PRE>
__global__ __launch_bounds__(64 * kSmallWaves) void gated_small_grads_kernel(GatedArgs p) {
  __shared__ SmallSums red;
  __shared__ EntryPlan plan;
  make_entries<64 * kSmallWaves, 32, kMaxGroups>(p, plan);
  const long long dx = p.dx ? small_items<GatedPart::kDx>(p, plan) : 0;
  const long long total = dx + (p.dw_gate ? small_items<GatedPart::kDw>(p, plan) : 0);
  for (long long it = blockIdx.x; it < total; it += gridDim.x) {
    if (it < dx) small_item<T, GatedPart::kDx, FROM_PRE>(p, plan, it, red);
    else small_item<T, GatedPart::kDw, FROM_PRE>(p, plan, it - dx, red);
  }
}

__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(bf16_t* p, const float (&v)[4]) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2(f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16),
                 f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16));
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
      gate_grad<T>(a[e], u[e], g[e], da[e], du[e]);
    }
    T* o = dau + row * 2 * F + c;
    if (vec) {
      store4(o, da);
      store4(o + F, du);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e >= n) break;
        ActTraits<T>::store(o + e, da[e]);
        ActTraits<T>::store(o + F + e, du[e]);
      }
    }
  }
}

template <typename T, GatedPart PART>
void run(const GatedArgs& a, hipStream_t st) {
  // tiles of 64 while 128 would leave compute units without one
  const long long cols = PART == GatedPart::kForward ? 2 * a.F : a.d;
  const long long rows = PART == GatedPart::kDw ? 2LL * a.F * a.E : a.M;
  if ((rows + 127) / 128 * ((cols + 127) / 128) < 256)
    gated_tile_kernel<1, T, PART><<<1024, kT32Threads, 0, st>>>(a);
  else
    gated_tile_kernel<2, T, PART><<<1024, kT32Threads, 0, st>>>(a);
}

template <typename T>
void run(const GatedArgs& a, GatedPart part, hipStream_t st) {
  if (part == GatedPart::kForward) run<T, GatedPart::kForward>(a, st);
  else if (part == GatedPart::kDx) run<T, GatedPart::kDx>(a, st);
  else run<T, GatedPart::kDw>(a, st);
}

// Workgroups for a product's blocks of 32 x 32, of which there are that many at most.
unsigned small_grid(const GatedArgs& a, GatedPart part) {
  const double entries = std::ceil(a.M / 32.0) + (a.E > 1 ? std::min(a.M, a.E) : 0);
  const double blocks = part == GatedPart::kForward ? entries * std::ceil(a.F / 16.0)
                        : part == GatedPart::kDx    ? entries * std::ceil(a.d / 32.0)
                                                    : std::ceil(a.F / 16.0) * a.E * std::ceil(a.d / 32.0);
  return static_cast<unsigned>(std::min(1024.0, blocks));
}

template <typename T>
void run_small(const GatedArgs& a, GatedPart part, hipStream_t st) {
  auto go = [&](auto kernel) { kernel<<<small_grid(a, part), 64 * kSmallWaves, 0, st>>>(a); };
  if (part == GatedPart::kForward) go(gated_small_kernel<T, GatedPart::kForward>);
  else if (part == GatedPart::kDx) go(gated_small_kernel<T, GatedPart::kDx>);
  else go(gated_small_kernel<T, GatedPart::kDw>);
}

}  // namespace

hipError_t launch_gated_tile(const GatedArgs& a, GatedPart part, hipStream_t st) {
  if (a.bf16) run<bf16_t>(a, part, st);
  else run<float>(a, part, st);
  return hipGetLastError();
}

hipError_t launch_gated_small(const GatedArgs& a, GatedPart part, hipStream_t st) {
  if (a.bf16) run_small<bf16_t>(a, part, st);
  else run_small<float>(a, part, st);
  return hipGetLastError();
}

hipError_t launch_gated_small_grads(const GatedArgs& a, bool from_pre, hipStream_t st) {
  const unsigned grid = std::min(1024u, (a.dx ? small_grid(a, GatedPart::kDx) : 0) +
                                           (a.dw_gate ? small_grid(a, GatedPart::kDw) : 0));
  auto go = [&](auto kernel) { kernel<<<grid, 64 * kSmallWaves, 0, st>>>(a); };
  if (a.bf16)
    from_pre ? go(gated_small_grads_kernel<bf16_t, true>) : go(gated_small_grads_kernel<bf16_t, false>);
  else
    from_pre ? go(gated_small_grads_kernel<float, true>) : go(gated_small_grads_kernel<float, false>);
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
