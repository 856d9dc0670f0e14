// Products of groups with few rows: a stream of the weights through the matrix
// cores (e4m3 with block scales; the gated block in bf16 and fp32).
//
// The rows of a group are cut into entries of up to 16.  A unit is an entry and one
// or two tiles of 16 weight rows (gated: with two, 16 rows of Wg and the same 16 of
// Wu, so that a lane ends with a and u of the same column; with one, 8 and 8).  A
// wave walks a unit's K in steps of 128
// bytes a row, lane l taking 32 bytes of row l % 16 of each tile and of the
// activations, straight into registers: RING - 1 steps are in flight, and the next
// unit's first steps are loaded before this one ends.  Where there are fewer units
// than waves, `split` waves of a workgroup share a unit's K and add their sums through
// LDS, in a fixed order.
//
// Bound by the weight loads: nothing is staged, so nothing waits at a barrier in the
// stream.  The matrix instructions take 16 rows whatever there are; e4m3 codes go
// through the bf16 instruction (as bf16 they are exact, and it adds in fp32, which
// v_mfma_f32_16x16x128_f8f6f4 does not): the matrix units are idle most of the time
// all the same.
#include "stream.h"

namespace moe {

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 1024, kWaves = kThreads / 64, kLogWaves = 4;
constexpr int kEntryRows = 16;
constexpr int kStep = 128;  // bytes of a row per step

__device__ const uint4 kZeros16 = {0, 0, 0, 0};

// 32 bytes of a row
struct Piece {
  u32x4_t v[2];
};

__device__ __forceinline__ bf16x8_t fp8_wide(uint32_t lo, uint32_t hi) {
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

// acc[t] += the products of a step; lane l: activation row l % 16, weight rows
// 4 (l / 16) + 0..3 of tile t.
template <StreamKind KIND, int TILES>
__device__ __forceinline__ void multiply(const Piece& a, const Piece (&w)[TILES], float as,
                                         float ws, f32x4_t (&acc)[TILES]) {
  if constexpr (KIND == StreamKind::kFp8) {
    f32x4_t p[TILES] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const bf16x8_t av = fp8_wide(a.v[h][2 * q], a.v[h][2 * q + 1]);
#pragma unroll
        for (int t = 0; t < TILES; ++t)
          p[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              fp8_wide(w[t].v[h][2 * q], w[t].v[h][2 * q + 1]), av, p[t], 0, 0, 0);
      }
    const float s = as * ws;
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(p[t][e], s, acc[t][e]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        if constexpr (KIND == StreamKind::kGatedBf16) {
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_t, w[t].v[h]), __builtin_bit_cast(bf16x8_t, a.v[h]),
              acc[t], 0, 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[t].v[h][e]),
                                                          __uint_as_float(a.v[h][e]), acc[t], 0,
                                                          0, 0);
        }
      }
  }
}

// GROUPED: rows of groups by the offsets; otherwise one group of all M rows, and no
// plan of entries to make first.  RING: steps in registers.
template <StreamKind KIND, bool GROUPED, int TILES, int RING>
__global__ __launch_bounds__(kThreads, 4) void stream_kernel(StreamArgs p, int log_split) {
  constexpr bool GATED = KIND != StreamKind::kFp8;
  constexpr int SIZE = KIND == StreamKind::kFp8 ? 1 : KIND == StreamKind::kGatedBf16 ? 2 : 4;
  constexpr int NOUT = GATED ? 8 * TILES : 16 * TILES;
  __shared__ EntryPlan plan;  // (none where it is not used)
  __shared__ f32x4_t red[kWaves][TILES][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, quad = lane >> 4;
  if constexpr (GROUPED) make_entries<kThreads, kEntryRows>(p, plan);
  const long long ld = static_cast<long long>(p.K) * SIZE;  // bytes of a row
  const int nk = static_cast<int>((ld + kStep - 1) / kStep);
  const int per = (p.N + NOUT - 1) / NOUT;
  const int nb = (p.N + 127) / 128;
  const int entries = GROUPED ? plan.start[p.E] : (p.M + kEntryRows - 1) / kEntryRows;
  // (32 bits hold the units: E N K < 2^40, and no more than 2.5 E entries come here)
  const int units = entries * per, share = units / gridDim.x, rest = units % gridDim.x;
  const int u0 = blockIdx.x * share + min(static_cast<int>(blockIdx.x), rest);
  const int u1 = u0 + share + (static_cast<int>(blockIdx.x) < rest ? 1 : 0);
  // this wave's units: a run of the workgroup's, or every teams-th of them
  const int split = 1 << log_split, teams = kWaves >> log_split;
  const int team = wave >> log_split, part = wave & (split - 1);
  const int first = split == 1 ? u0 + (u1 - u0) * wave / kWaves : u0 + team;
  const int last = split == 1 ? u0 + (u1 - u0) * (wave + 1) / kWaves : u1;
  const int log_stride = split == 1 ? 0 : kLogWaves - log_split, stride = 1 << log_stride;
  const int count = last > first ? (last - first + stride - 1) >> log_stride : 0;
  const int rounds = split == 1 ? 0 : (u1 - u0 + teams - 1) >> log_stride;
  const int s0 = (nk * part) >> log_split;
  const int ns = ((nk * (part + 1)) >> log_split) - s0;

  struct Place {
    int g, tile, rows;
    long long row0;
  };
  auto place = [&](int u) __attribute__((always_inline)) {
    Place q;
    const int ent = entries == 1 ? 0 : u / per;
    q.tile = u - ent * per;
    if constexpr (GROUPED) {
      q.g = entry_group(plan, p.E, ent);
      const int m0 = (ent - plan.start[q.g]) * kEntryRows;
      q.rows = min(plan.rows[q.g] - m0, kEntryRows);
      q.row0 = static_cast<long long>(plan.lo[q.g]) + m0;
    } else {
      q.g = 0;
      q.rows = min(p.M - ent * kEntryRows, kEntryRows);
      q.row0 = static_cast<long long>(ent) * kEntryRows;
    }
    return q;
  };

  if (count > 0) {
    // ---- load side
    int lu = first;
    int ls = 0, lleft = count;
    const char* ap;
    const char* wp[TILES];
    const float *asp = nullptr, *wsp = nullptr;
    int kb;  // byte of K of this lane's piece
    auto enter_load = [&]() __attribute__((always_inline)) {
      const Place q = place(lu);
      const long long row = q.row0 + min(r16, q.rows - 1);
      kb = s0 * kStep + quad * 32;
      ap = static_cast<const char*>(p.a) + row * ld + kb;
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const bool up = GATED && (TILES == 1 ? r16 >= 8 : t == 1);
        const int in = GATED ? (TILES == 1 ? r16 & 7 : r16) : 16 * t + r16;
        const int col = min(q.tile * NOUT + in, p.N - 1);
        wp[t] = static_cast<const char*>(up ? p.w1 : p.w0) +
                (static_cast<long long>(q.g) * p.N + col) * ld + kb;
      }
      if constexpr (!GATED) {
        asp = p.a_scale + row * nk + s0;
        wsp = p.w_scale + (static_cast<long long>(q.g) * nb + q.tile * NOUT / 128) * nk + s0;
      }
      ls = 0;
    };
    enter_load();
    Piece a[RING], w[RING][TILES];
    float as[RING], ws[RING];
    auto load = [&](int s) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // what lies behind the end of a row is another row's, or nobody's
        const bool in = !GATED || kb + 16 * h < ld;
        auto at = [&](const char* b) {
          return *(in ? reinterpret_cast<const u32x4_t*>(b + 16 * h)
                      : reinterpret_cast<const u32x4_t*>(&kZeros16));
        };
        a[s].v[h] = at(ap);
#pragma unroll
        for (int t = 0; t < TILES; ++t) w[s][t].v[h] = at(wp[t]);
      }
      if constexpr (!GATED) {
        as[s] = asp[ls];
        ws[s] = wsp[ls];
      }
      // on to the next step; past the last one the loads are repeated
      if (ls + 1 < ns) {
        ++ls;
        kb += kStep;
        ap += kStep;
#pragma unroll
        for (int t = 0; t < TILES; ++t) wp[t] += kStep;
      } else if (lleft > 1) {
        --lleft;
        lu += stride;
        enter_load();
      }
    };
#pragma unroll
    for (int i = 0; i < RING - 1; ++i) load(i);

    // ---- compute side
    int cu = first;
    int cs = 0;
    f32x4_t acc[TILES] = {};
    const long long total = static_cast<long long>(count) * ns;
    for (long long b = 0; b < total; b += RING) {
#pragma unroll
      for (int i = 0; i < RING; ++i) {
        if (b + i >= total) break;
        load((i + RING - 1) % RING);
        multiply<KIND, TILES>(a[i], w[i], GATED ? 0.0f : as[i], GATED ? 0.0f : ws[i], acc);
        if (++cs < ns) continue;
        cs = 0;
        if (split > 1) {
#pragma unroll
          for (int t = 0; t < TILES; ++t) red[wave][t][lane] = acc[t];
          __syncthreads();
          if (part == 0)
            for (int o = 1; o < split; ++o)
#pragma unroll
              for (int t = 0; t < TILES; ++t) acc[t] += red[wave + o][t][lane];
        }
        if (part == 0) {
          const Place q = place(cu);
          f32x4_t other;  // one tile: lanes 32 to 63 hold u of the columns of lanes 0 to 31
          if constexpr (GATED && TILES == 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) other[e] = __shfl_xor(acc[0][e], 32);
          if (r16 < q.rows) {
            const size_t row = static_cast<size_t>(q.row0) + r16;
            if constexpr (GATED) {
              const int c = q.tile * NOUT + 4 * (TILES == 1 ? quad & 1 : quad);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (c + e >= p.N || (TILES == 1 && quad >= 2)) break;
                const float av = acc[0][e], u = TILES == 1 ? other[e] : acc[TILES - 1][e];
                const float h = av * (1.0f / (1.0f + expf(-av))) * u;
                if (p.out) {
                  if (SIZE == 2) static_cast<bf16_t*>(p.out)[row * p.N + c + e] = f32_to_bf16(h);
                  else static_cast<float*>(p.out)[row * p.N + c + e] = h;
                }
                if (p.pre) {
                  p.pre[row * 2 * p.N + c + e] = av;
                  p.pre[row * 2 * p.N + p.N + c + e] = u;
                }
              }
            } else {
#pragma unroll
              for (int t = 0; t < TILES; ++t) {
                const int c = q.tile * NOUT + 16 * t + 4 * quad;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if (c + e >= p.N) break;
                  if (p.out_bf16) static_cast<bf16_t*>(p.out)[row * p.N + c + e] = f32_to_bf16(acc[t][e]);
                  else static_cast<float*>(p.out)[row * p.N + c + e] = acc[t][e];
                }
              }
            }
          }
        }
        if (split > 1) __syncthreads();  // red is free again
#pragma unroll
        for (int t = 0; t < TILES; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        cu += stride;
      }
    }
  }
  // a team without a unit in the last round takes part in its barriers
  for (int r = count; r < rounds; ++r) {
    __syncthreads();
    __syncthreads();
  }
}

template <StreamKind KIND>
hipError_t run(const StreamArgs& a, hipStream_t st) {
  constexpr bool GATED = KIND != StreamKind::kFp8;
  constexpr int SIZE = KIND == StreamKind::kFp8 ? 1 : KIND == StreamKind::kGatedBf16 ? 2 : 4;
  constexpr int kGrid = 256;
  const long long nk = (static_cast<long long>(a.K) * SIZE + kStep - 1) / kStep;
  // units there may be: an entry for each 16 rows of a group, one at least for each
  // group with rows
  const long long entries = a.E == 1 ? (a.M + 15) / 16 : (a.M < a.E ? a.M : a.E);
  const int cols = GATED ? 8 : 16;
  const bool two = entries * ((a.N + 2 * cols - 1) / (2 * cols)) >= kGrid;
  const long long units = entries * ((a.N + (two ? 2 : 1) * cols - 1) / ((two ? 2 : 1) * cols));
  // waves that share a unit: as many as leave no more than a unit a team, with two
  // steps each at least
  int split = 0;  // as a power of two
  while (split < kLogWaves && (units << (split + 1)) <= static_cast<long long>(kGrid) * kWaves &&
         nk >= 4LL << split)
    ++split;
  const long long teams = kWaves >> split;
  const long long want = (units + teams - 1) / teams;
  const int grid = split == 0 || want > kGrid ? kGrid : static_cast<int>(want);
  if (a.offsets) {
    if (two) stream_kernel<KIND, true, 2, 3><<<grid, kThreads, 0, st>>>(a, split);
    else stream_kernel<KIND, true, 1, 4><<<grid, kThreads, 0, st>>>(a, split);
  } else {
    if (two) stream_kernel<KIND, false, 2, 3><<<grid, kThreads, 0, st>>>(a, split);
    else stream_kernel<KIND, false, 1, 4><<<grid, kThreads, 0, st>>>(a, split);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_stream(const StreamArgs& a, StreamKind kind, hipStream_t st) {
  switch (kind) {
    case StreamKind::kFp8: return run<StreamKind::kFp8>(a, st);
    case StreamKind::kGatedBf16: return run<StreamKind::kGatedBf16>(a, st);
    default: return run<StreamKind::kGatedF32>(a, st);
  }
}

}  // namespace moe
