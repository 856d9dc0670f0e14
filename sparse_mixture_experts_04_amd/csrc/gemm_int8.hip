// Grouped products of 8-bit integer rows: y = s_r t_n (q . w), and the SwiGLU
// pair of them for the experts' gate/up half.
//
// The sums are exact in int32 (K <= 131072), so the only rounding is the
// scaling in fp32 and the store.
#include "int8.h"
#include "stream.h"

namespace moe {

// Groups' row tiles of MT rows as an exclusive prefix in LDS (256 threads).
struct RowPlan {
  int start[kInt8MaxGroups + 2 + 1];  // prefix over groups
  int lo[kInt8MaxGroups + 2];         // first row of the group
  int rows[kInt8MaxGroups + 2];
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

// First row and row count of group g (offsets clamped to the M rows there are).
__device__ __forceinline__ void group_rows(const Int8Args& p, int g, int& lo, int& n) {
  if (g >= p.E) {
    lo = 0;
    n = p.T;
  } else if (!p.offsets) {
    lo = 0;
    n = p.M;
  } else {
    lo = clampi(p.offsets[g], 0, p.M);
    n = clampi(p.offsets[g + 1], lo, p.M) - lo;
  }
}

__device__ __forceinline__ void make_row_plan(const Int8Args& p, int MT, RowPlan& s) {
  __shared__ int wsum[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int G = p.E + p.S;
  int base = 0;
  for (int g0 = 0; g0 < G; g0 += 256) {
    const int g = g0 + tid;
    int lo = 0, n = 0;
    if (g < G) group_rows(p, g, lo, n);
    const int t = (n + MT - 1) / MT;
    int v = t;  // inclusive scan over the 256 threads
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(v, o);
      if (lane >= o) v += u;
    }
    if (lane == 63) wsum[wave] = v;
    __syncthreads();
    int before = base;
    for (int w = 0; w < wave; ++w) before += wsum[w];
    if (g < G) {
      s.start[g] = before + v - t;
      s.lo[g] = lo;
      s.rows[g] = n;
    }
    base += wsum[0] + wsum[1] + wsum[2] + wsum[3];
    __syncthreads();
  }
  if (tid == 0) s.start[G] = base;
  __syncthreads();
}

// Tile: up to 16 NT rows of one group x 16 output columns (GATED: 16 gate and
// 16 up rows of weights) or 32 (plain), four waves splitting K.
template <bool GATED, int NT>
__global__ __launch_bounds__(256) void gemm_int8_stream_kernel(Int8Args p) {
  constexpr int CT = 2, W = 4, MT = 16 * NT;
  constexpr int NOUT = GATED ? 16 : 32;
  __shared__ RowPlan plan;
  __shared__ i32x4_t red[W][CT][NT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, piece = (lane >> 4) * 16;
  make_row_plan(p, MT, plan);
  const int G = p.E + p.S;
  const int ncol = (p.N + NOUT - 1) / NOUT;
  const long long total = static_cast<long long>(plan.start[G]) * ncol;
  const int steps = p.Kp / kStepBytes;
  const int s0 = wave * steps / W, s1 = (wave + 1) * steps / W;

  for (long long it = blockIdx.x; it < total; it += gridDim.x) {
    int lo = 0, hi = G;  // last group whose first item is at or before it
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (static_cast<long long>(plan.start[mid]) * ncol <= it) lo = mid;
      else hi = mid;
    }
    const int g = lo;
    const int tiles = plan.start[g + 1] - plan.start[g];
    const int local = static_cast<int>(it - static_cast<long long>(plan.start[g]) * ncol);
    const int n0 = local / tiles * NOUT;       // row tiles inner: they share weights
    const int m0 = local % tiles * MT;
    const int rows = plan.rows[g];
    const bool routed = g < p.E;
    const int ge = routed ? g : g - p.E;

    // this lane's activation row of each row tile (clamped; extra rows are
    // computed and not stored)
    long long arow[NT];
    const char* ap[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      int r = m0 + t * 16 + r16;
      r = r < rows ? r : rows - 1;
      if (!routed) arow[t] = GATED ? r : static_cast<long long>(p.M) + static_cast<long long>(ge) * p.T + r;
      else if (GATED) arow[t] = clampi(p.sorted_pair[plan.lo[g] + r] / p.k, 0, p.T - 1);
      else arow[t] = plan.lo[g] + r;
      ap[t] = reinterpret_cast<const char*>(p.a) + arow[t] * p.Kp +
              static_cast<size_t>(s0) * kStepBytes + piece;
    }
    const char* wp[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int8_t* w = GATED && c == 1 ? (routed ? p.w1 : p.ws1) : (routed ? p.w0 : p.ws0);
      int n = n0 + r16 + (GATED ? 0 : 16 * c);
      n = n < p.N ? n : p.N - 1;
      wp[c] = reinterpret_cast<const char*>(w) + (static_cast<size_t>(ge) * p.N + n) * p.Kp +
              static_cast<size_t>(s0) * kStepBytes + piece;
    }
    i32x4_t acc[CT][NT];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[c][t] = i32x4_t{0, 0, 0, 0};
    stream_dot<OpI8, CT, NT, 4>(wp, ap, s1 - s0, acc);
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int t = 0; t < NT; ++t) red[wave][c][t][lane] = acc[c][t];
    __syncthreads();

    // sums over the waves; wave w finishes output tiles w, w + 4, ...
    const float* t0 = (routed ? p.t0 : p.ts0) + static_cast<size_t>(ge) * p.N;
    const float* t1 = GATED ? (routed ? p.t1 : p.ts1) + static_cast<size_t>(ge) * p.N : nullptr;
    constexpr int OT = GATED ? NT : CT * NT;
#pragma unroll
    for (int o0 = 0; o0 < OT; o0 += W) {
      const int o = o0 + wave;
      if (o >= OT) break;
      const int c = GATED ? 0 : o % CT, t = GATED ? o : o / CT;
      i32x4_t s{0, 0, 0, 0}, u{0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        s += red[w][c][t][lane];
        if (GATED) u += red[w][1][t][lane];
      }
      const int r = m0 + t * 16 + r16;
      if (r >= rows) continue;
      long long ar = 0;
#pragma unroll
      for (int tt = 0; tt < NT; ++tt) ar = tt == t ? arow[tt] : ar;
      const float sr = p.a_scale[ar];
      const size_t orow = routed ? static_cast<size_t>(plan.lo[g]) + r
                                 : static_cast<size_t>(ge) * p.T + r;
      void* out = routed ? p.out : p.out_shared;
      const int n = n0 + 16 * c + 4 * (lane >> 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (n + i >= p.N) break;
        const float v = static_cast<float>(s[i]) * (sr * t0[n + i]);
        if (GATED) {
          const float up = static_cast<float>(u[i]) * (sr * t1[n + i]);
          static_cast<float*>(out)[orow * p.N + n + i] = v / (1.0f + expf(-v)) * up;
        } else if (p.out_bf16) {
          static_cast<bf16_t*>(out)[orow * p.N + n + i] = f32_to_bf16(v);
        } else {
          static_cast<float*>(out)[orow * p.N + n + i] = v;
        }
      }
    }
    __syncthreads();
  }
}

size_t gemm_int8_plan_ints(int groups) { return static_cast<size_t>(groups) + 64; }

hipError_t launch_gemm_int8(const Int8Args& a, bool gated, int32_t* plan, hipStream_t st) {
  (void)plan;
  if (a.M == 0 && (a.S == 0 || a.T == 0)) return hipSuccess;
  const int nout = gated ? 16 : 32;
  // upper bound of the items: every group's last row tile may be partial
  const long long mean = a.M / (a.E > 0 ? a.E : 1);
  const int nt = mean <= 16 ? 1 : mean <= 32 ? 2 : 4;
  const long long ncol = (a.N + nout - 1) / nout;
  const long long tiles = (a.M + 16LL * nt - 1) / (16 * nt) + a.E +
                          static_cast<long long>(a.S) * ((a.T + 16LL * nt - 1) / (16 * nt));
  const long long want = tiles * ncol;
  const unsigned grid = static_cast<unsigned>(want < 2048 ? want : 2048);
  if (gated) {
    if (nt == 1) gemm_int8_stream_kernel<true, 1><<<grid, 256, 0, st>>>(a);
    else if (nt == 2) gemm_int8_stream_kernel<true, 2><<<grid, 256, 0, st>>>(a);
    else gemm_int8_stream_kernel<true, 4><<<grid, 256, 0, st>>>(a);
  } else {
    if (nt == 1) gemm_int8_stream_kernel<false, 1><<<grid, 256, 0, st>>>(a);
    else if (nt == 2) gemm_int8_stream_kernel<false, 2><<<grid, 256, 0, st>>>(a);
    else gemm_int8_stream_kernel<false, 4><<<grid, 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

}  // namespace moe
