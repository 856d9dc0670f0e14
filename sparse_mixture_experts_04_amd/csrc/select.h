// Selection of the top-k experts of a token by one wave, and its gates
// (shared by the router's kernels and the few-token layer).
#pragma once

#include "common.h"

namespace moe {

// ------------------------------------------------------------- selection

__device__ __forceinline__ bool better(double ka, int ia, double kb, int ib) {
  return ka > kb || (ka == kb && ia < ib);
}

// Lane exchanges of the wave reductions: step STEP returns the value of
// lane l's partner.  Within a row of 16 lanes by DPP (xor 1, xor 2, then
// each 4-lane group against the other half of its 8 lanes, each 8-lane
// group against the other half of its row: lane i <-> 7 - i and 15 - i);
// across rows by the gfx950 permlane swaps (l <-> l ^ 16, l <-> l ^ 32).
// Every pairing is an involution, so after the six steps every lane holds
// the reduction of all 64 (an associative and commutative one, or a sum
// whose order is the same on every lane).  No exchange goes through LDS.
template <int STEP>
__device__ __forceinline__ int lane_xchg(int v, int lane) {
  if constexpr (STEP == 0) {
    return __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, false);   // quad_perm 1,0,3,2
  } else if constexpr (STEP == 1) {
    return __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, false);   // quad_perm 2,3,0,1
  } else if constexpr (STEP == 2) {
    return __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, false);  // row_half_mirror
  } else if constexpr (STEP == 3) {
    return __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, false);  // row_mirror
  } else if constexpr (STEP == 4) {
    // odd rows of the first result hold the even rows' values, and the
    // even rows of the second the odd rows'
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (lane & 16) ? static_cast<int>(r[0]) : static_cast<int>(r[1]);
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (lane & 32) ? static_cast<int>(r[0]) : static_cast<int>(r[1]);
  }
}

template <int STEP>
__device__ __forceinline__ double lane_xchg64(double v, int lane) {
  const long long u = __double_as_longlong(v);
  const int lo = lane_xchg<STEP>(static_cast<int>(u), lane);
  const int hi = lane_xchg<STEP>(static_cast<int>(u >> 32), lane);
  return __longlong_as_double((static_cast<long long>(hi) << 32) |
                              static_cast<unsigned int>(lo));
}

template <int STEP>
__device__ __forceinline__ void argmax_step(double& bk, int& bj, int lane) {
  const double ok = lane_xchg64<STEP>(bk, lane);
  const int oj = lane_xchg<STEP>(bj, lane);
  if (better(ok, oj, bk, bj)) {
    bk = ok;
    bj = oj;
  }
}

// (bk, bj) := the best pair over the wave (descending key, lower number on
// an exact tie: a total order, so the result does not depend on the order
// of the steps), on every lane.
__device__ __forceinline__ void wave_argmax(double& bk, int& bj, int lane) {
  argmax_step<0>(bk, bj, lane);
  argmax_step<1>(bk, bj, lane);
  argmax_step<2>(bk, bj, lane);
  argmax_step<3>(bk, bj, lane);
  argmax_step<4>(bk, bj, lane);
  argmax_step<5>(bk, bj, lane);
}

// Sum over the wave in a fixed order (the same on every lane).
__device__ __forceinline__ double wave_sum(double v, int lane) {
  v += lane_xchg64<0>(v, lane);
  v += lane_xchg64<1>(v, lane);
  v += lane_xchg64<2>(v, lane);
  v += lane_xchg64<3>(v, lane);
  v += lane_xchg64<4>(v, lane);
  v += lane_xchg64<5>(v, lane);
  return v;
}

// Value of a double on a wave-uniform lane.
__device__ __forceinline__ double read_lane64(double v, int src) {
  const long long u = __double_as_longlong(v);
  const int lo = __builtin_amdgcn_readlane(static_cast<int>(u), src);
  const int hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), src);
  return __longlong_as_double((static_cast<long long>(hi) << 32) |
                              static_cast<unsigned int>(lo));
}

// K + 1 rounds of a wave-wide argmax over the candidates the lanes hold:
// candidate j = lane + 64q sits on lane j % 64 (valid[q]; keys, affinities
// s and logits z).  The candidates are numbered in ascending expert id, so
// rank order is descending key with exact ties to the lower number.  Fills,
// on every lane, the numbers, s and z of the K picks and the keys of the
// K + 1 best (the last one for the margin).
template <int K, int Q>
__device__ __forceinline__ void rank_rounds(int lane, const bool (&valid)[Q],
                                            const double (&key)[Q], const double (&sv)[Q],
                                            const double (&zv)[Q], int (&j_sel)[K],
                                            double (&s_sel)[K], double (&z_sel)[K],
                                            double (&k_sel)[K + 1]) {
  bool taken[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) taken[q] = !valid[q];
#pragma unroll
  for (int r = 0; r <= K; ++r) {
    double bk = -INFINITY;
    int bj = 0x7fffffff;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int j = lane + 64 * q;
      if (!taken[q] && better(key[q], j, bk, bj)) {
        bk = key[q];
        bj = j;
      }
    }
    wave_argmax(bk, bj, lane);
    bj = __builtin_amdgcn_readfirstlane(bj);  // the same on every lane
    k_sel[r] = bk;
    if (r < K) {
      const int q = bj >> 6;
      const int owner = bj & 63;
      double my = sv[0], mz = zv[0];
#pragma unroll
      for (int qq = 1; qq < Q; ++qq) {
        my = q == qq ? sv[qq] : my;
        mz = q == qq ? zv[qq] : mz;
      }
      s_sel[r] = read_lane64(my, owner);
      z_sel[r] = read_lane64(mz, owner);
      if (lane == owner) {
#pragma unroll
        for (int qq = 0; qq < Q; ++qq) taken[qq] = taken[qq] || q == qq;
      }
      j_sel[r] = bj;
    }
  }
}

// Gates of the K picks and the S shared experts (s_sh, z_sh: shared expert
// j's affinity and logit on lane j), then the outputs of token t: topk in
// rank order, gates in slot order, margin = key_K - key_(K+1).  Gates:
// s_j / sum s, or exp(logsigmoid(z_j) - logsumexp logsigmoid(z)), over the
// K + S contributors in slot order, times gate_scale.
template <int K, int S>
__device__ __forceinline__ void write_token(int t, int lane, const int (&i_sel)[K],
                                            const double (&s_pick)[K], const double (&z_pick)[K],
                                            double s_sh, double z_sh,
                                            const double (&k_sel)[K + 1],
                                            int32_t* __restrict__ topk, float* __restrict__ gates,
                                            float* __restrict__ margin, bool logsumexp_norm,
                                            double gate_scale) {
  double s_sel[K + S], z_sel[K + S];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    s_sel[j] = s_pick[j];
    z_sel[j] = z_pick[j];
  }
#pragma unroll
  for (int j = 0; j < S; ++j) {
    s_sel[K + j] = read_lane64(s_sh, j);
    z_sel[K + j] = read_lane64(z_sh, j);
  }
  double denom = 0.0;
  if (logsumexp_norm) {
#pragma unroll
    for (int j = 0; j < K + S; ++j) {
      const double z = z_sel[j];  // logsigmoid(z) = min(z, 0) - log1p(exp(-|z|))
      s_sel[j] = fmin(z, 0.0) - log1p(exp(-fabs(z)));
    }
    double m = s_sel[0];
#pragma unroll
    for (int j = 1; j < K + S; ++j) m = fmax(m, s_sel[j]);
#pragma unroll
    for (int j = 0; j < K + S; ++j) denom += exp(s_sel[j] - m);
    const double lse = m + log(denom);
#pragma unroll
    for (int j = 0; j < K + S; ++j) s_sel[j] = exp(s_sel[j] - lse) * gate_scale;
    denom = 1.0;
  } else {
#pragma unroll
    for (int j = 0; j < K + S; ++j) denom += s_sel[j];
    denom /= gate_scale;
  }
  if (lane < K) {
    int id = i_sel[0];
#pragma unroll
    for (int j = 1; j < K; ++j) id = lane == j ? i_sel[j] : id;
    topk[static_cast<size_t>(t) * K + lane] = id;
  }
  if (lane < K + S) {
    double sj = s_sel[0];
#pragma unroll
    for (int j = 1; j < K + S; ++j) sj = lane == j ? s_sel[j] : sj;
    gates[static_cast<size_t>(t) * (K + S) + lane] = static_cast<float>(sj / denom);
  }
  if (margin && lane == 0) margin[t] = static_cast<float>(k_sel[K - 1] - k_sel[K]);
}

__device__ __forceinline__ double sigmoid64(double z) { return 1.0 / (1.0 + exp(-z)); }

}  // namespace moe
