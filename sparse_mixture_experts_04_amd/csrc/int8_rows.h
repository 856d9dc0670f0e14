// Rows of the groups of an 8-bit product.
#pragma once

#include "int8.h"

namespace moe {

constexpr int kPlanGroups = kInt8MaxGroups + 2;  // with the shared experts

__device__ __forceinline__ int clampi(int v, int lo, int hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

// First row and row count of group g of a workgroup's thread g (NT threads, more
// than there are groups).  Offsets are clamped to the M rows there are, and one
// that is smaller than an offset before it counts as that one: no row lies in
// two groups.
template <int NT>
__device__ __forceinline__ void group_rows(const Int8Args& p, int& lo, int& n) {
  __shared__ int wmax[NT / 64];
  const int g = threadIdx.x, lane = g & 63, wave = g >> 6;
  int v = 0, next = 0;
  if (p.offsets && g < p.E) {
    v = clampi(p.offsets[g], 0, p.M);
    next = clampi(p.offsets[g + 1], 0, p.M);
  }
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o);
    if (lane >= o) v = v > u ? v : u;
  }
  if (lane == 63) wmax[wave] = v;
  __syncthreads();
  for (int w = 0; w < wave; ++w) v = v > wmax[w] ? v : wmax[w];
  lo = 0;
  n = 0;
  if (g < p.E) {
    lo = v;
    n = p.offsets ? (next > v ? next - v : 0) : p.M;
  } else if (g < p.E + p.S) {
    n = p.T;
  }
}

// Row of a that row r of a group is (first row lo of the group's rows).
template <bool GATED>
__device__ __forceinline__ long long source_row(const Int8Args& p, bool routed, int ge, int lo,
                                                int r) {
  if (!routed) return GATED ? r : static_cast<long long>(p.M) + static_cast<long long>(ge) * p.T + r;
  return GATED ? clampi(p.sorted_pair[lo + r] / p.k, 0, p.T - 1) : lo + r;
}

// The groups cut into entries of up to MR rows, in LDS.
struct EntryPlan {
  int start[kPlanGroups + 1];  // entries before each group
  int lo[kPlanGroups], rows[kPlanGroups];
};

// Fills the plan (a workgroup of NT >= kPlanGroups threads).
template <int NT, int MR>
__device__ __forceinline__ void make_entries(const Int8Args& p, EntryPlan& s) {
  static_assert(NT >= kPlanGroups, "a thread per group");
  __shared__ int wsum[NT / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, G = p.E + p.S;
  int lo = 0, n = 0;
  group_rows<NT>(p, lo, n);
  const int t = (n + MR - 1) / MR;
  int v = t;
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  if (lane == 63) wsum[wave] = v;
  __syncthreads();
  for (int w = 0; w < wave; ++w) v += wsum[w];
  if (tid < G) {
    s.start[tid] = v - t;
    s.lo[tid] = lo;
    s.rows[tid] = n;
  }
  if (tid == G - 1) s.start[G] = v;
  __syncthreads();
}

// Group of entry ent: the last one that starts at or before it.
__device__ __forceinline__ int entry_group(const EntryPlan& s, int G, int ent) {
  int g = 0;
  for (int hi = G; hi - g > 1;) {
    const int mid = (g + hi) >> 1;
    if (s.start[mid] <= ent) g = mid;
    else hi = mid;
  }
  return g;
}

hipError_t launch_gemm_int8_tiles(const Int8Args& a, bool gated, hipStream_t st);

}  // namespace moe
