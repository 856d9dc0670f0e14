// Rows of the groups of a grouped product.
#pragma once

#include "common.h"

namespace moe {

// Groups of a grouped product, at most.
constexpr int kMaxGroups = 256;
constexpr int kPlanGroups = kMaxGroups + 2;  // with the shared experts

__device__ __forceinline__ int clampi(int v, int lo, int hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

// First row and row count of group g of a workgroup's thread g (NT threads, as
// many as there are groups): groups 0..E-1 own the rows between their offsets
// (without offsets group 0 owns all M), S more groups T rows each.  Offsets are
// clamped to the M rows there are, and one that is smaller than an offset before
// it counts as that one: no row lies in two groups.
template <int NT, class Args>
__device__ __forceinline__ void group_rows(const Args& p, int& lo, int& n) {
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

// The groups cut into entries of up to MR rows, in LDS.
struct EntryPlan {
  int start[kPlanGroups + 1];  // entries before each group
  int lo[kPlanGroups], rows[kPlanGroups];
};

// Fills the plan (a workgroup of NT threads, one for each of up to GROUPS groups).
template <int NT, int MR, int GROUPS = kPlanGroups, class Args>
__device__ __forceinline__ void make_entries(const Args& p, EntryPlan& s) {
  static_assert(NT >= GROUPS && GROUPS <= kPlanGroups, "a thread per group");
  __shared__ int wsum[NT / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, G = p.E + p.S;
  if (!p.offsets && G == 1) {  // nothing to read or to add up
    if (tid == 0) {
      s.start[0] = 0;
      s.start[1] = static_cast<int>((static_cast<long long>(p.M) + MR - 1) / MR);
      s.lo[0] = 0;
      s.rows[0] = p.M;
    }
    __syncthreads();
    return;
  }
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

}  // namespace moe
