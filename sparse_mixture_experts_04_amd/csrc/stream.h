// Products of few activation rows with streamed weight rows, shared by the
// 8-bit decode GEMMs and the few-token layer.
//
// One wave multiplies CT tiles of 16 weight rows with NT tiles of 16
// activation rows over a range of K.  Both operands come straight from global
// memory in matrix-core fragment order: on the 16x16 instructions lane l
// holds, of row l % 16, the 16 bytes of K piece l / 16, so one load of 16
// bytes per lane covers 64 bytes (a "step") of 16 rows whatever the element
// type:
//   bf16   8 values  one  v_mfma_f32_16x16x32_bf16
//   int8  16 values  one  v_mfma_i32_16x16x64_i8
//   fp32   4 values  four v_mfma_f32_16x16x4_f32 (value j of every lane)
// The order of K inside a step is the same for both operands, so any lane to
// K assignment gives the same product.  The weights are read once and never
// again: their loads carry the non-temporal hint.  What bounds such a kernel
// is the rate of these loads, so each wave keeps a block of U steps in flight
// while it multiplies the block before.
#pragma once

#include "common.h"

namespace moe {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));

struct OpBf16 {
  using Acc = f32x4_t;
  using Val = float;
  __device__ static void mul(u32x4_t w, u32x4_t a, Acc& acc) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w),
                                                  __builtin_bit_cast(bf16x8_t, a), acc, 0, 0, 0);
  }
};
struct OpI8 {
  using Acc = i32x4_t;
  using Val = int32_t;
  __device__ static void mul(u32x4_t w, u32x4_t a, Acc& acc) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, w),
                                                __builtin_bit_cast(i32x4_t, a), acc, 0, 0, 0);
  }
};
struct OpF32 {
  using Acc = f32x4_t;
  using Val = float;
  __device__ static void mul(u32x4_t w, u32x4_t a, Acc& acc) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[j]), __uint_as_float(a[j]),
                                                 acc, 0, 0, 0);
  }
};

constexpr int kStepBytes = 64;  // K bytes of a row that one step covers

// Data that workgroups of one launch hand to each other: the eight XCDs have an
// L2 each, so it is written through to memory and read past the caches (relaxed
// accesses at agent scope).  One release or acquire fence instead writes back
// or drops a whole L2: with one of each per wave such fences took 150 us of a
// 1024-wave kernel here.
__device__ __forceinline__ void agent_store(uint64_t* p, uint64_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void agent_store(float* p, float v) {
  __hip_atomic_store(reinterpret_cast<uint32_t*>(p), __float_as_uint(v), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void agent_store(int32_t* p, int32_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t agent_load(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float agent_load(const float* p) {
  return __uint_as_float(__hip_atomic_load(reinterpret_cast<const uint32_t*>(p), __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT));
}
__device__ __forceinline__ int32_t agent_load(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// An activation fragment (AGENT: written by another workgroup of this launch).
template <bool AGENT>
__device__ __forceinline__ u32x4_t load_a(const char* p) {
  if constexpr (AGENT) {
    const uint64_t* q = reinterpret_cast<const uint64_t*>(p);
    const uint64_t lo = agent_load(q), hi = agent_load(q + 1);
    return u32x4_t{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32),
                   static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
  } else {
    return *reinterpret_cast<const u32x4_t*>(p);
  }
}

// Fragments of U consecutive steps.
template <int CT, int NT, int U>
struct StreamBlock {
  u32x4_t w[U][CT];
  u32x4_t a[U][NT];
};

template <int CT, int NT, int U, bool AGENT>
__device__ __forceinline__ void stream_load_step(const char* const (&wp)[CT],
                                                 const char* const (&ap)[NT], size_t off, int u,
                                                 StreamBlock<CT, NT, U>& f) {
#pragma unroll
  for (int c = 0; c < CT; ++c)
    f.w[u][c] = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4_t*>(wp[c] + off + u * kStepBytes));
#pragma unroll
  for (int t = 0; t < NT; ++t)
    f.a[u][t] = load_a<AGENT>(ap[t] + off + u * kStepBytes);
}

// Loads the steps s..s+U-1 that lie below n (per-lane pointers to step 0).
template <int CT, int NT, int U, bool AGENT>
__device__ __forceinline__ void stream_load(const char* const (&wp)[CT],
                                            const char* const (&ap)[NT], int s, int n,
                                            StreamBlock<CT, NT, U>& f) {
  const size_t off = static_cast<size_t>(s) * kStepBytes;
  if (n - s >= U) {
#pragma unroll
    for (int u = 0; u < U; ++u) stream_load_step<CT, NT, U, AGENT>(wp, ap, off, u, f);
  } else {
#pragma unroll
    for (int u = 0; u < U - 1; ++u)
      if (s + u < n) stream_load_step<CT, NT, U, AGENT>(wp, ap, off, u, f);
  }
}

template <class Op, int CT, int NT, int U>
__device__ __forceinline__ void stream_mul(const StreamBlock<CT, NT, U>& f, int steps,
                                           typename Op::Acc (&acc)[CT][NT]) {
  if (steps >= U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int t = 0; t < NT; ++t) Op::mul(f.w[u][c], f.a[u][t], acc[c][t]);
  } else {
#pragma unroll
    for (int u = 0; u < U - 1; ++u) {
      if (u < steps) {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int t = 0; t < NT; ++t) Op::mul(f.w[u][c], f.a[u][t], acc[c][t]);
      }
    }
  }
}

// acc[c][t] += W tile c times A tile t over n steps (n >= 0, the same on
// every lane).  Lane l of acc[c][t] holds weight rows 4 (l / 16) + 0..3 of
// activation row l % 16.
template <class Op, int CT, int NT, int U, bool AGENT = false>
__device__ __forceinline__ void stream_dot(const char* const (&wp)[CT],
                                           const char* const (&ap)[NT], int n,
                                           typename Op::Acc (&acc)[CT][NT]) {
  if (n <= 0) return;
  StreamBlock<CT, NT, U> f0, f1;
  stream_load<CT, NT, U, AGENT>(wp, ap, 0, n, f0);
  for (int s = 0;;) {
    if (s + U < n) stream_load<CT, NT, U, AGENT>(wp, ap, s + U, n, f1);
    stream_mul<Op, CT, NT, U>(f0, n - s, acc);
    s += U;
    if (s >= n) break;
    if (s + U < n) stream_load<CT, NT, U, AGENT>(wp, ap, s + U, n, f0);
    stream_mul<Op, CT, NT, U>(f1, n - s, acc);
    s += U;
    if (s >= n) break;
  }
}

}  // namespace moe
