// AdamW over many tensors in one launch.
//
//   m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2      (g: gradient times a factor)
//   p' = p (1 - lr wd) - lr (m' / (1 - b1^t)) / (sqrt(v' / (1 - b2^t)) + eps)
//
// The tensors are cut into chunks of 2048 values; a table in device memory, written
// once, has their addresses and the chunks before each, so that one launch serves
// any number of them.  Bound by memory: every value of p, m and v is read and
// written once, g read once, 16 bytes a lane where the addresses allow it.
//
// States in 8 bits: 256 consecutive values share an fp32 scale, the largest of them.
//   m = s sign(c) (c / 127)^2,  c = round(127 sqrt(|m'| / s)),  |c| <= 127
//   v = z (c / 255)^4,          c = round(255 (v' / z)^(1/4)),  1 <= c <= 255 where v' > 0
// Roots spread the codes over the range of a block that matters: neighbours differ by
// 1.6% at its top, and the smallest code stands for 6e-5 of the largest m and 2.4e-10
// of the largest v.  A v that is not 0 never becomes 0, for p divides by its root.
// m' and v' are taken in 64 bits: a code hangs on which side of a border they lie,
// and on a cancelling sum 32 bits would not say.  The root is taken in 32 bits, and
// where it lies within 1/2048 of a border, the border itself decides, in 64 bits
// and without a root: |m'| against s ((k + 1/2) / 127)^2.
#include <cmath>

#include "adamw.h"
#include "int8_quant.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                       // values a thread takes
static_assert(kThreads * kPer == kAdamwChunk, "a chunk a turn");

__global__ void adamw_table_kernel(AdamwBatch b, int first, AdamwTable t, int count) {
  const int i = threadIdx.x;
  if (i < b.n) {
    t.tensors[first + i] = b.tensors[i];
    t.start[first + i] = b.start[i];
  }
  if (i == 0 && first + b.n == count) t.start[count] = b.end;
}

// 8 values at p; n of them exist.
template <typename T>
__device__ __forceinline__ void get8(const T* p, int n, bool vec, float (&v)[8]) {
  uint4 h[sizeof(T) / 2];
  if (vec) hold8<T, true>(p, 8, h);
  else hold8<T, false>(p, n, h);
  values(h, v);
}
template <typename T>
__device__ __forceinline__ void put8(T* p, int n, bool vec, const float (&v)[8]) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = f32_to_bf16(v[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) ActTraits<T>::store(p + i, v[i]);
  }
}
template <typename T>
__device__ __forceinline__ bool on16(const T* p) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// 8 codes at p (a byte each).
__device__ __forceinline__ uint2 get_codes(const uint8_t* p, int n) {
  uint2 w = make_uint2(0u, 0u);
  if (n >= 8) {
    __builtin_memcpy(&w, p, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) reinterpret_cast<uint8_t*>(&w)[i] = p[i];
  }
  return w;
}
__device__ __forceinline__ void put_codes(uint8_t* p, int n, uint2 w) {
  if (n >= 8) {
    __builtin_memcpy(p, &w, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = reinterpret_cast<const uint8_t*>(&w)[i];
  }
}
__device__ __forceinline__ uint32_t code_at(uint2 w, int i) {
  return ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xffu;
}

// Largest over the 32 lanes that hold a block of 256 values.
__device__ __forceinline__ double block_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o));
  return v;
}

// round(levels (x / top)^(1 / P)), P = 2 or 4; inv = 1 / top.
template <int P>
__device__ __forceinline__ int root_code(double x, float top, float inv, float levels) {
  const float r = static_cast<float>(x) * inv;
  const float t = levels * (P == 2 ? sqrtf(r) : sqrtf(sqrtf(r)));
  const float k = floorf(t);
  int c = static_cast<int>(k) + (t - k > 0.5f ? 1 : 0);
  if (fabsf(t - k - 0.5f) < 0x1p-11f) {
    const double h = (static_cast<double>(k) + 0.5) * (static_cast<double>(k) + 0.5);
    const double n = static_cast<double>(levels) * levels;
    const double border = P == 2 ? h : h * h, whole = P == 2 ? n : n * n;
    c = static_cast<int>(k) + (x * whole > border * top ? 1 : 0);
  }
  return min(c, static_cast<int>(levels));
}

struct Rates {
  float decay, lr, inv_c1, inv_c2, eps, b1, b2, a1, a2, factor;
};

template <typename P, typename G, bool BITS8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwTable t, AdamwStep s) {
  __shared__ Rates shared;
  if (threadIdx.x == 0) {
    const double lr = s.lr_dev ? static_cast<double>(*s.lr_dev) : s.lr;
    const double step = static_cast<double>(s.step_dev ? *s.step_dev : s.step);
    shared.decay = static_cast<float>(1.0 - lr * s.weight_decay);
    shared.lr = static_cast<float>(lr);
    shared.inv_c1 = static_cast<float>(1.0 / (1.0 - pow(s.beta1, step)));
    shared.inv_c2 = static_cast<float>(1.0 / (1.0 - pow(s.beta2, step)));
    shared.eps = static_cast<float>(s.eps);
    shared.b1 = static_cast<float>(s.beta1);
    shared.b2 = static_cast<float>(s.beta2);
    shared.a1 = static_cast<float>(1.0 - s.beta1);
    shared.a2 = static_cast<float>(1.0 - s.beta2);
    shared.factor = s.grad_scale ? *s.grad_scale : 1.0f;
  }
  __syncthreads();
  const Rates r = shared;
  if (!(fabsf(r.factor) < INFINITY)) return;  // the whole step is skipped

  const long long total = t.start[t.count];
  const long long end = total * (blockIdx.x + 1) / gridDim.x;
  long long c = total * blockIdx.x / gridDim.x;
  if (c >= end) return;
  int lo = 0, hi = t.count;  // last tensor that starts at or before chunk c
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.start[mid] <= c) lo = mid;
    else hi = mid;
  }
  for (; c < end; ++c) {
    while (t.start[lo + 1] <= c) ++lo;
    const moe_adamw_tensor e = t.tensors[lo];
    const long long at = (c - t.start[lo]) * kAdamwChunk + threadIdx.x * kPer;
    const long long left = e.n - at;
    const int n = left >= kPer ? kPer : left > 0 ? static_cast<int>(left) : 0;
    P* pp = static_cast<P*>(e.p) + at;
    const G* gp = static_cast<const G*>(e.g) + at;
    const bool whole = n == kPer;
    float p[8], g[8], m[8], v[8];
    get8(pp, n, whole && on16(pp), p);
    get8(gp, n, whole && on16(gp), g);
    if constexpr (!BITS8) {
      float* mp = static_cast<float*>(e.m) + at;
      float* vp = static_cast<float*>(e.v) + at;
      get8(mp, n, whole && on16(mp), m);
      get8(vp, n, whole && on16(vp), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float gi = g[i] * r.factor;
        m[i] = r.b1 * m[i] + r.a1 * gi;
        v[i] = r.b2 * v[i] + r.a2 * gi * gi;
      }
      put8(mp, n, whole && on16(mp), m);
      put8(vp, n, whole && on16(vp), v);
    } else {
      uint8_t* mp = static_cast<uint8_t*>(e.m) + at;
      uint8_t* vp = static_cast<uint8_t*>(e.v) + at;
      const long long block = at / kAdamwBlock;
      double md[8], vd[8], mtop = 0.0, vtop = 0.0;
      bool fine = true;
      if (n > 0) {
        const uint2 cm = get_codes(mp, n), cv = get_codes(vp, n);
        const double ms = s.beta1 * (static_cast<double>(e.m_scale[block]) / 16129.0);
        const double vs = s.beta2 * (static_cast<double>(e.v_scale[block]) / 4228250625.0);
        const double a1 = 1.0 - s.beta1, a2 = 1.0 - s.beta2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int km = static_cast<int8_t>(code_at(cm, i));
          const uint32_t kv = code_at(cv, i), kv2 = kv * kv;
          const double gd = i < n ? static_cast<double>(g[i]) * r.factor : 0.0;
          md[i] = ms * (km * (km < 0 ? -km : km)) + a1 * gd;
          vd[i] = vs * static_cast<double>(kv2 * kv2) + a2 * (gd * gd);
          fine = fine && fabs(md[i]) < INFINITY && vd[i] < INFINITY;
          mtop = fmax(mtop, fabs(md[i]));
          vtop = fmax(vtop, vd[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) md[i] = vd[i] = 0.0;
      }
      const float ms = static_cast<float>(block_max(mtop));
      const float vs = static_cast<float>(block_max(vtop));
      // lanes of a block: the half wave
      const uint32_t half = static_cast<uint32_t>(__ballot(!fine) >> (threadIdx.x & 32));
      const bool good = half == 0 && ms < INFINITY && vs < INFINITY;
      uint2 cm = make_uint2(0u, 0u), cv = make_uint2(0u, 0u);
      if (good) {
        const float im = ms > 0.0f ? 1.0f / ms : 0.0f, iv = vs > 0.0f ? 1.0f / vs : 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          int k = root_code<2>(fabs(md[i]), ms, im, 127.0f);
          k = md[i] < 0.0 ? -k : k;
          int q = root_code<4>(vd[i], vs, iv, 255.0f);
          q = vd[i] > 0.0 && q < 1 ? 1 : q;
          (i < 4 ? cm.x : cm.y) |= static_cast<uint32_t>(k & 0xff) << (8 * (i & 3));
          (i < 4 ? cv.x : cv.y) |= static_cast<uint32_t>(q) << (8 * (i & 3));
        }
      }
      if (n > 0) {
        put_codes(mp, n, cm);
        put_codes(vp, n, cv);
        if (threadIdx.x % 32 == 0) {
          e.m_scale[block] = good ? ms : NAN;
          e.v_scale[block] = good ? vs : NAN;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m[i] = static_cast<float>(md[i]);
        v[i] = static_cast<float>(vd[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      p[i] = p[i] * r.decay - r.lr * (m[i] * r.inv_c1) / (sqrtf(v[i] * r.inv_c2) + r.eps);
    put8(pp, n, whole && on16(pp), p);
    if (sizeof(P) == 4 && e.copy) {
      bf16_t* cp = static_cast<bf16_t*>(e.copy) + at;
      put8(cp, n, whole && on16(cp), p);
    }
  }
}

// The fp32 values that 8-bit states stand for.
__global__ __launch_bounds__(kThreads) void adamw_values_kernel(AdamwTable t) {
  const long long total = t.start[t.count];
  const long long end = total * (blockIdx.x + 1) / gridDim.x;
  long long c = total * blockIdx.x / gridDim.x;
  if (c >= end) return;
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.start[mid] <= c) lo = mid;
    else hi = mid;
  }
  for (; c < end; ++c) {
    while (t.start[lo + 1] <= c) ++lo;
    const moe_adamw_tensor e = t.tensors[lo];
    const long long at = (c - t.start[lo]) * kAdamwChunk + threadIdx.x * kPer;
    const long long left = e.n - at;
    const int n = left >= kPer ? kPer : left > 0 ? static_cast<int>(left) : 0;
    if (n == 0) continue;
    const uint2 cm = get_codes(static_cast<const uint8_t*>(e.m) + at, n);
    const uint2 cv = get_codes(static_cast<const uint8_t*>(e.v) + at, n);
    const double ms = static_cast<double>(e.m_scale[at / kAdamwBlock]) / 16129.0;
    const double vs = static_cast<double>(e.v_scale[at / kAdamwBlock]) / 4228250625.0;
    float m[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int km = static_cast<int8_t>(code_at(cm, i));
      const uint32_t kv = code_at(cv, i), kv2 = kv * kv;
      m[i] = static_cast<float>(ms * (km * (km < 0 ? -km : km)));
      v[i] = static_cast<float>(vs * static_cast<double>(kv2 * kv2));
    }
    put8(e.m_values + at, n, n == kPer && on16(e.m_values + at), m);
    put8(e.v_values + at, n, n == kPer && on16(e.v_values + at), v);
  }
}

unsigned grid_of(long long chunks) {
  constexpr long long kMost = 256 * 8;  // 8 workgroups a compute unit
  return static_cast<unsigned>(chunks < kMost ? chunks : kMost);
}

}  // namespace

hipError_t launch_adamw_table(const AdamwBatch& b, int first, const AdamwTable& t,
                              hipStream_t st) {
  adamw_table_kernel<<<1, 64, 0, st>>>(b, first, t, t.count);
  return hipGetLastError();
}

hipError_t launch_adamw(const AdamwTable& t, const AdamwStep& s, long long chunks,
                        bool param_bf16, bool grad_bf16, bool bits8, hipStream_t st) {
  const unsigned grid = grid_of(chunks);
  auto go = [&](auto kernel) { kernel<<<grid, kThreads, 0, st>>>(t, s); };
  if (param_bf16) {
    if (grad_bf16) bits8 ? go(adamw_kernel<bf16_t, bf16_t, true>) : go(adamw_kernel<bf16_t, bf16_t, false>);
    else bits8 ? go(adamw_kernel<bf16_t, float, true>) : go(adamw_kernel<bf16_t, float, false>);
  } else {
    if (grad_bf16) bits8 ? go(adamw_kernel<float, bf16_t, true>) : go(adamw_kernel<float, bf16_t, false>);
    else bits8 ? go(adamw_kernel<float, float, true>) : go(adamw_kernel<float, float, false>);
  }
  return hipGetLastError();
}

hipError_t launch_adamw_values(const AdamwTable& t, long long chunks, hipStream_t st) {
  adamw_values_kernel<<<grid_of(chunks), kThreads, 0, st>>>(t);
  return hipGetLastError();
}

}  // namespace moe
