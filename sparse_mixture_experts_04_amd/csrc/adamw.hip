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
// and on a cancelling sum 32 bits would not say.  The root is taken in 32 bits, within
// 7e-5 of the exact one.  Where one of a lane's codes lies within 1/8192 (1.2e-4) of a
// border, the lane looks at its codes again, and at each within 1/4096 of one the border
// itself decides, in 64 bits and without a root: |m'| against s ((k + 1/2) / 127)^2.
#include <cmath>
#include <type_traits>

#include "adamw.h"
#include "int8_quant.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
// A thread takes two quads of values, 256 values apart: a wave's loads and stores of
// a quad are contiguous, and a quad of a wave is a block of 256 values that share a
// scale.  (Eight values in a row to a lane leave fp32 stores with gaps: the values of
// 604 million 8-bit states took 1.91 ms that way, 1.23 with quads.)
constexpr int kQuads = 2;
static_assert(kThreads * 4 * kQuads == kAdamwChunk && kAdamwBlock == 64 * 4, "a chunk a turn");

__global__ void adamw_table_kernel(AdamwBatch b, int first, AdamwTable t, int count) {
  const int i = threadIdx.x;
  if (i < b.n) {
    t.tensors[first + i] = b.tensors[i];
    t.start[first + i] = b.start[i];
  }
  if (i == 0 && first + b.n == count) t.start[count] = b.end;
}

// Four values as they lie in memory.  FAST: all there and aligned to one access;
// otherwise n of them, one by one.  (The pointers come from the table: without their
// address space a load would wait for LDS too.)
template <typename T> struct Quad;
template <> struct Quad<float> {
  f32x4_t w;
  __device__ __forceinline__ void split(float (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = w[i];
  }
  __device__ __forceinline__ void join(const float (&v)[4]) { w = f32x4_t{v[0], v[1], v[2], v[3]}; }
};
template <> struct Quad<bf16_t> {
  typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
  u32x2_t w;
  __device__ __forceinline__ void split(float (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void join(const float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = f32_to_bf16(v[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(v[2 * i + 1])) << 16);
  }
};
template <> struct Quad<uint8_t> {
  uint32_t w;
};
template <typename T>
using Global = __attribute__((address_space(1))) T;
template <bool FAST, typename T>
__device__ __forceinline__ void get4(const void* from, long long at, int n, Quad<T>& q) {
  const Global<T>* p = (const Global<T>*)from + at;
  if constexpr (FAST) {
    q.w = *(const Global<decltype(q.w)>*)p;
  } else {
    T v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? p[i] : T{0};
    __builtin_memcpy(&q, v, sizeof(q));
  }
}
template <bool FAST, typename T>
__device__ __forceinline__ void put4(void* to, long long at, int n, const Quad<T>& q) {
  Global<T>* p = (Global<T>*)to + at;
  if constexpr (FAST) {
    *(Global<decltype(q.w)>*)p = q.w;
  } else {
    T v[4];
    __builtin_memcpy(v, &q, sizeof(q));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ float get_scale(const float* s, long long at, int n) {
  return n > 0 ? ((const Global<float>*)s)[at / kAdamwBlock] : 0.0f;
}

// k |k| of a signed code, k^4 of an unsigned one, k = byte i of w.  (24-bit products:
// the 32-bit one takes four times as long.)
__device__ __forceinline__ double signed_square(uint32_t w, int i) {
  const int k = static_cast<int8_t>(w >> (8 * i));
  return static_cast<double>(__mul24(k, k < 0 ? -k : k));
}
__device__ __forceinline__ double fourth_power(uint32_t w, int i) {
  const int k = static_cast<int>((w >> (8 * i)) & 0xffu);
  const double k2 = static_cast<double>(__mul24(k, k));
  return k2 * k2;
}

// Largest of a wave's values, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto step = [&](auto ctrl) {
    const uint32_t u = __builtin_amdgcn_update_dpp(0u, v, decltype(ctrl)::value, 0xf, 0xf, true);
    v = u > v ? u : v;
  };
  step(std::integral_constant<int, 0xb1>{});   // lanes 1 apart
  step(std::integral_constant<int, 0x4e>{});   // 2
  step(std::integral_constant<int, 0x141>{});  // 4 (mirrored eights)
  step(std::integral_constant<int, 0x140>{});  // 8 (mirrored sixteens)
  const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  const uint32_t x = a > b ? a : b, y = c > d ? c : d;
  return x > y ? x : y;
}

// t to the nearest integer, in the low bits of the result; `off` collects how far
// from it the values lie.
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
__device__ __forceinline__ float round_low(float t, float& off) {
  const float f = t + kMagic;
  off = fmaxf(off, fabsf(t - (f - kMagic)));
  return f;
}
// A root in 32 bits is within 7e-5 of the exact one (some 2^-22 of it, times 255);
// beyond this distance from its integer the exact one could round otherwise.
constexpr float kNearBorder = 0.5f - 0x1p-13f;
// Scales under this one leave no accuracy to 32-bit roots.
constexpr float kTinyScale = 0x1p-100f;

// round(levels (x / top)^(1 / P)), the border between the two integers around the
// root t deciding.
template <int P>
__device__ __forceinline__ int exact_code(double x, double top, float t, int levels) {
  if (top < kTinyScale) {
    const double r = sqrt(x / top);
    t = static_cast<float>(levels * (P == 2 ? r : sqrt(r)));
  }
  const double k = floor(static_cast<double>(t)), h = (k + 0.5) * (k + 0.5);
  const double n = static_cast<double>(levels) * levels;
  const int c = fabsf(t - static_cast<float>(k) - 0.5f) > 0x1p-12f
                    ? static_cast<int>(rintf(t))
                    : static_cast<int>(k) +
                          (x * (P == 2 ? n : n * n) > (P == 2 ? h : h * h) * top ? 1 : 0);
  return c < levels ? c : levels;
}
// The low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(const float (&f)[4]) {
  const uint32_t a = __float_as_uint(f[0]), b = __float_as_uint(f[1]);
  const uint32_t c = __float_as_uint(f[2]), d = __float_as_uint(f[3]);
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0c0c0400u),
                               __builtin_amdgcn_perm(b, a, 0x0c0c0400u), 0x05040100u);
}

// Walks the chunks of the grid, this workgroup's one in every gridDim.x:
// work.load<FAST>(e, at, n, k) starts the loads of this thread's quad k (values at ..
// at + n of tensor e), work.use<FAST>(e, at, n, k) works on it.  FAST where a chunk is
// whole and work.aligned(e).
template <class Work>
__device__ __forceinline__ void walk_chunks(const AdamwTable& t, Work& work) {
  const long long total = t.start[t.count];
  // wave w of the workgroup takes 512 values of a chunk, lane l its values 4 l ..
  const int in = (threadIdx.x >> 6) * (256 * kQuads) + (threadIdx.x & 63) * 4;
  int lo = 0;  // last tensor that starts at or before chunk c
  for (long long c = blockIdx.x; c < total;) {
    // 64 places at a time: with 300 tensors two loads in turn, not nine
    for (int hi = t.count; hi - lo > 1;) {
      const int step = (hi - lo + 63) / 64, mid = lo + static_cast<int>(threadIdx.x & 63) * step;
      const int below = __popcll(__ballot(mid < hi && t.start[mid] <= c));
      lo += (below - 1) * step;
      hi = lo + step < hi ? lo + step : hi;
    }
    const moe_adamw_tensor e = t.tensors[lo];
    const long long first = t.start[lo], stop = t.start[lo + 1];
    const bool aligned = work.aligned(e);
    for (; c < stop; c += gridDim.x) {
      const long long at = (c - first) * kAdamwChunk + in;
      if (aligned && (c - first + 1) * kAdamwChunk <= e.n) {
#pragma unroll
        for (int k = 0; k < kQuads; ++k) work.template load<true>(e, at + 256 * k, 4, k);
#pragma unroll
        for (int k = 0; k < kQuads; ++k) work.template use<true>(e, at + 256 * k, 4, k);
      } else {
#pragma unroll 1
        for (int k = 0; k < kQuads; ++k) {
          const long long left = e.n - at - 256 * k;
          const int n = left >= 4 ? 4 : left > 0 ? static_cast<int>(left) : 0;
          work.template load<false>(e, at + 256 * k, n, 0);
          work.template use<false>(e, at + 256 * k, n, 0);
        }
      }
    }
  }
}

struct Rates {
  double b1, b2, a1, a2;
  float decay, lr, rate, inv_c1, inv_c2, eps, factor;
  float inv_root_c2;  // of 1 - b2^t's root: v' / (1 - b2^t) itself may pass fp32 where v' does not
};

template <typename P, typename G, bool BITS8>
struct StepWork {
  Rates r;
  Quad<P> hp[kQuads];
  Quad<G> hg[kQuads];
  Quad<float> hm[kQuads], hv[kQuads];
  Quad<uint8_t> hcm[kQuads], hcv[kQuads];
  float hms[kQuads], hvs[kQuads];

  static __device__ __forceinline__ bool aligned(const moe_adamw_tensor& e) {
    const auto on = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
    constexpr size_t kState = BITS8 ? 4 : 16;
    return on(e.p, 4 * sizeof(P)) && on(e.g, 4 * sizeof(G)) && on(e.m, kState) &&
           on(e.v, kState) && on(e.copy, 8);
  }
  template <bool FAST>
  __device__ __forceinline__ void load(const moe_adamw_tensor& e, long long at, int n, int k) {
    get4<FAST>(e.p, at, n, hp[k]);
    get4<FAST>(e.g, at, n, hg[k]);
    if constexpr (!BITS8) {
      get4<FAST>(e.m, at, n, hm[k]);
      get4<FAST>(e.v, at, n, hv[k]);
    } else {
      get4<FAST>(e.m, at, n, hcm[k]);
      get4<FAST>(e.v, at, n, hcv[k]);
      hms[k] = get_scale(e.m_scale, at, n);
      hvs[k] = get_scale(e.v_scale, at, n);
    }
  }
  template <bool FAST>
  __device__ __forceinline__ void use(const moe_adamw_tensor& e, long long at, int n, int k) {
    float p[4], g[4];
    hp[k].split(p);
    hg[k].split(g);
    if constexpr (!BITS8) {
      float m[4], v[4];
      hm[k].split(m);
      hv[k].split(v);
      const float b1 = static_cast<float>(r.b1), a1 = static_cast<float>(r.a1);
      const float b2 = static_cast<float>(r.b2), a2 = static_cast<float>(r.a2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float gi = g[i] * r.factor;
        m[i] = b1 * m[i] + a1 * gi;
        v[i] = b2 * v[i] + a2 * gi * gi;
        p[i] = p[i] * r.decay - r.lr * (m[i] * r.inv_c1) / (sqrtf(v[i]) * r.inv_root_c2 + r.eps);
      }
      hm[k].join(m);
      hv[k].join(v);
      put4<FAST>(e.m, at, n, hm[k]);
      put4<FAST>(e.v, at, n, hv[k]);
    } else {
      const double ma = r.b1 * (static_cast<double>(hms[k]) * (1.0 / 16129.0));
      const double va = r.b2 * (static_cast<double>(hvs[k]) * (1.0 / 4228250625.0));
      const double mb = r.a1 * r.factor, vb = r.a2 * r.factor * r.factor;
      double md[4], vd[4];
      float m[4], v[4];
      // the largest magnitudes of the values rounded to fp32 are the largest values
      // rounded to fp32; what is not finite counts as larger than all others
      uint32_t mtop = 0, vtop = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double gd = static_cast<double>(g[i]);
        md[i] = fma(ma, signed_square(hcm[k].w, i), mb * gd);
        vd[i] = fma(va, fourth_power(hcv[k].w, i), vb * (gd * gd));
        m[i] = static_cast<float>(md[i]);
        v[i] = static_cast<float>(vd[i]);
        const uint32_t mu = __float_as_uint(m[i]) & 0x7fffffffu;
        const uint32_t vu = __float_as_uint(v[i]) & 0x7fffffffu;
        mtop = i < n && mu > mtop ? mu : mtop;
        vtop = i < n && vu > vtop ? vu : vtop;
      }
      mtop = wave_max(mtop);
      vtop = wave_max(vtop);
      const bool good = mtop < kNotFinite && vtop < kNotFinite;
      const float ms = __uint_as_float(mtop), vs = __uint_as_float(vtop);
      const float im = 1.0f / fmaxf(ms, kTinyScale), iv = 1.0f / fmaxf(vs, kTinyScale);
      float tm[4], tv[4], fm[4], fv[4], den[4], off = 0.0f, least = INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tm[i] = 127.0f * __builtin_amdgcn_sqrtf(fabsf(m[i]) * im);
        tv[i] = 255.0f * __builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf(v[i] * iv));
        fm[i] = round_low(copysignf(tm[i], m[i]), off);
        fv[i] = round_low(tv[i], off);
        fv[i] = vd[i] > 0.0 ? fmaxf(fv[i], kMagic + 1.0f) : fv[i];
        den[i] = __builtin_amdgcn_sqrtf(v[i] * r.inv_c2) + r.eps;
        least = fminf(least, den[i]);
      }
      float upd[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) upd[i] = m[i] * r.rate * __builtin_amdgcn_rcpf(den[i]);
      // near a border, a scale or a denominator that the short forms do not reach
      const bool far = (ms < kTinyScale && ms > 0.0f) || (vs < kTinyScale && vs > 0.0f) ||
                       !(vs * r.inv_c2 < INFINITY);
      if (off > kNearBorder || far || least < 0x1p-50f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = ms > 0.0f ? exact_code<2>(fabs(md[i]), ms, tm[i], 127) : 0;
          fm[i] = kMagic + static_cast<float>(md[i] < 0.0 ? -c : c);
          const int q = vs > 0.0f ? exact_code<4>(vd[i], vs, tv[i], 255) : 0;
          fv[i] = kMagic + static_cast<float>(vd[i] > 0.0 && q < 1 ? 1 : q);
          upd[i] = r.lr * (m[i] * r.inv_c1) / (sqrtf(v[i]) * r.inv_root_c2 + r.eps);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = p[i] * r.decay - upd[i];
      hcm[k].w = good ? low_bytes(fm) : 0u;
      hcv[k].w = good ? low_bytes(fv) : 0u;
      put4<FAST>(e.m, at, n, hcm[k]);
      put4<FAST>(e.v, at, n, hcv[k]);
      if (n > 0 && threadIdx.x % 64 == 0) {
        e.m_scale[at / kAdamwBlock] = good ? ms : NAN;
        e.v_scale[at / kAdamwBlock] = good ? vs : NAN;
      }
    }
    hp[k].join(p);
    put4<FAST>(e.p, at, n, hp[k]);
    if (sizeof(P) == 4 && e.copy) {
      Quad<bf16_t> copy;
      copy.join(p);
      put4<FAST>(e.copy, at, n, copy);
    }
  }
};

template <typename P, typename G, bool BITS8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamwTable t, AdamwStep s) {
  __shared__ Rates shared;
  if (threadIdx.x == 0) {
    const double lr = s.lr_dev ? static_cast<double>(*s.lr_dev) : s.lr;
    double c1 = s.c1, c2 = s.c2;
    if (s.step_dev) {
      const double step = static_cast<double>(*s.step_dev);
      c1 = 1.0 - pow(s.beta1, step);
      c2 = 1.0 - pow(s.beta2, step);
    }
    shared.b1 = s.beta1;
    shared.b2 = s.beta2;
    shared.a1 = 1.0 - s.beta1;
    shared.a2 = 1.0 - s.beta2;
    shared.decay = static_cast<float>(1.0 - lr * s.weight_decay);
    shared.lr = static_cast<float>(lr);
    shared.rate = static_cast<float>(lr / c1);
    shared.inv_c1 = static_cast<float>(1.0 / c1);
    shared.inv_c2 = static_cast<float>(1.0 / c2);
    shared.inv_root_c2 = static_cast<float>(1.0 / sqrt(c2));
    shared.eps = static_cast<float>(s.eps);
    shared.factor = s.grad_scale ? *s.grad_scale : 1.0f;
  }
  __syncthreads();
  StepWork<P, G, BITS8> work;
  work.r = shared;
  if (!(fabsf(work.r.factor) < INFINITY)) return;  // the whole step is skipped

  walk_chunks(t, work);
}

// The fp32 values that 8-bit states stand for.
struct ValuesWork {
  Quad<uint8_t> cm[kQuads], cv[kQuads];
  float ms[kQuads], vs[kQuads];

  static __device__ __forceinline__ bool aligned(const moe_adamw_tensor& e) {
    return ((reinterpret_cast<uintptr_t>(e.m) | reinterpret_cast<uintptr_t>(e.v)) & 3) == 0 &&
           ((reinterpret_cast<uintptr_t>(e.m_values) | reinterpret_cast<uintptr_t>(e.v_values)) & 15) == 0;
  }
  template <bool FAST>
  __device__ __forceinline__ void load(const moe_adamw_tensor& e, long long at, int n, int k) {
    get4<FAST>(e.m, at, n, cm[k]);
    get4<FAST>(e.v, at, n, cv[k]);
    ms[k] = get_scale(e.m_scale, at, n);
    vs[k] = get_scale(e.v_scale, at, n);
  }
  template <bool FAST>
  __device__ __forceinline__ void use(const moe_adamw_tensor& e, long long at, int n, int k) {
    if (!e.m_values) return;  // a tensor without a place for them
    const double ma = static_cast<double>(ms[k]) * (1.0 / 16129.0);
    const double va = static_cast<double>(vs[k]) * (1.0 / 4228250625.0);
    float m[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = static_cast<float>(ma * signed_square(cm[k].w, i));
      v[i] = static_cast<float>(va * fourth_power(cv[k].w, i));
    }
    Quad<float> q;
    q.join(m);
    put4<FAST>(e.m_values, at, n, q);
    q.join(v);
    put4<FAST>(e.v_values, at, n, q);
  }
};

__global__ __launch_bounds__(kThreads) void adamw_values_kernel(AdamwTable t) {
  ValuesWork work;
  walk_chunks(t, work);
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
