// 8-bit products of groups with up to some 16 rows each: a stream of weight
// tiles through the matrix cores.
//
// The rows of a group are cut into entries of up to 16; the weight tiles of all
// entries (16 weight rows, all of K; GATED: 8 W_gate rows and the 8 W_up rows of
// the same columns) form one list that the workgroups, and the waves inside,
// split evenly.  A wave reads its tiles one after another in the order of
// v_mfma_i32_16x16x64_i8's operand: lane l takes, of row l % 16, 32 bytes of
// each 128-byte step (two fragments; the same bytes of K of the activation rows,
// which lie in LDS), so that every load touches whole 128-byte lines.  The sums
// of a tile end in one wave's registers: no reduction, no barrier in the
// stream.
//
// Bound by the weight loads.  kRing steps of a wave are in registers, all but
// one in flight; loads are issued unconditionally so that the compiler can
// count them; without the non-temporal hint, for the two loads of a step share
// their lines (the experts of T=64, d=7168, F=2048, which now take the 128-row
// tiles, ran on this kernel in 864 us with it and 794 without).  A stream of whole
// weight rows multiplied by v_dot4 needs one LDS byte per weight byte and
// row, this needs one whatever the rows: 8 rows a group, N=K=2048, 256 groups
// 397 against 216 us.  The matrix and vector units are mostly idle.
#include "int8_rows.h"

namespace moe {

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kGridTiles = 256;        // one workgroup per compute unit
constexpr int kEntryRows = 16;
constexpr int kStep = 128;             // bytes of K of a row per step
constexpr int kRing = 4;               // steps in registers
constexpr int kPad = 16;               // bytes between rows in LDS: no bank conflicts
constexpr int kOperBytes = 120 * 1024;
constexpr int kPartTiles = 32;         // tiles of a workgroup between passes over K

template <bool GATED>
__global__ __launch_bounds__(kThreads, 4) void gemm_int8_tiles_kernel(Int8Args p) {
  constexpr int NOUT = GATED ? 8 : 16;  // output columns of a tile
  __shared__ __attribute__((aligned(1024))) char oper[kOperBytes];
  __shared__ i32x4_t part[kPartTiles][64];
  __shared__ EntryPlan plan;
  __shared__ long long src[kEntryRows];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, quad = lane >> 4;
  const int G = p.E + p.S;
  make_entries<kThreads, kEntryRows>(p, plan);
  const int per = (p.N + NOUT - 1) / NOUT;  // tiles of an entry
  const long long list = static_cast<long long>(plan.start[G]) * per;
  const long long end = list * (blockIdx.x + 1) / gridDim.x;

  int staged_entry = -1, staged_k = -1;
  for (long long c = list * blockIdx.x / gridDim.x; c < end;) {
    const int ent = static_cast<int>(c / per);
    const int t0 = static_cast<int>(c - static_cast<long long>(ent) * per);
    const int g = entry_group(plan, G, ent);
    const bool routed = g < p.E;
    const int ge = routed ? g : g - p.E;
    const int row0 = (ent - plan.start[g]) * kEntryRows;
    const int R = min(plan.rows[g] - row0, kEntryRows);
    // bytes of K of a pass: all of it when R rows fit
    const int kmax = (kOperBytes / R - kPad) / kStep * kStep;
    const int kpass = min(p.Kp, kmax);
    const bool whole = kpass == p.Kp;
    const int n = static_cast<int>(min(min(static_cast<long long>(per - t0), end - c),
                                       static_cast<long long>(whole ? per : kPartTiles)));
    const int stride = kpass + kPad;
    const int ta = t0 + n * wave / kWaves, tb = t0 + n * (wave + 1) / kWaves;  // this wave's tiles
    const int8_t* w = GATED && r16 >= 8 ? (routed ? p.w1 : p.ws1) : (routed ? p.w0 : p.ws0);
    const int8_t* wbase = w + static_cast<size_t>(ge) * p.N * p.Kp + quad * 32;
    const float* s0 = (routed ? p.t0 : p.ts0) + static_cast<size_t>(ge) * p.N;
    const float* s1 = GATED ? (routed ? p.t1 : p.ts1) + static_cast<size_t>(ge) * p.N : nullptr;
    void* out = routed ? p.out : p.out_shared;

    for (int k0 = 0; k0 < p.Kp; k0 += kpass) {
      const int kbytes = min(kpass, p.Kp - k0);
      if (staged_entry != ent || staged_k != k0) {
        __syncthreads();
        if (tid < R) src[tid] = source_row<GATED>(p, routed, ge, plan.lo[g], row0 + tid);
        __syncthreads();
        const int pieces = kbytes / 16;
        for (int i = tid; i < R * pieces; i += kThreads) {
          const int r = i / pieces, o = (i - r * pieces) * 16;
          *reinterpret_cast<u32x4_t*>(oper + r * stride + o) = *reinterpret_cast<const u32x4_t*>(
              p.a + src[r] * static_cast<long long>(p.Kp) + k0 + o);
        }
        staged_entry = ent;
        staged_k = k0;
      }
      __syncthreads();
      const int steps = kbytes / kStep, total = (tb - ta) * steps;
      if (total > 0) {
        const char* arow = oper + (r16 < R ? r16 : 0) * stride + quad * 32;
        const float sr = p.a_scale[src[r16 < R ? r16 : 0]];
        u32x4_t f[kRing][2];
        // load side: tile lt, step ls
        int lt = ta, ls = 0;
        auto place = [&](int t) __attribute__((always_inline)) {
          int col = t * NOUT + (GATED ? r16 & 7 : r16);
          col = col < p.N ? col : p.N - 1;
          return reinterpret_cast<const char*>(wbase + static_cast<size_t>(col) * p.Kp + k0);
        };
        const char* lp = place(lt);
        auto load = [&](u32x4_t (&b)[2]) __attribute__((always_inline)) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            b[h] = *reinterpret_cast<const u32x4_t*>(lp + 16 * h);
          if (ls + 1 < steps) {
            ++ls;
            lp += kStep;
          } else if (lt + 1 < tb) {
            ++lt;
            ls = 0;
            lp = place(lt);
          }
        };
#pragma unroll
        for (int i = 0; i < kRing - 1; ++i) load(f[i]);
        i32x4_t acc;
        float sc[4];  // channel scales of this lane's columns, ahead of their use
        int ct = ta, cs = 0;
        auto enter = [&]() __attribute__((always_inline)) {
          const int col = ct * NOUT + (GATED ? 4 * (quad & 1) : 4 * quad);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[e] = (GATED && quad >= 2 ? s1 : s0)[col + e < p.N ? col + e : p.N - 1];
          acc = i32x4_t{0, 0, 0, 0};
          if (k0 > 0) acc = part[ct - t0][lane];
        };
        enter();
        for (int b = 0; b < total; b += kRing) {
#pragma unroll
          for (int i = 0; i < kRing; ++i) {
            if (b + i >= total) break;
            load(f[(i + kRing - 1) % kRing]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const u32x4_t a = *reinterpret_cast<const u32x4_t*>(arow + cs * kStep + 16 * h);
              acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, f[i][h]),
                                                          __builtin_bit_cast(i32x4_t, a), acc, 0, 0,
                                                          0);
            }
            if (++cs < steps) continue;
            // ---- tile done: lane holds weight rows 4 quad + 0..3 of row r16
            cs = 0;
            if (k0 + kbytes < p.Kp) {
              part[ct - t0][lane] = acc;
            } else {
              const int col = ct * NOUT + (GATED ? 4 * (quad & 1) : 4 * quad);
              float v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[e] = static_cast<float>(acc[e]) * (sr * sc[e]);
                if (GATED) {
                  const float up = __shfl_xor(v[e], 32);  // lanes 32-63 hold up
                  v[e] = v[e] / (1.0f + expf(-v[e])) * up;
                }
              }
              if (r16 < R && (!GATED || quad < 2)) {
                const size_t at =
                    (static_cast<size_t>(routed ? plan.lo[g] : ge * p.T) + row0 + r16) * p.N + col;
                const bool vec = p.N % 4 == 0 && col + 4 <= p.N;
                if (!GATED && p.out_bf16) {
                  bf16_t* o = static_cast<bf16_t*>(out) + at;
                  if (vec) {
                    *reinterpret_cast<uint2*>(o) =
                        make_uint2(f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16),
                                   f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16));
                  } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      if (col + e < p.N) o[e] = f32_to_bf16(v[e]);
                  }
                } else {
                  float* o = static_cast<float*>(out) + at;
                  if (vec) {
                    *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
                  } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      if (col + e < p.N) o[e] = v[e];
                  }
                }
              }
            }
            if (++ct < tb) enter();
          }
        }
      }
    }
    c += n;
  }
}

}  // namespace

hipError_t launch_gemm_int8_tiles(const Int8Args& a, bool gated, hipStream_t st) {
  if (gated) gemm_int8_tiles_kernel<true><<<kGridTiles, kThreads, 0, st>>>(a);
  else gemm_int8_tiles_kernel<false><<<kGridTiles, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
