// 8-bit products of groups with few rows: a stream of weight rows
// (rowstream.h).
//
// The rows of a group are cut into entries of up to 8; the columns of all
// entries form one list, which the workgroups split evenly.  A workgroup stages
// the codes of an entry's rows in LDS, its waves read the weight rows of the
// entry's columns that lie in its part of the list, and the exact int32 sums
// are scaled (GATED: SwiGLU applied) and stored when the columns are done.
#include "int8_rows.h"
#include "rowstream.h"

namespace moe {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kGridRows = 256;      // one workgroup per compute unit
constexpr int kPartUnits = 1024;    // weight rows between two epilogues
constexpr int kOperBytes = 96 * 1024;

// n columns from column c on; units are weight rows: column c + u, or (GATED)
// W_gate and W_up rows of column c + u / 2 in turn.
template <bool GATED>
struct ColumnWalk {
  const char *r0, *r1;  // next W (or W_gate) row, next W_up row
  size_t kfull;
  int n, rows, stride;
  int32_t (*part)[kUnitRows];
  bool more;            // not the first pass over K: add
  __device__ __forceinline__ int units() const { return GATED ? 2 * n : n; }
  __device__ __forceinline__ const char* row(int u) {
    if (GATED) {
      if (u & 1) return r1;
      if (u > 0) {
        r0 += kfull;
        r1 += kfull;
      }
    } else if (u > 0) {
      r0 += kfull;
    }
    return r0;
  }
  __device__ __forceinline__ int enter(int u, int (&off)[kUnitRows]) {
    if (u == 0) {
#pragma unroll
      for (int r = 0; r < kUnitRows; ++r)
        off[r] = (r < rows ? r : 0) * stride + (threadIdx.x & 63) * 16;
    }
    return rows;
  }
  __device__ __forceinline__ void leave(int u, int nr, const int32_t (&acc)[kUnitRows]) {
#pragma unroll
    for (int r = 0; r < kUnitRows; ++r) {
      if (r >= nr) break;
      const int32_t s = wave_total(acc[r]);
      if ((threadIdx.x & 63) == 0) part[u][r] = more ? part[u][r] + s : s;
    }
  }
};

template <bool GATED>
__global__ __launch_bounds__(kThreads, 4) void gemm_int8_rows_kernel(Int8Args p) {
  constexpr int UPC = GATED ? 2 : 1;  // units per column
  constexpr int kCols = kPartUnits / UPC;
  __shared__ __attribute__((aligned(1024))) char oper[kOperBytes];
  __shared__ int32_t part[kPartUnits][kUnitRows];
  __shared__ EntryPlan plan;
  __shared__ long long src[kUnitRows];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = p.E + p.S;

  make_entries<kThreads, kUnitRows>(p, plan);
  const long long list = static_cast<long long>(plan.start[G]) * p.N;
  const long long end = list * (blockIdx.x + 1) / gridDim.x;
  const size_t kfull = p.Kp;
  const int kall = (p.Kp + kChunk - 1) / kChunk;

  int staged_entry = -1, staged_k = -1;
  for (long long c = list * blockIdx.x / gridDim.x; c < end;) {
    const int ent = static_cast<int>(c / p.N);
    const int col = static_cast<int>(c - static_cast<long long>(ent) * p.N);
    const int g = entry_group(plan, G, ent);
    const bool routed = g < p.E;
    const int ge = routed ? g : g - p.E;
    const int r0 = (ent - plan.start[g]) * kUnitRows;
    const int R = min(plan.rows[g] - r0, kUnitRows);
    const int n = static_cast<int>(min(min(static_cast<long long>(p.N - col), end - c),
                                       static_cast<long long>(kCols)));
    const int kpass = min((kall + 1) / 2 * 2, kOperBytes / kChunk / R / 2 * 2);
    const int stride = kpass * kChunk;
    for (int k0 = 0; k0 < kall; k0 += kpass) {
      const int kbytes = static_cast<int>(min(kfull - static_cast<size_t>(k0) * kChunk,
                                              static_cast<size_t>(stride)));
      if (staged_entry != ent || staged_k != k0) {
        __syncthreads();
        if (tid < R) src[tid] = source_row<GATED>(p, routed, ge, plan.lo[g], r0 + tid);
        __syncthreads();
        const int pieces = stride / 16;
        for (int i = tid; i < R * pieces; i += kThreads) {
          const int r = i / pieces, o = (i - r * pieces) * 16;
          u32x4_t v{0, 0, 0, 0};
          if (o < kbytes)
            v = *reinterpret_cast<const u32x4_t*>(p.a + src[r] * static_cast<long long>(kfull) +
                                                  static_cast<size_t>(k0) * kChunk + o);
          *reinterpret_cast<u32x4_t*>(oper + r * stride + o) = v;
        }
        staged_entry = ent;
        staged_k = k0;
      }
      __syncthreads();
      const int a = n * wave / kWaves, b = n * (wave + 1) / kWaves;
      const size_t at = (static_cast<size_t>(ge) * p.N + col + a) * kfull +
                        static_cast<size_t>(k0) * kChunk;
      ColumnWalk<GATED> walk;
      walk.r0 = reinterpret_cast<const char*>(routed ? p.w0 : p.ws0) + at;
      walk.r1 = GATED ? reinterpret_cast<const char*>(routed ? p.w1 : p.ws1) + at : nullptr;
      walk.kfull = kfull;
      walk.n = b - a;
      walk.rows = R;
      walk.stride = stride;
      walk.part = part + a * UPC;
      walk.more = k0 > 0;
      stream_rows<DotI8, 1>(walk, kbytes, oper, 0);
    }
    __syncthreads();
    const float* t0 = (routed ? p.t0 : p.ts0) + static_cast<size_t>(ge) * p.N + col;
    const float* t1 = GATED ? (routed ? p.t1 : p.ts1) + static_cast<size_t>(ge) * p.N + col : nullptr;
    for (int i = tid; i < R * n; i += kThreads) {
      const int r = i / n, j = i - r * n;
      const float sr = p.a_scale[src[r]];
      const size_t at = (static_cast<size_t>(routed ? plan.lo[g] : ge * p.T) + r0 + r) * p.N + col + j;
      void* out = routed ? p.out : p.out_shared;
      const float v = static_cast<float>(part[j * UPC][r]) * (sr * t0[j]);
      if (GATED) {
        const float up = static_cast<float>(part[j * UPC + (UPC - 1)][r]) * (sr * t1[j]);
        static_cast<float*>(out)[at] = v / (1.0f + expf(-v)) * up;
      } else if (p.out_bf16) {
        static_cast<bf16_t*>(out)[at] = f32_to_bf16(v);
      } else {
        static_cast<float*>(out)[at] = v;
      }
    }
    __syncthreads();  // part is free again
    c += n;
  }
}

}  // namespace

hipError_t launch_gemm_int8_rows(const Int8Args& a, bool gated, hipStream_t st) {
  if (gated) gemm_int8_rows_kernel<true><<<kGridRows, kThreads, 0, st>>>(a);
  else gemm_int8_rows_kernel<false><<<kGridRows, kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
