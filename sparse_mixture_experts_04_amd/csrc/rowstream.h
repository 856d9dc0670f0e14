// Dot products of streamed weight rows with a few activation rows in LDS.
//
// A wave reads weight rows ("units") as contiguous KiB pieces ("chunks": 16
// bytes per lane), one after another, and multiplies each with the 1 to 8
// activation rows its expert holds; lane partial sums are added over the wave
// at a unit's end (row_totals).  Nothing is shared between waves, so there is no barrier in
// the stream, and the units split evenly over any number of waves.
//
// What bounds it is the rate of the weight loads.  Reading a row in whole KiB
// pieces matters: the matrix cores' fragment order, 16 rows at a time in pieces
// of 64 or 128 bytes, reached 2 to 4 TB/s on the same weights.  A chunk costs 4
// dot instructions per activation row whatever the type (v_dot2_f32_bf16,
// v_dot4_i32_i8, v_fma_f32), 16 cycles of a SIMD's time; at 8 rows that is a
// third of the time the chunk takes to arrive.
//
// kRing blocks of kBlock chunks are held in registers, all but one of them in
// flight.  Loads are issued unconditionally (past the last unit the last block
// is read again) so that the compiler can count them.  Small is fast here: code
// that the weights have driven out of the caches costs 0.4 us per 128 bytes, and
// a register too many (scratch memory) cost the whole kernel 10 to 20%.  Measured
// on the few-token layer, us at T=1 d=2048 F=768 / T=1 d=7168 F=2048 / T=16 there:
// ring 6 of 2 chunks 56 / 174 / 1516, 4 of 2 43 / 152 / 1244, 4 of 1 35 / 145 /
// 1261, and with products of 1, 3 and 8 rows instead of 1, 2, 4 and 8 (and the
// kernel's arguments not held in registers) 30 / 120 / 1192.
#pragma once

#include <type_traits>

#include "select.h"
#include "agent.h"

namespace moe {

constexpr int kChunk = 1024;     // bytes of a row per load instruction
constexpr int kBlock = 1;        // chunks per block
constexpr int kRing = 4;         // blocks in registers
constexpr int kUnitRows = 8;     // activation rows of a unit, at most

struct DotBf16 {
  using Acc = float;
  __device__ static void mul(u32x4_t w, u32x4_t x, float& a) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // through scalars: a bit cast of a vector's element takes element 0
      const uint32_t wi = w[i], xi = x[i];
      a = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, wi),
                                          __builtin_bit_cast(bf16x2_t, xi), a, false);
    }
  }
};
struct DotF32 {
  using Acc = float;
  __device__ static void mul(u32x4_t w, u32x4_t x, float& a) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a = fmaf(__uint_as_float(w[i]), __uint_as_float(x[i]), a);
  }
};
struct DotI8 {
  using Acc = int32_t;
  __device__ static void mul(u32x4_t w, u32x4_t x, int32_t& a) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a = __builtin_amdgcn_sdot4(static_cast<int>(w[i]), static_cast<int>(x[i]), a, false);
  }
};

// Sums over the wave of up to kUnitRows values a lane: lane l gets that of row
// total_row(l).  A swap of half a wave (or of every other 16 lanes) between two
// rows' values makes one value of both, so 8 rows take 10 exchanges instead of
// 48.  Every row is added in the same order, by lanes 32 apart, then 16, then
// within 16, whatever its place and the number of rows.
__device__ __forceinline__ int total_row(int lane) {
  return (lane >> 5 & 1) | (lane >> 3 & 2) | (lane >> 1 & 4);
}
template <class Acc>
__device__ __forceinline__ Acc row_totals(int nr, const Acc (&acc)[kUnitRows], int lane) {
  static_assert(sizeof(Acc) == 4 && kUnitRows == 8, "32-bit sums of 8 rows");
  auto fold32 = [](Acc a, Acc b) __attribute__((always_inline)) {  // a's in the low half, b's in the high
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a),
                                                    __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t x = r[0], y = r[1];
    return __builtin_bit_cast(Acc, x) + __builtin_bit_cast(Acc, y);
  };
  auto fold16 = [](Acc a, Acc b) __attribute__((always_inline)) {  // a's in even rows of 16, b's in odd
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a),
                                                    __builtin_bit_cast(uint32_t, b), false, false);
    const uint32_t x = r[0], y = r[1];
    return __builtin_bit_cast(Acc, x) + __builtin_bit_cast(Acc, y);
  };
  auto other = [&](auto step, Acc v) __attribute__((always_inline)) {
    return __builtin_bit_cast(Acc, lane_xchg<decltype(step)::value>(__builtin_bit_cast(int, v), lane));
  };
  Acc v = fold16(fold32(acc[0], acc[1]), fold32(acc[2], acc[3])), give = v;
  if (nr > 4) {
    const Acc w = fold16(fold32(acc[4], acc[5]), fold32(acc[6], acc[7]));
    give = lane & 8 ? v : w;
    v = lane & 8 ? w : v;
  }
  v += other(std::integral_constant<int, 3>{}, give);
  v += other(std::integral_constant<int, 2>{}, v);
  v += other(std::integral_constant<int, 1>{}, v);
  v += other(std::integral_constant<int, 0>{}, v);
  return v;
}

// The stream of one wave's units.  Walk tells where they are and takes the sums
// (everything but the row offsets is the same on every lane):
//   units()          number of units
//   row(u)           address of the row's first byte of this pass; called with
//                    u = 0, 1, 2, ... in order, each once
//   enter(u, off)    before unit u is multiplied, in order: sets the LDS offsets
//                    of its activation rows (lane's 16 bytes included) and
//                    returns their number
//   leave(u, n, acc) takes the n lane sums of unit u
// begin() issues the first loads; it needs the weights' addresses only, so it
// comes before what the activation rows wait for.  run() does the rest.
// kbytes: bytes of a row in this pass; planes of activation rows lie plane_bytes
// apart (their sums are added).
template <class Dot, int PL, class Walk>
struct RowStream {
  using Acc = typename Dot::Acc;
  u32x4_t w[kRing][kBlock];
  const char* lrow;  // load side: the next block is block lk of unit lu
  int lu, lk, units, kbytes, nkb;

  __device__ __forceinline__ void load(Walk& walk, u32x4_t (&f)[kBlock]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < kBlock; ++j) {
      int o = (lk * kBlock + j) * kChunk + lane * 16;
      o = o < kbytes ? o : 0;  // past the row: any byte of it (times zero)
      f[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(lrow + o));
    }
    if (lk + 1 < nkb) {
      ++lk;
    } else if (lu + 1 < units) {
      ++lu;
      lk = 0;
      lrow = walk.row(lu);
    }
  }

  __device__ __forceinline__ void begin(Walk& walk, int kb) {
    units = walk.units();
    kbytes = kb;
    nkb = (kb + kBlock * kChunk - 1) / (kBlock * kChunk);
    lu = lk = 0;
    if (units <= 0) return;
    lrow = walk.row(0);
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) load(walk, w[i]);
  }

  // Brings the load side of a walk made anew to where begin() left it.
  __device__ __forceinline__ void resume(Walk& walk) {
    for (int u = 1; u <= lu; ++u) walk.row(u);
  }

  __device__ __forceinline__ void run(Walk& walk, const char* oper, int plane_bytes) {
    const int total = units * nkb;
    if (total <= 0) return;
    int cu = 0, ck = 0;
    int off[kUnitRows];
    Acc acc[kUnitRows];
#pragma unroll
    for (int r = 0; r < kUnitRows; ++r) {
      acc[r] = Acc{0};
      off[r] = 0;
    }
    int rows = walk.enter(0, off);
    for (int b = 0; b < total; b += kRing) {
#pragma unroll
      for (int i = 0; i < kRing; ++i) {
        if (b + i >= total) break;
        load(walk, w[(i + kRing - 1) % kRing]);
        auto mul = [&](auto nr) __attribute__((always_inline)) {
          constexpr int N = decltype(nr)::value;
#pragma unroll
          for (int r = 0; r < N; ++r) {
#pragma unroll
            for (int j = 0; j < kBlock; ++j)
#pragma unroll
              for (int p = 0; p < PL; ++p)
                Dot::mul(w[i][j],
                         *reinterpret_cast<const u32x4_t*>(oper + off[r] + p * plane_bytes +
                                                           (ck * kBlock + j) * kChunk),
                         acc[r]);
            // no more than two rows' operands in registers at once
            if (r & 1) __builtin_amdgcn_sched_barrier(0);
          }
        };
        if (rows == 1) mul(std::integral_constant<int, 1>{});
        else if (rows <= 3) mul(std::integral_constant<int, 3>{});
        else mul(std::integral_constant<int, 8>{});
        if (++ck == nkb) {
          walk.leave(cu, rows, acc);
          ck = 0;
#pragma unroll
          for (int r = 0; r < kUnitRows; ++r) acc[r] = Acc{0};
          if (++cu < units) rows = walk.enter(cu, off);
        }
      }
    }
  }
};

}  // namespace moe
