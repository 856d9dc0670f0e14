// K loop of the large tiles for operands that are contiguous along K or along their
// rows, with ends of K that no step divides (bf16).
//
// Tile, rings and ping-pong are those of big_tile.h.  An operand that is contiguous
// along K lies in LDS as there.  One that is contiguous along its rows (the weights
// of dx = dau W, both operands of dW = dau^T x) lies as [k][row]: a K value's NC rows
// are one LDS line, copied by the same direct loads, and the matrix instruction's
// fragments (8 values of K of a row) are read turned, by two ds_read_b64_tr_b16:
// 16 lanes read 4 K values x 16 rows and each is given one row's 4 values.  Nothing is
// turned round in memory beforehand.
// 16-byte chunk c of line k sits in slot c ^ lines_swz(k): the 4 lines that 16 lanes
// read lie in different quarters of the banks, and those of lanes 32 to 63 (8 lines
// on) in the other half of each.
//
// K runs over up to two segments (dau's two halves against Wg, then Wu), each of
// them `kend` long; values past its end are read from zeros, in both operands, for
// what lies there may be a NaN.
#pragma once

#include "big_tile.h"

namespace moe {

__device__ const uint4 kTileZeros = {0, 0, 0, 0};

__device__ __forceinline__ int lines_swz(int k) { return ((k & 3) << 2) | (((k >> 3) & 1) << 1); }

// Direct global -> LDS loads to an LDS address (as dma16 in ffn_common.h, which takes
// a pointer: turning one into an address costs a comparison with null each time).
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(LDS_PTR(p)));
}
__device__ __forceinline__ void dma16_to(const bf16_t* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(src), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "m0");
}
// From a wave-uniform base and a lane's offset in bytes: one register a load instead
// of two, and the base moves along K for all of them.
__device__ __forceinline__ void dma16_at(const bf16_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "m0");
}
// 4 bytes a lane.
__device__ __forceinline__ void dma4_to(const float* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :
               : "v"(src), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "m0");
}
__device__ __forceinline__ void dma4_at(const float* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "m0");
}

// LDS addresses of the slots of rings that start at lds (operand A's slots first).
template <class C>
__device__ __forceinline__ uint32_t slot_a(uint32_t lds, int i) { return lds + i * C::A_STAGE * 2; }
template <class C>
__device__ __forceinline__ uint32_t slot_b(uint32_t lds, int i) {
  return lds + (C::NSA * C::A_STAGE + i * C::B_STAGE) * 2;
}

// One operand's loads of a wave: up to L of 1 KiB a stage.  kpos: the K value that
// this lane's part of load 0 starts at inside a stage; that of load q follows from
// how the stage is laid out (LINES: K lines a load of an operand that is contiguous
// along its rows, 0: contiguous along K).
template <int L>
struct KtLoads {
  const bf16_t* base;     // wave-uniform
  uint32_t off[L];        // bytes from it to this lane's source at K 0
  int kpos;
  long long kstride;      // elements from one K value to the next
  long long jump;         // elements from the first segment to the second
  int kend;               // K values of a segment
  int nseg;               // steps of a segment
  int first;              // step that the loop begins at
  long long upper;        // TWO: elements from the base of the first half of the
                          // loads to that of the second

  template <int BK, int LW, int LINES, bool TWO>
  __device__ __forceinline__ void issue(int ks, uint32_t slot, int wig) const {
    static_assert(LW <= L && LW % 2 == 0, "loads of a stage");
    ks += first;
    const bool second = ks >= nseg;
    const int k0 = (second ? ks - nseg : ks) * BK;
    const bf16_t* at = base + k0 * kstride + (second ? jump : 0);
    if (k0 + BK <= kend) {
#pragma unroll
      for (int q = 0; q < LW; ++q)
        dma16_at(TWO && q >= LW / 2 ? at + upper : at, off[q], slot + (wig * LW + q) * 1024);
    } else {
#pragma unroll
      for (int q = 0; q < LW; ++q) {
        const int kq = LINES > 0 ? kpos + q * LINES : BK == 64 && (q & 1) ? kpos ^ 8 : kpos;
        const bf16_t* p = k0 + kq < kend
                              ? reinterpret_cast<const bf16_t*>(
                                    reinterpret_cast<const char*>(TWO && q >= LW / 2 ? at + upper : at) +
                                    off[q])
                              : reinterpret_cast<const bf16_t*>(&kTileZeros);
        dma16_to(p, slot + (wig * LW + q) * 1024);
      }
    }
  }
};

// Place of load j (of a stage, 1 KiB) of an operand that is contiguous along its NC
// rows: the K line and the first row that this lane fetches.
template <int NC>
constexpr int kLinesOfLoad = 512 / NC;
template <int NC>
__device__ __forceinline__ void lines_place(int lane, int j, int& k, int& row) {
  constexpr int CH = NC / 8;        // chunks of a line
  k = j * kLinesOfLoad<NC> + lane / CH;
  row = ((lane % CH) ^ lines_swz(k)) * 8;
}

// The fragment of a 32-row block: `off` from lines_off, K substep kk.
template <int NC>
__device__ __forceinline__ int lines_off(int lane, int block) {
  const int i = lane & 15, k = 8 * (lane >> 5) + (i >> 2);
  const int chunk = 4 * block + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
  return k * NC + ((chunk ^ lines_swz(k)) << 3) + 4 * (i & 1);
}
template <int NC>
__device__ __forceinline__ bf16x8_t lines_frag(const bf16_t* s, int off, int kk) {
  typedef short s16x4_t __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4_t* lds_s16x4;
  union {
    s16x4_t half[2];
    bf16x8_t all;
  } u;
#pragma unroll
  for (int t = 0; t < 2; ++t)
    u.half[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (lds_s16x4)LDS_PTR(s + off + (16 * kk + 4 * t) * NC));
  return u.all;
}

// TA, TB: the operand is contiguous along its rows.
template <class C, bool TA, bool TB>
struct KtFrags {
  int offa[TA ? C::BM : C::KK];
  int offb[TB ? C::BN : C::KK];

  template <int GRP>
  __device__ __forceinline__ void init(int lane, int wig) {
    const int r32 = lane & 31;
#pragma unroll
    for (int kk = 0; kk < C::KK; ++kk) {
      const int o = r32 * C::BK + (((2 * kk + (lane >> 5)) ^ row_swz<C>(r32)) << 3);
      if constexpr (!TA) offa[kk] = o;
      if constexpr (!TB) offb[kk] = o;
    }
    if constexpr (TA)
#pragma unroll
      for (int i = 0; i < C::BM; ++i) offa[i] = lines_off<C::MT>(lane, 2 * i + GRP);
    if constexpr (TB)
#pragma unroll
      for (int j = 0; j < C::BN; ++j) offb[j] = lines_off<C::NB>(lane, 2 * wig + j);
  }

  template <int GRP, int NV>
  __device__ __forceinline__ void read(const bf16_t* sA, const bf16_t* sB, int wig,
                                       BigFrags<C>& f) const {
    constexpr int BLK = 32 * C::BK;
#pragma unroll
    for (int kk = 0; kk < C::KK; ++kk) {
#pragma unroll
      for (int j = 0; j < C::BN; ++j) {
        if constexpr (TB) f.b[kk][j] = lines_frag<C::NB>(sB, offb[j], kk);
        else f.b[kk][j] = *reinterpret_cast<const bf16x8_t*>(sB + (wig * 2 + j) * BLK + offb[kk]);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if constexpr (TA) f.a[kk][i] = lines_frag<C::MT>(sA, offa[i], kk);
        else f.a[kk][i] = *reinterpret_cast<const bf16x8_t*>(sA + (2 * i + GRP) * BLK + offa[kk]);
      }
    }
  }
};

template <class C, bool TA, bool TB, int U, int GRP, int NV, class Loads>
__device__ __forceinline__ void kt_step(const Loads& t, const KtFrags<C, TA, TB>& fr, int kt,
                                        int nk, bf16_t* const (&sA)[C::NSA],
                                        bf16_t* const (&sB)[C::NSB], uint32_t lds, int wig,
                                        f32x16_t (&acc)[C::BM][C::BN]) {
  BigFrags<C> f;
  fr.template read<GRP, NV>(sA[U % C::NSA], sB[U % C::NSB], wig, f);
  if constexpr (GRP == 0) {
    const int ks = kt + C::NSB - 1 < nk ? kt + C::NSB - 1 : nk - 1;
    t.template issue<C::BK, C::LPW_B, TB ? kLinesOfLoad<C::NB> : 0, !TB>(ks, slot_b<C>(lds, (U + C::NSB - 1) % C::NSB), wig);
  } else {
    const int ks = kt + C::NSA - 1 < nk ? kt + C::NSA - 1 : nk - 1;
    t.template issue<C::BK, C::LPW_A, TA ? kLinesOfLoad<C::MT> : 0, false>(ks, slot_a<C>(lds, (U + C::NSA - 1) % C::NSA), wig);
  }
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): fragments in registers
  if constexpr (GRP == 1) wait_vm<(C::NSA - 2) * C::LPW_A>();
  lds_barrier();
  big_mfma<C, NV>(f, acc);
  if constexpr (GRP == 0) wait_vm<(C::NSB - 2) * C::LPW_B>();
  lds_barrier();
}

// The sums over nk > 0 steps, for group GRP and NV row blocks that hold rows.
template <class C, bool TA, bool TB, int GRP, int NV, class Loads>
__device__ __forceinline__ void kt_kloop(const Loads& t, int nk, bf16_t* const (&sA)[C::NSA],
                                         bf16_t* const (&sB)[C::NSB], int wave, int lane,
                                         f32x16_t (&acc)[C::BM][C::BN]) {
  const int wig = wave & 3;
  const uint32_t lds = lds_address(sA[0]);
  KtFrags<C, TA, TB> fr;
  fr.template init<GRP>(lane, wig);
  if constexpr (GRP == 0) {
#pragma unroll
    for (int s = 0; s < C::NSB - 1; ++s)
      t.template issue<C::BK, C::LPW_B, TB ? kLinesOfLoad<C::NB> : 0, !TB>(s < nk ? s : nk - 1, slot_b<C>(lds, s), wig);
    wait_vm<(C::NSB - 2) * C::LPW_B>();
  } else {
#pragma unroll
    for (int s = 0; s < C::NSA - 1; ++s)
      t.template issue<C::BK, C::LPW_A, TA ? kLinesOfLoad<C::MT> : 0, false>(s < nk ? s : nk - 1, slot_a<C>(lds, s), wig);
    wait_vm<(C::NSA - 2) * C::LPW_A>();
  }
  lds_barrier();                // point 0: stage 0 complete
  if (GRP == 1) lds_barrier();  // point 1 for group 1
  for (int kt = 0; kt < nk; kt += 6) {
    kt_step<C, TA, TB, 0, GRP, NV>(t, fr, kt, nk, sA, sB, lds, wig, acc);
    if (kt + 1 < nk) kt_step<C, TA, TB, 1, GRP, NV>(t, fr, kt + 1, nk, sA, sB, lds, wig, acc);
    if (kt + 2 < nk) kt_step<C, TA, TB, 2, GRP, NV>(t, fr, kt + 2, nk, sA, sB, lds, wig, acc);
    if (kt + 3 < nk) kt_step<C, TA, TB, 3, GRP, NV>(t, fr, kt + 3, nk, sA, sB, lds, wig, acc);
    if (kt + 4 < nk) kt_step<C, TA, TB, 4, GRP, NV>(t, fr, kt + 4, nk, sA, sB, lds, wig, acc);
    if (kt + 5 < nk) kt_step<C, TA, TB, 5, GRP, NV>(t, fr, kt + 5, nk, sA, sB, lds, wig, acc);
  }
  if (GRP == 0) lds_barrier();
}

template <class C, bool TA, bool TB, int GRP, int NV, class Loads>
__device__ __forceinline__ void kt_kloop_nv(const Loads& t, int nk, bf16_t* const (&sA)[C::NSA],
                                            bf16_t* const (&sB)[C::NSB], int wave, int lane,
                                            int nv, f32x16_t (&acc)[C::BM][C::BN]) {
  if constexpr (NV == 0) {
    kt_kloop<C, TA, TB, GRP, 0>(t, nk, sA, sB, wave, lane, acc);
  } else {
    if (nv == NV) kt_kloop<C, TA, TB, GRP, NV>(t, nk, sA, sB, wave, lane, acc);
    else kt_kloop_nv<C, TA, TB, GRP, NV - 1>(t, nk, sA, sB, wave, lane, nv, acc);
  }
}

}  // namespace moe
