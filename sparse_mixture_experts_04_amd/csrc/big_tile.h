// Tile and K loop of the large-batch GEMMs (bf16 experts in ffn_big.hip, 8-bit
// products in gemm_int8.hip).
//
// Elements are counted in 16-bit units: a 16-byte fragment is 8 bf16 values or
// 16 int8 values of K, and the two matrix instructions take their operands in
// the same layout of bytes (32 rows, K piece lane / 32), so one K loop serves
// both.
#pragma once

#include "ffn_common.h"

namespace moe {

typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));
typedef int32_t i32x4v_t __attribute__((ext_vector_type(4)));

struct MmaBf16 {
  using Acc = f32x16_t;
  __device__ static __forceinline__ Acc mul(bf16x8_t b, bf16x8_t a, Acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(b, a, c, 0, 0, 0);
  }
};
struct MmaI8 {
  using Acc = i32x16_t;
  __device__ static __forceinline__ Acc mul(bf16x8_t b, bf16x8_t a, Acc c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4v_t, b),
                                                 __builtin_bit_cast(i32x4v_t, a), c, 0, 0, 0);
  }
};

// Tile shape: MT rows x 256 weight rows, K step BK (64-byte LDS rows for
// BK = 32, 128-byte rows for BK = 64), NSA / NSB ring slots for the two
// operands.
template <int MT_, int BK_, int NSA_, int NSB_, class Op_ = MmaBf16>
struct BigShape {
  using Op = Op_;
  using Acc = typename Op::Acc;
  static constexpr int THREADS = 512;
  static constexpr int WAVES = THREADS / 64;
  static constexpr int MT = MT_;
  static constexpr int NB = 256;
  static constexpr int BK = BK_;
  static constexpr int NSA = NSA_;                    // A (activation) ring slots
  static constexpr int NSB = NSB_;                    // B (weight) ring slots
  static constexpr int BM = MT / 32 / 2;              // row blocks per wave
  static constexpr int BN = 2;                        // column blocks per wave
  static constexpr int KK = BK / 16;                  // MFMA substeps per stage
  static constexpr int CPR = BK / 8;                  // 16-byte chunks per LDS row
  static constexpr int RPL = 64 / CPR;                // LDS rows per 1 KiB load
  static constexpr int A_STAGE = MT * BK;             // bf16 elements of one A stage
  static constexpr int B_STAGE = NB * BK;             // ... and of one B stage
  static constexpr int LPW_A = A_STAGE * 2 / 1024 / (WAVES / 2);  // 1 KiB loads per loading wave
  static constexpr int LPW_B = B_STAGE * 2 / 1024 / (WAVES / 2);
  static constexpr int LPW_MAX = LPW_A > LPW_B ? LPW_A : LPW_B;
  static constexpr int LDS_ELEMS = NSA * A_STAGE + NSB * B_STAGE;
  static_assert((NSB - 2) * LPW_B < 64 && (NSA - 2) * LPW_A < 64, "vmcnt range");
  static_assert(BK == 32 || BK == 64, "LDS row layouts");
  static_assert(6 % NSA == 0 && 6 % NSB == 0, "the K loop is unrolled by 6");
};
// 256-row tiles with K step 32 (the most MFMA work per loaded byte), and
// 128-row tiles with K step 64 for experts of up to ~200 rows: twice the
// bytes per barrier, for groups whose K steps carry few MFMAs.
using BigCfg = BigShape<256, 32, 3, 6>;
using MidCfg = BigShape<128, 64, 3, 3>;
static_assert(BigCfg::MT == BigCfgRows && MidCfg::MT == MidCfgRows, "row tiles");
static_assert(BigCfg::LDS_ELEMS * 2 <= 147456 && MidCfg::LDS_ELEMS * 2 <= 147456, "LDS");

// Slot of chunk c in LDS row r is c ^ row_swz(r).  gfx950 serves a ds_read_b128
// 16 lanes per cycle over 64 banks of 4 bytes (one 256-byte bank row); the
// 16 lanes of a cycle are 4 lane quads whose quad indices within the half
// wave have equal parity (lanes 0-3, 12-15, 20-27 together).  A fragment
// read (lane l: row l % 32, chunk 2kk + l / 32) then touches the 16 slots of
// a bank row exactly once per cycle when row_swz(r) = (r >> 2) & 3 for
// 64-byte rows (measured: no bank-conflict cycles), and with
// row_swz(r) = (r & 7) ^ ((r >> 3) & 1) for 128-byte rows (the layout of
// the 32-row kernel, also measured conflict-free).  Rows of a 32-row block
// differ only above bit 4, so the slot depends on the row inside its block.
template <class C>
__device__ __forceinline__ int row_swz(int row) {
  if constexpr (C::BK == 32) return (row >> 2) & 3;
  else return (row & 7) ^ ((row >> 3) & 1);
}

// Source chunk (in elements) that lane l fetches for load j of a stage: the
// load fills LDS rows RPL*j.. and the lane lands in slot l % CPR of row
// RPL*j + l / CPR, so it fetches chunk (l % CPR) ^ row_swz(that row).
template <class C>
__device__ __forceinline__ int src_chunk(int lane, int j) {
  if constexpr (C::BK == 32) return ((lane & 3) ^ ((lane >> 4) & 3)) * 8;
  else return ((lane & 7) ^ (lane >> 3) ^ (j & 1)) * 8;
}

// Wave group 0 loads the weight (B) tiles, group 1 the activation (A)
// tiles; each wave issues L 1 KiB loads per stage (LPW_B or LPW_A), load
// j = L * (wave % 4) + q filling LDS rows RPL*j.. of its operand's slot.
// KCAT (the fused shared-expert down + combine): K runs over the S shared
// experts one after the other, and from K offset kcat on a load's source
// moves on by `jump` elements (to the next expert's h rows or W_down rows).
template <class C, bool KCAT = false>
struct BigCtx {
  const bf16_t* src[C::LPW_MAX];  // per-lane source of each load (chunk applied)
  long long jump = 0;             // wave-uniform (KCAT only)
  int kcat = 0x7fffffff;

  template <int L>
  __device__ __forceinline__ void issue(int k0, bf16_t* slot, int wig) const {
    long long off = k0;
    if constexpr (KCAT) off += k0 >= kcat ? jump : 0;
#pragma unroll
    for (int q = 0; q < L; ++q) dma16(src[q] + off, slot + (wig * L + q) * 512);
  }
};

// Fragments of one stage for one wave: KK MFMA substeps x (BM row blocks of
// A, 2 column blocks of B).  Row block i of group grp is tile row block
// 2i + grp (groups interleave so a partly filled tile stays balanced).
template <class C>
struct BigFrags {
  bf16x8_t a[C::KK][C::BM];
  bf16x8_t b[C::KK][C::BN];
};

// Fragment reads.  Rows of a 32-row block differ only above bit 4, so the
// swizzle depends only on the lane's row inside the block: one per-lane
// offset per substep (`off[kk]`, in elements) plus a compile-time block
// offset addresses every fragment.  NV is the number of this wave's row
// blocks that hold rows of the tile (a compile-time count, so that the
// reads and MFMAs of a step are straight-line code).
template <class C, int GRP, int NV>
__device__ __forceinline__ void big_read_frags(const bf16_t* sA, const bf16_t* sB, int wn,
                                               const int (&off)[C::KK], BigFrags<C>& f) {
  constexpr int BLK = 32 * C::BK;  // elements of a 32-row block
#pragma unroll
  for (int kk = 0; kk < C::KK; ++kk) {
#pragma unroll
    for (int j = 0; j < C::BN; ++j)
      f.b[kk][j] =
          *reinterpret_cast<const bf16x8_t*>(sB + (wn * 2 + j) * BLK + off[kk]);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      f.a[kk][i] = *reinterpret_cast<const bf16x8_t*>(sA + (2 * i + GRP) * BLK + off[kk]);
  }
}

// The weight fragment is the MFMA's first operand, so each accumulator block
// is the transposed product (output columns down the lane's registers, tile
// rows across lanes): a lane then holds 4 consecutive output columns of one
// row, which the epilogue writes as one 8-byte word.
template <class C, int NV>
__device__ __forceinline__ void big_mfma(const BigFrags<C>& f, typename C::Acc (&acc)[C::BM][C::BN]) {
#pragma unroll
  for (int kk = 0; kk < C::KK; ++kk)
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < C::BN; ++j)
          acc[i][j] = C::Op::mul(f.b[kk][j], f.a[kk][i], acc[i][j]);
}

// The K loop with the two wave groups in ping-pong.  Barrier points are
// numbered 0, 1, 2, ...; group 0 runs memory(j) between points 2j and 2j+1
// and compute(j) between 2j+1 and 2j+2, group 1 the same one point later.
// So on every SIMD one wave issues MFMAs while its partner reads fragments
// and issues loads.
//   memory(j): read stage j's fragments into registers; group 0 issues its
//              share of the B loads of stage j+5 into the B slot of stage
//              j-1, group 1 its share of the A loads of stage j+2 into the
//              A slot of stage j-1 (both groups finished reading those one
//              point earlier); wait for the fragment reads;
//   compute(j): the MFMAs of stage j from registers.
// Before every even point 2j, every wave has waited for its loads of stage
// j (the loads of later stages stay in flight: four for B, one for A), so
// stage j is complete in LDS when group 0 starts reading it.  Weights come
// from HBM with a long latency and get the deep ring; activation rows are
// mostly L2 hits.  A wave's loads complete in issue order, so keeping each
// operand on its own waves lets the B loads run far ahead without the A
// waits depending on them.  Past the last K step the loads repeat the last
// step (L2 hits into slots never read), which keeps the counts uniform.
// GRP (the wave's group) and NV are compile-time, so a step has no
// branches: the MFMAs and fragment reads of a step are straight-line code.
template <class C, int U, bool GATED, int GRP, int NV, class Ctx>
__device__ __forceinline__ void big_pp_step(const Ctx& t, int kt, int nk,
                                            bf16_t* const (&sA)[C::NSA],
                                            bf16_t* const (&sB)[C::NSB], int wig,
                                            const int (&off)[C::KK],
                                            typename C::Acc (&acc)[C::BM][C::BN]) {
  BigFrags<C> f;
  big_read_frags<C, GRP, NV>(sA[U % C::NSA], sB[U % C::NSB], wig, off, f);
  if constexpr (GRP == 0) {
    const int ks = kt + C::NSB - 1 < nk ? kt + C::NSB - 1 : nk - 1;
    t.template issue<C::LPW_B>(ks * C::BK, sB[(U + C::NSB - 1) % C::NSB], wig);
  } else {
    const int ks = kt + C::NSA - 1 < nk ? kt + C::NSA - 1 : nk - 1;
    t.template issue<C::LPW_A>(ks * C::BK, sA[(U + C::NSA - 1) % C::NSA], wig);
  }
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): fragments in registers
  if constexpr (GRP == 1) wait_vm<(C::NSA - 2) * C::LPW_A>();
  lds_barrier();
  big_mfma<C, NV>(f, acc);
  if constexpr (GRP == 0) wait_vm<(C::NSB - 2) * C::LPW_B>();
  lds_barrier();
}

template <class C, bool GATED, int GRP, int NV, class Ctx>
__device__ __forceinline__ void big_kloop(const Ctx& t, int nk,
                                          bf16_t* const (&sA)[C::NSA],
                                          bf16_t* const (&sB)[C::NSB], int wave, int lane,
                                          typename C::Acc (&acc)[C::BM][C::BN]) {
  constexpr int grp = GRP;
  const int wig = wave & 3;
  const int r32 = lane & 31;
  int off[C::KK];
#pragma unroll
  for (int kk = 0; kk < C::KK; ++kk)
    off[kk] = r32 * C::BK + (((2 * kk + (lane >> 5)) ^ row_swz<C>(r32)) << 3);
  if (grp == 0) {
#pragma unroll
    for (int s = 0; s < C::NSB - 1; ++s)
      t.template issue<C::LPW_B>((s < nk ? s : nk - 1) * C::BK, sB[s], wig);
    wait_vm<(C::NSB - 2) * C::LPW_B>();
  } else {
#pragma unroll
    for (int s = 0; s < C::NSA - 1; ++s)
      t.template issue<C::LPW_A>((s < nk ? s : nk - 1) * C::BK, sA[s], wig);
    wait_vm<(C::NSA - 2) * C::LPW_A>();
  }
  lds_barrier();                  // point 0: stage 0 complete
  if (grp == 1) lds_barrier();    // point 1 for group 1 (its phase 0 is idle)
  for (int kt = 0; kt < nk; kt += 6) {
    big_pp_step<C, 0, GATED, GRP, NV>(t, kt, nk, sA, sB, wig, off, acc);
    if (kt + 1 < nk) big_pp_step<C, 1, GATED, GRP, NV>(t, kt + 1, nk, sA, sB, wig, off, acc);
    if (kt + 2 < nk) big_pp_step<C, 2, GATED, GRP, NV>(t, kt + 2, nk, sA, sB, wig, off, acc);
    if (kt + 3 < nk) big_pp_step<C, 3, GATED, GRP, NV>(t, kt + 3, nk, sA, sB, wig, off, acc);
    if (kt + 4 < nk) big_pp_step<C, 4, GATED, GRP, NV>(t, kt + 4, nk, sA, sB, wig, off, acc);
    if (kt + 5 < nk) big_pp_step<C, 5, GATED, GRP, NV>(t, kt + 5, nk, sA, sB, wig, off, acc);
  }
  if (grp == 0) lds_barrier();    // both groups pass the same number of points
}

// The K loop instantiated for the wave's group and its count of row blocks
// holding rows (nv, 0..BM; chosen once per item).
template <class C, bool GATED, int GRP, int NV, class Ctx>
__device__ __forceinline__ void big_kloop_nv(const Ctx& t, int nk, bf16_t* const (&sA)[C::NSA],
                                             bf16_t* const (&sB)[C::NSB], int wave, int lane,
                                             int nv, typename C::Acc (&acc)[C::BM][C::BN]) {
  if constexpr (NV == 0) {
    big_kloop<C, GATED, GRP, 0>(t, nk, sA, sB, wave, lane, acc);
  } else {
    if (nv == NV) big_kloop<C, GATED, GRP, NV>(t, nk, sA, sB, wave, lane, acc);
    else big_kloop_nv<C, GATED, GRP, NV - 1>(t, nk, sA, sB, wave, lane, nv, acc);
  }
}

inline int device_cus_big() {
  int dev = 0, cus = 256;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return 256;
  return cus > 0 ? cus : 256;
}

}  // namespace moe
