// e4m3 products for large batches.
//
// Tiles of 128 rows x 256 weight rows with the operand rings and the two wave groups
// in ping-pong of big_tile.h (K steps of 128 codes = 64 16-bit units, three slots
// each), or of 256 x 256 with two slots and one barrier a step (below).  A K step is
// one block of the scales.  The matrix instruction
// (v_mfma_f32_32x32x64_f8f6f4, twice the bf16 rate) starts each block's sum at
// zero, and the block joins the running sum by one fused multiply-add a value with
// s_row s_column: 16 of them (64 cycles) beside two instructions of 64, on the
// vector unit that the partner wave leaves idle.
//
// That instruction adds 8 consecutive products with 13 bits behind the exponent of the
// largest, each cut towards zero to a multiple of 2^(x - 13) (x: the largest sum of two
// codes' exponents among the 8, as measured; sums of 8 are added in fp32).  What 8 lose
// is less than 7 * 2^-13 of the largest of them: 1.4e-5 of a result on random values
// (2-norm, K = 128, 1024 and 7168), at most a quarter of the half step of a bf16 y where
// products do not cancel, any part of y where they do.  A bf16 y takes it, at twice the
// rate; an fp32 y takes the bf16 instruction on the codes as bf16 (exact; 1.4e-7 at
// K = 7168), and so do few rows of either type (blocks.hip).
//
// The scales travel like the operands: each wave of the activation group loads, per
// step, 32 row scales and the two weight scales of the tile into the stage's slot by
// one 4-byte direct-to-LDS load, so that no load of theirs disturbs the count of
// loads in flight.
#include <algorithm>
#include <cmath>

#include "fp8.h"
#include "tile_kt.h"

namespace moe {

namespace {

using MidF8 = BigShape<128, 64, 3, 3>;
using BigF8 = BigShape<256, 64, 2, 2>;
typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kScaleSlot = 8 * 64;  // floats: waves x (32 rows, 2 weight blocks, rest unused)

// 64 codes of K; the fragment's pieces of K are the same ones for both operands.
__device__ __forceinline__ f32x16_t mul64(i32x8_t b, i32x8_t a, f32x16_t c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, 0, 0, 0, 0, 0, 0);
}

// Has the sums made here and now: the compiler would put the additions off to the end
// of the loop and keep every block's p in registers until then.
__device__ __forceinline__ void pin(f32x16_t& v) {
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    float x = v[r];
    asm volatile("" : "+v"(x));
    v[r] = x;
  }
}

// Eight codes of a fragment (words 2q and 2q + 1) as bf16, which holds every e4m3
// value.
__device__ __forceinline__ bf16x8_t wide8(i32x8_t f, int q) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  union {
    bf16x2_t pair[4];
    bf16x8_t all;
  } u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    u.pair[2 * i] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * q + i], 1.0f, false);
    u.pair[2 * i + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[2 * q + i], 1.0f, true);
  }
  return u.all;
}

// The loads of a wave of the 128-row tiles: B's for group 0, A's and the scales' for
// group 1, from a wave-uniform base.
template <class C>
struct MidLoads {
  const bf16_t* base;
  uint32_t off[C::LPW_MAX];  // bytes from it to this lane's source of each load
  const float* scale;        // this lane's scale of step 0 (activation group)

  template <int L>
  __device__ __forceinline__ void issue(int ks, uint32_t slot, int wig) const {
#pragma unroll
    for (int q = 0; q < L; ++q)
      dma16_at(base + ks * C::BK, off[q], slot + (wig * L + q) * 1024);
  }
};

template <class C, bool FAST, int U, int GRP, int NV>
__device__ __forceinline__ void f8_step(const MidLoads<C>& c, uint32_t lds, uint32_t scales, int kt, int nk,
                                        bf16_t* const (&sA)[C::NSA], bf16_t* const (&sB)[C::NSB],
                                        float* sS, int wig, int lane, const int (&off)[C::KK],
                                        f32x16_t (&acc)[C::BM][C::BN]) {
  constexpr int BLK = 32 * C::BK;
  constexpr int NM = NV > 0 ? NV : 1;
  constexpr int H = C::KK / 2;
  i32x8_t a[H][NM], b[H][C::BN];
  float s[NM];
  const bf16_t* pa = sA[U % C::NSA];
  const bf16_t* pb = sB[U % C::NSB];
  const float* ps = sS + U % C::NSA * kScaleSlot;
  auto frag = [&](const bf16_t* blk, int h) __attribute__((always_inline)) {
    union {
      bf16x8_t half[2];
      i32x8_t all;
    } u;
    u.half[0] = *reinterpret_cast<const bf16x8_t*>(blk + off[2 * h]);
    u.half[1] = *reinterpret_cast<const bf16x8_t*>(blk + off[2 * h + 1]);
    return u.all;
  };
#pragma unroll
  for (int h = 0; h < H; ++h) {
#pragma unroll
    for (int j = 0; j < C::BN; ++j) b[h][j] = frag(pb + (wig * 2 + j) * BLK, h);
#pragma unroll
    for (int i = 0; i < NV; ++i) a[h][i] = frag(pa + (2 * i + GRP) * BLK, h);
  }
  // row block 2i + grp lies with wave 2i + grp's 32 scales; the two weight blocks
  // (128 columns each) behind the first wave's
  const float sw = ps[32 + (wig >> 1)];
#pragma unroll
  for (int i = 0; i < NV; ++i) s[i] = ps[(2 * i + GRP) * 64 + (lane & 31)] * sw;
  if constexpr (GRP == 0) {
    const int ks = kt + C::NSB - 1 < nk ? kt + C::NSB - 1 : nk - 1;
    c.template issue<C::LPW_B>(ks, slot_b<C>(lds, (U + C::NSB - 1) % C::NSB), wig);
  } else {
    const int ks = kt + C::NSA - 1 < nk ? kt + C::NSA - 1 : nk - 1;
    c.template issue<C::LPW_A>(ks, slot_a<C>(lds, (U + C::NSA - 1) % C::NSA), wig);
    dma4_to(c.scale + ks, scales + ((U + C::NSA - 1) % C::NSA * kScaleSlot + wig * 64) * 4);
  }
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): fragments in registers
  if constexpr (GRP == 1) wait_vm<(C::NSA - 2) * (C::LPW_A + 1)>();
  lds_barrier();
  if constexpr (FAST && NV > 0) {
    // block n's instructions between the two halves of block n - 1's additions, so
    // that the matrix unit does not wait for the vector unit
    constexpr int NBLK = NV * C::BN;
    static_assert(H == 2, "two instructions a block");
    f32x16_t p[2];
    auto join = [&](int n, int r0) __attribute__((always_inline)) {
#pragma unroll
      for (int r = r0; r < r0 + 8; ++r)
        acc[n / C::BN][n % C::BN][r] = fmaf(p[n & 1][r], s[n / C::BN], acc[n / C::BN][n % C::BN][r]);
    };
#pragma unroll
    for (int n = 0; n < NBLK; ++n) {
      p[n & 1] = mul64(b[0][n % C::BN], a[0][n / C::BN], f32x16_t{});
      __builtin_amdgcn_sched_barrier(0);
      if (n > 0) join(n - 1, 0);
      __builtin_amdgcn_sched_barrier(0);
      p[n & 1] = mul64(b[1][n % C::BN], a[1][n / C::BN], p[n & 1]);
      __builtin_amdgcn_sched_barrier(0);
      if (n > 0) {
        join(n - 1, 8);
        pin(acc[(n - 1) / C::BN][(n - 1) % C::BN]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    join(NBLK - 1, 0);
    join(NBLK - 1, 8);
    pin(acc[NV - 1][C::BN - 1]);
  } else if constexpr (NV > 0) {
    // a column block at a time (both at once do not fit in the registers)
#pragma unroll
    for (int j = 0; j < C::BN; ++j) {
      f32x16_t p[NM] = {};
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bf16x8_t wb = wide8(b[h][j], q);
#pragma unroll
          for (int i = 0; i < NV; ++i)
            p[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb, wide8(a[h][i], q), p[i], 0, 0, 0);
        }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = fmaf(p[i][r], s[i], acc[i][j][r]);
        pin(acc[i][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if constexpr (GRP == 0) wait_vm<(C::NSB - 2) * C::LPW_B>();
  lds_barrier();
}

template <class C, bool FAST, int GRP, int NV>
__device__ __forceinline__ void f8_kloop(const MidLoads<C>& c, uint32_t lds, uint32_t scales, int nk,
                                         bf16_t* const (&sA)[C::NSA],
                                         bf16_t* const (&sB)[C::NSB], float* sS, int wave,
                                         int lane, f32x16_t (&acc)[C::BM][C::BN]) {
  static_assert(C::NSA == 3 && C::NSB == 3, "unrolled by 3");
  const int wig = wave & 3, r32 = lane & 31;
  int off[C::KK];
#pragma unroll
  for (int kk = 0; kk < C::KK; ++kk)
    off[kk] = r32 * C::BK + (((2 * kk + (lane >> 5)) ^ row_swz<C>(r32)) << 3);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int ks = s < nk ? s : nk - 1;
    if constexpr (GRP == 0) {
      c.template issue<C::LPW_B>(ks, slot_b<C>(lds, s), wig);
    } else {
      c.template issue<C::LPW_A>(ks, slot_a<C>(lds, s), wig);
      dma4_to(c.scale + ks, scales + (s * kScaleSlot + wig * 64) * 4);
    }
  }
  if constexpr (GRP == 0) wait_vm<C::LPW_B>();
  else wait_vm<C::LPW_A + 1>();
  lds_barrier();                // point 0: stage 0 complete
  if (GRP == 1) lds_barrier();  // point 1 for group 1
  for (int kt = 0; kt < nk; kt += 3) {
    f8_step<C, FAST, 0, GRP, NV>(c, lds, scales, kt, nk, sA, sB, sS, wig, lane, off, acc);
    if (kt + 1 < nk) f8_step<C, FAST, 1, GRP, NV>(c, lds, scales, kt + 1, nk, sA, sB, sS, wig, lane, off, acc);
    if (kt + 2 < nk) f8_step<C, FAST, 2, GRP, NV>(c, lds, scales, kt + 2, nk, sA, sB, sS, wig, lane, off, acc);
  }
  if (GRP == 0) lds_barrier();
}

template <class C, bool FAST, int GRP, int NV>
__device__ __forceinline__ void f8_kloop_nv(const MidLoads<C>& c, uint32_t lds, uint32_t scales, int nk,
                                            bf16_t* const (&sA)[C::NSA],
                                            bf16_t* const (&sB)[C::NSB], float* sS, int wave,
                                            int lane, int nv, f32x16_t (&acc)[C::BM][C::BN]) {
  if constexpr (NV == 0) {
    f8_kloop<C, FAST, GRP, 0>(c, lds, scales, nk, sA, sB, sS, wave, lane, acc);
  } else {
    if (nv == NV) f8_kloop<C, FAST, GRP, NV>(c, lds, scales, nk, sA, sB, sS, wave, lane, acc);
    else f8_kloop_nv<C, FAST, GRP, NV - 1>(c, lds, scales, nk, sA, sB, sS, wave, lane, nv, acc);
  }
}

// ------------------------------------------------------------- 256-row tiles
//
// Twice the products for 4/3 of the 128-row tile's bytes.  Each wave owns 128 rows x
// 64 columns and walks its four row blocks with two sets of fragments of A in turn;
// two slots an operand, one barrier a step: behind it stage j is there (each wave has
// waited for its own loads) and nobody reads stage j - 1 any more, whose slot takes
// stage j + 1 while this one is multiplied.
struct F8Loads {
  const bf16_t* a;       // (all wave-uniform) tile's first row, first weight row
  const bf16_t* b;
  const float* a_scale;  // scales of the tile's first row
  const float* w_scale;  // of this wave's 64 weight rows
  int last_a, last_b;    // last row there is
  uint32_t ld;           // bytes of a row
};

__device__ __forceinline__ float sload_f32(const float* p, int i) {
  typedef const float __attribute__((address_space(4)))* scalar_f32;
  return ((scalar_f32)p)[__builtin_amdgcn_readfirstlane(i)];
}

template <class C, int NV>
__device__ __forceinline__ void f8b_kloop(const F8Loads& t, int nk, uint32_t lds,
                                          uint32_t scales, const float* sS, int wave, int lane,
                                          f32x16_t (&acc)[C::BM][C::BN]) {
  constexpr int BLK = 32 * C::BK, H = C::KK / 2;
  static_assert(H == 2 && C::BM == 4 && C::BN == 2, "256 x 256, 128 codes");
  const int r32 = lane & 31, wm = wave >> 2, wn = wave & 3;
  // LDS addresses of this lane's pieces in slot 0, row block wm of A and column block
  // 2 wn of B: what else an address has is a constant that the load instruction adds
  typedef const bf16x8_t __attribute__((address_space(3)))* lds_piece;
  uint32_t at_a[C::KK], at_b[C::KK];
#pragma unroll
  for (int kk = 0; kk < C::KK; ++kk) {
    const uint32_t o = 2 * (r32 * C::BK + (((2 * kk + (lane >> 5)) ^ row_swz<C>(r32)) << 3));
    at_a[kk] = slot_a<C>(lds, 0) + wm * BLK * 2 + o;
    at_b[kk] = slot_b<C>(lds, 0) + wn * BLK * 4 + o;
  }
  auto frag = [&](const uint32_t (&at)[C::KK], uint32_t more, int h) __attribute__((always_inline)) {
    union {
      bf16x8_t half[2];
      i32x8_t all;
    } u;
    u.half[0] = *(lds_piece)(at[2 * h] + more);
    u.half[1] = *(lds_piece)(at[2 * h + 1] + more);
    return u.all;
  };
  // Load q (0 to 8) of a stage.  Offsets are made where they are used (two
  // instructions; nine registers would not fit): row 64 w' + 8 q + lane / 8 of an
  // operand, chunk as src_chunk has it.
  int lrow = wave * 32 + (lane >> 3);
  const uint32_t chunk = ((lane & 7) ^ (lane >> 3)) * 16;
  auto load = [&](int ks, int slot, int q) __attribute__((always_inline)) {
    ks = ks < nk ? ks : nk - 1;  // past the end: again, into a slot nobody reads
    if (q < 8) {
      const int r = min(lrow + 8 * (q & 3), q < 4 ? t.last_a : t.last_b);
      const uint32_t at = __umul24(r, t.ld) + (chunk ^ ((q & 1) << 4));
      dma16_at((q < 4 ? t.a : t.b) + ks * C::BK, at,
               (q < 4 ? slot_a<C>(lds, slot) : slot_b<C>(lds, slot)) + (wave * 4 + (q & 3)) * 1024);
    } else {
      dma4_at(t.a_scale + ks, 4u * __umul24(min(wave * 32 + r32, t.last_a), nk),
              scales + (slot * kScaleSlot + wave * 64) * 4);
    }
  };
  float sw = sload_f32(t.w_scale, 0);
  auto step = [&](int kt, int slot) __attribute__((always_inline)) {
    i32x8_t b[H][2], a[2][H];
    float s[2];
    asm volatile("" : "+v"(lrow));  // (keeps the offsets from being made, and kept, before the loop)
    wait_vm<0>();
    lds_barrier();
    auto read_a = [&](int i) __attribute__((always_inline)) {
#pragma unroll
      for (int h = 0; h < H; ++h) a[i & 1][h] = frag(at_a, slot * C::A_STAGE * 2 + i * BLK * 4, h);
      s[i & 1] = sS[slot * kScaleSlot + (2 * i + wm) * 64 + r32] * sw;
    };
    if (NV > 0) {
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) b[h][j] = frag(at_b, slot * C::B_STAGE * 2 + j * BLK * 2, h);
      read_a(0);
    }
    if (NV > 1) read_a(1);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      // (the other wave of the SIMD has the matrix unit while this one adds)
      if (n < 2 * NV) {
        f32x16_t p = mul64(b[0][n % 2], a[n / 2 & 1][0], f32x16_t{});
        p = mul64(b[1][n % 2], a[n / 2 & 1][1], p);
        __builtin_amdgcn_sched_barrier(0);
        if (n < 3)
#pragma unroll
          for (int q = 3 * n; q < 3 * n + 3; ++q) load(kt + 1, slot ^ 1, q);
        // the fragments of the row block before are used up: those of the next one
        if (n % 2 == 0 && n > 0 && n / 2 + 1 < NV) read_a(n / 2 + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[n / 2][n % 2][r] = fmaf(p[r], s[n / 2 & 1], acc[n / 2][n % 2][r]);
        pin(acc[n / 2][n % 2]);
        __builtin_amdgcn_sched_barrier(0);
      } else if (n < 3) {
#pragma unroll
        for (int q = 3 * n; q < 3 * n + 3; ++q) load(kt + 1, slot ^ 1, q);
      }
    }
    sw = sload_f32(t.w_scale, kt + 1 < nk ? kt + 1 : kt);
  };
#pragma unroll
  for (int q = 0; q < 9; ++q) load(0, 0, q);
  for (int kt = 0; kt < nk; kt += 2) {
    step(kt, 0);
    if (kt + 1 < nk) step(kt + 1, 1);
  }
}

template <class C, int NV>
__device__ __forceinline__ void f8b_kloop_nv(const F8Loads& t, int nk, uint32_t lds,
                                             uint32_t scales, const float* sS, int wave, int lane,
                                             int nv, f32x16_t (&acc)[C::BM][C::BN]) {
  if constexpr (NV == 0) {
    f8b_kloop<C, 0>(t, nk, lds, scales, sS, wave, lane, acc);
  } else {
    if (nv == NV) f8b_kloop<C, NV>(t, nk, lds, scales, sS, wave, lane, acc);
    else f8b_kloop_nv<C, NV - 1>(t, nk, lds, scales, sS, wave, lane, nv, acc);
  }
}

// FAST: the e4m3 instruction (see above).  SPLIT: K is cut into p.splits slices, each
// an item of its own, whose fp32 sums go to slice s of p.part [splits, M, N].
template <class C, bool FAST, bool OUT_BF16, bool SPLIT = false>
__global__ __launch_bounds__(512, 1) void gemm_fp8_big_kernel(Fp8Args p) {
  __shared__ __attribute__((aligned(1024))) bf16_t lds[C::LDS_ELEMS];
  __shared__ __attribute__((aligned(256))) float sS[C::NSA * kScaleSlot];
  __shared__ EntryPlan plan;
  bf16_t* sA[C::NSA];
  bf16_t* sB[C::NSB];
#pragma unroll
  for (int i = 0; i < C::NSA; ++i) sA[i] = lds + i * C::A_STAGE;
#pragma unroll
  for (int i = 0; i < C::NSB; ++i) sB[i] = lds + C::NSA * C::A_STAGE + i * C::B_STAGE;
  constexpr int NOUT = C::NB;
  constexpr int OB = OUT_BF16 ? 2 : 4;
  static_assert(C::MT * NOUT * OB <= C::LDS_ELEMS * 2, "output tile");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  make_entries<C::THREADS, C::MT>(p, plan);
  const int n_tiles = (p.N + NOUT - 1) / NOUT, nb = (p.N + kFp8Block - 1) / kFp8Block;
  const int splits = SPLIT ? p.splits : 1;
  const long long total = static_cast<long long>(plan.start[p.E]) * n_tiles * splits;
  const int xcd = blockIdx.x % kXcds;
  const int kld = p.Kp / 2;  // row length in 16-bit units
  const int kb = p.Kp / kFp8Block;
  const int lrow = lane / C::CPR;
  const bf16_t* A = reinterpret_cast<const bf16_t*>(p.a);
  const bf16_t* W = reinterpret_cast<const bf16_t*>(p.w);

  const long long chunk = (total + kXcds - 1) / kXcds;
  for (long long mine = blockIdx.x / kXcds;; mine += gridDim.x / kXcds) {
    const long long turn = xcd * chunk + mine;
    if (mine >= chunk || turn >= total) break;
    __syncthreads();  // the item before is done with the LDS
    const long long it = SPLIT ? turn / splits : turn;
    const int slice = SPLIT ? static_cast<int>(turn % splits) : 0;
    const int k0 = SPLIT ? kb * slice / splits : 0;                // first step
    const int nk = SPLIT ? kb * (slice + 1) / splits - k0 : kb;    // and how many
    // (uniform, but read from LDS: tell the compiler)
    auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    const int g = uni(entry_group(plan, p.E, static_cast<int>(it / n_tiles)));
    Item item = place_item(it, plan.start, g, n_tiles, C::MT, plan.rows[g], true);
    item.m0 = uni(item.m0);
    item.rows = uni(item.rows);
    item.n = uni(item.n);
    const long long row0 = static_cast<long long>(uni(plan.lo[g])) + item.m0;
    auto source = [&](int r) { return row0 + (r < item.rows ? r : item.rows - 1); };
    f32x16_t acc[C::BM][C::BN];
#pragma unroll
    for (int i = 0; i < C::BM; ++i)
#pragma unroll
      for (int j = 0; j < C::BN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    const int nblk = (item.rows + 31) >> 5;
    const int nv = min((nblk - wm + 1) >> 1, C::BM);
    const float* wscale = p.w_scale + static_cast<long long>(g) * nb * kb + k0;
    if constexpr (C::MT == 256) {
      static_assert(!SPLIT, "128-row tiles");
      F8Loads t;
      t.a = A + row0 * kld;
      t.b = W + (static_cast<long long>(g) * p.N + item.n * NOUT) * kld;
      t.a_scale = p.a_scale + row0 * kb;
      t.w_scale = wscale + static_cast<long long>(min(item.n * 2 + (wn >> 1), nb - 1)) * kb;
      t.last_a = item.rows - 1;
      t.last_b = p.N - 1 - item.n * NOUT;
      t.ld = p.Kp;
      f8b_kloop_nv<C, C::BM>(t, nk, lds_address(lds), lds_address(sS), sS, wave, lane, nv, acc);
    } else {
      MidLoads<C> c;
      c.base = (wm == 1 ? A + row0 * kld
                        : W + (static_cast<long long>(g) * p.N + item.n * NOUT) * kld) + k0 * C::BK;
      const int last = wm == 1 ? item.rows - 1 : p.N - 1 - item.n * NOUT;
#pragma unroll
      for (int q = 0; q < C::LPW_MAX; ++q) {
        const int j = wn * (wm == 1 ? C::LPW_A : C::LPW_B) + q;
        c.off[q] = 2u * (static_cast<uint32_t>(min(j * C::RPL + lrow, last)) * kld +
                         src_chunk<C>(lane, j));
      }
      c.scale = lane < 32 ? p.a_scale + source(32 * wn + lane) * kb + k0
                          : wscale + static_cast<long long>(min(item.n * 2 + (lane & 1), nb - 1)) * kb;
      if (wm == 0) f8_kloop_nv<C, FAST, 0, C::BM>(c, lds_address(lds), lds_address(sS), nk, sA, sB, sS, wave, lane, nv, acc);
      else f8_kloop_nv<C, FAST, 1, C::BM>(c, lds_address(lds), lds_address(sS), nk, sA, sB, sS, wave, lane, nv, acc);
    }
    wait_vm<0>();
    __syncthreads();

    // ---- epilogue: block (i, j) holds the transposed product: lane l -> tile
    // row (2i + wm) * 32 + l % 32, registers 4q..4q+3 -> output columns
    // 8q + 4 (l / 32) + 0..3 of column block j.  Staged: 16-byte chunk c of row r in
    // slot c ^ (r % CPR) of the LDS tile.
    constexpr int CPR = NOUT * OB / 16;
    char* tile = reinterpret_cast<char*>(lds);
#pragma unroll
    for (int i = 0; i < C::BM; ++i) {
      const int row = (2 * i + wm) * 32 + (lane & 31);
#pragma unroll
      for (int j = 0; j < C::BN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = wn * 64 + j * 32 + 8 * q + 4 * (lane >> 5);
          const float* v = reinterpret_cast<const float*>(&acc[i][j]) + 4 * q;
          if constexpr (OUT_BF16) {
            const uint32_t w0 = f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16);
            const uint32_t w1 = f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16);
            *reinterpret_cast<uint2*>(tile + row * NOUT * OB +
                                      (((col >> 3) ^ (row & (CPR - 1))) << 4) + (col & 4) * 2) =
                make_uint2(w0, w1);
          } else {
            *reinterpret_cast<float4*>(tile + row * NOUT * OB +
                                       (((col >> 2) ^ (row & (CPR - 1))) << 4)) =
                make_float4(v[0], v[1], v[2], v[3]);
          }
        }
    }
    __syncthreads();
    constexpr int PER = 16 / OB;  // values of a chunk
    const int col0 = item.n * NOUT;
    char* out = SPLIT ? reinterpret_cast<char*>(p.part + static_cast<size_t>(slice) * p.M * p.N)
                      : static_cast<char*>(p.out);
    out += (row0 * p.N + col0) * OB;
    if (p.N % PER == 0) {  // rows of y start on 16 bytes
      for (int c = tid; c < item.rows * CPR; c += C::THREADS) {
        const int row = c / CPR, ch = c % CPR;
        if (col0 + ch * PER < p.N)
          *reinterpret_cast<uint4*>(out + (static_cast<size_t>(row) * p.N + ch * PER) * OB) =
              *reinterpret_cast<const uint4*>(tile + row * NOUT * OB + ((ch ^ (row & (CPR - 1))) << 4));
      }
    } else {  // a value a thread
      const int cols = min(NOUT, p.N - col0);
      for (int c = tid; c < item.rows * NOUT; c += C::THREADS) {
        const int row = c / NOUT, col = c % NOUT;
        if (col >= cols) continue;
        const char* from = tile + row * NOUT * OB + (((col / PER) ^ (row & (CPR - 1))) << 4) + col % PER * OB;
        const size_t to = static_cast<size_t>(row) * p.N + col;
        if (OB == 2) reinterpret_cast<uint16_t*>(out)[to] = *reinterpret_cast<const uint16_t*>(from);
        else reinterpret_cast<uint32_t*>(out)[to] = *reinterpret_cast<const uint32_t*>(from);
      }
    }
  }
}

// y from the slices' sums, in order; a thread per 4 values (VEC: N a multiple of 4).
// Rows outside the one group keep what y held.
template <bool VEC>
__global__ __launch_bounds__(256) void gemm_fp8_reduce_kernel(Fp8Args p) {
  long long first = 0, last = p.M;
  if (p.offsets) {
    first = clampi(p.offsets[0], 0, p.M);
    last = clampi(p.offsets[1], 0, p.M);
  }
  const long long n = static_cast<long long>(p.M) * p.N, end = last * p.N;
  constexpr int PER = VEC ? 4 : 1;
  for (long long i = first * p.N + (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * PER;
       i < end; i += static_cast<long long>(gridDim.x) * 256 * PER) {
    float v[PER] = {};
    for (int s = 0; s < p.splits; ++s) {
      if constexpr (VEC) {
        const float4 f = *reinterpret_cast<const float4*>(p.part + s * n + i);
        v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
      } else {
        v[0] += p.part[s * n + i];
      }
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      if (p.out_bf16) static_cast<bf16_t*>(p.out)[i + e] = f32_to_bf16(v[e]);
      else static_cast<float*>(p.out)[i + e] = v[e];
    }
  }
}

}  // namespace

// Slices of K of a product of one group on 128-row tiles: where there are few tiles a
// workgroup walks all of K alone (a step of 128 takes 0.75 us of it), while others
// have none.  Estimated (us): the walk, and for slices 6 and their sums written and
// read at 4 TB/s.  Measured (us, one walk / slices): N=2048 K=7168 128 rows 46 / 21.5,
// 256 rows 47 / 24, 512 rows 46 / 29, 1024 rows 47 / 38; N=K=7168 256 rows 47 / 36.
static int splits_of(int M, int N, int Kp, int E, double& time) {
  const double entries = std::ceil(M / 128.0) + (E > 1 ? std::min(M, E) : 0);
  const double items = entries * std::ceil(N / 256.0), nk = Kp / kFp8Block;
  int best = 1;
  time = nk * 0.75 * std::ceil(items / 256.0);
  for (int s = 2; E == 1 && s <= 16 && s * 2 <= nk; ++s) {
    const double t = 6.0 + std::ceil(nk / s) * 0.75 * std::ceil(items * s / 256.0) +
                     8.0 * s * M * N / 4e6;
    if (t < 0.9 * time) {
      time = t;
      best = s;
    }
  }
  return best;
}

int fp8_splits(int M, int N, int Kp, int E) {
  double time;
  return splits_of(M, N, Kp, E, time);
}

double fp8_tiles_time(int M, int N, int Kp, int E) {
  double time;
  return (splits_of(M, N, Kp, E, time) > 1 ? 12.0 : 6.5) + time;
}

// Whether a bf16 y takes the 256-row tiles: groups that fill one to 5/8, and as many
// values of y as 192 tiles have, for with fewer the 128-row tiles keep more compute
// units busy.  Measured (us, 256 / 128 rows):
//   16384 x 7168 by 2048   184 / 227      8192 x 2048 by 1024    32 / 23
//   8192 x 7168 by 2048    104 / 117      4096 x 7168 by 2048    95 / 62
//   8192 x 2048 by 2048    39 / 41.5      3500 x 4096 by 3500    66 / 70
//   2048 x 2048 by 7168    36.4 / 38      3000 x 4096 by 3000    55 / 61
//   24576 x 768 by 2048, 128 groups  98 / 104    24576 x 2048 by 768, 256 groups  120 / 110
//   24576 x 2048 by 768, 128 groups  78 / 79     the same, 64 groups  63 / 56
// (3500, 3000 rows and 64 groups are 6, 10 and 13% off the better kernel: there the
// rounds of tiles decide, which the rule does not count)
static bool large_tiles(const Fp8Args& a) {
  return a.M / a.E >= 160 && static_cast<long long>(a.M) * a.N >= 192LL * 256 * 256;
}

hipError_t launch_gemm_fp8_big(const Fp8Args& a, hipStream_t st) {
  const int grid = (device_cus_big() + kXcds - 1) / kXcds * kXcds;
  auto go = [&](auto kernel) { kernel<<<grid, MidF8::THREADS, 0, st>>>(a); };
  if (a.splits > 1) {
    a.out_bf16 ? go(gemm_fp8_big_kernel<MidF8, true, false, true>)
               : go(gemm_fp8_big_kernel<MidF8, false, false, true>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const long long blocks = (static_cast<long long>(a.M) * a.N + 1023) / 1024;
    const unsigned g = static_cast<unsigned>(blocks < 4096 ? blocks : 4096);
    if (a.N % 4 == 0) gemm_fp8_reduce_kernel<true><<<g, 256, 0, st>>>(a);
    else gemm_fp8_reduce_kernel<false><<<g, 256, 0, st>>>(a);
  } else if (!a.out_bf16) {
    go(gemm_fp8_big_kernel<MidF8, false, false>);
  } else if (large_tiles(a)) {
    go(gemm_fp8_big_kernel<BigF8, true, true>);
  } else {
    go(gemm_fp8_big_kernel<MidF8, true, true>);
  }
  return hipGetLastError();
}

}  // namespace moe
