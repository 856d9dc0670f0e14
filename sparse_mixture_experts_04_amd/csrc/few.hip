// The whole layer for 1 to 16 tokens in two kernels.
//
// Few tokens visit few experts (6 and the shared ones for one token), so the
// layer is one pass over those experts' weights; what it costs beyond that is
// launches and the waits between its stages.  few_route_kernel takes the
// router's logits and clears the flags below.  few_ffn_kernel does the rest
// with kFewGrid workgroups:
//
//   selection    workgroup t < T: top-6 and gates of token t;
//   gate/up      every workgroup's share ("chunk") of the shared experts'
//                columns, which needs no routing and so hides the selection,
//                then its share of the routed experts' columns;
//   down         its share of the output columns, all contributors of a column,
//                so that each y is summed where it is made.
//
// Between the stages workgroups wait for flags that others set.  A wait ends
// whatever else runs on the device: a flag says not started, started or done;
// work that has been started is held by a running workgroup and finishes
// (gate/up waits for the selection only, the selection for nothing), and work
// that no workgroup has started is done by the one that waits for it.  Two
// workgroups may then do the same piece: they write the same bits.  Nobody waits
// for the down stage.  (Handing items out by one counter cost 70 ns an item on
// this device, more than an item's weights take; release and acquire fences, a
// pair for each of 4096 waves, 150 us a call.)
//
// No sum depends on timing or on the other tokens' values: a dot product is
// added over the same lanes in the same order wherever its row lies, and a
// token's contributors in the order of moe_combine (its picks by rank, then the
// shared experts).
//
// Precision: logits, affinities and gates in fp64 (the selection is that of
// exact arithmetic but for keys within ~1e-15); products with fp32 (or exact
// int32, in the down product per pass over K) accumulation; h and the experts'
// outputs in fp32, one rounding into y.
// With bf16 weights h enters the down product as two bf16 terms (h = hi + lo
// to 2^-17): the second product costs no memory traffic.  With 8-bit weights x
// is quantised per token and h per row.
//
// Bound by the weight rows' loads (rowstream.h): T=16, d=7168, F=2048, bf16
// reads 7.63 GB in 1.20 to 1.23 ms, 6.2 to 6.3 TB/s; T=1 there 706 MB in 119 us,
// 5.9 TB/s; T=4 with 8-bit weights 0.98 GB in 175 to 179 us, 5.5 TB/s (bytes as
// counted).  At T=1, d=2048, F=768 the 77 MB need 12 us and the kernel takes 27:
// the selection (9 us, of which the shared experts' share hides half), the plan
// once the picks are known, the wait before the down stage and the latency of each
// stage's first loads, and the fetch of code that the weights have driven out of
// the caches (some 0.4 us per 128 bytes: hence loops where they can be).
// few_route_kernel adds 4 to 5 us, 13.6 at T=16, d=7168, where
// each of its workgroups reads all of x (512 threads a half of the tokens each: 14.9).
// Many experts of short rows are bound by what a row costs besides its bytes, in
// the down stage above all: T=16, d=1280, F=256 takes 67 us for the 26 that its
// 157 MB need; 82 entries of 1280 rows of 512 bytes, 1 us a row and wave.
#include <type_traits>

#include "few.h"
#include "int8_quant.h"
#include "select.h"
#include "rowstream.h"

namespace moe {

// ----------------------------------------------------------------- routing

// 4 consecutive values of x.
__device__ __forceinline__ void load4(const float* p, double (&v)[4]) {
  const float4 u = *reinterpret_cast<const float4*>(p);
  v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
}
__device__ __forceinline__ void load4(const bf16_t* p, double (&v)[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(u.x << 16);
  v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16);
  v[3] = __uint_as_float(u.y & 0xffff0000u);
}

// Block b < E + S: the logits of router row b for all tokens (products exact
// in fp64, sums in a fixed order) as sigmoids (and their logarithms).  Block E + S clears the control block of
// few_ffn_kernel.  INT8: block E + S + 1 + t quantises token t.  TM: tokens
// rounded up to a power of two.
template <typename X, int TM, bool INT8>
__global__ __launch_bounds__(512) void few_route_kernel(FewArgs p, int ctrl_ints) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = blockIdx.x;
  const int rows = p.E + p.S;
  const X* x = static_cast<const X*>(p.x);
  if (b == rows) {
    for (int i = tid; i < ctrl_ints; i += 512) p.ctrl[i] = 0;  // kIdle
    return;
  }
  if (INT8 && b > rows) {
    const int t = b - rows - 1;
    const float s = quantize_row<X, true, 512>(x + static_cast<size_t>(t) * p.d, p.d, p.d,
                                          p.xq + static_cast<size_t>(t) * p.d);
    if (tid == 0) p.xs[t] = s;
    return;
  }
  double acc[TM];
#pragma unroll
  for (int t = 0; t < TM; ++t) acc[t] = 0.0;
  const float* w = p.w_router + static_cast<size_t>(b) * p.d;
  for (int c = tid * 4; c < p.d; c += 2048) {
    double wv[4];
    load4(w + c, wv);
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      const int tt = t < p.T ? t : p.T - 1;
      double xv[4];
      load4(x + static_cast<size_t>(tt) * p.d + c, xv);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t] = fma(xv[i], wv[i], acc[t]);
    }
  }
  __shared__ double sum[8][TM];
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const double v = wave_sum(acc[t], lane);
    if (lane == 0) sum[wave][t] = v;
  }
  __syncthreads();
  if (tid < p.T) {
    double z = sum[0][tid];
#pragma unroll
    for (int i = 1; i < 8; ++i) z += sum[i][tid];
    // log sigmoid(z) for gates by logsumexp, and sigmoid(z)
    const double l = p.logsumexp ? fmin(z, 0.0) - log1p(exp(-fabs(z))) : 0.0;
    p.zs[static_cast<size_t>(tid) * rows + b] = double2{l, sigmoid64(z)};
  }
}

// --------------------------------------------------------------- the experts

// exp(x) for x <= 0, to a few 2^-53: x = n ln 2 + r with |r| <= ln 2 / 2, and the
// Taylor series of exp(r) to r^13 / 13! (the next term is below 2^-56) in a loop
// whose factors come from memory.  Below -800, where exp(x) is 0 in fp64 all the
// same, the argument is -800: r is small only while n fits the 53 bits of its
// products, and logits reach 1e80.  The library's exp is straight-line code with
// its constants in registers: two of those spilled, and scratch memory costs the
// whole kernel (8-bit, T=4, d=7168: 184 us with it, 177 without).
__device__ const double kOneOver[14] = {0.0, 1.0, 1.0 / 2, 1.0 / 3, 1.0 / 4, 1.0 / 5, 1.0 / 6,
                                        1.0 / 7, 1.0 / 8, 1.0 / 9, 1.0 / 10, 1.0 / 11, 1.0 / 12,
                                        1.0 / 13};
__device__ __forceinline__ double few_exp(double x) {
  x = x < -800.0 ? -800.0 : x;  // a NaN stays
  const double n = rint(x * 1.4426950408889634);
  // ln 2 = 45426 / 65536 + the rest; n times the first part is exact
  const double r = fma(n, -1.4286068203094173e-06, fma(n, -45426.0 / 65536.0, x));
  double e = 1.0;
#pragma unroll 1
  for (int k = 13; k > 0; --k) e = fma(e, r * kOneOver[k], 1.0);
  return ldexp(e, static_cast<int>(fmax(n, -2000.0)));  // fmax: a NaN has no integer
}

// Top-6 and gates of token t by one wave, in little code: a workgroup that runs
// this waits for every line of it to come from memory (the weights have
// streamed it out of the caches since the last call), so the rounds are a loop
// and the gates are taken a lane each.  A NaN key ranks last (the gates of such
// a token are NaN, and so is its output).
template <int S>
__device__ __forceinline__ void few_select(const FewArgs& p, int t, int lane) {
  constexpr int EPL = 4;  // experts per lane; those past E are no candidates
  const double2* zs = p.zs + static_cast<size_t>(t) * (p.E + S);
  double key[EPL];
  int open = 0;  // bit q: expert lane + 64 q is a candidate
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    const int e = lane + 64 * q;
    key[q] = -INFINITY;
    if (e < p.E) {
      const double k = zs[e].y + static_cast<double>(p.bias[e]);
      key[q] = k == k ? k : -INFINITY;
      open |= 1 << q;
    }
  }
  int id = p.E + (lane - kFewTopK < S ? lane - kFewTopK : 0);  // this lane's contributor
#pragma unroll 1
  for (int r = 0; r < kFewTopK; ++r) {
    double bk = -INFINITY;
    int bj = 0x7fffffff;
#pragma unroll
    for (int q = 0; q < EPL; ++q) {
      if (((open >> q) & 1) && better(key[q], lane + 64 * q, bk, bj)) {
        bk = key[q];
        bj = lane + 64 * q;
      }
    }
    wave_argmax(bk, bj, lane);
    if ((bj & 63) == lane) open &= ~(1 << (bj >> 6));
    if (lane == r) id = bj;
  }
  // lane j < 6 + S: contributor j
  const bool mine = lane < kFewTopK + S;
  const double2 v = mine ? zs[id] : double2{0.0, 0.0};
  double e = v.y;  // the gates are e / sum e, times gate_scale
  if (p.logsumexp) {  // exp(l - logsumexp l) = exp(l - m) / sum exp(l - m)
    double m = mine ? v.x : -INFINITY;
    int who = lane;
    wave_argmax(m, who, lane);
    e = mine ? few_exp(v.x - m) : 0.0;
  }
  const double g = e / (wave_sum(e, lane) / p.gate_scale);
  if (!mine) return;
  const int at = t * (kFewTopK + S) + lane;
  agent_store(p.gates + at, static_cast<float>(g));
  if (p.gates_out) p.gates_out[at] = static_cast<float>(g);
  if (lane < kFewTopK) {
    agent_store(p.topk + t * kFewTopK + lane, id);
    if (p.topk_out) p.topk_out[t * kFewTopK + lane] = id;
  }
}

// States of a flag.
enum { kIdle = 0, kStarted = 1, kDone = 2 };

// i / n for 0 <= i < 2^20 and a quotient below 128 (inv = 1 / n): the product is off
// by less than 128 * 2^-22, the quotient of i + 1/2 lies at least 1 / (2 n) from an
// integer, and every n here is at most 8192.  An integer division is 40
// instructions, all of them to be fetched.
__device__ __forceinline__ int quotient(int i, float inv) {
  return static_cast<int>((static_cast<float>(i) + 0.5f) * inv);
}

constexpr int kFewThreads = 1024;
constexpr int kFewWaves = kFewThreads / 64;
constexpr int kPatience = 64;  // polls before a waiter looks for work not started

// Every wave's agent stores have reached memory when it passes.
__device__ __forceinline__ void drain_stores() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  __syncthreads();
}

// Marks piece i of `flags` done, after everything the workgroup wrote for it
// with agent stores.
__device__ __forceinline__ void mark_done(int32_t* flags, int i) {
  drain_stores();
  if (threadIdx.x == 0) agent_store(flags + i, kDone);
}

// Waits until all n flags are done and returns -1, or, when some piece has
// still not been started after a while, returns that piece (the first from
// `from` on, cyclically) for the caller to do.  The same on every thread.
__device__ __forceinline__ int wait_all(const int32_t* flags, int n, int from, int* s_idle) {
  for (int poll = 0;; ++poll) {
    bool done = true;
    int idle = 0x7fffffff;
    for (int i = threadIdx.x; i < n; i += kFewThreads) {
      const int v = agent_load(flags + i);
      done = done && v == kDone;
      if (v == kIdle) {
        const int at = i >= from ? i - from : i - from + n;
        idle = at < idle ? at : idle;
      }
    }
    if (__syncthreads_and(done)) break;
    if (poll >= kPatience) {
      if (threadIdx.x == 0) *s_idle = 0x7fffffff;
      __syncthreads();
      if (idle != 0x7fffffff) atomicMin(s_idle, idle);
      __syncthreads();
      const int at = *s_idle;
      __syncthreads();
      if (at != 0x7fffffff) return (at + from) % n;
    }
    __builtin_amdgcn_s_sleep(2);
  }
  return -1;
}

// The rows of all contributors as one list: the shared experts' tokens, then the
// pairs of the routed experts in ascending expert (and pair) order; entries are
// runs of up to kUnitRows rows of one expert.
constexpr int kFewRows = kFewMaxTokens * (kFewTopK + 2);
constexpr int kFewEntries = kFewMaxTokens * kFewTopK + 2 * ((kFewMaxTokens + kUnitRows - 1) / kUnitRows);
struct FewPlan {
  int tok[kFewRows + kUnitRows];    // token of a list row
  int hrow[kFewRows + kUnitRows];   // its row of h
  float scale[kFewRows + kUnitRows];  // its scale of h (8-bit weights)
  float gate[kFewRows];             // gates [T, 6 + S]
  int first[kFewEntries + 1];       // first list row of an entry
  int expert[kFewEntries + 1];      // its row of the weight stack
  int shared_entries, entries;
};

// Entries of the shared experts (all threads, a barrier after it).
template <int S>
__device__ __forceinline__ void plan_shared(int T, FewPlan& s) {
  static_assert(S <= 2 && kFewMaxTokens <= 2 * kUnitRows, "two shared experts of two entries");
  const int per = T > kUnitRows ? 2 : 1;
  const int tid = threadIdx.x;
  if (tid < S * T) {
    const int e = tid >= T ? 1 : 0, t = tid - e * T;
    s.tok[tid] = t;
    s.hrow[tid] = T * kFewTopK + tid;
  }
  if (tid < S * per) {
    const int e = per == 2 ? tid >> 1 : tid, half = per == 2 ? tid & 1 : 0;
    s.first[tid] = e * T + half * kUnitRows;
    s.expert[tid] = e;
  }
  if (tid == 0) {
    s.shared_entries = S * per;
    s.first[S * per] = S * T;
  }
}

// Entries of the routed experts: thread e stands for expert e and finds its
// pairs in a bit mask of the 6 T pairs.
template <int S>
__device__ __forceinline__ void plan_routed(const FewArgs& p, FewPlan& s) {
  constexpr int MW = (kFewMaxTokens * kFewTopK + 31) / 32;
  __shared__ uint32_t mask[256][MW];
  __shared__ int wrow[4], went[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = p.T * kFewTopK;
  for (int i = tid; i < 256 * MW; i += kFewThreads) (&mask[0][0])[i] = 0;
  __syncthreads();
  if (tid < n) {
    const int e = agent_load(p.topk + tid);
    atomicOr(&mask[e < 0 ? 0 : e >= p.E ? p.E - 1 : e][tid / 32], 1u << (tid % 32));
  }
  __syncthreads();
  int cnt = 0, rows = 0, ent = 0;
  if (tid < 256) {
    for (int i = 0; i < MW; ++i) cnt += __popc(mask[tid][i]);
    rows = cnt;
    ent = (cnt + kUnitRows - 1) / kUnitRows;
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(rows, o), v = __shfl_up(ent, o);
      if (lane >= o) {
        rows += u;
        ent += v;
      }
    }
    if (lane == 63) {
      wrow[wave] = rows;
      went[wave] = ent;
    }
  }
  __syncthreads();
  if (tid < 256) {
    for (int w = 0; w < wave; ++w) {
      rows += wrow[w];
      ent += went[w];
    }
    int at = S * p.T + rows - cnt;
    const int e0 = s.shared_entries + ent - (cnt + kUnitRows - 1) / kUnitRows;
    for (int i = 0; i * kUnitRows < cnt; ++i) {
      s.first[e0 + i] = at + i * kUnitRows;
      s.expert[e0 + i] = tid;
    }
    for (int i = 0; i < MW; ++i)
      for (uint32_t m = mask[tid][i]; m; m &= m - 1) {
        const int pair = i * 32 + __ffs(m) - 1;
        s.tok[at] = pair / kFewTopK;
        s.hrow[at++] = pair;
      }
    if (tid == 255) {
      s.entries = s.shared_entries + ent;
      s.first[s.shared_entries + ent] = S * p.T + rows;
    }
  }
  __syncthreads();
}

// LDS of a workgroup: sums (gate and up of kPartCols columns, or the down products
// of its columns with every row of h), then activation rows.
constexpr int kPool = 144 * 1024;
constexpr int kPartCols = 512;     // gate/up columns between two epilogues
constexpr int kPartBytes = kPartCols * 2 * kUnitRows * 4;
static_assert(kFewMaxWidth / kFewGrid * kFewRows * 4 + 8 * kUnitRows * kChunk <= kPool,
              "8 chunks of 8 rows beside the widest layer's products");

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The units of a workgroup go to its waves in turn (unit i kFewWaves + wave is
// the wave's i-th): the waves read neighbouring rows at the same time, and their
// shares differ by one unit at most.

// Gate/up units of n columns from cbase on: unit 2 c is the W_gate row of column
// cbase + c, 2 c + 1 its W_up row; sums go to part[c].  Column cbase is column f_
// of entry ent_.
template <class Acc>
struct GateWalk {
  const FewPlan& plan;
  Acc (*part)[2][kUnitRows];
  const char* base;   // of the matrix stack this wave reads: W_gate or W_up
  size_t kfull;       // bytes of a weight row
  int F, n, up, xstride, lane;
  bool more;          // not the first pass over K: add
  const char* lrow;   // load side: the next unit's row
  int lf, lent;
  int f, ent, rows, col;  // multiply side
  static constexpr int kStep = kFewWaves / 2;  // columns from one unit to the next

  __device__ __forceinline__ GateWalk(const FewPlan& pl, Acc (*pt)[2][kUnitRows], const void* g,
                                      const void* u, size_t kf, size_t koff, int F_, int cols,
                                      int wave, int ent_, int f_, int xs, bool m)
      : plan(pl), part(pt), base(static_cast<const char*>(wave & 1 ? u : g) + koff), kfull(kf),
        F(F_), n((2 * cols - wave + kFewWaves - 1) / kFewWaves), up(wave & 1), xstride(xs),
        lane(threadIdx.x & 63), more(m) {
    static_assert(kFewWaves % 2 == 0, "a wave reads one of the two matrices");
    lent = ent_;
    lf = f_ + (wave >> 1);
    for (; lf >= F; lf -= F) ++lent;
    ent = lent;
    f = lf;
    col = wave >> 1;
    rows = 0;
    lrow = nullptr;
    if (n > 0) place();
  }
  __device__ __forceinline__ void place() {
    lrow = base + (static_cast<size_t>(uniform(plan.expert[lent])) * F + lf) * kfull;
  }
  __device__ __forceinline__ int units() const { return n; }
  __device__ __forceinline__ const char* row(int u) {
    if (u > 0) {
      lrow += kStep * kfull;
      lf += kStep;
      if (lf >= F) {  // F >= 128: one entry further
        lf -= F;
        ++lent;
        place();
      }
    }
    return lrow;
  }
  __device__ __forceinline__ int enter(int u, int (&off)[kUnitRows]) {
    if (u > 0) {
      f += kStep;
      col += kStep;
    }
    if (u == 0 || f >= F) {
      if (f >= F) {
        f -= F;
        ++ent;
      }
      const int r0 = plan.first[ent];
      rows = uniform(plan.first[ent + 1] - r0);
#pragma unroll
      for (int r = 0; r < kUnitRows; ++r)
        off[r] = plan.tok[r0 + (r < rows ? r : 0)] * xstride + lane * 16;
    }
    return rows;
  }
  __device__ __forceinline__ void leave(int, int nr, const Acc (&acc)[kUnitRows]) {
    const Acc s = row_totals(nr, acc, lane);
    const int r = total_row(lane);
    if ((lane & 7) == 0 && r < nr) {
      Acc* out = part[col][up] + r;
      *out = more ? *out + s : s;
    }
  }
};

// Down units of a pass over entries e0..e0+ne-1: unit u is column u / ne of the
// workgroup's columns and entry e0 + u % ne.
template <class Acc, bool I8>
struct DownWalk {
  const FewPlan& plan;
  float* yrow;             // [columns, rows of h]
  int rows_h;
  bool more;               // not the first pass over K: add
  const char *w, *ws;      // routed and shared W_down at the pass's K offset
  const float *t, *ts;     // 8-bit scales [E or S, d]
  size_t kfull;
  int d, n0, e0, ne, n, stride, lane, se, base;
  int lcol, lent, col, ent;
  float channel = 0.0f;    // 8-bit scale of the unit's channel
  int mine = 0;            // list row whose sum this lane gets (total_row)

  __device__ __forceinline__ DownWalk(const FewPlan& pl, float* ys, int rh, const FewArgs& p,
                                      size_t kf, size_t koff, int n0_, int e0_, int ne_, int cols,
                                      int wave, int st)
      : plan(pl), yrow(ys), rows_h(rh), more(koff > 0), w(static_cast<const char*>(p.w_down) + koff),
        ws(static_cast<const char*>(p.ws_down) + koff), t(p.t_down), ts(p.ts_down), kfull(kf),
        d(p.d), n0(n0_), e0(e0_), ne(ne_), n((cols * ne_ - wave + kFewWaves - 1) / kFewWaves),
        stride(st), lane(threadIdx.x & 63), se(uniform(pl.shared_entries)), base(pl.first[e0_]) {
    lcol = col = 0;
    lent = ent = wave;
    for (; lent >= ne; lent -= ne) ++lcol;
    ent = lent;
    col = lcol;
  }
  __device__ __forceinline__ int units() const { return n; }
  __device__ __forceinline__ const char* row(int u) {
    if (u > 0)
      for (lent += kFewWaves; lent >= ne; lent -= ne) ++lcol;
    const int i = e0 + lent;
    return (i < se ? ws : w) +
           (static_cast<size_t>(uniform(plan.expert[i])) * d + n0 + lcol) * kfull;
  }
  __device__ __forceinline__ int enter(int u, int (&off)[kUnitRows]) {
    if (u > 0)
      for (ent += kFewWaves; ent >= ne; ent -= ne) ++col;
    const int i = e0 + ent, r0 = plan.first[i];
    const int rows = uniform(plan.first[i + 1] - r0);
#pragma unroll
    for (int r = 0; r < kUnitRows; ++r)
      off[r] = (r0 - base + (r < rows ? r : 0)) * stride + lane * 16;
    const int tr = total_row(lane);
    mine = r0 + (tr < rows ? tr : 0);
    if (I8) {
      const int32_t* tp = reinterpret_cast<const int32_t*>(i < se ? ts : t) +
                          static_cast<size_t>(uniform(plan.expert[i])) * d;
      channel = __int_as_float(((const_words)tp)[n0 + col]);
    }
    return rows;
  }
  __device__ __forceinline__ void leave(int, int nr, const Acc (&acc)[kUnitRows]) {
    const Acc s = row_totals(nr, acc, lane);
    if ((lane & 7) == 0 && total_row(lane) < nr) {
      float v = static_cast<float>(s);
      if (I8) v *= plan.scale[mine] * channel;
      float* y = yrow + col * rows_h + plan.hrow[mine];
      *y = more ? *y + v : v;
    }
  }
  // reads through the scalar cache do not count as vector loads
  typedef const int32_t __attribute__((address_space(4)))* const_words;
};

// Work of one expert weight type.
template <class Dot> struct FewTraits;
template <> struct FewTraits<DotBf16> { static constexpr int ESZ = 2, PLANES = 2; };
template <> struct FewTraits<DotF32> { static constexpr int ESZ = 4, PLANES = 1; };
template <> struct FewTraits<DotI8> { static constexpr int ESZ = 1, PLANES = 1; };

// The kernel's arguments, read again where they are needed.  Kept from the start,
// they take most of the scalar registers through every loop, and what does not
// fit is spilled: with that the kernel was 5 to 25% slower.
__device__ __forceinline__ FewArgs args_again() {
  typedef const FewArgs __attribute__((address_space(4)))* arg_ptr;
  arg_ptr k = (arg_ptr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(k));  // not the loads from before
  FewArgs a;
  __builtin_memcpy(&a, (const FewArgs*)k, sizeof(a));
  return a;
}

// The arguments (args_again reads them).
template <class Dot, typename Y, int S>
__global__ __launch_bounds__(kFewThreads, 4) void few_ffn_kernel(FewArgs) {
  using Acc = typename Dot::Acc;
  constexpr int ESZ = FewTraits<Dot>::ESZ, PL = FewTraits<Dot>::PLANES;
  constexpr bool I8 = ESZ == 1;
  __shared__ __attribute__((aligned(1024))) char pool[kPool];
  __shared__ FewPlan plan;
  __shared__ int s_word;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const FewArgs p0 = args_again();
  const int T = p0.T, F = p0.F, d = p0.d;
  const int rows = T * (kFewTopK + S);
  int32_t* chunk_flag = p0.ctrl;                   // [grid]
  int32_t* token_flag = chunk_flag + kFewGrid;     // [T]
  int32_t* row_flag = token_flag + kFewMaxTokens;  // [rows] (8-bit weights)
  bool planned = false;

  if (tid == 0) {
    const int state = agent_load(chunk_flag + blockIdx.x);
    if (state == kIdle) {
      if (blockIdx.x < T) agent_store(token_flag + blockIdx.x, kStarted);
      agent_store(chunk_flag + blockIdx.x, kStarted);
    }
    s_word = state == kDone;  // started late: others have done this chunk
  }
  plan_shared<S>(T, plan);
  __syncthreads();
  bool skip = s_word;

  // The down stage: this workgroup's output columns, in passes over the
  // contributors (and over K, for wide experts) of as many rows of h as fit.
  // (Taken while the selection is waited for.)
  int n0 = 0, cols = 0, ybytes = 0, fall = 0, fpass = 0, stride = 0, capacity = 0;
  const size_t ffull = static_cast<size_t>(F) * ESZ;
  float* yrow = reinterpret_cast<float*>(pool);
  auto down_shape = [&]() __attribute__((always_inline)) {
    n0 = static_cast<int>(d * blockIdx.x / kFewGrid);
    cols = static_cast<int>(d * (blockIdx.x + 1) / kFewGrid) - n0;
    fall = static_cast<int>((ffull + kChunk - 1) / kChunk);
    ybytes = (cols * rows * 4 + kChunk - 1) / kChunk * kChunk;
    // every entry fits a pass: 8 rows of fpass chunks
    fpass = min(fall, (kPool - ybytes) / kChunk / PL / kUnitRows);
    stride = fpass * kChunk * PL;  // of a row of h in oper
    capacity = (kPool - ybytes) / stride;
  };
  using Down = DownWalk<Acc, I8>;
  auto pass_end = [&](int e0) {  // entries e0..pass_end-1 make a pass
    int e1 = e0 + 1;
    while (e1 < plan.entries && plan.first[e1 + 1] - plan.first[e0] <= capacity) ++e1;
    return e1;
  };
  auto down_walk = [&](int k0, int e0, int e1) __attribute__((always_inline)) {
    return Down(plan, yrow, rows, args_again(), ffull, static_cast<size_t>(k0) * kChunk, n0, e0, e1 - e0,
                cols, wave, stride);
  };
  RowStream<Dot, PL, Down> down;

  // ---- gate/up: this workgroup's chunk, then any that nobody has started.
  // Passes over K of as many chunks of every token as `oper` holds.
  const size_t kfull = static_cast<size_t>(d) * ESZ;
  const int kall = static_cast<int>((kfull + kChunk - 1) / kChunk);
  auto part_sums = reinterpret_cast<Acc(*)[2][kUnitRows]>(pool);
  char* oper = pool + kPartBytes;
  const int kpass = min(kall, (kPool - kPartBytes) / kChunk / T);
  int staged = -1;  // first K chunk of the pass that oper holds
  int token = blockIdx.x < T ? static_cast<int>(blockIdx.x) : -1;  // to be selected here
  for (int chunk = blockIdx.x; chunk >= 0;) {
    for (int part = 0; part < 2;) {  // shared, then routed experts
      if (token >= 0) {
        if (wave == 0) few_select<S>(args_again(), token, lane);
        mark_done(token_flag, token);
        token = -1;
      }
      if (part == 1 && !planned) {
        down_shape();
        token = wait_all(token_flag, T, 0, &s_word);
        if (token >= 0) continue;
        plan_routed<S>(args_again(), plan);
        planned = true;
      }
      // columns of this chunk: the workgroups that select tokens have no share of
      // the shared experts
      const int ent0 = part == 0 ? 0 : plan.shared_entries;
      // (at most 104 entries of 16384 columns, times 256: 32 bits)
      const unsigned n = static_cast<unsigned>(part == 0 ? plan.shared_entries
                                                         : plan.entries - ent0) * F;
      const int share = part == 0 ? chunk - T : chunk;
      int c = 0, cend = 0;
      if (skip) {
      } else if (part == 1) {
        c = static_cast<int>(n * share / kFewGrid);
        cend = static_cast<int>(n * (share + 1) / kFewGrid);
      } else if (share >= 0) {
        const unsigned of = kFewGrid - T;
        c = static_cast<int>(n * share / of);
        cend = static_cast<int>(n * (share + 1) / of);
      }
      int ent = ent0 + c / F, f = c - (ent - ent0) * F;  // entry and column of c
      for (; c < cend; c += kPartCols) {
        const int c1 = min(c + kPartCols, cend);
        for (int k0 = 0; k0 < kall; k0 += kpass) {
          const int kbytes = static_cast<int>(min(kfull - static_cast<size_t>(k0) * kChunk,
                                                  static_cast<size_t>(kpass) * kChunk));
          const FewArgs p = args_again();
          GateWalk<Acc> walk(plan, part_sums, part == 0 ? p.ws_gate : p.w_gate,
                             part == 0 ? p.ws_up : p.w_up, kfull,
                             static_cast<size_t>(k0) * kChunk, F, c1 - c, wave, ent, f,
                             kpass * kChunk, k0 > 0);
          RowStream<Dot, 1, GateWalk<Acc>> stream;
          stream.begin(walk, kbytes);
          if (staged != k0) {  // x of every token, zeros behind its last value
            __syncthreads();
            const char* x = I8 ? reinterpret_cast<const char*>(p.xq) : static_cast<const char*>(p.x);
            const int pieces = kpass * (kChunk / 16);
            const float inv = 1.0f / static_cast<float>(pieces);
            for (int i = tid; i < T * pieces; i += kFewThreads) {
              const int t = quotient(i, inv), o = (i - t * pieces) * 16;
              u32x4_t v{0, 0, 0, 0};
              if (o < kbytes)
                v = *reinterpret_cast<const u32x4_t*>(x + t * kfull +
                                                      static_cast<size_t>(k0) * kChunk + o);
              *reinterpret_cast<u32x4_t*>(oper + t * kpass * kChunk + o) = v;
            }
            staged = k0;
          }
          __syncthreads();
          stream.run(walk, oper, 0);
        }
        __syncthreads();
        // h = silu(gate) * up
        const FewArgs p = args_again();
        const float inv = 1.0f / static_cast<float>(c1 - c);
        for (int i = tid; i < (c1 - c) * kUnitRows; i += kFewThreads) {
          const int r = quotient(i, inv), j = i - r * (c1 - c);
          int je = ent, jf = f + j;  // entry and column of c + j
          for (; jf >= F; jf -= F) ++je;
          const int lr = plan.first[je] + r;
          if (lr >= plan.first[je + 1]) continue;
          float gt = static_cast<float>(part_sums[j][0][r]);
          float up = static_cast<float>(part_sums[j][1][r]);
          if (I8) {
            const float sx = p.xs[plan.tok[lr]];
            const size_t at = static_cast<size_t>(plan.expert[je]) * F + jf;
            gt *= sx * (part == 0 ? p.ts_gate : p.t_gate)[at];
            up *= sx * (part == 0 ? p.ts_up : p.t_up)[at];
          }
          agent_store(p.h + static_cast<size_t>(plan.hrow[lr]) * F + jf,
                      gt / (1.0f + expf(-gt)) * up);
        }
        for (f += kPartCols; f >= F; f -= F) ++ent;
      }
      ++part;
    }
    mark_done(chunk_flag, chunk);
    skip = false;
    // the first weights of the down stage come while the others finish
    Down walk = down_walk(0, 0, pass_end(0));
    down.begin(walk, static_cast<int>(min(ffull, static_cast<size_t>(fpass) * kChunk)));
    chunk = wait_all(chunk_flag, kFewGrid, blockIdx.x, &s_word);
  }

  // ---- 8-bit weights: row r of h quantised by workgroup r
  if (I8) {
    if (tid == 0 && static_cast<int>(blockIdx.x) < rows &&
        agent_load(row_flag + blockIdx.x) == kIdle)
      agent_store(row_flag + blockIdx.x, kStarted);
    for (int r = static_cast<int>(blockIdx.x) < rows ? static_cast<int>(blockIdx.x) : -2;
         r != -1; r = wait_all(row_flag, rows, blockIdx.x % rows, &s_word)) {
      if (r < 0) continue;
      const FewArgs p = args_again();
      const uint64_t* hr = reinterpret_cast<const uint64_t*>(p.h + static_cast<size_t>(r) * F);
      uint64_t* qr = reinterpret_cast<uint64_t*>(p.hq + static_cast<size_t>(r) * F);
      const float s = quantize_row<kFewThreads>(
          F, F,
          [&](int c, int, float (&v)[8]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t u = agent_load(hr + c * 4 + i);
              v[2 * i] = __uint_as_float(static_cast<uint32_t>(u));
              v[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(u >> 32));
            }
          },
          [&](int c, uint2 q) { agent_store(qr + c, q.x | (static_cast<uint64_t>(q.y) << 32)); });
      if (tid == 0) agent_store(p.hs + r, s);
      mark_done(row_flag, r);
    }
  }

  // ---- down: the passes
  // (what the passes' barriers make visible)
  if (tid < rows) {
    const FewArgs p = args_again();
    plan.gate[tid] = agent_load(p.gates + tid);
    if (I8) plan.scale[tid] = agent_load(p.hs + plan.hrow[tid]);
  }
  oper = pool + ybytes;
  for (int k0 = 0; k0 < fall; k0 += fpass) {
    const int kbytes = static_cast<int>(min(ffull - static_cast<size_t>(k0) * kChunk,
                                            static_cast<size_t>(fpass) * kChunk));
    for (int e0 = 0; e0 < plan.entries;) {
      const int first = plan.first[e0], e1 = pass_end(e0);
      Down walk = down_walk(k0, e0, e1);
      if (k0 > 0 || e0 > 0) down.begin(walk, kbytes);
      else down.resume(walk);
      const int n = plan.first[e1] - first;
      __syncthreads();  // the pass before is done with oper
      // 8 values of K at a time, zeros behind the last
      const FewArgs p = args_again();
      const int pieces = fpass * kChunk / (8 * ESZ);
      const float inv = 1.0f / static_cast<float>(pieces);
      for (int i = tid; i < n * pieces; i += kFewThreads) {
        const int r = quotient(i, inv), k = (i - r * pieces) * 8;
        char* at = oper + r * stride + k * ESZ;
        const size_t src = static_cast<size_t>(plan.hrow[first + r]) * F +
                           static_cast<size_t>(k0) * kChunk / ESZ + k;
        const bool in = k * ESZ < kbytes;
        if (I8) {
          *reinterpret_cast<uint64_t*>(at) =
              in ? agent_load(reinterpret_cast<const uint64_t*>(p.hq + src)) : 0;
        } else {
          uint64_t v[4] = {0, 0, 0, 0};
          if (in) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              v[q] = agent_load(reinterpret_cast<const uint64_t*>(p.h + src) + q);
          }
          if constexpr (PL == 2) {  // h = hi + lo in bf16
            u32x4_t hi, lo;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float a = __uint_as_float(static_cast<uint32_t>(v[q]));
              const float b = __uint_as_float(static_cast<uint32_t>(v[q] >> 32));
              const bf16_t ah = f32_to_bf16(a), bh = f32_to_bf16(b);
              hi[q] = ah | (static_cast<uint32_t>(bh) << 16);
              lo[q] = f32_to_bf16(a - bf16_to_f32(ah)) |
                      (static_cast<uint32_t>(f32_to_bf16(b - bf16_to_f32(bh))) << 16);
            }
            *reinterpret_cast<u32x4_t*>(at) = hi;
            *reinterpret_cast<u32x4_t*>(at + fpass * kChunk) = lo;
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) reinterpret_cast<uint64_t*>(at)[q] = v[q];
          }
        }
      }
      __syncthreads();
      down.run(walk, oper, fpass * kChunk);
      e0 = e1;
    }
  }
  __syncthreads();
  const FewArgs p = args_again();
  for (int i = tid; i < T * cols; i += kFewThreads) {
    const int t = i / cols, c = i - t * cols;
    const float* g = plan.gate + t * (kFewTopK + S);
    const float* y = yrow + c * rows;
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < kFewTopK; ++j) v = fmaf(g[j], y[t * kFewTopK + j], v);
#pragma unroll
    for (int s = 0; s < S; ++s) v = fmaf(g[kFewTopK + s], y[(kFewTopK + s) * T + t], v);
    ActTraits<Y>::store(static_cast<Y*>(p.y) + static_cast<size_t>(t) * d + n0 + c, v);
  }
}

// ------------------------------------------------------------------ host

template <typename X, bool INT8>
static void route(const FewArgs& a, int ctrl, hipStream_t st) {
  const unsigned grid = a.E + a.S + 1 + (INT8 ? a.T : 0);
  if (a.T == 1) few_route_kernel<X, 1, INT8><<<grid, 512, 0, st>>>(a, ctrl);
  else if (a.T == 2) few_route_kernel<X, 2, INT8><<<grid, 512, 0, st>>>(a, ctrl);
  else if (a.T <= 4) few_route_kernel<X, 4, INT8><<<grid, 512, 0, st>>>(a, ctrl);
  else if (a.T <= 8) few_route_kernel<X, 8, INT8><<<grid, 512, 0, st>>>(a, ctrl);
  else few_route_kernel<X, 16, INT8><<<grid, 512, 0, st>>>(a, ctrl);
}

template <class Dot, typename Y>
static void experts(const FewArgs& a, hipStream_t st) {
  if (a.S == 0) few_ffn_kernel<Dot, Y, 0><<<kFewGrid, kFewThreads, 0, st>>>(a);
  else if (a.S == 1) few_ffn_kernel<Dot, Y, 1><<<kFewGrid, kFewThreads, 0, st>>>(a);
  else few_ffn_kernel<Dot, Y, 2><<<kFewGrid, kFewThreads, 0, st>>>(a);
}

hipError_t launch_few(const FewArgs& a, bool act_bf16, FewWeight w, hipStream_t st) {
  if (a.T == 0) return hipSuccess;
  Shape s;
  s.T = a.T;
  s.E = a.E;
  s.S = a.S;
  s.d = a.d;
  const int ctrl = static_cast<int>(few_ctrl_ints(s));
  if (w == FewWeight::kInt8) {
    if (act_bf16) route<bf16_t, true>(a, ctrl, st);
    else route<float, true>(a, ctrl, st);
  } else if (act_bf16) {
    route<bf16_t, false>(a, ctrl, st);
  } else {
    route<float, false>(a, ctrl, st);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (w == FewWeight::kInt8) {
    if (act_bf16) experts<DotI8, bf16_t>(a, st);
    else experts<DotI8, float>(a, st);
  } else if (w == FewWeight::kBf16) {
    experts<DotBf16, bf16_t>(a, st);
  } else {
    experts<DotF32, float>(a, st);
  }
  return hipGetLastError();
}

}  // namespace moe
