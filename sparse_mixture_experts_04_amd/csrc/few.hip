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
//   down         blocks of 16 output columns, all contributors of a block by
//                one workgroup (or `parts` of them), so that each y is summed
//                where it is made.
//
// Between the stages workgroups wait for flags that others set.  A wait ends
// whatever else runs on the device: a flag says not started, started or done;
// work that has been started is held by a running workgroup and finishes
// (gate/up waits for the selection only, the selection for nothing), and work
// that no workgroup has started is done by the one that waits for it.  Two
// workgroups may then do the same piece: they write the same bits.  The down
// stage is waited for by nobody, except that the last of a block's parts adds
// them up.  (Handing items out by one counter cost 70 ns an item on this
// device, more than an item's weights take.)
//
// No sum depends on timing: products are split over waves and parts by the
// sizes alone, and added in a fixed order.
//
// Precision: logits, affinities and gates in fp64 (the selection is that of
// exact arithmetic but for keys within ~1e-15); products on the matrix cores
// with fp32 (or exact int32) accumulation; h and the experts' outputs in fp32.
// With bf16 weights h enters the down product as two bf16 terms (h = hi + lo
// to 2^-17): the second product costs no memory traffic.  With 8-bit weights x
// is quantised per token and h per row.
#include "few.h"
#include "int8_quant.h"
#include "select.h"
#include "stream.h"

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
// in fp64, sums in a fixed order).  Block E + S clears the control block of
// few_ffn_kernel.  INT8: block E + S + 1 + t quantises token t.  TM: tokens
// rounded up to a power of two.
template <typename X, int TM, bool INT8>
__global__ __launch_bounds__(256) void few_route_kernel(FewArgs p, int ctrl_ints) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = blockIdx.x;
  const int rows = p.E + p.S;
  const X* x = static_cast<const X*>(p.x);
  if (b == rows) {
    for (int i = tid; i < ctrl_ints; i += 256) p.ctrl[i] = 0;  // kIdle
    return;
  }
  if (INT8 && b > rows) {
    const int t = b - rows - 1;
    const float s = quantize_row<X, true, 256>(x + static_cast<size_t>(t) * p.d, p.d, p.d,
                                          p.xq + static_cast<size_t>(t) * p.d);
    if (tid == 0) p.xs[t] = s;
    return;
  }
  double acc[TM];
#pragma unroll
  for (int t = 0; t < TM; ++t) acc[t] = 0.0;
  const float* w = p.w_router + static_cast<size_t>(b) * p.d;
  for (int c = tid * 4; c < p.d; c += 1024) {
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
  __shared__ double sum[4][TM];
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const double v = wave_sum(acc[t], lane);
    if (lane == 0) sum[wave][t] = v;
  }
  __syncthreads();
  if (tid < p.T)
    p.z[static_cast<size_t>(tid) * rows + b] =
        ((sum[0][tid] + sum[1][tid]) + sum[2][tid]) + sum[3][tid];
}

// --------------------------------------------------------------- the experts

// Top-6, gates of token t by one wave.  A NaN key ranks last (the gates of
// such a token are NaN, and so is its output).
template <int S>
__device__ __forceinline__ void few_select(const FewArgs& p, int t, int lane) {
  __shared__ int32_t s_topk[kFewTopK];
  __shared__ float s_gates[kFewTopK + S];
  constexpr int EPL = 4;  // experts per lane; those past E are no candidates
  const double* z = p.z + static_cast<size_t>(t) * (p.E + S);
  double zv[EPL], sv[EPL], key[EPL];
  bool valid[EPL];
#pragma unroll
  for (int q = 0; q < EPL; ++q) {
    const int e = lane + 64 * q;
    valid[q] = e < p.E;
    zv[q] = valid[q] ? z[e] : 0.0;
    sv[q] = sigmoid64(zv[q]);
    const double k = valid[q] ? sv[q] + static_cast<double>(p.bias[e]) : 0.0;
    key[q] = k == k ? k : -INFINITY;
  }
  const double z_sh = lane < S ? z[p.E + lane] : 0.0;
  int i_sel[kFewTopK];
  double s_pick[kFewTopK], z_pick[kFewTopK], k_sel[kFewTopK + 1];
  rank_rounds<kFewTopK, EPL>(lane, valid, key, sv, zv, i_sel, s_pick, z_pick, k_sel);
  write_token<kFewTopK, S>(0, lane, i_sel, s_pick, z_pick, sigmoid64(z_sh), z_sh, k_sel, s_topk,
                           s_gates, nullptr, p.logsumexp, p.gate_scale);
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");  // LDS of one wave, in order
  if (lane < kFewTopK) {
    agent_store(p.topk + t * kFewTopK + lane, s_topk[lane]);
    if (p.topk_out) p.topk_out[t * kFewTopK + lane] = s_topk[lane];
  }
  if (lane < kFewTopK + S) {
    agent_store(p.gates + t * (kFewTopK + S) + lane, s_gates[lane]);
    if (p.gates_out) p.gates_out[t * (kFewTopK + S) + lane] = s_gates[lane];
  }
}

// States of a flag.
enum { kIdle = 0, kStarted = 1, kDone = 2 };

constexpr int kFewThreads = 512;
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

struct FewPlan {
  int topk[kFewMaxTokens * kFewTopK];
  int pair[kFewMaxTokens * kFewTopK];     // pairs grouped by expert, ascending
  int expert[kFewMaxTokens * kFewTopK];   // active experts, ascending
  int start[kFewMaxTokens * kFewTopK + 1];  // first entry of pair[] per active expert
  int active;
};

// Groups the 6 T pairs by expert (the first 256 threads stand for an expert
// each).
__device__ __forceinline__ void few_plan(const FewArgs& p, FewPlan& s) {
  __shared__ int wact[kFewWaves], wrow[kFewWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = p.T * kFewTopK;
  if (tid < n) {
    const int e = agent_load(p.topk + tid);
    s.topk[tid] = e < 0 ? 0 : e >= p.E ? p.E - 1 : e;
  }
  __syncthreads();
  int cnt = 0;  // pairs of expert tid
  for (int i = 0; i < n; ++i) cnt += s.topk[i] == tid ? 1 : 0;
  int rows = cnt, act = cnt > 0 ? 1 : 0;
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(rows, o), v = __shfl_up(act, o);
    if (lane >= o) {
      rows += u;
      act += v;
    }
  }
  if (lane == 63) {
    wrow[wave] = rows;
    wact[wave] = act;
  }
  __syncthreads();
  for (int w = 0; w < wave; ++w) {
    rows += wrow[w];
    act += wact[w];
  }
  if (cnt > 0) {
    s.expert[act - 1] = tid;
    int at = rows - cnt;
    s.start[act - 1] = at;
    for (int i = 0; i < n; ++i)
      if (s.topk[i] == tid) s.pair[at++] = i;
  }
  if (tid == kFewThreads - 1) {
    s.active = act;
    s.start[act] = rows;
  }
  __syncthreads();
}

template <class Op> struct FewTraits;
template <> struct FewTraits<OpBf16> { static constexpr int ESZ = 2, PLANES = 2; };
template <> struct FewTraits<OpF32> { static constexpr int ESZ = 4, PLANES = 1; };
template <> struct FewTraits<OpI8> { static constexpr int ESZ = 1, PLANES = 1; };

// Shared memory of few_ffn_kernel outside the plan.
template <class Op>
union FewLds {
  typename Op::Acc red[2][kFewWaves][4][64];              // gate/up: partial tiles
  float ysum[kFewWaves][kFewMaxTokens][16];               // down: each wave's share of y
};

// Group of CT tiles of expert e: tile c is 8 columns from f0 + 8 c on, its 16
// weight rows the 8 W_gate rows of these columns, then the 8 W_up rows.  The
// waves split K.  wave c then finishes tile c: h = silu(gate) * up of the R
// rows of the group.
template <class Op, int CT>
__device__ __forceinline__ void few_gate_up(const FewArgs& p, const void* wg, const void* wu,
                                            const float* tg, const float* tu, int e, int f0,
                                            int R, int tok, int row, int rows,
                                            typename Op::Acc (&red)[kFewWaves][4][64]) {
  using Acc = typename Op::Acc;
  constexpr int ESZ = FewTraits<Op>::ESZ, PL = FewTraits<Op>::PLANES;
  constexpr bool I8 = ESZ == 1;
  constexpr int U = CT == 1 ? 4 : CT == 2 ? 2 : 1;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, quad = lane >> 4;
  const size_t kbytes = static_cast<size_t>(p.d) * ESZ;
  const int steps = static_cast<int>(kbytes / kStepBytes);
  const int s0 = wave * steps / kFewWaves, s1 = (wave + 1) * steps / kFewWaves;
  const size_t at = static_cast<size_t>(s0) * kStepBytes + quad * 16;
  const char* w0 = static_cast<const char*>(r16 < 8 ? wg : wu) +
                   (static_cast<size_t>(e) * p.F + f0 + (r16 & 7)) * kbytes + at;
  const char* wp[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) wp[c] = w0 + 8 * c * kbytes;
  const char* a = I8 ? reinterpret_cast<const char*>(p.xq) : static_cast<const char*>(p.x);
  const char* ap[1] = {a + tok * kbytes + at};
  Acc acc[CT][1];
#pragma unroll
  for (int c = 0; c < CT; ++c) acc[c][0] = Acc{0, 0, 0, 0};
  stream_dot<Op, CT, 1, U>(wp, ap, s1 - s0, acc);
#pragma unroll
  for (int c = 0; c < CT; ++c) red[wave][c][lane] = acc[c][0];
  __syncthreads();
  if (wave >= CT) return;
  Acc v{0, 0, 0, 0};
#pragma unroll
  for (int w = 0; w < kFewWaves; ++w) v += red[w][wave][lane];
  const int f = f0 + 8 * wave + 4 * (quad & 1);
  float hv[4];
  float sx = 1.0f;
  if (I8) sx = p.xs[tok];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float gt = static_cast<float>(v[i]);
    if (I8) gt *= sx * (quad < 2 ? tg : tu)[static_cast<size_t>(e) * p.F + f + i];
    const float up = __shfl_xor(gt, 32);  // lanes 0-31 hold gate, 32-63 up
    hv[i] = gt / (1.0f + expf(-gt)) * up;
  }
  if (quad >= 2 || r16 >= R) return;
  if (PL == 2) {  // h = hi + lo in bf16
    bf16_t* hh = static_cast<bf16_t*>(p.h) + static_cast<size_t>(row) * p.F + f;
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bf16_t h0 = f32_to_bf16(hv[2 * i]), h1 = f32_to_bf16(hv[2 * i + 1]);
      hi[i] = h0 | (static_cast<uint32_t>(h1) << 16);
      lo[i] = f32_to_bf16(hv[2 * i] - bf16_to_f32(h0)) |
              (static_cast<uint32_t>(f32_to_bf16(hv[2 * i + 1] - bf16_to_f32(h1))) << 16);
    }
    agent_store(reinterpret_cast<uint64_t*>(hh), hi[0] | (static_cast<uint64_t>(hi[1]) << 32));
    agent_store(reinterpret_cast<uint64_t*>(hh + static_cast<size_t>(rows) * p.F),
                lo[0] | (static_cast<uint64_t>(lo[1]) << 32));
  } else {
    uint64_t* hh = reinterpret_cast<uint64_t*>(static_cast<float*>(p.h) +
                                               static_cast<size_t>(row) * p.F + f);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      agent_store(hh + i, __float_as_uint(hv[2 * i]) |
                              (static_cast<uint64_t>(__float_as_uint(hv[2 * i + 1])) << 32));
  }
}

template <class Op, typename Y, int S>
__global__ __launch_bounds__(kFewThreads, 4) void few_ffn_kernel(FewArgs p) {
  using Acc = typename Op::Acc;
  constexpr int ESZ = FewTraits<Op>::ESZ, PL = FewTraits<Op>::PLANES;
  constexpr bool I8 = ESZ == 1;
  __shared__ FewPlan plan;
  __shared__ FewLds<Op> lds;
  __shared__ int s_word;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, quad = lane >> 4;
  const int grid = gridDim.x;
  const int T = p.T, tiles = p.F / 8;  // gate/up tiles per expert
  const int pairs = T * kFewTopK, rows = pairs + S * T;
  int32_t* chunk_flag = p.ctrl;                 // [grid]
  int32_t* token_flag = p.ctrl + kFewGrid;      // [T]
  int32_t* row_flag = token_flag + kFewMaxTokens;  // [rows] (8-bit weights)
  int32_t* col_count = row_flag + rows;         // [d / 16]
  bool planned = false;

  if (tid == 0 && agent_load(chunk_flag + blockIdx.x) == kIdle) {
    if (blockIdx.x < T) agent_store(token_flag + blockIdx.x, kStarted);
    agent_store(chunk_flag + blockIdx.x, kStarted);
  }
  // ---- gate/up: this workgroup's chunk, then any that nobody has started
  int buf = 0;
  int token = blockIdx.x < T ? static_cast<int>(blockIdx.x) : -1;  // to be selected here
  for (int chunk = blockIdx.x; chunk >= 0;
       chunk = wait_all(chunk_flag, grid, blockIdx.x, &s_word)) {
    for (int part = S > 0 ? 0 : 1; part < 2;) {  // shared, then routed experts
      if (token >= 0) {
        if (wave == 0) few_select<S>(p, token, lane);
        mark_done(token_flag, token);
        token = -1;
      }
      if (part == 1 && !planned) {
        token = wait_all(token_flag, T, 0, &s_word);
        if (token >= 0) continue;
        few_plan(p, plan);
        planned = true;
      }
      const long long n = static_cast<long long>(part == 0 ? S : plan.active) * tiles;
      const int t1 = static_cast<int>(n * (chunk + 1) / grid);
      for (int t = static_cast<int>(n * chunk / grid); t < t1;) {
        const int g = t / tiles, left = min(t1, (g + 1) * tiles) - t;
        const int ct = left < 4 ? left : 4;
        const bool shared = part == 0;
        const int e = shared ? g : plan.expert[g];
        const int R = shared ? T : plan.start[g + 1] - plan.start[g];
        const int rr = r16 < R ? r16 : 0;  // spare columns repeat row 0
        const int pair = shared ? 0 : plan.pair[plan.start[g] + rr];
        const int row = shared ? pairs + g * T + rr : pair;
        const int tok = shared ? rr : pair / kFewTopK;
        const int f0 = (t - g * tiles) * 8;
        const void* wg = shared ? p.ws_gate : p.w_gate;
        const void* wu = shared ? p.ws_up : p.w_up;
        const float* tg = shared ? p.ts_gate : p.t_gate;
        const float* tu = shared ? p.ts_up : p.t_up;
        // two sets of partial tiles in turn: one barrier per group
        auto& red = lds.red[buf];
        buf ^= 1;
        if (ct == 4) few_gate_up<Op, 4>(p, wg, wu, tg, tu, e, f0, R, tok, row, rows, red);
        else if (ct == 3) few_gate_up<Op, 3>(p, wg, wu, tg, tu, e, f0, R, tok, row, rows, red);
        else if (ct == 2) few_gate_up<Op, 2>(p, wg, wu, tg, tu, e, f0, R, tok, row, rows, red);
        else few_gate_up<Op, 1>(p, wg, wu, tg, tu, e, f0, R, tok, row, rows, red);
        t += ct;
      }
      ++part;
    }
    mark_done(chunk_flag, chunk);
  }

  // ---- 8-bit weights: row r of h quantised by workgroup r
  if (I8) {
    if (tid == 0 && static_cast<int>(blockIdx.x) < rows &&
        agent_load(row_flag + blockIdx.x) == kIdle)
      agent_store(row_flag + blockIdx.x, kStarted);
    for (int r = static_cast<int>(blockIdx.x) < rows ? static_cast<int>(blockIdx.x) : -2;
         r != -1; r = wait_all(row_flag, rows, blockIdx.x % rows, &s_word)) {
      if (r < 0) continue;
      const uint64_t* hr = reinterpret_cast<const uint64_t*>(static_cast<const float*>(p.h) +
                                                             static_cast<size_t>(r) * p.F);
      uint64_t* qr = reinterpret_cast<uint64_t*>(p.hq + static_cast<size_t>(r) * p.F);
      const float s = quantize_row<kFewThreads>(
          p.F, p.F,
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

  // ---- down: unit u is block u / parts of 16 output columns, part u % parts.
  // The steps of all contributors (shared experts, then the active ones in
  // ascending order) form one list; part and wave take an equal share of it.
  const int contributors = S + plan.active;
  const size_t kbytes = static_cast<size_t>(p.F) * ESZ;
  const int steps = static_cast<int>(kbytes / kStepBytes);
  const long long list = static_cast<long long>(contributors) * steps;
  const int slices = p.parts * kFewWaves;
  for (int u = blockIdx.x; u < p.d / 16 * p.parts; u += grid) {
    const int blk = u / p.parts, part = u % p.parts;
    for (int i = tid; i < kFewWaves * kFewMaxTokens * 16; i += kFewThreads)
      (&lds.ysum[0][0][0])[i] = 0.0f;
    __syncthreads();
    const int slice = part * kFewWaves + wave;
    const long long l1 = list * (slice + 1) / slices;
    for (long long l = list * slice / slices; l < l1;) {
      const int ci = static_cast<int>(l / steps);
      const int s0 = static_cast<int>(l - static_cast<long long>(ci) * steps);
      const int n = static_cast<int>(min(static_cast<long long>(steps - s0), l1 - l));
      const bool shared = ci < S;
      const int g = ci - S;
      const int e = shared ? ci : plan.expert[g];
      const int R = shared ? T : plan.start[g + 1] - plan.start[g];
      const int rr = r16 < R ? r16 : 0;
      const int pair = shared ? 0 : plan.pair[plan.start[g] + rr];
      const int row = shared ? pairs + ci * T + rr : pair;
      const size_t at = static_cast<size_t>(s0) * kStepBytes + quad * 16;
      const char* wp[1] = {static_cast<const char*>(shared ? p.ws_down : p.w_down) +
                           (static_cast<size_t>(e) * p.d + blk * 16 + r16) * kbytes + at};
      const char* hb = I8 ? reinterpret_cast<const char*>(p.hq) : static_cast<const char*>(p.h);
      const char* ap[PL];
#pragma unroll
      for (int t = 0; t < PL; ++t)
        ap[t] = hb + (static_cast<size_t>(t) * rows + row) * kbytes + at;
      Acc acc[1][PL];
#pragma unroll
      for (int t = 0; t < PL; ++t) acc[0][t] = Acc{0, 0, 0, 0};
      stream_dot<Op, 1, PL, PL == 2 ? 3 : 4, true>(wp, ap, n, acc);
      if (r16 < R) {
        const int tok = shared ? rr : pair / kFewTopK;
        const int slot = shared ? kFewTopK + ci : pair % kFewTopK;
        float gate = agent_load(p.gates + tok * (kFewTopK + S) + slot);
        if (I8) gate *= agent_load(p.hs + row);
        float4* ys = reinterpret_cast<float4*>(&lds.ysum[wave][tok][4 * quad]);
        float4 o = *ys;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = static_cast<float>(acc[0][0][i]);
          if (PL == 2) v[i] += static_cast<float>(acc[0][PL - 1][i]);
          if (I8)
            v[i] *= (shared ? p.ts_down : p.t_down)[static_cast<size_t>(e) * p.d + blk * 16 +
                                                    4 * quad + i];
        }
        o.x = fmaf(gate, v[0], o.x);
        o.y = fmaf(gate, v[1], o.y);
        o.z = fmaf(gate, v[2], o.z);
        o.w = fmaf(gate, v[3], o.w);
        *ys = o;
      }
      l += n;
    }
    __syncthreads();
    const int t = tid >> 4, c = blk * 16 + (tid & 15);  // 16 T <= 256 threads
    float v = 0.0f;
    if (t < T) {
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w) v += lds.ysum[w][t][tid & 15];
    }
    if (p.parts > 1) {
      if (t < T) agent_store(p.ypart + (static_cast<size_t>(part) * T + t) * p.d + c, v);
      drain_stores();
      if (tid == 0)
        s_word = __hip_atomic_fetch_add(col_count + blk, 1, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT) == p.parts - 1;
      __syncthreads();
      if (s_word && t < T) {
        v = 0.0f;
        for (int q = 0; q < p.parts; ++q)
          v += agent_load(p.ypart + (static_cast<size_t>(q) * T + t) * p.d + c);
        ActTraits<Y>::store(static_cast<Y*>(p.y) + static_cast<size_t>(t) * p.d + c, v);
      }
      __syncthreads();
    } else if (t < T) {
      ActTraits<Y>::store(static_cast<Y*>(p.y) + static_cast<size_t>(t) * p.d + c, v);
    }
  }
}

// ------------------------------------------------------------------ host

template <typename X, bool INT8>
static void route(const FewArgs& a, int ctrl, hipStream_t st) {
  const unsigned grid = a.E + a.S + 1 + (INT8 ? a.T : 0);
  if (a.T == 1) few_route_kernel<X, 1, INT8><<<grid, 256, 0, st>>>(a, ctrl);
  else if (a.T == 2) few_route_kernel<X, 2, INT8><<<grid, 256, 0, st>>>(a, ctrl);
  else if (a.T <= 4) few_route_kernel<X, 4, INT8><<<grid, 256, 0, st>>>(a, ctrl);
  else if (a.T <= 8) few_route_kernel<X, 8, INT8><<<grid, 256, 0, st>>>(a, ctrl);
  else few_route_kernel<X, 16, INT8><<<grid, 256, 0, st>>>(a, ctrl);
}

template <class Op, typename Y>
static void experts(const FewArgs& a, hipStream_t st) {
  if (a.S == 0) few_ffn_kernel<Op, Y, 0><<<kFewGrid, kFewThreads, 0, st>>>(a);
  else if (a.S == 1) few_ffn_kernel<Op, Y, 1><<<kFewGrid, kFewThreads, 0, st>>>(a);
  else few_ffn_kernel<Op, Y, 2><<<kFewGrid, kFewThreads, 0, st>>>(a);
}

// Parts of the column blocks: enough that the last round of workgroups is
// nearly full (a narrow layer has fewer blocks than there are workgroups).
static int column_parts(int d) {
  const int blocks = d / 16;
  int best = 1;
  double least = 0.0;
  for (int q = 1; q <= kFewMaxParts; ++q) {
    const double rounds = static_cast<double>((blocks * q + kFewGrid - 1) / kFewGrid);
    const double cost = rounds / q;  // of one round over whole blocks
    if (q == 1 || cost < 0.9 * least) {
      best = q;
      least = cost;
    }
  }
  return best;
}

hipError_t launch_few(const FewArgs& args, bool act_bf16, FewWeight w, hipStream_t st) {
  if (args.T == 0) return hipSuccess;
  FewArgs a = args;
  a.parts = column_parts(a.d);
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
    if (act_bf16) experts<OpI8, bf16_t>(a, st);
    else experts<OpI8, float>(a, st);
  } else if (w == FewWeight::kBf16) {
    experts<OpBf16, bf16_t>(a, st);
  } else {
    experts<OpF32, float>(a, st);
  }
  return hipGetLastError();
}

}  // namespace moe
