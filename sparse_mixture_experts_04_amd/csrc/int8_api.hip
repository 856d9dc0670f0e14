// C ABI of the 8-bit products and of the few-token layer: host-side
// validation, workspace layout and the order of launches.  Declarations and
// the meaning of every argument are in include/moe.h.
#include <initializer_list>

#include "../../include/moe.h"
#include "api.h"
#include "few.h"
#include "int8.h"

using namespace moe;

namespace {

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// A workspace of `need` bytes at an address that its atomics can take.
moe_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE;
  return aligned16(ws) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

moe_status check_gemm(const moe_gemm_int8_desc* d) {
  if (!d) return MOE_ERR_NULL;
  if (d->M < 0 || d->N < 0 || d->K <= 0 || d->E <= 0) return MOE_ERR_SHAPE;
  if (d->out != MOE_F32 && d->out != MOE_BF16) return MOE_ERR_DTYPE;
  if (d->K > kInt8MaxK || d->E > kInt8MaxGroups || d->M > kInt8MaxRows || d->N > kInt8MaxRows)
    return MOE_ERR_UNSUPPORTED;
  const long long lim = 1LL << 40, kp = code_row(d->K);
  const long long wide = d->N > kp ? d->N : kp;
  if (static_cast<long long>(d->E) * d->N >= lim / kp || d->M >= lim / wide)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The layer descriptor of the 8-bit experts: an ordinary one, without MXFP4.
moe_status check_int8_desc(const moe_desc* d) {
  const moe_status st = check_ffn_desc(d);
  if (st != MOE_OK) return st;
  if (d->weight == MOE_MXFP4) return MOE_ERR_DTYPE;
  if (d->d > kInt8MaxK || d->F > kInt8MaxK) return MOE_ERR_UNSUPPORTED;
  // int32 row numbers: the shared experts' rows follow the T * k routed ones
  if (static_cast<long long>(d->T) * (d->k + d->S) > kInt8MaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_few_desc(const moe_desc* d) {
  const moe_status st = check_ffn_desc(d);
  if (st != MOE_OK) return st;
  if (d->weight == MOE_MXFP4 || d->T > kFewMaxTokens || d->capacity_factor != 0.0f ||
      d->d > kFewMaxWidth || d->F > kFewMaxWidth)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Whether the T tokens' x and y share memory: a workgroup of the few-token layer
// that starts late may still read x when others store y.
bool in_place(const Shape& s, const void* x, const void* y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  const uintptr_t n = static_cast<uintptr_t>(s.T) * s.d * (s.bf16 ? 2 : 4);
  return a < b + n && b < a + n;
}

// Every matrix that is read in 16-byte pieces (pointers a layer does not use
// may hold anything).
bool weights_aligned(const Shape& s, std::initializer_list<const void*> routed,
                     std::initializer_list<const void*> shared) {
  for (const void* p : routed)
    if (!aligned16(p)) return false;
  if (s.S > 0)
    for (const void* p : shared)
      if (!aligned16(p)) return false;
  return true;
}

bool int8_weights_ok(const moe_weights_int8* w, const Shape& s) {
  if (!(w && w->w_gate && w->t_gate && w->w_up && w->t_up && w->w_down && w->t_down)) return false;
  return s.S == 0 || (w->ws_gate && w->ts_gate && w->ws_up && w->ts_up && w->ws_down && w->ts_down);
}

struct FfnInt8Ws {
  int8_t* xq;
  float* xs;
  float* h;
  int8_t* hq;
  float* hs;
  int32_t* counters;
};
FfnInt8Ws carve_ffn_int8(Carver& c, const Shape& s) {
  FfnInt8Ws w;
  const size_t rows = static_cast<size_t>(s.k + s.S) * s.T;
  w.xq = c.take<int8_t>(static_cast<size_t>(s.T) * s.d);
  w.xs = c.take<float>(s.T);
  w.h = c.take<float>(rows * s.F);
  w.hq = c.take<int8_t>(rows * s.F);
  w.hs = c.take<float>(rows);
  w.counters = c.take<int32_t>(gemm_int8_counter_ints());
  return w;
}

// Carves the workspace into a.
void carve_few(Carver& c, const Shape& s, FewArgs& a) {
  const size_t rows = static_cast<size_t>(kFewTopK + s.S) * s.T;
  a.zs = c.take<double2>(static_cast<size_t>(s.T) * (s.E + s.S));
  a.ctrl = c.take<int32_t>(few_ctrl_ints(s));
  a.topk = c.take<int32_t>(static_cast<size_t>(s.T) * kFewTopK);
  a.gates = c.take<float>(static_cast<size_t>(s.T) * (kFewTopK + s.S));
  a.xq = c.take<int8_t>(static_cast<size_t>(s.T) * s.d);
  a.xs = c.take<float>(s.T);
  a.h = c.take<float>(rows * s.F);
  a.hq = c.take<int8_t>(rows * s.F);
  a.hs = c.take<float>(rows);
}

size_t few_ws_bytes(const Shape& s) {
  Carver c{nullptr};
  FewArgs a{};
  carve_few(c, s, a);
  return c.used;
}

// The parts of FewArgs that both forms share, from checked arguments.
FewArgs few_args(const Shape& s, const void* x, const float* w_router, const float* bias, void* y,
                 int32_t* topk, float* gates, void* ws) {
  FewArgs a{};
  a.x = x;
  a.w_router = w_router;
  a.bias = bias;
  a.y = y;
  a.topk_out = topk;
  a.gates_out = gates;
  a.T = s.T;
  a.d = s.d;
  a.F = s.F;
  a.E = s.E;
  a.S = s.S;
  a.logsumexp = s.gate_logsumexp;
  a.gate_scale = s.gate_scale;
  Carver c{static_cast<char*>(ws)};
  carve_few(c, s, a);
  return a;
}

}  // namespace

extern "C" {

moe_status moe_quantize_int8(int64_t rows, int32_t K, moe_dtype dtype, const void* x,
                             int8_t* codes, float* scales, hipStream_t stream) {
  if (rows < 0 || K <= 0) return MOE_ERR_SHAPE;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (K > kInt8MaxK || rows >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales) return MOE_ERR_NULL;
  if (!aligned16(codes)) return MOE_ERR_UNSUPPORTED;
  return hip_status(launch_quantize_int8(rows, K, dtype == MOE_BF16, x, codes, scales, stream));
}

moe_status moe_gemm_int8_workspace_size(const moe_gemm_int8_desc* desc, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const moe_status st = check_gemm(desc);
  if (st != MOE_OK) return st;
  *bytes = gemm_int8_counter_ints() * sizeof(int32_t);
  return MOE_OK;
}

moe_status moe_gemm_int8(const moe_gemm_int8_desc* desc, const int8_t* a, const float* a_scale,
                         const int8_t* w, const float* w_scale, const int32_t* offsets, void* y,
                         void* ws, size_t ws_bytes, hipStream_t stream) {
  moe_status st = check_gemm(desc);
  if (st != MOE_OK) return st;
  if (desc->M == 0 || desc->N == 0) return MOE_OK;
  if (!a || !a_scale || !w || !w_scale || !y || (!offsets && desc->E != 1)) return MOE_ERR_NULL;
  if (!aligned16(a) || !aligned16(w) || !aligned16(y)) return MOE_ERR_UNSUPPORTED;
  st = check_ws(ws, ws_bytes, gemm_int8_counter_ints() * sizeof(int32_t));
  if (st != MOE_OK) return st;
  Int8Args g{};
  g.a = a;
  g.a_scale = a_scale;
  g.w0 = w;
  g.t0 = w_scale;
  g.offsets = offsets;
  g.out = y;
  g.M = desc->M;
  g.N = desc->N;
  g.Kp = static_cast<int>(code_row(desc->K));
  g.E = desc->E;
  g.k = 1;
  g.out_bf16 = desc->out == MOE_BF16;
  bool cleared = false;
  return hip_status(launch_gemm_int8(g, false, static_cast<int32_t*>(ws), cleared, stream));
}

moe_status moe_expert_ffn_int8_workspace_size(const moe_desc* desc, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const moe_status st = check_int8_desc(desc);
  if (st != MOE_OK) return st;
  Carver c{nullptr};
  carve_ffn_int8(c, to_shape(desc));
  *bytes = c.used;
  return MOE_OK;
}

moe_status moe_expert_ffn_int8(const moe_desc* desc, const void* x, const moe_weights_int8* w,
                               const int32_t* offsets, const int32_t* sorted_pair, void* y_routed,
                               void* y_shared, void* ws, size_t ws_bytes, hipStream_t stream) {
  size_t need = 0;
  moe_status st = moe_expert_ffn_int8_workspace_size(desc, &need);
  if (st != MOE_OK) return st;
  const Shape s = to_shape(desc);
  if (!int8_weights_ok(w, s) || !offsets) return MOE_ERR_NULL;
  if (s.T > 0 && (!x || !sorted_pair || !y_routed || (s.S > 0 && !y_shared))) return MOE_ERR_NULL;
  if (!aligned16(x) || !aligned16(y_routed) || (s.S > 0 && !aligned16(y_shared)) ||
      !weights_aligned(s, {w->w_gate, w->w_up, w->w_down}, {w->ws_gate, w->ws_up, w->ws_down}))
    return MOE_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, need)) != MOE_OK) return st;
  if (s.T == 0) return MOE_OK;
  Carver c{static_cast<char*>(ws)};
  const FfnInt8Ws f = carve_ffn_int8(c, s);
  const int pairs = s.T * s.k, rows = s.T * (s.k + s.S);
  hipError_t e = launch_quantize_int8(s.T, s.d, s.bf16, x, f.xq, f.xs, stream);
  Int8Args g{};
  g.a = f.xq;
  g.a_scale = f.xs;
  g.w0 = w->w_gate;
  g.w1 = w->w_up;
  g.t0 = w->t_gate;
  g.t1 = w->t_up;
  g.ws0 = w->ws_gate;
  g.ws1 = w->ws_up;
  g.ts0 = w->ts_gate;
  g.ts1 = w->ts_up;
  g.offsets = offsets;
  g.sorted_pair = sorted_pair;
  g.out = f.h;
  g.out_shared = f.h + static_cast<size_t>(pairs) * s.F;
  g.M = pairs;
  g.N = s.F;
  g.Kp = s.d;
  g.E = s.E;
  g.S = s.S;
  g.T = s.T;
  g.k = s.k;
  bool cleared = false;
  if (e == hipSuccess) e = launch_gemm_int8(g, true, f.counters, cleared, stream);
  if (e == hipSuccess) e = launch_quantize_int8(rows, s.F, false, f.h, f.hq, f.hs, stream);
  g.a = f.hq;
  g.a_scale = f.hs;
  g.w0 = w->w_down;
  g.t0 = w->t_down;
  g.ws0 = w->ws_down;
  g.ts0 = w->ts_down;
  g.out = y_routed;
  g.out_shared = y_shared;
  g.N = s.d;
  g.Kp = s.F;
  g.out_bf16 = s.bf16;
  if (e == hipSuccess) e = launch_gemm_int8(g, false, f.counters, cleared, stream);
  return hip_status(e);
}

moe_status moe_forward_few_workspace_size(const moe_desc* desc, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const moe_status st = check_few_desc(desc);
  if (st != MOE_OK) return st;
  *bytes = few_ws_bytes(to_shape(desc));
  return MOE_OK;
}

moe_status moe_forward_few(const moe_desc* desc, const void* x, const moe_weights* w,
                           const float* bias, void* y, int32_t* topk_idx, float* gates, void* ws,
                           size_t ws_bytes, hipStream_t stream) {
  moe_status st = check_few_desc(desc);
  if (st != MOE_OK) return st;
  const Shape s = to_shape(desc);
  if (!weights_ok(w, s) || !w->w_router || !bias) return MOE_ERR_NULL;
  if (s.T > 0 && (!x || !y)) return MOE_ERR_NULL;
  // MXFP4 codes are a quarter of the bytes this call would read
  if (w->sc_gate || w->sc_up || w->sc_down) return MOE_ERR_DTYPE;
  if (in_place(s, x, y) || !aligned16(x) || !aligned16(w->w_router) ||
      !weights_aligned(s, {w->w_gate, w->w_up, w->w_down}, {w->ws_gate, w->ws_up, w->ws_down}))
    return MOE_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, few_ws_bytes(s))) != MOE_OK) return st;
  FewArgs a = few_args(s, x, w->w_router, bias, y, topk_idx, gates, ws);
  a.w_gate = w->w_gate;
  a.w_up = w->w_up;
  a.w_down = w->w_down;
  a.ws_gate = w->ws_gate;
  a.ws_up = w->ws_up;
  a.ws_down = w->ws_down;
  return hip_status(launch_few(a, s.bf16, s.bf16 ? FewWeight::kBf16 : FewWeight::kF32, stream));
}

moe_status moe_forward_few_int8(const moe_desc* desc, const void* x, const moe_weights_int8* w,
                                const float* bias, void* y, int32_t* topk_idx, float* gates,
                                void* ws, size_t ws_bytes, hipStream_t stream) {
  moe_status st = check_few_desc(desc);
  if (st != MOE_OK) return st;
  const Shape s = to_shape(desc);
  if (!int8_weights_ok(w, s) || !w->w_router || !bias) return MOE_ERR_NULL;
  if (s.T > 0 && (!x || !y)) return MOE_ERR_NULL;
  if (in_place(s, x, y) || !aligned16(x) || !aligned16(w->w_router) ||
      !weights_aligned(s, {w->w_gate, w->w_up, w->w_down}, {w->ws_gate, w->ws_up, w->ws_down}))
    return MOE_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, few_ws_bytes(s))) != MOE_OK) return st;
  FewArgs a = few_args(s, x, w->w_router, bias, y, topk_idx, gates, ws);
  a.w_gate = w->w_gate;
  a.w_up = w->w_up;
  a.w_down = w->w_down;
  a.ws_gate = w->ws_gate;
  a.ws_up = w->ws_up;
  a.ws_down = w->ws_down;
  a.t_gate = w->t_gate;
  a.t_up = w->t_up;
  a.t_down = w->t_down;
  a.ts_gate = w->ts_gate;
  a.ts_up = w->ts_up;
  a.ts_down = w->ts_down;
  return hip_status(launch_few(a, s.bf16, FewWeight::kInt8, stream));
}

}  // extern "C"
