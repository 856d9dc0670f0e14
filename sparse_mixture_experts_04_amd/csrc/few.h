// Internal declarations of the few-token layer.
#pragma once

#include "common.h"

namespace moe {

constexpr int kFewMaxTokens = 16;
constexpr int kFewTopK = 6;

// Weight element type of the few-token layer.
enum class FewWeight { kBf16, kF32, kInt8 };

// Workgroups of the experts' kernel: one per compute unit.
constexpr int kFewGrid = 256;
// Largest d and F.
constexpr int kFewMaxWidth = 16384;
// int32 words of the control block: a flag per workgroup, per token and per
// row of h.
inline size_t few_ctrl_ints(const Shape& s) {
  return kFewGrid + kFewMaxTokens + static_cast<size_t>(kFewTopK + s.S) * s.T;
}

struct FewArgs {
  const void* x;           // [T, d] act
  const float* w_router;   // [E+S, d]
  const float* bias;       // [E]
  const void *w_gate, *w_up, *w_down;      // routed
  const void *ws_gate, *ws_up, *ws_down;   // shared
  const float *t_gate, *t_up, *t_down;     // int8 scales, routed
  const float *ts_gate, *ts_up, *ts_down;  // int8 scales, shared
  void* y;                 // [T, d] act
  int32_t* topk_out;       // [T, 6] or null
  float* gates_out;        // [T, 6 + S] or null
  // workspace; rows of h are the 6 T pairs, then shared expert s's T rows
  double2* zs;             // [T, E+S] log sigmoid (logsumexp gates) and sigmoid of z
  int32_t* topk;           // [T, 6]
  float* gates;            // [T, 6 + S]
  int32_t* ctrl;           // few_ctrl_ints
  int8_t* xq;              // [T, d] codes (int8)
  float* xs;               // [T]
  float* h;                // [rows, F]
  int8_t* hq;              // [rows, F] codes (int8)
  float* hs;               // [rows]
  int T, d, F, E, S;
  bool logsumexp;
  double gate_scale;
};

hipError_t launch_few(const FewArgs& a, bool act_bf16, FewWeight w, hipStream_t st);

}  // namespace moe
