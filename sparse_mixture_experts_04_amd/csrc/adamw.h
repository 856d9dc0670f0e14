// Internal declarations of the AdamW step.
#pragma once

#include "../../include/moe.h"
#include "common.h"

namespace moe {

constexpr int kAdamwChunk = 2048;  // values of a work chunk
constexpr int kAdamwBlock = 256;   // values that share a scale of 8-bit states

// The table in device memory: count tensors and the chunks before each.
struct AdamwTable {
  int64_t* start;              // [count + 1]
  moe_adamw_tensor* tensors;   // [count]
  int count;
};

// Tensors that one launch writes into the table, as its arguments.
constexpr int kAdamwBatch = 32;
struct AdamwBatch {
  moe_adamw_tensor tensors[kAdamwBatch];
  int64_t start[kAdamwBatch];
  int64_t end;
  int n;
};
static_assert(sizeof(AdamwBatch) <= 3584, "kernel arguments");

struct AdamwStep {
  double lr, beta1, beta2, eps, weight_decay;
  double c1, c2;   // 1 - beta^step, where the step is known to the host
  const float* lr_dev;
  const int64_t* step_dev;
  const float* grad_scale;
};

hipError_t launch_adamw_table(const AdamwBatch& b, int first, const AdamwTable& t, hipStream_t st);
hipError_t launch_adamw(const AdamwTable& t, const AdamwStep& s, long long chunks, bool param_bf16,
                        bool grad_bf16, bool bits8, hipStream_t st);
hipError_t launch_adamw_values(const AdamwTable& t, long long chunks, hipStream_t st);

}  // namespace moe
