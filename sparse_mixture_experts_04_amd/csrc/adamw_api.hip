// C ABI of the AdamW step: host-side validation, the table of tensors and launches
// (include/moe.h has the meaning of every argument).
#include <algorithm>
#include <cmath>
#include <new>
#include <utility>
#include <vector>

#include "../../include/moe.h"
#include "adamw.h"
#include "api.h"

using namespace moe;

namespace {

constexpr int kAdamwMaxTensors = 1 << 20;
constexpr long long kAdamwMaxValues = 1LL << 40;  // of a table

bool on(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

moe_status check_desc(const moe_adamw_desc* d) {
  if (!d) return MOE_ERR_NULL;
  if (d->count < 0) return MOE_ERR_SHAPE;
  if ((d->param != MOE_F32 && d->param != MOE_BF16) || (d->grad != MOE_F32 && d->grad != MOE_BF16))
    return MOE_ERR_DTYPE;
  if (d->state_bits != 32 && d->state_bits != 8) return MOE_ERR_DTYPE;
  return d->count > kAdamwMaxTensors ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

size_t table_bytes(int count) {
  return align_up(sizeof(int64_t) * (static_cast<size_t>(count) + 1)) +
         sizeof(moe_adamw_tensor) * count;
}

AdamwTable table_at(void* p, int count) {
  char* base = static_cast<char*>(p);
  return AdamwTable{reinterpret_cast<int64_t*>(base),
                    reinterpret_cast<moe_adamw_tensor*>(
                        base + align_up(sizeof(int64_t) * (static_cast<size_t>(count) + 1))),
                    count};
}

moe_status check_tensor(const moe_adamw_desc* d, const moe_adamw_tensor& t) {
  if (t.n < 0) return MOE_ERR_SHAPE;
  if (t.n > kAdamwMaxValues) return MOE_ERR_UNSUPPORTED;
  if (t.n == 0) return MOE_OK;
  const bool bits8 = d->state_bits == 8;
  if (!t.p || !t.g || !t.m || !t.v || (bits8 && (!t.m_scale || !t.v_scale))) return MOE_ERR_NULL;
  if ((t.m_values == nullptr) != (t.v_values == nullptr)) return MOE_ERR_NULL;
  if (t.copy && d->param != MOE_F32) return MOE_ERR_DTYPE;
  const size_t ps = d->param == MOE_F32 ? 4 : 2, gs = d->grad == MOE_F32 ? 4 : 2;
  const size_t ss = bits8 ? 1 : 4;
  if (!on(t.p, ps) || !on(t.g, gs) || !on(t.m, ss) || !on(t.v, ss) || !on(t.copy, 2) ||
      !on(t.m_scale, 4) || !on(t.v_scale, 4) || !on(t.m_values, 4) || !on(t.v_values, 4))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Whether two tensors share parameters: both would take the step.
bool shared(const moe_adamw_desc* d, const moe_adamw_tensor* t) {
  std::vector<std::pair<uintptr_t, uintptr_t>> spans;  // first byte, one past the last
  const uintptr_t size = d->param == MOE_F32 ? 4 : 2;
  for (int i = 0; i < d->count; ++i)
    if (t[i].n > 0) {
      const uintptr_t p = reinterpret_cast<uintptr_t>(t[i].p);
      spans.emplace_back(p, p + size * static_cast<uintptr_t>(t[i].n));
    }
  std::sort(spans.begin(), spans.end());
  for (size_t i = 1; i < spans.size(); ++i)
    if (spans[i].first < spans[i - 1].second) return true;
  return false;
}

long long chunks_of(int64_t n) { return (n + kAdamwChunk - 1) / kAdamwChunk; }

}  // namespace

extern "C" {

moe_status moe_adamw_table_size(const moe_adamw_desc* desc, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const moe_status st = check_desc(desc);
  if (st != MOE_OK) return st;
  *bytes = table_bytes(desc->count);
  return MOE_OK;
}

moe_status moe_adamw_prepare(const moe_adamw_desc* desc, const moe_adamw_tensor* tensors,
                             int64_t* chunks, void* table, size_t bytes, hipStream_t stream) {
  moe_status st = check_desc(desc);
  if (st != MOE_OK) return st;
  if (!chunks || (desc->count > 0 && !tensors)) return MOE_ERR_NULL;
  long long total = 0, values = 0;
  for (int i = 0; i < desc->count; ++i) {
    st = check_tensor(desc, tensors[i]);
    if (st != MOE_OK) return st;
    total += chunks_of(tensors[i].n);
    values += tensors[i].n;
    if (values > kAdamwMaxValues) return MOE_ERR_UNSUPPORTED;
  }
  if (!table || bytes < table_bytes(desc->count)) return MOE_ERR_WORKSPACE;
  if (!on(table, 16)) return MOE_ERR_UNSUPPORTED;
  try {
    if (shared(desc, tensors)) return MOE_ERR_UNSUPPORTED;
  } catch (const std::bad_alloc&) {
    return MOE_ERR_WORKSPACE;
  }
  *chunks = total;
  const AdamwTable t = table_at(table, desc->count);
  long long at = 0;
  for (int first = 0; first < desc->count; first += kAdamwBatch) {
    AdamwBatch b{};
    b.n = desc->count - first < kAdamwBatch ? desc->count - first : kAdamwBatch;
    for (int i = 0; i < b.n; ++i) {
      b.tensors[i] = tensors[first + i];
      b.start[i] = at;
      at += chunks_of(tensors[first + i].n);
    }
    b.end = at;
    const hipError_t e = launch_adamw_table(b, first, t, stream);
    if (e != hipSuccess) return MOE_ERR_HIP;
  }
  return MOE_OK;
}

moe_status moe_adamw(const moe_adamw_desc* desc, const moe_adamw_step* step, int64_t chunks,
                     const void* table, hipStream_t stream) {
  const moe_status st = check_desc(desc);
  if (st != MOE_OK) return st;
  if (!step) return MOE_ERR_NULL;
  if (chunks < 0 || (!step->step_dev && step->step < 1)) return MOE_ERR_SHAPE;
  if (!(step->beta1 >= 0.0 && step->beta1 < 1.0) || !(step->beta2 >= 0.0 && step->beta2 < 1.0) ||
      !(step->eps >= 0.0 && step->eps < INFINITY) || !std::isfinite(step->weight_decay) ||
      (!step->lr_dev && !std::isfinite(step->lr)))
    return MOE_ERR_SHAPE;
  if (desc->count == 0 || chunks == 0) return MOE_OK;
  if (!table) return MOE_ERR_NULL;
  if (!on(table, 16) || !on(step->lr_dev, 4) || !on(step->step_dev, 8) ||
      !on(step->grad_scale_dev, 4))
    return MOE_ERR_UNSUPPORTED;
  const double t = static_cast<double>(step->step);
  const AdamwStep s{step->lr,
                    step->beta1,
                    step->beta2,
                    step->eps,
                    step->weight_decay,
                    1.0 - std::pow(step->beta1, t),
                    1.0 - std::pow(step->beta2, t),
                    step->lr_dev,
                    step->step_dev,
                    step->grad_scale_dev};
  return hip_status(launch_adamw(table_at(const_cast<void*>(table), desc->count), s, chunks,
                                 desc->param == MOE_BF16, desc->grad == MOE_BF16,
                                 desc->state_bits == 8, stream));
}

moe_status moe_adamw_state_values(const moe_adamw_desc* desc, int64_t chunks, const void* table,
                                  hipStream_t stream) {
  const moe_status st = check_desc(desc);
  if (st != MOE_OK) return st;
  if (desc->state_bits != 8) return MOE_ERR_DTYPE;
  if (chunks < 0) return MOE_ERR_SHAPE;
  if (desc->count == 0 || chunks == 0) return MOE_OK;
  if (!table) return MOE_ERR_NULL;
  if (!on(table, 16)) return MOE_ERR_UNSUPPORTED;
  return hip_status(
      launch_adamw_values(table_at(const_cast<void*>(table), desc->count), chunks, stream));
}

}  // extern "C"
