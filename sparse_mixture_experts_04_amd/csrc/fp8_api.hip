// C ABI of the e4m3 products: host-side validation and launches (include/moe.h has
// the meaning of every argument).
#include "../../include/moe.h"
#include "api.h"
#include "fp8.h"

using namespace moe;

namespace {

constexpr int kFp8MaxK = 131072;
constexpr long long kFp8MaxRows = (1LL << 31) - 1024;  // rounded up to a tile: 32 bits

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }
bool on_value(const void* p, moe_dtype t) {
  return reinterpret_cast<uintptr_t>(p) % (t == MOE_BF16 ? 2 : 4) == 0;
}

moe_status check_gemm(const moe_gemm_fp8_desc* d) {
  if (!d) return MOE_ERR_NULL;
  if (d->M < 0 || d->N < 0 || d->K <= 0 || d->E <= 0) return MOE_ERR_SHAPE;
  if (d->out != MOE_F32 && d->out != MOE_BF16) return MOE_ERR_DTYPE;
  if (d->K > kFp8MaxK || d->E > kMaxGroups || d->M > kFp8MaxRows || d->N > kFp8MaxRows)
    return MOE_ERR_UNSUPPORTED;
  const long long lim = 1LL << 40, kp = fp8_row(d->K), wide = d->N > kp ? d->N : kp;
  if (static_cast<long long>(d->E) * d->N >= lim / kp || d->M >= lim / wide)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Slices of K whose sums the workspace holds (1: none).
int slices(const moe_gemm_fp8_desc* d) {
  const int kp = static_cast<int>(fp8_row(d->K));
  return d->M == 0 || d->N == 0 || fp8_blocks(d->M, d->N, kp, d->E)
             ? 1
             : fp8_splits(d->M, d->N, kp, d->E);
}
size_t ws_bytes_of(const moe_gemm_fp8_desc* d) {
  const int s = slices(d);
  return s > 1 ? static_cast<size_t>(s) * d->M * d->N * sizeof(float) : 0;
}

}  // namespace

extern "C" {

moe_status moe_quantize_fp8(int64_t rows, int32_t K, moe_dtype dtype, const void* x,
                            uint8_t* codes, float* scales, hipStream_t stream) {
  if (rows < 0 || K <= 0) return MOE_ERR_SHAPE;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (K > kFp8MaxK || rows > kFp8MaxRows) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales) return MOE_ERR_NULL;
  if (!aligned16(codes) || !aligned4(scales) || !on_value(x, dtype)) return MOE_ERR_UNSUPPORTED;
  return hip_status(launch_quantize_fp8(rows, K, dtype == MOE_BF16, x, codes, scales, stream));
}

moe_status moe_quantize_fp8_weights(int32_t E, int32_t N, int32_t K, moe_dtype dtype,
                                    const void* w, uint8_t* codes, float* scales,
                                    hipStream_t stream) {
  if (E < 0 || N < 0 || K <= 0) return MOE_ERR_SHAPE;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
  // a workgroup for each block: its place is a grid index
  if (K > kFp8MaxK || E > 65535 || N > 65535 * kFp8Block) return MOE_ERR_UNSUPPORTED;
  if (E == 0 || N == 0) return MOE_OK;
  if (static_cast<long long>(E) * N >= (1LL << 40) / fp8_row(K)) return MOE_ERR_UNSUPPORTED;
  if (!w || !codes || !scales) return MOE_ERR_NULL;
  if (!aligned16(codes) || !aligned4(scales) || !on_value(w, dtype)) return MOE_ERR_UNSUPPORTED;
  return hip_status(
      launch_quantize_fp8_weights(E, N, K, dtype == MOE_BF16, w, codes, scales, stream));
}

moe_status moe_gemm_fp8_workspace_size(const moe_gemm_fp8_desc* desc, size_t* bytes) {
  if (!bytes) return MOE_ERR_NULL;
  const moe_status st = check_gemm(desc);
  if (st != MOE_OK) return st;
  *bytes = ws_bytes_of(desc);
  return MOE_OK;
}

moe_status moe_gemm_fp8(const moe_gemm_fp8_desc* desc, const uint8_t* a, const float* a_scale,
                        const uint8_t* w, const float* w_scale, const int32_t* offsets, void* y,
                        void* ws, size_t ws_bytes, hipStream_t stream) {
  moe_status st = check_gemm(desc);
  if (st != MOE_OK) return st;
  if (desc->M == 0 || desc->N == 0) return MOE_OK;
  if (!a || !a_scale || !w || !w_scale || !y || (!offsets && desc->E != 1)) return MOE_ERR_NULL;
  if (!aligned16(a) || !aligned16(w) || !aligned16(y) || !aligned4(a_scale) ||
      !aligned4(w_scale) || !aligned4(offsets))
    return MOE_ERR_UNSUPPORTED;
  const size_t need = ws_bytes_of(desc);
  if (need > 0 && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  if (!aligned16(ws)) return MOE_ERR_UNSUPPORTED;
  Fp8Args g{};
  g.part = static_cast<float*>(ws);
  g.splits = slices(desc);
  g.a = a;
  g.a_scale = a_scale;
  g.w = w;
  g.w_scale = w_scale;
  g.offsets = offsets;
  g.out = y;
  g.M = desc->M;
  g.N = desc->N;
  g.Kp = static_cast<int>(fp8_row(desc->K));
  g.E = desc->E;
  g.out_bf16 = desc->out == MOE_BF16;
  return hip_status(launch_gemm_fp8(g, stream));
}

}  // extern "C"
