// Kernel of an e4m3 product.
#include "fp8.h"
#include "stream.h"

namespace moe {

bool fp8_streams(int M, int N, int Kp, int E) { return E == 1 ? M <= 16 : M / E < 1; }

hipError_t launch_gemm_fp8(const Fp8Args& a, hipStream_t st) {
  if (!fp8_streams(a.M, a.N, a.Kp, a.E)) return launch_gemm_fp8_big(a, st);
  StreamArgs s{};
  s.a = a.a;
  s.w0 = a.w;
  s.a_scale = a.a_scale;
  s.w_scale = a.w_scale;
  s.offsets = a.offsets;
  s.out = a.out;
  s.M = a.M;
  s.N = a.N;
  s.K = a.Kp;
  s.E = a.E;
  s.out_bf16 = a.out_bf16;
  return launch_stream(s, StreamKind::kFp8, st);
}

}  // namespace moe
