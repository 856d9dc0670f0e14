// Kernel of an e4m3 product.
#include "fp8.h"
#include "stream.h"

namespace moe {

// Up to 8 rows in all take the stream, more the 128-row tiles (with K in slices where
// they are few).  Measured (us, stream / tiles, bf16):
//   7168 by 2048   1 row 11 / 15, 8 rows 13.7 / 14.5, 16 rows 17.2 / 15.2, 64 rows 21 / 15
//   2048 by 7168   16 rows 13.4 / 14.7, 64 rows 22 / 13
//   2048 by 2048, 256 groups   16 rows 20 / 17, 256 rows 130 / 120, 4096 rows 364 / 197
//   900 by 1500, 7 groups      7 rows 12 / 11, 60 rows 16 / 11
bool fp8_streams(int M) { return M <= 8; }

hipError_t launch_gemm_fp8(const Fp8Args& a, hipStream_t st) {
  if (!fp8_streams(a.M)) return launch_gemm_fp8_big(a, st);
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
