// Kernel of an e4m3 product.
#include <algorithm>
#include <cmath>

#include "fp8.h"
#include "stream.h"

namespace moe {

// Few results: blocks of 32 x 32 whose K the waves of a workgroup share, where blocks
// times K is small enough that the operands, read again for every 32 rows, do not
// count.  Otherwise up to 8 rows in all take the stream, more the 128-row tiles (with
// K in slices where they are few).  Measured (us, bf16 y, blocks / stream or tiles):
//   333 x 1111 by 770    7.3 / 16.7       16 x 2048 by 7168    5.9 / 10.8
//   1000 x 500 by 500    5.4 / 13.5       64 x 2048 by 7168    10.7 / 13
//   400 x 4000 by 500    11 / 16          128 x 2048 by 7168   20 / 17
//   1000 x 1000 by 1000  12.2 / 11.6      256 x 7168 by 2048   32 / 22
//   60 x 1500 by 900, 7 groups  7.5 / 12  16 x 2048 by 2048, 256 groups  26 / 17
bool fp8_small(int M, int N, int Kp, int E) {
  const double entries = std::ceil(M / 32.0) + (E > 1 ? std::min(M, E) : 0);
  return entries * std::ceil(N / 32.0) * (Kp / kFp8Block) <= 7168.0;
}

// (us, stream / tiles: 2048 by 2048, 256 groups, 16 rows 20 / 17, 256 rows 130 / 120,
// 4096 rows 364 / 197)
bool fp8_streams(int M) { return M <= 8; }

hipError_t launch_gemm_fp8(const Fp8Args& a, hipStream_t st) {
  if (fp8_small(a.M, a.N, a.Kp, a.E)) return launch_gemm_fp8_small(a, st);
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
