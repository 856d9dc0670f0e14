// Kernel of an e4m3 product.
#include <algorithm>
#include <cmath>

#include "fp8.h"
#include "stream.h"

namespace moe {

// Blocks of 32 x 32 whose K the waves of a workgroup share, where their estimated time
// (two workgroups a compute unit; a start and an end for each block and a step for
// each 128 of K) is below that of 128-row tiles; instead of the stream while there are
// no more blocks than run at once.  Measured (us, bf16 y, blocks / tiles or, up to 8
// rows, the stream):
//   333 x 1111 by 770    5.6 / 16.7       1 x 7168 by 2048     6.8 / 10
//   1000 x 500 by 500    5.4 / 13.5       8 x 2048 by 7168     4.7 / 11
//   128 x 7168 by 2048   9.1 / 20         256 x 7168 by 2048   15.8 / 22.5
//   256 x 2048 by 7168   18.8 / 17.5      4000 x 200 by 1000   22.8 / 8.7
//   60 x 1500 by 900, 7 groups  7.8 / 12  16 x 2048 by 2048, 256 groups  18 / 17.2
bool fp8_small(int M, int N, int Kp, int E) {
  const double entries = std::ceil(M / 32.0) + (E > 1 ? std::min(M, E) : 0);
  const double blocks = entries * std::ceil(N / 32.0), nk = Kp / kFp8Block;
  if (fp8_streams(M)) return blocks <= 512;
  return 3.0 + std::max(1.0, blocks / 512) * (2.3 + 0.18 * nk) < fp8_tiles_time(M, N, Kp, E);
}

// Up to 8 rows of many weights (us, stream / tiles: 2048 by 2048, 256 groups, 16 rows
// 20 / 17, 256 rows 130 / 120, 4096 rows 364 / 197).
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
