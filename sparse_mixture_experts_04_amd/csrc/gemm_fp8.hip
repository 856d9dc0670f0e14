// Kernel of an e4m3 product.
#include "blocks.h"
#include "fp8.h"

namespace moe {

// Blocks of 32 rows (blocks.hip) up to 8 rows, and where their estimated time is below
// that of the 128-row tiles.  Measured (us, bf16 y, blocks / tiles):
//   333 x 1111 by 770    5.6 / 16.7       16 x 2048 by 7168    5.0 / 10.8
//   1000 x 500 by 500    5.4 / 13.5       128 x 7168 by 2048   9.1 / 20
//   256 x 7168 by 2048   15.8 / 22.5      512 x 7168 by 2048   29.2 / 28.0
//   256 x 2048 by 7168   18.8 / 17.5      4000 x 200 by 1000   22.8 / 8.7
//   60 x 1500 by 900, 7 groups  7.8 / 12  256 x 2048 by 2048, 256 groups  142 / 127
// (512 x 7168 by 2048 is in blocks, its tiles estimated at 38: 4% lost.  An fp32 y,
// slower in tiles, goes by the same choice.)
bool fp8_blocks(int M, int N, int Kp, int E) {
  return M <= 8 || blocks_time(M, N, Kp, E, false) < fp8_tiles_time(M, N, Kp, E);
}

hipError_t launch_gemm_fp8(const Fp8Args& a, hipStream_t st) {
  if (!fp8_blocks(a.M, a.N, a.Kp, a.E)) return launch_gemm_fp8_big(a, st);
  BlockArgs b{};
  b.a = a.a;
  b.w0 = a.w;
  b.a_scale = a.a_scale;
  b.w_scale = a.w_scale;
  b.offsets = a.offsets;
  b.out = a.out;
  b.M = a.M;
  b.N = a.N;
  b.K = a.Kp;
  b.E = a.E;
  b.out_bf16 = a.out_bf16;
  return launch_blocks(b, BlockKind::kFp8, st);
}

}  // namespace moe
