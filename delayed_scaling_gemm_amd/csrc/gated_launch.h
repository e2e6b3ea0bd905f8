// Tile choice and launch of the gated feed-forward products; see gated.h and gemm_kernel.h.
#pragma once

#include "gemm_kernel.h"

namespace fp8ds {

template <int BM, int BN, int FA, bool EXACT, bool DIRECT, int KS, int EPI>
static hipError_t launch_gated_cfg(const GatedProblem& q, hipStream_t stream) {
  GatedArgs a = {};
  a.M = q.M; a.N = q.F; a.K = q.K;
  a.A = q.A; a.lda = q.lda; a.scale_a = q.scale_a;
  a.B = q.B; a.ldb = q.ldb; a.scale_b = q.scale_b;
  constexpr int BNO = EPI == kEpiGate ? BN / 2 : BN;
  a.tiles_m = (int)((q.M + BM - 1) / BM);
  a.tiles_n = (int)((q.F + BNO - 1) / BNO);
  a.act = q.act;
  a.gu = static_cast<uint16_t*>(q.gu); a.ldgu = q.ldgu;
  a.y = q.y; a.ldy = q.ldy; a.y_f32 = q.y_bf16 ? 0 : 1;
  a.q = q.q; a.ldq = q.ldq; a.fmt = q.fmt;
  a.scale = q.scale; a.scale_used = q.scale_used;
  a.amax = reinterpret_cast<uint32_t*>(q.amax);
  a.sat = reinterpret_cast<unsigned long long*>(q.sat);
  a.vec = q.vec ? 1 : 0;
  hipLaunchKernelGGL((gemm_kernel<BM, BN, true, true, FA, kE4M3, EXACT, DIRECT, false, false, KS, EPI>),
                     dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(256 * KS), 0, stream, a);
  return hipGetLastError();
}

// Bound by the matrix cores, and by the epilogues, which nothing overlaps on a CU that holds one tile:
// 8192 x 2*14336 x 4096 with g, u and codes stored 1.36 ms (1.42 PFLOP/s, matrix unit 73% busy in the
// first passes), its backward pass 0.80 ms (1.21 PFLOP/s, 56%: g and u read, two halves
// written).  128 x 128 tiles: 1.54 and 0.90 ms.
// The choice is the plain products' (gemm_kernel.h): 256 x 256 tiles where they give every CU one, K is
// long and rows are aligned; 128 x 128 tiles with at most one per CU in two K halves; operands that direct loads
// cannot take (K no multiple of a stage, 2^31 bytes and more) through registers.
template <int FA, bool EXACT, int EPI>
static hipError_t launch_gated_path(const GatedProblem& q, int num_cus, hipStream_t stream) {
  const int64_t rows_b = EPI == kEpiGate ? 2 * q.F : q.F;
  auto fits = [&](int64_t rows, int64_t ld) { return (rows + 256) * ld + q.K < (int64_t(1) << 31); };
  const bool direct = q.K % 128 == 0 && fits(q.M, q.lda) && fits(rows_b, q.ldb);
  if (!direct) return launch_gated_cfg<128, 128, FA, EXACT, false, 1, EPI>(q, stream);
  auto tiles = [&](int64_t b) {
    const int64_t bo = EPI == kEpiGate ? b / 2 : b;
    return ((q.M + b - 1) / b) * ((q.F + bo - 1) / bo);
  };
  if (q.vec && tiles(256) >= num_cus && q.K >= kBigTileMinK)
    return launch_gated_cfg<256, 256, FA, EXACT, true, 1, EPI>(q, stream);
  if (tiles(128) <= num_cus && q.K >= kSplitMinK && q.K % 256 == 0)
    return launch_gated_cfg<128, 128, FA, EXACT, true, 2, EPI>(q, stream);
  return launch_gated_cfg<128, 128, FA, EXACT, true, 1, EPI>(q, stream);
}

}  // namespace fp8ds
