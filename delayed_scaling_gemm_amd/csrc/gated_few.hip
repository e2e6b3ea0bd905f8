// Forward product of a gated feed-forward block for a few rows (decoding): reads every weight once.
//
//   g, u = d sum_k x w  of gate and up,  a = act(g) u       (gated.h; exact products, fp32 sums)
//
// Bound by the weights' bytes, 2 F K.  A workgroup owns 16 output columns (32 weight rows), its
// waves share K in segments of 128: lane l reads 32 consecutive bytes of weight row l % 16, so
// a wave's loads cover whole cache lines of 16 rows, straight into registers (no LDS: nothing is
// read twice), widens them to F16 and multiplies them with the tokens on the 16 x 16 x 32 matrix
// instruction, whose columns are the tokens.  The waves' sums meet in LDS, in wave order, and a
// thread finishes one output.
#include "gemm_kernel.h"

namespace fp8ds {

typedef float v4f __attribute__((ext_vector_type(4)));

// 16 bytes of a row from k on, zeros past K (ld is a multiple of 16: the chunk is in the row)
__device__ __forceinline__ u32x4 few_chunk(const uint8_t* row, int64_t k, int64_t K, bool live) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (live && k < K) {
    v = *reinterpret_cast<const u32x4*>(row + k);
    const int64_t valid = K - k;
    if (valid < 16) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int64_t b = valid - 4 * w;
        v[w] &= b >= 4 ? 0xFFFFFFFFu : b <= 0 ? 0u : (1u << (8 * b)) - 1u;
      }
    }
  }
  return v;
}

__device__ __forceinline__ v8h few_widen(const u32x4& v, int half) {
  const uint32_t a = v[2 * half], b = v[2 * half + 1];
  return __builtin_bit_cast(v8h, u32x4{widen_pair<kE4M3>(a, false), widen_pair<kE4M3>(a, true),
                                       widen_pair<kE4M3>(b, false), widen_pair<kE4M3>(b, true)});
}

// MT groups of 16 tokens; NW waves share K.
template <int MT, int NW>
__global__ __launch_bounds__(64 * NW) void gated_few_kernel(GatedArgs p) {
  constexpr int kBatch = 4;  // segments of a wave whose loads are in flight together
  __shared__ float part[NW][2][MT][16][17];
  __shared__ uint32_t red[2 * NW];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, kq = (lane >> 4) * 32;
  const int64_t F = p.N, K = p.K, n0 = (int64_t)blockIdx.x * 16;
  const bool live = n0 + r < F;
  const uint8_t* wrow[2] = {p.B + (live ? n0 + r : 0) * p.ldb, p.B + (F + (live ? n0 + r : 0)) * p.ldb};
  const uint8_t* xrow[MT];
  bool xlive[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    xlive[t] = t * 16 + r < p.M;
    xrow[t] = p.A + (xlive[t] ? t * 16 + r : 0) * p.lda;
  }
  v4f acc[2][MT];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[h][t] = v4f{0.f, 0.f, 0.f, 0.f};

  const int64_t nseg = (K + 127) / 128;
  for (int64_t s0 = wave; s0 < nseg; s0 += NW * kBatch) {
    u32x4 w[kBatch][2][2], x[kBatch][MT][2];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int64_t k = (s0 + b * NW) * 128 + kq;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        w[b][0][c] = few_chunk(wrow[0], k + 16 * c, K, live);
        w[b][1][c] = few_chunk(wrow[1], k + 16 * c, K, live);
#pragma unroll
        for (int t = 0; t < MT; ++t) x[b][t][c] = few_chunk(xrow[t], k + 16 * c, K, xlive[t]);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const v8h wg = few_widen(w[b][0][c], half), wu = few_widen(w[b][1][c], half);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const v8h xv = few_widen(x[b][t][c], half);
            acc[0][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wg, xv, acc[0][t], 0, 0, 0);
            acc[1][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wu, xv, acc[1][t], 0, 0, 0);
          }
        }
  }
  // lane l holds token l % 16, weight rows 4 (l / 16) + {0..3}
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[wave][h][t][r][4 * (lane >> 4) + v] = acc[h][t][v];
  __syncthreads();

  const float d = __fdiv_rn(1.0f, p.scale_a[0] * p.scale_b[0]);
  const float s = p.q ? *p.scale : 1.0f;
  if (p.scale_used && blockIdx.x == 0 && tid == 0) *p.scale_used = s;
  uint32_t amax = 0, sat = 0;
  for (int o = tid; o < MT * 256; o += 64 * NW) {
    const int64_t m = o >> 4, n = n0 + (o & 15);
    if (m >= p.M || n >= F) continue;
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      g += part[i][0][o >> 8][m & 15][o & 15];
      u += part[i][1][o >> 8][m & 15][o & 15];
    }
    g *= d;
    u *= d;
    const float a = act_value<false>(g, p.act).a * u;
    amax = max(amax, __float_as_uint(a) & 0x7FFFFFFFu);
    if (p.gu) {
      const uint32_t gu = pack_bf16x2(g, u);
      p.gu[m * p.ldgu + n] = (uint16_t)gu;
      p.gu[m * p.ldgu + F + n] = (uint16_t)(gu >> 16);
    }
    if (p.q) {
      const float v = a * s;
      const bool e5m2 = p.fmt == kE5M2;
      p.q[m * p.ldq + n] = (uint8_t)(e5m2 ? encode_fp8<kE5M2>(v) : encode_fp8<kE4M3>(v));
      sat += (uint32_t)(fabsf(v) > (e5m2 ? FmtTraits<kE5M2>::kMax : FmtTraits<kE4M3>::kMax));
    }
    if (p.y) {
      if (p.y_f32) static_cast<float*>(p.y)[m * p.ldy + n] = a;
      else static_cast<uint16_t*>(p.y)[m * p.ldy + n] = (uint16_t)pack_bf16x2(a, 0.f);
    }
  }
  if (p.amax || p.sat) {
    Health h;
    block_commit<false>(amax, sat, h, p.amax, p.sat, nullptr, red);
  }
}

hipError_t launch_gated_few(const GatedProblem& q, hipStream_t stream) {
  GatedArgs a = {};
  a.M = q.M; a.N = q.F; a.K = q.K;
  a.A = q.A; a.lda = q.lda; a.scale_a = q.scale_a;
  a.B = q.B; a.ldb = q.ldb; a.scale_b = q.scale_b;
  a.act = q.act;
  a.gu = static_cast<uint16_t*>(q.gu); a.ldgu = q.ldgu;
  a.y = q.y; a.ldy = q.ldy; a.y_f32 = q.y_bf16 ? 0 : 1;
  a.q = q.q; a.ldq = q.ldq; a.fmt = q.fmt;
  a.scale = q.scale; a.scale_used = q.scale_used;
  a.amax = reinterpret_cast<uint32_t*>(q.amax);
  a.sat = reinterpret_cast<unsigned long long*>(q.sat);
  const dim3 grid((unsigned)((q.F + 15) / 16));
  if (q.M <= 16) hipLaunchKernelGGL((gated_few_kernel<1, 4>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((gated_few_kernel<2, 4>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace fp8ds
