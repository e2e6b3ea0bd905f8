// Products with MXFP4 weights: C = A B^T, B [N x K] in MXFP4, A [M x K] in MXFP4 or
// MXFP8, every block of 32 along K with its own E8M0 scale, FP32 accumulation.
//
// What is computed:
//   C[i][j] = sum_k Pa[i][k] 2^(sa[i][k/32] - 127) Pb[j][k] 2^(sb[j][k/32] - 127)
// on gfx950's block-scaled matrix instruction v_mfma_scale_f32_16x16x128_f8f6f4,
// which takes each lane's E8M0 code for the block that the lane supplies.  An E2M1
// lane (row r = lane % 16, group g = lane / 16) holds k = 32 g .. 32 g + 31 of its row,
// one whole block; an FP8 lane holds k = 16 g .. 16 g + 15 and 64 + 16 g .. 64 + 16 g + 15,
// and the scale that lane group g hands in is still the one of block g.

#include "cast_common.h"
#include "fp4_common.h"
#include "launch.h"

namespace fp8ds {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// matrix-instruction code of an element format
template <int F>
constexpr int mfma_format() { return F == kE4M3 ? 0 : F == kE5M2 ? 1 : 4; }

template <int FA>
__device__ __forceinline__ f32x4 mfma_a_fp4(const i32x8& a, const i32x8& b, const f32x4& c, int sa,
                                            int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, mfma_format<FA>(), 4, 0, sa, 0,
                                                          sb);
}

// One lane's operand of rows [0, rows) of a matrix with `ld` bytes per row, at K offset
// k0 (elements): row r, group g.  Rows and blocks out of range give zeros (with the
// scale of 1, so that 0 * scale is 0).
template <int F>
__device__ __forceinline__ void load_frag(const uint8_t* p, int64_t ld, const uint8_t* sc,
                                          int64_t lds, int64_t r, int64_t rows, int64_t k0,
                                          int64_t K, int g, i32x8& v, int& s) {
  v = i32x8{0, 0, 0, 0, 0, 0, 0, 0};
  s = 127;
  if (r >= rows) return;
  if (k0 + 32 * g < K) s = sc[r * lds + k0 / 32 + g];
  if constexpr (F == kE2M1) {
    if (k0 + 32 * g < K) {
      const u32x4 d = *reinterpret_cast<const u32x4*>(p + r * ld + (k0 + 32 * g) / 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (int)d[i];
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t k = k0 + 64 * h + 16 * g;
      if (k < K) {
        const u32x4 d = *reinterpret_cast<const u32x4*>(p + r * ld + k);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = (int)d[i];
      }
    }
  }
}

// A workgroup of KW waves makes a tile of 16 MT x 16 NT outputs; wave w takes the K steps
// w, w + KW, ... of 128, straight from memory to registers, and the waves' sums are
// joined in LDS in a fixed order.
template <int FA, int MT, int NT, int KW>
__global__ __launch_bounds__(64 * KW) void gemm_mxfp4_direct_kernel(Mxfp4Gemm p) {
  constexpr int BM = 16 * MT, BN = 16 * NT;
  __shared__ float part[KW][BM][BN + 1];
  __shared__ uint32_t red[2 * KW];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * BN, m0 = (int64_t)blockIdx.y * BM;
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t lda = FA == kE2M1 ? p.lda / 2 : p.lda, ldb = p.ldb / 2;
  for (int64_t k = 128 * w; k < p.K; k += 128 * KW) {
    i32x8 a[MT], b[NT];
    int sa[MT], sb[NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
      load_frag<FA>(p.A, lda, p.sc_a, p.ldsa, m0 + 16 * i + r, p.M, k, p.K, g, a[i], sa[i]);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      load_frag<kE2M1>(p.B, ldb, p.sc_b, p.ldsb, n0 + 16 * j + r, p.N, k, p.K, g, b[j], sb[j]);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[i][j] = mfma_a_fp4<FA>(a[i], b[j], acc[i][j], sa[i], sb[j]);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[w][16 * i + 4 * g + e][16 * j + r] = acc[i][j][e];
  __syncthreads();
  uint32_t amax = 0;
  for (int u = threadIdx.x; u < BM * BN; u += 64 * KW) {
    const int m = u / BN, n = u % BN;
    float v = 0.0f;
#pragma unroll
    for (int x = 0; x < KW; ++x) v += part[x][m][n];
    if (m0 + m < p.M && n0 + n < p.N) {
      const int64_t at = (m0 + m) * p.ldc + n0 + n;
      if (p.out_bf16) {
        const uint16_t b = bf16_bits_rne(v);
        static_cast<uint16_t*>(p.C)[at] = b;
        amax = max(amax, (uint32_t)(b & 0x7FFFu) << 16);
      } else {
        static_cast<float*>(p.C)[at] = v;
        amax = max(amax, __float_as_uint(v) & 0x7FFFFFFFu);
      }
    }
  }
  if (p.amax_c) {
    Health h;
    block_commit<false>(amax, 0u, h, reinterpret_cast<uint32_t*>(p.amax_c), nullptr, nullptr, red);
  }
}

// ------------------------------------------------------------------ host launcher

template <int FA, int MT, int NT, int KW>
static hipError_t launch_direct(const Mxfp4Gemm& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 16 * NT - 1) / (16 * NT)),
                  (unsigned)((p.M + 16 * MT - 1) / (16 * MT)));
  hipLaunchKernelGGL((gemm_mxfp4_direct_kernel<FA, MT, NT, KW>), grid, dim3(64 * KW), 0, stream, p);
  return hipGetLastError();
}

template <int FA>
static hipError_t launch_fa(const Mxfp4Gemm& p, hipStream_t stream) {
  if (p.M <= 16) return launch_direct<FA, 1, 1, 8>(p, stream);
  return launch_direct<FA, 4, 4, 1>(p, stream);
}

hipError_t launch_gemm_mxfp4(const Mxfp4Gemm& p, int fa, int num_cus, hipStream_t stream) {
  switch (fa) {
    case kE4M3: return launch_fa<kE4M3>(p, stream);
    case kE5M2: return launch_fa<kE5M2>(p, stream);
    default: return launch_fa<kE2M1>(p, stream);
  }
}

}  // namespace fp8ds
