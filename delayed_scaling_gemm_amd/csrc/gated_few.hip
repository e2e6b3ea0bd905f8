// Forward product of a gated feed-forward block for a few rows (decoding): reads every weight once.
//
//   g, u = d sum_k x w  of gate and up,  a = act(g) u       (gated.h; exact products, fp32 sums)
//
// Bound by the weights' bytes, 2 F K.  A workgroup of eight waves stays on its CU and takes 8 output
// columns at a time: 8 gate rows and 8 up rows are the 16 rows of the 16 x 16 x 32 matrix
// instruction, the tokens its columns.  The waves share K in segments of 128, lane l reading 32
// consecutive bytes of row l % 16 straight into registers (nothing is read twice, so LDS has no part
// in it); the weights of the next two steps are on their way while one is widened to F16 and
// multiplied, and the tokens, whose part of K is a wave's own, are widened once for all columns
// where K fits (4096).  The waves' sums meet in LDS, in wave order, and a thread finishes one
// output.  One row of 4096 through 2 x 14336 columns: 117 MB; a workgroup per 16 columns that reads
// its tokens anew and ends with them took 30 us, this 26.
#include "gemm_kernel.h"

namespace fp8ds {

typedef float v4f __attribute__((ext_vector_type(4)));

// Zeros in the bytes of a chunk at and past K: `left` of the 16 are inside.
__device__ __forceinline__ u32x4 few_mask(u32x4 v, int left) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int b = left - 4 * w;
    v[w] &= b >= 4 ? 0xFFFFFFFFu : b <= 0 ? 0u : (1u << (8 * b)) - 1u;
  }
  return v;
}

__device__ __forceinline__ v8h few_widen(const u32x4& v, int half) {
  const uint32_t a = v[2 * half], b = v[2 * half + 1];
  return __builtin_bit_cast(v8h, u32x4{widen_pair<kE4M3>(a, false), widen_pair<kE4M3>(a, true),
                                       widen_pair<kE4M3>(b, false), widen_pair<kE4M3>(b, true)});
}

constexpr int kFewWaves = 8;
constexpr int kFewSegs = 4;                                // segments of a wave in a step

__global__ __launch_bounds__(64 * kFewWaves, 2) void gated_few_kernel(GatedArgs p, int groups) {
  constexpr int NW = kFewWaves, NS = kFewSegs;
  __shared__ float part[2][NW][16][17];
  __shared__ uint32_t red[2 * NW];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, kq = (lane >> 4) * 32;
  const int F = (int)p.N, K = (int)p.K, ldb = (int)p.ldb;
  // (offsets below 2^31: the launcher sees to that; what is past the last row reads as zeros.  Rows
  // start at 16 bytes, so the piece that K ends in is read whole and masked.)
  const int64_t row = (p.K + 15) / 16 * 16;
  const __amdgpu_buffer_rsrc_t bw = byte_rsrc(p.B, (2 * p.N - 1) * p.ldb + row);
  const __amdgpu_buffer_rsrc_t bx = byte_rsrc(p.A, (p.M - 1) * p.lda + row);
  const int vx = r * (int)p.lda + kq;
  // K in equal chunks of a step each
  const int segs = (K + 127) / 128, chunks = segs == 0 ? 1 : (segs + NW * NS - 1) / (NW * NS);
  const int per = (segs + chunks - 1) / chunks;  // segments of a chunk
  const int mine = groups > (int)blockIdx.x ? (groups - (int)blockIdx.x - 1) / (int)gridDim.x + 1 : 0;
  const int steps = mine * chunks;
  auto load = [](const __amdgpu_buffer_rsrc_t& b, int voff, int soff) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, voff, soff, 0));
  };
  struct Step {
    u32x4 v[NS][2];
  };
  auto seg_of = [&](int chunk, int i) {  // past the end where a wave has none
    return i * NW + wave < per ? chunk * per + i * NW + wave : segs;
  };
  auto fetch_w = [&](int step, Step& s) {  // (columns past F read the last one's, and are not used)
    if (step >= steps) return;
    const int group = (int)blockIdx.x + step / chunks * (int)gridDim.x, chunk = step % chunks;
    const int col = min(group * 8 + (r & 7), F - 1), voff = (r < 8 ? col : F + col) * ldb + kq;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      if (seg_of(chunk, i) * 128 >= K) continue;
#pragma unroll
      for (int c = 0; c < 2; ++c) s.v[i][c] = load(bw, voff + 16 * c, seg_of(chunk, i) * 128);
    }
  };
  auto fetch_x = [&](int chunk, Step& s) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      if (seg_of(chunk, i) * 128 >= K) continue;
#pragma unroll
      for (int c = 0; c < 2; ++c) s.v[i][c] = load(bx, vx + 16 * c, seg_of(chunk, i) * 128);
    }
  };
  // the bytes past K, in the segment that K ends in
  auto mask = [&](int seg, u32x4 (&v)[2]) {
    if (seg * 128 + 128 <= K) return;
#pragma unroll
    for (int c = 0; c < 2; ++c) v[c] = few_mask(v[c], K - (seg * 128 + kq + 16 * c));
  };
  v8h xf[NS][2][2];
  auto widen_x = [&](int chunk, Step& s) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int seg = seg_of(chunk, i);
      if (seg * 128 >= K) continue;
      mask(seg, s.v[i]);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int half = 0; half < 2; ++half) xf[i][c][half] = few_widen(s.v[i][c], half);
    }
  };
  const float d = __fdiv_rn(1.0f, p.scale_a[0] * p.scale_b[0]);
  const float s = p.q ? *p.scale : 1.0f;
  if (p.scale_used && blockIdx.x == 0 && tid == 0) *p.scale_used = s;
  uint32_t amax = 0, sat = 0;
  const Act act(p.act);
  const bool e5m2 = p.fmt == kE5M2;

  Step w0, w1, w2, xr;
  fetch_x(0, xr);
  fetch_w(0, w0);
  fetch_w(1, w1);
  widen_x(0, xr);
  v4f acc = {0.f, 0.f, 0.f, 0.f};
  for (int step = 0; step < steps; ++step) {
    const int chunk = step % chunks, next = chunk + 1 < chunks ? chunk + 1 : 0;
    if (chunks > 1) fetch_x(next, xr);
    fetch_w(step + 2, w2);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int seg = seg_of(chunk, i);
      if (seg * 128 >= K) continue;
      mask(seg, w0.v[i]);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int half = 0; half < 2; ++half)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(few_widen(w0.v[i][c], half), xf[i][c][half], acc, 0, 0, 0);
    }
    if (chunks > 1) widen_x(next, xr);
    w0 = w1;
    w1 = w2;
    if (chunk + 1 < chunks) continue;
    // lane l holds token l % 16, rows 4 (l / 16) + {0..3}: gate, gate, up, up.  Two buffers in
    // turn: one barrier keeps a group's readers and the next but one's writers apart.
    const int group = step / chunks;
    float (&sums)[NW][16][17] = part[group & 1];
#pragma unroll
    for (int v = 0; v < 4; ++v) sums[wave][4 * (lane >> 4) + v][r] = acc[v];
    acc = v4f{0.f, 0.f, 0.f, 0.f};
    __syncthreads();
    const int64_t m = tid >> 3, n = ((int64_t)blockIdx.x + (int64_t)group * gridDim.x) * 8 + (tid & 7);
    if (tid < 128 && m < p.M && n < F) {
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        g += sums[i][tid & 7][m];
        u += sums[i][8 + (tid & 7)][m];
      }
      g *= d;
      u *= d;
      const float a = act_value<false>(g, act).a * u;
      amax = max(amax, __float_as_uint(a) & 0x7FFFFFFFu);
      if (p.gu) {
        const uint32_t gu = pack_bf16x2(g, u);
        p.gu[m * p.ldgu + n] = (uint16_t)gu;
        p.gu[m * p.ldgu + F + n] = (uint16_t)(gu >> 16);
      }
      if (p.q) {
        const float v = a * s;
        p.q[m * p.ldq + n] = (uint8_t)(e5m2 ? encode_fp8<kE5M2>(v) : encode_fp8<kE4M3>(v));
        sat += (uint32_t)(fabsf(v) > (e5m2 ? FmtTraits<kE5M2>::kMax : FmtTraits<kE4M3>::kMax));
      }
      if (p.y) {
        if (p.y_f32) static_cast<float*>(p.y)[m * p.ldy + n] = a;
        else static_cast<uint16_t*>(p.y)[m * p.ldy + n] = (uint16_t)pack_bf16x2(a, 0.f);
      }
    }
  }
  if (p.amax || p.sat) {
    Health h;
    block_commit<false>(amax, sat, h, p.amax, p.sat, nullptr, red);
  }
}

hipError_t launch_gated_few(const GatedProblem& q, int num_cus, hipStream_t stream) {
  GatedArgs a = {};
  a.M = q.M; a.N = q.F; a.K = q.K;
  a.A = q.A; a.lda = q.M > 1 ? q.lda : 0; a.scale_a = q.scale_a;
  a.B = q.B; a.ldb = q.ldb; a.scale_b = q.scale_b;
  a.act = q.act;
  a.gu = static_cast<uint16_t*>(q.gu); a.ldgu = q.ldgu;
  a.y = q.y; a.ldy = q.ldy; a.y_f32 = q.y_bf16 ? 0 : 1;
  a.q = q.q; a.ldq = q.ldq; a.fmt = q.fmt;
  a.scale = q.scale; a.scale_used = q.scale_used;
  a.amax = reinterpret_cast<uint32_t*>(q.amax);
  a.sat = reinterpret_cast<unsigned long long*>(q.sat);
  const int groups = (int)((q.F + 7) / 8);
  hipLaunchKernelGGL(gated_few_kernel, dim3((unsigned)(groups < num_cus ? groups : num_cus)),
                     dim3(64 * kFewWaves), 0, stream, a, groups);
  return hipGetLastError();
}

}  // namespace fp8ds
