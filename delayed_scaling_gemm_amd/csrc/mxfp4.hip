// MXFP4 quantisation and its inverse: E2M1 elements, two to a byte, in blocks of 32
// consecutive elements of a row that share an E8M0 scale.
//
// What is computed (the block rule of the OCP Microscaling Formats specification, as
// the MXFP8 cast applies it to FP8 elements):
//   a = max |x_i| over the block
//   code = floor(log2 a) - 2 + 127 clamped to [0, 254], 0 for a zero block, 255 (NaN)
//          for a block that holds an infinity or NaN
//   P_i = the element of {0, 0.5, 1, 1.5, 2, 3, 4, 6} nearest |x_i| 2^(127 - code), ties
//         to the even code, saturating at 6, with x_i's sign
// and back: x_i = P_i 2^(code - 127), NaN where the code is 255.
//
// Design for gfx950: HBM-bound (BF16: 2 B read, 17/32 B written per element and copy).
// Lanes take consecutive 16-byte pieces, the 4 (BF16) or 8 (FP32) lanes of a block
// join its amax by shuffles, and gfx950's packed conversion makes the codes.
//
// Measured in BF16: 14336 x 4096 cast 26.5 us and back 26.2 us, 5.6 and 5.7 TB/s (a copy of
// 1 GiB: 5.1); with the transposed copy 16384 x 4096 48 us, 4.3 TB/s of 49/16 B per element.

#include "cast_common.h"
#include "fp4_common.h"
#include "launch.h"

namespace fp8ds {

template <bool BF16>
__device__ __forceinline__ void piece_values(const u32x4& d, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (BF16) {
      v[2 * k] = bf16_lo(d[k]);
      v[2 * k + 1] = bf16_hi(d[k]);
    } else {
      v[k] = __uint_as_float(d[k]);
      v[4 + k] = 0.0f;
    }
  }
}

// amax bits of the row block that this lane's piece belongs to.
template <bool BF16>
__device__ __forceinline__ uint32_t row_block_amax(const u32x4& d) {
  uint32_t a = piece_amax<BF16>(d);
  a = max(a, (uint32_t)__shfl_xor((int)a, 1));
  a = max(a, (uint32_t)__shfl_xor((int)a, 2));
  if constexpr (!BF16) a = max(a, (uint32_t)__shfl_xor((int)a, 4));
  return a;
}

template <bool BF16>
__device__ __forceinline__ void store_piece(uint8_t* q, int64_t piece, const u32x4& d,
                                            uint32_t code) {
  float v[8];
  piece_values<BF16>(d, v);
  const uint32_t c = code == 255u ? kFp4NanBlock : fp4_codes8(v, code);
  if constexpr (BF16)
    __builtin_nontemporal_store(c, reinterpret_cast<uint32_t*>(q) + piece);
  else
    __builtin_nontemporal_store((uint16_t)c, reinterpret_cast<uint16_t*>(q) + piece);
}

// P 16-byte pieces per thread: 8, or 1 where 8 would leave CUs without a workgroup
// (13 x 14336 BF16: 4.1 us with 8).
template <bool BF16, int P>
__global__ __launch_bounds__(256) void mxfp4_cast_kernel(const void* __restrict__ x,
                                                         int64_t npieces, uint8_t* __restrict__ q,
                                                         uint8_t* __restrict__ scales) {
  constexpr int PPB = BF16 ? 4 : 8;  // pieces (lanes) per block
  const int64_t base = (int64_t)blockIdx.x * 256 * P + threadIdx.x;
  const u32x4* xv = static_cast<const u32x4*>(x);
  u32x4 v[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int64_t pc = base + 256 * j;
    v[j] = pc < npieces ? __builtin_nontemporal_load(xv + pc) : u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int64_t pc = base + 256 * j;  // a block's lanes are all in range or all out
    const uint32_t code = mx_code(row_block_amax<BF16>(v[j]), 2u);
    if (pc < npieces) {
      store_piece<BF16>(q, pc, v[j], code);
      if ((threadIdx.x & (PPB - 1)) == 0) scales[pc / PPB] = (uint8_t)code;
    }
  }
}

// Both orientations from one read: q [rows x cols / 2] as above and q_t [cols x rows / 2],
// the transpose blocked along its own rows.  A 128 x 128 tile per workgroup is parked
// in LDS as it came; each thread then walks down the 32 rows of a column block (a pair
// of adjacent columns for BF16: one dword), which is one whole block of q_t, so its
// amax needs no exchange.  The 16 code bytes of a column block go through LDS once more
// so that a wave writes runs of 64 bytes.  rows and cols are multiples of 32; the last
// tiles may be partial, a 32 x 32 block never is.
// It moves 7% more than it has to: the 4 scale codes of a column are a write of 32 bytes.
// Tried and slower for 16384 x 4096: tiles dealt out so that each XCD has neighbours, whose
// parts of lines could meet in its L2 (56 to 59 us, then 52), workgroups that go on to
// further tiles with the next one's loads in flight (61 us), and BF16 pairs converted
// without widening (1% slower).
template <bool BF16>
__global__ __launch_bounds__(256) void mxfp4_cast_transpose_kernel(
    const void* __restrict__ xp, int64_t rows, int64_t cols, uint8_t* __restrict__ q,
    uint8_t* __restrict__ scales, uint8_t* __restrict__ qt, uint8_t* __restrict__ scales_t) {
  constexpr int T = 128;
  constexpr int PER = BF16 ? 8 : 4;         // elements per piece
  constexpr int PPR = T / PER;              // pieces per tile row
  constexpr int NP = T * PPR / 256;         // pieces per thread
  constexpr int RD = BF16 ? T / 2 : T;      // dwords per tile row
  __shared__ __attribute__((aligned(16))) uint32_t tile[T * RD];
  __shared__ __attribute__((aligned(16))) uint8_t codes_t[T * 64];
  const int tid = threadIdx.x;
  const int64_t c0 = (int64_t)blockIdx.x * T, r0 = (int64_t)blockIdx.y * T;
  const int nr = (int)(rows - r0 < T ? rows - r0 : T), nc = (int)(cols - c0 < T ? cols - c0 : T);
  u32x4 v[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int u = 256 * i + tid, r = u / PPR, c = (u % PPR) * PER;
    v[i] = r < nr && c < nc
               ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(
                     static_cast<const char*>(xp) + ((r0 + r) * cols + c0 + c) * (BF16 ? 2 : 4)))
               : u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int u = 256 * i + tid, r = u / PPR, c = (u % PPR) * PER;
    *reinterpret_cast<u32x4*>(&tile[r * RD + (u % PPR) * 4]) = v[i];
    const uint32_t code = mx_code(row_block_amax<BF16>(v[i]), 2u);
    if (r < nr && c < nc) {
      const int64_t at = (r0 + r) * cols + c0 + c;
      store_piece<BF16>(q, at / PER, v[i], code);
      if ((c & 31) == 0) scales[at / 32] = (uint8_t)code;
    }
  }
  __syncthreads();
  // one unit: dword column `dc` (two BF16 columns, or one FP32 column), row block `rb`
  constexpr int W = BF16 ? 2 : 1;  // columns per unit
  // (the 8 pieces of a pair of columns change places with the pair: in order, all the lanes
  // of a store would meet in the same banks)
  auto slot = [](int c, int rb) {
    return (c >> 1) * 128 + (((c & 1) * 4 + rb) ^ ((c >> 1) & 7)) * 16;
  };
#pragma unroll 1
  for (int u = tid; u < RD * 4; u += 256) {
    const int dc = u % RD, rb = u / RD;
    if (rb * 32 >= nr || dc * W >= nc) continue;
    uint32_t d[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) d[i] = tile[(rb * 32 + i) * RD + dc];
    uint32_t scale_codes = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      uint32_t a = 0;
      float f[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        f[i] = BF16 ? (w ? bf16_hi(d[i]) : bf16_lo(d[i])) : __uint_as_float(d[i]);
        a = max(a, __float_as_uint(f[i]) & 0x7FFFFFFFu);
      }
      const uint32_t code = mx_code(a, 2u);
      const int c = dc * W + w;
      u32x4 o;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float g[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = f[8 * k + i];
        o[k] = code == 255u ? kFp4NanBlock : fp4_codes8(g, code);
      }
      *reinterpret_cast<u32x4*>(&codes_t[slot(c, rb)]) = o;
      scale_codes |= code << (8 * w);
    }
    tile[rb * 32 * RD + dc] = scale_codes;  // (these 32 dwords are this thread's own)
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = 256 * i + tid, c = u >> 2, rb = u & 3;
    if (rb * 32 < nr && c < nc)
      *reinterpret_cast<u32x4*>(qt + (c0 + c) * (rows / 2) + r0 / 2 + rb * 16) =
          *reinterpret_cast<const u32x4*>(&codes_t[slot(c, rb)]);
  }
  // the scale codes of a column of the tile: one dword where they are four and aligned
  // (a byte at a time, each in a line of its own, the stores cost 10% of the call)
  if (tid < nc) {
    uint8_t* to = scales_t + (c0 + tid) * (rows / 32) + r0 / 32;
    uint32_t four = 0;
#pragma unroll
    for (int rb = 0; rb < 4; ++rb)
      four |= (tile[rb * 32 * RD + tid / W] >> (8 * (tid % W)) & 255u) << (8 * rb);
    if (nr == T && (reinterpret_cast<uintptr_t>(to) & 3) == 0)
      *reinterpret_cast<uint32_t*>(to) = four;
    else
      for (int rb = 0; rb * 32 < nr; ++rb) to[rb] = (uint8_t)(four >> (8 * rb));
  }
}

// A lane takes 8 elements (4 bytes of codes) per step.
template <bool BF16>
__global__ __launch_bounds__(256) void mxfp4_dequant_kernel(const uint8_t* __restrict__ q,
                                                            const uint8_t* __restrict__ scales,
                                                            int64_t nwords, void* __restrict__ y) {
  const int64_t base = (int64_t)blockIdx.x * 256 * 4 + threadIdx.x;
  uint32_t c[4], s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t w = base + 256 * j;
    c[j] = w < nwords ? reinterpret_cast<const uint32_t*>(q)[w] : 0u;
    s[j] = w < nwords ? scales[w / 4] : 0u;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t w = base + 256 * j;
    if (w >= nwords) continue;
    float v[8];
    fp4_values8(c[j], s[j], v);
    if constexpr (BF16) {
      // exact: two significant bits, and BF16 has fp32's exponents and subnormals of 2^-133
      u32x4 d;
#pragma unroll
      for (int k = 0; k < 4; ++k) d[k] = bf16_pair_rne(v[2 * k], v[2 * k + 1]);
      __builtin_nontemporal_store(d, static_cast<u32x4*>(y) + w);
    } else {
      u32x4 d[2];
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k >> 2][k & 3] = __float_as_uint(v[k]);
      __builtin_nontemporal_store(d[0], static_cast<u32x4*>(y) + 2 * w);
      __builtin_nontemporal_store(d[1], static_cast<u32x4*>(y) + 2 * w + 1);
    }
  }
}

// ------------------------------------------------------------------ host launchers

template <bool BF16>
static hipError_t launch_cast4(const void* x, int64_t n, uint8_t* q, uint8_t* scales, int num_cus,
                               hipStream_t stream) {
  const int64_t npieces = n / (BF16 ? 8 : 4);
  if (npieces < 256 * 8 * (int64_t)num_cus)
    hipLaunchKernelGGL((mxfp4_cast_kernel<BF16, 1>), dim3((unsigned)((npieces + 255) / 256)), dim3(256),
                       0, stream, x, npieces, q, scales);
  else
    hipLaunchKernelGGL((mxfp4_cast_kernel<BF16, 8>), dim3((unsigned)((npieces + 2047) / 2048)),
                       dim3(256), 0, stream, x, npieces, q, scales);
  return hipGetLastError();
}

hipError_t launch_mxfp4_cast(const void* x, bool bf16, int64_t n, uint8_t* q, uint8_t* scales,
                             int num_cus, hipStream_t stream) {
  return bf16 ? launch_cast4<true>(x, n, q, scales, num_cus, stream)
              : launch_cast4<false>(x, n, q, scales, num_cus, stream);
}

hipError_t launch_mxfp4_cast_transpose(const void* x, bool bf16, int64_t rows, int64_t cols,
                                       uint8_t* q, uint8_t* scales, uint8_t* qt, uint8_t* scales_t,
                                       hipStream_t stream) {
  const dim3 grid((unsigned)((cols + 127) / 128), (unsigned)((rows + 127) / 128));
  if (bf16)
    hipLaunchKernelGGL((mxfp4_cast_transpose_kernel<true>), grid, dim3(256), 0, stream, x, rows,
                       cols, q, scales, qt, scales_t);
  else
    hipLaunchKernelGGL((mxfp4_cast_transpose_kernel<false>), grid, dim3(256), 0, stream, x, rows,
                       cols, q, scales, qt, scales_t);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequant(const uint8_t* q, const uint8_t* scales, int64_t n, void* y,
                                bool bf16, hipStream_t stream) {
  const int64_t nwords = n / 8;
  const dim3 grid((unsigned)((nwords + 1023) / 1024));
  if (bf16)
    hipLaunchKernelGGL((mxfp4_dequant_kernel<true>), grid, dim3(256), 0, stream, q, scales, nwords, y);
  else
    hipLaunchKernelGGL((mxfp4_dequant_kernel<false>), grid, dim3(256), 0, stream, q, scales, nwords, y);
  return hipGetLastError();
}

}  // namespace fp8ds
