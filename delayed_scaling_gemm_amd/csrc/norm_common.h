// What the norm kernels share: rows held in registers as groups of 8 elements, row reductions,
// and the casts of a row's values.
#pragma once

#include <type_traits>

#include "cast_common.h"
#include "fp4_common.h"
#include "launch.h"

namespace fp8ds {

enum { kQNone = 0, kQTensor = 1, kQRow = 2, kQMx = 3 };

template <bool BF>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF)
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  else
    return static_cast<const float*>(p)[i];
}

template <bool BF>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (BF)
    static_cast<uint16_t*>(p)[i] = bf16_bits_rne(v);
  else
    static_cast<float*>(p)[i] = v;
}

// Vectors at the alignment of the elements: gfx950 takes 8- and 16-byte accesses at any
// address, an unaligned one costs the extra cache line that it touches.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

// Eight elements as they lie in memory.  All of a row's loads are issued before any is
// unpacked, and without a branch between them (each would wait for the load before it):
// groups past the row's end read its last whole group, and are not used.
template <bool BF>
struct Raw8 {
  u32x4 v[BF ? 1 : 2];
};

template <bool BF, bool AL>
__device__ __forceinline__ Raw8<BF> load8(const void* p, int64_t i) {
  using V = std::conditional_t<AL, u32x4, u32x4_any>;
  const V* s = BF ? reinterpret_cast<const V*>(static_cast<const uint16_t*>(p) + i)
                  : reinterpret_cast<const V*>(static_cast<const float*>(p) + i);
  Raw8<BF> r;
#pragma unroll
  for (int k = 0; k < (BF ? 1 : 2); ++k) r.v[k] = AL ? (u32x4)__builtin_nontemporal_load(s + k) : (u32x4)s[k];
  return r;
}

// The first n of them as floats, zeros after.
template <bool BF, bool AL>
__device__ __forceinline__ void unpack8(const Raw8<BF>& r, int n, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float x;
    if constexpr (BF) x = k & 1 ? bf16_hi(r.v[0][k >> 1]) : bf16_lo(r.v[0][k >> 1]);
    else x = __uint_as_float(r.v[k >> 2][k & 3]);
    v[k] = n == 8 ? x : 0.0f;
  }
}
// A row's last n < 8 elements, one by one.
template <bool BF>
__device__ __forceinline__ void load_tail(const void* p, int64_t i, int n, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 7; ++k) v[k] = k < n ? load1<BF>(p, i + k) : 0.0f;
}

template <bool BF, bool AL>
__device__ __forceinline__ void store8(void* p, int64_t i, int n, const float (&v)[8]) {
  using V = std::conditional_t<AL, u32x4, u32x4_any>;
  if (!AL && n < 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) store1<BF>(p, i + k, v[k]);
  } else if constexpr (BF) {
    u32x4 d;
#pragma unroll
    for (int k = 0; k < 4; ++k) d[k] = bf16_pair_rne(v[2 * k], v[2 * k + 1]);
    V* s = reinterpret_cast<V*>(static_cast<uint16_t*>(p) + i);
    if constexpr (AL) __builtin_nontemporal_store(d, s);
    else *s = d;
  } else {
    u32x4 a, b;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = __float_as_uint(v[k]);
      b[k] = __float_as_uint(v[4 + k]);
    }
    V* s = reinterpret_cast<V*>(static_cast<float*>(p) + i);
    if constexpr (AL) {
      __builtin_nontemporal_store(a, s);
      __builtin_nontemporal_store(b, s + 1);
    } else {
      s[0] = a;
      s[1] = b;
    }
  }
}

// Eight codes, or the first n of them.
template <bool AL>
__device__ __forceinline__ void store_codes(uint8_t* q, int n, const u32x2& c) {
  if (!AL && n < 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < n) q[k] = (uint8_t)(c[k >> 2] >> (8 * (k & 3)));
  } else if constexpr (AL) {
    __builtin_nontemporal_store(c, reinterpret_cast<u32x2*>(q));
  } else {
    *reinterpret_cast<u32x2_any*>(q) = c;
  }
}

// gamma is read by every row: ordinary (cached) loads, of either type without a branch
// (BF16 reads its piece twice).
template <bool AL>
__device__ __forceinline__ Raw8<false> gamma8(const void* g, bool bf, int64_t i) {
  using V = std::conditional_t<AL, u32x4, u32x4_any>;
  const char* s = static_cast<const char*>(g) + (i << (bf ? 1 : 2));
  Raw8<false> r;
  r.v[0] = *reinterpret_cast<const V*>(s);
  r.v[1] = *reinterpret_cast<const V*>(s + (bf ? 0 : 16));
  return r;
}
template <bool AL>
__device__ __forceinline__ void unpack_gamma(const Raw8<false>& r, bool bf, int n, float (&v)[8]) {
  if (bf) unpack8<true, AL>(Raw8<true>{{r.v[0]}}, n, v);
  else unpack8<false, AL>(r, n, v);
}
__device__ __forceinline__ float gamma1(const void* g, bool bf, int64_t i) {
  return bf ? load1<true>(g, i) : load1<false>(g, i);
}

// Sum over the TPR threads of a row; every thread gets it.  TPR > 64: through LDS
// (`red`: one word per wave; two barriers keep successive calls apart).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = (TPR < 64 ? TPR : 64) / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) t += red[w];
    __syncthreads();
    v = t;
  }
  return v;
}

template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
#pragma unroll
  for (int o = (TPR < 64 ? TPR : 64) / 2; o > 0; o >>= 1)
    v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    uint32_t t = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) t = max(t, red[w]);
    __syncthreads();
    v = t;
  }
  return v;
}

// 1 / sqrt(ss / C + eps), each operation correctly rounded.
__device__ __forceinline__ float norm_rstd(float ss, int64_t C, float eps) {
  return __fdiv_rn(1.0f, __builtin_sqrtf(__fdiv_rn(ss, (float)C) + eps));
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// FP8 codes of the N groups of v s, and what they add to the saturation count.  `amax`:
// the largest |v| bits of this thread.  Without a NaN among the values, and with a scale
// that makes none of them (Inf * 0), the packed converts alone encode.
template <int FMT, int N>
__device__ __forceinline__ void codes_fmt(const float (&v)[N][8], float s, uint32_t amax, u32x2 (&c)[N],
                                          uint32_t& sat, bool want_sat) {
  const uint32_t sb = __float_as_uint(s) & 0x7FFFFFFFu;
  const bool slow = amax > 0x7F800000u || sb >= 0x7F800000u || sb == 0u;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = v[j][k] * s;
    c[j] = u32x2{encode4_hw<FMT>(t[0], t[1], t[2], t[3]), encode4_hw<FMT>(t[4], t[5], t[6], t[7])};
    if (want_sat) sat += sat4<FMT>(t[0], t[1], t[2], t[3]) + sat4<FMT>(t[4], t[5], t[6], t[7]);
  }
  if (slow) {
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        c[j][q] = encode4_sw<FMT>(v[j][4 * q] * s, v[j][4 * q + 1] * s, v[j][4 * q + 2] * s,
                                  v[j][4 * q + 3] * s);
  }
}
template <int N>
__device__ __forceinline__ void codes8(const float (&v)[N][8], float s, bool e5m2, uint32_t amax,
                                       u32x2 (&c)[N], uint32_t& sat, bool want_sat) {
  if (e5m2) codes_fmt<kE5M2>(v, s, amax, c, sat, want_sat);
  else codes_fmt<kE4M3>(v, s, amax, c, sat, want_sat);
}
__device__ __forceinline__ uint32_t code1(float t, bool e5m2) {
  return e5m2 ? encode_fp8<kE5M2>(t) : encode_fp8<kE4M3>(t);
}
__device__ __forceinline__ uint32_t sat1(float t, bool e5m2) {
  return (uint32_t)(fabsf(t) > (e5m2 ? FmtTraits<kE5M2>::kMax : FmtTraits<kE4M3>::kMax));
}

// Commit of a workgroup's amax bits and saturation count for any thread count.
__device__ __forceinline__ void commit(uint32_t amax, uint32_t sat, float* g_amax, uint64_t* g_sat,
                                       uint32_t* smem) {
  Health h;
  block_commit<false>(amax, sat, h, reinterpret_cast<uint32_t*>(g_amax),
                      reinterpret_cast<unsigned long long*>(g_sat), nullptr, smem);
}

// Threads per row and groups of 8 per thread.  Few threads per row keep small rows
// from leaving lanes idle, and up to 8192 columns stay with 256 threads: 1024 threads with
// one group each were no faster for few rows (64 x 8192: 5.2 us both) and slower for more
// (511 x 8192: 10.4 us, 7.7 with 256).
struct RowShape {
  int tpr, vpt;  // vpt 0: the long-row kernel
};
static RowShape row_shape(int64_t cols) {
  const int64_t g = (cols + 7) / 8;
  if (cols < 8) return {1024, 0};  // no whole group to read
  if (g <= 16) return {16, 1};
  if (g <= 64) return {64, 1};
  if (g <= 128) return {64, 2};
  if (g <= 256) return {256, 1};
  if (g <= 512) return {256, 2};
  if (g <= 1024) return {256, 4};
  if (g <= 2048) return {1024, 2};
  if (g <= 4096) return {1024, 4};
  return {1024, 0};
}

}  // namespace fp8ds
