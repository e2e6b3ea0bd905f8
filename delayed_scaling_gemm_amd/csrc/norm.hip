// RMSNorm with the residual's addition and an output in 8 (or 4) bits, forward
// and backward.
//
// What is computed, per row of C elements:
//   h = x + res            rounded to the residual's type when it is BF16: that is
//                          the value the residual stream carries, and everything
//                          below uses it, so the codes, rstd and the backward pass
//                          are functions of what is stored
//   r = 1 / sqrt(sum h^2 / C + eps)
//   y = (h r) gamma
// and from the fp32 y, without a rounding to 16 bits in between, the operand of the
// next product: FP8 with a given (delayed) per-tensor scale, FP8 with a scale per
// row, or blocks of 32 with E8M0 scales (FP8 or FP4 elements).  Sums are fp32: each
// lane adds at most 32 squares in order, lanes are joined as a tree.  Rows longer than the
// registers hold are added in 64 bits by a lane, joined in fp32.
// Backward, with xhat = h r and g = dy gamma:
//   dx = r (g - xhat sum(g xhat) / C) + dres,   dgamma = sum over rows of dy xhat
// (d r / d h_j = -r^3 h_j / C gives the middle term; dres is the gradient that
// reaches h from above, and dx the gradient of both x and res).
//
// Design for gfx950: both directions are HBM-bound, so a row is read once and held
// in registers between its reduction and its output.  TPR threads share a row (16,
// 64, 256 or 1024, so that a thread holds 1 to 4 groups of 8 elements), a workgroup
// takes 256 / TPR rows at a time and goes on to others, the next ones' loads in flight.
// A group of 8 consecutive elements per lane makes 16-byte BF16 accesses, at the
// elements' alignment where rows have no better; a row that is no multiple of 8 long
// has its last elements taken one by one.
//
// Measured, 16384 x 4096 in BF16 with the residual: forward with FP8 output 84 us, 5.6 TB/s
// of 7 B per element (a copy of 1 GiB runs at 5.1); backward with FP8 output 119 us, 5.1 TB/s
// of 9 B, and 6.6 us for the join of dgamma's partials.  Traffic is the algorithm's within
// 1% (backward 3%, the partials).  1531 x 1023 with an FP32 stream and a scale per row, whose rows
// start at odd addresses: 8.4 us, 2.1 TB/s, one round of 383 workgroups and so one chain of
// load, two reductions and store.  At 1024 columns that is 5.7 us; unaligned rows cost 0.6,
// and the last 7 elements 2.0: they are loaded one by one, after the rest and after one another
// for x, the residual and gamma (the backward pass does so for its four operands), and
// stored so too.  One row of 4096: 3.5 us, the launch and a chain of two loads, a reduction
// and a store.

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

// ------------------------------------------------------------------ forward

template <bool XBF, bool HBF, int TPR, int VPT, int MODE, bool AL>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_fwd_kernel(NormArgs p) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  constexpr int RPB = NT / TPR;
  __shared__ uint32_t red[2 * (NT / 64)];
  const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int64_t C = p.cols;
  // group j of this thread: its first column, where it is read, how many elements it has
  auto col = [&](int j) -> int64_t { return ((int64_t)t + TPR * j) * 8; };
  auto at = [&](int j) -> int64_t { return col(j) + 8 <= C ? col(j) : C - 8; };
  auto count = [&](int j) -> int {
    const int64_t left = C - col(j);
    return left <= 0 ? 0 : AL || left >= 8 ? 8 : (int)left;
  };
  struct RowData {
    Raw8<XBF> x[VPT];
    Raw8<HBF> res[VPT];
  };
  // a row's loads; rows past the end read the last one, and are not used
  auto load_row = [&](int64_t row, RowData& d) {
    row = row < p.rows ? row : p.rows - 1;
#pragma unroll
    for (int j = 0; j < VPT; ++j) d.x[j] = load8<XBF, AL>(p.x, row * p.ldx + at(j));
    if (p.res) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) d.res[j] = load8<HBF, AL>(p.res, row * p.ldr + at(j));
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  // The next row is on its way while this one is computed, as far as the registers go: not
  // where 1024 threads, of 128 registers each, hold 4 groups (4096 x 20480: 243 us with it,
  // 184 without).  Those take gamma anew for each row, too, after its reduction (129).
  constexpr bool kFull = TPR == 1024 && VPT == 4;
  constexpr bool kAhead = !kFull && VPT * (XBF ? 4 : 8) + VPT * (HBF ? 4 : 8) <= 32;
  RowData now;
  load_row((int64_t)blockIdx.x * RPB + slot, now);
  Raw8<false> rg[VPT];
  auto load_gamma = [&] {
#pragma unroll
    for (int j = 0; j < VPT; ++j) rg[j] = gamma8<AL>(p.gamma, p.gamma_bf16, at(j));
  };
  if constexpr (!kFull) load_gamma();
  const bool e5m2 = p.fmt == kE5M2;
  const float given = MODE == kQTensor ? *p.scale_in : 1.0f;
  if (MODE == kQTensor && p.scale_used && blockIdx.x == 0 && threadIdx.x == 0) *p.scale_used = given;
  uint32_t amax = 0, sat = 0;  // of all this workgroup's rows (kQTensor)
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < p.rows; r0 += step) {
    const int64_t row = r0 + slot;
    const bool live = row < p.rows;
    RowData next;
    if constexpr (kAhead) {
      if (r0 + step < p.rows) load_row(row + step, next);
    }
    float h[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int n = live ? count(j) : 0;
      unpack8<XBF, AL>(now.x[j], n, h[j]);
      if (!AL && n > 0 && n < 8) load_tail<XBF>(p.x, row * p.ldx + col(j), n, h[j]);
    }
    if (p.res) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int n = live ? count(j) : 0;
        float r[8];
        unpack8<HBF, AL>(now.res[j], n, r);
        if (!AL && n > 0 && n < 8) load_tail<HBF>(p.res, row * p.ldr + col(j), n, r);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          h[j][k] += r[k];
          if constexpr (HBF) h[j][k] = bf16_round(h[j][k]);
        }
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) ss += h[j][k] * h[j][k];
    if (p.h) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (live && count(j) > 0) store8<HBF, AL>(p.h, row * p.ldh + col(j), count(j), h[j]);
    }
    ss = row_sum<TPR>(ss, reinterpret_cast<float*>(red));
    const float rstd = norm_rstd(ss, C, p.eps);
    if (p.rstd && live && t == 0) p.rstd[row] = rstd;
    if constexpr (kFull) load_gamma();
    // y in place of h
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int n = live ? count(j) : 0;
      float g[8];
      unpack_gamma<AL>(rg[j], p.gamma_bf16, n, g);
      if (!AL && n > 0 && n < 8) {
        if (p.gamma_bf16) load_tail<true>(p.gamma, col(j), n, g);
        else load_tail<false>(p.gamma, col(j), n, g);
      }
      // (past the row h is 0, but r may be infinite)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        h[j][k] = k < n ? (h[j][k] * rstd) * g[k] : 0.0f;
        mine = max(mine, abs_bits(h[j][k]));
      }
    }
    if (p.y) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (!live || count(j) == 0) continue;
        if (p.y_bf16) store8<true, AL>(p.y, row * p.ldy + col(j), count(j), h[j]);
        else store8<false, AL>(p.y, row * p.ldy + col(j), count(j), h[j]);
      }
    }
    if constexpr (MODE == kQTensor || MODE == kQRow) {
      float s = given;
      if constexpr (MODE == kQTensor) {
        amax = max(amax, mine);
      } else {
        const uint32_t a = canonical_amax_bits(row_max<TPR>(mine, red));
        s = scale_from_amax(__uint_as_float(a),
                            e5m2 ? FmtTraits<kE5M2>::kMax : FmtTraits<kE4M3>::kMax, p.margin);
        if (live && t == 0) {
          p.scale_out[row] = s;
          if (p.scale_inv) p.scale_inv[row] = __fdiv_rn(1.0f, s);
          if (p.amax) p.amax[row] = __uint_as_float(a);
        }
      }
      // (elements past the row are zeros: they add nothing to the count)
      u32x2 c[VPT];
      codes8(h, s, e5m2, mine, c, sat, MODE == kQTensor && p.sat);
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (live && count(j) > 0) store_codes<AL>(p.q + row * p.ldq + col(j), count(j), c[j]);
    } else if constexpr (MODE == kQMx) {
      // a block of 32 is 4 consecutive lanes (AL only; C is a multiple of 32)
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        uint32_t a = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) a = max(a, abs_bits(h[j][k]));
        a = max(a, (uint32_t)__shfl_xor((int)a, 1));
        a = max(a, (uint32_t)__shfl_xor((int)a, 2));
        const int64_t c0 = col(j);
        if (!live || count(j) == 0) continue;
        const uint32_t code = mx_code(a, p.fmt == kE2M1 ? 2u : e5m2 ? 15u : 8u);
        if ((t & 3) == 0) p.mx_scales[row * p.ldms + c0 / 32] = (uint8_t)code;
        if (p.fmt == kE2M1) {
          const uint32_t c = code == 255u ? kFp4NanBlock : fp4_codes8(h[j], code);
          *reinterpret_cast<uint32_t*>(p.q + row * p.ldq + c0 / 2) = c;
        } else {
          // (with a finite block no product is NaN)
          float u[1][8];
          u32x2 c[1];
          uint32_t unused = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) u[0][k] = h[j][k];
          codes8(u, mx_multiplier(code == 255u ? 127u : code), e5m2, 0u, c, unused, false);
          if (code == 255u) c[0] = u32x2{0x7F7F7F7Fu, 0x7F7F7F7Fu};
          store_codes<true>(p.q + row * p.ldq + c0, 8, c[0]);
        }
      }
    }
    if constexpr (kAhead) {
      now = next;
    } else {
      if (r0 + step < p.rows) load_row(row + step, now);
    }
  }
  if constexpr (MODE == kQTensor) commit(amax, sat, p.amax, p.sat, red);
}

// Rows longer than a workgroup's registers hold, and rows without a whole group of 8: one
// workgroup per row, from row0 on, passes over it two or three times (sum of squares; row
// amax; output).  h is taken back from p.h where it is stored, since p.h may be the
// residual's own buffer.
template <bool XBF, bool HBF, int MODE>
__global__ __launch_bounds__(1024) void norm_fwd_long_kernel(NormArgs p, int64_t row0) {
  __shared__ uint32_t red[2 * 16];
  const int t = threadIdx.x;
  const int64_t row = row0 + blockIdx.x, C = p.cols;
  const int64_t ox = row * p.ldx, orr = row * p.ldr, oh = row * p.ldh;
  auto fresh = [&](int64_t c) {
    float v = load1<XBF>(p.x, ox + c);
    if (p.res) {
      v += load1<HBF>(p.res, orr + c);
      if constexpr (HBF) v = bf16_round(v);
    }
    return v;
  };
  double mine = 0.0;  // cols / 1024 squares, too many for fp32 beyond 65536 columns
  for (int64_t c = t; c < C; c += 1024) {
    const float v = fresh(c);
    mine = fma((double)v, (double)v, mine);
    if (p.h) store1<HBF>(p.h, oh + c, v);
  }
  const float ss = row_sum<1024>((float)mine, reinterpret_cast<float*>(red));
  const float rstd = norm_rstd(ss, C, p.eps);
  if (p.rstd && t == 0) p.rstd[row] = rstd;
  auto value = [&](int64_t c) {
    const float v = p.h ? load1<HBF>(p.h, oh + c) : fresh(c);
    return (v * rstd) * gamma1(p.gamma, p.gamma_bf16, c);
  };
  const bool e5m2 = p.fmt == kE5M2;
  uint32_t amax = 0, sat = 0;
  float s = 1.0f;
  if constexpr (MODE == kQTensor) {
    s = *p.scale_in;
    if (p.scale_used && row == 0 && t == 0) *p.scale_used = s;
  }
  if constexpr (MODE == kQRow) {
    for (int64_t c = t; c < C; c += 1024) amax = max(amax, abs_bits(value(c)));
    amax = canonical_amax_bits(row_max<1024>(amax, red));
    s = scale_from_amax(__uint_as_float(amax),
                        e5m2 ? FmtTraits<kE5M2>::kMax : FmtTraits<kE4M3>::kMax, p.margin);
    if (t == 0) {
      p.scale_out[row] = s;
      if (p.scale_inv) p.scale_inv[row] = __fdiv_rn(1.0f, s);
      if (p.amax) p.amax[row] = __uint_as_float(amax);
    }
  }
  // the lanes of a block of 32 stay together: C is a multiple of 32 with kQMx, and a
  // wave's 64 lanes hold two whole blocks
  for (int64_t c = t; c < C; c += 1024) {
    const float v = value(c);
    if (p.y) {
      if (p.y_bf16)
        store1<true>(p.y, row * p.ldy + c, v);
      else
        store1<false>(p.y, row * p.ldy + c, v);
    }
    if constexpr (MODE == kQTensor) amax = max(amax, abs_bits(v));
    if constexpr (MODE == kQTensor || MODE == kQRow) {
      p.q[row * p.ldq + c] = (uint8_t)code1(v * s, e5m2);
      if (MODE == kQTensor && p.sat) sat += sat1(v * s, e5m2);
    }
    if constexpr (MODE == kQMx) {
      uint32_t a = abs_bits(v);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) a = max(a, (uint32_t)__shfl_xor((int)a, o));
      const uint32_t code = mx_code(a, p.fmt == kE2M1 ? 2u : e5m2 ? 15u : 8u);
      if ((t & 31) == 0) p.mx_scales[row * p.ldms + c / 32] = (uint8_t)code;
      const float m = __uint_as_float(code == 255u ? 0x3F800000u : (254u - code) << 23);
      if (p.fmt == kE2M1) {
        const uint32_t c4 = code == 255u ? (kFp4NanBlock & 15u) : fp4_code1(v * m);
        const uint32_t up = (uint32_t)__shfl_xor((int)c4, 1);
        if ((t & 1) == 0) p.q[row * p.ldq + c / 2] = (uint8_t)(c4 | (up << 4));
      } else {
        p.q[row * p.ldq + c] = code == 255u ? 0x7Fu : (uint8_t)code1(v * m, e5m2);
      }
    }
  }
  if constexpr (MODE == kQTensor) commit(amax, sat, p.amax, p.sat, red);
}

// ------------------------------------------------------------------ backward

// A workgroup takes rows blockIdx.x * RPB + slot, then gridDim.x * RPB further, and
// keeps its share of dgamma in registers: partial [gridDim.x][C] in `work`, summed by
// norm_dgamma_kernel in a fixed order (no atomics: the same inputs give the same
// bits).
template <bool XBF, bool HBF, int TPR, int VPT, bool AL>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_bwd_kernel(NormBwdArgs p) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  constexpr int RPB = NT / TPR;
  __shared__ uint32_t red[2 * (NT / 64)];
  __shared__ float dg_lds[RPB > 1 ? TPR * VPT * 8 : 1];
  const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int64_t C = p.cols;
  auto col = [&](int j) -> int64_t { return ((int64_t)t + TPR * j) * 8; };
  auto count = [&](int j) -> int {
    const int64_t left = C - col(j);
    return left <= 0 ? 0 : AL || left >= 8 ? 8 : (int)left;
  };
  const bool e5m2 = p.fmt == kE5M2;
  float s = 1.0f;
  if (p.q) {
    s = *p.scale_in;
    if (p.scale_used && blockIdx.x == 0 && threadIdx.x == 0) *p.scale_used = s;
  }
  float acc[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[j][k] = 0.0f;
  uint32_t amax = 0, sat = 0;
  const int64_t step = (int64_t)gridDim.x * RPB;
  auto at = [&](int j) -> int64_t { return col(j) + 8 <= C ? col(j) : C - 8; };
  struct RowData {
    Raw8<HBF> h[VPT], dr[VPT];
    Raw8<XBF> dy[VPT];
    float rstd;
  };
  // a row's loads; rows past the end read the last one, and are not used
  auto load_row = [&](int64_t row, RowData& d) {
    row = row < p.rows ? row : p.rows - 1;
#pragma unroll
    for (int j = 0; j < VPT; ++j) d.h[j] = load8<HBF, AL>(p.h, row * p.ldh + at(j));
#pragma unroll
    for (int j = 0; j < VPT; ++j) d.dy[j] = load8<XBF, AL>(p.dy, row * p.lddy + at(j));
    if (p.dres) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) d.dr[j] = load8<HBF, AL>(p.dres, row * p.lddr + at(j));
    }
    d.rstd = p.rstd[row];
  };
  Raw8<false> rg[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) rg[j] = gamma8<AL>(p.gamma, p.gamma_bf16, at(j));
  // The next row is on its way while this one is computed, as far as the registers go.
  constexpr bool kAhead = VPT * ((HBF ? 8 : 16) + (XBF ? 4 : 8)) <= 32;
  RowData now;
  if constexpr (kAhead) load_row((int64_t)blockIdx.x * RPB + slot, now);
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < p.rows; r0 += step) {
    const int64_t row = r0 + slot;
    const bool live = row < p.rows;
    RowData next;
    if constexpr (kAhead) load_row(row + step, next);
    else load_row(row, now);
    float xh[VPT][8], g[VPT][8];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int n = live ? count(j) : 0;
      float gm[8];
      unpack8<HBF, AL>(now.h[j], n, xh[j]);
      unpack8<XBF, AL>(now.dy[j], n, g[j]);
      unpack_gamma<AL>(rg[j], p.gamma_bf16, n, gm);
      if (!AL && n > 0 && n < 8) {
        load_tail<HBF>(p.h, row * p.ldh + col(j), n, xh[j]);
        load_tail<XBF>(p.dy, row * p.lddy + col(j), n, g[j]);
        if (p.gamma_bf16) load_tail<true>(p.gamma, col(j), n, gm);
        else load_tail<false>(p.gamma, col(j), n, gm);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        xh[j][k] = k < n ? xh[j][k] * now.rstd : 0.0f;  // (rstd may be infinite)
        acc[j][k] += g[j][k] * xh[j][k];
        g[j][k] *= gm[k];
        dot += g[j][k] * xh[j][k];
      }
    }
    const float mean = row_sum<TPR>(dot, reinterpret_cast<float*>(red)) / (float)C;
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int n = live ? count(j) : 0;
      float dr[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (p.dres) {
        unpack8<HBF, AL>(now.dr[j], n, dr);
        if (!AL && n > 0 && n < 8) load_tail<HBF>(p.dres, row * p.lddr + col(j), n, dr);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        g[j][k] = k < n ? now.rstd * (g[j][k] - xh[j][k] * mean) + dr[k] : 0.0f;
        mine = max(mine, abs_bits(g[j][k]));
      }
      if (n > 0) store8<HBF, AL>(p.dx, row * p.lddx + col(j), n, g[j]);
    }
    if (p.q) {
      amax = max(amax, mine);
      u32x2 c[VPT];
      codes8(g, s, e5m2, mine, c, sat, p.sat != nullptr);
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (live && count(j) > 0) store_codes<AL>(p.q + row * p.ldq + col(j), count(j), c[j]);
    }
    if constexpr (kAhead) now = next;
  }
  // dgamma: the slots of a workgroup one after the other, then one partial row
  float* out = p.work + (int64_t)blockIdx.x * C;
  if constexpr (RPB > 1) {
    for (int w = 0; w < RPB; ++w) {
      if (slot == w) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float* d = &dg_lds[(j * 8 + k) * TPR + t];
            *d = w == 0 ? acc[j][k] : *d + acc[j][k];
          }
      }
      __syncthreads();
    }
    if (slot == 0) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < count(j)) out[col(j) + k] = dg_lds[(j * 8 + k) * TPR + t];
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < count(j)) out[col(j) + k] = acc[j][k];
  }
  if (p.q) commit(amax, sat, p.amax, p.sat, red);
}

// Rows longer than the registers: one workgroup walks its rows, each read twice; its
// dgamma partial is kept in `work` (each element by one thread).
template <bool XBF, bool HBF>
__global__ __launch_bounds__(1024) void norm_bwd_long_kernel(NormBwdArgs p) {
  __shared__ uint32_t red[2 * 16];
  const int t = threadIdx.x;
  const int64_t C = p.cols;
  const bool e5m2 = p.fmt == kE5M2;
  float s = 1.0f;
  if (p.q) {
    s = *p.scale_in;
    if (p.scale_used && blockIdx.x == 0 && t == 0) *p.scale_used = s;
  }
  float* out = p.work + (int64_t)blockIdx.x * C;
  uint32_t amax = 0, sat = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float rstd = p.rstd[row];
    double dot = 0.0;
    for (int64_t c = t; c < C; c += 1024) {
      const float xh = load1<HBF>(p.h, row * p.ldh + c) * rstd;
      const float dy = load1<XBF>(p.dy, row * p.lddy + c);
      dot += (double)(dy * gamma1(p.gamma, p.gamma_bf16, c) * xh);
      out[c] = dy * xh + (row == (int64_t)blockIdx.x ? 0.0f : out[c]);
    }
    const float mean = row_sum<1024>((float)dot, reinterpret_cast<float*>(red)) / (float)C;
    for (int64_t c = t; c < C; c += 1024) {
      const float xh = load1<HBF>(p.h, row * p.ldh + c) * rstd;
      const float g = load1<XBF>(p.dy, row * p.lddy + c) * gamma1(p.gamma, p.gamma_bf16, c);
      float d = rstd * (g - xh * mean);
      if (p.dres) d += load1<HBF>(p.dres, row * p.lddr + c);
      store1<HBF>(p.dx, row * p.lddx + c, d);
      if (p.q) {
        amax = max(amax, abs_bits(d));
        p.q[row * p.ldq + c] = (uint8_t)code1(d * s, e5m2);
        if (p.sat) sat += sat1(d * s, e5m2);
      }
    }
  }
  if (p.q) commit(amax, sat, p.amax, p.sat, red);
}

// dgamma[c] = sum of `parts` partial rows: 32 columns x 16 shares of the rows per
// workgroup, joined in LDS in a fixed order; columns from c0 on.
__global__ __launch_bounds__(512) void norm_dgamma_kernel(const float* __restrict__ work, int parts,
                                                          int64_t C, float* __restrict__ dgamma,
                                                          int64_t c0) {
  __shared__ float part[16][33];
  const int cl = threadIdx.x & 31, sh = threadIdx.x >> 5;
  const int64_t c = c0 + (int64_t)blockIdx.x * 32 + cl;
  float v = 0.0f;
  if (c < C) {
#pragma unroll 4
    for (int i = sh; i < parts; i += 16) v += work[(int64_t)i * C + c];
  }
  part[sh][cl] = v;
  __syncthreads();
  if (sh == 0 && c < C) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += part[i][cl];
    dgamma[c] = t;
  }
}

// ------------------------------------------------------------------ host launchers

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

// Workgroups: as many as run at once, 8 per CU of 256 threads, one of 1024 (two: 512 x 16384
// 16.1 us, one 12.3).  Reading a row twice from memory, as longer ones are, took 347 us for
// 4096 x 20480 and 534 for 4096 x 32768; in registers 129 and 176.
template <bool XBF, bool HBF, int MODE, bool AL>
static hipError_t launch_fwd(const NormArgs& a, RowShape sh, int num_cus, hipStream_t stream) {
#define FP8DS_NORM_CASE(T, V)                                                                    \
  if (sh.tpr == T && sh.vpt == V) {                                                              \
    const int64_t rpb = T > 256 ? 1 : 256 / T, blocks = (a.rows + rpb - 1) / rpb;                \
    const int64_t most = (int64_t)num_cus * (T > 256 ? 1 : 8);                                   \
    hipLaunchKernelGGL((norm_fwd_kernel<XBF, HBF, T, V, MODE, AL>),                              \
                       dim3((unsigned)(blocks < most ? blocks : most)), dim3(T > 256 ? T : 256), \
                       0, stream, a);                                                            \
    return hipGetLastError();                                                                    \
  }
  FP8DS_NORM_CASE(16, 1)
  FP8DS_NORM_CASE(64, 1)
  FP8DS_NORM_CASE(64, 2)
  FP8DS_NORM_CASE(256, 1)
  FP8DS_NORM_CASE(256, 2)
  FP8DS_NORM_CASE(256, 4)
  FP8DS_NORM_CASE(1024, 2)
  FP8DS_NORM_CASE(1024, 4)
#undef FP8DS_NORM_CASE
  // A grid holds fewer than 2^32 threads; of a larger one HIP drops the excess without an error.
  // (Workgroups that go on to further rows instead: 4096 x 40000 981 us, a row each 656.)
  constexpr int64_t kSlice = 1 << 21;
  for (int64_t r0 = 0; r0 < a.rows; r0 += kSlice) {
    const int64_t n = a.rows - r0 < kSlice ? a.rows - r0 : kSlice;
    hipLaunchKernelGGL((norm_fwd_long_kernel<XBF, HBF, MODE>), dim3((unsigned)n), dim3(1024), 0,
                       stream, a, r0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool XBF, bool HBF>
static hipError_t launch_fwd_t(const NormArgs& a, RowShape sh, int n, hipStream_t s) {
  switch (a.mode) {
    case kQNone: return a.vec ? launch_fwd<XBF, HBF, kQNone, true>(a, sh, n, s)
                              : launch_fwd<XBF, HBF, kQNone, false>(a, sh, n, s);
    case kQTensor: return a.vec ? launch_fwd<XBF, HBF, kQTensor, true>(a, sh, n, s)
                                : launch_fwd<XBF, HBF, kQTensor, false>(a, sh, n, s);
    case kQRow: return a.vec ? launch_fwd<XBF, HBF, kQRow, true>(a, sh, n, s)
                             : launch_fwd<XBF, HBF, kQRow, false>(a, sh, n, s);
    default: return launch_fwd<XBF, HBF, kQMx, true>(a, sh, n, s);
  }
}

hipError_t launch_norm_fwd(const NormArgs& a, int num_cus, hipStream_t stream) {
  const RowShape sh = row_shape(a.cols);
  if (a.x_bf16 && a.h_bf16) return launch_fwd_t<true, true>(a, sh, num_cus, stream);
  if (a.x_bf16) return launch_fwd_t<true, false>(a, sh, num_cus, stream);
  return launch_fwd_t<false, false>(a, sh, num_cus, stream);
}

// The backward pass holds four values per element: 512 threads, whose waves may have
// 256 registers, take up to 16384 columns (4096 x 16384: 134 us, read twice 362); 1024
// threads (128 registers) would spill.
static RowShape bwd_shape(int64_t cols) {
  const int64_t g = (cols + 7) / 8;
  if (cols < 8) return {1024, 0};
  if (g <= 1024) return row_shape(cols);
  if (g <= 2048) return {512, 4};
  return {1024, 0};
}

// Workgroups of the backward pass: at most 1024, so that the dgamma partials stay a
// small part of the traffic.
int norm_bwd_parts(int64_t rows, int64_t cols) {
  const RowShape sh = bwd_shape(cols);
  const int64_t rpb = sh.tpr > 256 ? 1 : 256 / sh.tpr;
  const int64_t blocks = (rows + rpb - 1) / rpb;
  return (int)(blocks < 1024 ? blocks : 1024);
}

template <bool XBF, bool HBF, bool AL>
static hipError_t launch_bwd(const NormBwdArgs& a, RowShape sh, int parts, hipStream_t stream) {
#define FP8DS_NORM_CASE(T, V)                                                                     \
  if (sh.tpr == T && sh.vpt == V) {                                                               \
    hipLaunchKernelGGL((norm_bwd_kernel<XBF, HBF, T, V, AL>), dim3((unsigned)parts),             \
                       dim3(T > 256 ? T : 256), 0, stream, a);                                    \
    return hipGetLastError();                                                                     \
  }
  FP8DS_NORM_CASE(16, 1)
  FP8DS_NORM_CASE(64, 1)
  FP8DS_NORM_CASE(64, 2)
  FP8DS_NORM_CASE(256, 1)
  FP8DS_NORM_CASE(256, 2)
  FP8DS_NORM_CASE(256, 4)
  FP8DS_NORM_CASE(512, 4)
#undef FP8DS_NORM_CASE
  hipLaunchKernelGGL((norm_bwd_long_kernel<XBF, HBF>), dim3((unsigned)parts), dim3(1024), 0, stream,
                     a);
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormBwdArgs& a, hipStream_t stream) {
  const RowShape sh = bwd_shape(a.cols);
  const int parts = norm_bwd_parts(a.rows, a.cols);
  hipError_t e = hipSuccess;
  if (parts > 0) {
    if (a.x_bf16 && a.h_bf16)
      e = a.vec ? launch_bwd<true, true, true>(a, sh, parts, stream)
                : launch_bwd<true, true, false>(a, sh, parts, stream);
    else if (a.x_bf16)
      e = a.vec ? launch_bwd<true, false, true>(a, sh, parts, stream)
                : launch_bwd<true, false, false>(a, sh, parts, stream);
    else
      e = a.vec ? launch_bwd<false, false, true>(a, sh, parts, stream)
                : launch_bwd<false, false, false>(a, sh, parts, stream);
  }
  if (e != hipSuccess) return e;
  constexpr int64_t kSlice = 1 << 27;  // columns; 2^31 threads, of fewer than 2^32 in a grid
  for (int64_t c0 = 0; c0 < a.cols; c0 += kSlice) {
    const int64_t n = a.cols - c0 < kSlice ? a.cols - c0 : kSlice;
    hipLaunchKernelGGL(norm_dgamma_kernel, dim3((unsigned)((n + 31) / 32)), dim3(512), 0, stream,
                       a.work, parts, a.cols, a.dgamma, c0);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp8ds
