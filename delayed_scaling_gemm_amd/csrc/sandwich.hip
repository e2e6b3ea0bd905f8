// The norms around a residual addition, with the branch's gate and the residual scale, forward and
// backward: what stands between two blocks whose output is normalised before it is added.
//
// Per row of C elements, x the branch's output, res the residual stream:
//   r1 = 1 / sqrt(sum x^2 / C + e1),   p = (x r1) k,   k = alpha gate gamma1
//   h  = res + t p                     rounded to the stream's type; everything below uses it so
//   r2 = 1 / sqrt(sum h^2 / C + e2),   y = (h r2) gamma2, cast as the norm's output is
// gate [C] and t [rows] (one factor per token) may be absent.  Backward, xh1 = x r1, xh2 = h r2:
//   g2 = dy gamma2,  dh = r2 (g2 - xh2 sum(g2 xh2) / C) + dres     the gradient of res
//   g1 = t k dh,     dx = r1 (g1 - xh1 sum(g1 xh1) / C)            from the fp32 dh
//   dgamma2 = sum over rows dy xh2,  S = sum over rows alpha t dh xh1,
//   dgamma1 = gate S,  dgate = gamma1 S,  dt = sum_c k dh xh1
// so two column sums serve three parameters, and the sum that dx needs is t dt.
//
// Design for gfx950: HBM-bound, as the norm (norm.hip), whose row layout this shares: rows once
// through registers, two reductions one after the other in each direction, a row's loads issued
// together and the next row's ahead.  k is computed once per workgroup.  dgamma goes through one
// partial row per workgroup and sum, joined in a fixed order.
// 16384 x 4096 in BF16: forward to FP8 90 us (5.2 TB/s), backward with the FP8 copy of dx 149
// (5.0 TB/s; 8 of them the join).  One row of 4096: 5.0 to 5.4 on the device.

#include "norm_common.h"

namespace fp8ds {

// A row's last group, where it is not whole, is read as the row's last eight elements: the first 8 - n
// of them are the group before's too and only left out of the sums, so a ragged row has no element that
// is loaded by itself (each row waited for those: 8000 x 6999 forward 412 us, so 116; backward 764,
// 282).  Those 8 - n are not stored either, nor in a maximum: where the output is an input's storage the
// group before may have stored its own before this group's loads have come back (a barrier of a workgroup
// does not wait for loads), so what is worked out for them may be anything.  Groups past the row read the
// same eight, and count for nothing.
template <bool BF, bool AL>
__device__ __forceinline__ void take8(const Raw8<BF>& r, int n, float (&v)[8]) {
  unpack8<BF, AL>(r, AL ? n : 8, v);
}
template <bool AL>
__device__ __forceinline__ void take_gamma(const Raw8<false>& r, bool bf, int n, float (&v)[8]) {
  unpack_gamma<AL>(r, bf, AL ? n : 8, v);
}
// Aligned rows have whole groups only, and groups past the row are kept at zero (`held`: r may be
// infinite); of others each element is asked whether it counts.
template <bool AL>
__device__ __forceinline__ float held(int n, float v) {
  return !AL || n > 0 ? v : 0.0f;
}
template <bool AL>
__device__ __forceinline__ float counted(int i, int n, float v) {
  return AL || i >= 8 - n ? v : 0.0f;
}

// A group's own elements; i is where its eight stand (`at`).
template <bool BF, bool AL>
__device__ __forceinline__ void store_own(void* p, int64_t i, int n, const float (&v)[8]) {
  if (AL || n == 8) {
    store8<BF, AL>(p, i, 8, v);
    return;
  }
#pragma unroll
  for (int k = 1; k < 8; ++k)
    if (k >= 8 - n) store1<BF>(p, i + k, v[k]);
}
template <bool AL>
__device__ __forceinline__ void store_own_codes(uint8_t* p, int n, const u32x2& c) {
  if (AL || n == 8) {
    store_codes<AL>(p, 8, c);
    return;
  }
#pragma unroll
  for (int k = 1; k < 8; ++k)
    if (k >= 8 - n) p[k] = (uint8_t)(c[k >> 2] >> (8 * (k & 3)));
}
template <bool AL>
__device__ __forceinline__ uint32_t counted_bits(int i, int n, float v) {
  return AL || i >= 8 - n ? abs_bits(v) : 0u;
}

// codes8 of a row's groups, each element counted once.
template <int VPT, bool AL, typename Count>
__device__ __forceinline__ void cast_row(const float (&v)[VPT][8], float s, bool e5m2, uint32_t amax,
                                         bool live, const Count& count, u32x2 (&c)[VPT], uint32_t& sat,
                                         bool want_sat) {
  uint32_t unused = 0;
  codes8(v, s, e5m2, amax, c, unused, false);
  if (want_sat) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int n = live ? count(j) : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sat += i >= 8 - n ? sat1(v[j][i] * s, e5m2) : 0u;
    }
  }
}

// A row's output, from h in registers: y = (h rstd) gamma in place of h, stored and cast as MODE says
// (norm.hip has these lines in its kernels: as a function they cost its longest rows 5 to 20 times the
// spilled registers).
// `given`: the per-tensor scale; amax and sat: this workgroup's, of kQTensor.
// `at`, `count`: where a group is read and its elements, as the kernel has them.
template <int TPR, int VPT, int MODE, bool AL, typename Args, typename At, typename Count>
__device__ __forceinline__ void emit_row(const Args& p, const int64_t row, const bool live, const int t,
                                         const float rstd, float (&h)[VPT][8],
                                         const Raw8<false> (&rg)[VPT], const float given,
                                         const bool e5m2, uint32_t& amax, uint32_t& sat, uint32_t* red,
                                         const At& at, const Count& count) {
  uint32_t mine = 0;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int n = live ? count(j) : 0;
    float g[8];
    take_gamma<AL>(rg[j], p.gamma_bf16, n, g);
    // (past the row r may be infinite)
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      h[j][k] = (h[j][k] * rstd) * g[k];
      most = max(most, counted_bits<AL>(k, n, h[j][k]));
    }
    mine = max(mine, n > 0 ? most : 0u);
  }
  if (p.y) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (!live || count(j) == 0) continue;
      if (p.y_bf16) store_own<true, AL>(p.y, row * p.ldy + at(j), count(j), h[j]);
      else store_own<false, AL>(p.y, row * p.ldy + at(j), count(j), h[j]);
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
    u32x2 c[VPT];
    cast_row<VPT, AL>(h, s, e5m2, mine, live, count, c, sat, MODE == kQTensor && p.sat);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (live && count(j) > 0) store_own_codes<AL>(p.q + row * p.ldq + at(j), count(j), c[j]);
  } else if constexpr (MODE == kQMx) {
    // a block of 32 is 4 consecutive lanes (AL only; C is a multiple of 32)
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      uint32_t a = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) a = max(a, abs_bits(h[j][k]));
      a = max(a, (uint32_t)__shfl_xor((int)a, 1));
      a = max(a, (uint32_t)__shfl_xor((int)a, 2));
      const int64_t c0 = at(j);
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
}

// The same for rows that are read again: value(c) is y of column c.  1024 threads.
template <int MODE, typename Args, typename Value>
__device__ __forceinline__ void emit_long(const Args& p, int64_t row, const Value& value, uint32_t* red) {
  const int t = threadIdx.x;
  const int64_t C = p.cols;
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

// A thread's groups of a parameter row [C] of either type.
template <int TPR, int VPT, bool AL>
__device__ __forceinline__ void load_param(const void* g, bool bf, int t, int64_t C, float (&v)[VPT][8]) {
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int64_t c = ((int64_t)t + TPR * j) * 8, left = C - c;
    const int n = left <= 0 ? 0 : AL || left >= 8 ? 8 : (int)left;
    take_gamma<AL>(gamma8<AL>(g, bf, c + 8 <= C ? c : C - 8), bf, n, v[j]);
  }
}

// k = alpha gate gamma1 of this thread's columns.
template <int TPR, int VPT, bool AL, typename Args>
__device__ __forceinline__ void load_k(const Args& p, int t, int64_t C, float (&k)[VPT][8]) {
  load_param<TPR, VPT, AL>(p.post_gamma, p.post_gamma_bf16, t, C, k);
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) k[j][i] *= p.alpha;
  if (p.gate) {
    float g[VPT][8];
    load_param<TPR, VPT, AL>(p.gate, p.gate_bf16, t, C, g);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) k[j][i] *= g[j][i];
  }
}
template <typename Args>
__device__ __forceinline__ float k1(const Args& p, int64_t c) {
  const float k = gamma1(p.post_gamma, p.post_gamma_bf16, c) * p.alpha;
  return p.gate ? k * gamma1(p.gate, p.gate_bf16, c) : k;
}

// ------------------------------------------------------------------ forward

// h = res + (x r1) t k in 64 bits, rounded to fp32 once (rows of 8 to 16384 columns).  In fp32 its error of a
// unit or so put one BF16 value in 190000 on the other side of a border; memory's time hides the 64-bit
// arithmetic, which has fp32's rate (16384 x 4096 in BF16: 86 us with either; 8192 x 8192: 90, 86 in fp32;
// 4096 x 16384 with an FP32 stream: 138, 168).  k in 64 bits is kept in LDS: in registers it would take the
// room of the next row's loads.  Squares are added in pairs in fp32, whose errors average out, and in 64
// bits from there on.
typedef double v2d __attribute__((ext_vector_type(2)));
template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 15, 15, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 15, 15, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int W>  // lanes W apart, 16 or 32
__device__ __forceinline__ double add_swapped(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t l = (uint32_t)b, h = (uint32_t)(b >> 32);
  const auto p = W == 16 ? __builtin_amdgcn_permlane16_swap(l, l, false, false)
                         : __builtin_amdgcn_permlane32_swap(l, l, false, false);
  const auto q = W == 16 ? __builtin_amdgcn_permlane16_swap(h, h, false, false)
                         : __builtin_amdgcn_permlane32_swap(h, h, false, false);
  return __builtin_bit_cast(double, (uint64_t)q[0] << 32 | p[0]) +
         __builtin_bit_cast(double, (uint64_t)q[1] << 32 | p[1]);
}
// Sum over the TPR threads of a row, as row_sum, but within a wave without LDS's way there and back
// (8192 x 8192: 92 us with shuffles of both words, 90).
template <int TPR>
__device__ __forceinline__ double row_sum64(double v, double* red) {
  v = add_dpp<0xB1>(v);   // lanes 1 apart
  v = add_dpp<0x4E>(v);   // 2
  v = add_dpp<0x141>(v);  // the halves of 8 lanes, mirrored
  v = add_dpp<0x140>(v);  // of 16
  if constexpr (TPR > 16) v = add_swapped<32>(add_swapped<16>(v));
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < NW; ++w) t += red[w];
    __syncthreads();
    v = t;
  }
  return v;
}
// 1 / sqrt(mean + eps): the hardware's, 2^-26 and better, and one step that squares the error.
__device__ __forceinline__ double rstd64(double mean, float eps) {
  const double v = mean + (double)eps, y = __builtin_amdgcn_rsq(v);
  const double e = __builtin_fma(-v * y, y, 1.0);
  return fabs(e) < 1.0 ? __builtin_fma(0.5 * e, y, y) : y;  // (0, infinite, NaN: as it came)
}
template <typename Args>
__device__ __forceinline__ double k64(const Args& p, float post_gamma, float gate) {
  return (double)p.alpha * (double)post_gamma * (double)gate;
}

// BF16 rows of 2049 to 4096 columns fit into 128 registers, four waves a SIMD, which the compiler has to be
// told (16384 x 4096 with a scale per row: 94 us with three, 88; with an FP32 x or stream it would spill).
template <bool XBF, bool HBF, int TPR, int VPT, int MODE, bool AL>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256, XBF && HBF && TPR == 256 && VPT == 2 ? 4 : 1)
void sandwich_fwd_kernel(SandwichArgs p) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  constexpr int RPB = NT / TPR;
  __shared__ __attribute__((aligned(8))) uint32_t red[2 * (NT / 64)];
  constexpr bool kFull = TPR == 1024 && VPT == 4;
  __shared__ v2d k_lds[kFull ? 1 : TPR * VPT * 4];  // k of every column
  const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int64_t C = p.cols;
  auto col = [&](int j) -> int64_t { return ((int64_t)t + TPR * j) * 8; };
  auto at = [&](int j) -> int64_t { return col(j) + 8 <= C ? col(j) : C - 8; };
  auto count = [&](int j) -> int {
    const int64_t left = C - col(j);
    return left <= 0 ? 0 : AL || left >= 8 ? 8 : (int)left;
  };
  // Rows of more than 16384 columns: parameters again for each row and group, the stream's group
  // when x has been taken (4096 x 20480: 463 us with all of them held, 245).
  struct RowData {
    Raw8<XBF> x[VPT];
    Raw8<HBF> res[kFull ? 1 : VPT];
    float t;
  };
  // a row's loads; rows past the end read the last one, and are not used
  auto load_row = [&](int64_t row, RowData& d) {
    row = row < p.rows ? row : p.rows - 1;
#pragma unroll
    for (int j = 0; j < VPT; ++j) d.x[j] = load8<XBF, AL>(p.x, row * p.ldx + at(j));
    if constexpr (!kFull) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) d.res[j] = load8<HBF, AL>(p.res, row * p.ldr + at(j));
    }
    d.t = p.row_gate ? p.row_gate[row] : 1.0f;
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  constexpr bool kAhead = !kFull && VPT * (XBF ? 4 : 8) + VPT * (HBF ? 4 : 8) <= 32;
  RowData now;
  load_row((int64_t)blockIdx.x * RPB + slot, now);
  Raw8<false> rg[VPT];
  auto load_gamma = [&] {
#pragma unroll
    for (int j = 0; j < VPT; ++j) rg[j] = gamma8<AL>(p.gamma, p.gamma_bf16, at(j));
  };
  if constexpr (!kFull) {
    if (slot == 0) {
      float pg[VPT][8], g[VPT][8];
      load_param<TPR, VPT, AL>(p.post_gamma, p.post_gamma_bf16, t, C, pg);
      if (p.gate) load_param<TPR, VPT, AL>(p.gate, p.gate_bf16, t, C, g);
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          k_lds[(j * 4 + i / 2) * TPR + t] = v2d{k64(p, pg[j][i], p.gate ? g[j][i] : 1.0f),
                                                 k64(p, pg[j][i + 1], p.gate ? g[j][i + 1] : 1.0f)};
    }
    load_gamma();
    __syncthreads();
  }
  const bool e5m2 = p.fmt == kE5M2;
  const double inv_c = 1.0 / (double)C;
  const float given = MODE == kQTensor ? *p.scale_in : 1.0f;
  if (MODE == kQTensor && p.scale_used && blockIdx.x == 0 && threadIdx.x == 0) *p.scale_used = given;
  uint32_t amax = 0, sat = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < p.rows; r0 += step) {
    const int64_t row = r0 + slot;
    const bool live = row < p.rows;
    RowData next;
    if constexpr (kAhead) {
      if (r0 + step < p.rows) load_row(row + step, next);
    }
    float h[VPT][8];
    double sx = 0.0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int n = live ? count(j) : 0;
      take8<XBF, AL>(now.x[j], n, h[j]);
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        sx += (double)(counted<AL>(i, n, h[j][i] * h[j][i]) + counted<AL>(i + 1, n, h[j][i + 1] * h[j][i + 1]));
    }
    const double r1 = rstd64(row_sum64<TPR>(sx, reinterpret_cast<double*>(red)) * inv_c, p.post_eps);
    if (p.post_rstd && live && t == 0) p.post_rstd[row] = (float)r1;
    const double r1t = r1 * (double)now.t;
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int n = live ? count(j) : 0;
      float r[8];
      float k[8];
      if constexpr (kFull) {
        now.res[0] = load8<HBF, AL>(p.res, (live ? row : p.rows - 1) * p.ldr + at(j));
        take_gamma<AL>(gamma8<AL>(p.post_gamma, p.post_gamma_bf16, at(j)), p.post_gamma_bf16, n, k);
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] *= p.alpha;
        if (p.gate) {
          float g[8];
          take_gamma<AL>(gamma8<AL>(p.gate, p.gate_bf16, at(j)), p.gate_bf16, n, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) k[i] *= g[i];
        }
      }
      take8<HBF, AL>(now.res[kFull ? 0 : j], n, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (kFull) {
          h[j][i] = held<AL>(n, __builtin_fmaf(h[j][i], (float)r1t * k[i], r[i]));
        } else {
          const double k2 = k_lds[(j * 4 + i / 2) * TPR + t][i & 1];
          h[j][i] = held<AL>(n, (float)__builtin_fma((double)h[j][i], r1t * k2, (double)r[i]));
        }
        if constexpr (HBF) h[j][i] = bf16_round(h[j][i]);
        ss += counted<AL>(i, n, h[j][i] * h[j][i]);
      }
      if (n > 0) store_own<HBF, AL>(p.h, row * p.ldh + at(j), n, h[j]);
    }
    ss = (float)row_sum64<TPR>((double)ss, reinterpret_cast<double*>(red));
    const float rstd = norm_rstd(ss, C, p.eps);
    if (p.rstd && live && t == 0) p.rstd[row] = rstd;
    if constexpr (kFull) load_gamma();
    emit_row<TPR, VPT, MODE, AL>(p, row, live, t, rstd, h, rg, given, e5m2, amax, sat, red, at,
                                 count);
    if constexpr (kAhead) {
      now = next;
    } else {
      if (r0 + step < p.rows) load_row(row + step, now);
    }
  }
  if constexpr (MODE == kQTensor) commit(amax, sat, p.amax, p.sat, red);
}

// Rows longer than a workgroup's registers hold, and rows without a whole group of 8: one
// workgroup per row, from row0 on.  h is taken back from where it is stored.
template <bool XBF, bool HBF, int MODE>
__global__ __launch_bounds__(1024) void sandwich_fwd_long_kernel(SandwichArgs p, int64_t row0) {
  __shared__ uint32_t red[2 * 16];
  const int t = threadIdx.x;
  const int64_t row = row0 + blockIdx.x, C = p.cols;
  double mine = 0.0;  // cols / 1024 squares, too many for fp32 beyond 65536 columns
  for (int64_t c = t; c < C; c += 1024) {
    const double v = load1<XBF>(p.x, row * p.ldx + c);
    mine = fma(v, v, mine);
  }
  const float r1 = norm_rstd(row_sum<1024>((float)mine, reinterpret_cast<float*>(red)), C, p.post_eps);
  if (p.post_rstd && t == 0) p.post_rstd[row] = r1;
  const float tok = p.row_gate ? p.row_gate[row] : 1.0f;
  mine = 0.0;
  for (int64_t c = t; c < C; c += 1024) {
    float v = __builtin_fmaf(load1<XBF>(p.x, row * p.ldx + c), (r1 * tok) * k1(p, c),
                             load1<HBF>(p.res, row * p.ldr + c));
    if constexpr (HBF) v = bf16_round(v);
    store1<HBF>(p.h, row * p.ldh + c, v);
    mine = fma((double)v, (double)v, mine);
  }
  const float rstd = norm_rstd(row_sum<1024>((float)mine, reinterpret_cast<float*>(red)), C, p.eps);
  if (p.rstd && t == 0) p.rstd[row] = rstd;
  auto value = [&](int64_t c) {
    return (load1<HBF>(p.h, row * p.ldh + c) * rstd) * gamma1(p.gamma, p.gamma_bf16, c);
  };
  emit_long<MODE>(p, row, value, red);
}

// ------------------------------------------------------------------ backward

// Partial column sums of a workgroup: [2][gridDim.x][C] in `work`, dy xh2 and alpha t dh xh1.
template <bool XBF, bool HBF, int TPR, int VPT, bool AL>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void sandwich_bwd_kernel(SandwichBwdArgs p) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  constexpr int RPB = NT / TPR;
  __shared__ uint32_t red[2 * (NT / 64)];
  __shared__ float part_lds[RPB > 1 ? TPR * VPT * 8 : 1];
  // Rows of 8192 to 16384 columns, 1024 threads of 128 registers: the column sums are kept in LDS, the
  // parameters read again for each row, dres and x only when h and dy have been taken (7404 x 9063 in
  // 512 threads, all in registers: 1442 us, so 489; 4096 x 16384 526, 218).
  constexpr bool kLean = TPR == 1024;
  __shared__ float acc_lds[kLean ? 2 * TPR * VPT * 8 : 1];
  const int t = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int64_t C = p.cols;
  auto col = [&](int j) -> int64_t { return ((int64_t)t + TPR * j) * 8; };
  auto at = [&](int j) -> int64_t { return col(j) + 8 <= C ? col(j) : C - 8; };
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
  float acc2[kLean ? 1 : VPT][8], acc1[kLean ? 1 : VPT][8];
  auto sum2 = [&](int j, int i) -> float& {
    if constexpr (kLean) return acc_lds[(j * 8 + i) * TPR + t];
    else return acc2[j][i];
  };
  auto sum1 = [&](int j, int i) -> float& {
    if constexpr (kLean) return acc_lds[((VPT + j) * 8 + i) * TPR + t];
    else return acc1[j][i];
  };
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum2(j, i) = sum1(j, i) = 0.0f;
  uint32_t amax = 0, sat = 0;
  struct RowData {
    Raw8<HBF> h[VPT], dr[VPT];
    Raw8<XBF> dy[VPT], x[VPT];
    float r1, r2, t;
  };
  auto load_first = [&](int64_t row, RowData& d) {
    row = row < p.rows ? row : p.rows - 1;
#pragma unroll
    for (int j = 0; j < VPT; ++j) d.h[j] = load8<HBF, AL>(p.h, row * p.ldh + at(j));
#pragma unroll
    for (int j = 0; j < VPT; ++j) d.dy[j] = load8<XBF, AL>(p.dy, row * p.lddy + at(j));
    d.r1 = p.post_rstd[row];
    d.r2 = p.rstd[row];
    d.t = p.row_gate ? p.row_gate[row] : 1.0f;
  };
  auto load_second = [&](int64_t row, RowData& d) {
    row = row < p.rows ? row : p.rows - 1;
    if (p.dres) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) d.dr[j] = load8<HBF, AL>(p.dres, row * p.lddr + at(j));
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) d.x[j] = load8<XBF, AL>(p.x, row * p.ldx + at(j));
  };
  auto load_row = [&](int64_t row, RowData& d) {
    load_first(row, d);
    if constexpr (!kLean) load_second(row, d);
  };
  float k[kLean ? 1 : VPT][8];
  Raw8<false> rg[kLean ? 1 : VPT];
  if constexpr (!kLean) {
    load_k<TPR, VPT, AL>(p, t, C, k);
#pragma unroll
    for (int j = 0; j < VPT; ++j) rg[j] = gamma8<AL>(p.gamma, p.gamma_bf16, at(j));
  }
  auto param8 = [&](const void* v, bool bf, int j, int n, float (&out)[8]) {
    take_gamma<AL>(gamma8<AL>(v, bf, at(j)), bf, n, out);
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  constexpr bool kAhead = !kLean && VPT * ((HBF ? 8 : 16) + (XBF ? 8 : 16)) <= 32;
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
      take8<HBF, AL>(now.h[j], n, xh[j]);
      take8<XBF, AL>(now.dy[j], n, g[j]);
      if constexpr (kLean) param8(p.gamma, p.gamma_bf16, j, n, gm);
      else take_gamma<AL>(rg[j], p.gamma_bf16, n, gm);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[j][i] = held<AL>(n, xh[j][i] * now.r2);
        // (an unaligned row past the end holds the last one's values)
        sum2(j, i) += AL || n > 0 ? g[j][i] * xh[j][i] : 0.0f;
        g[j][i] *= gm[i];
        dot += counted<AL>(i, n, g[j][i] * xh[j][i]);
      }
    }
    if constexpr (kLean) load_second(row, now);
    const float mean2 = row_sum<TPR>(dot, reinterpret_cast<float*>(red)) / (float)C;
    // dh in place of g, the branch's xh in place of the stream's
    const float at1 = p.alpha * now.t;
    dot = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int n = live ? count(j) : 0;
      float dr[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (p.dres) {
        take8<HBF, AL>(now.dr[j], n, dr);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        g[j][i] = held<AL>(n, now.r2 * (g[j][i] - xh[j][i] * mean2) + dr[i]);
      if (n > 0) store_own<HBF, AL>(p.dh, row * p.lddh + at(j), n, g[j]);
      take8<XBF, AL>(now.x[j], n, xh[j]);
      float kj[8];
      if constexpr (kLean) {
        param8(p.post_gamma, p.post_gamma_bf16, j, n, kj);
#pragma unroll
        for (int i = 0; i < 8; ++i) kj[i] *= p.alpha;
        if (p.gate) {
          float gt[8];
          param8(p.gate, p.gate_bf16, j, n, gt);
#pragma unroll
          for (int i = 0; i < 8; ++i) kj[i] *= gt[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) kj[i] = k[j][i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[j][i] = held<AL>(n, xh[j][i] * now.r1);
        sum1(j, i) += AL || n > 0 ? (at1 * g[j][i]) * xh[j][i] : 0.0f;
        g[j][i] *= kj[i];
        dot += counted<AL>(i, n, g[j][i] * xh[j][i]);
      }
    }
    dot = row_sum<TPR>(dot, reinterpret_cast<float*>(red));
    if (p.drow_gate && live && t == 0) p.drow_gate[row] = dot;
    const float mean1 = dot / (float)C, rt = now.r1 * now.t;
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int n = live ? count(j) : 0;
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[j][i] = rt * (g[j][i] - xh[j][i] * mean1);
        most = max(most, counted_bits<AL>(i, n, g[j][i]));
      }
      mine = max(mine, n > 0 ? most : 0u);
      if (p.dx && n > 0) store_own<XBF, AL>(p.dx, row * p.lddx + at(j), n, g[j]);
    }
    if (p.q) {
      amax = max(amax, mine);
      u32x2 c[VPT];
      cast_row<VPT, AL>(g, s, e5m2, mine, live, count, c, sat, p.sat != nullptr);
#pragma unroll
      for (int j = 0; j < VPT; ++j)
        if (live && count(j) > 0) store_own_codes<AL>(p.q + row * p.ldq + at(j), count(j), c[j]);
    }
    if constexpr (kAhead) now = next;
  }
  // partial rows: the slots of a workgroup one after the other
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    auto acc = [&](int j, int i) { return which ? sum1(j, i) : sum2(j, i); };
    float* out = p.work + ((int64_t)which * gridDim.x + blockIdx.x) * C;
    if constexpr (RPB > 1) {
      for (int w = 0; w < RPB; ++w) {
        if (slot == w) {
#pragma unroll
          for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float* d = &part_lds[(j * 8 + i) * TPR + t];
              *d = w == 0 ? acc(j, i) : *d + acc(j, i);
            }
        }
        __syncthreads();
      }
      if (slot == 0) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i >= 8 - count(j)) out[at(j) + i] = part_lds[(j * 8 + i) * TPR + t];
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i >= 8 - count(j)) out[at(j) + i] = acc(j, i);
    }
  }
  if (p.q) commit(amax, sat, p.amax, p.sat, red);
}

// Rows longer than the registers: one workgroup walks its rows, each read three times (dh may be
// dres, so dh is stored only in the last pass, where nothing reads dres again).
template <bool XBF, bool HBF>
__global__ __launch_bounds__(1024) void sandwich_bwd_long_kernel(SandwichBwdArgs p) {
  __shared__ uint32_t red[2 * 16];
  const int t = threadIdx.x;
  const int64_t C = p.cols;
  const bool e5m2 = p.fmt == kE5M2;
  float s = 1.0f;
  if (p.q) {
    s = *p.scale_in;
    if (p.scale_used && blockIdx.x == 0 && t == 0) *p.scale_used = s;
  }
  float* out2 = p.work + (int64_t)blockIdx.x * C;
  float* out1 = p.work + ((int64_t)gridDim.x + blockIdx.x) * C;
  uint32_t amax = 0, sat = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const bool first = row == (int64_t)blockIdx.x;
    const float r1 = p.post_rstd[row], r2 = p.rstd[row], tok = p.row_gate ? p.row_gate[row] : 1.0f;
    double sum = 0.0;
    for (int64_t c = t; c < C; c += 1024) {
      const float xh = load1<HBF>(p.h, row * p.ldh + c) * r2, dy = load1<XBF>(p.dy, row * p.lddy + c);
      sum += (double)(dy * gamma1(p.gamma, p.gamma_bf16, c) * xh);
      out2[c] = dy * xh + (first ? 0.0f : out2[c]);
    }
    const float mean2 = row_sum<1024>((float)sum, reinterpret_cast<float*>(red)) / (float)C;
    auto dh_of = [&](int64_t c) {
      const float xh = load1<HBF>(p.h, row * p.ldh + c) * r2;
      const float g = load1<XBF>(p.dy, row * p.lddy + c) * gamma1(p.gamma, p.gamma_bf16, c);
      const float d = r2 * (g - xh * mean2);
      return p.dres ? d + load1<HBF>(p.dres, row * p.lddr + c) : d;
    };
    sum = 0.0;
    for (int64_t c = t; c < C; c += 1024) {
      const float dh = dh_of(c), xh = load1<XBF>(p.x, row * p.ldx + c) * r1;
      sum += (double)(dh * k1(p, c) * xh);
      out1[c] = (p.alpha * tok * dh) * xh + (first ? 0.0f : out1[c]);
    }
    const float dot = row_sum<1024>((float)sum, reinterpret_cast<float*>(red));
    if (p.drow_gate && t == 0) p.drow_gate[row] = dot;
    const float mean1 = dot / (float)C;
    for (int64_t c = t; c < C; c += 1024) {
      const float dh = dh_of(c), xh = load1<XBF>(p.x, row * p.ldx + c) * r1;
      const float d = (r1 * tok) * (dh * k1(p, c) - xh * mean1);
      store1<HBF>(p.dh, row * p.lddh + c, dh);
      if (p.dx) store1<XBF>(p.dx, row * p.lddx + c, d);
      if (p.q) {
        amax = max(amax, abs_bits(d));
        p.q[row * p.ldq + c] = (uint8_t)code1(d * s, e5m2);
        if (p.sat) sat += sat1(d * s, e5m2);
      }
    }
  }
  if (p.q) commit(amax, sat, p.amax, p.sat, red);
}

// The two column sums over `parts` partial rows: 32 columns x 16 shares of the rows per
// workgroup, joined in LDS in a fixed order; columns from c0 on, blockIdx.y the sum.
__global__ __launch_bounds__(512) void sandwich_join_kernel(SandwichBwdArgs p, int parts, int64_t c0) {
  __shared__ float part[16][33];
  const int cl = threadIdx.x & 31, sh = threadIdx.x >> 5;
  const int64_t c = c0 + (int64_t)blockIdx.x * 32 + cl, C = p.cols;
  const float* work = p.work + (int64_t)blockIdx.y * parts * C;
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
    if (blockIdx.y == 0) {
      p.dgamma[c] = t;
    } else {
      p.dpost_gamma[c] = p.gate ? t * gamma1(p.gate, p.gate_bf16, c) : t;
      if (p.dgate) p.dgate[c] = t * gamma1(p.post_gamma, p.post_gamma_bf16, c);
    }
  }
}

// ------------------------------------------------------------------ host launchers

template <bool XBF, bool HBF, int MODE, bool AL>
static hipError_t launch_fwd(const SandwichArgs& a, RowShape sh, int num_cus, hipStream_t stream) {
#define FP8DS_NORM_CASE(T, V)                                                                    \
  if (sh.tpr == T && sh.vpt == V) {                                                              \
    const int64_t rpb = T > 256 ? 1 : 256 / T, blocks = (a.rows + rpb - 1) / rpb;                \
    const int64_t most = (int64_t)num_cus * (T > 256 ? 1 : 8);                                   \
    hipLaunchKernelGGL((sandwich_fwd_kernel<XBF, HBF, T, V, MODE, AL>),                          \
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
  constexpr int64_t kSlice = 1 << 21;  // rows; 2^31 threads, of fewer than 2^32 in a grid
  for (int64_t r0 = 0; r0 < a.rows; r0 += kSlice) {
    const int64_t n = a.rows - r0 < kSlice ? a.rows - r0 : kSlice;
    hipLaunchKernelGGL((sandwich_fwd_long_kernel<XBF, HBF, MODE>), dim3((unsigned)n), dim3(1024), 0,
                       stream, a, r0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool XBF, bool HBF>
static hipError_t launch_fwd_t(const SandwichArgs& a, RowShape sh, int n, hipStream_t s) {
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

hipError_t launch_sandwich_fwd(const SandwichArgs& a, int num_cus, hipStream_t stream) {
  const RowShape sh = row_shape(a.cols);
  if (a.x_bf16 && a.h_bf16) return launch_fwd_t<true, true>(a, sh, num_cus, stream);
  if (a.x_bf16) return launch_fwd_t<true, false>(a, sh, num_cus, stream);
  return launch_fwd_t<false, false>(a, sh, num_cus, stream);
}

static RowShape bwd_shape(int64_t cols) {
  const int64_t g = (cols + 7) / 8;
  if (cols < 8) return {1024, 0};
  if (g <= 1024) return row_shape(cols);
  if (g <= 2048) return {1024, 2};
  return {1024, 0};
}

// Workgroups of the backward pass: at most 1024, so that the partial sums stay a small part of
// the traffic.
int sandwich_bwd_parts(int64_t rows, int64_t cols) {
  const RowShape sh = bwd_shape(cols);
  const int64_t rpb = sh.tpr > 256 ? 1 : 256 / sh.tpr;
  const int64_t blocks = (rows + rpb - 1) / rpb;
  return (int)(blocks < 1024 ? blocks : 1024);
}

template <bool XBF, bool HBF, bool AL>
static hipError_t launch_bwd(const SandwichBwdArgs& a, RowShape sh, int parts, hipStream_t stream) {
#define FP8DS_NORM_CASE(T, V)                                                                     \
  if (sh.tpr == T && sh.vpt == V) {                                                               \
    hipLaunchKernelGGL((sandwich_bwd_kernel<XBF, HBF, T, V, AL>), dim3((unsigned)parts),         \
                       dim3(T > 256 ? T : 256), 0, stream, a);                                    \
    return hipGetLastError();                                                                     \
  }
  FP8DS_NORM_CASE(16, 1)
  FP8DS_NORM_CASE(64, 1)
  FP8DS_NORM_CASE(64, 2)
  FP8DS_NORM_CASE(256, 1)
  FP8DS_NORM_CASE(256, 2)
  FP8DS_NORM_CASE(256, 4)
  FP8DS_NORM_CASE(1024, 2)
#undef FP8DS_NORM_CASE
  hipLaunchKernelGGL((sandwich_bwd_long_kernel<XBF, HBF>), dim3((unsigned)parts), dim3(1024), 0,
                     stream, a);
  return hipGetLastError();
}

hipError_t launch_sandwich_bwd(const SandwichBwdArgs& a, hipStream_t stream) {
  const RowShape sh = bwd_shape(a.cols);
  const int parts = sandwich_bwd_parts(a.rows, a.cols);
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
  constexpr int64_t kSlice = 1 << 26;  // columns; two sums of 2^30 threads, of fewer than 2^32
  for (int64_t c0 = 0; c0 < a.cols; c0 += kSlice) {
    const int64_t n = a.cols - c0 < kSlice ? a.cols - c0 : kSlice;
    hipLaunchKernelGGL(sandwich_join_kernel, dim3((unsigned)((n + 31) / 32), 2), dim3(512), 0, stream,
                       a, parts, c0);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp8ds
