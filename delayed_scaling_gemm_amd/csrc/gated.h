// The elementwise part of a gated feed-forward block, in the epilogues of its two products
// (included by gemm_kernel.h).
//
//   forward   g = acc_g d, u = acc_u d,  a = act(g) u          A = X, B = [W_gate; W_up]
//   backward  da = acc d,  dg = da u act'(g),  du = da act(g)  A = dY, B = W_down, g and u stored
//
// both activations being g times a sigmoid: SiLU g s(g); GELU (tanh form) g s(2 z) with
// z = sqrt(2 / pi) (g + 0.044715 g^3), since (1 + tanh z) / 2 = s(2 z).  With p the sigmoid and
// z' the derivative of its argument, act' = p + g p (1 - p) z'.  All of it in fp32 from the fp32
// sums; g and u are rounded to BF16 where they are kept for the backward pass, which reads
// them so: 2^-9 of each, against gradients that are rounded to 8 bits after it.
#pragma once

namespace fp8ds {

constexpr int kActSilu = 0, kActGelu = 1;

// Both sigmoids' argument is g (k1 + k3 g^2), k3 = 0 for SiLU: no branch on the activation.  e1 and e3
// are -k1 and -k3 over ln 2.
struct Act {
  float k1, k33, e1, e3;
  __device__ __forceinline__ explicit Act(int act) {
    constexpr float kL = 1.4426950408889634f;
    constexpr float kG = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    k1 = act == kActGelu ? kG : 1.0f;
    k33 = act == kActGelu ? 3.0f * 0.044715f * kG : 0.0f;
    e1 = act == kActGelu ? -kG * kL : -kL;
    e3 = act == kActGelu ? -0.044715f * kG * kL : 0.0f;
  }
};
struct ActValue {
  float a, d;  // act(g), act'(g)
};
// exp2 and the reciprocal are the hardware's, 1 ulp each: relative errors of a few 2^-24 (2^-24 |g|
// where the sigmoid is small), far below the 8 or 16 bits that the result is rounded to.  g^2 is
// kept finite, so that k3 = 0 and a sigmoid of 0 make zeros of it; NaN stays NaN.
template <bool GRAD>
__device__ __forceinline__ ActValue act_value(float g, const Act& c) {
  const float g2 = fminf(g * g, 1e37f);
  const float e = __builtin_amdgcn_exp2f(g * __builtin_fmaf(c.e3, g2, c.e1));
  const float p = __builtin_amdgcn_rcpf(1.0f + e);
  ActValue v;
  v.a = g * p;
  if constexpr (GRAD) {
    const float t = __builtin_fmaf(-p, p, p);
    v.d = __builtin_fmaf(g * t, __builtin_fmaf(c.k33, g2, c.k1), p);
  }
  return v;
}

// Eight elements of a row in memory: vectors, of unaligned type where rows are not at 16 bytes.  Of a
// ragged row's end n < 8: stored one by one, but read as the row's last eight and shifted down (`whole`: it
// has that many), since the wave waits for loads under a branch one after the other (300 x 1037 x 528
// backward: 25.7 us, so 21.1).
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

template <bool AL>
__device__ __forceinline__ u32x4 gated_load8(const uint16_t* p, int n, bool whole) {
  if constexpr (AL) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  u32x4 v = {0u, 0u, 0u, 0u};
  if (whole) {
    v = *reinterpret_cast<const u32x4_a2*>(p + (n - 8));
    const int by = 8 - n;
    if (by & 4) v = u32x4{v[2], v[3], 0u, 0u};
    if (by & 2) v = u32x4{v[1], v[2], v[3], 0u};
    if (by & 1)
      v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
  } else {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < n) v[k >> 1] |= (uint32_t)p[k] << (16 * (k & 1));
  }
  return v;
}
template <bool AL>
__device__ __forceinline__ void gated_store16(uint16_t* p, int n, const float (&v)[8]) {
  const u32x4 d = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7])};
  if constexpr (AL) {
    __builtin_nontemporal_store(d, reinterpret_cast<u32x4*>(p));
  } else if (n >= 8) {
    *reinterpret_cast<u32x4_a2*>(p) = d;
  } else {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < n) p[k] = (uint16_t)(d[k >> 1] >> (16 * (k & 1)));
  }
}
template <bool AL>
__device__ __forceinline__ void gated_store32(float* p, int n, const float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    if constexpr (AL) {
      *reinterpret_cast<f32x4_t*>(p + k) = f32x4_t{v[k], v[k + 1], v[k + 2], v[k + 3]};
    } else {
#pragma unroll
      for (int j = k; j < k + 4; ++j)
        if (j < n) p[j] = v[j];
    }
  }
}
template <bool AL>
__device__ __forceinline__ void gated_store8(uint8_t* p, int n, const u32x2& c) {
  if constexpr (AL) {
    __builtin_nontemporal_store(c, reinterpret_cast<u32x2*>(p));
  } else if (n >= 8) {
    *reinterpret_cast<u32x2_a1*>(p) = c;
  } else {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < n) p[k] = (uint8_t)(c[k >> 2] >> (8 * (k & 3)));
  }
}

// Eight codes of v s (the converts round as the definition does inside the format's range, which the
// clamp makes of every value but NaN; `nan`: some value of the eight may be one).
__device__ __forceinline__ u32x2 gated_codes(const float (&v)[8], float s, bool e5m2, bool nan,
                                             uint32_t& sat, bool want) {
  const float top = e5m2 ? FmtTraits<kE5M2>::kMax : FmtTraits<kE4M3>::kMax;
  float t[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    t[k] = v[k] * s;
    if (want) sat += (uint32_t)(fabsf(t[k]) > top);
    t[k] = __builtin_amdgcn_fmed3f(t[k], -top, top);
  }
  int w[2] = {0, 0};
  if (e5m2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = __builtin_amdgcn_cvt_pk_bf8_f32(t[4 * h], t[4 * h + 1], w[h], false);
      w[h] = __builtin_amdgcn_cvt_pk_bf8_f32(t[4 * h + 2], t[4 * h + 3], w[h], true);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * h], t[4 * h + 1], w[h], false);
      w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * h + 2], t[4 * h + 3], w[h], true);
    }
  }
  u32x2 c = {(uint32_t)w[0], (uint32_t)w[1]};
  if (nan) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = __float_as_uint(v[k]), at = 8 * (k & 3);
      if ((b & 0x7FFFFFFFu) > 0x7F800000u)
        c[k >> 2] = (c[k >> 2] & ~(0xFFu << at)) | ((0x7Fu | ((b >> 24) & 0x80u)) << at);
    }
  }
  return c;
}

// Barriers that a gated epilogue executes.
__device__ __forceinline__ int gated_barriers(const GatedArgs& p) {
  return 1 + (p.amax || p.sat ? 1 : 0);
}

// Lane l holds, for each 32 x 32 block (i, j), row l % 32 and the columns 8 g + 4 (l / 32) + {0..3},
// g = 0 .. 3.  Forward: blocks j and j + FN / 2 are gate and up of the same columns.
//
// A wave passes its sums, 32 rows at a time, through a part of the operand tiles' LDS of its own
// (in fp32, chunk c of 16 bytes of row r at c ^ (r % 8)) and takes them back with eight
// consecutive columns of a row in a lane: every access to memory is then 8 or 16 bytes of a run
// of a row, the elementwise work is written once, and the sums, which fill half of the
// registers, are only ever indexed by constants.
template <bool BWD, int BM, int BNO, int FM, int FN, int WTM, int WTN>
__device__ __forceinline__ void gated_epilogue(const GatedArgs& p, const v16f (&acc)[FM][FN],
                                               int64_t m0, int64_t n0, int wm, int wn, int tid, float d,
                                               uint32_t* red, uint8_t* stage0, uint8_t* stage1) {
  constexpr int WTO = BWD ? WTN : WTN / 2;  // output columns of a wave
  constexpr int NO = BWD ? 2 : 1;           // values per output place
  constexpr int UPR = WTO / 8;              // lanes of a row
  constexpr int RPT = 64 / UPR;             // rows of a turn
  constexpr int NT = 32 / RPT < 4 ? 32 / RPT : 4;  // turns taken together
  constexpr int NG = 32 / RPT / NT;         // such groups of turns in 32 rows
  const int lane = tid & 63, wave = tid >> 6;
  const int64_t M = p.M, F = p.N;
  const int64_t mw = m0 + wm * WTM, nw = n0 + wn * WTO;  // the wave's block
  const bool e5m2 = p.fmt == kE5M2;
  const float s = p.q ? *p.scale : 1.0f;
  if (p.scale_used && blockIdx.x == 0 && tid == 0) *p.scale_used = s;
  float top = 0.0f;
  uint32_t amax = 0, sat = 0;
  const Act act(p.act);
  const bool want_sat = p.sat != nullptr;
  // two buffers of 32 rows, used in turn
  uint8_t* st = (wave < 2 ? stage0 : stage1) + (wave & 1) * (BM * kRowBytes);
  static_assert(2 * 32 * WTN * 4 <= BM * kRowBytes && WTM * 2 == BM && WTN * 2 <= BM,
                "two buffers in a wave's part, half of an operand's two stages");
  __syncthreads();  // every wave has finished reading the operand tiles

  const int ur = lane / UPR, uc = (lane % UPR) * 8;  // of a turn: this lane's row and first column
  const int64_t n = nw + uc;
  const int left = F - n >= 8 ? 8 : (int)(F - n);
  auto rows = [&](auto al_tag) {
    constexpr bool AL = decltype(al_tag)::value;
    u32x4 pre[NT][2];  // backward: g and u of the group to come
    auto load_pre = [&](int group) {
      if constexpr (BWD) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int64_t m = mw + (group * NT + t) * RPT + ur;
          if (m < M && m < mw + WTM && left > 0) {
            const uint16_t* r = p.gu + m * p.ldgu + n;
            pre[t][0] = gated_load8<AL>(r, left, F >= 8);
            pre[t][1] = gated_load8<AL>(r + F, left, F >= 8);
          }
        }
      }
    };
    load_pre(0);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      uint8_t* buf = st + (i & 1) * (32 * WTN * 4);
      {
        const int r = lane & 31;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int c = 8 * j + 2 * g + (lane >> 5);
            *reinterpret_cast<f32x4_t*>(buf + r * (WTN * 4) + ((c ^ (r & 7)) << 4)) =
                f32x4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
          }
      }
      // lanes of this wave read what others of it wrote
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll 1  // (code size: unrolled, the loop over i would not be)
      for (int o = 0; o < NG; ++o) {
      u32x4 now[NT][2];
      if constexpr (BWD) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) now[t][h] = pre[t][h];
        load_pre(i * NG + o + 1);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = (o * NT + t) * RPT + ur;
        const int64_t m = mw + i * 32 + r;
        auto take = [&](int col, float (&v)[8]) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = col / 4 + h;
            const f32x4_t x =
                *reinterpret_cast<const f32x4_t*>(buf + r * (WTN * 4) + ((c ^ (r & 7)) << 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * h + k] = x[k] * d;
          }
        };
        float out[NO][8];
        if constexpr (!BWD) {
          float g[8], u[8];
          take(uc, g);
          take(WTO + uc, u);
#pragma unroll
          for (int k = 0; k < 8; ++k) out[0][k] = act_value<false>(g[k], act).a * u[k];
          if (m >= M || left <= 0) continue;
          if (p.gu) {
            gated_store16<AL>(p.gu + m * p.ldgu + n, left, g);
            gated_store16<AL>(p.gu + m * p.ldgu + F + n, left, u);
          }
        } else {
          float da[8];
          take(uc, da);
          if (m >= M || left <= 0) continue;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float g = k & 1 ? bf16_hi(now[t][0][k >> 1]) : bf16_lo(now[t][0][k >> 1]);
            const float u = k & 1 ? bf16_hi(now[t][1][k >> 1]) : bf16_lo(now[t][1][k >> 1]);
            const ActValue a = act_value<true>(g, act);
            out[0][k] = da[k] * u * a.d;
            out[1][k] = da[k] * a.a;
          }
        }
#pragma unroll
        for (int h = 0; h < NO; ++h) {
          // the largest magnitude as a float, which passes over NaN; 0 times a value that is not
          // finite tells of one
          float odd = 0.0f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (!AL && k >= left) out[h][k] = 0.0f;
            odd = __builtin_fmaf(out[h][k], 0.0f, odd);
            top = fmaxf(top, fabsf(out[h][k]));
          }
          if (odd != 0.0f) {
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = max(amax, __float_as_uint(out[h][k]) & 0x7FFFFFFFu);
          }
          if (p.q) {
            const u32x2 c = gated_codes(out[h], s, e5m2, odd != 0.0f, sat, want_sat);
            gated_store8<AL>(p.q + m * p.ldq + n + h * F, left, c);
          }
          if (p.y) {
            const int64_t at = m * p.ldy + n + h * F;
            if (p.y_f32) gated_store32<AL>(static_cast<float*>(p.y) + at, left, out[h]);
            else gated_store16<AL>(static_cast<uint16_t*>(p.y) + at, left, out[h]);
          }
        }
      }
      }
    }
  };
  // (256 x 256 tiles are launched for aligned rows only: with both, the compiler gives up unrolling)
  if (BM == 256 || p.vec) rows(std::true_type{});
  else if constexpr (BM < 256) rows(std::false_type{});

  if (p.amax || p.sat) {  // four waves: one word each
    amax = wave_max_u32(max(amax, __float_as_uint(top)));
    if (lane == 0) red[wave] = amax;
    if (p.sat && __any(sat != 0)) {
      sat = wave_sum_u32(sat);
      if (lane == 0) atomicAdd(p.sat, (unsigned long long)sat);
    }
    __syncthreads();
    if (tid == 0 && p.amax) {
      const uint32_t m = canonical_amax_bits(max(max(red[0], red[1]), max(red[2], red[3])));
      if (m > __hip_atomic_load(p.amax, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(p.amax, m);
    }
  }
}

}  // namespace fp8ds
