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
//
// An FP8 A has two datapaths.  That instruction adds the products of an FP8 operand in
// groups of 8 at a fixed point 13 bits below the group's largest (FP4 x FP4 products have too
// few bits to lose any there).  EXACT, the default, widens both operands to BF16 times
// their block's scale instead and multiplies those, v_mfma_f32_{16x16x32,32x32x16}_bf16:
// exact products (4 and 2 significant bits), FP32 sums.  A lane then holds one whole block
// of A too.
//
// BF16 has the exponents of fp32, so the widened value is exact but where it leaves the normal
// range: an element of A below 2^-126 (scale codes up to 9 for E4M3, 16 for E5M2) keeps
// what bits of it are left there, one of 2^128 or more (codes from 247 and 240, of B from 253)
// is infinite.  The conversions take the scale code itself as an exponent; 255 gives NaN.

#include "cast_common.h"
#include "fp4_common.h"
#include "gemm_kernel.h"
#include "launch.h"

namespace fp8ds {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// matrix-instruction code of an element format
template <int F>
constexpr int kMfmaFormat = F == kE4M3 ? 0 : F == kE5M2 ? 1 : 4;

template <int FA, int OP>
__device__ __forceinline__ f32x4 mfma_a_fp4(const i32x8& a, const i32x8& b, const f32x4& c, int sa,
                                            int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, kMfmaFormat<FA>, 4, OP, sa, OP,
                                                          sb);
}

// Byte u of a dword of scale codes as the conversions take it.
__device__ __forceinline__ float code_scale(int codes, int u) {
  return __uint_as_float(((uint32_t)codes >> (8 * u) & 255u) << 23);
}
// Eight elements as BF16 times the scale: of FP8 in two dwords, of FP4 in one.
template <int F>
__device__ __forceinline__ v8bf widen_fp8(int lo, int hi, float x) {
  const u32x4 d = {widen_pair_mx<F>(lo, false, x), widen_pair_mx<F>(lo, true, x),
                   widen_pair_mx<F>(hi, false, x), widen_pair_mx<F>(hi, true, x)};
  return __builtin_bit_cast(v8bf, d);
}
__device__ __forceinline__ v8bf widen_fp4(int c, float x) {
  const u32x4 d = {
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)c, x, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)c, x, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)c, x, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4((uint32_t)c, x, 3))};
  return __builtin_bit_cast(v8bf, d);
}

// ------------------------------------------------------------------ few rows

// 512 elements of K of one lane's row of an operand, for four MFMA steps.  Step u takes, in
// lane group g, block 4 g + u, so that a lane's elements are 64 consecutive bytes (FP4)
// and its codes one dword, of which the instruction picks byte u.
struct Span {
  i32x8 v[4];
  int s;
};
constexpr int kSpan = 512;

template <int F, bool EXACT>
struct RowPtr {
  const uint8_t *p, *sc;
  __device__ __forceinline__ RowPtr(const uint8_t* base, int64_t ld, const uint8_t* codes,
                                    int64_t ldc, int64_t row, int64_t rows) {
    // rows past the end read the last one: what they give is not stored
    row = row < rows ? row : rows - 1;
    p = base + row * (F == kE2M1 ? ld / 2 : ld);
    sc = codes + row * ldc;
  }
  // The span at k (a multiple of 512).  Blocks past the end of K: the row's start is read
  // in their place and the code is 0; zeros for an FP8 operand (a NaN element would
  // survive the code; the products of two FP4 elements at 2^-254 vanish).
  __device__ __forceinline__ void load(Span& d, int64_t k, int64_t K, int g) const {
    const int64_t b = k / 32 + 4 * g, nblk = K / 32;
    if (b + 4 <= nblk) {
      __builtin_memcpy(&d.s, sc + b, 4);  // rows of codes may start anywhere
    } else {
      d.s = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (b + u < nblk) d.s |= (int)sc[b + u] << (8 * u);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if constexpr (F == kE2M1) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(p + (b + u < nblk ? (b + u) * 16 : 0));
        d.v[u] = i32x8{(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
      } else {
        // EXACT: the group's own block; else half g % 2 of those of lane groups g / 2 and 2 + g / 2
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t c = EXACT ? b + u : k / 32 + 4 * (2 * h + (g >> 1)) + u;
          const u32x4 x = *reinterpret_cast<const u32x4*>(p + (c < nblk ? c * 32 : 0) +
                                                          16 * (EXACT ? h : g & 1));
#pragma unroll
          for (int i = 0; i < 4; ++i) d.v[u][4 * h + i] = c < nblk ? (int)x[i] : 0;
        }
      }
    }
  }
};

// A workgroup of KW waves makes 16 MT x 16 NT outputs; the waves share K, a span each at a
// time, straight from memory to registers, and their sums are joined in LDS in a fixed
// order.  A wave has the loads of its next span in flight while it multiplies: with few
// rows the product is the reading of B, (1/2 + 1/32) byte per weight.  Measured: 1 token x
// 14336 x 4096 8.4 us, 3.7 TB/s of B; with B from HBM each time and an FP8 A 10.6 us on the
// FP8 datapath and 11.5 on the exact one, whose conversions (8 to 16 for one to four matrix
// instructions) come on top.  What is over the copy's 6.1 us is the launch, the first loads'
// latency and the join: with 4 waves a K of 4096 is two spans for each.
template <int FA, bool EXACT, int MT, int NT, int KW>
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
  int64_t k = (int64_t)kSpan * w;
  if (k < p.K) {
    struct Operands {
      Span a[MT], b[NT];
    };
    Operands now;
    auto load = [&](int64_t at, Operands& x) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
        RowPtr<kE2M1, false>(p.B, p.ldb, p.sc_b, p.ldsb, n0 + 16 * j + r, p.N).load(x.b[j], at, p.K, g);
#pragma unroll
      for (int i = 0; i < MT; ++i)
        RowPtr<FA, EXACT>(p.A, p.lda, p.sc_a, p.ldsa, m0 + 16 * i + r, p.M).load(x.a[i], at, p.K, g);
    };
    auto mfmas = [&](auto step) {
      constexpr int u = decltype(step)::value;
      if constexpr (EXACT) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // 8 elements of each block
          v8bf wa[MT], wb[NT];
#pragma unroll
          for (int i = 0; i < MT; ++i)
            wa[i] = widen_fp8<FA>(now.a[i].v[u][2 * q], now.a[i].v[u][2 * q + 1],
                                  code_scale(now.a[i].s, u));
#pragma unroll
          for (int j = 0; j < NT; ++j) wb[j] = widen_fp4(now.b[j].v[u][q], code_scale(now.b[j].s, u));
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wa[i], wb[j], acc[i][j], 0, 0, 0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            acc[i][j] =
                mfma_a_fp4<FA, u>(now.a[i].v[u], now.b[j].v[u], acc[i][j], now.a[i].s, now.b[j].s);
      }
    };
    load(k, now);
    while (true) {
      k += kSpan * KW;
      const bool more = k < p.K;
      Operands next;
      if (more) load(k, next);
      mfmas(std::integral_constant<int, 0>{});
      mfmas(std::integral_constant<int, 1>{});
      mfmas(std::integral_constant<int, 2>{});
      mfmas(std::integral_constant<int, 3>{});
      if (!more) break;
      now = next;
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[w][16 * i + 4 * g + e][16 * j + r] = acc[i][j][e];
  __syncthreads();
  uint32_t amax = 0;
#pragma unroll 1
  for (int u = threadIdx.x; u < BM * BN; u += 64 * KW) {
    const int m = u / BN, n = u % BN;
    float v = 0.0f;
#pragma unroll
    for (int x = 0; x < KW; ++x) v += part[x][m][n];
    if (m0 + m < p.M && n0 + n < p.N) {
      const int64_t at = (m0 + m) * p.ldc + n0 + n;
      if (p.out_bf16) {
        const uint16_t c = bf16_bits_rne(v);
        static_cast<uint16_t*>(p.C)[at] = c;
        amax = max(amax, (uint32_t)(c & 0x7FFFu) << 16);
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

// ------------------------------------------------------------------ tiles through LDS

// A workgroup of GM x GN waves makes a BM x BN tile of C; a wave owns
// (BM / GM) x (BN / GN) of it as 32 x 32 blocks of v_mfma_scale_f32_32x32x64_f8f6f4.  The
// operands reach LDS by loads straight into it, a stage of K at a time: rows of 128 bytes
// (64 for the FP4 operand beside an FP8 one) whose 16-byte chunks are permuted by the row
// against bank conflicts, and each row's E8M0 codes.  K may be walked in any order as long
// as both operands agree: MFMA step s of a stage takes, in lane half h, block steps h + s,
// so that a half's codes lie next to each other and the instruction picks byte s.
//
// Stages: 256 elements of K and two buffers for FP4 x FP4, 128 elements and three for
// FP8 x FP4, which is what 160 KB of LDS hold of a 256 x 256 tile in rows of 128 bytes.
// Four buffers of 128 elements (rows of 64 bytes) for FP4 x FP4 have longer to arrive, but
// L2 serves rows of 64 bytes at half the rate of 128: 132 us became 164 at
// 4096 x 4096 x 16384.  Two buffers for FP8 x FP4: 416 us instead of 395 at
// 8192 x 14336 x 4096.
//
// Measured with random codes (FP4 x FP4, M x N x K): 4096 x 4096 x 16384 123 us = 4.5 PFLOP/s,
// 8192 x 14336 x 4096 239 us = 4.0, 16384 x 4096 x 4096 143 us = 3.8; FP8 x FP4
// 8192 x 14336 x 4096 348 us = 2.8 on the FP8 datapath, 675 us = 1.4 on the exact one, whose
// BF16 instructions have half the FP8 rate and share their issue with 24 conversions for 8 of
// them.  These are times in a loop that has run for some 200 launches; before that power
// control lowers the clock for a while, and the same calls take up to a fifth longer.  The
// comparisons in this file are of loops of 24 to 60 launches, both sides alike.  The instruction
// alone, fed from registers with random codes, reaches 6.6 (4.2 for FP8 x FP8).  The matrix
// unit is busy 65, 47 and 56% of the time (4096 x 4096 x 16384, 16384 x 4096 x 4096,
// 8192 x 14336 x 4096).  What holds it up: LDS, of whose time a step of
// MFMAs (512 cycles of a SIMD) takes 384 for fragment reads and 128 for the next stage's
// arrival; and at K = 4096 the start and end of each tile, 5 to 9 us a round of tiles, of
// which the stores of C are 1.5 to 3.5.  Waves of 128 x 128 outputs (4 a workgroup) read
// 2/3 of the fragments and were no faster; nor did a higher wave priority around the MFMAs help.
template <int FA>
struct Stage {
  static constexpr int K = FA == kE2M1 ? 256 : 128;
  static constexpr int kSteps = K / 64;
  static constexpr int kBuffers = FA == kE2M1 ? 2 : 3;
  static constexpr int kRowA = 128;  // bytes of a row of A
  static constexpr int kRowB = K / 2;
};

// LDS byte offset of 16-byte chunk c of row r, for rows of RB bytes.  A fragment read
// serves 16 consecutive rows at a time from the 16 16-byte columns of LDS; the chunks are
// permuted by the row so that those 16 pieces lie in 16 columns (two rows of 128 bytes, or
// four of 64, share the columns).
template <int RB>
__device__ __forceinline__ int chunk_off(int r, int c) {
  if constexpr (RB == 128) return r * 128 + ((c ^ ((r >> 1) & 7)) << 4);
  else return r * 64 + ((c ^ ((r >> 2) & 3)) << 4);
}

__device__ __forceinline__ void load_to_lds16(__amdgpu_buffer_rsrc_t rsrc, uint8_t* lds, int voff,
                                              int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      rsrc, (void __attribute__((address_space(3)))*)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void load_to_lds4(__amdgpu_buffer_rsrc_t rsrc, uint8_t* lds, int voff,
                                             int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      rsrc, (void __attribute__((address_space(3)))*)lds, 4, voff, soff, 0, 0);
}
// An offset past every buffer: such a load gives zeros and does not reach memory.
constexpr int kNowhere = 0x40000000;

// This wave's share of the loads of one operand tile (ROWS rows of RB bytes a stage).
template <int ROWS, int RB, int NW>
struct TileLoader {
  static constexpr int kRowsPer = 1024 / RB;  // rows per load instruction of a wave
  static constexpr int kPerWave = ROWS / kRowsPer / NW;
  static_assert(RB != 128 || kPerWave % 2 == 0, "a wave's first rows start a group of 16");
  __amdgpu_buffer_rsrc_t rsrc;
  int ld, w, row_off, col;

  __device__ __forceinline__ TileLoader(const uint8_t* src, int64_t ld_, int64_t row0, int64_t rows,
                                        int64_t row_bytes, int tid) {
    const int lane = tid & 63;
    ld = (int)ld_;
    w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the lane's place in the 1 KB that an instruction fills, and the chunk that belongs there
    const int row = lane / (RB / 16), place = lane % (RB / 16);
    col = (RB == 128 ? place ^ (row >> 1) : place ^ (row >> 2)) * 16;
    row_off = row * ld;
    const int64_t left = rows - row0 < ROWS ? rows - row0 : ROWS;
    rsrc = byte_rsrc(src + row0 * ld_, (left - 1) * ld_ + row_bytes);
  }

  // Bytes [k0, k0 + RB) of every row; what lies at or past row_bytes reads as zeros, and
  // so do rows past the matrix.
  __device__ __forceinline__ void issue(int k0, int row_bytes, uint8_t* lds) const {
    // rows 8 .. 15 of every 16 rows of 128 bytes have the other half of the permutations
    const int even = k0 + col < row_bytes ? row_off + col : kNowhere;
    const int odd = k0 + (col ^ 64) < row_bytes ? row_off + (col ^ 64) : kNowhere;
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int seg = w * kPerWave + i;
      load_to_lds16(rsrc, lds + seg * 1024, RB == 128 && (i & 1) ? odd : even,
                    seg * kRowsPer * ld + k0);
    }
  }
};

// The E8M0 codes of a tile's rows (A's, then B's) by loads straight into LDS.  L2 answers
// a load of 4 bytes per row with as many requests as one of 64, and the tile kernels come
// near its request rate: read by every lane for its own rows and stage, the codes took 20%
// of the kernel at 4096 x 4096 x 16384, loaded as dwords for every stage 4%.
//
// !WIDE: rows of codes that start at dwords and K a multiple of 128 of at least 512.  A load takes 16
// codes of a row, which serve the kBuffers stages of one turn of the loop.
// WIDE: rows of codes that start anywhere, any K.  The dwords that hold a row's codes of a
// stage, one load each: plane d has dword d of every row, and a shift brings the codes
// down.  The outer bytes of those dwords may belong to the neighbouring rows, or to
// nothing: they share a dword with a code of this row, so they can be read, and they are
// not used.
template <int BM, int BN, int NW, int STEPS, bool WIDE>
struct CodeLoader {
  static constexpr int kPlane = (BM + BN) * 4;
  static constexpr int kDwords = STEPS / 2 + 1;           // WIDE: per stage
  static constexpr int kBytes = WIDE ? kDwords * kPlane : (BM + BN) * 16;
  static constexpr int kPerWave = (BM + BN) / (64 * NW);  // groups of 64 rows per wave
  static constexpr int kLoads = kPerWave * (WIDE ? kDwords : 1);
  __amdgpu_buffer_rsrc_t ra, rb;
  int lda, ldb, w, lane, mis_a, mis_b, nblk;

  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const uint8_t* sc, int64_t ld,
                                                                int64_t row0, int64_t rows,
                                                                int64_t most, int nblk, int& mis) {
    const uint8_t* p = sc + row0 * ld;
    mis = WIDE ? (int)(reinterpret_cast<uintptr_t>(p) & 3u) : 0;
    const int64_t left = rows - row0 < most ? rows - row0 : most;
    return byte_rsrc(p - mis, ((left - 1) * ld + nblk + mis + 3) & ~int64_t(3));
  }
  __device__ __forceinline__ CodeLoader(const Mxfp4Gemm& p, int64_t m0, int64_t n0, int tid) {
    lda = (int)p.ldsa;
    ldb = (int)p.ldsb;
    lane = tid & 63;
    w = __builtin_amdgcn_readfirstlane(tid >> 6);
    nblk = (int)(p.K / 32);
    ra = rsrc(p.sc_a, p.ldsa, m0, p.M, BM, nblk, mis_a);
    rb = rsrc(p.sc_b, p.ldsb, n0, p.N, BN, nblk, mis_b);
  }
  // !WIDE: the first block of the load that serves the stages from k on (in the row still)
  __device__ __forceinline__ int first(int k) const { return min(2 * STEPS * k, nblk - 16); }

  // the codes of stage k (WIDE) or of the stages from k on
  __device__ __forceinline__ void issue(int k, uint8_t* lds) const {
#pragma unroll
    for (int x = 0; x < kPerWave; ++x) {
      constexpr int kSegA = BM / 64;
      const int seg = NW * x + w;
      const bool of_a = kSegA % NW == 0 ? x < kSegA / NW : seg < kSegA;
      const int ld = of_a ? lda : ldb, row = (of_a ? seg : seg - kSegA) * 64;
      if constexpr (!WIDE) {
        load_to_lds16(of_a ? ra : rb, lds + seg * 1024, lane * ld, row * ld + first(k));
      } else {
        const int at = ((row + lane) * ld + (of_a ? mis_a : mis_b)) & ~3;
        const int to = 2 * STEPS * k < nblk ? at : kNowhere;
#pragma unroll
        for (int d = 0; d < kDwords; ++d)
          load_to_lds4(of_a ? ra : rb, lds + d * kPlane + seg * 256, to, 2 * STEPS * k + 4 * d);
      }
    }
  }
  // Codes of half h of row i of the tile (A's rows, then B's), byte s for step s.  `off`
  // (!WIDE): the half's first block of the stage less first(); `shift` (WIDE): 8 times the
  // place of the row's first code in its dword.
  static __device__ __forceinline__ uint32_t read(const uint8_t* lds, int i, int h, int off,
                                                  uint32_t shift) {
    if constexpr (WIDE) {
      const uint8_t* q = lds + i * 4 + (STEPS == 4 ? h * kPlane : 0);
      const uint32_t lo = *reinterpret_cast<const uint32_t*>(q);
      const uint32_t hi = *reinterpret_cast<const uint32_t*>(q + kPlane);
      return (uint32_t)((((uint64_t)hi << 32) | lo) >> (shift + (STEPS == 4 ? 0 : 16 * h)));
    } else if constexpr (STEPS == 4) {
      return *reinterpret_cast<const uint32_t*>(lds + i * 16 + off);
    } else {
      return *reinterpret_cast<const uint16_t*>(lds + i * 16 + off);
    }
  }
};

// Barrier of a stage: every wave's reads of LDS are done, and all but its last N loads.
// (__syncthreads would wait for all loads.)  The fences order this thread's accesses for
// the compiler and wait for nothing.
template <int N>
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  // vmcnt N, lgkmcnt 0, expcnt unconstrained
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The order of a step: DS fragment reads and VM loads spread over its MF MFMAs, the reads
// over the first three quarters so that the last of them has arrived for the next step.
template <int MF, int DS, int VM, int I = 0>
__device__ __forceinline__ void interleave() {
  if constexpr (I < MF) {
    constexpr int kSpan = MF * 3 / 4;
    constexpr int d0 = I < kSpan ? DS * I / kSpan : DS, d1 = I + 1 < kSpan ? DS * (I + 1) / kSpan : DS;
    constexpr int v0 = VM * I / MF, v1 = VM * (I + 1) / MF;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                              // MFMA
    if constexpr (d1 > d0) __builtin_amdgcn_sched_group_barrier(0x100, d1 - d0, 0);  // LDS read
    if constexpr (v1 > v0) __builtin_amdgcn_sched_group_barrier(0x020, v1 - v0, 0);  // VMEM read
    interleave<MF, DS, VM, I + 1>();
  }
}

template <int FA, int OP>
__device__ __forceinline__ v16f mfma_tile(const v8i& b, const v8i& a, const v16f& c, int sb, int sa) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, c, 4, kMfmaFormat<FA>, OP, sb, OP, sa);
}

// Tile of workgroup wg.  XCD x = wg % 8 takes a contiguous share of the tiles, which are
// numbered down groups of ROWS tile rows, so that the tiles an XCD works on at a time are
// near a square: 4 x 8 of the 32 of 256 x 256 (8 x 4: 258 us instead of 254 at
// 8192 x 14336 x 4096, 172 instead of 168 at 16384 x 4096 x 4096; 2 x 16: 258 and 171),
// 8 x 8 of the 64 of 128 x 128 (4 x 16: 47 us instead of 44 at 1000 x 14336 x 4096).
template <int ROWS>
__device__ __forceinline__ void tile_of(int wg, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int total = tiles_m * tiles_n, x = wg & 7;
  const int i = total < 8 ? wg : x * (total >> 3) + min(x, total & 7) + (wg >> 3);
  const int first = i / (ROWS * tiles_n) * ROWS, rows = min(tiles_m - first, ROWS);
  const int j = i - first * tiles_n;
  tm = first + j % rows;
  tn = j / rows;
}

// The stages are variables of their own, and the loop names them: the compiler then knows
// that a fragment read does not touch a buffer being loaded, and does not wait for the
// loads in flight before each of them.
template <int FA, bool EXACT, int BM, int BN, int GM, int GN, bool WIDE>
__global__ __launch_bounds__(64 * GM * GN, 2) void gemm_mxfp4_tile_kernel(Mxfp4Gemm p, int tiles_m,
                                                                         int tiles_n) {
  using S = Stage<FA>;
  constexpr int NW = GM * GN, WM = BM / GM, WN = BN / GN, MI = WM / 32, NI = WN / 32;
  constexpr int NS = S::kSteps, NBUF = S::kBuffers, RA = S::kRowA, RB = S::kRowB;
  using Codes = CodeLoader<BM, BN, NW, NS, WIDE>;
  constexpr int kA = BM * RA, kB = BN * RB, kStage = kA + kB + (WIDE ? Codes::kBytes : 0);
  // the BF16 tile on its way out takes the stages' place, kOutWaves waves to each
  constexpr int kOutWaves = (NW + NBUF - 1) / NBUF, kOut = kOutWaves * WM * WN * 2;
  constexpr int kBuf = kStage > kOut ? kStage : kOut;
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[kBuf];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[kBuf];
  __shared__ __attribute__((aligned(1024))) uint8_t lds2[NBUF == 3 ? kBuf : 16];
  __shared__ __attribute__((aligned(16))) uint8_t codes[WIDE ? 16 : Codes::kBytes];
  __shared__ uint32_t red[2 * NW];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int r = lane & 31, h = lane >> 5;
  const int wm = (w / GN) * WM, wn = (w % GN) * WN;
  int tm, tn;
  tile_of<BM == 256 ? 4 : 8>(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int row_a = (int)(FA == kE2M1 ? p.K / 2 : p.K), row_b = (int)(p.K / 2);
  const int nblk = (int)(p.K / 32);
  const TileLoader<BM, RA, NW> la(p.A, FA == kE2M1 ? p.lda / 2 : p.lda, m0, p.M, row_a, tid);
  const TileLoader<BN, RB, NW> lb(p.B, p.ldb / 2, n0, p.N, row_b, tid);
  const Codes lc(p, m0, n0, tid);
  // this lane's fragment chunks in a row of LDS
  int oa[FA == kE2M1 ? NS : 2 * NS], ob[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    if constexpr (FA == kE2M1) {
      oa[s] = chunk_off<RA>(r, NS * h + s);
    } else if constexpr (EXACT) {  // a lane holds its half's block, in two chunks
      oa[s] = chunk_off<RA>(r, 2 * (NS * h + s));
      oa[NS + s] = chunk_off<RA>(r, 2 * (NS * h + s) + 1);
    } else {  // a lane holds half h of the blocks of both lane halves: s and NS + s
      oa[s] = chunk_off<RA>(r, 2 * s + h);
      oa[NS + s] = chunk_off<RA>(r, 2 * (NS + s) + h);
    }
    ob[s] = chunk_off<RB>(r, NS * h + s);
  }
  uint32_t sha[MI], shb[NI];  // WIDE: the shift of each row's codes
#pragma unroll
  for (int i = 0; i < MI; ++i)
    sha[i] = WIDE ? 8u * (((wm + 32 * i + r) * lc.lda + lc.mis_a) & 3) : 0u;
#pragma unroll
  for (int j = 0; j < NI; ++j)
    shb[j] = WIDE ? 8u * (((wn + 32 * j + r) * lc.ldb + lc.mis_b) & 3) : 0u;
  v16f acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  const int nst = (int)((p.K + S::K - 1) / S::K);
  int sa[MI], sb[NI];
  uint32_t pa_next[MI], pb_next[NI];  // codes read a stage ahead
  v8i fa[2][MI], fb[2][NI];
  // the loads of stage k (zeros for k >= nst)
  auto issue = [&](int k, uint8_t* dst) {
    la.issue(k * RA, row_a, dst);
    lb.issue(k * RB, row_b, dst + kA);
    if constexpr (WIDE) lc.issue(k, dst + kA + kB);
  };
  constexpr int kLoads = la.kPerWave + lb.kPerWave + (WIDE ? lc.kLoads : 0);
  // Codes of stage k for this lane's rows and half, out of the load for the stages from k0
  // on.  Blocks past the end of K take code 0: their elements are zeros, and a zero times
  // any power of two is zero, while the byte there may be the code of NaN.
  auto read_codes = [&](int k, int k0, const uint8_t* src, uint32_t (&ca)[MI], uint32_t (&cb)[NI]) {
    const int block = 2 * NS * k + NS * h, left = nblk - block;
    const uint32_t mask = left >= NS ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
    const int off = WIDE ? 0 : min(block - lc.first(k0), 16 - NS);
#pragma unroll
    for (int i = 0; i < MI; ++i) ca[i] = Codes::read(src, wm + 32 * i + r, h, off, sha[i]) & mask;
#pragma unroll
    for (int j = 0; j < NI; ++j) cb[j] = Codes::read(src, BM + wn + 32 * j + r, h, off, shb[j]) & mask;
  };
  // fragments of step s of the stage in `src`, into register set s & 1
  auto frags = [&](const uint8_t* src, auto step) {
    constexpr int s = decltype(step)::value;
    const uint8_t *pa = src + wm * RA, *pb = src + kA + wn * RB;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const u32x4 d = *reinterpret_cast<const u32x4*>(pa + oa[s] + 32 * i * RA);
      fa[s & 1][i] = v8i{(int)d[0], (int)d[1], (int)d[2], (int)d[3], 0, 0, 0, 0};
      if constexpr (FA != kE2M1) {
        const u32x4 e = *reinterpret_cast<const u32x4*>(pa + oa[NS + s] + 32 * i * RA);
#pragma unroll
        for (int x = 0; x < 4; ++x) fa[s & 1][i][4 + x] = (int)e[x];
      }
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const u32x4 d = *reinterpret_cast<const u32x4*>(pb + ob[s] + 32 * j * RB);
      fb[s & 1][j] = v8i{(int)d[0], (int)d[1], (int)d[2], (int)d[3], 0, 0, 0, 0};
    }
  };
  auto mfmas = [&](auto step) {
    constexpr int s = decltype(step)::value;
    if constexpr (EXACT) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // 8 elements of each block
        v8bf wa[MI], wb[NI];
#pragma unroll
        for (int i = 0; i < MI; ++i)
          wa[i] = widen_fp8<FA>(fa[s & 1][i][2 * q], fa[s & 1][i][2 * q + 1], code_scale(sa[i], s));
#pragma unroll
        for (int j = 0; j < NI; ++j) wb[j] = widen_fp4(fb[s & 1][j][q], code_scale(sb[j], s));
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NI; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j], wa[i], acc[i][j], 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
          acc[i][j] = mfma_tile<FA, s>(fb[s & 1][j], fa[s & 1][i], acc[i][j], sb[j], sa[i]);
    }
  };
  using std::integral_constant;
  // Stage k, from its barrier on, as number G of a turn of the loop.  The fragments of a
  // step are read while the step before it is multiplied, so the previous stage's last step
  // comes first here; and the loads of stage k + NBUF - 1 start beside it, into the buffer
  // that this barrier freed.  !WIDE: the turn's last stage has had its codes read by the
  // one before it, and loads the next turn's into their place.
  auto stage = [&](int k, const uint8_t* rd, uint8_t* wr, auto number) {
    constexpr int G = decltype(number)::value;
    constexpr bool kLast = !WIDE && G == NBUF - 1, kAhead = !WIDE && G == NBUF - 2;
    stage_barrier<(NBUF - 2) * kLoads>();  // all but the loads of later stages have arrived
    uint32_t ca[MI], cb[NI];
    if constexpr (kLast) {
#pragma unroll
      for (int i = 0; i < MI; ++i) ca[i] = pa_next[i];
#pragma unroll
      for (int j = 0; j < NI; ++j) cb[j] = pb_next[j];
      lc.issue(k + 1, codes);
      // no load may pass them: the next barrier counts on the codes being the older ones
      __builtin_amdgcn_sched_barrier(0x78F);
    } else {
      read_codes(k, k - G, WIDE ? rd + kA + kB : codes, ca, cb);
      if constexpr (kAhead) read_codes(k + 1, k - G, codes, pa_next, pb_next);
    }
    frags(rd, integral_constant<int, 0>{});
    issue(k + NBUF - 1, wr);
    mfmas(integral_constant<int, NS - 1>{});
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = (int)ca[i];
#pragma unroll
    for (int j = 0; j < NI; ++j) sb[j] = (int)cb[j];
    frags(rd, integral_constant<int, 1>{});
    mfmas(integral_constant<int, 0>{});
    if constexpr (NS == 4) {
      frags(rd, integral_constant<int, 2>{});
      mfmas(integral_constant<int, 1>{});
      frags(rd, integral_constant<int, 3>{});
      mfmas(integral_constant<int, 2>{});
    }
    // issue order: fragment reads and loads between the MFMAs that hide them
    constexpr int kReads = MI * (FA == kE2M1 ? 1 : 2) + NI, kMf = MI * NI * (EXACT ? 4 : 1);
    constexpr int kCodeReads = (MI + NI) * (WIDE ? 2 : kLast ? 0 : kAhead ? 2 : 1);
    interleave<kMf, kReads + kCodeReads, kLoads>();
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) interleave<kMf, kReads, 0>();
  };
  if (nst > 0) {
    // "the last step of the stage before the first": zeros
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      sa[i] = 127;
      fa[1][i] = v8i{0, 0, 0, 0, 0, 0, 0, 0};
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      sb[j] = 127;
      fb[1][j] = v8i{0, 0, 0, 0, 0, 0, 0, 0};
    }
    // Stages go NBUF at a time.  Of two, an odd one comes first and by itself (a loop that
    // can end between them was compiled to copies of the accumulators); of three, the last
    // turn is filled up with stages of zeros.  The loads past the last stage are issued too:
    // they give zeros and do not reach memory.
    constexpr integral_constant<int, 0> k0th{};
    constexpr integral_constant<int, 1> k1st{};
    int k = 0;
    if constexpr (!WIDE) lc.issue(0, codes);
    if constexpr (NBUF == 2) {
      if (nst & 1) {
        issue(0, lds1);
        if constexpr (!WIDE) {
          stage_barrier<0>();
          read_codes(0, 0, codes, pa_next, pb_next);
        }
        stage(0, lds1, lds0, k1st);
        k = 1;
      } else {
        issue(0, lds0);
      }
      for (; k < nst; k += 2) {
        stage(k, lds0, lds1, k0th);
        stage(k + 1, lds1, lds0, k1st);
      }
    } else {
      issue(0, lds0);
      issue(1, lds1);
      for (; k < nst; k += 3) {
        stage(k, lds0, lds2, k0th);
        stage(k + 1, lds1, lds0, k1st);
        stage(k + 2, lds2, lds1, integral_constant<int, 2>{});
      }
    }
    mfmas(integral_constant<int, NS - 1>{});
  }

  // Epilogue.  Lane (r, h) holds, of block (i, j), row r and columns 8 q + 4 h + {0..3} in
  // elements 4 q .. 4 q + 3.  BF16: each wave parks its rows in LDS (16-byte chunks
  // permuted by the row) and writes whole row runs; FP32: 16-byte pieces.
  uint32_t amax = 0;
  const int64_t cm = m0 + wm, cn = n0 + wn;
  if (p.out_bf16) {
    vmem_wait_all();
    __syncthreads();  // the stages in LDS are done with
    const int part = w / kOutWaves;
    uint8_t* out = (part == 0 ? lds0 : part == 1 ? lds1 : lds2) + w % kOutWaves * (WM * WN * 2);
    constexpr int CH = WN / 8;  // 16-byte chunks per row
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const u32x2 d = {bf16_pair_rne(acc[i][j][4 * q], acc[i][j][4 * q + 1]),
                           bf16_pair_rne(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3])};
          const int row = 32 * i + r, c = 4 * j + q;
          *reinterpret_cast<u32x2*>(out + row * (WN * 2) + ((c ^ (row & (CH - 1))) << 4) + 8 * h) = d;
        }
    __builtin_amdgcn_wave_barrier();
    uint16_t* C = static_cast<uint16_t*>(p.C);
    const bool wide = ((reinterpret_cast<uintptr_t>(C) | (uint64_t)(p.ldc * 2)) & 15u) == 0;
    constexpr int RPI = 64 / CH;  // rows per wave instruction
#pragma unroll 4
    for (int it = 0; it < WM / RPI; ++it) {
      const int row = it * RPI + lane / CH, c = lane % CH;
      const u32x4 d = *reinterpret_cast<const u32x4*>(out + row * (WN * 2) + ((c ^ (row & (CH - 1))) << 4));
      const int64_t m = cm + row, n = cn + 8 * c;
      if (m >= p.M || n >= p.N) continue;
      if (wide && n + 8 <= p.N) {
        __builtin_nontemporal_store(d, reinterpret_cast<u32x4*>(C + m * p.ldc + n));
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = max(amax, max((d[e] & 0x7FFFu) << 16, d[e] & 0x7FFF0000u));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (n + e >= p.N) continue;
          const uint32_t v = (d[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
          C[m * p.ldc + n + e] = (uint16_t)v;
          amax = max(amax, (v & 0x7FFFu) << 16);
        }
      }
    }
  } else {
    float* C = static_cast<float*>(p.C);
    const bool wide = ((reinterpret_cast<uintptr_t>(C) | (uint64_t)(p.ldc * 4)) & 15u) == 0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int64_t m = cm + 32 * i + r;
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t n = cn + 32 * j + 8 * q + 4 * h;
          if (m >= p.M || n >= p.N) continue;
          u32x4 d;
#pragma unroll
          for (int e = 0; e < 4; ++e) d[e] = __float_as_uint(acc[i][j][4 * q + e]);
          if (wide && n + 4 <= p.N) {
            __builtin_nontemporal_store(d, reinterpret_cast<u32x4*>(C + m * p.ldc + n));
#pragma unroll
            for (int e = 0; e < 4; ++e) amax = max(amax, d[e] & 0x7FFFFFFFu);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (n + e >= p.N) continue;
              C[m * p.ldc + n + e] = __uint_as_float(d[e]);
              amax = max(amax, d[e] & 0x7FFFFFFFu);
            }
          }
        }
    }
  }
  if (p.amax_c) {
    Health hh;
    block_commit<false>(amax, 0u, hh, reinterpret_cast<uint32_t*>(p.amax_c), nullptr, nullptr, red);
  }
}

// ------------------------------------------------------------------ host launcher

template <int FA, bool EXACT, int MT, int NT, int KW>
static hipError_t launch_direct(const Mxfp4Gemm& p, hipStream_t stream) {
  // A grid holds fewer than 2^32 threads along x; of a larger one HIP drops the excess without
  // an error.  2^27 columns are at most 2^27 / 16 workgroups of 512 (KW = 8) threads.
  constexpr int64_t kSlice = 1 << 27;
  for (int64_t n0 = 0; n0 < p.N; n0 += kSlice) {
    Mxfp4Gemm s = p;
    s.N = p.N - n0 < kSlice ? p.N - n0 : kSlice;
    s.B = p.B + n0 * (p.ldb / 2);
    s.sc_b = p.sc_b + n0 * p.ldsb;
    s.C = static_cast<char*>(p.C) + n0 * (p.out_bf16 ? 2 : 4);
    const dim3 grid((unsigned)((s.N + 16 * NT - 1) / (16 * NT)),
                    (unsigned)((s.M + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL((gemm_mxfp4_direct_kernel<FA, EXACT, MT, NT, KW>), grid, dim3(64 * KW), 0,
                       stream, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int FA, bool EXACT, int BM, int BN, int GM, int GN, bool WIDE>
static hipError_t launch_tile(const Mxfp4Gemm& p, hipStream_t stream) {
  const int tm = (int)((p.M + BM - 1) / BM), tn = (int)((p.N + BN - 1) / BN);
  hipLaunchKernelGGL((gemm_mxfp4_tile_kernel<FA, EXACT, BM, BN, GM, GN, WIDE>), dim3((unsigned)(tm * tn)),
                     dim3(64 * GM * GN), 0, stream, p, tm, tn);
  return hipGetLastError();
}

// Which kernel (times in us, one MI355X, FP4 x FP4 unless stated; "FP8 datapath" and
// "exact" are those of an FP8 A):
//  - up to 16 rows, direct: 16 x 16 outputs and 8 waves, or 16 x 32 and 4 waves where those
//    still give every CU a workgroup: 1 x 14336 x 4096 8.7 and 8.4 (FP8 datapath 11.6 and
//    9.3), 13 x 4096 x 14336 9.9 and 14.8;
//  - few outputs, direct with 32 x 32: up to one workgroup per CU (64 x 4096 x 4096: 6.9, on
//    128 x 128 tiles 13.2), with 8 waves, or 4 for an FP8 A, whose operands would spill; up
//    to two per CU with 4 waves for an FP4 A (32 x 14336 x 4096: 12.6, tiles 14.2) and on the
//    exact datapath (32 x 14336 x 4096: 23.8, tiles 27.9; 128 x 4096 x 14336: 55, tiles 80),
//    not on the FP8 datapath (18.5, tiles 16);
//  - 256 x 256 tiles where they give every CU one, else 128 x 128 (8192 x 1024 x 4096: 24,
//    on 256 x 256 tiles 33; 4096 x 4096 x 4128 on the FP8 datapath: 90, on 128 x 128 tiles 122;
//    8192 x 14336 x 4096 exact: 692, on 128 x 128 tiles 769).
template <int FA, bool EXACT>
static hipError_t launch_fa(const Mxfp4Gemm& p, int num_cus, hipStream_t stream) {
  if (p.M <= 16) {
    if ((p.N + 31) / 32 >= num_cus) return launch_direct<FA, EXACT, 1, 2, 4>(p, stream);
    return launch_direct<FA, EXACT, 1, 1, 8>(p, stream);
  }
  const int64_t small = ((p.M + 31) / 32) * ((p.N + 31) / 32);
  if constexpr (FA == kE2M1) {
    if (small <= num_cus) return launch_direct<FA, EXACT, 2, 2, 8>(p, stream);
  }
  // the tile loads address their rows with 30 bits
  const int64_t most = 1 << 21;
  if (p.lda >= most || p.ldb >= most || p.ldsa >= most || p.ldsb >= most ||
      small <= (FA == kE2M1 || EXACT ? 2 : 1) * num_cus)
    return launch_direct<FA, EXACT, 2, 2, 4>(p, stream);
  // where a load may take 16 codes of a row at a dword address (CodeLoader)
  const bool wide = p.K < 512 || ((reinterpret_cast<uintptr_t>(p.sc_a) | (uint64_t)p.ldsa |
                                   reinterpret_cast<uintptr_t>(p.sc_b) | (uint64_t)p.ldsb |
                                   (uint64_t)(p.K / 32)) & 3u) != 0;
  const int64_t big = ((p.M + 255) / 256) * ((p.N + 255) / 256);
  if (big >= num_cus)
    return wide ? launch_tile<FA, EXACT, 256, 256, 4, 2, true>(p, stream)
                : launch_tile<FA, EXACT, 256, 256, 4, 2, false>(p, stream);
  return wide ? launch_tile<FA, EXACT, 128, 128, 2, 2, true>(p, stream)
              : launch_tile<FA, EXACT, 128, 128, 2, 2, false>(p, stream);
}

hipError_t launch_gemm_mxfp4(const Mxfp4Gemm& p, int fa, bool exact, int num_cus,
                             hipStream_t stream) {
  switch (fa) {
    case kE4M3: return exact ? launch_fa<kE4M3, true>(p, num_cus, stream)
                             : launch_fa<kE4M3, false>(p, num_cus, stream);
    case kE5M2: return exact ? launch_fa<kE5M2, true>(p, num_cus, stream)
                             : launch_fa<kE5M2, false>(p, num_cus, stream);
    default: return launch_fa<kE2M1, false>(p, num_cus, stream);
  }
}

}  // namespace fp8ds
