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
#include "gemm_kernel.h"
#include "launch.h"

namespace fp8ds {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// matrix-instruction code of an element format
template <int F>
constexpr int kMfmaFormat = F == kE4M3 ? 0 : F == kE5M2 ? 1 : 4;

template <int FA>
__device__ __forceinline__ f32x4 mfma_a_fp4(const i32x8& a, const i32x8& b, const f32x4& c, int sa,
                                            int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, kMfmaFormat<FA>, 4, 0, sa, 0,
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

// ------------------------------------------------------------------ tiles through LDS

// A workgroup of GM x GN waves makes a BM x BN tile of C; a wave owns
// (BM / GM) x (BN / GN) of it as 32 x 32 blocks of v_mfma_scale_f32_32x32x64_f8f6f4.  The
// operands reach LDS by loads straight into it, two stages of KST elements of K deep,
// in rows of 128 bytes (64 for the FP4 operand beside an FP8 one) whose 16-byte
// chunks are permuted by the row, so that consecutive lanes of a fragment read fall in
// different banks.  K may be walked in any order as long as both operands agree: MFMA
// step s of a stage takes, in lane half h, block (KST / 64) h + s, so that the E8M0 codes
// of all of a half's steps lie next to each other, and one 4-byte load per 32 rows and
// stage serves them; the instruction picks byte s.
template <int FA>
struct TileShape {
  static constexpr int KST = FA == kE2M1 ? 256 : 128;  // elements of K per stage
  static constexpr int NS = KST / 64;                  // MFMA steps per stage
  static constexpr int RA = 128;                       // bytes per LDS row of A
  static constexpr int RB = KST / 2;                   // bytes per LDS row of B
};

// LDS byte offset of 16-byte chunk c of row r, for rows of RB bytes.  The permutation
// depends on the row modulo 8 only: rows 32 apart are a constant apart, and the loads'
// rows (8 or 16 per instruction) all have the same lane pattern.
template <int RB>
__device__ __forceinline__ int chunk_off(int r, int c) {
  if constexpr (RB == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  else return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// This wave's share of the loads of one operand tile (ROWS rows of RB bytes).
template <int ROWS, int RB, int NW>
struct TileLoader {
  static constexpr int kRowsPer = 1024 / RB;  // rows per load instruction of a wave
  static constexpr int kPerWave = ROWS / kRowsPer / NW;
  __amdgpu_buffer_rsrc_t rsrc;
  int ld, w, col, voff;

  __device__ __forceinline__ TileLoader(const uint8_t* src, int64_t ld_, int64_t row0, int64_t rows,
                                        int64_t row_bytes, int tid) {
    const int lane = tid & 63;
    ld = (int)ld_;
    w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the lane's place in the 1 KB that an instruction fills, and the chunk that belongs there
    const int row = lane / (RB / 16), place = lane % (RB / 16);
    col = (RB == 128 ? place ^ (row & 7) : place ^ ((row >> 1) & 3)) * 16;
    voff = row * ld + col;
    const int64_t left = rows - row0 < ROWS ? rows - row0 : ROWS;
    rsrc = byte_rsrc(src + row0 * ld_, (left - 1) * ld_ + row_bytes);
  }

  // Bytes [k0, k0 + RB) of every row; what lies at or past row_bytes reads as zeros.
  __device__ __forceinline__ void issue(int k0, int row_bytes, uint8_t* lds) const {
    const int v = k0 + col < row_bytes ? voff : 0x40000000;
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int seg = w * kPerWave + i;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (void __attribute__((address_space(3)))*)(lds + seg * 1024), 16, v,
          seg * kRowsPer * ld + k0, 0, 0);
    }
  }
};

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

// E8M0 codes of a tile's rows, 16 blocks of each at a time, by loads straight into LDS
// (16 bytes per row: row i of A, then of B).  Read from memory by every lane for its own
// rows and stage, they cost as many cache lines as the elements themselves: half the
// kernel's time at 4096 x 4096 x 16384.
template <int FA, int BM, int BN, int NW>
struct ScaleTiles {
  static constexpr int NS = TileShape<FA>::NS;
  static constexpr int kStages = 16 / (2 * NS);      // stages served by a load
  static constexpr int kBytes = (BM + BN) * 16;
  static constexpr int kPerWave = (BM + BN) / (64 * NW);

  // The first block of group g's load: the last group stays inside the row.
  static __device__ __forceinline__ int first(int g, int nblk) { return min(16 * g, nblk - 16); }

  static __device__ __forceinline__ void issue(__amdgpu_buffer_rsrc_t ca, __amdgpu_buffer_rsrc_t cb,
                                               int lda, int ldb, int g, int nblk, int w, int lane,
                                               uint8_t* dst) {
    const int wv = __builtin_amdgcn_readfirstlane(w), f = first(g, nblk);
    // 64 rows per instruction, no branch
#pragma unroll
    for (int x = 0; x < kPerWave; ++x) {
      constexpr int kSegA = BM / 64;
      const int seg = NW * x + wv;
      const bool of_a = kSegA % NW == 0 ? x < kSegA / NW : seg < kSegA;
      const int ld = of_a ? lda : ldb, row = (of_a ? seg : seg - kSegA) * 64;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          of_a ? ca : cb, (void __attribute__((address_space(3)))*)(dst + seg * 1024), 16, lane * ld,
          row * ld + f, 0, 0);
    }
  }
};

// The codes of a tile's rows: reads outside them give 0.
template <int ROWS>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scale_rsrc(const uint8_t* sc, int64_t ld,
                                                             int64_t row0, int64_t rows, int nblk) {
  const int64_t left = rows - row0 < ROWS ? rows - row0 : ROWS;
  return byte_rsrc(sc + row0 * ld, (left - 1) * ld + nblk);
}

template <int FA, int BM, int BN, int GM, int GN>
__global__ __launch_bounds__(64 * GM * GN, 2) void gemm_mxfp4_tile_kernel(Mxfp4Gemm p, int tiles_m,
                                                                         int tiles_n) {
  using S = TileShape<FA>;
  constexpr int NS = S::NS, NW = GM * GN, WM = BM / GM, WN = BN / GN, MI = WM / 32, NI = WN / 32;
  using SC = ScaleTiles<FA, BM, BN, NW>;
  constexpr int kA = BM * S::RA, kB = BN * S::RB, kStage = kA + kB + SC::kBytes;
  constexpr int kOut = BM * BN;  // half of the BF16 tile on its way out
  // The two stages are two variables, and the loop below names them: the compiler then
  // knows that a fragment read does not touch the buffer being loaded, and does not wait
  // for the loads in flight before each of them.
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[kStage > kOut ? kStage : kOut];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[kStage > kOut ? kStage : kOut];
  __shared__ uint32_t red[2 * NW];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int r = lane & 31, h = lane >> 5;
  const int wm = (w / GN) * WM, wn = (w % GN) * WN;
  int tm, tn;
  tile_coords(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int row_a = (int)(FA == kE2M1 ? p.K / 2 : p.K), row_b = (int)(p.K / 2);
  const TileLoader<BM, S::RA, NW> la(p.A, FA == kE2M1 ? p.lda / 2 : p.lda, m0, p.M, row_a, tid);
  const TileLoader<BN, S::RB, NW> lb(p.B, p.ldb / 2, n0, p.N, row_b, tid);
  const int nblk = (int)(p.K / 32);
  const __amdgpu_buffer_rsrc_t ca = scale_rsrc<BM>(p.sc_a, p.ldsa, m0, p.M, nblk);
  const __amdgpu_buffer_rsrc_t cb = scale_rsrc<BN>(p.sc_b, p.ldsb, n0, p.N, nblk);
  // this lane's fragment chunks in a row of LDS, one per load of a stage
  int oa[S::RA == 128 && FA != kE2M1 ? 2 * NS : NS], ob[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    if constexpr (FA == kE2M1) {
      oa[s] = chunk_off<S::RA>(r, NS * h + s);
    } else {  // a lane holds half h of the blocks of both lane halves: s and NS + s
      oa[s] = chunk_off<S::RA>(r, 2 * s + h);
      oa[NS + s] = chunk_off<S::RA>(r, 2 * (NS + s) + h);
    }
    ob[s] = chunk_off<S::RB>(r, NS * h + s);
  }
  v16f acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  const int nst = (int)((p.K + S::KST - 1) / S::KST);
  int sa[MI], sb[NI];
  v8i fa[2][MI], fb[2][NI];
  // the loads of stage k: elements of A, of B, codes of both
  auto issue = [&](int k, uint8_t* dst) {
    la.issue(k * S::RA, row_a, dst);
    lb.issue(k * S::RB, row_b, dst + kA);
    SC::issue(ca, cb, (int)p.ldsa, (int)p.ldsb, k / SC::kStages, nblk, w, lane, dst + kA + kB);
  };
  // fragments of step s of the stage in `src`, into register set s & 1
  auto frags = [&](const uint8_t* src, auto step) {
    constexpr int s = decltype(step)::value;
    const uint8_t *pa = src + wm * S::RA, *pb = src + kA + wn * S::RB;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const u32x4 d = *reinterpret_cast<const u32x4*>(pa + oa[s] + 32 * i * S::RA);
      fa[s & 1][i] = v8i{(int)d[0], (int)d[1], (int)d[2], (int)d[3], 0, 0, 0, 0};
      if constexpr (FA != kE2M1) {
        const u32x4 e = *reinterpret_cast<const u32x4*>(pa + oa[NS + s] + 32 * i * S::RA);
#pragma unroll
        for (int x = 0; x < 4; ++x) fa[s & 1][i][4 + x] = (int)e[x];
      }
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const u32x4 d = *reinterpret_cast<const u32x4*>(pb + ob[s] + 32 * j * S::RB);
      fb[s & 1][j] = v8i{(int)d[0], (int)d[1], (int)d[2], (int)d[3], 0, 0, 0, 0};
    }
  };
  auto mfmas = [&](auto step) {
    constexpr int s = decltype(step)::value;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
        acc[i][j] = mfma_tile<FA, s>(fb[s & 1][j], fa[s & 1][i], acc[i][j], sb[j], sa[i]);
  };
  using std::integral_constant;
  // One stage, from its barrier on.  The fragments of a step are read while the step
  // before it is multiplied, so the previous stage's last step comes first here, and the
  // loads of the next stage start beside it, into the buffer that this barrier freed.
  auto stage = [&](int k, const uint8_t* rd, uint8_t* wr) {
    // the codes of this lane's rows and half, byte s for step s; blocks past the end of K
    // take code 0 (their elements are zeros), and so do rows past the edge
    const int off = k * (2 * NS) + NS * h - SC::first(k / SC::kStages, nblk);
    const bool in = off <= 16 - NS;
    const uint8_t* src = rd + kA + kB + r * 16 + (in ? off : 0);
    int na[MI], nb[NI];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const uint8_t* q = src + (wm + 32 * i) * 16;
      na[i] = NS == 4 ? *reinterpret_cast<const int*>(q) : *reinterpret_cast<const uint16_t*>(q);
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const uint8_t* q = src + (BM + wn + 32 * j) * 16;
      nb[j] = NS == 4 ? *reinterpret_cast<const int*>(q) : *reinterpret_cast<const uint16_t*>(q);
    }
    frags(rd, integral_constant<int, 0>{});
    issue(k + 1, wr);
    mfmas(integral_constant<int, NS - 1>{});
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = in ? na[i] : 0;
#pragma unroll
    for (int j = 0; j < NI; ++j) sb[j] = in ? nb[j] : 0;
    frags(rd, integral_constant<int, 1>{});
    mfmas(integral_constant<int, 0>{});
    if constexpr (NS == 4) {
      frags(rd, integral_constant<int, 2>{});
      mfmas(integral_constant<int, 1>{});
      frags(rd, integral_constant<int, 3>{});
      mfmas(integral_constant<int, 2>{});
    }
    // issue order: fragment reads and loads between the MFMAs that hide them
    constexpr int kReads = MI * (FA == kE2M1 ? 1 : 2) + NI, kMf = MI * NI;
    interleave<kMf, kReads + MI + NI, la.kPerWave + lb.kPerWave + SC::kPerWave>();
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) interleave<kMf, kReads, 0>();
  };
  // this wave's loads have arrived, then everyone's
  auto arrived = [] {
    vmem_wait_all();
    __syncthreads();
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
    // Stages go in pairs, an odd first one by itself.  The last one's loads are issued
    // too (what lies past K reads as zeros without reaching memory): a loop that leaves
    // them out, or that can end between the two stages, was compiled to copies of the
    // accumulators.
    int k = 0;
    if (nst & 1) {
      issue(0, lds1);
      arrived();
      stage(0, lds1, lds0);
      k = 1;
    } else {
      issue(0, lds0);
    }
    for (; k < nst; k += 2) {
      arrived();
      stage(k, lds0, lds1);
      arrived();
      stage(k + 1, lds1, lds0);
    }
    mfmas(integral_constant<int, NS - 1>{});
  }

  // Epilogue.  Lane (r, h) holds, of block (i, j), row r and columns 8 q + 4 h + {0..3} in
  // elements 4 q .. 4 q + 3.  BF16: each wave parks its rows in LDS (16-byte chunks
  // permuted by the row) and writes whole row runs; FP32: 16-byte pieces.
  uint32_t amax = 0;
  const int64_t cm = m0 + wm, cn = n0 + wn;
  if (p.out_bf16) {
    arrived();  // the tiles in LDS are done with
    uint8_t* out = (w >= NW / 2 ? lds1 : lds0) + w % (NW / 2) * (WM * WN * 2);
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

template <int FA, int MT, int NT, int KW>
static hipError_t launch_direct(const Mxfp4Gemm& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 16 * NT - 1) / (16 * NT)),
                  (unsigned)((p.M + 16 * MT - 1) / (16 * MT)));
  hipLaunchKernelGGL((gemm_mxfp4_direct_kernel<FA, MT, NT, KW>), grid, dim3(64 * KW), 0, stream, p);
  return hipGetLastError();
}

template <int FA, int BM, int BN, int GM, int GN>
static hipError_t launch_tile(const Mxfp4Gemm& p, hipStream_t stream) {
  const int tm = (int)((p.M + BM - 1) / BM), tn = (int)((p.N + BN - 1) / BN);
  hipLaunchKernelGGL((gemm_mxfp4_tile_kernel<FA, BM, BN, GM, GN>), dim3((unsigned)(tm * tn)), dim3(64 * GM * GN), 0,
                     stream, p, tm, tn);
  return hipGetLastError();
}

template <int FA>
static hipError_t launch_fa(const Mxfp4Gemm& p, int num_cus, hipStream_t stream) {
  if (p.M <= 16) return launch_direct<FA, 1, 1, 8>(p, stream);
  // The tile loads address their rows with 30 bits; the codes' loads take 16 blocks of a
  // row at a time, at addresses that are a multiple of 4.
  const bool scales_aligned = ((reinterpret_cast<uintptr_t>(p.sc_a) | (uint64_t)p.ldsa |
                                reinterpret_cast<uintptr_t>(p.sc_b) | (uint64_t)p.ldsb |
                                (uint64_t)(p.K / 32)) & 3u) == 0;
  const bool fits = p.lda < (1 << 21) && p.ldb < (1 << 21) && p.ldsa < (1 << 21) &&
                    p.ldsb < (1 << 21) && p.K >= 512 && scales_aligned;
  if (!fits) return launch_direct<FA, 4, 4, 1>(p, stream);
  const int64_t big = ((p.M + 255) / 256) * ((p.N + 255) / 256);
  if (big >= num_cus) return launch_tile<FA, 256, 256, 4, 2>(p, stream);
  return launch_tile<FA, 128, 128, 2, 2>(p, stream);
}

hipError_t launch_gemm_mxfp4(const Mxfp4Gemm& p, int fa, int num_cus, hipStream_t stream) {
  switch (fa) {
    case kE4M3: return launch_fa<kE4M3>(p, num_cus, stream);
    case kE5M2: return launch_fa<kE5M2>(p, num_cus, stream);
    default: return launch_fa<kE2M1>(p, num_cus, stream);
  }
}

}  // namespace fp8ds
