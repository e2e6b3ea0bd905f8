// Muon's update: momentum, orthogonalisation by Newton-Schulz products, and (muon_apply in adamw.hip)
// the weights' step.
//
//   m = mu m + g',  U = g' + mu m (Nesterov) or m,  X = U / (|U|_F + eps)
//   A = X X^T,  B = a I + b A + c A A,  X = B X         once per step, with its own a, b, c
// for X with no more rows than columns (else its transpose).  With singular values s of X a step
// maps s to a s + b s^3 + c s^5: with the usual coefficients five steps bring all but the smallest
// near 1.
//
// Precision.  A step multiplies small singular values by a = 3.4, five steps by 485, and what the
// operands' rounding adds to the weak directions grows with them: with X, A and B rounded once to
// BF16 the result was 1e-2 (Gaussian matrices) to 1e-1 (a few strong directions over weak ones)
// off the one in 64 bits, once to F16 1e-3 to 1e-2.  So every operand is a pair of F16, hi + lo (22
// significant bits), and a product is hi hi + hi lo + lo hi in fp32, at three times the matrix
// instructions: 7e-7 to 6e-6 (Gaussian) and up to 3.4e-5 (decaying singular values), where the same
// iteration in fp32 is as far off.  (Pairs of BF16, 16 bits: 1.5e-5 to 3.5e-5 and up to 8e-4; 3%
// faster at 4096 x 14336.)
// F16's range: a matrix is stored times a power of two that brings its largest singular value, which
// bounds its elements, to 2^14 .. 2^15; what F16 cannot hold is then 2^-39 of that.  The bounds follow
// from the coefficients (poly_max, step_max), from |X| <= 1 on; twice of them still fits, and a bound's
// rounding errors are far less (a polynomial of degree 5 has a slope of at most 25 times its bound, so
// errors of 2^-21 of the operands stay such).
//
// Design for gfx950: the products are bound by the matrix cores.  All of them are C = P Q^T over
// K-contiguous pair matrices: X and its transpose are both kept (A and B are symmetric), so no
// operand is read across its rows.  A row of a pair matrix holds, for each 32 columns, 32 hi and then
// 32 lo values: 128 bytes, the row of a stage in LDS.  A stage serves 6 matrix instructions per
// block pair from 8 fragment reads, half of what single operands would read per instruction.  A and
// B are computed for the tiles on and below the diagonal only and stored with their mirror image;
// all sizes are padded with zeros to whole tiles, so no tile has an edge.
// 4096 x 14336, five steps: 6.9 to 7.0 ms.  In 256 x 256 tiles the steps' products run at 1.3 PFLOP/s of F16
// (matrix unit 83 to 91% busy), the symmetric ones of 4096^3 at 1.1 (136 tiles for 256 CUs); momentum
// with the norm's sum 0.13 ms and the split 0.16 are passes over memory.  333 x 130: 96 us, twenty
// launches of 3 to 6.5 us, each a chain of load - product - store.

#include <algorithm>

#include "tile_common.h"

namespace fp8ds {

namespace {

// ------------------------------------------------------------------ pairs

// Byte offset of column c of a pair row (lo: 64 bytes further).
__device__ __forceinline__ int64_t pair_at(int64_t c) { return (c >> 5) * 128 + (c & 31) * 2; }

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
struct Pair8 {
  u32x4 hi, lo;
};
__device__ __forceinline__ Pair8 split8(const float (&v)[8]) {
  Pair8 p;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const v2h h = {(_Float16)v[2 * k], (_Float16)v[2 * k + 1]};
    const v2h l = {(_Float16)(v[2 * k] - (float)h.x), (_Float16)(v[2 * k + 1] - (float)h.y)};
    p.hi[k] = __builtin_bit_cast(uint32_t, h);
    p.lo[k] = __builtin_bit_cast(uint32_t, l);
  }
  return p;
}
__device__ __forceinline__ void store_pair8(uint8_t* row, int64_t c, const float (&v)[8]) {
  const Pair8 p = split8(v);
  *reinterpret_cast<u32x4*>(row + pair_at(c)) = p.hi;
  *reinterpret_cast<u32x4*>(row + pair_at(c) + 64) = p.lo;
}

// A 64 x 64 tile of fp32 values in LDS as pairs: rows row0 .. of `dst` from column col0 on, or its
// transpose.  256 threads.
__device__ __forceinline__ void write_pairs64(const float (&tile)[64][65], bool transposed, uint8_t* dst,
                                              int64_t ld, int64_t row0, int64_t col0) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = threadIdx.x + 256 * i, r = u >> 3, c = (u & 7) * 8;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = transposed ? tile[c + k][r] : tile[r][c + k];
    store_pair8(dst + (row0 + r) * ld, col0 + c, v);
  }
}

// ------------------------------------------------------------------ momentum, norm, first X

__device__ __forceinline__ bool skipped(const float* amax) {
  return amax && (__float_as_uint(*amax) & 0x7FFFFFFFu) >= 0x7F800000u;
}

struct MuonIn {
  const void* g;
  float* m;              // or null
  int64_t n, cols, ldg;  // elements; row length and distance of g's rows
  int vec;               // four elements of g at a time
  float mu;
  int nesterov;
  float grad_scale;
  const float* grad_coef;  // or null
  const float* grad_amax;  // or null
};
// Place of element i in g.
__device__ __forceinline__ int64_t grad_at(const MuonIn& p, int64_t i) {
  return p.ldg == p.cols ? i : i / p.cols * p.ldg + i % p.cols;
}
template <bool GBF>
__device__ __forceinline__ float grad1(const MuonIn& p, int64_t i, float s) {
  if constexpr (GBF)
    return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.g)[i] << 16) * s;
  else
    return static_cast<const float*>(p.g)[i] * s;
}
// U from the gradient and the new momentum, each operation rounded once.
__device__ __forceinline__ float update1(const MuonIn& p, float g, float m) {
#pragma clang fp contract(off)
  return p.nesterov ? g + p.mu * m : m;
}

constexpr int kParts = 2048;  // partial sums of squares, one per workgroup

// Where U is small beside eps, X = U / (|U| + eps) is far below its bound of 1 and would leave F16's range.
// With rho = |U| / (|U| + eps), known on the device alone, X is stored times a further 2^e, the largest
// that its bound allows: after some steps |X| <= growth rho, and e = floor(log2(limit / rho)) >= 0 with
// limit the bound over the growth.  e is 0 where |U| is above eps.
constexpr int kMaxGroups = kMuonMaxSteps;
struct XScales {
  int groups;                // products with X
  double limit[kMaxGroups];  // of X before each
  float* mul;                // [groups][2]: what the extra scales leave to do in X X^T, and in the next X
};
__device__ __forceinline__ int extra_scale(double limit, double rho) {
  const double q = limit / rho;
  if (!(q >= 2.0)) return 0;  // (NaN too)
  const int e = (int)((__double_as_longlong(q) >> 52) & 0x7FF) - 1023;
  return e < 200 ? e : 200;   // (fp32's range of U against the largest eps: 277; what is below is 0)
}

// m, and sum U^2 in 64 bits: a share of the elements per workgroup, four at a time.
template <bool GBF>
__global__ __launch_bounds__(256) void muon_sum_kernel(MuonIn p, double* __restrict__ parts) {
  __shared__ double red[4];
  double sum = 0.0;
  if (!skipped(p.grad_amax)) {
    const float s = p.grad_coef ? p.grad_scale * *p.grad_coef : p.grad_scale;
    const int64_t step = (int64_t)gridDim.x * 1024;
    auto one = [&](int64_t i, float g, float mo) {
#pragma clang fp contract(off)
      float u = g;
      if (p.m) {
        const float m = p.mu * mo + g;
        p.m[i] = m;
        u = update1(p, g, m);
      }
      sum = fma((double)u, (double)u, sum);
    };
    for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x * 4; i < p.n; i += step) {
      if (p.vec && i + 4 <= p.n) {
        float g[4], m[4] = {0.f, 0.f, 0.f, 0.f};
        const int64_t at = grad_at(p, i);
        if constexpr (GBF) {
          const u32x2 d = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p.g) + at);
          g[0] = bf16_lo(d.x); g[1] = bf16_hi(d.x); g[2] = bf16_lo(d.y); g[3] = bf16_hi(d.y);
        } else {
          const f32x4_t d = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p.g) + at);
#pragma unroll
          for (int k = 0; k < 4; ++k) g[k] = d[k];
        }
        if (p.m) {
          const f32x4_t d = *reinterpret_cast<const f32x4_t*>(p.m + i);
#pragma unroll
          for (int k = 0; k < 4; ++k) m[k] = d[k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) one(i + k, g[k] * s, m[k]);
      } else {
        for (int64_t k = i; k < p.n && k < i + 4; ++k)
          one(k, grad1<GBF>(p, grad_at(p, k), s), p.m ? p.m[k] : 0.f);
      }
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) parts[blockIdx.x] = ((red[0] + red[1]) + red[2]) + red[3];
}

// X = U / (|U| + eps) as pairs, as it lies and transposed, 64 x 64 per workgroup; zeros past the
// matrix.
template <bool GBF>
__global__ __launch_bounds__(256) void muon_split_kernel(MuonIn p, const double* __restrict__ parts,
                                                         int nparts, float eps, float scale,
                                                         XScales xs, int64_t rows, int64_t cols,
                                                         uint8_t* __restrict__ x,
                                                         int64_t ldx, uint8_t* __restrict__ xt,
                                                         int64_t ldxt) {
  __shared__ float tile[64][65];
  __shared__ double red[4];
  const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
  const int c = (threadIdx.x & 15) * 4;
  // all loads before the norm's sum, those past the matrix from its last row and column (one by one, each
  // under its own branch: 235 us at 4096 x 14336, so 162)
  float g[4][4], m[4][4];
  const bool quads = p.vec && cols % 4 == 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = min(r0 + (threadIdx.x >> 4) + 16 * i, rows - 1);
    if (quads) {
      const int64_t col = min(c0 + c, cols - 4);
      if constexpr (GBF) {
        const u32x2 d = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p.g) + row * p.ldg + col);
        g[i][0] = bf16_lo(d.x); g[i][1] = bf16_hi(d.x); g[i][2] = bf16_lo(d.y); g[i][3] = bf16_hi(d.y);
      } else {
        const f32x4_t d = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p.g) + row * p.ldg + col);
#pragma unroll
        for (int k = 0; k < 4; ++k) g[i][k] = d[k];
      }
      if (p.m) {
        const f32x4_t d = *reinterpret_cast<const f32x4_t*>(p.m + row * cols + col);
#pragma unroll
        for (int k = 0; k < 4; ++k) m[i][k] = d[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t col = min(c0 + c + k, cols - 1);
        g[i][k] = grad1<GBF>(p, row * p.ldg + col, 1.0f);
        if (p.m) m[i][k] = p.m[row * cols + col];
      }
    }
  }
  double sum = 0.0;
  for (int i = threadIdx.x; i < nparts; i += 256) sum += parts[i];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  // (in 64 bits up to the product: the reciprocal of a tiny eps is beyond fp32's range, that of a norm
  // above 2^126 below its normal numbers)
  const double norm = sqrt(((red[0] + red[1]) + red[2]) + red[3]);
  const double rho = norm > 0.0 ? norm / (norm + (double)eps) : 1.0;
  const double inv = ldexp((double)scale, extra_scale(xs.limit[0], rho)) / (norm + (double)eps);
  if (blockIdx.x == 0 && blockIdx.y == 0 && (int)threadIdx.x < xs.groups) {
    const int k = threadIdx.x, e = extra_scale(xs.limit[k], rho);
    xs.mul[2 * k] = (float)ldexp(1.0, -2 * e);
    xs.mul[2 * k + 1] = (float)ldexp(1.0, (k + 1 < xs.groups ? extra_scale(xs.limit[k + 1], rho) : 0) - e);
  }
  const float s = p.grad_coef ? p.grad_scale * *p.grad_coef : p.grad_scale;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (threadIdx.x >> 4) + 16 * i;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = r0 + r < rows && c0 + c + k < cols;
      const float gs = g[i][k] * s;
      tile[r][c + k] = in ? (float)((double)(p.m ? update1(p, gs, m[i][k]) : gs) * inv) : 0.0f;
    }
  }
  __syncthreads();
  write_pairs64(tile, false, x, ldx, r0, c0);
  write_pairs64(tile, true, xt, ldxt, c0, r0);
}

// ------------------------------------------------------------------ products

constexpr int kGram = 0;   // C = P Q^T where that is symmetric: X X^T, products of polynomials of one A
constexpr int kPart = 1;   // the same over a share of K, fp32 sums for muon_join_kernel
constexpr int kPoly = 2;   // B = a I + b A + c A A, symmetric (P is A)
constexpr int kStep = 3;   // X = P Q^T and its transpose (P is B, Q is X^T)
constexpr int kLast = 4;   // the result

struct NsArgs {
  const uint8_t *P, *Q;  // pair matrices of the same K
  int ld;                // bytes of a row of both
  int nk;                // stages of 32 columns of a share (a multiple of 4, but for the whole of K)
  int tiles_m, tiles_n;
  uint8_t *C, *Ct;       // pair matrices: the result and its transpose
  int64_t ldc, ldct;
  float a, b, c;         // kPoly, with the scales of A and B in them
  float f;               // of the sums: the result's scale over the operands'
  const float* mul;      // or null: a further factor
  float* part;           // kPart: [share][tile pair][T][T]
  void* o;               // kLast: [orows][ldo]
  int o_bf16, o_t;       // o_t: o holds the transpose
  int64_t orows, ocols, ldo;
  int o_vec;             // eight elements at a time
  const float* skip;
};

// Tile pair of number i on and below the diagonal: tm >= tn.
__device__ __forceinline__ void pair_of(int i, int& tm, int& tn) {
  tm = (int)((__builtin_sqrtf(8.0f * (float)i + 1.0f) - 1.0f) * 0.5f);
  while (tm * (tm + 1) / 2 > i) --tm;
  while ((tm + 1) * (tm + 2) / 2 <= i) ++tm;
  tn = i - tm * (tm + 1) / 2;
}

// NBUF stages in LDS.  Two where a CU has a tile of 256 x 256, or two of 128 x 128 that hide each
// other's loads; four where it has one small tile, whose stage is shorter than a load takes
// (916 x 2368: 387 us with two, 231 with four and the accumulators below, 236 with eight; 333 x 130:
// 95 with four, 111 with eight, whose turns end in more stages of zeros).
template <int T, int GM, int GN, int NBUF, int MODE>
__global__ __launch_bounds__(64 * GM * GN, 2) void muon_gemm_kernel(NsArgs p) {
  constexpr int NW = GM * GN, WM = T / GM, WN = T / GN, MI = WM / 32, NI = WN / 32;
  // a block of its own gets an accumulator for each of its three products: they need not wait for
  // one another
  constexpr int NA = MI * NI == 1 ? 3 : 1;
  constexpr bool SYM = MODE == kGram || MODE == kPart || MODE == kPoly;
  constexpr int kA = T * 128, kBuf = 2 * kA;
  // the waves' sums on their way out, 32 rows of fp32 each, take the stages' place
  constexpr int kOut = 32 * WN * 4, kOutWaves = kBuf / kOut < NW ? kBuf / kOut : NW;
  static_assert(kOutWaves * 2 >= NW, "two stages hold every wave's part");
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[kBuf];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[kBuf];
  __shared__ __attribute__((aligned(1024))) uint8_t lds2[NBUF == 4 ? kBuf : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t lds3[NBUF == 4 ? kBuf : 16];
  if (MODE == kLast && skipped(p.skip)) return;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int r = lane & 31, h = lane >> 5;
  const int wm = (w / GN) * WM, wn = (w % GN) * WN;
  int tm, tn, pair = 0;
  if constexpr (SYM) {
    const int total = gridDim.x, x = blockIdx.x & 7;
    pair = total < 8 ? (int)blockIdx.x : x * (total >> 3) + min(x, total & 7) + (int)(blockIdx.x >> 3);
    pair_of(pair, tm, tn);
  } else {
    tile_of<T == 256 ? 4 : 8>(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
  }
  const int64_t m0 = (int64_t)tm * T, n0 = (int64_t)tn * T;
  const int share = MODE == kPart ? blockIdx.y * p.nk : 0;  // first stage
  const TileLoader<T, 128, NW> la(p.P, p.ld, m0, m0 + T, p.ld, tid);
  const TileLoader<T, 128, NW> lb(p.Q, p.ld, n0, n0 + T, p.ld, tid);
  // this lane's chunks of a row: hi of step s, lo of step s
  int of[2][2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int l = 0; l < 2; ++l) of[s][l] = chunk_off<128>(r, 4 * l + 2 * s + h);
  v16f acc[MI][NI], more[2];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  if constexpr (NA == 3) {
#pragma unroll
    for (int e = 0; e < 16; ++e) more[0][e] = more[1][e] = 0.0f;
  }

  auto issue = [&](int k, uint8_t* dst) {  // (zeros past the last stage)
    la.issue((share + k) * 128, p.ld, dst);
    lb.issue((share + k) * 128, p.ld, dst + kA);
  };
  constexpr int kLoads = 2 * la.kPerWave;
  u32x4 fa[2][MI][2], fb[2][NI][2];
  auto frags = [&](const uint8_t* src, auto step) {
    constexpr int s = decltype(step)::value;
    const uint8_t *pa = src + wm * 128, *pb = src + kA + wn * 128;
#pragma unroll
    for (int l = 0; l < 2; ++l) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
        fa[s][i][l] = *reinterpret_cast<const u32x4*>(pa + of[s][l] + 32 * i * 128);
#pragma unroll
      for (int j = 0; j < NI; ++j)
        fb[s][j][l] = *reinterpret_cast<const u32x4*>(pb + of[s][l] + 32 * j * 128);
    }
  };
  auto mfmas = [&](auto step) {
    constexpr int s = decltype(step)::value;
#pragma unroll
    for (int q = 0; q < 3; ++q)  // lo hi, hi lo, hi hi: the small terms first
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          v16f& c = NA == 3 && q < 2 ? more[q] : acc[i][j];
          c = __builtin_amdgcn_mfma_f32_32x32x16_f16(
              __builtin_bit_cast(v8h, fb[s][j][q == 0 ? 1 : 0]),
              __builtin_bit_cast(v8h, fa[s][i][q == 1 ? 1 : 0]), c, 0, 0, 0);
        }
  };
  using std::integral_constant;
  constexpr integral_constant<int, 0> k0th{};
  constexpr integral_constant<int, 1> k1st{};
  // Stage k from its barrier on: a step's fragments are read while the step before it is
  // multiplied, so the previous stage's second step comes first here; the loads of stage
  // k + NBUF - 1 go into the buffer that this barrier freed.
  constexpr int kMf = 3 * MI * NI, kReads = 2 * (MI + NI);
  auto stage = [&](int k, const uint8_t* rd, uint8_t* wr) {
    stage_barrier<(NBUF - 2) * kLoads>();  // all but the loads of later stages have arrived
    frags(rd, k0th);
    issue(k + NBUF - 1, wr);
    mfmas(k1st);
    frags(rd, k1st);
    mfmas(k0th);
    interleave<kMf, kReads, kLoads>();
    interleave<kMf, kReads, 0>();
  };
#pragma unroll
  for (int l = 0; l < 2; ++l) {  // "the second step of the stage before the first": zeros
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[1][i][l] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < NI; ++j) fb[1][j][l] = u32x4{0u, 0u, 0u, 0u};
  }
  // (a last turn is filled up with stages of zeros: a row ends with its last stage, and shares of K
  // are whole turns)
  issue(0, lds0);
  if constexpr (NBUF == 2) {
    for (int k = 0; k < p.nk; k += 2) {
      stage(k, lds0, lds1);
      stage(k + 1, lds1, lds0);
    }
  } else {
    issue(1, lds1);
    issue(2, lds2);
    for (int k = 0; k < p.nk; k += 4) {
      stage(k, lds0, lds3);
      stage(k + 1, lds1, lds0);
      stage(k + 2, lds2, lds1);
      stage(k + 3, lds3, lds2);
    }
  }
  mfmas(k1st);
  if constexpr (NA == 3) {
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[0][0][e] += more[0][e] + more[1][e];
  }

  // Out through LDS, 32 rows of a wave at a time in fp32, chunk c of 16 bytes of row r at
  // c ^ swz32(r): lane (r, h) holds, of block (i, j), row r and columns 8 q + 4 h + {0..3} in
  // elements 4 q .. 4 q + 3.
  vmem_wait_all();
  __syncthreads();
  uint8_t* out = (w < kOutWaves ? lds0 : lds1) + w % kOutWaves * kOut;
  auto swz32 = [](int row) { return WN >= 64 ? (row & 7) ^ ((row >> 3) << 2) : row & 7; };
  auto place = [&](int row, int c) {
    return reinterpret_cast<float*>(out + row * (WN * 4) + (((c >> 2) ^ swz32(row)) << 4) + (c & 3) * 4);
  };
  constexpr int UPR = WN / 8, RPT = 64 / UPR;  // lanes of a row, rows of a turn
  const float f = MODE == kPart || MODE == kPoly ? 1.0f : p.f;
  const float f2 = MODE != kPart && MODE != kPoly && p.mul ? *p.mul : 1.0f;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    if (i > 0) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4_t*>(place(r, 32 * j + 8 * q + 4 * h)) =
            f32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int64_t mi = m0 + wm + 32 * i, nw = n0 + wn;
    // eight consecutive columns of a row in a lane
    auto by_rows = [&](auto&& body) {
#pragma unroll 2
      for (int t = 0; t < 32 / RPT; ++t) {
        const int row = t * RPT + lane / UPR, c = (lane % UPR) * 8;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
          const f32x4_t d = *reinterpret_cast<const f32x4_t*>(place(row, c + k));
#pragma unroll
          for (int e = 0; e < 4; ++e) v[k + e] = d[e] * f * f2;
        }
        body(row, c, v);
      }
    };
    // eight consecutive rows of a column in a lane
    auto by_columns = [&](auto&& body) {
#pragma unroll 2
      for (int t = 0; t < WN / 16; ++t) {
        const int c = t * 16 + (lane & 15), row = (lane >> 4) * 8;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = *place(row + k, c) * f * f2;
        body(row, c, v);
      }
    };
    if constexpr (MODE == kPart) {
      float* dst = p.part + ((int64_t)blockIdx.y * gridDim.x + pair) * T * T;
      by_rows([&](int row, int c, const float (&v)[8]) {
        f32x4_t* o = reinterpret_cast<f32x4_t*>(dst + (wm + 32 * i + row) * T + wn + c);
        o[0] = f32x4_t{v[0], v[1], v[2], v[3]};
        o[1] = f32x4_t{v[4], v[5], v[6], v[7]};
      });
    } else if constexpr (MODE == kLast) {
      const int64_t R = p.orows, C = p.ocols;
      const bool vec = p.o_vec != 0;
      auto put = [&](int64_t row, int64_t c, const float (&v)[8]) {
        if (row >= R || c >= C) return;
        const int64_t at = row * p.ldo + c;
        if (p.o_bf16) {
          const u32x4 d = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                           pack_bf16x2(v[6], v[7])};
          uint16_t* o = static_cast<uint16_t*>(p.o) + at;
          if (vec) {
            *reinterpret_cast<u32x4*>(o) = d;
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (c + k < C) o[k] = (uint16_t)(d[k >> 1] >> (16 * (k & 1)));
          }
        } else {
          float* o = static_cast<float*>(p.o) + at;
          if (vec) {
            reinterpret_cast<f32x4_t*>(o)[0] = f32x4_t{v[0], v[1], v[2], v[3]};
            reinterpret_cast<f32x4_t*>(o)[1] = f32x4_t{v[4], v[5], v[6], v[7]};
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (c + k < C) o[k] = v[k];
          }
        }
      };
      if (p.o_t) by_columns([&](int row, int c, const float (&v)[8]) { put(nw + c, mi + row, v); });
      else by_rows([&](int row, int c, const float (&v)[8]) { put(mi + row, nw + c, v); });
    } else {
      if constexpr (MODE == kPoly) {
        by_rows([&](int row, int c, float (&v)[8]) {
          const uint8_t* a = p.P + (mi + row) * p.ld + pair_at(nw + c);
          const u32x4 hi = *reinterpret_cast<const u32x4*>(a), lo = *reinterpret_cast<const u32x4*>(a + 64);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t wh = hi[k >> 1], wl = lo[k >> 1];  // (a bit_cast of the element itself takes [0])
            const v2h xh = __builtin_bit_cast(v2h, wh), xl = __builtin_bit_cast(v2h, wl);
            const float x = (float)xh[k & 1] + (float)xl[k & 1];
            v[k] = p.c * v[k] + p.b * x;
            if (mi + row == nw + c + k) v[k] += p.a;
          }
          store_pair8(p.C + (mi + row) * p.ldc, nw + c, v);
          if (tm != tn) {  // the mirror image takes the same values
#pragma unroll
            for (int k = 0; k < 8; ++k) *place(row, c + k) = v[k];
          }
        });
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      } else {
        by_rows([&](int row, int c, const float (&v)[8]) {
          store_pair8(p.C + (mi + row) * p.ldc, nw + c, v);
        });
      }
      if (!SYM || tm != tn)
        by_columns([&](int row, int c, const float (&v)[8]) {
          store_pair8(p.Ct + (nw + c) * p.ldct, mi + row, v);
        });
    }
  }
}

// A from the shares of K: a tile pair per workgroup, the shares in order.
__global__ __launch_bounds__(256) void muon_join_kernel(const float* __restrict__ part, int shares,
                                                        int pairs, float f, const float* __restrict__ mul,
                                                        uint8_t* __restrict__ A, int64_t ld) {
  __shared__ float tile[64][65];
  int tm, tn;
  pair_of(blockIdx.x, tm, tn);
  const int c = (threadIdx.x & 15) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (threadIdx.x >> 4) + 16 * i;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < shares; ++s) {
      const f32x4_t d = *reinterpret_cast<const f32x4_t*>(
          part + (((int64_t)s * pairs + blockIdx.x) * 64 + r) * 64 + c);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += d[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) tile[r][c + k] = v[k] * f * *mul;
  }
  __syncthreads();
  const int64_t m0 = (int64_t)tm * 64, n0 = (int64_t)tn * 64;
  write_pairs64(tile, false, A, ld, m0, n0);
  if (tm != tn) write_pairs64(tile, true, A, ld, n0, m0);
}

// ------------------------------------------------------------------ host

// gfx950's, and not the current device's: the workspace must not depend on which device is current when
// its size is asked for.
constexpr int kCus = 256;

// The largest tiles that still give most of the CUs one, but none that the shorter side (m) fills to
// half or less (8 x 128256: in tiles of 256 439 us and a workspace of 398 MB, of 64 366 and 100).
int tile_for(int64_t m, int64_t n, bool sym, int most) {
  for (int t = 256; t > 64; t /= 2) {
    const int64_t a = (m + t - 1) / t, b = (n + t - 1) / t;
    if (t <= most && t / 2 < m && (sym ? a * (a + 1) / 2 : a * b) >= kCus / 2) return t;
  }
  return 64;
}

struct MuonPlan {
  bool tall;            // more rows than columns: X is the transpose
  int64_t m, n;         // padded sizes of X
  int step_tile, sym_tile, shares, share_stages;
  bool grouped;         // steps in groups (launch_muon_direction)
  int64_t parts, mul, x, xt[2], a, t, b[3], share, total;  // offsets in the workspace, bytes
};
MuonPlan muon_plan(int64_t rows, int64_t cols) {
  MuonPlan p = {};
  p.tall = rows > cols;
  const int64_t m = p.tall ? cols : rows, n = p.tall ? rows : cols;
  p.step_tile = tile_for(m, n, false, 256);
  auto pad = [&](int64_t v) { return (v + p.step_tile - 1) / p.step_tile * p.step_tile; };
  p.m = pad(m);
  p.n = pad(n);
  p.sym_tile = tile_for(p.m, p.m, true, p.step_tile);
  // X X^T with few tiles and a long K: shares of K, of 16 stages and more, up to a tile per CU.  Tiles of
  // 128 and 256 are taken from 128 tile pairs on, which leaves no CU for a second share.
  // (Shares that even out 136 tiles over 256 CUs, 3 or 7, were no faster at 4096 x 14336: the CUs
  // that work run at a higher clock.)
  const int64_t st = p.m / p.sym_tile, pairs = st * (st + 1) / 2, stages = p.n / 32;
  int64_t shares = 1;
  while (p.sym_tile == 64 && pairs * shares * 2 <= kCus && stages / (shares * 2) >= 16) shares *= 2;
  p.share_stages = (int)(shares == 1 ? stages : (stages + 4 * shares - 1) / (4 * shares) * 4);
  p.shares = (int)shares;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  p.parts = take(kParts * (int64_t)sizeof(double));
  p.mul = take(kMaxGroups * 2 * (int64_t)sizeof(float));
  p.x = take(p.m * p.n * 4);
  p.xt[0] = take(p.m * p.n * 4);
  p.xt[1] = take(p.m * p.n * 4);
  p.grouped = 2 * p.n >= 3 * p.m;
  p.a = take(p.m * p.m * 4);
  p.b[0] = take(p.m * p.m * 4);
  if (p.grouped) {
    p.t = take(p.m * p.m * 4);
    p.b[1] = take(p.m * p.m * 4);
    p.b[2] = take(p.m * p.m * 4);
  }
  p.share = take(p.shares > 1 ? p.shares * pairs * p.sym_tile * p.sym_tile * 4 : 0);
  p.total = at;
  return p;
}

template <int MODE>
hipError_t launch_product(const NsArgs& a, int tile, unsigned grid, hipStream_t stream) {
  if (tile == 256)
    hipLaunchKernelGGL((muon_gemm_kernel<256, 4, 2, 2, MODE>), dim3(grid), dim3(512), 0, stream, a);
  else if (tile == 128 && grid > kCus)
    hipLaunchKernelGGL((muon_gemm_kernel<128, 2, 2, 2, MODE>), dim3(grid), dim3(256), 0, stream, a);
  else if (tile == 128)
    hipLaunchKernelGGL((muon_gemm_kernel<128, 2, 2, 4, MODE>), dim3(grid), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((muon_gemm_kernel<64, 2, 2, 4, MODE>), dim3(grid), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// Largest |a + b t + c t^2| of 0 <= t <= top, and largest |s (a + b s^2 + c s^4)| of 0 <= s <= top: what a
// step makes of singular values up to there.
double poly_max(const float* abc, double top) {
  const double a = abc[0], b = abc[1], c = abc[2];
  auto at = [&](double t) { return std::fabs(a + t * (b + t * c)); };
  double m = std::fmax(at(0.0), at(top));
  if (c != 0.0) {
    const double t = -b / (2.0 * c);
    if (t > 0.0 && t < top) m = std::fmax(m, at(t));
  }
  return m;
}
double step_max(const float* abc, double top) {
  const double a = abc[0], b = abc[1], c = abc[2];
  auto at = [&](double t) { return std::sqrt(t) * std::fabs(a + t * (b + t * c)); };
  double m = at(top * top);
  auto root = [&](double t) {  // of a + 3 b t + 5 c t^2
    if (t > 0.0 && t < top * top) m = std::fmax(m, at(t));
  };
  const double d = 9.0 * b * b - 20.0 * a * c;
  if (c != 0.0 && d >= 0.0) {
    root((-3.0 * b + std::sqrt(d)) / (10.0 * c));
    root((-3.0 * b - std::sqrt(d)) / (10.0 * c));
  } else if (c == 0.0 && b != 0.0) {
    root(-a / (3.0 * b));
  }
  return m;
}
// The power of two that brings a matrix of this largest singular value to 2^14 .. 2^15: within 2^-400 ..
// 2^400, so that A of any X that fp32 holds has one, and a product's three scales are finite here.
double scale_of(double bound) {
  int e = 0;
  if (std::isfinite(bound) && std::frexp(bound, &e) == 0.5) --e;  // (a zero stays as it is)
  if (!std::isfinite(bound) || e > 400) e = 400;
  return std::ldexp(1.0, 15 - (e < -400 ? -400 : e));
}

}  // namespace

int64_t muon_workspace(int64_t rows, int64_t cols) {
  return rows == 0 || cols == 0 ? 0 : muon_plan(rows, cols).total;
}

hipError_t launch_muon_direction(const MuonLaunch& q, hipStream_t stream) {
  const MuonPlan pl = muon_plan(q.rows, q.cols);
  uint8_t* ws = static_cast<uint8_t*>(q.workspace);
  const bool gvec = reinterpret_cast<uintptr_t>(q.g) % 16 == 0 &&
                    (q.ldg == q.cols || (q.ldg % 4 == 0 && q.cols % 4 == 0));
  MuonIn in = {q.g, q.momentum, q.rows * q.cols, q.cols, q.ldg, gvec ? 1 : 0, q.mu, q.nesterov ? 1 : 0,
               q.grad_scale, q.grad_coef, q.grad_amax};
  double* parts = reinterpret_cast<double*>(ws + pl.parts);
  const int64_t want = (in.n + 1023) / 1024;
  const int nparts = (int)(want < kParts ? want : kParts);
  if (q.g_bf16) hipLaunchKernelGGL((muon_sum_kernel<true>), dim3(nparts), dim3(256), 0, stream, in, parts);
  else hipLaunchKernelGGL((muon_sum_kernel<false>), dim3(nparts), dim3(256), 0, stream, in, parts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;

  uint8_t *x = ws + pl.x, *a = ws + pl.a;
  const int64_t ldx = pl.n * 4, ldxt = pl.m * 4;  // bytes of a pair row of X, of X^T, A and B
  // the matrix as it lies is X, or X's transpose
  uint8_t *as_is = pl.tall ? ws + pl.xt[0] : x, *turned = pl.tall ? x : ws + pl.xt[0];
  const int64_t ld_is = pl.tall ? ldxt : ldx, ld_turned = pl.tall ? ldx : ldxt;
  const int64_t prows = pl.tall ? pl.n : pl.m, pcols = pl.tall ? pl.m : pl.n;
  const dim3 grid((unsigned)(pcols / 64), (unsigned)(prows / 64));
  // X: a bound of its singular values, the scale it is stored with (times its extra scale), and how often it
  // may have become its first self.
  double xb = 1.0, xs = scale_of(xb), growth = 1.0;
  XScales extra = {};
  extra.mul = reinterpret_cast<float*>(ws + pl.mul);
  auto group_size = [&](int k) { return !pl.grouped ? 1 : std::min(q.steps - k, k ? 3 : 2); };
  for (int k = 0, n; k < q.steps; k += n) {
    extra.limit[extra.groups++] = xb / growth;
    n = group_size(k);
    for (int i = 0; i < n; ++i) {
      growth *= poly_max(q.coefs + 3 * (k + i), xb * xb);
      xb = step_max(q.coefs + 3 * (k + i), xb);
    }
  }
  xb = 1.0;
  if (q.g_bf16)
    hipLaunchKernelGGL((muon_split_kernel<true>), grid, dim3(256), 0, stream, in, parts, nparts, q.eps,
                       (float)xs, extra, q.rows, q.cols, as_is, ld_is, turned, ld_turned);
  else
    hipLaunchKernelGGL((muon_split_kernel<false>), grid, dim3(256), 0, stream, in, parts, nparts, q.eps,
                       (float)xs, extra, q.rows, q.cols, as_is, ld_is, turned, ld_turned);
  e = hipGetLastError();

  const int st = (int)(pl.m / pl.sym_tile), pairs = st * (st + 1) / 2;
  // C = P Q^T over m columns, symmetric; ps, qs, cs: their scales
  auto symmetric = [&](auto mode_tag, const uint8_t* P, double ps, const uint8_t* Q, double qs, uint8_t* C,
                       double cs, const float* abc) {
    NsArgs g = {};
    g.P = P; g.Q = Q; g.ld = (int)ldxt; g.nk = (int)(pl.m / 32);
    g.C = g.Ct = C; g.ldc = g.ldct = ldxt;
    g.f = (float)(cs / (ps * qs));
    if (abc) {
      g.a = (float)(abc[0] * cs);
      g.b = (float)(abc[1] * (cs / ps));
      g.c = (float)(abc[2] * (cs / (ps * ps)));
    }
    if (e == hipSuccess) e = launch_product<decltype(mode_tag)::value>(g, pl.sym_tile, pairs, stream);
  };
  const std::integral_constant<int, kGram> product{};
  const std::integral_constant<int, kPoly> poly{};
  int turn = 0;  // of the two transposes
  for (int k = 0; e == hipSuccess && k < q.steps; ++turn) {
    const uint8_t* xt = ws + pl.xt[turn & 1];
    NsArgs g = {};
    g.P = g.Q = x; g.ld = (int)ldx; g.nk = pl.share_stages;
    g.C = g.Ct = a; g.ldc = g.ldct = ldxt;
    double as = scale_of(xb * xb);
    g.f = (float)(as / (xs * xs));
    g.mul = extra.mul + 2 * turn;
    if (pl.shares > 1) {
      g.part = reinterpret_cast<float*>(ws + pl.share);
      hipLaunchKernelGGL((muon_gemm_kernel<64, 2, 2, 4, kPart>), dim3(pairs, pl.shares), dim3(256), 0,
                         stream, g);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL(muon_join_kernel, dim3(pairs), dim3(256), 0, stream, g.part, pl.shares, pairs,
                         g.f, g.mul, a, ldxt);
      e = hipGetLastError();
    } else {
      e = launch_product<kGram>(g, pl.sym_tile, pairs, stream);
    }
    // A group of steps is one product with X: with B_0 of A_0 = X X^T, the next step's A_1 is
    // B_0 A_0 B_0, and X becomes (B_1 B_0) X.  Every factor is a polynomial of A_0, so all of them
    // are symmetric and commute.
    const int size = group_size(k);
    uint8_t *const b0 = ws + pl.b[0], *const b1 = ws + pl.b[1], *const b2 = ws + pl.b[2];
    uint8_t *last = b0, *sofar = b0;  // B of the last step, the product of all
    const float* abc = q.coefs + 3 * k;
    double bound = poly_max(abc, xb * xb), after = step_max(abc, xb);  // of B so far, of X after the steps
    double ls = scale_of(bound), js = ls;                             // scales of `last` and `sofar`
    symmetric(poly, a, as, a, as, b0, ls, abc);
    for (int i = 1; i < size; ++i) {  // (three steps at most: b0 and then b1 are free again by then)
      const double ts = scale_of(xb * after), next = scale_of(after * after);  // (B A is s (s p(s^2)))
      symmetric(product, last, ls, a, as, ws + pl.t, ts, nullptr);
      symmetric(product, ws + pl.t, ts, last, ls, a, next, nullptr);
      as = next;
      xb = after;
      uint8_t *fresh = i == 1 ? b1 : b0, *joined = i == 1 ? b2 : b1;
      abc += 3;
      const double more = poly_max(abc, xb * xb);
      bound *= more;
      ls = scale_of(more);
      symmetric(poly, a, as, a, as, fresh, ls, abc);
      symmetric(product, fresh, ls, sofar, js, joined, scale_of(bound), nullptr);
      js = scale_of(bound);
      after = step_max(abc, xb);
      last = fresh;
      sofar = joined;
    }
    k += size;
    xb = after;
    if (e != hipSuccess) return e;
    g = NsArgs{};
    g.P = sofar; g.Q = xt; g.ld = (int)ldxt; g.nk = (int)(pl.m / 32);
    g.mul = extra.mul + 2 * turn + 1;
    g.tiles_m = (int)(pl.m / pl.step_tile); g.tiles_n = (int)(pl.n / pl.step_tile);
    const unsigned tiles = (unsigned)(g.tiles_m * g.tiles_n);
    if (k < q.steps) {
      const double scale = scale_of(xb);
      g.f = (float)(scale / (js * xs));
      xs = scale;
      g.C = x; g.ldc = ldx;
      g.Ct = ws + pl.xt[(turn + 1) & 1]; g.ldct = ldxt;
      e = launch_product<kStep>(g, pl.step_tile, tiles, stream);
    } else {
      g.f = (float)(1.0 / (js * xs));
      g.o = q.o; g.o_bf16 = q.o_bf16 ? 1 : 0; g.o_t = pl.tall ? 1 : 0;
      g.orows = q.rows; g.ocols = q.cols; g.ldo = q.ldo;
      g.o_vec = q.cols % 8 == 0 && reinterpret_cast<uintptr_t>(q.o) % 16 == 0 &&
                (q.ldo * (q.o_bf16 ? 2 : 4)) % 16 == 0;
      g.skip = q.grad_amax;
      e = launch_product<kLast>(g, pl.step_tile, tiles, stream);
    }
  }
  return e;
}

}  // namespace fp8ds
