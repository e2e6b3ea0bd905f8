// C ABI of the FP8 delayed-scaling Linear: host-side validation, error
// reporting and dispatch to the HIP launchers.  See include/fp8ds.h for the
// contract of each entry point.

#include "fp8ds.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "launch.h"

namespace {

thread_local char g_err[512] = "";

int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return status;
}

int ok() {
  g_err[0] = '\0';
  return FP8DS_OK;
}

int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(FP8DS_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxElems = int64_t(1) << 40;

// Compute units of the current device, cached per device id.
int num_cus() {
  static std::mutex mu;
  static int cache[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    int n = 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      n = 256;
    cache[dev] = n;
  }
  return cache[dev];
}

bool valid_fmt(int f) { return f == FP8DS_E4M3 || f == FP8DS_E5M2; }
bool valid_mx_fmt(int f) { return valid_fmt(f) || f == FP8DS_E2M1; }
bool valid_dtype(int t) { return t == FP8DS_F32 || t == FP8DS_BF16; }
// A transposing cast's tiles of 128 x 128, of 256 threads each, columns along x: of a grid of 2^32
// threads and more HIP drops a part without an error.
bool too_many_tiles(int64_t rows, int64_t cols) {
  return (rows + 127) / 128 > 65535 || (cols + 127) / 128 >= (int64_t(1) << 24);
}

}  // namespace

extern "C" {

int fp8ds_abi_version(void) { return FP8DS_ABI_VERSION; }

const char* fp8ds_status_string(int status) {
  switch (status) {
    case FP8DS_OK: return "ok";
    case FP8DS_ERR_NULL: return "required pointer is null";
    case FP8DS_ERR_SHAPE: return "invalid size or leading dimension";
    case FP8DS_ERR_ENUM: return "enum value out of range";
    case FP8DS_ERR_ALIGN: return "pointer or leading dimension not 16-byte aligned";
    case FP8DS_ERR_HIP: return "HIP runtime error";
    case FP8DS_ERR_UNSUPPORTED: return "unsupported combination";
    case FP8DS_ERR_VALUE: return "scalar argument out of range";
    default: return "unknown status";
  }
}

const char* fp8ds_last_error(void) { return g_err; }

int fp8ds_amax(const void* x, fp8ds_dtype xt, int64_t n, float* amax, hipStream_t stream) {
  if (!amax) return fail(FP8DS_ERR_NULL, "fp8ds_amax: amax is null");
  if (!valid_dtype(xt)) return fail(FP8DS_ERR_ENUM, "fp8ds_amax: bad dtype %d", (int)xt);
  if (n < 0 || n > kMaxElems) return fail(FP8DS_ERR_SHAPE, "fp8ds_amax: bad n %lld", (long long)n);
  if (n > 0 && !x) return fail(FP8DS_ERR_NULL, "fp8ds_amax: x is null");
  if (n > 0 && !aligned16(x)) return fail(FP8DS_ERR_ALIGN, "fp8ds_amax: x not 16-byte aligned");
  hipError_t e = fp8ds::launch_prologue(1, nullptr, nullptr, amax, nullptr, stream);
  if (e == hipSuccess && n > 0)
    e = fp8ds::launch_cast(x, xt == FP8DS_BF16, 1, n, n, 0, nullptr, nullptr, 0, amax, nullptr,
                           nullptr, num_cus(), stream);
  return hip_status(e, "fp8ds_amax");
}

// acc: amax / sat_count are combined into (max / add) instead of reset, and the
// cast kernel writes scale_used itself: no reset kernel before the cast.
static int cast_common(const char* who, const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols,
                       fp8ds_format fmt, const float* scale, uint8_t* q, uint8_t* q_t,
                       float* scale_used, float* amax, uint64_t* sat_count, uint64_t* health,
                       hipStream_t stream, bool acc = false) {
  if (!scale) return fail(FP8DS_ERR_NULL, "%s: scale is null", who);
  if (!valid_dtype(xt)) return fail(FP8DS_ERR_ENUM, "%s: bad dtype %d", who, (int)xt);
  if (!valid_fmt(fmt)) return fail(FP8DS_ERR_ENUM, "%s: bad format %d", who, (int)fmt);
  if (rows < 0 || cols < 0 || (cols > 0 && rows > kMaxElems / cols))
    return fail(FP8DS_ERR_SHAPE, "%s: bad shape %lld x %lld", who, (long long)rows,
                (long long)cols);
  const int64_t n = rows * cols;
  if (n > 0) {
    if (!x || !q) return fail(FP8DS_ERR_NULL, "%s: x or q is null", who);
    if (!aligned16(x) || !aligned16(q) || (q_t && !aligned16(q_t)))
      return fail(FP8DS_ERR_ALIGN, "%s: x, q and q_t must be 16-byte aligned", who);
  }
  if (q_t && too_many_tiles(rows, cols))
    return fail(FP8DS_ERR_SHAPE, "%s: a transposed copy supports at most %d rows and 2^31 - 128 "
                "columns", who, 65535 * 128);
  hipError_t e = hipSuccess;
  if (!acc)  // with health counts, sat_count is counts[0] and the four others follow it
    e = fp8ds::launch_prologue(1, scale, scale_used, amax, sat_count, stream,
                               health ? FP8DS_HEALTH_COUNTS : 1);
  else if (n == 0)  // nothing to combine; the snapshot is still written
    e = fp8ds::launch_prologue(1, scale, scale_used, nullptr, nullptr, stream);
  float* snap = acc ? scale_used : nullptr;
  if (e == hipSuccess && n > 0) {
    if (q_t)
      e = fp8ds::launch_cast_transpose(x, xt == FP8DS_BF16, rows, cols, (int)fmt, scale, q, q_t,
                                       amax, sat_count, health, stream, snap);
    else
      e = fp8ds::launch_cast(x, xt == FP8DS_BF16, 1, n, n, (int)fmt, scale, q, n, amax, sat_count,
                             health, num_cus(), stream, snap);
  }
  return hip_status(e, who);
}

int fp8ds_cast(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols, fp8ds_format fmt,
               const float* scale, uint8_t* q, uint8_t* q_t, float* scale_used, float* amax,
               uint64_t* sat_count, hipStream_t stream) {
  return cast_common("fp8ds_cast", x, xt, rows, cols, fmt, scale, q, q_t, scale_used, amax,
                     sat_count, nullptr, stream);
}

int fp8ds_cast_acc(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols, fp8ds_format fmt,
                   const float* scale, uint8_t* q, uint8_t* q_t, float* scale_used, float* amax,
                   uint64_t* sat_count, hipStream_t stream) {
  return cast_common("fp8ds_cast_acc", x, xt, rows, cols, fmt, scale, q, q_t, scale_used, amax,
                     sat_count, nullptr, stream, true);
}

int fp8ds_cast_health(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols, fp8ds_format fmt,
                      const float* scale, uint8_t* q, uint8_t* q_t, float* scale_used, float* amax,
                      uint64_t* counts, hipStream_t stream) {
  if (!counts) return fail(FP8DS_ERR_NULL, "fp8ds_cast_health: counts is null");
  return cast_common("fp8ds_cast_health", x, xt, rows, cols, fmt, scale, q, q_t, scale_used, amax,
                     counts, counts + 1, stream);
}

int fp8ds_cast_batched(const void* x, fp8ds_dtype xt, int64_t batch, int64_t n, int64_t stride_x,
                       fp8ds_format fmt, const float* scale, uint8_t* q, int64_t stride_q,
                       float* scale_used, float* amax, uint64_t* sat_count, hipStream_t stream) {
  if (!scale) return fail(FP8DS_ERR_NULL, "fp8ds_cast_batched: scale is null");
  if (!valid_dtype(xt)) return fail(FP8DS_ERR_ENUM, "fp8ds_cast_batched: bad dtype %d", (int)xt);
  if (!valid_fmt(fmt)) return fail(FP8DS_ERR_ENUM, "fp8ds_cast_batched: bad format %d", (int)fmt);
  if (batch < 0 || batch > 65535 || n < 0 || n > kMaxElems)
    return fail(FP8DS_ERR_SHAPE, "fp8ds_cast_batched: bad batch %lld or n %lld", (long long)batch,
                (long long)n);
  if (batch == 0) return ok();
  const int esz = xt == FP8DS_BF16 ? 2 : 4;
  if (n > 0) {
    if (!x || !q) return fail(FP8DS_ERR_NULL, "fp8ds_cast_batched: x or q is null");
    if (stride_x < n || stride_q < n || stride_x > kMaxElems || stride_q > kMaxElems)
      return fail(FP8DS_ERR_SHAPE, "fp8ds_cast_batched: strides must be >= n");
    if (!aligned16(x) || !aligned16(q) || (stride_x * esz) % 16 || stride_q % 16)
      return fail(FP8DS_ERR_ALIGN, "fp8ds_cast_batched: operands and strides must keep 16-byte "
                                   "alignment");
  }
  return hip_status(fp8ds::launch_cast_batched(x, xt == FP8DS_BF16, batch, n, stride_x, (int)fmt,
                                               scale, q, stride_q, scale_used, amax, sat_count,
                                               stream),
                    "fp8ds_cast_batched");
}

static int scale_update_common(const char* who, int n_tensors, int hist_len, float* history,
                               int32_t* cursor, const float* amax, const fp8ds_format* fmt,
                               fp8ds_algo algo, int margin, float* scale, float* scale_inv,
                               void* clear, int64_t clear_bytes, hipStream_t stream);

int fp8ds_scale_update(int n_tensors, int hist_len, float* history, int32_t* cursor,
                       const float* amax, const fp8ds_format* fmt, fp8ds_algo algo, int margin,
                       float* scale, float* scale_inv, hipStream_t stream) {
  return scale_update_common("fp8ds_scale_update", n_tensors, hist_len, history, cursor, amax,
                             fmt, algo, margin, scale, scale_inv, nullptr, 0, stream);
}

int fp8ds_scale_update_clear(int n_tensors, int hist_len, float* history, int32_t* cursor,
                             const float* amax, const fp8ds_format* fmt, fp8ds_algo algo,
                             int margin, float* scale, float* scale_inv, void* clear,
                             int64_t clear_bytes, hipStream_t stream) {
  const char* who = "fp8ds_scale_update_clear";
  if (clear_bytes < 0 || clear_bytes % 4 || clear_bytes > (int64_t(1) << 30))
    return fail(FP8DS_ERR_SHAPE, "%s: clear_bytes %lld must be a multiple of 4 in [0, 2^30]", who,
                (long long)clear_bytes);
  if (clear_bytes > 0 && !clear) return fail(FP8DS_ERR_NULL, "%s: clear is null", who);
  if (clear && (reinterpret_cast<uintptr_t>(clear) & 3u))
    return fail(FP8DS_ERR_ALIGN, "%s: clear must be 4-byte aligned", who);
  if (clear && amax && n_tensors > 0) {
    const uintptr_t c0 = reinterpret_cast<uintptr_t>(clear), c1 = c0 + (uintptr_t)clear_bytes;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(amax), a1 = a0 + 4u * (uintptr_t)n_tensors;
    if (c0 < a1 && a0 < c1)
      return fail(FP8DS_ERR_VALUE, "%s: the cleared bytes overlap the amax being consumed", who);
  }
  return scale_update_common(who, n_tensors, hist_len, history, cursor, amax, fmt, algo, margin,
                             scale, scale_inv, clear, clear_bytes, stream);
}

static int scale_update_common(const char* who, int n_tensors, int hist_len, float* history,
                               int32_t* cursor, const float* amax, const fp8ds_format* fmt,
                               fp8ds_algo algo, int margin, float* scale, float* scale_inv,
                               void* clear, int64_t clear_bytes, hipStream_t stream) {
  if (n_tensors < 1 || n_tensors > 4096)
    return fail(FP8DS_ERR_SHAPE, "%s: n_tensors %d not in [1, 4096]", who, n_tensors);
  if (hist_len < 1 || hist_len > 65536)
    return fail(FP8DS_ERR_SHAPE, "%s: hist_len %d not in [1, 65536]", who, hist_len);
  if (!history || !cursor || !amax || !fmt || !scale)
    return fail(FP8DS_ERR_NULL, "%s: history, cursor, amax, fmt and scale are "
                                "required", who);
  if (algo != FP8DS_ALGO_MAX && algo != FP8DS_ALGO_MOST_RECENT)
    return fail(FP8DS_ERR_ENUM, "%s: bad algo %d", who, (int)algo);
  if (margin < -126 || margin > 126)
    return fail(FP8DS_ERR_SHAPE, "%s: margin %d not in [-126, 126]", who, margin);
  fp8ds::FmtBits bits;
  std::memset(&bits, 0, sizeof(bits));
  for (int t = 0; t < n_tensors; ++t) {
    if (!valid_fmt(fmt[t]))
      return fail(FP8DS_ERR_ENUM, "%s: bad format %d for tensor %d", who, (int)fmt[t], t);
    if (fmt[t] == FP8DS_E5M2) bits.w[t >> 5] |= 1u << (t & 31);
  }
  return hip_status(fp8ds::launch_scale_update(n_tensors, hist_len, history, cursor, amax, bits,
                                               (int)algo, margin, scale, scale_inv, stream,
                                               static_cast<uint32_t*>(clear), clear_bytes / 4),
                    who);
}

static int gemm_common(const char* who, fp8ds_op opa, fp8ds_op opb, int64_t M, int64_t N,
                       int64_t K, int64_t batch, const uint8_t* A, fp8ds_format fa, int64_t lda,
                       int64_t stride_a, const float* scale_a, const uint8_t* B, fp8ds_format fb,
                       int64_t ldb, int64_t stride_b, const float* scale_b, void* C,
                       fp8ds_dtype ct, int64_t ldc, int64_t stride_c, float* amax_c,
                       fp8ds_mma mma, hipStream_t stream, bool rowcol = false,
                       bool reset = true) {
  // rowcol: scale_a / scale_b are inverse-scale vectors [M] / [N] (exact datapath)
  if (mma != FP8DS_MMA_EXACT && mma != FP8DS_MMA_FP8)
    return fail(FP8DS_ERR_ENUM, "%s: bad mma %d", who, (int)mma);
  if ((opa != FP8DS_OP_N && opa != FP8DS_OP_T) || (opb != FP8DS_OP_N && opb != FP8DS_OP_T))
    return fail(FP8DS_ERR_ENUM, "%s: bad op", who);
  if (opa == FP8DS_OP_T && opb == FP8DS_OP_T)
    return fail(FP8DS_ERR_UNSUPPORTED, "%s: (T, T) is not supported", who);
  if (!valid_fmt(fa) || !valid_fmt(fb)) return fail(FP8DS_ERR_ENUM, "%s: bad format", who);
  if (!valid_dtype(ct)) return fail(FP8DS_ERR_ENUM, "%s: bad output dtype", who);
  const int64_t lim = int64_t(1) << 31;
  if (M < 0 || N < 0 || K < 0 || M >= lim || N >= lim || K >= lim)
    return fail(FP8DS_ERR_SHAPE, "%s: bad M/N/K %lld/%lld/%lld", who, (long long)M, (long long)N,
                (long long)K);
  if (batch < 0 || batch > 65535) return fail(FP8DS_ERR_SHAPE, "%s: bad batch", who);
  // the launch grid counts 128 x 128 output tiles in one dimension
  if (((M + 127) / 128) * ((N + 127) / 128) >= lim)
    return fail(FP8DS_ERR_SHAPE, "%s: M x N %lld x %lld has too many tiles", who, (long long)M,
                (long long)N);
  if (M == 0 || N == 0 || batch == 0) {
    if (amax_c && batch > 0 && reset)
      return hip_status(fp8ds::launch_prologue(batch, nullptr, nullptr, amax_c, nullptr, stream),
                        who);
    return ok();
  }
  // Stored shapes: A is [M x K] (N) or [K x M] (T); B is [K x N] (N) or [N x K] (T).
  const int64_t a_cols = opa == FP8DS_OP_N ? K : M;
  const int64_t b_cols = opb == FP8DS_OP_N ? N : K;
  if (lda < a_cols || ldb < b_cols || ldc < N || lda < 1 || ldb < 1)
    return fail(FP8DS_ERR_SHAPE, "%s: leading dimension too small (lda %lld >= %lld, ldb %lld >= "
                "%lld, ldc %lld >= %lld)", who, (long long)lda, (long long)a_cols, (long long)ldb,
                (long long)b_cols, (long long)ldc, (long long)N);
  if (!C || !scale_a || !scale_b || (K > 0 && (!A || !B)))
    return fail(FP8DS_ERR_NULL, "%s: A, B, C and the two scales are required", who);
  if (rowcol && !aligned16(scale_b))
    return fail(FP8DS_ERR_ALIGN, "%s: scale_inv_b must be 16-byte aligned", who);
  const int esz = ct == FP8DS_BF16 ? 2 : 4;
  if ((K > 0 && (!aligned16(A) || !aligned16(B) || lda % 16 || ldb % 16)) || !aligned16(C) ||
      (ldc * esz) % 16)
    return fail(FP8DS_ERR_ALIGN, "%s: A, B, C and lda, ldb, ldc*elem_size must be 16-byte aligned",
                who);
  if (batch > 1 && (stride_a % 16 || stride_b % 16 || (stride_c * esz) % 16 || stride_a < 0 ||
                    stride_b < 0 || stride_c < 0))
    return fail(FP8DS_ERR_ALIGN, "%s: batch strides must keep 16-byte alignment", who);
  hipError_t e = hipSuccess;
  if (amax_c && reset) e = fp8ds::launch_prologue(batch, nullptr, nullptr, amax_c, nullptr, stream);
  if (e == hipSuccess) {
    fp8ds::GemmProblem p;
    p.opa = (int)opa; p.opb = (int)opb;
    p.M = M; p.N = N; p.K = K;
    p.A = A; p.fa = (int)fa; p.lda = lda; p.scale_a = scale_a;
    p.B = B; p.fb = (int)fb; p.ldb = ldb; p.scale_b = scale_b;
    p.C = C; p.out_bf16 = ct == FP8DS_BF16; p.ldc = ldc; p.amax_c = amax_c;
    p.batch = batch; p.stride_a = stride_a; p.stride_b = stride_b; p.stride_c = stride_c;
    if (rowcol) {
      p.inv_a = scale_a;
      p.inv_b = scale_b;
      e = fp8ds::launch_gemm_rowcol(p, num_cus(), stream);
    } else {
      e = mma == FP8DS_MMA_EXACT ? fp8ds::launch_gemm_exact(p, num_cus(), stream)
                                 : fp8ds::launch_gemm_fp8(p, num_cus(), stream);
    }
  }
  return hip_status(e, who);
}

int fp8ds_gemm(fp8ds_op opa, fp8ds_op opb, int64_t M, int64_t N, int64_t K, const uint8_t* A,
               fp8ds_format fa, int64_t lda, const float* scale_a, const uint8_t* B,
               fp8ds_format fb, int64_t ldb, const float* scale_b, void* C, fp8ds_dtype ct,
               int64_t ldc, float* amax_c, fp8ds_mma mma, hipStream_t stream) {
  return gemm_common("fp8ds_gemm", opa, opb, M, N, K, 1, A, fa, lda, 0, scale_a, B, fb, ldb, 0,
                     scale_b, C, ct, ldc, 0, amax_c, mma, stream);
}

int fp8ds_gemm_acc(fp8ds_op opa, fp8ds_op opb, int64_t M, int64_t N, int64_t K, const uint8_t* A,
                   fp8ds_format fa, int64_t lda, const float* scale_a, const uint8_t* B,
                   fp8ds_format fb, int64_t ldb, const float* scale_b, void* C, fp8ds_dtype ct,
                   int64_t ldc, float* amax_c, fp8ds_mma mma, hipStream_t stream) {
  return gemm_common("fp8ds_gemm_acc", opa, opb, M, N, K, 1, A, fa, lda, 0, scale_a, B, fb, ldb, 0,
                     scale_b, C, ct, ldc, 0, amax_c, mma, stream, false, false);
}

int fp8ds_gemm_batched(fp8ds_op opa, fp8ds_op opb, int64_t M, int64_t N, int64_t K, int64_t batch,
                       const uint8_t* A, fp8ds_format fa, int64_t lda, int64_t stride_a,
                       const float* scale_a, const uint8_t* B, fp8ds_format fb, int64_t ldb,
                       int64_t stride_b, const float* scale_b, void* C, fp8ds_dtype ct,
                       int64_t ldc, int64_t stride_c, float* amax_c, fp8ds_mma mma,
                       hipStream_t stream) {
  return gemm_common("fp8ds_gemm_batched", opa, opb, M, N, K, batch, A, fa, lda, stride_a, scale_a,
                     B, fb, ldb, stride_b, scale_b, C, ct, ldc, stride_c, amax_c, mma, stream);
}

int fp8ds_linear_batched(int64_t batch, int64_t M, int64_t N, int64_t K, fp8ds_dtype xt,
                         const void* x, int64_t stride_x, fp8ds_format fx, const void* w,
                         int64_t stride_w, fp8ds_format fw, int hist_len, float* history,
                         int32_t* cursor, fp8ds_algo algo, int margin, float* scale,
                         float* scale_used, float* amax, uint64_t* sat_count, uint8_t* xq,
                         int64_t stride_xq, uint8_t* wq, int64_t stride_wq, void* y,
                         int64_t stride_y, float* amax_y, hipStream_t stream) {
  const char* who = "fp8ds_linear_batched";
  if (!valid_dtype(xt)) return fail(FP8DS_ERR_ENUM, "%s: bad dtype %d", who, (int)xt);
  if (xt != FP8DS_BF16) return fail(FP8DS_ERR_UNSUPPORTED, "%s: only BF16 inputs", who);
  if (!valid_fmt(fx) || !valid_fmt(fw)) return fail(FP8DS_ERR_ENUM, "%s: bad format", who);
  if (algo != FP8DS_ALGO_MAX && algo != FP8DS_ALGO_MOST_RECENT)
    return fail(FP8DS_ERR_ENUM, "%s: bad algo %d", who, (int)algo);
  if (batch < 1 || batch > 65535)
    return fail(FP8DS_ERR_SHAPE, "%s: batch %lld not in [1, 65535]", who, (long long)batch);
  auto dim_ok = [](int64_t v) { return v >= 16 && v <= 256 && v % 16 == 0; };
  if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K))
    return fail(FP8DS_ERR_SHAPE, "%s: M, N, K (%lld, %lld, %lld) must be multiples of 16 in "
                "[16, 256]", who, (long long)M, (long long)N, (long long)K);
  if (hist_len < 1 || hist_len > 65536)
    return fail(FP8DS_ERR_SHAPE, "%s: hist_len %d not in [1, 65536]", who, hist_len);
  if (margin < -126 || margin > 126)
    return fail(FP8DS_ERR_SHAPE, "%s: margin %d not in [-126, 126]", who, margin);
  if (!x || !w || !history || !cursor || !scale || !amax || !y)
    return fail(FP8DS_ERR_NULL, "%s: x, w, history, cursor, scale, amax and y are required", who);
  if (stride_x < M * K || stride_w < K * N || stride_y < M * N || (xq && stride_xq < M * K) ||
      (wq && stride_wq < K * N) || stride_x > kMaxElems || stride_w > kMaxElems ||
      stride_y > kMaxElems || stride_xq > kMaxElems || stride_wq > kMaxElems)
    return fail(FP8DS_ERR_SHAPE, "%s: every stride must be at least its problem's size", who);
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || (xq && !aligned16(xq)) ||
      (wq && !aligned16(wq)) || (stride_x * 2) % 16 || (stride_w * 2) % 16 ||
      (stride_y * 2) % 16 || (xq && stride_xq % 16) || (wq && stride_wq % 16))
    return fail(FP8DS_ERR_ALIGN, "%s: pointers and strides must keep 16-byte alignment", who);
  fp8ds::LinearBatchedArgs a;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.batch = (int)batch;
  a.x = static_cast<const uint16_t*>(x);
  a.stride_x = stride_x;
  a.w = static_cast<const uint16_t*>(w);
  a.stride_w = stride_w;
  a.xq = xq;
  a.stride_xq = xq ? stride_xq : 0;
  a.wq = wq;
  a.stride_wq = wq ? stride_wq : 0;
  a.y = static_cast<uint16_t*>(y);
  a.stride_y = stride_y;
  a.amax_y = amax_y;
  a.history = history;
  a.cursor = cursor;
  a.hist_len = hist_len;
  a.algo = (int)algo;
  a.margin = margin;
  a.scale = scale;
  a.scale_used = scale_used;
  a.amax = amax;
  a.sat = reinterpret_cast<unsigned long long*>(sat_count);
  return hip_status(fp8ds::launch_linear_batched(a, (int)fx, (int)fw, stream), who);
}

static int adamw_common(const char* who, float* w, const void* g, fp8ds_dtype gt, float* m, float* v,
                        int64_t rows, int64_t cols, float lr, float beta1, float beta2, float eps,
                        float weight_decay, float grad_scale, const float* grad_coef, int64_t step,
                        const float* grad_amax, fp8ds_format fmt, const float* scale, uint8_t* q,
                        uint8_t* q_t, float* scale_used, float* amax, uint64_t* sat_count,
                        hipStream_t stream) {
#pragma clang fp contract(off)
  if (!valid_dtype(gt)) return fail(FP8DS_ERR_ENUM, "%s: bad gradient dtype %d", who, (int)gt);
  if (rows < 0 || cols < 0 || (cols > 0 && rows > kMaxElems / cols))
    return fail(FP8DS_ERR_SHAPE, "%s: bad shape %lld x %lld", who, (long long)rows,
                (long long)cols);
  if (!(std::isfinite(lr) && std::isfinite(weight_decay) && beta1 >= 0.0f && beta1 < 1.0f &&
        beta2 >= 0.0f && beta2 < 1.0f && std::isfinite(eps) && eps > 0.0f &&
        std::isfinite(grad_scale) && grad_scale > 0.0f && step >= 1))
    return fail(FP8DS_ERR_VALUE,
                "%s: need finite lr and weight_decay, 0 <= beta1, beta2 < 1, finite eps > 0, "
                "finite grad_scale > 0 and step >= 1",
                who);
  // the FP8 copy is requested by a scale
  const bool cast = scale != nullptr;
  if (cast && !valid_fmt(fmt)) return fail(FP8DS_ERR_ENUM, "%s: bad format %d", who, (int)fmt);
  if (!cast && (q || q_t || scale_used || amax || sat_count))
    return fail(FP8DS_ERR_NULL, "%s: q, q_t, scale_used, amax and sat_count need scale", who);
  const int64_t n = rows * cols;
  if (n > 0) {
    if (!w || !g || !m || !v) return fail(FP8DS_ERR_NULL, "%s: w, g, m and v are required", who);
    if (cast && !q) return fail(FP8DS_ERR_NULL, "%s: q is null", who);
    if (!aligned16(w) || !aligned16(g) || !aligned16(m) || !aligned16(v) || (q && !aligned16(q)) ||
        (q_t && !aligned16(q_t)))
      return fail(FP8DS_ERR_ALIGN, "%s: w, g, m, v, q and q_t must be 16-byte aligned", who);
  }
  if (q_t && too_many_tiles(rows, cols))
    return fail(FP8DS_ERR_SHAPE, "%s: a transposed copy supports at most %d rows and 2^31 - 128 "
                "columns", who, 65535 * 128);
  // Per-step constants: float64 from the fp32 hyperparameters, one rounding to fp32.
  const double lr_d = lr, wd_d = weight_decay, b1 = beta1, b2 = beta2;
  fp8ds::AdamWConsts c;
  c.b1 = beta1;
  c.b2 = beta2;
  c.omb1 = (float)(1.0 - b1);
  c.omb2 = (float)(1.0 - b2);
  c.eps = eps;
  c.decay = (float)(1.0 - lr_d * wd_d);
  c.step_size = (float)(lr_d / (1.0 - std::pow(b1, (double)step)));
  c.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(b2, (double)step)));
  c.grad_scale = grad_scale;
  fp8ds::AdamWLaunch a{w, g, gt == FP8DS_BF16, m, v, rows, cols, c, grad_amax, (int)fmt, scale,
                       cast ? q : nullptr, cast ? q_t : nullptr, amax, sat_count, grad_coef};
  hipError_t e = hipSuccess;
  if (cast) e = fp8ds::launch_prologue(1, scale, scale_used, amax, sat_count, stream);
  if (e == hipSuccess && n > 0) e = fp8ds::launch_adamw(a, stream);
  return hip_status(e, who);
}

int fp8ds_adamw(float* w, const void* g, fp8ds_dtype gt, float* m, float* v, int64_t rows,
                int64_t cols, float lr, float beta1, float beta2, float eps, float weight_decay,
                float grad_scale, int64_t step, const float* grad_amax, fp8ds_format fmt,
                const float* scale, uint8_t* q, uint8_t* q_t, float* scale_used, float* amax,
                uint64_t* sat_count, hipStream_t stream) {
  return adamw_common("fp8ds_adamw", w, g, gt, m, v, rows, cols, lr, beta1, beta2, eps,
                      weight_decay, grad_scale, nullptr, step, grad_amax, fmt, scale, q, q_t,
                      scale_used, amax, sat_count, stream);
}

int fp8ds_adamw_clip(float* w, const void* g, fp8ds_dtype gt, float* m, float* v, int64_t rows,
                     int64_t cols, float lr, float beta1, float beta2, float eps,
                     float weight_decay, float grad_scale, const float* grad_coef, int64_t step,
                     const float* grad_amax, fp8ds_format fmt, const float* scale, uint8_t* q,
                     uint8_t* q_t, float* scale_used, float* amax, uint64_t* sat_count,
                     hipStream_t stream) {
  if (!grad_coef) return fail(FP8DS_ERR_NULL, "fp8ds_adamw_clip: grad_coef is null");
  return adamw_common("fp8ds_adamw_clip", w, g, gt, m, v, rows, cols, lr, beta1, beta2, eps,
                      weight_decay, grad_scale, grad_coef, step, grad_amax, fmt, scale, q, q_t,
                      scale_used, amax, sat_count, stream);
}

int fp8ds_gemm_rowcol(fp8ds_op opa, fp8ds_op opb, int64_t M, int64_t N, int64_t K,
                      const uint8_t* A, fp8ds_format fa, int64_t lda, const float* scale_inv_a,
                      const uint8_t* B, fp8ds_format fb, int64_t ldb, const float* scale_inv_b,
                      void* C, fp8ds_dtype ct, int64_t ldc, float* amax_c, hipStream_t stream) {
  return gemm_common("fp8ds_gemm_rowcol", opa, opb, M, N, K, 1, A, fa, lda, 0, scale_inv_a, B, fb,
                     ldb, 0, scale_inv_b, C, ct, ldc, 0, amax_c, FP8DS_MMA_EXACT, stream, true);
}

int fp8ds_cast_rowwise(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols, fp8ds_format fmt,
                       int margin, uint8_t* q, float* scale, float* scale_inv, float* amax,
                       hipStream_t stream) {
  const char* who = "fp8ds_cast_rowwise";
  if (!valid_dtype(xt)) return fail(FP8DS_ERR_ENUM, "%s: bad dtype %d", who, (int)xt);
  if (!valid_fmt(fmt)) return fail(FP8DS_ERR_ENUM, "%s: bad format %d", who, (int)fmt);
  if (rows < 0 || cols < 0 || rows >= (int64_t(1) << 31) || (cols > 0 && rows > kMaxElems / cols))
    return fail(FP8DS_ERR_SHAPE, "%s: bad shape %lld x %lld", who, (long long)rows,
                (long long)cols);
  if (margin < -126 || margin > 126)
    return fail(FP8DS_ERR_SHAPE, "%s: margin %d not in [-126, 126]", who, margin);
  if (rows > 0 && !scale) return fail(FP8DS_ERR_NULL, "%s: scale is null", who);
  if (rows * cols > 0) {
    if (!x || !q) return fail(FP8DS_ERR_NULL, "%s: x or q is null", who);
    if (!aligned16(x) || !aligned16(q))
      return fail(FP8DS_ERR_ALIGN, "%s: x and q must be 16-byte aligned", who);
  }
  return hip_status(fp8ds::launch_rowwise_cast(x, xt == FP8DS_BF16, rows, cols, (int)fmt, margin,
                                               q, scale, scale_inv, amax, stream),
                    who);
}

int fp8ds_cast_current(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols,
                       fp8ds_format fmt, int margin, uint8_t* q, uint8_t* q_t, float* scale,
                       float* scale_inv, float* amax, uint64_t* sat_count, hipStream_t stream) {
  const char* who = "fp8ds_cast_current";
  if (!scale || !amax) return fail(FP8DS_ERR_NULL, "%s: scale and amax are required", who);
  if (margin < -126 || margin > 126)
    return fail(FP8DS_ERR_SHAPE, "%s: margin %d not in [-126, 126]", who, margin);
  if (!valid_dtype(xt)) return fail(FP8DS_ERR_ENUM, "%s: bad dtype %d", who, (int)xt);
  if (!valid_fmt(fmt)) return fail(FP8DS_ERR_ENUM, "%s: bad format %d", who, (int)fmt);
  if (rows < 0 || cols < 0 || (cols > 0 && rows > kMaxElems / cols))
    return fail(FP8DS_ERR_SHAPE, "%s: bad shape %lld x %lld", who, (long long)rows,
                (long long)cols);
  const int64_t n = rows * cols;
  if (n > 0) {
    if (!x || !q) return fail(FP8DS_ERR_NULL, "%s: x or q is null", who);
    if (!aligned16(x) || !aligned16(q) || (q_t && !aligned16(q_t)))
      return fail(FP8DS_ERR_ALIGN, "%s: x, q and q_t must be 16-byte aligned", who);
  }
  if (q_t && too_many_tiles(rows, cols))
    return fail(FP8DS_ERR_SHAPE, "%s: a transposed copy supports at most %d rows and 2^31 - 128 "
                "columns", who, 65535 * 128);
  // amax pass, scale from it, then the cast with that scale
  hipError_t e = fp8ds::launch_prologue(1, nullptr, nullptr, amax, sat_count, stream);
  if (e == hipSuccess && n > 0)
    e = fp8ds::launch_cast(x, xt == FP8DS_BF16, 1, n, n, 0, nullptr, nullptr, n, amax, nullptr,
                           nullptr, num_cus(), stream);
  if (e == hipSuccess) e = fp8ds::launch_current_scale(amax, (int)fmt, margin, scale, scale_inv,
                                                       stream);
  if (e == hipSuccess && n > 0) {
    if (q_t)
      e = fp8ds::launch_cast_transpose(x, xt == FP8DS_BF16, rows, cols, (int)fmt, scale, q, q_t,
                                       nullptr, sat_count, nullptr, stream);
    else
      e = fp8ds::launch_cast(x, xt == FP8DS_BF16, 1, n, n, (int)fmt, scale, q, n, nullptr,
                             sat_count, nullptr, num_cus(), stream);
  }
  return hip_status(e, who);
}

}  // extern "C"

extern "C" {

int fp8ds_cast_mx(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols, fp8ds_format fmt,
                  uint8_t* q, uint8_t* scales, uint8_t* q_t, uint8_t* scales_t,
                  hipStream_t stream) {
  const char* who = "fp8ds_cast_mx";
  if (!valid_dtype(xt)) return fail(FP8DS_ERR_ENUM, "%s: bad dtype %d", who, (int)xt);
  if (!valid_fmt(fmt)) return fail(FP8DS_ERR_ENUM, "%s: bad format %d", who, (int)fmt);
  if (rows < 0 || cols < 0 || (cols > 0 && rows > kMaxElems / cols))
    return fail(FP8DS_ERR_SHAPE, "%s: bad shape %lld x %lld", who, (long long)rows,
                (long long)cols);
  if (cols % 32 != 0)
    return fail(FP8DS_ERR_SHAPE, "%s: the row length %lld is not a multiple of the block (32)",
                who, (long long)cols);
  const int64_t n = rows * cols;
  if (n == 0) return ok();
  if (!x || !q || !scales) return fail(FP8DS_ERR_NULL, "%s: x, q and scales are required", who);
  if (!aligned16(x) || !aligned16(q))
    return fail(FP8DS_ERR_ALIGN, "%s: x and q must be 16-byte aligned", who);
  if (!q_t != !scales_t)
    return fail(FP8DS_ERR_NULL, "%s: q_t and scales_t go together", who);
  if (q_t) {
    if (rows % 128 || cols % 128)
      return fail(FP8DS_ERR_SHAPE, "%s: a transposed copy needs rows and cols in multiples of "
                  "128 (got %lld x %lld)", who, (long long)rows, (long long)cols);
    if (rows / 128 > 65535 || cols / 128 > (int64_t(1) << 31) - 1)
      return fail(FP8DS_ERR_SHAPE, "%s: too many 128-row tiles for a transposed copy", who);
    if (!aligned16(q_t)) return fail(FP8DS_ERR_ALIGN, "%s: q_t must be 16-byte aligned", who);
    return hip_status(fp8ds::launch_mx_cast_transpose(x, xt == FP8DS_BF16, rows, cols, (int)fmt,
                                                      q, scales, q_t, scales_t, stream),
                      who);
  }
  return hip_status(fp8ds::launch_mx_cast(x, xt == FP8DS_BF16, n, (int)fmt, q, scales, stream),
                    who);
}

int fp8ds_gemm_mx(int64_t M, int64_t N, int64_t K, const uint8_t* A, fp8ds_format fa, int64_t lda,
                  const uint8_t* scales_a, int64_t ld_scales_a, const uint8_t* B, fp8ds_format fb,
                  int64_t ldb, const uint8_t* scales_b, int64_t ld_scales_b, void* C,
                  fp8ds_dtype ct, int64_t ldc, float* amax_c, fp8ds_mma mma, hipStream_t stream) {
  const char* who = "fp8ds_gemm_mx";
  if (mma != FP8DS_MMA_EXACT && mma != FP8DS_MMA_FP8)
    return fail(FP8DS_ERR_ENUM, "%s: bad mma %d", who, (int)mma);
  if (!valid_fmt(fa) || !valid_fmt(fb)) return fail(FP8DS_ERR_ENUM, "%s: bad format", who);
  if (!valid_dtype(ct)) return fail(FP8DS_ERR_ENUM, "%s: bad output dtype", who);
  const int64_t lim = int64_t(1) << 31;
  if (M < 0 || N < 0 || K < 0 || M >= lim || N >= lim || K >= lim)
    return fail(FP8DS_ERR_SHAPE, "%s: bad M/N/K %lld/%lld/%lld", who, (long long)M, (long long)N,
                (long long)K);
  if (K % 128 != 0)
    return fail(FP8DS_ERR_SHAPE, "%s: K = %lld is not a multiple of 128", who, (long long)K);
  if (((M + 127) / 128) * ((N + 127) / 128) >= lim)
    return fail(FP8DS_ERR_SHAPE, "%s: M x N %lld x %lld has too many tiles", who, (long long)M,
                (long long)N);
  if (M == 0 || N == 0) {
    if (amax_c)
      return hip_status(fp8ds::launch_prologue(1, nullptr, nullptr, amax_c, nullptr, stream), who);
    return ok();
  }
  if (lda < K || ldb < K || ldc < N || ld_scales_a < K / 32 || ld_scales_b < K / 32)
    return fail(FP8DS_ERR_SHAPE, "%s: leading dimension too small", who);
  if (!C || (K > 0 && (!A || !B || !scales_a || !scales_b)))
    return fail(FP8DS_ERR_NULL, "%s: A, B, their scales and C are required", who);
  const int esz = ct == FP8DS_BF16 ? 2 : 4;
  if ((K > 0 && (!aligned16(A) || !aligned16(B) || lda % 16 || ldb % 16)) || !aligned16(C) ||
      (ldc * esz) % 16)
    return fail(FP8DS_ERR_ALIGN, "%s: A, B, C and lda, ldb, ldc*elem_size must be 16-byte aligned",
                who);
  if (K > 0 && ((reinterpret_cast<uintptr_t>(scales_a) & 3u) ||
                (reinterpret_cast<uintptr_t>(scales_b) & 3u) || ld_scales_a % 4 || ld_scales_b % 4))
    return fail(FP8DS_ERR_ALIGN, "%s: the scale arrays and their leading dimensions must be "
                "4-byte aligned", who);
  hipError_t e = hipSuccess;
  if (amax_c) e = fp8ds::launch_prologue(1, nullptr, nullptr, amax_c, nullptr, stream);
  if (e == hipSuccess) {
    fp8ds::GemmProblem p;
    p.opa = 0; p.opb = 1;
    p.M = M; p.N = N; p.K = K;
    p.A = A; p.fa = (int)fa; p.lda = lda; p.scale_a = nullptr;
    p.B = B; p.fb = (int)fb; p.ldb = ldb; p.scale_b = nullptr;
    p.C = C; p.out_bf16 = ct == FP8DS_BF16; p.ldc = ldc; p.amax_c = amax_c;
    p.batch = 1; p.stride_a = 0; p.stride_b = 0; p.stride_c = 0;
    p.sc_a = scales_a; p.sc_b = scales_b; p.ldsa = ld_scales_a; p.ldsb = ld_scales_b;
    e = fp8ds::launch_gemm_mx(p, mma == FP8DS_MMA_EXACT, num_cus(), stream);
  }
  return hip_status(e, who);
}

}  // extern "C"

// ------------------------------------------------------------------ RMSNorm

namespace {

// One matrix argument of the norm: rows of `cols` elements of `esz` bytes, `ld` apart.
struct RowsArg {
  const char* name;
  const void* p;
  int64_t ld;
  int esz;
};

// Elementwise alignment of every matrix, ld >= cols; *vec: rows on 16-byte borders.
int check_rows(const char* who, const RowsArg* args, int n, int64_t rows, int64_t cols, bool* vec) {
  *vec = cols % 8 == 0;
  for (int i = 0; i < n; ++i) {
    const RowsArg& a = args[i];
    if (!a.p) continue;
    if (a.ld < cols || a.ld > kMaxElems || (rows > 1 && a.ld > kMaxElems / rows))
      return fail(FP8DS_ERR_SHAPE, "%s: leading dimension %lld of %s (rows of %lld)", who,
                  (long long)a.ld, a.name, (long long)cols);
    if (reinterpret_cast<uintptr_t>(a.p) % a.esz)
      return fail(FP8DS_ERR_ALIGN, "%s: %s is not aligned to its elements", who, a.name);
    // 8 elements of one byte are stored as 8 bytes
    const uintptr_t need = a.esz == 1 ? 8 : 16;
    if (reinterpret_cast<uintptr_t>(a.p) % need || (rows > 1 && (a.ld * a.esz) % need)) *vec = false;
  }
  return FP8DS_OK;
}

int check_norm_shape(const char* who, int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31) ||
      (cols > 0 && rows > kMaxElems / cols))
    return fail(FP8DS_ERR_SHAPE, "%s: bad shape %lld x %lld", who, (long long)rows, (long long)cols);
  return FP8DS_OK;
}

// What the three forward calls share: checks, and all of NormArgs but the quantised output.
int norm_args(const char* who, fp8ds::NormArgs& a, const void* x, fp8ds_dtype xt, int64_t ldx,
              const void* residual, int64_t ldr, fp8ds_dtype ht, const void* gamma, fp8ds_dtype gt,
              int64_t rows, int64_t cols, float eps, void* h, int64_t ldh, void* y, fp8ds_dtype yt,
              int64_t ldy, float* rstd, uint8_t* q, int64_t ldq, int64_t qcols) {
  if (!valid_dtype(xt) || !valid_dtype(ht) || !valid_dtype(gt) || !valid_dtype(yt))
    return fail(FP8DS_ERR_ENUM, "%s: bad dtype", who);
  if (xt == FP8DS_F32 && ht == FP8DS_BF16)
    return fail(FP8DS_ERR_UNSUPPORTED, "%s: an FP32 x with a BF16 residual stream", who);
  if (!(std::isfinite(eps) && eps >= 0.0f)) return fail(FP8DS_ERR_VALUE, "%s: bad eps", who);
  if (int e = check_norm_shape(who, rows, cols)) return e;
  if (rows > 0 && cols > 0) {
    if (!x || !gamma) return fail(FP8DS_ERR_NULL, "%s: x and gamma are required", who);
    const int hs = ht == FP8DS_BF16 ? 2 : 4, gs = gt == FP8DS_BF16 ? 2 : 4;
    const RowsArg m[] = {{"x", x, ldx, xt == FP8DS_BF16 ? 2 : 4},
                         {"residual", residual, ldr, hs},
                         {"h", h, ldh, hs},
                         {"y", y, ldy, yt == FP8DS_BF16 ? 2 : 4}};
    if (int e = check_rows(who, m, 4, rows, cols, &a.vec)) return e;
    bool qvec = true;
    const RowsArg qm[] = {{"q", q, ldq, 1}};
    if (int e = check_rows(who, qm, 1, rows, qcols, &qvec)) return e;
    // (q's own column count does not decide: packed rows are cols / 2 bytes long)
    if (q && (reinterpret_cast<uintptr_t>(q) % 8 || (rows > 1 && ldq % 8))) a.vec = false;
    if (reinterpret_cast<uintptr_t>(gamma) % gs)
      return fail(FP8DS_ERR_ALIGN, "%s: gamma is not aligned to its elements", who);
    if (reinterpret_cast<uintptr_t>(gamma) % 16) a.vec = false;
  }
  if (reinterpret_cast<uintptr_t>(rstd) % 4)
    return fail(FP8DS_ERR_ALIGN, "%s: rstd is not aligned to its elements", who);
  a.x = x; a.x_bf16 = xt == FP8DS_BF16; a.ldx = ldx;
  a.res = residual; a.ldr = ldr; a.h_bf16 = ht == FP8DS_BF16;
  a.gamma = gamma; a.gamma_bf16 = gt == FP8DS_BF16;
  a.rows = rows; a.cols = cols; a.eps = eps;
  a.h = h; a.ldh = ldh;
  a.y = y; a.y_bf16 = yt == FP8DS_BF16; a.ldy = ldy;
  a.rstd = rstd;
  a.q = q; a.ldq = ldq;
  return FP8DS_OK;
}

}  // namespace

extern "C" {

int fp8ds_rmsnorm(const void* x, fp8ds_dtype xt, int64_t ldx, const void* residual, int64_t ldr,
                  fp8ds_dtype ht, const void* gamma, fp8ds_dtype gt, int64_t rows, int64_t cols,
                  float eps, void* h, int64_t ldh, void* y, fp8ds_dtype yt, int64_t ldy,
                  float* rstd, fp8ds_format fmt, const float* scale, uint8_t* q, int64_t ldq,
                  float* scale_used, float* amax, uint64_t* sat_count, hipStream_t stream) {
  const char* who = "fp8ds_rmsnorm";
  fp8ds::NormArgs a = {};
  const bool cast = scale != nullptr;
  if (cast && !valid_fmt(fmt)) return fail(FP8DS_ERR_ENUM, "%s: bad format %d", who, (int)fmt);
  if (!cast && (q || scale_used || amax || sat_count))
    return fail(FP8DS_ERR_NULL, "%s: q, scale_used, amax and sat_count need scale", who);
  if (int e = norm_args(who, a, x, xt, ldx, residual, ldr, ht, gamma, gt, rows, cols, eps, h, ldh, y,
                        yt, ldy, rstd, q, ldq, cols))
    return e;
  if (cast && rows > 0 && cols > 0 && !q) return fail(FP8DS_ERR_NULL, "%s: q is null", who);
  if (rows == 0 || cols == 0)  // nothing to combine; the snapshot is still written
    return scale_used ? hip_status(fp8ds::launch_prologue(1, scale, scale_used, nullptr, nullptr,
                                                          stream), who)
                      : ok();
  a.mode = cast ? 1 : 0;
  a.fmt = (int)fmt;
  a.scale_in = scale; a.scale_used = scale_used; a.amax = amax; a.sat = sat_count;
  return hip_status(fp8ds::launch_norm_fwd(a, num_cus(), stream), who);
}

int fp8ds_rmsnorm_rowwise(const void* x, fp8ds_dtype xt, int64_t ldx, const void* residual,
                          int64_t ldr, fp8ds_dtype ht, const void* gamma, fp8ds_dtype gt,
                          int64_t rows, int64_t cols, float eps, void* h, int64_t ldh, void* y,
                          fp8ds_dtype yt, int64_t ldy, float* rstd, fp8ds_format fmt, int margin,
                          uint8_t* q, int64_t ldq, float* scale, float* scale_inv, float* amax,
                          hipStream_t stream) {
  const char* who = "fp8ds_rmsnorm_rowwise";
  fp8ds::NormArgs a = {};
  if (!valid_fmt(fmt)) return fail(FP8DS_ERR_ENUM, "%s: bad format %d", who, (int)fmt);
  if (margin < -126 || margin > 126)
    return fail(FP8DS_ERR_SHAPE, "%s: margin %d not in [-126, 126]", who, margin);
  if (int e = norm_args(who, a, x, xt, ldx, residual, ldr, ht, gamma, gt, rows, cols, eps, h, ldh, y,
                        yt, ldy, rstd, q, ldq, cols))
    return e;
  if (rows == 0 || cols == 0) return ok();
  if (!q || !scale) return fail(FP8DS_ERR_NULL, "%s: q and scale are required", who);
  a.mode = 2;
  a.fmt = (int)fmt; a.margin = margin;
  a.scale_out = scale; a.scale_inv = scale_inv; a.amax = amax;
  return hip_status(fp8ds::launch_norm_fwd(a, num_cus(), stream), who);
}

int fp8ds_rmsnorm_mx(const void* x, fp8ds_dtype xt, int64_t ldx, const void* residual, int64_t ldr,
                     fp8ds_dtype ht, const void* gamma, fp8ds_dtype gt, int64_t rows, int64_t cols,
                     float eps, void* h, int64_t ldh, void* y, fp8ds_dtype yt, int64_t ldy,
                     float* rstd, fp8ds_format fmt, uint8_t* q, int64_t ldq, uint8_t* scales,
                     int64_t ld_scales, hipStream_t stream) {
  const char* who = "fp8ds_rmsnorm_mx";
  fp8ds::NormArgs a = {};
  if (!valid_mx_fmt(fmt)) return fail(FP8DS_ERR_ENUM, "%s: bad format %d", who, (int)fmt);
  if (cols > 0 && cols % 32 != 0)
    return fail(FP8DS_ERR_SHAPE, "%s: the row length %lld is not a multiple of the block (32)", who,
                (long long)cols);
  if (int e = norm_args(who, a, x, xt, ldx, residual, ldr, ht, gamma, gt, rows, cols, eps, h, ldh, y,
                        yt, ldy, rstd, q, ldq, fmt == FP8DS_E2M1 ? cols / 2 : cols))
    return e;
  if (rows == 0 || cols == 0) return ok();
  if (!q || !scales) return fail(FP8DS_ERR_NULL, "%s: q and scales are required", who);
  if (ld_scales < cols / 32 || ld_scales > kMaxElems / rows)
    return fail(FP8DS_ERR_SHAPE, "%s: ld_scales %lld for %lld blocks a row", who,
                (long long)ld_scales, (long long)(cols / 32));
  if (!a.vec)
    return fail(FP8DS_ERR_ALIGN, "%s: the rows of x, residual, h, y and gamma must be 16-byte "
                "aligned, those of q 8-byte", who);
  a.mode = 3;
  a.fmt = (int)fmt;
  a.mx_scales = scales; a.ldms = ld_scales;
  return hip_status(fp8ds::launch_norm_fwd(a, num_cus(), stream), who);
}

int64_t fp8ds_rmsnorm_bwd_workspace(int64_t rows, int64_t cols) {
  if (check_norm_shape("fp8ds_rmsnorm_bwd_workspace", rows, cols)) return FP8DS_ERR_SHAPE;
  ok();
  return rows == 0 ? 0 : (int64_t)fp8ds::norm_bwd_parts(rows, cols) * cols * (int64_t)sizeof(float);
}

int fp8ds_rmsnorm_bwd(const void* dy, fp8ds_dtype dt, int64_t lddy, const void* h, fp8ds_dtype ht,
                      int64_t ldh, const float* rstd, const void* gamma, fp8ds_dtype gt,
                      const void* dres, int64_t lddr, int64_t rows, int64_t cols, void* dx,
                      int64_t lddx, float* dgamma, void* workspace, int64_t workspace_bytes,
                      fp8ds_format fmt, const float* scale, uint8_t* q, int64_t ldq,
                      float* scale_used, float* amax, uint64_t* sat_count, hipStream_t stream) {
  const char* who = "fp8ds_rmsnorm_bwd";
  fp8ds::NormBwdArgs a = {};
  if (!valid_dtype(dt) || !valid_dtype(ht) || !valid_dtype(gt))
    return fail(FP8DS_ERR_ENUM, "%s: bad dtype", who);
  if (dt == FP8DS_F32 && ht == FP8DS_BF16)
    return fail(FP8DS_ERR_UNSUPPORTED, "%s: an FP32 dy with a BF16 residual stream", who);
  const bool cast = scale != nullptr;
  if (cast && !valid_fmt(fmt)) return fail(FP8DS_ERR_ENUM, "%s: bad format %d", who, (int)fmt);
  if (!cast && (q || scale_used || amax || sat_count))
    return fail(FP8DS_ERR_NULL, "%s: q, scale_used, amax and sat_count need scale", who);
  if (int e = check_norm_shape(who, rows, cols)) return e;
  if (cols == 0)
    return scale_used ? hip_status(fp8ds::launch_prologue(1, scale, scale_used, nullptr, nullptr,
                                                          stream), who)
                      : ok();
  if (!dgamma) return fail(FP8DS_ERR_NULL, "%s: dgamma is required", who);
  if (reinterpret_cast<uintptr_t>(dgamma) % 4 || reinterpret_cast<uintptr_t>(rstd) % 4)
    return fail(FP8DS_ERR_ALIGN, "%s: dgamma and rstd are fp32", who);
  if (rows > 0) {
    if (!dy || !h || !rstd || !gamma || !dx)
      return fail(FP8DS_ERR_NULL, "%s: dy, h, rstd, gamma and dx are required", who);
    if (cast && !q) return fail(FP8DS_ERR_NULL, "%s: q is null", who);
    const int hs = ht == FP8DS_BF16 ? 2 : 4;
    const RowsArg m[] = {{"dy", dy, lddy, dt == FP8DS_BF16 ? 2 : 4}, {"h", h, ldh, hs},
                         {"dres", dres, lddr, hs}, {"dx", dx, lddx, hs}, {"q", q, ldq, 1}};
    if (int e = check_rows(who, m, 5, rows, cols, &a.vec)) return e;
    if (reinterpret_cast<uintptr_t>(gamma) % (gt == FP8DS_BF16 ? 2 : 4))
      return fail(FP8DS_ERR_ALIGN, "%s: gamma is not aligned to its elements", who);
    if (reinterpret_cast<uintptr_t>(gamma) % 16) a.vec = false;
    const int64_t need = fp8ds_rmsnorm_bwd_workspace(rows, cols);
    if (!workspace || workspace_bytes < need)
      return fail(workspace ? FP8DS_ERR_SHAPE : FP8DS_ERR_NULL, "%s: workspace of %lld bytes, %lld "
                  "needed", who, (long long)(workspace ? workspace_bytes : 0), (long long)need);
    if (!aligned16(workspace))
      return fail(FP8DS_ERR_ALIGN, "%s: workspace not 16-byte aligned", who);
  }
  a.dy = dy; a.x_bf16 = dt == FP8DS_BF16; a.lddy = lddy;
  a.h = h; a.h_bf16 = ht == FP8DS_BF16; a.ldh = ldh;
  a.dres = dres; a.lddr = lddr;
  a.rstd = rstd; a.gamma = gamma; a.gamma_bf16 = gt == FP8DS_BF16;
  a.rows = rows; a.cols = cols;
  a.dx = dx; a.lddx = lddx; a.dgamma = dgamma; a.work = static_cast<float*>(workspace);
  a.fmt = (int)fmt; a.scale_in = scale; a.q = q; a.ldq = ldq;
  a.scale_used = scale_used; a.amax = amax; a.sat = sat_count;
  hipError_t e = hipSuccess;
  if (rows == 0 && scale_used)
    e = fp8ds::launch_prologue(1, scale, scale_used, nullptr, nullptr, stream);
  if (e == hipSuccess) e = fp8ds::launch_norm_bwd(a, stream);
  return hip_status(e, who);
}

}  // extern "C"

// ------------------------------------------------------------------ gradient norm, clip

namespace {

constexpr int kMaxGrads = 4096;
constexpr int kNormBlocks = 1024;                      // partial sums per launch
// Up to here one workgroup takes the norm: 24 thousand elements 4.7 us against 5.8 in two
// launches; 60 thousand 6.4 against 6.0, but a second launch costs the host 1.5 us more;
// 128 thousand 6.9 against 5.8.
constexpr int64_t kSingleElems = 65536;

int check_grads(const char* who, int n, const void* const* grads, const fp8ds_dtype* types,
                const int64_t* counts, void* const* out, const fp8ds_dtype* out_types) {
  int64_t total = 0;  // bounds a launch's chunk numbers too (2^40 elements: 2^27 chunks)
  if (n < 0 || n > kMaxGrads)
    return fail(FP8DS_ERR_SHAPE, "%s: n_tensors %d not in [0, %d]", who, n, kMaxGrads);
  if (n > 0 && (!grads || !types || !counts || (out && !out_types)))
    return fail(FP8DS_ERR_NULL, "%s: the arrays of addresses, types and counts are required", who);
  for (int i = 0; i < n; ++i) {
    if (!valid_dtype(types[i]) || (out && !valid_dtype(out_types[i])))
      return fail(FP8DS_ERR_ENUM, "%s: bad dtype of tensor %d", who, i);
    if (counts[i] < 0 || counts[i] > kMaxElems)
      return fail(FP8DS_ERR_SHAPE, "%s: bad count %lld of tensor %d", who, (long long)counts[i], i);
    total += counts[i];
    if (total > kMaxElems) return fail(FP8DS_ERR_SHAPE, "%s: too many elements", who);
    if (counts[i] == 0) continue;
    if (!grads[i] || (out && !out[i]))
      return fail(FP8DS_ERR_NULL, "%s: tensor %d is null", who, i);
    if (reinterpret_cast<uintptr_t>(grads[i]) % (types[i] == FP8DS_BF16 ? 2 : 4) ||
        (out && reinterpret_cast<uintptr_t>(out[i]) % (out_types[i] == FP8DS_BF16 ? 2 : 4)))
      return fail(FP8DS_ERR_ALIGN, "%s: tensor %d is not aligned to its elements", who, i);
    if (out && out[i] == grads[i] && out_types[i] != types[i])
      return fail(FP8DS_ERR_UNSUPPORTED, "%s: tensor %d in place with another type", who, i);
  }
  return FP8DS_OK;
}

// Fills a table from tensor *i on (empty tensors left out) and advances *i.
void fill_table(fp8ds::TensorTable& tb, int* i, int n, const void* const* grads,
                const fp8ds_dtype* types, const int64_t* counts, void* const* out,
                const fp8ds_dtype* out_types) {
  std::memset(&tb, 0, sizeof(tb));
  int64_t chunks = 0;
  for (; *i < n && tb.count < fp8ds::kTensors; ++*i) {
    if (counts[*i] == 0) continue;
    const int64_t c = fp8ds::table_chunks(counts[*i]);
    const int k = tb.count++;
    tb.src[k] = grads[*i];
    tb.dst[k] = out ? out[*i] : const_cast<void*>(grads[*i]);
    tb.n[k] = counts[*i];
    tb.start[k] = (uint32_t)chunks;
    if (types[*i] == FP8DS_BF16) tb.src_bf16[k >> 5] |= 1u << (k & 31);
    if ((out ? out_types[*i] : types[*i]) == FP8DS_BF16) tb.dst_bf16[k >> 5] |= 1u << (k & 31);
    chunks += c;
    tb.start[k + 1] = (uint32_t)chunks;
  }
}

}  // namespace

extern "C" {

// one row of partial sums per launch
int64_t fp8ds_grad_norm_workspace(void) {
  return (int64_t)(kMaxGrads / fp8ds::kTensors) * kNormBlocks * (int64_t)sizeof(double);
}

int fp8ds_grad_norm(int n_tensors, const void* const* grads, const fp8ds_dtype* types,
                    const int64_t* counts, float grad_scale, float max_norm, float* norm,
                    float* coef, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  const char* who = "fp8ds_grad_norm";
  if (int e = check_grads(who, n_tensors, grads, types, counts, nullptr, nullptr)) return e;
  if (!norm) return fail(FP8DS_ERR_NULL, "%s: norm is required", who);
  if (!(std::isfinite(grad_scale) && grad_scale > 0.0f))
    return fail(FP8DS_ERR_VALUE, "%s: grad_scale must be finite and > 0", who);
  if (coef && !(max_norm > 0.0f)) return fail(FP8DS_ERR_VALUE, "%s: max_norm must be > 0", who);
  if (reinterpret_cast<uintptr_t>(norm) % 4 || reinterpret_cast<uintptr_t>(coef) % 4)
    return fail(FP8DS_ERR_ALIGN, "%s: norm and coef are fp32", who);
  int64_t total = 0;
  for (int i = 0; i < n_tensors; ++i) total += counts[i];
  fp8ds::TensorTable tb;
  int i = 0;
  fill_table(tb, &i, n_tensors, grads, types, counts, nullptr, nullptr);
  if (i == n_tensors && total <= kSingleElems)
    return hip_status(fp8ds::launch_grad_norm_single(tb, grad_scale, max_norm, norm, coef, stream),
                      who);
  if (!workspace || workspace_bytes < fp8ds_grad_norm_workspace())
    return fail(workspace ? FP8DS_ERR_SHAPE : FP8DS_ERR_NULL, "%s: workspace of %lld bytes, %lld "
                "needed", who, (long long)(workspace ? workspace_bytes : 0),
                (long long)fp8ds_grad_norm_workspace());
  if (!aligned16(workspace)) return fail(FP8DS_ERR_ALIGN, "%s: workspace not 16-byte aligned", who);
  double* parts = static_cast<double*>(workspace);
  int used = 0;
  hipError_t e = hipSuccess;
  while (e == hipSuccess && tb.count > 0) {
    const uint32_t chunks = tb.start[tb.count];
    const int blocks = (int)(chunks < (uint32_t)kNormBlocks ? chunks : (uint32_t)kNormBlocks);
    e = fp8ds::launch_grad_norm_part(tb, blocks, parts + used, stream);
    used += blocks;
    fill_table(tb, &i, n_tensors, grads, types, counts, nullptr, nullptr);
  }
  if (e == hipSuccess)
    e = fp8ds::launch_grad_norm_join(parts, used, grad_scale, max_norm, norm, coef, stream);
  return hip_status(e, who);
}

int fp8ds_grad_clip(int n_tensors, const void* const* grads, const fp8ds_dtype* types,
                    const int64_t* counts, void* const* out, const fp8ds_dtype* out_types,
                    const float* coef, hipStream_t stream) {
  const char* who = "fp8ds_grad_clip";
  if (int e = check_grads(who, n_tensors, grads, types, counts, out, out_types)) return e;
  if (!coef) return fail(FP8DS_ERR_NULL, "%s: coef is required", who);
  hipError_t e = hipSuccess;
  for (int i = 0; e == hipSuccess && i < n_tensors;) {
    fp8ds::TensorTable tb;
    fill_table(tb, &i, n_tensors, grads, types, counts, out, out_types);
    e = fp8ds::launch_grad_clip(tb, coef, stream);
  }
  return hip_status(e, who);
}

// ------------------------------------------------------------------ MXFP4

int fp8ds_cast_mxfp4(const void* x, fp8ds_dtype xt, int64_t rows, int64_t cols, uint8_t* q,
                     uint8_t* scales, uint8_t* q_t, uint8_t* scales_t, hipStream_t stream) {
  const char* who = "fp8ds_cast_mxfp4";
  if (!valid_dtype(xt)) return fail(FP8DS_ERR_ENUM, "%s: bad dtype %d", who, (int)xt);
  if (rows < 0 || cols < 0 || (cols > 0 && rows > kMaxElems / cols))
    return fail(FP8DS_ERR_SHAPE, "%s: bad shape %lld x %lld", who, (long long)rows,
                (long long)cols);
  if (cols % 32 != 0)
    return fail(FP8DS_ERR_SHAPE, "%s: the row length %lld is not a multiple of the block (32)",
                who, (long long)cols);
  const int64_t n = rows * cols;
  if (n == 0) return ok();
  if (!x || !q || !scales) return fail(FP8DS_ERR_NULL, "%s: x, q and scales are required", who);
  if (!q_t != !scales_t) return fail(FP8DS_ERR_NULL, "%s: q_t and scales_t go together", who);
  if (!aligned16(x) || !aligned16(q) || (q_t && !aligned16(q_t)))
    return fail(FP8DS_ERR_ALIGN, "%s: x, q and q_t must be 16-byte aligned", who);
  if (!q_t)
    return hip_status(fp8ds::launch_mxfp4_cast(x, xt == FP8DS_BF16, n, q, scales, num_cus(), stream), who);
  if (rows % 32 != 0)
    return fail(FP8DS_ERR_SHAPE, "%s: a transposed copy needs rows in multiples of 32 (got %lld)",
                who, (long long)rows);
  if (too_many_tiles(rows, cols))
    return fail(FP8DS_ERR_SHAPE, "%s: too many tiles for a transposed copy", who);
  return hip_status(fp8ds::launch_mxfp4_cast_transpose(x, xt == FP8DS_BF16, rows, cols, q, scales,
                                                       q_t, scales_t, stream),
                    who);
}

int fp8ds_dequant_mxfp4(const uint8_t* q, const uint8_t* scales, int64_t rows, int64_t cols,
                        void* y, fp8ds_dtype yt, hipStream_t stream) {
  const char* who = "fp8ds_dequant_mxfp4";
  if (!valid_dtype(yt)) return fail(FP8DS_ERR_ENUM, "%s: bad dtype %d", who, (int)yt);
  if (rows < 0 || cols < 0 || (cols > 0 && rows > kMaxElems / cols))
    return fail(FP8DS_ERR_SHAPE, "%s: bad shape %lld x %lld", who, (long long)rows,
                (long long)cols);
  if (cols % 32 != 0)
    return fail(FP8DS_ERR_SHAPE, "%s: the row length %lld is not a multiple of the block (32)",
                who, (long long)cols);
  if (rows * cols == 0) return ok();
  if (!q || !scales || !y) return fail(FP8DS_ERR_NULL, "%s: q, scales and y are required", who);
  if (!aligned16(q) || !aligned16(y))
    return fail(FP8DS_ERR_ALIGN, "%s: q and y must be 16-byte aligned", who);
  return hip_status(fp8ds::launch_mxfp4_dequant(q, scales, rows * cols, y, yt == FP8DS_BF16, stream),
                    who);
}

static int gemm_mxfp4_common(const char* who, int64_t M, int64_t N, int64_t K, const uint8_t* A,
                             fp8ds_format fa, int64_t lda, const uint8_t* scales_a,
                             int64_t ld_scales_a, const uint8_t* B, int64_t ldb,
                             const uint8_t* scales_b, int64_t ld_scales_b, void* C, fp8ds_dtype ct,
                             int64_t ldc, float* amax_c, fp8ds_mma mma, hipStream_t stream) {
  if (mma != FP8DS_MMA_EXACT && mma != FP8DS_MMA_FP8)
    return fail(FP8DS_ERR_ENUM, "%s: bad mma %d", who, (int)mma);
  if (!valid_mx_fmt(fa)) return fail(FP8DS_ERR_ENUM, "%s: bad format %d", who, (int)fa);
  if (!valid_dtype(ct)) return fail(FP8DS_ERR_ENUM, "%s: bad output dtype", who);
  const int64_t lim = int64_t(1) << 31;
  if (M < 0 || N < 0 || K < 0 || M >= lim || N >= lim || K >= lim)
    return fail(FP8DS_ERR_SHAPE, "%s: bad M/N/K %lld/%lld/%lld", who, (long long)M, (long long)N,
                (long long)K);
  if (K % 32 != 0)
    return fail(FP8DS_ERR_SHAPE, "%s: K = %lld is not a multiple of the block (32)", who,
                (long long)K);
  if (M > 65535 * int64_t(64))
    return fail(FP8DS_ERR_SHAPE, "%s: M = %lld is too large", who, (long long)M);
  if (amax_c && reinterpret_cast<uintptr_t>(amax_c) % 4)
    return fail(FP8DS_ERR_ALIGN, "%s: amax_c is fp32", who);
  if (M == 0 || N == 0) {
    if (amax_c)
      return hip_status(fp8ds::launch_prologue(1, nullptr, nullptr, amax_c, nullptr, stream), who);
    return ok();
  }
  if (lda < K || ldb < K || ldc < N || ld_scales_a < K / 32 || ld_scales_b < K / 32 ||
      lda > kMaxElems / M || ldb > kMaxElems / N || ldc > kMaxElems / M ||
      ld_scales_a > kMaxElems / M || ld_scales_b > kMaxElems / N)
    return fail(FP8DS_ERR_SHAPE, "%s: bad leading dimension", who);
  if (!C || (K > 0 && (!A || !B || !scales_a || !scales_b)))
    return fail(FP8DS_ERR_NULL, "%s: A, B, their scales and C are required", who);
  const int esz = ct == FP8DS_BF16 ? 2 : 4;
  if (K > 0 && (!aligned16(A) || !aligned16(B) || (M > 1 && lda % (fa == FP8DS_E2M1 ? 32 : 16)) ||
                (N > 1 && ldb % 32)))
    return fail(FP8DS_ERR_ALIGN, "%s: the rows of A and B must be 16-byte aligned", who);
  if (reinterpret_cast<uintptr_t>(C) % esz)
    return fail(FP8DS_ERR_ALIGN, "%s: C is not aligned to its elements", who);
  hipError_t e = hipSuccess;
  if (amax_c) e = fp8ds::launch_prologue(1, nullptr, nullptr, amax_c, nullptr, stream);
  if (e == hipSuccess) {
    fp8ds::Mxfp4Gemm p;
    p.M = M; p.N = N; p.K = K;
    p.A = A; p.lda = lda; p.sc_a = scales_a; p.ldsa = ld_scales_a;
    p.B = B; p.ldb = ldb; p.sc_b = scales_b; p.ldsb = ld_scales_b;
    p.C = C; p.out_bf16 = ct == FP8DS_BF16; p.ldc = ldc; p.amax_c = amax_c;
    e = fp8ds::launch_gemm_mxfp4(p, (int)fa, mma == FP8DS_MMA_EXACT, num_cus(), stream);
  }
  return hip_status(e, who);
}

int fp8ds_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const uint8_t* A, fp8ds_format fa,
                     int64_t lda, const uint8_t* scales_a, int64_t ld_scales_a, const uint8_t* B,
                     int64_t ldb, const uint8_t* scales_b, int64_t ld_scales_b, void* C,
                     fp8ds_dtype ct, int64_t ldc, float* amax_c, hipStream_t stream) {
  return gemm_mxfp4_common("fp8ds_gemm_mxfp4", M, N, K, A, fa, lda, scales_a, ld_scales_a, B, ldb,
                           scales_b, ld_scales_b, C, ct, ldc, amax_c, FP8DS_MMA_EXACT, stream);
}

int fp8ds_gemm_mxfp4_mma(int64_t M, int64_t N, int64_t K, const uint8_t* A, fp8ds_format fa,
                         int64_t lda, const uint8_t* scales_a, int64_t ld_scales_a,
                         const uint8_t* B, int64_t ldb, const uint8_t* scales_b,
                         int64_t ld_scales_b, void* C, fp8ds_dtype ct, int64_t ldc, float* amax_c,
                         fp8ds_mma mma, hipStream_t stream) {
  return gemm_mxfp4_common("fp8ds_gemm_mxfp4_mma", M, N, K, A, fa, lda, scales_a, ld_scales_a, B,
                           ldb, scales_b, ld_scales_b, C, ct, ldc, amax_c, mma, stream);
}

}  // extern "C"
