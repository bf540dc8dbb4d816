// The C ABI of the expert-training operators (include/gemm_gb300.h): the
// grouped products, their gradients and the Newton-Schulz orthogonalisation.
#include <cmath>

#include "gemm_gb300.h"
#include "grouped_host.h"

using namespace gb300;

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxPitch = int64_t(1) << 36;
constexpr int64_t kMaxStride = (int64_t(1) << 39) - 8;   // TMA: under 2^40 bytes

bool dim_ok(int64_t x) { return x >= 0 && x <= kMaxDim; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Sizes, offsets and output type shared by the three grouped products.
int check_grouped(const int32_t* offsets, int64_t groups, int64_t M, int64_t N, int64_t K, int out_dtype) {
  if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K) || groups < 0 || groups > GEMM_MAX_GROUPS ||
      (out_dtype != GEMM_DTYPE_BF16 && out_dtype != GEMM_DTYPE_F32))
    return GEMM_ERR_INVALID_ARG;
  if (groups > 0 && offsets == nullptr) return GEMM_ERR_INVALID_ARG;
  return groups > 0 && !aligned(offsets, 4) ? GEMM_ERR_ALIGNMENT : GEMM_OK;
}

// An operand of `cols` bf16 a row that TMA reads.
int check_operand(const void* p, int64_t cols, int64_t ld) {
  if (p == nullptr || ld < cols || ld > kMaxPitch) return GEMM_ERR_INVALID_ARG;
  return aligned(p, 16) && ld % 8 == 0 ? GEMM_OK : GEMM_ERR_ALIGNMENT;
}

int check_output(const void* p, int64_t cols, int64_t ld, int out_dtype) {
  if (p == nullptr || ld < cols || ld > kMaxPitch) return GEMM_ERR_INVALID_ARG;
  return aligned(p, out_dtype == GEMM_DTYPE_F32 ? 4 : 2) ? GEMM_OK : GEMM_ERR_ALIGNMENT;
}

// The groups' matrices [groups, N, K]: stride >= N * ld, a product that 64 bits
// need not hold.
int check_stride(int64_t groups, int64_t N, int64_t ld, int64_t stride) {
  const bool bad = stride < 0 || stride > kMaxStride || (N > 0 && ld > stride / N);
  return groups > 1 && bad ? GEMM_ERR_INVALID_ARG : GEMM_OK;
}

// Forward (dgrad = false): X = A [M, K], out = D [M, N]; else X = dD [M, N], out = dA [M, K].
int grouped_rows(bool dgrad, const void* X, const void* B, void* out, const int32_t* offsets, int64_t groups,
                 int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldb, int64_t stride_b, int64_t ldo,
                 int out_dtype, cudaStream_t stream) {
  int rc = check_grouped(offsets, groups, M, N, K, out_dtype);
  if (rc != GEMM_OK) return rc;
  const int64_t L = dgrad ? K : N, red = dgrad ? N : K;
  if (groups == 0 || M == 0 || L == 0) return GEMM_OK;
  if ((rc = check_output(out, L, ldo, out_dtype)) != GEMM_OK) return rc;
  if (red > 0) {
    if ((rc = check_operand(X, red, ldx)) != GEMM_OK || (rc = check_operand(B, K, ldb)) != GEMM_OK ||
        (rc = check_stride(groups, N, ldb, stride_b)) != GEMM_OK)
      return rc;
    if (groups > 1 && stride_b % 8 != 0) return GEMM_ERR_ALIGNMENT;
  }
  LaunchCtx ctx;
  if ((rc = launch_context(red, &ctx)) != GEMM_OK) return rc;
  if (!device_pointer_ok(out, ctx) || !device_pointer_ok(offsets, ctx)) return GEMM_ERR_INVALID_ARG;
  if (red == 0)
    return launch_grouped_zero(out, out_dtype == GEMM_DTYPE_F32, offsets, static_cast<uint32_t>(groups),
                               static_cast<uint32_t>(M), static_cast<uint32_t>(L), static_cast<uint64_t>(ldo), 0, ctx,
                               stream);
  if (!device_pointer_ok(X, ctx) || !device_pointer_ok(B, ctx)) return GEMM_ERR_INVALID_ARG;
  GroupedProblem p = {};
  p.M = static_cast<uint32_t>(M);
  p.N = static_cast<uint32_t>(N);
  p.K = static_cast<uint32_t>(K);
  p.groups = static_cast<uint32_t>(groups);
  p.offsets = offsets;
  p.B = B;
  p.ldb = static_cast<uint64_t>(ldb);
  p.stride_b = static_cast<uint64_t>(stride_b);
  p.out = out;
  p.ldo = static_cast<uint64_t>(ldo);
  p.out_f32 = out_dtype == GEMM_DTYPE_F32;
  p.stall_iter = take_stall_request();
  if (dgrad) {
    p.dD = X;
    p.ldd = static_cast<uint64_t>(ldx);
    return launch_grouped_dgrad(p, ctx, stream);
  }
  p.A = X;
  p.lda = static_cast<uint64_t>(ldx);
  return launch_grouped_forward(p, ctx, stream);
}

}  // namespace

extern "C" {

int gemm_bf16_grouped(const void* A, const void* B, void* D, const int32_t* offsets, int64_t groups, int64_t M,
                      int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t stride_b, int64_t ldd, int out_dtype,
                      cudaStream_t stream) {
  return grouped_rows(false, A, B, D, offsets, groups, M, N, K, lda, ldb, stride_b, ldd, out_dtype, stream);
}

int gemm_bf16_grouped_dgrad(const void* dD, const void* B, void* dA, const int32_t* offsets, int64_t groups,
                            int64_t M, int64_t N, int64_t K, int64_t ldd, int64_t ldb, int64_t stride_b, int64_t lda,
                            int out_dtype, cudaStream_t stream) {
  return grouped_rows(true, dD, B, dA, offsets, groups, M, N, K, ldd, ldb, stride_b, lda, out_dtype, stream);
}

int gemm_bf16_grouped_wgrad(const void* dD, const void* A, void* dB, const int32_t* offsets, int64_t groups,
                            int64_t M, int64_t N, int64_t K, int64_t ldd, int64_t lda, int64_t ldb, int64_t stride_b,
                            int out_dtype, int accumulate, cudaStream_t stream) {
  int rc = check_grouped(offsets, groups, M, N, K, out_dtype);
  if (rc != GEMM_OK) return rc;
  if (accumulate != 0 && accumulate != 1) return GEMM_ERR_INVALID_ARG;
  if (groups == 0 || N == 0 || K == 0) return GEMM_OK;
  if ((rc = check_output(dB, K, ldb, out_dtype)) != GEMM_OK || (rc = check_stride(groups, N, ldb, stride_b)) != GEMM_OK)
    return rc;
  if (M > 0 && ((rc = check_operand(dD, N, ldd)) != GEMM_OK || (rc = check_operand(A, K, lda)) != GEMM_OK)) return rc;
  LaunchCtx ctx;
  if ((rc = launch_context(M, &ctx)) != GEMM_OK) return rc;
  if (!device_pointer_ok(dB, ctx) || !device_pointer_ok(offsets, ctx)) return GEMM_ERR_INVALID_ARG;
  if (M == 0)
    return accumulate ? GEMM_OK
                      : launch_grouped_zero(dB, out_dtype == GEMM_DTYPE_F32, nullptr, static_cast<uint32_t>(groups),
                                            static_cast<uint32_t>(N), static_cast<uint32_t>(K),
                                            static_cast<uint64_t>(ldb), static_cast<uint64_t>(stride_b), ctx, stream);
  if (!device_pointer_ok(dD, ctx) || !device_pointer_ok(A, ctx)) return GEMM_ERR_INVALID_ARG;
  GroupedProblem p = {};
  p.M = static_cast<uint32_t>(M);
  p.N = static_cast<uint32_t>(N);
  p.K = static_cast<uint32_t>(K);
  p.groups = static_cast<uint32_t>(groups);
  p.offsets = offsets;
  p.A = A;
  p.lda = static_cast<uint64_t>(lda);
  p.dD = dD;
  p.ldd = static_cast<uint64_t>(ldd);
  p.out = dB;
  p.ldo = static_cast<uint64_t>(ldb);
  p.stride_o = static_cast<uint64_t>(stride_b);
  p.out_f32 = out_dtype == GEMM_DTYPE_F32;
  p.accumulate = accumulate != 0;
  p.stall_iter = take_stall_request();
  return launch_grouped_wgrad(p, ctx, stream);
}

int64_t gemm_newton_schulz_workspace_bytes(int64_t batch, int64_t rows, int64_t cols) {
  if (batch < 0 || batch > 65535 || rows < 0 || cols < 0 || rows > GEMM_NEWTON_SCHULZ_MAX_DIM ||
      cols > GEMM_NEWTON_SCHULZ_MAX_DIM)
    return GEMM_ERR_INVALID_ARG;
  return static_cast<int64_t>(newton_schulz_bytes(static_cast<uint64_t>(batch), static_cast<uint64_t>(rows),
                                                  static_cast<uint64_t>(cols)));
}

int gemm_newton_schulz(const void* G, void* O, int64_t batch, int64_t rows, int64_t cols, int64_t ldg,
                       int64_t stride_g, int64_t ldo, int64_t stride_o, int in_dtype, int out_dtype, int steps,
                       float a, float b, float c, float eps, void* workspace, int64_t workspace_bytes,
                       cudaStream_t stream) {
  const int64_t need = gemm_newton_schulz_workspace_bytes(batch, rows, cols);
  if (need < 0) return static_cast<int>(need);
  if ((in_dtype != GEMM_DTYPE_BF16 && in_dtype != GEMM_DTYPE_F32) ||
      (out_dtype != GEMM_DTYPE_BF16 && out_dtype != GEMM_DTYPE_F32) || steps < 1 || steps > 64 ||
      !std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c) || !(eps >= 0.0f) || !std::isfinite(eps))
    return GEMM_ERR_INVALID_ARG;
  if (batch == 0 || rows == 0 || cols == 0) return GEMM_OK;
  int rc = check_output(G, cols, ldg, in_dtype);   // plain loads: any pitch, element alignment
  if (rc == GEMM_OK) rc = check_output(O, cols, ldo, out_dtype);
  if (rc != GEMM_OK) return rc;
  if (check_stride(batch, rows, ldg, stride_g) != GEMM_OK || check_stride(batch, rows, ldo, stride_o) != GEMM_OK ||
      workspace == nullptr || workspace_bytes < need)
    return GEMM_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return GEMM_ERR_ALIGNMENT;
  LaunchCtx ctx;
  if ((rc = launch_context(rows > cols ? rows : cols, &ctx)) != GEMM_OK) return rc;
  if (!device_pointer_ok(G, ctx) || !device_pointer_ok(O, ctx) || !device_pointer_ok(workspace, ctx))
    return GEMM_ERR_INVALID_ARG;
  NewtonSchulzProblem p = {};
  p.batch = static_cast<uint32_t>(batch);
  p.rows = static_cast<uint32_t>(rows);
  p.cols = static_cast<uint32_t>(cols);
  p.G = G;
  p.g_f32 = in_dtype == GEMM_DTYPE_F32;
  p.ldg = static_cast<uint64_t>(ldg);
  p.stride_g = static_cast<uint64_t>(stride_g);
  p.out = O;
  p.out_f32 = out_dtype == GEMM_DTYPE_F32;
  p.ldo = static_cast<uint64_t>(ldo);
  p.stride_o = static_cast<uint64_t>(stride_o);
  p.steps = steps;
  p.a = a;
  p.b = b;
  p.c = c;
  p.eps = eps;
  p.workspace = workspace;
  return launch_newton_schulz(p, ctx, stream);
}

}  // extern "C"
