// The C ABI of the losses over a vocabulary (include/gemm_gb300.h): cross entropy and
// distillation from a teacher's top logits, with their gradients.
#include <cmath>

#include "gemm_gb300.h"
#include "grouped_host.h"
#include "loss_host.h"

using namespace gb300;

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxPitch = int64_t(1) << 36;

// (exponents are taken in base 2)
bool scale_ok(float scale) { return scale > 0.0f && std::isfinite(scale * 1.4426950408889634f); }
bool dim_ok(int64_t x) { return x >= 0 && x <= kMaxDim; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A [rows, cols] matrix of `size` bytes an element, at `unit` elements' alignment and pitch.
int check_matrix(const void* p, int64_t cols, int64_t ld, uintptr_t size, int64_t unit) {
  if (p == nullptr || ld < cols || ld > kMaxPitch) return GEMM_ERR_INVALID_ARG;
  return aligned(p, size * static_cast<uintptr_t>(unit)) && ld % unit == 0 ? GEMM_OK : GEMM_ERR_ALIGNMENT;
}
int check_vector(const void* p, uintptr_t size) {
  if (p == nullptr) return GEMM_ERR_INVALID_ARG;
  return aligned(p, size) ? GEMM_OK : GEMM_ERR_ALIGNMENT;
}
bool index_code_ok(int code) { return code == GEMM_INDEX_I32 || code == GEMM_INDEX_I64; }
bool float_code_ok(int code) { return code == GEMM_DTYPE_BF16 || code == GEMM_DTYPE_F32; }
uintptr_t index_size(int code) { return code == GEMM_INDEX_I64 ? 8 : 4; }
uintptr_t float_size(int code) { return code == GEMM_DTYPE_F32 ? 4 : 2; }

struct Sizes {
  int64_t M, N, K, top;        // top: 0 for a target per row
};

int64_t workspace_bytes(const Sizes& z, int grad) {
  if (!dim_ok(z.M) || !dim_ok(z.N) || !dim_ok(z.K) || (grad != 0 && grad != 1)) return GEMM_ERR_INVALID_ARG;
  if (z.M == 0 || z.N == 0) return 0;
  const uint64_t M = static_cast<uint64_t>(z.M), N = static_cast<uint64_t>(z.N), K = static_cast<uint64_t>(z.K),
                 top = static_cast<uint64_t>(z.top);
  const uint64_t n = grad ? loss_backward_bytes(M, N, K, top) : loss_forward_bytes(M, N, K, top);
  return n == kNoWorkspace ? static_cast<int64_t>(GEMM_ERR_INVALID_ARG) : static_cast<int64_t>(n);
}

// Sizes, operands and workspace shared by all four calls; the rest of `p` is the caller's.
int check_common(const Sizes& z, const void* A, const void* B, int64_t lda, int64_t ldb, const void* ws, int64_t ws_bytes,
                 int grad) {
  int rc;
  if (z.K > 0 && ((rc = check_matrix(A, z.K, lda, 2, 8)) != GEMM_OK || (rc = check_matrix(B, z.K, ldb, 2, 8)) != GEMM_OK))
    return rc;
  const int64_t need = workspace_bytes(z, grad);
  if (ws == nullptr || need < 0 || ws_bytes < need) return GEMM_ERR_INVALID_ARG;
  return aligned(ws, 256) ? GEMM_OK : GEMM_ERR_ALIGNMENT;
}

void fill(LossProblem& p, const Sizes& z, const void* A, const void* B, int64_t lda, int64_t ldb, void* ws) {
  p.M = static_cast<uint32_t>(z.M);
  p.N = static_cast<uint32_t>(z.N);
  p.K = static_cast<uint32_t>(z.K);
  p.top = static_cast<uint32_t>(z.top);
  p.A = A;
  p.B = B;
  p.lda = static_cast<uint64_t>(lda);
  p.ldb = static_cast<uint64_t>(ldb);
  p.workspace = ws;
}

bool operands_ok(const LossProblem& p, const LaunchCtx& ctx) {
  return device_pointer_ok(p.workspace, ctx) &&
         (p.K == 0 || (device_pointer_ok(p.A, ctx) && device_pointer_ok(p.B, ctx))) &&
         (p.top > 0 ? device_pointer_ok(p.teacher, ctx) && device_pointer_ok(p.ids, ctx)
                    : device_pointer_ok(p.targets, ctx));
}

int forward(LossProblem& p, const Sizes& z, const void* A, const void* B, int64_t lda, int64_t ldb, float* loss, float* lse,
            void* ws, int64_t ws_bytes, cudaStream_t stream) {
  int rc;
  if ((rc = check_vector(loss, 4)) != GEMM_OK || (rc = check_vector(lse, 4)) != GEMM_OK ||
      (rc = check_common(z, A, B, lda, ldb, ws, ws_bytes, 0)) != GEMM_OK)
    return rc;
  fill(p, z, A, B, lda, ldb, ws);
  p.loss = loss;
  p.lse_out = lse;
  LaunchCtx ctx;
  if ((rc = launch_context(z.K, &ctx)) != GEMM_OK) return rc;
  if (!operands_ok(p, ctx) || !device_pointer_ok(loss, ctx) || !device_pointer_ok(lse, ctx)) return GEMM_ERR_INVALID_ARG;
  p.stall_iter = take_stall_request();
  return launch_loss_forward(p, ctx, stream);
}

int backward(LossProblem& p, const Sizes& z, const float* dloss, int64_t inc_dloss, const void* A, const void* B,
             const float* lse, void* dA, void* dB, int64_t lda, int64_t ldb, int64_t ld_da, int64_t ld_db, int da_dtype,
             int db_dtype, int accumulate, void* ws, int64_t ws_bytes, cudaStream_t stream) {
  if (!float_code_ok(da_dtype) || !float_code_ok(db_dtype) || (accumulate != 0 && accumulate != 1) || inc_dloss < 0 ||
      inc_dloss > kMaxPitch)
    return GEMM_ERR_INVALID_ARG;
  if (z.K == 0 || (dA == nullptr && dB == nullptr)) return GEMM_OK;   // nothing to write
  int rc;
  if (dB != nullptr && (rc = check_matrix(dB, z.K, ld_db, float_size(db_dtype), 1)) != GEMM_OK) return rc;
  LaunchCtx ctx;
  if (z.M == 0) {   // an empty sum
    if (dB == nullptr || z.N == 0 || accumulate) return GEMM_OK;
    if ((rc = launch_context(z.K, &ctx)) != GEMM_OK) return rc;
    if (!device_pointer_ok(dB, ctx)) return GEMM_ERR_INVALID_ARG;
    return launch_grouped_zero(dB, db_dtype == GEMM_DTYPE_F32, nullptr, 1, static_cast<uint32_t>(z.N),
                               static_cast<uint32_t>(z.K), static_cast<uint64_t>(ld_db), 0, ctx, stream);
  }
  if (dA != nullptr && (rc = check_matrix(dA, z.K, ld_da, float_size(da_dtype), 1)) != GEMM_OK) return rc;
  if ((rc = check_vector(dloss, 4)) != GEMM_OK || (rc = check_vector(lse, 4)) != GEMM_OK ||
      (rc = check_common(z, A, B, lda, ldb, ws, ws_bytes, 1)) != GEMM_OK)
    return rc;
  fill(p, z, A, B, lda, ldb, ws);
  p.dloss = dloss;
  p.inc_dloss = static_cast<uint64_t>(inc_dloss);
  p.lse = lse;
  p.dA = dA;
  p.dB = dB;
  p.ld_da = static_cast<uint64_t>(ld_da);
  p.ld_db = static_cast<uint64_t>(ld_db);
  p.da_f32 = da_dtype == GEMM_DTYPE_F32;
  p.db_f32 = db_dtype == GEMM_DTYPE_F32;
  p.accumulate = accumulate != 0;
  // a wait's limit covers the longest reduction: over the width, a piece of the vocabulary, the rows
  const int64_t longest = z.K > z.N ? (z.K > z.M ? z.K : z.M) : (z.N > z.M ? z.N : z.M);
  if ((rc = launch_context(longest, &ctx)) != GEMM_OK) return rc;
  if (!operands_ok(p, ctx) || !device_pointer_ok(dloss, ctx) || !device_pointer_ok(lse, ctx) ||
      (dA != nullptr && !device_pointer_ok(dA, ctx)) || (dB != nullptr && !device_pointer_ok(dB, ctx)))
    return GEMM_ERR_INVALID_ARG;
  p.stall_iter = take_stall_request();
  return launch_loss_backward(p, ctx, stream);
}

bool sizes_ok(const Sizes& z) { return dim_ok(z.M) && dim_ok(z.N) && dim_ok(z.K) && (z.N > 0 || z.M == 0); }

int cross_entropy_problem(LossProblem& p, const Sizes& z, const void* targets, int target_dtype, float scale, float smoothing,
                          float z_loss) {
  if (!sizes_ok(z) || !index_code_ok(target_dtype) || !scale_ok(scale) || !(smoothing >= 0.0f) ||
      !(smoothing <= 1.0f) || !std::isfinite(z_loss))
    return GEMM_ERR_INVALID_ARG;
  p = {};
  p.targets = targets;
  p.target64 = target_dtype == GEMM_INDEX_I64;
  p.scale = scale;
  p.smoothing = smoothing;
  p.z_coef = z_loss;
  return z.M > 0 ? check_vector(targets, index_size(target_dtype)) : GEMM_OK;
}

int distill_problem(LossProblem& p, const Sizes& z, const void* teacher, int teacher_dtype, const void* ids, int id_dtype,
                    int64_t ld_teacher, int64_t ld_ids, float temperature) {
  if (!sizes_ok(z) || z.top < 1 || z.top > GEMM_MAX_TOP || !float_code_ok(teacher_dtype) || !index_code_ok(id_dtype) ||
      !(temperature > 0.0f) || !std::isfinite(temperature) || !scale_ok(1.0f / temperature))
    return GEMM_ERR_INVALID_ARG;
  p = {};
  p.teacher = teacher;
  p.teacher_f32 = teacher_dtype == GEMM_DTYPE_F32;
  p.ids = ids;
  p.ids64 = id_dtype == GEMM_INDEX_I64;
  p.ld_teacher = static_cast<uint64_t>(ld_teacher);
  p.ld_ids = static_cast<uint64_t>(ld_ids);
  p.scale = 1.0f / temperature;
  if (z.M == 0) return GEMM_OK;
  const int rc = check_matrix(teacher, z.top, ld_teacher, float_size(teacher_dtype), 1);
  return rc != GEMM_OK ? rc : check_matrix(ids, z.top, ld_ids, index_size(id_dtype), 1);
}

}  // namespace

extern "C" {

int64_t gemm_bf16_cross_entropy_workspace_bytes(int64_t M, int64_t N, int64_t K, int grad) {
  return workspace_bytes({M, N, K, 0}, grad);
}

int gemm_bf16_cross_entropy(const void* A, const void* B, const void* targets, float* loss, float* lse, int64_t M, int64_t N,
                            int64_t K, int64_t lda, int64_t ldb, int target_dtype, float scale, float smoothing,
                            float z_loss, void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
  const Sizes z = {M, N, K, 0};
  LossProblem p;
  const int rc = cross_entropy_problem(p, z, targets, target_dtype, scale, smoothing, z_loss);
  if (rc != GEMM_OK || M == 0) return rc;
  return forward(p, z, A, B, lda, ldb, loss, lse, workspace, workspace_bytes, stream);
}

int gemm_bf16_cross_entropy_grad(const float* dloss, const void* A, const void* B, const void* targets, const float* lse,
                                 void* dA, void* dB, int64_t M, int64_t N, int64_t K, int64_t inc_dloss, int64_t lda,
                                 int64_t ldb, int64_t ld_da, int64_t ld_db, int target_dtype, int da_dtype, int db_dtype,
                                 float scale, float smoothing, float z_loss, int accumulate, void* workspace,
                                 int64_t workspace_bytes, cudaStream_t stream) {
  const Sizes z = {M, N, K, 0};
  LossProblem p;
  const int rc = cross_entropy_problem(p, z, targets, target_dtype, scale, smoothing, z_loss);
  if (rc != GEMM_OK) return rc;
  return backward(p, z, dloss, inc_dloss, A, B, lse, dA, dB, lda, ldb, ld_da, ld_db, da_dtype, db_dtype, accumulate, workspace,
                  workspace_bytes, stream);
}

int64_t gemm_bf16_distill_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t top, int grad) {
  return top < 1 || top > GEMM_MAX_TOP ? static_cast<int64_t>(GEMM_ERR_INVALID_ARG) : workspace_bytes({M, N, K, top}, grad);
}

int gemm_bf16_distill(const void* A, const void* B, const void* teacher, const void* ids, float* loss, float* lse, int64_t M,
                      int64_t N, int64_t K, int64_t top, int64_t lda, int64_t ldb, int64_t ld_teacher, int64_t ld_ids,
                      int teacher_dtype, int id_dtype, float temperature, void* workspace, int64_t workspace_bytes,
                      cudaStream_t stream) {
  const Sizes z = {M, N, K, top};
  LossProblem p;
  const int rc = distill_problem(p, z, teacher, teacher_dtype, ids, id_dtype, ld_teacher, ld_ids, temperature);
  if (rc != GEMM_OK || M == 0) return rc;
  return forward(p, z, A, B, lda, ldb, loss, lse, workspace, workspace_bytes, stream);
}

int gemm_bf16_distill_grad(const float* dloss, const void* A, const void* B, const void* teacher, const void* ids,
                           const float* lse, void* dA, void* dB, int64_t M, int64_t N, int64_t K, int64_t top,
                           int64_t inc_dloss, int64_t lda, int64_t ldb, int64_t ld_teacher, int64_t ld_ids, int64_t ld_da,
                           int64_t ld_db, int teacher_dtype, int id_dtype, int da_dtype, int db_dtype, float temperature,
                           int accumulate, void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
  const Sizes z = {M, N, K, top};
  LossProblem p;
  const int rc = distill_problem(p, z, teacher, teacher_dtype, ids, id_dtype, ld_teacher, ld_ids, temperature);
  if (rc != GEMM_OK) return rc;
  return backward(p, z, dloss, inc_dloss, A, B, lse, dA, dB, lda, ldb, ld_da, ld_db, da_dtype, db_dtype, accumulate, workspace,
                  workspace_bytes, stream);
}

}  // extern "C"
