// Losses over a vocabulary: softmax cross entropy and distillation from a teacher's
// top logits, with their gradients, from rows A [M, K] and the vocabulary's matrix
// B [N, K].  z = scale A B^T is never stored:
//
//   forward    list     a teacher's entries of a row, sorted by token, with their
//                       probabilities (distillation only)
//              rows     which rows count, compact (more than kInPlace rows only)
//              gather   their rows of A, where some are left out
//              product  per tile the largest logit, the sum of exponentials and the
//                       entries' logits (loss_kernel)
//              finish   the tiles' results joined, losses and lse
//   backward   list, rows, gather as above, with each row's factors; then for each
//              piece of the vocabulary
//              product  g = dloss dloss/dz of the piece, bf16 (loss_kernel)
//              dA      += g B[piece]         in fp32, the reduction in parts
//              dB[piece] (+)= g^T A
//              spread   dA's parts joined, its rows to where they belong, zeros to the
//                       others
//
// Every kernel but a call's first is launched while the one before it runs, and waits for
// it before it touches memory.
// Only a piece's g is held: kPieceBytes, or a piece of kLeastPiece columns.
#include <cuda_bf16.h>

#include "gemm_gb300.h"
#include "grouped_host.h"
#include "loss_host.h"
#include "loss_kernels.cuh"

namespace gb300 {
namespace {

constexpr uint32_t kInPlace = 256;             // up to so many rows, a forward pass takes them as they lie
constexpr uint64_t kPieceBytes = 256ull << 20;
constexpr uint64_t kLeastPiece = 4096;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

uint64_t up(uint64_t n, uint64_t m) { return (n + m - 1) / m * m; }

struct Layout {
  uint64_t offs, index, pos, ids, prob, len, entropy, entry_z, part, part_sum, compact, row, piece, sums;
  uint64_t ld_compact, ld_part, ld_sums, stride_sums, width, bytes;   // width: of a piece
  LossRowsPlan plan;
};

Layout layout_of(uint64_t M, uint64_t N, uint64_t K, uint64_t top, bool back) {
  Layout w = {};
  const auto take = [&](uint64_t bytes) {
    const uint64_t at = w.bytes;
    w.bytes += up(bytes, 256);
    return at;
  };
  w.offs = take(16);
  w.index = take(4 * M);
  w.pos = take(4 * M);
  if (top > 0) {
    w.ids = take(4 * M * top);
    w.prob = take(4 * M * top);
    w.len = take(4 * M);
    w.entropy = take(4 * M);
  }
  w.ld_compact = up(K, 64);
  if (back) {
    w.compact = take(2 * M * w.ld_compact);
    w.row = take(16 * M);
    uint64_t width = kPieceBytes / 2 / (M > 0 ? M : 1);
    width = width < kLeastPiece ? kLeastPiece : width;
    const uint64_t pieces = (N + width - 1) / width;
    w.width = up((N + pieces - 1) / (pieces > 0 ? pieces : 1), 256);
    w.piece = take(2 * M * w.width);
    w.ld_sums = up(K, 32);
    w.stride_sums = M * w.ld_sums;
    w.plan = loss_rows_plan(M, w.width < N ? w.width : N, K);
    w.sums = take(4 * w.stride_sums * w.plan.split);
  } else {
    if (M > kInPlace) w.compact = take(2 * M * w.ld_compact);
    w.entry_z = take(4 * M * (top > 0 ? top : 1));
    const uint64_t slots = loss_tiles(M, N, K).slots(M, N);
    w.ld_part = up(M, 32);
    w.part = take(16 * slots * w.ld_part);
    w.part_sum = take(8 * slots * w.ld_part);
  }
  return w;
}

__device__ __forceinline__ int64_t index_at(const void* p, bool wide, uint64_t i) {
  return wide ? static_cast<const int64_t*>(p)[i] : static_cast<int64_t>(static_cast<const int32_t*>(p)[i]);
}

__device__ __forceinline__ float warp_all(float v, bool largest) {
#pragma unroll
  for (uint32_t d = 16; d > 0; d /= 2) {
    const float x = __shfl_xor_sync(0xffffffffu, v, d);
    v = largest ? fmaxf(v, x) : v + x;
  }
  return v;
}
// The same over a block; `slots` holds a value per warp.
__device__ __forceinline__ float block_all(float v, bool largest, float* slots) {
  v = warp_all(v, largest);
  __syncthreads();
  if ((threadIdx.x & 31u) == 0) slots[threadIdx.x / 32] = v;
  __syncthreads();
  v = slots[0];
  for (uint32_t i = 1; i < blockDim.x / 32; ++i) v = largest ? fmaxf(v, slots[i]) : v + slots[i];
  return v;
}

// A block per row: p = softmax(teacher scale) over the entries that are there (id >= 0,
// logit not -Inf), sorted by id, and sum p log p, which is NaN where an id lies past the
// vocabulary or a logit is NaN or +Inf.  The place of an entry is the number of entries
// before it: top^2 / threads comparisons from shared memory.
__global__ void __launch_bounds__(256) loss_list_kernel(const void* teacher, bool f32, uint64_t ld_teacher, const void* ids,
                                                        bool ids64, uint64_t ld_ids, uint32_t top, uint32_t N, float scale,
                                                        int32_t* out_ids, float* out_prob, uint32_t* len, float* entropy) {
  grid_dependents_launch();
  grid_dependency_wait();
  __shared__ int32_t s_id[GEMM_MAX_TOP];
  __shared__ float slots[8];
  const uint64_t r = blockIdx.x;
  const auto logit = [&](uint32_t i) {
    const uint64_t at = r * ld_teacher + i;
    return scale * (f32 ? static_cast<const float*>(teacher)[at]
                        : bf16_bits_to_f32(static_cast<const uint16_t*>(teacher)[at]));
  };
  float most = -INFINITY;
  bool wrong = false;
  uint32_t mine = 0;
  for (uint32_t i = threadIdx.x; i < top; i += blockDim.x) {
    const int64_t id = index_at(ids, ids64, r * ld_ids + i);
    const float t = logit(i);
    const bool there = id >= 0 && t != -INFINITY;
    wrong |= there && id >= N;
    s_id[i] = there ? static_cast<int32_t>(min(id, static_cast<int64_t>(0x7FFFFFFF))) : -1;
    if (there) {
      most = fmaxf(most, t);
      ++mine;
    }
  }
  most = block_all(most, true, slots);
  float sum = 0.0f;
  for (uint32_t i = threadIdx.x; i < top; i += blockDim.x)
    if (s_id[i] >= 0) sum += expf(logit(i) - most);
  sum = block_all(sum, false, slots);
  const float log_sum = logf(sum);
  float h = wrong ? NAN : 0.0f;
  for (uint32_t i = threadIdx.x; i < top; i += blockDim.x) {
    const int32_t id = s_id[i];
    if (id < 0) continue;
    uint32_t place = 0;
    for (uint32_t k = 0; k < top; ++k) place += s_id[k] >= 0 && (s_id[k] < id || (s_id[k] == id && k < i)) ? 1u : 0u;
    const float d = logit(i) - most, p = expf(d) / sum;
    out_ids[r * top + place] = id;
    out_prob[r * top + place] = p;
    h += p == 0.0f ? 0.0f : p * (d - log_sum);
  }
  h = block_all(h, false, slots);
  const uint32_t n = static_cast<uint32_t>(block_all(static_cast<float>(mine), false, slots));
  if (threadIdx.x == 0) {
    len[r] = n;
    entropy[r] = h;
  }
}

// One block: index[i] = the i-th row that counts, pos[r] its place (-1: left out), offs =
// {0, their number}; a forward pass's results for the rows left out.  8192 rows at a time,
// their flags on the way together.
__global__ void __launch_bounds__(1024) loss_rows_kernel(uint32_t M, const void* targets, bool target64, const uint32_t* len,
                                                         int32_t* offs, uint32_t* index, int32_t* pos, float* loss, float* lse) {
  __shared__ uint32_t votes[256], sums[8];
  grid_dependents_launch();
  grid_dependency_wait();
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x / 32;
  uint32_t before = 0;
  for (uint32_t r0 = 0; r0 < M; r0 += 8192) {   // (M < 2^31)
    bool in[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      const uint32_t r = r0 + i * 1024 + threadIdx.x;
      in[i] = r < M && (len != nullptr ? len[r] > 0 : index_at(targets, target64, r) >= 0);
    }
    uint32_t vote[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      vote[i] = __ballot_sync(0xffffffffu, in[i]);
      if (lane == 0) votes[i * 32 + warp] = __popc(vote[i]);
    }
    __syncthreads();
    // votes[w]: rows that count in the warps before w of this turn
    if (warp < 8) {
      const uint32_t n = votes[threadIdx.x];
      uint32_t incl = n;
#pragma unroll
      for (uint32_t d = 1; d < 32; d *= 2) {
        const uint32_t lower = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += lower;
      }
      votes[threadIdx.x] = incl - n;
      if (lane == 31) sums[warp] = incl;
    }
    __syncthreads();
    uint32_t base = before;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      const uint32_t r = r0 + i * 1024 + threadIdx.x;
      const uint32_t at = base + votes[i * 32 + warp] + __popc(vote[i] & ((1u << lane) - 1u));
      if (in[i]) index[at] = r;
      if (r < M) {
        pos[r] = in[i] ? static_cast<int32_t>(at) : -1;
        if (!in[i] && loss != nullptr) loss[r] = lse[r] = 0.0f;
      }
      base += sums[i];
    }
    before = base;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    offs[0] = 0;
    offs[1] = static_cast<int32_t>(before);
  }
}

// What a row's gradient is made of: g = gq exp(z - lse) - gs - gt (at the target; times p
// at a list's entries).
struct RowFactors {
  const float* dloss;
  uint64_t inc_dloss;
  const float* lse;
  const void* targets;
  bool target64;
  const float* entropy;        // a list's: NaN where it is wrong
  float scale, smoothing, z_coef;
  uint32_t N;
  float4* row;
};

// A warp per row that counts: its row of A (where some row is left out, or `back`) and,
// for a backward pass, its factors, and zeros up to a multiple of 64 rows.
__global__ void __launch_bounds__(256) loss_gather_kernel(const uint16_t* A, uint64_t lda, uint32_t M, uint32_t K,
                                                          const uint32_t* count, const uint32_t* index, uint16_t* out,
                                                          uint64_t ldo, bool back, const RowFactors f) {
  grid_dependents_launch();
  grid_dependency_wait();
  const uint32_t lane = lane_idx(), n = *count;
  const bool copy = back || n < M;
  for (uint32_t i = blockIdx.x * 8 + threadIdx.x / 32; i < (back ? min((n + 63) / 64 * 64, M) : n); i += gridDim.x * 8) {
    if (i >= n) {
      for (uint32_t c = lane; c < ldo / 8; c += 32) reinterpret_cast<uint4*>(out + i * ldo)[c] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint32_t r = index[i];
    if (copy) {
      const uint16_t* const from = A + r * lda;
      uint16_t* const to = out + i * ldo;
      const uint32_t whole = K / 8;
      for (uint32_t c = lane; c < whole; c += 32)
        reinterpret_cast<uint4*>(to)[c] = __ldg(reinterpret_cast<const uint4*>(from) + c);
      if (8 * whole + lane < K) to[8 * whole + lane] = from[8 * whole + lane];
    }
    if (back && lane == 0) {
      const float g = f.dloss[r * f.inc_dloss] * f.scale, l = f.lse[r];
      float gq = g * (1.0f + 2.0f * f.z_coef * l);
      const bool wrong = f.entropy != nullptr ? isnan(f.entropy[r]) : index_at(f.targets, f.target64, r) >= f.N;
      if (wrong) gq = NAN;
      f.row[i] = make_float4(l * kLog2e, gq, g * f.smoothing / static_cast<float>(f.N), g * (1.0f - f.smoothing));
    }
  }
}

struct FinishArgs {
  uint32_t M, N, slots, top;
  const uint32_t* count;       // (nullptr: all rows, in place)
  const uint32_t* index;
  const float2* part;
  const float* part_sum;
  uint64_t ld_part;
  float scale, smoothing, z_coef;
  const void* targets;
  bool target64;
  const float *entry_z, *prob, *entropy;
  const uint32_t* len;
  float *loss, *lse;
};

// A lane per row, the block's 32 warps share its partial results, joined in a fixed order.
__global__ void __launch_bounds__(1024) loss_finish_kernel(const FinishArgs a) {
  __shared__ float s_m[32][33], s_s[32][33], s_z[32][33];
  grid_dependency_wait();
  const uint32_t lane = lane_idx(), warp = threadIdx.x / 32;
  const uint32_t n = a.count != nullptr ? *a.count : a.M;
  const uint32_t i = blockIdx.x * 32 + lane;
  if (blockIdx.x * 32 >= n) return;
  const bool in = i < n;
  const uint32_t r = in ? (a.index != nullptr ? a.index[i] : i) : 0u;
  float m = -INFINITY, s = 0.0f, sum = 0.0f;
  const uint32_t parts = 2 * a.slots;
  // (a lane without a row takes the last one's, eight loads on their way at a time)
  const uint32_t at = in ? i : n - 1;
  for (uint32_t p0 = warp; p0 < parts; p0 += 256) {
    float2 x[8];
    float z[8];
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
      const uint32_t p = p0 + 32 * k;
      x[k] = p < parts ? a.part[p * a.ld_part + at] : make_float2(-INFINITY, 0.0f);
      z[k] = p < parts && a.part_sum != nullptr ? a.part_sum[p * a.ld_part + at] : 0.0f;
    }
    float top = m;
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) top = fmaxf(top, x[k].x);
    const float shift = top == -INFINITY ? 0.0f : top;
    s *= exp2_approx(m - shift);
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
      s += x[k].y * exp2_approx(x[k].x - shift);
      sum += z[k];
    }
    m = top;
  }
  s_m[warp][lane] = m;
  s_s[warp][lane] = s;
  s_z[warp][lane] = sum;
  __syncthreads();
  float top = -INFINITY;
  for (uint32_t w = 0; w < 32; ++w) top = fmaxf(top, s_m[w][lane]);
  const float shift = top == -INFINITY ? 0.0f : top;
  s = sum = 0.0f;
  for (uint32_t w = 0; w < 32; ++w) {
    s += s_s[w][lane] * exp2_approx(s_m[w][lane] - shift);
    sum += s_z[w][lane];
  }
  if (a.slots == 0) {   // no width: all logits are 0
    top = 0.0f;
    s = static_cast<float>(a.N);
  }
  const float lse = kLn2 * (top + log2f(s));
  float loss;
  bool counts;
  if (a.top > 0) {
    // sum p log p + sum p (lse - z), the entries dealt to the warps
    const uint32_t len = in ? a.len[r] : 0u;
    const uint64_t at = static_cast<uint64_t>(r) * a.top;
    float x = 0.0f;
    for (uint32_t e = warp; e < len; e += 32) x += a.prob[at + e] * (lse - (a.slots == 0 ? 0.0f : a.entry_z[at + e]));
    __syncthreads();
    s_z[warp][lane] = x;
    __syncthreads();
    loss = in ? a.entropy[r] : 0.0f;
    x = 0.0f;
    for (uint32_t w = 0; w < 32; ++w) x += s_z[w][lane];
    loss += x;
    counts = len > 0;
  } else {
    const int64_t t = in ? index_at(a.targets, a.target64, r) : -1;
    counts = t >= 0;
    const float z = a.slots != 0 && counts && t < a.N ? a.entry_z[r] : 0.0f;
    loss = (1.0f - a.smoothing) * (lse - z) + a.z_coef * lse * lse;
    if (a.smoothing > 0.0f) loss += a.smoothing * (lse - a.scale * sum / static_cast<float>(a.N));
    if (t >= a.N) loss = NAN;
  }
  if (warp == 0 && in) {
    a.loss[r] = counts ? loss : 0.0f;
    a.lse[r] = counts ? lse : 0.0f;
  }
}

// dA[r] = the parts' sums[pos[r]] in order, rounded once, or zeros.
template <class T>
__global__ void __launch_bounds__(256) loss_spread_kernel(const float* sums, uint64_t ld_sums, uint64_t stride_sums,
                                                          uint32_t split, const int32_t* pos, uint32_t M, uint32_t K, T* dA,
                                                          uint64_t ldo) {
  grid_dependency_wait();
  const uint32_t lane = lane_idx();
  const bool vec = ((reinterpret_cast<uintptr_t>(dA) | (ldo * sizeof(T))) & (4 * sizeof(T) - 1)) == 0;
  // a warp takes 128 columns of a row at a time: rows alone could be too few
  const uint32_t pieces = (K + 127) / 128;
  const uint64_t units = static_cast<uint64_t>(M) * pieces;
  for (uint64_t u = blockIdx.x * 8ull + threadIdx.x / 32; u < units; u += gridDim.x * 8ull) {
    const uint32_t r = static_cast<uint32_t>(u / pieces), c = static_cast<uint32_t>(u % pieces) * 128 + 4 * lane;
    const int32_t i = pos[r];
    T* const to = dA + r * ldo;
    if (c < K) {
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i >= 0) {
        const float* from = sums + static_cast<uint32_t>(i) * ld_sums + c;
#pragma unroll 8
        for (uint32_t p = 0; p < split; ++p, from += stride_sums) {
          const float4 y = *reinterpret_cast<const float4*>(from);
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
      }
      if constexpr (sizeof(T) == 2) {
        const uint2 h = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
        if (vec && c + 4 <= K) {
          *reinterpret_cast<uint2*>(to + c) = h;
        } else {
          const uint32_t v[2] = {h.x, h.y};
          for (uint32_t e = 0; e < 4 && c + e < K; ++e) to[c + e] = static_cast<T>(v[e / 2] >> (16 * (e % 2)));
        }
      } else {
        if (vec && c + 4 <= K) {
          *reinterpret_cast<float4*>(to + c) = x;
        } else {
          const float v[4] = {x.x, x.y, x.z, x.w};
          for (uint32_t e = 0; e < 4 && c + e < K; ++e) to[c + e] = v[e];
        }
      }
    }
  }
}

template <class... P, class... A>
int launch(void (*kern)(P...), unsigned grid, unsigned block, bool chained, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = chained ? 1 : 0;
  if (const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...); e != cudaSuccess) {
    note_cuda_error(e);
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

unsigned row_blocks(uint64_t rows, uint64_t per, int num_sms) {
  const uint64_t n = (rows + per - 1) / per, most = 16ull * static_cast<uint64_t>(num_sms);
  return static_cast<unsigned>(n < most ? n : most);
}

int launch_list(const LossProblem& p, const Layout& w, uint8_t* ws, cudaStream_t stream) {
  const uint32_t threads = p.top >= 256 ? 256u : (p.top + 31) / 32 * 32;
  return launch(loss_list_kernel, p.M, threads, false, stream, p.teacher, p.teacher_f32, p.ld_teacher, p.ids, p.ids64, p.ld_ids,
                p.top, p.N, p.scale, reinterpret_cast<int32_t*>(ws + w.ids), reinterpret_cast<float*>(ws + w.prob),
                reinterpret_cast<uint32_t*>(ws + w.len), reinterpret_cast<float*>(ws + w.entropy));
}

LossArgs logits_args(const LossProblem& p, const Layout& w, uint8_t* ws) {
  LossArgs a = {};
  a.M = p.M;
  a.N = p.N;
  a.K = p.K;
  a.c = p.scale * kLog2e;
  a.scale = p.scale;
  a.target = p.targets;
  a.target64 = p.target64 ? 1u : 0u;
  a.top = p.top;
  if (p.top > 0) {
    a.ids = reinterpret_cast<const int32_t*>(ws + w.ids);
    a.prob = reinterpret_cast<const float*>(ws + w.prob);
    a.len = reinterpret_cast<const uint32_t*>(ws + w.len);
  }
  a.stall_iter = p.stall_iter;
  return a;
}

}  // namespace

uint64_t loss_forward_bytes(uint64_t M, uint64_t N, uint64_t K, uint64_t top) { return layout_of(M, N, K, top, false).bytes; }
uint64_t loss_backward_bytes(uint64_t M, uint64_t N, uint64_t K, uint64_t top) { return layout_of(M, N, K, top, true).bytes; }

int launch_loss_forward(const LossProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  const Layout w = layout_of(p.M, p.N, p.K, p.top, false);
  uint8_t* const ws = static_cast<uint8_t*>(p.workspace);
  int rc;
  if (p.top > 0 && (rc = launch_list(p, w, ws, stream)) != GEMM_OK) return rc;
  LossArgs a = logits_args(p, w, ws);
  LossOperands o = {p.A, p.lda, nullptr, 0, p.B, p.ldb, p.top > 0};
  if (p.M > kInPlace) {
    int32_t* const offs = reinterpret_cast<int32_t*>(ws + w.offs);
    uint32_t* const index = reinterpret_cast<uint32_t*>(ws + w.index);
    if ((rc = launch(loss_rows_kernel, 1, 1024, p.top > 0, stream, p.M, p.targets, p.target64, a.len, offs, index,
                     reinterpret_cast<int32_t*>(ws + w.pos), p.loss, p.lse_out)) != GEMM_OK)
      return rc;
    a.count = reinterpret_cast<const uint32_t*>(offs + 1);
    a.index = index;
    o.compact = ws + w.compact;
    o.ld_compact = w.ld_compact;
    o.chained = true;
    if ((rc = launch(loss_gather_kernel, row_blocks(p.M, 8, ctx.num_sms), 256, true, stream, static_cast<const uint16_t*>(p.A),
                     p.lda, p.M, p.K, a.count, a.index, reinterpret_cast<uint16_t*>(ws + w.compact), w.ld_compact, false,
                     RowFactors{})) != GEMM_OK)
      return rc;
  }
  a.part = reinterpret_cast<float2*>(ws + w.part);
  a.part_sum = p.smoothing > 0.0f ? reinterpret_cast<float*>(ws + w.part_sum) : nullptr;
  a.ld_part = w.ld_part;
  a.entry_z = reinterpret_cast<float*>(ws + w.entry_z);
  uint32_t slots = 0;
  if (p.K > 0 && (rc = launch_loss_logits_forward(o, a, ctx, &slots, stream)) != GEMM_OK) return rc;
  FinishArgs f = {};
  f.M = p.M;
  f.N = p.N;
  f.slots = slots;
  f.top = p.top;
  f.count = a.count;
  f.index = a.index;
  f.part = a.part;
  f.part_sum = a.part_sum;
  f.ld_part = a.ld_part;
  f.scale = p.scale;
  f.smoothing = p.smoothing;
  f.z_coef = p.z_coef;
  f.targets = p.targets;
  f.target64 = p.target64;
  f.entry_z = a.entry_z;
  f.prob = a.prob;
  f.len = a.len;
  f.entropy = reinterpret_cast<const float*>(ws + w.entropy);
  f.loss = p.loss;
  f.lse = p.lse_out;
  return launch(loss_finish_kernel, (p.M + 31) / 32, 1024, p.K > 0 || o.chained, stream, f);
}

int launch_loss_backward(const LossProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  const Layout w = layout_of(p.M, p.N, p.K, p.top, true);
  uint8_t* const ws = static_cast<uint8_t*>(p.workspace);
  int rc;
  if (p.top > 0 && (rc = launch_list(p, w, ws, stream)) != GEMM_OK) return rc;
  LossArgs a = logits_args(p, w, ws);
  int32_t* const offs = reinterpret_cast<int32_t*>(ws + w.offs);
  uint32_t* const index = reinterpret_cast<uint32_t*>(ws + w.index);
  int32_t* const pos = reinterpret_cast<int32_t*>(ws + w.pos);
  uint16_t* const compact = reinterpret_cast<uint16_t*>(ws + w.compact);
  float* const sums = reinterpret_cast<float*>(ws + w.sums);
  if ((rc = launch(loss_rows_kernel, 1, 1024, p.top > 0, stream, p.M, p.targets, p.target64, a.len, offs, index, pos, nullptr,
                   nullptr)) != GEMM_OK)
    return rc;
  a.count = reinterpret_cast<const uint32_t*>(offs + 1);
  a.index = index;
  a.row = reinterpret_cast<const float4*>(ws + w.row);
  RowFactors f = {};
  f.dloss = p.dloss;
  f.inc_dloss = p.inc_dloss;
  f.lse = p.lse;
  f.targets = p.targets;
  f.target64 = p.target64;
  f.entropy = p.top > 0 ? reinterpret_cast<const float*>(ws + w.entropy) : nullptr;
  f.scale = p.scale;
  f.smoothing = p.smoothing;
  f.z_coef = p.z_coef;
  f.N = p.N;
  f.row = reinterpret_cast<float4*>(ws + w.row);
  if ((rc = launch(loss_gather_kernel, row_blocks(p.M, 8, ctx.num_sms), 256, true, stream, static_cast<const uint16_t*>(p.A),
                   p.lda, p.M, p.K, a.count, a.index, compact, w.ld_compact, true, f)) != GEMM_OK)
    return rc;
  const LossOperands all = {compact, w.ld_compact, compact, w.ld_compact, p.B, p.ldb, true};
  a.out = reinterpret_cast<uint16_t*>(ws + w.piece);
  a.ld_out = w.width;
  for (uint64_t v0 = 0; v0 < p.N; v0 += w.width) {
    const uint32_t n = static_cast<uint32_t>(p.N - v0 < w.width ? p.N - v0 : w.width);
    LossOperands o = all;
    o.B = static_cast<const uint16_t*>(p.B) + v0 * p.ldb;
    a.N = n;
    a.first = static_cast<uint32_t>(v0);
    if ((rc = launch_loss_logits_backward(o, a, ctx, stream)) != GEMM_OK) return rc;
    a.stall_iter = 0xFFFFFFFFu;
    LossProduct g = {};
    g.M = p.M;
    g.n = n;
    g.K = p.K;
    g.count = a.count;
    g.g = a.out;
    g.ldg = w.width;
    if (p.dA != nullptr) {
      g.X = o.B;
      g.ldx = p.ldb;
      g.out = sums;
      g.ldo = w.ld_sums;
      g.stride_o = w.stride_sums;
      g.out_f32 = true;
      g.add = v0 > 0;
      if ((rc = launch_loss_rows(g, w.plan, ctx, stream)) != GEMM_OK) return rc;
    }
    if (p.dB != nullptr) {
      g.X = compact;
      g.ldx = w.ld_compact;
      g.out = static_cast<uint8_t*>(p.dB) + v0 * p.ld_db * (p.db_f32 ? 4 : 2);
      g.ldo = p.ld_db;
      g.out_f32 = p.db_f32;
      g.add = p.accumulate;
      if (loss_matrix_ok(g.out, g.ldo, g.out_f32)) {
        if ((rc = launch_loss_matrix(g, ctx, stream)) != GEMM_OK) return rc;
      } else {
        // rows that start inside sectors: the grouped product, whose warps store along rows
        GroupedProblem d = {};
        d.M = p.M;
        d.N = n;
        d.K = p.K;
        d.groups = 1;
        d.offsets = offs;
        d.dD = a.out;
        d.ldd = w.width;
        d.A = compact;
        d.lda = w.ld_compact;
        d.out = g.out;
        d.ldo = p.ld_db;
        d.out_f32 = p.db_f32;
        d.accumulate = p.accumulate;
        d.stall_iter = 0xFFFFFFFFu;
        if ((rc = launch_grouped_wgrad(d, ctx, stream)) != GEMM_OK) return rc;
      }
    }
  }
  if (p.dA == nullptr) return GEMM_OK;
  const unsigned blocks = row_blocks(static_cast<uint64_t>(p.M) * ((p.K + 127) / 128), 8, ctx.num_sms);
  return p.da_f32 ? launch(loss_spread_kernel<float>, blocks, 256, true, stream, sums, w.ld_sums, w.stride_sums, w.plan.split,
                           pos, p.M, p.K, static_cast<float*>(p.dA), p.ld_da)
                  : launch(loss_spread_kernel<uint16_t>, blocks, 256, true, stream, sums, w.ld_sums, w.stride_sums,
                           w.plan.split, pos, p.M, p.K, static_cast<uint16_t*>(p.dA), p.ld_da);
}

}  // namespace gb300
