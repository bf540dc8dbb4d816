// Losses over a vocabulary: softmax cross entropy and distillation from a teacher's
// top logits, with their gradients, from rows A [M, K] and the vocabulary's matrix
// B [N, K].  z = scale A B^T is never stored:
//
//   forward    list     a teacher's entries of a row, sorted by token, with their
//                       probabilities (distillation only)
//              rows     which rows count, and a compact copy of them where some are left
//                       out (more than kInPlace rows only)
//              product  per tile the largest logit, the sum of exponentials and the
//                       entries' products (loss_kernel)
//              finish   the tiles' results joined, losses and lse
//   backward   list, rows as above, with each row's factors; then for each piece of the
//              vocabulary
//              product  g = dloss dloss/dz of the piece, bf16 (loss_kernel; up to kInPlace
//                       rows it also copies the rows that count, without the others)
//              products dA += g B[piece] in fp32, the reduction in parts, and
//                       dB[piece] (+)= g^T A (loss_product_kernel)
//              spread   dA's parts joined, its rows to where they belong, zeros to the
//                       others
//
// Every kernel but a call's first is launched while the one before it runs, and waits for
// it before it touches memory.  Two exceptions: in place, the first logits' kernel loads A and
// B, which no kernel of the call writes, before that wait; and the product that stores rows
// TMA cannot, the grouped one, is launched when the one before it has ended.  Only a piece's g
// is held: kPieceBytes, or a piece of kLeastPiece columns.
#include <cuda_bf16.h>

#include "gemm_gb300.h"
#include "grouped_host.h"
#include "loss_host.h"
#include "loss_kernels.cuh"
#include "loss_products.cuh"

namespace gb300 {
namespace {

constexpr uint32_t kInPlace = 256;             // up to so many rows are taken as they lie
// (4099 rows, 50021 tokens of width 1040: 572 us in one piece of 410 MB, 587 in two)
constexpr uint64_t kPieceBytes = 512ull << 20;
constexpr uint64_t kLeastPiece = 4096;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

constexpr uint64_t kMostWorkspace = 1ull << 62;

uint64_t up(uint64_t n, uint64_t m) { return (n + m - 1) / m * m; }

// Whether a list's entries are found by buckets.  Few rows have a tile or two a cluster, whose
// search hides behind the first loads, and a short list is searched in three loads.
bool bucketed(uint64_t M, uint64_t top) { return M > kInPlace && top > 8; }

// Up to so many rows, one tile's, g keeps two bf16 halves: the products are bound by what they
// read and write there, not by the MMAs of twice the rows (64 rows, 131072 tokens of width
// 4096: 640 us, 623 with one half; 128 rows: 613, 640).  Over thousands it would double them.
constexpr uint64_t kTwoHalves = 128;

struct Layout {
  uint64_t count, deal, index, pos, start, ids, prob, len, entropy, entry, part, part_sum, compact, row, piece, sums, sums_db;
  uint64_t ld_compact, ld_part, ld_sums, stride_sums, width, bytes;   // width: of a piece
  uint32_t parts, parts_db;                              // of dA's and dB's sums at most
  uint64_t lo, rows;                                     // where g's lower halves follow (0: none), rows of g
};

Layout layout_of(uint64_t M, uint64_t N, uint64_t K, uint64_t top, bool back) {
  Layout w = {};
  // (sizes that no memory holds: kNoWorkspace)
  const auto take = [&](uint64_t n, uint64_t size) {
    const uint64_t at = w.bytes;
    w.bytes = at > kMostWorkspace || n > (kMostWorkspace - at) / size ? kNoWorkspace : at + up(n * size, 256);
    return at;
  };
  w.count = take(1, 8);
  w.deal = back ? take(1, sizeof(LossDeal)) : 0;
  w.index = take(M, 4);
  w.pos = take(M, 4);
  if (top > 0) {
    w.ids = take(M * top, 4);
    w.prob = take(M * top, 4);
    w.len = take(M, 4);
    if (bucketed(M, top)) w.start = take((kLossBuckets + 1) * M, 2);
    w.entropy = take(M, 4);
  }
  w.ld_compact = up(K, 64);
  if (back) {
    w.lo = M <= kTwoHalves ? up(M, 64) : 0;
    w.rows = w.lo + M;
    w.compact = take(w.rows * w.ld_compact, 2);
    w.row = take(M, 16);
    uint64_t width = kPieceBytes / 2 / (w.rows > 0 ? w.rows : 1);
    width = width < kLeastPiece ? kLeastPiece : width;
    const uint64_t pieces = (N + width - 1) / width;
    w.width = up((N + pieces - 1) / (pieces > 0 ? pieces : 1), 256);
    w.piece = take(w.rows * w.width, 2);
    w.ld_sums = up(K, 32);
    w.stride_sums = w.rows * w.ld_sums;
    w.parts = loss_most_parts(w.rows, w.width < N ? w.width : N, K);
    w.sums = take(w.stride_sums * w.parts, 4);
    w.parts_db = M > kInPlace && w.width >= N ? loss_most_parts_db(M, N, K) : 1;
    if (w.parts_db > 1) w.sums_db = take(N * w.ld_sums * w.parts_db, 4);
  } else {
    if (M > kInPlace) w.compact = take(M * w.ld_compact, 2);
    w.entry = take(M * (top > 0 ? top : 1), 4);
    const uint64_t slots = loss_tiles(M, N, K).slots(M, N);
    w.ld_part = up(M, 32);
    w.part = take(slots * w.ld_part, 16);
    w.part_sum = take(slots * w.ld_part, 8);
  }
  return w;
}

__device__ __forceinline__ float warp_all(float v, bool largest) {
#pragma unroll
  for (uint32_t d = 16; d > 0; d /= 2) {
    const float x = __shfl_xor_sync(0xffffffffu, v, d);
    v = largest ? fmaxf(v, x) : v + x;
  }
  return v;
}
// The same over T threads, a warp or a block of 256; `slots` holds a value per warp.
template <uint32_t T>
__device__ __forceinline__ float all_of(float v, bool largest, float* slots) {
  v = warp_all(v, largest);
  if constexpr (T > 32) {
    __syncthreads();
    if ((threadIdx.x & 31u) == 0) slots[threadIdx.x / 32] = v;
    __syncthreads();
    v = slots[0];
    for (uint32_t i = 1; i < T / 32; ++i) v = largest ? fmaxf(v, slots[i]) : v + slots[i];
  }
  return v;
}

// T threads per row: p = softmax(teacher scale) over the entries that are there (id >= 0,
// logit not -Inf), sorted by id, and sum p log p, which is NaN where an id lies past the
// vocabulary or a logit is NaN or +Inf.  The scale is applied to differences of halves, which
// finite logits do not leave fp32 in: the type's lowest value is a logit like any other.  The place of an entry is the number of entries
// before it: top^2 / T comparisons from shared memory.  A warp has room for 128 entries.
constexpr uint32_t kWarpTop = 128;
struct ListArgs {
  const void* teacher;
  const void* ids;
  uint64_t ld_teacher, ld_ids;
  bool f32, ids64;
  uint32_t M, top, N;
  float scale;
  int32_t* out_ids;
  float* out_prob;
  uint32_t* len;
  uint16_t* start;             // (nullptr: not wanted)
  uint32_t bucket;
  float* entropy;
};
template <uint32_t T>
__global__ void __launch_bounds__(256) loss_list_kernel(const ListArgs a) {
  constexpr uint32_t kRows = 256 / T, kRoom = T == 32 ? kWarpTop : GEMM_MAX_TOP;
  __shared__ alignas(16) int32_t ids_of[kRows][kRoom];
  __shared__ float logits_of[kRows][kRoom];
  __shared__ float slots[8];
  grid_dependents_launch();
  grid_dependency_wait();
  const uint32_t me = threadIdx.x % T, top = a.top;
  const uint64_t r = blockIdx.x * static_cast<uint64_t>(kRows) + threadIdx.x / T;
  if (r >= a.M) return;   // (a whole warp; a block has one row)
  int32_t* const s_id = ids_of[threadIdx.x / T];
  float* const s_t = logits_of[threadIdx.x / T];
  float most = -INFINITY;
  bool wrong = false;
  uint32_t mine = 0;
  for (uint32_t i = me; i < top; i += T) {
    const int64_t id = loss_index_at(a.ids, a.ids64, r * a.ld_ids + i);
    const uint64_t at = r * a.ld_teacher + i;
    const float t = 0.5f * (a.f32 ? static_cast<const float*>(a.teacher)[at]
                                  : bf16_bits_to_f32(static_cast<const uint16_t*>(a.teacher)[at]));
    const bool there = id >= 0 && t != -INFINITY;
    wrong |= there && id >= a.N;
    s_id[i] = there ? static_cast<int32_t>(min(id, static_cast<int64_t>(0x7FFFFFFF))) : -1;
    s_t[i] = t;
    if (there) {
      most = fmaxf(most, t);
      ++mine;
    }
  }
  most = all_of<T>(most, true, slots);
  const auto behind = [&](uint32_t i) { return 2.0f * (a.scale * (s_t[i] - most)); };   // the largest, scaled
  float sum = 0.0f;
  for (uint32_t i = me; i < top; i += T) {
    if (s_id[i] >= 0) sum += expf(behind(i));
  }
  sum = all_of<T>(sum, false, slots);
  const float log_sum = logf(sum);
  float h = wrong ? NAN : 0.0f;
  __syncwarp();   // (T > 32: all_of's barriers)
  // the places of this thread's entries, four others at a time (absent ones come after all)
  constexpr uint32_t kMine = kRoom / T;
  uint32_t place[kMine] = {}, id_of[kMine];
#pragma unroll
  for (uint32_t j = 0; j < kMine; ++j) id_of[j] = me + j * T < top ? static_cast<uint32_t>(s_id[me + j * T]) : 0xFFFFFFFFu;
  for (uint32_t k = 0; k < top; k += 4) {
    const int4 x = *reinterpret_cast<const int4*>(s_id + k);
    const uint32_t other[4] = {static_cast<uint32_t>(x.x), static_cast<uint32_t>(x.y), static_cast<uint32_t>(x.z),
                               static_cast<uint32_t>(x.w)};
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e)
#pragma unroll
      for (uint32_t j = 0; j < kMine; ++j)
        place[j] += k + e < top && (other[e] < id_of[j] || (other[e] == id_of[j] && k + e < me + j * T)) ? 1u : 0u;
  }
#pragma unroll
  for (uint32_t j = 0; j < kMine; ++j) {
    const uint32_t i = me + j * T;
    if (static_cast<int32_t>(id_of[j]) < 0) continue;
    const float d = behind(i), p = expf(d) / sum;
    a.out_ids[r * top + place[j]] = static_cast<int32_t>(id_of[j]);
    a.out_prob[r * top + place[j]] = p;
    h += p == 0.0f ? 0.0f : p * (d - log_sum);
  }
  h = all_of<T>(h, false, slots);
  const uint32_t n = static_cast<uint32_t>(all_of<T>(static_cast<float>(mine), false, slots));
  if (me == 0) {
    a.len[r] = n;
    a.entropy[r] = h;
  }
  if (a.start == nullptr) return;
  // how many lie before each bucket, from the sorted ids
  const auto sync = [] {
    if constexpr (T > 32) __syncthreads();
    else __syncwarp();
  };
  sync();
#pragma unroll
  for (uint32_t j = 0; j < kMine; ++j)
    if (static_cast<int32_t>(id_of[j]) >= 0) s_id[place[j]] = static_cast<int32_t>(id_of[j]);
  sync();
  for (uint32_t b = me; b <= kLossBuckets; b += T) {
    const uint64_t border = static_cast<uint64_t>(b) * a.bucket;
    uint32_t lo = 0, hi = n;
    while (lo < hi && b < kLossBuckets) {
      const uint32_t mid = (lo + hi) / 2;
      if (static_cast<uint32_t>(s_id[mid]) < border) lo = mid + 1; else hi = mid;
    }
    a.start[b * static_cast<uint64_t>(a.M) + r] = static_cast<uint16_t>(b < kLossBuckets ? lo : n);
  }
}

// Which rows count: index[i] = the i-th of them, pos[r] its place (-1: left out), count =
// {0, their number}.  A forward pass's results for the rows left out, a backward pass's
// factors of the others; where there are some left out, the compact copy of the others, for
// a backward pass with zeros up to a multiple of 64 rows.
struct RowsArgs {
  uint32_t M, K, per;          // per: rows a block
  const void* targets;
  bool target64, back, always;  // always: the copy is wanted where no row is left out, too
  const uint32_t* len;         // (nullptr: targets)
  int32_t* count;
  uint32_t* index;
  int32_t* pos;
  float *loss, *lse;
  const uint16_t* A;
  uint64_t lda;
  uint16_t* compact;
  uint64_t ld_compact;
  LossFactors factors;
  float4* row;
  LossDeal* deal;              // the products' items (nullptr: not wanted)
  LossProductArgs products;
  uint32_t lt, clusters;
};

// Blocks of 256 threads, each for `per` rows of its own; to know their places, each counts
// all rows: at most 1024 blocks read M targets each, from L2.
__global__ void __launch_bounds__(256) loss_rows_kernel(const RowsArgs a) {
  __shared__ uint32_t sums[2][8], votes[8];
  grid_dependents_launch();
  grid_dependency_wait();
  const uint32_t lane = lane_idx(), warp = threadIdx.x / 32;
  const auto counts = [&](uint32_t r) {
    return a.len != nullptr ? a.len[r] > 0 : loss_index_at(a.targets, a.target64, r) >= 0;
  };
  const uint32_t first = blockIdx.x * a.per, last = min(first + a.per, a.M);
  uint32_t before = 0, all = 0;
  for (uint32_t r0 = 0; r0 < a.M; r0 += 2048) {   // (M < 2^31)
    bool in[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) in[i] = r0 + i * 256 + threadIdx.x < a.M && counts(r0 + i * 256 + threadIdx.x);
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      all += in[i] ? 1u : 0u;
      before += in[i] && r0 + i * 256 + threadIdx.x < first ? 1u : 0u;
    }
  }
  before = __reduce_add_sync(0xffffffffu, before);
  all = __reduce_add_sync(0xffffffffu, all);
  if (lane == 0) sums[0][warp] = before, sums[1][warp] = all;
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i) before += sums[0][i], all += sums[1][i];
  if (blockIdx.x == 0 && threadIdx.x == 0) a.count[0] = 0, a.count[1] = static_cast<int32_t>(all);
  const bool copy = a.always || all < a.M;
  for (uint32_t r0 = first; r0 < last; r0 += 256) {
    const uint32_t r = r0 + threadIdx.x;
    const bool in = r < last && counts(r);
    const uint32_t vote = __ballot_sync(0xffffffffu, in);
    if (lane == 0) votes[warp] = __popc(vote);
    __syncthreads();
    uint32_t lower = 0, turn = 0;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      lower += i < warp ? votes[i] : 0u;
      turn += votes[i];
    }
    const uint32_t at = before + lower + __popc(vote & ((1u << lane) - 1u));
    if (r < last) {
      a.pos[r] = in ? static_cast<int32_t>(at) : -1;
      if (in) {
        a.index[at] = r;
        if (a.back) a.row[at] = loss_row_factors(a.factors, a.targets, a.target64, r);
      } else if (!a.back) {
        a.loss[r] = a.lse[r] = 0.0f;
      }
    }
    before += turn;
    __syncthreads();
  }
  if (a.deal != nullptr && blockIdx.x == 0 && warp == 7) {
    const LossDeal d = loss_deal(a.products, all, a.lt, a.clusters);
    if (lane == 0) *a.deal = d;
  }
  if (!copy) return;
  // (a block's own writes of pos, which the last turn's barrier ordered before)
  const uint32_t whole = a.K / 8;
  for (uint32_t r = first + warp; r < last; r += 8) {
    const int32_t i = a.pos[r];
    if (i < 0) continue;
    const uint16_t* const from = a.A + r * a.lda;
    uint16_t* const to = a.compact + static_cast<uint32_t>(i) * a.ld_compact;
#pragma unroll 4
    for (uint32_t c = lane; c < whole; c += 32)
      reinterpret_cast<uint4*>(to)[c] = __ldg(reinterpret_cast<const uint4*>(from) + c);
    if (8 * whole + lane < a.K) to[8 * whole + lane] = from[8 * whole + lane];
  }
  if (a.back && blockIdx.x == gridDim.x - 1) {
    for (uint32_t i = all + warp; i < min((all + 63) / 64 * 64, a.M); i += 8)
      for (uint32_t c = lane; c < a.ld_compact / 8; c += 32)
        reinterpret_cast<uint4*>(a.compact + i * a.ld_compact)[c] = make_uint4(0, 0, 0, 0);
  }
}

struct FinishArgs {
  uint32_t M, N, slots, top;
  const uint32_t* count;       // (nullptr: in place)
  const uint32_t* index;
  const float2* part;
  const float* part_sum;
  uint64_t ld_part;
  float c, smoothing, z_coef;  // c: exp(z) = 2^(c a.b)
  const void* targets;
  bool target64;
  const float *entry, *prob, *entropy;   // entry: the entries' products with B
  const uint32_t* len;
  float *loss, *lse;
};

// A row's partial results: 2^top times `sum`, and the sum of its products with B.
struct RowPart {
  float top, sum, products;
};
// Joins N of them.
template <uint32_t N>
__device__ __forceinline__ void join(RowPart& r, const float2 (&x)[N], const float (&z)[N]) {
  float top = r.top;
#pragma unroll
  for (uint32_t k = 0; k < N; ++k) top = fmaxf(top, x[k].x);
  const float shift = top == -INFINITY ? 0.0f : top;   // (nothing yet: sums of 0)
  r.sum *= exp2_approx(r.top - shift);
#pragma unroll
  for (uint32_t k = 0; k < N; ++k) {
    r.sum += x[k].y * exp2_approx(x[k].x - shift);
    r.products += z[k];
  }
  r.top = top;
}
// Joins the warp's, in an order that does not depend on timing; every lane gets the result.
__device__ __forceinline__ void join_warp(RowPart& r) {
  const float top = warp_all(r.top, true), shift = top == -INFINITY ? 0.0f : top;
  r.sum = warp_all(r.sum * exp2_approx(r.top - shift), false);
  r.products = warp_all(r.products, false);
  r.top = top;
}

// Row r's loss and lse, by one warp.  lse - z of an entry is taken in base 2, its product with B
// subtracted from the largest in one fused multiply-add: what all of a row's logits share cancels
// before anything is rounded (8192 in every logit: losses off by 9e-4 where lse and z are rounded
// first, by 9e-6 so).  What is never below 0 is not let below it by roundings either.
__device__ __forceinline__ void finish_row(const FinishArgs& a, uint32_t r, RowPart p) {
  const uint32_t lane = lane_idx();
  if (a.slots == 0) p = RowPart{0.0f, static_cast<float>(a.N), 0.0f};   // no width: all logits are 0
  const float log_sum = log2f(p.sum), lse = kLn2 * (p.top + log_sum);
  const auto behind = [&](float product) { return kLn2 * (fmaf(-a.c, product, p.top) + log_sum); };
  float loss;
  bool counts;
  if (a.top > 0) {
    // sum p log p + sum p (lse - z)
    const uint32_t len = a.len[r];
    const uint64_t at = static_cast<uint64_t>(r) * a.top;
    float x = 0.0f;
    for (uint32_t e = lane; e < len; e += 32) x += a.prob[at + e] * behind(a.slots == 0 ? 0.0f : a.entry[at + e]);
    loss = a.entropy[r] + warp_all(x, false);
    if (loss < 0.0f) loss = 0.0f;
    counts = len > 0;
  } else {
    const int64_t t = loss_index_at(a.targets, a.target64, r);
    counts = t >= 0;
    loss = (1.0f - a.smoothing) * behind(a.slots != 0 && counts && t < a.N ? a.entry[r] : 0.0f);
    if (a.smoothing > 0.0f) loss += a.smoothing * behind(p.products / static_cast<float>(a.N));
    if (loss < 0.0f) loss = 0.0f;
    loss += a.z_coef * lse * lse;
    if (t >= a.N) loss = NAN;
  }
  if (lane == 0) {
    a.loss[r] = counts ? loss : 0.0f;
    a.lse[r] = counts ? lse : 0.0f;
  }
}

// In place: a warp per row, its partial results dealt to the lanes.
__global__ void __launch_bounds__(128) loss_finish_few_kernel(const FinishArgs a) {
  grid_dependency_wait();
  const uint32_t lane = lane_idx(), r = blockIdx.x * 4 + threadIdx.x / 32, parts = 2 * a.slots;
  if (r >= a.M) return;
  RowPart p = {-INFINITY, 0.0f, 0.0f};
  for (uint32_t p0 = lane; p0 < parts; p0 += 320) {
    float2 x[10];
    float z[10];
#pragma unroll
    for (uint32_t k = 0; k < 10; ++k) {
      const uint32_t i = p0 + 32 * k;
      x[k] = i < parts ? a.part[i * a.ld_part + r] : make_float2(-INFINITY, 0.0f);
      z[k] = i < parts && a.part_sum != nullptr ? a.part_sum[i * a.ld_part + r] : 0.0f;
    }
    join(p, x, z);
  }
  join_warp(p);
  finish_row(a, r, p);
}

// Rows that count, compact: 32 to a block, a lane per row while the 32 warps read its partial
// results (whole lines), a warp per row from there on.
__global__ void __launch_bounds__(1024) loss_finish_kernel(const FinishArgs a) {
  __shared__ float s_m[32][33], s_s[32][33], s_z[32][33];
  grid_dependency_wait();
  const uint32_t lane = lane_idx(), warp = threadIdx.x / 32, n = *a.count, parts = 2 * a.slots;
  if (blockIdx.x * 32 >= n) return;
  const uint32_t at = min(blockIdx.x * 32 + lane, n - 1);
  RowPart p = {-INFINITY, 0.0f, 0.0f};
  for (uint32_t p0 = warp; p0 < parts; p0 += 256) {
    float2 x[8];
    float z[8];
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) {
      const uint32_t i = p0 + 32 * k;
      x[k] = i < parts ? a.part[i * a.ld_part + at] : make_float2(-INFINITY, 0.0f);
      z[k] = i < parts && a.part_sum != nullptr ? a.part_sum[i * a.ld_part + at] : 0.0f;
    }
    join(p, x, z);
  }
  s_m[warp][lane] = p.top;
  s_s[warp][lane] = p.sum;
  s_z[warp][lane] = p.products;
  __syncthreads();
  const uint32_t i = blockIdx.x * 32 + warp;
  if (i >= n) return;
  p = RowPart{s_m[lane][warp], s_s[lane][warp], s_z[lane][warp]};
  join_warp(p);
  finish_row(a, a.index[i], p);
}

struct SpreadArgs {
  LossProductArgs products;    // by which the number of parts is found
  uint32_t clusters;
  const float* sums;
  uint64_t ld_sums, stride_sums;
  uint32_t M, lo;              // rows; where g's lower halves' sums follow (0: none)
  const int32_t* pos;          // (nullptr: in place, by targets or len)
  const void* targets;
  bool target64;
  const uint32_t* len;
  void* dA;                    // (nullptr: not wanted)
  uint64_t ldo;
  bool da_f32;
  // the matrix's rows dealt in parts
  const float* sums_db;        // (nullptr: never)
  uint64_t stride_db;
  uint32_t N;
  void* dB;
  uint64_t ld_db;
  bool db_f32, add_db;
};

// Four columns of a row from c on, rounded once (add: fp32, to what is there).
__device__ __forceinline__ void store_joined(void* out, uint64_t ld, bool f32, bool add, uint32_t K, uint64_t r, uint32_t c,
                                             float4 x) {
  const uint64_t size = f32 ? 4 : 2;
  const bool vec = ((reinterpret_cast<uintptr_t>(out) | (ld * size)) & (4 * size - 1)) == 0 && c + 4 <= K;
  if (!f32) {
    uint16_t* const to = static_cast<uint16_t*>(out) + r * ld + c;
    const uint2 h = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
    if (vec) {
      *reinterpret_cast<uint2*>(to) = h;
    } else {
      const uint32_t v[2] = {h.x, h.y};
      for (uint32_t e = 0; e < 4 && c + e < K; ++e) to[e] = static_cast<uint16_t>(v[e / 2] >> (16 * (e % 2)));
    }
    return;
  }
  float* const to = static_cast<float*>(out) + r * ld + c;
  if (vec) {
    if (add) {
      const float4 had = *reinterpret_cast<const float4*>(to);
      x = make_float4(had.x + x.x, had.y + x.y, had.z + x.z, had.w + x.w);
    }
    *reinterpret_cast<float4*>(to) = x;
  } else {
    const float v[4] = {x.x, x.y, x.z, x.w};
    for (uint32_t e = 0; e < 4 && c + e < K; ++e) to[e] = add ? to[e] + v[e] : v[e];
  }
}

// dA[r] = the parts' sums[pos[r]] in order, rounded once, or zeros, and dB (+)= its parts'
// sums; nothing where the products have stored it themselves.  A block per 128 columns
// of a row where there are many parts, which its warps share; a warp where there are few.
// DB: Matrix's rows may have been dealt in parts.
template <int CG, bool DB>
__global__ void __launch_bounds__(256) loss_spread_kernel(const SpreadArgs a) {
  __shared__ float4 joined[8][32];
  if (a.pos != nullptr) grid_dependency_wait();          // (in place the deal needs no earlier kernel's count)
  const uint32_t lane = lane_idx(), warp = threadIdx.x / 32;
  const uint32_t K = a.products.K;
  const LossDeal deal = loss_deal_of<CG>(a.products, a.clusters);
  const uint32_t M = a.dA == nullptr || deal.direct ? 0u : a.M, N = !DB || deal.parts_db == 1 ? 0u : a.N;
  if (M + N == 0) return;
  if (a.pos == nullptr) grid_dependency_wait();
  const uint32_t pieces = (K + 127) / 128;
  // `rows` rows; where(r): where row r's sums lie (nullptr: zeros)
  const auto join = [&](uint32_t rows, uint32_t parts, uint64_t stride, uint64_t lo, const auto& where, const auto& store) {
    const uint32_t share = parts > 4 ? 8u : 1u;          // warps a piece
    const uint64_t units = static_cast<uint64_t>(rows) * pieces, step = static_cast<uint64_t>(gridDim.x) * (8 / share);
    // (a block's warps take the same turns)
    for (uint64_t u0 = blockIdx.x * static_cast<uint64_t>(8 / share); u0 < units; u0 += step) {
      const uint64_t u = u0 + (share == 1 ? warp : 0u);
      const uint32_t r = static_cast<uint32_t>(u / pieces), c = static_cast<uint32_t>(u % pieces) * 128 + 4 * lane;
      const bool in = u < units && c < K;
      const float* from = in ? where(r) : nullptr;
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (from != nullptr) {
        from += c;
#pragma unroll 4
        for (uint32_t p = share == 1 ? 0u : warp; p < parts; p += share) {
          const float4 y = *reinterpret_cast<const float4*>(from + p * stride);
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
          if (lo != 0) {
            const float4 z = *reinterpret_cast<const float4*>(from + p * stride + lo);
            x.x += z.x, x.y += z.y, x.z += z.z, x.w += z.w;
          }
        }
      }
      if (share > 1) {
        joined[warp][lane] = x;
        __syncthreads();
        if (warp == 0) {
#pragma unroll
          for (uint32_t w = 1; w < 8; ++w) {
            const float4 y = joined[w][lane];
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
          }
        }
        __syncthreads();
        if (warp != 0) continue;
      }
      if (in) store(r, c, x);
    }
  };
  join(M, deal.parts, a.stride_sums, a.lo * a.ld_sums,
       [&](uint32_t r) -> const float* {
         int32_t i = -1;
         if (a.pos != nullptr) i = a.pos[r];
         else if (a.len != nullptr ? a.len[r] > 0 : loss_index_at(a.targets, a.target64, r) >= 0) i = static_cast<int32_t>(r);
         return i >= 0 ? a.sums + static_cast<uint32_t>(i) * a.ld_sums : nullptr;
       },
       [&](uint32_t r, uint32_t c, const float4& x) { store_joined(a.dA, a.ldo, a.da_f32, false, K, r, c, x); });
  if constexpr (DB)
    join(N, deal.parts_db, a.stride_db, 0,
         [&](uint32_t v) -> const float* { return a.sums_db + v * a.ld_sums; },
         [&](uint32_t v, uint32_t c, const float4& x) { store_joined(a.dB, a.ld_db, a.db_f32, a.add_db, K, v, c, x); });
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

int launch_list(const LossProblem& p, const Layout& w, uint8_t* ws, cudaStream_t stream) {
  ListArgs a = {};
  a.teacher = p.teacher;
  a.ids = p.ids;
  a.ld_teacher = p.ld_teacher;
  a.ld_ids = p.ld_ids;
  a.f32 = p.teacher_f32;
  a.ids64 = p.ids64;
  a.M = p.M;
  a.top = p.top;
  a.N = p.N;
  a.scale = p.scale;
  a.out_ids = reinterpret_cast<int32_t*>(ws + w.ids);
  a.out_prob = reinterpret_cast<float*>(ws + w.prob);
  a.len = reinterpret_cast<uint32_t*>(ws + w.len);
  a.entropy = reinterpret_cast<float*>(ws + w.entropy);
  a.start = bucketed(p.M, p.top) ? reinterpret_cast<uint16_t*>(ws + w.start) : nullptr;
  a.bucket = (p.N + kLossBuckets - 1) / kLossBuckets;
  return p.top <= kWarpTop ? launch(loss_list_kernel<32>, (p.M + 7) / 8, 256, false, stream, a)
                           : launch(loss_list_kernel<256>, p.M, 256, false, stream, a);
}

LossArgs logits_args(const LossProblem& p, const Layout& w, uint8_t* ws) {
  LossArgs a = {};
  a.M = p.M;
  a.N = p.N;
  a.K = p.K;
  a.c = p.scale * kLog2e;
  a.target = p.targets;
  a.target64 = p.target64 ? 1u : 0u;
  a.top = p.top;
  if (p.top > 0) {
    a.ids = reinterpret_cast<const int32_t*>(ws + w.ids);
    a.prob = reinterpret_cast<const float*>(ws + w.prob);
    a.len = reinterpret_cast<const uint32_t*>(ws + w.len);
    a.start = bucketed(p.M, p.top) ? reinterpret_cast<const uint16_t*>(ws + w.start) : nullptr;
    a.bucket = (p.N + kLossBuckets - 1) / kLossBuckets;
  }
  a.stall_iter = p.stall_iter;
  return a;
}

LossFactors factors_of(const LossProblem& p, const Layout& w, uint8_t* ws) {
  LossFactors f = {};
  f.dloss = p.dloss;
  f.inc_dloss = p.inc_dloss;
  f.lse = p.lse;
  f.entropy = p.top > 0 ? reinterpret_cast<const float*>(ws + w.entropy) : nullptr;
  f.scale = p.scale;
  f.smoothing = p.smoothing;
  f.z_coef = p.z_coef;
  f.N = p.N;
  return f;
}

// More than kInPlace rows: those that count, compact.
int launch_rows(const LossProblem& p, const Layout& w, uint8_t* ws, LossArgs& a, RowsArgs r, bool back, bool always,
                cudaStream_t stream) {
  r.M = p.M;
  r.K = p.K;
  r.per = p.M <= 16 * 1024 ? 16u : (p.M + 1023) / 1024;
  r.targets = p.targets;
  r.target64 = p.target64;
  r.back = back;
  r.always = always;
  r.len = a.len;
  r.count = reinterpret_cast<int32_t*>(ws + w.count);
  r.index = reinterpret_cast<uint32_t*>(ws + w.index);
  r.pos = reinterpret_cast<int32_t*>(ws + w.pos);
  r.loss = p.loss;
  r.lse = p.lse_out;
  r.A = static_cast<const uint16_t*>(p.A);
  r.lda = p.lda;
  r.compact = reinterpret_cast<uint16_t*>(ws + w.compact);
  r.ld_compact = w.ld_compact;
  r.factors = factors_of(p, w, ws);
  r.row = reinterpret_cast<float4*>(ws + w.row);
  a.count = reinterpret_cast<const uint32_t*>(r.count + 1);
  a.index = r.index;
  return launch(loss_rows_kernel, (p.M + r.per - 1) / r.per, 256, p.top > 0, stream, r);
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
    if ((rc = launch_rows(p, w, ws, a, RowsArgs{}, false, false, stream)) != GEMM_OK) return rc;
    o.compact = ws + w.compact;
    o.ld_compact = w.ld_compact;
    o.chained = true;
  }
  a.part = reinterpret_cast<float2*>(ws + w.part);
  a.part_sum = p.smoothing > 0.0f ? reinterpret_cast<float*>(ws + w.part_sum) : nullptr;
  a.ld_part = w.ld_part;
  a.entry = reinterpret_cast<float*>(ws + w.entry);
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
  f.c = a.c;
  f.smoothing = p.smoothing;
  f.z_coef = p.z_coef;
  f.targets = p.targets;
  f.target64 = p.target64;
  f.entry = a.entry;
  f.prob = a.prob;
  f.len = a.len;
  f.entropy = reinterpret_cast<const float*>(ws + w.entropy);
  f.loss = p.loss;
  f.lse = p.lse_out;
  const bool chained = p.K > 0 || o.chained;
  return f.count == nullptr ? launch(loss_finish_few_kernel, (p.M + 3) / 4, 128, chained, stream, f)
                            : launch(loss_finish_kernel, (p.M + 31) / 32, 1024, chained, stream, f);
}

int launch_loss_backward(const LossProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  const Layout w = layout_of(p.M, p.N, p.K, p.top, true);
  uint8_t* const ws = static_cast<uint8_t*>(p.workspace);
  int rc;
  if (p.top > 0 && (rc = launch_list(p, w, ws, stream)) != GEMM_OK) return rc;
  LossArgs a = logits_args(p, w, ws);
  uint16_t* const compact = reinterpret_cast<uint16_t*>(ws + w.compact);
  LossOperands o = {p.A, p.lda, compact, w.ld_compact, p.B, p.ldb, true};
  const bool in_place = p.M <= kInPlace;
  // rows that TMA cannot store, and bf16 to be added to: the grouped product
  const bool whole = p.dB != nullptr && loss_matrix_ok(p.dB, p.ld_db, p.K, p.db_f32, p.accumulate);
  LossProduct g = {};
  g.M = static_cast<uint32_t>(w.rows);
  g.K = p.K;
  g.width = static_cast<uint32_t>(w.width < p.N ? w.width : p.N);
  g.deal = in_place ? nullptr : reinterpret_cast<const LossDeal*>(ws + w.deal);
  g.g = ws + w.piece;
  g.ldg = w.width;
  g.ldb = p.ldb;
  g.compact = compact;
  g.ld_compact = w.ld_compact;
  g.A = in_place ? compact : p.A;
  g.lda = in_place ? w.ld_compact : p.lda;
  g.sums = p.dA != nullptr ? reinterpret_cast<float*>(ws + w.sums) : nullptr;
  g.ld_sums = w.ld_sums;
  g.stride_sums = w.stride_sums;
  g.most = w.parts;
  // one piece of more rows than are taken in place: dA needs no joining where none is left out
  if (!in_place && w.width >= p.N && p.dA != nullptr && loss_matrix_ok(p.dA, p.ld_da, p.K, p.da_f32, false)) {
    g.dA = p.dA;
    g.ld_da = p.ld_da;
    g.da_f32 = p.da_f32;
  }
  g.dB = whole ? p.dB : nullptr;
  g.ld_db = p.ld_db;
  g.db_f32 = p.db_f32;
  g.add_db = p.accumulate;
  if (whole && w.parts_db > 1) {
    g.sums_db = reinterpret_cast<float*>(ws + w.sums_db);
    g.stride_db = static_cast<uint64_t>(p.N) * w.ld_sums;
    g.most_db = w.parts_db;
  }
  LossProductPlan plan = {};
  if ((g.sums != nullptr || whole) && (rc = loss_product_plan(g, ctx, &plan)) != GEMM_OK) return rc;
  if (in_place) {
    o.compact = nullptr;
    o.chained = p.top > 0;
    a.factors = factors_of(p, w, ws);
    a.A = static_cast<const uint16_t*>(p.A);
    a.lda = p.lda;
    a.clean = compact;
    a.ld_clean = w.ld_compact;
    a.offsets = reinterpret_cast<int32_t*>(ws + w.count);
  } else {
    RowsArgs r = {};
    if (g.sums != nullptr || whole) {
      r.deal = reinterpret_cast<LossDeal*>(ws + w.deal);
      r.products = loss_product_args(g, plan, ctx);
      r.lt = 128 * plan.cg;
      r.clusters = plan.clusters;
    }
    if ((rc = launch_rows(p, w, ws, a, r, true, p.dB != nullptr && !whole, stream)) != GEMM_OK) return rc;
    a.row = reinterpret_cast<const float4*>(ws + w.row);
  }
  a.out = reinterpret_cast<uint16_t*>(ws + w.piece);
  a.ld_out = w.width;
  o.out_rows = w.rows;
  a.lo_row = static_cast<uint32_t>(w.lo);

  for (uint64_t v0 = 0; v0 < p.N; v0 += w.width) {
    const uint32_t n = static_cast<uint32_t>(p.N - v0 < w.width ? p.N - v0 : w.width);
    o.B = static_cast<const uint16_t*>(p.B) + v0 * p.ldb;
    a.N = n;
    a.first = static_cast<uint32_t>(v0);
    if ((rc = launch_loss_logits_backward(o, a, ctx, stream)) != GEMM_OK) return rc;
    a.stall_iter = 0xFFFFFFFFu;
    a.clean = nullptr;
    o.chained = true;
    g.n = n;
    g.B = o.B;
    void* const dB = p.dB != nullptr ? static_cast<uint8_t*>(p.dB) + v0 * p.ld_db * (p.db_f32 ? 4 : 2) : nullptr;
    if (g.sums != nullptr || whole) {
      g.dB = whole ? dB : nullptr;
      if ((rc = launch_loss_products(g, plan, ctx, stream)) != GEMM_OK) return rc;
      g.add_sums = true;
    }
    if (dB != nullptr && !whole) {
      GroupedProblem d = {};
      d.M = g.M;
      d.N = n;
      d.K = p.K;
      d.groups = 1;
      d.offsets = reinterpret_cast<const int32_t*>(ws + w.count);
      d.dD = g.g;
      d.ldd = w.width;
      d.A = compact;
      d.lda = w.ld_compact;
      d.out = dB;
      d.ldo = p.ld_db;
      d.out_f32 = p.db_f32;
      d.accumulate = p.accumulate;
      d.stall_iter = 0xFFFFFFFFu;
      if ((rc = launch_grouped_wgrad(d, ctx, stream)) != GEMM_OK) return rc;
    }
  }
  if (p.dA == nullptr && g.sums_db == nullptr) return GEMM_OK;
  g.n = g.width;
  SpreadArgs d = {};
  d.products = loss_product_args(g, plan, ctx);
  d.sums = g.sums;
  d.ld_sums = w.ld_sums;
  d.stride_sums = w.stride_sums;
  d.clusters = plan.clusters;
  d.M = p.M;
  d.lo = a.lo_row;
  d.pos = in_place ? nullptr : reinterpret_cast<const int32_t*>(ws + w.pos);
  d.targets = p.targets;
  d.target64 = p.target64;
  d.len = a.len;
  d.dA = p.dA;
  d.ldo = p.ld_da;
  d.da_f32 = p.da_f32;
  d.sums_db = g.sums_db;
  d.stride_db = g.stride_db;
  d.N = p.N;
  d.dB = p.dB;
  d.ld_db = p.ld_db;
  d.db_f32 = p.db_f32;
  d.add_db = p.accumulate;
  const uint64_t rows = (p.dA != nullptr ? p.M : 0ull) + (g.sums_db != nullptr ? p.N : 0ull);
  const uint64_t units = rows * ((p.K + 127) / 128), most = 16ull * static_cast<uint64_t>(ctx.num_sms);
  const unsigned blocks = static_cast<unsigned>(units < most ? units : most);
  if (g.sums_db != nullptr)
    return plan.cg == 2 ? launch(loss_spread_kernel<2, true>, blocks, 256, true, stream, d)
                        : launch(loss_spread_kernel<1, true>, blocks, 256, true, stream, d);
  return plan.cg == 2 ? launch(loss_spread_kernel<2, false>, blocks, 256, true, stream, d)
                      : launch(loss_spread_kernel<1, false>, blocks, 256, true, stream, d);
}

}  // namespace gb300
