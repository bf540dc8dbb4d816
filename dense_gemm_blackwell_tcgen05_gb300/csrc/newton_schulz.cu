// Newton-Schulz orthogonalisation of a batch of matrices:
//
//     X = G / (|G|_F + eps);  steps times:  P = X X^T,  X <- a X + (b P + c P^2) X
//
// on the smaller side m of each rows x cols matrix (P = X^T X and
// X <- a X + X (b P + c P^2) where rows > cols), as three products a step:
// the Gram matrix P, the polynomial Y = b P + c P P -- both symmetric, so only
// the tiles on and below the diagonal are computed -- and X' = a X + Y X.
// Every operand lies as the tensor cores can take it, so neither orientation
// is transposed.
//
// Precision.  The operands are fp16: at the same rate as bf16 their rounding
// is 8 times finer, and the range fits, because X is held scaled by a power of
// two that brings its entries near 1 and P and Y have norms of a few units.  A
// matrix whose X starts far below 1 has a power of its own, which the steps use up
// as they may have grown X (|G| = 1e-12 with eps = 1e-7, 1024 x 1024: without it
// 5.8e-2 of the result are lost to fp16's smallest numbers).
// X itself is held as hi + lo, two fp16 halves, and only the terms outside
// the products see lo.  Directions with small singular values grow by a = 3.4
// a step through a X, and so would its rounding errors.  Y's diagonal, about
// -2.7 once singular values are near 1 and then most of Y, stays in fp32 and
// is applied outside the product as well: (a + d_i) X_i + (Y - diag d) X.
// Relative error of five steps against 64 bits, random 256 x 256 / rank 8,
// 512 x 1024: bf16 operands 1.0e-2 / 0.34, fp16 1.3e-3 / 4.2e-2, X as hi + lo
// 1.6e-3 / 3.3e-4, and with the diagonal apart 8.6e-4 / 5.8e-4.
//
// Measured, five steps: 4096 x 4096 bf16 925 us (1.5 PFLOP/s, the power limit), 16 of
// 1024 x 2048 fp32 667 us (X's traffic), 2053 x 1040 142 us and 256 x 256 60 us (the
// latency of 15 dependent products and two launches before them).
#include <cmath>

#include "launch_grouped.cuh"

namespace gb300 {
namespace {

constexpr uint32_t kSegment = 1024;      // columns a warp takes at a time
constexpr uint32_t kMaxPartials = 1024;  // partial sums per matrix

// Sum of squares of a lane's share of columns col .. of a row segment, each times
// `factor`: four consecutive columns out of each 128; and the largest magnitude seen.
// QUADS: as one load (rows of whole quadruples).  All loads come before the first use.
template <class T, bool QUADS>
__device__ __forceinline__ float segment_square_sum(const T* row, uint32_t col, uint32_t cols, float factor,
                                                    float& top) {
  constexpr uint32_t kN = kSegment / 128;
  float sum = 0.0f;
  const auto add = [&](float x, float y, float z, float w) {
    top = fmaxf(fmaxf(top, fmaxf(fabsf(x), fabsf(y))), fmaxf(fabsf(z), fabsf(w)));
    x *= factor, y *= factor, z *= factor, w *= factor;
    sum += x * x + y * y + (z * z + w * w);
  };
  row += col;
  if constexpr (QUADS) {
    using P = std::conditional_t<sizeof(T) == 4, float4, uint2>;
    P x[kN];
#pragma unroll
    for (uint32_t i = 0; i < kN; ++i) x[i] = col + i * 128 < cols ? __ldg(reinterpret_cast<const P*>(row + i * 128)) : P{};
#pragma unroll
    for (uint32_t i = 0; i < kN; ++i) {
      if constexpr (sizeof(T) == 4) add(x[i].x, x[i].y, x[i].z, x[i].w);
      else add(bf16_bits_to_f32(x[i].x & 0xFFFFu), bf16_bits_to_f32(x[i].x >> 16), bf16_bits_to_f32(x[i].y & 0xFFFFu),
               bf16_bits_to_f32(x[i].y >> 16));
    }
  } else {
    T x[4 * kN];
#pragma unroll
    for (uint32_t i = 0; i < 4 * kN; ++i) {
      const uint32_t at = i / 4 * 128 + i % 4;
      x[i] = col + at < cols ? __ldg(row + at) : T(0);
    }
#pragma unroll
    for (uint32_t i = 0; i < kN; ++i) {
      if constexpr (sizeof(T) == 4) add(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      else add(bf16_bits_to_f32(x[4 * i]), bf16_bits_to_f32(x[4 * i + 1]), bf16_bits_to_f32(x[4 * i + 2]),
               bf16_bits_to_f32(x[4 * i + 3]));
    }
  }
  return sum;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (uint32_t d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Sum over the 8 warps of the block, in a fixed order; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float* slots) {
  v = warp_sum(v);
  if ((threadIdx.x & 31u) == 0) slots[threadIdx.x / 32] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i) t += slots[i];
  return t;
}

// A sum of squares of any fp32 values: `sum` 2^(180 `range`), range -1, 0 or 1.  The
// sum stays between 2^-80 and 2^100 (or is 0, Inf or NaN), far from where squares
// and sums of 1024 such leave fp32.
constexpr float kSumMost = 0x1p100f, kSumLeast = 0x1p-80f;
__device__ __forceinline__ float range_factor(int range) { return range > 0 ? 0x1p-90f : range < 0 ? 0x1p90f : 1.0f; }

// partials[z][block]: sum of squares of this block's share of matrix z.  One
// warp takes a row segment of kSegment columns at a time.  A share whose squares
// leave the range is read once more with its values scaled.  A read of G: 16 of 1024
// x 2048 fp32 in 22.5 us, 6.0 TB/s.
template <class T>
__global__ void __launch_bounds__(256) ns_square_sum_kernel(const T* G, uint32_t rows, uint32_t cols, uint64_t ldg,
                                                            uint64_t stride_g, float2* partials) {
  __shared__ float slots[8];
  grid_dependents_launch();
  const uint32_t lane = lane_idx();
  const T* const g = G + blockIdx.y * stride_g;
  const bool vec = (reinterpret_cast<uintptr_t>(g) & (4 * sizeof(T) - 1)) == 0 && ldg % 4 == 0 && cols % 4 == 0;
  const uint32_t segs = (cols + kSegment - 1) / kSegment;
  const uint64_t units = static_cast<uint64_t>(rows) * segs;
  float sum = 0.0f, top = 0.0f;
  int range = 0;
  for (;;) {   // (every thread of the block takes the same turns)
    const float factor = range_factor(range);
    sum = 0.0f;
    for (uint64_t u = blockIdx.x * 8ull + threadIdx.x / 32; u < units; u += gridDim.x * 8ull) {
      const uint64_t r = u / segs;
      const uint32_t c0 = static_cast<uint32_t>(u - r * segs) * kSegment;
      const T* const row = g + r * ldg;
      sum += vec ? segment_square_sum<T, true>(row, c0 + lane * 4, cols, factor, top)
                 : segment_square_sum<T, false>(row, c0 + lane * 4, cols, factor, top);
    }
    const bool any = __syncthreads_or(top > 0.0f) != 0;   // (also: the slots are free again)
    sum = block_sum(sum, slots);
    if (range != 0) break;
    if (!(sum < kSumMost)) range = 1;
    else if (any && sum < kSumLeast) range = -1;
    else break;
  }
  if (threadIdx.x == 0) partials[blockIdx.y * kMaxPartials + blockIdx.x] = make_float2(sum, static_cast<float>(range));
}

// The sum of a matrix's `count` partial sums; every thread of the block gets it.
__device__ __forceinline__ float partial_sum(const float2* partials, uint32_t count, float* slots, int& range) {
  constexpr uint32_t kN = kMaxPartials / 256;
  float2 p[kN];
  bool high = false, mid = false, low = false;
#pragma unroll
  for (uint32_t i = 0; i < kN; ++i) {
    const uint32_t at = i * 256 + threadIdx.x;
    p[i] = at < count ? partials[at] : make_float2(0.0f, 0.0f);
    high |= p[i].y > 0.0f;
    mid |= p[i].y == 0.0f && p[i].x > 0.0f;
    low |= p[i].y < 0.0f;
  }
  range = 0;
  if (__syncthreads_or(high || low)) {   // (rare: every partial to the largest one's range)
    range = __syncthreads_or(high) ? 1 : __syncthreads_or(mid) ? 0 : -1;
#pragma unroll
    for (uint32_t i = 0; i < kN; ++i) {
      const int below = range - static_cast<int>(p[i].y);   // 2^-180 for each range
      if (below == 1) p[i].x = p[i].x * 0x1p-90f * 0x1p-90f;
      if (below == 2) p[i].x = 0.0f;
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (uint32_t i = 0; i < kN; ++i) sum += p[i].x;
  return block_sum(sum, slots);
}

// A lane's 16 pairs of elements of a block: columns col, col + 1 of every second
// row from row on (those outside the matrix read as 0).  PAIRS: as one load each.
// All loads come before the first use.
template <class T, bool PAIRS>
__device__ __forceinline__ void load_pairs(const T* g, uint64_t ld, uint32_t row, uint32_t col, uint32_t rows,
                                           uint32_t cols, float2 (&v)[16]) {
  g += row * ld + col;
  const bool in0 = col < cols, in1 = col + 1 < cols;
  if constexpr (PAIRS) {
    using P = std::conditional_t<sizeof(T) == 4, float2, uint32_t>;
    P x[16];
#pragma unroll
    for (uint32_t t = 0; t < 16; ++t, g += 2 * ld) x[t] = row + 2 * t < rows ? __ldg(reinterpret_cast<const P*>(g)) : P{};
#pragma unroll
    for (uint32_t t = 0; t < 16; ++t) {
      if constexpr (sizeof(T) == 4) v[t] = x[t];
      else v[t] = make_float2(bf16_bits_to_f32(x[t] & 0xFFFFu), bf16_bits_to_f32(x[t] >> 16));
    }
  } else {
    T x[16], y[16];
#pragma unroll
    for (uint32_t t = 0; t < 16; ++t, g += 2 * ld) {
      x[t] = in0 && row + 2 * t < rows ? __ldg(g) : T(0);
      y[t] = in1 && row + 2 * t < rows ? __ldg(g + 1) : T(0);
    }
#pragma unroll
    for (uint32_t t = 0; t < 16; ++t) {
      if constexpr (sizeof(T) == 4) v[t] = make_float2(x[t], y[t]);
      else v[t] = make_float2(bf16_bits_to_f32(x[t]), bf16_bits_to_f32(y[t]));
    }
  }
}

// A factor that fp32 need not hold: mantissa 2^(e0 + e1).
struct Factor {
  float first, second;   // mantissa 2^e0, 2^e1
  __device__ __forceinline__ float of(float x) const { return x * first * second; }
};

// X is lifted by this many powers of two at most (X = 2^-120 is far below any result of use).
constexpr int kMostLift = 120;

// The exponent of a positive normal number.
__device__ __forceinline__ int exponent(float x) { return (__float_as_int(x) >> 23) - 127; }

// scale 2^lift / (|G| + eps), scale a power of two, |G| = root 2^(90 range), which lies
// between 2^-149 and 2^144: |G| + eps as mantissa 2^e.  (In 64-bit arithmetic this made the
// kernel 12 % longer.)  lift: the norm of X = G / (|G| + eps) is at most 2^-lift, and
// above a quarter of it.
__device__ __forceinline__ Factor normalising_factor(float root, int range, float scale, float eps, int& lift) {
  lift = 0;
  if (root == 0.0f && eps > 0.0f) return {0.0f, 0.0f};   // (0 / eps)
  int unit = 90 * range;
  float norm = root + (range > 0 ? eps * 0x1p-90f : range < 0 ? eps * 0x1p90f : eps);   // times 2^unit
  if (range < 0 && eps > 0x1p30f) {                       // (|G| is below 2^-39)
    unit = 0;
    norm = eps;
  }
  if (!(norm > 0.0f) || isinf(norm)) return {scale / norm, 1.0f};   // Inf, NaN or 0
  const int e = exponent(norm) + unit;
  lift = min(max(e - (exponent(root) + 90 * range) - 1, 0), kMostLift);
  const float mantissa = __int_as_float((__float_as_int(norm) & 0x7FFFFF) | 0x3F800000);
  const int e0 = (lift - e) / 2;
  return {scale / mantissa * pow2(e0), pow2(lift - e - e0)};
}

// X = G * scale * 2^lift / (|G| + eps) as fp16 halves hi + lo, a 32 x 32 block at a time
// with a lane's elements as lo_block has them.  A read of G, a write of X: 16 of
// 1024 x 2048 fp32 in 39 us, 6.9 TB/s.
template <class T>
__global__ void __launch_bounds__(256) ns_normalise_kernel(const T* G, uint32_t rows, uint32_t cols, uint64_t ldg,
                                                           uint64_t stride_g, const float2* partials,
                                                           uint32_t num_partials, float scale, float eps,
                                                           __half* hi, __half* lo, uint64_t ldx, uint64_t stride_x,
                                                           int32_t* lifts) {
  __shared__ float slots[8];
  grid_dependents_launch();
  grid_dependency_wait();
  const uint32_t lane = lane_idx();
  int range, lift;
  const float root = sqrtf(partial_sum(partials + blockIdx.y * kMaxPartials, num_partials, slots, range));
  const Factor f = normalising_factor(root, range, scale, eps, lift);
  if (blockIdx.x == 0 && threadIdx.x == 0) lifts[blockIdx.y] = lift;
  const T* const g = G + blockIdx.y * stride_g;
  const bool vec = (reinterpret_cast<uintptr_t>(g) & (2 * sizeof(T) - 1)) == 0 && ldg % 2 == 0;
  const uint32_t across = (cols + 31) / 32;
  const uint64_t units = static_cast<uint64_t>((rows + 31) / 32) * across;
  for (uint64_t u = blockIdx.x * 8ull + threadIdx.x / 32; u < units; u += gridDim.x * 8ull) {
    const uint32_t rb = static_cast<uint32_t>(u / across);
    const uint32_t c = (static_cast<uint32_t>(u) - rb * across) * 32 + (lane & ~1u), r = rb * 32 + (lane & 1u);
    float2 v[16];
    if (vec && (c & ~31u) + 32 <= cols) load_pairs<T, true>(g, ldg, r, c, rows, cols, v);
    else load_pairs<T, false>(g, ldg, r, c, rows, cols, v);
    uint32_t low[16];
#pragma unroll
    for (uint32_t t = 0; t < 16; ++t) {
      const float x = f.of(v[t].x), y = f.of(v[t].y);
      const uint32_t h = pack_f16x2(x, y);
      const float2 got = __half22float2(*reinterpret_cast<const __half2*>(&h));
      low[t] = pack_f16x2(x - got.x, y - got.y);
      // the pitch is even: two columns from c < ldx fit
      if (r + 2 * t < rows && c < ldx)
        *reinterpret_cast<uint32_t*>(hi + blockIdx.y * stride_x + (r + 2 * t) * ldx + c) = h;
    }
    uint4* const l = reinterpret_cast<uint4*>(lo + lo_block(blockIdx.y, rb * 32, c, rows, cols)) + lane;
#pragma unroll
    for (uint32_t p = 0; p < 4; ++p) l[32 * p] = make_uint4(low[4 * p], low[4 * p + 1], low[4 * p + 2], low[4 * p + 3]);
  }
}

uint64_t round_up(uint64_t x, uint64_t a) { return (x + a - 1) / a * a; }

// Where the parts of the workspace start, in bytes.
struct Layout {
  uint64_t ldx, stride_x, ldp, stride_p;   // elements
  uint64_t hi[2], lo[2], gram, poly, diag, lift, partials, bytes;
};

Layout layout_of(uint64_t batch, uint64_t rows, uint64_t cols) {
  Layout w;
  const uint64_t m = rows < cols ? rows : cols;
  w.ldx = round_up(cols, 64);   // rows on whole lines: no store leaves a part of a sector
  w.stride_x = rows * w.ldx;
  w.ldp = round_up(m, 64);
  w.stride_p = m * w.ldp;
  uint64_t at = 0;
  const auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  for (int i = 0; i < 2; ++i) {
    w.hi[i] = take(batch * w.stride_x * 2);
    w.lo[i] = take(batch * round_up(rows, 32) * round_up(cols, 32) * 2);
  }
  w.gram = take(batch * w.stride_p * 2);
  w.poly = take(batch * w.stride_p * 2);
  w.diag = take(batch * m * 4);
  w.lift = take(batch * 4);
  w.partials = take(batch * kMaxPartials * sizeof(float2));
  w.bytes = at;
  return w;
}

int last_launch() {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return GEMM_OK;
  note_cuda_error(e);
  return GEMM_ERR_LAUNCH;
}

// hi + lo of the normalised matrices into the workspace.
template <class T>
int normalise(const NewtonSchulzProblem& p, const Layout& w, float scale, const LaunchCtx& ctx, cudaStream_t stream) {
  uint8_t* const ws = static_cast<uint8_t*>(p.workspace);
  const uint64_t share = ceil_div_u64(8ull * static_cast<uint64_t>(ctx.num_sms), p.batch);
  const auto blocks_of = [&](uint64_t units) {   // eight warps a block, one unit a warp at a time
    const uint64_t b = ceil_div_u64(units, 8), most = share < kMaxPartials ? share : kMaxPartials;
    return b < most ? b : most;
  };
  const uint64_t blocks = blocks_of(static_cast<uint64_t>(p.rows) * ceil_div_u64(p.cols, kSegment));
  float2* const partials = reinterpret_cast<float2*>(ws + w.partials);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), p.batch);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 0;
  const T* const g = static_cast<const T*>(p.G);
  if (cudaLaunchKernelEx(&cfg, ns_square_sum_kernel<T>, g, p.rows, p.cols, p.ldg, p.stride_g, partials) != cudaSuccess)
    return last_launch();
  cfg.numAttrs = 1;
  cfg.gridDim.x = static_cast<unsigned>(blocks_of(ceil_div_u64(p.rows, 32) * ceil_div_u64(p.cols, 32)));
  cudaLaunchKernelEx(&cfg, ns_normalise_kernel<T>, g, p.rows, p.cols, p.ldg, p.stride_g,
                     static_cast<const float2*>(partials), static_cast<uint32_t>(blocks), scale, p.eps,
                     reinterpret_cast<__half*>(ws + w.hi[0]), reinterpret_cast<__half*>(ws + w.lo[0]), w.ldx,
                     w.stride_x, reinterpret_cast<int32_t*>(ws + w.lift));
  return last_launch();
}

// Time of a product, us: rounds of tiles over the CTAs or pairs that run at once,
// each as long as its kt stages of 64 k or its epilogue, whichever is longer (the
// shorter one is seen once).  A stage is bound by its loads: 24, 32 and 32 KB into
// each SM at 64 bytes a clock are 0.20, 0.27 and 0.27 us, and X and X' use the same
// way.  Fitted to 1500 measured chains (101 sizes: 1 to 32 matrices, sides of 64 to
// 8192; 14 choices of the three products' tiles): choosing each product's tiles by
// it is 0.2 % behind the best choice, the same tiles for all three 1.1 %.
struct TileCost {
  uint32_t lt, nt;                        // output columns and rows
  double stage, sym, apply, launch;
};
constexpr TileCost kNarrow = {128, 64, 0.26, 0.0, 2.3, 2.3};
constexpr TileCost kWide = {128, 128, 0.31, 1.2, 3.9, 1.6};
constexpr TileCost kPair = {256, 256, 0.42, 3.0, 6.5, 0.0};   // (less than the others' by this fit)

double time_of(const TileCost& c, uint64_t tiles, uint32_t K, double epilogue, const LaunchCtx& ctx) {
  const uint64_t clusters = static_cast<uint64_t>(ctx.num_sms) * 128 / c.lt;
  const double load = static_cast<double>(ceil_div_u64(K, 64)) * c.stage;
  const double rounds = static_cast<double>(ceil_div_u64(tiles, clusters));
  return c.launch + (load > epilogue ? rounds * load + epilogue : rounds * epilogue + load);
}

// Tiles on and below the diagonal of m x m.
uint64_t sym_tiles(uint64_t lt, uint64_t nt, uint64_t m, uint64_t batch) {
  const uint64_t n = ceil_div_u64(m, lt);
  return lt / nt * (n * (n + 1) / 2) * batch;
}
uint64_t all_tiles(uint64_t lt, uint64_t nt, const GroupedArgs& a) {
  return ceil_div_u64(a.L, lt) * ceil_div_u64(a.C, nt) * a.groups;
}

// A symmetric product of P and Q, the same matrix; MN: by its columns.
template <bool MN>
int symmetric(const CUtensorMap& P, const CUtensorMap& Q, const GroupedArgs& a, const LaunchCtx& ctx,
              cudaStream_t stream) {
  const auto tiles = [&](const TileCost& c) { return sym_tiles(c.lt, c.nt, a.C, a.groups); };
  const auto time = [&](const TileCost& c) { return time_of(c, tiles(c), a.K, c.sym, ctx); };
  // Few tiles and a long reduction: a cluster of CTAs shares it.  Four cost 6.0 us more
  // a launch than one and save 0.17 us for each 64 k, two cost 4.6 and save 0.11.
  // Measured, five steps on a 64 x n matrix, us, one CTA / two / four: n = 1024:
  // 64 / 77 / 80, 2048: 82 / 87 / 84, 4096: 118 / 105 / 94, 8192: 191 / 140 / 111; four
  // matrices of 384 x 4096, whose tiles are too many for four: 194 / 179.
  const uint64_t fine = tiles(kNarrow);
  uint64_t room = 0;
  if (a.K >= 36 * 64 && fine <= static_cast<uint64_t>(ctx.num_sms / 4)) {
    if (const int rc = grouped_room<1, Op::Sym, MN, MN, 64, false, 4>(ctx, &room); rc != GEMM_OK) return rc;
    if (fine <= room) return launch_grouped<1, Op::Sym, MN, MN, 64, false, 4>(P, Q, a, fine, ctx, stream);
  }
  if (a.K >= 42 * 64 && fine <= static_cast<uint64_t>(ctx.num_sms / 2)) {
    if (const int rc = grouped_room<1, Op::Sym, MN, MN, 64, false, 2>(ctx, &room); rc != GEMM_OK) return rc;
    if (fine <= room) return launch_grouped<1, Op::Sym, MN, MN, 64, false, 2>(P, Q, a, fine, ctx, stream);
  }
  const double narrow = time(kNarrow), wide = time(kWide), pair = time(kPair);
  if (pair < wide && pair < narrow)
    return launch_grouped<2, Op::Sym, MN, MN, 256, false>(P, Q, a, tiles(kPair), ctx, stream);
  return wide < narrow ? launch_grouped<1, Op::Sym, MN, MN, 128, false>(P, Q, a, tiles(kWide), ctx, stream)
                       : launch_grouped<1, Op::Sym, MN, MN, 64, false>(P, Q, a, tiles(kNarrow), ctx, stream);
}

// X' from Y as P (K-major) and X as Q, or, MN, X as P (by its columns) and Y as Q.
template <Op OP, bool MN>
int apply(const CUtensorMap& P, const CUtensorMap& Q, const GroupedArgs& a, const LaunchCtx& ctx,
          cudaStream_t stream) {
  const auto tiles = [&](const TileCost& c) { return all_tiles(c.lt, c.nt, a); };
  const auto time = [&](const TileCost& c) { return time_of(c, tiles(c), a.K, c.apply, ctx); };
  const double narrow = time(kNarrow), wide = time(kWide), pair = time(kPair);
  if (pair < wide && pair < narrow)
    return launch_grouped<2, OP, MN, false, 256, false>(P, Q, a, tiles(kPair), ctx, stream);
  return wide < narrow ? launch_grouped<1, OP, MN, false, 128, false>(P, Q, a, tiles(kWide), ctx, stream)
                       : launch_grouped<1, OP, MN, false, 64, false>(P, Q, a, tiles(kNarrow), ctx, stream);
}

// A step's p(s) = a s + b s^3 + c s^5 makes singular values s <= 1 at most this many
// times larger: the largest |a + b u + c u^2| for u = s^2 <= 1 (1 if it is less).
double largest_growth(double a, double b, double c) {
  const auto at = [&](double u) { return std::fabs(a + b * u + c * u * u); };
  double most = std::fmax(1.0, std::fmax(at(0.0), at(1.0)));
  if (c != 0.0 && -b / (2.0 * c) > 0.0 && -b / (2.0 * c) < 1.0) most = std::fmax(most, at(-b / (2.0 * c)));
  return most;
}

int iterate(const NewtonSchulzProblem& p, const Layout& w, float scale, const LaunchCtx& ctx, cudaStream_t stream) {
  uint8_t* const ws = static_cast<uint8_t*>(p.workspace);
  const bool tall = p.rows > p.cols;
  const uint32_t m = tall ? p.cols : p.rows;
  __half* const gram = reinterpret_cast<__half*>(ws + w.gram);
  __half* const poly = reinterpret_cast<__half*>(ws + w.poly);

  GroupedArgs base = {};
  base.groups = p.batch;
  base.pdl = 1;
  base.status = ctx.status;
  base.timeout_ns = ctx.timeout_ns;
  base.stall_iter = 0xFFFFFFFFu;
  base.diag = reinterpret_cast<float*>(ws + w.diag);
  base.diag_n = m;
  base.lift = reinterpret_cast<const int32_t*>(ws + w.lift);

  // Y as an operand: K-major P or Q; P as both operands of its square.  The boxes
  // are those of every tile size.
  using Any = GroupedCfg<1, Op::Sym, false, false, 64, false>;
  constexpr uint32_t kP = p_box_rows<Any, false>(), kQ = q_box_rows<Any, false>(), kMN = p_box_rows<Any, true>();
  static_assert(kQ == GroupedCfg<1, Op::Sym, false, false, 128, false>::Q_BOX &&
                    kQ == GroupedCfg<2, Op::Sym, false, false, 256, false>::Q_BOX,
                "one tensor map for all tiles");
  CUtensorMap gramP, gramQ, polyP, polyQ;
  if (!operand_map(&gramP, gram, m, m, p.batch, w.ldp, w.stride_p, kP) ||
      !operand_map(&gramQ, gram, m, m, p.batch, w.ldp, w.stride_p, kQ) ||
      !operand_map(&polyP, poly, m, m, p.batch, w.ldp, w.stride_p, kP) ||
      !operand_map(&polyQ, poly, m, m, p.batch, w.ldp, w.stride_p, kQ))
    return GEMM_ERR_LAUNCH;
  CUtensorMap byRows[2], byRowsQ[2], byCols[2];   // X, of either buffer, by its rows (as P, as Q) and by its columns
  for (int i = 0; i < (p.steps > 1 ? 2 : 1); ++i) {
    const void* const hi = ws + w.hi[i];
    if ((!tall && !operand_map(&byRows[i], hi, p.cols, p.rows, p.batch, w.ldx, w.stride_x, kP)) ||
        !operand_map(&byRowsQ[i], hi, p.cols, p.rows, p.batch, w.ldx, w.stride_x, kQ) ||
        !operand_map(&byCols[i], hi, p.cols, p.rows, p.batch, w.ldx, w.stride_x, kMN))
      return GEMM_ERR_LAUNCH;
  }

  // Where |G| is far below eps (an idle expert's decayed momentum), X starts far below 1,
  // where fp16 halves hold little: it is then held times 2^lift too.  Singular values up
  // to 2^-lift can have grown to 2^(spent - lift) by a step, so that many powers remain.
  const double growth = std::log2(largest_growth(p.a, p.b, p.c));
  const auto spent = [&](int step) {
    const double e = std::ceil(growth * step);
    return e < kMostLift ? static_cast<int32_t>(e) : kMostLift;
  };
  for (int step = 0; step < p.steps; ++step) {
    const int cur = step & 1;
    base.spent = spent(step);
    base.spent_next = spent(step + 1);
    const bool last = step + 1 == p.steps;
    __half* const hi = reinterpret_cast<__half*>(ws + w.hi[cur]);
    const CUtensorMap &xK = byRows[cur], &xKq = byRowsQ[cur], &xMN = byCols[cur];

    GroupedArgs s = base;   // P = X X^T (or X^T X), the scale taken out
    s.L = s.C = m;
    s.K = tall ? p.rows : p.cols;
    s.out = gram;
    s.ldo = w.ldp;
    s.stride_o = w.stride_p;
    s.alpha = 1.0f / (scale * scale);
    int rc = tall ? symmetric<true>(xMN, xMN, s, ctx, stream) : symmetric<false>(xK, xKq, s, ctx, stream);
    if (rc != GEMM_OK) return rc;

    s.K = m;                // Y = b P + c P P, its diagonal apart
    s.out = poly;
    s.alpha = p.c;
    s.beta = p.b;
    s.R = gram;
    if ((rc = symmetric<false>(gramP, gramQ, s, ctx, stream)) != GEMM_OK) return rc;

    GroupedArgs t = base;   // X' = (a + d) X + Y X (or X (a + d) + X Y)
    t.L = p.cols;
    t.C = p.rows;
    t.K = m;
    t.alpha = p.a;
    t.x_hi = hi;
    t.x_lo = reinterpret_cast<const __half*>(ws + w.lo[cur]);
    t.ldx = w.ldx;
    t.stride_x = w.stride_x;
    if (last) {
      t.out = p.out;
      t.ldo = p.ldo;
      t.stride_o = p.stride_o;
      t.out_scale = 1.0f / scale;
      t.out_f32 = p.out_f32 ? 1u : 0u;
    } else {
      t.out = ws + w.hi[cur ^ 1];
      t.out_lo = reinterpret_cast<__half*>(ws + w.lo[cur ^ 1]);
      t.ldo = w.ldx;
      t.stride_o = w.stride_x;
    }
    if (last)
      rc = tall ? apply<Op::ApplyOut, false>(polyP, xKq, t, ctx, stream)
                : apply<Op::ApplyOut, true>(xMN, polyQ, t, ctx, stream);
    else
      rc = tall ? apply<Op::Apply, false>(polyP, xKq, t, ctx, stream)
                : apply<Op::Apply, true>(xMN, polyQ, t, ctx, stream);
    if (rc != GEMM_OK) return rc;
  }
  return GEMM_OK;
}

}  // namespace

uint64_t newton_schulz_bytes(uint64_t batch, uint64_t rows, uint64_t cols) {
  return layout_of(batch, rows, cols).bytes;
}

int launch_newton_schulz(const NewtonSchulzProblem& p, const LaunchCtx& ctx, cudaStream_t stream) {
  const Layout w = layout_of(p.batch, p.rows, p.cols);
  if (ceil_div_u64(p.cols, 128) * ceil_div_u64(p.rows, 64) * p.batch > 0x7FFFFFFFull) return GEMM_ERR_INVALID_ARG;
  // X is held times 2^k, near the square root of its longer side: its entries
  // are then near 1 once its singular values are, and the fp16 halves far
  // from their range's ends
  const uint32_t n = p.rows > p.cols ? p.rows : p.cols;
  const float scale = std::ldexp(1.0f, static_cast<int>(std::floor(0.5 * std::log2(static_cast<double>(n)))));
  const int rc = p.g_f32 ? normalise<float>(p, w, scale, ctx, stream) : normalise<uint16_t>(p, w, scale, ctx, stream);
  return rc != GEMM_OK ? rc : iterate(p, w, scale, ctx, stream);
}

}  // namespace gb300
