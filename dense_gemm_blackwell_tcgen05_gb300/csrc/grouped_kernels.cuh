// Grouped (ragged) and symmetric bf16/fp16 products on the tensor cores:
//
//     out[c, l] = sum_k P[l, k] Q[c, k]          fp32 accumulation in TMEM
//
// l runs along the contiguous dimension of the output and sits in the TMEM
// lanes (the MMA's M), c is the output row and sits in the TMEM columns (the
// MMA's N).  Each operand is K-major (its rows hold k contiguously) or
// MN-major (k runs over its rows), as it lies in memory: nothing is
// transposed beforehand.  The products built on it:
//
//   Op::Rows   rows sorted by group times the group's matrix.  c = the row,
//              so a group's ragged last tile costs what its rows need: the
//              MMA's N is those rows rounded up to 16 (32 for a CTA pair).
//                D[r, n]  = sum_k B[e][n, k] A[r, k]    P = B[e] K-major
//                dA[r, k] = sum_n B[e][n, k] dD[r, n]   P = B[e] MN-major
//   Op::Sum    each group's rows summed: dB[e][n, k] = sum_r A[r, k] dD[r, n],
//              P = A and Q = dD, both MN-major; the reduction is ragged.
//   Op::Sym    a symmetric product (P and Q the same matrix): only the tiles
//              on and below the diagonal are computed and each is stored
//              twice.  out = alpha P P^T, or b R + c R R^T with R symmetric.
//              With R the diagonal goes to fp32 values of its own, and zeros
//              to the matrix.
//   Op::Apply  X' = (a + d) X + B X (B symmetric without its diagonal d; P_MN),
//              or X (a + d) + X B (P K-major), X held as two halves hi + lo
//              of which hi feeds the tensor cores.  ApplyOut: the last one,
//              whose X' is rounded once to the result's type.
//   Op::SumAdd is Op::Sum added to what the output holds.
//   Op::SumLane, Op::SumLaneAdd are these with the operands' places exchanged:
//              P = dD and Q = A, l the output row and c along its contiguous
//              dimension, for 16-bit outputs whose rows hold whole pieces of 16
//              bytes: a lane then stores its row's elements in whole sectors.
//
// Persistent, warp-specialised: warp 0 lane 0 loads operand tiles of 64 k by
// TMA (128-byte swizzle) into a ring of stages, warp 1 lane 0 issues the MMAs
// into one of two TMEM accumulators, eight epilogue warps (two per lane
// quarter, alternating 32-column chunks) drain the other one straight to
// global memory: with l in the lanes, a warp's store covers 32 consecutive
// elements of an output row and needs no staging.  Op::Sum adds a warp that
// clears the operand rows of the next group at the end of a ragged reduction.
//
// What bounds it.  A stage of 64 k brings 32 KB into an SM, 512 clocks at 64 bytes
// each; a pair's tile of 256 x 256 has MMAs of 512 clocks for it, one CTA's of 128 x
// 128 of 256.  So large products run on pairs (32 groups of 4096 x 2048, 16384
// rows: 175 us, 1.57 PFLOP/s at the power limit), few rows a group read the weights
// and little else (64 groups of 2048 x 4096, 256 rows: 152 us, 7.1 TB/s), short
// reductions write (79 groups of 1536 x 4096 in bf16, 427 rows: 166 us, 6.0 TB/s),
// and Apply's X adds its traffic to the operands' (16 of 1024 x 2048: 64 us a
// product, 36 without X).  Stores move whole sectors wherever the pitch allows it.
#pragma once


#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "gemm_kernels.cuh"
#include "ptx_grouped.cuh"

namespace gb300 {

// Wait sites of the status word, after those that all kernels share.
enum GroupedWaitSite : uint32_t {
  kSiteTail = 11,           // tail warp waiting for a ragged reduction end
  kSiteSplit = 12,          // epilogue waiting for the other CTAs' parts of a reduction
};

enum class Op { Rows, Sum, SumAdd, SumLane, SumLaneAdd, Sym, Apply, ApplyOut };

// Groups a launch can hold: the offsets and the tile table sit in shared memory.
constexpr uint32_t kMaxGroups = 1024;
// Up to this many groups, they are sorted by size before they are dealt out.
constexpr uint32_t kMaxSortedGroups = 256;

struct GroupedArgs {
  uint32_t L;                  // output columns (lanes)
  uint32_t C;                  // output rows: in all (Rows), per group (Sum), per matrix (Sym, Apply)
  uint32_t K;                  // reduction length (Rows, Sym, Apply); rows in all (Sum)
  uint32_t groups;             // groups (Rows, Sum) or matrices (Sym, Apply)
  const int32_t* offsets;      // [groups + 1] first row of each group (Rows, Sum)
  void* out;                   // bf16 / fp32 (Rows, Sum), fp16 (Sym), fp16 hi or the result (Apply)
  uint64_t ldo, stride_o;      // pitch and matrix stride of `out` in elements
  uint32_t fmt;                // operand type: 1 bf16, 0 fp16
  uint32_t pdl;                // launched while its predecessor runs: wait for it before touching memory
  // Sym: out = alpha acc + beta R[l, c].   Apply: v = (alpha + diag) X + acc
  float alpha, beta;
  // Sym, Apply: X is held times 2^now, now = max(lift[matrix] - spent, 0), X' times 2^next,
  // from spent_next; P and, apart from the factor 2^(next - now) it brings to X', Y are not
  const int32_t* lift;
  int32_t spent, spent_next;
  float* diag;                 // [matrix][C]: written by Sym with R, read by Apply
  uint32_t diag_n;             // values of diag per matrix
  const __half* R;             // Sym: the symmetric matrix of the beta term (nullptr: none)
  const __half* x_hi;          // Apply: X as hi + lo: hi by rows (pitch ldx, stride stride_x),
  const __half* x_lo;          //   lo in blocks as the epilogue's lanes take it (lo_block)
  uint64_t ldx, stride_x;
  __half* out_lo;              // Apply: the lo half of X'
  float out_scale;             // ApplyOut: factor on the way out
  uint32_t out_f32;            // ApplyOut: fp32 (else bf16)
  unsigned long long* status;
  unsigned long long timeout_ns;
  uint32_t stall_iter;         // watchdog test hook (0xFFFFFFFF: none)
};

// One tile of work.  P rows l0.., Q rows c0.. of group / matrix z; Rows: Q's
// rows start at memory row row0 + c0; Sum: the reduction covers memory rows
// row0 .. row0 + k_len - 1.
struct __align__(16) TileItem {
  uint32_t z, l0, c0, live, row0, k_len;
  uint32_t mirror;   // Sym: store the tile's mirror image too
  uint32_t valid;    // 0: past the cluster's last tile
};

// A cluster's first tiles are worked out ahead by all threads at once; the
// division-heavy arithmetic (0.5 us of one thread's time) would otherwise
// stand between two tiles' MMAs.
constexpr uint32_t kAheadItems = 128;

// Columns [c0, c0 + live) of the tile as the MMA's N: CTA pairs take
// multiples of 32 (16 rows of Q from each CTA), one CTA multiples of 16.
template <int CG>
__device__ __forceinline__ uint32_t mma_n(uint32_t live) {
  constexpr uint32_t g = 16u * CG;
  return live == 0 ? g : (live + g - 1) / g * g;
}

// SPLIT: a cluster of that many CTAs shares each tile's reduction (one tile a
// cluster: the launcher splits only where there are clusters for all tiles).
template <int CG, Op OP, bool P_MN, bool Q_MN, uint32_t NT, bool OUT32, uint32_t SPLIT = 1>
struct GroupedCfg {
  static_assert(CG == 1 || CG == 2, "cta_group is 1 or 2");
  static constexpr uint32_t BK = 64;                     // k per stage: one 128-byte row
  static constexpr uint32_t LT = 128 * CG;               // lanes (output columns) per tile
  static constexpr uint32_t Q_ROWS = NT / CG;            // Q rows staged by one CTA
  static_assert(!Q_MN || Q_ROWS == 128 || (Q_ROWS == 64 && OP == Op::Sym), "an MN-major Q tile is 64-wide boxes");
  static_assert(Q_ROWS % 16 == 0 && Q_ROWS <= 256 && NT <= 256, "tile width");
  // rows per load of a K-major Q: ragged tiles load what they need, the others 64
  // rows at a time (Newton-Schulz products 1 % shorter than with 32)
  static constexpr uint32_t Q_BOX = OP == Op::Rows ? 32 : 64;
  static constexpr uint32_t P_BYTES = 128 * 128;
  static constexpr uint32_t Q_BYTES = Q_ROWS * 128;
  static constexpr uint32_t STAGE_BYTES = P_BYTES + Q_BYTES;
  static constexpr bool ADD = OP == Op::SumAdd || OP == Op::SumLaneAdd;   // out += instead of out =
  static constexpr bool LANE = OP == Op::SumLane || OP == Op::SumLaneAdd; // output rows in the lanes
  static constexpr bool SUM = OP == Op::Sum || LANE || ADD;
  static_assert(!LANE || !OUT32, "fp32 rows are stored as whole lines either way");
  static constexpr bool APPLY = OP == Op::Apply || OP == Op::ApplyOut;
  static constexpr bool TAIL = SUM;                      // a warp clears ragged reduction ends
  static constexpr uint32_t kEpiWarps = 8;
  static constexpr uint32_t kTailWarp = 2 + kEpiWarps;
  static constexpr uint32_t kThreads = 32 * (2 + kEpiWarps + (TAIL ? 1 : 0));
  // fp32 outputs: the tensor core adds each MMA to the accumulator with
  // truncation, a bias of about 1.1e-9 of the result per k (measured: 2e-6 at
  // 2048).  Every SEG_TILES stages (512 k, 5e-7) the epilogue takes the
  // accumulator over into registers, where the segments are added rounded to
  // nearest.  bf16 and fp16 outputs round far above that and take one segment.
  static constexpr uint32_t SEG_TILES = OUT32 ? 8u : 0xFFFFFFFFu;
  static constexpr uint32_t NCH = (NT + 63) / 64;        // 32-column chunks per epilogue warp
  static constexpr bool GROUPED = OP == Op::Rows || SUM;
  static_assert(SPLIT == 1 || (CG == 1 && (OP == Op::Rows || OP == Op::Sym) && NT == 64), "split reductions");
  static constexpr uint32_t kCluster = CG * SPLIT;       // CTAs a cluster
  // the other CTAs' sums, fp32, in the first one: for each of them a tile of
  // 128 lanes by NT columns, 16 bytes a lane after another
  static constexpr uint32_t PART_BYTES = 128 * NT * 4;
  static constexpr uint32_t SPLIT_BYTES = (SPLIT - 1) * PART_BYTES;
  static constexpr uint32_t ITEM_BYTES = kAheadItems * sizeof(TileItem);
  static constexpr uint32_t TABLE_BYTES = ITEM_BYTES + (GROUPED ? 2 * 4 * (kMaxGroups + 8) : 0);
  static constexpr uint32_t BAR_BYTES = 512;
  static constexpr uint32_t SMEM_LIMIT = 232448;
  static constexpr uint32_t ALIGN_SLACK = 1024;
  static constexpr uint32_t FIT = (SMEM_LIMIT - ALIGN_SLACK - BAR_BYTES - TABLE_BYTES - SPLIT_BYTES) / STAGE_BYTES;
  static constexpr uint32_t STAGES = FIT > 12 ? 12 : FIT;
  static constexpr uint32_t SMEM_BYTES = ALIGN_SLACK + STAGES * STAGE_BYTES + SPLIT_BYTES + BAR_BYTES + TABLE_BYTES;
  static_assert((3 * STAGES + 6) * 8 + 16 <= BAR_BYTES, "barrier area");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t ACC_COLS = 256;              // second accumulator's first column
};

// Shared-memory descriptor of an MN-major operand tile as SWIZZLE_128B boxes
// of 64 (mn) x 64 (k) elements leave it: k rows of 128 bytes in 8-row atoms
// (stride byte offset 1024 along k), 64-element blocks along mn one box
// (leading byte offset 8192) apart.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192 >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// idesc_bf16 with the operand type (fmt: 1 bf16, 0 fp16) and majors chosen.
__device__ __forceinline__ uint32_t idesc_f16(uint32_t M, uint32_t N, uint32_t fmt, bool p_mn, bool q_mn) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(p_mn) << 15) |
         (static_cast<uint32_t>(q_mn) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_dependents_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Tiles along the C columns of a Sum.  LANE: neighbours share 8 columns, so that
// each row can pass from one to the next at a boundary of its sectors.
template <class C, uint32_t NT>
__host__ __device__ __forceinline__ uint32_t sum_column_tiles(uint32_t columns) {
  if (!C::LANE) return (columns + NT - 1) / NT;
  return columns <= NT ? 1u : (columns - 8 + NT - 9) / (NT - 8);
}

// The wi-th tile of cluster c among G; false past the last.  Every role of
// every CTA walks the same sequence.  offs: the clamped offsets; tab: the
// first tile of each group and their number (Rows), or the groups in the order
// they are walked (Sum).
template <class C, int CG, Op OP, uint32_t NT>
__device__ __forceinline__ bool tile_item(const GroupedArgs& a, const uint32_t* offs, const uint32_t* tab,
                                          uint32_t c, uint32_t G, uint32_t wi, TileItem& w) {
  const uint32_t lt = (a.L + C::LT - 1) / C::LT;
  w.mirror = 0u;
  w.row0 = 0;
  w.k_len = a.K;
  if constexpr (OP == Op::Rows) {
    // Group by group, dealt round-robin: a group's matrix is read by all
    // clusters at about the same time.  (Groups by falling tile width, equal
    // tiles within a group and alternating directions measured the same on
    // uneven groups of 512 rows: what is left to even out is the power limit's.)
    const uint32_t x = c + wi * G;
    if (x >= tab[a.groups]) return false;
    uint32_t lo = 0, hi = a.groups;        // tab[lo] <= x < tab[hi]
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) / 2;
      if (tab[mid] <= x) lo = mid; else hi = mid;
    }
    w.z = lo;
    w.row0 = offs[lo];
    const uint32_t rows = offs[lo + 1] - w.row0;
    uint32_t cb, lb;
    tile_coords(x - tab[lo], (rows + NT - 1) / NT, lt, 8u, cb, lb);
    w.c0 = cb * NT;
    w.l0 = lb * C::LT;
    w.live = w.c0 < rows ? min(NT, rows - w.c0) : 0u;
    return true;
  } else if constexpr (C::SUM) {
    // Large and small groups in turn, so that a tile bound by its MMAs runs
    // beside one bound by its store; rounds in alternating directions.
    const uint32_t ct = sum_column_tiles<C, NT>(a.C), per = lt * ct;
    const uint32_t t = wi * G + ((wi & 1u) ? G - 1u - c : c);
    if (t >= per * a.groups) return false;
    // tiles of the groups 2p and 2p + 1 of the order alternate
    const uint32_t pr = t / (2 * per), r = t - pr * 2 * per;
    const bool both = 2 * pr + 1 < a.groups;
    const uint32_t g = both ? 2 * pr + (r & 1u) : 2 * pr;
    w.z = tab[g];
    w.row0 = offs[w.z];
    w.k_len = offs[w.z + 1] - w.row0;
    uint32_t cb, lb;
    tile_coords(both ? r / 2 : r, ct, lt, 8u, cb, lb);
    w.c0 = cb * (C::LANE ? NT - 8 : NT);
    w.l0 = lb * C::LT;
    w.live = min(NT, a.C - w.c0);
    return true;
  } else if constexpr (OP == Op::Sym) {
    // blocks of LT x LT on and below the diagonal, row by row, each as LT / NT
    // tiles; those on it are stored as they are, the others twice
    constexpr uint32_t kPer = C::LT / NT;
    static_assert(OP != Op::Sym || C::LT % NT == 0, "tiles divide the diagonal's blocks");
    const uint32_t per = kPer * (lt * (lt + 1) / 2);
    const uint32_t t = c + wi * G;
    if (t >= per * a.groups) return false;
    w.z = t / per;
    const uint32_t r = (t - w.z * per) / kPer;
    uint32_t i = static_cast<uint32_t>((sqrtf(8.0f * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > r) --i;
    while ((i + 1) * (i + 2) / 2 <= r) ++i;
    const uint32_t j = r - i * (i + 1) / 2;
    w.l0 = i * C::LT;
    w.c0 = j * C::LT + t % kPer * NT;      // (per is a multiple of kPer)
    w.live = w.c0 < a.C ? min(NT, a.C - w.c0) : 0u;
    w.mirror = i != j ? 1u : 0u;
    return true;
  } else {
    const uint32_t ct = (a.C + NT - 1) / NT, per = lt * ct;
    const uint32_t t = c + wi * G;
    if (t >= per * a.groups) return false;
    w.z = t / per;
    uint32_t cb, lb;
    tile_coords(t - w.z * per, ct, lt, 8u, cb, lb);
    w.c0 = cb * NT;
    w.l0 = lb * C::LT;
    w.live = min(NT, a.C - w.c0);
    return true;
  }
}

// Zeros in rows 0 .. rows - 1, columns 0 .. cols - 1 (cols <= 128) of a tile at
// `out`, by 256 threads, 16 bytes a thread where `vec` says that every row starts
// on such a boundary.
template <class T>
__device__ __forceinline__ void zero_tile(T* out, uint64_t ldo, uint32_t rows, uint32_t cols, bool vec,
                                          uint32_t thread) {
  constexpr uint32_t kPer = 16 / sizeof(T), kPieces = 128 / kPer;   // a row's elements a piece, pieces
  const uint32_t c = thread % kPieces * kPer;
  out += static_cast<uint64_t>(thread / kPieces) * ldo + c;
  for (uint32_t r = thread / kPieces; r < rows; r += 256 / kPieces, out += 256 / kPieces * ldo) {
    if (vec && c + kPer <= cols) {
      *reinterpret_cast<uint4*>(out) = make_uint4(0, 0, 0, 0);
    } else {
      for (uint32_t i = 0; i < kPer && c + i < cols; ++i) out[i] = T(0);
    }
  }
}

// Two neighbouring output columns of one row per lane instead of two rows of
// one column: lanes 2j and 2j + 1 hold columns 2j, 2j + 1 of rows 2i (v0) and
// 2i + 1 (v1); afterwards lane 2j has row 2i's pair, lane 2j + 1 row 2i + 1's.
__device__ __forceinline__ void pair_columns(float v0, float v1, uint32_t odd, float& x0, float& x1) {
  const float got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
  x0 = odd ? got : v0;
  x1 = odd ? v1 : got;
}

// The same with both rounded to bf16 first: one conversion, one exchange and one
// permutation of bytes for two elements.
__device__ __forceinline__ uint32_t pair_columns_bf16(float v0, float v1, uint32_t odd) {
  const uint32_t own = pack_bf16x2(v0, v1);   // rows 2i, 2i + 1 of this lane's column
  const uint32_t got = __shfl_xor_sync(0xffffffffu, own, 1);
  return __byte_perm(own, got, odd ? 0x3276u : 0x5410u);
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// fp16 bits plus, or minus, an fp32 value, in fp32.
__device__ __forceinline__ float f16_plus(uint32_t bits, float x) {
  float r;
  asm("add.f32.f16 %0, %1, %2;" : "=f"(r) : "h"(static_cast<uint16_t>(bits)), "f"(x));
  return r;
}
__device__ __forceinline__ float f16_minus(uint32_t bits, float x) {
  float r;
  asm("sub.f32.f16 %0, %1, %2;" : "=f"(r) : "h"(static_cast<uint16_t>(bits)), "f"(x));
  return r;
}

// First element of a 32 x 32 block of X's lo half, whose layout is private to the
// kernels that write and read it: blocks of 1024 along the rows; in a block piece p
// (of 4) of lane l is 8 elements at 256 p + 8 l: columns 2 (l / 2) and the next of
// rows 2 t + l % 2, t = 4 p .. 4 p + 3.  Four 16-byte accesses a lane, all in order.
__device__ __forceinline__ uint64_t lo_block(uint64_t z, uint32_t row, uint32_t col, uint32_t rows, uint32_t cols) {
  return ((z * ((rows + 31) / 32) + row / 32) * ((cols + 31) / 32) + col / 32) * 1024;
}

// wait_bounded for a thread that does not itself wait for the kernel's predecessor:
// the limit is for this kernel's loads, so when it runs out before the predecessor is
// known to have ended (`alone`), the thread waits for that and starts it anew.
// (Waiting for the predecessor beforehand makes every launch 0.1 to 0.2 us longer.)
__device__ __forceinline__ bool wait_bounded_alone(uint32_t bar, uint32_t parity, const Watchdog& wd, uint32_t site,
                                                   bool& alone) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = global_timer_ns();
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 31u) == 0) {
      if (*wd.abort_flag) return false;
      if (global_timer_ns() - t0 > wd.timeout_ns) {
        if (alone) {
          *wd.abort_flag = 1u;
          report_error(wd.status, kDevTimeout, site);
          return false;
        }
        grid_dependency_wait();
        alone = true;
        t0 = global_timer_ns();
      }
    }
  }
}

template <int CG, Op OP, bool P_MN, bool Q_MN, uint32_t NT, bool OUT32, uint32_t SPLIT = 1>
__global__ void __launch_bounds__(GroupedCfg<CG, OP, P_MN, Q_MN, NT, OUT32, SPLIT>::kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                   const GroupedArgs args) {
  using C = GroupedCfg<CG, OP, P_MN, Q_MN, NT, OUT32, SPLIT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  const uint32_t part0 = base + C::STAGES * C::STAGE_BYTES;
  const uint32_t bar0 = part0 + C::SPLIT_BYTES;
  const auto full_bar = [&](uint32_t s) { return bar0 + 8 * s; };
  const auto empty_bar = [&](uint32_t s) { return bar0 + 8 * (C::STAGES + s); };
  const auto tail_bar = [&](uint32_t s) { return bar0 + 8 * (2 * C::STAGES + s); };
  constexpr uint32_t kAccBar0 = 3 * C::STAGES;
  const auto accf_bar = [&](uint32_t b) { return bar0 + 8 * (kAccBar0 + b); };
  const auto acce_bar = [&](uint32_t b) { return bar0 + 8 * (kAccBar0 + 2 + b); };
  const uint32_t drain_bar = bar0 + 8 * (kAccBar0 + 4);
  const uint32_t part_bar = bar0 + 8 * (kAccBar0 + 5);   // SPLIT: the other CTAs' sums are here
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + (bar0 - base) + 8 * (kAccBar0 + 6));
  volatile uint32_t* const abort_flag = tmem_slot + 1;
  TileItem* const ahead = reinterpret_cast<TileItem*>(base_ptr + (bar0 - base) + C::BAR_BYTES);
  uint32_t* const offs = reinterpret_cast<uint32_t*>(ahead + kAheadItems);
  uint32_t* const tab = offs + kMaxGroups + 8;

  const uint32_t warp = warp_idx_sync();
  const uint32_t lane = lane_idx();
  const uint32_t rank = (CG == 2) ? cluster_cta_rank() : 0u;
  const bool leader = rank == 0;
  const uint32_t k_rank = SPLIT > 1 ? cluster_cta_rank() : 0u;   // which part of the reduction
  const uint32_t cluster_id = blockIdx.x / C::kCluster;
  const uint32_t G = gridDim.x / C::kCluster;
  const Watchdog wd{args.status, args.timeout_ns, abort_flag};

  // ---- set-up ------------------------------------------------------------------
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmP);
      tma_prefetch_desc(&tmQ);
      *abort_flag = 0u;
    }
    // arrivals: a full barrier gets the leader's expect_tx (its producer's, or
    // its tail warp's on a ragged tile); an accumulator is handed back by
    // every epilogue warp
    for (uint32_t i = lane; i < kAccBar0 + 6; i += 32) {
      uint32_t count = 1;
      if (i == kAccBar0 + 2 || i == kAccBar0 + 3) count = C::kEpiWarps * CG;
      mbar_init(bar0 + 8 * i, count);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc<CG>(smem_addr(tmem_slot), C::TMEM_COLS);
    tmem_relinquish<CG>();
  }
  if (args.pdl) grid_dependents_launch();
  if constexpr (C::GROUPED) {
    // offsets clamped into [0, rows] and made to rise: whatever they hold, no
    // access leaves the operands and the groups do not overlap
    const int32_t rows = static_cast<int32_t>(OP == Op::Rows ? args.C : args.K);
    if (warp == 2) {
      int32_t top = 0;
      for (uint32_t e0 = 0; e0 <= args.groups; e0 += 32) {
        const uint32_t e = e0 + lane;
        int32_t v = e <= args.groups ? min(max(__ldg(args.offsets + e), 0), rows) : 0;
#pragma unroll
        for (uint32_t d = 1; d < 32; d *= 2) {
          const int32_t up = __shfl_up_sync(0xffffffffu, v, d);
          if (lane >= d) v = max(v, up);
        }
        v = max(v, top);
        if (e <= args.groups) offs[e] = static_cast<uint32_t>(v);
        top = __shfl_sync(0xffffffffu, v, 31);
      }
      __syncwarp();
    }
    if constexpr (OP == Op::Rows) {
      // first tile of each group: an exclusive sum
      if (warp == 2) {
        const uint32_t lt = (args.L + C::LT - 1) / C::LT;
        uint32_t sum = 0;
        for (uint32_t e0 = 0; e0 < args.groups; e0 += 32) {
          const uint32_t e = e0 + lane;
          const uint32_t n = e < args.groups ? (offs[e + 1] - offs[e] + NT - 1) / NT * lt : 0u;
          uint32_t incl = n;
#pragma unroll
          for (uint32_t d = 1; d < 32; d *= 2) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += up;
          }
          if (e < args.groups) tab[e] = sum + incl - n;
          sum += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) tab[args.groups] = sum;
      }
    } else {
      // the group with most rows, the one with fewest, the next, ...
      __syncthreads();
      for (uint32_t e = threadIdx.x; e < args.groups; e += C::kThreads) {
        uint32_t place = e;
        if (args.groups <= kMaxSortedGroups) {
          const uint32_t n = offs[e + 1] - offs[e];
          place = 0;
          for (uint32_t f = 0; f < args.groups; ++f) {
            const uint32_t m = offs[f + 1] - offs[f];
            place += (m > n || (m == n && f < e)) ? 1u : 0u;
          }
          place = 2 * place < args.groups ? 2 * place : 2 * (args.groups - 1 - place) + 1;
        }
        tab[place] = e;
      }
    }
    __syncthreads();
  }
  static_assert(kAheadItems <= C::kThreads, "one item per thread");
  if (threadIdx.x < kAheadItems) {
    TileItem w;
    w.valid = tile_item<C, CG, OP, NT>(args, offs, tab, cluster_id, G, threadIdx.x, w) ? 1u : 0u;
    ahead[threadIdx.x] = w;
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (C::kCluster > 1) cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const auto item = [&](uint32_t wi, TileItem& w) {
    if (wi < kAheadItems) {
      w = ahead[wi];
      return w.valid != 0u;
    }
    return tile_item<C, CG, OP, NT>(args, offs, tab, cluster_id, G, wi, w);
  };

  // this CTA's stages of a reduction of kt_n: all of them, or its part
  const auto k_first = [&](uint32_t kt_n) { return SPLIT > 1 ? kt_n * k_rank / SPLIT : 0u; };
  const auto k_last = [&](uint32_t kt_n) { return SPLIT > 1 ? kt_n * (k_rank + 1) / SPLIT : kt_n; };

  if (warp == 0) {
    // ==================== TMA producer: one thread ==============================
    if (lane == 0) {
      // (the threads that touch memory wait for the predecessor; every CTA
      // has some, so none ends before it)
      if (args.pdl) grid_dependency_wait();
      const uint64_t pol = l2_policy_evict_last();
      uint32_t it = 0;
      uint32_t tail_last = 0, tail_phase = 0;   // per stage: its last tile was ragged; its tail barrier's parity
      bool ok = true;
      TileItem w;
      for (uint32_t wi = 0; ok && item(wi, w); ++wi) {
        const uint32_t kt_n = (w.k_len + C::BK - 1) / C::BK;
        const uint32_t h = mma_n<CG>(w.live) / CG;     // Q rows this CTA contributes to the MMA
        // a K-major Q arrives in boxes of Q_BOX rows, as many as the MMA reads
        const uint32_t q_boxes = Q_MN ? 0u : (h + C::Q_BOX - 1) / C::Q_BOX;
        const uint32_t tx = C::P_BYTES + (Q_MN ? C::Q_BYTES : q_boxes * C::Q_BOX * 128);
        const int32_t px = static_cast<int32_t>(w.l0 + rank * 128);
        const int32_t qy = static_cast<int32_t>(w.c0 + rank * h);
        if (SPLIT > 1 && k_rank == 0)
          mbar_arrive_expect_tx(part_bar, (SPLIT - 1) * ((w.live + 31) / 32) * (128 * 32 * 4));
        for (uint32_t kt = k_first(kt_n); kt < k_last(kt_n); ++kt, ++it) {
          const uint32_t s = it % C::STAGES;
          if (it == args.stall_iter) continue;   // watchdog test: this stage never fills
          if (!wait_bounded(empty_bar(s), ((it / C::STAGES) & 1u) ^ 1u, wd, kSiteProducerEmpty)) {
            ok = false;
            break;
          }
          const uint32_t sb = base + s * C::STAGE_BYTES;
          const int32_t k0 = static_cast<int32_t>(kt * C::BK);
          const bool ragged = C::TAIL && (kt + 1) * C::BK > w.k_len;
          // a ragged tile lands on this CTA's own tail barrier; its tail warp
          // passes it on to the leader's full barrier
          uint32_t bar = full_bar(s);
          bool pair = false;
          if (ragged) {
            bar = tail_bar(s);
            mbar_arrive_expect_tx(bar, tx);
            tail_last |= 1u << s;
            tail_phase ^= 1u << s;
          } else {
            tail_last &= ~(1u << s);
            if constexpr (CG == 2) {
              pair = true;
              bar = mapa_shared(full_bar(s), 0);
            }
            if (leader) mbar_arrive_expect_tx(full_bar(s), CG * tx);
          }
          const auto load = [&](uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y, int32_t z) {
            if (CG == 2 && pair) tma_load_3d_pair(dst, m, bar, x, y, z, pol);
            else tma_load_3d(dst, m, bar, x, y, z, pol);
          };
          const int32_t pz = static_cast<int32_t>(C::SUM ? 0u : w.z);
          const int32_t qz = static_cast<int32_t>(C::GROUPED ? 0u : w.z);
          const int32_t kr = static_cast<int32_t>((C::SUM ? w.row0 : 0u)) + k0;
          if constexpr (P_MN) {
            load(sb, &tmP, px, kr, pz);
            load(sb + 8192, &tmP, px + 64, kr, pz);
          } else {
            load(sb, &tmP, k0, px, pz);
          }
          if constexpr (Q_MN) {
#pragma unroll
            for (uint32_t x = 0; x < C::Q_ROWS; x += 64)
              load(sb + C::P_BYTES + x * 128, &tmQ, qy + static_cast<int32_t>(x), kr, qz);
          } else {
            const int32_t y = static_cast<int32_t>(OP == Op::Rows ? w.row0 : 0u) + qy;
            for (uint32_t r = 0; r < q_boxes; ++r)
              load(sb + C::P_BYTES + r * C::Q_BOX * 128, &tmQ, k0, y + static_cast<int32_t>(r * C::Q_BOX), qz);
          }
        }
      }
      // Exit path after a give-up: let this CTA's issued loads, and sums on their
      // way to it, land first.
      if (*abort_flag) {
        if (SPLIT > 1 && k_rank == 0) drain_wait(part_bar, 0, wd, kSiteProducerDrain);
        const uint32_t first = it > C::STAGES ? it - C::STAGES : 0u;
        for (uint32_t i = first; i < it; ++i) {
          const uint32_t s = i % C::STAGES;
          if (i == args.stall_iter) continue;
          if ((tail_last >> s) & 1u) drain_wait(tail_bar(s), ((tail_phase >> s) & 1u) ^ 1u, wd, kSiteProducerDrain);
          if (leader) drain_wait(full_bar(s), (i / C::STAGES) & 1u, wd, kSiteProducerDrain);
        }
      }
    }
  } else if (warp == 1) {
    // ==================== MMA issuer: one thread of the leader CTA ==============
    if (leader && lane == 0) {
      bool alone = !args.pdl;   // known: the predecessor has ended
      uint32_t it = 0, j = 0;
      bool ok = true, issued = false;
      TileItem w;
      for (uint32_t wi = 0; ok && item(wi, w); ++wi) {
        const uint32_t kt_n = (w.k_len + C::BK - 1) / C::BK;
        const uint32_t idesc = idesc_f16(C::LT, mma_n<CG>(w.live), args.fmt, P_MN, Q_MN);
        const uint32_t k_stop = k_last(kt_n);
        for (uint32_t k_begin = k_first(kt_n); ok && k_begin < k_stop; ++j) {
          const uint32_t k_end = k_stop - k_begin > C::SEG_TILES ? k_begin + C::SEG_TILES : k_stop;
          const uint32_t b = j & 1u;
          // accumulator b must have been drained by every epilogue warp
          if (!wait_bounded(acce_bar(b), ((j >> 1) & 1u) ^ 1u, wd, kSiteMmaAccEmpty)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t d_tmem = tmem_base + b * C::ACC_COLS;
          const auto stage = [&](uint32_t kt, uint32_t steps) {
            const uint32_t s = it % C::STAGES;
            if (!wait_bounded_alone(full_bar(s), (it / C::STAGES) & 1u, wd, kSiteMmaFull, alone)) {
              ok = false;
              return;
            }
            tc_fence_after_sync();
            const uint32_t sb = base + s * C::STAGE_BYTES;
            const uint64_t pd = P_MN ? smem_desc_mn_sw128(sb) : smem_desc_sw128(sb);
            const uint64_t qd = Q_MN ? smem_desc_mn_sw128(sb + C::P_BYTES) : smem_desc_sw128(sb + C::P_BYTES);
            // 16 k per MMA: 32 bytes along a K-major row, 16 rows of an MN-major tile
            constexpr uint32_t kPStep = P_MN ? 128 : 2, kQStep = Q_MN ? 128 : 2;
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
              if (k == steps) break;
              mma_bf16<CG>(d_tmem, pd + kPStep * k, qd + kQStep * k, idesc, (kt != k_begin || k != 0u));
            }
            commit_to<CG>(empty_bar(s));   // frees the stage once these MMAs finish
            issued = true;
            ++it;
          };
          // Whole stages in a loop of their own, without a step's condition between two
          // MMAs.  A pair's MMAs of a stage take 512 clocks and the issuing thread nearly
          // as long: unrolled, one group of 4096 x 4096 x 4096 takes 82 us to the weights
          // instead of 92 (fp32: 98, 106).  One CTA's narrower MMAs leave it time, and calls as short
          // as those that use them wait for its instructions.
          constexpr uint32_t kUnroll = CG == 2 ? 4 : 1;
          const uint32_t whole = C::TAIL && k_end == k_stop ? w.k_len / C::BK : k_end;
          uint32_t kt = k_begin;
#pragma unroll kUnroll
          for (; ok && kt < whole; ++kt) stage(kt, 4);
          if (C::TAIL && ok && kt < k_end) stage(kt, (w.k_len % C::BK + 15) / 16);
          if (!ok) break;
          commit_to<CG>(accf_bar(b));
          k_begin = k_end;
        }
      }
      // Exit path: every tcgen05 op this thread issued completes before TMEM is released.
      if (issued) {
        if constexpr (CG == 1)
          tc_commit(drain_bar);
        else
          tc_commit_pair_multicast(drain_bar, 0x1);
        drain_wait(drain_bar, 0, wd, kSiteMmaDrain);
      }
    }
  } else if (C::TAIL && warp == C::kTailWarp) {
    // ==================== ragged reduction ends (Op::Sum) ========================
    // The last tile of a group's reduction also holds rows of the next group
    // (or nothing): those up to the next multiple of 16 k, which the MMA
    // reads, are cleared in both operands, so that not even an Inf or NaN of
    // another group's rows reaches this one.
    uint32_t it = 0, phase = 0;
    bool ok = true;
    TileItem w;
    for (uint32_t wi = 0; ok && item(wi, w); ++wi) {
      const uint32_t kt_n = (w.k_len + C::BK - 1) / C::BK;
      const uint32_t tail = w.k_len % C::BK;
      it += kt_n;
      if (tail == 0) continue;
      const uint32_t s = (it - 1) % C::STAGES;
      if (!warp_wait(tail_bar(s), (phase >> s) & 1u, wd, kSiteTail, lane)) {
        ok = false;
        break;
      }
      phase ^= 1u << s;
      uint8_t* const sp = base_ptr + s * C::STAGE_BYTES;
      const uint32_t end = (tail + 15) / 16 * 16;
      // 4 boxes (two 64-wide blocks of each operand), rows tail .. end - 1, 8 pieces of 16 bytes
      const uint32_t n = (end - tail) * 32;
      for (uint32_t i = lane; i < n; i += 32) {
        const uint32_t r = tail + i / 32, box = (i / 8) & 3u, piece = i & 7u;
        *reinterpret_cast<uint4*>(sp + box * 8192 + r * 128 + piece * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        // the leader's barrier: its own arrival, and 4 bytes from the peer CTA
        if (leader) mbar_arrive_expect_tx(full_bar(s), CG == 2 ? 4u : 0u);
        else st_async_u32(mapa_shared(smem_addr(tmem_slot + 2), 0), s, mapa_shared(full_bar(s), 0));
      }
    }
  } else {
    // ==================== epilogue: eight warps, two per TMEM lane quarter =======
    const uint32_t q = warp & 3u;              // TMEM lanes 32q .. 32q + 31
    const uint32_t eg = (warp - 2u) / 4u;      // chunks eg, eg + 2, ...
    const uint32_t odd = lane & 1u;
    uint32_t j = 0;
    bool ok = true;
    TileItem w;
    if (args.pdl) grid_dependency_wait();
    for (uint32_t wi = 0; ok && item(wi, w); ++wi) {
      const uint32_t kt_n = (w.k_len + C::BK - 1) / C::BK;
      const uint32_t lbase = w.l0 + rank * 128 + q * 32;   // this warp's first output column
      const uint32_t col = lbase + lane;
      const uint32_t nch = (w.live + 31) / 32;
      // output row of tile column c: matrix z, row c0 + c (Rows: memory row row0 + c0 + c)
      const uint64_t out0 = OP == Op::Rows
                                ? static_cast<uint64_t>(w.row0 + w.c0) * args.ldo
                                : w.z * args.stride_o + static_cast<uint64_t>(w.c0) * args.ldo;
      // The hand-back of an accumulator whose reads are complete
      // (tcgen05.wait::ld): it publishes nothing.
      const auto release = [&](uint32_t b) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 1) mbar_arrive(acce_bar(b));
          else mbar_arrive_cluster_relaxed(mapa_shared(acce_bar(b), 0));
        }
      };
      if (C::SUM && kt_n == 0) {
        // a group without rows: no accumulator, zeros, or (+=) nothing at all
        if (!C::ADD) {
          using T = std::conditional_t<OUT32, uint32_t, uint16_t>;
          const uint32_t l = w.l0 + rank * 128;
          const bool vec = ((reinterpret_cast<uintptr_t>(args.out) | (args.ldo * sizeof(T)) |
                             (args.stride_o * sizeof(T))) & 15u) == 0;
          if (C::LANE && l < args.L) {
            T* const o = static_cast<T*>(args.out) + w.z * args.stride_o + l * args.ldo + w.c0;
            for (uint32_t c = 0; c < w.live; c += 128)
              zero_tile(o + c, args.ldo, min(128u, args.L - l), min(128u, w.live - c), vec, threadIdx.x - 64);
          } else if (l < args.L) {
            zero_tile(static_cast<T*>(args.out) + out0 + l, args.ldo, w.live, min(128u, args.L - l), vec,
                      threadIdx.x - 64);
          }
        }
        continue;
      }
      const auto t_addr = [&](uint32_t ch) {
        return tmem_base + ((q * 32u) << 16) + (j & 1u) * C::ACC_COLS + ch * 32;
      };
      // SPLIT: the first CTA adds the others' sums of a chunk in their order; the
      // others send theirs and are done (true: the chunk is not theirs to store)
      const auto combine = [&](uint32_t ch, uint32_t (&v)[32]) -> bool {
        const uint32_t at = (ch * 4 + q) * 4096 + lane * 16;
        if (k_rank != 0) {
          const uint32_t dst = mapa_shared(part0 + (k_rank - 1) * C::PART_BYTES + at, 0);
          const uint32_t bar = mapa_shared(part_bar, 0);
#pragma unroll
          for (uint32_t i = 0; i < 8; ++i)
            st_async_v4(dst + i * 512, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], bar);
          return true;
        }
        if (!warp_wait(part_bar, 0, wd, kSiteSplit, lane)) {
          ok = false;
          return true;
        }
#pragma unroll 1
        for (uint32_t r = 0; r + 1 < SPLIT; ++r) {
          const uint8_t* const src = base_ptr + (part0 - base) + r * C::PART_BYTES + at;
#pragma unroll
          for (uint32_t i = 0; i < 8; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(src + i * 512);
            v[4 * i] = __float_as_uint(__uint_as_float(v[4 * i]) + x.x);
            v[4 * i + 1] = __float_as_uint(__uint_as_float(v[4 * i + 1]) + x.y);
            v[4 * i + 2] = __float_as_uint(__uint_as_float(v[4 * i + 2]) + x.z);
            v[4 * i + 3] = __float_as_uint(__uint_as_float(v[4 * i + 3]) + x.w);
          }
        }
        return false;
      };
      const auto acc_wait = [&]() {
        ok = warp_wait(accf_bar(j & 1u), (j >> 1) & 1u, wd, kSiteEpiAccFull, lane);
        tc_fence_after_sync();
        return ok;
      };
      if constexpr (OUT32) {
        float acc[C::NCH][32];
#pragma unroll
        for (uint32_t i = 0; i < C::NCH; ++i)
#pragma unroll
          for (uint32_t t = 0; t < 32; ++t) acc[i][t] = 0.0f;
        for (uint32_t k = k_first(kt_n); k < k_last(kt_n); k += C::SEG_TILES, ++j) {
          if (!acc_wait()) break;
#pragma unroll
          for (uint32_t i = 0; i < C::NCH; ++i) {
            if (2 * i + eg < nch) {
              uint32_t v[32];
              tmem_ld_32x32b_x32_sync(t_addr(2 * i + eg), v);
#pragma unroll
              for (uint32_t t = 0; t < 32; ++t) acc[i][t] += __uint_as_float(v[t]);
            }
          }
          release(j & 1u);
        }
        if (!ok) break;
        float* const o = static_cast<float*>(args.out) + out0 + col;
#pragma unroll
        for (uint32_t i = 0; i < C::NCH; ++i) {
          const uint32_t c0 = (2 * i + eg) * 32;
          if constexpr (SPLIT > 1) {
            uint32_t v[32];
#pragma unroll
            for (uint32_t t = 0; t < 32; ++t) v[t] = __float_as_uint(acc[i][t]);
            if (2 * i + eg >= nch || combine(2 * i + eg, v)) continue;
#pragma unroll
            for (uint32_t t = 0; t < 32; ++t) acc[i][t] = __uint_as_float(v[t]);
          }
          float* p = o + static_cast<uint64_t>(c0) * args.ldo;
          if (c0 + 32 <= w.live && lbase + 32 <= args.L && !(C::ADD)) {
#pragma unroll
            for (uint32_t t = 0; t < 32; ++t, p += args.ldo) *p = acc[i][t];
          } else if (col < args.L) {
            if constexpr (C::ADD) {
              // 16 rows' old values are on their way at a time: a store could alias the
              // next load for all the compiler knows, so each row would wait for the last
#pragma unroll
              for (uint32_t h = 0; h < 32; h += 16) {
                float had[16];
#pragma unroll
                for (uint32_t t = 0; t < 16; ++t) had[t] = c0 + h + t < w.live ? p[t * args.ldo] : 0.0f;
#pragma unroll
                for (uint32_t t = 0; t < 16; ++t)
                  if (c0 + h + t < w.live) p[t * args.ldo] = had[t] + acc[i][h + t];
                p += 16 * args.ldo;
              }
            } else {
#pragma unroll
              for (uint32_t t = 0; t < 32; ++t, p += args.ldo)
                if (c0 + t < w.live) *p = acc[i][t];
            }
          }
        }
      } else if constexpr (C::LANE) {
        // This lane's row as whole sectors of 32 bytes.  Rows start on 16 bytes and
        // hold whole pieces of 8 columns.  Where the tile starts inside a sector of
        // this row (`late`), its first piece is the tile before's, which shares 8
        // columns, and a chunk's last piece waits for the next chunk (`kept`).
        const uint32_t half = (nch + 1) / 2;
        const uint32_t first = eg * half, last = min(nch, first + half);
        uint16_t* const row = static_cast<uint16_t*>(args.out) + w.z * args.stride_o + col * args.ldo + w.c0;
        const bool late = ((reinterpret_cast<uintptr_t>(row) >> 4) & 1u) != 0;
        const bool row_end = w.c0 + NT >= args.C;
        uint32_t kept[4] = {};
        if (!acc_wait()) break;
        const uint32_t b = j & 1u;
        bool held = true;
#pragma unroll 1
        for (uint32_t ch = first == 0 ? 0 : first - 1; ch < last; ++ch) {   // (first - 1: for the piece kept)
          uint16_t* const o = row + ch * 32;
          const uint32_t pieces = col < args.L ? min(4u, (w.live - ch * 32) / 8) : 0u;
          uint32_t v[32];
          tmem_ld_32x32b_x32_sync(t_addr(ch), v);
          if (ch + 1 == last) {
            release(b);
            held = false;
          }
          uint32_t h[16];
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) {
            uint4 had = make_uint4(0, 0, 0, 0);   // what the output holds
            if (C::ADD && i < pieces) had = *reinterpret_cast<const uint4*>(o + 8 * i);
            const uint32_t had4[4] = {had.x, had.y, had.z, had.w};
#pragma unroll
            for (uint32_t t = 0; t < 4; ++t) {
              float x0 = __uint_as_float(v[8 * i + 2 * t]), x1 = __uint_as_float(v[8 * i + 2 * t + 1]);
              if (C::ADD) {
                x0 += bf16_bits_to_f32(had4[t] & 0xFFFFu);
                x1 += bf16_bits_to_f32(had4[t] >> 16);
              }
              h[4 * i + t] = pack_bf16x2(x0, x1);
            }
          }
          // two sectors: pieces 0 1 2 3, or the one kept and 0 1 2
          uint32_t x[16];
#pragma unroll
          for (uint32_t t = 0; t < 4; ++t) x[t] = late ? kept[t] : h[t];
#pragma unroll
          for (uint32_t t = 4; t < 16; ++t) x[t] = late ? h[t - 4] : h[t];
#pragma unroll
          for (uint32_t t = 0; t < 4; ++t) kept[t] = h[12 + t];
          if (ch < first || pieces == 0) continue;
          uint16_t* const at = o - (late ? 8 : 0);
          const uint32_t have = pieces + (late ? 1u : 0u);
          if (late && ch == 0) {
            if (w.c0 == 0) st_global_v4(o, x + 4);   // the row's first piece
          } else if (have >= 2) {
            st_global_v8(at, x);
          } else {
            st_global_v4(at, x);
          }
          if (have >= 4) st_global_v8(at + 16, x + 8);
          else if (have == 3) st_global_v4(at + 16, x + 8);
          if (have == 5 && row_end && ch + 1 == nch) st_global_v4(o + 24, kept);
        }
        if (held) release(b);   // (a warp without a chunk)
        ++j;
      } else {
        // 16-bit outputs, one 32-column chunk at a time.  The code of a chunk is
        // kept short and rolled: run once or twice a kernel, it costs what its
        // instructions cost to fetch.
        const uint32_t pcol = lbase + (lane & ~1u);   // this lane's column pair
        // What the epilogue adds to a chunk is loaded a chunk ahead, the first
        // chunk's before the accumulator is waited for.
        //   Sym: row `col` of the symmetric R, whose 32 values from column
        //     w.c0 + c0 on are the chunk's (rows are whole lines of 64)
        //   Apply: X's halves at this lane's column pair, row 2 t + odd
        const auto sym_at = [&](uint32_t c0) {
          return w.z * args.stride_o + static_cast<uint64_t>(col) * args.ldo + w.c0 + c0;
        };
        // the arguments with this matrix's powers of two
        float alpha = args.alpha, beta = args.beta, out_scale = args.out_scale;
        if constexpr (OP == Op::Sym || C::APPLY) {
          const int lift = args.lift[w.z], now = max(lift - args.spent, 0), next = max(lift - args.spent_next, 0);
          if (OP == Op::Sym && args.R == nullptr) {
            alpha = alpha * pow2(-now) * pow2(-now);
          } else {
            alpha *= pow2(next - now);
            beta *= pow2(next - now);
          }
          out_scale *= pow2(-next);
        }
        uint32_t add0[16], add1[16];         // Sym: R in add0; Apply: hi, lo
        float rowf = 0.0f;                   // Apply, Y X: this lane's row's alpha + diag
        const float* const dg = args.diag + static_cast<uint64_t>(w.z) * args.diag_n;
        const auto fetch = [&](uint32_t ch) {
          const uint32_t c0 = ch * 32;
          if constexpr (OP == Op::Sym) {
            const bool live = args.R != nullptr && ch < nch && col < args.L;
            const uint4* const r = reinterpret_cast<const uint4*>(args.R + sym_at(c0));
#pragma unroll
            for (uint32_t p = 0; p < 4; ++p) {
              const uint4 x = live ? r[p] : make_uint4(0, 0, 0, 0);
              add0[4 * p] = x.x;
              add0[4 * p + 1] = x.y;
              add0[4 * p + 2] = x.z;
              add0[4 * p + 3] = x.w;
            }
          } else if constexpr (C::APPLY) {
            const uint64_t at =
                w.z * args.stride_x + static_cast<uint64_t>(w.c0 + c0 + odd) * args.ldx + pcol;
            const uint32_t* h = reinterpret_cast<const uint32_t*>(args.x_hi + at);
            const uint4* l =
                reinterpret_cast<const uint4*>(args.x_lo + lo_block(w.z, w.c0 + c0, lbase, args.C, args.L)) + lane;
            const uint32_t left = pcol < args.L && c0 + odd < w.live ? w.live - c0 - odd : 0u;
            if (P_MN) rowf = c0 + lane < w.live ? alpha + dg[w.c0 + c0 + lane] : 0.0f;
#pragma unroll
            for (uint32_t t = 0; t < 16; ++t, h += args.ldx) add0[t] = 2 * t < left ? *h : 0u;
            // (the block's rows and columns past the matrix's are never stored as hi)
            const bool live = ch < nch && lbase < args.L;
#pragma unroll
            for (uint32_t p = 0; p < 4; ++p) {
              const uint4 x = live ? l[32 * p] : make_uint4(0, 0, 0, 0);
              add1[4 * p] = x.x;
              add1[4 * p + 1] = x.y;
              add1[4 * p + 2] = x.z;
              add1[4 * p + 3] = x.w;
            }
          }
        };
        float colf0 = 0.0f, colf1 = 0.0f;    // Apply, X Y: this lane's columns' alpha + diag
        if constexpr (C::APPLY && !P_MN) {
          if (pcol < args.L) colf0 = alpha + dg[pcol];
          if (pcol + 1 < args.L) colf1 = alpha + dg[pcol + 1];
        }
        // a row's column pairs start on 4 bytes
        const bool pairs = ((reinterpret_cast<uintptr_t>(args.out) & 3u) == 0) && (args.ldo & 1u) == 0 &&
                           (args.stride_o & 1u) == 0;
        fetch(eg);
        if (!acc_wait()) break;
        const uint32_t b = j & 1u;
        bool held = true;
#pragma unroll 1
        for (uint32_t ch = eg; ch < nch; ch += 2) {
          const uint32_t c0 = ch * 32;
          uint32_t v[32];
          tmem_ld_32x32b_x32_sync(t_addr(ch), v);
          if (held && ch + 2 >= nch) {   // all of it is in registers: hand it back before the last stores
            release(b);
            held = false;
          }
          if constexpr (SPLIT > 1) {
            if (combine(ch, v)) continue;
          }
          if constexpr (OP == Op::Sym) {
#pragma unroll
            for (uint32_t t = 0; t < 16; ++t) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&add0[t]));
              v[2 * t] = __float_as_uint(fmaf(beta, f.x, alpha * __uint_as_float(v[2 * t])));
              v[2 * t + 1] = __float_as_uint(fmaf(beta, f.y, alpha * __uint_as_float(v[2 * t + 1])));
            }
            fetch(ch + 2);
            if (args.R != nullptr && !w.mirror && col - w.c0 - c0 < 32u && col < args.L) {
              // (an unrolled search: registers have no addresses)
#pragma unroll
              for (uint32_t t = 0; t < 32; ++t)
                if (w.c0 + c0 + t == col) {
                  args.diag[static_cast<uint64_t>(w.z) * args.diag_n + col] = __uint_as_float(v[t]);
                  v[t] = 0u;
                }
            }
            if (w.mirror && col < args.L) {
              // the values also belong to row `col`: two sectors a lane
              uint16_t* const m = static_cast<uint16_t*>(args.out) + sym_at(c0);
#pragma unroll
              for (uint32_t p = 0; p < 2; ++p) {
                uint32_t h[8];
#pragma unroll
                for (uint32_t t = 0; t < 8; ++t)
                  h[t] = pack_f16x2(__uint_as_float(v[16 * p + 2 * t]), __uint_as_float(v[16 * p + 2 * t + 1]));
                st_global_v8(m + 16 * p, h);
              }
            }
          }
          if constexpr (OP == Op::Rows || OP == Op::Sum) {
            if (!pairs) {
              // rows that start on 2 bytes: this lane's column, row by row
              uint16_t* p = static_cast<uint16_t*>(args.out) + out0 + static_cast<uint64_t>(c0) * args.ldo + col;
#pragma unroll
              for (uint32_t t = 0; t < 16; ++t, p += 2 * args.ldo) {
                const uint32_t h = pack_bf16x2(__uint_as_float(v[2 * t]), __uint_as_float(v[2 * t + 1]));
                if (c0 + 2 * t < w.live && col < args.L) p[0] = static_cast<uint16_t>(h & 0xFFFFu);
                if (c0 + 2 * t + 1 < w.live && col < args.L) p[args.ldo] = static_cast<uint16_t>(h >> 16);
              }
              continue;
            }
          }
          // this lane's column pair of row 2 t + odd: rounded in st0 (Apply: and the
          // lo halves in st1), or the two fp32 values
          uint32_t st0[16], st1[16];
#pragma unroll
          for (uint32_t t = 0; t < 16; ++t) {
            if constexpr (OP == Op::Rows || OP == Op::Sum) {
              st0[t] = pair_columns_bf16(__uint_as_float(v[2 * t]), __uint_as_float(v[2 * t + 1]), odd);
              continue;
            }
            float x0, x1;
            pair_columns(__uint_as_float(v[2 * t]), __uint_as_float(v[2 * t + 1]), odd, x0, x1);
            if constexpr (C::APPLY) {
              const float2 l = __half22float2(*reinterpret_cast<const __half2*>(&add1[t]));
              const float f = P_MN ? __shfl_sync(0xffffffffu, rowf, 2 * t + odd) : 0.0f;
              x0 = fmaf(P_MN ? f : colf0, f16_plus(add0[t] & 0xFFFFu, l.x), x0);
              x1 = fmaf(P_MN ? f : colf1, f16_plus(add0[t] >> 16, l.y), x1);
            }
            if constexpr (OP == Op::Apply) {
              const uint32_t p = pack_f16x2(x0, x1);
              st0[t] = p;
              st1[t] = pack_f16x2(-f16_minus(p & 0xFFFFu, x0), -f16_minus(p >> 16, x1));
            } else if constexpr (OP == Op::ApplyOut) {
              st0[t] = __float_as_uint(x0 * out_scale);
              st1[t] = __float_as_uint(x1 * out_scale);
            } else {
              // (SumAdd: unrounded)
              st0[t] = OP == Op::Sym ? pack_f16x2(x0, x1) : __float_as_uint(x0);
              st1[t] = __float_as_uint(x1);
            }
          }
          if constexpr (C::APPLY) fetch(ch + 2);
          const uint64_t at = out0 + static_cast<uint64_t>(c0 + odd) * args.ldo;
          const uint32_t rows_left = c0 + odd < w.live ? w.live - c0 - odd : 0u;   // row 2 t is live: 2 t < rows_left
          if constexpr (OP == Op::Sym || OP == Op::Apply) {
            // the workspace: even pitches, and the column past an odd last one is padding
            uint32_t* p = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(args.out) + at + pcol);
            const uint32_t left = pcol < args.L ? rows_left : 0u;
#pragma unroll
            for (uint32_t t = 0; t < 16; ++t, p += args.ldo)
              if (2 * t < left) *p = st0[t];
            if (OP == Op::Apply && lbase < args.L) {
              uint4* l =
                  reinterpret_cast<uint4*>(args.out_lo + lo_block(w.z, w.c0 + c0, lbase, args.C, args.L)) + lane;
#pragma unroll
              for (uint32_t p = 0; p < 4; ++p)
                l[32 * p] = make_uint4(st1[4 * p], st1[4 * p + 1], st1[4 * p + 2], st1[4 * p + 3]);
            }
          } else if (OP == Op::ApplyOut && args.out_f32) {
            float* p = static_cast<float*>(args.out) + at + pcol;
#pragma unroll
            for (uint32_t t = 0; t < 16; ++t, p += 2 * args.ldo)
              if (2 * t < rows_left) {
                if (pcol < args.L) p[0] = __uint_as_float(st0[t]);
                if (pcol + 1 < args.L) p[1] = __uint_as_float(st1[t]);
              }
          } else {
            uint16_t* p = static_cast<uint16_t*>(args.out) + at + pcol;
            if (C::ADD) {
#pragma unroll
              for (uint32_t t = 0; t < 16; ++t) {
                uint16_t* const o = p + static_cast<uint64_t>(2 * t) * args.ldo;
                const bool live = 2 * t < rows_left;
                float x0 = __uint_as_float(st0[t]), x1 = __uint_as_float(st1[t]);
                if (live && pcol < args.L) x0 += bf16_bits_to_f32(o[0]);
                if (live && pcol + 1 < args.L) x1 += bf16_bits_to_f32(o[1]);
                st0[t] = pack_bf16x2(x0, x1);
              }
            }
            if (OP == Op::ApplyOut) {
#pragma unroll
              for (uint32_t t = 0; t < 16; ++t)
                st0[t] = pack_bf16x2(__uint_as_float(st0[t]), __uint_as_float(st1[t]));
            }
            if (pairs && lbase + 32 <= args.L && c0 + 32 <= w.live) {
              uint32_t* o = reinterpret_cast<uint32_t*>(p);
#pragma unroll
              for (uint32_t t = 0; t < 16; ++t, o += args.ldo) *o = st0[t];
            } else if (pairs && lbase + 32 <= args.L) {
#pragma unroll
              for (uint32_t t = 0; t < 16; ++t, p += 2 * args.ldo)
                if (2 * t < rows_left) *reinterpret_cast<uint32_t*>(p) = st0[t];
            } else {
#pragma unroll
              for (uint32_t t = 0; t < 16; ++t, p += 2 * args.ldo) {
                if (2 * t < rows_left && pcol < args.L) p[0] = static_cast<uint16_t>(st0[t] & 0xFFFFu);
                if (2 * t < rows_left && pcol + 1 < args.L) p[1] = static_cast<uint16_t>(st0[t] >> 16);
              }
            }
          }
        }
        if (held) release(b);   // (a warp without a chunk)
        ++j;
      }
    }
  }

  // ---- teardown: every role is done with TMEM and with the peer's barriers ----
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (C::kCluster > 1) cluster_sync();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc<CG>(tmem_base, C::TMEM_COLS);
  }
}

}  // namespace gb300
