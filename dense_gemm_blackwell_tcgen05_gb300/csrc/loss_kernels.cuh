// Losses over a vocabulary: the logits z = scale A B^T (A [M, K] rows, B [N, K]
// the vocabulary's matrix, bf16) as tiles in TMEM that are never stored.
//
//     out of a tile, forward:   per row its largest logit m, the sum of exp(z - m),
//                               the logits at the row's entries (its target, or a
//                               teacher's list), and for label smoothing sum z
//     out of a tile, backward:  the logits' gradient, rounded to bf16, into a
//                               buffer that holds one piece of the vocabulary:
//                               g = gq exp(z - lse) - gs - (gt or gt p at the entries)
//
// Rows sit in the TMEM lanes (the MMA's M) and the vocabulary in its columns (N), so
// that a thread holds 32 consecutive logits of one row: maxima and sums need no other
// thread, an entry's logit is in one thread's registers, and a gradient's row is
// stored by its thread in whole sectors.
//
// Persistent, warp-specialised like the grouped products: a TMA producer, an MMA
// issuer with two accumulators, eight epilogue warps, two per lane quarter, each with
// half of the tile's columns.  The gradient leaves through shared memory by TMA (4096 rows,
// 32768 tokens of width 2048: 11 us of 285 less than from registers, each lane its own row in
// whole sectors; 128 rows, a million tokens of width 64: 393 for 508, both gradients), but for
// single CTAs' up to 64 rows, whose boxes would be half empty (64 rows, 200000 tokens of width 256:
// 87 us, 91 with boxes), or over a long width, which the loads of B bound: there another stage of
// them is worth more (64 rows, 131072 tokens of width 4096: 164 us, 170 with boxes).  Rows left out
// of the loss are left out of the product: the rows that count lie compact, and their number is
// read on the GPU.
//
// Bounds.  Thousands of rows are bound by the MMAs (4096 rows, 32768 tokens of width 4096:
// 523 us forward, 2.10 PFLOP/s, tensor pipes 98.8 % busy; 549 backward), few by the read of B
// (48 rows, 131072 tokens: 159 us, 6.8 TB/s), a few thousand tokens by latency.
//
// Precision.  The tensor core's additions truncate (1.1e-9 of the result a term), so both
// passes add up segments of 256 or 512 terms in registers: a row's loss is the difference of its
// logits, and where it is sure of its target its gradient is that of two numbers near 1
// (1 - exp(z - lse) of 2.2e-4 at a logit of 16, width 8192: 4.1e-4 off in one sum, 5e-6 in
// segments).
// exp is 2^x of the multiprocessor's special function unit (2 units in the last place)
// on arguments in fp32.  The gradient g is rounded to bf16 for the products with it, at
// 2^-9 of itself: over many rows as much as rounding the products' bf16 results adds (2.4e-3
// of dA and dB where fp32 logits, rounded once at the end, give 1.7e-3).  Of few rows a
// row's error shows, and what g's rounding left follows as rows of its own (1.7e-3).
#pragma once

#include <cstdint>

#include "gemm_kernels.cuh"
#include "grouped_kernels.cuh"
#include "ptx_grouped.cuh"
#include "ptx_loss.cuh"

namespace gb300 {

// What a row's gradient is made of: g = gq exp(z - lse) - gs - gt (at the target; times p
// at a list's entries).
struct LossFactors {
  const float* dloss;
  uint64_t inc_dloss;
  const float* lse;
  const float* entropy;        // a list's: NaN where it is wrong (nullptr: targets)
  float scale, smoothing, z_coef;
  uint32_t N;                  // the whole vocabulary
};

// A list's entries are found from the number of them before each of so many buckets of
// tokens: a row's own search would be seven loads, one after another.
constexpr uint32_t kLossBuckets = 64;

struct LossArgs {
  uint32_t M, N, K;            // rows in all, vocabulary (of this piece, backward), width
  uint32_t nt;                 // columns of a tile, a multiple of 32
  const uint32_t* count;       // rows that count (nullptr: all of them, in place)
  const uint32_t* index;       // [count] where each of them lies among all rows (nullptr: in place)
  float c;                     // scale log2(e): exp(z) = 2^(c a.b)
  uint32_t first;              // number of this piece's first token
  // entries: a target per row, or a sorted list
  const void* target;          // [M] int32 or int64, by all rows
  uint32_t target64;
  const int32_t* ids;          // [M][top] rising, by all rows
  const float* prob;           // [M][top] their probabilities (backward)
  const uint32_t* len;         // [M] how many
  const uint16_t* start;       // [kLossBuckets + 1][M] how many lie before a bucket of tokens (nullptr: not known)
  uint32_t bucket;             // its tokens
  uint32_t top;
  // forward
  float2* part;                // [slots][2][ld_part]: largest c a.b, sum of 2^(c a.b - largest)
  float* part_sum;             // [slots][2][ld_part] sum of a.b (nullptr: not wanted)
  uint64_t ld_part;
  uint32_t runs;               // one block of rows: a slot for each cluster, else for each tile of columns
  float* entry;                // [M] or [M][top], by all rows: the entries' a.b
  // backward
  const float4* row;           // [count] (lse log2(e), gq, gs, gt) (nullptr: in place, from `factors`)
  LossFactors factors;
  const uint16_t* A;           // in place: rows copied to `clean` (nullptr: not by this launch),
  uint64_t lda;                //   zeros for those left out
  uint16_t* clean;
  uint64_t ld_clean;
  int32_t* offsets;            //   and {0, M}, as one group's offsets
  uint16_t* out;               // [count][ld_out] the gradient's piece; zeros up to a multiple of 64 rows
  uint64_t ld_out;
  bool boxes;                  // it leaves by TMA, where the kernel can
  uint32_t lo_row;             // its row from which on what rounding left follows (0: it is dropped)
  unsigned long long* status;
  unsigned long long timeout_ns;
  uint32_t stall_iter;         // watchdog test hook (0xFFFFFFFF: none)
};

// Stages in a sum of the tensor core's: 512 terms, and 256 forward on one CTA, whose epilogue has the
// time (48 rows, 131072 tokens of width 4096: 161.1 us for 160.5, losses 3.2e-6 off for 5.2e-6; on
// pairs 3 to 6 % of the time, and of a gradient of 128 rows 3 % at a width of 512).
constexpr uint32_t loss_segment(uint32_t cg, bool back) { return cg == 1 && !back ? 4 : 8; }

// NT: columns of a tile at most.  BACK, SEG: as loss_kernel's.
template <int CG, uint32_t NT, bool BACK, bool SEG>
struct LossCfg {
  static_assert(CG == 1 || CG == 2, "cta_group is 1 or 2");
  static constexpr uint32_t BK = 64;                     // k per stage: one 128-byte row
  static constexpr uint32_t LT = 128 * CG;               // rows per tile
  static_assert(NT % 64 == 0 && NT <= 256, "two halves of whole 32-column chunks");
  // rows per load of A: few rows load what they need, pairs all at once
  static constexpr uint32_t P_BOX = CG == 2 ? 128 : 32;
  static constexpr uint32_t P_BYTES = 128 * 128;
  static constexpr uint32_t Q_BYTES = NT / CG * 128;     // vocabulary rows staged by one CTA
  static constexpr uint32_t STAGE_BYTES = P_BYTES + Q_BYTES;
  static constexpr uint32_t kEpiWarps = 8;
  static constexpr uint32_t kThreads = 32 * (4 + kEpiWarps);   // producer, MMA issuer, two that idle; the epilogue
  // A pair's epilogue holds 128 columns' sums a thread between segments: it takes registers that the
  // other four warps leave (without, 64 bytes a thread are spilled: backward, 4096 lists of 64 over
  // 32768 tokens of width 2048, 304 us instead of 278).
  static constexpr bool kSplit = CG == 2 && SEG;
  static constexpr uint32_t kFewRegs = 56, kManyRegs = 224, kLeastRegs = kSplit ? 168 : 0;   // least: of a launch
  static_assert(!kSplit || 128 * kFewRegs + 32 * kEpiWarps * kManyRegs <= kThreads * kLeastRegs, "more than the launch's");
  static constexpr uint32_t SEG_TILES = loss_segment(CG, BACK);
  static constexpr uint32_t NCH = NT / 64;               // 32-column chunks per epilogue warp at most
  static constexpr uint32_t BAR_BYTES = 512;
  static constexpr uint32_t SMEM_LIMIT = 232448;
  static constexpr uint32_t ALIGN_SLACK = 1024;
  static constexpr uint32_t BOX_BYTES = 32 * 64;         // a warp's 32 rows of a chunk on their way out
  static constexpr bool kBoxes = BACK && (CG == 2 || !SEG);   // the gradient leaves through them
  static constexpr uint32_t OUT_BYTES = kBoxes ? kEpiWarps * 2 * BOX_BYTES : 0;
  static constexpr uint32_t FIT = (SMEM_LIMIT - ALIGN_SLACK - BAR_BYTES - OUT_BYTES) / STAGE_BYTES;
  static constexpr uint32_t STAGES = FIT > 12 ? 12 : FIT;
  static constexpr uint32_t SMEM_BYTES = ALIGN_SLACK + STAGES * STAGE_BYTES + OUT_BYTES + BAR_BYTES;
  static_assert((2 * STAGES + 5) * 8 + 16 <= BAR_BYTES, "barrier area");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t ACC_COLS = 256;              // second accumulator's first column
};

// Row blocks swept together along the vocabulary.
constexpr uint32_t kLossRaster = 16;

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Element t (< 32) of a register array.
__device__ __forceinline__ float select32(const float (&v)[32], uint32_t t) {
  float x = v[0];
#pragma unroll
  for (uint32_t i = 1; i < 32; ++i) x = t == i ? v[i] : x;
  return x;
}

__device__ __forceinline__ int64_t loss_index_at(const void* p, bool wide, uint64_t i) {
  return wide ? static_cast<const int64_t*>(p)[i] : static_cast<int64_t>(static_cast<const int32_t*>(p)[i]);
}

// (lse log2(e), gq, gs, gt) of row r; NaN for a target or an entry past the vocabulary.
__device__ __forceinline__ float4 loss_row_factors(const LossFactors& f, const void* targets, bool target64, uint32_t r) {
  const float g = f.dloss[r * f.inc_dloss] * f.scale, l = f.lse[r];
  const bool wrong = f.entropy != nullptr ? isnan(f.entropy[r]) : loss_index_at(targets, target64, r) >= f.N;
  return make_float4(l * 1.4426950408889634f, wrong ? NAN : g * (1.0f + 2.0f * f.z_coef * l),
                     g * f.smoothing / static_cast<float>(f.N), g * (1.0f - f.smoothing));
}

// LIST: a list of entries per row, else one target.  SEG: several segments of the width, else one,
// whose sums a backward pass takes a chunk at a time.
template <int CG, uint32_t NT, bool BACK, bool LIST, bool SEG>
__global__ void __launch_bounds__(LossCfg<CG, NT, BACK, SEG>::kThreads, 1)
    loss_kernel(const __grid_constant__ CUtensorMap tmAll, const __grid_constant__ CUtensorMap tmCompact,
                const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmOut, const LossArgs args) {
  using C = LossCfg<CG, NT, BACK, SEG>;
  static_assert(BACK || SEG, "a forward pass takes any width");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const base_ptr = smem_raw + (base - raw);
  const uint32_t out0 = base + C::STAGES * C::STAGE_BYTES;
  const uint32_t bar0 = out0 + C::OUT_BYTES;
  const auto full_bar = [&](uint32_t s) { return bar0 + 8 * s; };
  const auto empty_bar = [&](uint32_t s) { return bar0 + 8 * (C::STAGES + s); };
  constexpr uint32_t kAccBar0 = 2 * C::STAGES;
  const auto accf_bar = [&](uint32_t b) { return bar0 + 8 * (kAccBar0 + b); };
  const auto acce_bar = [&](uint32_t b) { return bar0 + 8 * (kAccBar0 + 2 + b); };
  const uint32_t drain_bar = bar0 + 8 * (kAccBar0 + 4);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + (bar0 - base) + 8 * (kAccBar0 + 5));
  volatile uint32_t* const abort_flag = tmem_slot + 1;

  const uint32_t warp = warp_idx_sync();
  const uint32_t lane = lane_idx();
  const uint32_t rank = (CG == 2) ? cluster_cta_rank() : 0u;
  const bool leader = rank == 0;
  const uint32_t cluster_id = blockIdx.x / CG;
  const uint32_t G = gridDim.x / CG;
  const Watchdog wd{args.status, args.timeout_ns, abort_flag};

  // ---- set-up ------------------------------------------------------------------
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmAll);
      tma_prefetch_desc(&tmCompact);
      tma_prefetch_desc(&tmQ);
      if constexpr (C::kBoxes) tma_prefetch_desc(&tmOut);
      *abort_flag = 0u;
    }
    for (uint32_t i = lane; i < kAccBar0 + 5; i += 32)
      mbar_init(bar0 + 8 * i, (i == kAccBar0 + 2 || i == kAccBar0 + 3) ? C::kEpiWarps * CG : 1u);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc<CG>(smem_addr(tmem_slot), C::TMEM_COLS);
    tmem_relinquish<CG>();
  }
  grid_dependents_launch();
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

  // the rows, their number and their entries are earlier kernels'.  In place, ahead of the
  // first piece, there are only entries, which the epilogue takes: the operands are on their
  // way while a few rows' lists are sorted (by a kernel that writes no operand and began after
  // all work before the call).  Before later pieces the wait would count as the watchdog's.
  if (warp > 1 || args.count != nullptr || args.first != 0) grid_dependency_wait();
  const uint32_t count = args.count != nullptr ? min(*args.count, args.M) : args.M;
  const uint32_t rbs = (count + C::LT - 1) / C::LT, vts = (args.N + args.nt - 1) / args.nt;
  const uint32_t tiles = rbs * vts;
  const uint32_t kt_n = (args.K + C::BK - 1) / C::BK;

  if (warp < 4) {
    if constexpr (C::kSplit) regs_dec<C::kFewRegs>();
    if (warp == 0) {
      // ==================== TMA producer: one thread issues =======================
      const uint64_t pol = l2_policy_evict_last();
      const uint32_t q_rows = args.nt / CG, q_bytes = q_rows * 128;
      const CUtensorMap* const tmP = args.index != nullptr && count < args.M ? &tmCompact : &tmAll;
      RingStage r;
      uint32_t it = 0;
      bool ok = true;
      for (uint32_t t = cluster_id; ok && t < tiles; t += G) {
        uint32_t rb, vt;
        tile_coords(t, rbs, vts, kLossRaster, rb, vt);
        // boxes of A that a CTA of the tile loads (one without rows loads one: its stage is waited for)
        const auto boxes = [&](uint32_t p) {
          const uint32_t live = count > p ? min(128u, count - p) : 1u;
          return (live + C::P_BOX - 1) / C::P_BOX;
        };
        const uint32_t p0 = rb * C::LT + rank * 128, p_boxes = boxes(p0);
        const uint32_t tx = CG * q_bytes + (CG == 2 ? boxes(rb * C::LT) + boxes(rb * C::LT + 128) : p_boxes) * C::P_BOX * 128;
        const int32_t px = static_cast<int32_t>(p0), qy = static_cast<int32_t>(vt * args.nt + rank * q_rows);
        for (uint32_t kt = 0; kt < kt_n; ++kt, ++it, r.next<C::STAGES>()) {
          if (it == args.stall_iter) continue;   // watchdog test: this stage never fills
          if (!uniform_wait(empty_bar(r.s), r.round ^ 1u, wd, kSiteProducerEmpty, lane)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const uint32_t sb = base + r.s * C::STAGE_BYTES;
            const int32_t k0 = static_cast<int32_t>(kt * C::BK);
            uint32_t bar = full_bar(r.s);
            if constexpr (CG == 2) bar = mapa_shared(full_bar(r.s), 0);
            if (leader) mbar_arrive_expect_tx(full_bar(r.s), tx);
            const auto load = [&](uint32_t dst, const CUtensorMap* m, int32_t y) {
              if (CG == 2) tma_load_3d_pair(dst, m, bar, k0, y, 0, pol);
              else tma_load_3d(dst, m, bar, k0, y, 0, pol);
            };
            for (uint32_t i = 0; i < (CG == 2 ? 1u : p_boxes); ++i)
              load(sb + i * C::P_BOX * 128, tmP, px + static_cast<int32_t>(i * C::P_BOX));
            load(sb + C::P_BYTES, &tmQ, qy);
          }
          __syncwarp();
        }
      }
      // Exit path after a give-up: let this CTA's issued loads land first.
      if (lane == 0 && leader && *abort_flag) {
        const uint32_t first = it > C::STAGES ? it - C::STAGES : 0u;
        for (uint32_t i = first; i < it; ++i) {
          if (i == args.stall_iter) continue;
          drain_wait(full_bar(i % C::STAGES), (i / C::STAGES) & 1u, wd, kSiteProducerDrain);
        }
      }
    } else if (warp == 1) {
      // ==================== MMA issuer: the leader CTA's, one thread issues ========
      if (leader) {
        const uint32_t idesc = idesc_f16(C::LT, args.nt, 1u, false, false);
        const uint64_t pd0 = smem_desc_sw128(base), qd0 = smem_desc_sw128(base + C::P_BYTES);
        RingStage r;
        uint32_t j = 0;
        bool ok = true, issued = false;
        for (uint32_t t = cluster_id; ok && t < tiles; t += G) {
          for (uint32_t k_begin = 0; ok && k_begin < kt_n; ++j) {
            const uint32_t k_end = kt_n - k_begin > C::SEG_TILES ? k_begin + C::SEG_TILES : kt_n;
            const uint32_t b = j & 1u;
            // accumulator b must have been drained by every epilogue warp
            if (!uniform_wait(acce_bar(b), ((j >> 1) & 1u) ^ 1u, wd, kSiteMmaAccEmpty, lane)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint32_t d_tmem = tmem_base + b * C::ACC_COLS;
            for (uint32_t kt = k_begin; kt < k_end; ++kt) {
              if (!uniform_wait(full_bar(r.s), r.round, wd, kSiteMmaFull, lane)) {
                ok = false;
                break;
              }
              tc_fence_after_sync();
              const uint64_t step = static_cast<uint64_t>(r.s * (C::STAGE_BYTES / 16));
              const uint32_t left = args.K - kt * C::BK;   // (no MMAs over nothing but the zeros past the width)
              if (lane == 0) {
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k)   // 16 k per MMA: 32 bytes along a row
                  if (16 * k < left)
                    mma_bf16<CG>(d_tmem, pd0 + step + 2 * k, qd0 + step + 2 * k, idesc, (kt != k_begin || k != 0u));
                commit_to<CG>(empty_bar(r.s));     // frees the stage once these MMAs finish
              }
              __syncwarp();
              issued = true;
              r.next<C::STAGES>();
            }
            if (!ok) break;
            if (lane == 0) commit_to<CG>(accf_bar(b));
            k_begin = k_end;
          }
        }
        // Exit path: every tcgen05 op this thread issued completes before TMEM is released.
        if (issued && lane == 0) {
          if constexpr (CG == 1)
            tc_commit(drain_bar);
          else
            tc_commit_pair_multicast(drain_bar, 0x1);
          drain_wait(drain_bar, 0, wd, kSiteMmaDrain);
        }
      }
    }
  } else {
    // ==================== epilogue: eight warps, two per TMEM lane quarter =======
    if constexpr (C::kSplit) regs_inc<C::kManyRegs>();
    const uint32_t q = warp & 3u;              // TMEM lanes 32q .. 32q + 31
    const uint32_t eg = (warp - 4u) / 4u;      // this warp's half of the tile's chunks of 32 columns
    const uint32_t ch0 = eg == 0 ? 0u : (args.nt / 32 + 1) / 2, chunks = eg == 0 ? (args.nt / 32 + 1) / 2 : args.nt / 32 - ch0;
    uint32_t j = 0, sent = 0;
    bool ok = true;
    const auto counts = [&](uint32_t r) {      // in place: whether row r does
      return LIST ? args.len[r] > 0 : loss_index_at(args.target, args.target64, r) >= 0;
    };
    // Backward, in place: A's rows copied without those left out, in pieces of 8 elements, the last of a
    // row element by element.  Between segments, whose sums would else wait for it (105 rows, 1598
    // tokens of width 6488: 26.2 us for 31.1); ahead of everything where there is one.
    const uint32_t rows = args.lo_row + args.M, per = (args.K + 7) / 8;
    const uint64_t pieces = BACK && args.clean != nullptr ? static_cast<uint64_t>(rows) * per : 0ull;   // (few rows, of any width)
    uint64_t piece = blockIdx.x * 256u + threadIdx.x - 128u;
    const auto copy = [&]() {                  // four of them
      uint4 v[4];
      uint32_t to_row[4], e[4];
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k, piece += gridDim.x * 256u) {
        to_row[k] = 0xFFFFFFFFu;
        if (piece >= pieces) continue;
        to_row[k] = static_cast<uint32_t>(pieces >> 32 ? piece / per : static_cast<uint32_t>(piece) / per);
        e[k] = static_cast<uint32_t>(piece - static_cast<uint64_t>(to_row[k]) * per) * 8;
        const uint32_t r = args.lo_row != 0 && to_row[k] >= args.lo_row ? to_row[k] - args.lo_row : to_row[k];
        const uint16_t* const from = args.A + r * args.lda + e[k];
        v[k] = make_uint4(0, 0, 0, 0);
        if (r < args.M && counts(r)) {
          if (e[k] + 8 <= args.K) {
            v[k] = __ldg(reinterpret_cast<const uint4*>(from));
          } else {
            uint16_t x[8] = {};
#pragma unroll
            for (uint32_t i = 0; i < 7; ++i)
              if (e[k] + i < args.K) x[i] = from[i];
            v[k] = make_uint4(x[0] | static_cast<uint32_t>(x[1]) << 16, x[2] | static_cast<uint32_t>(x[3]) << 16,
                              x[4] | static_cast<uint32_t>(x[5]) << 16, x[6]);
          }
        }
      }
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)         // (the pitch has room for whole pieces)
        if (to_row[k] != 0xFFFFFFFFu) *reinterpret_cast<uint4*>(args.clean + to_row[k] * args.ld_clean + e[k]) = v[k];
    };
    if constexpr (BACK) {
      if (blockIdx.x == 0 && threadIdx.x == 128 && pieces > 0) args.offsets[0] = 0, args.offsets[1] = static_cast<int32_t>(rows);
      if constexpr (!SEG)
        while (piece < pieces) copy();
    }
    // forward, `runs`: largest and sums over this cluster's tiles so far
    float run_m = -INFINITY, run_s = 0.0f, run_z = 0.0f;
    // a tile's place, and this lane's row among all rows: loaded a tile ahead
    uint32_t rb = 0, vt = 0, at_ahead = 0;
    const auto look = [&](uint32_t t) {
      if (t >= tiles) return;
      tile_coords(t, rbs, vts, kLossRaster, rb, vt);
      const uint32_t row = rb * C::LT + rank * 128 + q * 32 + lane;
      at_ahead = row < count ? (args.index != nullptr ? args.index[row] : row) : 0u;
    };
    look(cluster_id);
    for (uint32_t t = cluster_id; ok && t < tiles; t += G) {
      const uint32_t row = rb * C::LT + rank * 128 + q * 32 + lane, at = at_ahead, column = vt;
      const bool live = row < count && (!BACK || args.row != nullptr || counts(row));
      const bool any = row - lane < count;               // some lane of the warp has a row
      const uint32_t n0 = vt * args.nt + ch0 * 32;       // this warp's first column
      const uint32_t cols = args.N > n0 ? min(chunks * 32, args.N - n0) : 0u;
      // The first entry in this warp's columns: its offset from n0, 0xFFFFFFFF where there is none; a
      // list's next one is known ahead.  Three loads that wait for each other, of a target one: where the
      // sums have segments, each is on its way while a segment is added up.
      const uint32_t here = chunks * 32, from = args.first + n0;
      uint32_t next = 0xFFFFFFFFu, ahead = 0xFFFFFFFFu;
      uint32_t cur = 0, end = 0xFFFFFFFFu, len = 0, id[3];
      float p_next = 0.0f, p_ahead = 0.0f;
      int64_t target = -1;
      float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);    // backward: the row's factors
      const uint64_t list = LIST ? static_cast<uint64_t>(at) * args.top : 0ull;
      const auto look_up = [&]() {
        if (!live) return;
        if constexpr (LIST) {
          len = args.len[at];
          if (args.start != nullptr) {
            const uint64_t bucket = min(from / args.bucket, kLossBuckets - 1);
            cur = args.start[bucket * args.M + at];
            end = args.start[(bucket + 1) * args.M + at];
          }
        } else {
          target = loss_index_at(args.target, args.target64, at);
        }
      };
      const auto search = [&]() {
        if (!live) return;
        if constexpr (BACK) r = args.row != nullptr ? args.row[row] : loss_row_factors(args.factors, args.target, args.target64, row);
        if constexpr (LIST) {
          end = min(end, len);
          while (end - cur > 2) {
            const uint32_t mid = (cur + end) / 2;
            if (static_cast<uint32_t>(args.ids[list + mid]) < from) cur = mid + 1; else end = mid;
          }
#pragma unroll
          for (uint32_t e = 0; e < 3; ++e) id[e] = cur + e < len ? static_cast<uint32_t>(args.ids[list + cur + e]) : 0xFFFFFFFFu;
        } else {
          const int64_t d = target - from;
          next = d >= 0 && d < here ? static_cast<uint32_t>(d) : 0xFFFFFFFFu;
        }
      };
      // (an offset's probability: only where the offset is this tile's)
      const auto entry = [&](uint32_t e, uint32_t token, float& p) {
        if (token == 0xFFFFFFFFu || token - from >= here) return 0xFFFFFFFFu;
        if constexpr (BACK) p = args.prob[list + e];
        return token - from;
      };
      const auto settle = [&]() {
        if (!LIST || !live) return;
#pragma unroll
        for (uint32_t e = 0; e < 2; ++e)
          if (id[0] < from) {
            ++cur;
            id[0] = id[1];
            id[1] = id[2];
            id[2] = 0u;   // not loaded
          }
        if (id[1] < from && cur + 1 < len) id[1] = static_cast<uint32_t>(args.ids[list + cur + 1]);
        next = entry(cur, id[0], p_next);
        ahead = entry(cur + 1, id[1], p_ahead);
      };
      const auto take = [&]() {
        ++cur;
        next = ahead;
        p_next = p_ahead;
        ahead = 0xFFFFFFFFu;
        if (next != 0xFFFFFFFFu && cur + 1 < len) ahead = entry(cur + 1, static_cast<uint32_t>(args.ids[list + cur + 1]), p_ahead);
      };
      look(t + G);
      // The hand-back of an accumulator whose reads are complete: it publishes nothing.
      const auto release = [&](uint32_t b) {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 1) mbar_arrive(acce_bar(b));
          else mbar_arrive_cluster_relaxed(mapa_shared(acce_bar(b), 0));
        }
      };
      const auto t_addr = [&](uint32_t ch) {
        return tmem_base + ((q * 32u) << 16) + (j & 1u) * C::ACC_COLS + (ch0 + ch) * 32;
      };
      const auto acc_wait = [&]() {
        ok = uniform_wait(accf_bar(j & 1u), (j >> 1) & 1u, wd, kSiteEpiAccFull, lane);
        tc_fence_after_sync();
        return ok;
      };
      look_up();
      if (!SEG || kt_n <= C::SEG_TILES) {
        search();
        settle();
      }
      // the tile's sums, by segments of the width
      float acc[C::NCH][32];
      const auto add_up = [&]() {
        for (uint32_t k = 0; k < kt_n; k += C::SEG_TILES, ++j) {
          if (!acc_wait()) return;
          if (any) {
#pragma unroll
            for (uint32_t i = 0; i < C::NCH; ++i) {
              if (i >= chunks) break;
              uint32_t v[32];
              tmem_ld_32x32b_x32_sync(t_addr(i), v);
              if (k == 0) {
#pragma unroll
                for (uint32_t e = 0; e < 32; ++e) acc[i][e] = __uint_as_float(v[e]);
              } else {
#pragma unroll
                for (uint32_t e = 0; e < 32; e += 2)
                  add_pair(acc[i][e], acc[i][e + 1], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              }
            }
          }
          release(j & 1u);
          if (kt_n > C::SEG_TILES) {
            if (k == 0) search();
            if (k == C::SEG_TILES) settle();
          }
          if constexpr (BACK)
            if (piece < pieces) copy();
        }
      };
      if constexpr (!BACK) {
        add_up();
        if (!ok) break;
        if (any) {
          // the entries' products
#pragma unroll
          for (uint32_t i = 0; i < C::NCH; ++i) {
            if (i >= chunks) break;
            while (__any_sync(0xffffffffu, next - 32 * i < 32u)) {
              const bool here = next - 32 * i < 32u;
              const float x = select32(acc[i], (next - 32 * i) & 31u);
              if (here && next < cols) args.entry[LIST ? static_cast<uint64_t>(at) * args.top + cur : at] = x;
              if (here) {
                if constexpr (LIST) take(); else next = 0xFFFFFFFFu;
              }
            }
          }
          float sum_z = 0.0f;
          if (cols < 32 * C::NCH) {   // columns past the tile's or the vocabulary's end
#pragma unroll
            for (uint32_t i = 0; i < C::NCH; ++i)
#pragma unroll
              for (uint32_t e = 0; e < 32; ++e) {
                const bool in = 32 * i + e < cols;
                sum_z += in ? acc[i][e] : 0.0f;
                if (!in) acc[i][e] = -INFINITY;
              }
          } else if (args.part_sum != nullptr) {
#pragma unroll
            for (uint32_t i = 0; i < C::NCH; ++i) {
              float part = 0.0f;
#pragma unroll
              for (uint32_t e = 0; e < 32; ++e) part += acc[i][e];
              sum_z += part;
            }
          }
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (uint32_t i = 0; i < C::NCH; ++i)
#pragma unroll
            for (uint32_t e = 0; e < 32; ++e) top[e & 3] = fmaxf(top[e & 3], acc[i][e]);
          float m = args.c * fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
          if (args.runs) m = fmaxf(m, run_m);
          const float shift = m == -INFINITY ? 0.0f : m;   // (nothing but masked columns: sums of 0)
          float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (uint32_t i = 0; i < C::NCH; ++i)
#pragma unroll
            for (uint32_t e = 0; e < 32; ++e) s[e & 3] += exp2_approx(fmaf(args.c, acc[i][e], -shift));
          float sum = (s[0] + s[1]) + (s[2] + s[3]);
          if (args.runs) {
            sum += run_s * exp2_approx(run_m - shift);
            run_m = m;
            run_s = sum;
            run_z += sum_z;
            sum_z = run_z;
          }
          if (live && (!args.runs || t + G >= tiles)) {
            const uint64_t o = ((args.runs ? cluster_id : column) * 2ull + eg) * args.ld_part + row;
            args.part[o] = make_float2(m, sum);
            if (args.part_sum != nullptr) args.part_sum[o] = sum_z;
          }
        }
      } else {
        // the product that sums over rows takes 64 at a time
        const uint32_t padded = args.lo_row != 0 ? args.lo_row : min((count + 63) / 64 * 64, args.M);
        // chunk i's gradient from its sums
        const auto finish = [&](uint32_t i, float(&g)[32], bool all_live) {
#pragma unroll
          for (uint32_t e = 0; e < 32; e += 2) {
            fma_pair(args.c, g[e], g[e + 1], -r.x);
            g[e] = exp2_approx(g[e]);
            g[e + 1] = exp2_approx(g[e + 1]);
            fma_pair(r.y, g[e], g[e + 1], -r.z);
          }
          while (__any_sync(0xffffffffu, next - 32 * i < 32u)) {
            const uint32_t w = next - 32 * i;
            const float x = LIST ? r.w * p_next : r.w;
            float xs[4];
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) xs[k] = (w & 3u) == k ? x : 0.0f;
#pragma unroll
            for (uint32_t e = 0; e < 32; ++e) g[e] = w / 4 == e / 4 ? g[e] - xs[e % 4] : g[e];
            if (w < 32u) {
              if constexpr (LIST) take(); else next = 0xFFFFFFFFu;
            }
          }
          if (!all_live) {   // (a padding row's accumulator is whatever its operand's rows held)
#pragma unroll
            for (uint32_t e = 0; e < 32; ++e) g[e] = live ? g[e] : 0.0f;
          }
          if (32 * i >= cols) return;
          // 32 rows of the piece from at_row on, which no multiple of 64 divides
          const auto send = [&](const uint32_t(&x)[16], uint32_t at_row) {
            if (C::kBoxes && args.boxes) {                 // (rows past the buffer's are left out)
              const uint32_t box = out0 + ((warp - 4u) * 2 + (sent & 1u)) * C::BOX_BYTES;
              ++sent;
              if (lane == 0) bulk_wait_group_read<1>();    // the store before the last has read it
              __syncwarp();
              stage_half_row(box, lane, x);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_3d(&tmOut, box, static_cast<int32_t>(n0 + 32 * i), static_cast<int32_t>(at_row), 0);
                bulk_commit_group();
              }
            } else if (row < (at_row >= padded ? args.M : padded)) {
              uint16_t* const o = args.out + static_cast<uint64_t>(at_row + lane) * args.ld_out + n0 + 32 * i;
              st_global_v8(o, x);
              st_global_v8(o + 16, x + 8);
            }
          };
          uint32_t x[16];
#pragma unroll
          for (uint32_t e = 0; e < 16; ++e) x[e] = pack_bf16x2(g[2 * e], g[2 * e + 1]);
          send(x, row - lane);
          if (args.lo_row != 0 && row - lane < args.M) {
#pragma unroll
            for (uint32_t e = 0; e < 16; ++e)
              x[e] = pack_bf16x2(g[2 * e] - bf16_bits_to_f32(x[e] & 0xFFFFu), g[2 * e + 1] - bf16_bits_to_f32(x[e] >> 16));
            send(x, args.lo_row + row - lane);
          }
        };
        if constexpr (SEG) {
          add_up();
          if (!ok) break;
          if (row - lane < padded) {
            const bool all_live = __all_sync(0xffffffffu, live);
#pragma unroll
            for (uint32_t i = 0; i < C::NCH; ++i)
              if (i < chunks) finish(i, acc[i], all_live);
          }
        } else {
          if (!acc_wait()) break;
          const uint32_t b = j & 1u;
          if (row - lane < padded && chunks > 0) {
            const bool all_live = __all_sync(0xffffffffu, live);
#pragma unroll 1
            for (uint32_t i = 0; i < chunks; ++i) {
              uint32_t v[32];
              tmem_ld_32x32b_x32_sync(t_addr(i), v);
              if (i + 1 == chunks) release(b);
              float g[32];
#pragma unroll
              for (uint32_t e = 0; e < 32; ++e) g[e] = __uint_as_float(v[e]);
              finish(i, g, all_live);
            }
          } else {
            release(b);
          }
          ++j;
        }
      }
    }
    if constexpr (BACK)
      while (piece < pieces) copy();
    if (C::kBoxes && lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  // ---- teardown: every role is done with TMEM and with the peer's barriers ----
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc<CG>(tmem_base, C::TMEM_COLS);
  }
}

}  // namespace gb300
