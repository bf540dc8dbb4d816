// The two products with a piece of the logits' gradient g [rows, n] (bf16, compact rows,
// zeros in the rows between `count` and the next multiple of 64):
//
//     Rows    sums[s][r, k] (+)= sum over the s-th part of the piece's v of g[r, v] B[v, k]
//     Matrix  dB[v, k]      (+)= sum_r g[r, v] A[r, k]
//
// Output rows sit in the TMEM lanes (the MMA's M), the width in its columns (N): a width
// that fills no tile costs what it holds, in steps of 32 (16 on one CTA).  A warp stages
// 32 rows of 128 bytes in shared memory and stores them by TMA, which leaves out what lies
// past the output's ends and adds in L2 what is to be added in fp32 (129 rows, 32768 tokens
// of width 2048, both gradients: 3 us of 100 less than from registers, each lane its own row
// in whole sectors).  Rows has few tiles and a long reduction,
// so it is dealt to the clusters in parts, whose sums lie apart and are joined in order:
// the same bits every time.  Matrix has many tiles, or, of a small matrix and many rows, goes in
// parts too.  One launch takes the items of both in turn, so that one last round is ragged
// instead of two.
//
// Bounds.  Thousands of rows are bound by the MMAs (4096 rows, 32768 tokens of width 4096:
// 1134 us for both, 1.94 PFLOP/s, tensor pipes 97.8 % busy), few by B's read and dB's write
// (48 rows, 131072 tokens: 402 us, 5.4 TB/s; the write alone goes at 5.9, a fill at 4.0).
//
// Persistent, warp-specialised like the other products: a TMA producer, an MMA issuer with
// two accumulators, eight epilogue warps (two per lane quarter, alternating 32-column
// chunks).
#pragma once

#include "gemm_kernels.cuh"
#include "grouped_kernels.cuh"
#include "loss_deal.h"
#include "ptx_grouped.cuh"
#include "ptx_loss.cuh"

namespace gb300 {

template <int CG>
struct LossProductCfg {
  static constexpr uint32_t BK = 64;
  static constexpr uint32_t LT = 128 * CG;               // output rows per tile
  static constexpr uint32_t NT = 128 * CG;               // columns per tile at most
  static constexpr uint32_t P_BYTES = 128 * 128, Q_BYTES = 128 * 128;   // a CTA's 128 rows, 128 columns
  static constexpr uint32_t STAGE_BYTES = P_BYTES + Q_BYTES;
  static constexpr uint32_t kEpiWarps = 8;
  static constexpr uint32_t kThreads = 32 * (2 + kEpiWarps);
  static constexpr uint32_t kLeastRegs = 0;              // (any number will do)
  static constexpr uint32_t BAR_BYTES = 512;
  static constexpr uint32_t SMEM_LIMIT = 232448;
  static constexpr uint32_t ALIGN_SLACK = 1024;
  static constexpr uint32_t BOX_BYTES = 32 * 128;        // a warp's rows on their way out
  static constexpr uint32_t OUT_BYTES = kEpiWarps * BOX_BYTES;
  static constexpr uint32_t STAGES = (SMEM_LIMIT - ALIGN_SLACK - BAR_BYTES - OUT_BYTES - 64 * 24) / STAGE_BYTES;
  static constexpr uint32_t ITEM_BYTES = 64 * 24;        // a cluster's first items
  static constexpr uint32_t SMEM_BYTES = ALIGN_SLACK + STAGES * STAGE_BYTES + OUT_BYTES + BAR_BYTES + ITEM_BYTES;
  static_assert((2 * STAGES + 5) * 8 + 16 <= BAR_BYTES, "barrier area");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t ACC_COLS = 256;
};

// The deal that ends first: the 32 lanes try a number of parts each.
struct LossPick {
  __device__ __forceinline__ void operator()(LossDeal& d, const LossWork& w, uint32_t G, uint32_t most) const {
    const uint32_t s = lane_idx() + 1, found = loss_shares(w, s, G, d), time = s <= most ? found : 0xFFFFFFFFu;
    const uint32_t best = __reduce_min_sync(0xffffffffu, time);
    const int lane = __ffs(__ballot_sync(0xffffffffu, time == best)) - 1;
    d.parts = static_cast<uint32_t>(lane) + 1;
    d.x = __shfl_sync(0xffffffffu, d.x, lane);
    d.r = __shfl_sync(0xffffffffu, d.r, lane);
    d.n1 = __shfl_sync(0xffffffffu, d.n1, lane);
    d.n0 = __shfl_sync(0xffffffffu, d.n0, lane);
  }
};

__device__ __forceinline__ LossDeal loss_deal(const LossProductArgs& a, uint32_t count, uint32_t lt, uint32_t G) {
  return loss_deal_by(a, count, lt, G, LossPick{});
}

// The same, once the kernels before the product's have ended: found ahead where rows may be left out.
template <int CG>
__device__ __forceinline__ LossDeal loss_deal_of(const LossProductArgs& a, uint32_t G) {
  constexpr uint32_t LT = 128 * CG;
  if (a.deal == nullptr) return loss_deal(a, a.M, LT, G);
  LossDeal d = *a.deal;
  d.rb_y = a.matrix ? (a.n + LT - 1) / LT : 0u;          // (by this piece)
  return d;
}

// Cluster c's i-th item: rows l0.., columns c0.., stages k0 .. k1 - 1; part s of Rows or of
// Matrix.  False past the last.
struct LossItem {
  uint32_t l0, c0, k0, k1, s;
  uint16_t matrix, valid;
};
// (a cluster's first kLossAhead are worked out ahead by as many threads: the divisions
// would otherwise stand between two tiles)
constexpr uint32_t kLossAhead = 64;
template <int CG>
__device__ __forceinline__ bool loss_item(const LossProductArgs& a, const LossDeal& d, uint32_t c, uint32_t G, uint32_t i,
                                          LossItem& w) {
  bool matrix;
  uint32_t t, rb, cb;
  if (!loss_item_at(d, c, G, i, matrix, t, w.s)) return false;
  w.matrix = matrix ? 1 : 0;
  tile_coords(t, matrix ? d.rb_y : d.rb_x, d.cb, 8u, rb, cb);
  w.l0 = rb * 128 * CG;
  w.c0 = cb * a.nt;
  const uint32_t kt = ((matrix ? d.count : a.n) + 63) / 64, parts = matrix ? d.parts_db : d.parts;
  // (several parts: 32 of at most 2^25 stages, or 152 of 2^24)
  w.k0 = parts == 1 ? 0u : kt * w.s / parts;
  w.k1 = parts == 1 ? kt : kt * (w.s + 1) / parts;
  return true;
}

// g by its rows (boxes of 128) and by its columns, B's piece and the rows of A, all and those
// that count (boxes of 64 x 64); the sums [parts][M][K] and [parts_db][n][K], dA and dB's rows
// of the piece (boxes of 128 bytes x 32).
struct LossMaps {
  CUtensorMap g_rows, g_columns, B, A, compact, sums, sums_db, dA, dB;
};

// T: dB's elements, uint32_t (fp32) or uint16_t (bf16).
template <int CG, class T>
__global__ void __launch_bounds__(LossProductCfg<CG>::kThreads, 1)
    loss_product_kernel(const __grid_constant__ LossMaps maps, const LossProductArgs args) {
  using C = LossProductCfg<CG>;
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
      tma_prefetch_desc(&maps.g_rows);
      tma_prefetch_desc(&maps.g_columns);
      tma_prefetch_desc(&maps.B);
      tma_prefetch_desc(&maps.A);
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
  // (every thread: g is an earlier kernel's; the number of rows only where some may be left out,
  // else the items are dealt ahead)
  if (args.deal != nullptr) grid_dependency_wait();
  const LossDeal deal = loss_deal_of<CG>(args, G);
  static_assert(sizeof(LossItem) == 24 && C::ITEM_BYTES == kLossAhead * sizeof(LossItem), "the items' table");
  LossItem* const ahead = reinterpret_cast<LossItem*>(base_ptr + (bar0 - base) + C::BAR_BYTES);
  if (threadIdx.x < kLossAhead) {
    LossItem w;
    w.valid = loss_item<CG>(args, deal, cluster_id, G, threadIdx.x, w) ? 1 : 0;
    ahead[threadIdx.x] = w;
  }
  __syncthreads();
  if (args.deal == nullptr) grid_dependency_wait();
  const auto item = [&](uint32_t i, LossItem& w) {
    if (i >= kLossAhead) return loss_item<CG>(args, deal, cluster_id, G, i, w);
    w = ahead[i];
    return w.valid != 0;
  };

  if (warp == 0) {
    // ==================== TMA producer: one thread issues =======================
    const uint64_t pol = l2_policy_evict_last();
    RingStage r;
    uint32_t it = 0;
    bool ok = true;
    LossItem w;
    for (uint32_t i = 0; ok && item(i, w); ++i) {
      const uint32_t h = mma_n<CG>(min(args.nt, args.K - w.c0)) / CG;   // columns this CTA contributes to the MMA
      const uint32_t q_boxes = (h + 63) / 64;
      const uint32_t tx = CG * (C::P_BYTES + q_boxes * 8192);
      const int32_t px = static_cast<int32_t>(w.l0 + rank * 128), qx = static_cast<int32_t>(w.c0 + rank * h);
      const CUtensorMap* const tmQ = w.matrix ? (deal.count < args.M ? &maps.compact : &maps.A) : &maps.B;
      for (uint32_t kt = w.k0; kt < w.k1; ++kt, ++it, r.next<C::STAGES>()) {
        if (!uniform_wait(empty_bar(r.s), r.round ^ 1u, wd, kSiteProducerEmpty, lane)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const uint32_t sb = base + r.s * C::STAGE_BYTES;
          const int32_t k = static_cast<int32_t>(kt * C::BK);
          uint32_t bar = full_bar(r.s);
          if constexpr (CG == 2) bar = mapa_shared(full_bar(r.s), 0);
          if (leader) mbar_arrive_expect_tx(full_bar(r.s), tx);
          const auto load = [&](uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y) {
            if (CG == 2) tma_load_3d_pair(dst, m, bar, x, y, 0, pol);
            else tma_load_3d(dst, m, bar, x, y, 0, pol);
          };
          if (w.matrix) {
            load(sb, &maps.g_columns, px, k);
            load(sb + 8192, &maps.g_columns, px + 64, k);
          } else {
            load(sb, &maps.g_rows, k, px);
          }
          for (uint32_t b = 0; b < q_boxes; ++b)
            load(sb + C::P_BYTES + b * 8192, tmQ, qx + static_cast<int32_t>(64 * b), k);
        }
        __syncwarp();
      }
    }
    // Exit path after a give-up: let this CTA's issued loads land first.
    if (lane == 0 && leader && *abort_flag) {
      const uint32_t first = it > C::STAGES ? it - C::STAGES : 0u;
      for (uint32_t k = first; k < it; ++k)
        drain_wait(full_bar(k % C::STAGES), (k / C::STAGES) & 1u, wd, kSiteProducerDrain);
    }
  } else if (warp == 1) {
    // ==================== MMA issuer: the leader CTA's, one thread issues ========
    if (leader) {
      const uint64_t gr0 = smem_desc_sw128(base), gc0 = smem_desc_mn_sw128(base), qd0 = smem_desc_mn_sw128(base + C::P_BYTES);
      RingStage r;
      uint32_t j = 0;
      bool ok = true, issued = false;
      LossItem w;
      for (uint32_t i = 0; ok && item(i, w); ++i) {
        if (w.k0 == w.k1) continue;
        const uint32_t idesc = idesc_f16(C::LT, mma_n<CG>(min(args.nt, args.K - w.c0)), 1u, w.matrix, true);
        // 16 k: 16 rows of an MN-major tile, 32 bytes along a K-major row
        const uint64_t pd0 = w.matrix ? gc0 : gr0, p_step = w.matrix ? 128 : 2;
        const uint32_t length = w.matrix ? deal.count : args.n;   // (no MMAs over nothing but zeros past it)
        const uint32_t b = j & 1u;
        // accumulator b must have been drained by every epilogue warp
        if (!uniform_wait(acce_bar(b), ((j >> 1) & 1u) ^ 1u, wd, kSiteMmaAccEmpty, lane)) break;
        ++j;
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + b * C::ACC_COLS;
        for (uint32_t kt = w.k0; kt < w.k1; ++kt) {
          if (!uniform_wait(full_bar(r.s), r.round, wd, kSiteMmaFull, lane)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t step = static_cast<uint64_t>(r.s * (C::STAGE_BYTES / 16));
          if (lane == 0) {
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
              if (kt * C::BK + 16 * k < length)
                mma_bf16<CG>(d_tmem, pd0 + step + p_step * k, qd0 + step + 128 * k, idesc, (kt != w.k0 || k != 0u));
            commit_to<CG>(empty_bar(r.s));   // frees the stage once these MMAs finish
          }
          __syncwarp();
          issued = true;
          r.next<C::STAGES>();
        }
        if (!ok) break;
        if (lane == 0) commit_to<CG>(accf_bar(b));
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
  } else {
    // ==================== epilogue: eight warps, two per TMEM lane quarter =======
    const uint32_t q = warp & 3u;              // TMEM lanes 32q .. 32q + 31
    const uint32_t eg = (warp - 2u) / 4u;      // chunks eg, eg + 2, ...
    const uint32_t box = out0 + (warp - 2u) * C::BOX_BYTES;
    uint32_t j = 0;
    LossItem w;
    for (uint32_t i = 0; item(i, w); ++i) {
      // columns of a box: 128 bytes a row
      const bool apart = w.matrix && deal.parts_db > 1;   // Matrix's sums are joined later
      const bool bf16 = w.matrix ? sizeof(T) == 2 && !apart : deal.direct && args.direct == 1u;
      const uint32_t wide = bf16 ? 64u : 32u;
      const uint32_t nch = (min(args.nt, args.K - w.c0) + wide - 1) / wide;
      const int32_t row = static_cast<int32_t>(w.l0 + rank * 128 + q * 32);
      const bool add = w.matrix ? args.add_db != 0u && !apart : args.add_sums != 0u;
      // a box on its way: rows past the output's are nobody's
      const auto send = [&](uint32_t ch) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row < static_cast<int32_t>(w.matrix ? args.n : deal.count)) {
          const CUtensorMap* const out = apart ? &maps.sums_db : w.matrix ? &maps.dB : deal.direct ? &maps.dA : &maps.sums;
          const int32_t x = static_cast<int32_t>(w.c0 + ch * wide), z = static_cast<int32_t>(w.s);
          if (add) tma_add_3d(out, box, x, row, z);
          else tma_store_3d(out, box, x, row, z);
          bulk_commit_group();
        }
      };
      const auto box_free = [&]() {
        if (lane == 0) bulk_wait_group_read<0>();   // its last store has read it
        __syncwarp();
      };
      if (w.k0 == w.k1) {   // nothing is added up: zeros
        if (add) continue;
        const uint32_t v[32] = {};
        box_free();
        stage_row(box, lane, 0, v);
        for (uint32_t ch = eg; ch < nch; ch += 2) send(ch);
        continue;
      }
      const uint32_t b = j & 1u;
      if (!uniform_wait(accf_bar(b), (j >> 1) & 1u, wd, kSiteEpiAccFull, lane)) break;
      tc_fence_after_sync();
      ++j;
      bool held = true;
      // The hand-back of an accumulator whose reads are complete: it publishes nothing.
      const auto release = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 1) mbar_arrive(acce_bar(b));
          else mbar_arrive_cluster_relaxed(mapa_shared(acce_bar(b), 0));
        }
        held = false;
      };
      const uint32_t acc = tmem_base + ((q * 32u) << 16) + b * C::ACC_COLS;
#pragma unroll 1
      for (uint32_t ch = eg; ch < nch; ch += 2) {
        const bool last = ch + 2 >= nch;   // all of it is in registers: hand it back
        if (!bf16) {
          uint32_t v[32];
          tmem_ld_32x32b_x32_sync(acc + ch * 32, v);
          if (last) release();
          box_free();
          stage_row(box, lane, 0, v);
        } else {
          uint32_t v0[32], v1[32], x[32];
          tmem_ld2_32x32b_x32_sync(acc + ch * 64, acc + ch * 64 + 32, v0, v1);
          if (last) release();
#pragma unroll
          for (uint32_t e = 0; e < 16; ++e) {
            x[e] = pack_bf16x2(__uint_as_float(v0[2 * e]), __uint_as_float(v0[2 * e + 1]));
            x[16 + e] = pack_bf16x2(__uint_as_float(v1[2 * e]), __uint_as_float(v1[2 * e + 1]));
          }
          box_free();
          stage_row(box, lane, 0, x);
        }
        send(ch);
      }
      if (held) release();   // (a warp without a chunk)
    }
    if (lane == 0) bulk_wait_group<0>();
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
