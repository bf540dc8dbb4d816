// How the products with a piece of the logits' gradient (loss_products.cuh) deal their items to
// clusters: whole numbers only, the same on the host and in every kernel that works them out.
#pragma once

#include <cstdint>

#if defined(__CUDACC__)
#define GB300_HD __host__ __device__ __forceinline__
#else
#define GB300_HD inline
#endif

namespace gb300 {

struct LossDeal;
struct LossProductArgs {
  uint32_t M, n, K;            // rows at most, columns of the piece, width
  const LossDeal* deal;        // the deal for the rows that count (nullptr: all of them do, it is found here)
  uint32_t nt;                 // columns of a tile, a multiple of 64
  uint32_t width;              // of the first piece, by which the parts are chosen
  uint32_t most, most_db;      // parts at most, of Rows and of Matrix
  uint32_t rows, matrix;       // which of them are wanted
  uint32_t direct;             // Rows to dA, bf16 (1) or fp32 (2), where there is nothing to join (0: never)
  uint32_t add_sums, add_db;   // added to what is there
  uint32_t db_cost;            // a tile of dB's store in stages
  uint32_t unit;               // times are counted in 2^unit stages (loss_unit)
  unsigned long long* status;
  unsigned long long timeout_ns;
};

// Matrix's reduction to the rows goes in `parts_db` where it has so few tiles that clusters would
// idle.  Rows' reduction over the piece goes in `parts`, and its items in turn to the G clusters,
// so that the first `r` have one more than the others' x; Matrix's follow, n1 at most to each of
// those and n0 to each of the others, who end no later for it.
struct LossDeal {
  uint32_t count, rb_x, rb_y, cb;      // rows that count; tiles down, of either, and across
  uint32_t parts, parts_db, x, r, n1, n0;
  bool direct;                         // Rows go to dA: one part, and no row left out
};

// What is dealt: `kt` stages a tile over `tiles` tiles of Rows, `others` items of Matrix of `cost`
// stages each; each part of Rows costs its sums' way to memory and back (`extra` stages over all
// clusters); times are counted in 2^unit stages.
struct LossWork {
  uint32_t tiles, others, kt, cost, extra, unit;
};

constexpr uint32_t kLossParts = 32;                      // Rows' at most, as a warp's lanes
constexpr uint32_t kLossEnds = 5;                        // an item's first loads and last store, in stages

GB300_HD uint32_t loss_units(uint32_t stages, uint32_t unit) { return (stages + (1u << unit) - 1) >> unit; }

// The deal of Rows in s parts, and the units until the last cluster ends.
GB300_HD uint32_t loss_shares(const LossWork& w, uint32_t s, uint32_t G, LossDeal& d) {
  const uint32_t items = w.tiles * s, x = items / G, r = items - x * G, rest = G - r;
  const uint32_t cost = loss_units(w.cost, w.unit), each = loss_units((w.kt + s - 1) / s + kLossEnds, w.unit);
  const uint32_t l0 = x * each, l1 = r > 0 ? l0 + each : l0;
  uint32_t t = (r * l1 + rest * l0 + w.others * cost + G - 1) / G;
  t = t > l1 ? t : l1;
  uint32_t n1 = 0, n0 = 0;
  for (uint32_t i = 0; i < 4; ++i) {
    n1 = (t - l1) / cost;
    n0 = (t - l0) / cost;
    if (r * n1 + rest * n0 >= w.others) break;
    const uint32_t a = l0 + (n0 + 1) * cost, b = l1 + (n1 + 1) * cost;
    t = a < b ? a : b;
  }
  if (r * n1 < w.others) {
    const uint32_t least = (w.others - r * n1 + rest - 1) / rest;
    n0 = n0 > least ? n0 : least;
  }
  d.parts = s;
  d.x = x;
  d.r = r;
  d.n1 = n1;
  d.n0 = n0;
  return t + loss_units(w.extra, w.unit) * s;
}

// For `count` rows, tiles of `lt` rows and G clusters; pick(d, work, G, most) finds the number of
// Rows' parts that ends first.
template <class Pick>
GB300_HD LossDeal loss_deal_by(const LossProductArgs& a, uint32_t count, uint32_t lt, uint32_t G, const Pick& pick) {
  LossDeal d;
  d.count = count;
  d.cb = (a.K + a.nt - 1) / a.nt;
  d.rb_x = a.rows ? (d.count + lt - 1) / lt : 0u;
  d.rb_y = a.matrix ? (a.n + lt - 1) / lt : 0u;
  // (by the first piece: later ones, which may be narrower, add to the same parts)
  const uint32_t tiles = a.matrix ? (a.width + lt - 1) / lt * d.cb : 0u, stages = (d.count + 63) / 64;
  // Matrix in parts of at least 8 stages, where that saves more than the sums' way to memory and
  // back (4 bytes at 5 TB/s, 0.3 us a stage) and the joining take: 4000 rows, 512 tokens of width
  // 256, 8 tiles of 63 stages, 19.5 us in parts and 28.3 whole; 1500, 512, 128, 4 of 24, 19.0 and 17.0
  d.parts_db = 1;
  if (tiles > 0 && a.most_db > 1 && stages <= 0x1000000u) {
    uint32_t n = G / tiles < stages / 8 ? G / tiles : stages / 8;
    n = n < a.most_db ? n : a.most_db;
    const uint32_t way = static_cast<uint32_t>(static_cast<uint64_t>(a.width) * a.K * n * 8 / 1500000);
    if (n > 1 && stages - (stages + n - 1) / n > way + 24) d.parts_db = n;
  }
  const uint32_t each = (stages + d.parts_db - 1) / d.parts_db + 3;
  LossWork w;
  w.tiles = d.rb_x * d.cb;
  w.others = tiles * d.parts_db;
  w.kt = (a.width + 63) / 64;
  w.cost = each > a.db_cost ? each : a.db_cost;
  // (Rows' sums, the same)
  w.extra = static_cast<uint32_t>(static_cast<uint64_t>(d.count) * a.K * 8 / 1500000);
  w.unit = a.unit;
  pick(d, w, G, a.most);
  d.direct = a.direct != 0u && d.parts == 1 && d.count == a.M;
  return d;
}

// The unit in which the times of all clusters together stay below 2^30, and with a unit more for
// each item (2^31 items at most) in 32 bits, whatever the number of rows that count.
inline uint32_t loss_unit(const LossProductArgs& a, uint32_t lt) {
  const uint64_t cb = (a.K + a.nt - 1) / a.nt, stages = (a.M + 63ull) / 64 + 3;
  const uint64_t cost = stages > a.db_cost ? stages : a.db_cost;
  const uint64_t all = (a.rows ? (a.M + lt - 1ull) / lt * cb * ((a.width + 63ull) / 64 + (kLossEnds + 1) * kLossParts) : 0) +
                       ((a.matrix ? (a.width + lt - 1ull) / lt * cb * a.most_db : 0) + 1) * cost +
                       static_cast<uint64_t>(a.M) * a.K * 8 / 1500000 * kLossParts;
  uint32_t unit = 0;
  while (all >> unit >> 30 != 0) ++unit;
  return unit;
}

// Cluster c's i-th item: tile t of part s of Rows or of Matrix.  False past the last.
GB300_HD bool loss_item_at(const LossDeal& d, uint32_t c, uint32_t G, uint32_t i, bool& matrix, uint32_t& t, uint32_t& s) {
  const uint32_t mine = d.x + (c < d.r ? 1u : 0u);
  matrix = i >= mine;
  const uint32_t per = (matrix ? d.rb_y : d.rb_x) * d.cb;
  t = c + i * G;
  if (matrix) {
    i -= mine;
    if (i >= (c < d.r ? d.n1 : d.n0)) return false;
    t = i < d.n1 ? c + i * G : d.n1 * G + (i - d.n1) * (G - d.r) + (c - d.r);
    if (t >= per * d.parts_db) return false;
  }
  s = t / per;
  t -= s * per;
  return true;
}

}  // namespace gb300
