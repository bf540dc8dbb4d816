// The losses' deal of items on the host, for test_loss_deal.py.
#include "loss_deal.h"

#include <vector>

using namespace gb300;

// A deal for these sizes, checked by walking all clusters' items: out = {parts, parts_db, items
// missing, items dealt twice, stages until the last cluster ends (x 16), the same if all ended
// together}.
extern "C" void loss_deal_walk(uint32_t M, uint32_t count, uint32_t n, uint32_t K, uint32_t width, uint32_t nt, uint32_t lt,
                               uint32_t most, uint32_t most_db, uint32_t rows, uint32_t matrix, uint32_t db_cost, uint32_t G,
                               uint64_t* out) {
  LossProductArgs a = {};
  a.M = M, a.n = n, a.K = K, a.nt = nt, a.width = width, a.most = most, a.most_db = most_db;
  a.rows = rows, a.matrix = matrix, a.db_cost = db_cost, a.unit = loss_unit(a, lt);
  const LossDeal d = loss_deal_by(a, count, lt, G, [&](LossDeal& best, const LossWork& w, uint32_t clusters, uint32_t limit) {
    uint32_t least = 0xFFFFFFFFu;
    for (uint32_t s = 1; s <= kLossParts && s <= limit; ++s) {
      LossDeal one = best;
      const uint32_t time = loss_shares(w, s, clusters, one);
      if (time < least) least = time, best = one;
    }
  });
  const uint64_t per_x = static_cast<uint64_t>(d.rb_x) * d.cb, per_y = static_cast<uint64_t>(d.rb_y) * d.cb;
  std::vector<uint8_t> x(per_x * d.parts), y(per_y * d.parts_db);
  uint64_t twice = 0, last = 0, sum = 0;
  const uint64_t kt_x = (n + 63) / 64, kt_y = (count + 63) / 64;
  for (uint32_t c = 0; c < G; ++c) {
    uint64_t time = 0;
    bool m;
    uint32_t t, s;
    for (uint32_t i = 0; loss_item_at(d, c, G, i, m, t, s); ++i) {
      uint8_t& seen = m ? y[s * per_y + t] : x[s * per_x + t];
      twice += seen;
      seen = 1;
      const uint64_t kt = m ? kt_y : kt_x, parts = m ? d.parts_db : d.parts;
      const uint64_t k = kt * (s + 1) / parts - kt * s / parts;
      time += m ? (k + 3 > db_cost ? k + 3 : db_cost) : k + kLossEnds;
    }
    sum += time;
    last = time > last ? time : last;
  }
  uint64_t missing = 0;
  for (const uint8_t v : x) missing += !v;
  for (const uint8_t v : y) missing += !v;
  out[0] = d.parts, out[1] = d.parts_db, out[2] = missing, out[3] = twice, out[4] = 16 * last, out[5] = 16 * sum / G;
}
