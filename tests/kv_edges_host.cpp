// Host build of the cache's index functions: the attention and the append place
// a row alike.
#include "kv_index.h"

#include <cmath>

using namespace kronq;

// 0, or 1 + the first row whose position in the attention (its sequence's end,
// counted back) is not the append's.  Positions before a sequence's start are alike.
extern "C" int places_differ(const int32_t* ctx, const int32_t* cu, int seqs, int rows) {
  KvView c{};
  c.ctx = ctx, c.cu = cu, c.seqs = seqs, c.rows = rows, c.lgp = 4;
  const AttnShape a{1, 0, 0, 1, INT32_MAX};
  for (int b = 0; b < seqs; ++b) {
    const Seq s = seq_at(c, a, b, 16, 32);
    for (int t = 0; t < s.len; ++t) {
      const int64_t pos = (int64_t)s.ctx - s.len + t;
      const Place p = place_of(c, b, s.row0 + t, cu[b + 1]);
      if (pos != p.pos && (pos >= 0 || p.pos >= 0)) return 1 + s.row0 + t;
    }
  }
  return 0;
}
