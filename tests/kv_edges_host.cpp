// Host build of the cache's index functions: the attention and the append place
// a row alike, and cut sequences have places for their chunks.
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

// Units of sequences that are cut, and all units, against what a launch has for
// them.  `sane`: rows are each one sequence's and `units` was made for that many
// row tiles, so that it has to suffice, too.
extern "C" int places_suffice(const int32_t* ctx, const int32_t* cu, int seqs, int columns, int rows, int share, int bm,
                              int kt, int units, int aim, int spare, int least, int sane, int* longest_chunks) {
  KvView c{};
  c.ctx = ctx, c.cu = cu, c.seqs = seqs, c.rows = rows, c.lgp = 4, c.columns = columns;
  const AttnShape a{share, 0, 0, 1, INT32_MAX};
  const Cut cut{units, aim, spare};
  double sum = 0, work = 0;
  for (int b = 0; b < seqs; ++b) {
    const Seq s = seq_at(c, a, b, bm, kt);
    sum += s.qtiles;
    work += (double)s.qtiles * s.tiles;
  }
  const int per = chunk_tiles(work, sum, used_units(cut, sum), least);
  int64_t all = 0, places = 0;
  *longest_chunks = 0;
  for (int b = 0; b < seqs; ++b) {
    const Seq s = seq_at(c, a, b, bm, kt);
    const int chunks = chunks_of(s, per);
    all += (int64_t)s.qtiles * chunks;
    if (chunks > 1) places += (int64_t)s.qtiles * chunks;
    if (chunks > *longest_chunks) *longest_chunks = chunks;
  }
  if (places > places_of(cut)) return 1;
  return sane && all > units ? 2 : 0;
}
