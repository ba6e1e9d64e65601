// Host build of the cache's index functions: what they return for any content
// of the batch arrays stays inside the buffers, and the attention's units cover
// every visible key of every row once.
#include "kv_index.h"

#include <cmath>
#include <vector>

using namespace kronq;

extern "C" int rows_in_bounds(const int32_t* table, const int32_t* ctx, const int32_t* cu, int seqs, int columns,
                              int pages, int lgp, int rows) {
  KvView c{};
  c.table = table, c.ctx = ctx, c.cu = cu, c.ldt = columns, c.seqs = seqs, c.columns = columns;
  c.pages = pages, c.lgp = lgp, c.rows = rows;
  for (int r = 0; r < rows; ++r) {
    const int b = seq_of(cu, seqs, r);
    if (b < 0) continue;
    if (b >= seqs) return 1;
    const Place p = place_of(c, b, r, cu[b + 1]);
    if (p.page < 0 || p.page >= pages || p.slot < 0 || p.slot >= (1 << lgp)) return 2;
    if (!p.bad && (p.pos < 0 || (p.pos >> lgp) >= columns || table[(int64_t)b * columns + (p.pos >> lgp)] != p.page)) return 3;
  }
  return 0;
}

// 0, or what is wrong.  `sane`: the arrays are a valid batch, so that coverage
// can be asked for; units_used is what the cut took of `units`.
extern "C" int units_cover(const int32_t* table, const int32_t* ctx, const int32_t* cu, int seqs, int columns,
                           int pages, int lgp, int rows, int share, int window, int sinks, int bm, int kt, int units,
                           int least, int sane, int* units_used) {
  KvView c{};
  c.table = table, c.ctx = ctx, c.cu = cu, c.ldt = columns, c.seqs = seqs, c.columns = columns;
  c.pages = pages, c.lgp = lgp, c.rows = rows;
  const AttnShape a{share, window, sinks, 1, INT32_MAX};
  double sum_rows = 0, work = 0;
  for (int b = 0; b < seqs; ++b) {
    const Seq s = seq_at(c, a, b, bm, kt);
    if (s.len < 0 || s.tiles < 0 || s.qtiles < 0 || s.row0 < 0 || s.row0 + s.len > rows) return 1;
    sum_rows += s.qtiles;
    work += (double)s.qtiles * s.tiles;
  }
  const int per = chunk_tiles(work, sum_rows, units, least);
  int base = 0;
  for (int b = 0; b < seqs; ++b) {
    const Seq s = seq_at(c, a, b, bm, kt);
    const int chunks = chunks_of(s, per);
    for (int q = 0; q < s.qtiles; ++q) {
      std::vector<int> count;
      Span span{};
      int pos_lo = 0, pos_hi = 0;
      for (int k = 0; k < chunks; ++k) {
        const Unit u{b, q, k, chunks, base, s.row0, s.len, s.ctx};
        span = span_of(c, a, u, bm, kt, pos_lo, pos_hi);
        if (span.sink < 0 || span.from < span.sink || span.upto < span.from) return 2;
        int v0, v1;
        chunk_of(span, u, v0, v1);
        if (v0 < 0 || v1 < v0 || v1 > span.sink + span.upto - span.from) return 3;
        if (v1 - v0 > per) return 4;
        for (int v = v0; v < v1; ++v) {
          const int key0 = key_of(span, v, kt);
          if (key0 < 0 || key0 >= room_of(c)) return 5;
          for (int j = key0; j < key0 + kt; j += 16) {
            const PageAt p = page_at(c, table + (int64_t)b * columns, j);
            if (p.page < 0 || p.page >= pages) return 6;
          }
          if (sane) {
            if ((int)count.size() < key0 + kt) count.resize(key0 + kt, 0);
            for (int j = key0; j < key0 + kt; ++j) ++count[j];
          }
        }
      }
      if (!sane) continue;
      for (int pos = pos_lo; pos <= pos_hi; ++pos)
        for (int j = 0; j <= pos; ++j)
          if ((!window || j > pos - window || j < sinks) && (j >= (int)count.size() || count[j] != 1)) return 7;
      for (int n : count)
        if (n > 1) return 8;
    }
    base += s.qtiles * chunks;
  }
  *units_used = base;
  return base > units ? 9 : 0;
}
