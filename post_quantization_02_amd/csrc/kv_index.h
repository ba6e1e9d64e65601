// Which memory a call on the 4-bit paged key/value cache touches: rows to
// sequences, positions to pages, and how the attention's work is cut.  Plain
// functions of the batch arrays (whose content no host check sees), so that
// what they may return is tested on the host.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace kronq {

struct KvView {
  uint8_t *kc, *vc;        // codes
  uint32_t *kg, *vg;       // grids
  uint32_t kcs, vcs;       // bytes between pages
  uint32_t kgs, vgs;       // words between pages
  const int32_t *table, *ctx, *cu;
  int64_t ldt;
  int pages, lgp, heads;   // page = 1 << lgp
  int seqs, columns;
  int rows;
};

// The sequence of a row: the last one that starts at or before it and ends
// behind it; -1 if there is none.  `cu` are the sequences' starts and the end.
__host__ __device__ inline int seq_of(const int32_t* cu, int seqs, int row) {
  int lo = 0, hi = seqs;   // cu[lo] <= row < cu[hi]
  if (row < cu[0] || row >= cu[seqs]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= row) lo = mid; else hi = mid;
  }
  return lo;
}

struct PageAt { int page; bool bad; };

// The page of a position >= 0 of the sequence whose table row is given; page 0
// where there is none in range, so that reading is safe.  In two parts, an entry
// (of the last column where there is no such column) and what it comes to, for
// those who ask early and look late.
__host__ __device__ inline int page_entry(const KvView& c, const int32_t* table, int pos) {
  const int col = pos >> c.lgp;
  return c.columns > 0 ? table[col < c.columns ? col : c.columns - 1] : -1;
}

__host__ __device__ inline PageAt page_from(const KvView& c, int entry, int pos) {
  const bool bad = (pos >> c.lgp) >= c.columns || entry < 0 || entry >= c.pages;
  return {bad ? 0 : entry, bad};
}

__host__ __device__ inline PageAt page_at(const KvView& c, const int32_t* table, int pos) {
  return page_from(c, page_entry(c, table, pos), pos);
}

// Where a row's token lives.  pos < 0: nowhere.  bad: no page in range.
struct Place { int pos, page, slot; bool bad; };

__host__ __device__ inline Place place_of(const KvView& c, int seq, int row, int end) {
  const int64_t pos = (int64_t)c.ctx[seq] - end + row;   // end: the sequence's, cu[seq + 1] > row
  if (pos < 0) return {-1, 0, 0, true};
  const PageAt p = page_at(c, c.table + seq * c.ldt, (int)pos);
  return {(int)pos, p.page, (int)(pos & ((1 << c.lgp) - 1)), p.bad};
}

// ---- attention: the work of a sequence
//
// Rows x share query heads of a key head in tiles of BM, keys in tiles of KT.
// A kernel takes the sequences whose rows x share are least .. most.

struct AttnShape { int share, window, sinks, least, most; };   // window 0: none

struct Seq { int row0, len, ctx, tiles, qtiles; };   // ctx: the position behind its last row

__host__ __device__ inline int tiles_of(int n, int kt) { return n / kt + (n % kt != 0); }

// Bytes (words) from the cache's start to a page: 32 x 32 bits, which is one
// instruction.
__host__ __device__ inline uint64_t page_offset(int page, uint32_t stride) { return (uint64_t)(uint32_t)page * stride; }

// Positions that have a column.
__host__ __device__ inline int64_t room_of(const KvView& c) { return (int64_t)c.columns << c.lgp; }

__host__ __device__ inline int cut_to_room(const KvView& c, int n) {
  const int64_t room = room_of(c);
  return n < 0 ? 0 : (int64_t)n < room ? n : (int)room;
}

// The key tiles that rows at pos_lo .. pos_hi see: `sink` first ones, then
// from .. upto - 1.
struct Span { int sink, from, upto; };

__host__ __device__ inline Span span_between(const KvView& c, const AttnShape& a, int pos_lo, int pos_hi, int kt) {
  const int end = cut_to_room(c, pos_hi < 0 ? 0 : pos_hi == INT32_MAX ? pos_hi : pos_hi + 1);
  Span s{0, 0, tiles_of(end, kt)};
  if (a.window) {
    const int first = pos_lo - a.window + 1;
    s.from = first > 0 ? first / kt : 0;
    if (s.from > s.upto) s.from = s.upto;
    s.sink = tiles_of(a.sinks < end ? a.sinks : end, kt);
    if (s.sink > s.from) s.sink = s.from;
  }
  return s;
}

__host__ __device__ inline Seq seq_at(const KvView& c, const AttnShape& a, int b, int bm, int kt) {
  Seq s{0, 0, 0, 0, 0};
  if (b >= c.seqs) return s;
  const int lo = c.cu[b] > 0 ? c.cu[b] : 0, hi = c.cu[b + 1] < c.rows ? c.cu[b + 1] : c.rows;
  if (hi <= lo) return s;
  const int64_t n = (int64_t)(hi - lo) * a.share;
  if (n < a.least || n > a.most) return s;
  s.row0 = lo;
  s.len = hi - lo;
  // where its last row of this call stands, which a batch that names more rows
  // than there are (cu beyond them) does not end with
  const int64_t end = (int64_t)c.ctx[b] - ((int64_t)c.cu[b + 1] - hi);
  s.ctx = end > 0 ? (int)end : 0;
  const Span all = span_between(c, a, s.ctx > s.len ? s.ctx - s.len : 0, s.ctx - 1, kt);
  s.tiles = all.sink + all.upto - all.from;
  s.qtiles = (int)((n + bm - 1) / bm);
  return s;
}

// The launch has a fixed number of units; a unit is (sequence, tile of rows,
// chunk of the keys).  The chunk length is the smallest at which all chunks fit:
// sum of qtiles * ceil(tiles / per) <= work / per + rows <= units, with
// work = sum of qtiles * tiles and rows = sum of qtiles.
__host__ __device__ inline int chunk_tiles(double work, double rows, int units, int least) {
  const double room = units - rows > 1.0 ? units - rows : 1.0;
  const int per = (int)ceil(work / room);
  return per > least ? per : least;
}

// How a launch is cut: its units, how many of them are to be used as a rule
// (`aim`), and how many at least are left for chunks (`spare`) where the row tiles
// alone are more than that, so that one long sequence among many is cut still.
struct Cut { int units, aim, spare; };

// Units to be used: a sequence's last row tile leaves half a chunk empty on average.
__host__ __device__ inline int used_units(const Cut& c, double rows) {
  const double some = rows + fmax(c.aim - 0.5 * rows, (double)c.spare);
  return some < c.units ? (int)some : c.units;
}

// Units of sequences that are cut in chunks, at most, which have a place for their
// partial results: the sum of qtiles * (chunks - 1) is below work / per <= used -
// rows <= max(aim, spare), whatever the batch holds, and chunks <= 2 (chunks - 1).
__host__ __device__ inline int places_of(const Cut& c) {
  const int64_t n = 2 * (int64_t)(c.aim > c.spare ? c.aim : c.spare);
  return n < c.units ? (int)n : c.units;
}

__host__ __device__ inline int chunks_of(const Seq& s, int per) {
  const int n = tiles_of(s.tiles, per);
  return n > 1 ? n : 1;
}

struct Unit {
  int b, qtile, chunk, chunks, base;   // base: the sequence's first unit
  int row0, len, ctx;
  int place;               // of its chunk's partial results, where chunks > 1
};

__host__ __device__ inline Span span_of(const KvView& c, const AttnShape& a, const Unit& u, int bm, int kt, int& pos_lo,
                                        int& pos_hi) {
  const int last = (u.qtile * bm + bm - 1) / a.share;
  pos_lo = u.ctx - u.len + u.qtile * bm / a.share;
  pos_hi = u.ctx - u.len + (last < u.len ? last : u.len - 1);
  return span_between(c, a, pos_lo, pos_hi, kt);
}

// The tiles v0 .. v1 - 1 of a span's (counted over both its parts) that are the
// unit's: equal parts of what the unit's rows see.
__host__ __device__ inline void chunk_of(const Span& s, const Unit& u, int& v0, int& v1) {
  const int tiles = s.sink + s.upto - s.from, per = tiles / u.chunks + (tiles % u.chunks != 0);
  v0 = (int64_t)u.chunk * per < tiles ? u.chunk * per : tiles;
  v1 = v0 + per < tiles ? v0 + per : tiles;
}

__host__ __device__ inline int key_of(const Span& s, int v, int kt) {
  return (v < s.sink ? v : v - s.sink + s.from) * kt;
}

}  // namespace kronq
