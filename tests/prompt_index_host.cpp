// Host build of the packed prompts' index functions: whatever cu holds, rows stay inside
// the buffers, and every pair of a row and a key that it sees is in a tile of both ways.
#include "prompt_index.h"

using namespace kronq;

extern "C" int rows_inside(int lo, int hi, int rows) {
  const Prompt p = prompt_between(lo, hi, rows);
  if (p.start < 0 || p.n < 0 || p.start > rows || p.n > rows - p.start) return 1;
  if (lo >= 0 && hi <= rows && hi >= lo && (p.start != lo || p.n != hi - lo)) return 2;
  return 0;
}

extern "C" int tiles_cover(int n, int window, int bm, int kt) {
  const int w = window > 0 ? window : 1 << 30;
  for (int r0 = 0; r0 < n; r0 += bm) {
    const TileSpan s = keys_of_rows(r0, bm, n, w, kt), k = rows_of_keys(r0, bm, n, w, kt);
    if (s.first < 0 || s.last < s.first || s.last * kt >= n) return 1;
    if (k.first < 0 || k.last < k.first || k.last * kt >= n) return 2;
    for (int i = r0; i < r0 + bm && i < n; ++i) {
      for (int j = 0; j <= i; ++j)           // i sees j
        if (j > i - w && (j / kt < s.first || j / kt > s.last)) return 3;
      for (int j = i; j < n; ++j)            // j sees i
        if (i > j - w && (j / kt < k.first || j / kt > k.last)) return 4;
    }
  }
  return 0;
}
