// Which rows a call on packed prompts touches.  Plain functions of cu, whose content no
// host check sees, so that what they may return is tested on the host.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace kronq {

// Rows start .. start + n - 1 of a sequence.
struct Prompt { int start, n; };

// The sequence whose rows are lo .. hi - 1, cut to the rows there are: any lo and hi.
__host__ __device__ inline Prompt prompt_between(int lo, int hi, int rows) {
  lo = lo < 0 ? 0 : lo > rows ? rows : lo;
  hi = hi < 0 ? 0 : hi > rows ? rows : hi;
  return {lo, hi > lo ? hi - lo : 0};
}

// Tiles first .. last (not empty).
struct TileSpan { int first, last; };

// Tiles of kt keys that rows r0 .. r0 + bm - 1 (r0 < n) of a sequence of n see.
// window: at most 2^30.
__host__ __device__ inline TileSpan keys_of_rows(int r0, int bm, int n, int window, int kt) {
  const int end = r0 + bm < n ? r0 + bm : n;
  return {r0 >= window ? (r0 - window + 1) / kt : 0, (end - 1) / kt};
}

// Tiles of qt rows that see keys k0 .. k0 + bn - 1 (k0 < n).
__host__ __device__ inline TileSpan rows_of_keys(int k0, int bn, int n, int window, int qt) {
  const int last = k0 + bn - 1 < n - window ? k0 + bn - 1 + window : n - 1;
  return {k0 / qt, last / qt};
}

}  // namespace kronq
