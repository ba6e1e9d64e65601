// What the attention's kernels share: their arguments, the search for a unit of
// work, queries on their way to the matrix cores, and the unpacking of codes.
#pragma once

#include "kv.h"

namespace kronq {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kNan = __builtin_nanf("");

// What kv_attention_cut leaves for a kernel and its join.
struct CutTold { int per, any; };   // tiles of a chunk, whether any sequence is cut

struct AttnView {
  KvView c;
  HeadsView q, out;
  RopeView rope;
  float* lse;
  int qheads;              // query heads
  float scale;
  AttnShape shape;
  Cut cut;                 // work units of a key head
  int min_tiles;           // tiles of a chunk at least
  const CutTold* told;     // how long chunks are, where that was worked out before
  int places;              // of partial results, for each key head
  float* part;             // [places][heads][BM][dim] unnormalized outputs
  float* stat;             // [places][heads][BM][2]   maximum (of f S), sum
};

// ---- work units
//
// The host knows neither the lengths nor the contexts, only how many rows and
// sequences there are, so the launch has a fixed number of units and the kernels
// cut the keys.  Every wave works its unit out from cu and ctx by itself, 64
// sequences at a time; how long a chunk is, too, unless kv_attention_cut did.

// Data-parallel moves within the wave (rows of 16 lanes, then their last lanes):
// they wait for nothing, where exchanges through LDS cost 100 cycles a step.
template <int CTRL, int ROWS>
__device__ inline int moved(int x) {                  // 0 where nothing comes
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, false);
}

template <int CTRL, int ROWS>
__device__ inline double moved(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = moved<CTRL, ROWS>((int)(uint32_t)b), hi = moved<CTRL, ROWS>((int)(uint32_t)(b >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

template <typename V>
__device__ inline V wave_scan(V x) {                  // inclusive
  x += moved<0x111, 0xF>(x);                          // row_shr:1, 2, 4, 8
  x += moved<0x112, 0xF>(x);
  x += moved<0x114, 0xF>(x);
  x += moved<0x118, 0xF>(x);
  x += moved<0x142, 0xA>(x);                          // row_bcast:15 to rows 1 and 3
  x += moved<0x143, 0xC>(x);                          // row_bcast:31 to rows 2 and 3
  return x;
}

__device__ inline double wave_sum(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, wave_scan(x));
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, 63), hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ inline int wave_max(int x) {               // x >= 0
  x = max(x, moved<0x111, 0xF>(x));
  x = max(x, moved<0x112, 0xF>(x));
  x = max(x, moved<0x114, 0xF>(x));
  x = max(x, moved<0x118, 0xF>(x));
  x = max(x, moved<0x142, 0xA>(x));
  x = max(x, moved<0x143, 0xC>(x));
  return __builtin_amdgcn_readlane(x, 63);
}

// The unit `want`; by_row: the sequence of row `want`, its first unit.  false:
// there is none.
template <int BM, int KT>
__device__ inline bool find_unit(const AttnView& a, int want, bool by_row, Unit& u) {
  const int lane = threadIdx.x & 63;
  Seq s = seq_at(a.c, a.shape, lane, BM, KT);
  int per = a.min_tiles;
  if (room_of(a.c) > (int64_t)per * KT) {             // else nothing is cut
    if (a.told) {
      per = a.told->per;
    } else {                                          // at most 64 sequences
      // sums of integers below 2^53: exact
      double rows = s.qtiles, work = (double)s.qtiles * s.tiles;
      if (a.c.seqs > 1) {                             // one sequence is lane 0's
        rows = wave_sum(rows);
        work = wave_sum(work);
      }
      per = chunk_tiles(work, rows, used_units(a.cut, rows), per);
    }
  }
  int before = 0, places = 0;
  for (int b0 = 0; b0 < a.c.seqs; b0 += 64) {
    if (a.c.seqs > 64) s = seq_at(a.c, a.shape, b0 + lane, BM, KT);
    const int chunks = chunks_of(s, per);
    const int n = s.qtiles * chunks, upto = before + wave_scan(n);
    int place = 0;                                    // of the sequence's first unit
    if (__any(chunks > 1)) {
      const int k = chunks > 1 ? n : 0, all = places + wave_scan(k);
      place = all - k;
      places = __builtin_amdgcn_readlane(all, 63);
    }
    const bool mine = by_row ? (want >= s.row0 && want < s.row0 + s.len) : (want < upto && want >= upto - n);
    const uint64_t hit = __ballot(mine);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      u.b = b0 + l;                                   // the same in all lanes, and known to be
      u.base = __builtin_amdgcn_readlane(upto - n, l);
      u.chunks = __builtin_amdgcn_readlane(chunks, l);
      u.row0 = __builtin_amdgcn_readlane(s.row0, l);
      u.len = __builtin_amdgcn_readlane(s.len, l);
      u.ctx = __builtin_amdgcn_readlane(s.ctx, l);
      const int rest = by_row ? 0 : want - u.base;
      u.qtile = rest / u.chunks;
      u.chunk = rest % u.chunks;
      u.place = u.chunks > 1 ? __builtin_amdgcn_readlane(place, l) + rest : 0;
      return true;
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// ---- queries

// Eight values of a query head from position d on, rotated in fp32.
template <typename T>
__device__ inline void query8(const T* p, int d, const RopeView& rope, int64_t pos, float* x) {
  load8(p + d, x);
  if (d >= 2 * rope.half) return;
  const float* ct = rope.cos + pos * rope.ld;
  const float* st = rope.sin + pos * rope.ld;
  if (rope.neighbours) {
    const f32x4 c = *reinterpret_cast<const f32x4*>(ct + d / 2);
    const f32x4 s = *reinterpret_cast<const f32x4*>(st + d / 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float y = x[2 * i], z = x[2 * i + 1];
      x[2 * i] = y * c[i] - z * s[i];
      x[2 * i + 1] = z * c[i] + y * s[i];
    }
  } else {
    const bool second = d >= rope.half;
    const int j = second ? d - rope.half : d;
    float o[8], c[8], s[8];
    load8(p + (second ? j : d + rope.half), o);
    load8(ct + j, c);
    load8(st + j, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = second ? x[i] * c[i] + o[i] * s[i] : x[i] * c[i] - o[i] * s[i];
  }
}

// Eight codes of a word in the order the unpacking yields them.
__device__ constexpr int kOrder[8] = {0, 4, 1, 5, 2, 6, 3, 7};

// A row's query as fp16, N runs of eight values at first + step k, times 2^e2 so
// that its largest value is in [2^10, 2^11), in PARTS parts (the second is what the
// first's rounding left).  Returns f, by which products with it become scores in
// powers of two; NaN for a row that has none (an entry that is not finite, a
// position without angles).  LANES lanes 64 / LANES apart share the row.
template <typename T, int PARTS, int N, int LANES>
__device__ inline float load_query(const AttnView& a, const Unit& u, int head, int r, int first, int step,
                                   half8_t (&q1)[N], half8_t (&q2)[PARTS > 1 ? N : 1]) {
  const int share = a.shape.share, t = min(r / share, u.len - 1), pos = u.ctx - u.len + t;
  const T* qp = static_cast<const T*>(a.q.data) + (int64_t)(u.row0 + t) * a.q.row +
                (int64_t)(head * share + r % share) * a.q.head;
  RopeView rope = a.rope;
  bool fine = !rope.half || pos < rope.positions;
  if (!fine || pos < 0) rope.half = 0;                // before the sequence's start: sees nothing
  float x[N][8], big = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    query8(qp, first + step * k, rope, pos, x[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      big = fmaxf(big, fabsf(x[k][e]));
      fine = fine && (x[k][e] - x[k][e] == 0);
    }
  }
  int bad = !fine;
#pragma unroll
  for (int d = 64 / LANES; d < 64; d <<= 1) {
    big = fmaxf(big, __shfl_xor(big, d));
    bad |= __shfl_xor(bad, d);
  }
  int e2 = 0;
  if (!bad && big > 0) {
    frexpf(big, &e2);                                 // big < 2^e2
    e2 = 11 - e2;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = bad ? 0.0f : ldexpf(x[k][kOrder[e]], e2);
      q1[k][e] = (_Float16)y;
      if constexpr (PARTS > 1) q2[k][e] = (_Float16)(y - (float)q1[k][e]);
    }
  }
  // f > 0, so that it takes -inf to -inf; of a row before the start, too
  const float f = fmaxf(ldexpf(a.scale * kLog2e, -e2), 0x1p-126f);
  return bad && pos >= 0 ? kNan : f;
}

__device__ inline half2_t as_half2(uint32_t x) { return __builtin_bit_cast(half2_t, x); }

// Codes as fp16 integers c - z.  1024 + c is the fp16 number 0x6400 | c, and
// 1024 + 16 c is 0x6400 | 16 c, so a code in bits 0..3 or 4..7 of a half becomes a
// number in one bit-field insert, and loses 1024 + z, or after a factor 1/16
// 64 + z, in one packed addition for two: all exact.  The constants live in
// registers that the compiler does not look into: as literals they would cost a
// second operation each.
struct Unpacker {
  uint32_t low, high, bias;
  __device__ inline Unpacker() : low(0x000F000Fu), high(0x00F000F0u), bias(0x64006400u) {
    asm("" : "+s"(low));
    asm("" : "+s"(high));
    asm("" : "+v"(bias));
  }
  __device__ inline half2_t low_pair(uint32_t x, half2_t zero1024) const {
    return as_half2((x & low) | (bias & ~low)) - zero1024;
  }
  __device__ inline half2_t high_pair(uint32_t x, half2_t zero64) const {
    return as_half2((x & high) | (bias & ~high)) * half2_t{(_Float16)0.0625f, (_Float16)0.0625f} - zero64;
  }
  // A word's eight codes minus their zero point, in kOrder.
  __device__ inline half8_t word(uint32_t w, half2_t zero1024, half2_t zero64) const {
    const half2_t a = low_pair(w, zero1024), b = high_pair(w, zero64);
    const half2_t c = low_pair(w >> 8, zero1024), d = high_pair(w >> 8, zero64);
    return half8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
  }
};

// A zero point's constants for it: 1024 + z (0x6400 | z) and 64 + z
// (0x5400 | 16 z), in both halves.
__device__ inline uint32_t zero1024_of(uint32_t z) { return (z * 0x00010001u) | 0x64006400u; }
__device__ inline uint32_t zero64_of(uint32_t z) { return (z * 0x00100010u) | 0x54005400u; }

// Products of weights and value scales enter the matrix cores as fp16 under a
// row's factor 2^-e.  e follows the row's largest such product: where that was
// last set it lies in [2^5, 2^6), and products up to 2^14 pass before it is set
// again, so that products 2^-20 of the largest are still normal numbers whatever
// the scales' range.  A row's maximum m is raised only where a score leaves it
// behind by 2^kLazy.
constexpr int kLazy = 8, kRoom = 6, kTop = 14;
constexpr int kLeast = -126, kMost = 120;             // of e; kLeast where nothing was seen yet

// Beyond this f S and its maximum, which is rounded to fp32, no longer cancel to 0 for
// the largest score (from 2^28 on its weight would overflow, or vanish): there what
// the rounding left is taken off, too.  Asking for it costs 0 to 2 % (dim 64
// and 256: up to 6).
constexpr float kSteep = 0x1p+16f;

// Exponent e for a row's largest product (positive).
__device__ inline int exponent_for(float largest) {
  return (int)(__float_as_uint(largest) >> 23) - 126 - kRoom;
}

// kvrows.hip: the kernel of many rows, 32 x waves (4 or 8; 4 for dim 256) a tile
kronq_status kv_rows_launch(const AttnView& a, int dim, int32_t dtype, int waves, hipStream_t s);

}  // namespace kronq
