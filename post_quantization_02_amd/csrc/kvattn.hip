// Attention over the 4-bit paged key/value cache.
//
// For each row's head: scores S_j = s_j (q . (c_j - z_j)) over the visible
// positions j, a running maximum m and sum l = sum_j 2^(f (S_j - m)) with
// f = scale log2(e), and O = sum_j 2^(f (S_j - m)) s'_j (c'_j - z'_j), all in
// one pass over the codes; out = O / l.  The matrix cores see codes minus zero
// points as fp16 integers (exact); the scales of keys multiply scores, those of
// values multiply weights, both in fp32.
#include <algorithm>
#include <cmath>

#include "kv.h"

namespace kronq {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct AttnView {
  KvView c;
  HeadsView q, out;
  RopeView rope;
  float* lse;
  int qheads;              // query heads
  float scale;
  AttnShape shape;
  int units;               // work units of a key head
  int min_tiles;           // tiles of a chunk at least
  float* part;             // [units][heads][BM][dim] unnormalized outputs
  float* stat;             // [units][heads][BM][2]   maximum (of f S), sum
};

// ---- work units
//
// The host knows neither the lengths nor the contexts, only how many rows and
// sequences there are, so the launch has a fixed number of units and the kernels
// cut the keys.  Every wave works its unit out from cu and ctx by itself, 64
// sequences at a time.

__device__ inline int wave_scan(int x) {              // inclusive
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if ((int)(threadIdx.x & 63) >= d) x += y;
  }
  return x;
}

__device__ inline double wave_sum(double x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  return x;
}

// The unit `want`; by_row: the sequence of row `want`, its first unit.  false:
// there is none.
template <int BM, int KT>
__device__ inline bool find_unit(const AttnView& a, int want, bool by_row, Unit& u) {
  const int lane = threadIdx.x & 63;
  // sums of integers below 2^53: exact
  double rows = 0, work = 0;
  Seq s = seq_at(a.c, a.shape, lane, BM, KT);
  for (int b0 = 0;;) {
    rows += s.qtiles;
    work += (double)s.qtiles * s.tiles;
    b0 += 64;
    if (b0 >= a.c.seqs) break;
    s = seq_at(a.c, a.shape, b0 + lane, BM, KT);
  }
  rows = wave_sum(rows);
  work = wave_sum(work);
  const int per = chunk_tiles(work, rows, a.units, a.min_tiles);
  int before = 0;
  for (int b0 = 0; b0 < a.c.seqs; b0 += 64) {
    if (a.c.seqs > 64) s = seq_at(a.c, a.shape, b0 + lane, BM, KT);
    const int chunks = chunks_of(s, per);
    const int n = s.qtiles * chunks, upto = before + wave_scan(n);
    const bool mine = by_row ? (want >= s.row0 && want < s.row0 + s.len) : (want < upto && want >= upto - n);
    const uint64_t hit = __ballot(mine);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      u.b = b0 + l;
      u.base = __shfl(upto - n, l);
      u.chunks = __shfl(chunks, l);
      u.row0 = __shfl(s.row0, l);
      u.len = __shfl(s.len, l);
      u.ctx = __shfl(s.ctx, l);
      const int rest = by_row ? 0 : want - u.base;
      u.qtile = rest / u.chunks;
      u.chunk = rest % u.chunks;
      return true;
    }
    before = __shfl(upto, 63);
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

__device__ inline half2_t as_half2(uint32_t x) { return __builtin_bit_cast(half2_t, x); }

// Pairs of values c - z.  1024 + c is the fp16 number 0x6400 | c, and
// 1024 + 16 c is 0x6400 | 16 c; zero holds z in both halves (0x6400 | z, and
// 64 + z = 0x5400 | 16 z).  All differences are exact.
__device__ inline half2_t low_pair(uint32_t x, half2_t zero1024) {
  return as_half2((x & 0x000F000Fu) | 0x64006400u) - zero1024;
}
__device__ inline half2_t high_pair(uint32_t x, half2_t zero64) {
  return as_half2((x & 0x00F000F0u) | 0x64006400u) * half2_t{(_Float16)0.0625f, (_Float16)0.0625f} - zero64;
}

// A word's eight codes minus their zero point, in kOrder.
__device__ inline half8_t unpack_word(uint32_t w, half2_t zero1024, half2_t zero64) {
  const half2_t a = low_pair(w, zero1024), b = high_pair(w, zero64);
  const half2_t c = low_pair(w >> 8, zero1024), d = high_pair(w >> 8, zero64);
  return half8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// ---- one tile of 16 rows
//
// A workgroup takes a unit of 16 rows (rows x share of one key head); its four
// waves take the unit's tiles of 32 keys in turn.  With 16x16x32 fp16 products
// everything stays in registers:
//   S^T = K Q^T: row i of the 16-key operand a (0, 1) is key 8 (i / 4) + 4 a +
//     i % 4 of the tile, and lane (i, g) holds values (dim / 4) g and up of it:
//     dim / 8 contiguous bytes, dim / 32 products of 32 values.
//   The lane (row, g) then has the scores of keys 8 g .. 8 g + 7, which is what
//   O^T = V^T P^T wants of P: k slots (g, 0..7) are those keys.  Lane (i, g)
//     holds values (dim / 16) i and up of them, dim / 16 products of 16 values.

template <int DIM>
struct RawTile {
  uint32_t k[2][DIM / 32];
  uint32_t kz[2];          // grid words of this lane's key rows
  u32x4 ks[2], vs[2];      // grid words of keys 8 g .. 8 g + 7
  uint32_t v[8][(DIM + 127) / 128];
  bool bad;                // the page of those keys is out of range
};

template <int DIM>
__device__ inline void load_tile(const KvView& c, const int32_t* table, int head, int key0, RawTile<DIM>& t) {
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int in_page = (1 << c.lgp) - 1;
  // a page holds at least 16 keys: each half of the tile lies in one
  const PageAt p0 = page_at(c, table, key0), p1 = page_at(c, table, key0 + 16);
  const int64_t slot0 = ((int64_t)head << c.lgp) + (key0 & in_page);
  const int64_t slot1 = ((int64_t)head << c.lgp) + ((key0 + 16) & in_page);
  {
    const bool up = (i >> 3) != 0;
    const int64_t page = up ? p1.page : p0.page;
    const int64_t slot = (up ? slot1 : slot0) + 8 * ((i >> 2) & 1) + (i & 3);
    const uint8_t* k = c.kc + page * c.kcs + slot * (DIM / 2) + g * (DIM / 8);
    const uint32_t* kg = c.kg + page * c.kgs + slot;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      if constexpr (DIM == 64) {
        *reinterpret_cast<u32x2*>(t.k[a]) = *reinterpret_cast<const u32x2*>(k + 4 * a * (DIM / 2));
      } else {
#pragma unroll
        for (int w = 0; w < DIM / 32; w += 4)
          *reinterpret_cast<u32x4*>(t.k[a] + w) = *reinterpret_cast<const u32x4*>(k + 4 * a * (DIM / 2) + 4 * w);
      }
      t.kz[a] = kg[4 * a];
    }
  }
  {
    const bool up = (g >> 1) != 0;
    const int64_t page = up ? p1.page : p0.page;
    const int64_t slot = (up ? slot1 : slot0) + 8 * (g & 1);
    const uint32_t* kg = c.kg + page * c.kgs + slot;
    const uint32_t* vg = c.vg + page * c.vgs + slot;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      t.ks[a] = *reinterpret_cast<const u32x4*>(kg + 4 * a);
      t.vs[a] = *reinterpret_cast<const u32x4*>(vg + 4 * a);
    }
    t.bad = up ? p1.bad : p0.bad;
    const uint8_t* v = c.vc + page * c.vcs + slot * (DIM / 2) + i * (DIM / 32);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (DIM == 64)
        t.v[j][0] = *reinterpret_cast<const uint16_t*>(v + j * (DIM / 2));
      else if constexpr (DIM == 128)
        t.v[j][0] = *reinterpret_cast<const uint32_t*>(v + j * (DIM / 2));
      else
        *reinterpret_cast<u32x2*>(t.v[j]) = *reinterpret_cast<const u32x2*>(v + j * (DIM / 2));
    }
  }
}

// What a row keeps while its keys go by: the maximum m of f S, its lane's part
// of l, and the factor 2^-e under which the products of weights and value scales
// enter the matrix cores as fp16.  e follows the row's largest such product:
// where that was last set it lies in [2^5, 2^6), and products up to 2^14 pass
// before it is set again, so that products 2^-20 of the largest are still normal
// numbers whatever the scales' range.  m is raised only where a score leaves it
// behind by 2^kLazy.
constexpr int kLazy = 8, kRoom = 6, kTop = 14, kNone = -127;

struct RowState {
  float m = -INFINITY, l = 0, limit = 0;   // limit 2^(kTop + e); 0: nothing seen yet
  int e = kNone;
};

template <int DIM, typename T, bool TWO>
__global__ __launch_bounds__(256) void kv_attention16(AttnView a) {
  constexpr int BM = 16, KT = 32, KS = DIM / 32, VT = DIM / 16, PAD = DIM + 4;
  __shared__ float lds_o[4][BM][PAD];
  __shared__ float lds_m[4][BM], lds_l[4][BM];
  Unit u;
  if (!find_unit<BM, KT>(a, blockIdx.x, false, u)) return;
  const int head = blockIdx.y;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, i = lane & 15, g = lane >> 4;
  int pos_lo, pos_hi;
  const Span span = span_of(a.c, a.shape, u, BM, KT, pos_lo, pos_hi);
  int v0, v1;
  chunk_of(span, u, v0, v1);
  const int share = a.shape.share, window = a.shape.window, sinks = a.shape.sinks;
  const int32_t* table = a.c.table + (int64_t)u.b * a.c.ldt;

  // this lane's query row
  const int r = u.qtile * BM + i;
  const int t = min(r / share, u.len - 1);
  const int pos = u.ctx - u.len + t;
  const bool real = r < u.len * share;
  float f;
  half8_t q1[KS], q2[TWO ? KS : 1];
  {
    const int qh = head * share + r % share;
    const T* qp = static_cast<const T*>(a.q.data) + (int64_t)(u.row0 + t) * a.q.row + (int64_t)qh * a.q.head;
    float x[KS][8], big = 0;
    const bool turned = !a.rope.half || (pos >= 0 && pos < a.rope.positions);
    bool fine = turned;
    RopeView rope = a.rope;
    if (!turned) rope.half = 0;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      query8(qp, g * (DIM / 4) + 8 * k, rope, pos, x[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        big = fmaxf(big, fabsf(x[k][e]));
        fine = fine && (x[k][e] - x[k][e] == 0);
      }
    }
    big = fmaxf(big, __shfl_xor(big, 16));
    big = fmaxf(big, __shfl_xor(big, 32));
    const uint64_t notfine = __ballot(!fine);
    fine = !((notfine >> i) & 0x0001000100010001ull);
    int e2 = 0;
    if (fine && big > 0) {
      frexpf(big, &e2);                               // big < 2^e2
      e2 = 4 - e2;                                    // the row's largest value in [2^3, 2^4)
    }
    // a row that is not finite has no score
    f = fine ? ldexpf(a.scale * kLog2e, -e2) : __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = fine ? ldexpf(x[k][kOrder[e]], e2) : 0.0f;
        q1[k][e] = (_Float16)y;
        if constexpr (TWO) q2[k][e] = (_Float16)(y - (float)q1[k][e]);
      }
    }
  }

  f32x4 o[VT];
#pragma unroll
  for (int k = 0; k < VT; ++k) o[k] = f32x4{0, 0, 0, 0};
  RowState st;
  RawTile<DIM> raw;
  if (v0 + wave < v1) load_tile<DIM>(a.c, table, head, key_of(span, v0 + wave, KT), raw);
  for (int v = v0 + wave; v < v1; v += 4) {
    const RawTile<DIM> cur = raw;
    const int key0 = key_of(span, v, KT);
    if (v + 4 < v1) load_tile<DIM>(a.c, table, head, key_of(span, v + 4, KT), raw);

    // scores
    f32x4 sc[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t z = cur.kz[b] & 15;
      const half2_t z1 = as_half2((z * 0x00010001u) | 0x64006400u), z2 = as_half2((z * 0x00100010u) | 0x54005400u);
      sc[b] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const half8_t kv = unpack_word(cur.k[b][k], z1, z2);
        sc[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv, q1[k], sc[b], 0, 0, 0);
        if constexpr (TWO) sc[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv, q2[k], sc[b], 0, 0, 0);
      }
    }
    // keys 8 g + x: which are visible?  All are, but in the tiles at the edges.
    const int first = key0 + 8 * g;
    const bool whole = key0 + KT - 1 <= pos_lo &&
                       (!window || key0 > pos_hi - window || key0 + KT <= sinks);
    bool seen[8];
    float s[8], vs[8], top = -INFINITY;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int j = first + x;
      seen[x] = whole || (j <= pos && (!window || j > pos - window || j < sinks));
      const float nan = __uint_as_float(0x7FC00000u);
      const float ks = cur.bad ? nan : __uint_as_float(cur.ks[x >> 2][x & 3] & ~15u);
      vs[x] = cur.bad ? nan : __uint_as_float(cur.vs[x >> 2][x & 3] & ~15u);
      s[x] = seen[x] ? sc[x >> 2][x & 3] * (ks * f) : -INFINITY;
      top = fmaxf(top, s[x]);
    }
    if (__any(top > st.m + kLazy || (st.m == -INFINITY && top > st.m))) {
      float nm = fmaxf(top, __shfl_xor(top, 16));
      nm = fmaxf(nm, __shfl_xor(nm, 32));
      nm = fmaxf(nm, st.m);
      if (st.m != -INFINITY) {
        const float down = fminf(nm - st.m, 300.0f);
        const int ne = st.e == kNone ? kNone : max(st.e - (int)ceilf(down), -126);
        const float by = __builtin_amdgcn_exp2f((float)(st.e - ne) - down);
        st.l *= __builtin_amdgcn_exp2f(-down);
#pragma unroll
        for (int k = 0; k < VT; ++k) o[k] *= by;
        st.e = ne;
        st.limit = ne == kNone ? 0.0f : ldexpf(1.0f, min(ne + kTop, 127));
      }
      st.m = nm;
    }
    const float base = st.m == -INFINITY ? 0.0f : st.m;
    float y[8], ytop = 0;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float p = __builtin_amdgcn_exp2f(s[x] - base);
      st.l += p;
      y[x] = seen[x] ? p * vs[x] : 0.0f;
      ytop = fmaxf(ytop, y[x]);
    }
    if (__any(ytop > st.limit)) {
      ytop = fmaxf(ytop, __shfl_xor(ytop, 16));
      ytop = fmaxf(ytop, __shfl_xor(ytop, 32));
      if (ytop > st.limit) {
        const int ne = min(max((int)(__float_as_uint(ytop) >> 23) - 126 - kRoom, -126), 120);
        const float by = ldexpf(1.0f, st.e - ne);
#pragma unroll
        for (int k = 0; k < VT; ++k) o[k] *= by;
        st.e = ne;
        st.limit = ldexpf(1.0f, min(ne + kTop, 127));
      }
    }
    const float unit = ldexpf(1.0f, min(-st.e, 126));
    half8_t p1, p2;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      y[x] *= unit;
      p1[x] = (_Float16)y[x];
      if constexpr (TWO) p2[x] = (_Float16)(y[x] - (float)p1[x]);
    }
    half2_t z1[4], z2[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t z = (cur.vs[x >> 1][2 * (x & 1)] & 15) | ((cur.vs[x >> 1][2 * (x & 1) + 1] & 15) << 16);
      z1[x] = as_half2(z | 0x64006400u);
      z2[x] = as_half2((z << 4) | 0x54005400u);
    }
#pragma unroll
    for (int b = 0; b < VT / 2; ++b) {                // byte b of the words: values 2 b, 2 b + 1
      half2_t lo[4], hi[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t w = __builtin_amdgcn_perm(cur.v[2 * x + 1][b >> 2], cur.v[2 * x][b >> 2],
                                                 0x0C000C00u | (uint32_t)(b & 3) | ((uint32_t)(4 + (b & 3)) << 16));
        lo[x] = low_pair(w, z1[x]);
        hi[x] = high_pair(w, z2[x]);
      }
      const half8_t va{lo[0].x, lo[0].y, lo[1].x, lo[1].y, lo[2].x, lo[2].y, lo[3].x, lo[3].y};
      const half8_t vb{hi[0].x, hi[0].y, hi[1].x, hi[1].y, hi[2].x, hi[2].y, hi[3].x, hi[3].y};
      o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(va, p1, o[2 * b], 0, 0, 0);
      o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vb, p1, o[2 * b + 1], 0, 0, 0);
      if constexpr (TWO) {
        o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(va, p2, o[2 * b], 0, 0, 0);
        o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vb, p2, o[2 * b + 1], 0, 0, 0);
      }
    }
  }

  // the four waves' parts
  st.l += __shfl_xor(st.l, 16);
  st.l += __shfl_xor(st.l, 32);
  if (lane < 16) {
    lds_m[wave][i] = st.m;
    lds_l[wave][i] = st.l;
  }
  const float back = ldexpf(1.0f, st.e);
#pragma unroll
  for (int rr = 0; rr < 4; ++rr) {
#pragma unroll
    for (int k = 0; k < VT; ++k) lds_o[wave][i][VT * (4 * g + rr) + k] = o[k][rr] * back;
  }
  __syncthreads();
  // thread: 8 values of one row at a time
  for (int c = tid; c < BM * DIM / 8; c += 256) {
    const int row = c / (DIM / 8), d = (c % (DIM / 8)) * 8;
    const int rg = u.qtile * BM + row;
    if (rg >= u.len * share) continue;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) mm = fmaxf(mm, lds_m[w][row]);
    float ll = 0, x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float by = lds_m[w][row] == -INFINITY ? 0.0f : exp2f(lds_m[w][row] - mm);
      ll += lds_l[w][row] * by;
#pragma unroll
      for (int y = 0; y < 8; ++y) x[y] += lds_o[w][row][d + y] * by;
    }
    const int tok = rg / share, qh = head * share + rg % share;
    // a position without a column: its row sees at least itself
    if (u.ctx - u.len + tok >= room_of(a.c)) ll = __uint_as_float(0x7FC00000u);
    if (u.chunks == 1) {
      const float inv = ll == 0 ? 0.0f : 1.0f / ll;
#pragma unroll
      for (int y = 0; y < 8; ++y) x[y] = ll == 0 ? 0.0f : x[y] * inv;
      store8(static_cast<T*>(a.out.data) + (int64_t)(u.row0 + tok) * a.out.row + (int64_t)qh * a.out.head + d, x);
      if (a.lse && d == 0)
        a.lse[(int64_t)(u.row0 + tok) * a.qheads + qh] = ll == 0 ? -INFINITY : (mm + log2f(ll)) * kLn2;
    } else {
      const int64_t at = ((int64_t)blockIdx.x * a.c.heads + head) * BM + row;
      store8(a.part + at * DIM + d, x);
      if (d == 0) {
        a.stat[2 * at] = mm;
        a.stat[2 * at + 1] = ll;
      }
    }
  }
}

// Joins the chunks of one row's head, in the order of the chunks.
template <int DIM, int BM, int KT, typename T>
__global__ __launch_bounds__(256) void kv_attention_join(AttnView a) {
  constexpr int LANES = DIM / 8, SLOTS = 256 / LANES;
  __shared__ float lds_x[SLOTS][DIM + 4];
  __shared__ float lds_l[SLOTS];
  Unit u;
  const int share = a.shape.share;
  const int row = blockIdx.x, qh = blockIdx.y, head = qh / share;
  if (!find_unit<BM, KT>(a, row, true, u) || u.chunks == 1) return;
  const int r = (row - u.row0) * share + qh % share;
  const int tid = threadIdx.x, slot = tid / LANES, d = (tid % LANES) * 8;
  auto at = [&](int chunk) {
    return ((int64_t)(u.base + r / BM * u.chunks + chunk) * a.c.heads + head) * BM + r % BM;
  };
  float m = -INFINITY;
  for (int c = tid & 63; c < u.chunks; c += 64) m = fmaxf(m, a.stat[2 * at(c)]);
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) m = fmaxf(m, __shfl_xor(m, s));
  float l = 0, x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
  for (int c = slot; c < u.chunks; c += SLOTS) {
    float y[8];
    load8(a.part + at(c) * DIM + d, y);
    const float mc = a.stat[2 * at(c)], by = mc == -INFINITY ? 0.0f : exp2f(mc - m);
    l += a.stat[2 * at(c) + 1] * by;
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] += y[k] * by;
  }
  store8(&lds_x[slot][d], x);
  if (d == 0) lds_l[slot] = l;
  __syncthreads();
  if (slot) return;
  l = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = 0;
  for (int s = 0; s < SLOTS; ++s) {
    float y[8];
    load8(&lds_x[s][d], y);
    l += lds_l[s];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] += y[k];
  }
  const float inv = l == 0 ? 0.0f : 1.0f / l;
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = l == 0 ? 0.0f : x[k] * inv;
  store8(static_cast<T*>(a.out.data) + (int64_t)row * a.out.row + (int64_t)qh * a.out.head + d, x);
  if (a.lse && d == 0) a.lse[(int64_t)row * a.qheads + qh] = l == 0 ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---- launch

constexpr int kMinTiles16 = 8;           // 256 keys: a chunk of 64 for each wave
constexpr int kUnits16 = 2048;           // chunks over all key heads that a launch aims at

// Units of the 16-row kernel: a bound of the row tiles, and the chunks on top.
int64_t units16(int64_t rows, int64_t seqs, int share, int heads) {
  const int64_t tiles = (rows * share + 15 * std::min(rows, seqs)) / 16;
  return tiles + std::max<int64_t>(kUnits16 / heads, 1);
}

template <int DIM, typename T, bool TWO>
kronq_status launch16(AttnView a, hipStream_t s) {
  hipLaunchKernelGGL((kv_attention16<DIM, T, TWO>), dim3((unsigned)a.units, (unsigned)a.c.heads), dim3(256), 0, s, a);
  KQ_LAUNCHED("kv_attention16");
  // no chunk can be cut when the longest context the table has room for fits one
  if (room_of(a.c) <= (int64_t)a.min_tiles * 32) return KRONQ_OK;
  hipLaunchKernelGGL((kv_attention_join<DIM, 16, 32, T>), dim3((unsigned)a.c.rows, (unsigned)a.qheads), dim3(256), 0, s, a);
  KQ_LAUNCHED("kv_attention_join");
  return KRONQ_OK;
}

template <int DIM>
kronq_status launch_dim(const AttnView& a, int32_t dtype, hipStream_t s) {
  if (dtype == KRONQ_F32) return launch16<DIM, float, true>(a, s);
  if (dtype == KRONQ_BF16) return launch16<DIM, bf16_t, false>(a, s);
  return launch16<DIM, _Float16, true>(a, s);
}

}  // namespace

size_t kv_attention_ws_bytes(int64_t rows, int64_t seqs, int q_heads, int heads, int dim) {
  const int64_t units = units16(rows, seqs, q_heads / heads, heads);
  return (size_t)units * heads * 16 * (dim + 2) * sizeof(float);
}

kronq_status kv_attention_launch(const KvView& c, int dim, int32_t dtype, const HeadsView& q, int q_heads,
                                 const RopeView& rope, float scale, int window, int sinks, const HeadsView& out,
                                 float* lse, void* ws, hipStream_t s) {
  AttnView a{};
  a.c = c;
  a.q = q;
  a.out = out;
  a.rope = rope;
  a.lse = lse;
  a.qheads = q_heads;
  a.shape = AttnShape{q_heads / c.heads, window, sinks};
  a.scale = scale;
  a.units = (int)units16(c.rows, c.seqs, a.shape.share, c.heads);
  a.min_tiles = kMinTiles16;
  a.part = static_cast<float*>(ws);
  a.stat = a.part + (int64_t)a.units * c.heads * 16 * dim;
  if (dim == 64) return launch_dim<64>(a, dtype, s);
  if (dim == 128) return launch_dim<128>(a, dtype, s);
  return launch_dim<256>(a, dtype, s);
}

}  // namespace kronq
