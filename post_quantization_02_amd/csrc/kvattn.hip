// Attention over the 4-bit paged key/value cache.
//
// For each row's head: scores S_j = s_j (q . (c_j - z_j)) over the visible
// positions j, a running maximum m of f S_j with f = scale log2(e), the sum
// l = sum_j 2^(f S_j - m), and O = sum_j 2^(f S_j - m) s'_j (c'_j - z'_j), all in
// one pass over the codes; out = O / l.  The matrix cores see codes as fp16
// numbers (exact); the scales of keys multiply scores, those of values multiply
// weights, both in fp32.
#include <algorithm>
#include <cmath>

#include "kvattn.h"

namespace kronq {
namespace {

// ---- one or two tiles of 16 rows
//
// A workgroup takes a unit of 16 QT rows (rows x share of one key head); its four
// waves take the unit's tiles of 32 keys in turn.  QT is 2 where sequences have
// more than 16 such rows on average, for a tile of keys is then unpacked once for
// 32 (40 sequences of 4 rows x 8, dim 128: 115 us against 135; 24 of 5 rows x 4,
// dim 64 in fp16: 47 against 51); not for dim 256, which has no registers for it.  With 16x16x32 fp16 products
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
  uint32_t v[8][(DIM + 127) / 128];
  uint32_t word;           // lanes 0..31: the key's grid word, 32..63: the value's, of key lane % 32
};

// The pages of a tile's two halves (a page holds at least 16 keys).
struct TilePages { PageAt a, b; };

template <bool SMALL>
__device__ inline TilePages tile_pages(const KvView& c, const int32_t* table, int key0) {
  TilePages p;
  p.a = page_at(c, table, key0);
  p.b = SMALL ? page_at(c, table, key0 + 16) : p.a;
  return p;
}

// A tile's data.  Key0 and pages are the same for all lanes, so with pages that
// hold whole tiles every address is a scalar base and a lane's constant offset;
// with pages of 16 keys (SMALL) a lane chooses between two bases.
template <int DIM, bool SMALL>
__device__ inline void load_tile(const KvView& c, const TilePages& p, int head, int key0, RawTile<DIM>& t) {
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int in_page = (1 << c.lgp) - 1;
  const int64_t first = (int64_t)head << c.lgp;
  const int64_t slot = first + (key0 & in_page), slot2 = SMALL ? first : slot + 16;
  auto pick = [&](bool up, const uint8_t* base, uint32_t stride, int row) {
    const uint8_t* lo = base + page_offset(p.a.page, stride) + slot * row;
    const uint8_t* hi = base + page_offset(p.b.page, stride) + slot2 * row;
    return up ? hi : lo;
  };
  {
    const int row = 8 * ((i >> 2) & 1) + (i & 3), up = i >> 3;
    const uint8_t* k;
    if constexpr (SMALL) k = pick(up, c.kc, c.kcs, DIM / 2) + (row * (DIM / 2) + g * (DIM / 8));
    else k = c.kc + page_offset(p.a.page, c.kcs) + slot * (DIM / 2) + (uint32_t)((16 * up + row) * (DIM / 2) + g * (DIM / 8));
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      if constexpr (DIM == 64) {
        *reinterpret_cast<u32x2*>(t.k[a]) = *reinterpret_cast<const u32x2*>(k + 4 * a * (DIM / 2));
      } else {
#pragma unroll
        for (int w = 0; w < DIM / 32; w += 4)
          *reinterpret_cast<u32x4*>(t.k[a] + w) = *reinterpret_cast<const u32x4*>(k + 4 * a * (DIM / 2) + 4 * w);
      }
    }
  }
  {
    const int row = 8 * (g & 1), up = g >> 1;
    const uint8_t* v;
    if constexpr (SMALL) v = pick(up, c.vc, c.vcs, DIM / 2) + (row * (DIM / 2) + i * (DIM / 32));
    else v = c.vc + page_offset(p.a.page, c.vcs) + slot * (DIM / 2) + (uint32_t)((16 * up + row) * (DIM / 2) + i * (DIM / 32));
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
  {
    const int up = (lane >> 4) & 1;
    const uint32_t* kg = c.kg + (SMALL && up ? page_offset(p.b.page, c.kgs) + slot2 : page_offset(p.a.page, c.kgs) + slot + 16 * up);
    const uint32_t* vg = c.vg + (SMALL && up ? page_offset(p.b.page, c.vgs) + slot2 : page_offset(p.a.page, c.vgs) + slot + 16 * up);
    t.word = (lane < 32 ? kg : vg)[lane & 15];
  }
}

// A tile's queries, made ready by all threads: a thread has eight values of a row
// (two such where dim is 256), asked for before the first keys, and leaves them as
// the products' operands in LDS.  What load_query does for a wave by itself.
template <typename T, int DIM, int QT>
struct QueryPiece {
  static constexpr int kLanes = DIM / 8, kRows = 16 * QT, kPieces = (kRows * kLanes + 255) / 256;
  float x[kPieces][8], o[kPieces][8], c[kPieces][8], s[kPieces][8];
  bool turn[kPieces], fine[kPieces], second[kPieces];

  __device__ __forceinline__ void ask(const AttnView& a, const Unit& u, int head) {
    const RopeView& rope = a.rope;
    const int share = a.shape.share;
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
      const int row = ((int)threadIdx.x / kLanes + n * (256 / kLanes)) & (kRows - 1), d = (int)threadIdx.x % kLanes * 8;
      const int r = u.qtile * kRows + row, tok = min(r / share, u.len - 1), pos = u.ctx - u.len + tok;
      const T* p = static_cast<const T*>(a.q.data) + (int64_t)(u.row0 + tok) * a.q.row +
                   (int64_t)(head * share + r % share) * a.q.head + d;
      fine[n] = !rope.half || pos < rope.positions;
      turn[n] = fine[n] && pos >= 0 && d < 2 * rope.half;   // before the sequence's start: sees nothing
      second[n] = !rope.neighbours && d >= rope.half;
      // every load happens, for branches would wait for theirs: what is not rotated
      // loads its own values in the angles' place
      const int other = !turn[n] || rope.neighbours ? 0 : second[n] ? -rope.half : rope.half;
      const int j = rope.neighbours ? d / 2 : second[n] ? d - rope.half : d;
      const float* ct = turn[n] ? rope.cos + (int64_t)pos * rope.ld + j : reinterpret_cast<const float*>(p);
      const float* st = turn[n] ? rope.sin + (int64_t)pos * rope.ld + j : reinterpret_cast<const float*>(p);
      const int more = turn[n] && !rope.neighbours ? 4 : 0;
      load8(p, x[n]);
      load8(p + other, o[n]);
      const f32x4 c0 = *reinterpret_cast<const f32x4*>(ct), c1 = *reinterpret_cast<const f32x4*>(ct + more);
      const f32x4 s0 = *reinterpret_cast<const f32x4*>(st), s1 = *reinterpret_cast<const f32x4*>(st + more);
#pragma unroll
      for (int k = 0; k < 4; ++k) c[n][k] = c0[k], c[n][4 + k] = c1[k], s[n][k] = s0[k], s[n][4 + k] = s1[k];
    }
  }

  template <int PARTS>
  __device__ __forceinline__ void put(const AttnView& a, const Unit& u, half8_t (*__restrict__ q)[DIM / 32][64],
                                      float* __restrict__ f) {
    const int share = a.shape.share;
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
      if (kRows * kLanes < 256 && (int)threadIdx.x >= kRows * kLanes) break;   // whole waves
      const int row = (int)threadIdx.x / kLanes + n * (256 / kLanes), d8 = (int)threadIdx.x % kLanes;
      float y[8], big = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float cc = a.rope.neighbours ? c[n][k / 2] : c[n][k], ss = a.rope.neighbours ? s[n][k / 2] : s[n][k];
        const float z = a.rope.neighbours ? x[n][k ^ 1] : o[n][k];
        const bool minus = a.rope.neighbours ? !(k & 1) : !second[n];
        const float by = minus ? -ss : ss;
        y[k] = turn[n] ? x[n][k] * cc + z * by : x[n][k];
        big = fmaxf(big, y[k] - y[k] == 0 ? fabsf(y[k]) : INFINITY);
      }
      if (!fine[n]) big = INFINITY;
      big = fmaxf(big, partner<0xB1>(big));
      big = fmaxf(big, partner<0x4E>(big));
      big = fmaxf(big, partner<0x141>(big));
      if constexpr (kLanes > 8) big = fmaxf(big, partner<0x140>(big));
      if constexpr (kLanes > 16) big = fmaxf(big, __shfl_xor(big, 16));
      const bool bad = big == INFINITY;
      int e2 = 0;
      if (!bad && big > 0) {
        frexpf(big, &e2);                                   // big < 2^e2
        e2 = 11 - e2;
      }
      half8_t q1, q2;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float z = bad ? 0.0f : ldexpf(y[kOrder[k]], e2);
        q1[k] = (_Float16)z;
        if constexpr (PARTS > 1) q2[k] = (_Float16)(z - (float)q1[k]);
      }
      const int lane = (row & 15) + 16 * (d8 / (DIM / 32)), k = d8 % (DIM / 32), at = (row >> 4) * PARTS;
      q[at][k][lane] = q1;
      if constexpr (PARTS > 1) q[at + 1][k][lane] = q2;
      if (d8 == 0) {
        const int tok = min((u.qtile * kRows + row) / share, u.len - 1);
        f[row] = bad && u.ctx - u.len + tok >= 0 ? kNan : fmaxf(ldexpf(a.scale * kLog2e, -e2), 0x1p-126f);
      }
    }
  }
};

// In its loop bound by HBM and the vector pipes alike: dim 128, bf16, 131071 keys of
// 8 key heads for one token 32 us (143 MB: 4.4 TB/s, 7 in the loop; 8 us pass before
// it, in three misses one behind the other), 40 sequences of up to 12000 keys 62 us
// (281 MB).  By the vector pipes alone with one query head a key head (fp32, 12 of
// up to 4095 keys, 32 heads: 38 us, 122 MB) and with dim 64 (fp16, 24 x 5 rows x 4 in a
// window of 4096: 43 us).  A wave issues 250 vector operations a tile for 16 rows and
// 8 products a part.  Tiles of 32 rows keep registers in scratch: fp32 and fp16 16 to
// 25 at dim 64, 5 or 6 at dim 128.
template <int DIM, typename T, int PARTS, bool SMALL, int QT>
__global__ __launch_bounds__(256, DIM == 256 ? 1 : QT > 1 && DIM == 128 ? 2 : 3) void kv_attention16(AttnView a) {
  constexpr int BM = 16 * QT, KT = 32, KS = DIM / 32, VT = DIM / 16, PAD = DIM + 4;
  constexpr int AHEAD = 2;                            // tiles in registers; a third one gained nothing
  __shared__ float lds_o[4][16][PAD];
  __shared__ float lds_m[4][16], lds_l[4][16];
  // of a tile's grids: scales (32 keys, 32 values) and the zero points' constants
  __shared__ __align__(16) float lds_s[4][64];
  __shared__ __align__(16) uint32_t lds_kz[4][32][2];
  __shared__ __align__(16) uint16_t lds_vz[4][2][32];
  __shared__ half8_t lds_q[QT * PARTS][KS][64];
  __shared__ float lds_f[BM];
  Unit u;
  if (!find_unit<BM, KT>(a, blockIdx.x, false, u)) return;
  const int head = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int pos_lo, pos_hi;
  const Span span = span_of(a.c, a.shape, u, BM, KT, pos_lo, pos_hi);
  int v0, v1;
  chunk_of(span, u, v0, v1);
  const int share = a.shape.share, window = a.shape.window, sinks = a.shape.sinks;
  const int32_t* table = a.c.table + (int64_t)u.b * a.c.ldt;

  // The first tiles are on their way while the query is made ready.  Past its last
  // tile a wave asks for that one again: a load that may not happen would have to
  // be waited for together with those that must have.
  RawTile<DIM> raw[AHEAD];
  TilePages at[AHEAD]{};
  const int w0 = v0 + wave;
  auto tile_key = [&](int v) { return key_of(span, min(v, v1 - 1), KT); };
  if (w0 < v1) {
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) at[n] = tile_pages<SMALL>(a.c, table, tile_key(w0 + 4 * n));
  }
  QueryPiece<T, DIM, QT> piece;
  piece.ask(a, u, head);
  __builtin_amdgcn_sched_barrier(0);
  if (w0 < v1) {
#pragma unroll
    for (int n = 0; n < AHEAD - 1; ++n) load_tile<DIM, SMALL>(a.c, at[n], head, tile_key(w0 + 4 * n), raw[n]);
  }
  __builtin_amdgcn_sched_barrier(0);

  // this lane's query rows
  piece.template put<PARTS>(a, u, lds_q, lds_f);
  __syncthreads();
  int pos[QT];
  half8_t q1[QT][KS], q2[QT][PARTS > 1 ? KS : 1];
  float f[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    pos[t] = u.ctx - u.len + min((u.qtile * BM + 16 * t + i) / share, u.len - 1);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      q1[t][k] = lds_q[t * PARTS][k][lane];
      if constexpr (PARTS > 1) q2[t][k] = lds_q[t * PARTS + 1][k][lane];
    }
    f[t] = lds_f[16 * t + i];
  }

  const Unpacker un;
  f32x4 o[QT][VT];
  float m[QT], l[QT];                                 // m of S; l of this lane's keys
  int e[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
#pragma unroll
    for (int k = 0; k < VT; ++k) o[t][k] = f32x4{0, 0, 0, 0};
    m[t] = -INFINITY;
    l[t] = 0;
    e[t] = kLeast;
  }

  // Tile v, whose data and pages are given: the data of tile v + 4 (AHEAD - 1) (of
  // pages looked up a tile before) and the pages of the tile after that are asked
  // for on the way.
  auto step = [&](int v, const RawTile<DIM>& cur, TilePages& pages, RawTile<DIM>& next, const TilePages& ahead) {
    const int key0 = key_of(span, v, KT);
    // keys 8 g + x are this lane's; all are seen, but in the tiles at the edges
    const bool edge = key0 + KT - 1 > pos_lo || (window && key0 <= pos_hi - window && key0 + KT > sinks) ||
                      pages.a.bad || pages.b.bad;
    const bool bad = (g >> 1) ? pages.b.bad : pages.a.bad;
    {
      const uint32_t z = cur.word & 15, z1 = zero1024_of(z), z2 = zero64_of(z);
      lds_s[wave][lane] = __uint_as_float(cur.word & ~15u);
      if (lane < 32) {
        *reinterpret_cast<u32x2_alias*>(lds_kz[wave][lane]) = u32x2_alias{z1, z2};
      } else {
        lds_vz[wave][0][lane - 32] = (uint16_t)z1;
        lds_vz[wave][1][lane - 32] = (uint16_t)z2;
      }
    }
    load_tile<DIM, SMALL>(a.c, ahead, head, tile_key(v + 4 * (AHEAD - 1)), next);
    pages = tile_pages<SMALL>(a.c, table, tile_key(v + 4 * AHEAD));
    __builtin_amdgcn_wave_barrier();                  // those parts of LDS are this wave's alone
    f32x4 sc[QT][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const u32x2_alias z = *reinterpret_cast<const u32x2_alias*>(lds_kz[wave][8 * (i >> 2) + 4 * b + (i & 3)]);
      const half2_t z1 = as_half2(z.x), z2 = as_half2(z.y);
#pragma unroll
      for (int t = 0; t < QT; ++t) sc[t][b] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const half8_t kv = un.word(cur.k[b][k], z1, z2);
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          sc[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv, q1[t][k], sc[t][b], 0, 0, 0);
          if constexpr (PARTS > 1) sc[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv, q2[t][k], sc[t][b], 0, 0, 0);
        }
      }
    }
    half8_t p1[QT], p2[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      float s[8], vs[8], top = -INFINITY;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const f32x4_alias ks = *reinterpret_cast<const f32x4_alias*>(&lds_s[wave][8 * g + 4 * b]);
        const f32x4_alias vv = *reinterpret_cast<const f32x4_alias*>(&lds_s[wave][32 + 8 * g + 4 * b]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[4 * b + x] = sc[t][b][x] * ks[x];
          vs[4 * b + x] = vv[x];
        }
      }
      if (edge) {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int j = key0 + 8 * g + x;
          const bool seen = (j <= pos[t]) & ((window == 0) | (j > pos[t] - window) | (j < sinks));
          s[x] = !seen ? -INFINITY : bad ? kNan : s[x];
          vs[x] = seen ? vs[x] : 0.0f;
        }
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) top = fmaxf(top, s[x]);
      if (__any(top * f[t] > fmaf(m[t], f[t], kLazy) || (m[t] == -INFINITY && top > m[t]))) {
        float nm = fmaxf(top, __shfl_xor(top, 16));
        nm = fmaxf(nm, __shfl_xor(nm, 32));
        nm = fmaxf(nm, m[t]);
        if (m[t] != -INFINITY) {
          const float down = fminf((nm - m[t]) * f[t], 300.0f);
          const int ne = max(e[t] - (int)ceilf(down), kLeast);
          const float by = __builtin_amdgcn_exp2f((float)(e[t] - ne) - down);
          l[t] *= __builtin_amdgcn_exp2f(-down);
#pragma unroll
          for (int k = 0; k < VT; ++k) o[t][k] *= by;
          e[t] = ne;
        }
        m[t] = nm;
      }
      // weights times 2^-ue, the part of the row's factor that they can carry (none
      // before the first is known)
      const int ue = e[t] == kLeast ? 0 : min(max(e[t], -60), 30);
      const float most = m[t] == -INFINITY ? 0.0f : m[t] * f[t];
      float base = most + (float)ue;
      if (__any(fabsf(most) > kSteep)) {
#pragma unroll
        for (int x = 0; x < 8; ++x) s[x] -= m[t] == -INFINITY ? 0.0f : m[t];
        base = (float)ue;
      }
      float y[8], ytop = 0, sum = 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float p = __builtin_amdgcn_exp2f(fmaf(s[x], f[t], -base));
        sum += p;
        y[x] = p * vs[x];
        ytop = fmaxf(ytop, fabsf(y[x]));              // a grid's scale may be below 0
      }
      l[t] += sum * ldexpf(1.0f, ue);
      if (__any(ytop > ldexpf(1.0f, min(kTop + e[t] - ue, 127)))) {
        ytop = fmaxf(ytop, __shfl_xor(ytop, 16));
        ytop = fmaxf(ytop, __shfl_xor(ytop, 32));
        if (ytop > ldexpf(1.0f, min(kTop + e[t] - ue, 127))) {
          const int ne = min(max(exponent_for(ytop) + ue, kLeast), kMost);
          const float by = ldexpf(1.0f, e[t] - ne);
#pragma unroll
          for (int k = 0; k < VT; ++k) o[t][k] *= by;
          e[t] = ne;
        }
      }
      if (__any(e[t] != ue)) {
        const float by = ldexpf(1.0f, ue - e[t]);
#pragma unroll
        for (int x = 0; x < 8; ++x) y[x] *= by;
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        p1[t][x] = (_Float16)y[x];
        if constexpr (PARTS > 1) p2[t][x] = (_Float16)(y[x] - (float)p1[t][x]);
      }
    }
    const u32x4_alias z1 = *reinterpret_cast<const u32x4_alias*>(&lds_vz[wave][0][8 * g]);
    const u32x4_alias z2 = *reinterpret_cast<const u32x4_alias*>(&lds_vz[wave][1][8 * g]);
#pragma unroll
    for (int b = 0; b < VT / 2; ++b) {                // byte b of the words: values 2 b, 2 b + 1
      half2_t lo[4], hi[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t w = __builtin_amdgcn_perm(cur.v[2 * x + 1][b >> 2], cur.v[2 * x][b >> 2],
                                                 0x0C000C00u | (uint32_t)(b & 3) | ((uint32_t)(4 + (b & 3)) << 16));
        lo[x] = un.low_pair(w, as_half2(z1[x]));
        hi[x] = un.high_pair(w, as_half2(z2[x]));
      }
      const half8_t va{lo[0].x, lo[0].y, lo[1].x, lo[1].y, lo[2].x, lo[2].y, lo[3].x, lo[3].y};
      const half8_t vb{hi[0].x, hi[0].y, hi[1].x, hi[1].y, hi[2].x, hi[2].y, hi[3].x, hi[3].y};
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        o[t][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(va, p1[t], o[t][2 * b], 0, 0, 0);
        o[t][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vb, p1[t], o[t][2 * b + 1], 0, 0, 0);
        if constexpr (PARTS > 1) {
          o[t][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(va, p2[t], o[t][2 * b], 0, 0, 0);
          o[t][2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vb, p2[t], o[t][2 * b + 1], 0, 0, 0);
        }
      }
    }
  };
  for (int v = w0; v < v1; v += 4 * AHEAD) {
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      if (v + 4 * n >= v1) break;
      step(v + 4 * n, raw[n], at[n], raw[(n + AHEAD - 1) % AHEAD], at[(n + AHEAD - 1) % AHEAD]);
    }
  }

  // the four waves' parts, sixteen rows at a time
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    if (t) __syncthreads();
    l[t] += __shfl_xor(l[t], 16);
    l[t] += __shfl_xor(l[t], 32);
    if (lane < 16) {
      lds_m[wave][i] = m[t] == -INFINITY ? -INFINITY : m[t] * f[t];
      lds_l[wave][i] = l[t];
    }
    const float back = ldexpf(1.0f, e[t]);
#pragma unroll
    for (int rr = 0; rr < 4; ++rr) {
#pragma unroll
      for (int k = 0; k < VT; k += 4)
        *reinterpret_cast<f32x4*>(&lds_o[wave][i][VT * (4 * g + rr) + k]) =
            f32x4{o[t][k][rr], o[t][k + 1][rr], o[t][k + 2][rr], o[t][k + 3][rr]} * back;
    }
    __syncthreads();
    // thread: 8 values of one row at a time
    for (int c = tid; c < 16 * DIM / 8; c += 256) {
      const int row = c / (DIM / 8), d = (c % (DIM / 8)) * 8;
      const int rg = u.qtile * BM + 16 * t + row;
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
      if (u.ctx - u.len + tok >= room_of(a.c)) ll = kNan;
      if (u.chunks == 1) {
        const float inv = ll == 0 ? 0.0f : 1.0f / ll;
#pragma unroll
        for (int y = 0; y < 8; ++y) x[y] = ll == 0 ? 0.0f : x[y] * inv;
        store8(static_cast<T*>(a.out.data) + (int64_t)(u.row0 + tok) * a.out.row + (int64_t)qh * a.out.head + d, x);
        if (a.lse && d == 0)
          a.lse[(int64_t)(u.row0 + tok) * a.qheads + qh] = ll == 0 ? -INFINITY : (mm + log2f(ll)) * kLn2;
      } else if (u.place < a.places) {
        const int64_t at = ((int64_t)u.place * a.c.heads + head) * BM + 16 * t + row;
        store8(a.part + at * DIM + d, x);
        if (d == 0) {
          a.stat[2 * at] = mm;
          a.stat[2 * at + 1] = ll;
        }
      }
    }
  }
}

// Joins the chunks of a row's heads, in the order of the chunks.  blockIdx.x: a
// row; or, where few rows of each sequence are this kernel's (per > 0), a
// sequence's row, per for each.  A head is joined by `slots` groups of lanes (a
// power of two), each of which adds up every slots-th chunk.  Latency: 5 to 6 us.
template <int DIM, int BM, int KT, typename T>
__global__ __launch_bounds__(256) void kv_attention_join(AttnView a, int per, int slots) {
  constexpr int LANES = DIM / 8, GROUPS = 256 / LANES;
  __shared__ float lds_x[GROUPS][DIM + 4];
  __shared__ float lds_l[GROUPS];
  if (a.told && !a.told->any) return;
  Unit u;
  const int share = a.shape.share;
  int row = blockIdx.x;
  if (per) {
    const Seq s = seq_at(a.c, a.shape, blockIdx.x / per, BM, KT);
    if ((int)blockIdx.x % per >= s.len) return;
    row = s.row0 + blockIdx.x % per;
  }
  if (!find_unit<BM, KT>(a, row, true, u) || u.chunks == 1) return;
  if (u.place + ((int64_t)u.len * share - 1) / BM * u.chunks + u.chunks > a.places) return;
  const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES, d = lane * 8;
  const int slot = group & (slots - 1), qh = (int)blockIdx.y * (GROUPS / slots) + group / slots;
  const bool in = qh < a.qheads;
  const int head = qh / share, r = (row - u.row0) * share + qh % share;
  auto at = [&](int chunk) {
    return ((int64_t)(u.place + r / BM * u.chunks + chunk) * a.c.heads + head) * BM + r % BM;
  };
  const int width = min(slots * LANES, 64);          // lanes of a wave that share the head
  float m = -INFINITY;
  if (in)
    for (int c = threadIdx.x & (width - 1); c < u.chunks; c += width) m = fmaxf(m, a.stat[2 * at(c)]);
  for (int s = 1; s < width; s <<= 1) m = fmaxf(m, __shfl_xor(m, s));
  float l = 0, x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (in) {
#pragma unroll 4
    for (int c = slot; c < u.chunks; c += slots) {
      float y[8];
      load8(a.part + at(c) * DIM + d, y);
      const float mc = a.stat[2 * at(c)], by = mc == -INFINITY ? 0.0f : exp2f(mc - m);
      l += a.stat[2 * at(c) + 1] * by;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] += y[k] * by;
    }
  }
  if (slots > 1) {
    store8(&lds_x[group][d], x);
    if (lane == 0) lds_l[group] = l;
    __syncthreads();
    if (slot) return;
    for (int s = 1; s < min(slots, u.chunks); ++s) {
      float y[8];
      load8(&lds_x[group + s][d], y);
      l += lds_l[group + s];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] += y[k];
    }
  }
  if (!in) return;
  const float inv = l == 0 ? 0.0f : 1.0f / l;
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = l == 0 ? 0.0f : x[k] * inv;
  store8(static_cast<T*>(a.out.data) + (int64_t)row * a.out.row + (int64_t)qh * a.out.head + d, x);
  if (a.lse && lane == 0) a.lse[(int64_t)row * a.qheads + qh] = l == 0 ? -INFINITY : (m + log2f(l)) * kLn2;
}

// How long the chunks of up to two launches are, where each of their waves adding
// that up for itself would cost more (more than 64 sequences: 1000 of 200 to 700
// keys, 8 key heads, 260 us with this kernel, 369 without), or a join that finds
// nothing (many rows).  A workgroup for each.  Latency: 4 us.
struct CutAsked {
  AttnShape shape;
  Cut cut;
  int min_tiles, bm, kt;
  CutTold* told;
};

__global__ __launch_bounds__(256) void kv_attention_cut(KvView c, CutAsked first, CutAsked second) {
  __shared__ double sums[2][4];
  __shared__ int most[4];
  const CutAsked a = blockIdx.x ? second : first;
  double rows = 0, work = 0;
  int longest = 0;
#pragma unroll 4
  for (int b = threadIdx.x; b < c.seqs; b += 256) {
    const Seq s = seq_at(c, a.shape, b, a.bm, a.kt);
    rows += s.qtiles;                                 // sums of integers below 2^53: exact
    work += (double)s.qtiles * s.tiles;
    longest = max(longest, s.tiles);
  }
  const int wave = threadIdx.x >> 6;
  rows = wave_sum(rows);
  work = wave_sum(work);
  longest = wave_max(longest);
  if ((threadIdx.x & 63) == 0) sums[0][wave] = rows, sums[1][wave] = work, most[wave] = longest;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < 4; ++w) rows += sums[0][w], work += sums[1][w], longest = max(longest, most[w]);
  const int per = chunk_tiles(work, rows, used_units(a.cut, rows), a.min_tiles);
  *a.told = CutTold{per, longest > per};
}

// ---- launch
//
// Sequences of up to kFewRows rows x share go to the kernel of few rows, which
// reads and unpacks the cache once for each 16 or 32 of them; longer ones to the
// kernel of 128 or 256.  Both take any length, so a batch whose sequences have few
// rows on average is one launch of the first (a launch that finds nothing costs
// 5 us).  8 sequences of up to 8000 keys, dim 128, bf16, with up to 64, 96, 128 rows x
// share: 32, 40, 44 us by the kernel of few, 70, 75, 77 by both; 24 sequences of up to
// 96, 128, 192: 105, 130, 181 and 129, 134, 158.  One prompt among 40 single tokens x
// 4, bf16: of 60, 250, 500 rows 78, 168, 228 by the kernel of few, 94, 156, 223 by
// both; among 140 of 500 and 2000 rows 342 and 653, 381 and 608 (fp16: 809 and over 1182).
// What the average gives up: dim 256 (250 rows among 40: 384 and 305; 2000 among 140:
// 1836 and 1202), and a batch padded to 256 sequences (one of 4000 rows: 795 and 629).

constexpr int kFewRows = 64;
// Tiles of a chunk at least: two for each wave (3000 keys: 14.4 us at 4, 13.8 at 8,
// 14.8 at 16; 6000 keys: 15.3, 16.4, 16.8).
constexpr int kMinTiles16 = 8;
// Where the table has room for no more than this, the keys are not cut: six steps
// of a wave cost less than a join behind two (one token, whole and cut: 613 keys
// 11.5 and 12.3 us, 1000 keys 14.7 and 12.3).
constexpr int kWholeTiles16 = 24;
// Chunks over all key heads that a launch aims at: a little under the 768
// workgroups that are resident at once (three on a CU), because a unit's start (its
// search, its query, the first tile) takes 8 us and all units' starts then pass
// together.  Call times at 672, 744, 768: 131071 keys 42, 41, 40 us (48 at 1450); 40
// sequences 77, 70, 71; 12 of 32 key heads 43, 42, 46.  Measured for dim 64 and 128:
// of dim 256 one workgroup fits a CU (its registers), and 744 are three rounds (60000
// keys 61 us; no other number was measured).
constexpr int kUnits16 = 744;
constexpr int kUnits32 = 496;            // of 512: two tiles of rows, dim 128
// The kernel of many rows: tiles of 128 or 256 rows, the latter where sequences
// have that many on average (a tile of keys is unpacked once for all of its rows).
// 2047 and 1774 rows x 4 behind 9001 and 4830 keys, dim 128: 616 us in tiles of 128
// rows, 575 in tiles of 256.
constexpr int kTallRows = 256;
constexpr int kMinTilesRows = 4;         // 256 keys
// Workgroups resident at once: two of four waves on a CU, or one of eight.  Row
// tiles that fill half of them or less are cut along the keys to fill 7/8 (one
// round), fewer than all to twice that (two rounds of smaller ones).  One sequence of
// up to 8000 keys, rows x 4, dim 128, bf16: 256 rows 74 us in one round, 91 in two;
// 1024 rows 188 and 231 (fp32: 314 and 397); two such sequences, more than half: 319
// and 287.  Of dim 256, and of 128 rows in fp32 and fp16 at dim 128, one workgroup
// fits a CU: for them these are twice as many, and no other number was measured.
constexpr int kResident = 512, kResidentTall = 256;

// The join gives each row's head as many groups of lanes as make this many
// workgroups (40 sequences, attention and join: 72 us at 128, 71 at 512, 76 at 2048).
constexpr int64_t kJoinGroups = 512;

// Tiles of a chunk at least where nothing may be cut: the units that a batch does
// not need for its row tiles (they are a bound) would otherwise be taken for chunks.
constexpr int kUncut = INT32_MAX;

// How a call is cut: units of each kernel (0: not launched; a bound of its row
// tiles, and chunks on top), and whether there can be chunks to join.
struct Plan {
  Cut few, rows;
  int waves;
  int tall;                              // the first's tiles are of 16 << tall rows
  bool join16, join_rows;
  bool told16, told_rows;                // kv_attention_cut runs before them
  size_t told, part16, part_rows;        // floats: what it leaves, partial results
};

// Where row tiles alone fill the chip, a kSpare-th part of it is left for chunks all
// the same, and the join is launched: one sequence may be longer than all others
// together.  131071 keys among 255 sequences of 200 to 700, 8 key heads x 4: 1047 us
// whole, 134 cut; 64 rows behind 131071 keys among 40 prompts of 512: 5035 and 946;
// 200 sequences of 1500 to 12000, x 8: 370 and 342.  Where nothing is cut the two
// launches cost 5 us (200 sequences of 200 to 700 keys: 44 and 49; 8 prompts of 1024:
// 200 and 206).
constexpr int kSpare = 2;

Plan plan_of(int64_t rows, int64_t seqs, int share, int heads, int dim) {
  Plan p{};
  const int64_t n = rows * share, some = std::min(rows, seqs);
  const bool few = n <= kFewRows * some;   // on average, or for sure
  if (few || seqs > 1) {
    p.tall = few && n > 16 * some && dim < 256;
    const int64_t bm = 16 << p.tall;
    const int64_t tiles = std::min((n + (bm - 1) * some) / bm, few ? n : some * ((kFewRows + 15) / 16));
    const int64_t aim = (p.tall && dim == 128 ? kUnits32 : kUnits16) / heads;
    const int64_t spare = std::max<int64_t>(aim / kSpare, 1), more = std::max(aim - tiles / 2, spare);
    p.few = Cut{(int)(tiles + more), (int)aim, (int)spare};
    p.join16 = more > 1;
  }
  if (!few) {
    p.waves = dim < 256 && n >= kTallRows * some ? 8 : 4;
    const int64_t bm = 32 * p.waves, resident = (p.waves == 8 ? kResidentTall : kResident) / heads;
    const int64_t tiles = (n + (bm - 1) * std::min<int64_t>(some, n / (kFewRows + 1))) / bm;
    if (2 * tiles <= resident) {
      const int64_t more = std::max<int64_t>(resident * 7 / 8 - tiles / 2, 1);
      p.rows = Cut{(int)(tiles + more), (int)(resident * 7 / 8), 1};
    } else if (tiles < resident) {
      p.rows = Cut{(int)(2 * resident), (int)(2 * resident), 1};
    } else {
      // tiles of one sequence are equally long but for their own rows
      const int64_t spare = some > 1 ? std::max<int64_t>(resident / kSpare, 1) : 1;
      p.rows = Cut{(int)(tiles + spare), (int)(some > 1 ? resident : 0), (int)spare};
    }
    p.join_rows = p.rows.units - tiles > 1;
    p.told_rows = p.join_rows && (seqs > 64 || tiles >= resident);
  }
  p.told16 = p.join16 && seqs > 64;
  if (p.told16 || p.told_rows) p.told = 4;
  if (p.join16) p.part16 = (size_t)places_of(p.few) * heads * (16 << p.tall) * (dim + 2);
  if (p.join_rows) p.part_rows = (size_t)places_of(p.rows) * heads * 32 * p.waves * (dim + 2);
  return p;
}

template <int DIM, int BM, int KT, typename T>
kronq_status join(const AttnView& a, int64_t per, hipStream_t s) {
  // no chunk can be cut when the longest context the table has room for fits one
  if (room_of(a.c) <= (int64_t)a.min_tiles * KT) return KRONQ_OK;
  const bool by_seq = per > 0 && per * a.c.seqs < a.c.rows;
  const int64_t grid = by_seq ? per * a.c.seqs : a.c.rows;
  constexpr int groups = 256 / (DIM / 8);
  int slots = 1;
  while (slots < groups && grid * a.qheads * slots / groups < kJoinGroups) slots *= 2;
  const int at_once = groups / slots;
  hipLaunchKernelGGL((kv_attention_join<DIM, BM, KT, T>),
                     dim3((unsigned)grid, (unsigned)((a.qheads + at_once - 1) / at_once)), dim3(256), 0, s, a,
                     by_seq ? (int)per : 0, slots);
  KQ_LAUNCHED("kv_attention_join");
  return KRONQ_OK;
}

template <int DIM, typename T, int PARTS, int QT>
kronq_status launch_few(const AttnView& a, const Plan& p, bool both, hipStream_t s) {
  const dim3 grid((unsigned)a.cut.units, (unsigned)a.c.heads);
  if (a.c.lgp == 4) hipLaunchKernelGGL((kv_attention16<DIM, T, PARTS, true, QT>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((kv_attention16<DIM, T, PARTS, false, QT>), grid, dim3(256), 0, s, a);
  KQ_LAUNCHED("kv_attention16");
  if (!p.join16) return KRONQ_OK;
  return join<DIM, 16 * QT, 32, T>(a, both ? std::max(kFewRows / a.shape.share, 1) : 0, s);
}

template <int DIM, typename T, int PARTS>
kronq_status launch(AttnView a, int dim, int32_t dtype, float* ws, hipStream_t s) {
  const Plan p = plan_of(a.c.rows, a.c.seqs, a.shape.share, a.c.heads, DIM);
  const bool both = p.few.units && p.rows.units;
  CutTold* told = reinterpret_cast<CutTold*>(ws);
  AttnView few = a, rows = a;
  int asked = 0;
  CutAsked ask[2] = {};
  // a kernel's part of the workspace, and what is asked for it beforehand
  auto ready = [&](AttnView& v, const Cut& cut, bool joined, bool ahead, int min_tiles, int bm, int kt, float* part) {
    v.cut = cut;
    v.min_tiles = joined ? min_tiles : kUncut;
    v.places = joined ? places_of(cut) : 0;
    v.part = part;
    v.stat = part + (size_t)v.places * a.c.heads * bm * DIM;
    if (!ahead || room_of(a.c) <= (int64_t)v.min_tiles * kt) return;
    v.told = told + asked;
    ask[asked] = CutAsked{v.shape, cut, v.min_tiles, bm, kt, told + asked};
    ++asked;
  };
  if (p.few.units) {
    few.shape.least = 1;
    few.shape.most = both ? kFewRows : INT32_MAX;
    ready(few, p.few, p.join16, p.told16, room_of(a.c) <= kWholeTiles16 * 32 ? kWholeTiles16 : kMinTiles16, 16 << p.tall,
          32, ws + p.told);
  }
  if (p.rows.units) {
    rows.shape.least = both ? kFewRows + 1 : 1;
    rows.shape.most = INT32_MAX;
    ready(rows, p.rows, p.join_rows, p.told_rows, kMinTilesRows, 32 * p.waves, 64, ws + p.told + p.part16);
  }
  if (asked) {
    hipLaunchKernelGGL(kv_attention_cut, dim3((unsigned)asked), dim3(256), 0, s, a.c, ask[0], ask[1]);
    KQ_LAUNCHED("kv_attention_cut");
  }
  if (p.few.units) {
    kronq_status st;
    if constexpr (DIM < 256)
      st = p.tall ? launch_few<DIM, T, PARTS, 2>(few, p, both, s) : launch_few<DIM, T, PARTS, 1>(few, p, both, s);
    else
      st = launch_few<DIM, T, PARTS, 1>(few, p, both, s);
    if (st) return st;
  }
  if (p.rows.units) {
    const kronq_status st = kv_rows_launch(rows, dim, dtype, p.waves, s);
    if (st || !p.join_rows) return st;
    if constexpr (DIM < 256)
      if (p.waves == 8) return join<DIM, 256, 64, T>(rows, 0, s);
    return join<DIM, 128, 64, T>(rows, 0, s);
  }
  return KRONQ_OK;
}

template <int DIM>
kronq_status launch_dim(const AttnView& a, int32_t dtype, float* ws, hipStream_t s) {
  // Operands in two fp16 parts are as good as fp32 ones (2^-22); in bf16 one part's
  // 2^-11 lies below the result's own 2^-8.
  if (dtype == KRONQ_F32) return launch<DIM, float, 2>(a, DIM, dtype, ws, s);
  if (dtype == KRONQ_BF16) return launch<DIM, bf16_t, 1>(a, DIM, dtype, ws, s);
  return launch<DIM, _Float16, 2>(a, DIM, dtype, ws, s);
}

}  // namespace

size_t kv_attention_ws_bytes(int64_t rows, int64_t seqs, int q_heads, int heads, int dim) {
  const Plan p = plan_of(rows, seqs, q_heads / heads, heads, dim);
  return std::max((p.told + p.part16 + p.part_rows) * sizeof(float), size_t(16));
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
  a.shape = AttnShape{q_heads / c.heads, window, sinks, 1, INT32_MAX};
  a.scale = scale;
  if (dim == 64) return launch_dim<64>(a, dtype, static_cast<float*>(ws), s);
  if (dim == 128) return launch_dim<128>(a, dtype, static_cast<float*>(ws), s);
  return launch_dim<256>(a, dtype, static_cast<float*>(ws), s);
}

}  // namespace kronq
