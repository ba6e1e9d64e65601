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

#include "kvattn.h"

namespace kronq {
namespace {

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

template <int DIM, typename T, int PARTS>
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
  const int r = u.qtile * BM + i, pos = u.ctx - u.len + min(r / share, u.len - 1);
  half8_t q1[KS], q2[PARTS > 1 ? KS : 1];
  const float f = load_query<T, PARTS, KS, 4>(a, u, head, r, g * (DIM / 4), 8, q1, q2);

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
        if constexpr (PARTS > 1) sc[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kv, q2[k], sc[b], 0, 0, 0);
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
      const float ks = cur.bad ? kNan : __uint_as_float(cur.ks[x >> 2][x & 3] & ~15u);
      vs[x] = cur.bad ? kNan : __uint_as_float(cur.vs[x >> 2][x & 3] & ~15u);
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
      if constexpr (PARTS > 1) p2[x] = (_Float16)(y[x] - (float)p1[x]);
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
      if constexpr (PARTS > 1) {
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
    if (u.ctx - u.len + tok >= room_of(a.c)) ll = kNan;
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

// Joins the chunks of one row's head, in the order of the chunks.  blockIdx.x:
// a row; or, where few rows of each sequence are this kernel's (per > 0), a
// sequence's row, per for each.
template <int DIM, int BM, int KT, typename T>
__global__ __launch_bounds__(256) void kv_attention_join(AttnView a, int per) {
  constexpr int LANES = DIM / 8, SLOTS = 256 / LANES;
  __shared__ float lds_x[SLOTS][DIM + 4];
  __shared__ float lds_l[SLOTS];
  Unit u;
  const int share = a.shape.share;
  int row = blockIdx.x;
  if (per) {
    const Seq s = seq_at(a.c, a.shape, blockIdx.x / per, BM, KT);
    if ((int)blockIdx.x % per >= s.len) return;
    row = s.row0 + blockIdx.x % per;
  }
  const int qh = blockIdx.y, head = qh / share;
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
//
// Sequences of up to kFewRows rows x share go to the 16-row kernel, which reads
// the cache once for each 16 of them; longer ones to the 128-row kernel.

constexpr int kFewRows = 32;
constexpr int kMinTiles16 = 8;           // 256 keys: a chunk of 64 for each wave
constexpr int kUnits16 = 2048;           // chunks over all key heads that a launch aims at
constexpr int kMinTiles128 = 4;          // 256 keys
constexpr int kUnits128 = 512;

// How a call is cut: units of each kernel (0: not launched; a bound of its row
// tiles, and chunks on top), and whether there can be chunks to join.
struct Plan {
  int units16, units128;
  bool join16, join128;
  size_t part16, part128;                // floats of partial results
};

Plan plan_of(int64_t rows, int64_t seqs, int share, int heads, int dim) {
  Plan p{};
  const int64_t n = rows * share, some = std::min(rows, seqs);
  // with one sequence the rows decide; with more, few rows for one may be many for another
  if (seqs > 1 || n <= kFewRows) {
    const int64_t tiles = std::min((n + 15 * some) / 16, some * ((kFewRows + 15) / 16));
    const int64_t more = std::max<int64_t>(kUnits16 / heads - tiles / 2, 1);
    p.units16 = (int)(tiles + more);
    p.join16 = more > 1;
  }
  if (n > kFewRows) {
    const int64_t tiles = (n + 127 * std::min<int64_t>(some, n / (kFewRows + 1))) / 128;
    const int64_t more = tiles * heads >= kUnits128 ? 1 : std::max<int64_t>(kUnits128 / heads, 1);
    p.units128 = (int)(tiles + more);
    p.join128 = more > 1;
  }
  if (p.join16) p.part16 = (size_t)p.units16 * heads * 16 * (dim + 2);
  if (p.join128) p.part128 = (size_t)p.units128 * heads * 128 * (dim + 2);
  return p;
}

template <int DIM, int BM, int KT, typename T>
kronq_status join(const AttnView& a, int64_t per, hipStream_t s) {
  // no chunk can be cut when the longest context the table has room for fits one
  if (room_of(a.c) <= (int64_t)a.min_tiles * KT) return KRONQ_OK;
  const bool by_seq = per > 0 && per * a.c.seqs < a.c.rows;
  const int64_t grid = by_seq ? per * a.c.seqs : a.c.rows;
  hipLaunchKernelGGL((kv_attention_join<DIM, BM, KT, T>), dim3((unsigned)grid, (unsigned)a.qheads), dim3(256), 0, s, a,
                     by_seq ? (int)per : 0);
  KQ_LAUNCHED("kv_attention_join");
  return KRONQ_OK;
}

template <int DIM, typename T, int PARTS>
kronq_status launch(AttnView a, int dim, int32_t dtype, float* ws, hipStream_t s) {
  const Plan p = plan_of(a.c.rows, a.c.seqs, a.shape.share, a.c.heads, DIM);
  const bool both = p.units16 && p.units128;
  if (p.units16) {
    a.shape.least = 1;
    a.shape.most = both ? kFewRows : INT32_MAX;
    a.units = p.units16;
    a.min_tiles = kMinTiles16;
    a.part = ws;
    a.stat = ws + (size_t)p.units16 * a.c.heads * 16 * DIM;
    hipLaunchKernelGGL((kv_attention16<DIM, T, PARTS>), dim3((unsigned)a.units, (unsigned)a.c.heads), dim3(256), 0, s, a);
    KQ_LAUNCHED("kv_attention16");
    if (p.join16) {
      const kronq_status st = join<DIM, 16, 32, T>(a, std::max(kFewRows / a.shape.share, 1), s);
      if (st) return st;
    }
  }
  if (p.units128) {
    a.shape.least = both ? kFewRows + 1 : 1;
    a.shape.most = INT32_MAX;
    a.units = p.units128;
    a.min_tiles = kMinTiles128;
    a.part = ws + p.part16;
    a.stat = a.part + (size_t)p.units128 * a.c.heads * 128 * DIM;
    const kronq_status st = kv_rows_launch(a, dim, dtype, s);
    if (st) return st;
    if (p.join128) return join<DIM, 128, 64, T>(a, 0, s);
  }
  return KRONQ_OK;
}

template <int DIM>
kronq_status launch_dim(const AttnView& a, int32_t dtype, float* ws, hipStream_t s) {
  if (dtype == KRONQ_F32) return launch<DIM, float, 2>(a, DIM, dtype, ws, s);
  if (dtype == KRONQ_BF16) return launch<DIM, bf16_t, 1>(a, DIM, dtype, ws, s);
  return launch<DIM, _Float16, 2>(a, DIM, dtype, ws, s);
}

}  // namespace

size_t kv_attention_ws_bytes(int64_t rows, int64_t seqs, int q_heads, int heads, int dim) {
  const Plan p = plan_of(rows, seqs, q_heads / heads, heads, dim);
  return std::max((p.part16 + p.part128) * sizeof(float), size_t(16));
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
