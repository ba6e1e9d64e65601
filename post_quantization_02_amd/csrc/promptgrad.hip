// Gradients of attention over whole packed prompts.  With S = scale Q K^T over what
// rows see, P = exp(S - lse), delta_i = sum_j P_ij dP_ij:
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q
//
// Two kernels, so that no sum needs atomics or a second pass: one takes 128 rows of a
// query head and goes through their keys (dQ), one takes 128 keys of a key head and
// goes through the rows of all its query heads (dK, dV stay in registers).  Both
// compute S and dP.  Where there are too few of these for the chip (SPLIT), a workgroup
// takes 32 rows or keys, its waves every fourth tile each, by themselves, and the four
// parts are joined in LDS.
//
// delta is dO . O, but O has been rounded to its type, and where one key has most of
// a row's weight dP - delta is small beside that rounding.  The rows of dS sum to 0,
// so with a delta that is off the sum is what it is off by, r_i: the first kernel
// sums it beside B = P K, takes r B off dQ and hands the right delta to the second.
// (Not for fp32, whose outputs hold it well enough.)  A row that sees one key has dS = 0,
// not what two ways to sum dO . V differ by (times 0: what is not a number stays).
//
// Bound by the matrix cores and the vector pipes, which overlap little: 9807 rows of 8
// sequences, 32 heads of 128 on 8, bf16, 305 + 320 us, the matrix cores busy 37 and 34 %
// of the time.  Of the eight products five are the formulas' (480 TFLOP/s); S and dP
// twice and B are what the two kernels and the right delta cost.  P and dS are rounded
// to the operands' type, half a step of it each, which makes dq and dk up to 1.6 times
// as far off as a plain form in fp32 on the same inputs that rounds its results only; dS
// in two parts would be nearer for two more products.  Statistics, delta and all sums
// are fp32.
#include "prompt.h"

namespace kronq {
namespace {

constexpr int NT = 256;

// Weights on their way into an operand of fp16, whose range is small: those of a
// lane's column are held times a power of two that follows the column's largest
// (below 2^15), and so are its results, until they are stored.  Other types hold
// them as they are.
template <typename T>
struct Fit {
  __device__ __forceinline__ float back() const { return 1; }
  template <int DN>
  __device__ __forceinline__ void scale(float (&)[16], f32x16 (&)[DN]) {}
};

template <>
struct Fit<_Float16> {
  float by = 0x1p127f;
  __device__ __forceinline__ float back() const { return 1 / by; }
  template <int DN>
  __device__ __forceinline__ void scale(float (&w)[16], f32x16 (&acc)[DN]) {
    float top = 0;
#pragma unroll
    for (int x = 0; x < 16; ++x) top = fmaxf(top, fabsf(w[x]));
    top = both_max(top);
    if (__any(top * by >= 0x1p15f)) {
      rarely();
      // 2^(13 - e) for a largest of 2^e and up
      const int e = (int)(__float_as_uint(top) >> 23);
      const float to = fminf(by, __uint_as_float((uint32_t)min(max(267 - e, 1), 254) << 23));
      const float f = to / by;
#pragma unroll
      for (int dt = 0; dt < DN; ++dt)
#pragma unroll
        for (int x = 0; x < 16; ++x) acc[dt][x] *= f;
      by = to;
    }
#pragma unroll
    for (int x = 0; x < 16; ++x) w[x] *= by;
  }
};

// While a wave has products to do it goes before the SIMD's others, which fill the vector
// pipes meanwhile.  Both kernels, us, without and with: bf16, dim 128, 594 and 582, one
// sequence of 1500 rows 188 and 170; dim 64 324 and 300, in fp16 266 and 271; dim 256,
// where a SIMD has one wave, 842 and 856 (not done there).
template <int D>
__device__ __forceinline__ void products(bool begin) {
  if (D == 256) return;
  if (begin) __builtin_amdgcn_s_setprio(1);
  else __builtin_amdgcn_s_setprio(0);
}

// ---------------------------------------------------------------- queries

constexpr int KT = 32;

template <typename T, int D, bool SPLIT>
struct RowsLds {
  static constexpr bool FIX = sizeof(T) == 2;      // delta is put right; dO is held here
  union {
    struct { LdsTile<T, D, KT> k[SPLIT ? 4 : 2], v[SPLIT ? 4 : 2]; } tile;
    typename std::conditional<SPLIT, JoinLds<D / 32>, int>::type join;
  };
  typename std::conditional<FIX, LdsTile<T, D, 32>, int>::type own[SPLIT ? 1 : 4];
  float off[4][64];
  // Of a tile that some row does not see all of: keys that are not finite.  Of a tile, the
  // next, and the one after, which is cleared while the others are in use (SPLIT: a wave's).
  uint32_t odd[4];
  __device__ RowsLds() {}
};

template <typename T, int D, bool SPLIT>
__global__ __launch_bounds__(NT, SPLIT || D == 256 || (D == 128 && sizeof(T) == 4) ? 1 : 2) void prompt_rows_grad(PromptArgs a) {
  constexpr int BM = SPLIT ? 32 : 128, DT = D / 32, STEPS = D / Op<T>::STEP, BY = SPLIT ? 4 : 1;
  typedef RowsLds<T, D, SPLIT> Lds;
  constexpr bool FIX = Lds::FIX;
  typedef LdsTile<T, D, KT> Tile;
  typedef Staged<T, D, KT, SPLIT ? 64 : NT> Stage;
  __shared__ Lds lds;
  const int g = blockIdx.x % a.heads, hs = blockIdx.x / a.heads % a.share, unit = blockIdx.x / (a.heads * a.share);
  const int head = g * a.share + hs;
  Prompt p;
  int much;
  if (!find_tile(a, BM, unit, p, much)) return;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = (much - 1) * BM, w0 = SPLIT ? r0 : r0 + 32 * wave, row = w0 + (lane & 31);
  const uint32_t to_lane = Stage::lane(), rows_lane = Tile::rows_lane(), d_lane = Tile::d_lane();
  auto& own = lds.own[SPLIT ? 0 : wave];           // SPLIT: all waves write the same

  typename Op<T>::frag qc[STEPS], oc[FIX ? 1 : STEPS];
  float neg_lse, neg_delta;
  {
    typename Op<T>::frag f[STEPS], o[STEPS];
    load_column<T, D>(a.dout, p.start, head, row, p.n, a.dim, f);
    load_column<T, D>(a.out, p.start, head, row, p.n, a.dim, o);
    float sum = 0;
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int i = 0; i < Op<T>::EPL; ++i) sum = fmaf(Op<T>::value(f[s], i), Op<T>::value(o[s], i), sum);
    neg_delta = -both_sum(sum);
    const float lse = a.lse[(int64_t)(p.start + min(row, p.n - 1)) * (a.heads * a.share) + head];
    // a row of no weight has none
    neg_lse = lse == -INFINITY ? -INFINITY : -lse * kPromptLog2e;
    if constexpr (FIX) {
      put_column<T, D>(lds_at(own) + rows_lane, f);
    } else {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) oc[s] = f[s];
    }
  }
  load_column<T, D>(a.q, p.start, head, row, p.n, a.dim, qc);
  const float c = a.scale * kPromptLog2e;
  f32x16 dq[DT], pk[FIX ? DT : 1];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int x = 0; x < 16; ++x) dq[dt][x] = pk[FIX ? dt : 0][x] = 0;
  Fit<T> fit;
  float off = 0;                          // what this lane's rows of dS sum to

  const TileSpan span = keys_of_rows(r0, BM, p.n, a.window, KT);
  const int t0 = span.first, t1 = span.last;
  Stage sk, sv;
  // whether some row of the workgroup does not see all of tile t
  auto cut = [&](int t) {
    return t * KT + KT - 1 > r0 || t * KT <= r0 + BM - 1 - a.window;
  };
  auto fetch = [&](int t) __attribute__((always_inline)) {
    sk.load(a.k, p.start, g, t * KT, p.n, a.dim);
    sv.load(a.v, p.start, g, t * KT, p.n, a.dim);
  };
  auto put = [&](int t, int to, int slot) __attribute__((always_inline)) {
    if (cut(t)) {
      rarely();
      // 0 times them would not be 0.  A row that sees one has no number for a maximum, or
      // no weight for the key.
      const uint32_t keys = sk.clean();
      if (keys) atomicOr(&lds.odd[slot], keys);
    }
    sk.store(hidden(lds_at(lds.tile.k[to]) + to_lane));
    sv.store(hidden(lds_at(lds.tile.v[to]) + to_lane));
  };
  if (tid < 4) lds.odd[tid] = 0;
  const int first = SPLIT ? t0 + wave : t0;
  if (first <= t1) fetch(first);
  __syncthreads();
  if (!SPLIT) put(first, first & 1, 0);
  int slot = SPLIT ? wave : 0;
  for (int t = first; t <= t1; t += BY) {
    const int from = SPLIT ? wave : t & 1;
    int next_slot = slot;
    if (SPLIT) {
      own_lds();
      if (lane == 0) lds.odd[slot] = 0;
      own_lds();
      put(t, from, slot);
      own_lds();
    } else {
      __syncthreads();
      next_slot = slot == 2 ? 0 : slot + 1;
      if (tid == 0) lds.odd[next_slot == 2 ? 0 : next_slot + 1] = 0;
    }
    if (t + BY <= t1) fetch(t + BY);
    const int k0 = t * KT;
    const bool none = k0 > w0 + 31 || k0 + KT - 1 <= w0 - a.window;
    if (!none) {
      f32x16 s, d;
#pragma unroll
      for (int x = 0; x < 16; ++x) s[x] = 0, d[x] = neg_delta;
      const uint32_t k_at = hidden(lds_at(lds.tile.k[from]) + rows_lane), v_at = hidden(lds_at(lds.tile.v[from]) + rows_lane);
      products<D>(true);
      s = scores<T, D>(k_at, 0, qc, s);
      if constexpr (FIX) d = scores<T, D>(v_at, hidden(lds_at(own) + rows_lane), d);
      else d = scores<T, D>(v_at, 0, oc, d);
      products<D>(false);
      float w[16], u[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        w[x] = __builtin_amdgcn_exp2f(fmaf(s[x], c, neg_lse));
        u[x] = w[x] * d[x];
      }
      if (k0 + KT - 1 > w0 || k0 <= w0 + 31 - a.window) {
        rarely();
        const int from_key = (int)hidden(row - k0 - 4 * h);
        const uint32_t fine = hidden(~lds.odd[slot] >> (4 * h));
        const float alone = row == 0 || a.window == 1 ? 0.0f : 1.0f;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int r = block_row(x, 0);
          const bool in = r <= from_key && r > from_key - a.window && (fine >> r & 1);
          w[x] = in ? w[x] : 0.0f;
          u[x] = in ? u[x] * alone : 0.0f;
        }
      }
      if constexpr (FIX) {
#pragma unroll
        for (int x = 0; x < 16; ++x) off += u[x];
      }
      fit.scale(u, dq);
      const uint32_t kd_at = hidden(lds_at(lds.tile.k[from]) + d_lane);
      products<D>(true);
      if constexpr (FIX) contract_two<T, D>(kd_at, u, dq, w, pk);
      else contract<T, D, 0, DT, 1>(kd_at, 0, u, dq);
      products<D>(false);
    }
    if (!SPLIT && t < t1) put(t + 1, from ^ 1, next_slot);
    slot = next_slot;
  }
  if constexpr (FIX) off = both_sum(off);
  if constexpr (SPLIT && FIX) {
    lds.off[wave][lane] = off;
    __syncthreads();
    off = (lds.off[0][lane] + lds.off[1][lane]) + (lds.off[2][lane] + lds.off[3][lane]);
  }
  if constexpr (FIX) {
    neg_delta -= off;
    const float by = off / fit.back();
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int x = 0; x < 16; ++x) dq[dt][x] -= by * pk[dt][x];
  }
  if constexpr (SPLIT) {
    if (!FIX) __syncthreads();
    put_part(lds.join, dq, fit.back());
    __syncthreads();
#pragma unroll
    for (int dt = 0; dt < DT; dt += 4)
      if (dt + wave < DT && row < p.n) {
        const f32x16 y[1] = {joined(lds.join, dt + wave)};
        store_column<T, 1>(a.dq, p.start, head, row, a.dim, 32 * (dt + wave), y, a.scale);
      }
  } else if (row < p.n) {
    store_column<T, DT>(a.dq, p.start, head, row, a.dim, 0, dq, a.scale * fit.back());
  }
  if (row < p.n && h == 0 && (!SPLIT || wave == 0)) {
    const int64_t at = (int64_t)head * a.rows + p.start + row;
    a.neg_lse[at] = neg_lse;
    a.neg_delta[at] = neg_delta;
  }
}

// ---------------------------------------------------------------- keys and values

// How a workgroup goes through its keys' rows: 128 keys by four waves, 32 keys split
// (SPLIT), or 128 keys by eight waves, of which the second four take the second half of
// each tile.  A key tile at a long sequence's start has many rows to go through, and where
// there are few workgroups a CU the launch is as long as that takes: with eight waves
// half as long for the same work.
enum Way { kFour, kSplit, kEight };

template <typename T, int D, int DN, Way WAY>
struct KeysLds {
  static constexpr bool SPLIT = WAY == kSplit;
  static constexpr int HALVES = WAY == kEight ? 2 : 1, QT = 32 * HALVES;
  static constexpr bool JOINED = SPLIT || HALVES == 2;
  static constexpr bool OWN = sizeof(T) == 2 && D == 128;   // values are held here: no registers left
  union {
    struct { LdsTile<T, D, QT> q[SPLIT ? 4 : 2], o[SPLIT ? 4 : 2]; } tile;
    typename std::conditional<JOINED, JoinLds<DN>, int>::type join;
  };
  typename std::conditional<OWN, LdsTile<T, D, 32>, int>::type own[SPLIT ? 1 : 4];
  alignas(16) float row[SPLIT ? 4 : 2][2][QT];   // -lse log2 e, -delta
  int odd;                                // gradients that were taken out of tiles
  __device__ KeysLds() {}
};

// Values 32 D0 .. of a head's: a head of 256 is taken in two halves, whose sums would
// not fit the registers together.
template <typename T, int D, int D0, int DN, Way WAY>
__device__ __forceinline__ void keys_grad(const PromptArgs& a, KeysLds<T, D, DN, WAY>& lds) {
  constexpr bool SPLIT = WAY == kSplit;
  constexpr int BN = SPLIT ? 32 : 128, STEPS = D / Op<T>::STEP, BY = SPLIT ? 4 : 1;
  typedef KeysLds<T, D, DN, WAY> Lds;
  constexpr bool OWN = Lds::OWN;
  constexpr int HALVES = Lds::HALVES, QT = Lds::QT;
  typedef LdsTile<T, D, QT> Tile;
  typedef Staged<T, D, QT, SPLIT ? 64 : NT * HALVES> Stage;
  const int g = blockIdx.x % a.heads, unit = blockIdx.x / a.heads;
  Prompt p;
  int much;
  if (!find_tile(a, BN, unit, p, much)) return;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = wave >> 2;             // of a tile's rows (SPLIT and four waves: 0)
  const int k0 = ((p.n + BN - 1) / BN - much) * BN, w0 = SPLIT ? k0 : k0 + 32 * (wave & 3), key = w0 + (lane & 31);
  const uint32_t to_lane = Stage::lane(), rows_lane = Tile::rows_lane(), d_lane = Tile::d_lane();
  auto& own = lds.own[SPLIT ? 0 : wave & 3];       // who has the same keys writes the same
  typename Op<T>::frag kc[STEPS], vc[OWN ? 1 : STEPS];
  if constexpr (OWN) {
    load_column<T, D>(a.v, p.start, g, key, p.n, a.dim, kc);
    put_column<T, D>(lds_at(own) + rows_lane, kc);
  } else {
    load_column<T, D>(a.v, p.start, g, key, p.n, a.dim, vc);
  }
  load_column<T, D>(a.k, p.start, g, key, p.n, a.dim, kc);
  const float c = a.scale * kPromptLog2e;
  f32x16 dk[DN], dv[DN];
#pragma unroll
  for (int dt = 0; dt < DN; ++dt)
#pragma unroll
    for (int x = 0; x < 16; ++x) dk[dt][x] = dv[dt][x] = 0;
  Fit<T> fit_p, fit_s;

  const TileSpan span = rows_of_keys(k0, BN, p.n, a.window, QT);
  const int t0 = span.first, t1 = span.last, total = (t1 - t0 + 1) * a.share;
  Stage sq, so;
  float srow = 0;
  const int at = SPLIT ? lane : tid;      // which of a tile's rows' constants it loads
  // the tile on its way: its query head and first row
  int next_head = g * a.share, next_row = t0 * QT;
  auto onward = [&](int n) __attribute__((always_inline)) {
    next_row += n * QT;
    while (next_row > t1 * QT) next_row -= (t1 - t0 + 1) * QT, ++next_head;
  };
  // whether some key of the workgroup is not seen by all rows of a tile
  auto cut = [&](int r0) { return r0 < k0 + BN - 1 || r0 + QT - 1 - a.window >= k0; };
  auto fetch = [&]() __attribute__((always_inline)) {
    sq.load(a.q, p.start, next_head, next_row, p.n, a.dim);
    so.load(a.dout, p.start, next_head, next_row, p.n, a.dim);
    if (SPLIT || tid < 2 * QT) {
      const int row = next_row + at % QT;
      const float* from = (at < QT ? a.neg_lse : a.neg_delta) + (int64_t)next_head * a.rows + p.start;
      const float y = from[min(row, p.n - 1)];
      srow = row < p.n ? y : at < QT ? -INFINITY : 0.0f;
    }
  };
  auto put = [&](int to) __attribute__((always_inline)) {
    if (cut(next_row)) {
      rarely();
      // 0 times them would not be 0.  A row of such a query has no lse, one of such a
      // gradient no delta; what of it belongs to dv is added in the end.
      sq.clean();
      if (so.clean()) lds.odd = 1;
    }
    sq.store(hidden(lds_at(lds.tile.q[to]) + to_lane));
    so.store(hidden(lds_at(lds.tile.o[to]) + to_lane));
    if (SPLIT || tid < 2 * QT) lds.row[to][at / QT][at % QT] = srow;
  };
  if (tid == 0) lds.odd = 0;
  const int first = SPLIT ? wave : 0;
  if (SPLIT) onward(wave);
  if (first < total) fetch();
  __syncthreads();
  if (!SPLIT) put(0);
  for (int it = first; it < total; it += BY) {
    const int from = SPLIT ? wave : it & 1, r0 = next_row + 32 * half;
    if (SPLIT) own_lds(), put(from), own_lds();
    else __syncthreads();
    if (it + BY < total) {
      onward(BY);
      fetch();
    }
    const bool none = r0 + 31 < w0 || r0 - a.window >= w0 + 31;
    constexpr int HALF = 32 * D * (int)sizeof(T);   // a half tile's bytes
    if (!none) {
      f32x16 s, d;
      float w[16], u[16];
#pragma unroll
      for (int x = 0; x < 16; x += 4) {
        const f32x4 z = *reinterpret_cast<const f32x4*>(&lds.row[from][1][32 * half + block_row(x, h)]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[x + i] = 0, d[x + i] = z[i];
      }
      products<D>(true);
      s = scores<T, D>(hidden(lds_at(lds.tile.q[from]) + half * HALF + rows_lane), 0, kc, s);
      const uint32_t do_at = hidden(lds_at(lds.tile.o[from]) + half * HALF + rows_lane);
      if constexpr (OWN) d = scores<T, D>(do_at, hidden(lds_at(own) + rows_lane), d);
      else d = scores<T, D>(do_at, 0, vc, d);
      products<D>(false);
#pragma unroll
      for (int x = 0; x < 16; x += 4) {
        const f32x4 y = *reinterpret_cast<const f32x4*>(&lds.row[from][0][32 * half + block_row(x, h)]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[x + i] = __builtin_amdgcn_exp2f(fmaf(s[x + i], c, y[i]));
          u[x + i] = w[x + i] * d[x + i];
        }
      }
      if (r0 < w0 + 31 || r0 + 31 - a.window >= w0) {
        rarely();
        const int from_row = (int)hidden(key - r0 - 4 * h);
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const bool in = block_row(x, 0) >= from_row && block_row(x, 0) < from_row + a.window;
          const bool alone = block_row(x, 0) == from_row && (key == 0 || a.window == 1);
          w[x] = in ? w[x] : 0.0f;
          u[x] = in ? u[x] * (alone ? 0.0f : 1.0f) : 0.0f;
        }
      }
      fit_p.scale(w, dv);
      fit_s.scale(u, dk);
      const uint32_t q_at = hidden(lds_at(lds.tile.q[from]) + half * HALF + d_lane);
      const uint32_t o_at = hidden(lds_at(lds.tile.o[from]) + half * HALF + d_lane);
      products<D>(true);
      contract<T, D, D0, DN, 1>(o_at, 0, w, dv);
      contract<T, D, D0, DN, 1>(q_at, 0, u, dk);
      products<D>(false);
    }
    if (!SPLIT && it + 1 < total) put(from ^ 1);
  }
  __syncthreads();
  if (lds.odd) {
    rarely();
    for (int hs = 0; hs < a.share; ++hs)
      for (int t = t0; t <= t1; ++t)
        if (cut(t * QT))
          add_odd<T, DN>(a.dout, p.start, g * a.share + hs, t * QT, min(t * QT + QT, p.n), a.dim, 32 * D0, dv,
                         [&](int i) { return key <= i && key > i - a.window; });
  }
  if constexpr (SPLIT) {
#pragma unroll
    for (int both = 0; both < 2; ++both) {
      put_part(lds.join, both ? dv : dk, both ? fit_p.back() : fit_s.back());
      __syncthreads();
#pragma unroll
      for (int dt = 0; dt < DN; dt += 4)
        if (dt + wave < DN && key < p.n) {
          const f32x16 y[1] = {joined(lds.join, dt + wave)};
          store_column<T, 1>(both ? a.dv : a.dk, p.start, g, key, a.dim, 32 * (D0 + dt + wave), y, both ? 1.0f : a.scale);
        }
      __syncthreads();
    }
  } else if constexpr (HALVES == 2) {
#pragma unroll
    for (int both = 0; both < 2; ++both) {
      f32x16 (&acc)[DN] = both ? dv : dk;
      const float by = both ? fit_p.back() : fit_s.back();
      if (half) put_part(lds.join, acc, by);
      __syncthreads();
      if (!half) {
#pragma unroll
        for (int dt = 0; dt < DN; ++dt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 y = lds.join.b[wave][dt][i][lane];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[dt][4 * i + j] = acc[dt][4 * i + j] * by + y[j];
          }
        if (key < p.n) store_column<T, DN>(both ? a.dv : a.dk, p.start, g, key, a.dim, 32 * D0, acc, both ? 1.0f : a.scale);
      }
      __syncthreads();
    }
  } else if (key < p.n) {
    store_column<T, DN>(a.dk, p.start, g, key, a.dim, 32 * D0, dk, a.scale * fit_s.back());
    store_column<T, DN>(a.dv, p.start, g, key, a.dim, 32 * D0, dv, fit_p.back());
  }
}

template <typename T, int D, Way WAY>
__global__ __launch_bounds__((WAY == kEight ? 2 * NT : NT), (WAY != kSplit && sizeof(T) == 2 && D <= 128) ? 2 : 1)
void prompt_keys_grad(PromptArgs a) {
  if constexpr (D == 256) {
    __shared__ KeysLds<T, D, 4, WAY> lds;
    if (blockIdx.y == 0) keys_grad<T, D, 0, 4, WAY>(a, lds);
    else keys_grad<T, D, 4, 4, WAY>(a, lds);
  } else {
    __shared__ KeysLds<T, D, D / 32, WAY> lds;
    keys_grad<T, D, 0, D / 32, WAY>(a, lds);
  }
}

template <typename T, int D, bool SPLIT>
kronq_status launch_rows(const PromptArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)a.rows / (SPLIT ? 32 : 128) + a.seqs;
  hipLaunchKernelGGL((prompt_rows_grad<T, D, SPLIT>), dim3((unsigned)(units * a.heads * a.share)), dim3(NT), 0, s, a);
  KQ_LAUNCHED("prompt_rows_grad");
  return KRONQ_OK;
}

template <typename T, int D, Way WAY>
kronq_status launch_keys(const PromptArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)a.rows / (WAY == kSplit ? 32 : 128) + a.seqs;
  hipLaunchKernelGGL((prompt_keys_grad<T, D, WAY>), dim3((unsigned)(units * a.heads), D == 256 ? 2 : 1),
                     dim3(WAY == kEight ? 2 * NT : NT), 0, s, a);
  KQ_LAUNCHED("prompt_keys_grad");
  return KRONQ_OK;
}

// SPLIT up to that many workgroups of 128 rows (keys).  Both kernels' time, us, with the
// one's work split and whole: rows, bf16, dim 128, 128 workgroups 86 and 99, 192 125 and
// 123, 288 58 and 42; dim 256, 64 285 and 357, 256 1317 and 846; dim 64, 192
// 60 and 71 or (shorter sequences) 42 and 41, 288 33 and 27; fp32, dim 64, 192 109 and
// 116, 288 76 and 70; dim 128, 96 271 and 473.  Keys, split and the way that follows,
// bf16, dim 128, 96 169 and 260, 160 357 and 427, 192 229 and 226, 256 325 and 295; dim 64,
// 256 174 and 197, 384 295 and 294, 760 825 and 784; dim 256, 116 826 and 851; fp32, dim
// 128, 344 2254 and 2382, 700 8716 and 7999.
template <typename T, int D>
constexpr int64_t kRowsSplitUpTo = D == 256 ? 64 : sizeof(T) == 4 || D == 64 ? 192 : 128;
template <typename T, int D>
constexpr int64_t kKeysSplitUpTo = sizeof(T) == 2 && D == 128 ? 192 : 384;
// Eight waves up to that many (fp32 and heads of 256 have no room for them).  Both kernels'
// time, us, eight and four: dim 128, 672 workgroups 583 and 719 and (longer sequences) 1374
// and 1534, 1340 1598 and 1530; dim 64, 680 470 and 506, 1360 923 and 830.
constexpr int64_t kEightUpTo = 1024;

template <typename T, int D>
kronq_status launch_dim(const PromptArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)a.rows / 128 + a.seqs;
  kronq_status st;
  // fp32 heads of 256 have no room for four waves' tiles
  if constexpr (!(sizeof(T) == 4 && D == 256)) {
    st = units * a.heads * a.share <= kRowsSplitUpTo<T, D> ? launch_rows<T, D, true>(a, s) : launch_rows<T, D, false>(a, s);
    if (st) return st;
    if (units * a.heads <= kKeysSplitUpTo<T, D>) return launch_keys<T, D, kSplit>(a, s);
    if constexpr (sizeof(T) == 2 && D <= 128)
      if (units * a.heads <= kEightUpTo) return launch_keys<T, D, kEight>(a, s);
    return launch_keys<T, D, kFour>(a, s);
  } else {
    st = launch_rows<T, D, false>(a, s);
    return st ? st : launch_keys<T, D, kFour>(a, s);
  }
}

template <typename T>
kronq_status launch(const PromptArgs& a, hipStream_t s) {
  if (a.dim <= 64) return launch_dim<T, 64>(a, s);
  if (a.dim <= 128) return launch_dim<T, 128>(a, s);
  return launch_dim<T, 256>(a, s);
}

}  // namespace

size_t prompt_grad_ws_bytes(int64_t rows, int q_heads) { return (size_t)rows * (size_t)q_heads * 2 * sizeof(float); }

kronq_status prompt_grad_launch(const PromptArgs& a, int32_t dtype, hipStream_t s) {
  if (dtype == KRONQ_F32) return launch<float>(a, s);
  if (dtype == KRONQ_BF16) return launch<bf16_t>(a, s);
  return launch<_Float16>(a, s);
}

}  // namespace kronq
