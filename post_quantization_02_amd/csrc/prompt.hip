// Causal attention over whole prompts, packed one behind the other, with grouped
// heads and a window:  out_i = sum_j w_ij v_j / sum_j w_ij,
// w_ij = exp(scale q_i . k_j - m_i) for the rows j that row i sees, in one pass with the
// running maximum and sum of a softmax.
//
// A workgroup takes 128 rows of one query head, four waves of 32, and goes through
// the keys in tiles that all waves share; a tile goes to LDS (two buffers) while the
// one before is multiplied:
//   S^T = K Q^T (a lane's column is its query), O^T = V^T P^T.
// Where there are too few of these for the chip (SPLIT), a workgroup takes 32 rows, and
// its waves go through every fourth tile each, by themselves; the four parts are joined
// in LDS.
//
// Long prompts are bound by the matrix cores and the vector pipes (exponentials,
// maxima), which overlap little: 24201 rows of 7 sequences, 32 heads of 128 on 8, bf16,
// 815 us, 880 TFLOP/s, the matrix cores busy 46 % of the time and the vector pipes 40.
// Scores of the next tile beside the weights of this one (twice the registers, a wave
// less a SIMD) took 1136 us against 830.  Weights are rounded to the operands' type, half
// a step of it each: in two parts, the second product would take twice as long.
// Statistics and sums are fp32.
#include "prompt.h"

namespace kronq {
namespace {

constexpr int NT = 256;

// SPLIT up to that many workgroups of 128 rows.  Split and whole, us: bf16, dim 128, 64
// workgroups (4000 rows of 2 heads) 34 and 99, 192 21 and 23, 320 36 and 37, 480 47 and 40;
// dim 64, 256 17 and 20, 480 25 and 24; dim 256, 64 40 and 55, 128 89 and 94, 420 477 and
// 183; fp32, whose products take longer than a tile's way to LDS, 544 253 and 376, 690 606
// and 629, 2800 2433 and 1860.
template <typename T, int D>
constexpr int64_t kSplitUpTo = sizeof(T) == 4 ? 704 : D == 256 ? 128 : 320;

// KT: keys of a tile.  More waves on a SIMD are worth more than longer tiles: dim 128
// in bf16 with tiles of 64 keys and two waves a SIMD 830 us, of 32 and three 808.
template <typename T, int D, bool SPLIT>
struct Shape {
  static constexpr int KT = sizeof(T) == 2 && D <= 64 && !SPLIT ? 64 : 32;
  static constexpr int PER_SIMD = D == 256 || (SPLIT && D * sizeof(T) == 512) ? 1 : SPLIT || sizeof(T) == 4 ? 2 : D == 64 ? 4 : 3;
};

// The maximum is raised when a tile's exceeds it by 2^kLazy: weights stay below that.
constexpr float kLazy = 8;

template <typename T, int D, bool SPLIT>
struct AttentionLds {
  union {
    struct { LdsTile<T, D, Shape<T, D, SPLIT>::KT> k[SPLIT ? 4 : 2], v[SPLIT ? 4 : 2]; } tile;
    typename std::conditional<SPLIT, JoinLds<D / 32>, int>::type join;
  };
  float m[4][64], l[4][64];
  int odd;                                // values that were taken out of tiles
  __device__ AttentionLds() {}
};

template <typename T, int D, bool SPLIT>
__global__ __launch_bounds__(NT, (Shape<T, D, SPLIT>::PER_SIMD)) void prompt_attention(PromptArgs a) {
  __shared__ AttentionLds<T, D, SPLIT> lds;
  constexpr int KT = Shape<T, D, SPLIT>::KT, SUB = KT / 32, DT = D / 32, BM = SPLIT ? 32 : 128;
  typedef LdsTile<T, D, KT> Tile;
  typedef Staged<T, D, KT, SPLIT ? 64 : NT> Stage;
  // key heads are the fastest index: an XCD's workgroups read few heads
  const int g = blockIdx.x % a.heads, hs = blockIdx.x / a.heads % a.share, unit = blockIdx.x / (a.heads * a.share);
  const int head = g * a.share + hs;
  Prompt p;
  int much;
  if (!find_tile(a, BM, unit, p, much)) return;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = (much - 1) * BM, w0 = SPLIT ? r0 : r0 + 32 * wave, row = w0 + (lane & 31);

  typename Op<T>::frag q[D / Op<T>::STEP];
  load_column<T, D>(a.q, p.start, head, row, p.n, a.dim, q);
  const float c = a.scale * kPromptLog2e;
  f32x16 o[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int x = 0; x < 16; ++x) o[dt][x] = 0;
  float m = -FLT_MAX, l = 0;              // of c S; this lane's share of the sum

  const TileSpan span = keys_of_rows(r0, BM, p.n, a.window, KT);
  const int t0 = span.first, t1 = span.last;
  if (tid == 0) lds.odd = 0;
  Stage sk, sv;
  // whether some row of the workgroup does not see all of tile t
  auto cut = [&](int t) {
    return t * KT + KT - 1 > r0 || t * KT <= r0 + BM - 1 - a.window;
  };
  auto fetch = [&](int t) __attribute__((always_inline)) {
    sk.load(a.k, p.start, g, t * KT, p.n, a.dim);
    sv.load(a.v, p.start, g, t * KT, p.n, a.dim);
  };
  const uint32_t to_lane = Stage::lane(), rows_lane = Tile::rows_lane(), d_lane = Tile::d_lane();
  auto put = [&](int t, int to) __attribute__((always_inline)) {
    sk.store(hidden(lds_at(lds.tile.k[to]) + to_lane));
    if (cut(t)) {
      rarely();
      if (sv.clean()) lds.odd = 1;
    }
    sv.store(hidden(lds_at(lds.tile.v[to]) + to_lane));
  };
  // the workgroup's tiles, or (SPLIT) this wave's of them
  constexpr int BY = SPLIT ? 4 : 1;
  const int first = SPLIT ? t0 + wave : t0;
  if (first <= t1) fetch(first);
  __syncthreads();
  if (!SPLIT) put(first, first & 1);
  for (int t = first; t <= t1; t += BY) {
    const int from = SPLIT ? wave : t & 1;
    if (SPLIT) own_lds(), put(t, from), own_lds();
    else __syncthreads();
    if (t + BY <= t1) fetch(t + BY);
    const int k0 = t * KT;
    const bool none = k0 > w0 + 31 || k0 + KT - 1 <= w0 - a.window;
    if (!none) {
      const bool part = k0 + KT - 1 > w0 || k0 <= w0 + 31 - a.window;
      const uint32_t k_at = hidden(lds_at(lds.tile.k[from]) + rows_lane), v_at = hidden(lds_at(lds.tile.v[from]) + d_lane);
      f32x16 s[SUB];
#pragma unroll
      for (int b = 0; b < SUB; ++b) {
#pragma unroll
        for (int x = 0; x < 16; ++x) s[b][x] = 0;
        s[b] = scores<T, D>(k_at, 32 * b, q, s[b]);
      }
      // whether a lane's row (`from` the tile's first key) sees the tile's key r
      auto seen = [&](int from, int r) { return r <= from && r > from - a.window; };
      if (part) {
        rarely();
        const int from = (int)hidden(row - k0 - 4 * h);
#pragma unroll
        for (int b = 0; b < SUB; ++b)
#pragma unroll
          for (int x = 0; x < 16; ++x) s[b][x] = seen(from, 32 * b + block_row(x, 0)) ? s[b][x] : -INFINITY;
      }
      float top = s[0][0];
#pragma unroll
      for (int b = 0; b < SUB; ++b)
#pragma unroll
        for (int x = 0; x < 16; ++x) top = fmaxf(top, s[b][x]);
      top = both_max(top) * c;
      if (__any(top > m + kLazy)) {
        rarely();
        const float up = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - up);
        m = up;
        l *= f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
          for (int x = 0; x < 16; ++x) o[dt][x] *= f;
      }
#pragma unroll
      for (int b = 0; b < SUB; ++b) {
        float w[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          w[x] = __builtin_amdgcn_exp2f(fmaf(s[b][x], c, -m));
          l += w[x];
        }
        contract<T, D, 0, DT, (sizeof(T) == 2 && D == 128 && !SPLIT ? 1 : 2)>(v_at, 32 * b, w, o);
      }
    }
    if (!SPLIT && t < t1) put(t + 1, from ^ 1);
  }
  // what was taken out of tiles, into the values 32 d0 and up of the results
  auto add_back = [&](auto& acc, int d0) __attribute__((always_inline)) {
    rarely();
    for (int t = t0; t <= t1; ++t)
      if (cut(t))
        add_odd<T>(a.v, p.start, g, t * KT, min(t * KT + KT, p.n), a.dim, 32 * d0, acc,
                   [&](int j) { return j <= row && j > row - a.window; });
  };
  __syncthreads();
  l = both_sum(l);
  if constexpr (SPLIT) {
    lds.m[wave][lane] = m;
    lds.l[wave][lane] = l;
    __syncthreads();
    float top = m, sum = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, lds.m[w][lane]);
#pragma unroll
    for (int w = 0; w < 4; ++w) sum += lds.l[w][lane] * __builtin_amdgcn_exp2f(lds.m[w][lane] - top);
    put_part(lds.join, o, __builtin_amdgcn_exp2f(m - top));
    __syncthreads();
    m = top;
    l = sum;
#pragma unroll
    for (int dt = 0; dt < DT; dt += 4)
      if (dt + wave < DT && row < p.n) {
        f32x16 y[1] = {joined(lds.join, dt + wave)};
        if (lds.odd) add_back(y, dt + wave);
        store_column<T, 1>(a.out, p.start, head, row, a.dim, 32 * (dt + wave), y, l == 0 ? 0.0f : 1 / l);
      }
  } else if (row < p.n) {
    if (lds.odd) add_back(o, 0);
    store_column<T, DT>(a.out, p.start, head, row, a.dim, 0, o, l == 0 ? 0.0f : 1 / l);
  }
  if (row < p.n && a.lse && h == 0 && (!SPLIT || wave == 0))
    a.lse[(int64_t)(p.start + row) * (a.heads * a.share) + head] = l == 0 ? -INFINITY : (m + __log2f(l)) * kPromptLn2;
}

template <typename T, int D>
kronq_status launch_dim(const PromptArgs& a, hipStream_t s) {
  const int64_t wide = ((int64_t)a.rows / 128 + a.seqs) * a.heads * a.share;
  // fp32 heads of 256 have no room for four waves' tiles
  if constexpr (!(sizeof(T) == 4 && D == 256)) {
    if (wide <= kSplitUpTo<T, D>) {
      const int64_t grid = ((int64_t)a.rows / 32 + a.seqs) * a.heads * a.share;
      hipLaunchKernelGGL((prompt_attention<T, D, true>), dim3((unsigned)grid), dim3(NT), 0, s, a);
      KQ_LAUNCHED("prompt_attention");
      return KRONQ_OK;
    }
  }
  hipLaunchKernelGGL((prompt_attention<T, D, false>), dim3((unsigned)wide), dim3(NT), 0, s, a);
  KQ_LAUNCHED("prompt_attention");
  return KRONQ_OK;
}

template <typename T>
kronq_status launch(const PromptArgs& a, hipStream_t s) {
  if (a.dim <= 64) return launch_dim<T, 64>(a, s);
  if (a.dim <= 128) return launch_dim<T, 128>(a, s);
  return launch_dim<T, 256>(a, s);
}

}  // namespace

kronq_status prompt_attention_launch(const PromptArgs& a, int32_t dtype, hipStream_t s) {
  if (dtype == KRONQ_F32) return launch<float>(a, s);
  if (dtype == KRONQ_BF16) return launch<bf16_t>(a, s);
  return launch<_Float16>(a, s);
}

}  // namespace kronq
