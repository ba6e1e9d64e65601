// Causal attention over whole prompts, packed one behind the other, with grouped
// heads and a window:  out_i = sum_j w_ij v_j / sum_j w_ij,
// w_ij = exp(scale q_i . k_j - m_i) for the rows j that row i sees, in one pass with the
// running maximum and sum of a softmax.
//
// A workgroup takes 128 rows of one query head, four waves of 32, and goes through
// the keys in tiles that all waves share; a tile goes to LDS (two buffers) while the
// one before is multiplied:
//   S^T = K Q^T (a lane's column is its query), O^T = V^T P^T.
#include <utility>

#include "prompt.h"

namespace kronq {
namespace {

constexpr int NT = 256, BM = 128;

template <typename T, int D>
struct Shape {
  static constexpr int KT = sizeof(T) == 2 && D <= 128 ? 64 : 32;
  static constexpr int PER_SIMD = D == 64 && sizeof(T) == 2 ? 4 : D <= 128 ? 2 : 1;
};

// The maximum is raised when a tile's exceeds it by 2^kLazy: weights stay below that.
constexpr float kLazy = 8;

template <typename T, int D>
struct AttentionLds {
  LdsTile<T, D, Shape<T, D>::KT> k[2], v[2];
  int odd[2];                             // the tile (its number + 1) whose values are not all finite
};

// A workgroup's work.  False, with nothing written, where a tile that some row does not
// see all of holds values that are not finite, unless CAREFUL.
template <typename T, int D, bool CAREFUL>
__device__ __forceinline__ bool attend(const PromptArgs& a, AttentionLds<T, D>& lds) {
  constexpr int KT = Shape<T, D>::KT, SUB = KT / 32, DT = D / 32;
  typedef LdsTile<T, D, KT> Tile;
  // key heads are the fastest index: an XCD's workgroups read few heads
  const int g = blockIdx.x % a.heads, hs = blockIdx.x / a.heads % a.share, unit = blockIdx.x / (a.heads * a.share);
  const int head = g * a.share + hs;
  Prompt p;
  int tile;
  if (!find_tile(a, BM, unit, p, tile)) return true;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = tile * BM, w0 = r0 + 32 * wave, row = w0 + (lane & 31);

  typename Op<T>::frag q[D / Op<T>::STEP];
  load_column<T, D>(a.q, p.start, head, row, p.n, a.dim, q);
  const float c = a.scale * kPromptLog2e;
  f32x16 o[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int x = 0; x < 16; ++x) o[dt][x] = 0;
  float m = -FLT_MAX, l = 0;              // of c S; this lane's share of the sum

  const int t0 = a.window && r0 >= a.window ? (r0 - a.window + 1) / KT : 0, t1 = min(r0 + BM - 1, p.n - 1) / KT;
  if (tid < 2) lds.odd[tid] = 0;
  Staged<T, D, KT, NT> sk, sv;
  // whether some row of the workgroup does not see all of tile t
  auto cut = [&](int t) {
    return t * KT + KT - 1 > r0 || (a.window && t * KT <= r0 + BM - 1 - a.window);
  };
  auto fetch = [&](int t) __attribute__((always_inline)) {
    sk.load(a.k, p.start, g, t * KT, p.n, a.dim);
    sv.load(a.v, p.start, g, t * KT, p.n, a.dim);
  };
  const uint32_t to_lane = Staged<T, D, KT, NT>::lane(), rows_lane = Tile::rows_lane(), d_lane = Tile::d_lane();
  auto put = [&](int t, int to) __attribute__((always_inline)) {
    sk.store(hidden(lds_at(lds.k[to]) + to_lane));
    sv.store(hidden(lds_at(lds.v[to]) + to_lane));
    if (cut(t)) {
      rarely();
      if (sv.odd()) lds.odd[to] = t + 1;
    }
  };
  fetch(t0);
  __syncthreads();
  put(t0, t0 & 1);
  for (int t = t0; t <= t1; ++t) {
    const int from = t & 1;
    __syncthreads();
    if (!CAREFUL && cut(t) && lds.odd[from] == t + 1) return false;
    if (t < t1) fetch(t + 1);
    const int k0 = t * KT;
    const bool none = k0 > w0 + 31 || (a.window && k0 + KT - 1 <= w0 - a.window);
    if (!none) {
      const bool part = k0 + KT - 1 > w0 || (a.window && k0 <= w0 + 31 - a.window);
      const uint32_t k_at = hidden(lds_at(lds.k[from]) + rows_lane), v_at = hidden(lds_at(lds.v[from]) + d_lane);
      f32x16 s[SUB];
#pragma unroll
      for (int b = 0; b < SUB; ++b) {
#pragma unroll
        for (int x = 0; x < 16; ++x) s[b][x] = 0;
        s[b] = scores<T, D>(k_at, 32 * b, q, s[b]);
      }
      auto seen = [&](int b, int r) {     // row r of block b
        const int j = k0 + 32 * b + r;
        return j <= row && (!a.window || j > row - a.window);
      };
      if (part) {
        rarely();
#pragma unroll
        for (int b = 0; b < SUB; ++b)
#pragma unroll
          for (int x = 0; x < 16; ++x) s[b][x] = seen(b, block_row(x, h)) ? s[b][x] : -INFINITY;
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
        if (CAREFUL && part) contract_seen<T, D, 0, DT, false>(v_at, 32 * b, w, o, [&](int r) { return seen(b, r); });
        else contract<T, D, 0, DT>(v_at, 32 * b, w, o);
      }
    }
    if (t < t1) put(t + 1, from ^ 1);
  }
  l = both_sum(l);
  if (row < p.n) {
    store_column<T, DT>(a.out, p.start, head, row, a.dim, 0, o, l == 0 ? 0.0f : 1 / l);
    if (a.lse && h == 0)
      a.lse[(int64_t)(p.start + row) * (a.heads * a.share) + head] = l == 0 ? -INFINITY : (m + __log2f(l)) * kPromptLn2;
  }
  return true;
}

// Called rather than a part of the kernel, so that it costs the usual way no registers.
template <typename T, int D>
__device__ __attribute__((noinline)) void attend_carefully(PromptArgs a, AttentionLds<T, D>* lds) {
  __syncthreads();
  attend<T, D, true>(a, *lds);
}

template <typename T, int D>
__global__ __launch_bounds__(NT, (Shape<T, D>::PER_SIMD)) void prompt_attention(PromptArgs a) {
  __shared__ AttentionLds<T, D> lds;
  if (!attend<T, D, false>(a, lds)) attend_carefully<T, D>(a, &lds);
}

template <typename T>
kronq_status launch(const PromptArgs& a, hipStream_t s) {
  const int64_t grid = ((int64_t)a.rows / BM + a.seqs) * a.heads * a.share;
  const dim3 blocks((unsigned)grid);
  if (a.dim <= 64) hipLaunchKernelGGL((prompt_attention<T, 64>), blocks, dim3(NT), 0, s, a);
  else if (a.dim <= 128) hipLaunchKernelGGL((prompt_attention<T, 128>), blocks, dim3(NT), 0, s, a);
  else hipLaunchKernelGGL((prompt_attention<T, 256>), blocks, dim3(NT), 0, s, a);
  KQ_LAUNCHED("prompt_attention");
  return KRONQ_OK;
}

}  // namespace

kronq_status prompt_attention_launch(const PromptArgs& a, int32_t dtype, hipStream_t s) {
  if (dtype == KRONQ_F32) return launch<float>(a, s);
  if (dtype == KRONQ_BF16) return launch<bf16_t>(a, s);
  return launch<_Float16>(a, s);
}

}  // namespace kronq
