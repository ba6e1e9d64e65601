// Gradients of attention over whole packed prompts.  With S = scale Q K^T over what
// rows see, P = exp(S - lse), delta_i = dO_i . O_i:
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q
//
// Two kernels, so that no sum needs atomics or a second pass: one takes 128 keys of
// a key head and goes through the rows of all its query heads (dK, dV stay in
// registers), one takes 128 rows of a query head and goes through its keys (dQ).
// Both compute S and dP: seven products instead of five.  Products start from
// -lse / scale and -delta, so that what comes out is S - lse and dP - delta.
#include <utility>

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

// ---------------------------------------------------------------- rows' constants

// Sixteen lanes a row of a head.
template <typename T>
__global__ __launch_bounds__(NT) void prompt_delta(PromptArgs a) {
  const int lane = threadIdx.x & 15, row = blockIdx.x * 16 + (threadIdx.x >> 4), head = blockIdx.y;
  float sum = 0;
  if (row < a.rows) {
    const T* o = static_cast<const T*>(a.out.data) + row * a.out.row + head * a.out.head;
    const T* g = static_cast<const T*>(a.dout.data) + row * a.dout.row + head * a.dout.head;
    for (int d = 8 * lane; d < a.dim; d += 128) {
      float x[8], y[8];
      load8(o + d, x);
      load8(g + d, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(x[i], y[i], sum);
    }
  }
#pragma unroll
  for (int o = 8; o; o >>= 1) sum += __shfl_xor(sum, o);
  if (row < a.rows && lane == 0) {
    const int q_heads = a.heads * a.share;
    const float lse = a.lse[(int64_t)row * q_heads + head];
    const int64_t at = (int64_t)head * a.rows + row;
    a.neg_lse[at] = lse == -INFINITY ? -INFINITY : -lse / a.scale;   // a row of no weight
    a.neg_delta[at] = -sum;
  }
}

// ---------------------------------------------------------------- keys and values

// Values 32 D0 .. of a head's: a head of 256 is taken in two halves, whose sums would
// not fit the registers together.
constexpr int QT = 32;

template <typename T, int D>
struct KeysLds {
  LdsTile<T, D, QT> q[2], o[2];
  alignas(16) float row[2][2][QT];        // -lse / scale, -delta
  int odd[2][2];
};

template <typename T, int D, int D0, int DN>
__device__ __forceinline__ void keys_grad(const PromptArgs& a, int g, int unit, KeysLds<T, D>& lds) {
  constexpr int BN = 128;
  typedef LdsTile<T, D, QT> Tile;
  auto& lq = lds.q;
  auto& lo = lds.o;
  auto& lrow = lds.row;
  auto& odd = lds.odd;
  Prompt p;
  int tile;
  if (!find_tile(a, BN, unit, p, tile)) return;
  tile = (p.n + BN - 1) / BN - 1 - tile;           // early keys are seen most: they come first
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int k0 = tile * BN, w0 = k0 + 32 * wave, key = w0 + (lane & 31);
  typename Op<T>::frag kc[D / Op<T>::STEP], vc[D / Op<T>::STEP];
  load_column<T, D>(a.k, p.start, g, key, p.n, a.dim, kc);
  load_column<T, D>(a.v, p.start, g, key, p.n, a.dim, vc);
  const float c = a.scale * kPromptLog2e;
  f32x16 dk[DN], dv[DN];
#pragma unroll
  for (int dt = 0; dt < DN; ++dt)
#pragma unroll
    for (int x = 0; x < 16; ++x) dk[dt][x] = dv[dt][x] = 0;
  Fit<T> fit_p, fit_s;

  const int t0 = k0 / QT, last = a.window && k0 + BN - 1 < p.n - a.window ? k0 + BN - 1 + a.window : p.n - 1;
  const int tiles = last / QT - t0 + 1, total = tiles * a.share;
  Staged<T, D, QT, NT> sq, so;
  float srow = 0;
  auto first_row = [&](int it) { return (t0 + it % tiles) * QT; };
  auto fetch = [&](int it) __attribute__((always_inline)) {
    const int head = g * a.share + it / tiles, r0 = first_row(it);
    sq.load(a.q, p.start, head, r0, p.n, a.dim);
    so.load(a.dout, p.start, head, r0, p.n, a.dim);
    if (tid < 64) {
      const int row = r0 + (tid & 31);
      const float* from = (tid < 32 ? a.neg_lse : a.neg_delta) + (int64_t)head * a.rows + p.start;
      const float y = from[min(row, p.n - 1)];
      srow = row < p.n ? y : tid < 32 ? -INFINITY : 0.0f;
    }
  };
  const uint32_t to_lane = Staged<T, D, QT, NT>::lane(), rows_lane = Tile::rows_lane(), d_lane = Tile::d_lane();
  auto put = [&](int it, int to) __attribute__((always_inline)) {
    sq.store(hidden(lds_at(lq[to]) + to_lane));
    so.store(hidden(lds_at(lo[to]) + to_lane));
    if (tid < 64) lrow[to][tid >> 5][tid & 31] = srow;
    const int r0 = first_row(it);
    if (r0 < k0 + BN - 1 || (a.window && r0 + QT - 1 >= k0 + a.window)) {
      if (sq.odd()) odd[to][0] = it + 1;
      if (so.odd()) odd[to][1] = it + 1;
    }
  };
  if (tid < 4) odd[tid >> 1][tid & 1] = 0;
  fetch(0);
  __syncthreads();
  put(0, 0);
  for (int it = 0; it < total; ++it) {
    const int from = it & 1;
    __syncthreads();
    if (it + 1 < total) fetch(it + 1);
    const int r0 = first_row(it);
    const bool none = r0 + QT - 1 < w0 || (a.window && r0 - a.window >= w0 + 31);
    if (!none) {
      const bool part = r0 < w0 + 31 || (a.window && r0 + QT - 1 - a.window >= w0);
      auto seen = [&](int r) {
        const int i = r0 + r;
        return key <= i && (!a.window || key > i - a.window);
      };
      f32x16 s, d;
#pragma unroll
      for (int x = 0; x < 16; x += 4) {
        const f32x4 y = *reinterpret_cast<const f32x4*>(&lrow[from][0][block_row(x, h)]);
        const f32x4 z = *reinterpret_cast<const f32x4*>(&lrow[from][1][block_row(x, h)]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[x + i] = y[i], d[x + i] = z[i];
      }
      s = scores<T, D>(hidden(lds_at(lq[from]) + rows_lane), 0, kc, s);
      d = scores<T, D>(hidden(lds_at(lo[from]) + rows_lane), 0, vc, d);
      float w[16], u[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        w[x] = __builtin_amdgcn_exp2f(s[x] * c);
        u[x] = w[x] * d[x];
      }
      if (part) {
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const bool in = seen(block_row(x, h));
          w[x] = in ? w[x] : 0.0f;
          u[x] = in ? u[x] : 0.0f;
        }
      }
      fit_p.scale(w, dv);
      fit_s.scale(u, dk);
      const uint32_t q_at = hidden(lds_at(lq[from]) + d_lane), o_at = hidden(lds_at(lo[from]) + d_lane);
      if (part && odd[from][1] == it + 1) contract_seen<T, D, D0, DN, false>(o_at, 0, w, dv, seen);
      else contract<T, D, D0, DN>(o_at, 0, w, dv);
      if (part && odd[from][0] == it + 1) contract_seen<T, D, D0, DN, true>(q_at, 0, u, dk, seen);
      else contract<T, D, D0, DN>(q_at, 0, u, dk);
    }
    if (it + 1 < total) put(it + 1, from ^ 1);
  }
  if (key < p.n) {
    store_column<T, DN>(a.dk, p.start, g, key, a.dim, 32 * D0, dk, a.scale * fit_s.back());
    store_column<T, DN>(a.dv, p.start, g, key, a.dim, 32 * D0, dv, fit_p.back());
  }
}

template <typename T, int D>
__global__ __launch_bounds__(NT, 1) void prompt_keys_grad(PromptArgs a) {
  __shared__ KeysLds<T, D> lds;
  const int g = blockIdx.x % a.heads, unit = blockIdx.x / a.heads;
  if constexpr (D == 256) {
    if (blockIdx.y == 0) keys_grad<T, D, 0, 4>(a, g, unit, lds);
    else keys_grad<T, D, 4, 4>(a, g, unit, lds);
  } else {
    keys_grad<T, D, 0, D / 32>(a, g, unit, lds);
  }
}

// ---------------------------------------------------------------- queries

template <typename T, int D>
__global__ __launch_bounds__(NT, D == 256 ? 1 : 2) void prompt_rows_grad(PromptArgs a) {
  constexpr int BM = 128, KT = 32, DT = D / 32;
  typedef LdsTile<T, D, KT> Tile;
  __shared__ Tile lk[2], lv[2];
  __shared__ int odd[2];
  const int g = blockIdx.x % a.heads, hs = blockIdx.x / a.heads % a.share, unit = blockIdx.x / (a.heads * a.share);
  const int head = g * a.share + hs;
  Prompt p;
  int tile;
  if (!find_tile(a, BM, unit, p, tile)) return;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = tile * BM, w0 = r0 + 32 * wave, row = w0 + (lane & 31);
  typename Op<T>::frag qc[D / Op<T>::STEP], oc[D / Op<T>::STEP];
  load_column<T, D>(a.q, p.start, head, row, p.n, a.dim, qc);
  load_column<T, D>(a.dout, p.start, head, row, p.n, a.dim, oc);
  const float c = a.scale * kPromptLog2e;
  const int64_t at = (int64_t)head * a.rows + p.start + min(row, p.n - 1);
  const float neg_lse = a.neg_lse[at], neg_delta = a.neg_delta[at];
  f32x16 dq[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt)
#pragma unroll
    for (int x = 0; x < 16; ++x) dq[dt][x] = 0;
  Fit<T> fit;

  const int t0 = a.window && r0 >= a.window ? (r0 - a.window + 1) / KT : 0, t1 = min(r0 + BM - 1, p.n - 1) / KT;
  if (tid < 2) odd[tid] = 0;
  Staged<T, D, KT, NT> sk, sv;
  auto cut = [&](int t) {
    return t * KT + KT - 1 > r0 || (a.window && t * KT <= r0 + BM - 1 - a.window);
  };
  auto fetch = [&](int t) __attribute__((always_inline)) {
    sk.load(a.k, p.start, g, t * KT, p.n, a.dim);
    sv.load(a.v, p.start, g, t * KT, p.n, a.dim);
  };
  const uint32_t to_lane = Staged<T, D, KT, NT>::lane(), rows_lane = Tile::rows_lane(), d_lane = Tile::d_lane();
  auto put = [&](int t, int to) __attribute__((always_inline)) {
    sk.store(hidden(lds_at(lk[to]) + to_lane));
    sv.store(hidden(lds_at(lv[to]) + to_lane));
    if (cut(t) && sk.odd()) odd[to] = t + 1;
  };
  fetch(t0);
  __syncthreads();
  put(t0, t0 & 1);
  for (int t = t0; t <= t1; ++t) {
    const int from = t & 1;
    __syncthreads();
    if (t < t1) fetch(t + 1);
    const int k0 = t * KT;
    const bool none = k0 > w0 + 31 || (a.window && k0 + KT - 1 <= w0 - a.window);
    if (!none) {
      const bool part = k0 + KT - 1 > w0 || (a.window && k0 <= w0 + 31 - a.window);
      auto seen = [&](int r) {
        const int j = k0 + r;
        return j <= row && (!a.window || j > row - a.window);
      };
      f32x16 s, d;
#pragma unroll
      for (int x = 0; x < 16; ++x) s[x] = neg_lse, d[x] = neg_delta;
      s = scores<T, D>(hidden(lds_at(lk[from]) + rows_lane), 0, qc, s);
      d = scores<T, D>(hidden(lds_at(lv[from]) + rows_lane), 0, oc, d);
      float u[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) u[x] = __builtin_amdgcn_exp2f(s[x] * c) * d[x];
      if (part) {
#pragma unroll
        for (int x = 0; x < 16; ++x) u[x] = seen(block_row(x, h)) ? u[x] : 0.0f;
      }
      fit.scale(u, dq);
      const uint32_t k_at = hidden(lds_at(lk[from]) + d_lane);
      if (part && odd[from] == t + 1) contract_seen<T, D, 0, DT, true>(k_at, 0, u, dq, seen);
      else contract<T, D, 0, DT>(k_at, 0, u, dq);
    }
    if (t < t1) put(t + 1, from ^ 1);
  }
  if (row < p.n) store_column<T, DT>(a.dq, p.start, head, row, a.dim, 0, dq, a.scale * fit.back());
}

template <typename T, int D>
kronq_status launch_dim(const PromptArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)a.rows / 128 + a.seqs;
  hipLaunchKernelGGL((prompt_keys_grad<T, D>), dim3((unsigned)(units * a.heads), D == 256 ? 2 : 1), dim3(NT), 0, s, a);
  KQ_LAUNCHED("prompt_keys_grad");
  hipLaunchKernelGGL((prompt_rows_grad<T, D>), dim3((unsigned)(units * a.heads * a.share)), dim3(NT), 0, s, a);
  KQ_LAUNCHED("prompt_rows_grad");
  return KRONQ_OK;
}

template <typename T>
kronq_status launch(const PromptArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((prompt_delta<T>), dim3((unsigned)((a.rows + 15) / 16), (unsigned)(a.heads * a.share)), dim3(NT), 0, s, a);
  KQ_LAUNCHED("prompt_delta");
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
