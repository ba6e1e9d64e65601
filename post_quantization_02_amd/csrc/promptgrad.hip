// Gradients of attention over whole packed prompts.  With S = scale Q K^T over what
// rows see, P = exp(S - lse), delta_i = sum_j P_ij dP_ij:
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q
//
// Two kernels, so that no sum needs atomics or a second pass: one takes 128 rows of a
// query head and goes through their keys (dQ), one takes 128 keys of a key head and
// goes through the rows of all its query heads (dK, dV stay in registers).  Both
// compute S and dP.
//
// delta is dO . O, but O has been rounded to its type, and where one key has most of
// a row's weight dP - delta is small beside that rounding.  The rows of dS sum to 0,
// so with a delta that is off the sum is what it is off by, r_i: the first kernel
// sums it beside B = P K, takes r B off dQ and hands the right delta to the second.
// (Not for fp32, whose outputs hold it well enough.)
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

// ---------------------------------------------------------------- queries

template <typename T, int D>
struct RowsLds {
  static constexpr bool FIX = sizeof(T) == 2;      // delta is put right; dO is held here
  LdsTile<T, D, 32> k[2], v[2];
  typename std::conditional<FIX, LdsTile<T, D, 32>, int>::type own[4];
  int odd[2];
};

// A workgroup's work.  False, with nothing written, where a tile that some row does not
// see all of holds keys that are not finite, unless CAREFUL.
template <typename T, int D, bool CAREFUL>
__device__ __forceinline__ bool rows_grad(const PromptArgs& a, RowsLds<T, D>& lds) {
  constexpr int BM = 128, KT = 32, DT = D / 32, STEPS = D / Op<T>::STEP;
  constexpr bool FIX = RowsLds<T, D>::FIX;
  typedef LdsTile<T, D, KT> Tile;
  const int g = blockIdx.x % a.heads, hs = blockIdx.x / a.heads % a.share, unit = blockIdx.x / (a.heads * a.share);
  const int head = g * a.share + hs;
  Prompt p;
  int tile;
  if (!find_tile(a, BM, unit, p, tile)) return true;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r0 = tile * BM, w0 = r0 + 32 * wave, row = w0 + (lane & 31);
  const uint32_t to_lane = Staged<T, D, KT, NT>::lane(), rows_lane = Tile::rows_lane(), d_lane = Tile::d_lane();

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
      put_column<T, D>(lds_at(lds.own[wave]) + rows_lane, f);
    } else {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) oc[s] = f[s];
    }
  }
  load_column<T, D>(a.q, p.start, head, row, p.n, a.dim, qc);
  const float c = a.scale * kPromptLog2e;
  f32x16 dq[DT], pk[FIX ? DT : 1];
  Fit<T> fit;
  float off;                              // what this lane's rows of dS sum to

  const int t0 = a.window && r0 >= a.window ? (r0 - a.window + 1) / KT : 0, t1 = min(r0 + BM - 1, p.n - 1) / KT;
  Staged<T, D, KT, NT> sk, sv;
  auto cut = [&](int t) {
    return t * KT + KT - 1 > r0 || (a.window && t * KT <= r0 + BM - 1 - a.window);
  };
  auto fetch = [&](int t) __attribute__((always_inline)) {
    sk.load(a.k, p.start, g, t * KT, p.n, a.dim);
    sv.load(a.v, p.start, g, t * KT, p.n, a.dim);
  };
  auto put = [&](int t, int to) __attribute__((always_inline)) {
    sk.store(hidden(lds_at(lds.k[to]) + to_lane));
    sv.store(hidden(lds_at(lds.v[to]) + to_lane));
    if (cut(t)) {
      rarely();
      if (sk.odd()) lds.odd[to] = t + 1;
    }
  };
  {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int x = 0; x < 16; ++x) dq[dt][x] = pk[FIX ? dt : 0][x] = 0;
    fit = Fit<T>();
    off = 0;
    if (tid < 2) lds.odd[tid] = 0;
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
        auto seen = [&](int r) {
          const int j = k0 + r;
          return j <= row && (!a.window || j > row - a.window);
        };
        f32x16 s, d;
#pragma unroll
        for (int x = 0; x < 16; ++x) s[x] = 0, d[x] = neg_delta;
        const uint32_t k_at = hidden(lds_at(lds.k[from]) + rows_lane), v_at = hidden(lds_at(lds.v[from]) + rows_lane);
        s = scores<T, D>(k_at, 0, qc, s);
        if constexpr (FIX) d = scores<T, D>(v_at, hidden(lds_at(lds.own[wave]) + rows_lane), d);
        else d = scores<T, D>(v_at, 0, oc, d);
        float w[16], u[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          w[x] = __builtin_amdgcn_exp2f(fmaf(s[x], c, neg_lse));
          u[x] = w[x] * d[x];
        }
        if (part) {
        rarely();
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const bool in = seen(block_row(x, h));
            w[x] = in ? w[x] : 0.0f;
            u[x] = in ? u[x] : 0.0f;
          }
        }
        if constexpr (FIX) {
#pragma unroll
          for (int x = 0; x < 16; ++x) off += u[x];
        }
        fit.scale(u, dq);
        const uint32_t kd_at = hidden(lds_at(lds.k[from]) + d_lane);
        bool done = false;
        if constexpr (CAREFUL) {
          if (part) {
            contract_seen<T, D, 0, DT, true>(kd_at, 0, u, dq, seen);
            if constexpr (FIX) contract_seen<T, D, 0, DT, true>(kd_at, 0, w, pk, seen);
            done = true;
          }
        }
        if (!done) {
          if constexpr (FIX) contract_two<T, D>(kd_at, u, dq, w, pk);
          else contract<T, D, 0, DT>(kd_at, 0, u, dq);
        }
      }
      if (t < t1) put(t + 1, from ^ 1);
    }
  }
  if constexpr (FIX) {
    off = both_sum(off);
    neg_delta -= off;
    const float by = off / fit.back();
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int x = 0; x < 16; ++x) dq[dt][x] -= by * pk[dt][x];
  }
  if (row < p.n) {
    store_column<T, DT>(a.dq, p.start, head, row, a.dim, 0, dq, a.scale * fit.back());
    if (h == 0) {
      const int64_t at = (int64_t)head * a.rows + p.start + row;
      a.neg_lse[at] = neg_lse;
      a.neg_delta[at] = neg_delta;
    }
  }
  return true;
}

// Called rather than a part of the kernel, so that it costs the usual way no registers.
template <typename T, int D>
__device__ __attribute__((noinline)) void rows_grad_carefully(PromptArgs a, RowsLds<T, D>* lds) {
  __syncthreads();
  rows_grad<T, D, true>(a, *lds);
}

template <typename T, int D>
__global__ __launch_bounds__(NT, D == 256 || (D == 128 && sizeof(T) == 4) ? 1 : 2) void prompt_rows_grad(PromptArgs a) {
  __shared__ RowsLds<T, D> lds;
  if (!rows_grad<T, D, false>(a, lds)) rows_grad_carefully<T, D>(a, &lds);
}

// ---------------------------------------------------------------- keys and values

constexpr int QT = 32;

template <typename T, int D>
struct KeysLds {
  static constexpr bool OWN = sizeof(T) == 2 && D == 128;   // values are held here: no registers left
  LdsTile<T, D, QT> q[2], o[2];
  typename std::conditional<OWN, LdsTile<T, D, 32>, int>::type own[4];
  alignas(16) float row[2][2][QT];        // -lse log2 e, -delta
  int odd[2];
};

// Values 32 D0 .. of a head's: a head of 256 is taken in two halves, whose sums would
// not fit the registers together.
template <typename T, int D, int D0, int DN, bool CAREFUL>
__device__ __forceinline__ bool keys_grad(const PromptArgs& a, KeysLds<T, D>& lds) {
  const int g = blockIdx.x % a.heads, unit = blockIdx.x / a.heads;
  constexpr int BN = 128, STEPS = D / Op<T>::STEP;
  constexpr bool OWN = KeysLds<T, D>::OWN;
  typedef LdsTile<T, D, QT> Tile;
  Prompt p;
  int tile;
  if (!find_tile(a, BN, unit, p, tile)) return true;
  tile = (p.n + BN - 1) / BN - 1 - tile;           // early keys are seen most: they come first
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int k0 = tile * BN, w0 = k0 + 32 * wave, key = w0 + (lane & 31);
  const uint32_t to_lane = Staged<T, D, QT, NT>::lane(), rows_lane = Tile::rows_lane(), d_lane = Tile::d_lane();
  typename Op<T>::frag kc[STEPS], vc[OWN ? 1 : STEPS];
  if constexpr (OWN) {
    load_column<T, D>(a.v, p.start, g, key, p.n, a.dim, kc);
    put_column<T, D>(lds_at(lds.own[wave]) + rows_lane, kc);
  } else {
    load_column<T, D>(a.v, p.start, g, key, p.n, a.dim, vc);
  }
  load_column<T, D>(a.k, p.start, g, key, p.n, a.dim, kc);
  const float c = a.scale * kPromptLog2e;
  f32x16 dk[DN], dv[DN];
  Fit<T> fit_p, fit_s;

  const int t0 = k0 / QT, last = a.window && k0 + BN - 1 < p.n - a.window ? k0 + BN - 1 + a.window : p.n - 1;
  const int tiles = last / QT - t0 + 1, total = tiles * a.share;
  Staged<T, D, QT, NT> sq, so;
  float srow = 0;
  int next_head, next_row;                // the tile on its way: its query head and first row
  // whether some key of the workgroup is not seen by all rows of a tile
  auto cut = [&](int r0) { return r0 < k0 + BN - 1 || (a.window && r0 + QT - 1 - a.window >= k0); };
  auto fetch = [&]() __attribute__((always_inline)) {
    sq.load(a.q, p.start, next_head, next_row, p.n, a.dim);
    so.load(a.dout, p.start, next_head, next_row, p.n, a.dim);
    if (tid < 64) {
      const int row = next_row + (tid & 31);
      const float* from = (tid < 32 ? a.neg_lse : a.neg_delta) + (int64_t)next_head * a.rows + p.start;
      const float y = from[min(row, p.n - 1)];
      srow = row < p.n ? y : tid < 32 ? -INFINITY : 0.0f;
    }
  };
  auto put = [&](int it, int to) __attribute__((always_inline)) {
    sq.store(hidden(lds_at(lds.q[to]) + to_lane));
    so.store(hidden(lds_at(lds.o[to]) + to_lane));
    if (tid < 64) lds.row[to][tid >> 5][tid & 31] = srow;
    if (cut(next_row)) {
      rarely();
      if (sq.odd() || so.odd()) lds.odd[to] = it + 1;
    }
  };
  {
#pragma unroll
    for (int dt = 0; dt < DN; ++dt)
#pragma unroll
      for (int x = 0; x < 16; ++x) dk[dt][x] = dv[dt][x] = 0;
    fit_p = fit_s = Fit<T>();
    next_head = g * a.share;
    next_row = t0 * QT;
    if (tid < 2) lds.odd[tid] = 0;
    fetch();
    __syncthreads();
    put(0, 0);
    for (int it = 0; it < total; ++it) {
      const int from = it & 1, r0 = next_row;
      __syncthreads();
      if (!CAREFUL && cut(r0) && lds.odd[from] == it + 1) return false;
      if (it + 1 < total) {
        next_row += QT;
        if (next_row > last) next_row = t0 * QT, ++next_head;
        fetch();
      }
      const bool none = r0 + QT - 1 < w0 || (a.window && r0 - a.window >= w0 + 31);
      if (!none) {
        const bool part = r0 < w0 + 31 || (a.window && r0 + QT - 1 - a.window >= w0);
        auto seen = [&](int r) {
          const int i = r0 + r;
          return key <= i && (!a.window || key > i - a.window);
        };
        f32x16 s, d;
        float w[16], u[16];
#pragma unroll
        for (int x = 0; x < 16; x += 4) {
          const f32x4 z = *reinterpret_cast<const f32x4*>(&lds.row[from][1][block_row(x, h)]);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[x + i] = 0, d[x + i] = z[i];
        }
        s = scores<T, D>(hidden(lds_at(lds.q[from]) + rows_lane), 0, kc, s);
        const uint32_t do_at = hidden(lds_at(lds.o[from]) + rows_lane);
        if constexpr (OWN) d = scores<T, D>(do_at, hidden(lds_at(lds.own[wave]) + rows_lane), d);
        else d = scores<T, D>(do_at, 0, vc, d);
#pragma unroll
        for (int x = 0; x < 16; x += 4) {
          const f32x4 y = *reinterpret_cast<const f32x4*>(&lds.row[from][0][block_row(x, h)]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            w[x + i] = __builtin_amdgcn_exp2f(fmaf(s[x + i], c, y[i]));
            u[x + i] = w[x + i] * d[x + i];
          }
        }
        if (part) {
        rarely();
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const bool in = seen(block_row(x, h));
            w[x] = in ? w[x] : 0.0f;
            u[x] = in ? u[x] : 0.0f;
          }
        }
        fit_p.scale(w, dv);
        fit_s.scale(u, dk);
        const uint32_t q_at = hidden(lds_at(lds.q[from]) + d_lane), o_at = hidden(lds_at(lds.o[from]) + d_lane);
        bool done = false;
        if constexpr (CAREFUL) {
          if (part) {
            contract_seen<T, D, D0, DN, false>(o_at, 0, w, dv, seen);
            contract_seen<T, D, D0, DN, true>(q_at, 0, u, dk, seen);
            done = true;
          }
        }
        if (!done) {
          contract<T, D, D0, DN>(o_at, 0, w, dv);
          contract<T, D, D0, DN>(q_at, 0, u, dk);
        }
      }
      if (it + 1 < total) put(it + 1, from ^ 1);
    }
  }
  if (key < p.n) {
    store_column<T, DN>(a.dk, p.start, g, key, a.dim, 32 * D0, dk, a.scale * fit_s.back());
    store_column<T, DN>(a.dv, p.start, g, key, a.dim, 32 * D0, dv, fit_p.back());
  }
  return true;
}

template <typename T, int D, bool CAREFUL>
__device__ __forceinline__ bool keys_grad_of(const PromptArgs& a, KeysLds<T, D>& lds) {
  if constexpr (D == 256) {
    return blockIdx.y == 0 ? keys_grad<T, D, 0, 4, CAREFUL>(a, lds) : keys_grad<T, D, 4, 4, CAREFUL>(a, lds);
  } else {
    return keys_grad<T, D, 0, D / 32, CAREFUL>(a, lds);
  }
}

template <typename T, int D>
__device__ __attribute__((noinline)) void keys_grad_carefully(PromptArgs a, KeysLds<T, D>* lds) {
  __syncthreads();
  keys_grad_of<T, D, true>(a, *lds);
}

template <typename T, int D>
__global__ __launch_bounds__(NT, (sizeof(T) == 2 && D <= 128) ? 2 : 1) void prompt_keys_grad(PromptArgs a) {
  __shared__ KeysLds<T, D> lds;
  if (!keys_grad_of<T, D, false>(a, lds)) keys_grad_carefully<T, D>(a, &lds);
}

template <typename T, int D>
kronq_status launch_dim(const PromptArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)a.rows / 128 + a.seqs;
  hipLaunchKernelGGL((prompt_rows_grad<T, D>), dim3((unsigned)(units * a.heads * a.share)), dim3(NT), 0, s, a);
  KQ_LAUNCHED("prompt_rows_grad");
  hipLaunchKernelGGL((prompt_keys_grad<T, D>), dim3((unsigned)(units * a.heads), D == 256 ? 2 : 1), dim3(NT), 0, s, a);
  KQ_LAUNCHED("prompt_keys_grad");
  return KRONQ_OK;
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
