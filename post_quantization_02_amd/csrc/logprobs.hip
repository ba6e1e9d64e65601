// Log probabilities of given tokens with entropy and top alternatives, and their
// gradients.
//
// A row of logits l:  m = max l,  S = sum exp(l - m),  T = sum exp(l - m) (l - m)
//   lse = m + log S,  logp(v) = (l_v - m) - log S,  entropy = log S - T / S
// in one pass: a thread keeps the maximum of what it has seen, and S and T
// relative to it; a new maximum m' turns them into f S and f (T + S (m - m')) with
// f = exp(m - m').  What is minus infinity counts as probability 0 in all of them.
//   d l_v = g ([v = target] - p_v) - h p_v (logp_v + entropy)
//           + sum_k t_k ([v = id_k] - p_v),  p_v = exp(l_v - lse)
//
// Top alternatives by (value, lowest index) without sorting the row: a thread's
// largest value is known from the pass.  tau, the K-th largest of the threads' 256
// largest, is a lower bound of the row's K-th, so that only threads whose largest
// reaches tau can hold a winner: their values are read again (from the caches), those
// from tau on are listed and ranked by counting.  Where more than the list holds
// reach tau (a mask's one value all over a row, or a row in order), the K-th value
// itself is found by bisection and values equal to it are taken in their order.
#include <algorithm>
#include <cfloat>

#include "kv.h"
#include "logprobs.h"

namespace kronq {
namespace {

constexpr int NT = 256, WAVES = NT / 64;
constexpr int kList = 1024;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kFar = -1.0e4f;           // exp of this and below is 0

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7FC00000u); }

// sixteen bytes of logits
__device__ __forceinline__ void unpack(u32x4 w, float (&x)[4], float) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void unpack(u32x4 w, float (&x)[8], bf16_t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(u32x4 w, float (&x)[8], _Float16) {
  const half8_t h = __builtin_bit_cast(half8_t, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (float)h[i];
}
__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(bf16_t x) { return __uint_as_float((uint32_t)x.bits << 16); }
__device__ __forceinline__ float value(_Float16 x) { return (float)x; }
__device__ __forceinline__ void set(float& y, float x) { y = x; }
__device__ __forceinline__ void set(bf16_t& y, float x) { y.bits = to_bf16(x); }
__device__ __forceinline__ void set(_Float16& y, float x) { y = (_Float16)x; }

// A row's values: up to the first sixteen-byte border one by one, then `chunks` of
// sixteen bytes, then the rest one by one.
template <typename T>
struct Row {
  static constexpr int N = 16 / sizeof(T);
  const T* data;
  int vocab, head, chunks;

  __device__ Row(const T* p, int n) : data(p), vocab(n) {
    const int to_border = (int)(-reinterpret_cast<uintptr_t>(p) & 15) / (int)sizeof(T);
    head = min(n, to_border);
    chunks = (n - head) / N;
  }
  __device__ u32x4 chunk(int c) const { return *reinterpret_cast<const u32x4*>(data + head + (int64_t)c * N); }
  __device__ int index(int c) const { return head + c * N; }
  __device__ int rest() const { return head + chunks * N; }     // the first value behind the chunks
};

// S and T relative to m; best: the largest value, minus infinity if there is none
struct Sums { float m, s, t, best; };

__device__ __forceinline__ Sums no_sums() { return {-FLT_MAX, 0, 0, -INFINITY}; }

__device__ __forceinline__ void raise(Sums& a, float m) {
  const float d = fmaxf(a.m - m, kFar), f = exp_of(d);
  a.t = f * (a.t + a.s * d);
  a.s *= f;
  a.m = m;
}

template <int N, bool ENTROPY>
__device__ __forceinline__ void add(Sums& a, const float (&x)[N]) {
  float top = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
  a.best = fmaxf(a.best, top);
  if (top > a.m) raise(a, top);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float d = x[i] - a.m, e = exp_of(d);
    a.s += e;
    if constexpr (ENTROPY) a.t = fmaf(e, fmaxf(d, kFar), a.t);
  }
}

__device__ __forceinline__ Sums join(Sums a, Sums b) {
  const float m = fmaxf(a.m, b.m);
  raise(a, m);
  raise(b, m);
  return {m, a.s + b.s, a.t + b.t, fmaxf(a.best, b.best)};
}

// A candidate, in descending order of value, ascending order of index: zeros of
// both signs are one value.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, int index) { return (uint64_t)ordered(x) << 32 | (uint32_t)~index; }
__device__ __forceinline__ float key_value(uint64_t k) { return from_ordered((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_index(uint64_t k) { return (int)~(uint32_t)k; }

struct Part { float m, s, t, pad; };      // a segment's sums

struct Shared {
  Sums sums[WAVES];
  alignas(16) float best[NT];
  float tau[WAVES];
  uint32_t count[WAVES + 1];
  int n, chosen;
  uint16_t who[NT];
  uint64_t list[kList];
};

// f(value, index) for this thread's share of what the chosen threads (who[0 ..
// chosen)) have seen, and of the row's ends; no further once the list has overflown.
template <typename T, typename F>
__device__ __forceinline__ void visit(const Row<T>& row, int c0, int c1, bool ends_lo, bool ends_hi, const Shared& sh, F f) {
  constexpr int N = Row<T>::N;
  const int tid = threadIdx.x;
  if (ends_lo && tid < row.head) f(value(row.data[tid]), tid);
  if (ends_hi && tid < row.vocab - row.rest()) f(value(row.data[row.rest() + tid]), row.rest() + tid);
  // their chunks one behind the other, one a lane
  const int each = (c1 - c0 + NT - 1) / NT, all = sh.chosen * each;
  for (int at = tid; at < all; at += NT) {
    if (*const_cast<const volatile int*>(&sh.n) > kList) return;
    const int w = at / each, c = c0 + sh.who[w] + NT * (at - w * each);
    if (c >= c1) continue;
    float x[N];
    unpack(row.chunk(c), x, T());
#pragma unroll
    for (int i = 0; i < N; ++i) f(x[i], row.index(c) + i);
  }
}

__device__ __forceinline__ void choose(Shared& sh, bool in) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid == 0) sh.chosen = 0;
  __syncthreads();
  if (in) sh.who[atomicAdd(&sh.chosen, 1)] = (uint16_t)tid;
  __syncthreads();
}

// Sum over the workgroup, known to all.
__device__ __forceinline__ uint32_t count_all(Shared& sh, uint32_t n) {
#pragma unroll
  for (int o = 32; o; o >>= 1) n += __shfl_xor(n, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.count[threadIdx.x >> 6] = n;
  __syncthreads();
  uint32_t all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) all += sh.count[w];
  return all;
}

// The K largest of chunks c0 .. c1 of a row (and of its ends) go to sh.list[0 ..
// n), in no order; all of them are in it, and others may be.  n <= kList; at least
// K unless there are fewer values.
template <typename T>
__device__ void collect(const Row<T>& row, int c0, int c1, bool lo, bool hi, float best, int K, Shared& sh) {
  constexpr int N = Row<T>::N;
  const int tid = threadIdx.x;
  sh.best[tid] = best;
  __syncthreads();
  int reach = 0;
  for (int i = 0; i < NT; i += 4) {
    const f32x4 b = *reinterpret_cast<const f32x4*>(&sh.best[i]);
    reach += (b[0] >= best) + (b[1] >= best) + (b[2] >= best) + (b[3] >= best);
  }
  float tau = reach >= K ? best : -INFINITY;
#pragma unroll
  for (int o = 32; o; o >>= 1) tau = fmaxf(tau, __shfl_xor(tau, o));
  if ((tid & 63) == 0) sh.tau[tid >> 6] = tau;
  if (tid == 0) sh.n = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WAVES; ++w) tau = fmaxf(tau, sh.tau[w]);
  auto put = [&](float x, int index) {
    const int at = atomicAdd(&sh.n, 1);
    if (at < kList) sh.list[at] = key_of(x, index);
  };
  choose(sh, best >= tau);
  visit(row, c0, c1, lo, hi, sh, [&](float x, int i) { if (x >= tau) put(x, i); });
  __syncthreads();
  if (sh.n <= kList) return;

  // more than the list holds: the K-th largest value is tau, or above it
  choose(sh, best > tau);
  if (tid == 0) sh.n = 0;
  __syncthreads();
  auto above = [&](float bound) {
    uint32_t n = 0;
    visit(row, c0, c1, lo, hi, sh, [&](float x, int) { n += x > bound; });
    return count_all(sh, n);
  };
  if (above(tau) >= (uint32_t)K) {
    // the largest value that K values reach: at least K are above `low`, fewer above `high`
    uint32_t low = ordered(tau), high = ordered(INFINITY);
    while (high - low > 1) {
      const uint32_t mid = low + (high - low) / 2;
      if (above(from_ordered(mid)) >= (uint32_t)K) low = mid;
      else high = mid;
    }
    tau = from_ordered(high);
  }
  visit(row, c0, c1, lo, hi, sh, [&](float x, int i) { if (x > tau) put(x, i); });     // fewer than K
  __syncthreads();
  // values equal to tau, in their order, until there are K
  int have = sh.n;
  __syncthreads();
  auto in_order = [&](uint32_t hits, int index) {      // bit i: value index + i equals tau
    const int mine = __popc(hits), lane = tid & 63;
    int before = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(before, o);
      before += lane >= o ? y : 0;
    }
    if (lane == 63) sh.count[tid >> 6] = before;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      if (w < (tid >> 6)) before += sh.count[w];
      all += sh.count[w];
    }
    int at = have + before - mine;
    for (uint32_t left = hits; left && at < K; left &= left - 1) sh.list[at++] = key_of(tau, index + __ffs(left) - 1);
    have += all;
    __syncthreads();
  };
  if (lo && row.head) in_order(tid < row.head && value(row.data[tid]) == tau, tid);
  for (int c = c0; c < c1 && have < K; c += NT) {
    uint32_t hits = 0;
    if (c + tid < c1) {
      float x[N];
      unpack(row.chunk(c + tid), x, T());
#pragma unroll
      for (int i = 0; i < N; ++i) hits |= (uint32_t)(x[i] == tau) << i;
    }
    in_order(hits, row.index(c + tid));
  }
  if (hi && have < K) {
    const int at = row.rest() + tid;
    in_order(at < row.vocab && value(row.data[at]) == tau, at);
  }
  if (tid == 0) sh.n = min(have, K);
  __syncthreads();
}

// f(rank, key) for each of the list's K first.
template <typename F>
__device__ __forceinline__ void ranked(Shared& sh, int K, F f) {
  const int n = sh.n;
  for (int i = threadIdx.x; i < n; i += NT) {
    const uint64_t k = sh.list[i];
    int rank = 0;
    int j = 0;
    for (; j + 16 <= n; j += 16) {        // reads in flight together: one behind the other they would be all of the time
#pragma unroll
      for (int x = 0; x < 16; ++x) rank += sh.list[j + x] > k;
    }
    for (; j < n; ++j) rank += sh.list[j] > k;
    if (rank < K) f(rank, k);
  }
}

__device__ __forceinline__ Sums sums_of_all(Sums a, Shared& sh) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const Sums b{__shfl_xor(a.m, o), __shfl_xor(a.s, o), __shfl_xor(a.t, o), __shfl_xor(a.best, o)};
    a = join(a, b);
  }
  if ((threadIdx.x & 63) == 0) sh.sums[threadIdx.x >> 6] = a;
  __syncthreads();
  a = sh.sums[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) a = join(a, sh.sums[w]);
  return a;
}

// What a row's sums come to.
template <typename T>
__device__ __forceinline__ void finish(const LogprobsArgs& a, int64_t r, const Row<T>& row, const Sums& s, Shared& sh) {
  const float log_s = logf(s.s);
  if (threadIdx.x == 0) {
    if (a.lse) a.lse[r] = s.m + log_s;
    if (a.entropy) a.entropy[r] = s.s == 0 ? 0.0f : log_s - s.t / s.s;
    if (a.logp) {
      const int t = a.targets[r];
      float p = 0;
      if (t >= 0) p = t < a.vocab && s.s == s.s ? s.s == 0 ? -INFINITY : (value(row.data[t]) - s.m) - log_s : quiet_nan();
      a.logp[r] = p;
    }
  }
  if (a.top > 0) {
    const bool nan = s.s != s.s;
    ranked(sh, a.top, [&](int rank, uint64_t k) {
      a.top_logp[r * a.top + rank] = nan ? quiet_nan() : s.s == 0 ? -INFINITY : (key_value(k) - s.m) - log_s;
      a.top_ids[r * a.top + rank] = nan ? -1 : key_index(k);
    });
    // a row with what is not a number may have too few others
    for (int i = threadIdx.x; i < a.top; i += NT)
      if (i >= sh.n) {
        a.top_logp[r * a.top + i] = quiet_nan();
        a.top_ids[r * a.top + i] = -1;
      }
  }
}

// A workgroup takes a segment of a row, or (segs 1) a row; four pieces a thread are in
// flight.  Bound by HBM: 4095 x 32000 in fp32 with entropy and five alternatives 98 us,
// 5.3 TB/s.  Few rows are bound by the steps that follow one another: 40 x 128256 in
// bf16, 20 alternatives, 12 us and 7 of the join, where the bytes take 2.
template <typename T, bool ENTROPY>
__global__ __launch_bounds__(NT) void token_logprobs(LogprobsArgs a, int segs, Part* __restrict__ parts,
                                                     uint64_t* __restrict__ keys) {
  constexpr int N = Row<T>::N;
  __shared__ Shared sh;
  const int64_t r = blockIdx.x / (unsigned)segs;
  const int seg = (int)(blockIdx.x % (unsigned)segs), tid = threadIdx.x;
  const Row<T> row(static_cast<const T*>(a.logits) + r * a.ld, a.vocab);
  const int c0 = (int)((int64_t)row.chunks * seg / segs), c1 = (int)((int64_t)row.chunks * (seg + 1) / segs);
  const bool lo = seg == 0, hi = seg == segs - 1;
  Sums s = no_sums();
  if (lo && tid < row.head) {
    const float x[1] = {value(row.data[tid])};
    add<1, ENTROPY>(s, x);
  }
  if (hi && tid < row.vocab - row.rest()) {
    const float x[1] = {value(row.data[row.rest() + tid])};
    add<1, ENTROPY>(s, x);
  }
  constexpr int AHEAD = 4;
  int c = c0 + tid;
  for (; c + (AHEAD - 1) * NT < c1; c += AHEAD * NT) {
    u32x4 w[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) w[i] = row.chunk(c + i * NT);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      float x[N];
      unpack(w[i], x, T());
      add<N, ENTROPY>(s, x);
    }
  }
  for (; c < c1; c += NT) {
    float x[N];
    unpack(row.chunk(c), x, T());
    add<N, ENTROPY>(s, x);
  }
  if (a.top > 0) collect(row, c0, c1, lo, hi, s.best, a.top, sh);
  s = sums_of_all(s, sh);
  if (segs == 1) {
    finish(a, r, row, s, sh);
    return;
  }
  if (tid == 0) parts[blockIdx.x] = Part{s.m, s.s, s.t, 0};
  if (a.top > 0) {
    uint64_t* mine = keys + (int64_t)blockIdx.x * a.top;
    ranked(sh, a.top, [&](int rank, uint64_t k) { mine[rank] = k; });
    for (int i = tid; i < a.top; i += NT)
      if (i >= sh.n) mine[i] = 0;         // below every value's
  }
}

template <typename T>
__global__ __launch_bounds__(NT) void token_logprobs_join(LogprobsArgs a, int segs, const Part* __restrict__ parts,
                                                          const uint64_t* __restrict__ keys) {
  __shared__ Shared sh;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  const Row<T> row(static_cast<const T*>(a.logits) + r * a.ld, a.vocab);
  Sums s = no_sums();
  for (int i = 0; i < segs; ++i) {        // in their order, by every thread
    const Part p = parts[r * segs + i];
    s = join(s, Sums{p.m, p.s, p.t, -INFINITY});
  }
  if (a.top > 0) {
    if (tid == 0) sh.n = 0;
    __syncthreads();
    // a segment's last key is reached by `top` of the row's
    uint64_t least = 1;
    for (int i = 0; i < segs; ++i) least = max(least, keys[(r * segs + i) * a.top + a.top - 1]);
    for (int i = tid; i < segs * a.top; i += NT) {
      const uint64_t k = keys[r * segs * a.top + i];
      if (k >= least) sh.list[atomicAdd(&sh.n, 1)] = k;
    }
    __syncthreads();
  }
  finish(a, r, row, s, sh);
}

// Segments of a row: where rows are fewer than the chip's CUs, about one workgroup a CU,
// of at least 8192 values each; what the join takes fits its list.
int segments(int64_t rows, int64_t vocab) {
  if (rows >= 256) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>({kList / kTopMost, (256 + rows - 1) / rows, vocab / 8192}));
}

template <typename T>
kronq_status logprobs_type(const LogprobsArgs& a, void* ws, hipStream_t s) {
  const int segs = segments(a.rows, a.vocab);
  Part* parts = static_cast<Part*>(ws);
  uint64_t* keys = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + a.rows * segs * sizeof(Part));
  const dim3 grid((unsigned)(a.rows * segs));
  if (a.entropy) hipLaunchKernelGGL((token_logprobs<T, true>), grid, dim3(NT), 0, s, a, segs, parts, keys);
  else hipLaunchKernelGGL((token_logprobs<T, false>), grid, dim3(NT), 0, s, a, segs, parts, keys);
  KQ_LAUNCHED("token_logprobs");
  if (segs > 1) {
    hipLaunchKernelGGL((token_logprobs_join<T>), dim3((unsigned)a.rows), dim3(NT), 0, s, a, segs, parts, keys);
    KQ_LAUNCHED("token_logprobs_join");
  }
  return KRONQ_OK;
}

// ---------------------------------------------------------------- gradients

constexpr int kSpan = 4096;               // values of a row that a workgroup takes (6144 x 128256 bf16: 518 us, 16384 620, 2048 589)

// One pass, a read and a write; bound by HBM: 6144 x 128256 in bf16 505 us, 6.2 TB/s.
// An output is rounded to its type once.  The few places that a target or an
// alternative names are computed again behind it, all their shares at once.  The
// logits may be where the gradients go: those places are read before the pass.
template <typename T>
__global__ __launch_bounds__(NT) void token_logprobs_grad(LogprobsGradArgs a, int spans) {
  constexpr int N = Row<T>::N;
  const int64_t r = blockIdx.x / (unsigned)spans;
  const int span = (int)(blockIdx.x % (unsigned)spans), tid = threadIdx.x;
  const T* in = static_cast<const T*>(a.logits) + r * a.ld;
  T* out = static_cast<T*>(a.out) + r * a.ld_out;
  const Row<T> row(in, a.vocab);
  const int target = a.targets ? a.targets[r] : -1;
  const float lse = a.lse[r], g = target >= 0 && a.d_logp ? a.d_logp[r] : 0.0f;
  const float h = a.d_entropy ? a.d_entropy[r] : 0.0f, ent = a.d_entropy ? a.entropy[r] : 0.0f;
  float whole = g;
  if (target >= a.vocab) whole = quiet_nan();
  if (a.d_top)
    for (int k = 0; k < a.top; ++k) {
      const int id = a.top_ids[r * a.top + k];
      if (id >= 0 && id < a.vocab) whole += a.d_top[r * a.top + k];
    }
  const bool none = lse == -INFINITY;     // nothing but minus infinity
  auto grad = [&](float x) {
    const float logp = x - lse, p = exp_of(logp);
    float d = whole;
    if (a.d_entropy) d += h * (fmaxf(logp, kFar) + ent);
    return none ? 0.0f : -p * d;
  };
  // this span's values from `first` on, whole chunks but at a row's ends
  const int per = kSpan / N, c0 = span * per, c1 = min(row.chunks, c0 + per);
  const bool lo = span == 0, hi = span == spans - 1;
  const int first = lo ? 0 : row.index(min(c0, row.chunks)), last = hi ? row.vocab : row.index(c1);
  // thread k's place: an alternative's, or behind them the target's
  int place = -1;
  float held = 0;
  if (tid <= a.top) {
    place = tid == a.top ? target : a.d_top ? a.top_ids[r * a.top + tid] : -1;
    if (place < first || place >= last) place = -1;
    if (place >= 0) held = value(in[place]);
  }
  __syncthreads();
  auto one = [&](int v) { set(out[v], grad(value(in[v]))); };
  if (lo && tid < row.head) one(tid);
  if (hi && tid < row.vocab - row.rest()) one(row.rest() + tid);
  if (((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(in)) & 15) == 0) {
    for (int c = c0 + tid; c < c1; c += NT) {
      float x[N];
      unpack(row.chunk(c), x, T());
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = grad(x[i]);
      T* to = out + row.index(c);
      if constexpr (N == 4) store4(to, x);
      else store8(to, x);
    }
  } else {                                // borders of sixteen bytes differ
    for (int v = row.index(c0) + tid; v < row.index(c1); v += NT) one(v);
  }
  __syncthreads();                        // what the pass wrote is there before
  if (place >= 0 && !none) {
    float d = grad(held) + (place == target ? g : 0.0f);
    if (a.d_top)
      for (int k = 0; k < a.top; ++k)
        if (a.top_ids[r * a.top + k] == place) d += a.d_top[r * a.top + k];
    set(out[place], d);
  }
}

int spans_of(int64_t vocab) { return (int)((vocab + kSpan - 1) / kSpan); }

}  // namespace

size_t logprobs_ws_bytes(int64_t rows, int64_t vocab, int top) {
  const int segs = segments(rows, vocab);
  return segs > 1 ? (size_t)rows * segs * (sizeof(Part) + (size_t)top * sizeof(uint64_t)) : 0;
}

kronq_status logprobs_launch(const LogprobsArgs& a, int32_t dtype, void* ws, hipStream_t s) {
  if (dtype == KRONQ_F32) return logprobs_type<float>(a, ws, s);
  if (dtype == KRONQ_BF16) return logprobs_type<bf16_t>(a, ws, s);
  return logprobs_type<_Float16>(a, ws, s);
}

int64_t logprobs_grad_grid(int64_t rows, int64_t vocab) { return rows * spans_of(vocab); }

kronq_status logprobs_grad_launch(const LogprobsGradArgs& a, int32_t dtype, hipStream_t s) {
  const int spans = spans_of(a.vocab);
  const dim3 grid((unsigned)(a.rows * spans));
  if (dtype == KRONQ_F32) hipLaunchKernelGGL((token_logprobs_grad<float>), grid, dim3(NT), 0, s, a, spans);
  else if (dtype == KRONQ_BF16) hipLaunchKernelGGL((token_logprobs_grad<bf16_t>), grid, dim3(NT), 0, s, a, spans);
  else hipLaunchKernelGGL((token_logprobs_grad<_Float16>), grid, dim3(NT), 0, s, a, spans);
  KQ_LAUNCHED("token_logprobs_grad");
  return KRONQ_OK;
}

}  // namespace kronq
