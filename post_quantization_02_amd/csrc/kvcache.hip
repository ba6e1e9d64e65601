// The 4-bit paged key/value cache: new tokens in (rotated and rounded to the
// grid), and the held values out.
//
// Both kernels give a lane eight consecutive values of one token's head, so
// dim / 8 neighbouring lanes hold a group (the unit that shares a scale and a
// zero point).  A group's lanes take one token and go through some of its heads:
// its sequence, its page and its rotation are found once for them.  A workgroup's
// tokens are neighbours, which share a page's lines of codes and grid words.
#include "kv.h"

#include <type_traits>

namespace kronq {
namespace {

constexpr int NT = 256;
constexpr int kCuLds = 1024;   // sequence starts kept in LDS

// Sequence starts in LDS while they fit: the search for a row's sequence is a
// chain of dependent reads.
__device__ inline const int32_t* stage_cu(const KvView& c, int32_t* lds) {
  if (c.seqs >= kCuLds) return c.cu;
  for (int i = threadIdx.x; i <= c.seqs; i += NT) lds[i] = c.cu[i];
  __syncthreads();
  return lds;
}

template <typename V>
__device__ inline V least(V a, V b) { return __builtin_elementwise_min(a, b); }
template <typename V>
__device__ inline V most(V a, V b) { return __builtin_elementwise_max(a, b); }

// Extremes over a group's LANES lanes.  Of V = float when the values are exact
// there (inputs as they came), of V = double for rotated ones.
template <int LANES, typename V>
__device__ inline void group_extremes(V& lo, V& hi) {
  auto step = [&](V l, V h) __attribute__((always_inline)) {
    lo = least(lo, l);
    hi = most(hi, h);
  };
  step(partner<0xB1>(lo), partner<0xB1>(hi));       // lane ^ 1
  step(partner<0x4E>(lo), partner<0x4E>(hi));       // lane ^ 2
  step(partner<0x141>(lo), partner<0x141>(hi));     // mirrored within eight
  if constexpr (LANES > 8) step(partner<0x140>(lo), partner<0x140>(hi));   // within sixteen
  if constexpr (LANES > 16) step(__shfl_xor(lo, 16), __shfl_xor(hi, 16));
}

// How near to a border between two codes fp32 is asked, see below.
constexpr float kSure = 0.5f - 0x1p-15f;

// One group's grid word and this lane's eight codes.  The grid is defined in
// fp64 (a code changes at a border, so both sides of a border have to agree on
// it), but only the group's extremes and their difference need it: zero point and
// codes are taken in fp32 unless a place on the grid is within 2^-15 of a border,
// where fp32 (places up to 16, each off by less than 2^-18: 1.5 x 2^-23 of the
// product of value and reciprocal, and half a last place) cannot tell.
template <int LANES, typename V>
__device__ inline uint32_t to_grid(const V (&x)[8], uint32_t& word) {
  V lo = 0, hi = 0, odd = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = least(lo, x[i]);
    hi = most(hi, x[i]);
    odd = __builtin_elementwise_fma(x[i], (V)0, odd);         // not 0: not finite
  }
  group_extremes<LANES>(lo, hi);
  const uint64_t lanes = LANES == 64 ? ~0ull : ((1ull << LANES) - 1);
  const int first = (threadIdx.x & 63) & ~(LANES - 1);
  if ((__ballot(!(odd == 0)) >> first) & lanes) {
    word = 0x7FC00000u;
    return 0;
  }
  double l = lo, h = hi;
  if (l == h) l = -1, h = 1;                        // both are 0
  // (h - l) / 15: the product with 1/15 (off by 2^-56) is one of the quotient's two
  // neighbours, from which one step with the exact remainder rounds it correctly
  const double d = h - l, by = 1.0 / 15.0, near = d * by;
  double want = fma(fma(-15.0, near, d), by, near);
  if (want < 0x1p-126) want = 0x1p-126;
  uint32_t w = __float_as_uint((float)want);
  w = (w + 7 + ((w >> 4) & 1)) & ~15u;              // 20 significant bits, ties to even
  const float s = __uint_as_float(w), inv = __builtin_amdgcn_rcpf(s);    // 2^-23
  const bool plain = inv > 0x1p-120f && inv < 0x1p+120f;   // fp32 holds it in full
  const float at = -(float)l * inv;
  float zf = rintf(at);
  if (!(fabsf(at - zf) < kSure) || !plain) zf = (float)rint(-l / s);
  zf = fminf(fmaxf(zf, 0.0f), 15.0f);
  word = w | (uint32_t)(int)zf;
  float q[8], off = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = fmaf((float)x[i], inv, zf), r = rintf(t);
    off = most(off, fabsf(t - r));
    q[i] = __builtin_amdgcn_fmed3f(r, 0.0f, 15.0f);
  }
  if (!(off < kSure) || !plain) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf((float)rint((double)x[i] / s + zf), 0.0f), 15.0f);
  }
  // four codes are a number below 2^16
  auto four = [&](int i) __attribute__((always_inline)) {
    return (uint32_t)fmaf(q[i + 3], 4096.0f, fmaf(q[i + 2], 256.0f, fmaf(q[i + 1], 16.0f, q[i])));
  };
  return four(0) | four(4) << 16;
}

// Eight values as they are in memory.
template <typename T>
struct Eight {
  u32x4_alias w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) w[i] = reinterpret_cast<const u32x4_alias*>(p)[i];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const { load8(reinterpret_cast<const T*>(w), x); }
};

// Which token and heads a thread works for: blockIdx.x counts NT / LANES tokens;
// blockIdx.y is twice the block of `per` heads, and 1 more for values.
struct Work { int row, d, head0, head1; bool keys; };

template <int LANES>
__device__ inline Work work_of(const KvView& c, int per) {
  const int row = (int)(blockIdx.x * (NT / LANES) + threadIdx.x / LANES);
  const int head0 = (int)(blockIdx.y >> 1) * per;
  return {row, (int)(threadIdx.x & (LANES - 1)) * 8, head0, min(head0 + per, c.heads), (blockIdx.y & 1) == 0};
}

// Bound by the vector pipes at size (28.6 operations a value by the counters: what a
// group's lanes do for their eight values each, extremes of rotated keys in fp64 and
// the grid among it), by the launch for few rows.  19000 rows of 8 heads of
// 128 bf16 values, keys and values: 40 us (118 MB: 2.9 TB/s); one row 4 us.  With
// a lane group for each (row, head), its sequence searched each time, 67 us.
template <typename T, int LANES>
__global__ __launch_bounds__(NT) void kv_append(KvView c, HeadsView k, HeadsView v, RopeView rope, int per) {
  __shared__ int32_t lds[kCuLds];
  const int32_t* cu = stage_cu(c, lds);
  const Work w = work_of<LANES>(c, per);
  if (w.row >= c.rows) return;
  const int seq = seq_of(cu, c.seqs, w.row);
  if (seq < 0) return;                                      // a row of no sequence
  const Place at = place_of(c, seq, w.row, cu[seq + 1]);
  if (at.pos < 0 || at.bad) return;
  if (rope.half && at.pos >= rope.positions) return;        // both halves of a token, or none
  const int d = w.d;
  const HeadsView src = w.keys ? k : v;
  const T* p = static_cast<const T*>(src.data) + w.row * src.row + w.head0 * src.head;
  const bool turn = w.keys && d < 2 * rope.half;
  // the other half's values (the same again where there is nothing to rotate)
  const int d2 = !turn || rope.neighbours ? d : d >= rope.half ? d - rope.half : d + rope.half;
  float cv[8], sv[8];
  if (turn) {
    const float* ct = rope.cos + at.pos * rope.ld;
    const float* st = rope.sin + at.pos * rope.ld;
    if (rope.neighbours) {                                  // pairs' angles, twice
      const f32x4 a = *reinterpret_cast<const f32x4*>(ct + d / 2), b = *reinterpret_cast<const f32x4*>(st + d / 2);
#pragma unroll
      for (int i = 0; i < 8; ++i) cv[i] = a[i / 2], sv[i] = i & 1 ? b[i / 2] : -b[i / 2];
    } else {
      const int j = min(d, d2);
      load8(ct + j, cv);
      load8(st + j, sv);
#pragma unroll
      for (int i = 0; i < 8; ++i) sv[i] = d > d2 ? sv[i] : -sv[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) cv[i] = 1, sv[i] = 0;
  }
  uint8_t* codes = (w.keys ? c.kc + page_offset(at.page, c.kcs) : c.vc + page_offset(at.page, c.vcs)) +
                   (((uint64_t)w.head0 << c.lgp) + at.slot) * (LANES * 4) + d / 2;
  uint32_t* grid = (w.keys ? c.kg + page_offset(at.page, c.kgs) : c.vg + page_offset(at.page, c.vgs)) +
                   ((uint64_t)w.head0 << c.lgp) + at.slot;
  // rotated: 0, 1 pairs of the halves, 2 neighbours
  auto go = [&](auto rotated) __attribute__((always_inline)) {
    Eight<T> mine, other;
    mine.load(p + d);
    if constexpr (rotated == 1) other.load(p + d2);
    for (int head = w.head0; head < w.head1; ++head) {
      float x[8], o[8];
      mine.get(x);
      if constexpr (rotated == 1) other.get(o);
      if (head + 1 < w.head1) p += src.head;                // asked for early; the last one twice
      mine.load(p + d);
      if constexpr (rotated == 1) other.load(p + d2);
      uint32_t word, out;
      if constexpr (rotated != 0) {
        // Products of two fp32 numbers are exact in fp64: each sum is rounded once.
        // Values behind the rotated ones: x 1 + x 0, which is x where x is finite.
        double y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[i] = fma((double)x[i], (double)cv[i], (double)(rotated == 1 ? o[i] : x[i ^ 1]) * (double)sv[i]);
        out = to_grid<LANES>(y, word);
      } else {
        out = to_grid<LANES>(x, word);
      }
      *reinterpret_cast<uint32_t*>(codes) = out;
      if (d == 0) *grid = word;
      codes += (size_t)(LANES * 4) << c.lgp;
      grid += 1 << c.lgp;
    }
  };
  if (!w.keys || !rope.half) go(std::integral_constant<int, 0>{});
  else if (rope.neighbours) go(std::integral_constant<int, 2>{});
  else go(std::integral_constant<int, 1>{});
}

// Bound by its writes.  32768 rows of 8 heads of 128 as bf16: 28 us (174 MB: 6.2 TB/s,
// the codes partly from the caches); one row 3 us.
template <typename T, int LANES>
__global__ __launch_bounds__(NT) void kv_read(KvView c, HeadsView k, HeadsView v, int per) {
  __shared__ int32_t lds[kCuLds];
  const int32_t* cu = stage_cu(c, lds);
  const Work w = work_of<LANES>(c, per);
  if (w.row >= c.rows) return;
  const int seq = seq_of(cu, c.seqs, w.row);
  if (seq < 0) return;                                      // a row of no sequence
  const Place at = place_of(c, seq, w.row, cu[seq + 1]);
  const bool there = at.pos >= 0 && !at.bad;
  const int d = w.d;
  const HeadsView dst = w.keys ? k : v;
  T* p = static_cast<T*>(dst.data) + w.row * dst.row + w.head0 * dst.head + d;
  const uint64_t slot = ((uint64_t)w.head0 << c.lgp) + at.slot;   // page 0 where there is none
  const uint8_t* codes = (w.keys ? c.kc + page_offset(at.page, c.kcs) : c.vc + page_offset(at.page, c.vcs)) +
                         slot * (LANES * 4) + d / 2;
  const uint32_t* grid = (w.keys ? c.kg + page_offset(at.page, c.kgs) : c.vg + page_offset(at.page, c.vgs)) + slot;
#pragma unroll 4
  for (int head = w.head0; head < w.head1; ++head) {
    const uint32_t word = there ? *grid : 0x7FC00000u, x8 = there ? *reinterpret_cast<const uint32_t*>(codes) : 0;
    const float s = __uint_as_float(word & ~15u), z = (float)(word & 15);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = s * ((float)((x8 >> (4 * i)) & 15) - z);
    store8(p, x);
    codes += (size_t)(LANES * 4) << c.lgp;
    grid += 1 << c.lgp;
    p += dst.head;
  }
}

// Heads a lane group goes through: as many as leave kGroups workgroups.  19000 rows
// appended, read: 41, 38 us at 1024 and 2048, 43, 37 at 4096, 69, 40 with one head
// each.
constexpr int64_t kGroups = 2048;
int heads_per(int64_t blocks, int heads) {
  int per = 8;
  while (per > 1 && (per > heads || 2 * blocks * ((heads + per - 1) / per) < kGroups)) per /= 2;
  return per;
}

template <typename T, int LANES>
void append_typed(const KvView& c, const HeadsView& k, const HeadsView& v, const RopeView& r, hipStream_t s) {
  const int blocks = (c.rows + NT / LANES - 1) / (NT / LANES), per = heads_per(blocks, c.heads);
  const dim3 grid((unsigned)blocks, 2 * (unsigned)((c.heads + per - 1) / per));
  hipLaunchKernelGGL((kv_append<T, LANES>), grid, dim3(NT), 0, s, c, k, v, r, per);
}

template <typename T, int LANES>
void read_typed(const KvView& c, const HeadsView& k, const HeadsView& v, hipStream_t s) {
  const int blocks = (c.rows + NT / LANES - 1) / (NT / LANES), per = heads_per(blocks, c.heads);
  const dim3 grid((unsigned)blocks, 2 * (unsigned)((c.heads + per - 1) / per));
  hipLaunchKernelGGL((kv_read<T, LANES>), grid, dim3(NT), 0, s, c, k, v, per);
}

template <typename T>
void append_dim(const KvView& c, int dim, const HeadsView& k, const HeadsView& v, const RopeView& r, hipStream_t s) {
  if (dim == 64) append_typed<T, 8>(c, k, v, r, s);
  else if (dim == 128) append_typed<T, 16>(c, k, v, r, s);
  else append_typed<T, 32>(c, k, v, r, s);
}

template <typename T>
void read_dim(const KvView& c, int dim, const HeadsView& k, const HeadsView& v, hipStream_t s) {
  if (dim == 64) read_typed<T, 8>(c, k, v, s);
  else if (dim == 128) read_typed<T, 16>(c, k, v, s);
  else read_typed<T, 32>(c, k, v, s);
}

}  // namespace

kronq_status kv_append_launch(const KvView& c, int dim, int32_t dtype, const HeadsView& k, const HeadsView& v,
                              const RopeView& r, hipStream_t s) {
  if (dtype == KRONQ_F32) append_dim<float>(c, dim, k, v, r, s);
  else if (dtype == KRONQ_BF16) append_dim<bf16_t>(c, dim, k, v, r, s);
  else append_dim<_Float16>(c, dim, k, v, r, s);
  KQ_LAUNCHED("kv_append");
  return KRONQ_OK;
}

kronq_status kv_read_launch(const KvView& c, int dim, int32_t dtype, const HeadsView& k, const HeadsView& v,
                            hipStream_t s) {
  if (dtype == KRONQ_F32) read_dim<float>(c, dim, k, v, s);
  else if (dtype == KRONQ_BF16) read_dim<bf16_t>(c, dim, k, v, s);
  else read_dim<_Float16>(c, dim, k, v, s);
  KQ_LAUNCHED("kv_read");
  return KRONQ_OK;
}

}  // namespace kronq
