// The 4-bit paged key/value cache: new tokens in (rotated and rounded to the
// grid), and the held values out.
//
// Both kernels give a lane eight consecutive values of one token's head, so
// dim / 8 neighbouring lanes hold a group (the unit that shares a scale and a
// zero point), and the group's extremes come from log2(dim / 8) exchanges.
#include "kv.h"

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

// Extremes over a group's LANES lanes.  Of V = float when the values are exact
// there (inputs as they came), of V = double for rotated ones.
template <int LANES, typename V>
__device__ inline void group_extremes(V& lo, V& hi) {
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1) {
    const V l = __shfl_xor(lo, d), h = __shfl_xor(hi, d);
    lo = l < lo ? l : lo;
    hi = h > hi ? h : hi;
  }
}

// One group's grid word and this lane's eight codes.  The grid is defined in
// fp64 (a code changes at a border, so both sides of a border have to agree on
// it), but only the group's scale and zero point need it: a code is taken in
// fp32 unless its place on the grid is within 2^-15 of a border, where the fp32
// arithmetic (off by at most 15 * 2^-22 there) cannot tell.
template <int LANES, typename V>
__device__ inline uint32_t to_grid(const V (&x)[8], uint32_t& word) {
  V lo = 0, hi = 0;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = x[i] < lo ? x[i] : lo;
    hi = x[i] > hi ? x[i] : hi;
    fine = fine && (x[i] - x[i] == 0);
  }
  group_extremes<LANES>(lo, hi);
  const uint64_t lanes = LANES == 64 ? ~0ull : ((1ull << LANES) - 1);
  const int first = (threadIdx.x & 63) & ~(LANES - 1);
  if ((__ballot(!fine) >> first) & lanes) {
    word = 0x7FC00000u;
    return 0;
  }
  double l = lo, h = hi;
  if (l == h) l = -1, h = 1;                        // both are 0
  double want = (h - l) / 15.0;
  if (want < 0x1p-126) want = 0x1p-126;
  uint32_t w = __float_as_uint((float)want);
  w = (w + 7 + ((w >> 4) & 1)) & ~15u;              // 20 significant bits, ties to even
  const double s = __uint_as_float(w);
  double z = rint(-l / s);
  z = z < 0 ? 0 : z > 15 ? 15 : z;
  word = w | (uint32_t)(int)z;
  const float inv = (float)(1.0 / s), zf = (float)z;
  const bool plain = inv > 0x1p-120f && inv < 0x1p+120f;   // fp32 holds it in full
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = fmaf((float)x[i], inv, zf);
    float q = rintf(t);
    if (!(fabsf(t - q) < 0.5f - 0x1p-15f) || !plain) q = (float)rint((double)x[i] / s + z);
    q = fminf(fmaxf(q, 0.0f), 15.0f);
    codes |= (uint32_t)q << (4 * i);
  }
  return codes;
}

// blockIdx.y: 0 keys, 1 values.  A lane group takes one (row, head); heads are
// the faster index, so a wave reads neighbouring heads of a row.
// Bound by memory at size and by latency for few rows; the only fp64 work over
// all values is the keys' rotation, two fused operations each.
template <typename T, int LANES>
__global__ __launch_bounds__(NT) void kv_append(KvView c, HeadsView k, HeadsView v, RopeView rope) {
  __shared__ int32_t lds[kCuLds];
  const int32_t* cu = stage_cu(c, lds);
  const int64_t item = ((int64_t)blockIdx.x * NT + threadIdx.x) / LANES;
  const int d = (threadIdx.x & (LANES - 1)) * 8;
  const bool in = item < (int64_t)c.rows * c.heads;
  const int row = in ? (int)(item / c.heads) : 0, head = in ? (int)(item % c.heads) : 0;
  const int seq = in ? seq_of(cu, c.seqs, row) : -1;
  Place at{-1, 0, 0, true};
  if (seq >= 0) at = place_of(c, seq, row, cu[seq + 1]);
  const bool keys = blockIdx.y == 0;
  if (rope.half && at.pos >= rope.positions) at.pos = -1;   // both halves of a token, or none
  const bool on = at.pos >= 0 && !at.bad;                   // one value for a group's lanes
  float x[8];
  uint32_t word = 0, codes;
  const HeadsView src = keys ? k : v;
  const T* p = static_cast<const T*>(src.data) + row * src.row + head * src.head;
  if (on) {
    load8(p + d, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0;
  }
  if (keys && rope.half) {
    double y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
    if (on && d < 2 * rope.half) {
      // products of two fp32 numbers are exact in fp64: each sum is rounded once
      const float* ct = rope.cos + at.pos * rope.ld;
      const float* st = rope.sin + at.pos * rope.ld;
      if (rope.neighbours) {
        const f32x4 cv = *reinterpret_cast<const f32x4*>(ct + d / 2);
        const f32x4 sv = *reinterpret_cast<const f32x4*>(st + d / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double a = x[2 * i], b = x[2 * i + 1], cc = cv[i], ss = sv[i];
          y[2 * i] = a * cc - b * ss;
          y[2 * i + 1] = b * cc + a * ss;
        }
      } else {
        const bool second = d >= rope.half;
        const int j = second ? d - rope.half : d;
        float o[8], cv[8], sv[8];
        load8(p + (second ? j : d + rope.half), o);
        load8(ct + j, cv);
        load8(st + j, sv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double a = x[i], b = o[i], cc = cv[i], ss = second ? sv[i] : -sv[i];
          y[i] = a * cc + b * ss;
        }
      }
    }
    codes = to_grid<LANES>(y, word);
  } else {
    codes = to_grid<LANES>(x, word);
  }
  if (!on) return;
  const int64_t slot = ((int64_t)head << c.lgp) + at.slot;
  if (keys) {
    *reinterpret_cast<uint32_t*>(c.kc + page_offset(at.page, c.kcs) + slot * (LANES * 4) + d / 2) = codes;
    if (d == 0) c.kg[page_offset(at.page, c.kgs) + slot] = word;
  } else {
    *reinterpret_cast<uint32_t*>(c.vc + page_offset(at.page, c.vcs) + slot * (LANES * 4) + d / 2) = codes;
    if (d == 0) c.vg[page_offset(at.page, c.vgs) + slot] = word;
  }
}

// As kv_append: one (row, head) for a lane group, blockIdx.y 0 keys, 1 values.
template <typename T, int LANES>
__global__ __launch_bounds__(NT) void kv_read(KvView c, HeadsView k, HeadsView v) {
  __shared__ int32_t lds[kCuLds];
  const int32_t* cu = stage_cu(c, lds);
  const int64_t item = ((int64_t)blockIdx.x * NT + threadIdx.x) / LANES;
  if (item >= (int64_t)c.rows * c.heads) return;
  const int d = (threadIdx.x & (LANES - 1)) * 8;
  const int row = (int)(item / c.heads), head = (int)(item % c.heads);
  const int seq = seq_of(cu, c.seqs, row);
  if (seq < 0) return;                                      // a row of no sequence
  const Place at = place_of(c, seq, row, cu[seq + 1]);
  const bool keys = blockIdx.y == 0;
  const HeadsView dst = keys ? k : v;
  T* p = static_cast<T*>(dst.data) + row * dst.row + head * dst.head + d;
  float x[8];
  float s = __uint_as_float(0x7FC00000u);
  uint32_t word = 0, w = 0;
  if (at.pos >= 0 && !at.bad) {
    const int64_t slot = ((int64_t)head << c.lgp) + at.slot;
    word = keys ? c.kg[page_offset(at.page, c.kgs) + slot] : c.vg[page_offset(at.page, c.vgs) + slot];
    const uint8_t* codes = keys ? c.kc + page_offset(at.page, c.kcs) : c.vc + page_offset(at.page, c.vcs);
    w = *reinterpret_cast<const uint32_t*>(codes + slot * (LANES * 4) + d / 2);
    s = __uint_as_float(word & ~15u);
  }
  const int z = word & 15;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = s * (float)((int)((w >> (4 * i)) & 15) - z);
  store8(p, x);
}

template <typename T, int LANES>
void append_typed(const KvView& c, const HeadsView& k, const HeadsView& v, const RopeView& r, hipStream_t s) {
  const int64_t items = (int64_t)c.rows * c.heads;
  const dim3 grid((unsigned)((items * LANES + NT - 1) / NT), 2);
  hipLaunchKernelGGL((kv_append<T, LANES>), grid, dim3(NT), 0, s, c, k, v, r);
}

template <typename T, int LANES>
void read_typed(const KvView& c, const HeadsView& k, const HeadsView& v, hipStream_t s) {
  const int64_t items = (int64_t)c.rows * c.heads;
  const dim3 grid((unsigned)((items * LANES + NT - 1) / NT), 2);
  hipLaunchKernelGGL((kv_read<T, LANES>), grid, dim3(NT), 0, s, c, k, v);
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
