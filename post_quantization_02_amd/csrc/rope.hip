// Rotary positions outside the cache: the tables of cosines and sines, plain or
// scaled for contexts longer than the model's, and the rotation of query and key
// heads in both directions.
//
// A pair (a, b) of a head at position p turns by the angle p f_i:
//   a' = a cos - b sin, b' = b cos + a sin     (back: the transpose, -sin for sin)
// The transpose is the gradient of the rotation and, but for the tables' common
// factor and rounding, its inverse.
#include <algorithm>
#include <cmath>

#include "kv.h"
#include "rope.h"

namespace kronq {
namespace {

// ---------------------------------------------------------------- tables

// Angles are products in fp64 (position 10^5 times a frequency: 10^-11 off).  A
// thread takes one pair through kSteps positions: cosine and sine of the first
// and of one step from the library, then one turn a step in fp64, four operations
// where a sine and a cosine cost above a hundred.  kSteps turns are off by at most
// kSteps 2^-52, far below the result's 2^-24, relative to a small sine as well (its
// terms then have one sign).  Bound by the writes: 131072 positions of 64 pairs 12.2 us,
// 5.5 TB/s.
constexpr int kSteps = 32;

struct Frequencies { double f[kRopePairs]; };

__global__ __launch_bounds__(256) void rope_tables(Frequencies fr, float* __restrict__ cos_out, float* __restrict__ sin_out,
                                                   int64_t ld, int64_t first, int64_t positions, int half,
                                                   double magnitude) {
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t block = at / half;
  const int i = (int)(at - block * half);
  const int64_t p0 = block * kSteps;
  if (p0 >= positions) return;
  const double f = fr.f[i];
  double s, c, ds, dc;
  sincos((double)(first + p0) * f, &s, &c);
  sincos(f, &ds, &dc);
  const int n = (int)min((int64_t)kSteps, positions - p0);
  for (int k = 0; k < n; ++k) {
    cos_out[(p0 + k) * ld + i] = (float)(c * magnitude);
    sin_out[(p0 + k) * ld + i] = (float)(s * magnitude);
    const double t = c * dc - s * ds;
    s = s * dc + c * ds;
    c = t;
  }
}

// ---------------------------------------------------------------- rotation

struct RotateArgs {
  HeadsView in[2], out[2];                // queries, keys
  int heads[2];
  const int32_t* pos;
  RopeView r;
  int rows, dim, back;
  bool same[2];                           // in place
};

// sixteen bytes of values
__device__ __forceinline__ void load_piece(const float* p, float (&x)[4]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = a[i];
}
template <typename T>
__device__ __forceinline__ void load_piece(const T* p, float (&x)[8]) { load8(p, x); }
__device__ __forceinline__ void store_piece(float* p, const float (&x)[4]) { store4(p, x); }
template <typename T>
__device__ __forceinline__ void store_piece(T* p, const float (&x)[8]) { store8(p, x); }

template <int E>
__device__ __forceinline__ void load_angles(const float* p, float (&x)[E]) {
  if constexpr (E == 2) x[0] = p[0], x[1] = p[1];
  else
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(p + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i + j] = a[j];
    }
}

// A lane takes two pieces of sixteen bytes of a token's head, half of the rotated values
// (of the others) apart: the two sides of its pairs, or, where neighbours are pairs, two
// pieces of them.  Neighbouring lanes are neighbouring pieces, then heads.  Bound by HBM:
// 15000 rows of 64 and 8 heads of 128 in bf16 70 us, 5.6 TB/s.
template <typename T, bool NEIGHBOURS>
__global__ __launch_bounds__(256) void rotate(RotateArgs a) {
  constexpr int E = 16 / sizeof(T);
  const uint32_t at = blockIdx.x * 256u + threadIdx.x, each = (uint32_t)a.dim / (2 * E);
  const uint32_t heads = (uint32_t)(a.heads[0] + a.heads[1]), unit = at / each;
  const int c = (int)(at - unit * each), row = (int)(unit / heads), h = (int)(unit - (uint32_t)row * heads);
  if (row >= a.rows) return;
  const int pos = a.pos[row];
  if (pos < 0) return;                    // a row of no sequence
  const int which = h >= a.heads[0];
  const HeadsView in = which ? a.in[1] : a.in[0], out = which ? a.out[1] : a.out[0];
  const int64_t head = which ? h - a.heads[0] : h;
  const T* x = static_cast<const T*>(in.data) + row * in.row + head * in.head;
  T* y = static_cast<T*>(out.data) + row * out.row + head * out.head;
  const int rot = 2 * a.r.half;
  const bool turns = c < a.r.half / E;
  const int d0 = turns ? E * c : rot + E * (c - a.r.half / E), d1 = d0 + (turns ? a.r.half : (a.dim - rot) / 2);
  if (pos >= a.r.positions) {
    float none[E];
#pragma unroll
    for (int i = 0; i < E; ++i) none[i] = __uint_as_float(0x7FC00000u);
    store_piece(y + d0, none);
    store_piece(y + d1, none);
    return;
  }
  if (!turns) {                           // as they are, bit for bit
    if (which ? a.same[1] : a.same[0]) return;
    const u32x4 u = *reinterpret_cast<const u32x4*>(x + d0), v = *reinterpret_cast<const u32x4*>(x + d1);
    *reinterpret_cast<u32x4*>(y + d0) = u;
    *reinterpret_cast<u32x4*>(y + d1) = v;
    return;
  }
  const float* cos = a.r.cos + pos * a.r.ld;
  const float* sin = a.r.sin + pos * a.r.ld;
  const float sign = a.back ? -1.0f : 1.0f;
  float u[E], v[E], p[E], q[E];
  load_piece(x + d0, u);
  load_piece(x + d1, v);
  if constexpr (NEIGHBOURS) {
    float cu[E / 2], su[E / 2], cv[E / 2], sv[E / 2];
    load_angles(cos + d0 / 2, cu);
    load_angles(sin + d0 / 2, su);
    load_angles(cos + d1 / 2, cv);
    load_angles(sin + d1 / 2, sv);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float s0 = sign * su[i], s1 = sign * sv[i];
      p[2 * i] = u[2 * i] * cu[i] - u[2 * i + 1] * s0;
      p[2 * i + 1] = u[2 * i + 1] * cu[i] + u[2 * i] * s0;
      q[2 * i] = v[2 * i] * cv[i] - v[2 * i + 1] * s1;
      q[2 * i + 1] = v[2 * i + 1] * cv[i] + v[2 * i] * s1;
    }
  } else {
    float cs[E], sn[E];
    load_angles(cos + d0, cs);
    load_angles(sin + d0, sn);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float s = sign * sn[i];
      p[i] = u[i] * cs[i] - v[i] * s;
      q[i] = v[i] * cs[i] + u[i] * s;
    }
  }
  store_piece(y + d0, p);
  store_piece(y + d1, q);
}

template <typename T>
void rotate_type(const RotateArgs& a, unsigned grid, hipStream_t s) {
  if (a.r.neighbours) hipLaunchKernelGGL((rotate<T, true>), dim3(grid), dim3(256), 0, s, a);
  else hipLaunchKernelGGL((rotate<T, false>), dim3(grid), dim3(256), 0, s, a);
}

}  // namespace

void rope_frequencies(const kronq_rope_scaling& c, int dim, double* f) {
  // the pair whose wave turns `turns` times over the original positions
  auto place = [&](double turns) {
    return dim * std::log(c.original / (turns * 2 * M_PI)) / (2 * std::log(c.base));
  };
  double lo = 0, hi = 0;
  if (c.scaling == KRONQ_ROPE_INDEX) {
    lo = std::max(std::floor(place(c.high)), 0.0);
    hi = std::min(std::ceil(place(c.low)), dim - 1.0);
  }
  for (int i = 0; i < dim / 2; ++i) {
    const double plain = std::pow(c.base, -2.0 * i / dim);
    double keep = 1;                      // share of the plain frequency, beside the one divided by factor
    if (c.scaling == KRONQ_ROPE_LINEAR) keep = 0;
    if (c.scaling == KRONQ_ROPE_PARTS) keep = (c.original * plain / (2 * M_PI) - c.low) / (c.high - c.low);
    if (c.scaling == KRONQ_ROPE_INDEX) keep = 1 - (i - lo) / std::max(hi - lo, 0.001);
    keep = std::min(std::max(keep, 0.0), 1.0);
    f[i] = plain * keep + plain / c.factor * (1 - keep);
  }
}

int64_t rope_tables_grid(int64_t positions, int dim) {
  return ((positions + kSteps - 1) / kSteps * (dim / 2) + 255) / 256;
}

int64_t rotate_grid(int64_t rows, int64_t heads, int dim, int32_t dtype) {
  return (rows * heads * (dim / (dtype == KRONQ_F32 ? 8 : 16)) + 255) / 256;
}

kronq_status rope_tables_launch(float* cos, float* sin, int64_t ld, int64_t first, int64_t positions, int dim,
                                const kronq_rope_scaling& c, hipStream_t s) {
  Frequencies fr{};
  rope_frequencies(c, dim, fr.f);
  const int half = dim / 2;
  hipLaunchKernelGGL(rope_tables, dim3((unsigned)rope_tables_grid(positions, dim)), dim3(256), 0, s, fr, cos, sin, ld, first,
                     positions, half, c.magnitude);
  KQ_LAUNCHED("rope_tables");
  return KRONQ_OK;
}

kronq_status rotate_launch(const HeadsView* in, const HeadsView* out, const int* heads, int32_t dtype, int64_t rows,
                           int dim, const int32_t* pos, const RopeView& r, int back, hipStream_t s) {
  RotateArgs a{};
  for (int w = 0; w < 2; ++w) {
    a.in[w] = in[w];
    a.out[w] = out[w];
    a.heads[w] = heads[w];
    a.same[w] = in[w].data == out[w].data;
  }
  a.pos = pos;
  a.r = r;
  a.rows = (int)rows;
  a.dim = dim;
  a.back = back;
  const int64_t grid = rotate_grid(rows, (int64_t)heads[0] + heads[1], dim, dtype);
  switch (dtype) {
    case KRONQ_F32: rotate_type<float>(a, (unsigned)grid, s); break;
    case KRONQ_BF16: rotate_type<bf16_t>(a, (unsigned)grid, s); break;
    default: rotate_type<_Float16>(a, (unsigned)grid, s); break;
  }
  KQ_LAUNCHED("rotate");
  return KRONQ_OK;
}

}  // namespace kronq
