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
// terms then have one sign).
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
  int rows, chunks;                       // chunks of sixteen values of a head
  int slices, back;
  bool same[2];                           // in place
};

// A lane takes sixteen values of a token's head, eight of each side of eight pairs
// (the rest of a head: sixteen neighbours, copied), and the same sixteen of
// every slices-th head: a token's angles are read once for them.  Neighbouring
// lanes are a head's chunks, then neighbouring heads.
template <typename T, bool NEIGHBOURS>
__global__ __launch_bounds__(256) void rotate(RotateArgs a) {
  const uint32_t at = blockIdx.x * 256u + threadIdx.x;
  const uint32_t unit = at / (uint32_t)a.chunks;
  const int chunk = (int)(at - unit * (uint32_t)a.chunks);
  const int row = (int)(unit / (uint32_t)a.slices), slice = (int)(unit - (uint32_t)row * (uint32_t)a.slices);
  if (row >= a.rows) return;
  const int pos = a.pos[row];
  if (pos < 0) return;                    // a row of no sequence
  const bool none = pos >= a.r.positions;
  const bool turns = chunk < a.r.half / 8;
  float c[8], s[8];
  if (turns && !none) {
    load8(a.r.cos + pos * a.r.ld + 8 * chunk, c);
    load8(a.r.sin + pos * a.r.ld + 8 * chunk, s);
    if (a.back) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = -s[i];
    }
  }
  const int d0 = NEIGHBOURS || !turns ? 16 * chunk : 8 * chunk;
  const int d1 = NEIGHBOURS || !turns ? d0 + 8 : d0 + a.r.half;
  for (int h = slice; h < a.heads[0] + a.heads[1]; h += a.slices) {
    const int which = h >= a.heads[0];
    const HeadsView in = which ? a.in[1] : a.in[0], out = which ? a.out[1] : a.out[0];
    const int64_t head = which ? h - a.heads[0] : h;
    const T* x = static_cast<const T*>(in.data) + row * in.row + head * in.head;
    T* y = static_cast<T*>(out.data) + row * out.row + head * out.head;
    float u[8], v[8];
    if (none) {
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = v[i] = __uint_as_float(0x7FC00000u);
      store8(y + d0, u);
      store8(y + d1, v);
      continue;
    }
    if (!turns) {
      if (which ? a.same[1] : a.same[0]) continue;
      // as they are, bit for bit
#pragma unroll
      for (int i = 0; i < 16 * (int)sizeof(T) / 16; ++i)
        reinterpret_cast<u32x4*>(y + d0)[i] = reinterpret_cast<const u32x4*>(x + d0)[i];
      continue;
    }
    load8(x + d0, u);
    load8(x + d1, v);
    float p[8], q[8];
    if constexpr (NEIGHBOURS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[2 * i] = u[2 * i] * c[i] - u[2 * i + 1] * s[i];
        p[2 * i + 1] = u[2 * i + 1] * c[i] + u[2 * i] * s[i];
        q[2 * i] = v[2 * i] * c[4 + i] - v[2 * i + 1] * s[4 + i];
        q[2 * i + 1] = v[2 * i + 1] * c[4 + i] + v[2 * i] * s[4 + i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = u[i] * c[i] - v[i] * s[i];
        q[i] = v[i] * c[i] + u[i] * s[i];
      }
    }
    store8(y + d0, p);
    store8(y + d1, q);
  }
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

kronq_status rope_tables_launch(float* cos, float* sin, int64_t ld, int64_t first, int64_t positions, int dim,
                                const kronq_rope_scaling& c, hipStream_t s) {
  Frequencies fr{};
  rope_frequencies(c, dim, fr.f);
  const int half = dim / 2;
  const int64_t threads = (positions + kSteps - 1) / kSteps * half;
  hipLaunchKernelGGL(rope_tables, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, fr, cos, sin, ld, first,
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
  a.chunks = dim / 16;
  a.back = back;
  // up to eight heads a lane once there are lanes for every wave slot of the chip
  const int total = heads[0] + heads[1];
  const int64_t lanes = rows * total * a.chunks;
  const int per = (int)std::min<int64_t>(8, std::max<int64_t>(1, lanes / (256 * 2048)));
  a.slices = (total + per - 1) / per;
  const int64_t grid = (rows * a.slices * a.chunks + 255) / 256;
  switch (dtype) {
    case KRONQ_F32: rotate_type<float>(a, (unsigned)grid, s); break;
    case KRONQ_BF16: rotate_type<bf16_t>(a, (unsigned)grid, s); break;
    default: rotate_type<_Float16>(a, (unsigned)grid, s); break;
  }
  KQ_LAUNCHED("rotate");
  return KRONQ_OK;
}

}  // namespace kronq
