// What the kernels of attention over whole packed prompts share: where a workgroup
// works, matrix operands of each type, tiles in LDS.
//
// All products are laid out so that a lane's column is its own: a 32 x 32 block of
// weights W^T has, in lane (c, h) (c = lane % 32, h = lane / 32), column c and rows
//   row(x, h) = x % 4 + 8 (x / 4) + 4 h,  x = 0 .. 15,
// and that is what the next product wants as its second operand, as long as its
// first operand's k slots are given the same order: weights never leave their
// registers, and statistics of a column are a lane's own.
#pragma once

#include <cfloat>
#include <type_traits>

#include "kv.h"
#include "prompt_index.h"

namespace kronq {

struct PromptArgs {
  HeadsView q, k, v, out, dout, dq, dk, dv;
  float* lse;               // rows x q_heads (forwards: NULL if not wanted)
  float *neg_lse, *neg_delta;   // backwards, workspace: q_heads x rows, -lse log2 e and -delta
  const int32_t* cu;
  int seqs, rows, heads, share, dim;
  float scale;              // > 0
  int window;               // of rows; more than there are: none
};

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr float kPromptLog2e = 1.44269504088896340736f, kPromptLn2 = 0.69314718055994530942f;

// ---------------------------------------------------------------- where a workgroup works

__device__ __forceinline__ int wave_sum(int x) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
  return __builtin_amdgcn_readfirstlane(x);
}
__device__ __forceinline__ int wave_max(int x) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x = max(x, __shfl_xor(x, o));
  return __builtin_amdgcn_readfirstlane(x);
}

// Tile number `unit` of all sequences' tiles of bm rows: its sequence, and how many tiles it
// has to do with (`much`: 1 .. the sequence's), the most first, so that the last
// workgroups to start are the short ones.  Sequences beyond 64 are taken one behind the
// other, each from its longest tile on.  False: there are fewer tiles.
__device__ __forceinline__ bool find_tile(const PromptArgs& a, int bm, int unit, Prompt& p, int& much) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int b0 = 0; b0 < a.seqs; b0 += 64) {
    Prompt mine{0, 0};
    if (b0 + lane < a.seqs) mine = prompt_between(a.cu[b0 + lane], a.cu[b0 + lane + 1], a.rows);
    const int tiles = (mine.n + bm - 1) / bm;
    if (a.seqs <= 64) {
      int lo = 0, hi = wave_max(tiles), upto = 0;  // tiles of more than hi: at most unit, of more than lo: more
      if (wave_sum(tiles) <= unit) return false;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1, n = wave_sum(max(tiles - mid, 0));
        if (n <= unit) hi = mid, upto = n;
        else lo = mid;
      }
      const uint64_t some = __ballot(tiles >= hi);
      const int rank = __builtin_amdgcn_mbcnt_hi((uint32_t)(some >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)some, 0));
      const int at = __ffsll((unsigned long long)__ballot(tiles >= hi && rank == unit - upto)) - 1;
      p.start = __builtin_amdgcn_readlane(mine.start, at);
      p.n = __builtin_amdgcn_readlane(mine.n, at);
      much = hi;
      return true;
    }
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(upto, o);
      upto += lane >= o ? y : 0;
    }
    const uint64_t past = __ballot(before + upto > unit);
    if (past) {
      const int at = __ffsll((unsigned long long)past) - 1;
      p.start = __builtin_amdgcn_readlane(mine.start, at);
      p.n = __builtin_amdgcn_readlane(mine.n, at);
      much = before + __builtin_amdgcn_readlane(upto, at) - unit;
      return true;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// ---------------------------------------------------------------- operands

// EPL: values of a lane in one step (16 bytes); STEP: k of a step; MULS: its products;
// TURNED: reads of a transposed operand.
template <typename T>
struct Op;

template <>
struct Op<bf16_t> {
  typedef s16x8 frag;
  static constexpr int EPL = 8, STEP = 16, MULS = 1, TURNED = 2;
  __device__ static f32x16 mul(frag a, frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  __device__ static float value(frag f, int i) { return __uint_as_float((uint32_t)(uint16_t)f[i] << 16); }
  __device__ static float value(bf16_t x) { return __uint_as_float((uint32_t)x.bits << 16); }
  __device__ static frag pack(const float* w) {
    bf16x8 f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (__bf16)w[i];
    return __builtin_bit_cast(frag, f);
  }
  // a word of values without what is not finite (an exponent of all ones)
  __device__ static uint32_t fine(uint32_t w) {
    return ((w & 0x7F80u) == 0x7F80u ? 0 : w & 0xFFFFu) | ((w & 0x7F800000u) == 0x7F800000u ? 0 : w & 0xFFFF0000u);
  }
};

template <>
struct Op<_Float16> {
  typedef s16x8 frag;
  static constexpr int EPL = 8, STEP = 16, MULS = 1, TURNED = 2;
  __device__ static f32x16 mul(frag a, frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
  }
  __device__ static float value(frag f, int i) { return (float)__builtin_bit_cast(half8_t, f)[i]; }
  __device__ static float value(_Float16 x) { return (float)x; }
  __device__ static frag pack(const float* w) {
    half8_t f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (_Float16)w[i];
    return __builtin_bit_cast(frag, f);
  }
  __device__ static uint32_t fine(uint32_t w) {
    return ((w & 0x7C00u) == 0x7C00u ? 0 : w & 0xFFFFu) | ((w & 0x7C000000u) == 0x7C000000u ? 0 : w & 0xFFFF0000u);
  }
};

// fp32 as it is: four products of k 2 a step
template <>
struct Op<float> {
  typedef f32x4 frag;
  static constexpr int EPL = 4, STEP = 8, MULS = 4, TURNED = 4;
  __device__ static f32x16 mul(frag a, frag b, f32x16 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
  __device__ static float value(frag f, int i) { return f[i]; }
  __device__ static float value(float x) { return x; }
  __device__ static frag pack(const float* w) { return frag{w[0], w[1], w[2], w[3]}; }
  __device__ static uint32_t fine(uint32_t w) { return (w & 0x7F800000u) == 0x7F800000u ? 0 : w; }
};

// Row of a 32 x 32 block that register x holds.
__device__ constexpr int block_row(int x, int h) { return (x & 3) + 8 * (x >> 2) + 4 * h; }

// Largest of a column: both halves hold some of its rows.
__device__ __forceinline__ float both_max(float x) {
  const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
}
__device__ __forceinline__ float both_sum(float x) {
  const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(y[0]) + __uint_as_float(y[1]);
}

// N groups of `muls` products with READS operand reads each from LDS, which run AHEAD
// groups before their products: left alone, the compiler has each product wait for a
// read just issued.
template <int N, int MULS, int READS, int AHEAD>
__device__ __forceinline__ void in_turn() {
  constexpr int kMul = 0x008, kRead = 0x100, kAhead = AHEAD < N ? AHEAD : N;
  __builtin_amdgcn_sched_group_barrier(kRead, kAhead * READS, 0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(kMul, MULS, 0);
    if (i < N - kAhead) __builtin_amdgcn_sched_group_barrier(kRead, READS, 0);
  }
}

// Keeps what follows a branch of its own: as selects it would cost every tile what few need.
__device__ __forceinline__ void rarely() { asm volatile(""); }

// ---------------------------------------------------------------- tiles in LDS

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// A tile's place in LDS.
template <typename Tile>
__device__ __forceinline__ uint32_t lds_at(const Tile& t) { return (uint32_t)(uintptr_t)(lds_u8*)&t; }

// Hides where a value comes from, so that what is added to it in a loop is added
// there: kept in a register each, those sums would leave none for the work.
__device__ __forceinline__ uint32_t hidden(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

// LDS is written in other units than it is read in.
template <typename V>
__device__ __forceinline__ V lds_read(uint32_t at) {
  typedef V __attribute__((may_alias)) Any;
  return *(const __attribute__((address_space(3))) Any*)(uintptr_t)at;
}
template <typename V>
__device__ __forceinline__ void lds_write(uint32_t at, V x) {
  typedef V __attribute__((may_alias)) Any;
  *(__attribute__((address_space(3))) Any*)(uintptr_t)at = x;
}

// Between what a wave writes to its own LDS and what its other lanes read of it: the
// hardware keeps their order, the compiler has to.
__device__ __forceinline__ void own_lds() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// ROWS rows of D values (D a power of two; what a head has fewer is 0), in 16-byte
// pieces that are exchanged within a row, piece c of a row at c ^ turn(row), so that
//   sixteen neighbouring rows' same pieces, and
//   four neighbouring pieces of rows 4 i .. 4 i + 3 (transposing reads)
// each lie in all 64 banks.  A lane's places are then one number, with a constant
// exclusive-or'd and a constant added for each read: tiles start at whole KiB.
template <typename T, int D, int ROWS>
struct LdsTile {
  static constexpr int PIECES = D * (int)sizeof(T) / 16, BYTES = D * (int)sizeof(T);
  alignas(1024) uint8_t b[ROWS * BYTES];

  __device__ static constexpr int turn(int row) {
    if (PIECES == 8) {                    // two rows in the banks
      const int m = (row >> 1) & 7;
      return (m & 1) << 2 | m >> 1;
    }
    return (row & 3) << 2 | ((row >> 2) & 3);
  }

  // This lane's number for rows_by_d: row c, piece h.
  __device__ static __forceinline__ uint32_t rows_lane() {
    const int lane = threadIdx.x & 63, row = lane & 31;
    return (uint32_t)(row * BYTES + (((lane >> 5) ^ turn(row)) << 4));
  }
  // First operand, rows r0 .. r0 + 31 by D, step s (of 2 pieces)
  __device__ static __forceinline__ typename Op<T>::frag rows_by_d(uint32_t at, int r0, int s) {
    return lds_read<typename Op<T>::frag>((at ^ (uint32_t)(2 * s) << 4) + (uint32_t)(r0 * BYTES));
  }

  // This lane's number for d_by_rows.
  __device__ static __forceinline__ uint32_t d_lane() {
    const int lane = threadIdx.x & 63, h = lane >> 5;
    if constexpr (sizeof(T) == 2) {       // rows 4 h .. 4 h + 3, a 16-lane group's two pieces
      const int row = 4 * h + ((lane >> 2) & 3), c = ((lane >> 4) & 1) * 2 + ((lane >> 1) & 1);
      return (uint32_t)(row * BYTES + ((c ^ turn(row)) << 4) + (lane & 1) * 8);
    } else {                              // row 4 h, value c
      return (uint32_t)(4 * h * BYTES + ((((lane & 31) >> 2) ^ turn(4 * h)) << 4) + (lane & 3) * 4);
    }
  }
  // First operand, values 32 dt .. 32 dt + 31 by rows r0 .. r0 + 31 (transposed), step s;
  // its k slots in the order that a block of weights has
  __device__ static __forceinline__ typename Op<T>::frag d_by_rows(uint32_t at, int r0, int dt, int s) {
    if constexpr (sizeof(T) == 2) {
      // rows 8 further turn by 2 more
      const uint32_t lo_at = (at ^ (uint32_t)(4 * dt) << 4) + (uint32_t)((r0 + 16 * s) * BYTES);
      const uint32_t hi_at = (at ^ (uint32_t)(4 * dt ^ 2) << 4) + (uint32_t)((r0 + 16 * s + 8) * BYTES);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)lo_at);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)hi_at);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      f32x4 f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[i] = lds_read<float>((at ^ (uint32_t)(8 * dt ^ turn(8 * s + i)) << 4) + (uint32_t)((r0 + 8 * s + i) * BYTES));
      return f;
    }
  }
};

// A tile on its way from memory to LDS by NT threads (a workgroup, or a wave each its
// own), 16 bytes a thread and load.
template <typename T, int D, int ROWS, int NT>
struct Staged {
  typedef LdsTile<T, D, ROWS> Tile;
  static constexpr int EACH = ROWS * Tile::PIECES / NT, APART = NT / Tile::PIECES;
  static_assert(EACH * NT == ROWS * Tile::PIECES && APART * EACH == ROWS, "whole rows");
  static_assert((APART & (APART - 1)) == 0, "the turn of a row is that of its multiple of APART and that of the rest");
  u32x4 w[EACH];

  // rows `row` .. of a head's n (row < n); `dim` of D values.  What lies behind the last
  // row's values is out of the buffer's range, and a load of it gives 0; so are a short
  // head's missing pieces, whose places are past any range.
  __device__ __forceinline__ void load(const HeadsView& x, int64_t first, int head, int row, int n, int dim) {
    const int c = threadIdx.x % Tile::PIECES, r = threadIdx.x % NT / Tile::PIECES;
    const uint32_t stride = (uint32_t)x.row * (uint32_t)sizeof(T);
    T* base = static_cast<T*>(x.data) + ((first + row) * x.row + head * x.head);
    const uint32_t range = (uint32_t)(min(n - row, ROWS) - 1) * stride + (uint32_t)dim * (uint32_t)sizeof(T);
    const auto rows = __builtin_amdgcn_make_buffer_rsrc(base, 0, range, 0x27000);
    const uint32_t mine = c * Op<T>::EPL < dim ? (uint32_t)r * stride + (uint32_t)c * 16 : 0x80000000u;
#pragma unroll
    for (int i = 0; i < EACH; ++i)
      w[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, mine + (uint32_t)(i * APART) * stride, 0, 0));
  }
  // This thread's number for store.
  __device__ static __forceinline__ uint32_t lane() {
    const int c = threadIdx.x % Tile::PIECES, r = threadIdx.x % NT / Tile::PIECES;
    return (uint32_t)(r * Tile::BYTES + ((c ^ Tile::turn(r)) << 4));
  }
  __device__ __forceinline__ void store(uint32_t at) const {
#pragma unroll
    for (int i = 0; i < EACH; ++i)
      lds_write((at ^ (uint32_t)Tile::turn(i * APART) << 4) + (uint32_t)(i * APART * Tile::BYTES), w[i]);
  }
  // Takes out what is not finite; the rows of the tile (from 0 on, of the first 32) that this
  // thread found any in.
  __device__ __forceinline__ uint32_t clean() {
    const int r = threadIdx.x % NT / Tile::PIECES;
    uint32_t rows = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      bool bad = false;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t y = Op<T>::fine(w[i][j]);
        bad |= y != w[i][j];
        w[i][j] = y;
      }
      rows |= bad ? 1u << ((r + i * APART) & 31) : 0u;
    }
    return rows;
  }
};

// Second operand, D by a lane's column: row `row` of a head (0 where row >= n).
template <typename T, int D>
__device__ __forceinline__ void load_column(const HeadsView& x, int64_t first, int head, int row, int n, int dim,
                                            typename Op<T>::frag (&f)[D / Op<T>::STEP]) {
  typedef typename Op<T>::frag frag;
  const int h = (threadIdx.x & 63) >> 5;
  const T* p = static_cast<const T*>(x.data) + (first + min(row, n - 1)) * x.row + head * x.head;
#pragma unroll
  for (int s = 0; s < D / Op<T>::STEP; ++s) {
    const int d = s * Op<T>::STEP + h * Op<T>::EPL;
    const bool ok = row < n && d < dim;
    const frag y = *reinterpret_cast<const frag*>(p + (ok ? d : 0));
    f[s] = ok ? y : frag{};
  }
}

// A lane's column into a tile of its wave's own, to be read as rows_by_d of row r0.
template <typename T, int D>
__device__ __forceinline__ void put_column(uint32_t at, const typename Op<T>::frag (&f)[D / Op<T>::STEP]) {
#pragma unroll
  for (int s = 0; s < D / Op<T>::STEP; ++s) lds_write(at ^ (uint32_t)(2 * s) << 4, f[s]);
  own_lds();
}

// A block of scores whose columns are such a tile's (at their place and rows_lane).
template <typename T, int D>
__device__ __forceinline__ f32x16 scores(uint32_t at, uint32_t col_at, f32x16 acc) {
#pragma unroll
  for (int s = 0; s < D / Op<T>::STEP; ++s)
    acc = Op<T>::mul(LdsTile<T, D, 32>::rows_by_d(at, 0, s), LdsTile<T, D, 32>::rows_by_d(col_at, 0, s), acc);
  in_turn<D / Op<T>::STEP, Op<T>::MULS, 2, 3>();
  return acc;
}

// A block of scores: rows r0 .. r0 + 31 of a tile (at: its place and rows_lane)
// against the lanes' columns.
template <typename T, int D>
__device__ __forceinline__ f32x16 scores(uint32_t at, int r0, const typename Op<T>::frag (&col)[D / Op<T>::STEP], f32x16 acc) {
#pragma unroll
  for (int s = 0; s < D / Op<T>::STEP; ++s) acc = Op<T>::mul(LdsTile<T, D, 32>::rows_by_d(at, r0, s), col[s], acc);
  in_turn<D / Op<T>::STEP, Op<T>::MULS, 1, 4>();
  return acc;
}

// acc^T += tile^T w: rows r0 .. r0 + 31 of a tile (at: its place and d_lane) by the
// lanes' columns of weights, values 32 D0 ..
template <typename T, int D, int D0, int DN, int AHEAD>
__device__ __forceinline__ void contract(uint32_t at, int r0, const float (&w)[16], f32x16 (&acc)[DN]) {
#pragma unroll
  for (int s = 0; s < 32 / Op<T>::STEP; ++s) {
    const typename Op<T>::frag b = Op<T>::pack(w + s * Op<T>::EPL);
#pragma unroll
    for (int dt = 0; dt < DN; ++dt) acc[dt] = Op<T>::mul(LdsTile<T, D, 32>::d_by_rows(at, r0, D0 + dt, s), b, acc[dt]);
  }
  in_turn<32 / Op<T>::STEP * DN, Op<T>::MULS, Op<T>::TURNED, AHEAD>();
}

// Two columns of weights by the same rows.
template <typename T, int D>
__device__ __forceinline__ void contract_two(uint32_t at, const float (&w)[16], f32x16 (&acc)[D / 32], const float (&w2)[16],
                                             f32x16 (&acc2)[D / 32]) {
#pragma unroll
  for (int s = 0; s < 32 / Op<T>::STEP; ++s) {
    const typename Op<T>::frag b = Op<T>::pack(w + s * Op<T>::EPL), b2 = Op<T>::pack(w2 + s * Op<T>::EPL);
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) {
      const typename Op<T>::frag f = LdsTile<T, D, 32>::d_by_rows(at, 0, dt, s);
      acc[dt] = Op<T>::mul(f, b, acc[dt]);
      acc2[dt] = Op<T>::mul(f, b2, acc2[dt]);
    }
  }
  in_turn<32 / Op<T>::STEP * (D / 32), 2 * Op<T>::MULS, Op<T>::TURNED, 2>();
}

// What rows `from` .. `upto` - 1 of x hold that is not finite, for the columns that see them
// (weights are positive): tiles that not all columns see are held without it, for 0 times
// that is not 0.  Rare.
template <typename T, int DN, typename Seen>
__device__ __forceinline__ void add_odd(const HeadsView& x, int64_t first, int head, int from, int upto, int dim, int d0,
                                        f32x16 (&acc)[DN], Seen seen) {
  const int h = (threadIdx.x & 63) >> 5;
#pragma clang loop unroll(disable)
  for (int r = from; r < upto; ++r) {
    if (!seen(r)) continue;
    const T* p = static_cast<const T*>(x.data) + (first + r) * x.row + head * x.head;
#pragma unroll
    for (int dt = 0; dt < DN; ++dt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = d0 + 32 * dt + 8 * i + 4 * h;
        if (d >= dim) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float y = Op<T>::value(p[d + j]);
          acc[dt][4 * i + j] += (__float_as_uint(y) & 0x7F800000u) == 0x7F800000u ? y : 0.0f;
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// Four neighbouring values of a lane's row of results.
template <typename T, int DN>
__device__ __forceinline__ void store_column(const HeadsView& x, int64_t first, int head, int row, int dim, int d0,
                                             const f32x16 (&acc)[DN], float by) {
  const int h = (threadIdx.x & 63) >> 5;
  T* p = static_cast<T*>(x.data) + (first + row) * x.row + head * x.head;
#pragma unroll
  for (int dt = 0; dt < DN; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = d0 + 32 * dt + 8 * i + 4 * h;
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = acc[dt][4 * i + j] * by;
      if (d < dim) store4(p + d, y);
    }
}

// Results of four waves that had a part of the same columns' sums each: this wave's
// into `all`, and after a barrier the sum of all four of the blocks that are its own.
template <int DN>
struct JoinLds { f32x4 b[4][DN][4][64]; };

template <int DN>
__device__ __forceinline__ void put_part(JoinLds<DN>& all, const f32x16 (&acc)[DN], float by) {
  const int lane = threadIdx.x & 63, wave = (threadIdx.x >> 6) & 3;
#pragma unroll
  for (int dt = 0; dt < DN; ++dt)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      all.b[wave][dt][i][lane] = f32x4{acc[dt][4 * i] * by, acc[dt][4 * i + 1] * by, acc[dt][4 * i + 2] * by, acc[dt][4 * i + 3] * by};
}

template <int DN>
__device__ __forceinline__ f32x16 joined(const JoinLds<DN>& all, int dt) {
  const int lane = threadIdx.x & 63;
  f32x16 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f32x4 x = all.b[0][dt][i][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) x += all.b[w][dt][i][lane];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[4 * i + j] = x[j];
  }
  return y;
}

kronq_status prompt_attention_launch(const PromptArgs& a, int32_t dtype, hipStream_t s);
size_t prompt_grad_ws_bytes(int64_t rows, int q_heads);
kronq_status prompt_grad_launch(const PromptArgs& a, int32_t dtype, hipStream_t s);

}  // namespace kronq
