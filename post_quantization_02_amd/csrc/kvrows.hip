// Attention over the 4-bit paged cache for sequences with many rows (a prompt
// that enters in pieces, a long draft): tiles of 32 WAVES rows x share of one key
// head, waves of 32 rows that share each tile of 64 keys.
//
// The codes of a tile are unpacked once, into LDS, as fp16 codes minus zero
// points, while the tile before is multiplied, by each wave some keys: keys as rows
// of dim values, values transposed as rows of 64 keys.  Both are read as whole
// 16-byte operands of the 32x32x16 products:
//   S^T = K Q^T: lane (row, h) gets, of each 16 keys, the eight keys 8 h and up
//     (the LDS rows of the keys are ordered for that),
//   O^T = V^T P^T: which are its k slots, so weights stay in registers.
// The 16-byte pieces of an LDS row are exchanged so that sixteen lanes that read or
// write at once use all banks.
//
// FOLD (bf16 results): the scales, too, go into the fp16 operands, as s 2^-e with
// e of the tile's largest scale; that costs two roundings (2^-11) of each key and
// value next to the result's 2^-8, and saves a product a score and two a weight.
// Keys whose scales are too far below the tile's largest to be held beside it
// (2^kKeySpread, 2^kValueSpread) are left for another pass over the tile, with an
// exponent of their own: no key's scale costs another key's precision.
// Otherwise scores and weights are multiplied in fp32 as in the kernel of few
// rows.
#include "kvattn.h"

#include <utility>

namespace kronq {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));

constexpr int KT = 64;

// FOLD.  Scales of a pass are in 2^-kKeySpread (2^-kValueSpread) to 1 of the
// largest, which times 2^-e is in [2^(kFoldSet - 1), 2^kFoldSet): times a code of
// at most 15 all are normal fp16 numbers.  Weights are up to 2^(kUp + kLazy), so
// normal ones reach 2^-(14 + kUp) of the row's largest: what is less precise than
// that, times a value 2^kValueSpread larger than the largest's, is below 2^-11 of
// the row's largest product.
constexpr int kFoldSet = 10, kKeySpread = 20, kValueSpread = 8, kUp = 6;

// How a tile goes to LDS.  Each wave takes kKeys keys: kParts lanes a key, kWords
// words of it each, as codes are loaded.  Values are unpacked by eight keys a lane,
// of them kVals values each, after an exchange within the wave.
template <int DIM, int WAVES>
struct Split {
  static constexpr int kKeys = KT / WAVES, kParts = 64 / kKeys, kWords = DIM / 8 / kParts;
  static constexpr int kCols = 64 / (kKeys / 8), kVals = DIM / kCols;
  // Where a piece (eight values of a key, or of eight keys a value) stands in its row:
  // sixteen neighbouring rows' same pieces lie in all 64 banks (256 bytes)
  __device__ static constexpr int key_piece(int piece, int row) {
    return DIM == 64 ? value_piece(piece, row) : piece ^ (row & 15);
  }
  __device__ static constexpr int value_piece(int piece, int d) { return piece ^ ((d ^ (d >> 3)) & 7); }
};

template <int DIM, int WAVES>
struct Raw {
  uint32_t k[Split<DIM, WAVES>::kWords], v[Split<DIM, WAVES>::kWords];
  uint32_t kw, vw;                        // grid words of key `lane`
  bool bad;                               // its page is out of range
};

// `n` words (a power of two) from memory that is aligned to them
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    *reinterpret_cast<u32x2*>(w) = *reinterpret_cast<const u32x2*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<u32x4*>(w + i) = *reinterpret_cast<const u32x4*>(p + 4 * i);
  }
}

// Asks for a tile's data.  `at` is the page of key `lane` or, WHOLE, of the tile.
template <int DIM, int WAVES>
__device__ __forceinline__ void load_raw(const KvView& c, PageAt at, bool whole, int head, int key0, int wave,
                                         Raw<DIM, WAVES>& t) {
  using S = Split<DIM, WAVES>;
  const int lane = threadIdx.x & 63, in_page = (1 << c.lgp) - 1;
  const int64_t head0 = (int64_t)head << c.lgp;
  const int key = wave * S::kKeys + lane / S::kParts;
  const int page = whole ? at.page : __shfl(at.page, key);
  const int64_t part = (head0 + ((key0 + key) & in_page)) * (DIM / 2) + lane % S::kParts * (4 * S::kWords);
  load_words(c.kc + page_offset(page, c.kcs) + part, t.k);
  load_words(c.vc + page_offset(page, c.vcs) + part, t.v);
  const int64_t slot = head0 + ((key0 + lane) & in_page);
  t.kw = c.kg[page_offset(at.page, c.kgs) + slot];
  t.vw = c.vg[page_offset(at.page, c.vgs) + slot];
  t.bad = at.bad;                         // for later: what is loaded is not waited for here
}

// Exponent of a grid word's scale (scale < 2^(x - 126)); 0 for one that is zero or
// not finite.
__device__ inline int exponent_of(uint32_t word) {
  const int x = (int)((word >> 23) & 0xFF);
  return x == 255 ? 0 : x;
}

// The n lowest bits (all for n > 31, none for n < 1).
__device__ inline uint32_t below(int n) { return n > 31 ? ~0u : n < 1 ? 0u : (1u << n) - 1; }

// A pass over a tile: the keys in it (bit: key of the tile) and, for FOLD, the
// exponents of what is in LDS.
struct Pass {
  int key0, ke, ve;
  uint64_t keys;
};

// FOLD: the largest exponents of scales that the current ke and ve were made for
// (0: none yet).  They stay while all keys fit them.
struct Most { int k, v; };

template <int DIM, bool FOLD>
struct Tile {
  alignas(16) _Float16 k[KT][DIM];
  alignas(16) _Float16 v[DIM][KT];
  alignas(16) float ks[FOLD ? 4 : KT];
  alignas(16) float vs[FOLD ? 4 : KT];
};

// What unpacking wants to know of key `lane`: its zero points, and for FOLD its
// scales times 2^-e as fp16 in the upper halves (0 for a key of another pass).
struct KeyInfo { uint32_t k, v; };

// Which keys of a tile's `left` the next pass takes: all of them unless FOLD.
template <int DIM, int WAVES, bool FOLD>
__device__ __forceinline__ Pass choose(const Raw<DIM, WAVES>& t, int key0, uint64_t& left, Most& most, KeyInfo& info) {
  const int lane = threadIdx.x & 63;
  Pass pass{key0, 0, 0, left};
  uint32_t kw = t.bad ? 0x7FC00000u : t.kw, vw = t.bad ? 0x7FC00000u : t.vw;
  info = {kw & 15, vw & 15};
  if constexpr (FOLD) {
    // a value scale that is not finite makes its key's scores not numbers, which
    // reaches the rows that see the key and no others
    const bool odd = (vw & 0x7F800000u) == 0x7F800000u;
    kw = odd || (kw & 0x7F800000u) == 0x7F800000u ? 0x7FC00000u : kw;
    vw = odd ? 0 : vw;
    const int kx = exponent_of(kw), vx = exponent_of(vw);
    auto fits = [](int x, int largest, int spread) __attribute__((always_inline)) {
      return (x == 0) | ((uint32_t)(largest - x) <= (uint32_t)spread);
    };
    bool in = (left >> lane) & 1;
    if (__ballot(in & !(fits(kx, most.k, kKeySpread) & fits(vx, most.v, kValueSpread)))) {
      most.k = wave_max(in ? kx : 0);
      in = in && fits(kx, most.k, kKeySpread);
      most.v = wave_max(in ? vx : 0);
      in = in && fits(vx, most.v, kValueSpread);
    }
    pass.keys = __ballot(in);
    pass.ke = most.k - 126 - kFoldSet;
    pass.ve = most.v - 126 - kFoldSet;
    auto half = [&](uint32_t word, int e) __attribute__((always_inline)) {
      const _Float16 s = (_Float16)ldexpf(__uint_as_float(word & ~15u), -e);
      return in ? (uint32_t)__builtin_bit_cast(uint16_t, s) << 16 : 0u;
    };
    info.k |= half(kw, pass.ke);
    info.v |= half(vw, pass.ve);
  }
  left &= ~pass.keys;
  return pass;
}

// A wave issues in order, and the compiler would put all vector work behind all
// products (or one operand read before each product): the order that fills both
// pipes is written out, and this keeps it.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// f(0), .., f(N - 1), each with a constant: register arrays want constant indices
// before loops are unrolled.
template <typename F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
  each_of(f, std::make_integer_sequence<int, N>{});
}

// Unpacking a wave's keys of one tile, cut into pieces to go between products: a
// word of a key each, then a pair of keys' kVals (at most four) values each.
template <int DIM, int WAVES, bool FOLD>
struct Unpacking {
  using S = Split<DIM, WAVES>;
  static constexpr int kRuns = (S::kVals + 3) / 4;    // of up to four values
  static constexpr int kPieces = S::kWords + 4 * kRuns;
  half2_t kz1, kz2, kby;
  half2_t z1[4], z2[4], by[4];
  u32x4 v0, v1, v2, v3;                               // of four values, pairs of keys
  uint32_t raw[8 * ((S::kVals + 7) / 8)];             // of each of eight keys, this lane's values

  // `mine`: LDS of the wave's own, for its keys' values
  __device__ __forceinline__ void begin(const KeyInfo& info, int wave, uint8_t* __restrict__ mine, const Raw<DIM, WAVES>& t) {
    const int lane = threadIdx.x & 63, group = lane / S::kCols;
#pragma unroll
    for (int w = 0; w < S::kWords; w += S::kWords < 4 ? S::kWords : 4) {
      uint8_t* p = mine + 4 * S::kWords * lane + 4 * w;
      if constexpr (S::kWords == 1) *reinterpret_cast<u32_alias*>(p) = t.v[0];
      else if constexpr (S::kWords == 2) *reinterpret_cast<u32x2_alias*>(p) = u32x2_alias{t.v[0], t.v[1]};
      else *reinterpret_cast<u32x4_alias*>(p) = u32x4_alias{t.v[w], t.v[w + 1], t.v[w + 2], t.v[w + 3]};
    }
    const uint32_t c = __shfl(info.k, wave * S::kKeys + lane / S::kParts), z = c & 0xFFFF;
    kz1 = as_half2(zero1024_of(z));
    kz2 = as_half2(zero64_of(z));
    kby = as_half2(__builtin_amdgcn_perm(c, c, 0x03020302u));
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t a, b;
      if constexpr (S::kCols == 64) {                 // the same eight keys for all lanes
        a = __builtin_amdgcn_readlane(info.v, wave * S::kKeys + 2 * x);
        b = __builtin_amdgcn_readlane(info.v, wave * S::kKeys + 2 * x + 1);
      } else {
        a = __shfl(info.v, wave * S::kKeys + 8 * group + 2 * x);
        b = __shfl(info.v, wave * S::kKeys + 8 * group + 2 * x + 1);
      }
      const uint32_t z = (a & 0xFFFF) | (b << 16);
      z1[x] = as_half2(z | 0x64006400u);
      z2[x] = as_half2((z << 4) | 0x54005400u);
      by[x] = as_half2((a >> 16) | (b & 0xFFFF0000u));
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint8_t* p = mine + (8 * group + j) * (DIM / 2) + lane % S::kCols * S::kVals / 2;
      if constexpr (S::kVals == 1) raw[j] = lane & 1 ? *p >> 4 : *p;
      else if constexpr (S::kVals == 2) raw[j] = *p;
      else if constexpr (S::kVals == 4) raw[j] = *reinterpret_cast<const u16_alias*>(p);
      else if constexpr (S::kVals == 8) raw[j] = *reinterpret_cast<const u32_alias*>(p);
      else raw[2 * j] = reinterpret_cast<const u32_alias*>(p)[0], raw[2 * j + 1] = reinterpret_cast<const u32_alias*>(p)[1];
    }
  }

  template <int W>
  __device__ __forceinline__ void piece(int wave, const Unpacker& un, const Raw<DIM, WAVES>& t,
                                        Tile<DIM, FOLD>* __restrict__ out) {
    const int lane = threadIdx.x & 63;
    if constexpr (W < S::kWords) {
      const int key = wave * S::kKeys + lane / S::kParts, part = lane % S::kParts;
      // bits 2 and 3 exchanged: see the scores' layout
      const int row = (key & ~12) | ((key & 4) << 1) | ((key & 8) >> 1);
      half8_t x = un.word(t.k[W], kz1, kz2);
      if constexpr (FOLD) x *= __builtin_shufflevector(kby, kby, 0, 1, 0, 1, 0, 1, 0, 1);
      *reinterpret_cast<half8_t*>(&out->k[row][8 * S::key_piece(part * S::kWords + W, row)]) = x;
    } else {
      // keys 2 x and 2 x + 1, values 4 n and up
      constexpr int n = (W - S::kWords) / 4, x = (W - S::kWords) % 4;
      const int kg = wave * (S::kKeys / 8) + lane / S::kCols, col = lane % S::kCols;
      const uint32_t wa = S::kVals > 8 ? raw[4 * x + (n >> 1)] : raw[2 * x];
      const uint32_t wb = S::kVals > 8 ? raw[4 * x + 2 + (n >> 1)] : raw[2 * x + 1];
      const uint32_t p = __builtin_amdgcn_perm(wb, wa, n & 1 ? 0x07060302u : 0x05040100u);
      auto put = [&](half2_t pair) __attribute__((always_inline)) {
        if constexpr (FOLD) pair *= by[x];
        return __builtin_bit_cast(uint32_t, pair);
      };
      v0[x] = put(un.low_pair(p, z1[x]));
      if constexpr (S::kVals > 1) v1[x] = put(un.high_pair(p, z2[x]));
      if constexpr (S::kVals > 2) {
        v2[x] = put(un.low_pair(p >> 8, z1[x]));
        v3[x] = put(un.high_pair(p >> 8, z2[x]));
      }
      if constexpr (x == 3) {
        const int d = col * S::kVals + 4 * n;
        auto store = [&](int y, u32x4 v) __attribute__((always_inline)) {
          *reinterpret_cast<half8_t*>(&out->v[d + y][8 * S::value_piece(kg, d + y)]) = __builtin_bit_cast(half8_t, v);
        };
        store(0, v0);
        if constexpr (S::kVals > 1) store(1, v1);
        if constexpr (S::kVals > 2) {
          store(2, v2);
          store(3, v3);
        }
      }
    }
  }
};

// One stage: the scores of the tile `cur`, and the next tile's codes into `out`.
// Operands are read a step ahead (further ahead there are no registers).
template <int DIM, int WAVES, bool FOLD, int PARTS, bool QLDS>
__device__ __forceinline__ void scores_and_unpack(const Tile<DIM, FOLD>* __restrict__ cur, Tile<DIM, FOLD>* __restrict__ out,
                                                  const Unpacker& un, const Raw<DIM, WAVES>& t,
                                                  const KeyInfo& info, int wave, uint8_t* __restrict__ mine,
                                                  const half8_t (&q1)[DIM / 16],
                                                  const half8_t (&q2)[PARTS > 1 ? DIM / 16 : 1],
                                                  const half8_t (*__restrict__ lds_q)[64], f32x16 (&sc)[2]) {
  using S = Split<DIM, WAVES>;
  constexpr int KS = DIM / 16, AHEAD = 1, RING = AHEAD + 1;
  const int lane = threadIdx.x & 63, i = lane & 31, h = lane >> 5;
  half8_t kv[RING][2], second[QLDS ? RING : 1];
  auto read = [&](int k) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
      kv[k % RING][s] = *reinterpret_cast<const half8_t*>(&cur->k[32 * s + i][8 * S::key_piece(2 * k + h, 32 * s + i)]);
    if constexpr (QLDS) second[k % RING] = lds_q[k][lane];
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) read(k);
  Unpacking<DIM, WAVES, FOLD> work;
  work.begin(info, wave, mine, t);
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int x = 0; x < 16; ++x) sc[s][x] = 0;
  in_order();
  // half step `at`: a product (or two) and its share of the pieces
  each<2 * KS>([&](auto at) __attribute__((always_inline)) {
    constexpr int k = at / 2, s = at % 2, N = Unpacking<DIM, WAVES, FOLD>::kPieces;
    if constexpr (s == 0 && k + AHEAD < KS) read(k + AHEAD);
    sc[s] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kv[k % RING][s], q1[k], sc[s], 0, 0, 0);
    if constexpr (PARTS > 1)
      sc[s] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kv[k % RING][s], QLDS ? second[QLDS ? k % RING : 0] : q2[PARTS > 1 ? k : 0],
                                                     sc[s], 0, 0, 0);
    each<N>([&](auto w) __attribute__((always_inline)) {
      if constexpr (w * 2 * KS / N == at) work.template piece<w>(wave, un, t, out);
    });
    in_order();
  });
}

// Bound by the vector pipes (the exponentials and what surrounds them, and
// unpacking: by the counters 400 operations a wave and 64 keys at dim 128 in bf16,
// 660 in fp16) and the matrix cores (32 products of 32 cycles, 64 where operands are
// in two parts) together, of which two waves on a SIMD overlap little, for one
// barrier a pass keeps all in one phase; LDS conflicts are 2 % of it.  2047 + 1774
// rows x 4 of 8 key heads behind 9001 and 4830 keys: 540 us, 700 TFLOP/s, and 570 once
// the clock has fallen under a run of such launches; fp16 in a window of 2048: 200 us
// (180 with weights in one part, whose error against 64 bits was 0.0003, not 0.0002).
// Dim 256 keeps 70 registers in scratch in fp32 and fp16.
template <int DIM, typename T, int PARTS, bool FOLD, int WAVES>
__global__ __launch_bounds__(64 * WAVES, DIM == 256 || (DIM == 128 && PARTS > 1 && WAVES == 4) ? 1 : 2)
void kv_attention_rows(AttnView a) {
  using S = Split<DIM, WAVES>;
  constexpr int BM = 32 * WAVES, KS = DIM / 16, VT = DIM / 32;
  constexpr bool QLDS = PARTS > 1 && DIM == 128 && WAVES == 8;   // queries' second parts: no registers left
  __shared__ Tile<DIM, FOLD> lds[2];
  __shared__ half8_t lds_q[QLDS ? WAVES : 1][QLDS ? KS : 1][64];
  __shared__ __align__(16) uint8_t packed[WAVES][256 * S::kWords];
  Unit u;
  // key heads are the faster index, so that workgroups on one XCD read few heads;
  // later row tiles see more keys: they come first
  const int head = blockIdx.x % a.c.heads, unit = a.cut.units - 1 - (int)(blockIdx.x / a.c.heads);
  if (!find_unit<BM, KT>(a, unit, false, u)) return;
  const int tid = threadIdx.x, lane = tid & 63, i = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int pos_lo, pos_hi;
  const Span span = span_of(a.c, a.shape, u, BM, KT, pos_lo, pos_hi);
  int v0, v1;
  chunk_of(span, u, v0, v1);
  const int share = a.shape.share, window = a.shape.window, sinks = a.shape.sinks;
  const int32_t* table = a.c.table + (int64_t)u.b * a.c.ldt;

  // this lane's query row, and the positions of the wave's 32
  const int r0 = u.qtile * BM + 32 * wave, r = r0 + i, pos0 = u.ctx - u.len;
  const int pos = pos0 + min(r / share, u.len - 1);
  const int wave_lo = pos0 + min(r0 / share, u.len - 1), wave_hi = pos0 + min((r0 + 31) / share, u.len - 1);
  half8_t q1[KS], q2[PARTS > 1 ? KS : 1];
  const float f = load_query<T, PARTS, KS, 2>(a, u, head, r, 8 * h, 16, q1, q2);
  if constexpr (QLDS) {
#pragma unroll
    for (int k = 0; k < KS; ++k) lds_q[wave][k][lane] = q2[k];
  }

  f32x16 o[VT];
#pragma unroll
  for (int k = 0; k < VT; ++k)
#pragma unroll
    for (int x = 0; x < 16; ++x) o[k][x] = 0;
  float m = -INFINITY, l = 0;                         // of f S; l of this lane's keys
  int e = kLeast;                                     // not FOLD: O is held times 2^-e
  float rest = 0;                                     // what rounding m left of f S
  float d = -INFINITY;                                // FOLD: O is held times 2^(kUp - m - d)

  // The tile `at` on its way to LDS, and its keys that are still to go there.  What
  // is asked for is asked for every time, the last tile again behind the end: see
  // the kernel of few rows.
  const Unpacker un;
  Raw<DIM, WAVES> raw;
  const bool whole = a.c.lgp >= 6;                    // pages hold whole tiles
  int at = v0;
  auto tile_key = [&](int v) __attribute__((always_inline)) { return key_of(span, min(v, v1 - 1), KT); };
  auto page_key = [&](int v) __attribute__((always_inline)) { return tile_key(v) + (whole ? 0 : lane); };
  auto unseen = [&]() __attribute__((always_inline)) {      // keys of tile `at` that some row sees
    const int key = tile_key(at) + lane;
    return (uint64_t)__ballot(key <= pos_hi && (!window || key > pos_lo - window || key < sinks));
  };
  Most most{0, 0};
  PageAt here{0, true};                               // of tile `at` (WHOLE), or of its key `lane`
  int next = -1;                                      // the table's entry of the tile after it
  uint64_t left = 0;
  if (v0 < v1) {
    here = page_at(a.c, table, page_key(v0));
    next = page_entry(a.c, table, page_key(v0 + 1));
    left = unseen();
  }
  KeyInfo info{};
  f32x16 sc[2];
  // chooses the next pass, for the buffer `to`
  auto take = [&](int to) __attribute__((always_inline)) {
    if constexpr (!FOLD)
      if (wave == 0) {
        lds[to].ks[lane] = raw.bad ? kNan : __uint_as_float(raw.kw & ~15u);
        lds[to].vs[lane] = raw.bad ? kNan : __uint_as_float(raw.vw & ~15u);
      }
    return choose<DIM, WAVES, FOLD>(raw, tile_key(at), left, most, info);
  };
  // the scores of the buffer `from` and the chosen pass into the other; when a tile
  // has gone there the next one's data are asked for
  auto stage = [&](int from) __attribute__((always_inline)) {
    scores_and_unpack<DIM, WAVES, FOLD, PARTS, QLDS>(&lds[from], &lds[from ^ 1], un, raw, info, wave, packed[wave], q1, q2,
                                                  lds_q[QLDS ? wave : 0], sc);
    if (!left) {
      ++at;
      here = page_from(a.c, next, page_key(at));
      left = unseen();
    }
    load_raw<DIM, WAVES>(a.c, here, whole, head, tile_key(at), wave, raw);
    next = page_entry(a.c, table, page_key(at + 1));
  };
  Pass cur{};
  bool more = v0 < v1;
  if (more) {
    load_raw<DIM, WAVES>(a.c, here, whole, head, tile_key(at), wave, raw);
    cur = take(0);
    stage(1);                                         // no scores yet
  }
  __syncthreads();
  for (int buf = 0; more; buf ^= 1) {
    const Tile<DIM, FOLD>& tile = lds[buf];
    const Pass pass = cur;
    const int key0 = pass.key0;
    more = at < v1;
    if (more) cur = take(buf ^ 1);
    stage(buf);                                       // past the last tile: its data again, which nobody reads
    {
      // entry x of sc[s] is key 32 s + 16 (x / 8) + 8 h + x % 8 of the tile
      // scores are ff sc (ff > 0, or not a number)
      const float ff = FOLD && f == f ? fmaxf(ldexpf(f, pass.ke), 0x1p-126f) : f;
      if constexpr (!FOLD) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int x = 0; x < 16; ++x) sc[s][x] *= tile.ks[32 * s + 16 * (x >> 3) + 8 * h + (x & 7)];
      }
      if (key0 + KT - 1 > wave_lo || (window && key0 <= wave_hi - window && key0 + KT > sinks) || ~pass.keys) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int first = key0 + 32 * s + 8 * h;    // bit b: key first + b
          uint32_t seen = below(pos - first + 1) & ((uint32_t)(pass.keys >> (32 * s)) >> (8 * h));
          if (window) seen &= ~below(pos - window + 1 - first) | below(sinks - first);
#pragma unroll
          for (int x = 0; x < 16; ++x) sc[s][x] = seen & (1u << (16 * (x >> 3) + (x & 7))) ? sc[s][x] : -INFINITY;
        }
      }
      float top = sc[0][0];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int x = 0; x < 16; ++x) top = fmaxf(top, sc[s][x]);
      const float mine = top * ff;
      if (__any(mine > m + kLazy || (m == -INFINITY && mine > m) || (FOLD && mine - m + (float)pass.ve > d + kLazy))) {
        top = fmaxf(top, __shfl_xor(top, 32));
        const float row = top * ff, nm = fmaxf(row, m);
        const float nrest = row > m ? fmaf(top, ff, -row) : rest;
        if (m != -INFINITY) {
          const float far = fmaxf(nm - m + (nrest - rest), 0.0f), down = fminf(far, 300.0f);
          float by = __builtin_amdgcn_exp2f(-down);
          l *= by;
          if constexpr (FOLD) {
            const float nd = fmaxf(row - nm + (float)pass.ve, d - far);
            by = __builtin_amdgcn_exp2f(fmaxf(d - far - nd, -300.0f));
            d = nd;
          } else {
            const int ne = max(e - (int)ceilf(down), kLeast);
            by = __builtin_amdgcn_exp2f((float)(e - ne) - down);
            e = ne;
          }
#pragma unroll
          for (int k = 0; k < VT; ++k) o[k] *= by;
        } else if (FOLD && nm != -INFINITY) {
          d = (float)pass.ve;
        }
        m = nm;
        rest = nrest;
      }
      // Weights are 2^(ff sc - base + up).  FOLD: as O is held; times 2^-up they are the
      // sum's, and where that is too far for one fp32 number to do for both (`far`),
      // they are added up by themselves.  Otherwise: times 2^-ue, the part of the row's
      // factor that they can carry (none before the first is known).
      const int ue = e == kLeast ? 0 : min(max(e, -60), 30);
      const float up = !FOLD ? -(float)ue : d == -INFINITY ? 0.0f : (float)(pass.ve + kUp) - d;
      const bool far = FOLD && __any(-up > 60.0f);
      float base = m == -INFINITY ? 0.0f : m, fx = ff;
      if (__any(fabsf(base) > kSteep)) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int x = 0; x < 16; ++x) sc[s][x] = fmaf(sc[s][x], ff, -base) - rest;
        base = 0;
        fx = 1;
      }
      const float off = up - base;
      float sum = 0, apart = 0;
      if (far) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int x = 0; x < 16; ++x) apart += __builtin_amdgcn_exp2f(fmaf(sc[s][x], fx, -base));
      }
      if constexpr (!FOLD) {
        float ytop = 0;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float p = __builtin_amdgcn_exp2f(fmaf(sc[s][x], fx, off));
            sum += p;
            const bool seen = sc[s][x] != -INFINITY;  // not seen: whatever scale is there
            sc[s][x] = seen ? p * tile.vs[32 * s + 16 * (x >> 3) + 8 * h + (x & 7)] : 0.0f;
            ytop = fmaxf(ytop, fabsf(sc[s][x]));      // a grid's scale may be below 0
          }
        if (__any(ytop > ldexpf(1.0f, min(kTop + e - ue, 127)))) {
          ytop = fmaxf(ytop, __shfl_xor(ytop, 32));
          if (ytop > ldexpf(1.0f, min(kTop + e - ue, 127))) {
            const int ne = min(max(exponent_for(ytop) + ue, kLeast), kMost);
            const float by = ldexpf(1.0f, e - ne);
#pragma unroll
            for (int k = 0; k < VT; ++k) o[k] *= by;
            e = ne;
          }
        }
        if (__any(e != ue)) {
          const float by = ldexpf(1.0f, ue - e);
#pragma unroll
          for (int s = 0; s < 2; ++s) sc[s] *= by;
        }
      }
      // Sixteen keys at a time: their products, and between them the next sixteen's
      // weights.
      half8_t p1[2], p2[PARTS > 1 ? 2 : 1], vv[2][VT];
      auto weigh = [&](int n, int x) __attribute__((always_inline)) {
        float y = sc[n >> 1][8 * (n & 1) + x];
        if constexpr (FOLD) {
          y = __builtin_amdgcn_exp2f(fmaf(y, fx, off));
          sum += y;
        }
        p1[n & 1][x] = (_Float16)y;
        if constexpr (PARTS > 1) p2[n & 1][x] = (_Float16)(y - (float)p1[n & 1][x]);
      };
      auto read = [&](int n) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < VT; ++k) {
          const int d = 32 * k + i;
          vv[n & 1][k] = *reinterpret_cast<const half8_t*>(&tile.v[d][8 * S::value_piece(2 * n + h, d)]);
        }
      };
      read(0);
#pragma unroll
      for (int x = 0; x < 8; ++x) weigh(0, x);
      in_order();
      each<4 * VT>([&](auto at) __attribute__((always_inline)) {
        constexpr int n = at / VT, k = at % VT;
        if constexpr (n < 3 && k == 0) read(n + 1);
        o[k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv[n & 1][k], p1[n & 1], o[k], 0, 0, 0);
        if constexpr (PARTS > 1) o[k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv[n & 1][k], p2[PARTS > 1 ? n & 1 : 0], o[k], 0, 0, 0);
        if constexpr (n < 3) {
#pragma unroll
          for (int x = 8 * k / VT; x < 8 * (k + 1) / VT; ++x) weigh(n + 1, x);
        }
        in_order();
      });
      l += !FOLD ? sum * ldexpf(1.0f, ue) : -up > 60.0f ? apart : sum * __builtin_amdgcn_exp2f(-up);
    }
    __syncthreads();
  }

  l += __shfl_xor(l, 32);
  if (r >= u.len * share) return;
  if (pos >= room_of(a.c)) l = kNan;               // a position without a column
  // O is held times 2^-(2 back): in two steps, each within fp32
  const float back = __builtin_amdgcn_exp2f(!FOLD ? 0.5f * e : d == -INFINITY ? 0.0f : 0.5f * (d - (float)kUp));
  if (u.chunks == 1) {
    const int tok = r / share, qh = head * share + r % share;
    const float by = l == 0 ? 0.0f : back / l;      // 0 of a row that sees nothing
    T* out = static_cast<T*>(a.out.data) + (int64_t)(u.row0 + tok) * a.out.row + (int64_t)qh * a.out.head;
#pragma unroll
    for (int k = 0; k < VT; ++k)
#pragma unroll
      for (int x = 0; x < 16; x += 4) {
        float y[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) y[z] = l == 0 ? 0.0f : o[k][x + z] * back * by;
        store4(out + 32 * k + 2 * x + 4 * h, y);
      }
    if (a.lse && h == 0)
      a.lse[(int64_t)(u.row0 + tok) * a.qheads + qh] = l == 0 ? -INFINITY : (m + log2f(l)) * kLn2;
  } else if (u.place < a.places) {
    const int64_t at = ((int64_t)u.place * a.c.heads + head) * BM + 32 * wave + i;
#pragma unroll
    for (int k = 0; k < VT; ++k)
#pragma unroll
      for (int x = 0; x < 16; x += 4) {
        float y[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) y[z] = o[k][x + z] * back * back;
        store4(a.part + at * DIM + 32 * k + 2 * x + 4 * h, y);
      }
    if (h == 0) {
      a.stat[2 * at] = m;
      a.stat[2 * at + 1] = l;
    }
  }
}

template <int DIM, int WAVES>
void rows_waves(const AttnView& a, int32_t dtype, hipStream_t s) {
  const dim3 grid((unsigned)(a.c.heads * a.cut.units)), block(64 * WAVES);
  if (dtype == KRONQ_F32)
    hipLaunchKernelGGL((kv_attention_rows<DIM, float, 2, false, WAVES>), grid, block, 0, s, a);
  else if (dtype == KRONQ_BF16)
    hipLaunchKernelGGL((kv_attention_rows<DIM, bf16_t, 1, true, WAVES>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((kv_attention_rows<DIM, _Float16, 2, false, WAVES>), grid, block, 0, s, a);
}

}  // namespace

kronq_status kv_rows_launch(const AttnView& a, int dim, int32_t dtype, int waves, hipStream_t s) {
  if (dim == 64 && waves == 8) rows_waves<64, 8>(a, dtype, s);
  else if (dim == 64) rows_waves<64, 4>(a, dtype, s);
  else if (dim == 128 && waves == 8) rows_waves<128, 8>(a, dtype, s);
  else if (dim == 128) rows_waves<128, 4>(a, dtype, s);
  else rows_waves<256, 4>(a, dtype, s);
  KQ_LAUNCHED("kv_attention_rows");
  return KRONQ_OK;
}

}  // namespace kronq
