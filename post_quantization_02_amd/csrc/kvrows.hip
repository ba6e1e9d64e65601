// Attention over the 4-bit paged cache for sequences with many rows (a prompt
// that enters in pieces, a long draft): tiles of 128 rows x share of one key
// head, four waves of 32 rows that share each tile of 64 keys.
//
// The codes of a tile are unpacked once, into LDS, as fp16 codes minus zero
// points, while the tile before is multiplied: keys as rows of dim values,
// values transposed as rows of 64 keys, both read as whole 16-byte operands of
// the 32x32x16 products:
//   S^T = K Q^T: lane (row, h) gets, of each 16 keys, the eight keys 8 h and up
//     (the LDS rows of the keys are ordered for that),
//   O^T = V^T P^T: which are its k slots, so weights stay in registers.
// 16-byte pieces of an LDS row are exchanged by an exclusive or with the row, so
// that eight lanes that read or write at once use all banks.
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

namespace kronq {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));

constexpr int BM = 128, KT = 64;

// FOLD.  Scales of a pass are in 2^-kKeySpread (2^-kValueSpread) to 1 of the
// largest, which times 2^-e is in [2^(kFoldSet - 1), 2^kFoldSet): times a code of
// at most 15 all are normal fp16 numbers.  Weights are up to 2^(kUp + kLazy), so
// normal ones reach 2^-(14 + kUp) of the row's largest: what is less precise than
// that, times a value 2^kValueSpread larger than the largest's, is below 2^-11 of
// the row's largest product.
constexpr int kFoldSet = 10, kKeySpread = 20, kValueSpread = 8, kUp = 6;

// What a thread holds of a tile on its way to LDS: a quarter of one key (key
// tid / 4), and dim / 16 values of four keys (4 (tid / 16) and up).
template <int DIM>
struct Raw {
  uint32_t k[DIM / 32];
  uint32_t v[4][(DIM + 127) / 128];
  uint32_t kw, vw;         // grid words of key `lane`
};

// The page of key `lane` of a tile; a tile past the table's end is not asked for.
__device__ inline PageAt lane_page(const KvView& c, const int32_t* table, int key0) {
  return page_at(c, table, key0 + (threadIdx.x & 63));
}

template <int DIM>
__device__ inline void load_raw(const KvView& c, const PageAt& at, int head, int key0, Raw<DIM>& t) {
  const int tid = threadIdx.x, lane = tid & 63, in_page = (1 << c.lgp) - 1;
  const int packed = at.bad ? -1 : at.page;
  const int64_t head0 = (int64_t)head << c.lgp;
  {
    const int key = tid >> 2, page = max(__shfl(packed, key), 0);
    const uint8_t* p = c.kc + (int64_t)page * c.kcs + (head0 + ((key0 + key) & in_page)) * (DIM / 2) + (tid & 3) * (DIM / 8);
    if constexpr (DIM == 64) {
      *reinterpret_cast<u32x2*>(t.k) = *reinterpret_cast<const u32x2*>(p);
    } else {
#pragma unroll
      for (int w = 0; w < DIM / 32; w += 4)
        *reinterpret_cast<u32x4*>(t.k + w) = *reinterpret_cast<const u32x4*>(p + 4 * w);
    }
  }
  {
    const int key = (tid >> 4) * 4, page = max(__shfl(packed, key), 0);   // four keys share a page
    const uint8_t* p = c.vc + (int64_t)page * c.vcs + (head0 + ((key0 + key) & in_page)) * (DIM / 2) + (tid & 15) * (DIM / 32);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DIM == 64)
        t.v[j][0] = *reinterpret_cast<const uint16_t*>(p + j * (DIM / 2));
      else if constexpr (DIM == 128)
        t.v[j][0] = *reinterpret_cast<const uint32_t*>(p + j * (DIM / 2));
      else
        *reinterpret_cast<u32x2*>(t.v[j]) = *reinterpret_cast<const u32x2*>(p + j * (DIM / 2));
    }
  }
  const int64_t slot = head0 + ((key0 + lane) & in_page);
  t.kw = at.bad ? 0x7FC00000u : c.kg[(int64_t)at.page * c.kgs + slot];
  t.vw = at.bad ? 0x7FC00000u : c.vg[(int64_t)at.page * c.vgs + slot];
}

// fp16 factor of a grid word's scale times 2^-e, in both halves.
__device__ inline half2_t scale_pair(uint32_t word, int e) {
  const _Float16 h = (_Float16)ldexpf(__uint_as_float(word & ~15u), -e);
  return half2_t{h, h};
}

// Exponent of a grid word's scale (scale < 2^(x - 126)); 0 for one that is zero or
// not finite.
__device__ inline int exponent_of(uint32_t word) {
  const int x = (int)((word >> 23) & 0xFF);
  return x == 255 ? 0 : x;
}

__device__ inline int wave_max(int x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x = max(x, __shfl_xor(x, d));
  return x;
}

// A pass over a tile: the keys in it (bit: key of the tile) and, for FOLD, the
// exponents of what is in LDS.
struct Pass {
  int key0, ke, ve;
  uint64_t keys;
};

template <int DIM, bool FOLD>
struct Tile {
  _Float16 k[KT][DIM];
  _Float16 v[DIM][KT];
  float ks[FOLD ? 1 : KT], vs[FOLD ? 1 : KT];
};

// Unpacks a tile's keys in `left` into LDS, or (FOLD) those of them that fit a
// pass, and takes them out of `left`.
template <int DIM, bool FOLD>
__device__ inline Pass unpack_tile(const Unpacker& un, const Raw<DIM>& t, Tile<DIM, FOLD>& out, int key0, uint64_t& left) {
  const int tid = threadIdx.x, lane = tid & 63;
  Pass pass{key0, 0, 0, left};
  uint32_t kw = t.kw, vw = t.vw;
  if constexpr (FOLD) {
    // a value scale that is not finite makes its key's scores not numbers, which
    // reaches the rows that see the key and no others
    if ((vw & 0x7F800000u) == 0x7F800000u) kw = 0x7FC00000u, vw = 0;
    if ((kw & 0x7F800000u) == 0x7F800000u) kw = 0x7FC00000u;
    bool in = (left >> lane) & 1;
    const int kx = exponent_of(kw), vx = exponent_of(vw);
    const int kmost = wave_max(in ? kx : 0);
    in = in && (kx == 0 || kx >= kmost - kKeySpread);
    const int vmost = wave_max(in ? vx : 0);
    in = in && (vx == 0 || vx >= vmost - kValueSpread);
    pass.keys = __ballot(in);
    pass.ke = kmost - 126 - kFoldSet;
    pass.ve = vmost - 126 - kFoldSet;
    if (!in) kw = vw = 0;                             // a scale of 0
  } else if (tid < KT) {
    out.ks[lane] = __uint_as_float(kw & ~15u);
    out.vs[lane] = __uint_as_float(vw & ~15u);
  }
  left &= ~pass.keys;
  {
    const int key = tid >> 2;
    const uint32_t word = __shfl(kw, key);
    const uint32_t z = word & 15;
    const half2_t z1 = as_half2(zero1024_of(z)), z2 = as_half2(zero64_of(z));
    // bits 2 and 3 exchanged: see the scores' layout
    const int row = (key & ~12) | ((key & 4) << 1) | ((key & 8) >> 1);
    half2_t by{};
    if constexpr (FOLD) by = scale_pair(word, pass.ke);
#pragma unroll
    for (int w = 0; w < DIM / 32; ++w) {
      half8_t x = un.word(t.k[w], z1, z2);
      if constexpr (FOLD) x *= __builtin_shufflevector(by, by, 0, 1, 0, 1, 0, 1, 0, 1);
      const int piece = ((tid & 3) * (DIM / 32) + w) ^ (row & 7);
      *reinterpret_cast<half8_t*>(&out.k[row][8 * piece]) = x;
    }
  }
  {
    const int kg = tid >> 4, col = tid & 15;
    half2_t z1[2], z2[2], by[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t w0 = __shfl(vw, 4 * kg + 2 * x), w1 = __shfl(vw, 4 * kg + 2 * x + 1);
      const uint32_t z = (w0 & 15) | ((w1 & 15) << 16);
      z1[x] = as_half2(z | 0x64006400u);
      z2[x] = as_half2((z << 4) | 0x54005400u);
      if constexpr (FOLD) by[x] = half2_t{scale_pair(w0, pass.ve).x, scale_pair(w1, pass.ve).x};
    }
#pragma unroll
    for (int b = 0; b < DIM / 32; ++b) {              // byte b of the words: values 2 b, 2 b + 1
      const uint32_t sel = 0x0C000C00u | (uint32_t)(b & 3) | ((uint32_t)(4 + (b & 3)) << 16);
      half2_t lo[2], hi[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t w = __builtin_amdgcn_perm(t.v[2 * x + 1][b >> 2], t.v[2 * x][b >> 2], sel);
        lo[x] = un.low_pair(w, z1[x]);
        hi[x] = un.high_pair(w, z2[x]);
        if constexpr (FOLD) lo[x] *= by[x], hi[x] *= by[x];
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int d = col * (DIM / 16) + 2 * b + n;
        const int piece = (kg >> 1) ^ ((d ^ (d >> 3)) & 7);
        const half4_t x = n ? half4_t{hi[0].x, hi[0].y, hi[1].x, hi[1].y} : half4_t{lo[0].x, lo[0].y, lo[1].x, lo[1].y};
        *reinterpret_cast<half4_t*>(&out.v[d][8 * piece + 4 * (kg & 1)]) = x;
      }
    }
  }
  return pass;
}

// Bound by the vector pipes (the exponentials and what surrounds them) and the
// matrix cores together.
template <int DIM, typename T, int QP, int PP, bool FOLD>
__global__ __launch_bounds__(256, DIM == 256 ? 1 : 2) void kv_attention_rows(AttnView a) {
  constexpr int KS = DIM / 16, VT = DIM / 32;
  __shared__ Tile<DIM, FOLD> lds[2];
  Unit u;
  // key heads are the faster index, so that workgroups on one XCD read few heads;
  // later row tiles see more keys: they come first
  const int head = blockIdx.x % a.c.heads, unit = a.units - 1 - (int)(blockIdx.x / a.c.heads);
  if (!find_unit<BM, KT>(a, unit, false, u)) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, i = lane & 31, h = lane >> 5;
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
  half8_t q1[KS], q2[QP > 1 ? KS : 1];
  const float f = load_query<T, QP, KS, 2>(a, u, head, r, 8 * h, 16, q1, q2);

  f32x16 o[VT];
#pragma unroll
  for (int k = 0; k < VT; ++k)
#pragma unroll
    for (int x = 0; x < 16; ++x) o[k][x] = 0;
  float m = -INFINITY, l = 0;                         // of f S; l of this lane's keys
  int e = kLeast;                                     // not FOLD: O is held times 2^-e
  float ref = -INFINITY;                              // FOLD: O is held times 2^(kUp - ref)

  // the tile on its way to LDS, its keys that are still to go there, and the page
  // of the one after it
  const Unpacker un;
  Raw<DIM> raw;
  uint64_t left = 0;
  PageAt next{0, true};
  int at = v0;
  auto fetch = [&]() {                                // tile `at`, whose pages are in `next`
    if (at >= v1) return;
    const int key0 = key_of(span, at, KT), key = key0 + lane;
    load_raw<DIM>(a.c, next, head, key0, raw);
    left = __ballot(key <= pos_hi && (!window || key > pos_lo - window || key < sinks));
    if (at + 1 < v1) next = lane_page(a.c, table, key_of(span, at + 1, KT));
  };
  auto unpack = [&](int buf) {
    const Pass p = unpack_tile<DIM, FOLD>(un, raw, lds[buf], key_of(span, at, KT), left);
    if (!left) ++at, fetch();
    return p;
  };
  if (v0 < v1) next = lane_page(a.c, table, key_of(span, v0, KT));
  fetch();
  Pass cur{};
  bool more = v0 < v1;
  if (more) cur = unpack(0);
  __syncthreads();
  for (int buf = 0; more; buf ^= 1) {
    const Tile<DIM, FOLD>& tile = lds[buf];
    const Pass pass = cur;
    const int key0 = pass.key0;
    more = at < v1;
    if (more) cur = unpack(buf ^ 1);
    // some row of the wave sees some key
    if (key0 <= wave_hi && (!window || key0 + KT - 1 > wave_lo - window || key0 < sinks)) {
      f32x16 sc[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int x = 0; x < 16; ++x) sc[s][x] = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const half8_t kv = *reinterpret_cast<const half8_t*>(&tile.k[32 * s + i][8 * ((2 * k + h) ^ (i & 7))]);
          sc[s] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kv, q1[k], sc[s], 0, 0, 0);
          if constexpr (QP > 1) sc[s] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kv, q2[k], sc[s], 0, 0, 0);
        }
      }
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
          const uint32_t in = (uint32_t)(pass.keys >> (32 * s)) >> (8 * h);
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const int bit = 16 * (x >> 3) + (x & 7), j = key0 + 32 * s + 8 * h + bit;
            if (j > pos || (window && j <= pos - window && j >= sinks) || !((in >> bit) & 1)) sc[s][x] = -INFINITY;
          }
        }
      }
      float top = sc[0][0];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int x = 0; x < 16; ++x) top = fmaxf(top, sc[s][x]);
      top *= ff;
      const float vtop = FOLD ? top + (float)pass.ve : top;
      if (__any(top > m + kLazy || (m == -INFINITY && top > m) || (FOLD && vtop > ref + kLazy))) {
        const float row = fmaxf(top, __shfl_xor(top, 32)), nm = fmaxf(row, m);
        if (m != -INFINITY) {
          const float down = fminf(nm - m, 300.0f);
          float by = __builtin_amdgcn_exp2f(-down);
          l *= by;
          if constexpr (FOLD) {
            const float nref = fmaxf(row + (float)pass.ve, ref);
            by = __builtin_amdgcn_exp2f(fmaxf(ref - nref, -300.0f));
            ref = nref;
          } else {
            const int ne = max(e - (int)ceilf(down), kLeast);
            by = __builtin_amdgcn_exp2f((float)(e - ne) - down);
            e = ne;
          }
#pragma unroll
          for (int k = 0; k < VT; ++k) o[k] *= by;
        } else if (FOLD && nm != -INFINITY) {
          ref = nm + (float)pass.ve;
        }
        m = nm;
      }
      const float base = m == -INFINITY ? 0.0f : m;
      // weights are 2^(ff sc + up).  FOLD: for O; times 2^(-base - up) they are the
      // sum's, and where that is too far for one fp32 number to do for both, they
      // are added up by themselves.  Otherwise: times 2^-ue, the part of the row's
      // factor that they can carry (none before the first is known).
      const int ue = e == kLeast ? 0 : min(max(e, -60), 30);
      const float up = !FOLD ? -base - (float)ue : ref == -INFINITY ? 0.0f : (float)(pass.ve + kUp) - ref;
      float ytop = 0, sum = 0;
      if (FOLD && __any(-base - up > 60.0f)) {
        float apart = 0;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int x = 0; x < 16; ++x) apart += __builtin_amdgcn_exp2f(fmaf(sc[s][x], ff, -base));
        l += -base - up > 60.0f ? apart : 0.0f;
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float p = __builtin_amdgcn_exp2f(fmaf(sc[s][x], ff, up));
          sum += p;
          if constexpr (FOLD) {
            sc[s][x] = p;
          } else {
            const bool seen = sc[s][x] != -INFINITY;  // not seen: whatever scale is there
            sc[s][x] = seen ? p * tile.vs[32 * s + 16 * (x >> 3) + 8 * h + (x & 7)] : 0.0f;
            ytop = fmaxf(ytop, sc[s][x]);
          }
        }
      l += !FOLD ? sum * ldexpf(1.0f, ue) : -base - up > 60.0f ? 0.0f : sum * __builtin_amdgcn_exp2f(-base - up);
      if constexpr (!FOLD) {
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
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          half8_t p1, p2;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float y = sc[s][8 * j + x];
            p1[x] = (_Float16)y;
            if constexpr (PP > 1) p2[x] = (_Float16)(y - (float)p1[x]);
          }
#pragma unroll
          for (int k = 0; k < VT; ++k) {
            const int d = 32 * k + i;
            const half8_t vv = *reinterpret_cast<const half8_t*>(&tile.v[d][8 * ((4 * s + 2 * j + h) ^ ((d ^ (d >> 3)) & 7))]);
            o[k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, p1, o[k], 0, 0, 0);
            if constexpr (PP > 1) o[k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vv, p2, o[k], 0, 0, 0);
          }
        }
    }
    __syncthreads();
  }

  l += __shfl_xor(l, 32);
  if (r >= u.len * share) return;
  if (pos >= room_of(a.c)) l = kNan;               // a position without a column
  // O is held times 2^-(2 back): in two steps, each within fp32
  const float back = __builtin_amdgcn_exp2f(!FOLD ? 0.5f * e : ref == -INFINITY ? 0.0f : 0.5f * (ref - m - (float)kUp));
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
  } else {
    const int64_t at = ((int64_t)unit * a.c.heads + head) * BM + 32 * wave + i;
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

template <int DIM>
void rows_dim(const AttnView& a, int32_t dtype, hipStream_t s) {
  const dim3 grid((unsigned)(a.c.heads * a.units));
  if (dtype == KRONQ_F32)
    hipLaunchKernelGGL((kv_attention_rows<DIM, float, 2, 2, false>), grid, dim3(256), 0, s, a);
  else if (dtype == KRONQ_BF16)
    hipLaunchKernelGGL((kv_attention_rows<DIM, bf16_t, 1, 1, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((kv_attention_rows<DIM, _Float16, 2, 1, false>), grid, dim3(256), 0, s, a);
}

}  // namespace

kronq_status kv_rows_launch(const AttnView& a, int dim, int32_t dtype, hipStream_t s) {
  if (dim == 64) rows_dim<64>(a, dtype, s);
  else if (dim == 128) rows_dim<128>(a, dtype, s);
  else rows_dim<256>(a, dtype, s);
  KQ_LAUNCHED("kv_attention_rows");
  return KRONQ_OK;
}

}  // namespace kronq
