// k12_tree.cu -- attention of drafted tokens over the paged cache
// (fs_tree_attn): out = sum p v / sum p over the prefix and the drafted tokens
// that a row's mask lets it see.
//
// Rows.  The R = count * G rows of one sequence and kv head (G query heads read
// one kv head) share its keys; row r is token r / G, query head r % G.  They
// are taken M at a time.
//
// Split.  The work is cut into units of 32 keys of one (sequence, kv head, row
// tile): a segment.  All units stand in one line and every block takes an
// equal stretch of it, so that ragged batches and few long sequences alike keep
// every SM busy.  Lengths are known on the device alone: each block works out
// the line for itself.  A segment that lies in one block is written by it; of
// the others each block leaves (m, l, O) in the workspace, and a second kernel
// adds them in block order (no atomics: the same bits every time).
//
// A block's warps take the segment's units in turn, each with all M rows and
// its own running maximum, sum and output, and a ring of units in flight
// (asynchronous copies into shared memory); they are joined once a segment.
//
// Products are mma.sync m16n8k16 with fp32 sums.  A fragment may hold the
// elements of a head in any order that q and k share, and the values in any
// order of columns: so every lane reads whole 16-byte (8, 4) pieces of codes
// and turns them into fragments in registers.  Codes of 8 and 4 bits are exact
// in fp16; q is brought into fp16's range by a power of two a row (exact but
// for elements below 2^-31 of the row's largest, which are rounded at 2^-39 of it, 2^-35
// where int4's odd ones are divided by 16).  The key's scale multiplies
// the score, the value's scale the probability: a weight.
//
// Weights go into the second product as fp16 (half a step 2^-11), the row's
// largest at least 2^7: half a step of the smallest is 2^-32 of the largest; with
// bf16 values as a bf16 pair (high and low part, 2^-16).  A row's reference follows
// the largest weight of the keys that it sees, lazily (tree.cuh): a common one
// for all rows, from the largest value scale of the unit, would let values that a row
// does not see, or sees with next to no probability, take its weights out of fp16's
// range.
#include <type_traits>

#include "tree.cuh"

namespace fs {
namespace {

constexpr int kUnit = 32;  // keys of a unit
constexpr uint32_t kNone = ~0u;

// ---------------------------------------------------------------------------
// fragments
// ---------------------------------------------------------------------------
// c = a b, or c += a b (a first product takes zeros in place of c, which costs
// no moves).
template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, bool add = true) {
  const float z0 = add ? c[0] : 0.f, z1 = add ? c[1] : 0.f, z2 = add ? c[2] : 0.f,
              z3 = add ? c[3] : 0.f;
  if constexpr (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};\n"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2),
          "f"(z3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};\n"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2),
          "f"(z3));
}

// MT sixteens of rows a tile; MT = 0: eight rows.
template <int F, int D, int MT>
struct Cfg {
  static constexpr int kBits = Fmt<F>::kBits;
  static constexpr int kRow = D * kBits / 8;  // bytes of a row
  static constexpr int P = kRow / 16;         // 16-byte pieces of a row
  static constexpr int kM = MT ? 16 * MT : 8;
  static constexpr int kWarps = kRow >= 256 ? 4 : 8;
  static constexpr int kCodes = kUnit * kRow;  // bytes of a unit's keys
  // keys, values, 32 + 32 scales, which keys can be read
  static constexpr int kStage = 2 * kCodes + 8 * kUnit + 16;
  static constexpr int kCtas =
      (MT == 0 || (MT == 1 && D == 64)) && kStage * kWarps * 3 <= 112 * 1024 ? 2 : 1;
  static constexpr int kRoom = (kCtas == 2 ? 110 : 220) * 1024;
  static constexpr int kFit = kRoom / (kStage * kWarps);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kJoin = kWarps * kM * (D + 6) * 4;  // the warps' results
  static constexpr int kRing = kStage * kWarps * kStages;
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
  static constexpr bool kBF = F == FS_CACHE_BF16;
  static_assert(kStages >= 2 && kSmem <= kRoom, "ring");
};

// The lane's registers of one row of q (null: zeros), two for every k step.  Lane column c
// (lane % 4) holds the elements that its key words hold:
//   bf16          8-element pieces c, c + 4, ...
//   8 bits        16-element pieces c, c + 4
//   4 bits        elements D / 4 c ..., in every eight the pairs (0, 4), (1, 5),
//                 (2, 6), (3, 7)
template <int F, int D>
__device__ __forceinline__ void q_words(const uint16_t *row, int c, uint32_t (&raw)[D / 16][2]) {
  constexpr int N = D / 8;  // words of a lane: a quarter of the row
  uint32_t w[N];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const int piece = F == FS_CACHE_BF16   ? c + 4 * i
                      : F == FS_CACHE_INT4 ? N / 4 * c + i
                                           : 2 * (c + 4 * (i / 2)) + i % 2;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (row) u = *reinterpret_cast<const uint4 *>(row + piece * 8);
    w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
  }
#pragma unroll
  for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (F == FS_CACHE_INT4)
        raw[ks][e] = __byte_perm(w[4 * (ks / 2) + ks % 2], w[4 * (ks / 2) + 2 + ks % 2],
                                 e ? 0x7632 : 0x5410);
      else
        raw[ks][e] = w[2 * ks + e];
    }
}
// Element that column n of value tile i stands for.
template <int F, int D>
__device__ __forceinline__ int v_element(int n, int i) {
  if constexpr (D == 64) return 8 * n + i;
  if constexpr (F == FS_CACHE_BF16) return 8 * n + i % 8 + 64 * (i / 8);
  return 16 * n + i;
}
// Places of 16-byte pieces, so that the lanes that read at one time hit
// different banks: keys are read by eight neighbouring rows at once, values by
// rows two apart.
template <int P>
__device__ __forceinline__ int k_place(int r, int piece) {
  return r * P + (P >= 8 ? piece ^ (4 * (r & 1)) : piece);
}
template <int P>
__device__ __forceinline__ int v_place(int r, int piece) {
  return (r * P + piece) ^ (P >= 4 ? 2 * ((r >> 1) & 3) : 2 * ((r >> 2) & 1));
}

// The k step's two key registers from the lane's code words.  Integer codes go
// in as code + bias (128 or 8), the bits of an fp16 subnormal: (code + bias)
// 2^-24, of an odd nibble 16 times that, which its elements of q make up for.
// The bias is the same for all keys of a row of q and leaves with one addition.
// It takes bits from the fp32 sum: two where codes fill their range, five to seven
// where a key row has one outlier and its other codes are a few units.  A score is then off
// by some (d + 3) 2^-24 of |q|_1 times twice the key row's largest magnitude.  (The values'
// codes below, whose sum runs over all keys, go in without one.)
template <int F>
constexpr float kBias = F == FS_CACHE_INT8 ? 128.f : F == FS_CACHE_INT4 ? 8.f : 0.f;
template <int F>
__device__ __forceinline__ void k_regs(const Magic &m, const uint32_t *w, int s, uint32_t &b0,
                                       uint32_t &b1) {
  if constexpr (F == FS_CACHE_BF16) {
    b0 = w[2 * s];
    b1 = w[2 * s + 1];
  } else if constexpr (F == FS_CACHE_E4M3) {
    e4m3_h2(w[s], b0, b1);
  } else if constexpr (F == FS_CACHE_INT8) {
    const uint32_t x = w[s] ^ 0x80808080u;
    b0 = __byte_perm(x, 0, 0x4140);
    b1 = __byte_perm(x, 0, 0x4342);
  } else {
    const uint32_t x = w[s / 2] >> (8 * (s % 2));
    b0 = (x & m.even) ^ 0x00080008u;
    b1 = (x & m.odd) ^ 0x00800080u;
  }
}
// Value register(s) of two keys' words: the elements 2 j and 2 j + 1 of the
// lane's 8 (of word set x, y), each paired over the two keys.
template <int F>
__device__ __forceinline__ void v_regs(const Magic &m, const uint32_t *x, const uint32_t *y, int j,
                                       uint32_t &r0, uint32_t &r1) {
  if constexpr (F == FS_CACHE_BF16) {
    r0 = __byte_perm(x[j], y[j], 0x5410);
    r1 = __byte_perm(x[j], y[j], 0x7632);
  } else if constexpr (F == FS_CACHE_E4M3) {
    e4m3_h2(__byte_perm(x[j / 2], y[j / 2], j % 2 ? 0x7362 : 0x5140), r0, r1);
  } else if constexpr (F == FS_CACHE_INT8) {
    const uint32_t z = __byte_perm(x[j / 2], y[j / 2], j % 2 ? 0x7362 : 0x5140) ^ 0x80808080u;
    r0 = h2add(__byte_perm(z, m.magic, 0x7170), kSub128);
    r1 = h2add(__byte_perm(z, m.magic, 0x7372), kSub128);
  } else {
    // byte j of both keys: its low and high nibble
    const uint32_t sel = (uint32_t)(j % 4) * 0x0011u + (uint32_t)(4 + j % 4) * 0x1100u;
    const uint32_t z = __byte_perm(x[j / 4], y[j / 4], sel);
    r0 = nib_even(m, z);
    r1 = nib_odd(m, z);
  }
}

template <int N>
__device__ __forceinline__ void lds_words(const char *p, uint32_t *w) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  } else if constexpr (N == 2) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    w[0] = u.x, w[1] = u.y;
  } else {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  }
}

// An 8 x 8 matrix of 16-bit elements, two of row g in lane (g, c), transposed.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
// Element el of value r of a unit (bf16).
template <int F, int D>
__device__ __forceinline__ float value_at(const char *vs, int r, int el) {
  constexpr int P = D * Fmt<F>::kBits / 128;
  const uint16_t bits =
      *reinterpret_cast<const uint16_t *>(vs + v_place<P>(r, el / 8) * 16 + (el % 8) * 2);
  return __uint_as_float((uint32_t)bits << 16);
}

// Where a lane's words of a unit lie, and the loads of them.
template <int F, int D>
struct Words {
  static constexpr int kBits = Fmt<F>::kBits, kRow = D * kBits / 8, P = kRow / 16;
  static constexpr bool kBF = F == FS_CACHE_BF16;
  static constexpr int KW = D * kBits / 128;  // of a key: a quarter of the row
  static constexpr int VW = D == 64 ? kBits / 4 : (kBF ? 4 : kBits / 2);  // of a value, at a time
  static constexpr int SETS = kBF ? D / 64 : 1;
  int g, c;
  int k_at, k_half, v_at[2];
  __device__ __forceinline__ Words(int lane) : g(lane >> 2), c(lane & 3) {
    const int v_byte = g * VW * 4;  // inside the row (its first set)
    k_at = KW == 2 ? g * kRow + c * 8 : k_place<P>(g, c) * 16;
    k_half = (k_at & 64) ? -64 : 64;
    v_at[0] = v_place<P>(2 * c, v_byte / 16) * 16 + v_byte % 16;
    v_at[1] = v_place<P>(2 * c + 1, v_byte / 16) * 16 + v_byte % 16;
  }
  // of key 8 nt + g
  __device__ __forceinline__ void key(const char *st, int nt, uint32_t (&w)[KW]) const {
    const char *row = st + k_at + nt * 8 * kRow;
    if constexpr (KW <= 4) {
      lds_words<KW>(row, w);
    } else {
      // (four pieces on: within a row of eight the place's other half)
#pragma unroll
      for (int j = 0; j < KW / 4; ++j)
        lds_words<4>(P == 8 ? st + (k_at ^ (64 * j)) + nt * 8 * kRow
                            : row + (j & 1 ? k_half : 0) + j / 2 * 128,
                     w + 4 * j);
    }
  }
  // of values 16 kk + 2 c + (i & 1) + 8 (i / 2): eight rows on, the places repeat
  __device__ __forceinline__ void values(const char *vs, int kk, int set,
                                         uint32_t (&w)[4][VW]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      lds_words<VW>(vs + v_at[i & 1] + (16 * kk + 8 * (i >> 1)) * kRow + 128 * set, w[i]);
  }
};

// What the rows of a tile see of a unit that not all of them see whole.
struct Sight {
  const uint64_t *bits;  // of the tile's rows: drafted tokens,
  const int *first;      // first key of the prefix
  int past, key0;
  uint32_t valid;  // keys that can be read
  __device__ __forceinline__ bool sees(uint64_t b, int f, int at) const {
    const int key = key0 + at;
    return (valid >> at & 1) && (key < past ? key >= f : (bool)(b >> (key - past) & 1));
  }
};

// One row of q as the lane holds it (q_words): to fp16 by a power of two.  f: the
// row's factor; sum: of its fp16 elements, over the row's four lanes, where the
// key codes have a bias.
template <int F, int D>
__device__ __forceinline__ void q_to_f16(const Magic &magic, uint32_t (&raw)[D / 16][2], float &f,
                                         float &sum) {
  f = 1.f;
  sum = 0.f;
  if constexpr (F != FS_CACHE_BF16) {
    uint32_t most = 0;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e) most = __vmaxu2(most, raw[ks][e] & 0x7fff7fffu);
    most = max(most & 0xffffu, most >> 16);
    most = max(most, __shfl_xor_sync(~0u, most, 1));
    most = max(most, __shfl_xor_sync(~0u, most, 2));
    // the largest magnitude goes to [2^14, 2^15)
    f = __uint_as_float((uint32_t)min(254, 268 - (int)(most >> 7)) << 23);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t x = pack_f16(bf16_lo(raw[ks][e]) * f, bf16_hi(raw[ks][e]) * f);
        if constexpr (kBias<F> != 0.f) {
          const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&x));
          sum += y.x + y.y;
        }
        if constexpr (F == FS_CACHE_INT4)
          if (e) x = h2fma(x, magic.sixteenth, 0u);
        raw[ks][e] = x;
      }
    if constexpr (kBias<F> != 0.f) {
      sum += __shfl_xor_sync(~0u, sum, 1);
      sum += __shfl_xor_sync(~0u, sum, 2);
    }
  }
}
// Product of the fragments -> log2 units, and what the bias adds to a product.
template <int F>
__device__ __forceinline__ float score_factor(float scale, float f) {
  const float rf = log2_factor(scale, f);
  return kBias<F> != 0.f ? rf * 0x1p24f : rf;
}
template <int F>
__device__ __forceinline__ float bias_of(float sum) {
  return -0x1p-24f * kBias<F> * sum;
}

// Up to 16 MT rows: S = Q K^T, O = P V, rows g and g + 8 of every sixteen in the
// lane.
template <int F, int D, int MT>
struct RowForm {
  static constexpr bool kBF = F == FS_CACHE_BF16;
  static constexpr int KS = D / 16, NT = D / 8;  // k steps, value tiles
  using W = Words<F, D>;
  const W &at;
  uint32_t raw[MT][2][KS][2];
  uint32_t q[MT][KS][4];
  float rf[MT][2], bias[MT][2];
  // reference, sum (of even and odd keys)
  float ref[MT][2], l[MT][2][2], o[MT][NT][4], sc[MT][4][4];

  __device__ __forceinline__ RowForm(const W &w) : at(w) {}
  // src(row): the row's elements, null past the last
  template <class Src>
  __device__ __forceinline__ void load(const Src &src) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) q_words<F, D>(src(mt * 16 + hf * 8 + at.g), at.c, raw[mt][hf]);
  }
  __device__ __forceinline__ void begin(const Magic &magic, float scale) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float f, sum;
        q_to_f16<F, D>(magic, raw[mt][hf], f, sum);
        rf[mt][hf] = score_factor<F>(scale, f);
        bias[mt][hf] = bias_of<F>(sum);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          q[mt][ks][hf] = raw[mt][hf][ks][0];
          q[mt][ks][2 + hf] = raw[mt][hf][ks][1];
        }
        ref[mt][hf] = FLT_MAX;
        l[mt][hf][0] = l[mt][hf][1] = 0.f;
#pragma unroll
        for (int i = 0; i < NT; ++i) o[mt][i][2 * hf] = o[mt][i][2 * hf + 1] = 0.f;
      }
  }
  __device__ __forceinline__ void scores(const Magic &magic, const char *st) {
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      uint32_t w[W::KW];
      at.key(st, nt, w);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t b0, b1;
        k_regs<F>(magic, w, ks, b0, b1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) mma16816<kBF>(sc[mt][nt], q[mt][ks], b0, b1, ks > 0);
      }
    }
  }
  __device__ __forceinline__ void scale_keys(const float *kscale) {
    if constexpr (!kBF) {
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const float2 ks = *reinterpret_cast<const float2 *>(kscale + nt * 8 + 2 * at.c);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float &x = sc[mt][nt][2 * hf], &y = sc[mt][nt][2 * hf + 1];
            if constexpr (kBias<F> != 0.f) add2(x, y, bias[mt][hf], bias[mt][hf]);
            mul2(x, y, ks.x, ks.y);
          }
      }
    }
  }
  __device__ __forceinline__ void mask(const Sight &si) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint64_t bits = si.bits[mt * 16 + hf * 8 + at.g];
        const int first = si.first[mt * 16 + hf * 8 + at.g];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!si.sees(bits, first, nt * 8 + 2 * at.c + e)) sc[mt][nt][2 * hf + e] = -INFINITY;
      }
  }
  __device__ __forceinline__ float top_of(int mt, int hf) const {
    float top = fmaxf(sc[mt][0][2 * hf], sc[mt][0][2 * hf + 1]);
#pragma unroll
    for (int nt = 1; nt < 4; ++nt) top = max3f(top, sc[mt][nt][2 * hf], sc[mt][nt][2 * hf + 1]);
    return top;
  }
  __device__ __forceinline__ void follow(const float *kscale, float high) {  // the rows' references
    bool raise = false;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
        raise = raise || fmaf(top_of(mt, hf), rf[mt][hf], ref[mt][hf]) > high;
    if (!__any_sync(~0u, raise)) return;
    [[maybe_unused]] float lv[8];
    if constexpr (!kBF) {
#pragma unroll
      for (int i = 0; i < 8; ++i) lv[i] = lg2(fabsf(kscale[kUnit + i / 2 * 8 + 2 * at.c + i % 2]));
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float score = top_of(mt, hf) * rf[mt][hf], weight = -INFINITY;
        if constexpr (!kBF) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            weight = fmaxf(weight, fmaf(sc[mt][i / 2][2 * hf + i % 2], rf[mt][hf], lv[i]));
        }
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
          score = fmaxf(score, __shfl_xor_sync(~0u, score, x));
          if constexpr (!kBF) weight = fmaxf(weight, __shfl_xor_sync(~0u, weight, x));
        }
        const float to = moved<F>(ref[mt][hf], score, weight);
        const Back back(ref[mt][hf], to);
        ref[mt][hf] = to;
        l[mt][hf][0] = back(l[mt][hf][0]);
        l[mt][hf][1] = back(l[mt][hf][1]);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          o[mt][i][2 * hf] = back(o[mt][i][2 * hf]);
          o[mt][i][2 * hf + 1] = back(o[mt][i][2 * hf + 1]);
        }
      }
  }
  template <bool MASKED>
  __device__ __forceinline__ void weigh(const float *kscale) {
    [[maybe_unused]] float2 vs[4];
    if constexpr (!kBF) {
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
        vs[nt] = *reinterpret_cast<const float2 *>(kscale + kUnit + nt * 8 + 2 * at.c);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          float &x = sc[mt][nt][2 * hf], &y = sc[mt][nt][2 * hf + 1];
          [[maybe_unused]] const bool sx = x != -INFINITY, sy = y != -INFINITY;
          fma2(x, y, x, y, rf[mt][hf], ref[mt][hf]);
          x = tc::ex2(x);
          y = tc::ex2(y);
          add2(l[mt][hf][0], l[mt][hf][1], x, y);
          if constexpr (!kBF) {
            mul2(x, y, vs[nt].x, vs[nt].y);
            if constexpr (MASKED) {  // (a masked key's scale may be NaN)
              x = sx ? x : 0.f;
              y = sy ? y : 0.f;
            }
          }
        }
      }
  }
  // One value at a time, for values that are not finite; pt: room for [key][row].
  __device__ __forceinline__ void add_values_singly(const char *vs, float *pt) {
    constexpr int M = 16 * MT;
    __syncwarp();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          pt[(nt * 8 + 2 * at.c + (e & 1)) * M + mt * 16 + (e >> 1) * 8 + at.g] = sc[mt][nt][e];
    __syncwarp();
#pragma unroll 1
    for (int r = 0; r < kUnit; ++r) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float v = value_at<F, D>(vs, r, v_element<F, D>(2 * at.c + e, i));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const float p = pt[r * M + mt * 16 + hf * 8 + at.g];
              if (p != 0.f) o[mt][i][2 * hf + e] += p * v;
            }
        }
    }
  }
  __device__ __forceinline__ void add_values(const Magic &magic, const char *vs) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      uint32_t p[MT][4], lo[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = sc[mt][2 * kk + j / 2][2 * (j % 2)];
          const float x1 = sc[mt][2 * kk + j / 2][2 * (j % 2) + 1];
          if constexpr (kBF) {
            p[mt][j] = pack_bf16(x0, x1);
            lo[mt][j] = pack_bf16(x0 - bf16_lo(p[mt][j]), x1 - bf16_hi(p[mt][j]));
          } else {
            p[mt][j] = pack_f16(x0, x1);
          }
        }
#pragma unroll
      for (int set = 0; set < W::SETS; ++set) {
        uint32_t w[4][W::VW];
        at.values(vs, kk, set, w);
#pragma unroll
        for (int j = 0; j < NT / W::SETS / 2; ++j) {
          uint32_t b00, b01, b10, b11;
          v_regs<F>(magic, w[0], w[1], j, b00, b10);
          v_regs<F>(magic, w[2], w[3], j, b01, b11);
          const int i = set * (NT / W::SETS) + 2 * j;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma16816<kBF>(o[mt][i], p[mt], b00, b01);
            mma16816<kBF>(o[mt][i + 1], p[mt], b10, b11);
            if constexpr (kBF) {
              mma16816<true>(o[mt][i], lo[mt], b00, b01);
              mma16816<true>(o[mt][i + 1], lo[mt], b10, b11);
            }
          }
        }
      }
    }
  }
  // The warp's results: rows of SD floats, references, sums.
  template <int SD>
  __device__ __forceinline__ void leave(float *jo, float *jm, float *jl, int live) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float sum = l[mt][hf][0] + l[mt][hf][1];
        sum += __shfl_xor_sync(~0u, sum, 1);
        sum += __shfl_xor_sync(~0u, sum, 2);
        const int row = mt * 16 + hf * 8 + at.g;
        if (row >= live) continue;
        if (at.c == 0) {
          jm[row] = -ref[mt][hf];
          jl[row] = sum;
        }
#pragma unroll
        for (int i = 0; i < NT; i += 4)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4 *>(jo + row * SD + v_element<F, D>(2 * at.c + e, i)) =
                make_float4(o[mt][i][2 * hf + e], o[mt][i + 1][2 * hf + e],
                            o[mt][i + 2][2 * hf + e], o[mt][i + 3][2 * hf + e]);
      }
  }
};

// Up to eight rows: S^T = K Q^T and O^T = V^T P^T, so that the keys and the
// elements of a head fill the products' sixteens and the rows their eight columns:
// half the products and weights of RowForm, from the same registers.  Rows 2 c and
// 2 c + 1 in the lane.
template <int F, int D>
struct ColForm {
  static constexpr bool kBF = F == FS_CACHE_BF16;
  static constexpr int KS = D / 16, NT = D / 8;
  using W = Words<F, D>;
  const W &at;
  uint32_t q[KS][2];  // of row g
  float rf[2], bias[2];
  float ref[2], l[2];
  float o[NT / 2][4];  // element v_element(g, 2 j + i / 2), row 2 c + i % 2
  float sc[2][4];      // key 16 mt + 8 (i / 2) + g, row 2 c + i % 2

  __device__ __forceinline__ ColForm(const W &w) : at(w) {}
  template <class Src>
  __device__ __forceinline__ void load(const Src &src) {
    q_words<F, D>(src(at.g), at.c, q);
  }
  __device__ __forceinline__ void begin(const Magic &magic, float scale) {
    float f, sum;
    q_to_f16<F, D>(magic, q, f, sum);
    const float r = score_factor<F>(scale, f), b = bias_of<F>(sum);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      rf[e] = __shfl_sync(~0u, r, 4 * (2 * at.c + e));
      bias[e] = __shfl_sync(~0u, b, 4 * (2 * at.c + e));
      ref[e] = FLT_MAX;
      l[e] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < NT / 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
  }
  __device__ __forceinline__ void scores(const Magic &magic, const char *st) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t w[2][W::KW];
      at.key(st, 2 * mt, w[0]);
      at.key(st, 2 * mt + 1, w[1]);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t a[4];
        k_regs<F>(magic, w[0], ks, a[0], a[2]);
        k_regs<F>(magic, w[1], ks, a[1], a[3]);
        mma16816<kBF>(sc[mt], a, q[ks][0], q[ks][1], ks > 0);
      }
    }
  }
  __device__ __forceinline__ void scale_keys(const float *kscale) {
    if constexpr (!kBF) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ks = kscale[8 * i + at.g];
        float &x = sc[i / 2][2 * (i % 2)], &y = sc[i / 2][2 * (i % 2) + 1];
        if constexpr (kBias<F> != 0.f) add2(x, y, bias[0], bias[1]);
        mul2(x, y, ks, ks);
      }
    }
  }
  __device__ __forceinline__ void mask(const Sight &si) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint64_t bits = si.bits[2 * at.c + e];
      const int first = si.first[2 * at.c + e];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!si.sees(bits, first, 8 * i + at.g)) sc[i / 2][2 * (i % 2) + e] = -INFINITY;
    }
  }
  __device__ __forceinline__ float top_of(int e) const {
    return fmaxf(max3f(sc[0][e], sc[0][2 + e], sc[1][e]), sc[1][2 + e]);
  }
  __device__ __forceinline__ void follow(const float *kscale, float high) {
    if (!__any_sync(~0u, fmaf(top_of(0), rf[0], ref[0]) > high ||
                             fmaf(top_of(1), rf[1], ref[1]) > high))
      return;
    [[maybe_unused]] float lv[4];
    if constexpr (!kBF) {
#pragma unroll
      for (int i = 0; i < 4; ++i) lv[i] = lg2(fabsf(kscale[kUnit + 8 * i + at.g]));
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float score = top_of(e) * rf[e], weight = -INFINITY;
      if constexpr (!kBF) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          weight = fmaxf(weight, fmaf(sc[i / 2][2 * (i % 2) + e], rf[e], lv[i]));
      }
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        score = fmaxf(score, __shfl_xor_sync(~0u, score, x));
        if constexpr (!kBF) weight = fmaxf(weight, __shfl_xor_sync(~0u, weight, x));
      }
      const float to = moved<F>(ref[e], score, weight);
      const Back back(ref[e], to);
      ref[e] = to;
      l[e] = back(l[e]);
#pragma unroll
      for (int j = 0; j < NT / 2; ++j) {
        o[j][e] = back(o[j][e]);
        o[j][2 + e] = back(o[j][2 + e]);
      }
    }
  }
  template <bool MASKED>
  __device__ __forceinline__ void weigh(const float *kscale) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float &x = sc[i / 2][2 * (i % 2)], &y = sc[i / 2][2 * (i % 2) + 1];
      [[maybe_unused]] const bool sx = x != -INFINITY, sy = y != -INFINITY;
      x = tc::ex2(fmaf(x, rf[0], ref[0]));
      y = tc::ex2(fmaf(y, rf[1], ref[1]));
      add2(l[0], l[1], x, y);
      if constexpr (!kBF) {
        const float vs = kscale[kUnit + 8 * i + at.g];
        mul2(x, y, vs, vs);
        if constexpr (MASKED) {  // (a masked key's scale may be NaN)
          x = sx ? x : 0.f;
          y = sy ? y : 0.f;
        }
      }
    }
  }
  __device__ __forceinline__ void add_values_singly(const char *vs, float *pt) {
    constexpr int M = 8;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        pt[(8 * i + at.g) * M + 2 * at.c + e] = sc[i / 2][2 * (i % 2) + e];
    __syncwarp();
#pragma unroll 1
    for (int r = 0; r < kUnit; ++r) {
      const float p0 = pt[r * M + 2 * at.c], p1 = pt[r * M + 2 * at.c + 1];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float v = value_at<F, D>(vs, r, v_element<F, D>(at.g, i));
        if (p0 != 0.f) o[i / 2][2 * (i % 2)] += p0 * v;
        if (p1 != 0.f) o[i / 2][2 * (i % 2) + 1] += p1 * v;
      }
    }
  }
  __device__ __forceinline__ void add_values(const Magic &magic, const char *vs) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      // a transposed 8 x 8: the lane's two rows of key g -> two keys of row g
      uint32_t p[2], lo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float x = sc[kk][2 * i], y = sc[kk][2 * i + 1];
        if constexpr (kBF) {
          const uint32_t hi = pack_bf16(x, y);
          p[i] = turned(hi);
          lo[i] = turned(pack_bf16(x - bf16_lo(hi), y - bf16_hi(hi)));
        } else {
          p[i] = turned(pack_f16(x, y));
        }
      }
#pragma unroll
      for (int set = 0; set < W::SETS; ++set) {
        uint32_t w[4][W::VW];
        at.values(vs, kk, set, w);
#pragma unroll
        for (int j = 0; j < NT / W::SETS / 2; ++j) {
          uint32_t a[4];
          v_regs<F>(magic, w[0], w[1], j, a[0], a[1]);
          v_regs<F>(magic, w[2], w[3], j, a[2], a[3]);
          const int i = set * (NT / W::SETS / 2) + j;
          mma16816<kBF>(o[i], a, p[0], p[1]);
          if constexpr (kBF) mma16816<true>(o[i], a, lo[0], lo[1]);
        }
      }
    }
  }
  template <int SD>
  __device__ __forceinline__ void leave(float *jo, float *jm, float *jl, int live) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[e];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(~0u, sum, x);
      const int row = 2 * at.c + e;
      if (row >= live) continue;
      if (at.g == 0) {
        jm[row] = -ref[e];
        jl[row] = sum;
      }
#pragma unroll
      for (int j = 0; j < NT / 2; j += 2)
        *reinterpret_cast<float4 *>(jo + row * SD + v_element<F, D>(at.g, 2 * j)) =
            make_float4(o[j][e], o[j][2 + e], o[j + 1][e], o[j + 1][2 + e]);
    }
  }
};
template <int F, int D, int MT>
struct FormOf {
  using type = RowForm<F, D, MT>;
};
template <int F, int D>
struct FormOf<F, D, 0> {
  using type = ColForm<F, D>;
};

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <int F, int D, int MT>
__global__ void __launch_bounds__(Cfg<F, D, MT>::kWarps * 32, Cfg<F, D, MT>::kCtas)
k12_tree_kernel(const __grid_constant__ TreeK k) {
  using C = Cfg<F, D, MT>;
  constexpr int P = C::P, W = C::kWarps, M = C::kM, NS = C::kStages;
  extern __shared__ __align__(128) char smem[];
  __shared__ uint64_t row_bits[M];
  __shared__ int row_first[M];
  const TreeArgs &a = k.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int shift = 31 - __clz(a.c.page);
  asm volatile("griddepcontrol.launch_dependents;");

  if (blockIdx.x == 0)
    for (int i = tid; i < a.c.batch; i += W * 32)
      if (a.c.status && seq_outside(k, i)) atomicCAS(a.c.status, 0, FS_ERR_CACHE);
  const Line line = line_of(k, [&](const Share &share, int, long long x, long long y) {
    const long long at = share.begin(blockIdx.x);
    return (int)blockIdx.x < share.blocks && at >= x && at < y;
  });
  const long long total = line.total;
  if (total == 0) return;
  const Share &share = line.share;
  if ((int)blockIdx.x >= share.blocks) return;
  const long long u0 = share.begin(blockIdx.x), u1 = share.begin(blockIdx.x + 1);
  int b = line.b;
  long long begin = line.begin;  // of sequence b
  Seq s = line.s;

  const Magic magic = make_magic();
  char *ring = smem + warp * (C::kStage * NS);
  const uint32_t ring_s = smem_u32(ring);
  const int v_off = a.c.Hkv * a.c.page;  // rows from a key to its value

  uint32_t whole_units = 0;  // stages whose 32 keys can all be read
  const Words<F, D> words(lane);
  typename FormOf<F, D, MT>::type form(words);

  long long u = u0;
  while (u < u1) {
    while (u >= begin + seq_units(k, s) && b + 1 < a.c.batch) {
      begin += seq_units(k, s);
      s = seq_of(k, ++b);
    }
    if (s.units == 0) break;  // (lengths that changed under the call)
    const int seg = (int)quot(u - begin, s.units);
    const long long seg0 = begin + (long long)seg * s.units;
    const int rt = seg % s.tiles, h = seg / s.tiles;
    const int from = (int)(u - seg0), to = (int)min((long long)s.units, u1 - seg0);
    const int rows = s.n * k.G;

    __syncthreads();  // the ring held the last segment's results
    // q first: loads behind the units' copies would wait for them
    form.load([&](int r) -> const uint16_t * {
      const int row = rt * M + r;
      if (row >= rows) return nullptr;
      const int t = row / k.G, head = h * k.G + row - t * k.G;
      return static_cast<const uint16_t *>(a.q) + (((size_t)b * a.H + head) * a.T + t) * D;
    });
    // Where sixteen of the warp's units lie, two halves of sixteen rows to a unit:
    // lane 2 i + j holds half j of unit x + W i, as its place among all groups of
    // sixteen rows (kNone: nothing to read).  The table is read sixteen units
    // ahead: a load behind the units in flight waits for them.
    const int groups = a.c.page >> 4;
    auto page_of = [&](int x) -> int {
      const int key = s.first + (x + W * (lane >> 1)) * kUnit + 16 * (lane & 1);
      return x + W * (lane >> 1) < to && key < s.end
                 ? a.c.table[(size_t)b * a.c.max_pages + (key >> shift)]
                 : INT_MIN;
    };
    auto place_of = [&](int x, int page) -> uint32_t {
      if ((unsigned)page >= (unsigned)a.c.pages) {
        if (page != INT_MIN && a.c.status) atomicCAS(a.c.status, 0, FS_ERR_CACHE);
        return kNone;
      }
      const int key = s.first + (x + W * (lane >> 1)) * kUnit + 16 * (lane & 1);
      return (uint32_t)(page * 2 * a.c.Hkv + h) * groups + ((key & (a.c.page - 1)) >> 4);
    };
    // the lane's first row and piece of a half, and its scale
    const char *lane_src =
        static_cast<const char *>(a.c.codes) + (lane / P) * C::kRow + (lane % P) * 16;
    const float *lane_scale = C::kBF ? nullptr : a.c.scales + (lane & 15);
    auto issue = [&](int x, int stage, uint32_t place, int at) {
      if (x < to) {
        const uint32_t dst = ring_s + stage * C::kStage;
        const uint32_t g0 = __shfl_sync(~0u, place, 2 * at), g1 = __shfl_sync(~0u, place, 2 * at + 1);
        const char *src[2] = {lane_src + (size_t)g0 * (16 * C::kRow),
                              lane_src + (size_t)g1 * (16 * C::kRow)};
        const float *sp = nullptr;
        const uint32_t to_s = dst + 2 * C::kCodes + lane * 4;
        if constexpr (!C::kBF) sp = lane_scale + (size_t)(lane >> 4 ? g1 : g0) * 16;
        if (g0 != kNone && g1 != kNone && s.first + (x + 1) * kUnit <= s.end) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const int r = lane / P + 32 / P * i;
            const char *from_k = src[i * 2 / P] + (32 / P * i - 16 * (i * 2 / P)) * C::kRow;
            cp_async16(dst + k_place<P>(r, lane % P) * 16, from_k);
            cp_async16(dst + C::kCodes + v_place<P>(r, lane % P) * 16, from_k + v_off * C::kRow);
          }
          if constexpr (!C::kBF) {
            cp_async4(to_s, sp);
            cp_async4(to_s + 4 * kUnit, sp + v_off);
          }
          whole_units |= 1u << stage;
        } else {  // zeros for what cannot be read
          const bool in = (lane >> 4 ? g1 : g0) != kNone && s.first + x * kUnit + lane < s.end;
          const uint32_t valid = __ballot_sync(~0u, in);
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const int r = lane / P + 32 / P * i;
            const bool have = valid >> r & 1;
            const char *from_k = have ? src[i * 2 / P] + (32 / P * i - 16 * (i * 2 / P)) * C::kRow
                                      : static_cast<const char *>(a.c.codes);
            cp_async16z(dst + k_place<P>(r, lane % P) * 16, from_k, have ? 16 : 0);
            cp_async16z(dst + C::kCodes + v_place<P>(r, lane % P) * 16,
                        have ? from_k + v_off * C::kRow : from_k, have ? 16 : 0);
          }
          if constexpr (!C::kBF) {
            cp_async4z(to_s, in ? sp : a.c.scales, in ? 4 : 0);
            cp_async4z(to_s + 4 * kUnit, in ? sp + v_off : a.c.scales, in ? 4 : 0);
          }
          whole_units &= ~(1u << stage);
          if (lane == 0)
            *reinterpret_cast<uint32_t *>(ring + stage * C::kStage + 2 * C::kCodes + 8 * kUnit) =
                valid;
        }
      }
      cp_async_commit();
    };

    int next = from + warp, at = 0;  // unit to issue, its place among sixteen
    const int page = page_of(next);
    int later = page_of(next + 16 * W);
    // what every row sees: its bits, and its first key of the prefix
    if (tid < M) {
      const int r = rt * M + tid;
      uint64_t bits = 0;
      int first = INT_MAX;
      if (r < rows) {
        const int t = r / k.G;
        bits = a.tree ? (uint64_t)a.tree[(size_t)b * a.T + t] : ~0ull >> (63 - t);
        if (s.n < 64) bits &= (1ull << s.n) - 1;
        first = a.window ? max(0, s.past + __popcll(bits) - a.window) : 0;
      }
      row_bits[tid] = bits;
      row_first[tid] = first;
    }
    __syncthreads();

    uint32_t place = place_of(next, page);
    auto issue_next = [&](int stage) {
      issue(next, stage, place, at);
      next += W;
      if (++at == 16) {
        at = 0;
        place = place_of(next, later);
        later = page_of(next + 16 * W);
      }
    };
#pragma unroll 1
    for (int i = 0; i < NS - 1; ++i) issue_next(i);
    form.begin(magic, a.scale);
    int lead = 0;  // no row's prefix begins later
    if (a.window)
      for (int r = 0; r < M; ++r) lead = max(lead, row_first[r] == INT_MAX ? 0 : row_first[r]);

    int stage = 0;
    for (int x = from + warp; x < to; x += W) {
      cp_async_wait<NS - 2>();
      __syncwarp();
      const char *st = ring + stage * C::kStage;
      const float *kscale = reinterpret_cast<const float *>(st + 2 * C::kCodes);
      uint32_t top = 0;  // of the value scales, before anything waits for the products
      if constexpr (!C::kBF) top = __reduce_max_sync(~0u, scale_bits(kscale[kUnit + lane]));
      const int key0 = s.first + x * kUnit;
      const bool whole = (whole_units >> stage & 1) && key0 + kUnit <= s.past && key0 >= lead;

      form.scores(magic, st);
      // the next unit's copies while the products are under way
      issue_next(stage == 0 ? NS - 1 : stage - 1);
      form.scale_keys(kscale);
      if (!whole)
        form.mask(Sight{row_bits, row_first, s.past, key0,
                        whole_units >> stage & 1
                            ? ~0u
                            : *reinterpret_cast<const uint32_t *>(st + 2 * C::kCodes + 8 * kUnit)});
      form.follow(kscale, border<F>(top));
      if (C::kBF || whole)
        form.template weigh<false>(kscale);
      else
        form.template weigh<true>(kscale);

      const char *vs = st + C::kCodes;
      bool plain = true;
      if constexpr (C::kBF) {
        // A value that is not finite may reach only the rows that see it: 0 *
        // inf in the matrix product would reach the others.
        if (!whole) {
          bool odd = false;
          for (int i = lane; i < kUnit * P; i += 32) {
            uint32_t w[4];
            lds_words<4>(vs + i * 16, w);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              odd = odd || (w[j] & 0x7f80u) == 0x7f80u || (w[j] & 0x7f800000u) == 0x7f800000u;
          }
          plain = !__any_sync(~0u, odd);
          if (!plain)  // (the keys of the stage have been used)
            form.add_values_singly(vs, reinterpret_cast<float *>(ring + stage * C::kStage));
        }
      }
      if (plain) form.add_values(magic, vs);
      __syncwarp();  // before the stage is filled again
      stage = stage + 1 == NS ? 0 : stage + 1;
    }
    cp_async_wait<0>();

    // join the warps
    __syncthreads();
    constexpr int SD = D + 4;  // (rows in different banks)
    float *jo = reinterpret_cast<float *>(smem);  // [warp][M][SD]
    float *jm = jo + W * M * SD, *jl = jm + W * M;  // [warp][M]
    const int live = min(M, rows - rt * M);
    form.template leave<SD>(jo + warp * M * SD, jm + warp * M, jl + warp * M, live);
    __syncthreads();
    const bool alone = from == 0 && to == s.units;
    float *part = k.part + ((size_t)blockIdx.x * 2 + (from == 0)) * M * (D + 2);
    if (tid < live) {  // a row: the warps' factors in place of their references
      float top = jm[tid], sum = 0.f;
#pragma unroll
      for (int w = 1; w < W; ++w) top = fmaxf(top, jm[w * M + tid]);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = root_of(jm[w * M + tid], top);
        jm[w * M + tid] = f;
        sum += joined(f, jl[w * M + tid]);
      }
      if (!alone) {
        part[M * D + tid] = top;
        part[M * D + M + tid] = sum;
      }
      jl[tid] = sum;
    }
    __syncthreads();
    for (int i = tid; i < live * (D / 4); i += W * 32) {
      const int r = i / (D / 4), e = i % (D / 4) * 4, row = rt * M + r;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = jm[w * M + r];
        const float4 y = *reinterpret_cast<const float4 *>(jo + (w * M + r) * SD + e);
        x.x += joined(f, y.x), x.y += joined(f, y.y), x.z += joined(f, y.z), x.w += joined(f, y.w);
      }
      if (alone)
        put_row<D>(k, b, h, row, e, x, jl[r]);
      else
        *reinterpret_cast<float4 *>(part + r * D + e) = x;
    }
    u = seg0 + to;
  }
}

// Adds what the blocks of the line left of a segment: a block for ROWS rows of
// one kv head and sequence (of one row tile: ROWS divides its size), 256 / ROWS
// threads a row.  One row a block where there are few, so that many blocks' parts
// are read at once (152 parts of one row: 5 us against 13); eight where there are
// many.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) k12_join_kernel(const __grid_constant__ TreeK k) {
  constexpr int L = D / 4, LANES = 256 / ROWS;  // lanes of a row's output, of a row
  __shared__ float wt[ROWS][2 * kTreeSMs];
  __shared__ float red[2][8];
  __shared__ float4 acc[LANES > 32 ? 8 * L : 1];
  const int b = blockIdx.z, h = blockIdx.y, tid = threadIdx.x, lane = tid % LANES;
  const Line line = line_of(k, [&](const Share &, int i, long long, long long) { return i == b; });
  const Seq s = line.s;
  // What the earlier kernel wrote is read after this; every block waits, so that
  // the end of this kernel is the end of both.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int rows = s.n * k.G, row0 = blockIdx.x * ROWS;
  if (row0 >= rows || s.units == 0) return;
  const Share &share = line.share;
  const int rt = row0 / k.M, M = k.M;
  const long long s0 = line.begin + ((long long)h * s.tiles + rt) * s.units;
  const int c0 = share.of(s0), c1 = share.of(s0 + s.units - 1);
  if (c0 == c1) return;  // written by its block
  const int n = c1 - c0 + 1, i0 = tid / LANES, row = row0 + i0, r = row % M;
  if (row >= rows) return;  // (whole warps, or the block)
  // the first block left it as its last segment (1), the others as their first (0)
  auto part = [&](int i) { return k.part + ((size_t)(c0 + i) * 2 + (i == 0)) * M * (D + 2); };
  auto over_block = [&](float *sh, float x, auto op) {  // of the warps' results
    if constexpr (LANES > 32) {
      if (tid % 32 == 0) sh[tid / 32] = x;
      __syncthreads();
      x = sh[0];
#pragma unroll
      for (int w = 1; w < 8; ++w) x = op(x, sh[w]);
    }
    return x;
  };
  float top = -FLT_MAX;
  for (int i = lane; i < n; i += LANES) top = fmaxf(top, part(i)[M * D + r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  top = over_block(red[0], top, [](float x, float y) { return fmaxf(x, y); });
  float sum = 0.f;
  for (int i = lane; i < n; i += LANES) {
    const float *p = part(i);
    const float f = root_of(p[M * D + r], top);
    wt[i0][i] = f;
    sum += joined(f, p[M * D + M + r]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  __syncwarp();
  sum = over_block(red[1], sum, [](float x, float y) { return x + y; });  // (and wt is whole)
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = lane / L; i < n; i += LANES / L) {
    const float4 y = *reinterpret_cast<const float4 *>(part(i) + r * D + lane % L * 4);
    const float f = wt[i0][i];
    x.x += joined(f, y.x), x.y += joined(f, y.y), x.z += joined(f, y.z), x.w += joined(f, y.w);
  }
  if constexpr (L == 16) {
    x.x += __shfl_xor_sync(~0u, x.x, 16);
    x.y += __shfl_xor_sync(~0u, x.y, 16);
    x.z += __shfl_xor_sync(~0u, x.z, 16);
    x.w += __shfl_xor_sync(~0u, x.w, 16);
  }
  if constexpr (LANES > 32) {
    if (tid % 32 < L) acc[tid / 32 * L + tid % 32] = x;
    __syncthreads();
    if (lane < L) {
#pragma unroll
      for (int w = 1; w < 8; ++w) {
        const float4 y = acc[w * L + lane];
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
    }
  }
  if (lane < L) put_row<D>(k, b, h, row, lane * 4, x, sum);
}

template <int F, int D, int MT>
cudaError_t launch_mt(TreeK k, cudaStream_t st) {
  using C = Cfg<F, D, MT>;
  k.M = C::kM;
  k.unit = kUnit;
  k.least = C::kWarps;
  k.blocks = kTreeSMs * C::kCtas;
  // no more blocks than the table has room for units
  const long long most = (long long)k.a.c.batch * k.a.c.Hkv * ((k.a.T * k.G + k.M - 1) / k.M) *
                         (((long long)k.a.c.max_pages * k.a.c.page + kUnit - 1) / kUnit);
  const long long need = (most + k.least - 1) / k.least;
  if (need < k.blocks) k.blocks = (int)need;
  auto fn = k12_tree_kernel<F, D, MT>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  fn<<<k.blocks, C::kWarps * 32, C::kSmem, st>>>(k);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_tree_join(k, st);
}

template <int F>
cudaError_t launch_f(const TreeK &k, cudaStream_t st) {
  const bool one = k.a.T * k.G <= 16;
  if (k.a.T * k.G <= 8) return k.a.c.d == 64 ? launch_mt<F, 64, 0>(k, st) : launch_mt<F, 128, 0>(k, st);
  if (k.a.c.d == 64) return one ? launch_mt<F, 64, 1>(k, st) : launch_mt<F, 64, 2>(k, st);
  return launch_mt<F, 128, 1>(k, st);
}

}  // namespace

// Whether 128 rows are taken at a time, on tcgen05: from more rows to a kv head
// than the kernel above does well.  Measured on 4 sequences of 16384 keys, 8 kv
// heads, cold caches, here against there (us):
//   d = 64    int8 64 rows 65, 65, 96 rows 82, 67   e4m3 61, 65 and 76, 66   int4 60, 63 and 76, 64
//   d = 128   int8 32 rows 78, 81, 40 rows 93, 80   e4m3 77, 79 and 90, 77   int4 69, 76 and 86, 75
//   bf16, whose probabilities are two products here and whose rows need no conversion there:
//   d = 64 32 rows 61, 70, 40 rows 77, 67           d = 128 16 rows 80, 88, 20 rows 123, 90
// The prefixes' lengths, which the host does not know, play no part: over a few hundred keys
// both take 18 to 35 us, and the rule costs up to 10 of them (4 x 400 bf16 keys, d = 128,
// 20 to 48 rows: 24 to 27 here, 34 to 37 there; 8-bit and int4 codes at most 8).
bool wide(const fs_cache &c, int H, int T) {
  return H / c.Hkv * T > (c.d == 64 ? 64 : 32) / (c.format == FS_CACHE_BF16 ? 2 : 1);
}

template <int D, int ROWS>
cudaError_t launch_join(const TreeK &k, cudaStream_t st) {
  // its blocks may start, and look up their rows, while the last ones of the
  // kernel before run
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((k.a.T * k.G + ROWS - 1) / ROWS), (unsigned)k.a.c.Hkv,
                     (unsigned)k.a.c.batch);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k12_join_kernel<D, ROWS>, k);
}

cudaError_t launch_tree_join(const TreeK &k, cudaStream_t st) {
  const bool few = (long long)k.a.T * k.a.H * k.a.c.batch <= kTreeSMs * 8;
  if (k.a.c.d == 64) return few ? launch_join<64, 1>(k, st) : launch_join<64, 8>(k, st);
  return few ? launch_join<128, 1>(k, st) : launch_join<128, 8>(k, st);
}

size_t tree_workspace_bytes(const fs_cache &c, int H, int T) {
  const int rows = wide(c, H, T) ? kTreeSMs * 128 : kTreeSMs * 2 * 32;
  return (size_t)rows * 2 * (c.d + 2) * sizeof(float);
}

cudaError_t launch_tree(const TreeArgs &a, cudaStream_t st) {
  TreeK k{};
  k.a = a;
  k.G = a.H / a.c.Hkv;
  k.part = static_cast<float *>(a.ws);
  if (wide(a.c, a.H, a.T)) return launch_tree_wide(k, st);
  switch (a.c.format) {
    case FS_CACHE_BF16: return launch_f<FS_CACHE_BF16>(k, st);
    case FS_CACHE_E4M3: return launch_f<FS_CACHE_E4M3>(k, st);
    case FS_CACHE_INT8: return launch_f<FS_CACHE_INT8>(k, st);
    default: return launch_f<FS_CACHE_INT4>(k, st);
  }
}

}  // namespace fs
