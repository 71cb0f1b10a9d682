// k13_tree_wide.cu -- fs_tree_attn where many rows share their keys (a wide
// tree, or grouped heads): 128 rows a block on the tensor cores (tcgen05).
//
// The line of units, its sharing and the joining of the blocks' results are
// k12_tree.cu's; a unit here is a tile of KT keys.  A block works on one
// segment at a time:
//   * warps 8-11 turn codes into fp16 tiles in shared memory (exact: codes have
//     at most 8 bits), rings of keys and of values, with the scales beside them; two
//     warps to a tile, the other two on the next one.  bf16 rows are tiles as they
//     lie: TMA brings them, keys and values of even and of odd tiles a warp each, and
//     warps 14, 15 look through the values that not all rows see;
//   * two streams of four warps take the tiles in turn, a thread a row, each
//     stream with its own scores, probabilities, output (TMEM), running
//     reference and sum, so that neither waits for the other;
//   * one thread of warp 12 (13) issues the first (second) stream's products:
//     S = Q K^T a tile or two ahead of the rows, O += P V with P from TMEM.
// The streams are joined through shared memory at the end of a segment.
//
// Scores, scales, references and weights are as in k12_tree.cu (q by a power of
// two a row, weights in fp16; bf16: the first 8 bits of a probability and the
// next 8, two products).  Where the largest score of 32 columns, with the largest of
// their value scales, could take a weight past fp16's range, the row's reference is
// moved by what the row sees before they are weighed: its sum, its O (between
// two products) and its earlier weights of the tile are multiplied by the
// difference.
//
// Tiles of 128 codes with heads of 64 (scores, probabilities and output fill a
// stream's half of TMEM), else of 64 with the scores held twice and P written over
// them: 64 tokens x 4 heads a kv head over 8 x 16384 keys take 167 us (int8) and 162
// (e4m3) with the former, 168 and 165 with the latter.  Four warps on the same tile, each
// waiting for the same barriers, were what everything waited for: 205 us when pairs in
// turn took 157 (bf16: one warp for all TMA copies 182, four 150).
//
// Bound by: with codes, the rows' warps, which read two scales a column from shared
// memory (26 us of an earlier 154 went with those reads) around the exponentials (128 x KT
// a tile); with bf16 and heads of 128 the products' issue and the keys that come twice,
// once for each 128 rows (4 of 107 us went with the rows' work).
#include <cuda.h>

#include "tree.cuh"

namespace fs {
namespace {

template <int F, int D>
struct Wide {
  static constexpr bool kBF = F == FS_CACHE_BF16;
  static constexpr int kBits = Fmt<F>::kBits;
  static constexpr int kRow = D * kBits / 8, P = kRow / 16;
  static constexpr int KT = D == 64 && !kBF ? 128 : 64;  // keys of a tile
  static constexpr bool kTwice = KT == 64;               // scores are held twice
  static constexpr int kCols = D / 64;           // 64-element column blocks
  static constexpr int kBlock = KT * 128;        // bytes of one of them
  static constexpr int kTile = kCols * kBlock;   // keys or values of a tile
  // tiles of keys and of values held
  static constexpr int NK = !kBF ? 2 : D == 64 ? 6 : 4, NV = !kBF ? 4 : D == 64 ? 8 : 6;
  // Codes: a tile is two warps' with half of its keys each, the next one the other two's,
  // so that the waits of one pair hide behind the work of the other.
  static constexpr int kMates = 2, KW = KT / kMates;
  // a warp's codes of a tile, a scale pair a key, valid words
  static constexpr int kRawScale = KW * kRow * 2, kRaw = kBF ? 0 : kRawScale + KW * 8 + 16;
  static constexpr int kQ = 128 * 128 * kCols;
  static constexpr int kMerge = 128 * (64 + 2) * 4;  // begins in place of q
  static constexpr int kRounds = D / 64;  // of handing it over
  // key scales, value scales, their log2, valid words and borders of 32 keys each; bf16: 2
  // valid words, 2 of odd values
  static constexpr int kSide = kBF ? 16 : KT * 12 + KT / 4;
  static constexpr int kBars = 496;
  static constexpr int kRest = 1024 + kTile * (NK + NV) + kMerge + kSide * NV + kBars;
  static constexpr int kFit = kBF ? 0 : (226 * 1024 - kRest) / (kBF ? 1 : 4 * kRaw);
  static constexpr int kRaws = kFit > 3 ? 3 : kFit;  // tiles of codes under way, a warp
  static constexpr int kSmem = kRest + 4 * kRaws * kRaw;
  // TMEM columns of a stream: S twice, O, and P in place of S, 32 columns at a time (16
  // of fp16, or of high parts and 16 of low ones); or S, P, O.
  static constexpr int kO = kTwice ? 2 * KT : KT + KT / 2, kTmem = 256;
  static_assert(kO + D <= kTmem && kQ <= kMerge && kSmem <= 226 * 1024, "sizes");
  // A wait by parity must not fall two phases behind.  A place in the rings holds tiles of
  // one parity, which are one loader's and, within a segment, one stream's; after a segment
  // with an odd number of tiles the streams change places, but no tile of the next
  // one is read before q_full, which follows the last reads of this one.
  static_assert(NK % 2 == 0 && NV % 2 == 0, "rings");
  static_assert(kBF || kRaws >= 2, "pieces");
  static constexpr int NP = KW * P / 32;  // pieces of a lane, keys or values
};

constexpr uint32_t kNone = ~0u;

// Element of a head at position i of the tiles' rows: int4 codes leave a word
// in the order 0 4 1 5 2 6 3 7.
template <int F>
__device__ __forceinline__ constexpr int element_of(int i) {
  return F == FS_CACHE_INT4 ? (i & ~7) | ((i & 7) >> 1) | ((i & 1) << 2) : i;
}

// tc::mbar_wait with a hint of how long the thread may sleep in a try: nearly
// all of these waits are long, and their polls would take issue slots from the
// rows' warps.
__device__ __forceinline__ bool wait_asleep(uint64_t *bar, uint32_t parity, int *fail,
                                            long long cycles) {
  if (tc::mbar_try_wait(bar, parity)) return true;  // (reading the clock takes as long)
  const long long t0 = clock64();
  const uint32_t ns = (uint32_t)min(cycles, 1000000ll);
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(ns)
        : "memory");
    if (ok) return true;
    if (clock64() - t0 > cycles) break;
    if (*reinterpret_cast<volatile int *>(fail) != 0) return false;
  }
  tc::report_error(fail, FS_ERR_TIMEOUT);
  return false;
}

// The segments of a block, one after the other.
struct Walk {
  long long u, u1, begin;
  int b;
  Seq s;
  int h, rt, from, to;
  __device__ __forceinline__ bool next(const TreeK &k) {
    if (u >= u1) return false;
    while (u >= begin + seq_units(k, s) && b + 1 < k.a.c.batch) {
      begin += seq_units(k, s);
      s = seq_of(k, ++b);
    }
    if (s.units == 0) return false;  // (lengths that changed under the call)
    const int seg = (int)quot(u - begin, s.units);
    const long long seg0 = begin + (long long)seg * s.units;
    rt = seg % s.tiles;
    h = seg / s.tiles;
    from = (int)(u - seg0);
    to = (int)min((long long)s.units, u1 - seg0);
    u = seg0 + to;
    return true;
  }
};

struct Bars {
  uint64_t kfull[8], kempty[8];         // tiles of keys
  uint64_t vfull[8], vempty[8];         // of values, with scales and valid words
  uint64_t landed[8];                   // values that are looked through first (bf16)
  uint64_t s_full[2][2], s_free[2];     // a stream's scores
  // A stream's probabilities and the products that read them, of even and of odd
  // tiles: a warp may be a tile ahead of another, the rows two ahead of the products.
  uint64_t p_full[2][2], p_free[2][2];
  uint64_t added[2];                    // values that are not finite were (bf16)
  uint64_t q_full, done, merge, merged;  // of a segment
  uint64_t drained[2];                  // a stream's products, when a wait has given up
};

// Sixteen bytes of codes -> fp16, eight elements to a 16-byte chunk.
template <int F>
__device__ __forceinline__ void to_chunk(const Magic &m, const uint32_t *w, uint4 &x) {
  if constexpr (F == FS_CACHE_E4M3) {
    e4m3_h2(w[0], x.x, x.y);
    e4m3_h2(w[1], x.z, x.w);
  } else if constexpr (F == FS_CACHE_INT8) {
    const uint32_t a = w[0] ^ 0x80808080u, b = w[1] ^ 0x80808080u;
    x.x = h2add(__byte_perm(a, m.magic, 0x7170), kSub128);
    x.y = h2add(__byte_perm(a, m.magic, 0x7372), kSub128);
    x.z = h2add(__byte_perm(b, m.magic, 0x7170), kSub128);
    x.w = h2add(__byte_perm(b, m.magic, 0x7372), kSub128);
  } else {
    x.x = nib_even(m, w[0]);
    x.y = nib_odd(m, w[0]);
    x.z = nib_even(m, w[0] >> 8);
    x.w = nib_odd(m, w[0] >> 8);
  }
}

// bf16 rows come by TMA: the map of all groups of sixteen rows.
struct NoMap {};
template <int F>
using MapOf = std::conditional_t<F == FS_CACHE_BF16, CUtensorMap, NoMap>;

// The box of 64 elements from x on of the groups from g on; zeros where one is outside.
__device__ __forceinline__ void load_group(void *dst, const void *map, uint64_t *bar, int x, int g) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%3, 0, %4}], [%2];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(g)
      : "memory");
}

// tc::desc_sw128 for elements in several blocks of 64, `apart` bytes from one to the next.
__device__ __forceinline__ uint64_t desc_blocks(uint32_t at, uint32_t apart) {
  return (tc::desc_sw128(at) & ~(0x3fffull << 16)) | (uint64_t)(apart >> 4) << 16;
}

// Bits of two bf16 elements that are NaN or infinite: their masks, 0 if both are finite.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) |
         ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

template <int F, int D>
__global__ void __launch_bounds__(512, 1)
k13_tree_wide_kernel(const __grid_constant__ TreeK k, const __grid_constant__ MapOf<F> map) {
  using C = Wide<F, D>;
  constexpr int KT = C::KT, P = C::P, NK = C::NK, NV = C::NV, NP = C::NP;
  constexpr int kRaws = C::kRaws;
  constexpr bool kBF = C::kBF;
  extern __shared__ char smem_raw[];
  char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  char *vals = smem + NK * C::kTile, *qs = vals + NV * C::kTile;
  float *mo = reinterpret_cast<float *>(qs);  // 64 columns of the second stream's O, over q
  float *mm = mo + 128 * 64, *ml = mm + 128;
  char *side = reinterpret_cast<char *>(ml + 128);
  static_assert(sizeof(Bars) <= C::kBars, "sizes");
  Bars &bar = *reinterpret_cast<Bars *>(side + NV * C::kSide);
  [[maybe_unused]] char *raw = side + NV * C::kSide + C::kBars;
  __shared__ uint32_t tmem_base;
  __shared__ int fail;
  // What a TMA warp has issued: the tile after its last one, the places whose last tile goes
  // by `landed`, and the phases of those.
  struct Issued {
    uint32_t next, looked, landed;
  };
  __shared__ Issued issued[4];
  const TreeArgs &a = k.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;");

  if (blockIdx.x == 0)
    for (int i = tid; i < a.c.batch; i += 512)
      if (a.c.status && seq_outside(k, i)) atomicCAS(a.c.status, 0, FS_ERR_CACHE);
  const Line line = line_of(k, [&](const Share &share, int, long long x, long long y) {
    const long long at = share.begin(blockIdx.x);
    return (int)blockIdx.x < share.blocks && at >= x && at < y;
  });
  if (line.total == 0) return;
  const Share &share = line.share;
  if ((int)blockIdx.x >= share.blocks) return;

  if (tid == 0) {
    fail = 0;
    for (int i = 0; i < 8; ++i) {
      tc::mbar_init(&bar.kfull[i], kBF ? 1 : C::kMates);
      tc::mbar_init(&bar.vfull[i], kBF ? 1 : C::kMates);
      tc::mbar_init(&bar.landed[i], 1);
      tc::mbar_init(&bar.kempty[i], 1);
      tc::mbar_init(&bar.vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bar.s_full[i][0], 1);
      tc::mbar_init(&bar.s_full[i][1], 1);
      tc::mbar_init(&bar.s_free[i], 128);
      tc::mbar_init(&bar.p_full[i][0], 128);
      tc::mbar_init(&bar.p_full[i][1], 128);
      tc::mbar_init(&bar.added[i], 128);
      tc::mbar_init(&bar.drained[i], 1);
      tc::mbar_init(&bar.p_free[i][0], 1);
      tc::mbar_init(&bar.p_free[i][1], 1);
    }
    // the rows of the first stream, and the second stream's issuing thread: a segment of
    // one tile has no other wait that ties it to the others
    tc::mbar_init(&bar.q_full, 129);
    tc::mbar_init(&bar.done, 128);
    tc::mbar_init(&bar.merge, 128);
    tc::mbar_init(&bar.merged, 128);
    tc::mbar_fence_init();
  }
  if (warp == 12) {
    tc::tmem_alloc(&tmem_base, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();

  Walk w{share.begin(blockIdx.x), share.begin(blockIdx.x + 1), line.begin, line.b, line.s, 0, 0, 0, 0};
  // Waits give up after a limit and say so in `fail`; every role then leaves its
  // loops for the barrier at the end, behind which the copies and products that are
  // still under way are waited for.
  auto wait_one = [&](uint64_t *b, uint32_t phase) {
    return wait_asleep(b, phase & 1, &fail, a.wait_cycles);
  };
  auto wait = [&](uint64_t *b, uint32_t phase) {  // the same answer in a warp
    return (bool)__all_sync(~0u, wait_one(b, phase));
  };
  uint32_t it = 0;  // tiles of the block before the current segment
  uint32_t seg = 0;

  if (warp < 8) {
    // ------------------------------------------------------------- a stream
    const int st = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's quarter of the lanes
    const uint32_t tm = tmem_base + st * C::kTmem + lanes;
    uint32_t jt = 0;  // tiles of the stream before the current one
    bool ok = true;
    for (; ok && w.next(k); ++seg) {
      const int n = w.to - w.from, rows = w.s.n * k.G, r = w.rt * 128 + row;
      const bool live = r < rows;
      const int t = live ? r / k.G : 0, head = w.h * k.G + (live ? r % k.G : 0);
      const size_t at = (((size_t)w.b * a.H + head) * a.T + t) * D;
      uint64_t bits = 0;
      int first = 0;
      if (live) {
        bits = a.tree ? (uint64_t)a.tree[(size_t)w.b * a.T + t] : ~0ull >> (63 - t);
        if (w.s.n < 64) bits &= (1ull << w.s.n) - 1;
        if (a.window) first = max(0, w.s.past + __popcll(bits) - a.window);
      }
      // the row's power of two; the first stream writes q
      const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + at);
      float f = 1.f;
      if constexpr (!kBF) {
        uint32_t most = 0;
#pragma unroll 8
        for (int i = 0; i < D / 8; ++i) {
          const uint4 x = live ? src[i] : make_uint4(0, 0, 0, 0);
          most = __vmaxu2(most, x.x & 0x7fff7fffu);
          most = __vmaxu2(most, x.y & 0x7fff7fffu);
          most = __vmaxu2(most, x.z & 0x7fff7fffu);
          most = __vmaxu2(most, x.w & 0x7fff7fffu);
        }
        most = max(most & 0xffffu, most >> 16);
        f = __uint_as_float((uint32_t)min(254, 268 - (int)(most >> 7)) << 23);
      }
      const float rf = log2_factor(a.scale, f);
      if (st == 0) {
#pragma unroll 1
        for (int c = 0; ok && c < C::kCols; ++c) {
          uint4 x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = live ? src[c * 8 + i] : make_uint4(0, 0, 0, 0);
          // (the second stream's results lay there)
          if (c == 0 && seg > 0 && !(ok = wait(&bar.merged, seg * C::kRounds - 1))) break;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t y[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t z[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if constexpr (kBF) {
                z[j] = y[j];
                continue;
              }
              const int e0 = element_of<F>(2 * j), e1 = element_of<F>(2 * j + 1);
              const float v0 = e0 % 2 ? bf16_hi(y[e0 / 2]) : bf16_lo(y[e0 / 2]);
              const float v1 = e1 % 2 ? bf16_hi(y[e1 / 2]) : bf16_lo(y[e1 / 2]);
              z[j] = pack_f16(v0 * f, v1 * f);
            }
            *reinterpret_cast<uint4 *>(qs + c * (128 * 128) + swz128(row, i)) =
                make_uint4(z[0], z[1], z[2], z[3]);
          }
        }
        if (!ok) break;
        tc::fence_async_smem();
        tc::mbar_arrive(&bar.q_full);
      } else if (!(ok = wait(&bar.q_full, seg))) {  // (the last segment's results have been taken)
        break;
      }

      float ref = FLT_MAX, l0 = 0.f, l1 = 0.f;
      bool begun = false;  // O holds something
      // O to a new reference, once the last tile's product has ended (this one's has not begun)
      auto rescale = [&](const Back &back) -> bool {
        if (jt > 0 && !wait(&bar.p_free[st][jt - 1 & 1], jt - 1 >> 1)) return false;
        tc::fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {  // (few registers: 32 columns wait meanwhile)
          uint32_t o[16];
          tc::tmem_ld16(tm + C::kO + c, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(back(__uint_as_float(o[i])));
          tc::tmem_st16(tm + C::kO + c, o);
        }
        tc::tmem_wait_st();
        return true;
      };

      for (int i = st; ok && i < n; i += 2, ++jt) {
        const uint32_t x = it + i, slot = x % NV;
        const uint32_t x2 = C::kTwice ? jt & 1 : 0, tile2 = C::kTwice ? jt >> 1 : jt;
        const uint32_t ts = tm + x2 * KT, tp = C::kTwice ? ts : tm + KT;  // S, P
        const float *ks = reinterpret_cast<const float *>(side + slot * C::kSide);
        const uint32_t *valid = reinterpret_cast<const uint32_t *>(ks + (kBF ? 0 : 3 * KT));
        const int key0 = w.s.first + (w.from + i) * KT;
        if (!(ok = wait(&bar.vfull[slot], x / NV))) break;
        const uint4 in = *reinterpret_cast<const uint4 *>(valid);
        if (!(ok = wait(&bar.s_full[st][x2], tile2))) break;
        tc::fence_after_sync();
        const bool whole = (KT == 128 ? in.x & in.y & in.z & in.w : in.x & in.y) == ~0u &&
                           __all_sync(~0u, key0 + KT <= w.s.past && key0 >= first);
        // The columns, 32 at a time.
        auto weigh = [&](int c0, auto masked) {
          uint32_t u[32];
          tc::tmem_ld32(ts + c0, u);
          [[maybe_unused]] uint32_t seen = ~0u;  // of these 32 keys
          if constexpr (masked.value) {
            const int key = key0 + c0;
            const int before = min(max(w.s.past - key, 0), 32);  // keys of the prefix
            const int skip = min(max(first - key, 0), before);   // outside the window
            seen = before - skip == 32 ? ~0u
                   : before > skip     ? ((1u << (before - skip)) - 1) << skip
                                       : 0u;
            if (before < 32) {  // drafted: bit (key + i - past)
              const int j = key - w.s.past;  // of key 0; negative inside the prefix
              const uint64_t z = j >= 64 ? 0 : j >= 0 ? bits >> j : bits << -j;
              seen |= (uint32_t)z & (before ? ~0u << before : ~0u);
            }
            seen &= valid[c0 / 32];
          }
          tc::tmem_wait_ld();
          if (!C::kTwice && c0 + 32 == KT) {  // the next tile's scores may be made
            tc::fence_before_sync();
            tc::mbar_arrive(&bar.s_free[st]);
          }
          // Step by step over all 32 columns: each step's operations do not wait
          // for one another.
          float y[32];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            y[j] = __uint_as_float(u[j]), y[j + 1] = __uint_as_float(u[j + 1]);
            y[j + 2] = __uint_as_float(u[j + 2]), y[j + 3] = __uint_as_float(u[j + 3]);
            if constexpr (!kBF) {
              const float4 kk = *reinterpret_cast<const float4 *>(ks + c0 + j);
              mul2(y[j], y[j + 1], kk.x, kk.y);
              mul2(y[j + 2], y[j + 3], kk.z, kk.w);
            }
          }
          if constexpr (masked.value) {
#pragma unroll
            for (int j = 0; j < 32; ++j) y[j] = seen >> j & 1 ? y[j] : -INFINITY;
          }
          float t0 = y[0], t1 = y[1];
#pragma unroll
          for (int j = 2; j < 32; j += 4) {
            t0 = max3f(t0, y[j], y[j + 1]);
            if (j + 2 < 32) t1 = max3f(t1, y[j + 2], y[j + 3]);
          }
          t0 = fmaxf(t0, t1);
          const float high =
              kBF ? Range<F>::kHigh : __uint_as_float(valid[KT / 32 + c0 / 32]);
          if (__any_sync(~0u, fmaf(t0, rf, ref) > high)) {  // move the rows' references
            float weight = -INFINITY;
            if constexpr (!kBF) {
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 lv = *reinterpret_cast<const float4 *>(ks + 2 * KT + c0 + j);
                weight = max3f(weight, fmaf(y[j], rf, lv.x), fmaf(y[j + 1], rf, lv.y));
                weight = max3f(weight, fmaf(y[j + 2], rf, lv.z), fmaf(y[j + 3], rf, lv.w));
              }
            }
            const float to = moved<F>(ref, t0 * rf, weight);
            const Back back(ref, to);
            // (none moves where the large values of a tile are hidden from all rows)
            const bool some = __any_sync(~0u, to != ref);
            ref = to;
            l0 = back(l0);
            l1 = back(l1);
            if (some && begun) ok = rescale(back);
#pragma unroll 1
            for (int c = 0; some && c < (C::kTwice ? c0 : c0 / 2);
                 c += C::kTwice && !kBF && c % 32 ? 24 : 8) {  // this tile's earlier columns
              uint32_t z[8];
              tc::tmem_wait_st();
              tc::tmem_ld8(tp + c, z);
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if constexpr (kBF) {
                  z[i] = pack_bf16(back(bf16_lo(z[i])), back(bf16_hi(z[i])));
                } else {
                  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&z[i]));
                  z[i] = pack_f16(back(f.x), back(f.y));
                }
              }
              tc::tmem_st8(tp + c, z);
            }
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2) fma2(y[j], y[j + 1], y[j], y[j + 1], rf, ref);
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] = tc::ex2(y[j]);
          float s2 = 0.f, s3 = 0.f;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            add2(l0, l1, y[j], y[j + 1]);
            add2(s2, s3, y[j + 2], y[j + 3]);
          }
          add2(l0, l1, s2, s3);
          if constexpr (!kBF) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 vv = *reinterpret_cast<const float4 *>(ks + KT + c0 + j);
              mul2(y[j], y[j + 1], vv.x, vv.y);
              mul2(y[j + 2], y[j + 3], vv.z, vv.w);
            }
            if constexpr (masked.value) {  // (a masked key's scale may be NaN)
#pragma unroll
              for (int j = 0; j < 32; ++j) y[j] = seen >> j & 1 ? y[j] : 0.f;
            }
          }
          uint32_t p[16];
          [[maybe_unused]] uint32_t rest[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            if constexpr (kBF) {  // cut off after 8 bits, and the next 8
              p[j / 2] = __byte_perm(__float_as_uint(y[j]), __float_as_uint(y[j + 1]), 0x7632);
              rest[j / 2] = pack_bf16(y[j] - bf16_lo(p[j / 2]), y[j + 1] - bf16_hi(p[j / 2]));
            } else {
              p[j / 2] = pack_f16(y[j], y[j + 1]);
            }
          }
          if (!C::kTwice && c0 == 0 && jt > 0) {  // the last tile's product has read P
            ok = wait(&bar.p_free[st][jt - 1 & 1], jt - 1 >> 1) && ok;
            tc::fence_after_sync();
          }
          tc::tmem_st16(tp + (C::kTwice ? c0 : c0 / 2), p);
          if constexpr (kBF) tc::tmem_st16(tp + c0 + 16, rest);
        };
        // (two copies: one with masks under a condition would test and select for
        // every element of every tile)
        if (whole) {
#pragma unroll 1
          for (int c0 = 0; ok && c0 < KT; c0 += 32) weigh(c0, std::false_type());
        } else {
#pragma unroll 1
          for (int c0 = 0; ok && c0 < KT; c0 += 32) weigh(c0, std::true_type());
        }
        if (!ok) break;
        tc::tmem_wait_st();
        tc::fence_before_sync();
        tc::mbar_arrive(&bar.p_full[st][jt & 1]);
        begun = true;
        if constexpr (kBF) {
          // Values that are not finite were taken out of the tile (0 * inf in the
          // product would reach the rows that do not see them) and are added here.
          for (uint64_t odd = (uint64_t)in.w << 32 | in.z; odd; odd &= odd - 1) {
            if (!(ok = wait(&bar.p_free[st][jt & 1], jt >> 1))) break;
            tc::fence_after_sync();
            const int i = __ffsll(odd) - 1, key = key0 + i, page = a.c.page;
            const int j = key - w.s.past;
            const bool sees = j < 0 ? key >= first : (bits >> j & 1) != 0;
            const size_t block =
                (size_t)a.c.table[(size_t)w.b * a.c.max_pages + key / page] * 2 + 1;
            const uint4 *v = reinterpret_cast<const uint4 *>(
                static_cast<const char *>(a.c.codes) +
                ((block * a.c.Hkv + w.h) * page + key % page) * C::kRow);
            uint32_t pw[8];
            tc::tmem_ld8(tp + (i & 32) + (i / 2 & 8), pw);
            tc::tmem_wait_ld();
            float p = 0.f;
#pragma unroll
            for (int x = 0; x < 8; ++x)
              if (x == (i / 2 & 7)) p = i & 1 ? bf16_hi(pw[x]) : bf16_lo(pw[x]);
#pragma unroll 1
            for (int c = 0; c < D; c += 8) {
              const uint4 x = v[c / 8];
              const uint32_t y[4] = {x.x & not_finite(x.x), x.y & not_finite(x.y),
                                     x.z & not_finite(x.z), x.w & not_finite(x.w)};
              if ((y[0] | y[1] | y[2] | y[3]) == 0) continue;  // the same for all rows
              uint32_t o[8];
              tc::tmem_ld8(tm + C::kO + c, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t bit = e & 1 ? y[e / 2] & 0xffff0000u : y[e / 2] << 16;
                if (sees && bit)
                  o[e] = __float_as_uint(__uint_as_float(o[e]) + p * __uint_as_float(bit));
              }
              tc::tmem_st8(tm + C::kO + c, o);
              tc::tmem_wait_st();
            }
          }
          if (!ok) break;
          if (in.z | in.w) {
            tc::fence_before_sync();
            tc::mbar_arrive(&bar.added[st]);
          }
        }
      }
      if (!ok) break;
      // the segment's end: all products of the stream
      if (begun) {
        if (!(ok = wait(&bar.p_free[st][jt - 1 & 1], jt - 1 >> 1))) break;
        tc::fence_after_sync();
      }
      const float l = l0 + l1;
      if (st == 1) {
        // (it goes where q lies: the first stream's scores must be done as well)
        if (!(ok = wait(&bar.done, seg))) break;
        mm[row] = -ref;
        ml[row] = l;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          if (c % 64 == 0 && c && !(ok = wait(&bar.merged, seg * C::kRounds + c / 64 - 1))) break;
          uint32_t o[32];
          if (begun) {
            tc::tmem_ld32(tm + C::kO + c, o);
            tc::tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i)
            mo[(c % 64 + i) * 128 + row] = begun ? __uint_as_float(o[i]) : 0.f;
          if (c % 64) tc::mbar_arrive(&bar.merge);
        }
        if (!ok) break;
        tc::fence_before_sync();
      } else {
        tc::mbar_arrive(&bar.done);
        const bool alone = w.from == 0 && w.to == w.s.units;
        float *part = k.part + ((size_t)blockIdx.x * 2 + (w.from == 0)) * 128 * (D + 2);
        float unit = 0.f, other = 0.f, inv = 0.f;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          if (c % 64 == 0) {
            if (!(ok = wait(&bar.merge, seg * C::kRounds + c / 64))) break;
            if (c == 0) {
              const float m1 = mm[row], top = fmaxf(-ref, m1);
              unit = root_of(-ref, top);
              other = root_of(m1, top);
              const float sum = joined(unit, l) + joined(other, ml[row]);
              inv = sum == 0.f ? 0.f : 1.f / sum;
              if (live && !alone) {
                part[128 * D + row] = top;
                part[128 * D + 128 + row] = sum;
              }
            }
          }
          uint32_t o[32];
          tc::tmem_ld32(tm + C::kO + c, o);  // (the first stream has a tile of every segment)
          tc::tmem_wait_ld();
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            y[element_of<F>(i)] = joined(unit, __uint_as_float(o[i])) +
                                  joined(other, mo[(c % 64 + i) * 128 + row]);
          if (c % 64) tc::mbar_arrive(&bar.merged);
          if (live && alone) {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at + c);
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              dst[i / 8] = make_uint4(pack_bf16(y[i] * inv, y[i + 1] * inv),
                                      pack_bf16(y[i + 2] * inv, y[i + 3] * inv),
                                      pack_bf16(y[i + 4] * inv, y[i + 5] * inv),
                                      pack_bf16(y[i + 6] * inv, y[i + 7] * inv));
          } else if (live) {
            float4 *dst = reinterpret_cast<float4 *>(part + row * D + c);
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              dst[i / 4] = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
          }
          __syncwarp();
        }
        if (!ok) break;
        tc::fence_before_sync();
      }
      it += n;
    }
    tc::tmem_wait_st();  // (where a wait has given up between a store and its own)
    tc::fence_before_sync();
  } else if (warp < 12 || warp >= 14) {
    // Where the tiles lie: lane l holds sixteen rows, group l % GP of the (l / GP)th of
    // the warp's next 32 / GP tiles, as their place among all groups of sixteen rows
    // (kNone: nothing to read); the following ones' pages are asked for meanwhile.
    constexpr int GP = KT / 16, AT = 32 / GP;
    const int shift = 31 - __clz(a.c.page), groups = a.c.page >> 4;
    int n = 0;
    auto key_of = [&](int i, int turn) {
      return w.s.first + (w.from + i + lane / GP * turn) * KT + 16 * (lane % GP);
    };
    auto page_of = [&](int i, int turn) {
      const int key = key_of(i, turn);
      return i + lane / GP * turn < n && key < w.s.end
                 ? a.c.table[(size_t)w.b * a.c.max_pages + (key >> shift)]
                 : INT_MIN;
    };
    auto place_of = [&](int i, int turn, int page) -> uint32_t {
      if ((unsigned)page >= (unsigned)a.c.pages) {
        if (page != INT_MIN && a.c.status) atomicCAS(a.c.status, 0, FS_ERR_CACHE);
        return kNone;
      }
      return (uint32_t)(page * 2 * a.c.Hkv + w.h) * groups +
             ((key_of(i, turn) & (a.c.page - 1)) >> 4);
    };
    bool ok = true;
    if constexpr (kBF) {
      // ------------------------ tiles by TMA: keys (warps 8, 9) and values (10, 11) of
      // the even and the odd ones, a warp's tiles one stream's.  Values of tiles that
      // not all rows see whole go through warps 14, 15 first: those of keys that are
      // not there and those that are not finite become zeros.
      const uint32_t mine = warp & 1;
      const bool look_only = warp >= 14, values = warp >= 10;
      const int box = min(groups, 4);      // groups of sixteen rows that come in one copy
      uint32_t looked = 0, landed = 0;     // places whose tile goes by `landed`, and its phases
      uint32_t next = mine;                // the tile after the last that was issued
      while (ok && w.next(k)) {
        n = w.to - w.from;
        const int lead = a.window ? w.s.past + w.s.n - a.window : 0;  // no row begins later
        const int i0 = (it & 1) == mine ? 0 : 1;
        uint32_t place = kNone;
        int later = look_only ? 0 : page_of(i0, 2), at = 0;
#pragma unroll 1
        for (int i = i0; i < n; i += 2) {
          const uint32_t t = it + i, slot = values ? t % NV : t % NK;
          char *dst = (values ? vals : smem) + slot * C::kTile;
          uint32_t *valid = reinterpret_cast<uint32_t *>(side + slot * C::kSide);
          const int key0 = w.s.first + (w.from + i) * KT;
          const bool look = key0 + KT > w.s.past || key0 < lead;
          if (!look_only) {
            if (at == 0) {
              place = place_of(i, 2, later);
              later = page_of(i + 2 * AT, 2);
            }
            const uint32_t turn = values ? t / NV : t / NK;
            if (turn > 0 &&
                !(ok = wait(values ? &bar.vempty[slot] : &bar.kempty[slot], turn - 1)))
              break;
            next = t + 2;
            const uint32_t have = __ballot_sync(~0u, place != kNone) >> (at * GP);
            uint64_t *to = values ? &bar.vfull[slot] : &bar.kfull[slot];
            if (values) {
              looked = looked & ~(1u << slot) | (uint32_t)look << slot;
              landed ^= (uint32_t)look << slot;
              if (look) to = &bar.landed[slot];
              if (lane == 0)
                *reinterpret_cast<uint4 *>(valid) =
                    make_uint4((have & 1 ? 0xffffu : 0u) | (have & 2 ? 0xffff0000u : 0u),
                               (have & 4 ? 0xffffu : 0u) | (have & 8 ? 0xffff0000u : 0u), 0, 0);
            }
            if (lane == 0) tc::mbar_arrive_expect_tx(to, C::kTile);
            __syncwarp();
            if (lane / GP == at && lane % GP % box == 0) {
              // (a group that is not there: before the first one, zeros)
              const int g = place == kNone ? -4 : (int)place + (values ? a.c.Hkv * groups : 0);
#pragma unroll
              for (int c = 0; c < C::kCols; ++c)
                load_group(dst + c * C::kBlock + lane % GP * 2048, &map, to, c * 64, g);
            }
            if (++at == AT) at = 0;
          } else if (look) {
            if (!(ok = wait(&bar.landed[slot], landed >> slot & 1))) break;
            landed ^= 1u << slot;
            uint32_t odd[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int r = half * 32 + lane;
              const bool in = key0 + r < w.s.end;
              uint32_t any = 0;
#pragma unroll 1
              for (int c = 0; c < C::kCols; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  uint4 *x = reinterpret_cast<uint4 *>(dst + c * C::kBlock + swz128(r, j));
                  const uint4 v = *x;
                  const uint4 z = make_uint4(not_finite(v.x), not_finite(v.y), not_finite(v.z),
                                             not_finite(v.w));
                  const uint32_t some = z.x | z.y | z.z | z.w;
                  any |= some;
                  if (!in) {
                    *x = make_uint4(0, 0, 0, 0);
                  } else if (some) {
                    *x = make_uint4(v.x & ~z.x, v.y & ~z.y, v.z & ~z.z, v.w & ~z.w);
                  }
                }
              odd[half] = __ballot_sync(~0u, in && any);
            }
            if (lane == 0) {
              valid[2] = odd[0];
              valid[3] = odd[1];
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bar.vfull[slot]);
          }
        }
        it += n;
      }
      if (!look_only && lane == 0) issued[warp - 8] = {next, looked, landed};
    } else {
      // ------------------------------------------------ codes -> fp16 tiles (warps 8-11)
      // A lane's pieces lie in rows row0 + lane / P + j (32 / P) of the tile, keys and
      // values; it copies them into a ring of its own and turns them into fp16 when
      // they have come.
      constexpr int KW = C::KW, TURN = 4 / C::kMates, CH = 128 / C::kBits / 8;  // chunks of a piece
      const int mate = (warp - 8) % C::kMates, mine = (warp - 8) / C::kMates, row0 = mate * KW;
      const Magic magic = make_magic();
      const int v_off = a.c.Hkv * a.c.page;  // rows from a key to its value
      char *ring = raw + (warp - 8) * kRaws * C::kRaw;
      const char *codes = static_cast<const char *>(a.c.codes) + lane / P * C::kRow + lane % P * 16;
      int chunk_at[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int chunk = lane % P * CH + c;  // of the row's D / 8
        chunk_at[c] = chunk / 8 * C::kBlock + swz128(row0 + lane / P, chunk % 8);
      }
      while (ok && warp < 12 && w.next(k)) {
        n = w.to - w.from;
        const int i0 = (int)((mine - it) % TURN);
        uint32_t place = kNone;
        int later = page_of(i0, TURN), at = 0, ahead = i0;  // the next tile to copy
        auto copy = [&](int slot) {
          if (at == 0) {
            place = place_of(ahead, TURN, later);
            later = page_of(ahead + TURN * AT, TURN);
          }
          char *to = ring + slot * C::kRaw;
          const uint32_t dst = smem_u32(to) + lane * 16;
          const uint32_t sc = smem_u32(to) + C::kRawScale + lane * 8;
          uint32_t *word = reinterpret_cast<uint32_t *>(to + C::kRawScale + KW * 8);
          const int left = w.s.end - w.s.first - (w.from + ahead) * KT;  // keys from the tile's first
          // (kNone in any of the tile's groups, or a tile that ends early)
          if (left >= KT && !__any_sync(~0u, lane / GP == at && place == kNone)) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
              const int r = j * (32 / P);
              const uint32_t g = __shfl_sync(~0u, place, at * GP + (row0 + r) / 16);
              const char *p = codes + ((size_t)g * 16 + r % 16) * C::kRow;
              cp_async16(dst + j * 512, p);
              cp_async16(dst + (NP + j) * 512, p + v_off * C::kRow);
            }
#pragma unroll
            for (int x = 0; x < KW; x += 32) {
              const uint32_t g = __shfl_sync(~0u, place, at * GP + (row0 + x + lane) / 16);
              const float *p = a.c.scales + (size_t)g * 16 + lane % 16;
              cp_async4(sc + x * 8, p);
              cp_async4(sc + x * 8 + 4, p + v_off);
              if (lane == 0) word[x / 32] = ~0u;
            }
          } else {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
              const int r = j * (32 / P);
              const uint32_t g = __shfl_sync(~0u, place, at * GP + (row0 + r) / 16);
              const bool have = g != kNone && row0 + r + lane / P < left;
              const char *p = have ? codes + ((size_t)g * 16 + r % 16) * C::kRow
                                   : static_cast<const char *>(a.c.codes);
              cp_async16z(dst + j * 512, p, have ? 16 : 0);
              cp_async16z(dst + (NP + j) * 512, have ? p + v_off * C::kRow : p, have ? 16 : 0);
            }
#pragma unroll
            for (int x = 0; x < KW; x += 32) {
              const uint32_t g = __shfl_sync(~0u, place, at * GP + (row0 + x + lane) / 16);
              const bool in = g != kNone && row0 + x + lane < left;
              const float *p = in ? a.c.scales + (size_t)g * 16 + lane % 16 : a.c.scales;
              cp_async4z(sc + x * 8, p, in ? 4 : 0);
              cp_async4z(sc + x * 8 + 4, in ? p + v_off : p, in ? 4 : 0);
              const uint32_t some = __ballot_sync(~0u, in);
              if (lane == 0) word[x / 32] = some;
            }
          }
          cp_async_commit();
          ahead += TURN;
          if (++at == AT) at = 0;
        };
#pragma unroll 1
        for (int i = 0; i < kRaws - 1; ++i) copy(i);
        int slot = 0;
#pragma unroll 1
        for (int i = i0; i < n; i += TURN) {
          copy(slot == 0 ? kRaws - 1 : slot - 1);
          cp_async_wait<kRaws - 1>();
          __syncwarp();
          const uint32_t t = it + i;
          const char *src = ring + slot * C::kRaw;
#pragma unroll 1
          for (int part = 0; part < 2; ++part) {  // keys, values
            const uint32_t place = part ? t % NV : t % NK, turn = part ? t / NV : t / NK;
            if (turn > 0 && !(ok = wait(part ? &bar.vempty[place] : &bar.kempty[place], turn - 1)))
              break;
            uint4 x[NP];
#pragma unroll
            for (int j = 0; j < NP; ++j)
              x[j] = *reinterpret_cast<const uint4 *>(src + (part * NP + j) * 512 + lane * 16);
            char *to = (part ? vals : smem) + place * C::kTile;
#pragma unroll
            for (int j = 0; j < NP; ++j) {
              const uint32_t wd[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
              for (int c = 0; c < CH; ++c) {
                uint4 y;
                to_chunk<F>(magic, wd + c * (4 / CH), y);
                // (the swizzle repeats after eight rows)
                *reinterpret_cast<uint4 *>(to + (chunk_at[c] ^ j * (32 / P) % 8 * 16) +
                                           j * (32 / P) * 128) = y;
              }
            }
            if (part) {
              float *sd = reinterpret_cast<float *>(side + place * C::kSide) + row0;
              uint32_t *valid = reinterpret_cast<uint32_t *>(sd - row0 + 3 * KT) + row0 / 32;
#pragma unroll
              for (int y = 0; y < KW; y += 32) {
                const float2 sc =
                    *reinterpret_cast<const float2 *>(src + C::kRawScale + (y + lane) * 8);
                const uint32_t top = __reduce_max_sync(~0u, scale_bits(sc.y));
                sd[y + lane] = sc.x;
                sd[KT + y + lane] = sc.y;
                sd[2 * KT + y + lane] = lg2(fabsf(sc.y));
                if (lane == 0) {
                  valid[y / 32] =
                      *reinterpret_cast<const uint32_t *>(src + C::kRawScale + KW * 8 + y / 8);
                  valid[KT / 32 + y / 32] = __float_as_uint(border<F>(top));
                }
              }
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(part ? &bar.vfull[place] : &bar.kfull[place]);
          }
          if (!ok) break;
          slot = slot + 1 == kRaws ? 0 : slot + 1;
        }
        cp_async_wait<0>();
        __syncwarp();
        it += n;
      }
    }
  } else if (warp < 14 && lane == 0) {
    // ------------------------------------------------------ a stream's products
    const int st = warp - 12;
    const uint32_t tm = tmem_base + st * C::kTmem;
    const uint32_t keys = smem_u32(smem), q = smem_u32(qs);
    constexpr uint32_t kQK = kBF ? tc::idesc_bf16(128, KT, 0) : tc::idesc_f16(128, KT, 0);
    constexpr uint32_t kPV = kBF ? tc::idesc_bf16(128, D, 1) : tc::idesc_f16(128, D, 1);
    constexpr int kPVs = KT / 16 * (kBF ? 2 : 1);  // steps: high parts, low parts
    uint32_t jt = 0, added = 0;
    bool ok = true;
    for (; ok && w.next(k); ++seg) {
      const int n = w.to - w.from;
      if (st == 1) tc::mbar_arrive(&bar.q_full);
      if (!(ok = wait_one(&bar.q_full, seg))) break;
      auto scores = [&](uint32_t j, uint32_t x) -> bool {
        const uint32_t slot = x % NK;
        if (!wait_one(&bar.kfull[slot], x / NK)) return false;
        if (!C::kTwice && j > 0 && !wait_one(&bar.s_free[st], j - 1)) return false;
        tc::fence_after_sync();
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t off = s / 4, in = s % 4 * 32;
          tc::mma_ss(tm + (C::kTwice ? (j & 1) * KT : 0), tc::desc_sw128(q + off * (128 * 128) + in),
                     tc::desc_sw128(keys + slot * C::kTile + off * C::kBlock + in), kQK, s > 0);
        }
        tc::mma_commit(&bar.s_full[st][C::kTwice ? j & 1 : 0]);
        tc::mma_commit(&bar.kempty[slot]);
        return true;
      };
      // one or two tiles of scores ahead of the rows
      if (st < n && !(ok = scores(jt, it + st))) break;
      if (C::kTwice && st + 2 < n && !(ok = scores(jt + 1, it + st + 2))) break;
      for (int i = st; i < n; i += 2, ++jt) {
        const uint32_t slot = (it + i) % NV;
        if (!C::kTwice && i + 2 < n && !(ok = scores(jt + 1, it + i + 2))) break;
        if (!(ok = wait_one(&bar.vfull[slot], (it + i) / NV) && wait_one(&bar.p_full[st][jt & 1], jt >> 1)))
          break;
        tc::fence_after_sync();
        const uint32_t v = smem_u32(vals) + slot * C::kTile;
        uint2 odd = make_uint2(0, 0);
        if constexpr (kBF) odd = *reinterpret_cast<const uint2 *>(side + slot * C::kSide + 8);
#pragma unroll
        for (int s = 0; s < kPVs; ++s)
          tc::mma_ts(tm + C::kO,
                     C::kTwice ? tm + (jt & 1) * KT + s % (KT / 16) / 2 * 32 + s % 2 * 8 +
                                     s / (KT / 16) * 16
                               : tm + KT + s * 8,
                     desc_blocks(v + s % (KT / 16) * 2048, C::kBlock), kPV, i != st || s > 0);
        tc::mma_commit(&bar.p_free[st][jt & 1]);
        tc::mma_commit(&bar.vempty[slot]);
        if ((odd.x | odd.y) && !(ok = wait_one(&bar.added[st], added++))) break;
        // (the scores after the next go where this tile's P lies)
        if (C::kTwice && i + 4 < n &&
            !(ok = wait_one(&bar.p_free[st][jt & 1], jt >> 1) && scores(jt + 2, it + i + 4)))
          break;
      }
      it += n;
    }
  }
  __syncthreads();
  if (fail) {  // nothing may write to shared memory or read TMEM when they are given back
    if constexpr (kBF) {
      if (warp >= 8 && warp < 12 && lane == 0) {
        const Issued s = issued[warp - 8];
        const bool values = warp >= 10;
        const uint32_t held = values ? NV : NK;
        for (uint32_t x = s.next > held ? s.next - held : warp & 1; x < s.next; x += 2)
          if (s.looked >> x % held & 1)
            tc::mbar_wait(&bar.landed[x % held], ~s.landed >> x % held & 1, nullptr);
          else
            tc::mbar_wait(values ? &bar.vfull[x % held] : &bar.kfull[x % held], x / held & 1,
                          nullptr);
      }
    }
    if ((warp == 12 || warp == 13) && lane == 0) {
      tc::mma_commit(&bar.drained[warp - 12]);
      tc::mbar_wait(&bar.drained[warp - 12], 0, nullptr);
    }
    __syncthreads();
    if (tid == 0 && a.c.status) tc::report_error(a.c.status, FS_ERR_TIMEOUT);
  }
  __syncwarp();
  if (warp == 12) tc::tmem_dealloc(tmem_base, 512);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
  static EncodeTiled fn = nullptr;
  if (!fn) {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(ptr);
  }
  return fn;
}

// All rows of the cache as [groups of sixteen][16][d], boxes of 64
// elements of the groups of a page, at most four (a tile).
bool make_cache_map(CUtensorMap *map, const fs_cache &c) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)c.d, 16,
                              (cuuint64_t)c.pages * 2 * c.Hkv * (c.page / 16)};
  const cuuint64_t strides[2] = {(cuuint64_t)c.d * 2, (cuuint64_t)c.d * 32};
  const cuuint32_t box[3] = {64, 16, (cuuint32_t)(c.page >= 64 ? 4 : c.page / 16)};
  const cuuint32_t steps[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, c.codes, dims, strides, box, steps,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int F, int D>
cudaError_t launch_fd(TreeK k, cudaStream_t st) {
  using C = Wide<F, D>;
  k.M = 128;
  k.unit = C::KT;
  k.least = 2;
  k.blocks = kTreeSMs;
  auto fn = k13_tree_wide_kernel<F, D>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  MapOf<F> map;
  if constexpr (C::kBF) {
    if (!make_cache_map(&map, k.a.c)) return cudaErrorInvalidValue;
  }
  fn<<<k.blocks, 512, C::kSmem, st>>>(k, map);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_tree_join(k, st);
}

}  // namespace

cudaError_t launch_tree_wide(const TreeK &k, cudaStream_t st) {
  const bool small = k.a.c.d == 64;
  switch (k.a.c.format) {
    case FS_CACHE_E4M3:
      return small ? launch_fd<FS_CACHE_E4M3, 64>(k, st) : launch_fd<FS_CACHE_E4M3, 128>(k, st);
    case FS_CACHE_INT8:
      return small ? launch_fd<FS_CACHE_INT8, 64>(k, st) : launch_fd<FS_CACHE_INT8, 128>(k, st);
    case FS_CACHE_INT4:
      return small ? launch_fd<FS_CACHE_INT4, 64>(k, st) : launch_fd<FS_CACHE_INT4, 128>(k, st);
    default:
      return small ? launch_fd<FS_CACHE_BF16, 64>(k, st) : launch_fd<FS_CACHE_BF16, 128>(k, st);
  }
}

}  // namespace fs
