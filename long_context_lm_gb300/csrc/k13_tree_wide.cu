// k13_tree_wide.cu -- fs_tree_attn where many rows share their keys (a wide
// tree, or grouped heads): 128 rows a block on the tensor cores (tcgen05).
//
// The line of units, its sharing and the joining of the blocks' results are
// k12_tree.cu's; a unit here is a tile of KT keys.  A block works on one
// segment at a time:
//   * warps 8-11 turn codes into fp16 tiles in shared memory (exact: codes have
//     at most 8 bits), a ring of them, with the scales beside them;
//   * two streams of four warps take the tiles in turn, a thread a row, each
//     stream with its own scores, probabilities, output (TMEM), running
//     reference and sum, so that neither waits for the other;
//   * one thread of warp 12 (13) issues the first (second) stream's products:
//     the next tile's S = Q K^T as soon as the rows have read this one's, then
//     O += P V with P from TMEM.
// The streams are joined through shared memory at the end of a segment.
//
// Scores, scales, references and probabilities are as in k12_tree.cu (q by a
// power of two a row, fp16 probabilities up to 2^15, value scales relative to a
// power of two that is part of the exponent here).  Where a score passes its
// row's reference by more than 8 (log2), the reference is raised to it before the 32
// columns are weighed: the row's sum, its O (between two products) and its
// earlier probabilities of the tile are multiplied by the difference.
//
// Bound by: the exponentials and the roughly five operations around each
// (128 x KT a tile), then the products' issue.
#include "tree.cuh"

namespace fs {
namespace {

template <int F, int D>
struct Wide {
  static constexpr int kBits = Fmt<F>::kBits;
  static constexpr int kRow = D * kBits / 8, P = kRow / 16;
  static constexpr int KT = D == 64 ? 128 : 64;  // keys of a tile
  static constexpr int kCols = D / 64;           // 64-element column blocks
  static constexpr int kBlock = KT * 128;        // bytes of one of them
  static constexpr int kStage = 2 * kCols * kBlock;
  static constexpr int kStages = 4;
  // a tile's codes, a scale pair a thread and four valid words
  static constexpr int kRawScale = KT * kRow * 2, kRaw = kRawScale + 1024 + 16;
  static constexpr int kQ = 128 * 128 * kCols;
  static constexpr int kMerge = 128 * (64 + 2) * 4;  // begins in place of q
  static constexpr int kRounds = D / 64;  // of handing it over
  static constexpr int kSide = KT * 8 + 64;  // scales, 4 valid words, 4 largest value scales
  static constexpr int kRest = 1024 + kStage * kStages + kMerge + kSide * kStages + 256;
  static constexpr int kFit = (226 * 1024 - kRest) / kRaw;
  static constexpr int kRaws = kFit > 5 ? 5 : kFit;  // tiles of codes under way
  static constexpr int kSmem = kRest + kRaws * kRaw;
  // TMEM columns of a stream: S, P, O
  static constexpr int kS = 0, kP = KT, kO = KT + KT / 2, kTmem = 256;
  static_assert(128 / P % 16 == 0 && kO + D <= kTmem && kRaws >= 2 && kQ <= kMerge, "sizes");
  static constexpr int NP = KT * P / 128;  // pieces of a thread, keys or values
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
__device__ __forceinline__ bool wait_asleep(uint64_t *bar, uint32_t parity, int *fail) {
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
        : "memory");
    if (ok) return true;
    if ((i & 15u) == 0) {
      if (clock64() - t0 > tc::kWaitCycles) break;
      if (*reinterpret_cast<volatile int *>(fail) != 0) return false;
    }
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
  uint64_t full[4], empty[4];           // tiles
  uint64_t s_full[2], s_free[2];     // a stream's scores
  uint64_t p_full[2], p_free[2];        // a stream's probabilities
  uint64_t q_full, done, merge, merged;  // of a segment
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

template <int F, int D>
__global__ void __launch_bounds__(512, 1) k13_tree_wide_kernel(const __grid_constant__ TreeK k) {
  using C = Wide<F, D>;
  constexpr int KT = C::KT, P = C::P, NS = C::kStages, NP = C::NP;
  constexpr int kRaws = C::kRaws;
  extern __shared__ char smem_raw[];
  char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  char *qs = smem + NS * C::kStage;
  float *mo = reinterpret_cast<float *>(qs);  // 64 columns of the second stream's O, over q
  float *mm = mo + 128 * 64, *ml = mm + 128;
  char *side = reinterpret_cast<char *>(ml + 128);
  Bars &bar = *reinterpret_cast<Bars *>(side + NS * C::kSide);
  char *raw = side + NS * C::kSide + 256;
  __shared__ uint32_t tmem_base;
  __shared__ int fail;
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
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(&bar.full[i], 128);
      tc::mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bar.s_full[i], 1);
      tc::mbar_init(&bar.s_free[i], 128);
      tc::mbar_init(&bar.p_full[i], 128);
      tc::mbar_init(&bar.p_free[i], 1);
    }
    tc::mbar_init(&bar.q_full, 128);
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
  // loops for the barrier at the end.
  auto wait_one = [&](uint64_t *b, uint32_t phase) { return wait_asleep(b, phase & 1, &fail); };
  auto wait = [&](uint64_t *b, uint32_t phase) {  // the same answer in a warp
    return (bool)__all_sync(~0u, wait_one(b, phase));
  };
  int it = 0;  // tiles of the block before the current segment
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
      const float f = __uint_as_float((uint32_t)min(254, 268 - (int)(most >> 7)) << 23);
      const float rf = fmaxf(a.scale * kLog2e * (1.f / f), FLT_MIN);
      if (st == 0) {
        // (the second stream's results lay there)
        if (seg > 0 && !(ok = wait(&bar.merged, seg * C::kRounds - 1))) break;
#pragma unroll 2
        for (int i = 0; i < D / 8; ++i) {
          const uint4 x = live ? src[i] : make_uint4(0, 0, 0, 0);
          const uint32_t y[4] = {x.x, x.y, x.z, x.w};
          uint32_t z[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e0 = element_of<F>(2 * j), e1 = element_of<F>(2 * j + 1);
            const float v0 = e0 % 2 ? bf16_hi(y[e0 / 2]) : bf16_lo(y[e0 / 2]);
            const float v1 = e1 % 2 ? bf16_hi(y[e1 / 2]) : bf16_lo(y[e1 / 2]);
            z[j] = pack_f16(v0 * f, v1 * f);
          }
          *reinterpret_cast<uint4 *>(qs + i / 8 * (128 * 128) + swz128(row, i % 8)) =
              make_uint4(z[0], z[1], z[2], z[3]);
        }
        tc::fence_async_smem();
        tc::mbar_arrive(&bar.q_full);
      } else if (!(ok = wait(&bar.q_full, seg))) {  // (the last segment's results have been taken)
        break;
      }

      float m = -FLT_MAX, thr = -INFINITY, l0 = 0.f, l1 = 0.f, vref = kLeast;
      bool begun = false;  // O holds something
      // O *= by, once the last tile's product has ended (this one's has not begun)
      auto rescale = [&](float by) -> bool {
        if (jt > 0 && !wait(&bar.p_free[st], jt - 1)) return false;
        tc::fence_after_sync();
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {  // (few registers: 32 columns wait meanwhile)
          uint32_t o[16];
          tc::tmem_ld16(tm + C::kO + c, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
          tc::tmem_st16(tm + C::kO + c, o);
        }
        tc::tmem_wait_st();
        return true;
      };

      int stage = (it + st) % NS;
      uint32_t round = (uint32_t)((it + st) / NS);
      for (int i = st; ok && i < n; i += 2, ++jt) {
        const float *ks = reinterpret_cast<const float *>(side + stage * C::kSide);
        const uint32_t *valid = reinterpret_cast<const uint32_t *>(ks + 2 * KT);
        if (!(ok = wait(&bar.full[stage], round) && wait(&bar.s_full[st], jt))) break;
        if ((stage += 2) >= NS) {
          stage -= NS;
          ++round;
        }
        tc::fence_after_sync();
        const int key0 = w.s.first + (w.from + i) * KT;
        const uint4 in = *reinterpret_cast<const uint4 *>(valid);
        const float4 tops = *reinterpret_cast<const float4 *>(valid + 4);
        const bool whole = (KT == 128 ? in.x & in.y & in.z & in.w : in.x & in.y) == ~0u &&
                           __all_sync(~0u, key0 + KT <= w.s.past && key0 >= first);
        const float top_v = KT == 128 ? fmaxf(fmaxf(tops.x, tops.y), fmaxf(tops.z, tops.w))
                                      : fmaxf(tops.x, tops.y);
        if (top_v > vref) {  // the same for all rows
          const float up =
              __uint_as_float((__float_as_uint(top_v) + 0x7fffffu) & 0x7f800000u);
          const float back = vref / up;
          if (begun && !(ok = rescale(back))) break;
          l0 *= back;
          l1 *= back;
          vref = up;
        }
        const float lift = 15.f - kRaise - (float)((int)(__float_as_uint(vref) >> 23) - 127);

        // The columns, 32 at a time.
        auto weigh = [&](int c0, auto masked) {
          uint32_t u[32];
          tc::tmem_ld32(tm + C::kS + c0, u);
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
          if (c0 + 32 == KT) {  // the next tile's scores may be made
            tc::fence_before_sync();
            tc::mbar_arrive(&bar.s_free[st]);
          }
          // Step by step over all 32 columns: each step's operations do not wait
          // for one another.
          float y[32];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 kk = *reinterpret_cast<const float4 *>(ks + c0 + j);
            y[j] = __uint_as_float(u[j]), y[j + 1] = __uint_as_float(u[j + 1]);
            y[j + 2] = __uint_as_float(u[j + 2]), y[j + 3] = __uint_as_float(u[j + 3]);
            mul2(y[j], y[j + 1], kk.x, kk.y);
            mul2(y[j + 2], y[j + 3], kk.z, kk.w);
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
          if (__any_sync(~0u, t0 > thr)) {  // raise the rows' references
            // by a whole number, so that the factor is a power of two: exact for the
            // fp16 probabilities that are made already
            const float by_log2 = ceilf(fmaxf(t0 * rf - m, 0.f));
            const bool none = m == -FLT_MAX;  // the row has seen no key
            const float back = none ? 0.f : exp2f(-by_log2);
            m = none ? fmaxf(t0 * rf, -FLT_MAX) : m + by_log2;
            if (m > -FLT_MAX) thr = (m + kRaise) / rf;
            l0 *= back;
            l1 *= back;
            if (begun) ok = rescale(back);
#pragma unroll 1
            for (int c = 0; c < c0 / 2; c += 8) {  // this tile's earlier columns
              uint32_t z[8];
              tc::tmem_wait_st();
              tc::tmem_ld8(tm + C::kP + c, z);
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&z[i]));
                z[i] = pack_f16(f.x * back, f.y * back);
              }
              tc::tmem_st8(tm + C::kP + c, z);
            }
          }
          const float ref = lift - m;
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
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) p[j / 2] = pack_f16(y[j], y[j + 1]);
          if (c0 == 0 && jt > 0) {  // the last tile's product has read P
            ok = wait(&bar.p_free[st], jt - 1) && ok;
            tc::fence_after_sync();
          }
          tc::tmem_st16(tm + C::kP + c0 / 2, p);
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
        tc::mbar_arrive(&bar.p_full[st]);
        begun = true;
      }
      if (!ok) break;
      // the segment's end: all products of the stream
      if (begun) {
        if (!(ok = wait(&bar.p_free[st], jt - 1))) break;
        tc::fence_after_sync();
      }
      const float l = (l0 + l1) * vref;
      if (st == 1) {
        // (it goes where q lies: the first stream's scores must be done as well)
        if (!(ok = wait(&bar.done, seg))) break;
        mm[row] = m;
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
            mo[(c % 64 + i) * 128 + row] = begun ? __uint_as_float(o[i]) * vref : 0.f;
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
              const float m1 = mm[row], top = fmaxf(m, m1), f0 = exp2f(m - top);
              other = exp2f(m1 - top);
              const float sum = f0 * l + other * ml[row];
              unit = f0 * vref;
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
            y[element_of<F>(i)] =
                __uint_as_float(o[i]) * unit + mo[(c % 64 + i) * 128 + row] * other;
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
  } else if (warp < 12) {
    // -------------------------------------------------- codes -> fp16 tiles
    const int t = tid - 256, shift = 31 - __clz(a.c.page);
    const Magic magic = make_magic();
    const int v_off = a.c.Hkv * a.c.page;  // rows from a key to its value
    bool ok = true;
    while (ok && w.next(k)) {
      // A thread's pieces lie in rows t / P + j (128 / P), keys and values; it
      // copies them into a ring of its own and turns them into fp16 when they
      // have come.  Its scale belongs to key t % KT.
      //
      // Where the tiles lie: lane l holds sixteen rows, group l % GP of tile
      // l / GP of the 32 / GP tiles looked up at a time, as their place among all
      // groups of sixteen rows (kNone: nothing to read); the next ones' pages are
      // asked for that many tiles ahead.
      constexpr int GP = KT / 16, AT = 32 / GP;
      const int n = w.to - w.from, key_s = t & (KT - 1), groups = a.c.page >> 4;
      auto key_of = [&](int i) {
        return w.s.first + (w.from + i + lane / GP) * KT + 16 * (lane % GP);
      };
      auto page_of = [&](int i) {
        const int key = key_of(i);
        return i + lane / GP < n && key < w.s.end
                   ? a.c.table[(size_t)w.b * a.c.max_pages + (key >> shift)]
                   : INT_MIN;
      };
      auto place_of = [&](int i, int page) -> uint32_t {
        if ((unsigned)page >= (unsigned)a.c.pages) {
          if (page != INT_MIN && a.c.status) atomicCAS(a.c.status, 0, FS_ERR_CACHE);
          return kNone;
        }
        return (uint32_t)(page * 2 * a.c.Hkv + w.h) * groups + ((key_of(i) & (a.c.page - 1)) >> 4);
      };
      uint32_t place = place_of(0, page_of(0));
      int later = page_of(AT), at = 0, left = w.s.end - w.s.first - w.from * KT;  // keys from here
      const char *codes = static_cast<const char *>(a.c.codes) +
                          (t / P % 16) * C::kRow + t % P * 16;  // the thread's piece of a group
      auto copy = [&](int slot) {
        const uint32_t dst = smem_u32(raw) + slot * C::kRaw + t * 16;
        const uint32_t to = smem_u32(raw) + slot * C::kRaw + C::kRawScale + t * 8;
        uint32_t *word = reinterpret_cast<uint32_t *>(raw + slot * C::kRaw + C::kRawScale + 1024) +
                         (t >> 5);
        const uint32_t gs = __shfl_sync(~0u, place, at * GP + key_s / 16);
        // (kNone in any of the tile's groups, or a tile that ends early)
        if (left >= KT && !__any_sync(~0u, lane / GP == at && place == kNone)) {
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const uint32_t g = __shfl_sync(~0u, place, at * GP + (t / P + j * (128 / P)) / 16);
            const char *p = codes + (size_t)g * (16 * C::kRow);
            cp_async16(dst + j * 2048, p);
            cp_async16(dst + (NP + j) * 2048, p + v_off * C::kRow);
          }
          const float *p = a.c.scales + (size_t)gs * 16 + key_s % 16;
          cp_async4(to, p);
          cp_async4(to + 4, p + v_off);
          if (lane == 0) *word = ~0u;
        } else {
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const int r = t / P + j * (128 / P);
            const uint32_t g = __shfl_sync(~0u, place, at * GP + r / 16);
            const bool have = g != kNone && r < left;
            const char *p = have ? codes + (size_t)g * (16 * C::kRow)
                                 : static_cast<const char *>(a.c.codes);
            cp_async16z(dst + j * 2048, p, have ? 16 : 0);
            cp_async16z(dst + (NP + j) * 2048, have ? p + v_off * C::kRow : p, have ? 16 : 0);
          }
          const bool in = gs != kNone && key_s < left;
          const float *p = in ? a.c.scales + (size_t)gs * 16 + key_s % 16 : a.c.scales;
          cp_async4z(to, p, in ? 4 : 0);
          cp_async4z(to + 4, in ? p + v_off : p, in ? 4 : 0);
          const uint32_t some = __ballot_sync(~0u, in);
          if (lane == 0) *word = some;
        }
        cp_async_commit();
        left -= KT;
        if (++at == AT) at = 0;
      };
      int ahead = 0;  // tiles copied
      auto copy_next = [&](int slot) {
        if (at == 0 && ahead) {
          place = place_of(ahead, later);
          later = page_of(ahead + AT);
        }
        copy(slot);
        ++ahead;
      };
#pragma unroll 1
      for (int i = 0; i < kRaws - 1; ++i) copy_next(i);
      int slot = 0, stage = it % NS;
      uint32_t round = (uint32_t)(it / NS);
      int chunk_at[128 / C::kBits / 8];
#pragma unroll
      for (int c = 0; c < 128 / C::kBits / 8; ++c) {
        const int chunk = t % P * (128 / C::kBits / 8) + c;  // of the row's D / 8
        chunk_at[c] = chunk / 8 * C::kBlock + swz128(t / P, chunk % 8);
      }
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        copy_next(slot == 0 ? kRaws - 1 : slot - 1);
        cp_async_wait<kRaws - 1>();
        if (round > 0 && !(ok = wait(&bar.empty[stage], round - 1))) break;
        const char *src = raw + slot * C::kRaw;
        char *dst = smem + stage * C::kStage;
        // (the row's place in the swizzle is the same for all of the thread's rows:
        // they lie a multiple of eight apart)
        constexpr int CH = 128 / C::kBits / 8;  // chunks of the piece: 2 or 4
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          uint4 x[NP];
#pragma unroll
          for (int j = 0; j < NP; ++j)
            x[j] = *reinterpret_cast<const uint4 *>(src + (part * NP + j) * 2048 + t * 16);
          char *to = dst + part * (C::kCols * C::kBlock);
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const uint32_t wd[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              uint4 y;
              to_chunk<F>(magic, wd + c * (4 / CH), y);
              *reinterpret_cast<uint4 *>(to + chunk_at[c] + j * (128 / P) * 128) = y;
            }
          }
        }
        const float2 sc = *reinterpret_cast<const float2 *>(src + C::kRawScale + t * 8);
        const uint32_t word = *reinterpret_cast<const uint32_t *>(src + C::kRawScale + 1024 + (t >> 5) * 4);
        const uint32_t top =
            __reduce_max_sync(~0u, sc.y <= FLT_MAX ? __float_as_uint(fmaxf(sc.y, 0.f)) : 0u);
        if (t < KT) {
          float *sd = reinterpret_cast<float *>(side + stage * C::kSide);
          sd[t] = sc.x;
          sd[KT + t] = sc.y;
          if (lane == 0) {
            uint32_t *valid = reinterpret_cast<uint32_t *>(sd + 2 * KT);
            valid[t / 32] = word;
            valid[4 + t / 32] = top;
          }
        }
        tc::fence_async_smem();
        tc::mbar_arrive(&bar.full[stage]);
        slot = slot + 1 == kRaws ? 0 : slot + 1;
        if (++stage == NS) {
          stage = 0;
          ++round;
        }
        __syncwarp();
      }
      cp_async_wait<0>();
      it += n;
    }
  } else if (warp < 14 && lane == 0) {
    // ------------------------------------------------------ a stream's products
    const int st = warp - 12;
    const uint32_t tm = tmem_base + st * C::kTmem;
    const uint32_t ring = smem_u32(smem), q = smem_u32(qs);
    constexpr uint32_t kQK = tc::idesc_f16(128, KT, 0), kPV = tc::idesc_f16(128, 64, 1);
    uint32_t jt = 0;
    bool ok = true;
    for (; ok && w.next(k); ++seg) {
      const int n = w.to - w.from;
      if (!(ok = wait_one(&bar.q_full, seg))) break;
      int stage = (it + st) % NS;  // of the next scores
      uint32_t round = (uint32_t)((it + st) / NS);
      auto scores = [&](uint32_t j) -> bool {
        if (!wait_one(&bar.full[stage], round)) return false;
        if (j > 0 && !wait_one(&bar.s_free[st], j - 1)) return false;
        tc::fence_after_sync();
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t off = s / 4, in = s % 4 * 32;
          tc::mma_ss(tm + C::kS, tc::desc_sw128(q + off * (128 * 128) + in),
                     tc::desc_sw128(ring + stage * C::kStage + off * C::kBlock + in), kQK, s > 0);
        }
        tc::mma_commit(&bar.s_full[st]);
        if ((stage += 2) >= NS) {
          stage -= NS;
          ++round;
        }
        return true;
      };
      int now = stage;  // of the values
      if (st < n && !(ok = scores(jt))) break;
      for (int i = st; i < n; i += 2, ++jt) {
        // the next tile's scores first: they are there when this one's rows are done
        if (i + 2 < n && !(ok = scores(jt + 1))) break;
        if (!(ok = wait_one(&bar.p_full[st], jt))) break;
        tc::fence_after_sync();
        const uint32_t v = ring + now * C::kStage + C::kCols * C::kBlock;
#pragma unroll
        for (int c = 0; c < C::kCols; ++c)
#pragma unroll
          for (int s = 0; s < KT / 16; ++s)
            tc::mma_ts(tm + C::kO + c * 64, tm + C::kP + s * 8,
                       tc::desc_sw128(v + c * C::kBlock + s * 2048), kPV, i != st || s > 0);
        tc::mma_commit(&bar.p_free[st]);
        tc::mma_commit(&bar.empty[now]);
        now = now + 2 >= NS ? now + 2 - NS : now + 2;
      }
      it += n;
    }
  }
  __syncthreads();
  if (tid == 0 && fail && a.c.status) tc::report_error(a.c.status, FS_ERR_TIMEOUT);
  __syncwarp();
  if (warp == 12) tc::tmem_dealloc(tmem_base, 512);
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
  fn<<<k.blocks, 512, C::kSmem, st>>>(k);
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
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fs
