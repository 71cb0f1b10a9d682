// tree.cuh -- what the two kernels of fs_tree_attn share: how the work is cut
// and shared out, where an output row lies, and codes as fp16 numbers.
#pragma once

#include <float.h>
#include <limits.h>

#include <type_traits>

#include "cache.cuh"
#include "tc05.cuh"

namespace fs {

constexpr float kLog2e = 1.4426950408889634f;

// Products with a row of q that was multiplied by f -> scores in log2 units.  Not 0, which a
// masked score's -inf may not meet; below fp32's normal range (q below 2^-110) it is
// off by 2^-150, a score by 2^-22.
__device__ __forceinline__ float log2_factor(float scale, float f) {
  return fmaxf(scale * kLog2e * (1.f / f), 0x1p-149f);
}

// ---------------------------------------------------------------------------
// references
// ---------------------------------------------------------------------------
// A row's probabilities are p = 2^(score + ref), scores in log2 units; its weights,
// which go into the product with the values, are p, or p times the value's scale where
// values are codes.  Sum and output are relative to the row's own reference, which what
// other rows see cannot move.  FLT_MAX: the row has seen no key.  A reference moves when a
// key that the row sees passes kHigh, and by so much that the largest is at kLow:
//   bf16   p alone; its parts are bf16 numbers, so that any range has the same bits.  2^-30
//          to 2^-14 leaves room for sums of 2^14 of bf16's largest values, and 96 binary
//          places below the largest p (the lower part's 8 bits: 87), which count where
//          a key of next to no probability has values that much larger.
//   codes  weights go to fp16, whose largest number is below 2^16; the row's largest stays
//          at 2^7 or more, 2^31 times the step of the smallest ones.  A second border, on p,
//          keeps the sums of 2^30 keys within fp32 where values are tiny or zero (it
//          costs weights bits where the largest value scale is below 2^-78, and p loses keys
//          2^-20 of the largest, below 2^-126, where that scale is above 2^113).
// Moving one costs the tcgen05 kernel a pass over its O: with 4, 8 and 12 between kLow and
// kHigh 64 tokens x 32 heads over 16384 int8 keys take 187, 167 and 158 us.
template <int F>
struct Range {
  static constexpr bool kBF = F == FS_CACHE_BF16;
  static constexpr float kLow = kBF ? -30.f : 8.f, kHigh = kBF ? -14.f : 15.99f;
  static constexpr float kSumLow = 85.f, kSumHigh = 93.f;
};

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// Bits of a value scale's magnitude, 0 for one that is not a number (its row's values are
// not either).
__device__ __forceinline__ uint32_t scale_bits(float x) {
  return fabsf(x) <= FLT_MAX ? __float_as_uint(fabsf(x)) : 0u;
}
// What a row's largest score plus reference may be, over keys whose value scales are at
// most the number with the bits `top`: below it no weight and no p passes its border.
template <int F>
__device__ __forceinline__ float border(uint32_t top) {
  using R = Range<F>;
  if constexpr (R::kBF) return R::kHigh;
  return R::kHigh - fmaxf(lg2(__uint_as_float(top)), R::kHigh - R::kSumHigh);
}
// A row's reference for keys whose largest score is `score`, and whose largest score plus
// log2 of the value scale is `weight` (codes), where some row of the warp has passed its border.
// It moves by whole numbers, so that what is there is multiplied by a power of two, and
// wherever the largest is above kLow: the warp pays for all its rows or none.
template <int F>
__device__ __forceinline__ float moved(float ref, float score, [[maybe_unused]] float weight) {
  using R = Range<F>;
  if (score == -INFINITY) return ref;  // none that the row sees
  if (ref == FLT_MAX)
    return R::kBF ? R::kLow - score : fminf(R::kLow - weight, R::kSumLow - score);
  if constexpr (R::kBF) return ref - ceilf(fmaxf(score + ref - R::kLow, 0.f));
  return ref - ceilf(fmaxf(fmaxf(weight + ref - R::kLow, score + ref - R::kSumLow), 0.f));
}
// 2^(to - from) as two factors: from the smallest values to the largest it is below 2^-149,
// while sums that it multiplies stay far above.  (The difference of two references is a
// whole number but for the last one's rounding.)
struct Back {
  float a, b;
  __device__ __forceinline__ Back(float from, float to) {
    const int n = __float2int_rn(fmaxf(to - from, -252.f)), h = n >> 1;
    a = __uint_as_float((uint32_t)(127 + h) << 23);
    b = __uint_as_float((uint32_t)(127 + n - h) << 23);
  }
  __device__ __forceinline__ float operator()(float x) const { return x * a * b; }
};
// Results with references -m are joined at the largest m of them: a factor of 2^(m - most),
// applied as its square root twice, for the same reason.
__device__ __forceinline__ float root_of(float m, float most) { return exp2f(0.5f * (m - most)); }
__device__ __forceinline__ float joined(float root, float x) { return root * x * root; }
// ---------------------------------------------------------------------------
// the line of units
// ---------------------------------------------------------------------------
struct Seq {
  int past, n, first, end;  // prefix, drafted tokens, keys [first, end) that any row sees
  int units, tiles;         // units of a segment, row tiles of a kv head
};

struct TreeK {
  TreeArgs a;
  int G, M;           // query heads of a kv head, rows of a tile
  int unit;           // keys of a unit (a power of two)
  int blocks, least;  // blocks of the launch, units that make a block worth it
  float *part;  // [blocks][2][M][D + 2]: O, m, l
};

constexpr int kTreeSMs = 152;
// The second kernel, and the first for many rows.
cudaError_t launch_tree_join(const TreeK &k, cudaStream_t st);
cudaError_t launch_tree_wide(const TreeK &k, cudaStream_t st);

__device__ __forceinline__ Seq seq_of(const TreeK &k, int b) {
  Seq s;
  const int limit = k.a.c.max_pages * k.a.c.page;  // at most 2^30
  const int past = k.a.past[b];
  s.n = k.a.count ? min(max(k.a.count[b], 0), k.a.T) : k.a.T;
  s.past = min(max(past, 0), limit);
  s.end = min(s.past + s.n, limit);
  // (a row that sees i drafted tokens begins at past + i - window)
  s.first = k.a.window ? max(0, s.past - k.a.window) & ~(k.unit - 1) : 0;
  s.units = (s.end - s.first + k.unit - 1) / k.unit;
  s.tiles = (s.n * k.G + k.M - 1) / k.M;
  if (s.n == 0) s.units = 0;
  return s;
}
__device__ __forceinline__ long long seq_units(const TreeK &k, const Seq &s) {
  return (long long)s.units * s.tiles * k.a.c.Hkv;
}
__device__ __forceinline__ bool seq_outside(const TreeK &k, int b) {
  const int past = k.a.past[b];
  const int n = k.a.count ? min(max(k.a.count[b], 0), k.a.T) : k.a.T;
  return n > 0 && (past < 0 || (long long)past + n > (long long)k.a.c.max_pages * k.a.c.page);
}

// a / b; nearly always both fit 32 bits, whose division is several times faster.
__device__ __forceinline__ long long quot(long long a, int b) {
  return a >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}
// How the line is shared: at most one block for every `least` units; the first `more` blocks have a unit more than the others.
struct Share {
  int blocks = 1, more = 0;
  long long each = 0;
  Share() = default;
  __device__ __forceinline__ Share(const TreeK &k, long long total) {
    const long long n = quot(total + k.least - 1, k.least);
    blocks = (int)(n < k.blocks ? (n < 1 ? 1 : n) : k.blocks);
    each = quot(total, blocks);
    more = (int)(total - each * blocks);
  }
  __device__ __forceinline__ long long begin(int c) const { return c * each + min(c, more); }
  // the block that holds unit u
  __device__ __forceinline__ int of(long long u) const {
    const long long first = more * (each + 1);
    if (each >> 31) return (int)(u < first ? u / (each + 1) : more + (u - first) / each);
    return (int)(u < first ? quot(u, (int)each + 1) : more + quot(u - first, (int)each));
  }
};

// Length of the line, how it is shared, and of the one sequence that
// `pick(share, b, begin, end)` chooses (the units [begin, end) are its own) the
// number, beginning and sizes.  Called by all threads of a block.
struct Line {
  long long total, begin;
  Share share;
  int b;
  Seq s;
};
template <class Pick>
__device__ __forceinline__ Line line_of(const TreeK &k, const Pick &pick) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  if (k.a.c.batch <= 32) {  // every warp for itself
    Seq s{};
    long long u = 0;
    if (lane < k.a.c.batch) {
      s = seq_of(k, lane);
      u = seq_units(k, s);
    }
    long long x = u;
#pragma unroll 1
    for (int o = 1; o < k.a.c.batch; o <<= 1) {
      const long long y = __shfl_up_sync(~0u, x, o);
      if (lane >= o) x += y;
    }
    Line out;
    out.total = __shfl_sync(~0u, x, k.a.c.batch - 1);
    out.share = Share(k, out.total);
    const uint32_t mine =
        __ballot_sync(~0u, lane < k.a.c.batch && pick(out.share, lane, x - u, x));
    out.b = mine ? __ffs(mine) - 1 : 0;
    out.begin = __shfl_sync(~0u, x - u, out.b);
    out.s.past = __shfl_sync(~0u, s.past, out.b);
    out.s.n = __shfl_sync(~0u, s.n, out.b);
    out.s.first = __shfl_sync(~0u, s.first, out.b);
    out.s.end = __shfl_sync(~0u, s.end, out.b);
    out.s.units = __shfl_sync(~0u, s.units, out.b);
    out.s.tiles = __shfl_sync(~0u, s.tiles, out.b);
    return out;
  }
  __shared__ long long sh[16];
  __shared__ Line found;
  const bool once = k.a.c.batch <= (int)blockDim.x;
  long long total = 0;
  Share share;
#pragma unroll 1
  for (int round = once ? 1 : 0; round < 2; ++round) {  // a long batch goes through twice
    long long before_all = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < k.a.c.batch; b0 += blockDim.x) {
      const int b = b0 + tid;
      Seq s{};
      long long u = 0;
      if (b < k.a.c.batch) {
        s = seq_of(k, b);
        u = seq_units(k, s);
      }
      long long x = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
      }
      if (b0) __syncthreads();
      if (lane == 31) sh[warp] = x;
      __syncthreads();
      long long all = 0;
      for (int w = 0; w < nw; ++w) {
        if (w < warp) x += sh[w];
        all += sh[w];
      }
      x += before_all;
      before_all += all;
      if (once) share = Share(k, total = all);
      if (round == 1 && b < k.a.c.batch && pick(share, b, x - u, x)) {
        found.b = b;
        found.begin = x - u;
        found.s = s;
      }
    }
    if (!once) share = Share(k, total = before_all);
    __syncthreads();
  }
  Line out = found;
  out.total = total;
  out.share = share;
  return out;
}

__device__ __forceinline__ uint32_t h2add(uint32_t a, uint32_t b) {
  __half2 r = __hadd2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
  return *reinterpret_cast<uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t h2fma(uint32_t a, uint32_t b, uint32_t c) {
  __half2 r = __hfma2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b),
                      *reinterpret_cast<__half2 *>(&c));
  return *reinterpret_cast<uint32_t *>(&r);
}
// Constants that stay in registers: the compiler would load one of the two that
// most of these operations take anew for every one of them.
struct Magic {
  uint32_t even, odd;   // nibbles 0 and 4, 1 and 5
  uint32_t magic;       // fp16 1024, whose step is 1
  uint32_t sixteenth, sub72;
};
__device__ __forceinline__ Magic make_magic() {
  Magic m;
  asm volatile("mov.b32 %0, 0x000f000f;" : "=r"(m.even));
  asm volatile("mov.b32 %0, 0x00f000f0;" : "=r"(m.odd));
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(m.magic));
  asm volatile("mov.b32 %0, 0x2c002c00;" : "=r"(m.sixteenth));
  asm volatile("mov.b32 %0, 0xd480d480;" : "=r"(m.sub72));  // -(64 + 8)
  return m;
}
constexpr uint32_t kSub128 = 0xe480e480u;  // -(1024 + 128)
constexpr uint32_t kSub8 = 0xe408e408u;    // -(1024 + 8)
// Nibbles 0 and 4, or 1 and 5, with their sign bits flipped (code + 8) in the
// same step that puts them into the magic number.
__device__ __forceinline__ uint32_t nib_even(const Magic &m, uint32_t x) {
  return h2add((x & m.even) ^ 0x64086408u, kSub8);
}
__device__ __forceinline__ uint32_t nib_odd(const Magic &m, uint32_t x) {
  return h2fma((x & m.odd) ^ 0x64806480u, m.sixteenth, m.sub72);
}

// (x, y) *= (a, b) and (x, y) = (x, y) * m + c on packed fp32 pairs.
__device__ __forceinline__ void mul2(float &x, float &y, float a, float b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(x, y)), "l"(f2_bits(a, b)));
  x = __uint_as_float((uint32_t)r);
  y = __uint_as_float((uint32_t)(r >> 32));
}

// Asynchronous copies of 16 and 4 bytes; with bytes = 0 zeros are written and
// nothing is read.
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src));
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src));
}
__device__ __forceinline__ void cp_async4z(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(bytes));
}

// Elements e .. e + 3 of a row's output; zeros where the row sees nothing.
template <int D>
__device__ __forceinline__ void put_row(const TreeK &k, int b, int h, int row, int e, float4 x,
                                        float sum) {
  const int t = row / k.G, head = h * k.G + row % k.G;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(k.a.out) +
                             (((size_t)b * k.a.H + head) * k.a.T + t) * D + e) =
      make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
}

}  // namespace fs
