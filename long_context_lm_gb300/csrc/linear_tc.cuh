// linear_tc.cuh -- what the chunked linear attention kernels share: the chunks of a
// sequence and their stretches, how states lie, and what the rows' warps do to a chunk.
#pragma once

#include <cuda.h>
#include <string.h>

#include "fs_common.cuh"
#include "fs_internal.h"
#include "linear.cuh"
#include "pairs.cuh"
#include "tc05.cuh"

namespace fs {
namespace lin {

constexpr int kC = 128;               // tokens of a chunk
constexpr uint32_t kAtom = kC * 128;  // bytes of 64 elements of a chunk's rows

// A band: the chunks [c0, c1) of every sequence, in the sweep's order.
struct Params {
  LinearArgs a;
  int c0, c1;
  bool first, last;   // band
  bool fused;         // the rows' pass makes states itself: only the stretches' own are wanted
  int splits;         // stretches of a band
  // Sweeps with states of their own, where those of a sweep are, and the sweep (or -1) whose states
  // are another's transposed.
  int own[3], slot[3], borrows;
  float *local;       // [own sweep, batch H, c1 - c0 - 1, D D]: the state before each chunk but the band's
                      // first, of its stretch alone (none before a stretch's first)
  float *slots;       // [own sweep, batch H, splits, D D]: what each stretch adds; then the state before it
  float *carry;       // [own sweep, batch H, D D]: the state behind the band
  uint8_t *odd;       // [own sweep, batch H, c1 - c0, 8]: not all of the values that a warp of the states'
                      // kernel saw of the chunk are finite
  int map[3][3];      // which map holds q, k, v of a sweep
  int axes[4][2];     // 0 where a map's sequences or heads are one
  int out_axes[3][2];
  int *err;
  uint32_t polls;     // between two looks at the clock, less one
};

struct Maps {
  CUtensorMap in[4], out[3];
};

// A sequence's part of the band: chunks [lo, hi) of `chunks`, in stretches of `per`.
struct Band {
  int n, chunks, lo, hi, per, stretches;
  __device__ __forceinline__ Band(const Params &p, int b) {
    n = p.a.count ? min(max(p.a.count[b], 0), p.a.T) : p.a.T;
    chunks = (n + kC - 1) / kC;
    lo = p.c0;
    hi = max(min(p.c1, chunks), lo);
    per = max((hi - lo + p.splits - 1) / p.splits, 1);
    stretches = (hi - lo + per - 1) / per;
  }
  __device__ __forceinline__ int chunk(int i, bool reverse) const { return reverse ? chunks - 1 - i : i; }
  __device__ __forceinline__ int size(int chunk) const { return min(n - chunk * kC, kC); }
  // tokens of the chunks [a, b) in the sweep's order: the sequence's last chunk may not be whole
  __device__ __forceinline__ int tokens(int a, int b, bool reverse) const {
    const int odd = chunks * kC - n;
    return (b - a) * kC - (b > a && (reverse ? a == 0 : b == chunks) ? odd : 0);
  }
  __device__ __forceinline__ int end(int r) const { return min(lo + (r + 1) * per, hi); }
};
// The last chunk of a sequence need not go into a state that nobody wants.
__device__ __forceinline__ bool wants_last(const Params &p, const LinearSweep &w) {
  return !p.last || (w.state_out && !p.fused);
}

// How the states' warps hold a D x D matrix (and how it lies in memory between the passes): warp
// w rows 16 (w % 4).. of 64 (32 (w % 4).. of 128) and columns 64 (w / 4).., a lane of each 8 x 8 block two
// columns of one row.
template <int D>
struct Frags {
  static constexpr int kWarps = D / 16, kThreads = 32 * kWarps;
  static constexpr int kHalves = D / 64;  // groups of 16 rows that a warp holds
  static __device__ __forceinline__ int row0(int t) { return (D == 64 ? t / 32 * 16 : t / 32 % 4 * 32) + t % 32 / 4; }
  static __device__ __forceinline__ int col0(int t) { return (D == 64 ? 0 : t / 128 * 64) + t % 4 * 2; }
  // pair e of group g: the row and the first column
  static __device__ __forceinline__ int row(int t, int g, int e) { return row0(t) + 16 * g + e % 2 * 8; }
  static __device__ __forceinline__ int col(int t, int e) { return col0(t) + e / 2 * 8; }
  // floats from a matrix's start to pairs e and e + 1 (e even) of group g
  static __device__ __forceinline__ int at(int t, int g, int e) { return ((g * 8 + e / 2) * kThreads + t) * 4; }
  // and to an element
  static __device__ __forceinline__ int index(int row, int col) {
    const int warp = D == 64 ? row / 16 : row / 32 + col / 64 * 4, g = D == 64 ? 0 : row / 16 % 2;
    return at(32 * warp + row % 8 * 4 + col % 8 / 2, g, col % 64 / 8 * 2) + row / 8 % 2 * 2 + col % 2;
  }
};

// tc::desc_sw128 for elements in several blocks of 64, `apart` bytes from one to the next.
__device__ __forceinline__ uint64_t desc_blocks(uint32_t at, uint32_t apart) {
  return (tc::desc_sw128(at) & ~(0x3fffull << 16)) | (uint64_t)(apart >> 4) << 16;
}

// 16 lanes x 64 columns, a warp's lane t holding of each eight columns 2 (t % 4) and the
// next, in lanes t / 4 and t / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t at, f2 (&r)[16]) {
  uint32_t u[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
        "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
        "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(at));
  tc::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = (f2)u[2 * i] | (f2)u[2 * i + 1] << 32;
}

// The 64 x 128 box of a map at token t of head h of sequence b.
__device__ __forceinline__ void load_rows(void *dst, const void *map, uint64_t *bar, int x, int t,
                                          int h, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%3, %4, %5, %6}], [%2];\n" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(t), "r"(h), "r"(b)
      : "memory");
}

// The other way, of `map`'s box size; for bulk_commit and bulk_wait_read of the same thread.
__device__ __forceinline__ void store_rows(const void *src, const void *map, int x, int t, int h, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];\n" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(x), "r"(t), "r"(h), "r"(b)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;\n" ::"n"(N) : "memory");
}

// Eight bf16 numbers, not all of them finite.
__device__ __forceinline__ bool not_finite(const uint4 &u) {
  auto biggest = [](uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
    return r;
  };
  const uint32_t m = biggest(biggest(u.x, u.y), biggest(u.z, u.w)) & 0x7fff7fffu;
  return (m & 0xffffu) >= 0x7f80u || (m >> 16) >= 0x7f80u;
}

__device__ __forceinline__ void stmatrix4(uint32_t at, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

// tc::mbar_wait with the call's own limit.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, const Params &p) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((i & p.polls) == 0) {
      if (clock64() - t0 > p.a.wait_cycles) break;
      if (*reinterpret_cast<volatile int *>(p.err) != 0) return false;
    }
  }
  tc::report_error(p.err, FS_ERR_TIMEOUT);
  return false;
}
#define WAIT(bar, k) __all_sync(0xffffffffu, wait_for(&(bar), (k) & 1, p))

// What the rows' warps need of a head: lam^n times the scale; columns' factors (see there).
struct Tables {
  float scaled[kC + 4];
  alignas(16) float cols[3][32];
};


__device__ __forceinline__ void fill_tables(Tables &tab, float decay, bool reverse, float scale, int t, int threads) {
  for (int k = t; k <= kC + 96; k += threads) {
    const int c = k - kC - 1;
    const int n = k <= kC ? k : 32 * (c / 32 + 1) + (reverse ? c % 32 - 31 : -(c % 32));
    const Factor x = decay_power(decay, n);
    if (k <= kC)
      tab.scaled[k] = (x.hi + x.lo) * scale;
    else
      tab.cols[c / 32][c % 32] = x.hi + x.lo;
  }
}

// Two parts of a state into shared memory as the factor of a product: [row][column], columns
// swizzled.  A lane names the row that it is to fill of one of four 8 x 8 blocks: rows + 0 and
// + 8 of two neighbours among the blocks of columns.
template <int D>
struct Publisher {
  uint32_t to;
  int lane;
  __device__ __forceinline__ Publisher(uint32_t place, int t)
      : to(place + Frags<D>::col0(t) / 64 * (D * 128) +
           (Frags<D>::row0(t) - t % 32 / 4 + t % 32 / 8 % 2 * 8 + t % 8) * 128),
        lane(t % 32) {}
  // pairs e .. e + 3 of group g, e a multiple of 4
  __device__ __forceinline__ void put(int g, int e, const f2 (&x)[4]) const {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f2 y = x[k];
      hi[k] = split2(y);
      lo[k] = pack2(y);
    }
    const uint32_t at = to + g * 16 * 128 + (((e / 2 + lane / 16) ^ (lane % 8)) << 4);
    stmatrix4(at, hi);
    stmatrix4(at + D / 64 * D * 128, lo);
  }
};

// Values that are not finite: per column the first such token of the block's chunk i, `at` tokens from
// the chunk's start in the sweep's order.  Marks of later chunks are greater, those of earlier tokens
// of one chunk too, so that nothing needs clearing: a row `at` is behind one if mark >= bad_mark(i, at).
__device__ __forceinline__ int bad_mark(int i, int at) { return (i + 1) << 8 | (255 - at); }

// A warp of the rows' eight: 32 rows, half of the columns.
template <int D>
struct RowWarp {
  int quarter, half, lane, row;
  uint32_t scores, out;  // its TMEM columns
  __device__ __forceinline__ RowWarp(int warp, int lane_, uint32_t scores_, uint32_t out_)
      : quarter(warp % 4), half(warp / 4), lane(lane_), row(quarter * 32 + lane_) {
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    scores = scores_ + lanes + 16 * half;
    out = out_ + lanes + half * (D / 2);
  }

  // Scores times scale lam^|i - j| as a bf16 high and low part, in place (sixteen keys: eight columns of
  // high parts, eight of low ones).  For 32 keys that all rows of the warp see, lam^|i - j| is a
  // factor of the row and one of the column, counted from the warp's near edge, so that neither passes 1.
  __device__ __forceinline__ void parts(const Tables &tab, bool reverse, int n) const {
    const float rowf = tab.scaled[reverse ? 31 - lane : lane];
    const f2 rowff = f2_bits(rowf, rowf);
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t part[2][8];
      const int off = reverse ? c - quarter : quarter - c;
      if (off < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) part[0][e] = part[1][e] = 0;
      } else {
        uint32_t x[16];
        tc::tmem_ld16(scores + 32 * c, x);
        tc::tmem_wait_ld();
        if (off > 0 && (!reverse || 32 * c + 32 <= n)) {
          const ulonglong2 *cw = reinterpret_cast<const ulonglong2 *>(tab.cols[off - 1] + 16 * half);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const ulonglong2 f = cw[e];
            f2 y = mul2(mul2((f2)x[4 * e] | (f2)x[4 * e + 1] << 32, f.x), rowff);
            f2 z = mul2(mul2((f2)x[4 * e + 2] | (f2)x[4 * e + 3] << 32, f.y), rowff);
            part[0][2 * e] = split2(y);
            part[1][2 * e] = pack2(y);
            part[0][2 * e + 1] = split2(z);
            part[1][2 * e + 1] = pack2(z);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float v[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int j = 32 * c + 16 * half + 2 * e + k, lag = reverse ? j - row : row - j;
              const bool seen = lag >= 0 && (!reverse || j < n);
              v[k] = seen ? __uint_as_float(x[2 * e + k]) * tab.scaled[abs(lag)] : 0.f;
            }
            f2 y = f2_bits(v[0], v[1]);
            part[0][e] = split2(y);
            part[1][e] = pack2(y);
          }
        }
      }
      tc::tmem_st8(scores + 32 * c, part[0]);
      tc::tmem_st8(scores + 32 * c + 8, part[1]);
    }
  }

  // Q S times scale lam^(i + 1) (in reverse lam^i, from the last token), in place.
  __device__ __forceinline__ void weigh(const Tables &tab, bool reverse, int n) const {
    const float f = tab.scaled[reverse ? max(n - 1 - row, 0) : row + 1];
    const f2 ff = f2_bits(f, f);
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t x[16];
      tc::tmem_ld16(out + 16 * c, x);
      tc::tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const f2 y = mul2((f2)x[e] | (f2)x[e + 1] << 32, ff);
        x[e] = (uint32_t)y;
        x[e + 1] = (uint32_t)(y >> 32);
      }
      tc::tmem_st16(out + 16 * c, x);
    }
    tc::tmem_wait_st();
  }

  // The finished rows.  Whole warps of bf16 rows leave by TMA by way of the values' place, 64 columns at
  // a time; the last rows of a sequence, and fp32 parts, from their threads.  `i`: which chunk of
  // the block's.  `bad` (or null): columns that are not finite, as bad_mark.  Arrives on o_free
  // when the accumulator is read.  True: the values' place is read until bulk_wait_read (lane 0).
  __device__ __forceinline__ bool store(const LinearSweep &w, const CUtensorMap *map, const int (&axes)[2], int b,
                                        int h, int chunk, int n, int i, bool reverse, const int *bad,
                                        unsigned char *values, uint64_t *o_free, uint64_t *pairs, const Params &p) const {
    const bool whole = 32 * quarter + 32 <= n && !w.out_f32;
    unsigned char *box = values + (D == 64 ? 0 : half * kAtom) + quarter * 4096;
    const long long to = b * w.os[0] + h * w.os[1] + (chunk * (long long)kC + row) * w.os[2] + half * (D / 2);
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t x[16];
      tc::tmem_ld16(out + 16 * c, x);
      tc::tmem_wait_ld();
      if (c == D / 32 - 1) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(o_free);
      }
      if (bad) {
#pragma unroll 1
        for (int e = 0; e < 16; ++e) {
          const bool gone = bad[half * (D / 2) + 16 * c + e] >= bad_mark(i, reverse ? kC - 1 - row : row);
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (k == e && gone) x[k] = 0x7fc00000u;
        }
      }
      if (w.out_f32) {
        if (row < n)
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             static_cast<float *>(w.out) + to + 16 * c + e),
                         "r"(x[e]), "r"(x[e + 1]), "r"(x[e + 2]), "r"(x[e + 3]), "r"(x[e + 4]), "r"(x[e + 5]),
                         "r"(x[e + 6]), "r"(x[e + 7])
                         : "memory");
        continue;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          y[k] = pack_bf16(__uint_as_float(x[8 * e + 2 * k]), __uint_as_float(x[8 * e + 2 * k + 1]));
        const uint4 z = make_uint4(y[0], y[1], y[2], y[3]);
        if (whole)
          *reinterpret_cast<uint4 *>(box + swz128(lane, (D == 64 ? 4 * half : 0) + 2 * c + e)) = z;
        else if (row < n)
          *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(w.out) + to + 16 * c + 8 * e) = z;
      }
    }
    if (whole) tc::fence_async_smem();
    __syncwarp();
    if (D == 64 && half != 0 && lane == 0) tc::mbar_arrive(&pairs[quarter]);  // two warps' halves of one box
    if (!whole || lane != 0 || (D == 64 && half != 0)) return false;
    if (D == 64 && !wait_for(&pairs[quarter], i & 1, p)) return false;
    store_rows(box, map, D == 64 ? 0 : 64 * half, chunk * kC + 32 * quarter, h * axes[1], b * axes[0]);
    bulk_commit();
    return true;
  }
};

// One pass over all chunks with the states in registers (k17_linear_fused.cu); with stretches,
// their states are in p.slots.
cudaError_t launch_fused(const Params &p, const Maps &maps, cudaStream_t st);

}  // namespace lin
}  // namespace fs
