// k16_linear_tc.cu -- linear attention with a decay for each head over prompts,
// in chunks of 128 tokens on the tensor cores.
//
// Within a chunk whose state before it is S (rows: elements of k, columns: of v)
//   out_i = scale (lam^(i+1) q_i S + sum over j <= i of lam^(i-j) (q_i . k_j) v_j)
//   S    <- lam^n S + sum over j of lam^(n-1-j) k_j v_j^T
// which are four products: Q K^T, Q S, (scores x powers) V and K^T (weighted V).
// In reverse (for gradients of k and v) a row sees the tokens behind it, S
// enters without a decay (lam^i in the place of lam^(i+1), counted from the last
// token) and a token's weight in it is one power higher.
//
// Precision.  q, k and v are bf16 and go in as they are.  The scores times their
// powers, and S as a factor, go in as a bf16 high and low part (2^-16 of
// themselves); the weighted values, of which states are made, in three parts
// (24 bits).  All sums are fp32; S itself is fp32, in registers.
//
// A block takes one (sequence, head), or one of `splits` stretches of it, chunk
// after chunk; S never leaves it.  Warps:
//   0-3       rows: Q S times the row's power in TMEM; scores to bf16 parts in their own
//             TMEM columns; the finished rows to memory
//   4..       states (D / 16 warps): weighted values into a ring of 32-token slabs, S in
//             registers, its bf16 parts into shared memory for the next chunk
//   then one  TMA loads, and one that issues the products.
// A chunk's q, k and v lie in shared memory once; each is loaded anew as soon as its
// last product has read it.  Heads of 64 leave room for two blocks an SM, which
// fill each other's waits; heads of 128 for one.
//
// With fewer (sequence, head) pairs than blocks fit, each is cut into stretches: a
// first pass of the same kernel without rows makes the states of the stretches
// alone (k and v are read twice then), a small kernel runs through them, and
// the main pass starts each stretch from its own.
#include <cuda.h>
#include <string.h>

#include "fs_common.cuh"
#include "fs_internal.h"
#include "linear.cuh"
#include "tc05.cuh"

namespace fs {
namespace {

constexpr int kC = 128;       // tokens of a chunk
constexpr int kSlab = 32;     // tokens of a slab of weighted values
constexpr int kSlabs = kC / kSlab;
constexpr int kRing = 2;      // slabs in the ring
constexpr uint32_t kAtom = kC * 128;  // 64 elements of a chunk's rows

struct Params {
  LinearArgs a;
  int splits;
  float *states;     // [sweep, batch H, splits, D D]: the state before each stretch
  int map[3][3];     // which map holds q, k, v of a sweep
  int axes[4][2];    // 0 where a map's sequences or heads are one
  int *err;
};

template <int D>
struct Cfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kStateWarps = D / 16;
  static constexpr int kTma = 4 + kStateWarps, kMma = kTma + 1;
  static constexpr int kThreads = 32 * (kMma + 1);
  static constexpr int kHalves = D / 64;  // groups of 16 rows that a state warp holds
  static constexpr uint32_t kTile = kAtoms * kAtom;              // q, k or v
  static constexpr uint32_t kPart = kAtoms * kSlab * 128;        // one part of a slab
  static constexpr uint32_t kSPart = kAtoms * D * 128;           // one part of S
  static constexpr uint32_t kQ = 0, kK = kTile, kV = 2 * kTile, kS = 3 * kTile,
                            kSlab0 = kS + 2 * kSPart, kBytes = kSlab0 + kRing * 3 * kPart;
  // TMEM columns: scores (then their parts), outputs, the chunk's addition to S
  static constexpr uint32_t kScores = 0, kOut = kC, kU = kC + D, kCols = D == 64 ? 256 : 512;
};

struct Shared {
  uint64_t qfull, kfull, vfull, qempty, kempty, vempty;
  uint64_t slab_full[kRing], slab_empty[kRing];
  uint64_t s_ready, s_free, scores, inter, parts, done, o_free, u_full, u_free, checked, fin;
  uint32_t tmem;
  int odd[2];                 // a chunk's values are not all finite
  float power[kC + 1];        // lam^n
  int bad[2][128];            // per column: the first such token in the sweep's order
};

// A stretch of a sweep: chunks [from, to) in the sweep's order of the `chunks` of a sequence of n tokens.
struct Stretch {
  int n, chunks, per, last, from, to;  // last: the last stretch with a token (0 if there is none)
  __device__ __forceinline__ Stretch(const Params &p, int b, int r) {
    n = p.a.count ? min(max(p.a.count[b], 0), p.a.T) : p.a.T;
    chunks = (n + kC - 1) / kC;
    per = max((chunks + p.splits - 1) / p.splits, 1);
    last = max((chunks + per - 1) / per - 1, 0);
    from = min(r * per, chunks);
    to = min(from + per, chunks);
  }
  __device__ __forceinline__ int chunk(int i, bool reverse) const { return reverse ? chunks - 1 - i : i; }
  __device__ __forceinline__ int size(int chunk) const { return min(n - chunk * kC, kC); }
  // tokens of the chunks [a, b) in the sweep's order
  __device__ __forceinline__ int tokens(int a, int b, bool reverse) const {
    const int whole = (b - a) * kC, odd = chunks * kC - n;  // the sequence's last chunk lacks `odd`
    return whole - ((reverse ? a == 0 : b == chunks) && b > a ? odd : 0);
  }
};

// tc::desc_sw128 for elements in several blocks of 64, `apart` bytes from one to the next.
__device__ __forceinline__ uint64_t desc_blocks(uint32_t at, uint32_t apart) {
  return (tc::desc_sw128(at) & ~(0x3fffull << 16)) | (uint64_t)(apart >> 4) << 16;
}

// 16 lanes x 64 columns, a warp's lane t holding of each eight columns 2 (t % 4) and the
// next, in lanes t / 4 and t / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t at, float (&r)[32]) {
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
  for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(u[i]);
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

// Two fp32 numbers as pairs of bf16: the nearest, and what is left.
__device__ __forceinline__ uint32_t split(float &x, float &y) {
  const uint32_t h = pack_bf16(x, y);
  x -= bf16_lo(h);
  y -= bf16_hi(h);
  return h;
}

__device__ __forceinline__ bool not_finite(const uint4 &u) {
  auto biggest = [](uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a & 0x7fff7fffu), "r"(b & 0x7fff7fffu));
    return r;
  };
  const uint32_t m = biggest(biggest(u.x, u.y), biggest(u.z, u.w)) & 0x7fff7fffu;
  return (m & 0xffffu) >= 0x7f80u || (m >> 16) >= 0x7f80u;
}

#define WAIT(bar, k) __all_sync(0xffffffffu, tc::mbar_wait(&(bar), (k) & 1, p.err))

// kRows: the whole sweep; without, only the states of the stretches (into p.states).
template <int D, bool kRows>
__global__ void __launch_bounds__(Cfg<D>::kThreads, D == 64 ? 2 : 1)
    k16_linear_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
                      const __grid_constant__ CUtensorMap map2, const __grid_constant__ CUtensorMap map3,
                      const __grid_constant__ Params p) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Shared s;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const LinearSweep &w = p.a.sweep[blockIdx.z];
  const int b = blockIdx.y / p.a.H, h = blockIdx.y % p.a.H, r = blockIdx.x;
  const Stretch st(p, b, r);
  const bool reverse = w.reverse;
  // nothing for this block: no such stretch, or the last one, whose state nobody starts from
  // (with one stretch the main pass reads the given state itself)
  if (kRows ? r > st.last : r >= st.last) return;
  const float decay = p.a.decay[h];

  if (threadIdx.x == 0) {
    for (uint64_t *x : {&s.qfull, &s.kfull, &s.vfull, &s.qempty, &s.kempty, &s.vempty, &s.s_free,
                        &s.scores, &s.inter, &s.done, &s.u_full, &s.fin})
      tc::mbar_init(x, 1);
    for (int i = 0; i < kRing; ++i) {
      tc::mbar_init(&s.slab_full[i], C::kStateWarps);
      tc::mbar_init(&s.slab_empty[i], 1);
    }
    for (uint64_t *x : {&s.s_ready, &s.u_free, &s.checked}) tc::mbar_init(x, C::kStateWarps);
    for (uint64_t *x : {&s.parts, &s.o_free}) tc::mbar_init(x, 4);
    tc::mbar_fence_init();
    s.odd[0] = s.odd[1] = 0;
  }
  for (int i = threadIdx.x; i <= kC; i += C::kThreads) {
    const Factor f = decay_power(decay, i);
    s.power[i] = f.hi + f.lo;
  }
  for (int i = threadIdx.x; i < 256; i += C::kThreads) s.bad[i / 128][i % 128] = kC;
  if (warp == C::kMma) {
    tc::tmem_alloc(&s.tmem, kRows ? C::kCols : D);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s.tmem, base = smem_u32(smem);
  const uint32_t tu = tmem + (kRows ? C::kU : 0);
  const int chunks = st.to - st.from;

  if (warp == C::kTma && lane == 0) {
    // ------------------------------------------------------------------ loads
    const CUtensorMap *maps[4] = {&map0, &map1, &map2, &map3};
    const int mq = p.map[blockIdx.z][0], mk = p.map[blockIdx.z][1], mv = p.map[blockIdx.z][2];
    auto load = [&](uint32_t at, int m, const LinearRows &x, uint64_t *bar, int t) {
      tc::mbar_arrive_expect_tx(bar, C::kTile);
      for (int i = 0; i < C::kAtoms; ++i)
        load_rows(smem + at + i * kAtom, maps[m], bar, 64 * i, t, h / x.share * p.axes[m][1],
                  b * p.axes[m][0]);
    };
    int i = 0;
    int loaded[3] = {0, 0, 0};
    for (; i < chunks; ++i) {
      const int t = st.chunk(st.from + i, reverse) * kC;
      if (kRows) {
        if (i && !tc::mbar_wait(&s.qempty, (i - 1) & 1, p.err)) break;
        load(C::kQ, mq, w.q, &s.qfull, t);
        ++loaded[0];
      }
      if (i && !tc::mbar_wait(&s.kempty, (i - 1) & 1, p.err)) break;
      load(C::kK, mk, w.k, &s.kfull, t);
      ++loaded[1];
      if (i && !tc::mbar_wait(&s.vempty, (i - 1) & 1, p.err)) break;
      load(C::kV, mv, w.v, &s.vfull, t);
      ++loaded[2];
    }
    // what is under way lands before the block ends
    uint64_t *full[3] = {&s.qfull, &s.kfull, &s.vfull};
    for (int j = 0; j < 3; ++j)
      if (loaded[j]) tc::mbar_wait(full[j], (loaded[j] - 1) & 1, nullptr);
  } else if (warp == C::kMma && lane == 0) {
    // --------------------------------------------------------------- products
    constexpr uint32_t kQK = tc::idesc_bf16(128, 128, 0), kB = tc::idesc_bf16(128, D, 1);
    constexpr uint32_t kUD = tc::idesc_bf16(D, D, 1) | 1u << 15;  // K^T: its rows run along M
    for (int i = 0; i < chunks; ++i) {
      if (kRows) {
        if (!tc::mbar_wait(&s.qfull, i & 1, p.err) || !tc::mbar_wait(&s.kfull, i & 1, p.err)) break;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_ss(tmem + C::kScores, tc::desc_sw128(base + C::kQ + k / 4 * kAtom + k % 4 * 32),
                     tc::desc_sw128(base + C::kK + k / 4 * kAtom + k % 4 * 32), kQK, k > 0);
        tc::mma_commit(&s.scores);
        if (!tc::mbar_wait(&s.s_ready, i & 1, p.err) ||
            (i && !tc::mbar_wait(&s.o_free, (i - 1) & 1, p.err)))
          break;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < 2 * D / 16; ++k) {
          const int kk = k % (D / 16), part = k / (D / 16);
          tc::mma_ss(tmem + C::kOut, tc::desc_sw128(base + C::kQ + kk / 4 * kAtom + kk % 4 * 32),
                     desc_blocks(base + C::kS + part * C::kSPart + kk * 2048, D * 128), kB, k > 0);
        }
        tc::mma_commit(&s.inter);
        tc::mma_commit(&s.s_free);
        tc::mma_commit(&s.qempty);
      } else if (!tc::mbar_wait(&s.kfull, i & 1, p.err)) {
        break;
      }
      if (i && !tc::mbar_wait(&s.u_free, (i - 1) & 1, p.err)) break;
      bool ok = true;
      for (int j = 0; j < kSlabs && ok; ++j) {
        const int at = i * kSlabs + j, slot = at % kRing;
        if (!(ok = tc::mbar_wait(&s.slab_full[slot], at / kRing & 1, p.err))) break;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < 3 * kSlab / 16; ++k) {
          const int kk = k % (kSlab / 16), part = k / (kSlab / 16);
          tc::mma_ss(tu, desc_blocks(base + C::kK + (j * kSlab + kk * 16) * 128, kAtom),
                     desc_blocks(base + C::kSlab0 + (slot * 3 + part) * C::kPart + kk * 2048, kSlab * 128),
                     kUD, j > 0 || k > 0);
        }
        tc::mma_commit(&s.slab_empty[slot]);
      }
      if (!ok) break;
      tc::mma_commit(&s.u_full);
      tc::mma_commit(&s.kempty);
      if (kRows) {
        if (!tc::mbar_wait(&s.parts, i & 1, p.err)) break;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < 2 * kC / 16; ++k) {
          const int kk = k % (kC / 16), part = k / (kC / 16);
          tc::mma_ts(tmem + C::kOut, tmem + C::kScores + kk / 2 * 32 + part * 16 + kk % 2 * 8,
                     desc_blocks(base + C::kV + kk * 2048, kAtom), kB, 1);
        }
        tc::mma_commit(&s.done);
      }
      tc::mma_commit(&s.vempty);
    }
    tc::mma_commit(&s.fin);
    tc::mbar_wait(&s.fin, 0, nullptr);
  } else if (warp >= 4 && warp < C::kTma) {
    // ------------------------------------------------------------------ states
    const int sw = warp - 4, t = threadIdx.x - 128, kT = 32 * C::kStateWarps;
    // this lane's places in S: rows row0 + 16 g (+ 8), columns col0 + 8 e (+ 1)
    const int row0 = (D == 64 ? sw * 16 : sw % 4 * 32) + lane / 4;
    const int col0 = (D == 64 ? 0 : sw / 4 * 64) + lane % 4 * 2;
    const uint32_t lanes = tu + ((uint32_t)(warp % 4 * 32) << 16) + (D == 64 ? 0 : sw / 4 * 64);
    const size_t bh = (size_t)blockIdx.z * gridDim.y + blockIdx.y;
    float S[C::kHalves][32];
    auto each = [&](auto f) {  // f(element, row, column)
#pragma unroll
      for (int g = 0; g < C::kHalves; ++g)
#pragma unroll
        for (int e = 0; e < 32; ++e)
          f(S[g][e], row0 + 16 * g + (e & 2) * 4, col0 + e / 4 * 8 + (e & 1));
    };
    // between the passes states lie as the lanes hold them
    auto slot = [&](int i) { return p.states + (bh * p.splits + i) * (D * D) + t * 4; };
    const float *given = w.state ? w.state + (size_t)blockIdx.y * D * D : nullptr;
    if (kRows && st.last > 0) {
      const float *from = slot(r);
#pragma unroll
      for (int g = 0; g < C::kHalves; ++g)
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 x = *reinterpret_cast<const float4 *>(from + (g * 8 + e / 4) * kT * 4);
          S[g][e] = x.x, S[g][e + 1] = x.y, S[g][e + 2] = x.z, S[g][e + 3] = x.w;
        }
    } else if (given && r == 0) {
      const int sr = w.transposed ? 1 : D, sc = w.transposed ? D : 1;
      each([&](float &x, int row, int col) { x = given[row * sr + col * sc] * w.state_mul; });
    } else {
      each([&](float &x, int, int) { x = 0.f; });
    }
    auto save = [&](float *to) {
#pragma unroll
      for (int g = 0; g < C::kHalves; ++g)
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4 *>(to + (g * 8 + e / 4) * kT * 4) =
              make_float4(S[g][e], S[g][e + 1], S[g][e + 2], S[g][e + 3]);
    };
    // S as the factor of the next product: two parts, [row][column] with the columns swizzled
    auto publish = [&]() {
#pragma unroll
      for (int g = 0; g < C::kHalves; ++g)
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const int row = row0 + 16 * g + (e & 2) * 4, col = col0 + e / 4 * 8;
          const uint32_t at = C::kS + col / 64 * (D * 128) + swz128(row, col % 64 / 8) + col % 8 * 2;
          float x = S[g][e], y = S[g][e + 1];
          *reinterpret_cast<uint32_t *>(smem + at) = split(x, y);
          *reinterpret_cast<uint32_t *>(smem + at + C::kSPart) = pack_bf16(x, y);
        }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&s.s_ready);
    };
    if (!kRows && r == 0) save(slot(0));
    if (kRows && chunks) publish();
    {
      const Factor whole = decay_power(decay, kC);
      int i = 0;
      bool ok = true;
      for (; i < chunks && ok; ++i) {
        const int n = st.size(st.chunk(st.from + i, reverse));
        if (!(ok = WAIT(s.vfull, i))) break;
        if (n < kC && !(ok = WAIT(s.kfull, i))) break;
        if (n < kC) {
          // what lies behind the sequence takes no part, whatever it is
          for (int u = t; u < (kC - n) * (D / 8); u += kT) {
            const int row = n + u / (D / 8), ch = u % (D / 8);
            const uint32_t at = ch / 8 * kAtom + swz128(row, ch % 8);
            *reinterpret_cast<uint4 *>(smem + C::kK + at) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(smem + C::kV + at) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kStateWarps) : "memory");
        }
        for (int j = 0; j < kSlabs; ++j) {
          const int at = i * kSlabs + j, place = at % kRing;
          if (at >= kRing && !(ok = WAIT(s.slab_empty[place], at / kRing - 1))) break;
          unsigned char *to = smem + C::kSlab0 + place * 3 * C::kPart;
#pragma unroll
          for (int u = t; u < kSlab * (D / 8); u += 32 * C::kStateWarps) {
            const int row = j * kSlab + u / (D / 8), ch = u % (D / 8);
            uint4 *from = reinterpret_cast<uint4 *>(smem + C::kV + ch / 8 * kAtom + swz128(row, ch % 8));
            const uint4 x = *from;
            const float f = row < n ? s.power[reverse ? row + 1 : n - 1 - row] : 0.f;
            const uint32_t in[4] = {x.x, x.y, x.z, x.w};
            uint32_t part[3][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float y = bf16_lo(in[c]) * f, z = bf16_hi(in[c]) * f;
              part[0][c] = split(y, z);
              part[1][c] = split(y, z);
              part[2][c] = pack_bf16(y, z);
            }
            const uint32_t off = ch / 8 * (kSlab * 128) + swz128(row % kSlab, ch % 8);
#pragma unroll
            for (int k = 0; k < 3; ++k)
              *reinterpret_cast<uint4 *>(to + k * C::kPart + off) =
                  make_uint4(part[k][0], part[k][1], part[k][2], part[k][3]);
            if (kRows && not_finite(x)) {
              // out of the tile, whose rows before it (scores 0) would become NaN too
              uint32_t keep[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                keep[c] = in[c];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  if ((in[c] >> 16 * k & 0x7f80u) == 0x7f80u) {
                    keep[c] &= k ? 0xffffu : 0xffff0000u;
                    atomicMin(&s.bad[i & 1][ch * 8 + 2 * c + k], reverse ? kC - 1 - row : row);
                  }
              }
              *from = make_uint4(keep[0], keep[1], keep[2], keep[3]);
              s.odd[i & 1] = 1;
            }
          }
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s.slab_full[place]);
        }
        if (!ok) break;
        if (kRows && lane == 0) tc::mbar_arrive(&s.checked);
        if (!(ok = WAIT(s.u_full, i))) break;
        tc::fence_after_sync();
        const Factor f = n == kC ? whole : decay_power(decay, n);
#pragma unroll
        for (int g = 0; g < C::kHalves; ++g) {
          float u[32];
          tmem_ld_16x64(lanes + ((uint32_t)(16 * g) << 16), u);
          if (g == C::kHalves - 1) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&s.u_free);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) S[g][e] = f.times(S[g][e], u[e]);
        }
        if (kRows && i + 1 < chunks) {
          if (!(ok = WAIT(s.s_free, i))) break;
          publish();
        }
      }
    }
    if (!kRows) {
      save(slot(r + 1));
    } else if (r == st.last && w.state_out) {
      float *to = w.state_out + (size_t)blockIdx.y * D * D;
      const int sr = w.transposed ? 1 : D, sc = w.transposed ? D : 1;
      const float mul = 1.f / w.state_mul;
      each([&](float &x, int row, int col) { to[row * sr + col * sc] = x * mul; });
    }
  } else if (kRows && warp < 4) {
    // -------------------------------------------------------------------- rows
    const int row = warp * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    const long long out0 = b * w.os[0] + h * w.os[1];
    for (int i = 0; i < chunks; ++i) {
      const int chunk = st.chunk(st.from + i, reverse), n = st.size(chunk);
      if (!WAIT(s.inter, i)) break;
      tc::fence_after_sync();
      {
        const float f = s.power[reverse ? max(n - 1 - row, 0) : row + 1];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[32];
          tc::tmem_ld32(lanes + C::kOut + 32 * c, x);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
          tc::tmem_st32(lanes + C::kOut + 32 * c, x);
        }
      }
      if (!WAIT(s.scores, i)) break;
      tc::fence_after_sync();
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t hi[16], lo[16];
        if (reverse ? c < warp : c > warp) {
#pragma unroll
          for (int e = 0; e < 16; ++e) hi[e] = lo[e] = 0;
        } else {
          uint32_t x[32];
          tc::tmem_ld32(lanes + C::kScores + 32 * c, x);
          tc::tmem_wait_ld();
          if (c != warp && (!reverse || 32 * c + 32 <= n)) {
            const float *pw = s.power + (reverse ? 32 * c - row : row - 32 * c);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float y = __uint_as_float(x[2 * e]) * (reverse ? pw[2 * e] : pw[-2 * e]);
              float z = __uint_as_float(x[2 * e + 1]) * (reverse ? pw[2 * e + 1] : pw[-2 * e - 1]);
              hi[e] = split(y, z);
              lo[e] = pack_bf16(y, z);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float v[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int j = 32 * c + 2 * e + k, lag = reverse ? j - row : row - j;
                const bool seen = lag >= 0 && (!reverse || j < n);
                v[k] = seen ? __uint_as_float(x[2 * e + k]) * s.power[abs(lag)] : 0.f;
              }
              hi[e] = split(v[0], v[1]);
              lo[e] = pack_bf16(v[0], v[1]);
            }
          }
        }
        tc::tmem_st16(lanes + C::kScores + 32 * c, hi);
        tc::tmem_st16(lanes + C::kScores + 32 * c + 16, lo);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&s.parts);
      if (!WAIT(s.checked, i) || !WAIT(s.done, i)) break;
      tc::fence_after_sync();
      const bool odd = s.odd[i & 1] != 0;
      const long long at = out0 + (chunk * (long long)kC + row) * w.os[2];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        tc::tmem_ld32(lanes + C::kOut + 32 * c, x);
        tc::tmem_wait_ld();
        if (c == D / 32 - 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s.o_free);
        }
        float y[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(x[e]) * p.a.scale;
        if (odd) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (s.bad[i & 1][32 * c + e] <= (reverse ? kC - 1 - row : row)) y[e] = __uint_as_float(0x7fc00000u);
        }
        if (row < n) {
          if (w.out_f32) {
            float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(w.out) + at + 32 * c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              to[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          } else {
            uint4 *to = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(w.out) + at + 32 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              to[e] = make_uint4(pack_bf16(y[8 * e], y[8 * e + 1]), pack_bf16(y[8 * e + 2], y[8 * e + 3]),
                                 pack_bf16(y[8 * e + 4], y[8 * e + 5]), pack_bf16(y[8 * e + 6], y[8 * e + 7]));
          }
        }
      }
      if (odd) {  // clean for the chunk after the next
        asm volatile("bar.sync 2, 128;" ::: "memory");
        if (row < D) s.bad[i & 1][row] = kC;
        if (row == 0) s.odd[i & 1] = 0;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::kMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kRows ? C::kCols : D);
  }
}

// Runs through the stretches' states in the sweep's order: slot r, the state that stretch r - 1
// alone adds (the first: with the given one), becomes the state before stretch r.
template <int D>
__global__ void __launch_bounds__(256) k16_join_kernel(const __grid_constant__ Params p) {
  const int b = blockIdx.y / p.a.H, h = blockIdx.y % p.a.H;
  const Stretch st(p, b, 0);
  const bool reverse = p.a.sweep[blockIdx.z].reverse;
  float4 *at = reinterpret_cast<float4 *>(
                   p.states + ((size_t)blockIdx.z * gridDim.y + blockIdx.y) * p.splits * (D * D)) +
               blockIdx.x * 256 + threadIdx.x;
  if (st.last < 2) return;
  constexpr int kAhead = 8;
  float4 x = at[D * D / 4];
  for (int r0 = 2; r0 <= st.last; r0 += kAhead) {
    float4 y[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (r0 + k <= st.last) y[k] = at[(size_t)(r0 + k) * (D * D / 4)];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int r = r0 + k;
      if (r > st.last) break;
      const Factor f = decay_power(p.a.decay[h], st.tokens((r - 1) * st.per, min(r * st.per, st.chunks), reverse));
      x = make_float4(f.times(x.x, y[k].x), f.times(x.y, y[k].y), f.times(x.z, y[k].z), f.times(x.w, y[k].w));
      at[(size_t)r * (D * D / 4)] = x;
    }
  }
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
  static EncodeTiled fn = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiled>(ptr);
    return static_cast<EncodeTiled>(nullptr);
  }();
  return fn;
}

// [batch, heads, T, D] bf16 rows in boxes of 128 tokens x 64 elements; an axis that all share
// (stride 0) is one long.
bool make_map(CUtensorMap *map, const LinearRows &x, const LinearArgs &a, int *axes) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  axes[0] = x.s[0] != 0;
  axes[1] = x.s[1] != 0;
  const cuuint64_t dims[4] = {(cuuint64_t)a.d, (cuuint64_t)a.T, (cuuint64_t)(axes[1] ? a.H / x.share : 1),
                              (cuuint64_t)(axes[0] ? a.batch : 1)};
  const cuuint64_t row = (cuuint64_t)a.d * 2;
  const cuuint64_t strides[3] = {(cuuint64_t)x.s[2] * 2, axes[1] ? (cuuint64_t)x.s[1] * 2 : row,
                                 axes[0] ? (cuuint64_t)x.s[0] * 2 : row};
  const cuuint32_t box[4] = {64, kC, 1, 1}, estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(x.x), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Stretches of a sweep: as many as blocks fit at once, two chunks each at least.
int splits_of(int sweeps, int pairs, int T, int d) {
  const int blocks = 152 * (d == 64 ? 2 : 1), most = ((T + kC - 1) / kC + 1) / 2;
  const int n = blocks / (sweeps * pairs < blocks ? sweeps * pairs : blocks);
  return n < most ? n : most < 1 ? 1 : most;
}

template <int D>
cudaError_t run(const Params &p, const CUtensorMap (&m)[4], cudaStream_t st) {
  constexpr int kSmem = Cfg<D>::kBytes + 1024;
  const int pairs = p.a.batch * p.a.H;
  if (p.splits > 1) {
    auto f = k16_linear_kernel<D, false>;
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    f<<<dim3(p.splits - 1, pairs, p.a.sweeps), Cfg<D>::kThreads, kSmem, st>>>(m[0], m[1], m[2], m[3], p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    k16_join_kernel<D><<<dim3(D * D / 1024, pairs, p.a.sweeps), 256, 0, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  auto f = k16_linear_kernel<D, true>;
  const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  f<<<dim3(p.splits, pairs, p.a.sweeps), Cfg<D>::kThreads, kSmem, st>>>(m[0], m[1], m[2], m[3], p);
  return cudaGetLastError();
}

}  // namespace

size_t linear_chunk_bytes(int sweeps, int batch, int H, int T, int d) {
  const int n = splits_of(sweeps, batch * H, T, d);
  return n > 1 ? (size_t)sweeps * batch * H * n * d * d * 4 : 0;
}

cudaError_t launch_linear_chunks(const LinearArgs &a, float *states, int *err, cudaStream_t st) {
  Params p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.splits = splits_of(a.sweeps, a.batch * a.H, a.T, a.d);
  p.states = states;
  p.err = err;
  // one map a tensor: the sweeps share theirs
  CUtensorMap maps[4];
  memset(maps, 0, sizeof(maps));
  const LinearRows *seen[4];
  auto same = [](const LinearRows &x, const LinearRows &y) {
    return x.x == y.x && x.share == y.share && x.s[0] == y.s[0] && x.s[1] == y.s[1] && x.s[2] == y.s[2];
  };
  int n = 0;
  for (int i = 0; i < a.sweeps; ++i) {
    const LinearRows *rows[3] = {&a.sweep[i].q, &a.sweep[i].k, &a.sweep[i].v};
    for (int j = 0; j < 3; ++j) {
      int m = 0;
      while (m < n && !same(*seen[m], *rows[j])) ++m;
      if (m == n) {
        if (n == 4) return cudaErrorInvalidValue;
        seen[n++] = rows[j];
        if (!make_map(&maps[m], *rows[j], a, p.axes[m])) return cudaErrorInvalidValue;
      }
      p.map[i][j] = m;
    }
  }
  return a.d == 64 ? run<64>(p, maps, st) : run<128>(p, maps, st);
}

}  // namespace fs
