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
//   0-7       rows, two warps to 32 of them, each with half of the columns: scores to bf16
//             parts in their own TMEM columns, Q S times the row's power in place, the
//             finished rows by way of the values' place in shared memory (a TMA store: rows
//             written by their own threads would be 32 places an instruction)
//   8..       states (D / 16 warps): weighted values into a slab, the next one's made in
//             registers while it is multiplied; S in registers, its bf16 parts into
//             shared memory for the next chunk
//   last four one for TMA loads, one that issues the products of the rows, one that issues
//             those of the slabs (issued by one thread, slabs waited behind the rows'
//             products, a slab at a time, and took 7000 cycles a chunk in place of 3000)
// Values are loaded a chunk ahead.  Heads of 64 leave room for two blocks an SM, which
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
#include "pairs.cuh"
#include "tc05.cuh"

namespace fs {
namespace {

constexpr int kC = 128;       // tokens of a chunk
constexpr uint32_t kAtom = kC * 128;       // 64 elements of a chunk's rows

struct Params {
  LinearArgs a;
  int splits;
  float *states;     // [sweep, batch H, splits, D D]: the state before each stretch
  int map[3][3];     // which map holds q, k, v of a sweep
  int axes[4][2];    // 0 where a map's sequences or heads are one
  int out_axes[3][2];
  int *err;
};

struct Maps {
  CUtensorMap in[4], out[3];
};

template <int D>
struct Cfg {
  static constexpr int kAtoms = D / 64;
  static constexpr int kStateWarps = D / 16;
  static constexpr int kTma = 8 + kStateWarps, kMma = kTma + 1, kMmaU = kTma + 2;
  static constexpr int kThreads = 32 * (kTma + 4);
  static constexpr int kSlab = 32, kSlabs = kC / kSlab;  // tokens of a slab, slabs
  static constexpr int kUnits = 2;  // 16-byte pieces of a slab for a state thread
  // registers a thread: at launch, then of the rows', states' and last four warps
  static constexpr int kRegs = D == 64 ? 64 : 96, kRowRegs = D == 64 ? 64 : 80, kStateRegs = D == 64 ? 88 : 128,
                       kLastRegs = 40;
  static_assert(8 * kRowRegs + kStateWarps * kStateRegs + 4 * kLastRegs <= (12 + kStateWarps) * kRegs, "registers");
  static constexpr uint32_t kSlabAtom = kSlab * 128;
  static constexpr int kHalves = D / 64;  // groups of 16 rows that a state warp holds
  static constexpr int kValues = 2;                              // chunks of v held
  static constexpr uint32_t kTile = kAtoms * kAtom;              // q, k or v
  static constexpr uint32_t kPart = kAtoms * kSlabAtom;          // one part of a slab
  static constexpr uint32_t kSPart = kAtoms * D * 128;           // one part of S
  static constexpr uint32_t kQ = 0, kK = kTile, kV = kK + kTile, kS = kV + kValues * kTile,
                            kSlab0 = kS + 2 * kSPart, kBytes = kSlab0 + 3 * kPart;
  // TMEM columns: scores (then their parts), outputs, the chunk's addition to S
  static constexpr uint32_t kScores = 0, kOut = kC, kU = kC + D, kCols = D == 64 ? 256 : 512;
};

struct Shared {
  uint64_t qfull, qempty, kfull, kempty, vfull[2], vempty[2];
  uint64_t slab_full, slab_empty;
  uint64_t s_ready, s_free, scores, inter, parts, done, o_free, u_full, u_free, fin, fin_u;
  // values looked through: the states' warps may be a chunk ahead of the rows', not two
  uint64_t checked[2];
  uint32_t tmem;
  int odd[2];                 // a chunk's values are not all finite
  float power[kC + 4];        // lam^n
  float scaled[kC + 4];       // scale lam^n
  alignas(16) float cols[3][32];  // see the rows' warps (read four at a time)
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

__device__ __forceinline__ void stmatrix4(uint32_t at, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(at), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

#define WAIT(bar, k) __all_sync(0xffffffffu, tc::mbar_wait(&(bar), (k) & 1, p.err))

// kRows: the whole sweep; without, only the states of the stretches (into p.states).
template <int D, bool kRows>
__global__ void __launch_bounds__(Cfg<D>::kThreads, D == 64 ? 2 : 1)
    k16_linear_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
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
    for (uint64_t *x : {&s.qfull, &s.qempty, &s.kfull, &s.s_free, &s.scores, &s.inter, &s.done, &s.u_full, &s.fin})
      tc::mbar_init(x, 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.vfull[i], 1);
      tc::mbar_init(&s.vempty[i], kRows ? 8 : C::kStateWarps);
    }
    tc::mbar_init(&s.slab_empty, 1);
    for (uint64_t *x : {&s.slab_full, &s.s_ready, &s.u_free, &s.checked[0], &s.checked[1]}) tc::mbar_init(x, C::kStateWarps);
    for (uint64_t *x : {&s.parts, &s.o_free}) tc::mbar_init(x, 8);
    tc::mbar_init(&s.kempty, kRows ? 2 : 1);  // read by the scores' product and by the slabs'
    tc::mbar_init(&s.fin_u, 1);
    tc::mbar_fence_init();
    s.odd[0] = s.odd[1] = 0;
  }
  for (int i = threadIdx.x; i <= kC; i += C::kThreads) {
    const Factor f = decay_power(decay, i);
    s.power[i] = f.hi + f.lo;
    s.scaled[i] = (f.hi + f.lo) * p.a.scale;
  }
  for (int i = threadIdx.x; i < 96; i += C::kThreads) {
    const Factor f = decay_power(decay, 32 * (i / 32 + 1) + (reverse ? i % 32 - 31 : -(i % 32)));
    s.cols[i / 32][i % 32] = f.hi + f.lo;
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
  if (warp >= C::kTma) {
    tc::regs_dec<C::kLastRegs>();
  if (warp == C::kTma && lane == 0) {
    // ------------------------------------------------------------------ loads
    const int mq = p.map[blockIdx.z][0], mk = p.map[blockIdx.z][1], mv = p.map[blockIdx.z][2];
    auto load = [&](uint32_t at, int m, const LinearRows &x, uint64_t *bar, int i) {
      const int t = st.chunk(st.from + i, reverse) * kC;
      tc::mbar_arrive_expect_tx(bar, C::kTile);
      for (int k = 0; k < C::kAtoms; ++k)
        load_rows(smem + at + k * kAtom, &maps.in[m], bar, 64 * k, t, h / x.share * p.axes[m][1],
                  b * p.axes[m][0]);
    };
    int nq = 0, nk = 0, nv = 0;  // loaded so far
    bool ok = true;
    auto load_q = [&]() {
      if (!kRows || !ok || nq >= chunks) return;
      if (nq && !(ok = tc::mbar_wait(&s.qempty, (nq - 1) & 1, p.err))) return;
      load(C::kQ, mq, w.q, &s.qfull, nq);
      ++nq;
    };
    auto load_k = [&]() {
      if (!ok || nk >= chunks) return;
      if (nk && !(ok = tc::mbar_wait(&s.kempty, (nk - 1) & 1, p.err))) return;
      load(C::kK, mk, w.k, &s.kfull, nk);
      ++nk;
    };
    auto load_v = [&]() {
      const int at = nv % C::kValues;
      if (!ok || nv >= chunks) return;
      if (nv >= C::kValues && !(ok = tc::mbar_wait(&s.vempty[at], (nv / C::kValues - 1) & 1, p.err))) return;
      load(C::kV + at * C::kTile, mv, w.v, &s.vfull[at], nv);
      ++nv;
    };
    // in the order in which places become free
    load_k();
    load_q();
    load_v();
    load_v();
    for (int i = 1; i < chunks && ok; ++i) {
      load_q();
      load_k();
      load_v();
    }
    // what is under way lands before the block ends
    if (nq) tc::mbar_wait(&s.qfull, (nq - 1) & 1, nullptr);
    if (nk) tc::mbar_wait(&s.kfull, (nk - 1) & 1, nullptr);
    for (int i = nv > C::kValues ? nv - C::kValues : 0; i < nv; ++i)
      tc::mbar_wait(&s.vfull[i % C::kValues], i / C::kValues & 1, nullptr);
  } else if (kRows && warp == C::kMma && lane == 0) {
    // ----------------------------------------------------- products of the rows
    constexpr uint32_t kQK = tc::idesc_bf16(128, 128, 0), kB = tc::idesc_bf16(128, D, 1);
    const uint32_t keys = base + C::kK;
    for (int i = 0; i < chunks; ++i) {
      const uint32_t values = base + C::kV + i % C::kValues * C::kTile;
      if (!tc::mbar_wait(&s.kfull, i & 1, p.err) || !tc::mbar_wait(&s.qfull, i & 1, p.err)) break;
      tc::fence_after_sync();
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        tc::mma_ss(tmem + C::kScores, tc::desc_sw128(base + C::kQ + k / 4 * kAtom + k % 4 * 32),
                   tc::desc_sw128(keys + k / 4 * kAtom + k % 4 * 32), kQK, k > 0);
      tc::mma_commit(&s.scores);
      tc::mma_commit(&s.kempty);
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
      if (!tc::mbar_wait(&s.parts, i & 1, p.err) || !tc::mbar_wait(&s.checked[i & 1], i >> 1 & 1, p.err)) break;
      tc::fence_after_sync();
#pragma unroll
      for (int k = 0; k < 2 * kC / 16; ++k) {
        const int kk = k % (kC / 16), part = k / (kC / 16);
        tc::mma_ts(tmem + C::kOut, tmem + C::kScores + kk * 16 + part * 8,
                   desc_blocks(values + kk * 2048, kAtom), kB, 1);
      }
      tc::mma_commit(&s.done);
    }
    tc::mma_commit(&s.fin);
    tc::mbar_wait(&s.fin, 0, nullptr);
  } else if (warp == C::kMmaU && lane == 0) {
    // ---------------------------------------------------- products of the slabs
    constexpr uint32_t kUD = tc::idesc_bf16(D, D, 1) | 1u << 15;  // K^T: its rows run along M
    const uint32_t keys = base + C::kK;
    bool ok = true;
    for (int i = 0; i < chunks && ok; ++i) {
      if (!tc::mbar_wait(&s.kfull, i & 1, p.err)) break;
      if (i && !tc::mbar_wait(&s.u_free, (i - 1) & 1, p.err)) break;
      for (int j = 0; j < C::kSlabs; ++j) {
        const int at = i * C::kSlabs + j;
        if (!(ok = tc::mbar_wait(&s.slab_full, at & 1, p.err))) break;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < 3 * C::kUnits; ++k) {
          const int kk = k % C::kUnits, part = k / C::kUnits;
          tc::mma_ss(tu, desc_blocks(keys + j * C::kSlabAtom + kk * 2048, kAtom),
                     desc_blocks(base + C::kSlab0 + part * C::kPart + kk * 2048, C::kSlabAtom),
                     kUD, j > 0 || k > 0);
        }
        tc::mma_commit(&s.slab_empty);
      }
      if (!ok) break;
      tc::mma_commit(&s.u_full);
      tc::mma_commit(&s.kempty);
    }
    tc::mma_commit(&s.fin_u);
    tc::mbar_wait(&s.fin_u, 0, nullptr);
  }
  } else if (warp >= 8) {
    tc::regs_inc<C::kStateRegs>();
    // ------------------------------------------------------------------ states
    constexpr int kT = 32 * C::kStateWarps;
    const int sw = warp - 8, t = threadIdx.x - 256;
    // this lane's places in S: rows row0 + 16 g (+ 8), columns col0 + 8 e (+ 1)
    const int row0 = (D == 64 ? sw * 16 : sw % 4 * 32) + lane / 4;
    const int col0 = (D == 64 ? 0 : sw / 4 * 64) + lane % 4 * 2;
    const uint32_t lanes = tu + ((uint32_t)(warp % 4 * 32) << 16) + (D == 64 ? 0 : sw / 4 * 64);
    const size_t bh = (size_t)blockIdx.z * gridDim.y + blockIdx.y;
    f2 S[C::kHalves][16];
    auto each = [&](auto f) {  // f(pair, row, column of its first)
#pragma unroll
      for (int g = 0; g < C::kHalves; ++g)
#pragma unroll
        for (int e = 0; e < 16; ++e) f(S[g][e], row0 + 16 * g + (e & 1) * 8, col0 + e / 2 * 8);
    };
    // between the passes states lie as the lanes hold them
    auto slot = [&](int i) { return p.states + (bh * p.splits + i) * (D * D) + t * 4; };
    const float *given = w.state ? w.state + (size_t)blockIdx.y * D * D : nullptr;
    if (kRows && st.last > 0) {
      const float *from = slot(r);
#pragma unroll
      for (int g = 0; g < C::kHalves; ++g)
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(from + (g * 8 + e / 2) * kT * 4);
          S[g][e] = x.x, S[g][e + 1] = x.y;
        }
    } else if (given && r == 0) {
      const int sr = w.transposed ? 1 : D, sc = w.transposed ? D : 1;
      each([&](f2 &x, int row, int col) {
        const float *at = given + row * sr + col * sc;
        x = f2_bits(at[0] * w.state_mul, at[sc] * w.state_mul);
      });
    } else {
      each([&](f2 &x, int, int) { x = 0; });
    }
    auto save = [&](float *to) {
#pragma unroll
      for (int g = 0; g < C::kHalves; ++g)
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          *reinterpret_cast<ulonglong2 *>(to + (g * 8 + e / 2) * kT * 4) = make_ulonglong2(S[g][e], S[g][e + 1]);
    };
    // S as the factor of the next product: two parts, [row][column] with the columns
    // swizzled.  A lane names the row that it is to fill of one of four 8 x 8 blocks:
    // rows + 0 and + 8 of two neighbours among the blocks of columns.
    const uint32_t sat = base + C::kS + col0 / 64 * (D * 128) + (row0 - lane / 4 + lane / 8 % 2 * 8 + lane % 8) * 128;
    auto publish = [&]() {
#pragma unroll
      for (int g = 0; g < C::kHalves; ++g)
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f2 x = S[g][e + k];
            hi[k] = split2(x);
            lo[k] = pack2(x);
          }
          const uint32_t at = sat + g * 16 * 128 + (((e / 2 + lane / 16) ^ (lane % 8)) << 4);
          stmatrix4(at, hi);
          stmatrix4(at + C::kSPart, lo);
        }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&s.s_ready);
    };
    if (!kRows && r == 0) save(slot(0));
    if (kRows && chunks) publish();
    const Factor whole = decay_power(decay, kC);
    // this thread's sixteen bytes of a slab's row r16 (and r16 + 16)
    const int r16 = t % 128 / 8, ch = t % 8, atom = t / 128;
    const uint32_t in = swz128(r16, ch);
    unsigned char *to = smem + C::kSlab0 + atom * C::kSlabAtom + in;
    for (int i = 0; i < chunks; ++i) {
      const int n = st.size(st.chunk(st.from + i, reverse));
      unsigned char *values = smem + C::kV + i % C::kValues * C::kTile;
      if (!WAIT(s.vfull[i % C::kValues], i / C::kValues)) break;
      if (n < kC) {
        // what lies behind the sequence takes no part, whatever it is
        if (!WAIT(s.kfull, i)) break;
        unsigned char *keys = smem + C::kK;
        for (int u = t; u < (kC - n) * (D / 8); u += kT) {
          const uint32_t at = u % (D / 8) / 8 * kAtom + swz128(n + u / (D / 8), u % 8);
          *reinterpret_cast<uint4 *>(keys + at) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(values + at) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_async_smem();
        asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kStateWarps) : "memory");
      }
      unsigned char *from = values + atom * kAtom + in;
      uint32_t some = 0;  // the bits of all third parts
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < C::kSlabs; ++j) {
        uint32_t part[C::kUnits][3][4];
#pragma unroll
        for (int k = 0; k < C::kUnits; ++k) {
          const int row = j * C::kSlab + r16 + 16 * k;
          const uint4 x = *reinterpret_cast<const uint4 *>(from + j * C::kSlabAtom + k * 2048);
          const float f = row < n ? s.power[reverse ? row + 1 : n - 1 - row] : 0.f;
          const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            f2 y = mul2(wide2(v[c]), f2_bits(f, f));
            part[k][0][c] = split2(y);
            part[k][1][c] = split2(y);
            part[k][2][c] = pack2(y);
            some |= part[k][2][c];
          }
        }
        const int at = i * C::kSlabs + j;
        if (at && !(ok = WAIT(s.slab_empty, at - 1))) break;
#pragma unroll
        for (int k = 0; k < C::kUnits; ++k)
#pragma unroll
          for (int q = 0; q < 3; ++q)
            *reinterpret_cast<uint4 *>(to + q * C::kPart + k * 2048) =
                make_uint4(part[k][q][0], part[k][q][1], part[k][q][2], part[k][q][3]);
        // A value that is not finite leaves NaN in the third part (and NaN in the state's column).
        // It leaves V before the scores' product, where scores of 0 would make NaN of the rows
        // before it as well; those after it get theirs at the end.
        if (kRows && j + 1 == C::kSlabs &&
            ((some & 0x7f80u) == 0x7f80u || (some & 0x7f800000u) == 0x7f800000u)) {
          for (int u = 0; u < kC / 16; ++u) {
            const int row = 16 * u + r16;
            uint32_t *word = reinterpret_cast<uint32_t *>(from + u * 2048);
            for (int c = 0; c < 8; ++c) {
              if ((word[c / 2] >> c % 2 * 16 & 0x7f80u) != 0x7f80u) continue;
              word[c / 2] &= c % 2 ? 0xffffu : 0xffff0000u;
              atomicMin(&s.bad[i & 1][atom * 64 + ch * 8 + c], reverse ? kC - 1 - row : row);
              s.odd[i & 1] = 1;
            }
          }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&s.slab_full);
      }
      if (!ok) break;
      if (lane == 0) tc::mbar_arrive(kRows ? &s.checked[i & 1] : &s.vempty[i % C::kValues]);
      if (!WAIT(s.u_full, i)) break;
      tc::fence_after_sync();
      const Factor f = n == kC ? whole : decay_power(decay, n);
      const f2 hi = f2_bits(f.hi, f.hi), lo = f2_bits(f.lo, f.lo);
#pragma unroll
      for (int g = 0; g < C::kHalves; ++g) {
        f2 u[16];
        tmem_ld_16x64(lanes + ((uint32_t)(16 * g) << 16), u);
        if (g == C::kHalves - 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s.u_free);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) S[g][e] = madd2(S[g][e], hi, madd2(S[g][e], lo, u[e]));
      }
      if (kRows && i + 1 < chunks) {
        if (!WAIT(s.s_free, i)) break;
        publish();
      }
    }
    if (!kRows) {
      save(slot(r + 1));
    } else if (r == st.last && w.state_out) {
      float *out = w.state_out + (size_t)blockIdx.y * D * D;
      const int sr = w.transposed ? 1 : D, sc = w.transposed ? D : 1;
      const float mul = 1.f / w.state_mul;
      each([&](f2 &x, int row, int col) {
        float *at = out + row * sr + col * sc;
        at[0] = lo2(x) * mul;
        at[sc] = hi2(x) * mul;
      });
    }
  } else {
    // (without rows too: the states' share counts on it)
    if constexpr (C::kRowRegs < C::kRegs) tc::regs_dec<C::kRowRegs>();
    if constexpr (kRows) {
    // -------------------------------------------------------------------- rows
    // lam^|i - j| for 32 columns that all rows of the warp see is a factor of the row and
    // one of the column, counted from the warp's near edge, so that neither passes 1
    const int quarter = warp % 4, half = warp / 4, row = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const float rowf = s.scaled[reverse ? 31 - lane : lane];
    const f2 rowff = f2_bits(rowf, rowf);
    const CUtensorMap *map = &maps.out[blockIdx.z];
    const int mh = h * p.out_axes[blockIdx.z][1], mb = b * p.out_axes[blockIdx.z][0];
    bool storing = false;  // (lane 0) a store may still read the values' place
    for (int i = 0; i < chunks; ++i) {
      const int chunk = st.chunk(st.from + i, reverse), n = st.size(chunk);
      if (!WAIT(s.scores, i)) break;
      tc::fence_after_sync();
      const uint32_t at = lanes + C::kScores + 16 * half;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t parts[2][8];
        const int off = reverse ? c - quarter : quarter - c;
        if (off < 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) parts[0][e] = parts[1][e] = 0;
        } else {
          uint32_t x[16];
          tc::tmem_ld16(at + 32 * c, x);
          tc::tmem_wait_ld();
          if (off > 0 && (!reverse || 32 * c + 32 <= n)) {
            const ulonglong2 *cw = reinterpret_cast<const ulonglong2 *>(s.cols[off - 1] + 16 * half);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const ulonglong2 f = cw[e];
              f2 y = mul2(mul2((f2)x[4 * e] | (f2)x[4 * e + 1] << 32, f.x), rowff);
              f2 z = mul2(mul2((f2)x[4 * e + 2] | (f2)x[4 * e + 3] << 32, f.y), rowff);
              parts[0][2 * e] = split2(y);
              parts[1][2 * e] = pack2(y);
              parts[0][2 * e + 1] = split2(z);
              parts[1][2 * e + 1] = pack2(z);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float v[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int j = 32 * c + 16 * half + 2 * e + k, lag = reverse ? j - row : row - j;
                const bool seen = lag >= 0 && (!reverse || j < n);
                v[k] = seen ? __uint_as_float(x[2 * e + k]) * s.scaled[abs(lag)] : 0.f;
              }
              f2 y = f2_bits(v[0], v[1]);
              parts[0][e] = split2(y);
              parts[1][e] = pack2(y);
            }
          }
        }
        tc::tmem_st8(at + 32 * c, parts[0]);
        tc::tmem_st8(at + 32 * c + 8, parts[1]);
      }
      if (i && lane == 0) {  // the last chunk's rows are on their way
        if (storing) bulk_wait_read<0>();
        tc::mbar_arrive(&s.vempty[(i - 1) % C::kValues]);
      }
      __syncwarp();
      if (!WAIT(s.inter, i)) break;
      tc::fence_after_sync();
      const uint32_t out = lanes + C::kOut + half * (D / 2);
      {
        const float f = s.scaled[reverse ? max(n - 1 - row, 0) : row + 1];
        const f2 ff = f2_bits(f, f);
#pragma unroll
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
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&s.parts);
      if (!WAIT(s.checked[i & 1], i >> 1) || !WAIT(s.done, i)) break;
      tc::fence_after_sync();
      const bool odd = s.odd[i & 1] != 0;
      // whole warps of bf16 rows leave by TMA, 64 columns at a time; the last rows of a
      // sequence, and fp32 parts, from their threads
      const bool whole = 32 * quarter + 32 <= n && !w.out_f32;
      unsigned char *box = smem + C::kV + i % C::kValues * C::kTile + (D == 64 ? 0 : half * kAtom) + quarter * 4096;
      const long long to = b * w.os[0] + h * w.os[1] + (chunk * (long long)kC + row) * w.os[2] + half * (D / 2);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[16];
        tc::tmem_ld16(out + 16 * c, x);
        tc::tmem_wait_ld();
        if (c == D / 32 - 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s.o_free);
        }
        if (odd) {
#pragma unroll 1
          for (int e = 0; e < 16; ++e) {
            const bool bad = s.bad[i & 1][half * (D / 2) + 16 * c + e] <= (reverse ? kC - 1 - row : row);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (k == e && bad) x[k] = 0x7fc00000u;
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
      storing = false;
      if (whole) {
        tc::fence_async_smem();
        if (D == 64)  // two warps' halves of one box
          asm volatile("bar.sync %0, 64;" ::"r"(3 + quarter) : "memory");
        else
          __syncwarp();
        if (lane == 0 && (D == 128 || half == 0)) {
          store_rows(box, map, D == 64 ? 0 : 64 * half, chunk * kC + 32 * quarter, mh, mb);
          bulk_commit();
          storing = true;
        }
      }
      if (odd) {  // clean for the chunk after the next
        asm volatile("bar.sync 2, 256;" ::: "memory");
        if (warp < 4 && row < D) s.bad[i & 1][row] = kC;
        if (warp == 0 && lane == 0) s.odd[i & 1] = 0;
      }
    }
    if (lane == 0) bulk_wait_read<0>();
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

// [batch, heads, T, D] rows in boxes of 128 bytes x `tokens`; an axis of stride 0 (one long, or the
// same for all) is one long.
bool make_map(CUtensorMap *map, const void *x, const long long (&s)[3], bool f32, int batch, int heads,
              int T, int d, int tokens, int *axes) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t size = f32 ? 4 : 2;
  axes[0] = s[0] != 0;
  axes[1] = s[1] != 0;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)(axes[1] ? heads : 1),
                              (cuuint64_t)(axes[0] ? batch : 1)};
  const cuuint64_t strides[3] = {(cuuint64_t)s[2] * size, (axes[1] ? (cuuint64_t)s[1] : d) * size,
                                 (axes[0] ? (cuuint64_t)s[0] : d) * size};
  const cuuint32_t box[4] = {(cuuint32_t)(128 / size), (cuuint32_t)tokens, 1, 1}, estr[4] = {1, 1, 1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void *>(x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Stretches of a sweep: as many as blocks fit at once, eight chunks each at least.  (Below that the
// two further launches and the second read of k and v cost what the shorter way saves: 8 x 16
// heads of 333 tokens 33 us in two stretches, 20 in one.)
int splits_of(int sweeps, int pairs, int T, int d) {
  const int blocks = 152 * (d == 64 ? 2 : 1), most = (T + kC - 1) / kC / 8;
  const int n = blocks / (sweeps * pairs < blocks ? sweeps * pairs : blocks);
  return n < most ? n : most < 1 ? 1 : most;
}

template <int D>
cudaError_t run(const Params &p, const Maps &m, cudaStream_t st) {
  constexpr int kSmem = Cfg<D>::kBytes + 1024;
  const int pairs = p.a.batch * p.a.H;
  if (p.splits > 1) {
    auto f = k16_linear_kernel<D, false>;
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    f<<<dim3(p.splits - 1, pairs, p.a.sweeps), Cfg<D>::kThreads, kSmem, st>>>(m, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    k16_join_kernel<D><<<dim3(D * D / 1024, pairs, p.a.sweeps), 256, 0, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  auto f = k16_linear_kernel<D, true>;
  const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  f<<<dim3(p.splits, pairs, p.a.sweeps), Cfg<D>::kThreads, kSmem, st>>>(m, p);
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
  Maps maps;
  memset(&maps, 0, sizeof(maps));
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
        if (!make_map(&maps.in[m], rows[j]->x, rows[j]->s, false, a.batch, a.H / rows[j]->share, a.T, a.d, kC,
                      p.axes[m]))
          return cudaErrorInvalidValue;
      }
      p.map[i][j] = m;
    }
    if (!make_map(&maps.out[i], a.sweep[i].out, a.sweep[i].os, a.sweep[i].out_f32, a.batch, a.H, a.T, a.d, 32,
                  p.out_axes[i]))
      return cudaErrorInvalidValue;
  }
  return a.d == 64 ? run<64>(p, maps, st) : run<128>(p, maps, st);
}

}  // namespace fs
