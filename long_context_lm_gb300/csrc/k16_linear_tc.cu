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
// (24 bits).  All sums are fp32; S itself is fp32.
//
// Two passes over the chunks, with a small kernel between them:
//   states  every (sequence, head) is cut into stretches, as many as fill the GPU; a
//           block goes through one with S in registers, from zeros, and leaves the
//           state before each chunk and the one after the last in memory
//   join    runs through the stretches: the state before each
//   rows    all chunks by themselves, in equal runs: S = (the stretch's own) + lam^m (the state
//           before it), then the three products of the outputs
// One pass (states in registers, rows beside them) reads and writes less, but with few
// heads needs the stretches' states beforehand, by a pass as long as the first here, and with
// any number of heads leaves blocks without work: 65536 tokens x 16 heads XX us, now XX;
// 5 ragged sequences of 8191 x 16 heads of 128 321, now XX.  The states between the passes
// (16 KB a chunk of 64 KB of rows; heads of 128: 64 of 128) are kept to what the L2 holds
// by going through long sequences in bands.
//
// What bounds it: XX
#include <cuda.h>
#include <string.h>

#include "fs_common.cuh"
#include "fs_internal.h"
#include "linear.cuh"
#include "pairs.cuh"
#include "tc05.cuh"

namespace fs {
namespace {

constexpr int kC = 128;               // tokens of a chunk
constexpr uint32_t kAtom = kC * 128;  // bytes of 64 elements of a chunk's rows

// A band: the chunks [c0, c1) of every sequence, in the sweep's order.
struct Params {
  LinearArgs a;
  int c0, c1;
  bool first, last;   // band
  int splits;         // stretches of a band
  float *local;       // [sweep, batch H, c1 - c0 - 1, D D]: the state before each chunk but the band's
                      // first, of its stretch alone (none before a stretch's first)
  float *slots;       // [sweep, batch H, splits, D D]: what each stretch adds; then the state before it
  float *carry;       // [sweep, batch H, D D]: the state behind the band
  uint8_t *odd;       // [sweep, batch H, c1 - c0, 8]: not all of the values that a warp of the states'
                      // kernel saw of the chunk are finite
  int map[3][3];      // which map holds q, k, v of a sweep
  int axes[4][2];     // 0 where a map's sequences or heads are one
  int out_axes[3][2];
  int *err;
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
  return !p.last || w.state_out;
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

// ---------------------------------------------------------------------------
// states
// ---------------------------------------------------------------------------
template <int D>
struct StateCfg {
  static constexpr int kAtoms = D / 64, kWarps = D / 16;
  static constexpr int kTma = kWarps, kMma = kWarps + 1, kThreads = 32 * (kWarps + 4);
  static constexpr int kSlab = 32, kSlabs = kC / kSlab;  // tokens of a slab of weighted values
  static constexpr uint32_t kSlabAtom = kSlab * 128;
  static constexpr uint32_t kTile = kAtoms * kAtom, kPart = kAtoms * kSlabAtom;
  static constexpr uint32_t kK = 0, kV = kTile, kSlab0 = 3 * kTile, kBytes = kSlab0 + 3 * kPart;
  static constexpr int kBlocks = D == 64 ? 3 : 1;  // of an SM
};

struct StateShared {
  uint64_t kfull, kempty, vfull[2], vempty[2], slab_full, slab_empty, u_full, u_free, fin;
  uint32_t tmem;
  float power[kC + 4];  // lam^n
};

// Warps: D / 16 that make weighted values (the next slab's in registers while one is
// multiplied) and hold S, then one for TMA loads (values a chunk ahead) and one that issues
// the products.  A thread has 16 bytes of rows r and r + 16 of every slab.
template <int D>
__global__ void __launch_bounds__(StateCfg<D>::kThreads, StateCfg<D>::kBlocks)
    k16_states_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using C = StateCfg<D>;
  using F = Frags<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ StateShared s;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const LinearSweep &w = p.a.sweep[blockIdx.z];
  const int b = blockIdx.y / p.a.H, h = blockIdx.y % p.a.H, r = blockIdx.x;
  const Band band(p, b);
  const bool reverse = w.reverse;
  if (r >= band.stretches) return;
  const int from = band.lo + r * band.per, to = band.end(r);
  const int chunks = to - from - (to == band.chunks && !wants_last(p, w) ? 1 : 0);
  const float decay = p.a.decay[h];

  if (threadIdx.x == 0) {
    for (uint64_t *x : {&s.kfull, &s.kempty, &s.vfull[0], &s.vfull[1], &s.slab_empty, &s.u_full, &s.fin})
      tc::mbar_init(x, 1);
    for (uint64_t *x : {&s.vempty[0], &s.vempty[1], &s.slab_full, &s.u_free}) tc::mbar_init(x, C::kWarps);
    tc::mbar_fence_init();
  }
  for (int i = threadIdx.x; i <= kC; i += C::kThreads) {
    const Factor f = decay_power(decay, i);
    s.power[i] = f.hi + f.lo;
  }
  if (warp == C::kMma) {
    tc::tmem_alloc(&s.tmem, D);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s.tmem, base = smem_u32(smem);

  if (warp == C::kTma && lane == 0) {
    const int mk = p.map[blockIdx.z][1], mv = p.map[blockIdx.z][2];
    auto load = [&](uint32_t at, int m, const LinearRows &x, uint64_t *bar, int i) {
      const int t = band.chunk(from + i, reverse) * kC;
      tc::mbar_arrive_expect_tx(bar, C::kTile);
      for (int k = 0; k < C::kAtoms; ++k)
        load_rows(smem + at + k * kAtom, &maps.in[m], bar, 64 * k, t, h / x.share * p.axes[m][1],
                  b * p.axes[m][0]);
    };
    int nk = 0, nv = 0;  // loaded so far
    bool ok = true;
    for (int i = -1; i < chunks && ok; ++i) {
      if (i + 1 < chunks) {
        if (nv > 1) ok = tc::mbar_wait(&s.vempty[nv & 1], (nv / 2 - 1) & 1, p.err);
        if (!ok) break;
        load(C::kV + (nv & 1) * C::kTile, mv, w.v, &s.vfull[nv & 1], nv);
        ++nv;
      }
      const int k = i < 0 ? 0 : i;
      if (nk == k && k < chunks) {
        if (nk) ok = tc::mbar_wait(&s.kempty, (nk - 1) & 1, p.err);
        if (!ok) break;
        load(C::kK, mk, w.k, &s.kfull, nk);
        ++nk;
      }
    }
    // what is under way lands before the block ends
    if (nk) tc::mbar_wait(&s.kfull, (nk - 1) & 1, nullptr);
    for (int i = nv > 2 ? nv - 2 : 0; i < nv; ++i) tc::mbar_wait(&s.vfull[i & 1], i / 2 & 1, nullptr);
  } else if (warp == C::kMma && lane == 0) {
    constexpr uint32_t kUD = tc::idesc_bf16(D, D, 1) | 1u << 15;  // K^T: its rows run along M
    const uint32_t keys = base + C::kK;
    bool ok = true;
    for (int i = 0; i < chunks && ok; ++i) {
      if (!tc::mbar_wait(&s.kfull, i & 1, p.err)) break;
      if (i && !tc::mbar_wait(&s.u_free, (i - 1) & 1, p.err)) break;
      for (int j = 0; j < C::kSlabs; ++j) {
        if (!(ok = tc::mbar_wait(&s.slab_full, (i * C::kSlabs + j) & 1, p.err))) break;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < 6; ++k)
          tc::mma_ss(tmem, desc_blocks(keys + j * C::kSlabAtom + k % 2 * 2048, kAtom),
                     desc_blocks(base + C::kSlab0 + k / 2 * C::kPart + k % 2 * 2048, C::kSlabAtom), kUD,
                     j > 0 || k > 0);
        tc::mma_commit(&s.slab_empty);
      }
      if (!ok) break;
      tc::mma_commit(&s.u_full);
      tc::mma_commit(&s.kempty);
    }
    tc::mma_commit(&s.fin);
    tc::mbar_wait(&s.fin, 0, nullptr);
  } else if (warp < C::kWarps) {
    const int t = threadIdx.x;
    const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16) + (D == 64 ? 0 : warp / 4 * 64);
    const size_t bh = (size_t)blockIdx.z * gridDim.y + blockIdx.y;
    f2 S[F::kHalves][16];
#pragma unroll
    for (int g = 0; g < F::kHalves; ++g)
#pragma unroll
      for (int e = 0; e < 16; ++e) S[g][e] = 0;
    auto save = [&](float *to) {
#pragma unroll
      for (int g = 0; g < F::kHalves; ++g)
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          *reinterpret_cast<ulonglong2 *>(to + F::at(t, g, e)) = make_ulonglong2(S[g][e], S[g][e + 1]);
    };
    const size_t nb = p.c1 - p.c0;
    // the matrix of the stretch's chunk i >= 1; the flag of chunk i
    auto local = [&](int i) { return p.local + (bh * (nb - 1) + (from - p.c0 + i - 1)) * (D * D); };
    auto flag = [&](int i) { return p.odd + (bh * nb + (from - p.c0 + i)) * 8 + warp; };
    const Factor whole = decay_power(decay, kC);
    const int r16 = t % 128 / 8, ch = t % 8, atom = t / 128;
    const uint32_t in = swz128(r16, ch);
    unsigned char *slab = smem + C::kSlab0 + atom * C::kSlabAtom + in;
    bool ok = true;
    for (int i = 0; i < chunks; ++i) {
      const int n = band.size(band.chunk(from + i, reverse));
      unsigned char *values = smem + C::kV + (i & 1) * C::kTile;
      if (!(ok = WAIT(s.vfull[i & 1], i / 2))) break;
      if (i) save(local(i));
      if (n < kC) {
        // what lies behind the sequence takes no part, whatever it is
        if (!(ok = WAIT(s.kfull, i))) break;
        for (int u = t; u < (kC - n) * (D / 8); u += F::kThreads) {
          const uint32_t at = u % (D / 8) / 8 * kAtom + swz128(n + u / (D / 8), u % 8);
          *reinterpret_cast<uint4 *>(smem + C::kK + at) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(values + at) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_async_smem();
        asm volatile("bar.sync 1, %0;" ::"n"(F::kThreads) : "memory");
      }
      const unsigned char *source = values + atom * kAtom + in;
      uint32_t some = 0;  // the bits of all third parts
#pragma unroll 1
      for (int j = 0; j < C::kSlabs; ++j) {
        uint32_t part[2][3][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int row = j * C::kSlab + r16 + 16 * k;
          const uint4 x = *reinterpret_cast<const uint4 *>(source + j * C::kSlabAtom + k * 2048);
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
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int q = 0; q < 3; ++q)
            *reinterpret_cast<uint4 *>(slab + q * C::kPart + k * 2048) =
                make_uint4(part[k][q][0], part[k][q][1], part[k][q][2], part[k][q][3]);
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&s.slab_full);
      }
      if (!ok) break;
      if (lane == 0) tc::mbar_arrive(&s.vempty[i & 1]);
      if (!(ok = WAIT(s.u_full, i))) break;
      tc::fence_after_sync();
      const Factor f = n == kC ? whole : decay_power(decay, n);
      const f2 hi = f2_bits(f.hi, f.hi), lo = f2_bits(f.lo, f.lo);
#pragma unroll
      for (int g = 0; g < F::kHalves; ++g) {
        f2 u[16];
        tmem_ld_16x64(lanes + ((uint32_t)(16 * g) << 16), u);
        if (g == F::kHalves - 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&s.u_free);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) S[g][e] = madd2(S[g][e], hi, madd2(S[g][e], lo, u[e]));
      }
      // A value that is not finite leaves NaN in its third part (some large finite ones leave bits
      // that look like it: the rows' pass looks again).
      const bool odd = (some & 0x7f80u) == 0x7f80u || (some & 0x7f800000u) == 0x7f800000u;
      const bool any = __any_sync(0xffffffffu, odd);
      if (lane == 0) *flag(i) = any;
    }
    if (ok && chunks < to - from) {  // the last chunk: only the state before it
      if (chunks) save(local(chunks));
      if (lane == 0) *flag(chunks) = 1;
    } else if (ok) {
      save(p.slots + (bh * p.splits + r) * (D * D));
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::kMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, D);
  }
}

// ---------------------------------------------------------------------------
// join
// ---------------------------------------------------------------------------
// Runs through the stretches in the sweep's order: a slot, what its stretch adds, becomes the
// state before the stretch.  Four floats of a matrix a thread.
template <int D>
__global__ void __launch_bounds__(256) k16_join_kernel(const __grid_constant__ Params p) {
  using F = Frags<D>;
  const LinearSweep &w = p.a.sweep[blockIdx.z];
  const int b = blockIdx.y / p.a.H, h = blockIdx.y % p.a.H;
  const Band band(p, b);
  const float decay = p.a.decay[h];
  const int i = blockIdx.x * 256 + threadIdx.x, t = i % F::kThreads, g = i / F::kThreads / 8,
            e = i / F::kThreads % 8 * 2;
  const int row = F::row(t, g, e), col = F::col(t, e);
  const int sr = w.transposed ? 1 : D, sc = w.transposed ? D : 1;
  const size_t bh = (size_t)blockIdx.z * gridDim.y + blockIdx.y;
  float4 *carry = reinterpret_cast<float4 *>(p.carry + bh * (D * D)) + i;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!p.first) {
    x = *carry;
  } else if (w.state) {
    const float *from = w.state + (size_t)blockIdx.y * (D * D) + row * sr + col * sc;
    x = make_float4(from[0] * w.state_mul, from[sc] * w.state_mul, from[8 * sr] * w.state_mul,
                    from[8 * sr + sc] * w.state_mul);
  }
  float4 *at = reinterpret_cast<float4 *>(p.slots + bh * p.splits * (D * D)) + i;
  const int adds = band.stretches - (band.stretches && band.hi == band.chunks && !wants_last(p, w) ? 1 : 0);
  constexpr int kAhead = 8;
  for (int r0 = 0; r0 < band.stretches; r0 += kAhead) {
    float4 y[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (r0 + k < adds) y[k] = at[(size_t)(r0 + k) * (D * D / 4)];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int r = r0 + k;
      if (r >= band.stretches) break;
      at[(size_t)r * (D * D / 4)] = x;
      if (r >= adds) break;
      const Factor f = decay_power(decay, band.tokens(band.lo + r * band.per, band.end(r), w.reverse));
      x = make_float4(f.times(x.x, y[k].x), f.times(x.y, y[k].y), f.times(x.z, y[k].z), f.times(x.w, y[k].w));
    }
  }
  if (!p.last) {
    *carry = x;
  } else if (w.state_out) {
    const float mul = 1.f / w.state_mul;
    float *to = w.state_out + (size_t)blockIdx.y * (D * D) + row * sr + col * sc;
    to[0] = x.x * mul;
    to[sc] = x.y * mul;
    to[8 * sr] = x.z * mul;
    to[8 * sr + sc] = x.w * mul;
  }
}

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
template <int D>
struct RowCfg {
  static constexpr int kAtoms = D / 64, kStateWarps = D / 16;
  static constexpr int kTma = 8 + kStateWarps, kMma = kTma + 1, kThreads = 32 * (kTma + 4);
  // registers a thread: at launch, then of the rows', states' and last four warps
  static constexpr int kRegs = D == 64 ? 64 : 96, kRowRegs = D == 64 ? 64 : 80, kStateRegs = D == 64 ? 88 : 128,
                       kLastRegs = 40;
  static_assert(8 * kRowRegs + kStateWarps * kStateRegs + 4 * kLastRegs <= (12 + kStateWarps) * kRegs, "registers");
  static constexpr uint32_t kTile = kAtoms * kAtom, kSPart = kAtoms * D * 128;  // q, k or v; one part of S
  static constexpr uint32_t kQ = 0, kK = kTile, kV = 2 * kTile, kS = 4 * kTile, kBytes = kS + 2 * kSPart;
  static constexpr uint32_t kScores = 0, kOut = kC, kCols = 256;  // TMEM columns
};

// What the rows' warps need of a head: lam^n times the scale; columns' factors (see there).
struct Tables {
  float scaled[kC + 4];
  alignas(16) float cols[3][32];
};

// A block's run of chunks in the order (sweep, sequence, head, the band's chunks from the last to the
// first: those whose states were written last come first out of the L2).
struct Start {
  int left, z, b, h, ci;
};
// By one warp: chunks of all sequences, then the place of this block's first.
__device__ __forceinline__ Start find_start(const Params &p, int lane) {
  Start s{0, 0, 0, 0, -1};
  const int H = p.a.H;
  auto chunks = [&](int b) {
    if (b >= p.a.batch) return 0;
    const Band band(p, b);
    return band.hi - band.lo;
  };
  auto sum = [](long long x) {
#pragma unroll
    for (int m = 16; m > 0; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
  };
  long long all = 0;
  if (p.a.count) {
    for (int b = lane; b < p.a.batch; b += 32) all += chunks(b);
    all = sum(all);
  } else {
    all = (long long)chunks(0) * p.a.batch;
  }
  const long long total = all * H * p.a.sweeps;
  long long at = total * blockIdx.x / gridDim.x;
  s.left = (int)(total * (blockIdx.x + 1) / gridDim.x - at);
  if (s.left <= 0) return s;
  s.z = (int)(at / (all * H));
  at -= s.z * all * H;
  int n;
  if (p.a.count) {
    for (int b = 0;; b += 32) {  // (the place is in front of the last sequence's end)
      const int mine = chunks(b + lane);
      long long before = mine;
#pragma unroll
      for (int m = 1; m < 32; m *= 2) {
        const long long x = __shfl_up_sync(0xffffffffu, before, m);
        if (lane >= m) before += x;
      }
      const unsigned found = __ballot_sync(0xffffffffu, at < before * H);
      if (found) {
        const int k = __ffs(found) - 1;
        n = __shfl_sync(0xffffffffu, mine, k);
        at -= (__shfl_sync(0xffffffffu, before, k) - n) * H;
        s.b = b + k;
        break;
      }
      at -= __shfl_sync(0xffffffffu, before, 31) * H;
    }
  } else {
    n = chunks(0);
    s.b = (int)(at / ((long long)n * H));
    at -= (long long)s.b * n * H;
  }
  s.h = (int)(at / n);
  s.ci = p.c0 + n - 1 - (int)(at % n);
  return s;
}

struct Walk : Start {
  const Params &p;
  bool reverse;
  __device__ __forceinline__ Walk(const Params &p_, const Start &s) : Start(s), p(p_), reverse(p_.a.sweep[s.z].reverse) {}
  // the next chunk; whether its head is another
  __device__ __forceinline__ bool next() {
    if (--ci >= p.c0) return false;
    if (++h == p.a.H) {
      h = 0;
      for (;;) {
        if (++b == p.a.batch) b = 0, ++z;
        if (z == p.a.sweeps) return true;  // (only behind the last chunk of all)
        const Band band(p, b);
        if (band.hi > band.lo) break;
      }
      reverse = p.a.sweep[z].reverse;
    }
    ci = Band(p, b).hi - 1;
    return true;
  }
};

struct RowShared {
  uint64_t qfull, qempty, kfull, kempty, vfull[2], vempty[2];
  uint64_t ready[2];  // S, tables and values: the states' warps may be a chunk ahead of the rows', not two
  uint64_t s_free, scores, inter, parts, done, o_free, fin;
  uint32_t tmem;
  int odd[2];         // a chunk's values are not all finite
  int bad[2][128];    // per column: the first such token in the sweep's order
  Tables tables[2];
  Start start;
};

// Warps:
//   0-7       rows, two warps to 32 of them, each with half of the columns: scores to bf16
//             parts in their own TMEM columns, Q S times the row's power in place, the
//             finished rows by way of the values' place in shared memory (a TMA store: rows
//             written by their own threads would be 32 places an instruction)
//   8..       states (D / 16 warps): S from its two parts, split, into shared memory; the
//             head's tables
//   last four one for TMA loads (values a chunk ahead), one that issues the products
// Heads of 64 leave room for two blocks an SM, which fill each other's waits; heads of 128
// for one.
template <int D>
__global__ void __launch_bounds__(RowCfg<D>::kThreads, D == 64 ? 2 : 1)
    k16_rows_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using C = RowCfg<D>;
  using F = Frags<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ RowShared s;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (uint64_t *x : {&s.qfull, &s.qempty, &s.kfull, &s.kempty, &s.vfull[0], &s.vfull[1], &s.s_free,
                        &s.scores, &s.inter, &s.done, &s.fin})
      tc::mbar_init(x, 1);
    for (uint64_t *x : {&s.ready[0], &s.ready[1]}) tc::mbar_init(x, C::kStateWarps);
    for (uint64_t *x : {&s.vempty[0], &s.vempty[1], &s.parts, &s.o_free}) tc::mbar_init(x, 8);
    tc::mbar_fence_init();
    s.odd[0] = s.odd[1] = 0;
  }
  for (int i = threadIdx.x; i < 256; i += C::kThreads) s.bad[i / 128][i % 128] = kC;
  if (warp == 0) {
    const Start start = find_start(p, lane);
    if (lane == 0) s.start = start;
  }
  if (warp == C::kMma) {
    tc::tmem_alloc(&s.tmem, C::kCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s.tmem, base = smem_u32(smem);

  if (warp >= C::kTma) {
    tc::regs_dec<C::kLastRegs>();
    if (warp == C::kTma && lane == 0) {
      // ---------------------------------------------------------------- loads
      Walk a(p, s.start), c(p, s.start);  // of q and k; of v, a chunk ahead
      const int chunks = a.left;
      auto load = [&](const Walk &u, uint32_t at, int which, uint64_t *bar) {
        const LinearSweep &w = p.a.sweep[u.z];
        const LinearRows &x = which == 0 ? w.q : which == 1 ? w.k : w.v;
        const int m = p.map[u.z][which], t = Band(p, u.b).chunk(u.ci, u.reverse) * kC;
        tc::mbar_arrive_expect_tx(bar, C::kTile);
        for (int k = 0; k < C::kAtoms; ++k)
          load_rows(smem + at + k * kAtom, &maps.in[m], bar, 64 * k, t, u.h / x.share * p.axes[m][1],
                    u.b * p.axes[m][0]);
      };
      int nq = 0, nk = 0, nv = 0;  // loaded so far
      bool ok = true;
      auto load_v = [&]() {
        if (!ok || nv >= chunks) return;
        if (nv > 1 && !(ok = tc::mbar_wait(&s.vempty[nv & 1], (nv / 2 - 1) & 1, p.err))) return;
        load(c, C::kV + (nv & 1) * C::kTile, 2, &s.vfull[nv & 1]);
        ++nv;
        c.next();
      };
      for (int i = 0; i < chunks && ok; ++i, a.next()) {
        if (nk && !(ok = tc::mbar_wait(&s.kempty, (nk - 1) & 1, p.err))) break;
        load(a, C::kK, 1, &s.kfull);
        ++nk;
        if (nq && !(ok = tc::mbar_wait(&s.qempty, (nq - 1) & 1, p.err))) break;
        load(a, C::kQ, 0, &s.qfull);
        ++nq;
        if (i != 1) load_v();
        if (i == 0) load_v();
      }
      // what is under way lands before the block ends
      if (nq) tc::mbar_wait(&s.qfull, (nq - 1) & 1, nullptr);
      if (nk) tc::mbar_wait(&s.kfull, (nk - 1) & 1, nullptr);
      for (int i = nv > 2 ? nv - 2 : 0; i < nv; ++i) tc::mbar_wait(&s.vfull[i & 1], i / 2 & 1, nullptr);
    } else if (warp == C::kMma && lane == 0) {
      // ------------------------------------------------------------- products
      constexpr uint32_t kQK = tc::idesc_bf16(128, 128, 0), kB = tc::idesc_bf16(128, D, 1);
      const int chunks = s.start.left;
      for (int i = 0; i < chunks; ++i) {
        const uint32_t values = base + C::kV + (i & 1) * C::kTile;
        if (!tc::mbar_wait(&s.kfull, i & 1, p.err) || !tc::mbar_wait(&s.qfull, i & 1, p.err)) break;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_ss(tmem + C::kScores, tc::desc_sw128(base + C::kQ + k / 4 * kAtom + k % 4 * 32),
                     tc::desc_sw128(base + C::kK + k / 4 * kAtom + k % 4 * 32), kQK, k > 0);
        tc::mma_commit(&s.scores);
        tc::mma_commit(&s.kempty);
        if (!tc::mbar_wait(&s.ready[i & 1], i >> 1 & 1, p.err) ||
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
        if (!tc::mbar_wait(&s.vfull[i & 1], i >> 1 & 1, p.err) || !tc::mbar_wait(&s.parts, i & 1, p.err)) break;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < 2 * kC / 16; ++k) {
          const int kk = k % (kC / 16), part = k / (kC / 16);
          tc::mma_ts(tmem + C::kOut, tmem + C::kScores + kk * 16 + part * 8, desc_blocks(values + kk * 2048, kAtom),
                     kB, 1);
        }
        tc::mma_commit(&s.done);
      }
      tc::mma_commit(&s.fin);
      tc::mbar_wait(&s.fin, 0, nullptr);
    }
  } else if (warp >= 8) {
    tc::regs_inc<C::kStateRegs>();
    // ------------------------------------------------------------------ states
    const int t = threadIdx.x - 256;
    // A lane names the row that it is to fill of one of four 8 x 8 blocks: rows + 0 and + 8 of
    // two neighbours among the blocks of columns ([row][column], columns swizzled).
    const uint32_t to = base + C::kS + F::col0(t) / 64 * (D * 128) +
                        (F::row0(t) - lane / 4 + lane / 8 % 2 * 8 + lane % 8) * 128;
    Walk u(p, s.start);
    const int chunks = u.left;
    int which = 0;             // of the tables
    bool fresh = true;         // another head than the last chunk's
    int stretch = -1;
    f2 before[F::kHalves][16];  // the state before the stretch
    for (int i = 0; i < chunks; ++i) {
      const Band band(p, u.b);
      const size_t bh = ((size_t)u.z * p.a.batch + u.b) * p.a.H + u.h;
      const int r = (u.ci - band.lo) / band.per, from = band.lo + r * band.per;
      const size_t nb = p.c1 - p.c0, place = u.ci - p.c0;
      if (fresh || r != stretch) {
        const float *at = p.slots + (bh * p.splits + r) * (D * D);
#pragma unroll
        for (int g = 0; g < F::kHalves; ++g)
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const ulonglong2 x = __ldg(reinterpret_cast<const ulonglong2 *>(at + F::at(t, g, e)));
            before[g][e] = x.x, before[g][e + 1] = x.y;
          }
        stretch = r;
      }
      const bool own = u.ci > from;  // (the first chunk of a stretch has only the state before it)
      const float *at = p.local + (bh * (nb - 1) + (own ? place - 1 : 0)) * (D * D);
      ulonglong2 local[8];
      auto fetch = [&](int g) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          local[e] = own ? __ldg(reinterpret_cast<const ulonglong2 *>(at + F::at(t, g, 2 * e))) : make_ulonglong2(0, 0);
      };
      fetch(0);
      bool look;
      if constexpr (D == 64) {
        look = *reinterpret_cast<const uint32_t *>(p.odd + (bh * nb + place) * 8) != 0;
      } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(p.odd + (bh * nb + place) * 8);
        look = (x.x | x.y) != 0;
      }
      const float decay = p.a.decay[u.h];
      const Factor f = decay_power(decay, band.tokens(from, u.ci, u.reverse));
      const f2 hi = f2_bits(f.hi, f.hi), lo = f2_bits(f.lo, f.lo);
      if (i && !WAIT(s.s_free, i - 1)) break;
      if (fresh) {
        which ^= 1;
        Tables &tab = s.tables[which];
        for (int k = t; k <= kC + 96; k += F::kThreads) {
          const int n = k <= kC ? k : 32 * ((k - kC - 1) / 32 + 1) + (u.reverse ? (k - kC - 1) % 32 - 31 : -((k - kC - 1) % 32));
          const Factor x = decay_power(decay, n);
          if (k <= kC)
            tab.scaled[k] = (x.hi + x.lo) * p.a.scale;
          else
            tab.cols[(k - kC - 1) / 32][(k - kC - 1) % 32] = x.hi + x.lo;
        }
      }
#pragma unroll
      for (int g = 0; g < F::kHalves; ++g) {
        if (g) fetch(g);
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          uint32_t a[4], c[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const f2 y = k % 2 ? local[e / 2 + k / 2].y : local[e / 2 + k / 2].x;
            f2 x = madd2(before[g][e + k], hi, madd2(before[g][e + k], lo, y));
            a[k] = split2(x);
            c[k] = pack2(x);
          }
          const uint32_t spot = to + g * 16 * 128 + (((e / 2 + lane / 16) ^ (lane % 8)) << 4);
          stmatrix4(spot, a);
          stmatrix4(spot + C::kSPart, c);
        }
      }
      const int n = band.size(band.chunk(u.ci, u.reverse));
      if (n < kC || look) {
        if (!WAIT(s.vfull[i & 1], i >> 1)) break;
        unsigned char *values = smem + C::kV + (i & 1) * C::kTile;
        for (int k = t; k < kC * (D / 8); k += F::kThreads) {
          const int row = k / (D / 8), ch = k % (D / 8);
          uint32_t *word = reinterpret_cast<uint32_t *>(values + ch / 8 * kAtom + swz128(row, ch % 8));
          for (int j = 0; j < 4; ++j) {
            if (row >= n) {  // what lies behind the sequence takes no part, whatever it is
              word[j] = 0;
              continue;
            }
            // A value that is not finite leaves the tile, where scores of 0 would make NaN of the rows
            // before it as well; those after it get theirs at the end.
#pragma unroll
            for (int m = 0; m < 2; ++m)
              if ((word[j] >> 16 * m & 0x7f80u) == 0x7f80u) {
                word[j] &= m ? 0xffffu : 0xffff0000u;
                atomicMin(&s.bad[i & 1][ch * 8 + 2 * j + m], u.reverse ? kC - 1 - row : row);
                s.odd[i & 1] = 1;
              }
          }
        }
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&s.ready[i & 1]);
      fresh = u.next();
    }
  } else {
    if constexpr (C::kRowRegs < C::kRegs) tc::regs_dec<C::kRowRegs>();
    // -------------------------------------------------------------------- rows
    // lam^|i - j| for 32 columns that all rows of the warp see is a factor of the row and
    // one of the column, counted from the warp's near edge, so that neither passes 1
    const int quarter = warp % 4, half = warp / 4, row = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    Walk u(p, s.start);
    const int chunks = u.left;
    int which = 0;
    bool fresh = true;
    bool storing = false;  // (lane 0) a store may still read the values' place
    for (int i = 0; i < chunks; ++i) {
      const Band band(p, u.b);
      const LinearSweep &w = p.a.sweep[u.z];
      const bool reverse = u.reverse;
      const int chunk = band.chunk(u.ci, reverse), n = band.size(chunk);
      if (fresh) which ^= 1;
      if (!WAIT(s.ready[i & 1], i >> 1) || !WAIT(s.scores, i)) break;
      tc::fence_after_sync();
      const Tables &tab = s.tables[which];
      const float rowf = tab.scaled[reverse ? 31 - lane : lane];
      const f2 rowff = f2_bits(rowf, rowf);
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
            const ulonglong2 *cw = reinterpret_cast<const ulonglong2 *>(tab.cols[off - 1] + 16 * half);
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
                v[k] = seen ? __uint_as_float(x[2 * e + k]) * tab.scaled[abs(lag)] : 0.f;
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
        tc::mbar_arrive(&s.vempty[(i - 1) & 1]);
      }
      __syncwarp();
      if (!WAIT(s.inter, i)) break;
      tc::fence_after_sync();
      const uint32_t out = lanes + C::kOut + half * (D / 2);
      {
        const float f = tab.scaled[reverse ? max(n - 1 - row, 0) : row + 1];
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
      if (!WAIT(s.done, i)) break;
      tc::fence_after_sync();
      const bool odd = s.odd[i & 1] != 0;
      // whole warps of bf16 rows leave by TMA, 64 columns at a time; the last rows of a
      // sequence, and fp32 parts, from their threads
      const bool whole = 32 * quarter + 32 <= n && !w.out_f32;
      unsigned char *box = smem + C::kV + (i & 1) * C::kTile + (D == 64 ? 0 : half * kAtom) + quarter * 4096;
      const long long to = u.b * w.os[0] + u.h * w.os[1] + (chunk * (long long)kC + row) * w.os[2] + half * (D / 2);
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
          store_rows(box, &maps.out[u.z], D == 64 ? 0 : 64 * half, chunk * kC + 32 * quarter,
                     u.h * p.out_axes[u.z][1], u.b * p.out_axes[u.z][0]);
          bulk_commit();
          storing = true;
        }
      }
      if (odd) {  // clean for the chunk after the next
        asm volatile("bar.sync 2, 256;" ::: "memory");
        if (warp < 4 && row < D) s.bad[i & 1][row] = kC;
        if (warp == 0 && lane == 0) s.odd[i & 1] = 0;
      }
      fresh = u.next();
    }
    if (lane == 0) bulk_wait_read<0>();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::kMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kCols);
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

// Chunks of a band, and the stretches that they are cut into.
struct Plan {
  int chunks, band, splits;
  size_t local, slots, carry, odd, total;  // bytes
};
constexpr size_t kBandBytes = (size_t)160 << 20;
Plan plan_of(int sweeps, int pairs, int T, int d) {
  Plan q;
  const size_t matrix = (size_t)d * d * 4, all = (size_t)sweeps * pairs;
  q.chunks = (T + kC - 1) / kC;
  // bands of equal length whose states stay within kBandBytes
  size_t most = kBandBytes / (all * matrix);
  if (most < 1) most = 1;
  const size_t bands = (q.chunks + most - 1) / most;
  q.band = (int)((q.chunks + bands - 1) / bands);
  const int blocks = 152 * (d == 64 ? StateCfg<64>::kBlocks : StateCfg<128>::kBlocks);
  int n = (int)(blocks / (all < (size_t)blocks ? all : blocks));
  const int longest = (q.band + 3) / 4;  // four chunks a stretch at least
  q.splits = n < longest ? n : longest;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  q.local = all * (q.band - 1) * matrix;
  q.slots = all * q.splits * matrix;
  q.carry = bands > 1 ? all * matrix : 0;
  q.odd = up(all * q.band * 8);
  q.total = q.local + q.slots + q.carry + q.odd;
  return q;
}

template <int D>
cudaError_t run(Params &p, const Maps &m, const Plan &q, cudaStream_t st) {
  auto states = k16_states_kernel<D>;
  auto rows = k16_rows_kernel<D>;
  constexpr int kStates = StateCfg<D>::kBytes + 1024, kRows = RowCfg<D>::kBytes + 1024;
  cudaError_t e = cudaFuncSetAttribute(states, cudaFuncAttributeMaxDynamicSharedMemorySize, kStates);
  if (e != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(rows, cudaFuncAttributeMaxDynamicSharedMemorySize, kRows)) != cudaSuccess) return e;
  const int pairs = p.a.batch * p.a.H;
  for (int c = 0; c < q.chunks; c += q.band) {
    p.c0 = c;
    p.c1 = c + q.band < q.chunks ? c + q.band : q.chunks;
    p.first = c == 0;
    p.last = p.c1 == q.chunks;
    states<<<dim3(p.splits, pairs, p.a.sweeps), StateCfg<D>::kThreads, kStates, st>>>(m, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    k16_join_kernel<D><<<dim3(D * D / 1024, pairs, p.a.sweeps), 256, 0, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const long long units = (long long)p.a.sweeps * pairs * (p.c1 - p.c0), blocks = 152 * (D == 64 ? 2 : 1);
    rows<<<(unsigned)(units < blocks ? units : blocks), RowCfg<D>::kThreads, kRows, st>>>(m, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t linear_chunk_bytes(int sweeps, int batch, int H, int T, int d) {
  return plan_of(sweeps, batch * H, T, d).total;
}

cudaError_t launch_linear_chunks(const LinearArgs &a, void *ws, int *err, cudaStream_t st) {
  const Plan q = plan_of(a.sweeps, a.batch * a.H, a.T, a.d);
  Params p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.splits = q.splits;
  char *at = static_cast<char *>(ws);
  p.local = reinterpret_cast<float *>(at);
  p.slots = reinterpret_cast<float *>(at + q.local);
  p.carry = reinterpret_cast<float *>(at + q.local + q.slots);
  p.odd = reinterpret_cast<uint8_t *>(at + q.local + q.slots + q.carry);
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
  return a.d == 64 ? run<64>(p, maps, q, st) : run<128>(p, maps, q, st);
}

}  // namespace fs
