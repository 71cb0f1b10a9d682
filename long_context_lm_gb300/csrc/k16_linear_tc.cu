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
// powers, and S as a factor, go in as a bf16 high and low part, off by 2^-17 of
// themselves at most: 2^9 times less than what the rounding of q, k and v to bf16, 2^-8, may
// have put into the same terms, so that no cancellation shows it before that.  Of the
// outputs 0.24% are the step beside the rounded value (with fp32 products 0.02%).  (A third
// part of the scores wants 64 TMEM columns more, where two blocks of one pass over heads
// of 64 take all 512; one of S 32 KB of shared memory, where heads of 128 take 217 of 227.)
// The weighted values, of which states are made, go in as three parts (24 bits), since a
// state adds up over thousands of chunks.  All sums are fp32; S itself is fp32.
//
// Two passes over the chunks, with a small kernel between them:
//   states  every (sequence, head) is cut into stretches, as many as fill the GPU; a
//           block goes through one with S in registers, from zeros, and leaves the
//           state before each chunk and the one after the last in memory
//   join    runs through the stretches: the state before each
//   rows    all chunks by themselves, in equal runs: S = (the stretch's own) + lam^m (the state
//           before it), then the three products of the outputs
// One pass (k17_linear_fused.cu: states in registers, rows beside them) reads and writes less,
// but with few heads needs the stretches' states beforehand, by a pass as long as the first here,
// and with any number of heads leaves blocks without work.  65536 tokens x 16 heads: 263 us in one
// pass, 210 in two.  States of heads of 128 are half of a chunk's rows (64 KB of 128; of 64 a
// quarter): 5 ragged sequences of 8191 x 16 heads of 128: 493 us in two passes, 292 in one.
//
// What bounds it: 65536 tokens x 16 heads move 1.07 GB in two passes (537 MB in and out have to, the
// keys and values go in twice, the states out and in), 158 us at the copy's rate; states 88 us, join
// 13, rows 110 (a chunk's three waits of rows on products and of products on rows, by two blocks an
// SM in turn).
#include <algorithm>

#include "linear_tc.cuh"

namespace fs {
namespace {

using namespace lin;

// ---------------------------------------------------------------------------
// states
// ---------------------------------------------------------------------------
// Heads of 128 are taken by two blocks, 64 columns (of v) each.
template <int D>
struct StateCfg {
  static constexpr int kAtoms = D / 64, kParts = D / 64, kWarps = D / 16, kStateThreads = 32 * kWarps;
  static constexpr int kTma = kWarps, kMma = kWarps + 1, kThreads = 32 * (kWarps + 4);
  static constexpr int kRows = kStateThreads / 8;              // rows that the threads take at once
  static constexpr int kSlab = 2 * kRows, kSlabs = kC / kSlab;  // tokens of a slab of weighted values
  static constexpr uint32_t kTile = kAtoms * kAtom, kPart = kSlab * 128;
  static constexpr uint32_t kK = 0, kV = kTile, kSlab0 = kV + 2 * kAtom, kBytes = kSlab0 + 3 * kPart;
  static constexpr int kBlocks = D == 64 ? 3 : 2;  // of an SM
};

struct StateShared {
  uint64_t kfull, kempty, vfull[2], vempty[2], slab_full, slab_empty, u_full, u_free, fin;
  uint32_t tmem;
  float power[kC + 4];  // lam^n
};

// Warps: D / 16 that make weighted values (the next slab's in registers while one is
// multiplied) and hold S, then one for TMA loads (values a chunk ahead) and one that issues
// the products.  A thread has 16 bytes of two rows of every slab, and in a state of 128 x 64 one of the two
// groups of 16 rows that Frags gives a warp.
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
  const int z = p.own[blockIdx.z];
  const LinearSweep &w = p.a.sweep[z];
  const int b = blockIdx.y / p.a.H, h = blockIdx.y % p.a.H;
  const int r = blockIdx.x / C::kParts, part0 = blockIdx.x % C::kParts;
  const Band band(p, b);
  const bool reverse = w.reverse;
  // (fused: nobody starts from the last stretch's)
  if (r >= band.stretches - (p.fused ? 1 : 0)) return;
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
    tc::tmem_alloc(&s.tmem, 64);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s.tmem, base = smem_u32(smem);

  if (warp == C::kTma && lane == 0) {
    const int mk = p.map[z][1], mv = p.map[z][2];
    // `atoms` times 64 columns from column x0 on
    auto load = [&](uint32_t at, int m, const LinearRows &x, uint64_t *bar, int i, int x0, int atoms) {
      const int t = band.chunk(from + i, reverse) * kC;
      tc::mbar_arrive_expect_tx(bar, atoms * kAtom);
      for (int k = 0; k < atoms; ++k)
        load_rows(smem + at + k * kAtom, &maps.in[m], bar, x0 + 64 * k, t, h / x.share * p.axes[m][1],
                  b * p.axes[m][0]);
    };
    int nk = 0, nv = 0;  // loaded so far
    bool ok = true;
    for (int i = -1; i < chunks && ok; ++i) {
      if (i + 1 < chunks) {
        if (nv > 1) ok = wait_for(&s.vempty[nv & 1], (nv / 2 - 1) & 1, p);
        if (!ok) break;
        load(C::kV + (nv & 1) * kAtom, mv, w.v, &s.vfull[nv & 1], nv, 64 * part0, 1);
        ++nv;
      }
      const int k = i < 0 ? 0 : i;
      if (nk == k && k < chunks) {
        if (nk) ok = wait_for(&s.kempty, (nk - 1) & 1, p);
        if (!ok) break;
        load(C::kK, mk, w.k, &s.kfull, nk, 0, C::kAtoms);
        ++nk;
      }
    }
    // what is under way lands before the block ends
    if (nk) tc::mbar_wait(&s.kfull, (nk - 1) & 1, nullptr);
    for (int i = nv > 2 ? nv - 2 : 0; i < nv; ++i) tc::mbar_wait(&s.vfull[i & 1], i / 2 & 1, nullptr);
  } else if (warp == C::kMma && lane == 0) {
    constexpr uint32_t kUD = tc::idesc_bf16(D, 64, 1) | 1u << 15;  // K^T: its rows run along M
    const uint32_t keys = base + C::kK;
    bool ok = true;
    for (int i = 0; i < chunks && ok; ++i) {
      if (!wait_for(&s.kfull, i & 1, p)) break;
      if (i && !wait_for(&s.u_free, (i - 1) & 1, p)) break;
      for (int j = 0; j < C::kSlabs; ++j) {
        if (!(ok = wait_for(&s.slab_full, (i * C::kSlabs + j) & 1, p))) break;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < 3 * C::kSlab / 16; ++k) {
          const int kk = k % (C::kSlab / 16), part = k / (C::kSlab / 16);
          tc::mma_ss(tmem, desc_blocks(keys + j * C::kPart + kk * 2048, kAtom),
                     tc::desc_sw128(base + C::kSlab0 + part * C::kPart + kk * 2048), kUD, j > 0 || k > 0);
        }
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
    const int group = D == 64 ? 0 : warp / 4, place = D == 64 ? t : part0 * 128 + t % 128;  // in Frags
    const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32 + 16 * group) << 16);
    const size_t bh = (size_t)blockIdx.z * gridDim.y + blockIdx.y;
    f2 S[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) S[e] = 0;
    auto save = [&](float *to) {
#pragma unroll
      for (int e = 0; e < 16; e += 2)
        *reinterpret_cast<ulonglong2 *>(to + F::at(place, group, e)) = make_ulonglong2(S[e], S[e + 1]);
    };
    const size_t nb = p.c1 - p.c0;
    // the matrix of the stretch's chunk i >= 1; the flag of chunk i
    auto local = [&](int i) { return p.local + (bh * (nb - 1) + (from - p.c0 + i - 1)) * (D * D); };
    auto flag = [&](int i) { return p.odd + (bh * nb + (from - p.c0 + i)) * 8 + warp; };
    const Factor whole = decay_power(decay, kC);
    const int r0 = t / 8;
    const uint32_t in = swz128(r0, t % 8);
    unsigned char *slab = smem + C::kSlab0 + in;
    bool ok = true;
    for (int i = 0; i < chunks; ++i) {
      const int n = band.size(band.chunk(from + i, reverse));
      unsigned char *values = smem + C::kV + (i & 1) * kAtom;
      if (!(ok = WAIT(s.vfull[i & 1], i / 2))) break;
      if (i && !p.fused) save(local(i));
      if (n < kC) {
        // what lies behind the sequence takes no part, whatever it is
        if (!(ok = WAIT(s.kfull, i))) break;
        for (int u = t; u < (kC - n) * (D / 8); u += C::kStateThreads)
          *reinterpret_cast<uint4 *>(smem + C::kK + u % (D / 8) / 8 * kAtom + swz128(n + u / (D / 8), u % 8)) =
              make_uint4(0, 0, 0, 0);
        // values: what this thread reads itself (the fence before the first slab's arrival is the keys')
#pragma unroll 1
        for (int row = r0; row < kC; row += C::kRows)
          if (row >= n) *reinterpret_cast<uint4 *>(values + in + (row - r0) * 128) = make_uint4(0, 0, 0, 0);
      }
      const unsigned char *source = values + in;
      uint32_t some = 0;  // the bits of all third parts
#pragma unroll 1
      for (int j = 0; j < C::kSlabs; ++j) {
        uint32_t part[2][3][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int row = j * C::kSlab + r0 + C::kRows * k;
          const uint4 x = *reinterpret_cast<const uint4 *>(source + j * C::kPart + k * C::kRows * 128);
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
            *reinterpret_cast<uint4 *>(slab + q * C::kPart + k * C::kRows * 128) =
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
      f2 u[16];
      tmem_ld_16x64(lanes, u);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&s.u_free);
#pragma unroll
      for (int e = 0; e < 16; ++e) S[e] = madd2(S[e], hi, madd2(S[e], lo, u[e]));
      // A value that is not finite leaves NaN in its third part (some large finite ones leave bits
      // that look like it: the rows' pass looks again).
      const bool odd = (some & 0x7f80u) == 0x7f80u || (some & 0x7f800000u) == 0x7f800000u;
      const bool any = __any_sync(0xffffffffu, odd);
      if (lane == 0 && !p.fused) *flag(i) = any;
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
    tc::tmem_dealloc(tmem, 64);
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
  const LinearSweep &w = p.a.sweep[p.own[blockIdx.z]];
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
  // (the last stretch of a sequence: not where nobody wants the state behind it)
  const int adds = band.stretches - (band.stretches && band.hi == band.chunks && !wants_last(p, w) ? 1 : 0);
  constexpr int kAhead = 8;
  const Factor whole = decay_power(decay, band.per * kC);
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
      const int n = band.tokens(band.lo + r * band.per, band.end(r), w.reverse);
      const Factor f = n == band.per * kC ? whole : decay_power(decay, n);
      x = make_float4(f.times(x.x, y[k].x), f.times(x.y, y[k].y), f.times(x.z, y[k].z), f.times(x.w, y[k].w));
    }
  }
  if (!p.last) {
    *carry = x;
  } else if (w.state_out && !p.fused) {
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
struct RowCfg {
  static constexpr int D = 64, kStateWarps = D / 16;
  static constexpr int kTma = 8 + kStateWarps, kMma = kTma + 1, kThreads = 32 * (kTma + 4);
  // registers a thread: at launch and the rows', then the states' and the last four warps'
  static constexpr int kRegs = 64, kStateRegs = 88, kLastRegs = 40;
  static_assert(8 * kRegs + kStateWarps * kStateRegs + 4 * kLastRegs <= (12 + kStateWarps) * kRegs, "registers");
  static constexpr uint32_t kTile = kAtom, kSPart = D * 128;  // q, k or v; one part of S
  static constexpr uint32_t kQ = 0, kK = kTile, kV = 2 * kTile, kS = 4 * kTile, kBytes = kS + 2 * kSPart;
  static constexpr uint32_t kScores = 0, kOut = kC, kCols = 256;  // TMEM columns
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
  Band band;
  __device__ __forceinline__ Walk(const Params &p_, const Start &s)
      : Start(s), p(p_), reverse(p_.a.sweep[s.z].reverse), band(p_, s.b) {}
  // the next chunk; whether its head is another
  __device__ __forceinline__ bool next() {
    if (--ci >= p.c0) return false;
    if (++h == p.a.H) {
      h = 0;
      for (;;) {
        if (++b == p.a.batch) b = 0, ++z;
        if (z == p.a.sweeps) return true;  // (only behind the last chunk of all)
        band = Band(p, b);
        if (band.hi > band.lo) break;
      }
      reverse = p.a.sweep[z].reverse;
    }
    ci = band.hi - 1;
    return true;
  }
};

struct RowShared {
  uint64_t qfull, qempty, kfull, kempty, vfull[2], vempty[2];
  // S and tables; values looked through: their warps may be a chunk ahead of the rows', not two
  uint64_t ready[2], checked[2];
  uint64_t s_free, scores, inter, parts, done, o_free, fin;
  uint64_t pairs[4];  // a chunk's rows of the second of two warps are in the values' place
  uint32_t tmem;
  bool turned[2];     // S is another sweep's, transposed
  int odd[2];         // i + 1: the values of the block's chunk i are not all finite
  int bad[2][128];    // per column, as bad_mark
  Tables tables[2];
  Start start;
};

// A chunk's values: what lies behind the sequence takes no part, whatever it is.  A value that
// is not finite leaves the tile, where scores of 0 would make NaN of the rows before it as well;
// those after it get theirs at the end.
__device__ __forceinline__ void look_through(RowShared &s, unsigned char *values, int i, int n, bool reverse, int t,
                                             int threads) {
  const int ch = t % 8;
#pragma unroll 1
  for (int row = t / 8; row < kC; row += threads / 8) {
    uint4 *place = reinterpret_cast<uint4 *>(values + swz128(row, ch));
    if (row >= n) {
      *place = make_uint4(0, 0, 0, 0);
      continue;
    }
    if (!not_finite(*place)) continue;
    uint32_t *word = reinterpret_cast<uint32_t *>(place);
    for (int j = 0; j < 8; ++j) {
      if ((word[j / 2] >> j % 2 * 16 & 0x7f80u) != 0x7f80u) continue;
      word[j / 2] &= j % 2 ? 0xffffu : 0xffff0000u;
      atomicMax(&s.bad[i & 1][ch * 8 + j], bad_mark(i, reverse ? kC - 1 - row : row));
      s.odd[i & 1] = i + 1;
    }
  }
  tc::fence_async_smem();
}

// Warps:
//   0-7       rows, two warps to 32 of them, each with half of the columns: scores to bf16
//             parts in their own TMEM columns, Q S times the row's power in place, the
//             finished rows by way of the values' place in shared memory (a TMA store: rows
//             written by their own threads would be 32 places an instruction)
//   8-11      states: S from its two parts, split, into shared memory; the head's tables
//   last four one for TMA loads (values a chunk ahead), one that issues the products, with
//             kTurns two that look through values
// Heads of 64 alone, for which there is room for two blocks an SM that fill each other's waits.
// kTurns: one of the sweeps borrows its states.  Then warps of their own look through the values
// (by the states' warps gradients of 4 x 4096 tokens x 16 heads 174 us, so 159); else the states'
// warps do, where the first pass has seen something (so 65536 tokens x 16 heads 210 us,
// with warps of their own 216).
template <bool kTurns>
__global__ void __launch_bounds__(RowCfg::kThreads, 2)
    k16_rows_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using C = RowCfg;
  constexpr int D = C::D;
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
    for (uint64_t &x : s.pairs) tc::mbar_init(&x, 1);
    for (uint64_t *x : {&s.ready[0], &s.ready[1]}) tc::mbar_init(x, C::kStateWarps);
    for (uint64_t *x : {&s.checked[0], &s.checked[1]}) tc::mbar_init(x, 2);
    for (uint64_t *x : {&s.vempty[0], &s.vempty[1], &s.parts, &s.o_free}) tc::mbar_init(x, 8);
    tc::mbar_fence_init();
    s.odd[0] = s.odd[1] = 0;
  }
  for (int i = threadIdx.x; i < 256; i += C::kThreads) s.bad[i / 128][i % 128] = 0;
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
      Walk a(p, s.start);
      const int chunks = a.left;
      auto load = [&](const Walk &u, uint32_t at, int which, uint64_t *bar) {
        const LinearSweep &w = p.a.sweep[u.z];
        const LinearRows &x = which == 0 ? w.q : which == 1 ? w.k : w.v;
        const int m = p.map[u.z][which], t = u.band.chunk(u.ci, u.reverse) * kC;
        tc::mbar_arrive_expect_tx(bar, C::kTile);
        load_rows(smem + at, &maps.in[m], bar, 0, t, u.h / x.share * p.axes[m][1], u.b * p.axes[m][0]);
      };
      int nq = 0, nk = 0, nv = 0;  // loaded so far
      for (; nv < chunks; a.next()) {
        if (nk && !wait_for(&s.kempty, (nk - 1) & 1, p)) break;
        load(a, C::kK, 1, &s.kfull);
        ++nk;
        if (nq && !wait_for(&s.qempty, (nq - 1) & 1, p)) break;
        load(a, C::kQ, 0, &s.qfull);
        ++nq;
        if (nv > 1 && !wait_for(&s.vempty[nv & 1], (nv / 2 - 1) & 1, p)) break;
        load(a, C::kV + (nv & 1) * C::kTile, 2, &s.vfull[nv & 1]);
        ++nv;
      }
      // what is under way lands before the block ends
      if (nq) tc::mbar_wait(&s.qfull, (nq - 1) & 1, nullptr);
      if (nk) tc::mbar_wait(&s.kfull, (nk - 1) & 1, nullptr);
      for (int i = nv > 2 ? nv - 2 : 0; i < nv; ++i) tc::mbar_wait(&s.vfull[i & 1], i / 2 & 1, nullptr);
    } else if (warp == C::kMma && lane == 0) {
      // ------------------------------------------------------------- products
      constexpr uint32_t kQK = tc::idesc_bf16(128, 128, 0), kB = tc::idesc_bf16(128, D, 1);
      constexpr uint32_t kBT = tc::idesc_bf16(128, D, 0);  // (S transposed: its columns along K)
      const int chunks = s.start.left;
      for (int i = 0; i < chunks; ++i) {
        // (kept from computing the descriptors beforehand, for which there are no registers)
        uint32_t here = base;
        asm volatile("" : "+r"(here));
        const uint32_t values = here + C::kV + (i & 1) * C::kTile;
        if (!wait_for(&s.kfull, i & 1, p) || !wait_for(&s.qfull, i & 1, p)) break;
        tc::fence_after_sync();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc::mma_ss(tmem + C::kScores, tc::desc_sw128(here + C::kQ + k / 4 * kAtom + k % 4 * 32),
                     tc::desc_sw128(here + C::kK + k / 4 * kAtom + k % 4 * 32), kQK, k > 0);
        tc::mma_commit(&s.scores);
        tc::mma_commit(&s.kempty);
        if (!wait_for(&s.ready[i & 1], i >> 1 & 1, p) ||
            (i && !wait_for(&s.o_free, (i - 1) & 1, p)))
          break;
        tc::fence_after_sync();
        const uint64_t sd = tc::desc_sw128(here + C::kS);
        if (kTurns && s.turned[i & 1]) {
#pragma unroll
          for (int k = 0; k < 2 * D / 16; ++k)
            tc::mma_ss(tmem + C::kOut, tc::desc_sw128(here + C::kQ + k % 4 * 32),
                       sd + (k / 4 * C::kSPart + k % 4 * 32) / 16, kBT, k > 0);
        } else {
#pragma unroll
          for (int k = 0; k < 2 * D / 16; ++k)
            tc::mma_ss(tmem + C::kOut, tc::desc_sw128(here + C::kQ + k % 4 * 32),
                       sd + (k / 4 * C::kSPart + k % 4 * 2048) / 16, kB, k > 0);
        }
        tc::mma_commit(&s.inter);
        tc::mma_commit(&s.s_free);
        tc::mma_commit(&s.qempty);
        if (!wait_for(kTurns ? &s.checked[i & 1] : &s.vfull[i & 1], i >> 1 & 1, p) ||
            !wait_for(&s.parts, i & 1, p))
          break;
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
    } else if (kTurns && warp > C::kMma) {
      // --------------------------------------------------------------- values
      const int t = threadIdx.x - 32 * (C::kMma + 1);
      Walk u(p, s.start);
      const int chunks = u.left;
      for (int i = 0; i < chunks; ++i, u.next()) {
        const size_t bh = ((size_t)p.slot[u.z] * p.a.batch + u.b) * p.a.H + u.h;
        const bool look =
            *reinterpret_cast<const uint32_t *>(p.odd + (bh * (p.c1 - p.c0) + (u.ci - p.c0)) * 8) != 0;
        const int n = u.band.size(u.band.chunk(u.ci, u.reverse));
        if (!WAIT(s.vfull[i & 1], i >> 1)) break;
        if (n < kC || look || u.z == p.borrows)  // (nobody has looked through a borrower's values)
          look_through(s, smem + C::kV + (i & 1) * C::kTile, i, n, u.reverse, t, 64);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&s.checked[i & 1]);
      }
    }
  } else if (warp >= 8) {
    tc::regs_inc<C::kStateRegs>();
    // ------------------------------------------------------------------ states
    const int t = threadIdx.x - 256;
    const Publisher<D> publisher(base + C::kS, t);
    Walk u(p, s.start);
    const int chunks = u.left;
    int which = 0;             // of the tables
    bool fresh = true;         // another head than the last chunk's
    int stretch = -1;
    f2 before[16];             // the state before the stretch
    for (int i = 0; i < chunks; ++i) {
      const Band &band = u.band;
      const size_t bh = ((size_t)p.slot[u.z] * p.a.batch + u.b) * p.a.H + u.h;
      const int r = (u.ci - band.lo) / band.per, from = band.lo + r * band.per;
      const size_t nb = p.c1 - p.c0, place = u.ci - p.c0;
      if (fresh || r != stretch) {
        const float *at = p.slots + (bh * p.splits + r) * (D * D);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const ulonglong2 x = __ldg(reinterpret_cast<const ulonglong2 *>(at + F::at(t, 0, e)));
          before[e] = x.x, before[e + 1] = x.y;
        }
        stretch = r;
      }
      const bool own = u.ci > from;  // (the first chunk of a stretch has only the state before it)
      const float *at = p.local + (bh * (nb - 1) + (own ? place - 1 : 0)) * (D * D);
      ulonglong2 local[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        local[e] = own ? __ldg(reinterpret_cast<const ulonglong2 *>(at + F::at(t, 0, 2 * e))) : make_ulonglong2(0, 0);
      const bool look = !kTurns && *reinterpret_cast<const uint32_t *>(p.odd + (bh * nb + place) * 8) != 0;
      const float decay = p.a.decay[u.h];
      const Factor f = decay_power(decay, band.tokens(from, u.ci, u.reverse));
      const f2 hi = f2_bits(f.hi, f.hi), lo = f2_bits(f.lo, f.lo);
      if (i && !WAIT(s.s_free, i - 1)) break;
      if (kTurns && t == 0) s.turned[i & 1] = u.z == p.borrows;
      if (fresh) {
        which ^= 1;
        fill_tables(s.tables[which], decay, u.reverse, p.a.scale, t, F::kThreads);
      }
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        f2 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f2 y = k % 2 ? local[e / 2 + k / 2].y : local[e / 2 + k / 2].x;
          x[k] = madd2(before[e + k], hi, madd2(before[e + k], lo, y));
        }
        publisher.put(0, e, x);
      }
      tc::fence_async_smem();
      if (!kTurns) {
        const int n = band.size(band.chunk(u.ci, u.reverse));
        if (n < kC || look) {
          if (!WAIT(s.vfull[i & 1], i >> 1)) break;
          look_through(s, smem + C::kV + (i & 1) * C::kTile, i, n, u.reverse, t, F::kThreads);
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&s.ready[i & 1]);
      fresh = u.next();
    }
  } else {
    // -------------------------------------------------------------------- rows
    const RowWarp<D> rows(warp, lane, tmem + C::kScores, tmem + C::kOut);
    Walk u(p, s.start);
    const int chunks = u.left;
    int which = 0;
    bool fresh = true;
    bool storing = false;  // (lane 0) a store may still read the values' place
    for (int i = 0; i < chunks; ++i) {
      const bool reverse = u.reverse;
      const int chunk = u.band.chunk(u.ci, reverse), n = u.band.size(chunk);
      if (fresh) which ^= 1;
      if (!WAIT(s.ready[i & 1], i >> 1) || !WAIT(s.scores, i)) break;
      tc::fence_after_sync();
      const Tables &tab = s.tables[which];
      rows.parts(tab, reverse, n);
      if (i && lane == 0) {  // the last chunk's rows are on their way
        if (storing) bulk_wait_read<0>();
        tc::mbar_arrive(&s.vempty[(i - 1) & 1]);
      }
      __syncwarp();
      if (!WAIT(s.inter, i)) break;
      tc::fence_after_sync();
      rows.weigh(tab, reverse, n);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&s.parts);
      if ((kTurns && !WAIT(s.checked[i & 1], i >> 1)) || !WAIT(s.done, i)) break;
      tc::fence_after_sync();
      storing = rows.store(p.a.sweep[u.z], &maps.out[u.z], p.out_axes[u.z], u.b, u.h, chunk, n, i, reverse,
                           s.odd[i & 1] == i + 1 ? s.bad[i & 1] : nullptr, smem + C::kV + (i & 1) * C::kTile,
                           &s.o_free, s.pairs, p);
      fresh = u.next();
    }
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
    tc::tmem_wait_st();  // (a wait that gave up may have left parts on their way into columns that are given back)
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

// [batch, heads, T, D] rows in boxes of 64 elements x `tokens`; an axis of stride 0 (one long, or the
// same for all) is one long.
bool make_map(CUtensorMap *map, const void *x, const long long (&s)[3], int batch, int heads, int T, int d,
              int tokens, int *axes) {
  EncodeTiled fn = encode_fn();
  if (!fn) return false;
  axes[0] = s[0] != 0;
  axes[1] = s[1] != 0;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)(axes[1] ? heads : 1),
                              (cuuint64_t)(axes[0] ? batch : 1)};
  const cuuint64_t strides[3] = {(cuuint64_t)s[2] * 2, (cuuint64_t)(axes[1] ? s[1] : d) * 2,
                                 (cuuint64_t)(axes[0] ? s[0] : d) * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)tokens, 1, 1}, estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(x), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Which way, chunks of a band, and the stretches that they are cut into.
struct Plan {
  bool fused;
  int chunks, band, splits;
  size_t local, slots, carry, odd, total;  // bytes
};
// (Bands small enough for the L2 to keep their states and keys between the passes cost more launches
// than they save: 65536 tokens x 16 heads in bands of 40 MB 289 us, of 80 MB 245, in one 210.)
constexpr size_t kBandBytes = (size_t)160 << 20;
constexpr size_t resident_of(int d) { return 152 * (d == 64 ? 2 : 1); }  // blocks of the fused kernel
// heads (of all sweeps) whose blocks fill the GPU
constexpr size_t filled_by(int sweeps, int d) { return sweeps == 3 ? resident_of(d) * 4 / 5 : resident_of(d); }
Plan plan_of(int sweeps, int pairs, int T, int d) {
  Plan q{};
  const size_t matrix = (size_t)d * d * 4;
  const size_t all = (size_t)sweeps * pairs;
  // Of the gradients' sweeps the second, over R^T, has the states of the third, over R.
  const size_t own = sweeps == 3 ? (size_t)2 * pairs : all;
  q.chunks = q.band = (T + kC - 1) / kC;
  const size_t resident = resident_of(d);
  // Heads of 64 in one pass: where blocks of whole heads fill the GPU (24 x 16 heads of 2048 tokens
  // 172 us, in two passes 173; 16 x 16: 146 and 136; gradients, whose sweeps are three, 6 x 16 of
  // 4096 197 and 233, 4 x 16 183 and 160), and where the chain of a head's chunks, 5.5 us each up to
  // a block an SM and 9 above, is shorter than two passes, 31 us and 24 ns a chunk of any head (2 x 16
  // heads of 640 tokens 27 us, in two passes 33; of 1024 38 and 36; 8 x 16 of 1024 40 and 55, of 2048
  // 95 and 80).
  q.fused = d == 128 || all >= filled_by(sweeps, d) ||
            (all > 152 ? q.chunks < 9 : q.chunks * (230 - all) < 1290);
  if (q.fused) {
    // Stretches of eight chunks at least, as many as fill the GPU once (heads of 128: 32 of 8191 tokens in
    // four stretches 159 us, in fourteen 163; 64 in two 262, in seven 293, ragged 262 and 239; gradients of
    // 16 three 241, six 255), and none where blocks of whole heads fill five eighths of it (128 heads of 4096
    // one 172, three 286; 96 of 8191 321 and 384, ragged 321 and 303; 160 of 4096 one 331, two 372; 256 335
    // and 489; gradients of 40 one 323, three 482).  Below that one stretch would leave too much empty, and
    // two pay for a pass more: three times what is resident (80 ragged heads of 8191 one 319, five 292; even
    // 319 and 347).
    size_t n = all < resident ? resident / all : 1;
    if (n == 1 && all < resident * 5 / 8) n = 3 * resident / all;
    const size_t most = q.chunks / 8;
    q.splits = (int)(n < most ? n : most < 1 ? 1 : most);
    q.slots = q.splits > 1 ? own * q.splits * matrix : 0;
    q.total = q.slots;
    return q;
  }
  // bands of equal length whose states stay within kBandBytes
  const size_t most = kBandBytes / (own * matrix) > 1 ? kBandBytes / (own * matrix) : 1;
  const size_t bands = (q.chunks + most - 1) / most;
  q.band = (int)((q.chunks + bands - 1) / bands);
  // four chunks a stretch at least
  const size_t n = 152 * StateCfg<64>::kBlocks / own, longest = (q.band + 3) / 4;
  q.splits = (int)(n < longest ? n : longest);
  q.local = own * (q.band - 1) * matrix;
  q.slots = own * q.splits * matrix;
  q.carry = bands > 1 ? own * matrix : 0;
  q.odd = (own * q.band * 8 + 255) / 256 * 256;
  q.total = q.local + q.slots + q.carry + q.odd;
  return q;
}

template <int D>
cudaError_t run(Params &p, const Maps &m, const Plan &q, cudaStream_t st) {
  auto states = k16_states_kernel<D>;
  constexpr int kStates = StateCfg<D>::kBytes + 1024, kRows = RowCfg::kBytes + 1024;
  cudaError_t e = cudaFuncSetAttribute(states, cudaFuncAttributeMaxDynamicSharedMemorySize, kStates);
  if (e != cudaSuccess) return e;
  auto rows = p.a.sweeps == 3 ? k16_rows_kernel<true> : k16_rows_kernel<false>;
  if ((e = cudaFuncSetAttribute(rows, cudaFuncAttributeMaxDynamicSharedMemorySize, kRows)) != cudaSuccess)
    return e;
  const int pairs = p.a.batch * p.a.H;
  p.fused = q.fused;
  const bool borrow = p.a.sweeps == 3;
  p.borrows = borrow ? 1 : -1;
  int owners = 0;
  for (int i = 0; i < p.a.sweeps; ++i)
    if (i != p.borrows) p.slot[i] = owners, p.own[owners++] = i;
  if (borrow) p.slot[1] = p.slot[2];
  for (int c = 0; c < q.chunks; c += q.band) {
    p.c0 = c;
    p.c1 = c + q.band < q.chunks ? c + q.band : q.chunks;
    p.first = c == 0;
    p.last = p.c1 == q.chunks;
    if (!q.fused || p.splits > 1) {
      const int stretches = q.fused ? p.splits - 1 : p.splits;
      states<<<dim3(stretches * StateCfg<D>::kParts, pairs, owners), StateCfg<D>::kThreads, kStates, st>>>(m, p);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      k16_join_kernel<D><<<dim3(D * D / 1024, pairs, owners), 256, 0, st>>>(p);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (q.fused) return lin::launch_fused(p, m, st);
    const long long units = (long long)p.a.sweeps * pairs * (p.c1 - p.c0), blocks = 152 * 2;
    rows<<<(unsigned)(units < blocks ? units : blocks), RowCfg::kThreads, kRows, st>>>(m, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

// What plan_of wants for this shape and for any with fewer sequences or tokens: plans change from two
// passes to one, and from one band to two, where the next larger shape wants less.
size_t linear_chunk_bytes(int sweeps, int batch, int H, int T, int d) {
  const size_t matrix = (size_t)d * d * 4, chunks = (T + kC - 1) / kC;
  const auto least = [](size_t a, size_t b) { return a < b ? a : b; };
  const int owners = sweeps == 3 ? 2 : 1;
  // One pass: two stretches or more of eight chunks or more, of which three times what is resident at most.
  size_t one = 0;
  if (chunks >= 16) one = least(3 * resident_of(d) * owners / sweeps, (size_t)owners * batch * H * (chunks / 8)) * matrix;
  // Two passes: the largest batch that takes them.
  size_t two = 0;
  if (d == 64) {
    const size_t own = owners * H * least(batch, (filled_by(sweeps, d) - 1) / ((size_t)sweeps * H));
    const size_t states = own * chunks * matrix;
    two = least(states, kBandBytes) + least(152 * StateCfg<64>::kBlocks, own * ((chunks + 3) / 4)) * matrix +
          (states > kBandBytes ? own * matrix : 0) + (least(states, kBandBytes) / matrix * 8 + 255) / 256 * 256;
  }
  const size_t now = plan_of(sweeps, batch * H, T, d).total;
  return std::max({one, two, now});
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
  p.polls = a.wait_cycles < tc::kWaitCycles ? 0 : 255;
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
        if (!make_map(&maps.in[m], rows[j]->x, rows[j]->s, a.batch, a.H / rows[j]->share, a.T, a.d, kC,
                      p.axes[m]))
          return cudaErrorInvalidValue;
      }
      p.map[i][j] = m;
    }
    // (fp32 parts leave from their threads)
    if (!a.sweep[i].out_f32 &&
        !make_map(&maps.out[i], a.sweep[i].out, a.sweep[i].os, a.batch, a.H, a.T, a.d, 32, p.out_axes[i]))
      return cudaErrorInvalidValue;
  }
  return a.d == 64 ? run<64>(p, maps, q, st) : run<128>(p, maps, q, st);
}

}  // namespace fs
