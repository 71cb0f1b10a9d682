// k17_linear_fused.cu -- linear attention over prompts in one pass: a block takes a
// (sequence, head), or a stretch of one, chunk after chunk, with its state in registers.
// The mathematics and the precision are k16_linear_tc.cu's, which chooses between the ways and
// makes the states before stretches.
//
// Every byte of q, k, v and out moves once (k and v twice but for a sequence's last
// stretch where there are stretches); states never leave the SM.  A chunk's q and k lie in
// shared memory once, its values twice (loaded a chunk ahead); each is loaded anew as
// soon as its last product has read it.  Warps:
//   0-7       rows, two warps to 32 of them, each with half of the columns (RowWarp)
//   8..       states (D / 16 warps): weighted values into a slab, the next one's made in
//             registers while it is multiplied; S in registers, its bf16 parts into
//             shared memory for the next chunk
//   last four one for TMA loads, one that issues the products of the rows, one that issues
//             those of the slabs (issued by one thread, slabs waited behind the rows'
//             products: 7000 cycles a chunk in place of 3000)
// Heads of 64 leave room for two blocks an SM, which fill each other's waits; heads of 128
// for one.
//
// What bounds it: the states' warps, 16-bit arithmetic on the ALU pipe (13 operations for a pair of
// weighted values in three parts) and its waits; some 9000 cycles a chunk of 128 x 128, the rows' warps
// 6500.  5 ragged sequences of 8191 x 16 heads of 128: 186 us beside 120 for the stretches' states.
#include "linear_tc.cuh"

namespace fs {
namespace {

using namespace lin;

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
                       kLastRegs = D == 64 ? 40 : 64;
  static_assert(8 * kRowRegs + kStateWarps * kStateRegs + 4 * kLastRegs <= (12 + kStateWarps) * kRegs, "registers");
  static constexpr uint32_t kSlabAtom = kSlab * 128;
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
  uint64_t pairs[4];  // a chunk's rows of the second of two warps are in the values' place
  uint32_t tmem;
  int odd[2];                 // i + 1: the values of the block's chunk i are not all finite
  float power[kC + 4];        // lam^n
  Tables tables;
  int bad[2][128];            // per column, as bad_mark
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, D == 64 ? 2 : 1)
    k17_linear_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using C = Cfg<D>;
  using F = Frags<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Shared s;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const LinearSweep &w = p.a.sweep[blockIdx.z];
  const int b = blockIdx.y / p.a.H, h = blockIdx.y % p.a.H, r = blockIdx.x;
  const Band st(p, b);
  const bool reverse = w.reverse;
  // (a sequence without tokens has one block, for its state)
  if (r >= max(st.stretches, 1)) return;
  const int from = st.lo + r * st.per;
  const float decay = p.a.decay[h];

  if (threadIdx.x == 0) {
    for (uint64_t *x : {&s.qfull, &s.qempty, &s.kfull, &s.s_free, &s.scores, &s.inter, &s.done, &s.u_full, &s.fin})
      tc::mbar_init(x, 1);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&s.vfull[i], 1);
      tc::mbar_init(&s.vempty[i], 8);
    }
    tc::mbar_init(&s.slab_empty, 1);
    for (uint64_t *x : {&s.slab_full, &s.s_ready, &s.u_free, &s.checked[0], &s.checked[1]})
      tc::mbar_init(x, C::kStateWarps);
    for (uint64_t *x : {&s.parts, &s.o_free}) tc::mbar_init(x, 8);
    tc::mbar_init(&s.kempty, 2);  // read by the scores' product and by the slabs'
    tc::mbar_init(&s.fin_u, 1);
    for (uint64_t &x : s.pairs) tc::mbar_init(&x, 1);
    tc::mbar_fence_init();
    s.odd[0] = s.odd[1] = 0;
  }
  for (int i = threadIdx.x; i <= kC; i += C::kThreads) {
    const Factor f = decay_power(decay, i);
    s.power[i] = f.hi + f.lo;
  }
  fill_tables(s.tables, decay, reverse, p.a.scale, threadIdx.x, C::kThreads);
  for (int i = threadIdx.x; i < 256; i += C::kThreads) s.bad[i / 128][i % 128] = 0;
  if (warp == C::kMma) {
    tc::tmem_alloc(&s.tmem, C::kCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s.tmem, base = smem_u32(smem);
  const uint32_t tu = tmem + C::kU;
  const int chunks = max(st.end(r) - from, 0);
  if (warp >= C::kTma) {
    tc::regs_dec<C::kLastRegs>();
  if (warp == C::kTma && lane == 0) {
    // ------------------------------------------------------------------ loads
    const int mq = p.map[blockIdx.z][0], mk = p.map[blockIdx.z][1], mv = p.map[blockIdx.z][2];
    auto load = [&](uint32_t at, int m, const LinearRows &x, uint64_t *bar, int i) {
      const int t = st.chunk(from + i, reverse) * kC;
      tc::mbar_arrive_expect_tx(bar, C::kTile);
      for (int k = 0; k < C::kAtoms; ++k)
        load_rows(smem + at + k * kAtom, &maps.in[m], bar, 64 * k, t, h / x.share * p.axes[m][1],
                  b * p.axes[m][0]);
    };
    int nq = 0, nk = 0, nv = 0;  // loaded so far
    bool ok = true;
    auto load_q = [&]() {
      if (!ok || nq >= chunks) return;
      if (nq && !(ok = wait_for(&s.qempty, (nq - 1) & 1, p))) return;
      load(C::kQ, mq, w.q, &s.qfull, nq);
      ++nq;
    };
    auto load_k = [&]() {
      if (!ok || nk >= chunks) return;
      if (nk && !(ok = wait_for(&s.kempty, (nk - 1) & 1, p))) return;
      load(C::kK, mk, w.k, &s.kfull, nk);
      ++nk;
    };
    auto load_v = [&]() {
      const int at = nv % C::kValues;
      if (!ok || nv >= chunks) return;
      if (nv >= C::kValues && !(ok = wait_for(&s.vempty[at], (nv / C::kValues - 1) & 1, p))) return;
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
  } else if (warp == C::kMma && lane == 0) {
    // ----------------------------------------------------- products of the rows
    constexpr uint32_t kQK = tc::idesc_bf16(128, 128, 0), kB = tc::idesc_bf16(128, D, 1);
    const uint32_t keys = base + C::kK;
    for (int i = 0; i < chunks; ++i) {
      const uint32_t values = base + C::kV + i % C::kValues * C::kTile;
      if (!wait_for(&s.kfull, i & 1, p) || !wait_for(&s.qfull, i & 1, p)) break;
      tc::fence_after_sync();
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        tc::mma_ss(tmem + C::kScores, tc::desc_sw128(base + C::kQ + k / 4 * kAtom + k % 4 * 32),
                   tc::desc_sw128(keys + k / 4 * kAtom + k % 4 * 32), kQK, k > 0);
      tc::mma_commit(&s.scores);
      tc::mma_commit(&s.kempty);
      if (!wait_for(&s.s_ready, i & 1, p) ||
          (i && !wait_for(&s.o_free, (i - 1) & 1, p)))
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
      if (!wait_for(&s.parts, i & 1, p) || !wait_for(&s.checked[i & 1], i >> 1 & 1, p)) break;
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
      if (!wait_for(&s.kfull, i & 1, p)) break;
      if (i && !wait_for(&s.u_free, (i - 1) & 1, p)) break;
      for (int j = 0; j < C::kSlabs; ++j) {
        const int at = i * C::kSlabs + j;
        if (!(ok = wait_for(&s.slab_full, at & 1, p))) break;
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
    const int t = threadIdx.x - 256;
    const uint32_t lanes = tu + ((uint32_t)(warp % 4 * 32) << 16) + (D == 64 ? 0 : t / 128 * 64);
    const int sr = w.transposed ? 1 : D, sc = w.transposed ? D : 1;
    f2 S[F::kHalves][16];
    const size_t slot = (size_t)p.slot[blockIdx.z] * gridDim.y + blockIdx.y;
    const float *given = w.state ? w.state + (size_t)blockIdx.y * D * D : nullptr;
#pragma unroll
    for (int g = 0; g < F::kHalves; ++g)
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        if (st.stretches > 1) {
          const float *at = p.slots + (slot * p.splits + r) * (D * D);
          if ((int)blockIdx.z == p.borrows) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int row = F::row(t, g, e + k), col = F::col(t, e + k);
              S[g][e + k] = f2_bits(at[F::index(col, row)], at[F::index(col + 1, row)]);
            }
          } else {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(at + F::at(t, g, e));
            S[g][e] = x.x, S[g][e + 1] = x.y;
          }
        } else if (given) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float *at = given + F::row(t, g, e + k) * sr + F::col(t, e + k) * sc;
            S[g][e + k] = f2_bits(at[0] * w.state_mul, at[sc] * w.state_mul);
          }
        } else {
          S[g][e] = S[g][e + 1] = 0;
        }
      }
    const Publisher<D> publisher(base + C::kS, t);
    auto publish = [&]() {
#pragma unroll
      for (int g = 0; g < F::kHalves; ++g)
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const f2 x[4] = {S[g][e], S[g][e + 1], S[g][e + 2], S[g][e + 3]};
          publisher.put(g, e, x);
        }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&s.s_ready);
    };
    if (chunks) publish();
    const Factor whole = decay_power(decay, kC);
    // this thread's sixteen bytes of a slab's row r16 (and r16 + 16)
    const int r16 = t % 128 / 8, ch = t % 8, atom = t / 128;
    const uint32_t in = swz128(r16, ch);
    unsigned char *slab = smem + C::kSlab0 + atom * C::kSlabAtom + in;
    for (int i = 0; i < chunks; ++i) {
      const int n = st.size(st.chunk(from + i, reverse));
      unsigned char *source = smem + C::kV + i % C::kValues * C::kTile + atom * kAtom + in;
      if (!WAIT(s.vfull[i % C::kValues], i / C::kValues)) break;
      if (n < kC) {
        // what lies behind the sequence takes no part, whatever it is
        if (!WAIT(s.kfull, i)) break;
        unsigned char *keys = smem + C::kK;
        for (int u = t; u < (kC - n) * (D / 8); u += F::kThreads)
          *reinterpret_cast<uint4 *>(keys + u % (D / 8) / 8 * kAtom + swz128(n + u / (D / 8), u % 8)) =
              make_uint4(0, 0, 0, 0);
        // values: those that this thread reads itself (the fence before the first slab's arrival is
        // for all of them)
#pragma unroll 1
        for (int row = r16; row < kC; row += 16)
          if (row >= n) *reinterpret_cast<uint4 *>(source + (row - r16) * 128) = make_uint4(0, 0, 0, 0);
      }
      uint32_t some = 0;  // the bits of all third parts
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < C::kSlabs; ++j) {
        uint32_t part[C::kUnits][3][4];
#pragma unroll
        for (int k = 0; k < C::kUnits; ++k) {
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
        for (int k = 0; k < C::kUnits; ++k)
#pragma unroll
          for (int q = 0; q < 3; ++q)
            *reinterpret_cast<uint4 *>(slab + q * C::kPart + k * 2048) =
                make_uint4(part[k][q][0], part[k][q][1], part[k][q][2], part[k][q][3]);
        // A value that is not finite leaves NaN in the third part (and NaN in the state's column).
        // It leaves V before the scores' product, where scores of 0 would make NaN of the rows
        // before it as well; those after it get theirs at the end.
        if (j + 1 == C::kSlabs &&
            ((some & 0x7f80u) == 0x7f80u || (some & 0x7f800000u) == 0x7f800000u)) {
          for (int u = 0; u < kC / 16; ++u) {
            const int row = 16 * u + r16;
            if (row >= n) break;
            uint32_t *word = reinterpret_cast<uint32_t *>(source + u * 2048);
            for (int c = 0; c < 8; ++c) {
              if ((word[c / 2] >> c % 2 * 16 & 0x7f80u) != 0x7f80u) continue;
              word[c / 2] &= c % 2 ? 0xffffu : 0xffff0000u;
              atomicMax(&s.bad[i & 1][atom * 64 + ch * 8 + c], bad_mark(i, reverse ? kC - 1 - row : row));
              s.odd[i & 1] = i + 1;
            }
          }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&s.slab_full);
      }
      if (!ok) break;
      if (lane == 0) tc::mbar_arrive(&s.checked[i & 1]);
      if (!WAIT(s.u_full, i)) break;
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
      if (i + 1 < chunks) {
        if (!WAIT(s.s_free, i)) break;
        publish();
      }
    }
    if (r == max(st.stretches, 1) - 1 && w.state_out) {
      float *out = w.state_out + (size_t)blockIdx.y * D * D;
      const float mul = 1.f / w.state_mul;
#pragma unroll
      for (int g = 0; g < F::kHalves; ++g)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float *at = out + F::row(t, g, e) * sr + F::col(t, e) * sc;
          at[0] = lo2(S[g][e]) * mul;
          at[sc] = hi2(S[g][e]) * mul;
        }
    }
  } else {
    if constexpr (C::kRowRegs < C::kRegs) tc::regs_dec<C::kRowRegs>();
    // -------------------------------------------------------------------- rows
    const RowWarp<D> rows(warp, lane, tmem + C::kScores, tmem + C::kOut);
    bool storing = false;  // (lane 0) a store may still read the values' place
    for (int i = 0; i < chunks; ++i) {
      const int chunk = st.chunk(from + i, reverse), n = st.size(chunk);
      if (!WAIT(s.scores, i)) break;
      tc::fence_after_sync();
      rows.parts(s.tables, reverse, n);
      if (i && lane == 0) {  // the last chunk's rows are on their way
        if (storing) bulk_wait_read<0>();
        tc::mbar_arrive(&s.vempty[(i - 1) & 1]);
      }
      __syncwarp();
      if (!WAIT(s.inter, i)) break;
      tc::fence_after_sync();
      rows.weigh(s.tables, reverse, n);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&s.parts);
      if (!WAIT(s.checked[i & 1], i >> 1) || !WAIT(s.done, i)) break;
      tc::fence_after_sync();
      storing = rows.store(w, &maps.out[blockIdx.z], p.out_axes[blockIdx.z], b, h, chunk, n, i, reverse,
                           s.odd[i & 1] == i + 1 ? s.bad[i & 1] : nullptr, smem + C::kV + (i & 1) * C::kTile,
                           &s.o_free, s.pairs, p);
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


template <int D>
cudaError_t run(const Params &p, const Maps &maps, cudaStream_t st) {
  constexpr int kSmem = Cfg<D>::kBytes + 1024;
  auto f = k17_linear_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  f<<<dim3(p.splits, p.a.batch * p.a.H, p.a.sweeps), Cfg<D>::kThreads, kSmem, st>>>(maps, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t lin::launch_fused(const Params &p, const Maps &maps, cudaStream_t st) {
  return p.a.d == 64 ? run<64>(p, maps, st) : run<128>(p, maps, st);
}

}  // namespace fs
