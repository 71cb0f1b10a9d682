// k15_norm.cu -- the norms after and before a block, with the block's gate and
// residual scale, and their gradients.
//
//   h = x r_g (r_g = 1 / sqrt(mean of x^2 over its group + eps); or h = x)
//   a = h gain silu(gate),   z = residual + scale a
//   y = z r next_gain,       r = 1 / sqrt(mean z^2 + eps)
//
// and with g = dz + r (w - z r^2 mean(w z)), w = dy next_gain, for the gradient
// that reaches z (mean over the row):
//   dresidual = g,   dnext_gain = sum over rows of dy z r
//   dgate = scale g h gain silu'(gate),   dgain = sum over rows of scale g silu(gate) h
//   dx = r_g (u - h mean_group(u h)),     u = scale g silu(gate) gain
//
// Every tensor is read or written once.  Memory bounds the forward pass: 65536 x 16 gated heads
// of 64 in bf16 67 us, 6.0 TB/s; 16384 x 8192 with an fp32 residual and the next norm 259 us, 6.2 TB/s.
// The backward pass is bound by its instructions (16384 x 16 gated heads 46 us, two thirds of
// all issue slots) and by its sums over a row, one after the other (8191 x 2500 in fp32 135 us,
// 4.9 TB/s).  A team of threads takes a
// row.  In the backward pass it takes one after another, each thread its own vectors, and the
// next row is under way into shared memory (asynchronous copies that nobody else waits
// for) while it works on this one: 16384 x 1024 gated heads in bf16 42 us instead of 65.  Of what
// is read to the row's end (x and the gate) there are always two rows, of the rest too (kTwice) or one,
// fetched anew once it has been read: less shared memory and fewer registers for one more block
// on the SM.  Rows too wide for that, and rows off sixteen bytes, are read where they lie.
// (The forward pass gained nothing from it: 77 us against 71, and 464 against 272 where rows are
// wide and one block had an SM to itself.)
// A thread has read an element of an input for the last time before it writes the
// output that may take its place.  Sums are fp32 in a fixed order.  The
// gradients of the gains are sums over rows: a thread keeps those of its columns over all
// rows that it takes, blocks put theirs into the workspace and a second kernel adds them
// in block order.
#include "fs_common.cuh"
#include "fs_internal.h"
#include "pairs.cuh"

namespace fs {
namespace {

// How a row's groups are added up.
enum Groups { kNone, kRow, kShuffle, kList };

__device__ __forceinline__ f2 both(float x) { return f2_bits(x, x); }

// V elements of a row as they are in memory: sixteen bytes of TX, as many elements of TR.
template <typename T, int V>
struct Raw {
  static constexpr int kPieces = V * sizeof(T) / 16;
  uint4 u[kPieces];
  __device__ __forceinline__ f2 get(int c) const {
    if constexpr (sizeof(T) == 2) {
      return wide2(c == 0 ? u[0].x : c == 1 ? u[0].y : c == 2 ? u[0].z : u[0].w);
    } else {
      const uint4 &w = u[c / 2];
      return c % 2 ? (f2)w.z | (f2)w.w << 32 : (f2)w.x | (f2)w.y << 32;
    }
  }
};

// V elements at p, of which the row has `left` more (kWhole: all or none).  `wide`: eight fp32
// elements lie on 32 bytes and go as one (as two of sixteen bytes each, a warp would touch every
// sector twice).
template <bool kWhole, typename T, int V>
__device__ __forceinline__ Raw<T, V> load(const T *p, int left, bool wide) {
  Raw<T, V> r;
  if constexpr (kWhole) {
#pragma unroll
    for (int i = 0; i < Raw<T, V>::kPieces; ++i) r.u[i] = make_uint4(0, 0, 0, 0);
    if (left > 0) {
      if constexpr (Raw<T, V>::kPieces == 2) {
        if (wide) {
          asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                       : "=r"(r.u[0].x), "=r"(r.u[0].y), "=r"(r.u[0].z), "=r"(r.u[0].w), "=r"(r.u[1].x),
                         "=r"(r.u[1].y), "=r"(r.u[1].z), "=r"(r.u[1].w)
                       : "l"(p)
                       : "memory");
          return r;
        }
      }
#pragma unroll
      for (int i = 0; i < Raw<T, V>::kPieces; ++i) r.u[i] = *(reinterpret_cast<const uint4 *>(p) + i);
    }
  } else {
    uint32_t w[4 * Raw<T, V>::kPieces];
#pragma unroll
    for (int c = 0; c < V / 2; ++c) {
      const float x = 2 * c < left ? static_cast<float>(p[2 * c]) : 0.f;
      const float y = 2 * c + 1 < left ? static_cast<float>(p[2 * c + 1]) : 0.f;
      if constexpr (sizeof(T) == 2) {
        w[c] = pack_bf16(x, y);  // (bf16 numbers: nothing is rounded)
      } else {
        w[2 * c] = __float_as_uint(x);
        w[2 * c + 1] = __float_as_uint(y);
      }
    }
#pragma unroll
    for (int i = 0; i < Raw<T, V>::kPieces; ++i)
      r.u[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  return r;
}
template <bool kWhole, typename T, int V>
__device__ __forceinline__ void store(T *p, int left, const f2 (&x)[V / 2], bool wide) {
  if constexpr (kWhole) {
    if (left <= 0) return;
    if constexpr (sizeof(T) == 4 && V == 8) {
      if (wide) {
        asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(x[0]), "l"(x[1]), "l"(x[2]), "l"(x[3])
                     : "memory");
        return;
      }
    }
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3]));
    } else {
#pragma unroll
      for (int c = 0; c < V / 2; c += 2)
        *reinterpret_cast<ulonglong2 *>(p + 2 * c) = make_ulonglong2(x[c], x[c + 1]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < V / 2; ++c) {
      if (2 * c < left) p[2 * c] = static_cast<T>(lo2(x[c]));
      if (2 * c + 1 < left) p[2 * c + 1] = static_cast<T>(hi2(x[c]));
    }
  }
}

// A thread's vectors of one tensor's rows.  kStaged: one or two of them in shared memory, piece
// after piece, threads side by side.
template <bool kStaged, bool kWhole, typename T, int V, int N>
struct Slot {
  enum { kPieces = Raw<T, V>::kPieces };
  uint32_t at;    // (shared memory) this thread's first piece of stage 0, 0 without the tensor
  uint32_t stage; // bytes from a stage to the next
  const T *row;   // the next row to fetch (not kStaged: to read), at this thread's first element
  long long step; // elements to the team's row after it
  __device__ __forceinline__ void init(uint32_t &free, int stages, const void *p, long long stride, long long first,
                                       int rows, int e0) {
    at = stage = 0;
    if constexpr (kStaged) {
      stage = N * kPieces * blockDim.x * 16;
      if (p) at = free + threadIdx.x * 16, free += stages * stage;
    }
    row = static_cast<const T *>(p) + first * stride + e0;
    step = rows * stride;
  }
  // `left` elements from the thread's first on, 0 without a row; `apart` elements from vector to vector.
  __device__ __forceinline__ void fetch(int which, int left, int apart) {
    if constexpr (kStaged) {
      if (!at) return;
      const uint32_t to = at + which * stage;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const bool have = left - i * apart > 0;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
          const uint32_t piece = to + (i * kPieces + k) * blockDim.x * 16;
          if (have)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(piece),
                         "l"(reinterpret_cast<const uint4 *>(row + i * apart) + k));
          else
            put(piece, make_uint4(0, 0, 0, 0));
        }
      }
      row += step;
    }
  }
  // A row that stays: the gains'.
  __device__ __forceinline__ void fill(int left, int apart) {
    if (!at) return;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const Raw<T, V> r = load<kWhole, T, V>(row + i * apart, left - i * apart, false);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) put(at + (i * kPieces + k) * blockDim.x * 16, r.u[k]);
    }
  }
  static __device__ __forceinline__ void put(uint32_t at, const uint4 &x) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w)
                 : "memory");
  }
  __device__ __forceinline__ void next() {
    if constexpr (!kStaged) row += step;
  }
  __device__ __forceinline__ Raw<T, V> get(int which, int i, int left, int apart) const {
    if constexpr (kStaged) {
      Raw<T, V> r;
#pragma unroll
      for (int k = 0; k < kPieces; ++k)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                     : "=r"(r.u[k].x), "=r"(r.u[k].y), "=r"(r.u[k].z), "=r"(r.u[k].w)
                     : "r"(at + which * stage + (i * kPieces + k) * blockDim.x * 16)
                     : "memory");
      return r;
    } else {
      return load<kWhole, T, V>(row + i * apart, left - i * apart, false);
    }
  }
};

// 1 / (1 + e^-x) by the special-function unit.
// kExact, where the residual stream and so z and its gradient are fp32: by e^-|x|, which is in (0, 1] for
// any x and keeps what lies below fp32's normal range; with the exponent's rounding put back and a Newton step
// on the reciprocal, 2^-22 of itself.
// Else: 2^-21, and |x| 2^-23 for the argument's rounding, which half a step of a bf16 result, 2^-8, hides; the
// gains' gradients are sums of such terms.  (65536 x 16 gated heads of 64 in bf16 67.6 us, with kExact 78.1;
// the gradients of 16384 x 16 47.1 and 53.3.)
template <bool kExact>
__device__ __forceinline__ float sigmoid(float x) {
  constexpr float kL = -1.44269504f, kRest = -1.92596303e-8f;  // -log2 e, what it lacks
  float e, r;
  if constexpr (kExact) {
    const float a = fabsf(x), t = a * kL;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
    if (t > -150.f) e = fmaf(e, (fmaf(a, kL, -t) + a * kRest) * 0.693147181f, e);  // (else e is 0, t may be infinite)
    const float d = 1.f + e;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    r = fmaf(r, fmaf(-d, r, 1.f), r);
    return x < 0.f ? e * r : r;
  } else {
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * kL));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
  }
}
template <bool kExact>
__device__ __forceinline__ f2 sigmoid2(f2 x) {
  return f2_bits(sigmoid<kExact>(lo2(x)), sigmoid<kExact>(hi2(x)));
}

// A number for each group, beside the elements of a vector: one for all where vectors are whole.
template <bool kWhole, int V>
struct PerGroup {
  f2 x[kWhole ? 1 : V / 2];
  __device__ __forceinline__ f2 get(int c) const { return x[kWhole ? 0 : c]; }
};

// A team's way to add: the block's threads (kTeam 0), or kTeam = 8 or 32 of a block of
// 256.  N vectors of V elements each: vector i of thread t is number t + i size of the row.
template <int kTeam, int V, int N, bool kWhole>
struct Team {
  static constexpr int kLanes = kTeam ? kTeam : 32;
  int t, team, size;  // thread within the team, team within the block, threads of a team
  float *scratch;     // two halves of the block's warps, in turn
  float *list;        // sums of vectors (elements), then of groups
  int turn;

  __device__ __forceinline__ void sync() const {
    if constexpr (kTeam)
      __syncwarp();
    else
      __syncthreads();
  }
  // K <= 2 sums over the team, the same in every thread.
  template <int K>
  __device__ __forceinline__ void add(float (&x)[K]) {
#pragma unroll
    for (int m = 1; m < kLanes; m *= 2)
#pragma unroll
      for (int k = 0; k < K; ++k) x[k] += __shfl_xor_sync(0xffffffffu, x[k], m);
    if (kTeam || size == 32) return;
    const int warps = size / 32, lane = t % 32;
    float *to = scratch + (turn ^= 1) * 2 * 16;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) to[k * 16 + t / 32] = x[k];
    sync();
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = lane < warps ? to[k * 16 + lane] : 0.f;  // at most sixteen
#pragma unroll
    for (int m = 8; m > 0; m /= 2)
#pragma unroll
      for (int k = 0; k < K; ++k) x[k] += __shfl_xor_sync(0xffffffffu, x[k], m);
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = __shfl_sync(0xffffffffu, x[k], 0);
  }
  // Sums over groups of the products f(i, c) (pair c of vector i).  Groups of a power of two
  // of whole vectors, up to a warp's: by shuffles.  Others through `list`: a group to a
  // warp (or small team) at a time.
  template <typename F>
  __device__ __forceinline__ void add_groups(PerGroup<kWhole, V> (&p)[N], const NormArgs &a, F f) {
    const int mode = a.mode;
    const int n = kWhole ? a.D / V : a.D;
    if (mode == kList) sync();  // (the list is free: its readers are past this)
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      f2 s = 0;
#pragma unroll
      for (int c = 0; c < V / 2; ++c) {
        const f2 x = f(i, c);
        s = c ? add2_bits(s, x) : x;
        if constexpr (!kWhole) {
          const int e = (t + i * size) * V + 2 * c;
          if (mode == kList && e < n) list[e] = lo2(x);
          if (mode == kList && e + 1 < n) list[e + 1] = hi2(x);
        }
      }
      v[i] = lo2(s) + hi2(s);
    }
    if (mode == kRow) {
      float s[1] = {v[0]};
#pragma unroll
      for (int i = 1; i < N; ++i) s[0] += v[i];
      add(s);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = s[0];
    } else if (mode == kShuffle) {
      for (int m = 1; m < a.per; m *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
    } else {
      if constexpr (kWhole) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (t + i * size < n) list[t + i * size] = v[i];
      }
      sync();
      for (int g = t / kLanes; g < a.groups; g += size / kLanes) {
        float s = 0.f;
        for (int j = t % kLanes; j < a.per; j += kLanes) s += list[g * a.per + j];
#pragma unroll
        for (int m = 1; m < kLanes; m *= 2) s += __shfl_xor_sync(0xffffffffu, s, m);
        if (t % kLanes == 0) list[n + g] = s;
      }
      sync();
      if constexpr (kWhole) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (t + i * size < n) v[i] = list[n + (t + i * size) / a.per];
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int c = 0; c < V / 2; ++c) {
            const int e = (t + i * size) * V + 2 * c;
            p[i].x[c] = f2_bits(e < n ? list[n + e / a.per] : 0.f, e + 1 < n ? list[n + (e + 1) / a.per] : 0.f);
          }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int c = 0; c < (kWhole ? 1 : V / 2); ++c) p[i].x[c] = both(v[i]);
  }
  // The factors that normalise x's groups (ones where they are not to be); x(i): vector i.  The row has `left`
  // elements from the thread's first on, 0 without a row.
  template <typename F>
  __device__ __forceinline__ void factors(PerGroup<kWhole, V> (&inv)[N], const NormArgs &a, int left, F x) {
    if (a.mode == kNone) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < (kWhole ? 1 : V / 2); ++c) inv[i].x[c] = both(1.f);
      return;
    }
    add_groups(inv, a, [&](int i, int c) {
      const f2 y = x(i).get(c);
      return mul2(y, y);
    });
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int c = 0; c < (kWhole ? 1 : V / 2); ++c) {
        // (past the row, and in a team without one, 0: with eps 0 the factor there would be infinite)
        const int e = i * size * V + 2 * c;
        const float f = e < left ? rsqrtf(fmaf(lo2(inv[i].x[c]), a.inv_n, a.eps)) : 0.f;
        const float g = kWhole ? f : e + 1 < left ? rsqrtf(fmaf(hi2(inv[i].x[c]), a.inv_n, a.eps)) : 0.f;
        inv[i].x[c] = f2_bits(f, g);
      }
  }
};

// Blocks of up to 512 threads, two or more to an SM; small teams share blocks of 256.  A team takes
// one row, all of whose loads are issued before anything else; other blocks' rows fill its waits.
template <typename TX, typename TR, int kTeam, int N, bool kWhole>
__global__ void __launch_bounds__(kTeam ? 256 : 512, sizeof(TX) == 4 || N * 8 > 16 ? 1 : 2)
    k15_norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int V = 16 / sizeof(TX);
  extern __shared__ uint4 slots[];
  __shared__ float scratch[64];
  Team<kTeam, V, N, kWhole> team;
  team.size = kTeam ? kTeam : blockDim.x;
  team.t = kTeam ? threadIdx.x % kTeam : threadIdx.x;
  team.team = kTeam ? threadIdx.x / kTeam : 0;
  team.scratch = scratch;
  team.list = reinterpret_cast<float *>(slots) + team.team * a.list;
  team.turn = 0;
  const int e0 = team.t * V, apart = team.size * V;
  // (a team without a row, in a block with one, keeps its warp company on zeros)
  const long long row = (long long)blockIdx.x * (kTeam ? 256 / kTeam : 1) + team.team;
  const int left = row < a.M ? a.D - e0 : 0;

  Raw<TX, V> x[N], gate[N];
  Raw<TR, V> res[N];
  const TX *xr = static_cast<const TX *>(a.x) + row * a.xs + e0;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = load<kWhole, TX, V>(xr + i * apart, left - i * apart, a.wide);
  if (a.gate) {
    const TX *gr = static_cast<const TX *>(a.gate) + row * a.gs + e0;
#pragma unroll
    for (int i = 0; i < N; ++i) gate[i] = load<kWhole, TX, V>(gr + i * apart, left - i * apart, a.wide);
  }
  if (a.residual) {
    const TR *rr = static_cast<const TR *>(a.residual) + row * a.rs + e0;
#pragma unroll
    for (int i = 0; i < N; ++i) res[i] = load<kWhole, TR, V>(rr + i * apart, left - i * apart, a.wide);
  }
  const f2 scale = both(a.scale);
  PerGroup<kWhole, V> inv[N];
  team.factors(inv, a, left, [&](int i) { return x[i]; });
  f2 z[N][V / 2], ss = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(x[i].get(c), inv[i].get(c));
    if (a.gain) {
      const Raw<float, V> g = load<kWhole, float, V>(a.gain + e0 + i * apart, a.D - e0 - i * apart, a.wide);
#pragma unroll
      for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(z[i][c], g.get(c));
    }
    if (a.gate) {
#pragma unroll
      for (int c = 0; c < V / 2; ++c) {
        const f2 g = gate[i].get(c);
        z[i][c] = mul2(z[i][c], mul2(g, sigmoid2<sizeof(TR) == 4>(g)));
      }
    }
    if (a.residual) {
#pragma unroll
      for (int c = 0; c < V / 2; ++c) z[i][c] = madd2(scale, z[i][c], res[i].get(c));
    } else {
#pragma unroll
      for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(scale, z[i][c]);
    }
  }
  if (a.z) {
    TR *zr = static_cast<TR *>(a.z) + row * a.zs + e0;
#pragma unroll
    for (int i = 0; i < N; ++i) store<kWhole, TR, V>(zr + i * apart, left - i * apart, z[i], a.wide);
  }
  f2 f = 0;
  if (a.next) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int c = 0; c < V / 2; ++c) ss = madd2(z[i][c], z[i][c], ss);
    float s[1] = {lo2(ss) + hi2(ss)};
    team.add(s);
    f = both(rsqrtf(fmaf(s[0], a.inv_D, a.eps)));
  }
  if (!a.next) return;
  TX *yr = static_cast<TX *>(a.y) + row * a.ys + e0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(z[i][c], f);
    if (a.next_gain) {
      const Raw<float, V> g = load<kWhole, float, V>(a.next_gain + e0 + i * apart, a.D - e0 - i * apart, a.wide);
#pragma unroll
      for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(z[i][c], g.get(c));
    }
    store<kWhole, TX, V>(yr + i * apart, left - i * apart, z[i], a.wide);
  }
}

template <typename TX, typename TR, int kTeam, int N, bool kWhole, bool kStaged, bool kTwice>
__global__ void __maxnreg__(!kTwice ? 96 : kTeam ? 255 : 128) k15_norm_bwd_kernel(const __grid_constant__ NormArgs a) {
  constexpr int V = 16 / sizeof(TX);
  constexpr bool kExact = sizeof(TR) == 4;
  extern __shared__ uint4 slots[];
  __shared__ float scratch[64];
  Team<kTeam, V, N, kWhole> team;
  team.size = kTeam ? kTeam : blockDim.x;
  team.t = kTeam ? threadIdx.x % kTeam : threadIdx.x;
  team.team = kTeam ? threadIdx.x / kTeam : 0;
  team.scratch = scratch;
  team.turn = 0;
  const int teams = kTeam ? 256 / kTeam : 1, rows = gridDim.x * teams;
  const int e0 = team.t * V, apart = team.size * V;
  long long row = (long long)blockIdx.x * teams + team.team;
  uint32_t free = smem_u32(slots);
  Slot<kStaged, kWhole, TX, V, N> x, gate, dy;
  Slot<kStaged, kWhole, TR, V, N> dz, res;
  Slot<kStaged, kWhole, float, V, N> gain, next;
  constexpr int stages = kTwice ? 2 : 1;
  x.init(free, 2, a.x, a.xs, row, rows, e0);
  gate.init(free, 2, a.gate, a.gs, row, rows, e0);
  dz.init(free, stages, a.dz, a.dzs, row, rows, e0);
  dy.init(free, stages, a.dy, a.dys, row, rows, e0);
  res.init(free, stages, a.next ? a.residual : nullptr, a.rs, row, rows, e0);
  gain.init(free, 1, a.gain, 0, 0, 0, e0);
  next.init(free, 1, a.next_gain, 0, 0, 0, e0);
  if constexpr (kStaged) gain.fill(a.D - e0, apart), next.fill(a.D - e0, apart);
  team.list = reinterpret_cast<float *>(slots) + (free - smem_u32(slots)) / 4 + team.team * a.list;
  TX *dxr = static_cast<TX *>(a.dx) + row * a.dxs + e0, *dgr = static_cast<TX *>(a.dgate) + row * a.dgs + e0;
  TR *drr = static_cast<TR *>(a.dres) + row * a.drs + e0;
  auto fetch = [&](int which, bool have) {
    const int left = have ? a.D - e0 : 0;
    x.fetch(which, left, apart);
    gate.fetch(which, left, apart);
  };
  auto fetch_rest = [&](int which, bool have) {
    const int left = have ? a.D - e0 : 0;
    dz.fetch(which, left, apart);
    dy.fetch(which, left, apart);
    res.fetch(which, left, apart);
  };
  if constexpr (kStaged) {
    fetch(0, row < a.M);
    fetch_rest(0, row < a.M);
    cp_async_commit();
  }
  f2 dgain[N][V / 2] = {}, dnext[N][V / 2] = {};  // (zeros and factors of 0, of a team without a row, add nothing)
  const f2 scale = both(a.scale);
  int which = 0;
  for (; row - team.team < a.M; row += rows, which ^= 1) {
    if constexpr (kStaged) {
      fetch(which ^ 1, row + rows < a.M);
      if constexpr (kTwice) fetch_rest(which ^ 1, row + rows < a.M);
      cp_async_commit();
      cp_async_wait<1>();
    }
    const int left = row < a.M ? a.D - e0 : 0, rest = kTwice ? which : 0;
    PerGroup<kWhole, V> inv[N];
    team.factors(inv, a, left, [&](int i) { return x.get(which, i, left, apart); });
    f2 sig[N][V / 2], g[N][V / 2];  // g: the gradient that reaches z
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (a.gate) {
        const Raw<TX, V> gv = gate.get(which, i, left, apart);
#pragma unroll
        for (int c = 0; c < V / 2; ++c) sig[i][c] = sigmoid2<kExact>(gv.get(c));
      }
      if (a.dz) {
        const Raw<TR, V> dv = dz.get(rest, i, left, apart);
#pragma unroll
        for (int c = 0; c < V / 2; ++c) g[i][c] = dv.get(c);
      } else {
#pragma unroll
        for (int c = 0; c < V / 2; ++c) g[i][c] = 0;
      }
    }
    if (a.next) {
      f2 z[N][V / 2], s0 = 0, s1 = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const Raw<TX, V> xv = x.get(which, i, left, apart);
#pragma unroll
        for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(xv.get(c), inv[i].get(c));
        if (a.gain) {
          const Raw<float, V> gv = gain.get(0, i, a.D - e0, apart);
#pragma unroll
          for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(z[i][c], gv.get(c));
        }
        if (a.gate) {
          const Raw<TX, V> gv = gate.get(which, i, left, apart);
#pragma unroll
          for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(z[i][c], mul2(gv.get(c), sig[i][c]));
        }
        if (a.residual) {
          const Raw<TR, V> rv = res.get(rest, i, left, apart);
#pragma unroll
          for (int c = 0; c < V / 2; ++c) z[i][c] = madd2(scale, z[i][c], rv.get(c));
        } else {
#pragma unroll
          for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(scale, z[i][c]);
        }
        const Raw<TX, V> dv = dy.get(rest, i, left, apart);
        if (a.next_gain) {
          const Raw<float, V> nv = next.get(0, i, a.D - e0, apart);
#pragma unroll
          for (int c = 0; c < V / 2; ++c) s1 = madd2(z[i][c], mul2(dv.get(c), nv.get(c)), s1);
        } else {
#pragma unroll
          for (int c = 0; c < V / 2; ++c) s1 = madd2(z[i][c], dv.get(c), s1);
        }
#pragma unroll
        for (int c = 0; c < V / 2; ++c) s0 = madd2(z[i][c], z[i][c], s0);
      }
      float s[2] = {lo2(s0) + hi2(s0), lo2(s1) + hi2(s1)};
      team.add(s);
      const float r = left > 0 ? rsqrtf(fmaf(s[0], a.inv_D, a.eps)) : 0.f;
      const f2 rf = both(r), mc = both(-r * r * s[1] * a.inv_D);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const Raw<TX, V> dv = dy.get(rest, i, left, apart);
        f2 w[V / 2];
#pragma unroll
        for (int c = 0; c < V / 2; ++c) {
          w[c] = dv.get(c);
          dnext[i][c] = madd2(mul2(w[c], rf), z[i][c], dnext[i][c]);
        }
        if (a.next_gain) {
          const Raw<float, V> nv = next.get(0, i, a.D - e0, apart);
#pragma unroll
          for (int c = 0; c < V / 2; ++c) w[c] = mul2(w[c], nv.get(c));
        }
#pragma unroll
        for (int c = 0; c < V / 2; ++c) g[i][c] = madd2(rf, madd2(mc, z[i][c], w[c]), g[i][c]);
      }
    }
    if constexpr (kStaged && !kTwice) {  // (these have been read)
      fetch_rest(0, row + rows < a.M);
      cp_async_commit();
    }
    if (a.dres) {
#pragma unroll
      for (int i = 0; i < N; ++i) store<kWhole, TR, V>(drr + i * apart, left - i * apart, g[i], a.wide);
      drr += rows * a.drs;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const Raw<TX, V> xv = x.get(which, i, left, apart);
      Raw<float, V> gn;
      if (a.gain) gn = gain.get(0, i, a.D - e0, apart);
#pragma unroll
      for (int c = 0; c < V / 2; ++c) g[i][c] = mul2(scale, g[i][c]);
      if (a.gate) {
        const Raw<TX, V> gv = gate.get(which, i, left, apart);
        f2 out[V / 2];
#pragma unroll
        for (int c = 0; c < V / 2; ++c) {
          f2 d = mul2(g[i][c], mul2(xv.get(c), inv[i].get(c)));
          if (a.gain) d = mul2(d, gn.get(c));
          const f2 sg = sig[i][c], silu = mul2(gv.get(c), sg);
          // silu' = sig + silu (1 - sig), the bracket first: past 17, where sig is 1, it is 0 whatever the gate
          out[c] = mul2(d, madd2(silu, sub2_bits(both(1.f), sg), sg));
          g[i][c] = mul2(g[i][c], silu);
        }
        if (a.dgate) store<kWhole, TX, V>(dgr + i * apart, left - i * apart, out, a.wide);
      }
#pragma unroll
      for (int c = 0; c < V / 2; ++c) {
        dgain[i][c] = madd2(g[i][c], mul2(xv.get(c), inv[i].get(c)), dgain[i][c]);
        if (a.gain) g[i][c] = mul2(g[i][c], gn.get(c));
      }
    }
    dgr += rows * a.dgs;
    if (a.mode != kNone) {
      PerGroup<kWhole, V> p[N];
      team.add_groups(p, a, [&](int i, int c) {
        return mul2(g[i][c], mul2(x.get(which, i, left, apart).get(c), inv[i].get(c)));
      });
      const f2 mn = both(-a.inv_n);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const Raw<TX, V> xv = x.get(which, i, left, apart);
#pragma unroll
        for (int c = 0; c < V / 2; ++c) {
          const f2 h = mul2(xv.get(c), inv[i].get(c));
          g[i][c] = mul2(inv[i].get(c), madd2(mul2(mn, p[i].get(c)), h, g[i][c]));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) store<kWhole, TX, V>(dxr + i * apart, left - i * apart, g[i], a.wide);
    dxr += rows * a.dxs;
    x.next(), gate.next(), dz.next(), dy.next(), res.next();
  }
  cp_async_wait<0>();

  // the block's gains: its teams' added in their order
  float *total = reinterpret_cast<float *>(slots);  // (no team is in a row any more once all are here)
#pragma unroll 1
  for (int k2 = 0; k2 < 2; ++k2) {
    if (!(k2 ? a.dnext : a.dgain)) continue;
    float *to = a.ws + ((size_t)(k2 && a.dgain ? gridDim.x : 0) + blockIdx.x) * a.D;
    for (int k = 0; k < teams; ++k) {
      if (teams > 1) __syncthreads();
      if (team.team != k) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int e = e0 + i * apart + j;
          if (e >= a.D) continue;
          const f2 pair = k2 ? dnext[i][j / 2] : dgain[i][j / 2];
          const float v = (k ? total[e] : 0.f) + (j % 2 ? hi2(pair) : lo2(pair));
          if (k + 1 < teams)
            total[e] = v;
          else
            to[e] = v;
        }
      }
    }
  }
}

// Column sums of the blocks' parts, in order: 32 columns a block, 32 runs of parts, each with
// what its additions lose carried beside it (in fp64, whose unit here adds two numbers a cycle,
// the sums took 16 us).
__global__ void __launch_bounds__(1024) k15_gain_kernel(const float *part, int blocks, int D,
                                                        float *first, float *second) {
  __shared__ float run[2][32][33];
  const int lane = threadIdx.x % 32, k = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  const float *p = part + (size_t)blockIdx.y * blocks * D + c;
  float x = 0.f, lost = 0.f;
  auto add = [&](float y) {
    const float s = x + y, z = s - x;
    lost += (x - (s - z)) + (y - z);
    x = s;
  };
  if (c < D) {
    constexpr int kAhead = 10;
    for (int i = k; i < blocks; i += 32 * kAhead) {
      float y[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) y[j] = i + 32 * j < blocks ? __ldg(p + (size_t)(i + 32 * j) * D) : 0.f;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) add(y[j]);
    }
  }
  run[0][k][lane] = x;
  run[1][k][lane] = lost;
  __syncthreads();
  // a warp to each column
  x = run[0][lane][k];
  lost = run[1][lane][k];
#pragma unroll
  for (int m = 16; m > 0; m /= 2) {
    const float y = __shfl_xor_sync(0xffffffffu, x, m), l = __shfl_xor_sync(0xffffffffu, lost, m);
    const float big = fmaxf(fabsf(x), fabsf(y)) == fabsf(x) ? x : y, small = big == x ? y : x;
    const float s = x + y;
    lost += l + (small - (s - big));
    x = s;
  }
  const int to = blockIdx.x * 32 + k;
  // (of a sum that is not finite nothing is lost: the difference of infinities would be NaN)
  if (lane == 0 && to < D) (blockIdx.y ? second : first)[to] = fabsf(x) <= 0x1.fffffep127f ? x + lost : x;
}

constexpr int kMaxBlocks = 152 * 4;

// Sixteen-byte vectors want every row of every tensor on sixteen bytes, and groups of whole vectors.
bool whole(const NormArgs &a) {
  const int V = a.x_f32 ? 4 : 8;
  if (a.D % V || (a.groups && a.D / a.groups % V)) return false;
  const struct { const void *p; long long s; bool f32; } all[] = {
      {a.x, a.xs, a.x_f32}, {a.gate, a.gs, a.x_f32}, {a.residual, a.rs, a.r_f32},
      {a.z, a.zs, a.r_f32}, {a.y, a.ys, a.x_f32}, {a.dz, a.dzs, a.r_f32},
      {a.dy, a.dys, a.x_f32}, {a.dx, a.dxs, a.x_f32}, {a.dgate, a.dgs, a.x_f32},
      {a.dres, a.drs, a.r_f32}, {a.gain, 0, true}, {a.next_gain, 0, true}};
  for (const auto &t : all)
    if (t.p && (reinterpret_cast<uintptr_t>(t.p) % 16 || t.s % (t.f32 ? 4 : 8))) return false;
  return true;
}

// Bytes of shared memory that the rows of a block's inputs and the gains take in the backward pass.
template <typename TX, typename TR, int N, bool kTwice>
size_t staged_bytes(const NormArgs &a, int threads) {
  constexpr int V = 16 / sizeof(TX);
  const size_t x = N * V * sizeof(TX) * threads, r = N * V * sizeof(TR) * threads;
  const size_t gain = N * V * sizeof(float) * threads;
  constexpr int k = kTwice ? 2 : 1;
  return 2 * x + (a.gate ? 2 * x : 0) + k * ((a.dz ? r : 0) + (a.dy ? x : 0)) + (a.next && a.residual ? k * r : 0) +
         (a.gain ? gain : 0) + (a.next_gain ? gain : 0);
}

// fp32 rows beside bf16 ones: all of them on 32 bytes.
bool wide(const NormArgs &a) {
  const struct { const void *p; long long s; bool f32; } all[] = {
      {a.residual, a.rs, a.r_f32}, {a.z, a.zs, a.r_f32}, {a.dz, a.dzs, a.r_f32}, {a.dres, a.drs, a.r_f32},
      {a.gain, 0, true}, {a.next_gain, 0, true}};
  for (const auto &t : all)
    if (t.p && t.f32 && (reinterpret_cast<uintptr_t>(t.p) % 32 || t.s % 8)) return false;
  return !a.x_f32;
}

template <bool kBack, typename TX, typename TR, int kTeam, int N, bool kWhole, bool kStaged, bool kTwice = true>
cudaError_t go(NormArgs a, int threads, cudaStream_t st) {
  constexpr int V = 16 / sizeof(TX);
  const int n = a.groups ? a.D / a.groups : 1, teams = kTeam ? 256 / kTeam : 1;
  a.per = kWhole ? n / V : n;
  a.inv_n = 1.f / (float)n;
  a.inv_D = 1.f / (float)a.D;
  a.wide = kWhole && wide(a);
  a.mode = !a.groups ? kNone
           : a.groups == 1 ? kRow
           : kWhole && a.per <= (kTeam ? kTeam : 32) && (a.per & (a.per - 1)) == 0 ? kShuffle : kList;
  a.list = a.mode == kList ? (kWhole ? a.D / V : a.D) + a.groups : 0;
  void (*f)(NormArgs);
  if constexpr (kBack)
    f = k15_norm_bwd_kernel<TX, TR, kTeam, N, kWhole, kStaged, kTwice>;
  else
    f = k15_norm_kernel<TX, TR, kTeam, N, kWhole>;
  size_t smem = (kBack && kStaged ? staged_bytes<TX, TR, N, kTwice>(a, threads) : 0) + (size_t)teams * a.list * 4;
  if (kBack && teams > 1 && smem < (size_t)a.D * 4) smem = (size_t)a.D * 4;
  cudaError_t e;
  if (smem + 1024 > 48 * 1024 &&
      (e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
    return e;
  const long long blocks = ((long long)a.M + teams - 1) / teams;
  if (!kBack) {
    f<<<(unsigned)blocks, threads, smem, st>>>(a);
    return cudaGetLastError();
  }
  // as many blocks as are resident at once: what registers, threads and shared memory leave
  static const int regs = [&] {
    cudaFuncAttributes attr;
    return cudaFuncGetAttributes(&attr, f) == cudaSuccess ? attr.numRegs : 255;
  }();
  int resident = kMaxBlocks / 152;
  for (int x : {65536 / ((regs + 7) / 8 * 8 * threads), 2048 / threads, (int)(227 * 1024 / (smem + 1024))})
    resident = x < resident ? x : resident;
  const int most = 152 * (resident < 1 ? 1 : resident);
  const int grid = (int)(blocks < most ? blocks : most);
  f<<<grid, threads, smem, st>>>(a);
  e = cudaGetLastError();
  const int sums = (a.dgain ? 1 : 0) + (a.dnext ? 1 : 0);
  if (e != cudaSuccess || !sums) return e;
  k15_gain_kernel<<<dim3((a.D + 31) / 32, sums), 1024, 0, st>>>(a.ws, grid, a.D,
                                                                a.dgain ? a.dgain : a.dnext, a.dnext);
  return cudaGetLastError();
}

// A thread's elements: 16 (forward) or 8 (backward, which has twice the values to hold), more
// where the row is wider than 512 threads of them.  Rows of up to 512 elements go to
// warps or parts of warps.  Rows are staged where both of all inputs leave room in an SM's
// shared memory.  Rows element by element are no path to be quick on.
template <bool kBack, typename TX, typename TR>
cudaError_t pick(const NormArgs &a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(TX), k8 = 8 / V, k16 = 16 / V, k32 = 32 / V;
  const int D = a.D;
  auto threads = [&](int N) { return ((D + V - 1) / V + N * 32 - 1) / (N * 32) * 32; };
  if (!whole(a)) {
    if (D <= 128) return go<kBack, TX, TR, 8, k16, false, false>(a, 256, st);
    return go<kBack, TX, TR, 0, k32, false, false>(a, threads(k32), st);
  }
  if (D <= 64) return go<kBack, TX, TR, 8, k8, true, true, false>(a, 256, st);
  if (D <= 256) return go<kBack, TX, TR, 32, k8, true, true, false>(a, 256, st);
  if (D <= 512) return go<kBack, TX, TR, 32, k16, true, true>(a, 256, st);
  if constexpr (kBack) {
    // Eight elements a thread want 128 registers and two rows in shared memory and can do with 96
    // and less (bf16 rows of 2048, two blocks an SM either way: 72 us and 78): where that makes
    // room for another block (of 2560, one or two: 132 us and 99; 2500 in fp32: 170 and 135).
    const int n = threads(k8), with96 = 65536 / 96 / n, with128 = 65536 / 128 / n;
    if (D <= 4096 && with128 < with96 && with128 < kMaxBlocks / 152)
      return go<kBack, TX, TR, 0, k8, true, true, false>(a, n, st);
    if (D <= 4096) return go<kBack, TX, TR, 0, k8, true, true>(a, n, st);
  }
  if constexpr (kBack) {
    const int n = threads(k16);
    if (n <= 512 && staged_bytes<TX, TR, k16, true>(a, n) + (D / V + a.groups) * 4 <= 226 * 1024)
      return go<kBack, TX, TR, 0, k16, true, true>(a, n, st);
  } else {
    if (D <= 8192) return go<kBack, TX, TR, 0, k16, true, true>(a, threads(k16), st);
  }
  return go<kBack, TX, TR, 0, k32, true, false>(a, threads(k32), st);
}

template <bool kBack>
cudaError_t launch(const NormArgs &a, cudaStream_t st) {
  if (a.x_f32) return pick<kBack, float, float>(a, st);
  if (a.r_f32) return pick<kBack, __nv_bfloat16, float>(a, st);
  return pick<kBack, __nv_bfloat16, __nv_bfloat16>(a, st);
}

}  // namespace

size_t norm_workspace_bytes(int M, int D) {
  // one part a block and gain; no more blocks than rows
  return (size_t)(M < kMaxBlocks ? M : kMaxBlocks) * D * 2 * sizeof(float);
}
cudaError_t launch_norm(const NormArgs &a, cudaStream_t st) { return launch<false>(a, st); }
cudaError_t launch_norm_bwd(const NormArgs &a, cudaStream_t st) { return launch<true>(a, st); }

}  // namespace fs
