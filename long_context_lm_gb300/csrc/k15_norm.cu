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
// Memory bounds both: every tensor is read or written once.  A team of
// threads holds a row in registers from its loads, all issued together, to
// its stores, so that z or y may take the place of an input.  Sums are fp32
// in a fixed order.  The gradients of the gains are sums over rows: a team
// keeps those of its columns over all rows that it takes, blocks put theirs
// into the workspace and a second kernel adds them in block order.
#include "fs_common.cuh"
#include "fs_internal.h"
#include "pairs.cuh"

namespace fs {
namespace {

// How a row's groups are added up.
enum Groups { kNone, kRow, kShuffle, kList };

// Sixteen bytes of a row of TX, or as many elements of TR: as they are in memory.
template <typename T, int V>
struct Raw {
  f2 x[V / 2];
  __device__ __forceinline__ f2 get(int c) const { return x[c]; }
};
template <int V>
struct Raw<__nv_bfloat16, V> {
  uint32_t x[V / 2];
  __device__ __forceinline__ f2 get(int c) const { return wide2(x[c]); }
};

// kWhole: rows are whole vectors on sixteen bytes.  Otherwise element by element.
template <bool kWhole, typename T, int V>
__device__ __forceinline__ void load(const void *row, int e, int D, Raw<T, V> &r) {
  const T *p = static_cast<const T *>(row) + e;
  if constexpr (kWhole) {
#pragma unroll
    for (int c = 0; c < V / 2; ++c) r.x[c] = 0;
    if (e >= D) return;
    if constexpr (sizeof(T) == 2) {
      const uint4 u = *reinterpret_cast<const uint4 *>(p);
      r.x[0] = u.x, r.x[1] = u.y, r.x[2] = u.z, r.x[3] = u.w;
    } else {
#pragma unroll
      for (int c = 0; c < V / 2; c += 2) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(p + 2 * c);
        r.x[c] = u.x, r.x[c + 1] = u.y;
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < V / 2; ++c) {
      const float x = e + 2 * c < D ? static_cast<float>(p[2 * c]) : 0.f;
      const float y = e + 2 * c + 1 < D ? static_cast<float>(p[2 * c + 1]) : 0.f;
      if constexpr (sizeof(T) == 2)
        r.x[c] = pack_bf16(x, y);  // (bf16 numbers: nothing is rounded)
      else
        r.x[c] = f2_bits(x, y);
    }
  }
}
template <bool kWhole, typename T, int V>
__device__ __forceinline__ void store(void *row, int e, int D, const f2 (&x)[V / 2]) {
  T *p = static_cast<T *>(row) + e;
  if constexpr (kWhole) {
    if (e >= D) return;
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
      if (e + 2 * c < D) p[2 * c] = static_cast<T>(lo2(x[c]));
      if (e + 2 * c + 1 < D) p[2 * c + 1] = static_cast<T>(hi2(x[c]));
    }
  }
}

// 1 / (1 + e^-x) by the special-function unit: 2^-20 of itself, enough for bf16 results.
// kExact: with the exponent's rounding put back and a Newton step on the reciprocal, 2^-22.
template <bool kExact>
__device__ __forceinline__ float sigmoid(float x) {
  constexpr float kL = -1.44269504f, kRest = -1.92596303e-8f;  // -log2 e, what it lacks
  float t = x * kL, e, r;
  if constexpr (kExact) t = fminf(t, 126.f);  // (past it the Newton step would meet an infinity)
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
  if constexpr (kExact) {
    const float rest = fmaf(x, kL, -t) + x * kRest;
    if (t < 126.f) e = fmaf(e, rest * 0.693147181f, e);
  }
  const float d = 1.f + e;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
  if constexpr (kExact) r = fmaf(r, fmaf(-d, r, 1.f), r);
  return r;
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

__device__ __forceinline__ f2 both(float x) { return f2_bits(x, x); }

// A team's way to add.  TPR threads take a row, N vectors of V elements each: vector i of
// thread t is number t + i TPR of the row.
template <int TPR, int V, int N, bool kWhole>
struct Team {
  static constexpr int kThreads = TPR < 256 ? 256 : TPR, kTeams = kThreads / TPR;
  static constexpr int kLanes = TPR < 32 ? TPR : 32;
  int t, team;    // thread within the team, team within the block
  float *scratch; // TPR > 32: two halves of the team's warps, in turn
  float *list;    // sums of vectors (elements), then of groups
  int turn;

  __device__ __forceinline__ void sync() const {
    if constexpr (TPR <= 32)
      __syncwarp();
    else if constexpr (kTeams == 1)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(TPR) : "memory");
  }
  // K sums over the team, the same in every thread.
  template <int K>
  __device__ __forceinline__ void add(float (&x)[K]) {
#pragma unroll
    for (int m = 1; m < kLanes; m *= 2)
#pragma unroll
      for (int k = 0; k < K; ++k) x[k] += __shfl_xor_sync(0xffffffffu, x[k], m);
    if constexpr (TPR > 32) {
      constexpr int kWarps = TPR / 32;
      float *to = scratch + (turn ^= 1) * 2 * kWarps;
      if (t % 32 == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) to[k * kWarps + t / 32] = x[k];
      sync();
      if constexpr (kWarps <= 4) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          x[k] = to[k * kWarps];
#pragma unroll
          for (int j = 1; j < kWarps; ++j) x[k] += to[k * kWarps + j];
        }
      } else {  // a warp adds them as it added its own
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] = t % 32 < kWarps ? to[k * kWarps + t % 32] : 0.f;
#pragma unroll
        for (int m = 1; m < kWarps; m *= 2)
#pragma unroll
          for (int k = 0; k < K; ++k) x[k] += __shfl_xor_sync(0xffffffffu, x[k], m);
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] = __shfl_sync(0xffffffffu, x[k], 0);
      }
    }
  }
  // Sums over groups of the products f(i, c) (pair c of vector i).  Groups of a power of two
  // of whole vectors, up to a warp's: by shuffles.  Others through `list`: a group to a
  // warp (or small team) at a time.
  template <typename F>
  __device__ __forceinline__ void add_groups(PerGroup<kWhole, V> (&p)[N], const NormArgs &a, F f) {
    const int mode = kWhole || a.mode <= kRow ? a.mode : kList;
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
          const int e = (t + i * TPR) * V + 2 * c;
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
          if (t + i * TPR < n) list[t + i * TPR] = v[i];
      }
      sync();
      for (int g = t / kLanes; g < a.groups; g += TPR / kLanes) {
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
          if (t + i * TPR < n) v[i] = list[n + (t + i * TPR) / a.per];
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int c = 0; c < V / 2; ++c) {
            const int e = (t + i * TPR) * V + 2 * c;
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
  // The factors that normalise x's groups (ones where they are not to be).
  template <typename T>
  __device__ __forceinline__ void factors(const Raw<T, V> (&x)[N], PerGroup<kWhole, V> (&inv)[N], const NormArgs &a) {
    if (a.mode == kNone) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < (kWhole ? 1 : V / 2); ++c) inv[i].x[c] = both(1.f);
      return;
    }
    add_groups(inv, a, [&](int i, int c) { return mul2(x[i].get(c), x[i].get(c)); });
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int c = 0; c < (kWhole ? 1 : V / 2); ++c) {
        // (past the row 0: with eps 0 the factor there would be infinite)
        const int e = (t + i * TPR) * V + 2 * c;
        const float f = e < a.D ? rsqrtf(fmaf(lo2(inv[i].x[c]), a.inv_n, a.eps)) : 0.f;
        const float g = kWhole ? f : e + 1 < a.D ? rsqrtf(fmaf(hi2(inv[i].x[c]), a.inv_n, a.eps)) : 0.f;
        inv[i].x[c] = f2_bits(f, g);
      }
  }
};

template <typename TX, typename TR, int TPR, int N, bool kWhole>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k15_norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int V = 16 / sizeof(TX);
  using T = Team<TPR, V, N, kWhole>;
  extern __shared__ float lists[];
  __shared__ float scratch[T::kTeams][TPR > 32 ? 4 * TPR / 32 : 1];
  T team{(int)threadIdx.x % TPR, (int)threadIdx.x / TPR, nullptr, nullptr, 0};
  team.scratch = scratch[team.team];
  team.list = lists + team.team * a.list;
  // (a small team without a row keeps its warp's shuffles and barriers company)
  const long long want = (long long)blockIdx.x * T::kTeams + team.team;
  if (TPR >= 32 && want >= a.M) return;
  const bool have = want < a.M;
  const long long row = have ? want : a.M - 1;
  const int e0 = team.t * V;

  Raw<TX, V> x[N], gate[N];
  f2 z[N][V / 2];
  {
    const TX *xr = static_cast<const TX *>(a.x) + row * a.xs;
#pragma unroll
    for (int i = 0; i < N; ++i) load<kWhole>(xr, e0 + i * TPR * V, a.D, x[i]);
  }
  if (a.gate) {
    const TX *gr = static_cast<const TX *>(a.gate) + row * a.gs;
#pragma unroll
    for (int i = 0; i < N; ++i) load<kWhole>(gr, e0 + i * TPR * V, a.D, gate[i]);
  }
  Raw<TR, V> res[N];
  if (a.residual) {
    const TR *rr = static_cast<const TR *>(a.residual) + row * a.rs;
#pragma unroll
    for (int i = 0; i < N; ++i) load<kWhole>(rr, e0 + i * TPR * V, a.D, res[i]);
  }
  {
    PerGroup<kWhole, V> inv[N];
    team.factors(x, inv, a);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(x[i].get(c), inv[i].get(c));
  }
  if (a.gain) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      Raw<float, V> g;
      load<kWhole>(a.gain, e0 + i * TPR * V, a.D, g);
#pragma unroll
      for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(z[i][c], g.x[c]);
    }
  }
  if (a.gate) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int c = 0; c < V / 2; ++c) {
        const f2 g = gate[i].get(c);
        z[i][c] = mul2(z[i][c], mul2(g, sigmoid2<sizeof(TX) == 4>(g)));
      }
  }
  const f2 scale = both(a.scale);
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int c = 0; c < V / 2; ++c) z[i][c] = madd2(scale, z[i][c], res[i].get(c));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(scale, z[i][c]);
  }
  float f = 0.f;
  if (a.next) {
    f2 s = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int c = 0; c < V / 2; ++c) s = madd2(z[i][c], z[i][c], s);
    float ss[1] = {lo2(s) + hi2(s)};
    team.add(ss);
    f = rsqrtf(fmaf(ss[0], a.inv_D, a.eps));
  }
  if (!have) return;
  if (a.z) {
    TR *zr = static_cast<TR *>(a.z) + row * a.zs;
#pragma unroll
    for (int i = 0; i < N; ++i) store<kWhole, TR, V>(zr, e0 + i * TPR * V, a.D, z[i]);
  }
  if (a.next) {
    TX *yr = static_cast<TX *>(a.y) + row * a.ys;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
      for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(z[i][c], both(f));
      if (a.next_gain) {
        Raw<float, V> g;
        load<kWhole>(a.next_gain, e0 + i * TPR * V, a.D, g);
#pragma unroll
        for (int c = 0; c < V / 2; ++c) z[i][c] = mul2(z[i][c], g.x[c]);
      }
      store<kWhole, TX, V>(yr, e0 + i * TPR * V, a.D, z[i]);
    }
  }
}

template <typename TX, typename TR, int TPR, int N, bool kWhole>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, 1) k15_norm_bwd_kernel(const __grid_constant__ NormArgs a) {
  constexpr int V = 16 / sizeof(TX);
  constexpr bool kExact = sizeof(TX) == 4;
  using T = Team<TPR, V, N, kWhole>;
  extern __shared__ float lists[];
  __shared__ float scratch[T::kTeams][TPR > 32 ? 4 * TPR / 32 : 1];
  T team{(int)threadIdx.x % TPR, (int)threadIdx.x / TPR, nullptr, nullptr, 0};
  team.scratch = scratch[team.team];
  team.list = lists + team.team * a.list;
  const int step = gridDim.x * T::kTeams, e0 = team.t * V;
  f2 dgain[N][V / 2] = {}, dnext[N][V / 2] = {};
  const f2 scale = both(a.scale);

  for (long long want = (long long)blockIdx.x * T::kTeams + team.team;
       TPR >= 32 ? want < a.M : want - team.team < a.M; want += step) {
    const bool have = want < a.M;
    const long long row = have ? want : a.M - 1;
    Raw<TX, V> x[N], gate[N], dy[N];
    Raw<TR, V> dz[N], res[N];
    {
      const TX *xr = static_cast<const TX *>(a.x) + row * a.xs;
#pragma unroll
      for (int i = 0; i < N; ++i) load<kWhole>(xr, e0 + i * TPR * V, a.D, x[i]);
    }
    if (a.gate) {
      const TX *gr = static_cast<const TX *>(a.gate) + row * a.gs;
#pragma unroll
      for (int i = 0; i < N; ++i) load<kWhole>(gr, e0 + i * TPR * V, a.D, gate[i]);
    }
    if (a.dz) {
      const TR *dr = static_cast<const TR *>(a.dz) + row * a.dzs;
#pragma unroll
      for (int i = 0; i < N; ++i) load<kWhole>(dr, e0 + i * TPR * V, a.D, dz[i]);
    }
    if (a.next) {
      const TX *dr = static_cast<const TX *>(a.dy) + row * a.dys;
#pragma unroll
      for (int i = 0; i < N; ++i) load<kWhole>(dr, e0 + i * TPR * V, a.D, dy[i]);
      if (a.residual) {
        const TR *rr = static_cast<const TR *>(a.residual) + row * a.rs;
#pragma unroll
        for (int i = 0; i < N; ++i) load<kWhole>(rr, e0 + i * TPR * V, a.D, res[i]);
      }
    }
    // h (x normalised) is worked out again where it is used: x in 16 bits and a group's
    // factor take fewer registers
    PerGroup<kWhole, V> inv[N];
    team.factors(x, inv, a);
    f2 sig[N][V / 2];
    if (a.gate) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < V / 2; ++c) sig[i][c] = sigmoid2<kExact>(gate[i].get(c));
    }
    f2 g[N][V / 2];  // the gradient that reaches z
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int c = 0; c < V / 2; ++c) g[i][c] = a.dz ? dz[i].get(c) : 0;
    if (a.next) {
      f2 z[N][V / 2], s0 = 0, s1 = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        Raw<float, V> gain, next;
        if (a.gain) load<kWhole>(a.gain, e0 + i * TPR * V, a.D, gain);
        if (a.next_gain) load<kWhole>(a.next_gain, e0 + i * TPR * V, a.D, next);
#pragma unroll
        for (int c = 0; c < V / 2; ++c) {
          f2 u = mul2(x[i].get(c), inv[i].get(c));
          if (a.gain) u = mul2(u, gain.x[c]);
          if (a.gate) u = mul2(u, mul2(gate[i].get(c), sig[i][c]));
          u = a.residual ? madd2(scale, u, res[i].get(c)) : mul2(scale, u);
          z[i][c] = u;
          s0 = madd2(u, u, s0);
          f2 w = dy[i].get(c);
          if (a.next_gain) w = mul2(w, next.x[c]);
          s1 = madd2(u, w, s1);
        }
      }
      float s[2] = {lo2(s0) + hi2(s0), lo2(s1) + hi2(s1)};
      team.add(s);
      const float r = rsqrtf(fmaf(s[0], a.inv_D, a.eps));
      const f2 rr = both(r), mc = both(-r * r * s[1] * a.inv_D);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        Raw<float, V> next;
        if (a.next_gain) load<kWhole>(a.next_gain, e0 + i * TPR * V, a.D, next);
#pragma unroll
        for (int c = 0; c < V / 2; ++c) {
          f2 w = dy[i].get(c);
          if (have) dnext[i][c] = madd2(mul2(w, rr), z[i][c], dnext[i][c]);
          if (a.next_gain) w = mul2(w, next.x[c]);
          g[i][c] = madd2(rr, madd2(mc, z[i][c], w), g[i][c]);
        }
      }
    }
    if (a.dres && have) {
      TR *dr = static_cast<TR *>(a.dres) + row * a.drs;
#pragma unroll
      for (int i = 0; i < N; ++i) store<kWhole, TR, V>(dr, e0 + i * TPR * V, a.D, g[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      Raw<float, V> gain;
      if (a.gain) load<kWhole>(a.gain, e0 + i * TPR * V, a.D, gain);
      f2 out[V / 2];
#pragma unroll
      for (int c = 0; c < V / 2; ++c) {
        const f2 h = mul2(x[i].get(c), inv[i].get(c));
        f2 u = mul2(scale, g[i][c]);
        if (a.gate) {
          const f2 gt = gate[i].get(c), sg = sig[i][c];
          f2 d = mul2(u, h);
          if (a.gain) d = mul2(d, gain.x[c]);
          const f2 silu = mul2(gt, sg);
          // silu' = sig (1 + gate (1 - sig)) = sig + silu - silu sig
          out[c] = mul2(d, sub2_bits(add2_bits(sg, silu), mul2(silu, sg)));
          u = mul2(u, silu);
        }
        if (have) dgain[i][c] = madd2(u, h, dgain[i][c]);
        if (a.gain) u = mul2(u, gain.x[c]);
        g[i][c] = u;
      }
      if (a.dgate && have)
        store<kWhole, TX, V>(static_cast<TX *>(a.dgate) + row * a.dgs, e0 + i * TPR * V, a.D, out);
    }
    if (a.mode != kNone) {
      PerGroup<kWhole, V> p[N];
      team.add_groups(p, a, [&](int i, int c) { return mul2(g[i][c], mul2(x[i].get(c), inv[i].get(c))); });
      const f2 mn = both(-a.inv_n);
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < V / 2; ++c) {
          const f2 h = mul2(x[i].get(c), inv[i].get(c));
          g[i][c] = mul2(inv[i].get(c), madd2(mul2(mn, p[i].get(c)), h, g[i][c]));
        }
    }
    if (have) {
      TX *dr = static_cast<TX *>(a.dx) + row * a.dxs;
#pragma unroll
      for (int i = 0; i < N; ++i) store<kWhole, TX, V>(dr, e0 + i * TPR * V, a.D, g[i]);
    }
  }

  // the block's gains: its teams' added in their order
  float *total = lists;  // (no team is in a row any more once all are here)
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (!(which ? a.dnext : a.dgain)) continue;
    float *to = a.ws + ((size_t)(which && a.dgain ? gridDim.x : 0) + blockIdx.x) * a.D;
    for (int k = 0; k < T::kTeams; ++k) {
      if (T::kTeams > 1) __syncthreads();
      if (team.team != k) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int e = e0 + i * TPR * V + j;
          if (e >= a.D) continue;
          const f2 pair = which ? dnext[i][j / 2] : dgain[i][j / 2];
          const float x = (k ? total[e] : 0.f) + (j % 2 ? hi2(pair) : lo2(pair));
          if (k + 1 < T::kTeams)
            total[e] = x;
          else
            to[e] = x;
        }
      }
    }
  }
}

// Column sums of the blocks' parts in fp64, in order: 32 columns a block, 32 runs of parts.
__global__ void __launch_bounds__(1024) k15_gain_kernel(const float *part, int blocks, int D,
                                                        float *first, float *second) {
  __shared__ double run[32][33];
  const int lane = threadIdx.x % 32, k = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  const float *p = part + (size_t)blockIdx.y * blocks * D + c;
  double x = 0.0;
  if (c < D) {
#pragma unroll 4
    for (int i = k; i < blocks; i += 32) x += __ldg(p + (size_t)i * D);
  }
  run[k][lane] = x;
  __syncthreads();
  // a warp to each column
  x = run[lane][k];
#pragma unroll
  for (int m = 16; m > 0; m /= 2) x += __shfl_xor_sync(0xffffffffu, x, m);
  const int to = blockIdx.x * 32 + k;
  if (lane == 0 && to < D) (blockIdx.y ? second : first)[to] = (float)x;
}

constexpr int kMaxBlocks = 152 * 2;

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

template <bool kBack, typename TX, typename TR, int TPR, int N, bool kWhole>
cudaError_t go(NormArgs a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(TX);
  using T = Team<TPR, V, N, kWhole>;
  const int n = a.groups ? a.D / a.groups : 1;
  a.per = kWhole ? n / V : n;
  a.inv_n = 1.f / (float)n;
  a.inv_D = 1.f / (float)a.D;
  a.mode = !a.groups ? kNone
           : a.groups == 1 ? kRow
           : kWhole && a.per <= T::kLanes && (a.per & (a.per - 1)) == 0 ? kShuffle : kList;
  a.list = a.mode == kList || (!kWhole && a.groups > 1) ? (kWhole ? a.D / V : a.D) + a.groups : 0;
  const long long blocks = ((long long)a.M + T::kTeams - 1) / T::kTeams;
  size_t smem = (size_t)T::kTeams * a.list * 4;
  if (kBack && T::kTeams > 1 && smem < (size_t)a.D * 4) smem = (size_t)a.D * 4;
  void (*f)(NormArgs);
  if constexpr (kBack)
    f = k15_norm_bwd_kernel<TX, TR, TPR, N, kWhole>;
  else
    f = k15_norm_kernel<TX, TR, TPR, N, kWhole>;
  cudaError_t e;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
    return e;
  if (!kBack) {
    f<<<(unsigned)blocks, T::kThreads, smem, st>>>(a);
    return cudaGetLastError();
  }
  const int grid = (int)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
  f<<<grid, T::kThreads, smem, st>>>(a);
  e = cudaGetLastError();
  const int sums = (a.dgain ? 1 : 0) + (a.dnext ? 1 : 0);
  if (e != cudaSuccess || !sums) return e;
  k15_gain_kernel<<<dim3((a.D + 31) / 32, sums), 1024, 0, st>>>(a.ws, grid, a.D,
                                                                a.dgain ? a.dgain : a.dnext, a.dnext);
  return cudaGetLastError();
}

// The smallest team whose threads hold the row, 16 elements each, 8 in the backward pass,
// which has twice the values to hold (more for the widest rows).  Rows element by
// element are no path to be quick on: fewer teams.
template <bool kBack, typename TX, typename TR>
cudaError_t pick(const NormArgs &a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(TX), k8 = 8 / V, k16 = 16 / V, k32 = 32 / V;
  const int D = a.D;
  if (!whole(a)) {
    if (D <= 128) return go<kBack, TX, TR, 8, k16, false>(a, st);
    if (D <= 2048) return go<kBack, TX, TR, 128, k16, false>(a, st);
    return go<kBack, TX, TR, 512, k32, false>(a, st);
  }
  if (D <= 64) return go<kBack, TX, TR, 8, k8, true>(a, st);
  if (D <= 256) return go<kBack, TX, TR, 32, k8, true>(a, st);
  if constexpr (kBack) {
    if (D <= 512) return go<kBack, TX, TR, 64, k8, true>(a, st);
    if (D <= 1024) return go<kBack, TX, TR, 128, k8, true>(a, st);
    if (D <= 2048) return go<kBack, TX, TR, 256, k8, true>(a, st);
    if (D <= 4096) return go<kBack, TX, TR, 512, k8, true>(a, st);
  } else {
    if (D <= 512) return go<kBack, TX, TR, 32, k16, true>(a, st);
    if (D <= 1024) return go<kBack, TX, TR, 64, k16, true>(a, st);
    if (D <= 2048) return go<kBack, TX, TR, 128, k16, true>(a, st);
    if (D <= 4096) return go<kBack, TX, TR, 256, k16, true>(a, st);
  }
  if (D <= 8192) return go<kBack, TX, TR, 512, k16, true>(a, st);
  return go<kBack, TX, TR, 512, k32, true>(a, st);
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
