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

namespace fs {
namespace {

// Up to 16 bytes of a row's elements as fp32.
template <typename T, int V>
__device__ __forceinline__ void load(const void *p, long long at, float (&x)[V]) {
  const T *s = static_cast<const T *>(p) + at;
  if constexpr (V == 1) {
    x[0] = static_cast<float>(*s);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 u = *reinterpret_cast<const float4 *>(s + i);
      x[i] = u.x, x[i + 1] = u.y, x[i + 2] = u.z, x[i + 3] = u.w;
    }
  } else {
    static_assert(V == 8, "sixteen bytes");
    const uint4 u = *reinterpret_cast<const uint4 *>(s);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store(void *p, long long at, const float (&x)[V]) {
  T *s = static_cast<T *>(p) + at;
  if constexpr (V == 1) {
    *s = static_cast<T>(x[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4 *>(s + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else {
    *reinterpret_cast<uint4 *>(s) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                               pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
}

// 1 / (1 + e^-x).  bf16 results need no more than the special-function unit's
// exponential and reciprocal (2^-20 or better); fp32 ones take the exact pair.
template <bool kExact>
__device__ __forceinline__ float sigmoid(float x) {
  if constexpr (kExact) return 1.f / (1.f + expf(-x));
  return __fdividef(1.f, 1.f + __expf(-x));
}

// A team's rows and its way to add.  TPR threads take a row, N vectors of V
// elements each: vector i of thread t is number t + i TPR of the row.
template <int TPR, int V, int N>
struct Team {
  static constexpr int kThreads = TPR < 256 ? 256 : TPR, kTeams = kThreads / TPR;
  int t, team;    // thread within the team, team within the block
  float *scratch; // TPR > 32: two halves of the team's warps, in turn
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
    for (int m = 1; m < (TPR < 32 ? TPR : 32); m *= 2)
#pragma unroll
      for (int k = 0; k < K; ++k) x[k] += __shfl_xor_sync(0xffffffffu, x[k], m);
    if constexpr (TPR > 32) {
      constexpr int kWarps = TPR / 32;
      float *to = scratch + (turn ^= 1) * 2 * kWarps;
      if (t % 32 == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) to[k * kWarps + t / 32] = x[k];
      sync();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        x[k] = 0.f;
        for (int j = 0; j < kWarps; ++j) x[k] += to[k * kWarps + j];
      }
    }
  }
  // x[i] (vector i's sum) becomes the sum over the group that the vector lies in.
  // Groups of whole vectors, a power of two of them up to a warp's: by shuffles.
  // Others: the vectors' sums in `list`, a group to a warp (or small team) at a time.
  __device__ __forceinline__ void add_groups(float (&x)[N], int D, int groups, float *list) {
    if (groups == 1) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < N; ++i) s[0] += x[i];
      add(s);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = s[0];
      return;
    }
    const int per = D / groups / V;  // vectors in a group
    constexpr int kLanes = TPR < 32 ? TPR : 32;
    if (per <= kLanes && (per & (per - 1)) == 0) {
      for (int m = 1; m < per; m *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], m);
      return;
    }
    const int vectors = D / V;
    sync();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (t + i * TPR < vectors) list[t + i * TPR] = x[i];
    sync();
    for (int g = t / kLanes; g < groups; g += TPR / kLanes) {
      float s = 0.f;
      for (int j = t % kLanes; j < per; j += kLanes) s += list[g * per + j];
#pragma unroll
      for (int m = 1; m < kLanes; m *= 2)
        s += __shfl_xor_sync(0xffffffffu, s, m);
      if (t % kLanes == 0) list[vectors + g] = s;
    }
    sync();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (t + i * TPR < vectors) x[i] = list[vectors + (t + i * TPR) / per];
  }
};

// What a team knows of its row: x (then h), the group factors, the gate's sigmoid, z.
template <typename TX, typename TR, int TPR, int V, int N>
struct Row {
  float h[N][V], gate[N][V], sig[N][V], z[N][V], inv[N];

  __device__ __forceinline__ void read(const NormArgs &a, long long row, int t, bool residual) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = (t + i * TPR) * V;
      const bool in = e < a.D;
#pragma unroll
      for (int j = 0; j < V; ++j) h[i][j] = gate[i][j] = z[i][j] = 0.f;
      if (in) load<TX, V>(a.x, row * a.xs + e, h[i]);
      if (in && a.gate) load<TX, V>(a.gate, row * a.gs + e, gate[i]);
      if (in && residual) load<TR, V>(a.residual, row * a.rs + e, z[i]);
    }
  }
  template <typename TeamT>
  __device__ __forceinline__ void normalise(const NormArgs &a, TeamT &team, float *list) {
    // (vectors past the row keep a factor of 0: with eps 0 theirs would be infinite)
    if (!a.groups) {
#pragma unroll
      for (int i = 0; i < N; ++i) inv[i] = 1.f;
      return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      inv[i] = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) inv[i] = fmaf(h[i][j], h[i][j], inv[i]);
    }
    team.add_groups(inv, a.D, a.groups, list);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      inv[i] = (team.t + i * TPR) * V < a.D
                   ? rsqrtf(inv[i] / (float)(a.D / a.groups) + a.eps)
                   : 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) h[i][j] *= inv[i];
    }
  }
};

template <int V>
__device__ __forceinline__ void load_gain(const float *p, int e, int D, float (&x)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = 1.f;
  if (p && e < D) load<float, V>(p, e, x);
}

template <typename TX, typename TR, int TPR, int V, int N>
__global__ void __launch_bounds__(Team<TPR, V, N>::kThreads) k15_norm_kernel(
    const __grid_constant__ NormArgs a) {
  using T = Team<TPR, V, N>;
  extern __shared__ float lists[];
  __shared__ float scratch[T::kTeams][TPR > 32 ? 4 * TPR / 32 : 1];
  T team{(int)threadIdx.x % TPR, (int)threadIdx.x / TPR, nullptr, 0};
  team.scratch = scratch[team.team];
  // (a small team without a row keeps its warp's shuffles and barriers company)
  const long long want = (long long)blockIdx.x * T::kTeams + team.team;
  if (TPR >= 32 && want >= a.M) return;
  const bool have = want < a.M;
  const long long row = have ? want : a.M - 1;
  float *list = lists + team.team * (a.D / V + a.groups);

  Row<TX, TR, TPR, V, N> r;
  r.read(a, row, team.t, a.residual != nullptr);
  r.normalise(a, team, list);
  float ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float gain[V];
    load_gain<V>(a.gain, (team.t + i * TPR) * V, a.D, gain);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float x = r.h[i][j] * gain[j];
      if (a.gate) x *= r.gate[i][j] * sigmoid<sizeof(TX) == 4>(r.gate[i][j]);
      r.z[i][j] = fmaf(a.scale, x, r.z[i][j]);
      ss[0] = fmaf(r.z[i][j], r.z[i][j], ss[0]);
    }
  }
  float f = 0.f;
  if (a.next) {
    team.add(ss);
    f = rsqrtf(ss[0] / (float)a.D + a.eps);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = (team.t + i * TPR) * V;
    if (e >= a.D || !have) continue;
    if (a.z) store<TR, V>(a.z, row * a.zs + e, r.z[i]);
    if (a.next) {
      float gain[V];
      load_gain<V>(a.next_gain, e, a.D, gain);
#pragma unroll
      for (int j = 0; j < V; ++j) gain[j] *= r.z[i][j] * f;
      store<TX, V>(a.y, row * a.ys + e, gain);
    }
  }
}

template <typename TX, typename TR, int TPR, int V, int N>
__global__ void __launch_bounds__(Team<TPR, V, N>::kThreads) k15_norm_bwd_kernel(
    const __grid_constant__ NormArgs a) {
  using T = Team<TPR, V, N>;
  extern __shared__ float lists[];
  __shared__ float scratch[T::kTeams][TPR > 32 ? 4 * TPR / 32 : 1];
  T team{(int)threadIdx.x % TPR, (int)threadIdx.x / TPR, nullptr, 0};
  team.scratch = scratch[team.team];
  const int step = gridDim.x * T::kTeams;
  float *list = lists + team.team * (a.D / V + a.groups);
  float dgain[N][V] = {}, dnext[N][V] = {};
  const float per_row = 1.f / (float)a.D, per_group = a.groups ? (float)a.groups / (float)a.D : 0.f;

  for (long long want = (long long)blockIdx.x * T::kTeams + team.team;
       TPR >= 32 ? want < a.M : want - team.team < a.M; want += step) {
    const bool have = want < a.M;
    const long long row = have ? want : a.M - 1;
    Row<TX, TR, TPR, V, N> r;
    float g[N][V];
    r.read(a, row, team.t, a.next && a.residual);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = (team.t + i * TPR) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) g[i][j] = 0.f;
      if (e < a.D && a.dz) load<TR, V>(a.dz, row * a.dzs + e, g[i]);
    }
    float dy[N][V];
    if (a.next) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = (team.t + i * TPR) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) dy[i][j] = 0.f;
        if (e < a.D) load<TX, V>(a.dy, row * a.dys + e, dy[i]);
      }
    }
    r.normalise(a, team, list);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j)
        r.sig[i][j] = a.gate ? sigmoid<sizeof(TX) == 4>(r.gate[i][j]) : 0.f;
    if (a.next) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = (team.t + i * TPR) * V;
        float gain[V], next[V];
        load_gain<V>(a.gain, e, a.D, gain);
        load_gain<V>(a.next_gain, e, a.D, next);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float x = r.h[i][j] * gain[j];
          if (a.gate) x *= r.gate[i][j] * r.sig[i][j];
          r.z[i][j] = fmaf(a.scale, x, r.z[i][j]);
          s[0] = fmaf(r.z[i][j], r.z[i][j], s[0]);
          s[1] = fmaf(r.z[i][j], dy[i][j] * next[j], s[1]);
        }
      }
      team.add(s);
      const float f = rsqrtf(s[0] * per_row + a.eps), c = f * f * s[1] * per_row;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float next[V];
        load_gain<V>(a.next_gain, (team.t + i * TPR) * V, a.D, next);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          g[i][j] = fmaf(f, fmaf(-c, r.z[i][j], dy[i][j] * next[j]), g[i][j]);
          if (have) dnext[i][j] = fmaf(dy[i][j] * f, r.z[i][j], dnext[i][j]);
        }
      }
    }
    float sums[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = (team.t + i * TPR) * V;
      const bool in = e < a.D && have;
      float gain[V], out[V];
      load_gain<V>(a.gain, e, a.D, gain);
      if (in && a.dres) store<TR, V>(a.dres, row * a.drs + e, g[i]);
      sums[i] = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float u = a.scale * g[i][j];
        if (a.gate) {
          const float gate = r.gate[i][j], sig = r.sig[i][j];
          out[j] = u * (r.h[i][j] * gain[j]) * (sig * fmaf(gate, 1.f - sig, 1.f));
          u *= gate * sig;
        }
        if (have) dgain[i][j] = fmaf(u, r.h[i][j], dgain[i][j]);
        g[i][j] = u * gain[j];
        sums[i] = fmaf(g[i][j], r.h[i][j], sums[i]);
      }
      if (in && a.dgate) store<TX, V>(a.dgate, row * a.dgs + e, out);
    }
    if (a.groups) team.add_groups(sums, a.D, a.groups, list);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = (team.t + i * TPR) * V;
      if (a.groups) {
        const float c = sums[i] * per_group;
#pragma unroll
        for (int j = 0; j < V; ++j) g[i][j] = r.inv[i] * fmaf(-c, r.h[i][j], g[i][j]);
      }
      if (e < a.D && have) store<TX, V>(a.dx, row * a.dxs + e, g[i]);
    }
  }

  // the block's gains: its teams' added in their order
  float *total = lists;  // (no team is in a row any more once all are here)
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (!(which ? a.dnext : a.dgain)) continue;
    float *to = a.ws + ((size_t)(which && a.dgain ? gridDim.x : 0) + blockIdx.x) * a.D;
    for (int k = 0; k < T::kTeams; ++k) {
      __syncthreads();
      if (team.team != k) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int e = (team.t + i * TPR) * V + j;
          if (e >= a.D) continue;
          const float x = (k ? total[e] : 0.f) + (which ? dnext[i][j] : dgain[i][j]);
          if (k + 1 < T::kTeams)
            total[e] = x;
          else
            to[e] = x;
        }
      }
    }
  }
}

// Column sums of the blocks' parts, in order: 32 columns a block, eight runs of parts.
__global__ void __launch_bounds__(256) k15_gain_kernel(const float *part, int blocks, int D,
                                                       float *first, float *second) {
  __shared__ double run[8][32];
  const int c = blockIdx.x * 32 + threadIdx.x % 32, k = threadIdx.x / 32;
  const float *p = part + (size_t)blockIdx.y * blocks * D;
  double x = 0.0;
  for (int i = k; i < blocks && c < D; i += 8) x += p[(size_t)i * D + c];
  run[k][threadIdx.x % 32] = x;
  __syncthreads();
  if (k || c >= D) return;
  for (int i = 1; i < 8; ++i) x += run[i][threadIdx.x];
  (blockIdx.y ? second : first)[c] = (float)x;
}

constexpr int kMaxBlocks = 152 * 4;

// Sixteen-byte vectors want every row of every tensor on sixteen bytes, and groups of whole vectors.
bool vectors(const NormArgs &a) {
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

template <typename TX, typename TR, int TPR, int V, int N>
cudaError_t go(const NormArgs &a, bool back, cudaStream_t st) {
  using T = Team<TPR, V, N>;
  const long long blocks = ((long long)a.M + T::kTeams - 1) / T::kTeams;
  size_t smem = a.groups > 1 ? (size_t)T::kTeams * (a.D / V + a.groups) * 4 : 0;
  if (!back) {
    auto f = k15_norm_kernel<TX, TR, TPR, V, N>;
    if (smem > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    f<<<(unsigned)blocks, T::kThreads, smem, st>>>(a);
    return cudaGetLastError();
  }
  auto f = k15_norm_bwd_kernel<TX, TR, TPR, V, N>;
  if (T::kTeams > 1 && smem < (size_t)a.D * 4) smem = (size_t)a.D * 4;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const int grid = (int)(blocks < kMaxBlocks ? blocks : kMaxBlocks);
  f<<<grid, T::kThreads, smem, st>>>(a);
  cudaError_t e = cudaGetLastError();
  const int n = (a.dgain ? 1 : 0) + (a.dnext ? 1 : 0);
  if (e != cudaSuccess || !n) return e;
  k15_gain_kernel<<<dim3((a.D + 31) / 32, n), 256, 0, st>>>(
      a.ws, grid, a.D, a.dgain ? a.dgain : a.dnext, a.dnext);
  return cudaGetLastError();
}

// The smallest team whose threads hold the row, 16 elements each (32 for the
// widest).  Rows by single elements are no path to be quick on: fewer teams.
template <typename TX, typename TR, int V>
cudaError_t pick(const NormArgs &a, bool back, cudaStream_t st) {
  constexpr int kN = 16 / V;  // vectors of sixteen elements
  const int D = a.D;
  if constexpr (V > 1) {
    if (D <= 64) return go<TX, TR, 8, V, 8 / V>(a, back, st);
    if (D <= 256) return go<TX, TR, 32, V, 8 / V>(a, back, st);
    if (D <= 512) return go<TX, TR, 32, V, kN>(a, back, st);
    if (D <= 1024) return go<TX, TR, 64, V, kN>(a, back, st);
    if (D <= 2048) return go<TX, TR, 128, V, kN>(a, back, st);
    if (D <= 4096) return go<TX, TR, 256, V, kN>(a, back, st);
  } else {
    if (D <= 128) return go<TX, TR, 8, V, kN>(a, back, st);
    if (D <= 2048) return go<TX, TR, 128, V, kN>(a, back, st);
  }
  if (D <= 8192) return go<TX, TR, 512, V, kN>(a, back, st);
  return go<TX, TR, 512, V, 2 * kN>(a, back, st);
}

template <typename TX, typename TR>
cudaError_t dispatch(const NormArgs &a, bool back, cudaStream_t st) {
  constexpr int kV = 16 / sizeof(TX);
  return vectors(a) ? pick<TX, TR, kV>(a, back, st) : pick<TX, TR, 1>(a, back, st);
}

cudaError_t launch(const NormArgs &a, bool back, cudaStream_t st) {
  if (a.x_f32) return dispatch<float, float>(a, back, st);
  if (a.r_f32) return dispatch<__nv_bfloat16, float>(a, back, st);
  return dispatch<__nv_bfloat16, __nv_bfloat16>(a, back, st);
}

}  // namespace

size_t norm_workspace_bytes(int M, int D) {
  // one part a block and gain; no more blocks than rows
  return (size_t)(M < kMaxBlocks ? M : kMaxBlocks) * D * 2 * sizeof(float);
}
cudaError_t launch_norm(const NormArgs &a, cudaStream_t st) { return launch(a, false, st); }
cudaError_t launch_norm_bwd(const NormArgs &a, cudaStream_t st) { return launch(a, true, st); }

}  // namespace fs
