// k10_rope.cu -- rotary positions of q and k in one launch (fs_rope), and the
// transposed rotation for their gradients.
//
// Pair i of a token at position p turns by the angle p f_i.  The plan holds
// f_i / 2 pi as a fraction F_i of 2^64, so p F_i modulo 2^64 is the fraction of
// a turn, exact for every 32-bit p apart from F_i's own last bit (2^-53
// relative, as a double holds f_i): no fp64 arithmetic.  The nearest quarter turn is
// taken off in whole numbers; 32 bits of what is left, an eighth of a turn at most
// either way and cut to 2^-34 of one, become a float (half a step: 2^-27 of a half
// turn) and go to sincospif.  Converted without that, angles near a half turn are off by
// four times as much.
//
// Bound by memory: 4 bytes per bf16 element against a handful of operations.  A
// thread takes V pairs of one token (two 16-byte pieces of a row), works out
// their V sines once and walks the heads with them.
#include <math.h>

#include "fs_common.cuh"

namespace fs {
namespace {

struct RopeTensor {
  const void *x;
  void *y;
  long long xb, xh, xt, yb, yh, yt;  // elements between batches, heads, tokens
};

struct RopeK {
  RopeTensor t[2];
  int H[2];
  int N, d, rot, pairs;   // pairs: adjacent-pair layout
  int batch, per, groups; // heads a thread walks, groups of heads
  const int32_t *pos;
  long long pos_stride;
  int pos0, inverse;
  fs_rope_plan plan;
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// V consecutive elements: one 16-byte access, or one element.
template <typename T, int V>
struct alignas(V * sizeof(T)) Piece {
  T e[V];
};

// A thread's item: V pairs of a token (item < rot / (2 V)), or 2 V elements
// that pass through.
template <typename T, int V>
__global__ void __launch_bounds__(256) k10_rope_kernel(const __grid_constant__ RopeK a) {
  const int items = a.d / (2 * V), turned = a.rot / (2 * V);
  const unsigned id = blockIdx.x * 256u + threadIdx.x;  // below 2^32: checked by the caller
  const unsigned bn = id / items;
  const int item = (int)(id - bn * items);
  const int b = (int)(bn / (unsigned)a.N), n = (int)(bn - (unsigned)b * a.N);
  if (b >= a.batch) return;
  // element offsets of the item's two pieces inside a row
  int e0, e1;
  const bool turn = item < turned;
  if (turn && !a.pairs) {
    e0 = item * V;
    e1 = e0 + a.rot / 2;
  } else {
    e0 = item * 2 * V;
    e1 = e0 + V;
  }
  float c[V], s[V];
  if (turn) {
    const int p = a.pos ? a.pos[b * a.pos_stride + n] : a.pos0 + n;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint64_t t = (uint64_t)(int64_t)p * a.plan.turns[item * V + i];
      const uint32_t hi = (uint32_t)(t >> 32), quarter = (hi + (1u << 29)) >> 30;
      const int32_t left = (int32_t)__funnelshift_l((uint32_t)t, hi - (quarter << 30), 2);
      float sn, cs;
      sincospif((float)left * 0x1p-33f, &sn, &cs);
      c[i] = quarter & 1 ? sn : cs;
      s[i] = quarter & 1 ? cs : sn;
      c[i] *= (quarter + 1) & 2 ? -a.plan.amplitude : a.plan.amplitude;
      s[i] *= (quarter >> 1) ^ (uint32_t)a.inverse ? -a.plan.amplitude : a.plan.amplitude;
    }
  }
  const int h0 = blockIdx.y * a.per, h1 = min(h0 + a.per, a.H[0] + a.H[1]);
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const int w = h >= a.H[0];
    const RopeTensor &t = a.t[w];
    const int hh = w ? h - a.H[0] : h;
    const T *x = static_cast<const T *>(t.x) + b * t.xb + hh * t.xh + n * t.xt;
    T *y = static_cast<T *>(t.y) + b * t.yb + hh * t.yh + n * t.yt;
    Piece<T, V> u = *reinterpret_cast<const Piece<T, V> *>(x + e0);
    Piece<T, V> v = *reinterpret_cast<const Piece<T, V> *>(x + e1);
    if (turn) {
      if (a.pairs) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          Piece<T, V> &z = 2 * i < V ? u : v;
          const int j = 2 * i < V ? 2 * i : 2 * i - V;
          if constexpr (V > 1) {
            const float p0 = to_f(z.e[j]), p1 = to_f(z.e[j + 1]);
            z.e[j] = from_f<T>(p0 * c[i] - p1 * s[i]);
            z.e[j + 1] = from_f<T>(p1 * c[i] + p0 * s[i]);
          } else {
            const float p0 = to_f(u.e[0]), p1 = to_f(v.e[0]);
            u.e[0] = from_f<T>(p0 * c[0] - p1 * s[0]);
            v.e[0] = from_f<T>(p1 * c[0] + p0 * s[0]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float p0 = to_f(u.e[i]), p1 = to_f(v.e[i]);
          u.e[i] = from_f<T>(p0 * c[i] - p1 * s[i]);
          v.e[i] = from_f<T>(p1 * c[i] + p0 * s[i]);
        }
      }
    }
    *reinterpret_cast<Piece<T, V> *>(y + e0) = u;
    *reinterpret_cast<Piece<T, V> *>(y + e1) = v;
  }
}

template <typename T, int V>
cudaError_t launch_v(RopeK &k, cudaStream_t st) {
  const int heads = k.H[0] + k.H[1];
  const long long threads = (long long)k.batch * k.N * (k.d / (2 * V));
  const long long blocks = (threads + 255) / 256;
  // Heads are split over blocks until some 32 blocks an SM exist (several waves: 64k
  // tokens x 32 heads of 64 take 83.5 us, with 4 blocks an SM 90); a thread walks
  // the rest with the sines it has.
  int groups = (int)((152 * 32 + blocks - 1) / blocks);
  groups = groups < 1 ? 1 : (groups > heads ? heads : groups);
  k.per = (heads + groups - 1) / groups;
  k.groups = (heads + k.per - 1) / k.per;
  k10_rope_kernel<T, V><<<dim3((unsigned)blocks, k.groups), 256, 0, st>>>(k);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st) {
  RopeK k{};
  const size_t size = a.f32 ? 4 : 2;
  const int V = a.f32 ? 4 : 8;
  // 16-byte pieces need aligned rows and pieces that do not straddle the
  // rotated part or its half; anything else goes element by element.
  bool wide = a.plan->rot % (2 * V) == 0 && a.d % (2 * V) == 0;
  for (int i = 0; i < 2; ++i) {
    RopeTensor &t = k.t[i];
    t.x = a.x[i];
    t.y = a.y[i];
    k.H[i] = a.H[i];
    if (!a.H[i]) continue;
    t.xb = a.xs[i][0], t.xh = a.xs[i][1], t.xt = a.xs[i][2];
    t.yb = a.ys[i][0], t.yh = a.ys[i][1], t.yt = a.ys[i][2];
    wide = wide && (reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.y)) % 16 == 0;
    for (long long s : {t.xb, t.xh, t.xt, t.yb, t.yh, t.yt}) wide = wide && s * (long long)size % 16 == 0;
  }
  k.N = a.N;
  k.d = a.d;
  k.rot = a.plan->rot;
  k.pairs = a.plan->layout == FS_ROPE_PAIRS;
  k.batch = a.batch;
  k.pos = a.pos;
  k.pos_stride = a.pos_stride;
  k.pos0 = a.pos0;
  k.inverse = a.inverse;
  k.plan = *a.plan;
  if (a.f32) return wide ? launch_v<float, 4>(k, st) : launch_v<float, 1>(k, st);
  return wide ? launch_v<__nv_bfloat16, 8>(k, st) : launch_v<__nv_bfloat16, 1>(k, st);
}

int rope_make_plan(const fs_rope_params &p, fs_rope_plan *plan) {
  if (p.rot < 2 || p.rot % 2) return FS_ERR_INVALID_ARG;
  if (p.layout != FS_ROPE_HALF && p.layout != FS_ROPE_PAIRS) return FS_ERR_INVALID_ARG;
  if (p.scaling < FS_ROPE_PLAIN || p.scaling > FS_ROPE_RAMP) return FS_ERR_INVALID_ARG;
  if (!(p.base > 1.0) || !isfinite(p.base)) return FS_ERR_INVALID_ARG;
  if (!(p.factor >= 1.0) || !isfinite(p.factor)) return FS_ERR_INVALID_ARG;
  if (!(p.amplitude >= 0.0) || !(p.amplitude <= 3e38)) return FS_ERR_INVALID_ARG;
  if (p.scaling == FS_ROPE_BASE && p.rot == 2) return FS_ERR_INVALID_ARG;
  if (p.scaling == FS_ROPE_RAMP &&
      (p.original < 1 || !(p.beta_slow > 0.0) || !(p.beta_fast >= p.beta_slow) ||
       !isfinite(p.beta_fast)))
    return FS_ERR_INVALID_ARG;
  if (p.rot > FS_ROPE_MAX_ROT) return FS_ERR_UNSUPPORTED;
  const double pi = 3.14159265358979323846;
  const double r = p.rot;
  double base = p.base;
  if (p.scaling == FS_ROPE_BASE) base *= pow(p.factor, r / (r - 2.0));
  double lo = 0.0, hi = 0.0;
  if (p.scaling == FS_ROPE_RAMP) {
    lo = floor(r * log(p.original / (2.0 * pi * p.beta_fast)) / (2.0 * log(base)));
    hi = ceil(r * log(p.original / (2.0 * pi * p.beta_slow)) / (2.0 * log(base)));
    lo = lo < 0.0 ? 0.0 : lo;
    hi = hi > r - 1 ? r - 1 : hi;  // (of the elements: beyond the last pair)
  }
  fs_rope_plan out{};
  out.rot = p.rot;
  out.layout = p.layout;
  out.amplitude = (float)p.amplitude;
  for (int i = 0; i < p.rot / 2; ++i) {
    double f = pow(base, -2.0 * i / r);
    if (p.scaling == FS_ROPE_LINEAR) f /= p.factor;
    if (p.scaling == FS_ROPE_RAMP) {
      double g = (i - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
      g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
      f = f * (1.0 - g) + f / p.factor * g;
    }
    // f <= 1 here, so the fraction of a turn is below 2^64
    out.turns[i] = (uint64_t)ldexp(f / (2.0 * pi), 64);
  }
  *plan = out;
  return FS_OK;
}

}  // namespace fs
