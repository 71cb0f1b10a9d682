// k14_linear.cu -- linear attention with a decay for each head, token by token.
//
//   S_t = lam S_{t-1} + k_t v_t^T,   out_t = scale q_t S_t,   lam = exp(decay)
//
// The columns of S (the elements of v and out) do not meet, so a block takes 32 of
// them: 128 bytes of every row, each thread four columns of d / 16 neighbouring rows.
// For a decoding step the state's bytes are everything (read once, written once:
// 2 x 4 d^2 bytes against 8 d bytes of rows), so all of a thread's state is under way
// before anything is computed, and a thread has enough of it (32 elements at d = 128)
// to carry the decay's exponential and the sums over rows.  128 sequences x 16 heads of
// 128: 268 MB of states in 43.6 us, 6.2 TB/s, 91% of a copy's rate.
// lam goes in as two fp32 numbers (linear.cuh): as one it would be off by up to
// 2^-25 in the same direction at every token, and a head with a long memory adds
// that up over thousands of them.
#include "fs_common.cuh"
#include "fs_internal.h"
#include "linear.cuh"
#include "pairs.cuh"

namespace fs {
namespace {

constexpr int kCols = 32, kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) k14_recurrent_kernel(const __grid_constant__ LinearArgs a) {
  constexpr int kRows = D / 16;
  const LinearSweep &w = a.sweep[blockIdx.z];
  const int b = blockIdx.y / a.H, h = blockIdx.y % a.H;
  const int tid = threadIdx.x, row = tid / 8 * kRows, col = blockIdx.x * kCols + tid % 8 * 4;
  __shared__ __align__(16) float part[2][kThreads / 32][kCols];

  f2 s[kRows][2];
  const size_t base = (size_t)blockIdx.y * D * D;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    s[r][0] = s[r][1] = 0;
    if (w.state && !w.transposed) {
      const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(w.state + base + (size_t)(row + r) * D + col);
      s[r][0] = x.x, s[r][1] = x.y;
    } else if (w.state) {
      const float *p = w.state + base + (size_t)col * D + row + r;
      s[r][0] = f2_bits(p[0], p[D]), s[r][1] = f2_bits(p[2 * D], p[3 * D]);
    }
  }
  const int n = a.count ? min(max(a.count[b], 0), a.T) : a.T;
  auto rows = [&](const LinearRows &x) {
    return static_cast<const __nv_bfloat16 *>(x.x) + b * x.s[0] + h / x.share * x.s[1];
  };
  const __nv_bfloat16 *q = rows(w.q) + row, *k = rows(w.k) + row, *v = rows(w.v) + col;
  const Factor lam = decay_power(a.decay[h], 1);
  const f2 hi = f2_bits(lam.hi, lam.hi), lo = f2_bits(lam.lo, lam.lo);
  if (w.state_mul != 1.f) {
    const f2 m = f2_bits(w.state_mul, w.state_mul);
#pragma unroll
    for (int r = 0; r < kRows; ++r) s[r][0] = mul2(s[r][0], m), s[r][1] = mul2(s[r][1], m);
  }

  for (int i = 0; i < n; ++i) {
    const long long t = w.reverse ? n - 1 - i : i;
    const uint2 vv = *reinterpret_cast<const uint2 *>(v + t * w.v.s[2]);
    uint32_t kk[kRows / 2], qq[kRows / 2];
    if constexpr (D == 128) {
      const uint4 x = *reinterpret_cast<const uint4 *>(k + t * w.k.s[2]);
      const uint4 y = *reinterpret_cast<const uint4 *>(q + t * w.q.s[2]);
      kk[0] = x.x, kk[1] = x.y, kk[2] = x.z, kk[3] = x.w;
      qq[0] = y.x, qq[1] = y.y, qq[2] = y.z, qq[3] = y.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2 *>(k + t * w.k.s[2]);
      const uint2 y = *reinterpret_cast<const uint2 *>(q + t * w.q.s[2]);
      kk[0] = x.x, kk[1] = x.y;
      qq[0] = y.x, qq[1] = y.y;
    }
    const f2 v2[2] = {wide2(vv.x), wide2(vv.y)};
    f2 o[2] = {0, 0};
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float kf = r % 2 ? bf16_hi(kk[r / 2]) : bf16_lo(kk[r / 2]);
      const float qf = r % 2 ? bf16_hi(qq[r / 2]) : bf16_lo(qq[r / 2]);
      const f2 k2 = f2_bits(kf, kf), q2 = f2_bits(qf, qf);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        f2 x = s[r][c];
        if (w.reverse) {
          x = madd2(k2, v2[c], x);
          s[r][c] = madd2(x, hi, mul2(x, lo));
        } else {
          x = s[r][c] = madd2(x, hi, madd2(x, lo, mul2(k2, v2[c])));
        }
        o[c] = madd2(q2, x, o[c]);
      }
    }
    float y[4] = {lo2(o[0]), hi2(o[0]), lo2(o[1]), hi2(o[1])};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      y[c] += __shfl_xor_sync(0xffffffffu, y[c], 8);
      y[c] += __shfl_xor_sync(0xffffffffu, y[c], 16);
    }
    if (tid % 32 < 8)
      *reinterpret_cast<float4 *>(&part[i & 1][tid / 32][tid % 32 * 4]) = make_float4(y[0], y[1], y[2], y[3]);
    __syncthreads();  // (the other half of `part` is free: its readers are past this token's barrier)
    if (tid < kCols / 2) {
      float x = 0.f, z = 0.f;
#pragma unroll
      for (int j = 0; j < kThreads / 32; ++j) {
        x += part[i & 1][j][2 * tid];
        z += part[i & 1][j][2 * tid + 1];
      }
      const long long at = b * w.os[0] + h * w.os[1] + t * w.os[2] + blockIdx.x * kCols + 2 * tid;
      x *= a.scale;
      z *= a.scale;
      if (w.out_f32)
        *reinterpret_cast<float2 *>(static_cast<float *>(w.out) + at) = make_float2(x, z);
      else
        *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(w.out) + at) = pack_bf16(x, z);
    }
  }
  if (!w.state_out) return;
  const float mul = 1.f / w.state_mul;
  const f2 m = f2_bits(mul, mul);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const f2 x = mul2(s[r][0], m), y = mul2(s[r][1], m);
    if (!w.transposed) {
      *reinterpret_cast<ulonglong2 *>(w.state_out + base + (size_t)(row + r) * D + col) = make_ulonglong2(x, y);
    } else {
      float *p = w.state_out + base + (size_t)col * D + row + r;
      p[0] = lo2(x), p[D] = hi2(x), p[2 * D] = lo2(y), p[3 * D] = hi2(y);
    }
  }
}

// Gradients of shared heads: the parts of `share` heads [batch, H, T, d] added in the heads' order.
__global__ void __launch_bounds__(256) k14_sum_kernel(const __grid_constant__ LinearSumArgs a) {
  const int per = a.d / 8;  // eight elements a thread
  const int Hkv = a.H / a.share, b = blockIdx.y / Hkv, hk = blockIdx.y % Hkv;
  const int n = a.count ? min(max(a.count[b], 0), a.T) : a.T;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long t = i / per;
  if (t >= n) return;
  const int e = (int)(i % per) * 8;
  float x[8] = {};
  for (int g = 0; g < a.share; ++g) {
    const float4 *p = reinterpret_cast<const float4 *>(
        a.part + (((size_t)b * a.H + hk * a.share + g) * a.T + t) * a.d + e);
    const float4 u = __ldg(p), w = __ldg(p + 1);
    x[0] += u.x, x[1] += u.y, x[2] += u.z, x[3] += u.w;
    x[4] += w.x, x[5] += w.y, x[6] += w.z, x[7] += w.w;
  }
  *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + b * a.os[0] + hk * a.os[1] +
                             t * a.os[2] + e) =
      make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                 pack_bf16(x[6], x[7]));
}

}  // namespace

cudaError_t launch_linear_sum(const LinearSumArgs &a, cudaStream_t st) {
  const long long blocks = ((long long)a.T * (a.d / 8) + 255) / 256;
  k14_sum_kernel<<<dim3((unsigned)blocks, a.batch * (a.H / a.share)), 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_linear_recurrent(const LinearArgs &a, cudaStream_t st) {
  const dim3 grid(a.d / kCols, a.batch * a.H, a.sweeps);
  if (a.d == 64)
    k14_recurrent_kernel<64><<<grid, kThreads, 0, st>>>(a);
  else
    k14_recurrent_kernel<128><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace fs
