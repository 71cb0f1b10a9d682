// k14_linear.cu -- linear attention with a decay for each head, token by token.
//
//   S_t = lam S_{t-1} + k_t v_t^T,   out_t = scale q_t S_t,   lam = exp(decay)
//
// The columns of S (the elements of v and out) do not meet, so a block takes
// kCols of them: d x kCols of the state in registers, four columns and
// d / kTeams rows a thread.  For a decoding step the state's bytes are
// everything (read once, written once: 2 x 4 d^2 bytes against 8 d bytes of
// rows), so all of a thread's state is under way before anything is computed.
// lam goes in as two fp32 numbers (linear.cuh): as one it would be off by up to
// 2^-25 in the same direction at every token, and a head with a long memory adds
// that up over thousands of them.
#include "fs_common.cuh"
#include "fs_internal.h"
#include "linear.cuh"

namespace fs {
namespace {

constexpr int kCols = 16, kThreads = 256, kTeams = kThreads / (kCols / 4);

template <int D>
__global__ void __launch_bounds__(kThreads) k14_recurrent_kernel(const __grid_constant__ LinearArgs a) {
  constexpr int kRows = D / kTeams;
  const LinearSweep &w = a.sweep[blockIdx.z];
  const int b = blockIdx.y / a.H, h = blockIdx.y % a.H;
  const int n = a.count ? min(max(a.count[b], 0), a.T) : a.T;
  const int tid = threadIdx.x, row = tid / (kCols / 4) * kRows;
  const int col = blockIdx.x * kCols + tid % (kCols / 4) * 4;
  __shared__ float part[2][kThreads / 32][kCols];

  float s[kRows][4];
  const size_t base = (size_t)blockIdx.y * D * D;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (w.state && !w.transposed) {
      x = *reinterpret_cast<const float4 *>(w.state + base + (size_t)(row + r) * D + col);
    } else if (w.state) {
      const float *p = w.state + base + (size_t)col * D + row + r;
      x = make_float4(p[0], p[D], p[2 * D], p[3 * D]);
    }
    s[r][0] = x.x * w.state_mul;
    s[r][1] = x.y * w.state_mul;
    s[r][2] = x.z * w.state_mul;
    s[r][3] = x.w * w.state_mul;
  }
  auto rows = [&](const LinearRows &x) {
    return static_cast<const __nv_bfloat16 *>(x.x) + b * x.s[0] + h / x.share * x.s[1];
  };
  const __nv_bfloat16 *q = rows(w.q), *k = rows(w.k), *v = rows(w.v);
  const Factor lam = decay_power(a.decay[h], 1);

  for (int i = 0; i < n; ++i) {
    const long long t = w.reverse ? n - 1 - i : i;
    const uint2 vv = *reinterpret_cast<const uint2 *>(v + t * w.v.s[2] + col);
    const float vf[4] = {bf16_lo(vv.x), bf16_hi(vv.x), bf16_lo(vv.y), bf16_hi(vv.y)};
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float kf = __bfloat162float(k[t * w.k.s[2] + row + r]);
      const float qf = __bfloat162float(q[t * w.q.s[2] + row + r]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float kv = kf * vf[c];
        const float x = w.reverse ? s[r][c] + kv : lam.times(s[r][c], kv);
        o[c] = fmaf(qf, x, o[c]);
        s[r][c] = w.reverse ? lam.times(x, 0.f) : x;
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int m = kCols / 4; m < 32; m *= 2) o[c] += __shfl_xor_sync(0xffffffffu, o[c], m);
    if (tid % 32 < kCols / 4)
      *reinterpret_cast<float4 *>(&part[i & 1][tid / 32][tid % 32 * 4]) =
          make_float4(o[0], o[1], o[2], o[3]);
    __syncthreads();  // (the other half of `part` is free: its readers are past this token's barrier)
    if (tid < kCols / 2) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int j = 0; j < kThreads / 32; ++j) {
        x += part[i & 1][j][2 * tid];
        y += part[i & 1][j][2 * tid + 1];
      }
      const long long at = b * w.os[0] + h * w.os[1] + t * w.os[2] + blockIdx.x * kCols + 2 * tid;
      x *= a.scale;
      y *= a.scale;
      if (w.out_f32)
        *reinterpret_cast<float2 *>(static_cast<float *>(w.out) + at) = make_float2(x, y);
      else
        *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(w.out) + at) = pack_bf16(x, y);
    }
  }
  if (!w.state_out) return;
  const float mul = 1.f / w.state_mul;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float4 x = make_float4(s[r][0] * mul, s[r][1] * mul, s[r][2] * mul, s[r][3] * mul);
    if (!w.transposed) {
      *reinterpret_cast<float4 *>(w.state_out + base + (size_t)(row + r) * D + col) = x;
    } else {
      float *p = w.state_out + base + (size_t)col * D + row + r;
      p[0] = x.x, p[D] = x.y, p[2 * D] = x.z, p[3 * D] = x.w;
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
