// k12_tree.cu -- attention of drafted tokens over the paged cache
// (fs_tree_attn).
#include "cache.cuh"

namespace fs {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// One block per (row, query head, sequence): tiles of 128 keys, a thread a key
// for the scores, then a thread a dimension for the values.
template <int F, int D>
__global__ void __launch_bounds__(128) k12_simple_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ float q[D], p[128], red[4];
  __shared__ long long at[128];
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int n = a.count ? min(a.count[b], a.T) : a.T;
  if (i >= n) return;
  const int G = a.H / a.c.Hkv, kvh = h / G;
  const long long past = max(a.past[b], 0);
  uint64_t bits = a.tree ? (uint64_t)a.tree[(size_t)b * a.T + i] : ~0ull >> (63 - i);
  if (n < 64) bits &= (1ull << n) - 1;
  long long first = 0;
  if (a.window) first = max(0ll, past + __popcll(bits) - a.window);
  const size_t qrow = (((size_t)b * a.H + h) * a.T + i) * D;
  if (tid < D) q[tid] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[qrow + tid]) *
                        (a.scale * kLog2e);
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (long long base = first; base < past + n; base += 128) {
    __syncthreads();
    const long long key = base + tid;
    float s = -INFINITY;
    int off = 0, page = -1;
    if (key < past + n && (key < past || (bits >> (key - past) & 1)))
      page = cache_page(a.c, b, key, &off);
    at[tid] = -1;
    if (page >= 0) {
      const size_t row = cache_row(a.c, page, 0, kvh, off);
      at[tid] = (long long)cache_row(a.c, page, 1, kvh, off);
      s = 0.f;
      for (int e = 0; e < D; e += 8) {
        uint32_t w[4];
        float x[8];
        load8<F>(a.c, row, e, w);
        decode8<F>(w, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) s += x[j] * q[e + j];
      }
      if constexpr (F != FS_CACHE_BF16) s *= a.c.scales[row];
    }
    float t = s;
    for (int o2 = 16; o2 > 0; o2 >>= 1) t = fmaxf(t, __shfl_xor_sync(~0u, t, o2));
    if (tid % 32 == 0) red[tid / 32] = t;
    __syncthreads();
    const float mt = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float ref = mt == -INFINITY ? 0.f : mt;
    p[tid] = at[tid] >= 0 ? exp2f(s - ref) : 0.f;
    const float back = exp2f(m - ref);
    m = mt;
    l *= back;
    o *= back;
    __syncthreads();
    for (int j = 0; j < 128; ++j) {
      const long long row = at[j];
      if (row < 0) continue;
      l += p[j];
      if (tid < D) {
        uint32_t w[4];
        float x[8];
        load8<F>(a.c, row, tid & ~7, w);
        decode8<F>(w, x);
        float v = x[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) v = (tid & 7) == e ? x[e] : v;
        if constexpr (F != FS_CACHE_BF16) v *= a.c.scales[row];
        o += p[j] * v;
      }
    }
  }
  if (tid < D)
    static_cast<__nv_bfloat16 *>(a.out)[qrow + tid] = __float2bfloat16_rn(l > 0.f ? o / l : (l == 0.f ? 0.f : l));
}

template <int D>
cudaError_t launch_simple(const TreeArgs &a, cudaStream_t st) {
  const dim3 grid(a.T, a.H, a.c.batch);
  switch (a.c.format) {
    case FS_CACHE_BF16: k12_simple_kernel<FS_CACHE_BF16, D><<<grid, 128, 0, st>>>(a); break;
    case FS_CACHE_E4M3: k12_simple_kernel<FS_CACHE_E4M3, D><<<grid, 128, 0, st>>>(a); break;
    case FS_CACHE_INT8: k12_simple_kernel<FS_CACHE_INT8, D><<<grid, 128, 0, st>>>(a); break;
    default: k12_simple_kernel<FS_CACHE_INT4, D><<<grid, 128, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace

size_t tree_workspace_bytes(const fs_cache &, int, int) { return 256; }

cudaError_t launch_tree(const TreeArgs &a, cudaStream_t st) {
  return a.c.d == 64 ? launch_simple<64>(a, st) : launch_simple<128>(a, st);
}

}  // namespace fs
