// k11_cache.cu -- writing rows into the paged cache (fs_cache_append), reading
// them back (fs_cache_read) and moving the rows of an accepted path
// (fs_cache_accept).
//
// A row of d elements belongs to d / 8 neighbouring lanes, eight elements (one
// 16-byte piece of bf16) each; the row's largest magnitude is a shuffle
// reduction over them.  Bound by memory (append: 2 d bytes in, d bits / 8 + 4
// out a row; read: the other way).
#include "cache.cuh"

namespace fs {
namespace {

// Token, head and part of a row, tokens running fastest (rows of one head lie
// together in the input and inside a page).
struct RowId {
  int b, h, part, t;
};
__device__ __forceinline__ RowId row_id(unsigned row, int T, int Hkv) {
  RowId r;
  const unsigned bhp = row / (unsigned)T;
  r.t = (int)(row - bhp * T);
  r.part = (int)(bhp & 1);
  const unsigned bh = bhp >> 1;
  r.b = (int)(bh / (unsigned)Hkv);
  r.h = (int)(bh - (unsigned)r.b * Hkv);
  return r;
}

template <int F>
__device__ __forceinline__ void encode8(const uint32_t (&x)[4], float amax, uint32_t (&w)[4]) {
  if constexpr (F == FS_CACHE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = x[i];
  } else {
    constexpr float Q = Fmt<F>::kTop;
    // Q x must not pass the fp32 range; the quotient is the same with both
    // sides scaled by a power of two (an x that this flushes has code 0).
    const float pre = amax > 0x1p64f ? 0x1p-32f : 1.f;
    const bool zero = !(amax > 0.f) || !(amax <= 3.4028235e38f);
    const float den = amax * pre;
    w[0] = w[1] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = 0.f, b = 0.f;
      if (!zero) {
        a = __fdiv_rn(bf16_lo(x[i]) * pre * Q, den);
        b = __fdiv_rn(bf16_hi(x[i]) * pre * Q, den);
      }
      if constexpr (F == FS_CACHE_E4M3) {
        const uint32_t two =
            __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        w[i / 2] |= two << (16 * (i % 2));
      } else if constexpr (F == FS_CACHE_INT8) {
        const uint32_t two = ((uint32_t)__float2int_rn(a) & 255u) |
                             (((uint32_t)__float2int_rn(b) & 255u) << 8);
        w[i / 2] |= two << (16 * (i % 2));
      } else {
        const uint32_t two = ((uint32_t)__float2int_rn(a) & 15u) |
                             (((uint32_t)__float2int_rn(b) & 15u) << 4);
        w[0] |= two << (8 * i);
      }
    }
  }
}

template <int F>
__device__ __forceinline__ void store8(const fs_cache &c, size_t index, int e,
                                       const uint32_t (&w)[4]) {
  constexpr int kBits = Fmt<F>::kBits;
  char *p = static_cast<char *>(c.codes) + (index * c.d + e) / 8 * kBits;
  if constexpr (kBits == 16)
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else if constexpr (kBits == 8)
    *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t *>(p) = w[0];
}

// L = d / 8 lanes a row.  Whole groups of lanes take part or not, and every
// lane reaches the shuffles.
template <int F, int L>
__global__ void __launch_bounds__(256) k11_append_kernel(const __grid_constant__ CacheRowsArgs a) {
  const unsigned row = (blockIdx.x * 256u + threadIdx.x) / L;
  const int lane = threadIdx.x % L;
  const RowId r = row_id(row, a.T, a.c.Hkv);
  bool live = r.b < a.c.batch;
  if (live && a.count) live = r.t < a.count[r.b];
  int page = -1, off = 0;
  if (live) page = cache_page(a.c, r.b, (long long)a.start[r.b] + r.t, &off);
  live = page >= 0;
  uint32_t x[4] = {0, 0, 0, 0}, w[4];
  if (live) {
    const long long(&s)[3] = r.part ? a.vs : a.ks;
    const uint16_t *p = static_cast<const uint16_t *>(r.part ? a.v : a.k) + r.b * s[0] +
                        r.h * s[1] + r.t * s[2] + lane * 8;
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
  }
  float amax = 0.f;
  if constexpr (F != FS_CACHE_BF16) {
    // Magnitudes of bf16 compare as integers, NaN above infinity.
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(x[i] << 16 & 0x7fffffffu, x[i] & 0x7fff0000u));
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    amax = __uint_as_float(m);
  }
  if (!live) return;
  encode8<F>(x, amax, w);
  const size_t index = cache_row(a.c, page, r.part, r.h, off);
  store8<F>(a.c, index, lane * 8, w);
  if constexpr (F != FS_CACHE_BF16) {
    if (lane == 0)
      a.c.scales[index] = amax <= 3.4028235e38f ? __fdiv_rn(amax, Fmt<F>::kTop)
                                                : __uint_as_float(0x7fc00000u);
  }
}

template <int F, int L, bool F32>
__global__ void __launch_bounds__(256) k11_read_kernel(const __grid_constant__ CacheRowsArgs a) {
  const unsigned row = (blockIdx.x * 256u + threadIdx.x) / L;
  const int lane = threadIdx.x % L;
  const RowId r = row_id(row, a.T, a.c.Hkv);
  if (r.b >= a.c.batch || (a.count && r.t >= a.count[r.b])) return;
  int off;
  const int page = cache_page(a.c, r.b, (long long)a.start[r.b] + r.t, &off);
  if (page < 0) return;
  const size_t index = cache_row(a.c, page, r.part, r.h, off);
  uint32_t w[4];
  load8<F>(a.c, index, lane * 8, w);
  const size_t at = (((size_t)r.b * a.c.Hkv + r.h) * a.T + r.t) * (L * 8) + lane * 8;
  void *out = r.part ? a.v_out : a.k_out;
  if constexpr (F == FS_CACHE_BF16 && !F32) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
  float x[8];
  decode8<F>(w, x);
  if constexpr (F != FS_CACHE_BF16) {
    const float s = a.c.scales[index];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= s;
  }
  if constexpr (F32) {
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
    o[0] = make_float4(x[0], x[1], x[2], x[3]);
    o[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                   pack_bf16(x[6], x[7]));
  }
}

// One block per (sequence, kv head, part): all source rows into shared memory,
// then out again.  At most 64 rows of 256 bytes.
__global__ void __launch_bounds__(256) k11_accept_kernel(const __grid_constant__ CacheRowsArgs a,
                                                         int words) {
  __shared__ uint4 rows[64 * 16];
  __shared__ float scale[64];
  __shared__ long long to[64];
  const int part = blockIdx.x & 1, h = (blockIdx.x >> 1) % a.c.Hkv, b = (blockIdx.x >> 1) / a.c.Hkv;
  const int n = a.count ? min(a.count[b], a.T) : a.T;
  uint4 *codes = static_cast<uint4 *>(a.c.codes);
  for (int i = threadIdx.x / 16; i < n; i += 16) {
    const int lane = threadIdx.x % 16;
    const int from = a.path[(size_t)b * a.T + i];
    int src_off, dst_off, src = -1, dst = -1;
    if (from >= 0 && from < 64) {
      src = cache_page(a.c, b, (long long)a.start[b] + from, &src_off);
      dst = cache_page(a.c, b, (long long)a.start[b] + i, &dst_off);
    } else if (a.c.status) {
      atomicCAS(a.c.status, 0, FS_ERR_CACHE);
    }
    const bool ok = src >= 0 && dst >= 0;
    if (ok) {
      const size_t index = cache_row(a.c, src, part, h, src_off);
      if (lane < words) rows[i * 16 + lane] = codes[index * words + lane];
      if (lane == 0 && a.c.format != FS_CACHE_BF16) scale[i] = a.c.scales[index];
    }
    if (lane == 0) to[i] = ok ? (long long)cache_row(a.c, dst, part, h, dst_off) : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x / 16; i < n; i += 16) {
    const int lane = threadIdx.x % 16;
    if (to[i] < 0) continue;
    if (lane < words) codes[(size_t)to[i] * words + lane] = rows[i * 16 + lane];
    if (lane == 0 && a.c.format != FS_CACHE_BF16) a.c.scales[to[i]] = scale[i];
  }
}

template <int L>
cudaError_t append(const CacheRowsArgs &a, unsigned blocks, cudaStream_t st) {
  switch (a.c.format) {
    case FS_CACHE_BF16: k11_append_kernel<FS_CACHE_BF16, L><<<blocks, 256, 0, st>>>(a); break;
    case FS_CACHE_E4M3: k11_append_kernel<FS_CACHE_E4M3, L><<<blocks, 256, 0, st>>>(a); break;
    case FS_CACHE_INT8: k11_append_kernel<FS_CACHE_INT8, L><<<blocks, 256, 0, st>>>(a); break;
    default: k11_append_kernel<FS_CACHE_INT4, L><<<blocks, 256, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

template <int L, bool F32>
cudaError_t read(const CacheRowsArgs &a, unsigned blocks, cudaStream_t st) {
  switch (a.c.format) {
    case FS_CACHE_BF16: k11_read_kernel<FS_CACHE_BF16, L, F32><<<blocks, 256, 0, st>>>(a); break;
    case FS_CACHE_E4M3: k11_read_kernel<FS_CACHE_E4M3, L, F32><<<blocks, 256, 0, st>>>(a); break;
    case FS_CACHE_INT8: k11_read_kernel<FS_CACHE_INT8, L, F32><<<blocks, 256, 0, st>>>(a); break;
    default: k11_read_kernel<FS_CACHE_INT4, L, F32><<<blocks, 256, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

// Blocks of 256 threads for the call's rows, d / 8 lanes each (below 2^32
// threads: checked by the caller).
unsigned row_blocks(const CacheRowsArgs &a) {
  const size_t threads = (size_t)a.c.batch * a.c.Hkv * 2 * a.T * (a.c.d / 8);
  return (unsigned)((threads + 255) / 256);
}

}  // namespace

cudaError_t launch_cache_append(const CacheRowsArgs &a, cudaStream_t st) {
  return a.c.d == 64 ? append<8>(a, row_blocks(a), st) : append<16>(a, row_blocks(a), st);
}

cudaError_t launch_cache_read(const CacheRowsArgs &a, cudaStream_t st) {
  const unsigned blocks = row_blocks(a);
  if (a.c.d == 64) return a.f32 ? read<8, true>(a, blocks, st) : read<8, false>(a, blocks, st);
  return a.f32 ? read<16, true>(a, blocks, st) : read<16, false>(a, blocks, st);
}

cudaError_t launch_cache_accept(const CacheRowsArgs &a, cudaStream_t st) {
  const int words = (int)(fs_cache_row_bytes(a.c.d, a.c.format) / 16);
  k11_accept_kernel<<<(unsigned)(a.c.batch * a.c.Hkv * 2), 256, 0, st>>>(a, words);
  return cudaGetLastError();
}

}  // namespace fs
