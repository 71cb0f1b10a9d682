// cache.cuh -- the paged cache's formats and addressing, shared by the kernels
// that write it, read it and attend over it.
//
// Codes come from exact quotients.  With bf16 inputs Q x has at most 17
// significant bits and amax 8, so a quotient Q x / amax that is not exactly on
// a border between two codes is at least 2^-17 (relative) away from it: any
// quotient good to 2^-20 falls on the right side, and only an exact border
// needs an exact quotient, which correctly rounded division gives (the border
// is representable).
#pragma once

#include <cuda_fp8.h>

#include "fs_common.cuh"

namespace fs {

template <int F>
struct Fmt;  // bits an element, Q
template <>
struct Fmt<FS_CACHE_BF16> {
  static constexpr int kBits = 16;
};
template <>
struct Fmt<FS_CACHE_E4M3> {
  static constexpr int kBits = 8;
  static constexpr float kTop = 448.f;
};
template <>
struct Fmt<FS_CACHE_INT8> {
  static constexpr int kBits = 8;
  static constexpr float kTop = 127.f;
};
template <>
struct Fmt<FS_CACHE_INT4> {
  static constexpr int kBits = 4;
  static constexpr float kTop = 7.f;
};

// Where token `pos` of sequence b lies: index of its page, or -1 (recorded in
// the cache's status word) when the table or the cache does not reach it.
__device__ __forceinline__ int cache_page(const fs_cache &c, int b, long long pos, int *row) {
  const int shift = 31 - __clz(c.page);
  const long long blk = pos >> shift;
  *row = (int)(pos & (c.page - 1));
  int page = -1;
  if (pos >= 0 && blk < c.max_pages) page = c.table[(size_t)b * c.max_pages + (size_t)blk];
  if (page < 0 || page >= c.pages) {
    if (c.status) atomicCAS(c.status, 0, FS_ERR_CACHE);
    return -1;
  }
  return page;
}

// Index of a row (part 0: key, 1: value) among all rows of the cache.
__device__ __forceinline__ size_t cache_row(const fs_cache &c, int page, int part, int h, int row) {
  return (((size_t)page * 2 + part) * c.Hkv + h) * (size_t)c.page + row;
}

// Two codes -> two floats.
__device__ __forceinline__ float2 e4m3x2(uint32_t two) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Eight consecutive elements of a row from their packed codes (16, 8 or 4
// bytes, in the low words of `c`), not yet scaled.
template <int F>
__device__ __forceinline__ void decode8(const uint32_t (&c)[4], float (&x)[8]) {
  if constexpr (F == FS_CACHE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(c[i]);
      x[2 * i + 1] = bf16_hi(c[i]);
    }
  } else if constexpr (F == FS_CACHE_E4M3) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = e4m3x2(c[i / 2] >> (16 * (i % 2)));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else if constexpr (F == FS_CACHE_INT8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)(int8_t)(c[i / 4] >> (8 * (i % 4)));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)((int32_t)(c[0] << (28 - 4 * i)) >> 28);
  }
}

// Eight elements' code words of row `index`, element offset e (a multiple of 8).
template <int F>
__device__ __forceinline__ void load8(const fs_cache &c, size_t index, int e, uint32_t (&w)[4]) {
  constexpr int kBits = Fmt<F>::kBits;
  const char *p = static_cast<const char *>(c.codes) + (index * c.d + e) / 8 * kBits;
  if constexpr (kBits == 16) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else if constexpr (kBits == 8) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t *>(p);
  }
}

}  // namespace fs
