// cache.cuh -- the paged cache's formats and addressing, shared by the kernels
// that write it, read it and attend over it.
#pragma once

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

// Four e4m3 codes -> two fp16 pairs.
__device__ __forceinline__ void e4m3_h2(uint32_t w, uint32_t &a, uint32_t &b) {
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n"
      " cvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
      : "=r"(a), "=r"(b)
      : "r"(w));
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
    for (int i = 0; i < 2; ++i) {
      uint32_t h[2];
      e4m3_h2(c[i], h[0], h[1]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        x[4 * i + 2 * j] = f.x;
        x[4 * i + 2 * j + 1] = f.y;
      }
    }
  } else if constexpr (F == FS_CACHE_INT8) {
    // 2^23 + (code + 128), an exact fp32 number, less 2^23 + 128
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = __uint_as_float(__byte_perm(c[i / 4] ^ 0x80808080u, 0x4b000000u, 0x7440 + i % 4)) -
             8388736.f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = __uint_as_float((c[0] >> (4 * i) & 15u) ^ 0x4b000008u) - 8388616.f;
  }
}

}  // namespace fs
