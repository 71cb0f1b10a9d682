// pairs.cuh -- pairs of fp32 numbers in one register pair (one instruction for two on
// this architecture), and pairs of bf16.
#pragma once

#include "fs_common.cuh"

namespace fs {

using f2 = unsigned long long;

__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 madd2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 add2_bits(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float lo2(f2 x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi2(f2 x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint32_t pack2(f2 x) { return pack_bf16(lo2(x), hi2(x)); }
__device__ __forceinline__ f2 wide2(uint32_t pair) {  // two bf16
  return (f2)(pair << 16) | (f2)(pair & 0xffff0000u) << 32;
}
// The nearest bf16 pair; x becomes what is left.
__device__ __forceinline__ uint32_t split2(f2 &x) {
  const uint32_t h = pack2(x);
  x = sub2_bits(x, wide2(h));
  return h;
}

}  // namespace fs
