// 8-bit codes of the cache as bf16 numbers, exactly, for the matrix units.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "lora_gb300.h"

namespace lgb {

// Two codes in the low bytes of x's halves (whose high bytes are not looked at) -> their
// values as bf16, exact.
__device__ __forceinline__ uint32_t int8_to_bf16x2(uint32_t x) {
  // 128 + low seven bits, minus 128 or (sign bit set) 256: all three are bf16 integers
  const uint32_t a = (x & 0x007F007Fu) | 0x43004300u, b = (x & 0x00800080u) | 0x43004300u;
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t e4m3_to_bf16x2(uint32_t x) {
  // sign, exponent and mantissa moved to bf16's places: the value times 2^-120, subnormals
  // included (the exponent biases are 7 and 127); one exact product puts it right
  const uint32_t a = ((x << 8) & 0x80008000u) | ((x << 4) & 0x07F007F0u), k = 0x7B807B80u;
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&k));
  return *reinterpret_cast<uint32_t*>(&r);
}
template <int FMT>
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t x) {
  return FMT == LORA_KV_INT8 ? int8_to_bf16x2(x) : e4m3_to_bf16x2(x);
}

}  // namespace lgb
