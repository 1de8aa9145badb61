// 8-bit codes of the cache as bf16 or f16 numbers, exactly, for the matrix units.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "lora_gb300.h"

namespace lgb {

// Two int8 codes in the low bytes of x's halves (the high bytes are not looked at): 128 +
// the low seven bits, minus 128 or (sign bit set) 256, all three bf16 integers.
__device__ __forceinline__ uint32_t int8_low_to_bf16x2(uint32_t x) {
  const uint32_t a = (x & 0x007F007Fu) | 0x43004300u, b = (x & 0x00800080u) | 0x43004300u;
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
// Two e4m3 codes in the high bytes of x's halves (the low bytes are not looked at): sign,
// exponent and mantissa moved to bf16's places are the value times 2^-120, subnormals
// included (the exponent biases are 7 and 127); one exact product puts it right.
__device__ __forceinline__ uint32_t e4m3_high_to_bf16x2(uint32_t x) {
  const uint32_t a = (x & 0x80008000u) | ((x >> 4) & 0x07F007F0u), k = 0x7B807B80u;
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&k));
  return *reinterpret_cast<uint32_t*>(&r);
}

// Codes 0, 1 and codes 2, 3 of a word of four.
template <int FMT>
__device__ __forceinline__ uint32_t codes01_to_bf16x2(uint32_t w) {
  return FMT == LORA_KV_INT8 ? int8_low_to_bf16x2(__byte_perm(w, 0, 0x4140)) : e4m3_high_to_bf16x2(__byte_perm(w, 0, 0x1404));
}
template <int FMT>
__device__ __forceinline__ uint32_t codes23_to_bf16x2(uint32_t w) {
  return FMT == LORA_KV_INT8 ? int8_low_to_bf16x2(__byte_perm(w, 0, 0x4342)) : e4m3_high_to_bf16x2(__byte_perm(w, 0, 0x3424));
}
// The same as f16.  int8: a byte in the low half of 1024's bits is 1024 + that byte, so with
// the sign bit turned 1152 + the code.
__device__ __forceinline__ uint32_t int8_from_biased_f16x2(uint32_t x) {
  const uint32_t k = 0x64806480u;
  __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&k));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t two) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
}
template <int FMT>
__device__ __forceinline__ uint32_t codes01_to_f16x2(uint32_t w) {
  return FMT == LORA_KV_INT8 ? int8_from_biased_f16x2(__byte_perm(w ^ 0x80808080u, 0x64646464u, 0x4140)) : e4m3_to_f16x2(w);
}
template <int FMT>
__device__ __forceinline__ uint32_t codes23_to_f16x2(uint32_t w) {
  return FMT == LORA_KV_INT8 ? int8_from_biased_f16x2(__byte_perm(w ^ 0x80808080u, 0x64646464u, 0x4342))
                             : e4m3_to_f16x2(w >> 16);
}
template <int FMT>
__device__ __forceinline__ uint32_t codes02_to_f16x2(uint32_t w) {
  return FMT == LORA_KV_INT8 ? int8_from_biased_f16x2((w & 0x00FF00FFu) ^ 0x64806480u) : e4m3_to_f16x2(__byte_perm(w, 0, 0x4420));
}
template <int FMT>
__device__ __forceinline__ uint32_t codes13_to_f16x2(uint32_t w) {
  return FMT == LORA_KV_INT8 ? int8_from_biased_f16x2(((w >> 8) & 0x00FF00FFu) ^ 0x64806480u)
                             : e4m3_to_f16x2(__byte_perm(w, 0, 0x4431));
}

}  // namespace lgb
