// 8-bit codes of the cache as f16 numbers, exactly, for the matrix units: codes 0, 1 and
// codes 2, 3 of a word of four; codes 0, 2 and codes 1, 3.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "lora_gb300.h"

namespace lgb {

// int8: a byte in the low half of 1024's bits is 1024 + that byte, so with
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
