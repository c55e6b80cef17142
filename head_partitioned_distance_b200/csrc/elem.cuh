// elem.cuh -- the two 16-bit element types of the query/key norm and of the
// paged cache: unpacking, packing, and the store of an fp32 row as 16 bits.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace spa {

struct Bf16 {
  static constexpr uint32_t kMmaFormat = 1;  // tcgen05 kind::f16 operand format
  static constexpr bool kIsBf16 = true;
  __device__ __forceinline__ static float2 unpack(uint32_t v) { return ptx::bf16x2_to_float2(v); }
  // round to nearest even; `lo` at the lower address
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) { return ptx::pack_bf16x2(lo, hi); }
};

struct Fp16 {
  static constexpr uint32_t kMmaFormat = 0;
  static constexpr bool kIsBf16 = false;
  __device__ __forceinline__ static float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// 32 fp32 values times `mul` -> 32 16-bit values at `dst` (64 bytes, 32-byte
// aligned).
template <class E>
__device__ __forceinline__ void store_row32(uint16_t* dst, const uint32_t (&g)[32], float mul) {
  uint32_t pk[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) pk[e] = E::pack(__uint_as_float(g[2 * e]) * mul, __uint_as_float(g[2 * e + 1]) * mul);
  ptx::st_global_v8(dst, pk);
  ptx::st_global_v8(dst + 16, pk + 8);
}

}  // namespace spa
