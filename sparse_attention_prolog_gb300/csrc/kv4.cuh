// Layout of the 4-bit latent cache row and its conversion to bf16, shared by
// the kernels that write, read and attend over it.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

namespace dsa {

constexpr int kKv4Row = 416;                      // bytes of a row
constexpr int kKv4Scales = 256, kKv4Rope = 288;   // byte offsets of the scale bytes and the rotary dims

// The scale of byte u enters the conversion as 16 s and -24 s, each twice in
// a register.  s = (1 + m/8) 2^(e-15) with u = 8e + m, so the bits of 16 s in
// bf16 are (u << 4) + (116 << 7): one multiply-add makes both halves.  -24 s =
// -1.5 * 16 s has at most 6 significant bits.  u = 255 stands for NaN.
struct Kv4Scale {
  uint32_t s16, m24;
};
__device__ __forceinline__ Kv4Scale kv4_scale(uint32_t u) {
  Kv4Scale r;
  r.s16 = u == 255u ? 0x7fc07fc0u : u * 0x00100010u + 0x3a003a00u;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r.m24) : "r"(r.s16), "r"(0xbfc0bfc0u));  // * -1.5
  return r;
}

// Four bytes of codes (8 dims) -> 8 bf16 in dim order.  A nibble c (two's
// complement, sign bit flipped) placed in mantissa bits 3..6 of 1.0 reads as
// 1.5 + c/16; one fused multiply-add with 16 s and -24 s gives c s, which bf16
// holds exactly: per pair of dims a shift, a three-input logic operation and
// the multiply-add.
__device__ __forceinline__ uint4 kv4_codes8(uint32_t w, const Kv4Scale& s) {
  uint32_t r[4];
  const uint32_t sh[4] = {w << 3, w >> 1, w >> 5, w >> 9};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t v = (sh[i] & 0x00780078u) ^ 0x3fc03fc0u;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r[i]) : "r"(v), "r"(s.s16), "r"(s.m24));
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace dsa
