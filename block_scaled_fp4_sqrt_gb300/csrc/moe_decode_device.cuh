// Device helpers of the decode-step operators.
#pragma once

#include "moe_decode_internal.h"
#include "moe_device.cuh"

namespace moe {

// Eight values times mul as E4M3 codes (round to nearest even, saturating), value i in byte i.
__device__ __forceinline__ uint2 e4m3_8(const float (&v)[8], float mul) {
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = e4m3x2(v[2 * i] * mul, v[2 * i + 1] * mul);
  return make_uint2((uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16));
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&v)[8]) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  return u;
}

// The largest magnitude of eight values as fp32 bits: above every finite value for infinities, and above those for NaN.
__device__ __forceinline__ uint32_t abs_max_bits(const float (&v)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return top;
}

// Eight values of an MXFP4 block whose largest magnitude is top (abs_max_bits over the block): their codes, value i in bits
// 4 i .., and the block's scale byte.  E2M1 has neither infinities nor NaN: a block that holds one gets the byte 255, which
// reads as NaN, and codes 0.
__device__ __forceinline__ uint8_t mxfp4_quad(const float (&v)[8], uint32_t top, uint32_t& codes) {
  const bool finite = top < 0x7F800000u;
  const int e = finite ? mxfp4_block_exp(__uint_as_float(top)) : 0;
  const float mul = exp2_neg_int(e);
  codes = e2m1x8(v[0] * mul, v[1] * mul, v[2] * mul, v[3] * mul, v[4] * mul, v[5] * mul, v[6] * mul, v[7] * mul);
  if (!finite) codes = 0;
  return finite ? (uint8_t)(e + 127) : (uint8_t)255;
}

// E8M0 byte j of w as a float, exact: two bytes at a time become bf16, which holds 2^-127 (byte 0) as a subnormal number.
// (Shifts and masks read byte 0 as 0, and one instruction more to mend that costs the few-token layer 9 % at one token and
// 3 % at eight, the attention 1 %: the conversion costs neither.)
__device__ __forceinline__ float e8m0_float(uint32_t w, int j) {
  uint32_t pair;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(pair) : "h"((uint16_t)(j & 2 ? w >> 16 : w)));
  return __uint_as_float(j & 1 ? pair & 0xFFFF0000u : pair << 16);
}

// n / page_size and n % page_size for 0 <= n < 2^31 (PageDiv, moe_decode_internal.h).
__device__ __forceinline__ int page_of(int n, PageDiv d, int page_size, int* row) {
  const int p = d.mul ? (int)(__umulhi((uint32_t)n, d.mul) >> d.shift) : n;
  *row = n - p * page_size;
  return p;
}

// The length of request b, clamped to what its block table can hold.
__device__ __forceinline__ int seq_len_of(const moe_kv_cache_t& c, int b) {
  const int n = __ldg(c.seq_lens + b);
  const int cap = c.max_pages * c.page_size;
  if (n >= 0 && n <= cap) return n;
  set_status(c.status, MOE_KV_BAD_LENGTH);
  return n < 0 ? 0 : cap;
}

}  // namespace moe
