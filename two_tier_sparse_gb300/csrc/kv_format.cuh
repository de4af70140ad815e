// Conversions of KV rows to and from the 4-bit cache format (DSA_KV_MXFP4):
// e2m1 codes under one power-of-two scale per 32 elements (OCP MX v1.0).
#pragma once

#include "kernels.h"

namespace dsa {

constexpr int kRow4Codes = kLatent / 2;                 // 256 bytes of codes, two a byte
constexpr int kRow4Scales = kLatent / 32;               // 16 scale bytes behind them
constexpr int kRow4Bytes = kRow4Codes + kRow4Scales;    // 272

// Bytes of one cache row of 512 elements.
__host__ __device__ constexpr int kv_row_bytes(int kv_fmt) {
  return kv_fmt == DSA_KV_MXFP4 ? kRow4Bytes : kv_fmt == DSA_KV_FP8_E4M3 ? kLatent : 2 * kLatent;
}

// The scale byte of 32 elements whose largest magnitude has the bits `amax`
// (an fp32 pattern without its sign): floor(log2 amax) - 2 above 2^-127, 2^0
// for a group of zeros, and 255 (NaN) for a group that holds a NaN or an
// infinity, whose fp32 patterns are the largest.
__device__ __forceinline__ uint32_t mx4_scale(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23);
  if (amax == 0u) return 127u;
  if (e == 255) return 255u;
  return static_cast<uint32_t>(max(e - 2, 0));
}

// 8 elements to 8 e2m1 codes, element i in bits 4 i .. 4 i + 3: each times
// 2^(127 - scale) (exact), rounded to the nearest code with ties to the even
// one, saturating at 6.
__device__ __forceinline__ uint32_t mx4_encode8(const float (&v)[8], uint32_t scale) {
  // 2^(127 - scale) in fp32; the scale is at most 252 here (255: the codes do not matter)
  const float inv = __uint_as_float((254u - min(scale, 253u)) << 23);
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 pr = make_float2(v[i] * inv, v[i + 1] * inv);
    c |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(pr, __NV_E2M1, cudaRoundNearest))
         << (4 * i);
  }
  return c;
}

// A scale byte as 2^(s - 127) in both halves of a bf16 pair: s is the exponent
// field, except 0 (2^-127, a subnormal) and 255 (NaN).
__device__ __forceinline__ uint32_t mx4_scale_bf16x2(uint32_t s) {
  const uint32_t h = s == 0u ? 0x0040u : s == 255u ? 0x7FC0u : s << 7;
  return h * 0x10001u;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;\n" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// 8 e2m1 codes times a scale (bf16 pair) to 8 bf16 values, element i in half
// i & 1 of word i / 2. Exact for scales up to 2^125: a code has two
// significant bits and bf16 the exponent range of the scale. The magnitudes
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 are looked up by byte permutes (a selector of
// three code bits picks one of the eight bytes), low and high bytes apart; the
// sign bits come from a permute whose selectors keep the codes' top bits (a
// selector with its top bit set replicates the byte's sign). About 20
// instructions for 8 elements.
__device__ __forceinline__ uint4 mx4_decode8(uint32_t c, uint32_t scale2) {
  uint32_t w[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t code = h ? c >> 16 : c;
    const uint32_t sel = code & 0x7777u;
    const uint32_t lo = prmt(0xC0800000u, 0xC0804000u, sel);
    const uint32_t sg = prmt(0x80808080u, 0x80808080u, code);  // 0xFF (negative) or 0x80
    const uint32_t hi = prmt(0x3F3F3F00u, 0x40404040u, sel) | ((sg << 1) & 0x80808080u);
    w[2 * h] = prmt(lo, hi, 0x5140u);
    w[2 * h + 1] = prmt(lo, hi, 0x7362u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]),
                                     *reinterpret_cast<const __nv_bfloat162*>(&scale2));
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace dsa
