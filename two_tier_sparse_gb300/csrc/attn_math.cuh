// Softmax arithmetic of one tile of attention scores, shared by the attention
// kernels: a thread holds one query head's scores of the tile.
#pragma once

#include "kernels.h"

namespace dsa {

// A tile's raw scores of this thread's head (TMEM columns [addr, addr + R)),
// -inf past the tile's valid rows: one TMEM load, one wait. The softmax scale
// (positive) is applied by max_scores and exp_pack.
template <int R>
__device__ __forceinline__ void load_scores(uint32_t addr, int valid, float (&z)[R]) {
  if constexpr (R == 64) {
    tmem_ld64(addr, z);
  } else {
    static_assert(R == 32, "tile rows");
    tmem_ld32(addr, z);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) z[i] = i < valid ? z[i] : -INFINITY;
}
// scale * max_i z[i] (log2 units; equal to max_i (scale * z[i]) for scale > 0),
// the maximum as four independent chains
template <int R>
__device__ __forceinline__ float max_scores(const float (&z)[R], float scale) {
  float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < R; ++i) m4[i & 3] = fmaxf(m4[i & 3], z[i]);
  return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale;
}
// 2^x by the ex2 instruction (flushing subnormal results to zero: a
// probability below 2^-126 of the running maximum's is dropped)
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// p_i = 2^(scale z_i - m) (one fused multiply-add a score) packed as bf16
// pairs into pk; returns sum_i p_i over the fp32 probabilities (four partial
// sums)
template <int R, bool F16 = false>
__device__ __forceinline__ float exp_pack(const float (&z)[R], float scale, float m,
                                          uint32_t (&pk)[R / 2]) {
  float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < R; i += 2) {
    const float p0 = ex2_ftz(fmaf(z[i], scale, -m)), p1 = ex2_ftz(fmaf(z[i + 1], scale, -m));
    s4[(i >> 1) & 3] += p0 + p1;
    if constexpr (F16) {  // the PV operands of an fp8 cache are f16
      const __half2 p2 = __floats2half2_rn(p0, p1);
      pk[i / 2] = *reinterpret_cast<const uint32_t*>(&p2);
    } else {
      const __nv_bfloat162 p2 = __floats2bfloat162_rn(p0, p1);
      pk[i / 2] = *reinterpret_cast<const uint32_t*>(&p2);
    }
  }
  return (s4[0] + s4[1]) + (s4[2] + s4[3]);
}

}  // namespace dsa
