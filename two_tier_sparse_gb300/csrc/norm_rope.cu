// Norms of queries and keys for each head, with the position rotation in the
// same pass: y = x / sqrt(mean(x^2) + eps) * w over a head's elements, then
// pairs of its rope_dim elements from rope_start on turned by the angle
// position * inv_freq. x is read once and y written once, so the pass is bound
// by memory (or, for a few tokens, by one trip through it).
//
// A CTA takes one token, or, when tokens are few, a part of a token's heads.
// A warp takes one head of more than 128 elements (lane l holds 8-element
// chunks l, l + 32, ...), or two, four ... smaller ones at a time. The angles
// are reduced to a fraction of a turn in fp64 (an fp32 product would lose the
// turn's fraction at far positions: half a radian at a million), once per token and frequency,
// and their cosines and sines shared by all heads through shared memory.
#include <algorithm>
#include <type_traits>

#include "kernels.h"

namespace dsa {

namespace {

constexpr int kWarps = 8;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
      } else {
        v[2 * i] = bf16_bits_to_float(w[i] & 0xFFFF);
        v[2 * i + 1] = bf16_bits_to_float(w[i] >> 16);
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// NV: 8-element chunks a lane holds (heads of up to 256 NV elements).
template <typename T, int NV>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  extern __shared__ float4 smem4[];
  float2* table = reinterpret_cast<float2*>(smem4);  // (cos, sin) of each pair, at the token
  griddep_wait();
  const int tok = blockIdx.x;
  if (a.n_valid && tok >= *a.n_valid) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pairs = a.pairs;
  if (pairs > 0) {
    const double pos = static_cast<double>(a.positions[tok]);
    for (int i = tid; i < pairs; i += 32 * kWarps) {
      const double turns = pos * a.inv_freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
      const float frac = static_cast<float>(turns - rint(turns));
      float s, c;
      sincospif(2.f * frac, &s, &c);
      table[i] = make_float2(c * a.rope_scale, s * a.rope_scale);
    }
    __syncthreads();
  }
  float* stage = reinterpret_cast<float*>(table + pairs) + warp * 256 * NV;  // halves rotated: a warp's rows
  const int first = blockIdx.y * a.units_per_cta;
  const int last = min(a.units, first + a.units_per_cta);
  int seg = 0;
  for (int u = first + warp; u < last; u += kWarps) {
    while (u >= a.seg[seg].unit_end) ++seg;
    const NormRopeSeg& sg = a.seg[seg];
    const int lanes = 1 << sg.lanes_log2;  // lanes of a head
    const int head = ((u - (seg ? a.seg[seg - 1].unit_end : 0)) << (5 - sg.lanes_log2)) +
                     (lane >> sg.lanes_log2);
    const int l = lane & (lanes - 1);
    const bool on = head < sg.heads;
    const T* x = static_cast<const T*>(sg.x) + tok * sg.x_token_stride + head * sg.x_head_stride;
    float v[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int e = 8 * (l + lanes * c);
      if (on && e < sg.dim) {
        load8(x + e, v[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[c][i], v[c][i], ss);
      }
    }
    if (sg.norm) {
      for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      const float r = rsqrtf(ss * sg.inv_dim + sg.eps);
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const int e = 8 * (l + lanes * c);
        if (on && e < sg.dim) {
          if (sg.weight) {
            float w[8];
            load8(sg.weight + e, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] *= r * w[i];
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] *= r;
          }
        }
      }
    }
    if (sg.rope) {
      const int rd = 2 * pairs;
      if (a.interleaved) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const int e = 8 * (l + lanes * c) - sg.rope_start;
          if (e >= 0 && e < rd) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 t = table[(e >> 1) + i];
              const float x0 = v[c][2 * i], x1 = v[c][2 * i + 1];
              v[c][2 * i] = x0 * t.x - x1 * t.y;
              v[c][2 * i + 1] = x0 * t.y + x1 * t.x;
            }
          }
        }
      } else {
        // element i and element i + rope_dim / 2 turn together: through shared memory
        float* mine = stage + (lane >> sg.lanes_log2) * rd;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const int e = 8 * (l + lanes * c) - sg.rope_start;
          if (e >= 0 && e < rd) store8(mine + e, v[c]);
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const int e = 8 * (l + lanes * c) - sg.rope_start;
          if (e >= 0 && e < rd) {
            const bool low = e < pairs;
            float other[8];
            load8(mine + (low ? e + pairs : e - pairs), other);
            const int p0 = low ? e : e - pairs;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 t = table[p0 + i];
              v[c][i] = low ? v[c][i] * t.x - other[i] * t.y : other[i] * t.y + v[c][i] * t.x;
            }
          }
        }
        __syncwarp();
      }
    }
    T* y = static_cast<T*>(sg.out) + tok * sg.out_token_stride + head * sg.out_head_stride;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int e = 8 * (l + lanes * c);
      if (on && e < sg.dim) store8(y + e, v[c]);
    }
  }
}

template <typename T, int NV>
cudaError_t launch_nv(const NormRopeArgs& a, dim3 grid, cudaStream_t s) {
  const int smem = a.pairs * 8 + (a.pairs && !a.interleaved ? kWarps * 256 * NV * 4 : 0);
  static std::atomic<int> smem_set[64]{};
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(norm_rope_kernel<T, NV>),
                              kWarps * 256 * NV * 4 + 4096 * 2, smem_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_rope_kernel<T, NV>, grid, dim3(32 * kWarps), static_cast<size_t>(smem), s, 1,
                    a);
}

template <typename T>
cudaError_t launch_t(const NormRopeArgs& a, int max_dim, dim3 grid, cudaStream_t s) {
  if (max_dim <= 256) return launch_nv<T, 1>(a, grid, s);
  if (max_dim <= 512) return launch_nv<T, 2>(a, grid, s);
  return launch_nv<T, 4>(a, grid, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& args, int dtype, int max_dim, cudaStream_t s) {
  if (args.n == 0 || args.units == 0) return cudaSuccess;
  NormRopeArgs a = args;
  // A token's heads are shared out while tokens alone do not give every SM two CTAs.
  const int want = (2 * device_sm_count() + a.n - 1) / a.n;
  const int parts = std::max(1, std::min(want, (a.units + kWarps - 1) / kWarps));
  a.units_per_cta = (a.units + parts - 1) / parts;
  const dim3 grid(a.n, (a.units + a.units_per_cta - 1) / a.units_per_cta);
  switch (dtype) {
    case DSA_DT_BF16: return launch_t<uint16_t>(a, max_dim, grid, s);
    case DSA_DT_F16: return launch_t<__half>(a, max_dim, grid, s);
    default: return launch_t<float>(a, max_dim, grid, s);
  }
}

}  // namespace dsa
