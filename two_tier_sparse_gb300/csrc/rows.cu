// KV rows to and from a cache through a slot map (the rows of a paged pool, or
// of the window buffer): one warp per row. Lane l holds elements [8 l, 8 l + 8)
// and [256 + 8 l, 256 + 8 l + 8), so every access of a warp is contiguous and
// a 32-element scale group is four neighbouring lanes. Bound by memory: 65536 rows to slots
// in any order take 15.5 us as MXFP4 (5.5 TB/s), 20.6 as E4M3 (4.9, its conversion in part), 22.3 as
// bf16 (6.0); out of the cache 16.0, 17.7 and 22.5. All 64 warps of an SM have a row on its way (48 to
// E4M3, whose quotients take 35 registers):
// with half of them MXFP4 takes 19.9 us.
#include <algorithm>

#include "kv_format.cuh"

namespace dsa {

namespace {

__device__ __forceinline__ void unpack8(uint4 x, float (&v)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_bits_to_float(w[i] & 0xFFFF);
    v[2 * i + 1] = bf16_bits_to_float(w[i] >> 16);
  }
}

// Rows of a call: the first n, or the first *n_valid of them.
__device__ __forceinline__ int valid_rows(const RowsArgs& a) {
  return a.n_valid ? min(a.n, *a.n_valid) : a.n;
}

// The row's slot, or -1 when it has none; a slot past the cache is reported.
__device__ __forceinline__ int64_t slot_of(const RowsArgs& a, int r, int lane) {
  const int s = a.slots[r];
  if (s >= a.n_rows) {
    if (lane == 0) record_status(a.status, DSA_ERR_DEVICE_CHECK, SITE_ROWS, static_cast<uint32_t>(r));
    return -1;
  }
  return s < 0 ? -1 : s;
}

// x / s rounded to fp32 as an E4M3 conversion that saturates sees it, for s between 2^-60 and 2^60 and
// y = 1 / s rounded: two corrections by the exact remainder q s - x (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990) make x y the
// rounded quotient. Beyond +-1000 x y does (E4M3 ends at 448), where a remainder could
// overflow, and for zeros, whose sign the corrections would lose.
__device__ __forceinline__ float quotient(float x, float s, float y) {
  const float q0 = x * y;
  const float q1 = fmaf(fmaf(-q0, s, x), y, q0);
  const float q2 = fmaf(fmaf(-q1, s, x), y, q1);
  return fabsf(q0) <= 1000.f && q0 != 0.f ? q2 : q0;
}

// x s for a further rounding to bf16: cut off to fp32, its last bit set where something was cut
// (rounding to odd: Boldo and Melquiond, "Emulation of FMA and correctly rounded sums: proved
// algorithms using rounding to odd", 2008). A product rounded to nearest here could come to lie
// halfway between two bf16 values when it does not. The remainder is exact down to products of
// 2^-122 (four bits of a code and 24 of a scale).
__device__ __forceinline__ float product_odd(float x, float s) {
  const float p = __fmul_rz(x, s);
  const bool cut = fmaf(x, s, -p) != 0.f;
  return __uint_as_float(__float_as_uint(p) | (cut ? 1u : 0u));
}

template <int FMT>
__global__ void __launch_bounds__(256) kv_write_kernel(RowsArgs a) {
  griddep_wait();
  // (65536 rows: 25.1 us with a division an element, 20.6 with these quotients)
  const bool by_reciprocal = a.kv_scale > 0x1p-60f && a.kv_scale < 0x1p60f;
  const float recip = 1.f / a.kv_scale;
  const int lane = threadIdx.x & 31;
  const int n = valid_rows(a);
  const int step = static_cast<int>(gridDim.x) * 8;
  for (int r = blockIdx.x * 8 + (threadIdx.x >> 5); r < n; r += step) {
    const int64_t slot = slot_of(a, r, lane);
    if (slot < 0) continue;
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(a.rows) + static_cast<int64_t>(r) * a.row_stride);
    const uint4 x0 = src[lane], x1 = src[32 + lane];
    uint8_t* dst = static_cast<uint8_t*>(a.cache) + slot * kv_row_bytes(FMT);
    if constexpr (FMT == DSA_KV_BF16) {
      reinterpret_cast<uint4*>(dst)[lane] = x0;
      reinterpret_cast<uint4*>(dst)[32 + lane] = x1;
    } else {
      float v[2][8];
      unpack8(x0, v[0]);
      unpack8(x1, v[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (FMT == DSA_KV_FP8_E4M3) {
          uint32_t w[2] = {0u, 0u};
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 pr =
                by_reciprocal ? make_float2(quotient(v[h][i], a.kv_scale, recip),
                                            quotient(v[h][i + 1], a.kv_scale, recip))
                              : make_float2(__fdiv_rn(v[h][i], a.kv_scale),
                                            __fdiv_rn(v[h][i + 1], a.kv_scale));
            w[i >> 2] |= static_cast<uint32_t>(
                             __nv_cvt_float2_to_fp8x2(pr, __NV_SATFINITE, __NV_E4M3))
                         << (16 * ((i >> 1) & 1));
          }
          reinterpret_cast<uint2*>(dst)[32 * h + lane] = make_uint2(w[0], w[1]);
        } else {
          // the group's largest magnitude as fp32 bits (NaN and infinity largest)
          uint32_t amax = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[h][i]) & 0x7FFFFFFFu);
          amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
          amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
          const uint32_t scale = mx4_scale(amax);
          reinterpret_cast<uint32_t*>(dst)[32 * h + lane] = mx4_encode8(v[h], scale);
          if ((lane & 3) == 0) {
            dst[kRow4Codes + 8 * h + (lane >> 2)] = static_cast<uint8_t>(scale);
          }
        }
      }
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(256) kv_read_kernel(RowsArgs a) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int n = valid_rows(a);
  const int step = static_cast<int>(gridDim.x) * 8;
  for (int r = blockIdx.x * 8 + (threadIdx.x >> 5); r < n; r += step) {
    const int64_t slot = slot_of(a, r, lane);
    if (slot < 0) continue;
    const uint8_t* src = static_cast<const uint8_t*>(a.cache) + slot * kv_row_bytes(FMT);
    uint4 x[2];
    if constexpr (FMT == DSA_KV_BF16) {
      x[0] = reinterpret_cast<const uint4*>(src)[lane];
      x[1] = reinterpret_cast<const uint4*>(src)[32 + lane];
    } else if constexpr (FMT == DSA_KV_FP8_E4M3) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 c = reinterpret_cast<const uint2*>(src)[32 * h + lane];
        const uint32_t cw[2] = {c.x, c.y};
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
              static_cast<__nv_fp8x2_storage_t>((cw[i >> 1] >> (16 * (i & 1))) & 0xFFFF), __NV_E4M3);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
          const __nv_bfloat162 p = __floats2bfloat162_rn(product_odd(f.x, a.kv_scale),
                                                         product_odd(f.y, a.kv_scale));
          w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
        x[h] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t c = reinterpret_cast<const uint32_t*>(src)[32 * h + lane];
        x[h] = mx4_decode8(c, mx4_scale_bf16x2(src[kRow4Codes + 8 * h + (lane >> 2)]));
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(const_cast<void*>(a.rows)) +
                                          static_cast<int64_t>(r) * a.row_stride);
    dst[lane] = x[0];
    dst[32 + lane] = x[1];
  }
}

template <typename K>
cudaError_t launch_rows(K* kernel, const RowsArgs& a, cudaStream_t s) {
  // one warp a row; beyond 8 CTAs an SM (all its warps) the warps loop
  const int64_t want = (static_cast<int64_t>(a.n) + 7) / 8;
  const int grid = static_cast<int>(std::min<int64_t>(want, int64_t{8} * device_sm_count()));
  return launch_pdl(kernel, dim3(grid), dim3(256), 0, s, 1, a);
}

}  // namespace

cudaError_t launch_kv_write(const RowsArgs& a, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  switch (a.kv_fmt) {
    case DSA_KV_BF16: return launch_rows(kv_write_kernel<DSA_KV_BF16>, a, s);
    case DSA_KV_FP8_E4M3: return launch_rows(kv_write_kernel<DSA_KV_FP8_E4M3>, a, s);
    default: return launch_rows(kv_write_kernel<DSA_KV_MXFP4>, a, s);
  }
}

cudaError_t launch_kv_read(const RowsArgs& a, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  switch (a.kv_fmt) {
    case DSA_KV_BF16: return launch_rows(kv_read_kernel<DSA_KV_BF16>, a, s);
    case DSA_KV_FP8_E4M3: return launch_rows(kv_read_kernel<DSA_KV_FP8_E4M3>, a, s);
    default: return launch_rows(kv_read_kernel<DSA_KV_MXFP4>, a, s);
  }
}

}  // namespace dsa
