// Norms of queries and keys for each head, with the position rotation in the
// same pass: y = x / sqrt(mean(x^2) + eps) * w over a head's elements, then
// pairs of its rope_dim elements from rope_start on turned by the angle
// position * inv_freq. x is read once and y written once, so the pass is bound
// by memory (or, for a few tokens, by one trip through it).
//
// A unit of work is one head of more than 128 elements (lane l holds 8-element
// chunks l, l + 32, ...), or two, four ... smaller ones: a warp's worth. Every warp of the
// grid takes an equal run of consecutive units (heads of a token, then the next
// token's) and works by itself: it copies the elements of the units ahead into a ring of its
// own (by cp.async; a lane reads back what it copied, so nothing waits for another lane),
// keeps its group's weights in registers, and works out the cosines and sines when
// its token changes. So there are always kAhead units of a warp on their way.
// The angles are reduced to a fraction of a turn in 64-bit integers (see turn_bits): an
// fp32 product would lose the turn's fraction at far positions, and the fp64 pipe would
// take longer for them than all the rest of a small call.
#include <algorithm>
#include <type_traits>

#include "kernels.h"

namespace dsa {

namespace {

constexpr int kWarps = 8;

constexpr int kAhead = 3;  // units on their way

// Two fp32 values in a register pair and their arithmetic (one instruction for both).
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 un2(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// 8 elements in shared or global memory as four pairs of fp32 values, and back.
template <typename T>
__device__ __forceinline__ F2 pair_of(uint32_t w) {  // two 16-bit elements
  if constexpr (std::is_same<T, __half>::value) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return f2(f.x, f.y);
  } else {
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
}
template <typename T>
__device__ __forceinline__ uint32_t word_of(F2 v) {
  const float2 f = un2(v);
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const F2 (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float2 a = un2(v[0]), b = un2(v[1]), c = un2(v[2]), d = un2(v[3]);
    reinterpret_cast<float4*>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
    reinterpret_cast<float4*>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(word_of<T>(v[0]), word_of<T>(v[1]), word_of<T>(v[2]),
                                              word_of<T>(v[3]));
  }
}
__device__ __forceinline__ void load8(const float* p, F2 (&v)[4]) {
  const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
  v[0] = f2(x.x, x.y), v[1] = f2(x.z, x.w), v[2] = f2(y.x, y.y), v[3] = f2(y.z, y.w);
}

// f / (2 pi) in units of 2^-64 turns, modulo whole turns, rounded down: the fp64 number
// f = m 2^(e - 1075) with its 53-bit integer m, times 1 / (2 pi) = inv_2pi 2^-66 (inv_2pi
// the 64-bit integer), is m inv_2pi 2^(e - 1077) of those units. A position times this,
// modulo 2^64, is the angle's fraction of a turn to within 2^-33 (positions below 2^31).
__device__ __forceinline__ uint64_t turn_bits(double f, uint64_t inv_2pi) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
  const int e = static_cast<int>(bits >> 52) & 0x7FF;
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | (e ? 1ull << 52 : 0ull);
  const uint64_t lo = m * inv_2pi, hi = __umul64hi(m, inv_2pi);
  const int sh = 1077 - max(e, 1);
  uint64_t t = 0;
  if (sh >= 64) {
    t = sh < 128 ? hi >> (sh - 64) : 0ull;
  } else if (sh > 0) {
    t = (hi << (64 - sh)) | (lo >> sh);
  } else {
    t = sh > -64 ? lo << -sh : 0ull;
  }
  return static_cast<int64_t>(bits) < 0 ? 0ull - t : t;
}

// Place of pair k in the table of cosines and sines: one place in nine is left out, so that
// lanes four or eight pairs apart read different banks.
__host__ __device__ constexpr int table_at(int k) { return k + (k >> 3); }
__host__ __device__ constexpr int table_len(int pairs) { return (table_at(pairs) + 1) & ~1; }

// A place in the run of units: the token, the unit of the token and its group of heads,
// this lane's head, its chunks of the group's heads (as bits) and its first element there
// (in x or in out), which moves by `step` from unit to unit of a group.
template <typename T>
struct Cursor {
  int tok, u, seg, head;
  uint32_t chunks;
  T* ptr;
  int64_t step;
};

// NV: 8-element chunks a lane holds (heads of up to 256 NV elements).
template <typename T, int NV>
__global__ void __launch_bounds__(32 * kWarps, NV == 1 ? 4 : NV == 2 ? 3 : 2)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  extern __shared__ float4 smem4[];
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = a.n_valid ? max(0, min(a.n, *a.n_valid)) : a.n;
  // Runs of `per` units, or of one more for the first `more` warps.
  const int64_t total = static_cast<int64_t>(n) * a.units;
  const int warps = static_cast<int>(gridDim.x) * kWarps;
  const int me = static_cast<int>(blockIdx.x) * kWarps + warp;
  int64_t per, more;
  if (total <= 0x7FFFFFFF) {  // (a 32-bit division takes a fraction of a 64-bit one)
    per = static_cast<int>(total) / warps;
    more = static_cast<int>(total) - static_cast<int>(per) * warps;
  } else {
    per = total / warps;
    more = total - per * warps;
  }
  const int64_t begin = me * per + min(static_cast<int64_t>(me), more);
  const int count = static_cast<int>(per) + (me < more ? 1 : 0);
  if (count == 0) return;
  const int pairs = a.pairs;
  // This warp's shared memory: the ring, (cos, sin) of each pair at its token, and (halves
  // rotated) the rotated elements of its heads.
  constexpr int kUnitBytes = 256 * NV * static_cast<int>(sizeof(T));
  constexpr int kQuads = static_cast<int>(sizeof(T)) / 2;  // 16-byte pieces of a chunk
  uint8_t* mem = reinterpret_cast<uint8_t*>(smem4) + warp * a.warp_bytes;
  float2* table = reinterpret_cast<float2*>(mem + kAhead * kUnitBytes);
  float* stage = reinterpret_cast<float*>(table + table_len(pairs));
  const uint32_t ring = smem_u32(mem);

  // A cursor's place in its group: the lane's head and pointer.
  auto enter = [&](Cursor<T>& c, bool in) {
    const NormRopeSeg& sg = a.seg[c.seg];
    const int lg = sg.lanes_log2;
    c.head = ((c.u - sg.unit_begin) << (5 - lg)) + (lane >> lg);
    const int64_t ts = in ? sg.x_token_stride : sg.out_token_stride;
    const int64_t hs = in ? sg.x_head_stride : sg.out_head_stride;
    const int l = lane & ((1 << lg) - 1);
    c.ptr = static_cast<T*>(in ? const_cast<void*>(sg.x) : sg.out) + c.tok * ts + c.head * hs + 8 * l;
    c.step = hs << (5 - lg);
    c.chunks = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (8 * (l + (k << lg)) < sg.dim) c.chunks |= 1u << k;
    }
  };
  auto advance = [&](Cursor<T>& c, bool in) {
    ++c.u;
    if (c.u < a.seg[c.seg].unit_end) {
      c.head += 32 >> a.seg[c.seg].lanes_log2;
      c.ptr += c.step;
      return;
    }
    if (c.u == a.units) {
      c.u = 0;
      c.seg = 0;
      ++c.tok;
    } else {
      ++c.seg;
    }
    enter(c, in);
  };
  Cursor<T> ahead;
  ahead.tok = total <= 0x7FFFFFFF ? static_cast<int>(begin) / a.units
                                  : static_cast<int>(begin / a.units);
  ahead.u = static_cast<int>(begin - static_cast<int64_t>(ahead.tok) * a.units);
  ahead.seg = 0;
  while (ahead.u >= a.seg[ahead.seg].unit_end) ++ahead.seg;
  Cursor<T> at;
  at.tok = ahead.tok, at.u = ahead.u, at.seg = ahead.seg;
  enter(ahead, true);
  enter(at, false);
  int issued = 0;
  uint32_t slot = ring;  // of the next unit to copy
  auto issue = [&]() {   // one copy group a unit, empty past the end
    if (issued < count) {
      const NormRopeSeg& sg = a.seg[ahead.seg];
      const uint32_t m = ahead.head < sg.heads ? ahead.chunks : 0u;
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        if (m >> c & 1u) {
#pragma unroll
          for (int k = 0; k < kQuads; ++k) {
            cp_async_16(slot + ((c * kQuads + k) * 32 + lane) * 16,
                        reinterpret_cast<const uint4*>(ahead.ptr + (8 * c << sg.lanes_log2)) + k);
          }
        }
      }
      advance(ahead, true);
    }
    ++issued;
    slot = slot == ring + (kAhead - 1) * kUnitBytes ? ring : slot + kUnitBytes;
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) issue();
  F2 w[NV][4];  // the group's weights
  int weights_of = -1, table_of = -1;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const NormRopeSeg& sg = a.seg[at.seg];
    const int lg = sg.lanes_log2, l = lane & ((1 << lg) - 1);
    if (weights_of != at.seg) {
      weights_of = at.seg;
#pragma unroll
      for (int c = 0; c < NV; ++c) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[c][k] = f2(1.f, 1.f);
        if (sg.weight && (at.chunks >> c & 1u)) load8(sg.weight + 8 * (l + (c << lg)), w[c]);
      }
    }
    if (sg.rope && table_of != at.tok) {
      table_of = at.tok;
      const int64_t pos = a.positions[at.tok];
      __syncwarp();
      for (int k = lane; k < pairs; k += 32) {
        const int64_t turn = pos * static_cast<int64_t>(turn_bits(a.inv_freq[k], a.inv_2pi));
        float s, c;
        sincospif(static_cast<float>(turn) * 0x1p-63f, &s, &c);  // half turns, from -1 to 1
        table[table_at(k)] = make_float2(c * a.rope_scale, s * a.rope_scale);
      }
      __syncwarp();
    }
    cp_async_wait<kAhead - 1>();
    const uint32_t m = at.head < sg.heads ? at.chunks : 0u;
    F2 v[NV][4];
    F2 ss0 = f2(0.f, 0.f), ss1 = ss0;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      // `slot` is the place of this unit, refilled below
      if (m >> c & 1u) {
        const uint4 x = ld_shared_v4(slot + (c * kQuads * 32 + lane) * 16);
        if constexpr (sizeof(T) == 4) {
          const uint4 y = ld_shared_v4(slot + ((c * kQuads + 1) * 32 + lane) * 16);
          v[c][0] = f2(__uint_as_float(x.x), __uint_as_float(x.y));
          v[c][1] = f2(__uint_as_float(x.z), __uint_as_float(x.w));
          v[c][2] = f2(__uint_as_float(y.x), __uint_as_float(y.y));
          v[c][3] = f2(__uint_as_float(y.z), __uint_as_float(y.w));
        } else {
          v[c][0] = pair_of<T>(x.x), v[c][1] = pair_of<T>(x.y);
          v[c][2] = pair_of<T>(x.z), v[c][3] = pair_of<T>(x.w);
        }
        ss0 = fma2(v[c][0], v[c][0], ss0);
        ss1 = fma2(v[c][1], v[c][1], ss1);
        ss0 = fma2(v[c][2], v[c][2], ss0);
        ss1 = fma2(v[c][3], v[c][3], ss1);
      }
    }
    issue();
    if (sg.norm) {
      const float2 s0 = un2(ss0), s1 = un2(ss1);
      float ss = (s0.x + s0.y) + (s1.x + s1.y);
      for (int o = (1 << lg) >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      const float r = rsqrtf(ss * sg.inv_dim + sg.eps);
      const F2 r2 = f2(r, r);
#pragma unroll
      for (int c = 0; c < NV; ++c) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[c][k] = mul2(v[c][k], mul2(r2, w[c][k]));
      }
    }
    if (sg.rope) {
      const int rd = 2 * pairs;
      if (a.interleaved) {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const int e = 8 * (l + (c << lg)) - sg.rope_start;
          if (e >= 0 && e < rd) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 t = table[table_at((e >> 1) + k)], x = un2(v[c][k]);
              v[c][k] = f2(x.x * t.x - x.y * t.y, x.x * t.y + x.y * t.x);
            }
          }
        }
      } else {
        // element i and element i + rope_dim / 2 turn together: through shared memory, the
        // first and the last four elements of the chunks apart (16 bytes from lane to lane)
        float4* heads = reinterpret_cast<float4*>(stage + (lane >> lg) * rd);
        const int last4 = rd >> 3;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const int e = 8 * (l + (c << lg)) - sg.rope_start;
          if (e >= 0 && e < rd) {
            const float2 x0 = un2(v[c][0]), x1 = un2(v[c][1]), x2 = un2(v[c][2]), x3 = un2(v[c][3]);
            heads[e >> 3] = make_float4(x0.x, x0.y, x1.x, x1.y);
            heads[last4 + (e >> 3)] = make_float4(x2.x, x2.y, x3.x, x3.y);
          }
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const int e = 8 * (l + (c << lg)) - sg.rope_start;
          if (e >= 0 && e < rd) {
            const bool low = e < pairs;
            const int there = (low ? e + pairs : e - pairs) >> 3;
            const float4 o0 = heads[there], o1 = heads[last4 + there];
            const float2 other[4] = {{o0.x, o0.y}, {o0.z, o0.w}, {o1.x, o1.y}, {o1.z, o1.w}};
            const int p0 = low ? e : e - pairs;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 t0 = table[table_at(p0 + 2 * k)], t1 = table[table_at(p0 + 2 * k + 1)];
              const float2 x = un2(v[c][k]), y = other[k];
              v[c][k] = low ? f2(x.x * t0.x - y.x * t0.y, x.y * t1.x - y.y * t1.y)
                            : f2(y.x * t0.y + x.x * t0.x, y.y * t1.y + x.y * t1.x);
            }
          }
        }
        __syncwarp();
      }
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      if (m >> c & 1u) store8(at.ptr + (8 * c << lg), v[c]);
    }
    advance(at, false);
  }
}

template <typename T, int NV>
cudaError_t launch_nv(NormRopeArgs a, cudaStream_t s) {
  const int stage = a.pairs && !a.interleaved ? 256 * NV * 4 : 0;
  a.inv_2pi = static_cast<uint64_t>(0x1p66L * 0.15915494309189533576888376337251436203445965L);
  a.warp_bytes = kAhead * 256 * NV * static_cast<int>(sizeof(T)) + table_len(a.pairs) * 8 + stage;
  const int smem = kWarps * a.warp_bytes;
  static std::atomic<int> smem_set[64]{};
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(norm_rope_kernel<T, NV>), smem, smem_set);
  if (e != cudaSuccess) return e;
  // As many CTAs as the SMs hold at once, or one for every eight units of fewer.
  // (The last answer is kept with the shared memory it is for, in one word.)
  static std::atomic<int64_t> last{0};
  const int64_t known = last.load(std::memory_order_relaxed);
  int per_sm = static_cast<int>(known & 0xFFFF);
  if (known >> 16 != smem + 1) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, norm_rope_kernel<T, NV>, 32 * kWarps,
                                                      static_cast<size_t>(smem)) != cudaSuccess ||
        per_sm < 1) {
      cudaGetLastError();  // clear the error the failed query left behind
      per_sm = 1;
    }
    last.store((int64_t{smem} + 1) << 16 | per_sm, std::memory_order_relaxed);
  }
  const int64_t want = (static_cast<int64_t>(a.n) * a.units + kWarps - 1) / kWarps;
  const int grid = static_cast<int>(std::min<int64_t>(want, int64_t{per_sm} * device_sm_count()));
  return launch_pdl(norm_rope_kernel<T, NV>, dim3(grid), dim3(32 * kWarps), static_cast<size_t>(smem),
                    s, 1, a);
}

template <typename T>
cudaError_t launch_t(const NormRopeArgs& a, int max_dim, cudaStream_t s) {
  if (max_dim <= 256) return launch_nv<T, 1>(a, s);
  if (max_dim <= 512) return launch_nv<T, 2>(a, s);
  return launch_nv<T, 4>(a, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int dtype, int max_dim, cudaStream_t s) {
  if (a.n == 0 || a.units == 0) return cudaSuccess;
  switch (dtype) {
    case DSA_DT_BF16: return launch_t<uint16_t>(a, max_dim, s);
    case DSA_DT_F16: return launch_t<__half>(a, max_dim, s);
    default: return launch_t<float>(a, max_dim, s);
  }
}

}  // namespace dsa
