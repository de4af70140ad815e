// Norms of queries and keys for each head, with the position rotation in the
// same pass: y = x / sqrt(mean(x^2) + eps) * w over a head's elements, then
// pairs of its rope_dim elements from rope_start on turned by the angle
// position * inv_freq. x is read once and y written once, so the pass is bound
// by memory (or, for a few tokens, by one trip through it).
//
// A lane holds 16-byte chunks of a head: l, l + 32, ... of one that fills a warp's row of
// chunks, so that every access of a warp is contiguous (fp32 heads in chunks of 32 bytes a
// lane took 261 us where this takes 186: 4096 tokens of 64 x 512). A unit of work is one
// such head, or two, four ... smaller ones: a warp's worth. Every warp of the
// grid takes an equal run of consecutive units (heads of a token, then the next
// token's) and works by itself: it copies the elements of the units ahead into a ring of its
// own (by cp.async; a lane reads back what it copied, so nothing waits for another lane),
// and works out the cosines and sines when its token changes. Within a run the units of one
// group of one token share their constants, and a loop for heads that fill every chunk
// has no branch for lanes without an element: a call that fits in the L2 is bound by the
// instructions (333 tokens of 89 heads of 128, f16: 9.1 -> 8.2 us; 4096 of them 67.5 -> 52.0).
// The weights stay in shared memory for their registers' sake. Two CTAs an SM with two
// units a warp on their way read and write faster than more of either: 4096 tokens of
// 64 heads of 512, bf16, 581 MB in 92.9 us (6.25 TB/s), a plain copy of as much by the same
// warps 97.
// The angles are reduced to a fraction of a turn in 64-bit integers (see turn_bits): an
// fp32 product would lose the turn's fraction at far positions, and the fp64 pipe would
// take longer for them than all the rest of a small call.
#include <algorithm>
#include <type_traits>

#include "kernels.h"

namespace dsa {

namespace {

constexpr int kWarps = 8;

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

// Two 16-bit elements as fp32 values, and back (rounded to nearest even).
template <typename T>
__device__ __forceinline__ F2 pair_of(uint32_t w) {
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
// A lane's chunk: 16 bytes of a head, as pairs of fp32 values.
template <typename T>
constexpr int kChunk = 16 / static_cast<int>(sizeof(T));  // elements
template <typename T>
__device__ __forceinline__ void unpack(uint4 x, F2 (&v)[kChunk<T> / 2]) {
  if constexpr (sizeof(T) == 4) {
    v[0] = f2(__uint_as_float(x.x), __uint_as_float(x.y));
    v[1] = f2(__uint_as_float(x.z), __uint_as_float(x.w));
  } else {
    v[0] = pair_of<T>(x.x), v[1] = pair_of<T>(x.y);
    v[2] = pair_of<T>(x.z), v[3] = pair_of<T>(x.w);
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const F2 (&v)[kChunk<T> / 2]) {
  if constexpr (sizeof(T) == 4) {
    const float2 a = un2(v[0]), b = un2(v[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                      __float_as_uint(b.y));
  } else {
    return make_uint4(word_of<T>(v[0]), word_of<T>(v[1]), word_of<T>(v[2]), word_of<T>(v[3]));
  }
}
__device__ __forceinline__ void st_shared_f2x2(uint32_t at, F2 a, F2 b) {
  asm volatile("st.shared.v2.b64 [%0], {%1, %2};\n" ::"r"(at), "l"(a), "l"(b) : "memory");
}
__device__ __forceinline__ void ld_shared_f2x2(uint32_t at, F2& a, F2& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];\n" : "=l"(a), "=l"(b) : "r"(at));
}

// f / (2 pi) in units of 2^-64 turns, modulo whole turns, rounded down: the fp64 number
// f = m 2^(e - 1075) with its 53-bit integer m, times 1 / (2 pi) = inv_2pi 2^-66 (inv_2pi
// the 64-bit integer), is m inv_2pi 2^(e - 1077) of those units. A position times this,
// modulo 2^64, is the angle's fraction of a turn to within 2^-33 and 2^-63 of the angle in turns
// (positions of either sign). f is finite: an infinity or NaN has no angle, see angle_exists.
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

__device__ __forceinline__ bool angle_exists(double f) {
  return (static_cast<uint32_t>(__double_as_longlong(f) >> 52) & 0x7FFu) != 0x7FFu;
}

// Shared memory of a warp's cosines and sines: (cos, sin) of each pair, or (halves) the
// cosines, the sines and the negated sines, which the first of a pair's elements take.
__host__ __device__ constexpr int table_bytes(int pairs, bool interleaved) {
  return (interleaved ? 8 : 12) * pairs;
}

// 16 bytes to shared memory by cp.async, or 16 zeros (n = 0: src is not read).
__device__ __forceinline__ void cp_async_or_zeros(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}

// How a group's heads are rotated.
enum { kStill = 0, kInterleaved = 1, kHalves = 2 };

// Units on their way. (4096 tokens of 64 heads of 512, bf16: 92.9 us with two, 103.9 with three,
// 112 with one. Heads of 256: 61.2 with two, 57.2 with three.)
template <int NV>
constexpr int kUnitsAhead = NV == 2 ? 2 : 3;

// NV: heads of up to 256 NV elements. (CTAs an SM: at NV = 1 three take 51.6 us where four take
// 53.4, 4096 tokens of 89 heads of 128; at NV = 4 two spill.)
template <typename T, int NV>
__global__ void __launch_bounds__(32 * kWarps, NV == 1 ? 3 : NV == 2 ? 2 : 1)
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
  constexpr int kAhead = kUnitsAhead<NV>;
  constexpr int E = kChunk<T>, NC = 256 * NV / (32 * E);  // a lane's chunks
  constexpr int kUnitBytes = 512 * NC;
  uint8_t* mem = reinterpret_cast<uint8_t*>(smem4) + warp * a.warp_bytes;
  const uint32_t weights = smem_u32(mem) + kAhead * kUnitBytes + 16u * lane;
  float* table = reinterpret_cast<float*>(mem + kAhead * kUnitBytes + 1024 * NV);
  float* stage = table + table_bytes(pairs, a.interleaved) / 4;
  const uint32_t ring = smem_u32(mem) + 16u * lane;

  // The run's first unit: token, group, unit of the token.
  int tok = total <= 0x7FFFFFFF ? static_cast<int>(begin) / a.units
                                : static_cast<int>(begin / a.units);
  int u = static_cast<int>(begin - static_cast<int64_t>(tok) * a.units);
  int s = 0;
  while (u >= a.seg[s].unit_end) ++s;

  // The copies: the next unit's place and what it takes to step on within its group.
  int in_tok = tok, in_s = s, in_u = u, in_left = count;
  const T* in;
  int64_t in_step;
  int in_end, in_lim, in_chunk;
  uint32_t in_bytes[NC];
  uint32_t slot = ring;  // of the next unit to copy
  auto in_enter = [&]() {
    const NormRopeSeg& sg = a.seg[in_s];
    const int lg = sg.lanes_log2, l = lane & ((1 << lg) - 1);
    const int head = ((in_u - sg.unit_begin) << (5 - lg)) + (lane >> lg);
    in = static_cast<const T*>(sg.x) + in_tok * sg.x_token_stride + head * sg.x_head_stride + E * l;
    in_step = sg.x_head_stride << (5 - lg);
    in_end = sg.unit_end;
    // the lane has a head in the units below in_lim
    in_lim = sg.unit_end - ((sg.heads - 1) % (32 >> lg) < (lane >> lg) ? 1 : 0);
    in_chunk = E << lg;
#pragma unroll
    for (int c = 0; c < NC; ++c) in_bytes[c] = E * (l + (c << lg)) < sg.dim ? 16u : 0u;
  };
  in_enter();
  auto issue = [&]() {  // one copy group a unit, empty past the end
    if (in_left > 0) {
      const bool mine = in_u < in_lim;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        cp_async_or_zeros(slot + c * 512, in + c * in_chunk, mine ? in_bytes[c] : 0u);
      }
      in += in_step;
      --in_left;
      if (++in_u == in_end) {
        if (++in_s == a.n_seg) {
          in_s = in_u = 0;
          ++in_tok;
        }
        in_enter();
      }
    }
    slot = slot == ring + (kAhead - 1) * kUnitBytes ? ring : slot + kUnitBytes;
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) issue();

  int table_of = -1, weights_of = -1, left = count;
  do {
    // The run's units of one group of one token.
    const NormRopeSeg& sg = a.seg[s];
    const int lg = sg.lanes_log2, l = lane & ((1 << lg) - 1), chunk = E << lg;
    const int units = min(left, sg.unit_end - u);
    const int head = ((u - sg.unit_begin) << (5 - lg)) + (lane >> lg);
    const int mine = ((sg.heads - 1 - head) >> (5 - lg)) + 1;  // of them, those with a head for the lane
    T* out = static_cast<T*>(sg.out) + tok * sg.out_token_stride + head * sg.out_head_stride + E * l;
    const int64_t out_step = sg.out_head_stride << (5 - lg);
    const float inv_dim = sg.inv_dim, eps = sg.eps;
    const bool norm = sg.norm != 0;
    const int dim = sg.dim, K = (dim + chunk - 1) >> (lg + (E == 8 ? 3 : 2));
    if (weights_of != s) {  // the group's weights: each lane its own elements'
      weights_of = s;
#pragma unroll
      for (int q = 0; q < NC * E / 4; ++q) {
        const int e = E * l + (4 * q / E) * chunk + 4 * q % E;
        float4 w = make_float4(1.f, 1.f, 1.f, 1.f);
        if (sg.weight && e < dim) w = *reinterpret_cast<const float4*>(sg.weight + e);
        st_shared_f2x2(weights + q * 512, f2(w.x, w.y), f2(w.z, w.w));
      }
    }
    if (sg.rope && table_of != tok) {
      table_of = tok;
      const uint64_t pos = static_cast<uint64_t>(int64_t{a.positions[tok]});
      __syncwarp();
      for (int k = lane; k < pairs; k += 32) {
        const double f = a.inv_freq[k];
        const int64_t turn = static_cast<int64_t>(pos * turn_bits(f, a.inv_2pi));  // (modulo 2^64)
        float sn, cs;
        sincospif(angle_exists(f) ? static_cast<float>(turn) * 0x1p-63f  // half turns, from -1 to 1
                                  : __int_as_float(0x7FC00000),          // (NaN)
                  &sn, &cs);
        cs *= a.rope_scale;
        sn *= a.rope_scale;
        if (a.interleaved) {
          reinterpret_cast<float2*>(table)[k] = make_float2(cs, sn);
        } else {
          table[k] = cs;
          table[pairs + k] = sn;
          table[2 * pairs + k] = -sn;
        }
      }
      __syncwarp();
    }
    const int start = sg.rope_start;
    // The units. `full`: heads of 256 NV elements, one a warp, so every lane has every chunk.
    auto run = [&](auto full_c, auto rope_c) {
      constexpr bool kFull = decltype(full_c)::value;
      constexpr int kRope = decltype(rope_c)::value;
      T* to = out;
#pragma unroll 1
      for (int i = 0; i < units; ++i) {
        cp_async_wait<kAhead - 1>();
        F2 v[NC][E / 2];
        F2 ss0 = f2(0.f, 0.f), ss1 = ss0;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (kFull || c == 0 || c < K) {
            unpack<T>(ld_shared_v4(slot + c * 512), v[c]);  // (the place refilled below)
#pragma unroll
            for (int k = 0; k < E / 2; k += 2) {
              ss0 = fma2(v[c][k], v[c][k], ss0);
              ss1 = fma2(v[c][k + 1], v[c][k + 1], ss1);
            }
          }
        }
        issue();
        const float2 s0 = un2(ss0), s1 = un2(ss1);
        float ss = (s0.x + s0.y) + (s1.x + s1.y);
        if constexpr (kFull) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        } else {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const float t = __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            if (o < 1 << lg) ss += t;
          }
        }
        const float r = norm ? rsqrtf(fmaf(ss, inv_dim, eps)) : 1.f;
        const F2 r2 = f2(r, r);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (kFull || c == 0 || c < K) {
#pragma unroll
            for (int k = 0; k < E / 2; k += 2) {
              F2 w0, w1;
              ld_shared_f2x2(weights + (c * E + 2 * k) / 4 * 512, w0, w1);
              v[c][k] = mul2(v[c][k], mul2(r2, w0));
              v[c][k + 1] = mul2(v[c][k + 1], mul2(r2, w1));
            }
          }
        }
        if constexpr (kRope == kInterleaved) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int e = E * l + c * chunk - start;
            if (static_cast<unsigned>(e) < static_cast<unsigned>(2 * pairs)) {
#pragma unroll
              for (int k = 0; k < E / 2; k += 2) {  // two pairs: cosine, sine, cosine, sine
                const float4 t = *reinterpret_cast<const float4*>(table + e + 2 * k);
                const float2 x = un2(v[c][k]), y = un2(v[c][k + 1]);
                v[c][k] = f2(x.x * t.x - x.y * t.y, x.x * t.y + x.y * t.x);
                v[c][k + 1] = f2(y.x * t.z - y.y * t.w, y.x * t.w + y.y * t.z);
              }
            }
          }
        } else if constexpr (kRope == kHalves) {
          // element i and element i + rope_dim / 2 turn together: through shared memory, the
          // chunks' quarters of four elements apart (16 bytes from lane to lane)
          const int rd = 2 * pairs;
          float4* heads = reinterpret_cast<float4*>(stage + (lane >> lg) * rd);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int e = E * l + c * chunk - start;
            if (static_cast<unsigned>(e) < static_cast<unsigned>(rd)) {
#pragma unroll
              for (int k = 0; k < E / 2; k += 2) {
                const float2 x = un2(v[c][k]), y = un2(v[c][k + 1]);
                heads[static_cast<unsigned>(e + k / 2 * rd) / E] = make_float4(x.x, x.y, y.x, y.y);
              }
            }
          }
          __syncwarp();
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int e = E * l + c * chunk - start;
            if (static_cast<unsigned>(e) < static_cast<unsigned>(rd)) {
              const bool low = e < pairs;
              const int there = low ? e + pairs : e - pairs;
              const float* cs = table + (low ? e : there);
              const float* sn = cs + (low ? rd : pairs);  // the low one's sine is negated
#pragma unroll
              for (int k = 0; k < E / 2; k += 2) {
                const float4 y = heads[static_cast<unsigned>(there + k / 2 * rd) / E];
                const float4 p = *reinterpret_cast<const float4*>(cs + 2 * k);
                const float4 q = *reinterpret_cast<const float4*>(sn + 2 * k);
                v[c][k] = fma2(f2(y.x, y.y), f2(q.x, q.y), mul2(v[c][k], f2(p.x, p.y)));
                v[c][k + 1] = fma2(f2(y.z, y.w), f2(q.z, q.w), mul2(v[c][k + 1], f2(p.z, p.w)));
              }
            }
          }
          __syncwarp();
        }
        if (kFull || i < mine) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            if (kFull || E * l + c * chunk < dim) {
              *reinterpret_cast<uint4*>(to + c * chunk) = pack<T>(v[c]);
            }
          }
        }
        to += out_step;
      }
    };
    using std::integral_constant;
    const bool full = dim == 256 * NV;
    const int rope = !sg.rope ? kStill : a.interleaved ? kInterleaved : kHalves;
    if (full && rope == kInterleaved) {
      run(std::true_type{}, integral_constant<int, kInterleaved>{});
    } else if (full && rope == kStill) {
      run(std::true_type{}, integral_constant<int, kStill>{});
    } else if (rope == kInterleaved) {
      run(std::false_type{}, integral_constant<int, kInterleaved>{});
    } else if (rope == kStill) {
      run(std::false_type{}, integral_constant<int, kStill>{});
    } else {
      run(std::false_type{}, integral_constant<int, kHalves>{});
    }
    left -= units;
    u += units;
    if (++s == a.n_seg) {
      s = u = 0;
      ++tok;
    }
  } while (left > 0);
}

template <typename T, int NV>
cudaError_t launch_nv(NormRopeArgs a, cudaStream_t s) {
  const int stage = a.pairs && !a.interleaved ? 256 * NV * 4 : 0;
  a.inv_2pi = static_cast<uint64_t>(0x1p66L * 0.15915494309189533576888376337251436203445965L);
  a.warp_bytes = kUnitsAhead<NV> * 256 * NV * static_cast<int>(sizeof(T)) + 1024 * NV +
                 table_bytes(a.pairs, a.interleaved) + stage;
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
