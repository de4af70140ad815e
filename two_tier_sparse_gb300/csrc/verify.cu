// Verification of drafted tokens against the target's probabilities, from given
// random numbers (rejection sampling, Leviathan, Kalman and Matias, "Fast inference from
// transformers via speculative decoding", 2023): draft i of a request stands while
// u_i q_i(x_i) < p_i(x_i); at the first that does not, a token is drawn from max(p_i - q_i, 0),
// behind the last one from p, as the first t whose running sum exceeds u' times the total.
//
// Only one position's probabilities are read whole, so a request is one pass over a row of p
// and a row of q: 1 MB at 129280 words. A cluster of up to 16 CTAs shares a request; its warps have
// consecutive spans of the row, each cut in at most 32 blocks whose sums its lanes keep. Once the
// cluster's total is known the warp whose span holds the drawn place finds the block among its
// lanes and reads that block again.
//
// Sums are whole numbers of 2^-44, so their order does not matter and no two ways of cutting a
// row differ: a value is taken to the nearest multiple of 2^-22 and its remainder to one of
// 2^-44 by adding 3 (a float's last place there is 2^-22) and reading the bits, which leaves
// two 32-bit additions where 64-bit ones would bound the pass.
//
// One request of 4 drafts and 129280 words takes 5.3 us (replayed from a graph), a chain of five trips
// through memory (tokens, their probabilities, the rows, the cluster's total, the place), 64 of 5 drafts
// 13.8, 256 of 4 45.6 (208 MB, one row of a request whose drafts all stand, two of another: 4.6 TB/s), 129 of 3
// over 50257 bf16 words 10.3 (13 MB). What bounds the large ones are loads in flight: a span is read in
// rounds of kUnroll iterations a warp, each behind the one before, and a scheduler issues a third of the
// time. Four iterations a round instead of two take 42.8 for the 256, but 14.3 for the 64, 8.7 for 7.2 with 512 requests of
// 5000 words (more code to fetch) and 15.4 for 13.7 with 129 of bf16 and two rows; CTAs of 128 threads 45.3, but 17.1 for the
// 64 and 6.4 for the one. (Of a kernel that took 46.4 for the 256: a ring in shared memory five iterations
// deep 52.6, the next units in registers ahead 49.3.)
#include <algorithm>
#include <type_traits>

#include "kernels.h"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPerSm = 4;        // CTAs an SM (64 registers a thread)
constexpr int kMaxCluster = 16;  // (8 is the portable size)
constexpr int kUnroll = 2;  // iterations whose loads are issued together

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

// A value as a probability: in [0, 1], 0 for a NaN.
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }

// A unit of a row that it does not fill or that crosses a 16-byte boundary, an element at a
// time, 0 before the row's start and past its end (out of line: few).
template <typename T>
__device__ __noinline__ uint4 load_elements(const T* row, int i0, int n) {
  constexpr int N = 16 / sizeof(T);
  T e[N];
#pragma unroll
  for (int k = 0; k < N; ++k) e[k] = i0 + k >= 0 && i0 + k < n ? row[i0 + k] : T(0.f);
  return *reinterpret_cast<const uint4*>(e);
}

// 16 bytes of a row.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  uint4 w;
  // Elements i0 .. of a row of n, 0 outside it. ALIGNED: they begin on a 16-byte boundary; else they
  // miss one by `off` bytes, and the aligned 16 bytes before and behind are read and shifted into
  // place.
  template <bool ALIGNED>
  __device__ __forceinline__ void load(const T* row, int i0, int n, uint32_t off) {
    const T* at = row + i0;
    if (ALIGNED ? i0 >= 0 && i0 + N <= n : i0 >= N && i0 + 2 * N <= n) {
      if constexpr (ALIGNED) {
        w = *reinterpret_cast<const uint4*>(at);
      } else {
        const uint4* v = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(at) - off);
        w = v[0];
        const uint4 x = v[1];
        uint32_t a[6] = {w.x, w.y, w.z, w.w, x.x, x.y};
        if (off & 8u) a[0] = a[2], a[1] = a[3], a[2] = a[4], a[3] = a[5], a[4] = x.z, a[5] = x.w;
        if (off & 4u) a[0] = a[1], a[1] = a[2], a[2] = a[3], a[3] = a[4], a[4] = a[5];
        const uint32_t s = 8u * (off & 3u);
        w = make_uint4(__funnelshift_r(a[0], a[1], s), __funnelshift_r(a[1], a[2], s),
                       __funnelshift_r(a[2], a[3], s), __funnelshift_r(a[3], a[4], s));
      }
    } else {
      w = i0 < n ? load_elements(row, i0, n) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  // elements 2 k and 2 k + 1
  __device__ __forceinline__ float2 pair(int k) const {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 4) {
      return make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
    } else if constexpr (std::is_same<T, __half>::value) {
      return __half22float2(*reinterpret_cast<const __half2*>(&x[k]));
    } else {
      return make_float2(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xFFFF0000u));
    }
  }
};

// Two floats in one register pair, and their packed arithmetic.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void bits_of(F2 x, uint32_t& a, uint32_t& b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=r"(a), "=r"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Sums of a few values in units of 2^-22 and of 2^-44 (of either sign, up to 2^22 a value).
struct Parts {
  uint32_t hi;
  int32_t lo;
};
__device__ __forceinline__ int64_t joined(const Parts& s) {
  return (static_cast<int64_t>(s.hi) << 22) + s.lo;
}
// The sum over a warp's lanes (32 values each at most): 8 bits of each part apart, so that
// 32 bits hold the sums.
__device__ __forceinline__ int64_t warp_joined(const Parts& s) {
  constexpr uint32_t all = 0xFFFFFFFFu;
  const int64_t hi = (static_cast<int64_t>(__reduce_add_sync(all, s.hi >> 8)) << 8) +
                     __reduce_add_sync(all, s.hi & 255u);
  const int64_t lo = static_cast<int64_t>(__reduce_add_sync(all, s.lo >> 8)) * 256 +
                     __reduce_add_sync(all, static_cast<uint32_t>(s.lo) & 255u);
  return (hi << 22) + lo;
}
constexpr uint32_t kThree = 0x40400000u;  // the bits of 3
// Two values d + e in [0, 1] (e below d's last place) as whole numbers: the bits of 3 + the nearest
// multiple of 2^-22 of d and of 3 + 2^22 times the rest.
__device__ __forceinline__ void split(F2 d, F2 e, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
  const F2 a = add2(d, f2(3.f, 3.f));
  const F2 rest = add2(fma2(add2(a, f2(-3.f, -3.f)), f2(-1.f, -1.f), d), e);
  bits_of(a, hi[0], hi[1]);
  bits_of(fma2(rest, f2(4194304.f, 4194304.f), f2(3.f, 3.f)), lo[0], lo[1]);
}

struct Row {
  const void *p, *q;  // q null: no draft to take off
  int n;              // words
  int drop;           // a word that does not count, or -1
  uint32_t p_off, q_off;  // bytes by which the rows miss a 16-byte boundary
  // Words that the first unit begins before the row, so that units begin on 16-byte boundaries
  // (both rows' where they miss them alike).
  int shift;
};

// The first `words` words of a 16-byte unit that begins at word i0, each word's share added to s:
// max(p, q) - q, which is p - q or nothing (a NaN or negative p counts as 0), exactly as the rounded
// difference d and what it lacks, e = (max(p, q) - d) - q. `top` collects the largest bits of q and
// of max(p, q): above those of 1 there are values that are no probabilities, and the sum is to be
// taken again with CLAMP.
template <typename T, bool HASQ, bool CLAMP>
__device__ __forceinline__ void add_unit(Parts& s, const Vec<T>& p, const Vec<T>& q, int i0, int drop,
                                         uint32_t& top, int words = Vec<T>::N) {
#pragma unroll
  for (int k = 0; k < Vec<T>::N; k += 2) {
    float2 pk = p.pair(k / 2), qk = make_float2(0.f, 0.f);
    if (!HASQ) {
      if (i0 + k == drop) pk.x = 0.f;
      if (i0 + k + 1 == drop) pk.y = 0.f;
    } else {
      qk = q.pair(k / 2);
      if (CLAMP) {
        qk = make_float2(prob(qk.x), prob(qk.y));
      } else {
        top = __vimax3_u32(top, __float_as_uint(qk.x), __float_as_uint(qk.y));
      }
    }
    pk = make_float2(fmaxf(pk.x, qk.x), fmaxf(pk.y, qk.y));
    if (CLAMP) {
      pk = make_float2(fminf(pk.x, 1.f), fminf(pk.y, 1.f));
    } else {
      top = __vimax3_u32(top, __float_as_uint(pk.x), __float_as_uint(pk.y));
    }
    uint32_t hi[2], lo[2];
    const F2 p2 = f2(pk.x, pk.y);
    if (HASQ) {
      const F2 m1 = f2(-1.f, -1.f), q2 = f2(qk.x, qk.y);
      const F2 d = fma2(q2, m1, p2);
      split(d, fma2(q2, m1, fma2(d, m1, p2)), hi, lo);
    } else {
      split(p2, f2(0.f, 0.f), hi, lo);
    }
    if (CLAMP) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (k + e < words) {
          s.hi += hi[e] - kThree;
          s.lo += static_cast<int32_t>(lo[e] - kThree);
        }
      }
    } else {
      s.hi += hi[0] + hi[1];
      s.lo += static_cast<int32_t>(lo[0] + lo[1]);
    }
  }
  if (!CLAMP) {
    s.hi -= Vec<T>::N * kThree;
    s.lo -= static_cast<int32_t>(Vec<T>::N * kThree);
  }
}

__device__ __forceinline__ int64_t shfl64(int64_t x, int lane) {
  return static_cast<int64_t>(__shfl_sync(0xFFFFFFFFu, static_cast<unsigned long long>(x), lane));
}
__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += t;
  }
  return x;
}

// A warp's span of a row: iterations [first, first + n) of 32 units, in blocks of `block`.
struct Span {
  int first, n, block;
};

// A unit's first `words` words again, with CLAMP.
template <typename T, bool HASQ, bool ALIGNED>
__device__ __noinline__ Parts clamped(const Row& r, int at, int words) {
  Vec<T> p, q;
  p.template load<ALIGNED>(static_cast<const T*>(r.p), at, r.n, r.p_off);
  if (HASQ) q.template load<ALIGNED>(static_cast<const T*>(r.q), at, r.n, r.q_off);
  Parts s{0u, 0};
  uint32_t top = 0;
  add_unit<T, HASQ, true>(s, p, q, at, r.drop, top, words);
  return s;
}

// kUnroll iterations' units of this lane from iteration i0 of the span on ...
template <typename T, bool HASQ, bool ALIGNED>
__device__ __forceinline__ void load_units(const Row& r, const Span& sp, int i0, int lane,
                                           Vec<T> (&p)[kUnroll], Vec<T> (&q)[kUnroll]) {
  constexpr int N = Vec<T>::N;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int at = i0 + u < sp.n ? ((sp.first + i0 + u) * 32 + lane) * N - r.shift : r.n;
    p[u].template load<ALIGNED>(static_cast<const T*>(r.p), at, r.n, r.p_off);
    if (HASQ) q[u].template load<ALIGNED>(static_cast<const T*>(r.q), at, r.n, r.q_off);
  }
}
// ... and each one's sum.
template <typename T, bool HASQ, bool ALIGNED>
__device__ __forceinline__ void sum_units(const Row& r, const Span& sp, int i0, int lane,
                                          const Vec<T> (&p)[kUnroll], const Vec<T> (&q)[kUnroll],
                                          Parts (&s)[kUnroll]) {
  constexpr int N = Vec<T>::N;
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    s[u] = Parts{0u, 0};
    add_unit<T, HASQ, false>(s[u], p[u], q[u], ((sp.first + i0 + u) * 32 + lane) * N - r.shift, r.drop, top);
  }
  if (top > 0x3F800000u) {  // (values that are no probabilities: rare, and out of the way)
#pragma unroll 1
    for (int u = 0; u < kUnroll; ++u) {
      const int at = i0 + u < sp.n ? ((sp.first + i0 + u) * 32 + lane) * N - r.shift : r.n;
      s[u] = clamped<T, HASQ, ALIGNED>(r, at, N);
    }
  }
}

// A lane's sums, below 2^52 each, over the warp.
__device__ __forceinline__ int64_t warp_total(int64_t x) {
  const uint32_t lo = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(x) & 0x3FFFFFFu);
  const uint32_t hi = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(x >> 26));
  return (static_cast<int64_t>(hi) << 26) + lo;
}

// Sums of the span's blocks, block j's in lane j.
template <typename T, bool HASQ, bool ALIGNED>
__device__ __forceinline__ int64_t span_sums(const Row& r, const Span& sp, int lane) {
  int64_t mine = 0, sum = 0;
  int j = 0, i0 = 0, left = sp.block;
#pragma unroll 1
  while (i0 < sp.n) {
    Vec<T> p[kUnroll], q[kUnroll];
    Parts s[kUnroll];
    load_units<T, HASQ, ALIGNED>(r, sp, i0, lane, p, q);
    sum_units<T, HASQ, ALIGNED>(r, sp, i0, lane, p, q, s);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) sum += joined(s[u]);
    i0 += kUnroll;
    left -= kUnroll;
    if (left == 0 || i0 >= sp.n) {
      const int64_t all = warp_total(sum);
      if (j == lane) mine = all;
      ++j;
      sum = 0;
      left = sp.block;
    }
  }
  return mine;
}

// The first word of block `j` of the span whose running sum, from `before` on, exceeds
// `place`; every lane gets it.
template <typename T, bool HASQ, bool ALIGNED>
__device__ __noinline__ int find_word(const Row& r, const Span& sp, int j, int64_t before,
                                      int64_t place, int lane) {
  constexpr int N = Vec<T>::N;
  const int end = min(sp.n, (j + 1) * sp.block);
#pragma unroll 1
  for (int i0 = j * sp.block; i0 < end; i0 += kUnroll) {
    Vec<T> p[kUnroll], q[kUnroll];
    Parts s[kUnroll];
    load_units<T, HASQ, ALIGNED>(r, sp, i0, lane, p, q);
    sum_units<T, HASQ, ALIGNED>(r, sp, i0, lane, p, q, s);
    // the iteration, ...
    int it = -1;
    Parts si = s[0];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t sum = warp_joined(s[u]);
      if (it < 0) {
        if (before + sum > place) {
          it = u;
          si = s[u];
        } else {
          before += sum;
        }
      }
    }
    if (it < 0) continue;
    // ... the lane and the word of its unit: lane k < N sums the unit's first k + 1 words
    const int64_t own = joined(si), incl = before + warp_scan(own, lane);
    const int who = __ffs(__ballot_sync(0xFFFFFFFFu, incl > place)) - 1;
    const int64_t start = shfl64(incl - own, who);
    const int at = ((sp.first + i0 + it) * 32 + who) * N - r.shift;
    const int64_t run = start + joined(clamped<T, HASQ, ALIGNED>(r, at, lane + 1));
    return at + __ffs(__ballot_sync(0xFFFFFFFFu, lane < N && run > place)) - 1;
  }
  return -1;
}

// floor(u R) for u in [0, 1) (others are taken to the nearer end), exactly.
__device__ __forceinline__ int64_t place_of(float u, int64_t R) {
  if (!(u > 0.f)) return 0;
  const uint32_t b = __float_as_uint(u);
  const int E = static_cast<int>(b >> 23);
  const uint64_t m = u >= 1.f ? 0xFFFFFFu : E == 0 ? (b & 0x7FFFFFu) : ((b & 0x7FFFFFu) | 0x800000u);
  const int s = u >= 1.f ? 24 : 150 - max(E, 1);  // u = m 2^-s, s >= 24
  const uint64_t r = static_cast<uint64_t>(R);
  const uint64_t lo = m * r, hi = __umul64hi(m, r);
  if (s >= 128) return 0;
  return static_cast<int64_t>(s >= 64 ? hi >> (s - 64) : (lo >> s) | (hi << (64 - s)));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kPerSm) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ int64_t warp_sum[kWarps];
  __shared__ __align__(16) int64_t cta_sum[2][kMaxCluster];  // written by the cluster's CTAs
  __shared__ int first_bad, bad_id;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = a.cluster, rank = blockIdx.y, b = blockIdx.x;
  if (S > 1) cluster_arrive_relaxed();
  if (tid == 0) {
    first_bad = a.n_draft;
    bad_id = 0;
  }
  griddep_wait();
  griddep_launch_dependents();

  // The drafts that stand: thread i looks at draft i.
  const int D = a.n_draft;
  int n = a.n_drafts != nullptr ? a.n_drafts[b] : D;
  const bool step = n >= 0, long_n = n > D;
  n = min(max(n, 0), D);
  const int32_t* drafts = a.draft_tokens + static_cast<int64_t>(b) * D;
  const float* uniform = a.uniform + static_cast<int64_t>(b) * (D + 1);
  int x = -1;
  if (tid < n) x = drafts[tid];
  const float u_last = uniform[D];
  __syncthreads();  // first_bad, bad_id
  if (tid < n) {
    bool stands = false;
    if (x >= 0 && x < a.vocab) {
      const float u = uniform[tid];
      const float p = prob(to_f<T>(static_cast<const T*>(a.target)[(int64_t{b} * (D + 1) + tid) * a.target_stride + x]));
      const float q = a.draft == nullptr
                          ? 1.f
                          : prob(to_f<T>(static_cast<const T*>(a.draft)[(int64_t{b} * D + tid) * a.draft_stride + x]));
      // (products of two 24-bit numbers: exact)
      stands = static_cast<double>(u) * static_cast<double>(q) < static_cast<double>(p);
    } else {
      bad_id = 1;
    }
    if (!stands) atomicMin(&first_bad, tid);
  }
  __syncthreads();
  const int kept = min(first_bad, n);
  if (rank == 0) {
    if (tid == 0) {
      if (long_n || bad_id) record_status(a.status, DSA_ERR_DEVICE_CHECK, SITE_VERIFY, static_cast<uint32_t>(b));
      a.n_kept[b] = step ? kept + 1 : 0;
      if (a.n_drop != nullptr) a.n_drop[b] = step ? n - kept : 0;
    }
    int32_t* out = a.tokens + static_cast<int64_t>(b) * (D + 1);
    for (int i = tid; i <= D; i += kThreads) {
      if (i != kept || !step) out[i] = step && i < kept ? x : -1;  // (i is tid for i < n)
    }
  }
  if (S > 1) cluster_wait();
  if (!step) return;

  Row r;
  r.n = a.vocab;
  r.p = static_cast<const T*>(a.target) + (int64_t{b} * (D + 1) + kept) * a.target_stride;
  const bool rejected = kept < n;
  r.q = rejected && a.draft != nullptr
            ? static_cast<const T*>(a.draft) + (int64_t{b} * D + kept) * a.draft_stride
            : nullptr;
  r.drop = rejected && a.draft == nullptr ? drafts[kept] : -1;
  constexpr int N = Vec<T>::N;

  // At most twice: where nothing of max(p - q, 0) is left, the token is drawn from p.
  for (int pass = 0; pass < 2; ++pass) {
    r.p_off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(r.p) & 15u);
    r.q_off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(r.q) & 15u);
    const bool alike = r.q == nullptr || r.p_off == r.q_off;
    r.shift = alike ? static_cast<int>(r.p_off / sizeof(T)) : 0;
    // The warp's span; at most 32 blocks of it.
    const int iters = (a.vocab + r.shift + 32 * N - 1) / (32 * N);
    const int per = (iters + S * kWarps - 1) / (S * kWarps);
    Span sp;
    sp.first = min(iters, (rank * kWarps + warp) * per);
    sp.n = min(iters, sp.first + per) - sp.first;
    sp.block = kUnroll * ((per + 32 * kUnroll - 1) / (32 * kUnroll));
    const int64_t block_sum = r.q == nullptr ? span_sums<T, false, true>(r, sp, lane)
                              : alike        ? span_sums<T, true, true>(r, sp, lane)
                                             : span_sums<T, true, false>(r, sp, lane);
    const int64_t incl = warp_scan(block_sum, lane);  // over the span's blocks
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t own = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int64_t s = warp_sum[w];
      own += s;
      if (w < warp) before += s;
    }
    int64_t total = own;
    if (S > 1) {
      if (tid < S) {
        const uint32_t there = mapa_shared(smem_u32(&cta_sum[pass][rank]), static_cast<uint32_t>(tid));
        st_cluster_u2(there, make_uint2(static_cast<uint32_t>(own), static_cast<uint32_t>(own >> 32)));
      }
      cluster_sync();
      total = 0;
      for (int k = 0; k < S; ++k) {
        const int64_t s = cta_sum[pass][k];
        total += s;
        if (k < rank) before += s;
      }
    }
    if (total > 0) {
      const int64_t place = place_of(u_last, total);
      const int64_t mine = shfl64(incl, 31);
      if (place >= before && place < before + mine) {  // (one warp of the cluster)
        const uint32_t over = __ballot_sync(0xFFFFFFFFu, before + incl > place);
        const int j = __ffs(over) - 1;
        const int64_t at = before + shfl64(incl - block_sum, j);
        const int word = r.q == nullptr ? find_word<T, false, true>(r, sp, j, at, place, lane)
                         : alike        ? find_word<T, true, true>(r, sp, j, at, place, lane)
                                        : find_word<T, true, false>(r, sp, j, at, place, lane);
        if (lane == 0) a.tokens[static_cast<int64_t>(b) * (D + 1) + kept] = word;
      }
      return;
    }
    if (pass == 1 || (r.q == nullptr && r.drop < 0)) break;
    r.q = nullptr;
    r.drop = -1;
    __syncthreads();  // warp_sum is read
  }
  if (rank == 0 && tid == 0) {  // no probability at all
    a.tokens[static_cast<int64_t>(b) * (D + 1) + kept] = -1;
    record_status(a.status, DSA_ERR_DEVICE_CHECK, SITE_VERIFY, static_cast<uint32_t>(b));
  }
}

template <typename T>
cudaError_t launch_type(const VerifyArgs& args, cudaStream_t s) {
  VerifyArgs a = args;
  // The most CTAs a request with which all requests' are resident at once.
  a.cluster = 1;
  for (int S = kMaxCluster; S > 1; S /= 2) {
    if (static_cast<int64_t>(S) * a.B <= (S > 8 ? 1 : kPerSm) * device_sm_count()) {
      a.cluster = S;
      break;
    }
  }
  if (a.cluster > 8) {
    static std::atomic<int> allowed[64]{};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || allowed[dev].load(std::memory_order_acquire) == 0) {
      e = cudaFuncSetAttribute(verify_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) allowed[dev].store(1, std::memory_order_release);
    }
  }
  return launch_pdl(verify_kernel<T>, dim3(a.B, a.cluster), dim3(kThreads), 0, s, a.cluster, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t s) {
  if (dtype == DSA_DT_F32) return launch_type<float>(a, s);
  return dtype == DSA_DT_F16 ? launch_type<__half>(a, s) : launch_type<__nv_bfloat16>(a, s);
}

}  // namespace dsa
