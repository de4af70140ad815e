// The plan of a serving step, from its request lengths: the block table grown
// by pages popped from a ring of free pages (an ended request's pages pushed
// back), and for every new token its request, position and the cache rows it
// will be written to.
//
// One launch. Every CTA works out the prefix sums over the requests (new
// tokens, pages popped, pages pushed) by itself from the lengths, so no CTA
// waits for another; tokens and pages are then dealt out over the grid. A page
// that a request gains in this step is known from the prefix sums and the
// ring, so a token's slot never reads a table entry that this launch writes.
// Popped and pushed positions of the ring never meet: free pages and pushed
// ones together are at most the pool, the ring's size. What may be updated in
// place (lengths, the ring's counters) is written by the last CTA to finish,
// when all have read it. The work is a few integer operations a token and four
// words written, so a small step costs its launch and two dependent reads.
#include <algorithm>

#include "kernels.h"

namespace dsa {

namespace {

constexpr int kThreads = 512;
constexpr int kPer = 4;  // consecutive tokens a thread takes: one 16-byte store an array

struct Sums {
  int64_t tok, pop, push;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return Sums{a.tok + b.tok, a.pop + b.pop, a.push + b.push};
}
__device__ __forceinline__ Sums shfl_up(const Sums& v, int o) {
  return Sums{__shfl_up_sync(0xFFFFFFFFu, v.tok, o), __shfl_up_sync(0xFFFFFFFFu, v.pop, o),
              __shfl_up_sync(0xFFFFFFFFu, v.push, o)};
}

// What one request adds: new tokens, pages popped and pushed. `bad`: lengths
// that no request can have.
__device__ __forceinline__ Sums request(const PlanArgs& a, int b, bool& bad) {
  const int n = a.n_tokens[b], add = a.n_new[b];
  const int R = a.page_rows;
  if (n < 0) {
    bad = true;
    return Sums{0, 0, 0};
  }
  const int have = (n / a.ratio + R - 1) / R;
  if (have > a.pages_per_seq) {
    bad = true;
    return Sums{0, 0, 0};
  }
  if (add < 0) return Sums{0, 0, have};  // the request ends
  const int64_t after = int64_t{n} + add;
  const int64_t need = (after / a.ratio + R - 1) / R;
  if (after > 0x7FFFFFFF || need > a.pages_per_seq) {
    bad = true;
    return Sums{0, 0, 0};
  }
  return Sums{add, need - have, 0};
}

// The last b with first[b] <= i, first[] ascending with first[0] = 0.
__device__ __forceinline__ int find(const int* first, int B, int i) {
  int lo = 0, hi = B;  // first[lo] <= i < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) {
      lo = mid;
    } else {
      hi = mid;
    }
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(PlanArgs a) {
  extern __shared__ int sm[];
  int* cu = sm;                    // [B + 1] new tokens before request b
  int* pop = cu + a.B + 1;         // [B + 1] pages popped
  int* push = pop + a.B + 1;       // [B + 1] pages pushed
  __shared__ Sums warp_sum[kThreads / 32];
  __shared__ int any_bad;
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = a.page_rows;
  const int64_t head = a.ring_state[0], tail = a.ring_state[1];
  if (tid == 0) any_bad = 0;
  __syncthreads();

  // Prefix sums: a thread takes `per` consecutive requests.
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  bool bad = false;
  Sums own{0, 0, 0};
  for (int b = b0; b < b1; ++b) own = own + request(a, b, bad);
  Sums incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums t = shfl_up(incl, o);
    if (lane >= o) incl = incl + t;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (bad) any_bad = 1;
  __syncthreads();
  Sums before{incl.tok - own.tok, incl.pop - own.pop, incl.push - own.push}, total{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before = before + warp_sum[w];
    total = total + warp_sum[w];
  }
  // All or nothing: the same decision in every CTA.
  const bool ok = !any_bad && total.tok <= a.max_new && head >= 0 && tail >= head &&
                  total.pop <= tail - head && tail - head + total.push <= a.n_pages;
  Sums at = before;
  for (int b = b0; b < b1; ++b) {
    cu[b] = ok ? static_cast<int>(at.tok) : 0;
    pop[b] = ok ? static_cast<int>(at.pop) : 0;
    push[b] = ok ? static_cast<int>(at.push) : 0;
    at = at + request(a, b, bad);
  }
  if (tid == 0) {
    cu[a.B] = ok ? static_cast<int>(total.tok) : 0;
    pop[a.B] = ok ? static_cast<int>(total.pop) : 0;
    push[a.B] = ok ? static_cast<int>(total.push) : 0;
    if (!ok && blockIdx.x == 0) record_status(a.status, DSA_ERR_DEVICE_CHECK, SITE_PLAN, any_bad);
  }
  __syncthreads();
  const int gtid = blockIdx.x * kThreads + tid, gstep = static_cast<int>(gridDim.x) * kThreads;
  const int n_tok = cu[a.B], n_pop = pop[a.B], n_push = push[a.B];
  const int head_m = ok ? static_cast<int>(head % a.n_pages) : 0;
  const int tail_m = ok ? static_cast<int>(tail % a.n_pages) : 0;
  auto ring_at = [&](int base, int k) -> int {  // position base + k of the ring
    const int64_t i = int64_t{base} + k;
    return static_cast<int>(i >= a.n_pages ? i - a.n_pages : i);
  };

  // The table's new entries, and the pages of ended requests back to the ring.
  for (int k = gtid; k < n_pop; k += gstep) {
    const int b = find(pop, a.B, k);
    const int have = (a.n_tokens[b] / a.ratio + R - 1) / R;
    a.table[static_cast<int64_t>(b) * a.pages_per_seq + have + (k - pop[b])] =
        a.ring[ring_at(head_m, k)];
  }
  for (int k = gtid; k < n_push; k += gstep) {
    const int b = find(push, a.B, k);
    a.ring[ring_at(tail_m, k)] = a.table[static_cast<int64_t>(b) * a.pages_per_seq + (k - push[b])];
  }

  // Tokens: kPer consecutive ones a thread; rows past the last token are empty.
  for (int i0 = kPer * gtid; i0 < a.max_new; i0 += kPer * gstep) {
    int seq[kPer], pos[kPer], lslot[kPer], wslot[kPer];
    int b = i0 < n_tok ? find(cu, a.B, i0) : 0;
    int nb = -1, n = 0, have = 0, after = 0;  // of request nb
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = i0 + k;
      seq[k] = lslot[k] = wslot[k] = -1;
      pos[k] = 0;
      if (i < n_tok) {
        while (i >= cu[b + 1]) ++b;
        if (b != nb) {
          nb = b;
          n = a.n_tokens[b];
          have = (n / a.ratio + R - 1) / R;
          after = n + (cu[b + 1] - cu[b]);
        }
        const int p = n + (i - cu[b]);
        seq[k] = b;
        pos[k] = p;
        if (p >= after - a.window) wslot[k] = b * a.window + p % a.window;
        const int j = (p + 1) / a.ratio - 1;
        if ((j + 1) * a.ratio == p + 1) {  // the token completes latent j
          const int pg = j / R;
          const int page = pg < have ? a.table[static_cast<int64_t>(b) * a.pages_per_seq + pg]
                                     : a.ring[ring_at(head_m, pop[b] + pg - have)];
          if (page >= 0 && page < a.n_pages) {
            lslot[k] = page * R + (j - pg * R);
          } else {
            record_status(a.status, DSA_ERR_DEVICE_CHECK, SITE_PLAN, static_cast<uint32_t>(b));
          }
        }
      }
    }
    if (i0 + kPer <= a.max_new) {
      *reinterpret_cast<int4*>(a.token_seq + i0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      *reinterpret_cast<int4*>(a.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(a.latent_slots + i0) =
          make_int4(lslot[0], lslot[1], lslot[2], lslot[3]);
      *reinterpret_cast<int4*>(a.window_slots + i0) =
          make_int4(wslot[0], wslot[1], wslot[2], wslot[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (i0 + k < a.max_new) {
          a.token_seq[i0 + k] = seq[k];
          a.positions[i0 + k] = pos[k];
          a.latent_slots[i0 + k] = lslot[k];
          a.window_slots[i0 + k] = wslot[k];
        }
      }
    }
  }

  // Per request. The lengths and the ring's counters may be updated in place:
  // the last CTA writes them, when every CTA has read what it needs.
  auto after_of = [&](int b) -> int {
    const int n = a.n_tokens[b];
    if (!ok) return n;
    return a.n_new[b] < 0 ? 0 : n + (cu[b + 1] - cu[b]);
  };
  for (int b = gtid; b <= a.B; b += gstep) {
    a.cu_new[b] = cu[b];
    if (b < a.B) {
      const int n = max(after_of(b), 0);
      a.n_latents[b] = n / a.ratio;
      a.swa_len[b] = min(n, a.window);
    }
  }
  __shared__ int last;
  __syncthreads();
  if (tid == 0) {
    last = 1;
    if (gridDim.x > 1) {
      last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
      if (last) *a.ticket = 0u;
    }
  }
  __syncthreads();
  if (!last) return;
  for (int b = tid; b < a.B; b += kThreads) a.n_tokens_out[b] = after_of(b);
  if (tid == 0) {
    a.ring_state_out[0] = ok ? head + total.pop : head;
    a.ring_state_out[1] = ok ? tail + total.push : tail;
  }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t s) {
  const int smem = 3 * (a.B + 1) * 4;
  static std::atomic<int> smem_set[64]{};
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(plan_kernel),
                              3 * (DSA_PLAN_MAX_REQUESTS + 1) * 4, smem_set);
  if (e != cudaSuccess) return e;
  // A CTA for every 2048 tokens (each thread one group of four), at most one an SM.
  const int64_t want = (static_cast<int64_t>(a.max_new) + kPer * kThreads - 1) / (kPer * kThreads);
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, device_sm_count())));
  return launch_pdl(plan_kernel, dim3(grid), dim3(kThreads), static_cast<size_t>(smem), s, 1, a);
}

}  // namespace dsa
