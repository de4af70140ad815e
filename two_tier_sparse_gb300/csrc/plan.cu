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
// ones together are at most the pool, the ring's size. An id outside the pool moves
// neither way: -1 takes its place. What may be updated in
// place (lengths, the ring's counters) is written by the last CTA to finish,
// when all have read it. The work is a few integer operations a token and four
// words written, so a small step costs its launch and two dependent reads: the
// lengths, then the table or the ring. Divisions are by constants of the call
// (page_rows, ratio, window), as a multiplication and a shift, and sums are held in
// 32 bits: 64 requests of one token take 4.4 us (6.9 with 64-bit sums and divisions), 301
// ragged ones with 9973 tokens 5.8, 1024 of 128 tokens 6.9 (11.0).
#include <algorithm>

#include "kernels.h"

namespace dsa {

namespace {

constexpr int kThreads = 512;
constexpr int kPer = 4;  // consecutive tokens a thread takes: one 16-byte store an array

// n / d for 0 <= n < 2^31: (n + floor(n mul / 2^32)) / 2^shift with shift = ceil(log2 d) and
// mul = floor(2^32 (2^shift - d) / d) + 1 (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994).
__device__ __forceinline__ int div_by(int n, const Divisor& d) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(n), d.mul) + static_cast<uint32_t>(n)) >>
                          d.shift);
}

// Sums over requests, each held at its own cap (one more than what is possible), so that
// 32 bits do.
struct Sums {
  uint32_t tok, pop, push;
};
__device__ __forceinline__ Sums add(const Sums& a, const Sums& b, const Sums& cap) {
  return Sums{min(a.tok + b.tok, cap.tok), min(a.pop + b.pop, cap.pop), min(a.push + b.push, cap.push)};
}

// What one request adds: new tokens, pages popped and pushed; `have` pages now. `bad`:
// lengths that no request can have.
__device__ __forceinline__ Sums request(const PlanArgs& a, int n, int more, int& have, bool& bad) {
  const Sums none{0, 0, 0};
  have = 0;
  if (n < 0) {
    bad = true;
    return none;
  }
  const int lat = div_by(n, a.by_ratio);
  have = div_by(lat, a.by_rows);
  have += have * a.page_rows < lat;
  if (have > a.pages_per_seq) {
    bad = true;
    return none;
  }
  if (more < 0) return Sums{0, 0, static_cast<uint32_t>(have)};  // the request ends
  if (more > 0x7FFFFFFF - n) {
    bad = true;
    return none;
  }
  const int lat1 = div_by(n + more, a.by_ratio);
  int need = div_by(lat1, a.by_rows);
  need += need * a.page_rows < lat1;
  if (need > a.pages_per_seq) {
    bad = true;
    return none;
  }
  return Sums{static_cast<uint32_t>(more), static_cast<uint32_t>(need - have), 0};
}

// The last b with first[b] <= i, first[] ascending with first[0] = 0 and first[B] > i.
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

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int sm[];
  int* cu = sm;                    // [B + 1] new tokens before request b
  int* pop = cu + a.B + 1;         // [B + 1] pages popped
  int* push = pop + a.B + 1;       // [B + 1] pages pushed
  int* len = push + a.B + 1;       // [B] lengths before the step
  int* held = len + a.B;           // [B] pages before the step
  __shared__ Sums warp_sum[kThreads / 32];
  __shared__ int any_bad, last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = a.page_rows;
  const Sums cap{static_cast<uint32_t>(a.max_new) + 1u, static_cast<uint32_t>(a.n_pages) + 1u,
                 static_cast<uint32_t>(a.n_pages) + 1u};
  if (tid == 0) any_bad = 0;
  griddep_wait();
  const int64_t head = a.ring_state[0], tail = a.ring_state[1];

  // Prefix sums: a thread takes `per` consecutive requests.
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  bool bad = false;
  Sums own{0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const int n = a.n_tokens[b], more = a.n_new[b];
    int have;
    const Sums r = request(a, n, more, have, bad);
    len[b] = n;
    held[b] = have;
    cu[b] = static_cast<int>(own.tok);  // (within the thread's requests, for now)
    pop[b] = static_cast<int>(own.pop);
    push[b] = static_cast<int>(own.push);
    own = add(own, r, cap);
  }
  Sums incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums t{__shfl_up_sync(0xFFFFFFFFu, incl.tok, o), __shfl_up_sync(0xFFFFFFFFu, incl.pop, o),
                 __shfl_up_sync(0xFFFFFFFFu, incl.push, o)};
    if (lane >= o) incl = add(incl, t, cap);
  }
  if (lane == 31) warp_sum[warp] = incl;
  Sums before{__shfl_up_sync(0xFFFFFFFFu, incl.tok, 1), __shfl_up_sync(0xFFFFFFFFu, incl.pop, 1),
              __shfl_up_sync(0xFFFFFFFFu, incl.push, 1)};
  if (lane == 0) before = Sums{0, 0, 0};
  __syncthreads();  // any_bad is cleared, the warps' sums are written
  if (bad) any_bad = 1;
  Sums total{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) before = add(before, total, cap);
    total = add(total, warp_sum[w], cap);
  }
  __syncthreads();  // any_bad is known
  // All or nothing: the same decision in every CTA.
  const int64_t free_pages = tail - head;
  const bool ok = !any_bad && total.tok <= static_cast<uint32_t>(a.max_new) && head >= 0 &&
                  free_pages >= 0 && total.pop <= free_pages &&
                  free_pages + total.push <= a.n_pages;
  for (int b = b0; b < b1; ++b) {
    cu[b] = ok ? cu[b] + static_cast<int>(before.tok) : 0;
    pop[b] = ok ? pop[b] + static_cast<int>(before.pop) : 0;
    push[b] = ok ? push[b] + static_cast<int>(before.push) : 0;
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
  auto in_pool = [&](int page) -> bool { return page >= 0 && page < a.n_pages; };

  // The table's new entries, and the pages of ended requests back to the ring: from the
  // grid's last thread down, so that in a small step they fall to other warps than the
  // tokens.
  for (int k = gstep - 1 - gtid; k < n_pop; k += gstep) {
    const int b = find(pop, a.B, k);
    const int pg = a.ring[ring_at(head_m, k)];  // (outside the pool: its tokens report it)
    a.table[static_cast<int64_t>(b) * a.pages_per_seq + held[b] + (k - pop[b])] = in_pool(pg) ? pg : -1;
  }
  for (int k = gstep - 1 - gtid; k < n_push; k += gstep) {
    const int b = find(push, a.B, k);
    const int pg = a.table[static_cast<int64_t>(b) * a.pages_per_seq + (k - push[b])];
    a.ring[ring_at(tail_m, k)] = in_pool(pg) ? pg : -1;
    if (!in_pool(pg) && pg != -1) {
      record_status(a.status, DSA_ERR_DEVICE_CHECK, SITE_PLAN, static_cast<uint32_t>(b));
    }
  }

  // Tokens: kPer consecutive ones a thread; rows past the last token are empty.
  for (int i0 = kPer * gtid; i0 < a.max_new; i0 += kPer * gstep) {
    int seq[kPer], pos[kPer], lslot[kPer], wslot[kPer], page[kPer];
    int b = i0 < n_tok ? find(cu, a.B, i0) : 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = i0 + k;
      seq[k] = lslot[k] = wslot[k] = -1;
      pos[k] = 0;
      page[k] = 0;
      if (i < n_tok) {
        while (i >= cu[b + 1]) ++b;
        const int n = len[b], p = n + (i - cu[b]), after = n + (cu[b + 1] - cu[b]);
        seq[k] = b;
        pos[k] = p;
        if (p >= after - a.window) {
          wslot[k] = b * a.window + (p - div_by(p, a.by_window) * a.window);
        }
        const int done = div_by(p + 1, a.by_ratio);
        if (done * a.ratio == p + 1) {  // the token completes latent done - 1
          const int j = done - 1, pg = div_by(j, a.by_rows), have = held[b];
          lslot[k] = j - pg * R;
          page[k] = pg < have ? a.table[static_cast<int64_t>(b) * a.pages_per_seq + pg]
                              : a.ring[ring_at(head_m, pop[b] + pg - have)];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (lslot[k] >= 0) {
        if (in_pool(page[k])) {
          lslot[k] += page[k] * R;
        } else {
          lslot[k] = -1;
          record_status(a.status, DSA_ERR_DEVICE_CHECK, SITE_PLAN, static_cast<uint32_t>(seq[k]));
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
    if (!ok) return len[b];
    return push[b + 1] > push[b] || a.n_new[b] < 0 ? 0 : len[b] + (cu[b + 1] - cu[b]);
  };
  for (int b = gtid; b <= a.B; b += gstep) {
    a.cu_new[b] = cu[b];
    if (b < a.B) {
      const int n = max(after_of(b), 0);
      a.n_latents[b] = div_by(n, a.by_ratio);
      a.swa_len[b] = min(n, a.window);
    }
  }
  if (gridDim.x > 1) {
    __syncthreads();
    if (tid == 0) {
      last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
      if (last) *a.ticket = 0u;
    }
    __syncthreads();
    if (!last) return;
  }
  for (int b = tid; b < a.B; b += kThreads) a.n_tokens_out[b] = after_of(b);
  if (tid == 0) {
    a.ring_state_out[0] = ok ? head + total.pop : head;
    a.ring_state_out[1] = ok ? tail + total.push : tail;
  }
}

Divisor divisor(int d) {
  Divisor r;
  r.shift = 0;
  while ((int64_t{1} << r.shift) < d) ++r.shift;
  r.mul = static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << r.shift) - d)) / d + 1);
  return r;
}

}  // namespace

cudaError_t launch_plan(const PlanArgs& args, cudaStream_t s) {
  PlanArgs a = args;
  a.by_ratio = divisor(a.ratio);
  a.by_rows = divisor(a.page_rows);
  a.by_window = divisor(a.window);
  const int smem = (5 * a.B + 3) * 4;
  static std::atomic<int> smem_set[64]{};
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(plan_kernel),
                              (5 * DSA_PLAN_MAX_REQUESTS + 3) * 4, smem_set);
  if (e != cudaSuccess) return e;
  // A CTA for every 2048 tokens (each thread one group of four), at most one an SM.
  const int64_t want = (static_cast<int64_t>(a.max_new) + kPer * kThreads - 1) / (kPer * kThreads);
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, device_sm_count())));
  return launch_pdl(plan_kernel, dim3(grid), dim3(kThreads), static_cast<size_t>(smem), s, 1, a);
}

}  // namespace dsa
