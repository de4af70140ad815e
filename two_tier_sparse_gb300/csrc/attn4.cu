// S5 - S7 over a cache held in 4 bits (DSA_KV_MXFP4): decode attention of 64
// heads over the selected latents and the sliding window under one softmax,
// the rows e2m1 codes with a power-of-two scale per 32 elements.
//
//   S   = Q . KV^T    (.ws, M = 64 heads, N = 64 rows, K = 512: rows 0..31 in lanes 0..63,
//                      rows 32..63 in lanes 64..127, 32 columns)
//   O^T += KV^T . P^T (four M = 128 slices of the 512 latent dims, N = 64 heads,
//                      K = the tile's rows; the KV tile is read as an MN-major operand)
//
// A row is 272 bytes, so a tile's rows fit in registers on their way: eight
// loader warps read the next tile's codes (16 bytes a lane: 32 elements, one scale) into
// one set of registers while they convert this tile's from another to bf16 in a swizzled
// operand slot (with one set, read after the conversion, the loads' latency was
// in every tile: 64 sequences took 17.5 us, 17.2 with two).
// bf16 holds every code times every scale exactly, so Q stays as it is given
// and the MMAs see the cache's own values.
//
// The MMAs are bound by the operands they read from shared memory at 128 bytes
// a clock (a step of K = 16 measured 31 clocks for M = 64, N = 64, 46 for
// M = 128, N = 64, whose extra lanes would hold no heads), provided that a
// converged warp issues them with one lane elected: from a lane that has
// branched off, a step took 58, descriptors moving through vector registers.
// 64 rows a tile use the Q operand twice as well as 32. The weight-stationary
// form's layout gives every math thread 32 scores of one head, so four warps
// share the softmax.
//
// A tile takes about 3300 clocks: the loaders ~2000 to convert it (two instructions of
// every three on the ALU pipe, at half rate) and ~650 to read the next one, the MMAs 1730 at
// least, and shared memory ~2300 for what all of them move, so they slow one
// another; the chain conversion - QK^T - softmax - PV over two slots is as long. 640 rows a
// sequence: 1 sequence 10.8 us, 64 x 131072 16.6 us, 152 22.4 us (of those ~6 before the first and
// after the last tile), 200 paged ragged 35.0 us.
//
// The split over a cluster of S CTAs, the lazy softmax maximum and the roles
// are those of the attention over bf16 rows. The CTAs of a cluster exchange their
// (max, sum) first, so each scales its partial output by its final weight and the
// merge is a sum. The partial outputs keep the upper 24 bits of their fp32 value
// (sign, exponent, 15 mantissa bits), as a 16-bit and an 8-bit part: with bf16 parts
// their rounding would add to the output's own, which is of the same size. The exchange is
// bound by what an SM can send to others: 14 bytes a clock measured, by 16-byte
// stores, bulk copies or remote loads alike (86 KB a CTA of eight: 6100 clocks; 49 KB a CTA
// of two: 3800).
#include <algorithm>
#include <cstddef>

#include "attn_math.cuh"
#include "kv_format.cuh"

namespace dsa {

namespace {

constexpr int kRows = 64;                          // rows of a tile
constexpr int kHalf = kRows / 2;                   // scores of a math thread
constexpr int kSlots = 2;
constexpr int kLoadWarp0 = 4;
constexpr int kLoadWarps = 8;
constexpr int kMmaWarp = kLoadWarp0 + kLoadWarps;  // 12: QK^T issuer (and TMEM owner)
constexpr int kPvWarp = kMmaWarp + 1;              // 13: PV issuer
constexpr int kThreads = 32 * (kPvWarp + 1);       // 448
constexpr int kMathBar = 1;                        // named barrier of the 128 math threads
constexpr int kEpiBar = 2;                         // of the epilogue (math and loader warps)
constexpr int kEpiThreads = 32 * kMmaWarp;         // 384
constexpr int kEpiGroups = kEpiThreads / 128;      // 3 groups of four warps (TMEM lane quarters)

// Shared memory, offsets from a 1024-aligned base.
constexpr int kAtomBytes = kRows * 128;            // 64 dims of a tile's rows
constexpr int kSlotBytes = 8 * kAtomBytes;
constexpr int kQ = 0;                              // 8 atoms x 64 heads x 128 B
constexpr uint32_t kQBytes = kHeads * kLatent * 2;
constexpr int kP = kQ + static_cast<int>(kQBytes); // 64 heads x 64 rows bf16
constexpr int kPBytes = kHeads * 128;
constexpr int kKV = kP + kPBytes;                  // the two slots
constexpr int kKVBytes = kSlots * kSlotBytes;
constexpr int kIds = kKV + kKVBytes;               // compacted latent rows
constexpr int kMl = kIds + kMaxKTokens * 4;        // [8][64] (max, sum) of each CTA's rows
constexpr int kMisc = kMl + kMaxAttnSplits * kHeads * 8;
constexpr int kMiscBytes = 2048;
constexpr int kSmemBytes = kMisc + kMiscBytes + 1024;  // + alignment slack of the base
static_assert(kSmemBytes <= 227 * 1024 && kIds % 16 == 0 && kMisc % 16 == 0, "shared memory");
constexpr int kTmemCols = 512;  // S[b]: cols [32 b, 32 b + 32); O^T slice m: [kTmemO + 64 m, ...)
constexpr int kTmemO = 64;

// What a CTA gives the one finishing dims [p D, p D + D), D = 512 / S (itself
// included): its part of the output for those dims, in planes of D x 16 bytes: plane u < 8 the upper 16 bits of heads
// 8 u .. 8 u + 7 for each dim, plane 8 + u the next 8 bits of heads 16 u ..
// 16 u + 15, so that a warp (32 dims) writes and reads 512 contiguous bytes.
__host__ __device__ constexpr int xchg_bytes(int S) { return (kLatent / S) * 192; }
static_assert(2 * xchg_bytes(2) <= kKVBytes && 4 * xchg_bytes(4) <= kKVBytes &&
                  kMaxAttnSplits * xchg_bytes(kMaxAttnSplits) <= kKVBytes,
              "receive areas fit the slots");

struct Misc {
  uint64_t kv_full[kSlots][2], kv_empty[kSlots][2], s_full[2], s_free[2], p_full, p_empty;
  uint64_t q_done, ids_ready;
  uint64_t o_done;  // every MMA of the CTA has completed
  uint32_t tmem_base;
  int abort;
  int n_sel;
  int warp_cnt[4];
  float mx[2][2][kHeads];  // a tile's largest score of each head in rows 0..31 and 32..63
  alignas(16) float alpha[kHeads];
  alignas(16) float wgt[kHeads];  // what a head's O is scaled by
};
static_assert(sizeof(Misc) <= kMiscBytes, "misc block");

// A converged warp's bounded wait; every lane gets the same answer (a lane whose
// wait ran out takes the warp with it), so that warp-wide instructions after it
// stay converged. The loop is kept out of line: the roles' code runs from a small
// instruction cache, and inlined at every wait it was a large part of it.
__device__ __noinline__ bool wait_loop(uint64_t* bar, uint32_t parity, volatile int* abort,
                                       DeviceStatus* st) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_abortable(bar, parity, abort, st, SITE_ATTN));
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Misc* m,
                                         DeviceStatus* st) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(smem_u32(bar), parity))) return true;
  return wait_loop(bar, parity, &m->abort, st);
}

__device__ __noinline__ void report(DeviceStatus* st, uint32_t detail) {
  record_status(st, DSA_ERR_DEVICE_CHECK, SITE_ATTN, detail);
}

// bf16(v[i]) to row h0 + i of a shared-memory image of the output (`row` bytes a head), lane
// l at dim d (2 bytes): a warp's lanes hold neighbouring dims, so a store touches
// each bank once. The image then leaves by coalesced 16-byte stores. (From the
// registers, 64-byte pieces of eight heads by exchanged 16-byte stores took 2300
// clocks for every 32 heads x 384 dims; this takes 700. Bulk copies, one a head, took
// a microsecond to read the image.)
template <int NH>
__device__ __forceinline__ void stage_heads(uint32_t image, uint32_t row, int h0, int d,
                                            const float (&v)[NH]) {
  const uint32_t at = image + static_cast<uint32_t>(h0) * row + 2u * static_cast<uint32_t>(d);
#pragma unroll
  for (int j = 0; j < NH; j += 2) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(v[j], v[j + 1]);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&x);
    asm volatile(
        "{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n st.shared.b16 [%0], a;\n"
        " st.shared.b16 [%1], b;\n}\n" ::"r"(at + j * row),
        "r"(at + (j + 1) * row), "r"(w)
        : "memory");
  }
}

// kParts: parts of a tile (in dims) that its slot is handed on in: QK^T begins with the first
// while the second is converted, and the tile after the next is converted into what PV has read
// first. (Two parts take a tile from 1.8 to 1.6 us; a CTA of two tiles, as clusters of
// eight have them, is faster in one part: 10.8 us where two take 11.1.)
template <int kParts>
__global__ void __launch_bounds__(kThreads, 1)
    attn4_kernel(AttnArgs a, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (sbase - raw);
  Misc* misc = reinterpret_cast<Misc*>(gbase + kMisc);
  int32_t* ids = reinterpret_cast<int32_t*>(gbase + kIds);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x;
  const int split = blockIdx.y;  // rank in the cluster
  const int S = a.splits;
  const bool paired = S > 1;
  int n_vis = 0, n_sw = 0;
  if (!a.wait_first) {  // (on their way while the barriers are set up)
    n_vis = a.n_latents[b];
    n_sw = a.swa_len[b];
  }
  // A math thread's token ids, read once the previous kernel's are final.
  constexpr int kPer = kMaxKTokens / 128;  // 4
  int my[kPer];
  auto read_ids = [&]() {
    const int32_t* tk = a.token_ids + static_cast<int64_t>(b) * a.k_tokens;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid * kPer + j;
      my[j] = i < a.k_tokens ? tk[i] : -1;
    }
  };

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      for (int p = 0; p < kParts; ++p) {
        mbar_init(&misc->kv_full[i][p], kLoadWarps);
        mbar_init(&misc->kv_empty[i][p], 1);
      }
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&misc->s_full[i], 1);
      mbar_init(&misc->s_free[i], 4);
    }
    mbar_init(&misc->p_full, 4);
    mbar_init(&misc->p_empty, 1);
    mbar_init(&misc->q_done, 1);     // the TMA loads of Q (expect-tx arrival + 64 KB)
    mbar_init(&misc->ids_ready, 1);  // the math warps compacted the token ids
    mbar_init(&misc->o_done, 1);     // the PV issuer's last commit
    misc->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(&misc->tmem_base, kTmemCols);
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();  // barriers initialised, tensor memory allocated
  tc_fence_after();
  // The peers' barriers are initialised before any remote access: every
  // thread arrives here and waits before its first cluster access.
  if (paired) cluster_arrive_relaxed();

  if (a.wait_first) {
    griddep_wait();
    n_vis = a.n_latents[b];
    n_sw = a.swa_len[b];
    if (tid < 128) read_ids();
  }
  if (n_sw < 0 || n_sw > a.window) {
    if (tid == 0 && split == 0) report(a.status, static_cast<uint32_t>(b));
    n_sw = n_sw < 0 ? 0 : a.window;
  }
  if (n_vis > a.lat_stride) n_vis = static_cast<int>(a.lat_stride);
  const bool paged = a.pages.table != nullptr;
  const int64_t lat_row0 = paged ? 0 : static_cast<int64_t>(b) * a.lat_stride;
  // This CTA's rows: its part of the window rows first (inputs of the step,
  // read while the previous kernel still selects the tokens), then its part of
  // the selected latents.
  const int64_t wrow0 = static_cast<int64_t>(b) * a.window;
  const int lg_s = 31 - __clz(S);
  const int w_part = (n_sw + S - 1) >> lg_s;
  const int w_begin = min(n_sw, split * w_part);
  const int w_cnt = min(n_sw, w_begin + w_part) - w_begin;
  auto sel_range = [&](int n_sel, int& s_begin, int& s_cnt) {
    const int h = (n_sel + S - 1) >> lg_s;
    s_begin = min(n_sel, split * h);
    s_cnt = min(n_sel, s_begin + h) - s_begin;
  };
  const uint32_t tmem = misc->tmem_base;

  if (warp == kLoadWarp0 && lane == 0) {
    // Q does not depend on the ids: eight boxes of 64 heads x 64 dims, each
    // landing as one 128-byte-swizzled atom of the QK^T A operand.
    tma_prefetch_map(&qmap);
    mbar_arrive_expect_tx(&misc->q_done, kQBytes);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      tma_load_2d(sbase + kQ + c * (kHeads * 128), &qmap, 64 * c, b * kHeads, &misc->q_done);
    }
  }

  // Compact the valid token ids (>= 0 and < n_vis) in order (math threads,
  // once the previous kernel's ids are final).
  if (tid < 128) {
    if (!a.wait_first) {
      griddep_wait();
      read_ids();
    }
    int cnt = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      int id = my[j];
      if (id >= n_vis) {
        if (split == 0) report(a.status, static_cast<uint32_t>(id));
        id = -1;
      }
      if (paged && id >= 0) {
        const int64_t row = paged_row(a.pages, b, id);
        if (row < 0 && split == 0) report(a.status, static_cast<uint32_t>(id));
        id = static_cast<int>(row);
      }
      my[j] = id;
      cnt += id >= 0 ? 1 : 0;
    }
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) misc->warp_cnt[warp] = incl;
    named_sync(kMathBar, 128);
    int before = incl - cnt;
    for (int w = 0; w < warp; ++w) before += misc->warp_cnt[w];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (my[j] >= 0) ids[before++] = my[j];
    }
    if (tid == 127) misc->n_sel = before;
    named_sync(kMathBar, 128);
    if (tid == 0) mbar_arrive(&misc->ids_ready);
  }

  // State the epilogue warps (math and loaders) share: the softmax statistics
  // of head tid (threads 0..63), whether every wait succeeded, the tile count.
  float m_run = -INFINITY, l_run = 0.f;
  bool ok = true;
  int n_tiles_e = 0;

  if (warp >= kLoadWarp0 && warp < kMmaWarp) {
    // ---------------- loaders ----------------
    // Loader warp w fills rows [8 w, 8 w + 8) of every tile. Lane l has row 8 w + r, r = l % 8,
    // and of it the 16-byte pieces g, g + 4, g + 8 and g + 12, g = l / 8: elements
    // [32 j, 32 j + 32) under scale j for piece j. The eight lanes of a 16-byte store then write
    // one chunk of eight different rows, which the swizzle spreads over all banks,
    // and every address is a lane's constant. The next tile's pieces are read into the
    // registers as soon as this tile's are converted; one copy of the code does every pass (the first only reads, the last only
    // converts). Rows without a source are zeros.
    const int w = warp - kLoadWarp0;
    const uint32_t r = lane & 7, g = lane >> 3;
    const uint8_t* lat = reinterpret_cast<const uint8_t*>(a.latents);
    const uint8_t* swa = reinterpret_cast<const uint8_t*>(a.swa);
    bool have_ids = false;
    int s_begin = 0, n_rows_cta = w_cnt, n_tiles = 0;
    uint32_t to[4];  // where word n of piece g goes in a slot (piece g + 4 i: two atoms on each)
#pragma unroll
    for (uint32_t n = 0; n < 4; ++n) {
      to[n] = sbase + kKV + (g >> 1) * kAtomBytes + (8u * w + r) * 128u +
              (((4u * (g & 1u) + n) ^ r) << 4);
    }
    int next = 0, done = 0;  // tiles read, tiles converted
    // Reads the next tile into (code, scales): 1; 0 if it needs ids that are not there yet (and
    // `block` is not set); -1 if there is none, or the wait for the ids ran out (ok is false).
    auto read = [&](uint4 (&code)[4], uint4& scales, bool block) -> int {
      if (!have_ids && (next + 1) * kRows > w_cnt) {
        if (!block && !__all_sync(0xFFFFFFFFu, mbar_try_wait(smem_u32(&misc->ids_ready), 0u))) return 0;
        if (!wait_bar(&misc->ids_ready, 0u, misc, a.status)) {
          ok = false;
          return -1;
        }
        int s_cnt;
        sel_range(misc->n_sel, s_begin, s_cnt);
        n_rows_cta = w_cnt + s_cnt;
        n_tiles = (n_rows_cta + kRows - 1) / kRows;
        have_ids = true;
      }
      if (have_ids && next >= n_tiles) return -1;
      const uint8_t* src = nullptr;  // this lane's row of the tile
      const int row_g = next * kRows + 8 * w + static_cast<int>(r);
      if (row_g < n_rows_cta) {
        if (row_g < w_cnt) {
          const int64_t row = wrow0 + w_begin + row_g;
          if (DSA_DCHECK(row >= 0 && row < a.swa_rows, a.status, SITE_ATTN, row)) {
            src = swa + row * kRow4Bytes;
          }
        } else {
          const int64_t row = lat_row0 + ids[s_begin + row_g - w_cnt];
          if (DSA_DCHECK(row >= 0 && row < a.lat_rows, a.status, SITE_ATTN, row)) {
            src = lat + row * kRow4Bytes;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) code[i] = make_uint4(0u, 0u, 0u, 0u);
      scales = make_uint4(0u, 0u, 0u, 0u);
      if (src != nullptr) {
        const uint4* p = reinterpret_cast<const uint4*>(src);
#pragma unroll
        for (int i = 0; i < 4; ++i) code[i] = ld_ordered(p + g + 4 * i);
        scales = ld_ordered(p + kRow4Codes / 16);
      }
      ++next;
      return 1;
    };
    // Converts tile `done` into its slot.
    auto convert = [&](const uint4 (&code)[4], const uint4& scales) {
      const int sl = done % kSlots;
      const uint32_t slot = static_cast<uint32_t>(sl * kSlotBytes);
      const uint32_t sw[4] = {scales.x, scales.y, scales.z, scales.w};
      // (a warp past the last step of 16 rows has nothing that PV reads)
      const bool needed = 8 * (w & ~1) < n_rows_cta - done * kRows;
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        if (done >= kSlots && !wait_bar(&misc->kv_empty[sl][p],
                                        static_cast<uint32_t>(((done / kSlots) - 1) & 1), misc,
                                        a.status)) {
          ok = false;
          return;
        }
        if (needed) {
#pragma unroll
          for (int i = p * (4 / kParts); i < (p + 1) * (4 / kParts); ++i) {
            // piece g + 4 i: its scale is byte g of word i
            const uint32_t f = mx4_scale_bf16x2((sw[i] >> (8u * g)) & 0xFFu);
            const uint32_t cw[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              st_shared_v4(to[n] + slot + 2 * i * kAtomBytes, mx4_decode8(cw[n], f));
            }
          }
        }
        fence_proxy_async_smem();  // the MMAs read the tile through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(&misc->kv_full[sl][p]);
      }
      ++done;
    };
    // One pass: the next tile is read into one set of registers (x) while the one before it
    // is converted from the other (y).
    auto pass = [&](uint4 (&x)[4], uint4& xs, const uint4 (&y)[4], const uint4& ys) -> bool {
      const bool at_hand = next > done;
      int got = read(x, xs, !at_hand);
      if (ok && at_hand) convert(y, ys);
      if (ok && got == 0) got = read(x, xs, true);
      return ok && got > 0;
    };
    uint4 code0[4], code1[4], scales0, scales1;
    while (pass(code0, scales0, code1, scales1) && pass(code1, scales1, code0, scales0)) {
    }
    n_tiles_e = have_ids ? n_tiles : 0;
  } else if (warp == kMmaWarp || warp == kPvWarp) {
    // ---------------- MMA issuers ----------------
    int n_rows_cta = 0;
    if (wait_bar(&misc->ids_ready, 0u, misc, a.status)) {
      int s_begin, s_cnt;
      sel_range(misc->n_sel, s_begin, s_cnt);
      n_rows_cta = w_cnt + s_cnt;
    }
    const int n_tiles = (n_rows_cta + kRows - 1) / kRows;
    // PV(t) is issued only after the softmax of tile t, hence after QK^T(t)
    // completed: its commit alone frees the tile's slot, and the PV issuer's
    // last commit means every MMA of the CTA has completed.
    const uint32_t leader = elect_leader();
    const uint64_t kv_mn = sw128_desc(sbase + kKV, kAtomBytes, 1024);  // slot 0, MN-major
    const uint64_t kv_k = sw128_desc(sbase + kKV, 16, 1024);           // slot 0, K-major
    const uint64_t q_k = sw128_desc(sbase + kQ, 16, 1024);
    const uint64_t p_k = sw128_desc(sbase + kP, 16, 1024);
    auto lo = [](uint64_t d) { return static_cast<uint32_t>(d); };
    auto hi = [](uint64_t d) { return static_cast<uint32_t>(d >> 32); };
    if (warp == kPvWarp) {
      constexpr uint32_t idesc_o = mma_idesc(128, kHeads, true, true, false);
      for (int t = 0; t < n_tiles; ++t) {
        const int sl = t % kSlots;
        if (!wait_bar(&misc->p_full, static_cast<uint32_t>(t & 1), misc, a.status)) break;
        tc_fence_after();
        fence_proxy_async_smem();
        uint32_t a_lo = lo(kv_mn) + static_cast<uint32_t>(sl * kSlotBytes >> 4);
        const int steps = (n_rows_cta - t * kRows + 15) >> 4;  // of 16 rows: those with any
#pragma unroll 1
        for (int p = 0; p < kParts; ++p) {
#pragma unroll 1
          for (int m = p * (4 / kParts); m < (p + 1) * (4 / kParts); ++m) {
#pragma unroll
            for (int ks = 0; ks < kRows / 16; ++ks) {
              mma_warp<false>(leader, tmem + kTmemO + 64 * m, a_lo + ((ks * 16 * 128) >> 4),
                              hi(kv_mn), lo(p_k) + ((ks * 32) >> 4), hi(p_k), idesc_o,
                              (t > 0 || ks > 0) ? 1u : 0u);
              if (ks + 1 >= steps) break;
            }
            a_lo += (2 * kAtomBytes) >> 4;
          }
          mma_commit_warp(leader, &misc->kv_empty[sl][p]);
        }
        mma_commit_warp(leader, &misc->p_empty);
      }
      if (n_tiles > 0) mma_commit_warp(leader, &misc->o_done);  // every MMA has completed
    } else {
      constexpr uint32_t idesc_s = mma_idesc(kHeads, kRows, true, false, false);
      bool qk_ok = n_tiles == 0 || wait_bar(&misc->q_done, 0u, misc, a.status);
      for (int t = 0; t < n_tiles && qk_ok; ++t) {
        const int sl = t % kSlots, sb = t & 1;
        if (t >= 2 && !wait_bar(&misc->s_free[sb], static_cast<uint32_t>(((t >> 1) - 1) & 1), misc,
                                a.status)) {
          break;
        }
        uint32_t a_lo = lo(q_k), b_lo = lo(kv_k) + static_cast<uint32_t>(sl * kSlotBytes >> 4);
#pragma unroll 1
        for (int p = 0; p < kParts; ++p) {
          if (!wait_bar(&misc->kv_full[sl][p], static_cast<uint32_t>((t / kSlots) & 1), misc,
                        a.status)) {
            qk_ok = false;
            break;
          }
          tc_fence_after();
          fence_proxy_async_smem();
#pragma unroll 1
          for (int c = 0; c < 8 / kParts; ++c) {  // atoms of 64 dims
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              mma_warp<true>(leader, tmem + 32 * sb, a_lo + ((ks * 32) >> 4), hi(q_k),
                             b_lo + ((ks * 32) >> 4), hi(kv_k), idesc_s,
                             (p > 0 || c > 0 || ks > 0) ? 1u : 0u);
            }
            a_lo += (kHeads * 128) >> 4;
            b_lo += kAtomBytes >> 4;
          }
        }
        if (qk_ok) mma_commit_warp(leader, &misc->s_full[sb]);
      }
    }
    __syncwarp();
    if (paired) {
      // the phases of the exchange below, which these warps only pass through
      cluster_wait();
      cluster_arrive();
      cluster_wait();
      cluster_arrive();
    }
  } else {
    // ---------------- math: softmax, rescale ----------------
    int s_begin, s_cnt;
    sel_range(misc->n_sel, s_begin, s_cnt);
    const int n_rows_cta = w_cnt + s_cnt;
    const int n_tiles = (n_rows_cta + kRows - 1) / kRows;
    // A failed (timed-out) wait makes `ok` false for good; the thread then
    // skips the work but still reaches every named barrier.
    n_tiles_e = n_tiles;
    // Thread (half, h) has head h's scores of rows 32 half .. 32 half + 31 of each
    // tile, and its share of the head's sum.
    const uint32_t la = tmem_addr(tmem, static_cast<uint32_t>(32 * warp), 0);
    const int half = warp >> 1, h = tid & (kHeads - 1);
    const float sl = a.scale_log2;
    // PV(t) is known complete through p_empty's phase t; a thread waits for every phase
    // in turn, so a parity wait is never more than one phase off.
    auto wait_pv = [&](int t) {
      if (ok) ok = wait_bar(&misc->p_empty, static_cast<uint32_t>(t & 1), misc, a.status);
    };
    for (int t = 0; t < n_tiles; ++t) {
      const int sb = t & 1;
      const int valid = n_rows_cta - t * kRows - kHalf * half;
      float z[kHalf];
      float mt = -INFINITY, alpha = 1.f;
      if (ok) ok = wait_bar(&misc->s_full[sb], static_cast<uint32_t>((t >> 1) & 1), misc, a.status);
      tc_fence_after();
      if (ok) {
        load_scores<kHalf>(la + 32 * sb, valid, z);
        mt = max_scores<kHalf>(z, sl);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&misc->s_free[sb]);
      // The buffer of tile t - 2 is free: its readers have passed tile t - 1's barrier.
      misc->mx[sb][half][h] = mt;
      // If any head's maximum moved by more than 2^8 (or there is none yet), both halves
      // take the larger one.
      if (named_sync_or(kMathBar, 128, t == 0 || mt > m_run + 8.f)) {
        mt = fmaxf(mt, misc->mx[sb][half ^ 1][h]);
        if (t == 0) {
          m_run = mt;
        } else {
          if (mt > m_run + 8.f) {
            alpha = exp2f(m_run - mt);
            m_run = mt;
          }
          // O^T holds PV(0..t-1): scale every head's column by its alpha (1 for heads
          // whose maximum stayed).
          if (half == 0) misc->alpha[h] = alpha;
          wait_pv(t - 1);
          tc_fence_after();
          named_sync(kMathBar, 128);
          if (ok) {
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                float v[16];
                const uint32_t addr = la + kTmemO + 64 * m + 16 * c;
                tmem_ld16(addr, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] *= misc->alpha[16 * c + i];
                tmem_st16(addr, v);
              }
            }
          }
          tc_fence_before();
          named_sync(kMathBar, 128);  // alpha is read by all before the next tile rewrites it
        }
      }
      if (t >= 1) wait_pv(t - 1);  // P was last read by PV(t - 1)
      if (ok) {
        uint32_t pk[kHalf / 2];
        // the denominator sums the fp32 probabilities; the MMA takes them in
        // bf16, the type of its other operand
        l_run = l_run * alpha + exp_pack<kHalf>(z, sl, m_run, pk);
        const uint32_t pb = sbase + kP;
#pragma unroll
        for (int c = 0; c < kHalf / 8; ++c) {
          st_shared_v4(pb + sw128_off(h, 4 * half + c),
                       make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&misc->p_full);
    }
    // the two halves' sums (the order is fixed); with a split, (max, sum) to every CTA of
    // the cluster, there by phase 1
    if (half == 1) misc->mx[0][0][h] = l_run;
    named_sync(kMathBar, 128);
    if (half == 0) l_run += misc->mx[0][0][h];
    if (paired) {
      cluster_wait();  // phase 0: every CTA's barriers are initialised
      if (half == 0) {
        const uint32_t mine = sbase + kMl + static_cast<uint32_t>(split * kHeads + h) * 8u;
        for (int p = 0; p < S; ++p) {
          st_cluster_f32x2(mapa_shared(mine, static_cast<uint32_t>(p)),
                           ok && n_tiles > 0 ? m_run : -INFINITY, ok ? l_run : 0.f);
        }
      }
    }
  }

  if (warp < kMmaWarp) {
    // ---------------- epilogue (math and loader warps) ----------------
    // Warp w reads TMEM lanes 32 (w % 4) .. + 31 (dims 128 m + 32 (w % 4) + lane of O^T
    // slice m); the (slice, 32 heads) pairs are dealt to the three warps of a lane
    // quarter in turn. The loops are rolled: the code runs once per CTA and is fetched
    // cold.
    const int grp = warp >> 2;
    const int et0 = 32 * (warp & 3);  // first dim within a slice = TMEM lane
    const uint32_t lq = tmem_addr(tmem, static_cast<uint32_t>(et0), kTmemO);
    const int n_tiles = n_tiles_e;
    if (n_tiles > 0) {
      if (ok) ok = wait_bar(&misc->o_done, 0u, misc, a.status);
    } else if (ok) {
      // no tiles: nothing else ordered the Q copies before the CTA's end
      ok = wait_bar(&misc->q_done, 0u, misc, a.status);
    }
    tc_fence_after();
    const bool have_o = ok && n_tiles > 0;
    uint16_t* out = a.out + static_cast<int64_t>(b) * kHeads * kLatent;
    // v = heads 32 hp .. + 31 of slice m's dim in this lane, times their weights
    auto load32 = [&](int m, int hp, float (&v)[32]) {
      if (have_o) {
        tmem_ld32(lq + 64 * m + 32 * hp, v);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
      }
      const uint32_t f = smem_u32(misc->wgt) + 128u * hp;
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 w4 = ld_shared_f4(f + 4u * i);
        v[i] *= w4.x;
        v[i + 1] *= w4.y;
        v[i + 2] *= w4.z;
        v[i + 3] *= w4.w;
      }
    };
    if (paired) {
      if (warp >= kLoadWarp0) cluster_wait();  // phase 0 (the math warps have waited)
      // phase 1: every CTA's MMAs are done, so its slots may be written, and every
      // CTA's (max, sum) is here
      cluster_arrive();
      cluster_wait();
    }
    // The weight of this CTA's O: 2^(m - M) / L with M = max_q m_q, L = sum_q 2^(m_q - M) l_q
    // over the cluster's CTAs (a range without rows has l_q = 0).
    if (warp < 2) {
      float M = m_run, L = l_run;
      if (paired) {
        const float2* ml = reinterpret_cast<const float2*>(gbase + kMl) + tid;
        float2 x[kMaxAttnSplits];
        M = -INFINITY;
#pragma unroll
        for (int q = 0; q < kMaxAttnSplits; ++q) {
          x[q] = q < S ? ml[q * kHeads] : make_float2(-INFINITY, 0.f);
        }
#pragma unroll
        for (int q = 0; q < kMaxAttnSplits; ++q) {
          if (!(x[q].y <= 0.f)) M = fmaxf(M, x[q].x);  // (a NaN counts)
        }
        L = 0.f;
#pragma unroll
        for (int q = 0; q < kMaxAttnSplits; ++q) {
          if (!(x[q].y <= 0.f)) L = fmaf(ex2_ftz(x[q].x - M), x[q].y, L);
        }
      }
      misc->wgt[tid] = L == 0.f || !have_o ? 0.f : ex2_ftz(m_run - M) / L;
      m_run = M;  // for the log-sum-exp at the end
      l_run = L;
    }
    named_sync(kEpiBar, kEpiThreads);
    const uint32_t image = sbase + kQ;  // Q is no longer read
    if (!paired) {
#pragma unroll 1
      for (int i = grp; i < 8; i += kEpiGroups) {
        float v[32];
        load32(i >> 1, i & 1, v);
        stage_heads<32>(image, kLatent * 2, 32 * (i & 1), 128 * (i >> 1) + et0 + lane, v);
      }
    } else {
      // CTA `split` finishes dims [split D, split D + D). Each CTA writes its part for
      // each CTA straight into that one's receive area (its slots). A warp's 32 dims
      // always go to one CTA.
      const int D = kLatent >> lg_s, lg_d = 9 - lg_s;
      const uint32_t pay = static_cast<uint32_t>(xchg_bytes(S));
      const uint32_t plane = static_cast<uint32_t>(D) * 16u;
#pragma unroll 1
      for (int i = grp; i < 8; i += kEpiGroups) {
        const int m = i >> 1, hp = i & 1;
        const int d = 128 * m + et0 + lane;
        const int p = d >> lg_d;
        const uint32_t mine = sbase + kKV + static_cast<uint32_t>(split) * pay +
                              static_cast<uint32_t>(d - p * D) * 16u +
                              static_cast<uint32_t>(4 * hp) * plane;
        const uint32_t mine_lo = mine + static_cast<uint32_t>(8 - 2 * hp) * plane;
        float v[32];
        load32(m, hp, v);
        uint4 hi[4], lo[2];
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 8 heads: the upper 16 bits ...
          const float* x = v + 8 * c;
          auto up = [&](int k) {
            return prmt(__float_as_uint(x[2 * k]), __float_as_uint(x[2 * k + 1]), 0x7632u);
          };
          hi[c] = make_uint4(up(0), up(1), up(2), up(3));
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // 16 heads: ... and the next 8
          const float* x = v + 16 * c;
          auto next = [&](int k) {
            return prmt(prmt(__float_as_uint(x[4 * k]), __float_as_uint(x[4 * k + 1]), 0x0051u),
                        prmt(__float_as_uint(x[4 * k + 2]), __float_as_uint(x[4 * k + 3]), 0x0051u),
                        0x5410u);
          };
          lo[c] = make_uint4(next(0), next(1), next(2), next(3));
        }
        if (p == split) {  // its own part, by plain stores
#pragma unroll
          for (int c = 0; c < 4; ++c) st_shared_v4(mine + c * plane, hi[c]);
#pragma unroll
          for (int c = 0; c < 2; ++c) st_shared_v4(mine_lo + c * plane, lo[c]);
        } else {
          const uint32_t there = mapa_shared(mine, static_cast<uint32_t>(p));
          const uint32_t there_lo = there + (mine_lo - mine);
#pragma unroll
          for (int c = 0; c < 4; ++c) st_cluster_u4(there + c * plane, hi[c]);
#pragma unroll
          for (int c = 0; c < 2; ++c) st_cluster_u4(there_lo + c * plane, lo[c]);
        }
      }
      cluster_arrive();  // phase 2: everything is written (release) ...
      cluster_wait();    // ... and visible here (acquire)
      // The output: the sum of the parts, (16 heads, 32 dims) pairs in turn over the warps.
#pragma unroll 1
      for (int i = warp; i < D >> 3; i += kEpiThreads / 32) {
        const uint32_t g = static_cast<uint32_t>(i & 3);
        const int d32 = 32 * (i >> 2);
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
        uint32_t src = sbase + kKV + static_cast<uint32_t>(d32 + lane) * 16u + 2u * g * plane;
        const uint32_t to_lo = (8u - g) * plane;
#pragma unroll 2
        for (int r = 0; r < S; ++r, src += pay) {
          const uint4 x0 = ld_shared_v4(src);
          const uint4 x1 = ld_shared_v4(src + plane);
          const uint4 y = ld_shared_v4(src + to_lo);
          const uint32_t hi[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
          const uint32_t lo[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // bytes from the top: the 16-bit part, the 8-bit part twice (the middle of
            // what was cut off, to within 2^-17)
            v[4 * e] += __uint_as_float(prmt(hi[2 * e], lo[e], 0x1044u));
            v[4 * e + 1] += __uint_as_float(prmt(hi[2 * e], lo[e], 0x3255u));
            v[4 * e + 2] += __uint_as_float(prmt(hi[2 * e + 1], lo[e], 0x1066u));
            v[4 * e + 3] += __uint_as_float(prmt(hi[2 * e + 1], lo[e], 0x3277u));
          }
        }
        stage_heads<16>(image, static_cast<uint32_t>(2 * D), 16 * static_cast<int>(g), d32 + lane,
                        v);
      }
    }
    named_sync(kEpiBar, kEpiThreads);
    {
      // 16-byte unit k of the image is unit k % (D / 8) of head k / (D / 8)
      const int lg_u = 6 - lg_s;
      uint16_t* dst = out + split * (kLatent >> lg_s);
      const int n = kHeads << lg_u;
#pragma unroll 4
      for (int k = tid; k < n; k += kEpiThreads) {
        const uint4 x = ld_shared_v4(image + 16u * static_cast<uint32_t>(k));
        *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(k >> lg_u) * kLatent +
                                  8 * (k & ((1 << lg_u) - 1))) = x;
      }
    }
    if (warp < 2 && a.lse && split == 0) {
      a.lse[static_cast<int64_t>(b) * kHeads + tid] =
          l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * 0.69314718055994531f;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // The epilogue warps have waited for phase 2 (no peer writes this CTA any
  // more); the MMA warps, which only arrived there, wait now.
  if (paired && warp >= kMmaWarp) cluster_wait();
}

template <int kParts>
cudaError_t launch_parts(const AttnArgs& a, const CUtensorMap& qmap, cudaStream_t s) {
  static std::atomic<int> smem_set[64]{};
  const cudaError_t e =
      ensure_smem(reinterpret_cast<const void*>(attn4_kernel<kParts>), kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn4_kernel<kParts>, dim3(a.B, a.splits), dim3(kThreads), kSmemBytes, s,
                    a.splits, a, qmap);
}

}  // namespace

cudaError_t launch_attn4(const AttnArgs& a, cudaStream_t s) {
  if (a.B == 0) return cudaSuccess;
  if (a.prefill || (a.splits != 1 && a.splits != 2 && a.splits != 4 && a.splits != 8)) {
    return cudaErrorInvalidValue;
  }
  CUtensorMap qmap;
  memset(&qmap, 0, sizeof(qmap));
  cudaError_t e = encode_tma_2d(&qmap, a.q, 2, kLatent, static_cast<uint64_t>(a.B) * kHeads,
                                kLatent * 2, 64, kHeads);
  if (e != cudaSuccess) return e;
  AttnArgs args = a;
  args.swa_rows = static_cast<int64_t>(a.B) * a.window;
  return a.splits == kMaxAttnSplits ? launch_parts<1>(args, qmap, s) : launch_parts<2>(args, qmap, s);
}

}  // namespace dsa
