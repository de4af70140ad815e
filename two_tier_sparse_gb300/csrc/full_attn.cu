// Attention of each query over its sequence's whole latent cache and the
// sliding window under one softmax, split over the cache's length and joined:
//   z_j = tau q_h . KV_j,  out_h = sum_j softmax(z)_j KV_j,  lse_h = log sum_j exp(z_j),
// for the 64 heads of a query and every row j its sequence holds for it.
//
// A query's rows are tiles of 64 (E4M3: 128), first its window rows, then its latents. 64 latents
// from a multiple of 64 on lie in one page. The tiles of all queries, one query's after
// another's (and kBegin more for each), are dealt out evenly: each CTA of one wave takes a run of consecutive tiles and works
// the run's ends out from the lengths by itself, so the split does not depend on how the rows are
// spread over the queries. A run crosses queries, and a query runs: the CTA leaves a query
// that is wholly its own finished, and of the others a part (the running maximum, the sum
// and the unnormalised output in fp32), which a second kernel joins. With few runs, 2 or 4 CTAs
// take the same one and leave a share of the output's dims each (half or a quarter of PV and of the
// part, which an SM writes at 32 bytes a clock: 2 us for all dims).
//
// Parts and their join cost 10 - 28 us where most queries are split (two thirds of it the parts' way out and
// in again, the rest more queries begun a CTA), so runs of whole queries are taken where the longest
// is not much longer than the even split's (kMore, kFew tiles): 140 sequences of 828 bf16 rows 46.2 ->
// 31.3 us, 100 of them 38.1 -> 29.8, 48 x 5 queries over 640 E4M3 rows 48.5 -> 35.9. 160 of 828, of which
// eight CTAs would have two, stay split (46.5; E4M3 38.8, whole 43.4).
//
// Per tile, weight-stationary MMAs with the 64 heads as M, whose result has its first N / 2 columns in
// lanes 0..63 and the others in lanes 64..127:
//   S  = Q . KV^T   (N = the tile's rows, K = 512)
//   O += P . KV     (N = 256 dims, twice; K = the tile's rows; KV is read as an MN-major operand)
// so a thread has one head's scores of half a tile's rows, and half of its output. They are
// bound by the operands read from shared memory at 128 bytes a clock: a step measured 38 clocks for
// N = 64, 49 for N = 128, 82 for N = 256 (in the form KV^T . P^T with 128 dims as M and N = 64
// heads 49 for a quarter of the dims), so 1860 clocks for 64 bf16 rows, 1450 for E4M3 ones.
//
// bf16 and E4M3 rows come by TMA straight into the swizzled operand layout, in four parts of
// 128 dims, refilled as soon as PV has read them. MXFP4 rows are read by loader warps that
// convert them to bf16 on the way (exactly).
//
// E4M3 codes are MMA operands as they are (K = 32 a step), so Q and P are E4M3 too, as sums of two:
// a bf16 has 8 significant bits and E4M3 4, so x = hi + lo with hi = RN(x) and lo = RN(x - hi)
// is exact down to E4M3's smallest step. Q, scaled by a power of two a head to at most 448, is exact for
// elements down to 2^-10 of the head's largest and within 2^-18 of that below. P is rounded to 8
// bits (as bf16 would) or by 2^-10, whichever is more. The second is a fixed step, and a long tail of small
// probabilities would get lost in it if P were in units of the largest so far. So the units follow
// the tiles, down too: of each tile the largest P is at least 2^5, whose sum the 128 roundings change by at
// most 2^-8, or the sum before it is at least 64 times the run's tiles of the query, whose sum all
// such tiles together change by at most 2^-9. Moving the unit scales the output in tensor memory; the
// sum soon suffices where no few rows have most of the weight (64 x 8192: 77 us with units of the largest
// and with these at scores spread by 0.6 nats, 79 -> 83 at 1.3, 83 -> 86 at 6; with units of the largest
// and a first row of half the weight, 0.03 of the sum was lost over 16384 rows, 0.38 over 131072).
// Both halves are products of their own with the same accumulators, so the MMAs cost
// what those of bf16 rows do (twice the products at twice the K), and rows are half the
// bytes. (Converted to f16 by loader warps 64 rows took 3.3 us.)
#include <algorithm>
#include <cstddef>

#include "attn_math.cuh"
#include "kv_format.cuh"

namespace dsa {

namespace {

constexpr int kMathBar = 1;                // named barrier of the 128 math threads
constexpr int kLoadWarp0 = 8;              // behind four math and four output warps

constexpr int kFmtE4m3 = DSA_KV_FP8_E4M3, kFmtMx4 = DSA_KV_MXFP4;

// Shared memory, offsets from a 1024-aligned base.
constexpr int kSub = 64;                   // rows that lie together: a box of TMA, a page's at least
constexpr int kQ = 0;                      // 8 atoms x 64 heads x 128 B
constexpr uint32_t kQBytes = kHeads * kLatent * 2;
constexpr int kQAtom = kHeads * 128;
constexpr int kP = kQ + static_cast<int>(kQBytes);  // 64 heads x 128 B (E4M3: hi, then lo)
constexpr int kPAtom = kHeads * 128;
constexpr int kKV = kP + 2 * kPAtom;       // two slots
constexpr int kSlots = 2;
constexpr int kSlotBytes = 64 * 1024;
constexpr int kStage = kKV + kSlots * kSlotBytes;  // an output warp's 64 bytes of 32 heads
constexpr int kStageBytes = 32 * 64;
constexpr int kMisc = kStage + 4 * kStageBytes;
constexpr int kMiscBytes = 6144;
constexpr int kSmemBytes = kMisc + kMiscBytes + 1024;  // + alignment slack of the base
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
constexpr int kTmemCols = 512;
constexpr int kTmemO = 128;  // O: 2 x 128 columns; below it S, two buffers of half a tile's rows

template <int FMT>
struct Shape {
  static constexpr bool kF8 = FMT == kFmtE4m3;      // E4M3 operands, bf16 otherwise
  static constexpr bool kTma = FMT != kFmtMx4;      // rows come as they are
  static constexpr int kRows = kF8 ? 128 : 64;      // of a tile
  static constexpr int kHalf = kRows / 2;           // scores of a math thread
  static constexpr int kSubs = kRows / kSub;
  static constexpr int kAtoms = kF8 ? 4 : 8;        // of a slot: 128 bytes of a tile's rows each
  static constexpr int kAtomBytes = kRows * 128;
  static constexpr int kParts = kTma ? 4 : 2;       // of a slot, in dims
  static constexpr int kStep = kF8 ? 32 : 16;       // rows of an MMA of PV
  static constexpr int kMinTiles = 128 / kRows;     // of a CTA's run, at least (but for the last)
  // Tiles by which the longest run of whole queries may exceed the even split's runs: kFew while
  // those are the shortest there are (few parts then: 16 sequences of 640 bf16 rows 14.4 us split, 22.0 whole).
  static constexpr int kMore = kF8 ? 7 : kTma ? 12 : 8, kFew = kF8 ? 3 : 5;
  // P = 2^(z - m + kUp), m the reference: a tile's largest z, moved up when another tile's is more
  // than kSlack above it (E4M3: P <= 2^8.8 < 448; else 2^8) ...
  static constexpr float kUp = kF8 ? 6.f : 0.f, kSlack = kF8 ? 2.8f : 8.f;
  // ... and, over E4M3 rows, down (by 2^kFar at most) when it is more than kDrop below it and the
  // sum so far less than kNeed times the run's tiles of the query.
  static constexpr float kDrop = 1.f, kNeed = 64.f, kFar = 24.f;
  static constexpr int kLoadWarps = kTma ? 1 : 8;
  static constexpr int kMmaWarp = kLoadWarp0 + kLoadWarps;
  static constexpr int kPvWarp = kMmaWarp + 1;
  static constexpr int kThreads = 32 * (kPvWarp + 1);
  static_assert(kAtoms * kAtomBytes == kSlotBytes && 2 * kHalf <= kTmemO, "a tile fits its slot");
};

// The rows of a query: n_win window rows from row win0 of its sequence's window
// buffer, then the first n_lat latents of its sequence.
struct Query {
  int seq, n_lat, n_win, win0;
  bool bad;  // a length that no sequence can have
};
__device__ __forceinline__ Query query_of(const FullAttnArgs& a, int x) {
  Query r;
  r.win0 = 0;
  r.n_win = 0;
  if (a.mq == 0) {
    const int n = a.lengths[x];
    r.seq = x;
    r.bad = n < 0 || n > a.max_latents;
    r.n_lat = static_cast<int>(min(max(int64_t{n}, int64_t{0}), a.max_latents));
    if (a.swa != nullptr) {
      const int w = a.swa_len[x];
      r.bad |= w < 0 || w > a.window;
      r.n_win = min(max(w, 0), a.window);
    }
  } else {
    r.seq = x / a.mq;
    const int i = x - r.seq * a.mq, n = a.lengths[r.seq];
    const int64_t seen = int64_t{n} - a.mq + i + 1;  // its position + 1
    const int64_t lat = seen > 0 ? seen / a.ratio : 0;
    r.bad = seen <= 0 || lat > a.max_latents;
    r.n_lat = static_cast<int>(min(lat, a.max_latents));
    if (a.swa != nullptr && seen > 0) {
      r.n_win = static_cast<int>(min(int64_t{a.window}, seen));
      r.win0 = i + a.window - r.n_win;
    }
  }
  return r;
}
// Tiles of a query; one without rows still has one (its output is written).
template <int ROWS>
__device__ __forceinline__ int window_tiles(const Query& r) { return (r.n_win + ROWS - 1) / ROWS; }
template <int ROWS>
__device__ __forceinline__ int tiles_of(const Query& r) {
  return max(1, window_tiles<ROWS>(r) + (r.n_lat + ROWS - 1) / ROWS);
}

// What beginning a query costs a CTA, in tiles, since nothing runs ahead of its Q (3.2 us in bf16, whose
// tile takes 1.6, 3.3 - 6 in E4M3, whose tile takes 2.2): runs count as many before each query's first. 48
// x 5 queries over 0 to 8192 E4M3 rows took 77 us with tiles alone, 64 with 1, 61 with 2, 63 with 3; 100
// sequences of 0 to 16384 MXFP4 rows 67, 58, 60, 61; 90 of 0 to 3000 bf16 rows 44.7, 45.6, 43.4, 44.6.
constexpr int kBegin = 2;

// A CTA's run, query by query: `take` tiles of query x from its tile `off` on.
struct Piece {
  int left;  // the run from this piece's first tile on
  int x, index;
  Query r;
  int tiles, off, take;
};
template <int ROWS>
__device__ __forceinline__ void next_piece(const FullAttnArgs& a, Piece& p) {
  p.left -= p.take + kBegin;
  ++p.x;
  ++p.index;
  p.take = 0;
  if (p.left > 0) {
    p.r = query_of(a, p.x);
    p.tiles = tiles_of<ROWS>(p.r);
    p.off = 0;
    p.take = min(p.left, p.tiles);
  }
}

struct Misc {
  uint64_t kv_full[kSlots][4], kv_empty[kSlots][4], s_full[2], s_free[2], p_full, p_empty;
  uint64_t q_full, q_conv, q_empty;  // Q in shared memory; split; read by the last QK^T
  uint64_t o_done, o_free;           // a query's last PV has completed; its output has left
  uint64_t stats_full[2];            // its maxima and sums are written (by its parity)
  uint64_t drain;                    // every MMA of the CTA has completed
  uint32_t tmem_base;
  int abort;
  int tile_rows[kSlots][2];  // rows of the slot's tile that count, of each 64
  Piece first;            // the CTA's run, at its first piece
  int2 warp_sum[8];        // of the tiles: the sum and the largest of a warp's queries
  int2 bound[kFullMaxCtas + 1];  // where runs of whole queries begin: the tile and its query
  float mx[2][2][kHeads];  // a tile's largest score of each head in its two halves
  float sum[2][2][kHeads];  // (E4M3) the two halves' sums before the tile
  // of a query, by its parity: the output warps may be one behind
  float m_of[2][kHeads], l_of[2][kHeads];
  float wgt[2][kHeads];    // 1 / the head's sum
  float q_unscale[2][kHeads];  // (E4M3) a head's scores, by the query's parity too
};
static_assert(sizeof(Misc) <= kMiscBytes, "misc block");

__device__ __noinline__ bool wait_loop(uint64_t* bar, uint32_t parity, volatile int* abort,
                                       DeviceStatus* st) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_abortable(bar, parity, abort, st, SITE_FULL));
}
// A converged warp's bounded wait; every lane gets the same answer.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, Misc* m,
                                         DeviceStatus* st) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(smem_u32(bar), parity))) return true;
  return wait_loop(bar, parity, &m->abort, st);
}

// Where 64 rows of a query's tile j lie, those of its part `sub`: their first row in the window buffer
// or the latent array, and how many of them count.
struct Rows {
  int64_t row;
  int rows;
};
template <int ROWS>
__device__ __forceinline__ Rows rows_at(const FullAttnArgs& a, const Query& r, int j, int sub) {
  Rows t;
  const int wt = window_tiles<ROWS>(r);
  if (j < wt) {
    const int first = j * ROWS + sub * kSub;
    t.rows = max(0, min(kSub, r.n_win - first));
    t.row = r.seq * a.swa_seq_rows + r.win0 + first;
    return t;
  }
  const int first = (j - wt) * ROWS + sub * kSub;
  t.rows = max(0, min(kSub, r.n_lat - first));
  t.row = a.pages.table == nullptr ? r.seq * a.lat_stride + first
          : t.rows > 0             ? paged_row(a.pages, r.seq, first)
                                   : 0;
  if (t.row < 0) {  // no such page
    record_status(a.status, DSA_ERR_DEVICE_CHECK, SITE_FULL, static_cast<uint32_t>(r.seq));
    t.rows = 0;
  }
  return t;
}

// Two values as sums of two E4M3 numbers, hi and lo (the first value in the low bytes).
__device__ __forceinline__ void split_e4m3(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  // x in f16 (exact for values of 11 bits, or to 2^-25); x - hi is exact there
  asm("{\n .reg .b16 h, l;\n .reg .b32 x, y;\n"
      " cvt.rn.f16x2.f32 x, %3, %2;\n cvt.rn.satfinite.e4m3x2.f16x2 h, x;\n"
      " cvt.rn.f16x2.e4m3x2 y, h;\n sub.rn.f16x2 x, x, y;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 l, x;\n cvt.u32.u16 %0, h;\n cvt.u32.u16 %1, l;\n}\n"
      : "=r"(hi), "=r"(lo)
      : "f"(x0), "f"(x1));
}
// p_i = 2^(scale z_i - m) as hi and lo, four to a word; returns sum_i p_i over the fp32 values.
template <int R>
__device__ __forceinline__ float exp_split(const float (&z)[R], float scale, float m,
                                           uint32_t (&ph)[R / 4], uint32_t (&pl)[R / 4]) {
  float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < R; i += 4) {
    float p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      p[k] = ex2_ftz(fmaf(z[i + k], scale, -m));
      s4[k] += p[k];
    }
    uint32_t h0, l0, h1, l1;
    split_e4m3(p[0], p[1], h0, l0);
    split_e4m3(p[2], p[3], h1, l1);
    ph[i / 4] = h0 | (h1 << 16);
    pl[i / 4] = l0 | (l1 << 16);
  }
  return (s4[0] + s4[1]) + (s4[2] + s4[3]);
}

// How `used` CTAs share the tiles: runs of len or, the first `more` of them, len + 1.
struct Runs {
  int used, len, more;
  __device__ __forceinline__ int begin_of(int c) const { return c * len + min(c, more); }
  __device__ __forceinline__ int run_of(int tile) const {
    const int longer = more * (len + 1);  // (tiles in longer runs)
    return tile < longer ? tile / (len + 1) : more + (tile - longer) / len;
  }
};

// Runs of whole queries in their place, each beginning where a query does that is nearest to the
// even split: run `run`'s first piece and true, if none is longer than `most` tiles. (Called by every
// thread; thread t < 256 has queries per * t and on, `own` tiles from tile `before` on.)
template <int ROWS>
__device__ __noinline__ bool whole_runs(const FullAttnArgs& a, Misc* misc, Runs runs, int run, int before,
                                        int own, int per, int most, int total) {
  const int tid = threadIdx.x;
  if (tid < 256 && own > 0) {
    int at = before, c = runs.run_of(before);
    for (int x = tid * per; at < before + own; ++x) {
      const int n = per > 1 ? kBegin + tiles_of<ROWS>(query_of(a, x)) : own;
      for (; c < runs.used && runs.begin_of(c) < at + n; ++c) {
        if (runs.begin_of(c) < at) continue;
        const bool next = 2 * (runs.begin_of(c) - at) >= n;
        misc->bound[c] = next ? make_int2(at + n, x + 1) : make_int2(at, x);
      }
      at += n;
    }
    if (tid == 0) misc->bound[runs.used] = make_int2(total, a.n_queries);
  }
  __syncthreads();
  if (__syncthreads_or(tid < runs.used && misc->bound[tid + 1].x - misc->bound[tid].x > most)) return false;
  if (run < runs.used && tid == 0) {
    const int2 b = misc->bound[run];
    Piece& p = misc->first;
    p.left = misc->bound[run + 1].x - b.x - kBegin;
    p.x = b.y;
    p.index = 0;
    p.off = 0;
    if (p.left > 0) {
      p.r = query_of(a, b.y);
      p.tiles = tiles_of<ROWS>(p.r);
      p.take = min(p.left, p.tiles);
    }
    a.records[run] = make_int4(-1, 0, 0, 0);
  }
  return true;
}

// 32 bytes, a sector (the address a multiple of 32).
__device__ __forceinline__ void st_global_v8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// Steps of PV that a tile takes, at least one: those up to its last row that counts (an absent page's
// rows in between are zeros).
template <int FMT>
__device__ __forceinline__ int rows_end(const int (&rows)[2]) {
  return Shape<FMT>::kSubs == 2 && rows[1] > 0 ? kSub + rows[1] : rows[0];
}
template <int FMT>
__device__ __forceinline__ int steps_of(const int (&rows)[2]) {
  return max(1, (rows_end<FMT>(rows) + Shape<FMT>::kStep - 1) / Shape<FMT>::kStep);
}

template <int FMT>
__global__ void __launch_bounds__(Shape<FMT>::kThreads, 1)
    full_attn_kernel(const __grid_constant__ FullAttnArgs a, const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap lmap,
                     const __grid_constant__ CUtensorMap wmap) {
  using Sh = Shape<FMT>;
  constexpr bool kF8 = Sh::kF8;
  constexpr int kRows = Sh::kRows, kHalf = Sh::kHalf, kParts = Sh::kParts, kAtomBytes = Sh::kAtomBytes;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (sbase - raw);
  Misc* misc = reinterpret_cast<Misc*>(gbase + kMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      for (int p = 0; p < kParts; ++p) {
        mbar_init(&misc->kv_full[i][p], Sh::kLoadWarps);
        mbar_init(&misc->kv_empty[i][p], 1);
      }
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&misc->s_full[i], 1);
      mbar_init(&misc->s_free[i], 4);
      mbar_init(&misc->stats_full[i], 4);
    }
    mbar_init(&misc->p_full, 4);
    mbar_init(&misc->p_empty, 1);
    mbar_init(&misc->q_full, 1);
    mbar_init(&misc->q_conv, 8);
    mbar_init(&misc->q_empty, 1);
    mbar_init(&misc->o_done, 1);
    mbar_init(&misc->o_free, 4);
    mbar_init(&misc->drain, 2);
    misc->abort = 0;
    misc->first.left = 0;
    misc->first.take = 0;
    fence_mbar_init();
  }
  if (warp == Sh::kMmaWarp) {
    tmem_alloc(&misc->tmem_base, kTmemCols);
    if (lane == 0) {
      tma_prefetch_map(&qmap);
      if (Sh::kTma) {
        tma_prefetch_map(&lmap);
        if (a.swa != nullptr) tma_prefetch_map(&wmap);
      }
    }
  }
  griddep_wait();
  griddep_launch_dependents();

  // The runs: thread t < 256 sums the tiles of `per` consecutive queries, and the
  // one whose queries hold the run's first tile looks for it. (All tiles are below 2^31.)
  int run, share, lg_share;
  {
    const int per = (a.n_queries + 255) / 256;
    const int x0 = min(a.n_queries, tid * per), x1 = min(a.n_queries, x0 + per);
    int own = 0, top = 0;
    Query r{};
    if (tid < 256) {
      for (int x = x0; x < x1; ++x) {
        r = query_of(a, x);
        const int n = kBegin + tiles_of<kRows>(r);
        own += n;
        top = max(top, n);
        if (r.bad && cta == 0) {
          record_status(a.status, DSA_ERR_DEVICE_CHECK, SITE_FULL, static_cast<uint32_t>(r.seq));
        }
      }
    }
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += t;
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 31 && warp < 8) misc->warp_sum[warp] = make_int2(incl, top);
    tc_fence_before();
    __syncthreads();  // (also: barriers initialised, tensor memory allocated)
    tc_fence_after();
    int before = incl - own, total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const int2 s = misc->warp_sum[w];
      if (w < warp) before += s.x;
      total += s.x;
      top = max(top, s.y);
    }
    // Where there are few runs, 2 or 4 CTAs have the same one and a share of the output's dims each.
    const int want = (total + Sh::kMinTiles - 1) / Sh::kMinTiles, ctas = static_cast<int>(gridDim.x);
    lg_share = want <= ctas / 4 ? 2 : want <= ctas / 2 ? 1 : 0;
    const int used = min(ctas >> lg_share, want);
    const int len = total / used, more = total - len * used;
    const Runs runs{used, len, more};
    run = cta >> lg_share;
    share = cta & ((1 << lg_share) - 1);
    const int begin = runs.begin_of(run);
    if (cta >= used && tid == 0) a.records[cta] = make_int4(-1, 0, 0, 0);
    const int most = len + (len > Sh::kMinTiles ? Sh::kMore : Sh::kFew);
    const bool whole_queries = lg_share == 0 && top <= most &&
                               whole_runs<kRows>(a, misc, runs, run, before, own, per, most, total);
    if (!whole_queries && run < used && tid < 256 && before <= begin && begin < before + own) {
      int x = x0, at = before, n = own;
      if (per > 1) {
        for (;; ++x) {
          r = query_of(a, x);
          n = kBegin + tiles_of<kRows>(r);
          if (begin < at + n) break;
          at += n;
        }
      }
      Piece& p = misc->first;
      const int first = at + kBegin;  // where its first tile is
      p.left = len + (run < more ? 1 : 0) - max(0, first - begin);
      p.x = x;
      p.index = 0;
      p.r = r;
      p.tiles = n - kBegin;
      p.off = max(0, begin - first);
      p.take = max(0, min(p.left, p.tiles - p.off));
      // A query to be joined is recorded by the run of its second part: the query, its
      // first run and the number of its parts.
      int4 rec = make_int4(-1, 0, 0, 0);
      if (begin > first && runs.begin_of(run - 1) <= first) {
        rec = make_int4(x, run - 1, runs.run_of(at + n - 1) - run + 2, 0);
      }
      if (share == 0) a.records[run] = rec;
    }
    __syncthreads();
  }
  const uint32_t tmem = misc->tmem_base;
  // Its dims: from dim0 on, in n_mma products of 2 n_cols dims.
  const int dim0 = share * (kLatent >> lg_share), n_mma = lg_share == 0 ? 2 : 1;
  const int n_cols = lg_share == 2 ? 64 : 128;

  if (warp >= kLoadWarp0 && warp < Sh::kMmaWarp) {
    // ---------------- loaders ----------------
    const int w = warp - kLoadWarp0;
    int tt = 0;  // tiles of the run, over its queries
    bool ok = true;
    if constexpr (Sh::kTma) {
      // one lane issues the tile's boxes of 64 rows x 128 bytes
      const uint64_t policy = l2_evict_first_policy();
      int part = 0;
      if (lane == 0) {
        for (Piece p = misc->first; ok && p.take > 0; next_piece<kRows>(a, p)) {
          for (int j = 0; j < p.take; ++j, ++tt) {
            const int sl = tt % kSlots;
            const CUtensorMap* map = p.off + j < window_tiles<kRows>(p.r) ? &wmap : &lmap;
            Rows r[Sh::kSubs];
#pragma unroll
            for (int s = 0; s < Sh::kSubs; ++s) {
              r[s] = rows_at<kRows>(a, p.r, p.off + j, s);
              // (without rows: a box past the end of what lmap covers, which reads zeros)
              if (r[s].rows == 0) r[s].row = max(a.lat_rows, int64_t{1});
            }
            for (part = 0; part < kParts; ++part) {
              if (tt >= kSlots &&
                  !mbar_wait_abortable(&misc->kv_empty[sl][part],
                                       static_cast<uint32_t>(((tt / kSlots) - 1) & 1),
                                       &misc->abort, a.status, SITE_FULL)) {
                ok = false;
                break;
              }
              if (part == 0) {
#pragma unroll
                for (int s = 0; s < Sh::kSubs; ++s) misc->tile_rows[sl][s] = r[s].rows;
              }
              uint64_t* bar = &misc->kv_full[sl][part];
              constexpr int kBoxes = Sh::kAtoms / kParts, kX = kLatent / Sh::kAtoms;
              mbar_arrive_expect_tx(bar, kBoxes * kAtomBytes);
#pragma unroll
              for (int c = kBoxes * part; c < kBoxes * (part + 1); ++c) {
#pragma unroll
                for (int s = 0; s < Sh::kSubs; ++s) {
                  const uint32_t dst = sbase + kKV + sl * kSlotBytes + c * kAtomBytes + s * kSub * 128;
                  const CUtensorMap* from = r[s].rows > 0 ? map : &lmap;
                  const int row = static_cast<int>(r[s].row);
                  if (a.mq > 1) {
                    tma_load_2d(dst, from, kX * c, row, bar);
                  } else {  // read once
                    tma_load_2d_hint(dst, from, kX * c, row, bar, policy);
                  }
                }
              }
            }
            if (!ok) break;
          }
        }
        if (!ok) {  // at part `part` of tile tt: the copies on their way land before the CTA ends
          for (int k = 0; k < kSlots * kParts; ++k) {
            const int sl = k / kParts, pt = k % kParts;
            // the slot's last tile of which this part was asked for
            const int at = tt - (tt - sl + kSlots) % kSlots;
            const int t = at == tt && pt >= part ? tt - kSlots : at;
            if (t >= 0) {
              mbar_wait(&misc->kv_full[sl][pt], static_cast<uint32_t>((t / kSlots) & 1), a.status,
                        SITE_FULL);
            }
          }
        }
      }
      __syncwarp();
    } else {
      // Loader warp w fills rows [8 w, 8 w + 8) of every tile. Lane l has row 8 w + r,
      // r = l % 8, and of it the 16-byte pieces g, g + 4, g + 8 and g + 12, g = l / 8: elements
      // [32 j, 32 j + 32) under scale j for piece j. The eight lanes of a
      // 16-byte store then write one chunk of eight different rows, which the swizzle spreads
      // over all banks. A tile's pieces are read while the tile before it is converted.
      constexpr int kPieces = 4;
      const uint32_t r = lane & 7, g = lane >> 3;
      uint32_t to[4];  // where word n of piece g goes in a slot (piece g + 4 i: two atoms on each)
#pragma unroll
      for (uint32_t n = 0; n < 4; ++n) {
        to[n] = sbase + kKV + (g >> 1) * kAtomBytes + (8u * w + r) * 128u +
                (((4u * (g & 1u) + n) ^ r) << 4);
      }
      auto read = [&](const Rows& t, bool window, uint4 (&code)[kPieces], uint4& scales) {
        const uint8_t* src = nullptr;
        const int row = 8 * w + static_cast<int>(r);
        if (row < t.rows) {
          src = static_cast<const uint8_t*>(window ? a.swa : a.latents) + (t.row + row) * kRow4Bytes;
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) code[i] = make_uint4(0u, 0u, 0u, 0u);
        scales = make_uint4(0u, 0u, 0u, 0u);
        if (src != nullptr) {
          // (64 x 8192 116.3 us as with read-only loads; left to the compiler 117.2, past the first-level
          // cache 124.2)
          const uint4* p = reinterpret_cast<const uint4*>(src);
#pragma unroll
          for (int i = 0; i < kPieces; ++i) code[i] = ld_ordered(p + g + 4 * i);
          scales = ld_ordered(p + kRow4Codes / 16);
        }
      };
      auto convert = [&](int t, int rows, const uint4 (&code)[kPieces], const uint4& scales) {
        const int sl = t % kSlots;
        const uint32_t slot = static_cast<uint32_t>(sl * kSlotBytes);
        const uint32_t sw[4] = {scales.x, scales.y, scales.z, scales.w};
        // (a warp past the last step of 16 rows has nothing that PV reads)
        const bool needed = 8 * (w & ~1) < max(rows, 1);
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          if (t >= kSlots && !wait_bar(&misc->kv_empty[sl][part],
                                       static_cast<uint32_t>(((t / kSlots) - 1) & 1), misc,
                                       a.status)) {
            ok = false;
            return;
          }
          if (needed) {
#pragma unroll
            for (int i = part * (kPieces / kParts); i < (part + 1) * (kPieces / kParts); ++i) {
              const uint32_t cw[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
              // piece g + 4 i: its scale is byte g of word i
              const uint32_t f = mx4_scale_bf16x2((sw[i] >> (8u * g)) & 0xFFu);
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                st_shared_v4(to[n] + slot + 2 * i * kAtomBytes, mx4_decode8(cw[n], f));
              }
            }
          }
          if (part == 0 && w == 0 && lane == 0) misc->tile_rows[sl][0] = rows;
          fence_proxy_async_smem();  // the MMAs read the tile through the async proxy
          __syncwarp();
          if (lane == 0) mbar_arrive(&misc->kv_full[sl][part]);
        }
      };
      Piece p = misc->first;
      int j = 0;
      // reads the next tile: its rows that count, -1 if there is none
      auto next_tile = [&](uint4 (&code)[kPieces], uint4& scales) -> int {
        if (p.take > 0 && j >= p.take) {
          next_piece<kRows>(a, p);
          j = 0;
        }
        if (p.take == 0) return -1;
        const int at = p.off + j++;
        const Rows t = rows_at<kRows>(a, p.r, at, 0);
        read(t, at < window_tiles<kRows>(p.r), code, scales);
        return t.rows;
      };
      uint4 code0[kPieces], code1[kPieces], scales0, scales1;
      int rows0 = next_tile(code0, scales0), rows1;
      while (ok && rows0 >= 0) {
        rows1 = next_tile(code1, scales1);
        convert(tt++, rows0, code0, scales0);
        if (!ok || rows1 < 0) break;
        rows0 = next_tile(code0, scales0);
        convert(tt++, rows1, code1, scales1);
      }
    }
  } else if (warp == Sh::kMmaWarp || warp == Sh::kPvWarp) {
    // ---------------- MMA issuers ----------------
    // PV(t) is issued only after the softmax of tile t, hence after QK^T(t) completed:
    // its commit alone frees the tile's slot.
    const uint32_t leader = elect_leader();
    const uint64_t kv_mn = sw128_desc(sbase + kKV, kAtomBytes, 1024);  // slot 0, MN-major
    const uint64_t kv_k = sw128_desc(sbase + kKV, 16, 1024);           // slot 0, K-major
    const uint64_t q_k = sw128_desc(sbase + kQ, 16, 1024);
    const uint64_t p_k = sw128_desc(sbase + kP, 16, 1024);
    auto lo = [](uint64_t d) { return static_cast<uint32_t>(d); };
    auto hi = [](uint64_t d) { return static_cast<uint32_t>(d >> 32); };
    int tt = 0, q_loads = 0;
    bool ok = true;
    if (warp == Sh::kPvWarp) {
      const uint32_t idesc_o = mma_idesc(kHeads, 2 * n_cols, !kF8, false, true);
      for (Piece p = misc->first; ok && p.take > 0; next_piece<kRows>(a, p)) {
        if (p.index > 0 && !wait_bar(&misc->o_free, static_cast<uint32_t>((p.index - 1) & 1), misc,
                                     a.status)) {
          break;
        }
        for (int j = 0; j < p.take; ++j, ++tt) {
          const int sl = tt % kSlots;
          if (!wait_bar(&misc->p_full, static_cast<uint32_t>(tt & 1), misc, a.status) ||
              !wait_bar(&misc->kv_full[sl][0], static_cast<uint32_t>((tt / kSlots) & 1), misc,
                        a.status)) {  // (complete already: tile_rows is visible behind it)
            ok = false;
            break;
          }
          const int steps = steps_of<FMT>(misc->tile_rows[sl]);  // of kStep rows: those with any
          tc_fence_after();
          fence_proxy_async_smem();
          const uint32_t kv = lo(kv_mn) + static_cast<uint32_t>(sl * kSlotBytes >> 4) +
                              static_cast<uint32_t>((dim0 * Sh::kAtoms / kLatent) * kAtomBytes >> 4);
#pragma unroll 1
          for (int i = 0; i < n_mma; ++i) {
            uint32_t b_lo = kv + static_cast<uint32_t>((i * Sh::kAtoms / 2 * kAtomBytes) >> 4);
#pragma unroll
            for (int ks = 0; ks < kRows / Sh::kStep; ++ks) {
              mma_warp<true, kF8>(leader, tmem + kTmemO + 128 * i, lo(p_k) + ((ks * 32) >> 4), hi(p_k),
                                  b_lo, hi(kv_mn), idesc_o, (j > 0 || ks > 0) ? 1u : 0u);
              if (kF8) {  // the low halves
                mma_warp<true, kF8>(leader, tmem + kTmemO + 128 * i, lo(p_k) + ((kPAtom + ks * 32) >> 4),
                                    hi(p_k), b_lo, hi(kv_mn), idesc_o, 1u);
              }
              if (ks + 1 >= steps) break;
              b_lo += (Sh::kStep * 128) >> 4;
            }
            // (with a share of the dims alone the other parts are free too: QK^T has read them)
            for (int part = i * kParts / 2; part < (i + 1 == n_mma ? kParts : kParts / 2); ++part) {
              mma_commit_warp(leader, &misc->kv_empty[sl][part]);
            }
          }
          mma_commit_warp(leader, &misc->p_empty);
        }
        if (ok) mma_commit_warp(leader, &misc->o_done);
      }
    } else {
      constexpr uint32_t idesc_s = mma_idesc(kHeads, kRows, !kF8, false, false);
      for (Piece p = misc->first; ok && p.take > 0; next_piece<kRows>(a, p)) {
        // The query's Q: eight boxes of 64 heads x 64 dims, each landing as one atom of the A
        // operand (E4M3: split in place then), once the last QK^T of the one before has read it.
        if (p.index > 0 && !wait_bar(&misc->q_empty, static_cast<uint32_t>((p.index - 1) & 1), misc,
                                     a.status)) {
          break;
        }
        if (leader) {
          mbar_arrive_expect_tx(&misc->q_full, kQBytes);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            tma_load_2d(sbase + kQ + c * kQAtom, &qmap, 64 * c, p.x * kHeads, &misc->q_full);
          }
        }
        __syncwarp();
        ++q_loads;
        if (!wait_bar(kF8 ? &misc->q_conv : &misc->q_full, static_cast<uint32_t>(p.index & 1), misc,
                      a.status)) {
          break;
        }
        for (int j = 0; ok && j < p.take; ++j, ++tt) {
          const int sl = tt % kSlots, sb = tt & 1;
          if (tt >= 2 && !wait_bar(&misc->s_free[sb], static_cast<uint32_t>(((tt >> 1) - 1) & 1),
                                   misc, a.status)) {
            ok = false;
            break;
          }
          uint32_t a_lo = lo(q_k), b_lo = lo(kv_k) + static_cast<uint32_t>(sl * kSlotBytes >> 4);
#pragma unroll 1
          for (int part = 0; part < kParts; ++part) {
            if (!wait_bar(&misc->kv_full[sl][part], static_cast<uint32_t>((tt / kSlots) & 1), misc,
                          a.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            fence_proxy_async_smem();
#pragma unroll 1
            for (int c = 0; c < Sh::kAtoms / kParts; ++c) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) {
                mma_warp<true, kF8>(leader, tmem + kHalf * sb, a_lo + ((ks * 32) >> 4), hi(q_k),
                                    b_lo + ((ks * 32) >> 4), hi(kv_k), idesc_s,
                                    (part > 0 || c > 0 || ks > 0) ? 1u : 0u);
                if (kF8) {  // the low halves
                  mma_warp<true, kF8>(leader, tmem + kHalf * sb,
                                      a_lo + ((Sh::kAtoms * kQAtom + ks * 32) >> 4), hi(q_k),
                                      b_lo + ((ks * 32) >> 4), hi(kv_k), idesc_s, 1u);
                }
              }
              a_lo += kQAtom >> 4;
              b_lo += kAtomBytes >> 4;
            }
          }
          if (ok) mma_commit_warp(leader, &misc->s_full[sb]);
        }
        if (ok) mma_commit_warp(leader, &misc->q_empty);
      }
    }
    // (after a timeout Q may be on its way)
    if (q_loads > 0) mbar_wait(&misc->q_full, static_cast<uint32_t>((q_loads - 1) & 1), a.status, SITE_FULL);
    __syncwarp();
    mma_commit_warp(leader, &misc->drain);
  } else {
    // ---------------- math: softmax, rescale; output: what a query leaves ----------------
    const bool math = warp < 4;
    const uint32_t la = tmem_addr(tmem, static_cast<uint32_t>(32 * (warp & 3)), 0);
    const int half = (warp >> 1) & 1, h = tid & (kHeads - 1);
    bool ok = true;
    int tt = 0;
    // (E4M3) The Q of piece `index` as hi + lo, in place: a head's row of eight atoms becomes its row
    // of four atoms of hi and four of lo. Eight warps take eight heads each, a lane 16 elements. A
    // head is scaled by a power of two to at most 448, and what undoes that recorded, times the
    // cache's scale. A head that holds an infinity or a NaN becomes NaN codes: its scores are NaN for
    // the rows that count, and for them alone.
    auto split_q = [&](int index) {
      if (ok) ok = wait_bar(&misc->q_full, static_cast<uint32_t>(index & 1), misc, a.status);
#pragma unroll 1
      for (int k = 0; k < 8; ++k) {
        const uint32_t hq = static_cast<uint32_t>(8 * warp + k), row = sbase + kQ;
        const uint32_t from = row + static_cast<uint32_t>(lane >> 2) * kQAtom;
        const uint4 v0 = ld_shared_v4(from + sw128_off(hq, 2 * lane)), v1 = ld_shared_v4(from + sw128_off(hq, 2 * lane + 1));
        const uint32_t vw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll
        for (int i = 0; i < 8; ++i) top = __vmaxu2(top, vw[i] & 0x7FFF7FFFu);
        top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));  // (every lane has read)
        const int E = static_cast<int>(top >> 7) - 127;
        int e = ((top & 0x7Fu) <= 0x60u ? 8 : 7) - E;
        e = min(126, max(-126, e));
        if (top == 0u) e = 0;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t h2[2], l2[2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t xw = vw[2 * i + n];
            split_e4m3(bf16_bits_to_float(xw & 0xFFFF) * up, bf16_bits_to_float(xw >> 16) * up, h2[n],
                       l2[n]);
          }
          hi[i] = top >= 0x7F80u ? 0x7F7F7F7Fu : h2[0] | (h2[1] << 16);
          lo[i] = l2[0] | (l2[1] << 16);
        }
        const uint32_t at = row + static_cast<uint32_t>(lane >> 3) * kQAtom + sw128_off(hq, lane & 7);
        st_shared_v4(at, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        st_shared_v4(at + Sh::kAtoms * kQAtom, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        if (lane == 0) {
          misc->q_unscale[index & 1][hq] = a.kv_scale * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        }
      }
      fence_proxy_async_smem();  // the MMA reads Q through the async proxy
      __syncwarp();
      if (lane == 0) mbar_arrive(&misc->q_conv);
    };
    Piece p = misc->first;
    if (kF8 && p.take > 0) split_q(0);
    for (; p.take > 0; next_piece<kRows>(a, p)) {
      const bool whole = p.take == p.tiles;
      const int pi = p.index & 1;
      if (math) {
        float m_run = -INFINITY, l_run = 0.f;
        // Thread (half, h) has head h's scores of a tile's rows kHalf half .. + kHalf - 1, its
        // share of the head's sum, and TMEM lane tid: half of the head's output.
        float sl = a.scale_log2;
        if (kF8) {
          if (ok) ok = wait_bar(&misc->q_conv, static_cast<uint32_t>(p.index & 1), misc, a.status);
          sl *= misc->q_unscale[pi][h];
          if (sl < 1.17549435e-38f) sl = 1.17549435e-38f;  // (by 0, a masked score would be NaN)
        }
        // PV(t) is known complete through p_empty's phase t; a thread waits for every phase
        // in turn, so a parity wait is never more than one phase off.
        auto wait_pv = [&](int t) {
          if (ok) ok = wait_bar(&misc->p_empty, static_cast<uint32_t>(t & 1), misc, a.status);
        };
        const float need = Sh::kNeed * static_cast<float>(p.take);
        for (int j = 0; j < p.take; ++j, ++tt) {
          const int sb = tt & 1, slot = tt % kSlots;
          float z[kHalf];
          float mt = -INFINITY, alpha = 1.f;
          if (ok) {
            ok = wait_bar(&misc->s_full[sb], static_cast<uint32_t>((tt >> 1) & 1), misc, a.status) &&
                 wait_bar(&misc->kv_full[slot][0], static_cast<uint32_t>((tt / kSlots) & 1), misc,
                          a.status);  // (complete already: tile_rows is visible behind it)
          }
          tc_fence_after();
          if (ok) {
            const int* rows = misc->tile_rows[slot];
            load_scores<kHalf>(la + kHalf * sb, Sh::kSubs == 2 ? rows[half] : rows[0] - kHalf * half, z);
            mt = max_scores<kHalf>(z, sl);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&misc->s_free[sb]);
          if (Sh::kTma && ok) {
            // The rows behind the tile's last, up to a whole step, are somebody else's or
            // stale; PV multiplies them by zeros, so they have to be numbers.
            constexpr int kChunks = 8 * Sh::kAtoms;  // 16-byte ones of a row
            const int end = rows_end<FMT>(misc->tile_rows[slot]);
            const int up_to = steps_of<FMT>(misc->tile_rows[slot]) * Sh::kStep;
            for (int k = tid; k < (up_to - end) * kChunks; k += 128) {
              const uint32_t row = static_cast<uint32_t>(end + k / kChunks), c = k % kChunks;
              st_shared_v4(sbase + kKV + slot * kSlotBytes + (c >> 3) * kAtomBytes +
                               sw128_off(row, c & 7),
                           make_uint4(0u, 0u, 0u, 0u));
            }
          }
          // The buffer of tile tt - 2 is free: its readers have passed tile tt - 1's barrier.
          misc->mx[sb][half][h] = mt;
          if (kF8) misc->sum[sb][half][h] = l_run;
          // If any head's reference may have to move (or there is none yet), both halves see
          // what is to be done with the larger maximum and the whole sum. (A half that alone is
          // low, or has little, asks in vain.)
          const bool low = kF8 && mt < m_run - Sh::kDrop && l_run < 0.5f * need;
          if (named_sync_or(kMathBar, 128, j == 0 || low || mt > m_run + Sh::kSlack)) {
            mt = fmaxf(mt, misc->mx[sb][half ^ 1][h]);
            if (j == 0) {
              m_run = mt;
            } else {
              float to = m_run;
              if (mt > m_run + Sh::kSlack) {
                to = mt;
              } else if (kF8 && mt < m_run - Sh::kDrop && l_run + misc->sum[sb][half ^ 1][h] < need) {
                to = fmaxf(mt, m_run - Sh::kFar);
              }
              if (to != m_run) {
                alpha = exp2f(m_run - to);
                m_run = to;
              }
              // O holds the tiles before: every thread scales its head's by alpha (1 for a
              // head whose reference stayed).
              wait_pv(tt - 1);
              tc_fence_after();
              if (ok && __any_sync(0xFFFFFFFFu, alpha != 1.f)) {
#pragma unroll 1
                for (int c = 0; c < n_mma * n_cols; c += 32) {
                  float v[32];
                  const uint32_t addr = la + kTmemO + c;
                  tmem_ld32(addr, v);
#pragma unroll
                  for (int i = 0; i < 32; ++i) v[i] *= alpha;
                  tmem_st32(addr, v);
                }
              }
              tc_fence_before();
            }
          }
          if (tt >= 1) wait_pv(tt - 1);  // P was last read by PV(tt - 1)
          if (ok) {
            // The denominator sums the fp32 probabilities; the MMA takes them in the type of
            // its other operand. (No rows so far: any finite maximum gives zeros.)
            const float m_at = m_run == -INFINITY ? 0.f : m_run - Sh::kUp;
            const uint32_t pb = sbase + kP;
            if constexpr (kF8) {
              uint32_t ph[kHalf / 4], pl[kHalf / 4];
              l_run = l_run * alpha + exp_split<kHalf>(z, sl, m_at, ph, pl);
#pragma unroll
              for (int c = 0; c < kHalf / 16; ++c) {
                const uint32_t at = pb + sw128_off(h, 4 * half + c);
                st_shared_v4(at, make_uint4(ph[4 * c], ph[4 * c + 1], ph[4 * c + 2], ph[4 * c + 3]));
                st_shared_v4(at + kPAtom,
                             make_uint4(pl[4 * c], pl[4 * c + 1], pl[4 * c + 2], pl[4 * c + 3]));
              }
            } else {
              uint32_t pk[kHalf / 2];
              l_run = l_run * alpha + exp_pack<kHalf>(z, sl, m_at, pk);
#pragma unroll
              for (int c = 0; c < kHalf / 8; ++c) {
                st_shared_v4(pb + sw128_off(h, 4 * half + c),
                             make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]));
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&misc->p_full);
        }
        // the two halves' sums (the order is fixed)
        if (half == 1) misc->mx[0][0][h] = l_run;
        named_sync(kMathBar, 128);
        if (half == 0) {
          l_run += misc->mx[0][0][h];
          misc->m_of[pi][h] = m_run - Sh::kUp;  // what l_run and O are in units of 2^ of
          misc->l_of[pi][h] = l_run;
          misc->wgt[pi][h] = l_run == 0.f ? 0.f : 1.f / l_run;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&misc->stats_full[pi]);
        if (kF8 && p.left > p.take + kBegin) split_q(p.index + 1);
        continue;
      }
      // (the next query's Q is there before this one's output)
      if (kF8 && p.left > p.take + kBegin) split_q(p.index + 1);
      if (ok) {
        ok = wait_bar(&misc->stats_full[pi], static_cast<uint32_t>((p.index >> 1) & 1), misc, a.status) &&
             wait_bar(&misc->o_done, static_cast<uint32_t>(pi), misc, a.status);
      }
      tc_fence_after();
      // Lane l of warp w reads TMEM lane 32 (w % 4) + l: head ho, and of each product's dims its
      // half.
      const int slot = 2 * run + (p.off > 0 ? 0 : 1);
      const int ho = (32 * warp + lane) & (kHeads - 1), d0 = dim0 + ((warp >> 1) & 1) * n_cols;
      // (E4M3: the cache's scale on its own, since its quotient by a large sum may be no normal number)
      const float f = misc->wgt[pi][ho], f2 = kF8 ? a.kv_scale : 1.f;
      if (whole && Sh::kTma) {
        // 64 bytes of each of the warp's heads at a time, over shared memory: the lanes' own stores
        // touch 32 rows each (608 sequences of 64 bf16 rows 26.2 us, this way 22.0).
        const uint32_t stage = sbase + kStage + static_cast<uint32_t>(warp - 4) * kStageBytes;
        const uint32_t put = stage + static_cast<uint32_t>(lane) * 64, put_x = (lane >> 1) & 3;
        uint16_t* out = static_cast<uint16_t*>(a.out) +
                        (static_cast<int64_t>(p.x) * kHeads + (ho & 32)) * kLatent + d0;
#pragma unroll 1
        for (int c = 0; ok && c < n_mma * n_cols; c += 32) {
          float v[32];
          tmem_ld32(la + kTmemO + c, v);
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * k + 2 * e] * f * f2, v[8 * k + 2 * e + 1] * f * f2);
              x[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
            st_shared_v4(put + ((k ^ put_x) << 4), make_uint4(x[0], x[1], x[2], x[3]));
          }
          __syncwarp();
          const int d = c + (c & 128);  // (the second product's columns begin at 128, its dims at 256)
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k) {
            const uint32_t hd = 8 * k + (lane >> 2), ch = lane & 3;  // head of the warp's, 16 bytes of its 64
            *reinterpret_cast<uint4*>(out + hd * kLatent + d + 8 * ch) =
                ld_shared_v4(stage + hd * 64 + ((ch ^ ((hd >> 1) & 3)) << 4));
          }
          __syncwarp();
        }
      } else {
        // (a whole output too where the registers are those of 18 warps: the staging spilled others)
        float* part = a.parts + (static_cast<int64_t>(slot) * kHeads + ho) * kLatent + d0;
        uint16_t* out = static_cast<uint16_t*>(a.out) + (static_cast<int64_t>(p.x) * kHeads + ho) * kLatent + d0;
#pragma unroll 1
        for (int c = 0; ok && c < n_mma * n_cols; c += 32) {
          float v[32];
          tmem_ld32(la + kTmemO + c, v);
          const int d = c + (c & 128);
          if (!Sh::kTma && whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t x[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * k + 2 * e] * f * f2, v[8 * k + 2 * e + 1] * f * f2);
                x[e] = *reinterpret_cast<const uint32_t*>(&b);
              }
              *reinterpret_cast<uint4*>(out + d + 8 * k) = make_uint4(x[0], x[1], x[2], x[3]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) st_global_v8(part + d + 8 * k, v + 8 * k);
          }
        }
      }
      if (warp < 6 && ok && share == 0) {
        const float m = misc->m_of[pi][h], l = misc->l_of[pi][h];
        if (!whole) {
          a.part_ml[slot * kHeads + h] = make_float2(m, l);
        } else if (a.lse != nullptr) {
          a.lse[static_cast<int64_t>(p.x) * kHeads + h] =
              l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&misc->o_free);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == Sh::kMmaWarp) {
    mbar_wait(&misc->drain, 0u, a.status, SITE_FULL);  // (after a timeout MMAs may be on their way)
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Four values of a part, which is read once (left to the compiler 1 x 131072 took 50.7 us, with
// read-only loads 45.3, this way 44.5).
__device__ __forceinline__ float4 ld_part(const float* p) {
  float4 x;
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "l"(p));
  return x;
}

// Joins the parts of the queries that several CTAs share: weights 2^(m_s - M) / L with M = max m_s
// and L = sum 2^(m_s - M) l_s. A unit of work is 128 dims of a head, a lane four of them;
// units are dealt out over the grid's warps, none of which waits for another, or, where there
// are few of many parts each, over its CTAs, whose warps share a unit's parts.
//
// A call with one split query runs each line of this code once, and fetching it took most of the
// kernel's 4.7 us. So it is kept short, and each CTA goes through it once without parts before it waits for
// the attention: while that still runs, where it leaves SMs idle (1 x 2048). Beside a CTA of the
// attention there is no room for one of these (4 KB of shared memory are left, and this takes 7), so in a full wave
// all of the join comes behind it.
constexpr int kUnits = kHeads * (kLatent / 128);  // of a query
constexpr int kJoinWarps = 4;
// A scheduler issues half the time, so what counts are instructions: four loads at once where most queries
// have two to four parts (64 x 8192 106.5 us with eight, 105.0 with four, 300 sequences of 0 to 1500 rows
// 75.9, 72.9), and CTAs of which none has many units (300 of 0 to 1500: 79.3 us with 4 an SM, 74.8 with
// 6, 73.6 with 10; a call without parts 0.9 us less with 4).
constexpr int kJoinPerSm = 8;  // CTAs
constexpr int kAhead = 4;      // parts whose loads are in flight together
__global__ void __launch_bounds__(32 * kJoinWarps, kJoinPerSm)
    full_join_kernel(const __grid_constant__ FullAttnArgs a, int n_ctas) {
  __shared__ int4 recs[kFullMaxCtas];
  __shared__ float wgts[kJoinWarps][kFullMaxCtas];
  __shared__ float4 accs[kJoinWarps][32];
  __shared__ int count[5];
  constexpr uint32_t all = 0xFFFFFFFFu;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  static_assert(kFullMaxCtas == 160 && kJoinWarps == 4 && kFullMaxCtas % kAhead == 0, "records");
  float* wgt = wgts[warp];
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int n_ctas_now = 0;
    if (pass == 1) {
      griddep_wait();
      griddep_launch_dependents();
      n_ctas_now = n_ctas;
    }
    // The records that name a query, in order (none in the first pass: a query without parts).
    const int4 none = make_int4(-1, 0, 0, 0);
    const int4 rec0 = tid < n_ctas_now ? a.records[tid] : none;
    const int4 rec1 = warp == 0 && 128 + lane < n_ctas_now ? a.records[128 + lane] : none;
    const uint32_t b0 = __ballot_sync(all, rec0.x >= 0), b1 = __ballot_sync(all, rec1.x >= 0);
    if (lane == 0) {
      count[warp] = __popc(b0);
      if (warp == 0) count[4] = __popc(b1);
    }
    __syncthreads();
    int n_rec = 0, at = 0;
#pragma unroll
    for (int w = 0; w < 5; ++w) {
      if (w < warp) at += count[w];
      n_rec += count[w];
    }
    const uint32_t below = (1u << lane) - 1u;
    if (rec0.x >= 0) recs[at + __popc(b0 & below)] = rec0;
    if (rec1.x >= 0) recs[n_rec - count[4] + __popc(b1 & below)] = rec1;
    if (pass == 0 && tid == 0) recs[0] = make_int4(0, 0, 0, 0);
    __syncthreads();
    const bool shared = pass == 0 || (n_rec * kUnits <= static_cast<int>(gridDim.x) && recs[0].z > kAhead);
    const int units = pass == 0 ? kUnits : n_rec * kUnits;
    const int step = pass == 0 ? kUnits : shared ? gridDim.x : gridDim.x * kJoinWarps;
#pragma unroll 1
    for (int u = pass == 0 ? 0 : shared ? blockIdx.x : blockIdx.x * kJoinWarps + warp; u < units;
         u += step) {
      const int4 rec = recs[u / kUnits];
      const int h = (u % kUnits) >> 2, d = 128 * (u & 3) + 4 * lane, n = rec.z;
      // part 0 is what run rec.y began, part k what run rec.y + k went on with
      auto slot_of = [&](int k) { return 2 * (rec.y + k) + (k == 0 ? 1 : 0); };
      const float* parts = a.parts + h * kLatent + d;
      const float2* mls = a.part_ml + h;
      // the warp's parts
      const int each = shared ? (n + kJoinWarps - 1) / kJoinWarps : n;
      const int k_begin = shared ? min(n, warp * each) : 0, k_end = min(n, k_begin + each);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float M = -INFINITY, L = 0.f;
      int k0 = k_begin;
#pragma unroll 1
      do {
        float4 x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k0 + k < k_end) {
            x[k] = ld_part(parts + static_cast<int64_t>(slot_of(k0 + k)) * (kHeads * kLatent));
          }
        }
        if (k0 == k_begin) {
          // (the first parts are on their way) A part without rows (sum 0) does not count, a
          // NaN sum does.
#pragma unroll 1
          for (int k = lane; k < n; k += 32) {
            const float2 ml = ld_ordered(mls + slot_of(k) * kHeads);
            if (!(ml.y == 0.f)) M = fmaxf(M, ml.x);
          }
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(all, M, o));
#pragma unroll 1
          for (int k = lane; k < n; k += 32) {
            const float2 ml = ld_ordered(mls + slot_of(k) * kHeads);  // (in the L1 by now)
            const float w = ml.y == 0.f ? 0.f : ex2_ftz(ml.x - M);
            L = fmaf(w, ml.y, L);
            wgt[k] = w;
          }
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) L += __shfl_xor_sync(all, L, o);
          __syncwarp();  // the weights are written
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (k0 + k < k_end) {
            const float w = wgt[k0 + k];
            acc.x = fmaf(w, x[k].x, acc.x);
            acc.y = fmaf(w, x[k].y, acc.y);
            acc.z = fmaf(w, x[k].z, acc.z);
            acc.w = fmaf(w, x[k].w, acc.w);
          }
        }
        k0 += kAhead;
      } while (k0 < k_end);
      __syncwarp();  // ... and read, before the next unit's
      if (shared) {
        accs[warp][lane] = acc;
        __syncthreads();
        if (warp == 0) {
#pragma unroll
          for (int w = 1; w < kJoinWarps; ++w) {
            const float4 x = accs[w][lane];
            acc = make_float4(acc.x + x.x, acc.y + x.y, acc.z + x.z, acc.w + x.w);
          }
        }
        __syncthreads();  // (accs, before the next unit)
      }
      if (n > 0 && (!shared || warp == 0)) {
        const float s = L == 0.f ? 0.f : 1.f / L, s2 = a.kv_fmt == kFmtE4m3 ? a.kv_scale : 1.f;
        const int64_t row = static_cast<int64_t>(rec.x) * kHeads + h;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * s * s2, acc.y * s * s2),
                             hi = __floats2bfloat162_rn(acc.z * s * s2, acc.w * s * s2);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * kLatent + d) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        if (a.lse != nullptr && d == 0) {
          a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
        }
      }
    }
    __syncthreads();  // (recs and count, before the second pass)
  }
}

template <int FMT>
cudaError_t launch_fmt(const FullAttnArgs& a, int grid, const CUtensorMap& qmap,
                       const CUtensorMap& lmap, const CUtensorMap& wmap, cudaStream_t s) {
  static std::atomic<int> smem_set[64]{};
  const cudaError_t e =
      ensure_smem(reinterpret_cast<const void*>(full_attn_kernel<FMT>), kSmemBytes, smem_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(full_attn_kernel<FMT>, dim3(grid), dim3(Shape<FMT>::kThreads), kSmemBytes, s, 1,
                    a, qmap, lmap, wmap);
}

}  // namespace

cudaError_t launch_full_attn(const FullAttnArgs& a, cudaStream_t s) {
  const int grid = std::min(device_sm_count(), kFullMaxCtas);
  CUtensorMap qmap, lmap, wmap;
  memset(&qmap, 0, sizeof(qmap));
  memset(&lmap, 0, sizeof(lmap));
  memset(&wmap, 0, sizeof(wmap));
  cudaError_t e = encode_tma_2d(&qmap, a.q, 2, kLatent, static_cast<uint64_t>(a.n_queries) * kHeads,
                                kLatent * 2, 64, kHeads);
  if (e != cudaSuccess) return e;
  if (a.kv_fmt != DSA_KV_MXFP4) {
    const int elem = a.kv_fmt == DSA_KV_BF16 ? 2 : 1;
    // (a cache without rows: a map of one row of the queries, which no box reads)
    const bool any = a.lat_rows > 0;
    e = encode_tma_2d(&lmap, any ? a.latents : a.q, elem, kLatent,
                      any ? static_cast<uint64_t>(a.lat_rows) : 1, kLatent * elem, 128 / elem, kSub);
    if (e != cudaSuccess) return e;
    if (a.swa != nullptr) {
      const int64_t seqs = a.mq > 0 ? a.n_queries / a.mq : a.n_queries;
      e = encode_tma_2d(&wmap, a.swa, elem, kLatent, static_cast<uint64_t>(seqs * a.swa_seq_rows),
                        kLatent * elem, 128 / elem, kSub);
      if (e != cudaSuccess) return e;
    }
  }
  if (a.kv_fmt == DSA_KV_BF16) {
    e = launch_fmt<DSA_KV_BF16>(a, grid, qmap, lmap, wmap, s);
  } else if (a.kv_fmt == DSA_KV_FP8_E4M3) {
    e = launch_fmt<DSA_KV_FP8_E4M3>(a, grid, qmap, lmap, wmap, s);
  } else {
    e = launch_fmt<DSA_KV_MXFP4>(a, grid, qmap, lmap, wmap, s);
  }
  if (e != cudaSuccess) return e;
  // at most one query a CTA but the first is split
  const int64_t units = int64_t{std::min(a.n_queries, grid - 1)} * kUnits;
  const int join = static_cast<int>(std::min<int64_t>(units, int64_t{kJoinPerSm} * device_sm_count()));
  return launch_pdl(full_join_kernel, dim3(std::max(join, 1)), dim3(32 * kJoinWarps), 0, s, 1, a, grid);
}

}  // namespace dsa
