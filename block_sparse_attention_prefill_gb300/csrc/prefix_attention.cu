// Dense causal attention over the paged E4M3 cache for a batch whose requests
// share their first pages: the part over the shared pages is computed once
// for all requests.  sm_103a: TMA, tcgen05, TMEM.
//
// With s_j = (q . k_j) c (c: the scales times log2 e) the kernel keeps, per
// query row, a reference m near the running maximum, l = sum 2^(s_j - m) and
// O = sum 2^(s_j - m) v_j over a range of pages; ranges are merged by their
// l and m (combine kernel below).  QK is an E4M3 MMA, exact products with
// fp32 sums; the probabilities are rounded to f16 (2^-11 of their value at
// most) and V widened to f16 (exact), so that the bf16 output is limited by
// its own rounding.
//
// Work.  Rows are (token, query head of one KV head).  A tile is up to 2 C
// tokens, C = floor(128 / G), with a range of pages: the shared pages for
// tiles over the whole batch's tokens (they lie before every query: no mask),
// a request's own pages for tiles over its tokens (and the shared pages with
// them where that costs less).  Both are the same kind of work.  A tile of
// more than C tokens is two 128-row halves that share every page (pair); a
// smaller one has its pages dealt in turn to the two streams, each with its
// own O (solo).  The tiles of all heads, laid end to end and weighted by
// pages, are cut into one equal range per CTA, so no CTA waits for a last
// wave and only tiles that a cut meets are split.
//
// Kernels: plan (one CTA: tiles and their place in the line; of a small batch
// every attend CTA makes it for itself), attend (one persistent CTA per SM),
// combine.
//
// Attend, by warps: 0 copies pages and Q (TMA), 3 issues the QKs, 1 and 2 the
// PVs of a stream, 4-7 and 8-11 are a stream's softmax (a row a thread), 12-15
// widen V.  Tensor memory holds, for each stream, two S of 64 keys (P takes
// its S's place) and O: all 512 columns.  The unit of 64 keys, not 128, is what
// lets QK of one unit, softmax of the next and PV run at the same time within
// a stream.
//
// Bounds and what was measured (GPU time of a call's launches, replayed from a
// graph; a call of its own takes 4-8 us more): 512 tokens x 16 heads over 128k
// shared keys 338 us, 1.64 PFLOP/s; QK at twice and PV at the bf16 rate would
// take 217.  A unit of both streams takes 1440 cycles, of which the tensor
// pipes are busy 0.6 (ncu), the issue slots 0.58: what is left is the latency
// of the hops S -> softmax -> P -> PV -> next QK, with all of tensor memory
// in use.  16 requests of 8 tokens over 83k keys of their own each: 130 us, 678 MB at
// 5.2 TB/s.  16 single tokens over 32k shared keys: 21.7 us, latency (plan
// and first loads 4, 6 units 5, epilogue 3, combine 5 us).
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "partial.cuh"
#include "ptx.cuh"

namespace msa {
namespace {

// ------------------------------------------------------------------- tiles

// Cost of a tile: its pages by kind, and its start and end (Q, epilogue), in
// the proportions measured (about 0.9, 1.8 and 4.5 us).
constexpr int kCostSolo = 2, kCostPair = 4, kCostTile = 10;
constexpr int kMinShare = 12;  // least cost of a CTA's range

// Behind every key (positions are below 2^30), with room for a tile's tokens.
constexpr int kNoMask = INT_MAX - 1024;

struct __align__(16) Tile {
  int b;       // row of block_table
  int tok0;    // first token
  int ntok;    // tokens
  int page0;   // first logical page
  int npages;
  uint32_t start;  // cost of the head's tiles before this one
  int pos0;    // position of tok0, or kNoMask (the shared pages)
  int seq;     // keys of the request (a page's keys behind it are not read)
};
struct PlanHead {
  int ntiles;
  uint32_t cost;  // of all tiles
  int shared_tiles;
  int bad;  // lengths inconsistent: every output row becomes empty
  int T;    // tokens of the batch
  int pad[3];
};
// The tiles of a head in line order: those over the shared pages, then each
// request's own.  In memory the own ones begin at a place that the sizes
// alone give, so that reading one need not wait for the plan's head.
__host__ __device__ inline int64_t own_base(int64_t T, int64_t C, int64_t prefix) {
  return prefix > 0 ? ceil_div(T, 2 * C) : 0;
}

__host__ __device__ inline int64_t max_tiles(int64_t B, int64_t T, int64_t C, int64_t prefix) {
  const int64_t n = ceil_div(T, 2 * C);
  return own_base(T, C, prefix) + (T < n + B ? T : n + B);
}

__device__ __forceinline__ int tile_rate(int ntok, int C) { return ntok > C ? kCostPair : kCostSolo; }
__device__ __forceinline__ int tile_cost(int ntok, int npages, int C) {
  return npages * tile_rate(ntok, C) + kCostTile;
}
// Cost of a page for all tiles of `tokens` consecutive tokens.
__device__ __forceinline__ int rate_of(int tokens, int C) {
  const int rest = tokens % (2 * C);
  return tokens / (2 * C) * kCostPair + (rest > C ? kCostPair : rest > 0 ? kCostSolo : 0);
}
// Pages of a tile in front of cost y of its own.
__device__ __forceinline__ int pages_before(int64_t y, int npages, int rate) {
  if (y <= kCostTile) return 0;
  const int64_t p = (y - kCostTile + rate - 1) / rate;
  return p < npages ? (int)p : npages;
}
__device__ __forceinline__ int64_t share_of(int64_t total, int ctas) {
  const int64_t s = total <= INT_MAX - ctas ? ((int)total + ctas - 1) / ctas
                                            : (total + ctas - 1) / ctas;
  return s > kMinShare ? s : kMinShare;
}

// Rows of the partials.  A tile's part at CTA i starts at row 256 i + (its
// head's rows) + (the rows before it): parts in line order never overlap,
// because a part has its tile's rows, at most 256 of them.
__device__ __forceinline__ int64_t part_row(int cta, int h, int tile, int shared_tiles, int tok0,
                                            int T, int G) {
  const int64_t rows = (int64_t)T * G;
  const int64_t per_head = shared_tiles > 0 ? 2 * rows : rows;
  return 256 * (int64_t)cta + h * per_head + (tile >= shared_tiles && shared_tiles > 0 ? rows : 0) +
         (int64_t)tok0 * G;
}

// Where a part's O of a row lies, in floats from its first row's: the rows of
// a stream go in blocks of 32 (a warp's), a block as 16 chunks of 8 columns,
// [chunk][row][8], so that a warp's stores of a chunk, and loads of
// neighbouring rows, are contiguous (rows one after another: 111 us instead of
// 105, before the plan's last change, for five chunks of 1 .. 700 tokens, by
// the cache's tag look-ups).
struct RowPlace {
  int first;  // of column 0
  int chunk;  // from one chunk to the next
};
__device__ __forceinline__ RowPlace row_place(int off, int ntok, int C, int G) {
  const int s0 = ntok > C && off >= C * G ? C * G : 0;
  const int rows = s0 > 0 ? (ntok - C) * G : (ntok > C ? C : ntok) * G;
  const int w = off - s0, block = w & ~31;
  return {(s0 + block) * kD + (w & 31) * 8, min(32, rows - block) * 8};
}

constexpr int kPlanThreads = 1024;

template <int kThreads>
__device__ __forceinline__ uint32_t block_excl_scan(uint32_t v, uint32_t* total) {
  __shared__ uint32_t sums[33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const uint32_t s = lane < kThreads / 32 ? sums[lane] : 0;
    uint32_t si = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t n = __shfl_up_sync(0xffffffffu, si, o);
      if (lane >= o) si += n;
    }
    sums[lane] = si - s;
    if (lane == 31) sums[32] = si;
  }
  __syncthreads();
  const uint32_t r = sums[warp] + incl - v;
  *total = sums[32];
  __syncthreads();
  return r;
}

struct PlanParams {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int B, T, C, prefix;
  int64_t max_q, max_k;
  PlanHead* head;
  Tile* tiles;
  int own_base;
  int* req;  // [B] own tiles of the requests before each
  uint32_t* status;
};

// Lists the tiles of one head (every head has the same): first those over the
// shared pages, then each request's own.  Run by a whole CTA; req is room for
// B ints that it can see.  Every thread gets the plan's head.
template <int kThreads>
__device__ __forceinline__ PlanHead make_plan(const PlanParams& p, int* req) {
  __shared__ int s_bad, s_first, s_rate;
  const int tid = threadIdx.x;
  if (tid == 0) s_bad = 0, s_first = INT_MAX, s_rate = 0;
  __syncthreads();
  const int T = p.cu_q[p.B];
  bool bad = p.cu_q[0] != 0 || T < 0 || T > p.T;
  int run = 0;  // tiles of the requests before this round's
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < p.B) {
      const int64_t q = (int64_t)p.cu_q[b + 1] - p.cu_q[b];
      const int64_t k = (int64_t)p.cu_k[b + 1] - p.cu_k[b];
      if (q < 0 || k < q || q > p.max_q || k > p.max_k ||
          (q > 0 && k - q < (int64_t)p.prefix * kPage))
        bad = true;
      else if (q > 0) {
        n = (int)((q + 2 * p.C - 1) / (2 * p.C));
        atomicMin(&s_first, b);
        atomicAdd(&s_rate, rate_of((int)q, p.C));
      }
    }
    uint32_t total;
    const int before = (int)block_excl_scan<kThreads>(n, &total);
    if (b < p.B) req[b] = run + before;
    run += (int)total;
  }
  if (bad) s_bad = 1;
  __syncthreads();  // also makes req visible to this CTA
  if (s_bad) {
    const PlanHead hd = {0, 0, 0, 1, 0, {0, 0, 0}};
    if (tid == 0) {
      *p.head = hd;
      if (p.status) atomicOr(p.status, (unsigned)MSA_STATUS_BAD_SEQLENS);
    }
    return hd;
  }
  // The shared pages as tiles of their own, or as part of each request's own
  // tiles (one request, chunks that fill tiles, a page or two): what costs less
  // (five chunks of 1 .. 700 tokens: 106.5 us and 102).
  int shared_tiles = p.prefix > 0 ? (T + 2 * p.C - 1) / (2 * p.C) : 0;
  if ((int64_t)p.prefix * (s_rate - rate_of(T, p.C)) <= (int64_t)shared_tiles * kCostTile)
    shared_tiles = 0;
  const int prefix = shared_tiles > 0 ? p.prefix : 0;
  const int ntiles = shared_tiles + run;
  uint32_t cost = 0;
  for (int i0 = 0; i0 < ntiles; i0 += kThreads) {
    const int i = i0 + tid;
    Tile t = {};
    int c = 0;
    if (i < ntiles) {
      if (i < shared_tiles) {
        t.b = s_first;
        t.tok0 = i * 2 * p.C;
        t.ntok = min(2 * p.C, T - t.tok0);
        t.page0 = 0;
        t.npages = prefix;
        t.pos0 = kNoMask;
        t.seq = prefix * kPage;
      } else {
        int lo = 0, hi = p.B - 1;  // the last request with req[b] <= i
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (req[mid] <= i - shared_tiles) lo = mid; else hi = mid - 1;
        }
        const int q = p.cu_q[lo + 1] - p.cu_q[lo], k = p.cu_k[lo + 1] - p.cu_k[lo];
        const int o = (i - shared_tiles - req[lo]) * 2 * p.C;
        t.b = lo;
        t.tok0 = p.cu_q[lo] + o;
        t.ntok = min(2 * p.C, q - o);
        t.page0 = prefix;
        t.pos0 = k - q + o;
        t.npages = (t.pos0 + t.ntok - 1) / kPage + 1 - prefix;
        t.seq = k;
      }
      c = tile_cost(t.ntok, t.npages, p.C);
    }
    uint32_t total;
    t.start = cost + block_excl_scan<kThreads>(c, &total);
    cost += total;
    if (i < ntiles)
      p.tiles[i < shared_tiles ? i : p.own_base + i - shared_tiles] = t;
  }
  const PlanHead hd = {ntiles, cost, shared_tiles, 0, T, {0, 0, 0}};
  if (tid == 0) *p.head = hd;
  return hd;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  pdl_wait();
  pdl_trigger();
  make_plan<kPlanThreads>(p, p.req);
}

// ------------------------------------------------------------------ attend

constexpr int kThreads = 512;
constexpr int kTileBytes = 128 * 128;       // an E4M3 tile of 128 x 128
constexpr int kRawK = 4, kRawV = 3;         // K and V pages in flight
constexpr int kWide = 4;                    // half pages of V widened to f16
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + 2 * kTileBytes;
constexpr int kOffV = kOffK + kRawK * kTileBytes;
constexpr int kOffW = kOffV + kRawV * kTileBytes;
constexpr int kOffBars = kOffW + kWide * kTileBytes;
constexpr int kThere = 16;  // more than the roles can be apart
constexpr int kIsThere = 1, kHasNan = 2;
struct Bars {
  uint64_t q_full, q_free;
  uint64_t k_full[kRawK], k_free[kRawK], v_full[kRawV], v_free[kRawV];
  uint64_t w_full[kWide], w_free[kWide];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // [stream][buffer]
  uint64_t part_done;
  uint64_t exchanged, read;  // the streams' results at the end of a solo part
  uint64_t mma_done[3];
  uint32_t tmem_base;
  int abort;
  int first_tile;
  float2 ml[2][128];  // a solo part's m and l by stream and row
  // whether a ring position's page is one, by the producer; kHasNan too where a
  // NaN lies among the V codes of its keys and not every row sees it whole
  uint8_t there[kThere];
};
constexpr int kSmem = kOffBars + (int)sizeof(Bars) + 1024;
static_assert(kSmem <= 232448, "shared memory of a CTA");
constexpr int kHalf = kPage / 2;  // keys of a unit: of one S, and one P
// Tensor memory, per stream s: two buffers of S (64 columns each) from column
// 128 s on, O at 256 + 128 s.  P (f16, 32 columns) replaces its S.
constexpr int kTmemCols = 512, kColO = 256;
// 512 threads with 128 registers each, shared out anew among the roles
// (of the launch's 128, 108 bytes are spilled)
constexpr int kRegsControl = 120, kRegsSoftmax = 144, kRegsWiden = 104;
static_assert(kRegsControl + 2 * kRegsSoftmax + kRegsWiden <= 512, "registers");
// P is kept as 2^(s - m + 7): a unit whose P add up to at most 2^15 has none
// outside f16's range, and f16's subnormals begin 2^-21 below the reference
// instead of 2^-14
constexpr float kPShift = 7.f, kMostSum = 32768.f;
constexpr float kLeftOut = -1.f;  // a weight in the merge of a part's streams

struct AttendParams {
  PlanParams plan;
  int plan_here;  // each CTA makes the plan for itself (all write the same)
  const Tile* tiles;
  int own_base;
  const int32_t* block_table;
  int64_t bt_stride;
  const uint8_t* kv;
  int num_pages;
  int T, G, C, Hkv;
  float score_log2;
  float* part_o;    // rows of 128 fp32, normalised, as in row_place
  float* part_lse;  // base-2 log-sum-exp of the row's part
  uint32_t* status;
  uint32_t wait_ns;
};

// One CTA's range of the line, tile by tile; each role walks it for itself.
struct Walk {
  const AttendParams& p;
  int ntiles, shared_tiles;
  int left;          // cost of the range still ahead
  int at;            // cost of the tile before the range
  int h, tile;
  Tile t, ahead;
  int p0, p1;        // pages of the tile in this range
  int cur_h, cur_tile;
  __device__ Walk(const AttendParams& prm, const PlanHead& hd, int first_tile)
      : p(prm), ntiles(hd.ntiles), shared_tiles(hd.shared_tiles), tile(first_tile) {
    const int64_t total = (int64_t)hd.cost * p.Hkv, share = share_of(total, gridDim.x);
    const int64_t x = blockIdx.x * share;
    left = x < total ? (int)min(share, total - x) : 0;
    h = left > 0 ? (int)(x / hd.cost) : 0;
    if (left > 0) {
      ahead = tile_at(tile);
      at = (int)(x - (int64_t)h * hd.cost - ahead.start);
    }
  }
  __device__ __forceinline__ const Tile& tile_at(int i) const {
    return p.tiles[i < shared_tiles ? i : p.own_base + i - shared_tiles];
  }
  // The next part with pages; false at the range's end.
  __device__ __forceinline__ bool next() {
    while (left > 0) {
      t = ahead;
      const int rate = tile_rate(t.ntok, p.C), cost = tile_cost(t.ntok, t.npages, p.C);
      const int take = min(left, cost - at);
      p0 = pages_before(at, t.npages, rate);
      p1 = pages_before(at + take, t.npages, rate);
      cur_h = h;
      cur_tile = tile;
      left -= take;
      at += take;
      if (at == cost) {
        at = 0;
        if (++tile == ntiles) tile = 0, ++h;
      }
      if (left > 0) ahead = tile_at(tile);  // in flight while this part is worked on
      if (p1 > p0) return true;
    }
    return false;
  }
  __device__ __forceinline__ bool pair() const { return t.ntok > p.C; }
  // pages that stream s handles of this part
  __device__ __forceinline__ int stream_pages(int s) const {
    return pair() ? p1 - p0 : (p1 - p0 + 1 - s) >> 1;
  }
  // the part's i-th page of stream s, counted from p0
  __device__ __forceinline__ int stream_page(int s, int i) const { return pair() ? i : 2 * i + s; }
};

// A ring of four slots that both streams use: in a pair part both use every
// item in turn (v: the item's number within the part); in a solo part each
// stream has two slots of its own (v: its number within the stream), so that
// neither waits for the other's progress.  A barrier tells a phase only from
// the next, so all who use a ring count every use of every slot: `odd` has a
// bit for each slot, set after an odd number of uses in earlier parts.
struct Ring {
  uint32_t odd = 0;
  static __device__ __forceinline__ uint32_t slot(bool pair, int s, uint32_t v) {
    return pair ? v & 3u : 2u * s + (v & 1u);
  }
  // the parity of this use's phase of the slot; its complement's phase is the
  // one before (complete at once on a new barrier)
  __device__ __forceinline__ uint32_t phase(bool pair, uint32_t slot, uint32_t v) const {
    return ((odd >> slot) ^ (pair ? v >> 2 : v >> 1)) & 1u;
  }
  // a part with n0 and n1 items of the two streams (pair: n0 in all) is over
  __device__ __forceinline__ void advance(bool pair, uint32_t n0, uint32_t n1) {
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
      const uint32_t n = pair ? n0 : k < 2 ? n0 : n1;
      odd ^= ((pair ? (n + 3 - k) >> 2 : (n + 1 - (k & 1)) >> 1) & 1u) << k;
    }
  }
};

__device__ __forceinline__ void give_up(Bars* bars, uint32_t* status) {
  *(volatile int*)&bars->abort = 1;
  if (status) atomicOr(status, (unsigned)MSA_STATUS_TIMEOUT);
}

// A wait of a whole warp: all lanes poll and agree, one vote a try (about 40
// cycles less than lanes that wait for themselves and vote in the end).
__device__ __forceinline__ bool all_wait(Bars* bars, uint64_t* bar, uint32_t parity,
                                         const AttendParams& p) {
  if (__all_sync(0xffffffffu, mbar_try_wait_long(bar, parity))) return true;
  const uint32_t t0 = (uint32_t)global_timer_ns();
  for (;;) {
    if (__all_sync(0xffffffffu, mbar_try_wait_long(bar, parity))) return true;
    const bool stop = *(volatile int*)&bars->abort || (uint32_t)global_timer_ns() - t0 > p.wait_ns;
    if (__any_sync(0xffffffffu, stop)) break;
  }
  if ((threadIdx.x & 31) == 0 && !*(volatile int*)&bars->abort) give_up(bars, p.status);
  return false;
}

// Four E4M3 codes -> four f16 in two words (exact).
__device__ __forceinline__ uint2 widen4(uint32_t c) {
  uint2 h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}\n"
      : "=r"(h.x), "=r"(h.y)
      : "r"(c));
  return h;
}
// 0x80 in each byte of w whose E4M3 code is NaN (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

__global__ void __launch_bounds__(kThreads, 1)
attend_kernel(const __grid_constant__ CUtensorMap kv_map, const __grid_constant__ CUtensorMap q_map,
              const AttendParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const volatile int* abort = &bars->abort;

  if (tid == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_free, 1);
    for (int i = 0; i < kRawK; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_free[i], 1);
    }
    for (int i = 0; i < kRawV; ++i) {
      mbar_init(&bars->v_full[i], 1);
      mbar_init(&bars->v_free[i], 4);
    }
    for (int i = 0; i < kWide; ++i) {
      mbar_init(&bars->w_full[i], 4);
      mbar_init(&bars->w_free[i], 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars->s_full[i >> 1][i & 1], 1);
      mbar_init(&bars->p_full[i >> 1][i & 1], 128);
      mbar_init(&bars->pv_done[i >> 1][i & 1], 1);
    }
    mbar_init(&bars->part_done, 2);
    mbar_init(&bars->exchanged, 256);
    mbar_init(&bars->read, 256);
    for (int i = 0; i < 3; ++i) mbar_init(&bars->mma_done[i], 1);
    bars->abort = 0;
    bars->first_tile = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  // Where G does not divide 128 no copy writes the last rows of Q.  They give
  // no output, but a NaN that shared memory held there would have the softmax
  // move its reference at every unit (94 us became 145).
  for (int i = p.C * p.G * kD + tid * 16; i < kTileBytes; i += kThreads * 16)
    for (int s = 0; s < 2; ++s)
      *reinterpret_cast<uint4*>(smem + kOffQ + s * kTileBytes + i) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  pdl_wait();
  pdl_trigger();
  // The workspace's plan: by a kernel of its own, or, while it takes one
  // round of this CTA's threads, here: the CTAs write the same values to the
  // same places, and each reads what it has written itself.
  PlanHead hd;
  if (p.plan_here)
    hd = make_plan<kThreads>(p.plan, reinterpret_cast<int*>(smem + kOffW));
  else
    hd = *p.plan.head;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  // the tile that this CTA's range starts in
  {
    const int64_t total = (int64_t)hd.cost * p.Hkv;
    const int64_t x = blockIdx.x * share_of(total, gridDim.x);
    if (x < total) {
      const uint32_t r = (uint32_t)(x % hd.cost);
      auto start = [&](int i) {
        return p.tiles[i < hd.shared_tiles ? i : p.own_base + i - hd.shared_tiles].start;
      };
      for (int i = tid; i < hd.ntiles; i += kThreads)
        if (start(i) <= r && (i + 1 == hd.ntiles || start(i + 1) > r)) bars->first_tile = i;
    }
  }
  __syncthreads();
  Walk walk(p, hd, bars->first_tile);

  if (warp >= 4 && warp < 12) {
    setmaxnreg_inc<kRegsSoftmax>();
    // ------------------------------------------------------------- softmax
    const int s = warp >= 8, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t s_tmem = tmem + lane_off + s * 128, o_tmem = s_tmem + kColO;
    const float c = p.score_log2;
    const int i_tok = row / p.G;
    uint32_t done = 0;  // units (half pages) of this stream so far
    uint32_t g0 = 0;    // pages of the parts before
    uint32_t solos = 0; // solo parts so far
    bool ok = true;
    while (ok && walk.next()) {
      const Tile& t = walk.t;
      const bool pair = walk.pair();
      const int n = walk.stream_pages(s);
      const int ntok = pair ? (s ? t.ntok - p.C : p.C) : t.ntok;
      const bool valid = i_tok < ntok;
      const int tok = i_tok + (pair && s ? p.C : 0);  // within the tile
      const int pos = t.pos0 + tok;
      const int32_t* table = p.block_table + t.b * p.bt_stride + t.page0;
      // the first position of the warp's rows: pages before it need no mask
      const int least = __reduce_min_sync(0xffffffffu, pos);
      float m = -INFINITY, l = 0.f;  // m: scores in units of 1 (not log2)
      float off = 0.f;
      int key0 = 0;  // the unit's first key
#pragma unroll 1
      for (int i = 0; i < 2 * n; ++i, ++done) {
        if ((i & 1) == 0) {
          key0 = (t.page0 + walk.p0 + walk.stream_page(s, i >> 1)) * kPage;
        } else {
          key0 += kHalf;
        }
        const uint32_t buf = done & 1, s_cols = s_tmem + buf * kHalf;
        if (!all_wait(bars, &bars->s_full[s][buf], (done >> 1) & 1, p)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t r[2][32];
        tmem_ld32(s_cols, r[0]);
        tmem_ld32(s_cols + 32, r[1]);
        tmem_wait_ld();
        const bool there = bars->there[(g0 + walk.stream_page(s, i >> 1)) % kThere];
        if (!there || key0 + kHalf - 1 > least) {
          const int lim = there ? pos - key0 : -1;  // the last key this row attends to
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (q * 32 + e > lim) r[q][e] = 0xFF800000u;  // -inf
        }
        const float2 c2 = make_float2(c, c);
        // The reference m is the maximum of the row's first unit.  Later
        // maxima are not waited for: only where the unit's P add up to more
        // than kMostSum (so that one could pass f16's range) m moves to the
        // maximum, O and l with it, and the unit is done again.
        bool move = m == -INFINITY;
        float sum;
#pragma unroll 1
        for (;;) {
          if (__any_sync(0xffffffffu, move)) {
            float mx[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(r[q][e]));
            // only the rows that need it move: what a row gives does not
            // depend on the others of its warp
            const float top = move ? fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) : m;
            if (i > 0) {
              // every PV of the stream has to be complete: the one before
              // this unit is the last issued
              if (!all_wait(bars, &bars->pv_done[s][buf ^ 1], ((done - 1) >> 1) & 1, p)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const float f = !move ? 1.f : m == -INFINITY ? 0.f : ex2_approx((m - top) * c);
              l *= f;
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                uint32_t o[32];
                tmem_ld32(o_tmem + q * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(o_tmem + q * 32, o);
              }
            }
            m = top;
            off = m == -INFINITY ? 0.f : kPShift - m * c;
          }
          // P into its buffer, in groups of 8 pairs, exponentials first, so
          // that their latencies overlap; each half is stored as it is done
          const float2 off2 = make_float2(off, off);
          float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; k += 8) {
              float2 a[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                a[e] = fma2(make_float2(__uint_as_float(r[q][2 * (k + e)]),
                                        __uint_as_float(r[q][2 * (k + e) + 1])),
                            c2, off2);
#pragma unroll
              for (int e = 0; e < 8; ++e) a[e].x = ex2_approx(a[e].x), a[e].y = ex2_approx(a[e].y);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                sums[e & 1] = add2(sums[e & 1], a[e]);
                const __half2 h = __floats2half2_rn(a[e].x, a[e].y);
                w[k + e] = *reinterpret_cast<const uint32_t*>(&h);
              }
            }
            tmem_st16(s_cols + q * 16, w);
          }
          sum = (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
          const bool again = !move && sum > kMostSum;
          if (!__any_sync(0xffffffffu, again)) break;
          move = again;
        }
        if (!ok) break;
        l += sum;
        tmem_wait_st();
        // the first PV of a part overwrites O: the other stream has read it
        if (i == 0 && solos > 0 && !all_wait(bars, &bars->read, (solos - 1) & 1, p)) {
          ok = false;
          break;
        }
        tc_fence_before();
        mbar_arrive(&bars->p_full[s][buf]);
      }
      if (!ok) break;
      // the part: O / l and log2 of the row's sum
      const int64_t first_row = part_row(blockIdx.x, walk.cur_h, walk.cur_tile, walk.shared_tiles,
                                         t.tok0, p.T, p.G);
      const int off_row = (pair && s ? p.C * p.G : 0) + row;
      g0 += walk.p1 - walk.p0;
      if (n > 0 &&
          !all_wait(bars, &bars->pv_done[s][(done - 1) & 1], ((done - 1) >> 1) & 1, p))
        break;
      tc_fence_after();
      // In a solo part the streams have the same rows, in the same lanes of
      // tensor memory: either writes half the columns of both streams' sum.
      // Weights of the own and the other stream's O.  What has no keys (l = 0)
      // is left out, whatever its O holds (weight kLeftOut); a weight that
      // underflows to 0 is no reason to, since a NaN in l (among the scores)
      // makes the row NaN and one in O (among V) its column.
      float wa = l == 0.f ? kLeftOut : 1.f, wb = kLeftOut, lt = l, mt = m;
      if (!pair) {
        if (solos > 0 && !all_wait(bars, &bars->read, (solos - 1) & 1, p)) break;
        bars->ml[s][row] = make_float2(m, l);
        tc_fence_before();
        mbar_arrive(&bars->exchanged);
        if (!all_wait(bars, &bars->exchanged, solos & 1, p)) break;
        tc_fence_after();
        const float2 z = bars->ml[s ^ 1][row];
        mt = fmaxf(m, z.x);
        wa = l == 0.f ? kLeftOut : m == -INFINITY ? 1.f : ex2_approx((m - mt) * c);
        wb = z.y == 0.f ? kLeftOut : z.x == -INFINITY ? 1.f : ex2_approx((z.x - mt) * c);
        lt = (wa < 0.f ? 0.f : l * wa) + (wb < 0.f ? 0.f : z.y * wb);
      }
      // Where a NaN lies among the V codes of a key in a page that some row
      // does not see whole, widening wrote it as 0, since a probability of 0
      // must hide it; now each warp finds, for each column, the first position
      // that has one (pages of that kind are the last three of a tile at most).
      bool poison = false;
      int nan_key[4] = {INT_MAX, INT_MAX, INT_MAX, INT_MAX};  // columns 4 lane ..
      for (int j = max(walk.p0, (t.pos0 + 1) / kPage - t.page0); j < walk.p1; ++j) {
        if (bars->there[(g0 + j - walk.p1) % kThere] & kHasNan) {
          poison = true;
          const int pg = __ldg(table + j);
          const uint8_t* v = p.kv + ((int64_t)pg * p.Hkv + walk.cur_h) * kPage * (2 * kD) + kD;
          const int first = (t.page0 + j) * kPage;
          for (int k = 0; k < kPage && first + k < t.seq; ++k) {
            const uint32_t bad = nan_bytes(
                __ldg(reinterpret_cast<const uint32_t*>(v + k * (2 * kD)) + lane));
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((bad >> (8 * e)) & 0x80u) nan_key[e] = min(nan_key[e], first + k);
          }
        }
      }
      const float inv = lt == 0.f ? 0.f : 1.f / lt;
      const float fa = wa < 0.f ? kLeftOut : wa * inv, fb = wb < 0.f ? kLeftOut : wb * inv;
      const RowPlace place = row_place(off_row, t.ntok, p.C, p.G);
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.part_o + first_row * kD) + place.first;
      const int q0 = pair ? 0 : 4 * s, q1 = pair ? 8 : q0 + 4;
#pragma unroll 1
      for (int q = q0; q < q1; ++q) {
        uint32_t o[16], x[16];
        tmem_ld16(o_tmem + q * 16, o);
        tmem_ld16(o_tmem + q * 16 + (s ? -128 : 128), x);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          o[e] = __float_as_uint((fa < 0.f ? 0.f : __uint_as_float(o[e]) * fa) +
                                 (fb < 0.f ? 0.f : __uint_as_float(x[e]) * fb));
        if (poison) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (__shfl_sync(0xffffffffu, nan_key[e & 3], q * 4 + (e >> 2)) <= pos)
              o[e] = 0x7FFFFFFFu;
        }
        if (valid) {
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            st_global_v8(dst + (2 * q + e / 8) * place.chunk, o[e], o[e + 1], o[e + 2], o[e + 3],
                         o[e + 4], o[e + 5], o[e + 6], o[e + 7]);
        }
      }
      tc_fence_before();
      if (!pair) {
        mbar_arrive(&bars->read);
        ++solos;
      }
      if (valid && (pair || s == 0))
        p.part_lse[first_row + off_row] = lt == 0.f ? -INFINITY : mt * c - kPShift + log2f(lt);
    }
  } else if (warp >= 12) {
    setmaxnreg_dec<kRegsWiden>();
    // -------------------------------------------------------------- widen
    // 128 threads: a page's V codes in pieces of 8; thread wt has piece
    // wt % 16 of keys wt / 16, + 8, ..., read through the TMA's 128-byte
    // swizzle and written as one 16-byte chunk of an f16 tile [64 keys][dims],
    // two blocks of 64 dims, 128-byte swizzle (its keys are alike modulo 8, so
    // the swizzle is the same for all; eight lanes write a whole row of a
    // block, without bank conflicts).
    const int wt = tid - 384, key0 = wt >> 4, piece = wt & 15;
    const int src0 = key0 * 128 + (((piece >> 1) ^ key0) << 4) + (piece & 1) * 8;
    const int dst0 = (piece >> 3) * (kTileBytes / 2) + key0 * 128 + (((piece & 7) ^ key0) << 4);
    int g = 0;
    Ring ring;
    bool ok = true;
    while (ok && walk.next()) {
      const Tile& t = walk.t;
      const bool pair = walk.pair();
      for (int j = walk.p0; j < walk.p1; ++j, ++g) {
        if (!all_wait(bars, &bars->v_full[g % kRawV], (g / kRawV) & 1, p)) {
          ok = false;
          break;
        }
        const int keys =
            bars->there[g % kThere] ? min(kPage, t.seq - (t.page0 + j) * kPage) : 0;
        // Every row of the tile sees all of a whole page: a NaN in it may
        // flow through PV.  In the others a probability of 0 has to hide one:
        // it is written as 0, and put back where it is seen in the end.
        const bool whole = keys == kPage && (t.page0 + j + 1) * kPage <= t.pos0 + 1;
        const uint8_t* src = smem + kOffV + (g % kRawV) * kTileBytes + src0;
        // all loads first, so that the conversions overlap
        uint2 w[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) w[u] = *reinterpret_cast<const uint2*>(src + u * 8 * 128);
        if (!whole) {
          uint32_t bad = 0;
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            if (key0 + u * 8 >= keys) w[u] = make_uint2(0u, 0u);
            const uint32_t x = nan_bytes(w[u].x), y = nan_bytes(w[u].y);
            bad |= x | y;
            w[u].x &= ~((x >> 7) * 0xFFu);
            w[u].y &= ~((y >> 7) * 0xFFu);
          }
          if (bad) bars->there[g % kThere] = kIsThere | kHasNan;
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int i = j - walk.p0;  // the page within the part
          const uint32_t x = pair ? 2 * i + half : (i & ~1) + half;
          const uint32_t slot = Ring::slot(pair, i & 1, x);
          if (!all_wait(bars, &bars->w_free[slot], ring.phase(pair, slot, x) ^ 1, p)) {
            ok = false;
            break;
          }
          uint8_t* dst = smem + kOffW + slot * kTileBytes + dst0;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint2 a = widen4(w[8 * half + u].x), b = widen4(w[8 * half + u].y);
            *reinterpret_cast<uint4*>(dst + u * 8 * 128) = make_uint4(a.x, a.y, b.x, b.y);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (half) mbar_arrive(&bars->v_free[g % kRawV]);
            mbar_arrive(&bars->w_full[slot]);
          }
        }
        if (!ok) break;
      }
      ring.advance(pair, 2 * walk.stream_pages(0), 2 * walk.stream_pages(1));
    }
  } else {
    setmaxnreg_dec<kRegsControl>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      int g = 0, part = 0;  // pages and parts so far
      int q_loads = 0, v_loads = 0;
      uint32_t k_used = 0, k_odd = 0;  // by slot: loaded, parity of the last load's phase
      Ring ring;
      bool ok = true;
      while (ok && walk.next()) {
        const Tile& t = walk.t;
        const bool pair = walk.pair();
        const int32_t* table = p.block_table + t.b * p.bt_stride + t.page0;
        for (int j0 = walk.p0; ok && j0 < walk.p1; j0 += 32) {
          const int mine = j0 + lane < walk.p1 ? __ldg(table + j0 + lane) : 0;
          const int n = min(32, walk.p1 - j0);
          for (int j = 0; j < n; ++j, ++g) {
            const int page = __shfl_sync(0xffffffffu, mine, j);
            if (lane == 0) {
              const int i = j0 + j - walk.p0;  // within the part
              const uint32_t v = pair ? i : i >> 1;
              const uint32_t slot = Ring::slot(pair, i & 1, v), ph = ring.phase(pair, slot, v);
              const bool there = page >= 0 && page < p.num_pages;
              bars->there[g % kThere] = there ? kIsThere : 0;
              if (!there && p.status) atomicOr(p.status, (unsigned)MSA_STATUS_BAD_BLOCK);
              const int y = there ? (page * p.Hkv + walk.cur_h) * kPage : 0;
              ok = bounded_wait_long(&bars->k_free[slot], ph ^ 1, abort, p.wait_ns);
              if (ok) {
                if (there) {
                  mbar_arrive_expect_tx(&bars->k_full[slot], kTileBytes);
                  tma_load_2d(smem + kOffK + slot * kTileBytes, &kv_map, &bars->k_full[slot], 0, y);
                } else {
                  mbar_arrive(&bars->k_full[slot]);
                }
                k_used |= 1u << slot;
                k_odd = (k_odd & ~(1u << slot)) | (ph << slot);
                ok = bounded_wait_long(&bars->v_free[g % kRawV], ((g / kRawV) & 1) ^ 1, abort,
                                       p.wait_ns);
              }
              if (ok) {
                const int vs = g % kRawV;
                if (there) {
                  mbar_arrive_expect_tx(&bars->v_full[vs], kTileBytes);
                  tma_load_2d(smem + kOffV + vs * kTileBytes, &kv_map, &bars->v_full[vs], kD, y);
                } else {
                  mbar_arrive(&bars->v_full[vs]);
                }
                ++v_loads;
              }
              // Q behind the part's first page (its copy needs no wait for the
              // part before, Q's does)
              if (ok && i == 0) {
                if (part > 0) ok = bounded_wait_long(&bars->q_free, (part - 1) & 1, abort, p.wait_ns);
                if (ok) {
                  const int boxes = pair ? 2 : 1;
                  mbar_arrive_expect_tx(&bars->q_full, (uint32_t)(boxes * p.C * p.G * kD));
                  for (int s = 0; s < boxes; ++s)
                    tma_load_3d(smem + kOffQ + s * kTileBytes, &q_map, &bars->q_full, 0,
                                walk.cur_h * p.G, t.tok0 + s * p.C);
                  ++q_loads;
                }
              }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
          }
        }
        ring.advance(pair, walk.stream_pages(0), walk.stream_pages(1));
        ++part;
      }
      if (lane == 0) {
        if (!ok && !*abort) give_up(bars, p.status);
        // every copy lands before the CTA may end
        for (int i = 0; i < kRawK; ++i)
          if (k_used >> i & 1u)
            bounded_wait_long(&bars->k_full[i], k_odd >> i & 1u, nullptr, kWaitLimitNs);
        for (int i = max(0, v_loads - kRawV); i < v_loads; ++i)
          bounded_wait_long(&bars->v_full[i % kRawV], (i / kRawV) & 1, nullptr, kWaitLimitNs);
        if (q_loads > 0)
          bounded_wait_long(&bars->q_full, (q_loads - 1) & 1, nullptr, kWaitLimitNs);
      }
      __syncwarp();
    } else if (elect_one()) {
      // ------------------------------------------------------- MMA issuers
      // The unit is a half page (64 keys): QK(u) into one of a stream's two S
      // buffers, PV(u) from the P that replaces it, QK(u + 2) when PV(u) is
      // complete, while the softmax works on unit u + 1.  One thread issues
      // the QKs of both streams, and one for each stream its PVs, so that a
      // PV whose P is ready does not wait behind a QK whose buffer is not.
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return bounded_wait_long(bar, parity, abort, p.wait_ns);
      };
      uint32_t part = 0;
      bool ok = true;
      if (warp == 3) {
        constexpr uint32_t kQk = idesc_e4m3_f32(128, kHalf, false);
        const uint64_t desc_k = smem_desc_sw128(smem_u32(smem + kOffK), 16, 1024);
        const uint64_t desc_q = smem_desc_sw128(smem_u32(smem + kOffQ), 16, 1024);
        uint32_t base[2] = {0, 0};  // units of the streams so far
        Ring ring;
        while (ok && walk.next()) {
          const bool pair = walk.pair();
          const uint32_t n[2] = {2u * walk.stream_pages(0), 2u * walk.stream_pages(1)};
          // Q is there when all QKs of the part before are complete
          ok = wait(&bars->q_full, part & 1);
          for (uint32_t i = 0; ok && i < n[0]; ++i) {  // n[0] >= n[1]
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              if (i >= n[s]) continue;
              const uint32_t u = base[s] + i, buf = u & 1, half = i & 1;
              const uint32_t slot = Ring::slot(pair, s, i >> 1);
              ok = (half || wait(&bars->k_full[slot], ring.phase(pair, slot, i >> 1))) &&
                   (u < 2 || wait(&bars->pv_done[s][buf], ((u >> 1) - 1) & 1));
              if (!ok) break;
              tc_fence_after();
              const uint64_t a = desc_q + (pair ? s : 0) * (kTileBytes / 16);
              const uint64_t b = desc_k + slot * (kTileBytes / 16) + half * (kHalf * 128 / 16);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_f8f6f4(tmem + s * 128 + buf * kHalf, a + kk * 2, b + kk * 2, kQk, kk > 0);
              mma_commit(&bars->s_full[s][buf]);
              // (stream 0's QKs of a pair's page are issued before stream 1's)
              if (half && (!pair || s == 1)) mma_commit(&bars->k_free[slot]);
            }
          }
          if (ok) mma_commit(&bars->q_free);
          ring.advance(pair, n[0] / 2, n[1] / 2);
          base[0] += n[0], base[1] += n[1];
          ++part;
        }
      } else {
        constexpr uint32_t kPv = idesc_f16_f32(128, 128, true);
        const int s = warp - 1;
        const uint64_t desc_w = smem_desc_sw128(smem_u32(smem + kOffW), kTileBytes / 2, 1024);
        const uint32_t s_tmem = tmem + s * 128, o_tmem = s_tmem + kColO;
        uint32_t base = 0;  // own units so far
        Ring ring;
        while (ok && walk.next()) {
          const bool pair = walk.pair();
          const uint32_t n0 = 2u * walk.stream_pages(0), n1 = 2u * walk.stream_pages(1);
          const uint32_t n = s ? n1 : n0;
          // the W slots' uses in the part before, of both streams, are over
          if (part > 0) ok = wait(&bars->part_done, (part - 1) & 1);
          for (uint32_t i = 0; ok && i < n; ++i) {
            const uint32_t u = base + i, buf = u & 1;
            const uint32_t slot = Ring::slot(pair, s, i);
            ok = wait(&bars->w_full[slot], ring.phase(pair, slot, i)) &&
                 wait(&bars->p_full[s][buf], (u >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b = desc_w + slot * (kTileBytes / 16);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f16_ts(o_tmem, s_tmem + buf * kHalf + kk * 8, b + kk * (16 * 128 / 16), kPv,
                         kk > 0 || i > 0);
            mma_commit(&bars->pv_done[s][buf]);
            // both streams free a slot; in a solo part its owner for both
            mma_commit(&bars->w_free[slot]);
            if (!pair) mma_commit(&bars->w_free[slot]);
          }
          if (ok) mma_commit(&bars->part_done);
          ring.advance(pair, n0, n1);
          base += n;
          ++part;
        }
      }
      if (!ok && !*abort) give_up(bars, p.status);
      mma_commit(&bars->mma_done[warp - 1]);
      bounded_wait_long(&bars->mma_done[warp - 1], 0, nullptr, kWaitLimitNs);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ----------------------------------------------------------------- combine

constexpr int kCombineWarps = 8;
constexpr int kMaxParts = 192;  // parts of a tile: one a CTA

struct CombineParams {
  const PlanHead* head;
  const Tile* own;  // the own tiles
  int T, Hq, Hkv, G, C, ctas, prefix;
  int rows;  // rows of a tile that a CTA takes
  const float* part_o;
  const float* part_lse;
  float v_scale;
  uint16_t* out;
  float* lse;
};

// A CTA takes some rows of a tile of a request's own pages (blockIdx.x) of a
// KV head (.y): first the parts of that tile and of the shared tiles (two at
// most) that its tokens lie in are listed, then each warp merges the parts of
// four neighbouring rows, 8 lanes a row, or kTeam warps together: weights
// 2^(lse - m), fp32 sums, eight or more 16-byte loads in flight per lane.  A
// batch that was refused gives empty rows.
template <int kTeam>
__global__ void __launch_bounds__(kCombineWarps * 32) combine_kernel(const CombineParams p) {
  // per listed tile: its parts' first rows (of the tile's first token and
  // head), in line order
  __shared__ int s_row[3][kMaxParts];
  __shared__ int s_n[3];
  __shared__ Tile s_tile[3];
  constexpr int kLanes = 8;
  constexpr int kQ = 32 / kLanes;             // float4 of a row per lane
  constexpr int kFlight = kTeam == 8 ? 8 : 2;  // parts in flight
  __shared__ __align__(16) float s_acc[kTeam > 1 ? kCombineWarps * 4 : 1][kD];  // (as float4)
  __shared__ float s_m[kCombineWarps * 4], s_l[kCombineWarps * 4];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y;
  const PlanHead hd = *p.head;
  const Tile own = p.own[blockIdx.x];
  if (hd.bad) {  // every row empty
    const int64_t n = (int64_t)p.T * p.G * (kD / 8);
    const int64_t step = (int64_t)gridDim.x * gridDim.z * blockDim.x;
    for (int64_t e = ((int64_t)blockIdx.z * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x;
         e < n; e += step) {
      const int64_t r = e / (kD / 8);
      const int64_t row = r / p.G * p.Hq + h * p.G + r % p.G;
      // 8-byte stores: out need not be aligned to more
      uint2* dst = reinterpret_cast<uint2*>(p.out + row * kD) + 2 * (e % (kD / 8));
      dst[0] = dst[1] = make_uint2(0u, 0u);
      if (p.lse && e % (kD / 8) == 0) p.lse[row] = -INFINITY;
    }
    return;
  }
  const int tile = hd.shared_tiles + blockIdx.x;
  if (tile >= hd.ntiles) return;
  const int row0 = blockIdx.z * p.rows, rows = min(p.rows, own.ntok * p.G - row0);
  if (rows <= 0) return;
  if (warp < 3) {  // warp 0: the own tile, 1 and 2: the shared ones
    const int first = own.tok0 / (2 * p.C), last = (own.tok0 + own.ntok - 1) / (2 * p.C);
    const int ti = warp == 0 ? tile : first + warp - 1;
    int n = 0;
    if (warp == 0 || (hd.shared_tiles > 0 && ti <= last)) {
      Tile t = own;
      if (warp > 0) {  // a shared tile: all of one size but the last
        t.tok0 = ti * 2 * p.C;
        t.ntok = min(2 * p.C, hd.T - t.tok0);
        t.npages = p.prefix;
        t.start = (uint32_t)ti * tile_cost(2 * p.C, p.prefix, p.C);
      }
      const int rate = tile_rate(t.ntok, p.C);
      const int64_t share = share_of((int64_t)hd.cost * p.Hkv, p.ctas);
      const int64_t t0 = (int64_t)h * hd.cost + t.start;
      const int64_t t1 = t0 + tile_cost(t.ntok, t.npages, p.C);
      // (64-bit divisions are slow; costs rarely need them)
      const bool small = t1 <= INT_MAX && share <= INT_MAX;
      const int i0 = small ? (int)t0 / (int)share : (int)(t0 / share);
      const int i1 = small ? (int)(t1 - 1) / (int)share : (int)((t1 - 1) / share);
      for (int c0 = i0; c0 <= i1; c0 += 32) {
        const int cta = c0 + lane;
        int pa = 0, pb = 0;
        if (cta <= i1) {
          pa = pages_before(max(cta * share, t0) - t0, t.npages, rate);
          pb = pages_before(min((cta + 1) * share, t1) - t0, t.npages, rate);
        }
        const uint32_t some = __ballot_sync(0xffffffffu, pb > pa);
        if (pb > pa) {
          const int at = n + __popc(some & ((1u << lane) - 1u));
          if (at < kMaxParts)
            s_row[warp][at] = (int)part_row(cta, h, ti, hd.shared_tiles, t.tok0, p.T, p.G);
        }
        n += __popc(some);
      }
      if (lane == 0) s_tile[warp] = t;
    }
    if (lane == 0) s_n[warp] = min(n, kMaxParts);
  }
  __syncthreads();
  const int sub = lane % kLanes, in_warp = lane / kLanes;
  const uint32_t peers = 0xFFu << (lane - sub);
  const int member = warp % kTeam, slot = warp / kTeam * 4 + in_warp;
  constexpr int kRows = kCombineWarps / kTeam * 4;  // rows at a time
  for (int r0 = 0; r0 < rows; r0 += kRows) {
    const int r = row0 + r0 + slot;
    const bool live = r0 + slot < rows;
    const int tok = own.tok0 + (live ? r / p.G : 0);
    float m = -INFINITY, l = 0.f;
    // lane `sub` has columns 4 (kLanes q + sub) .. + 3 of the row
    float4 acc[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
      for (int k = 0; k < 3; ++k) {
        const int n = s_n[k];
        if (n == 0) continue;
        const int o = tok - s_tile[k].tok0;  // the token within the listed tile
        if (o < 0 || o >= s_tile[k].ntok) continue;
        // rows of a pair: C tokens of the first stream, then the second's:
        // the same as token order
        const int off = o * p.G + r % p.G;
        const RowPlace place = row_place(off, s_tile[k].ntok, p.C, p.G);
        const float* col = p.part_o + place.first + (sub >> 1) * place.chunk + (sub & 1) * 4;
        // a member's parts are every kTeam-th, 8 of them a round
        for (int e0 = member; e0 < n; e0 += kTeam * kLanes) {
          const int e = e0 + kTeam * sub;
          int row = e < n ? s_row[k][e] : 0;
          const float le = e < n ? __ldcg(p.part_lse + row + off) : -INFINITY;
          // only a part without keys is left out: one whose weight underflows
          // may hold a NaN
          if (le == -INFINITY) row = -1;
          float top = le;
#pragma unroll
          for (int d = kLanes / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(peers, top, d));
          if (top > m) {
            const float f = m == -INFINITY ? 0.f : exp2f(m - top);
            l *= f;
#pragma unroll
            for (int q = 0; q < kQ; ++q) acc[q].x *= f, acc[q].y *= f, acc[q].z *= f, acc[q].w *= f;
            m = top;
          }
          // NaN (a NaN score) stays one
          const float w = le == -INFINITY ? 0.f : exp2f(le - (m == -INFINITY ? 0.f : m));
          const int count = min(kLanes, (n - e0 + kTeam - 1) / kTeam);
          for (int j = 0; j < count; j += kFlight) {
            float4 v[kFlight][kQ];
            float wj[kFlight];
#pragma unroll
            for (int d = 0; d < kFlight; ++d) {
              wj[d] = __shfl_sync(peers, w, j + d, kLanes);
              const int rj = __shfl_sync(peers, row, j + d, kLanes);
              const float* src = col + (int64_t)rj * kD;
#pragma unroll
              for (int q = 0; q < kQ; ++q)
                v[d][q] = rj >= 0
                              ? __ldcg(reinterpret_cast<const float4*>(src + 4 * q * place.chunk))
                              : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int d = 0; d < kFlight; ++d) {
              l += wj[d];
#pragma unroll
              for (int q = 0; q < kQ; ++q) {
                acc[q].x = fmaf(wj[d], v[d][q].x, acc[q].x);
                acc[q].y = fmaf(wj[d], v[d][q].y, acc[q].y);
                acc[q].z = fmaf(wj[d], v[d][q].z, acc[q].z);
                acc[q].w = fmaf(wj[d], v[d][q].w, acc[q].w);
              }
            }
          }
        }
      }
    }
    if constexpr (kTeam > 1) {
      const int mine = slot * kTeam + member;
      if (sub == 0) s_m[mine] = m, s_l[mine] = l;
#pragma unroll
      for (int q = 0; q < kQ; ++q)
        *reinterpret_cast<float4*>(&s_acc[mine][4 * (q * kLanes + sub)]) = acc[q];
      __syncthreads();
      if (member == 0 && live) {
        float top = -INFINITY;
        for (int k = 0; k < kTeam; ++k) top = fmaxf(top, s_m[mine + k]);
        l = 0.f;
#pragma unroll
        for (int q = 0; q < kQ; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < kTeam; ++k) {
          const float lk = s_l[mine + k];
          // a member without parts has l = 0; one with a NaN keeps it
          const float f = lk == 0.f ? 0.f
                          : lk == lk ? exp2f(s_m[mine + k] - (top == -INFINITY ? 0.f : top))
                                     : lk;
          l += f * lk;
#pragma unroll
          for (int q = 0; q < kQ; ++q) {
            const float4 v = *reinterpret_cast<const float4*>(&s_acc[mine + k][4 * (q * kLanes + sub)]);
            acc[q].x = fmaf(f, v.x, acc[q].x);
            acc[q].y = fmaf(f, v.y, acc[q].y);
            acc[q].z = fmaf(f, v.z, acc[q].z);
            acc[q].w = fmaf(f, v.w, acc[q].w);
          }
        }
        m = top;
      }
    }
    if (member == 0 && live) {
      const float scale = l == 0.f ? 0.f : p.v_scale / l;
      const int64_t row = (int64_t)tok * p.Hq + h * p.G + r % p.G;
#pragma unroll
      for (int q = 0; q < kQ; ++q)
        *reinterpret_cast<uint2*>(p.out + row * kD + 4 * (q * kLanes + sub)) =
            make_uint2(pack_bf16x2(acc[q].x * scale, acc[q].y * scale),
                       pack_bf16x2(acc[q].z * scale, acc[q].w * scale));
      if (p.lse && sub == 0)
        p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
    }
    if constexpr (kTeam > 1) __syncthreads();
  }
}

// -------------------------------------------------------------------- host

struct Layout {
  size_t head, tiles, req_tile, part_o, part_lse, total;
};

bool layout(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t prefix, int64_t max_k, int ctas,
            Layout* l) {
  const int64_t G = Hq / Hkv, C = kTileM / G;
  const int64_t tiles = max_tiles(B, T, C, prefix);
  // the cost of a head's tiles, that of a CTA's range and the rows of the
  // partials in range of their integers (64-bit places cost the attention
  // kernel 1 to 7 %, by its registers).  A machine without a GPU, where sizes
  // are asked too, counts as one SM.
  const double cost = (double)tiles * (double)(ceil_div(max_k, kPage) * kCostPair + kCostTile);
  if (cost > (double)UINT32_MAX || cost * (double)Hkv > (double)INT_MAX * (ctas > 1 ? ctas : 152))
    return false;
  const int64_t rows = 256 * ((int64_t)ctas + 1) + Hkv * (prefix > 0 ? 2 : 1) * T * G;
  if (rows >= INT_MAX || ctas > kMaxParts) return false;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  l->head = 0;
  l->tiles = 256;
  l->req_tile = l->tiles + up((size_t)tiles * sizeof(Tile));
  l->part_lse = l->req_tile + up((size_t)(B + 1) * sizeof(int32_t));
  l->part_o = l->part_lse + up((size_t)rows * sizeof(float));
  l->total = l->part_o + (size_t)rows * kD * sizeof(float);
  return true;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::atomic<EncodeTiledFn> fn{nullptr};
  EncodeTiledFn f = fn.load();
  if (!f) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn.store(f = reinterpret_cast<EncodeTiledFn>(ptr));
  }
  return f;
}

bool encode(EncodeTiledFn enc, CUtensorMap* map, const void* base, int dims, const cuuint64_t* size,
            const cuuint64_t* stride, const cuuint32_t* box) {
  const cuuint32_t one[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, const_cast<void*>(base), size, stride, box,
             one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t prefix_workspace(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t prefix_pages,
                        int64_t max_k) {
  Layout l;
  return layout(B, T, Hq, Hkv, prefix_pages, max_k, num_sms(), &l) ? l.total : 0;
}

cudaError_t launch_prefix_attention(const PrefixArgs& a, void* ws, cudaStream_t stream) {
  const int ctas = num_sms();
  const int G = (int)(a.Hq / a.Hkv), C = kTileM / G;
  Layout l;
  if (!layout(a.B, a.T, a.Hq, a.Hkv, a.prefix_pages, a.max_k, ctas, &l)) return cudaErrorInvalidValue;
  EncodeTiledFn enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  CUtensorMap kv_map, q_map;
  const cuuint64_t kv_size[2] = {2 * kD, (cuuint64_t)(std::max<int64_t>(a.num_pages, 1) * a.Hkv * kPage)};
  const cuuint64_t kv_stride[1] = {2 * kD};
  const cuuint32_t kv_box[2] = {kD, kPage};
  const cuuint64_t q_size[3] = {kD, (cuuint64_t)a.Hq, (cuuint64_t)a.T};
  const cuuint64_t q_stride[2] = {kD, (cuuint64_t)(a.Hq * kD)};
  const cuuint32_t q_box[3] = {kD, (cuuint32_t)G, (cuuint32_t)C};
  if (!encode(enc, &kv_map, a.kv, 2, kv_size, kv_stride, kv_box) ||
      !encode(enc, &q_map, a.q, 3, q_size, q_stride, q_box))
    return cudaErrorInvalidValue;
  char* base = static_cast<char*>(ws);
  PlanHead* head = reinterpret_cast<PlanHead*>(base + l.head);
  Tile* tiles = reinterpret_cast<Tile*>(base + l.tiles);
  int32_t* req_tile = reinterpret_cast<int32_t*>(base + l.req_tile);
  float* part_lse = reinterpret_cast<float*>(base + l.part_lse);
  float* part_o = reinterpret_cast<float*>(base + l.part_o);

  const int own0 = (int)own_base(a.T, C, a.prefix_pages);
  const PlanParams pp = {a.cu_q, a.cu_k, (int)a.B, (int)a.T, C, (int)a.prefix_pages, a.max_q,
                         a.max_k, head, tiles, own0, req_tile, a.status};
  cudaError_t e;
  // where the CTA's threads list all tiles in one round the plan is made in
  // the attention kernel's prologue: a launch less (16 requests over 32k keys:
  // 24.6 us, with a kernel for the plan 25.8; five chunks of 1 .. 700 tokens:
  // 111 and 127)
  const bool plan_here =
      a.B <= kThreads && max_tiles(a.B, a.T, C, a.prefix_pages) <= kThreads;
  if (!plan_here) {
    e = launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, pp);
    if (e != cudaSuccess) return e;
  }

  constexpr int kMaxDevices = 64;
  static std::atomic<bool> attr_set[kMaxDevices];
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) attr_set[dev].store(true, std::memory_order_release);
  }
  const AttendParams ap = {pp, plan_here, tiles, own0, a.block_table, a.bt_stride, a.kv, (int)a.num_pages,
                           (int)a.T, G, C, (int)a.Hkv, a.score_log2, part_o, part_lse, a.status,
                           (uint32_t)std::min<uint64_t>(pipeline_wait_limit_ns(), kWaitLimitNs)};
  e = launch_pdl(attend_kernel, dim3((unsigned)ctas), dim3(kThreads), (size_t)kSmem, stream, kv_map,
                 q_map, ap);
  if (e != cudaSuccess) return e;

  // Warps that share four rows in the combine, by about how many parts a row
  // has and how many rows there are.  Many parts of few rows: 8 (76 parts of
  // 256 rows: 22.0 us in all, with two warps 27.1, with one 40.9).  Some parts
  // of more rows: 2 (4 parts of 2048 rows: 128.1, with 8 warps 130.5, with one
  // 134.0).  Two parts of 25 thousand rows: 1 (105, with two warps 168).
  const int64_t tile_rows = std::min<int64_t>(2 * C, a.max_q) * G;
  const int64_t tiles_n =
      a.prefix_pages > 0 ? ceil_div(a.T, 2 * C) : std::min(a.T, ceil_div(a.T, 2 * C) + a.B);
  const int64_t parts = (int64_t)ctas / (a.Hkv * tiles_n);  // of a row, about
  const int64_t all_rows = a.T * a.Hq;
  const int team = parts >= 24 && all_rows <= 4096 ? 8 : parts >= 3 && all_rows <= 16384 ? 2 : 1;
  const int cta_rows = kCombineWarps / team * 4;
  const CombineParams cp = {head, tiles + own0, (int)a.T, (int)a.Hq, (int)a.Hkv, G, C, ctas,
                            (int)a.prefix_pages, cta_rows, part_o, part_lse, a.v_scale, a.out, a.lse};
  const int64_t own = std::min<int64_t>(a.T, ceil_div(a.T, 2 * C) + a.B);
  const dim3 grid((unsigned)own, (unsigned)a.Hkv, (unsigned)std::max<int64_t>(1, ceil_div(tile_rows, cta_rows)));
  const dim3 block(kCombineWarps * 32);
  if (team == 8) return launch_pdl(combine_kernel<8>, grid, block, 0, stream, cp);
  if (team == 2) return launch_pdl(combine_kernel<2>, grid, block, 0, stream, cp);
  return launch_pdl(combine_kernel<1>, grid, block, 0, stream, cp);
}

}  // namespace msa
