// Verification of drafted tokens against the target model's probabilities,
// from given random numbers (the step after msa_decode's speculative verify).
//
// With p_i the target's and q_i the draft's probabilities at draft i, x_i the
// drafted token and u_i a uniform number in [0, 1): draft i stands iff every
// draft before it stands and u_i q_i(x_i) < p_i(x_i); this product is taken
// in 64 bits, where it is exact.  At the first draft that falls the next
// token is drawn from max(p - q, 0), after the last draft from p, by the
// inverse of the distribution function: the lowest v whose cumulated weight
// exceeds u_{n-1} times the total.
//
// The weights are whole numbers of steps of 2^-44: floor(2^44 min(max(p - q,
// 0), 1)) with p - q rounded to fp32.  Their sums in 64-bit integers are
// exact (V < 2^19, so they stay below 2^63), so any split of the row gives
// the same token, and fp64 arithmetic, which this GPU has little of, is not
// needed.  A step of 2^-44 is far below the 2^-24 of a uniform fp32 number.
//
// One cluster of 8 CTAs per request, one launch: only the row that is drawn
// from is read (of p and of q), each CTA one eighth of it.  The CTAs'
// totals meet in distributed shared memory; the CTA, then the warp, that
// holds the threshold reads its own few hundred weights once more (from L2)
// to place it.  Bound: HBM for large batches, else the latency of the
// dependent steps (gather, row, cluster barrier, placing).
// Measured (GPU time, replayed from a graph): 64 requests, 200003 fp32 values
// a row 24.8 us, 102 MB at 4.1 TB/s, and 200000 (rows on 16 bytes) 21.3; one
// request of 32000 4.3 us.  64 registers a thread, four CTAs an SM; the odd
// rows' kernels spill 28 bytes.
//
// Greedy: draft i stands iff it is the first of the largest values of its
// row.  The same cluster scans the request's rows in order, each CTA its
// eighth, each warp by itself; a warp that has seen a draft beaten tells all
// CTAs (a minimum in their shared memory, no barrier), and rows behind it
// are left out: they cannot matter.
// Measured: 64 requests of 8 rows of 131072 bf16 values, three drafts of ten
// fall: 23.4 us.  The rows up to each request's first fallen draft are 51 MB
// (7.5 us at a copy's rate); 61 of 134 MB are read, at 2.6 TB/s: the requests
// whose drafts stand long are read row after row by their 8 CTAs, with too few
// bytes in flight for the SMs that are left.
#include <algorithm>
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <utility>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kCluster = 8;
constexpr int kVThreads = 256;
constexpr int kVWarps = kVThreads / 32;
constexpr int kMaxVerify = 32;  // rows of one request

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// N consecutive elements as they lie in memory (16 bytes, or one element).
template <typename T, int N>
struct Raw {
  static constexpr bool kVec = N * sizeof(T) == 16;
  uint32_t w[kVec ? 4 : 1];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kVec) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (sizeof(T) == 4) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
      w[0] = __ldg(reinterpret_cast<const uint16_t*>(p));
    }
  }
  __device__ __forceinline__ void fill(uint32_t bits) {
#pragma unroll
    for (int i = 0; i < (kVec ? 4 : 1); ++i) w[i] = bits;
  }
  // the elements from v on that lie before hi; the others' bits are `rest`
  // (a word of two equal elements for the 2-byte types)
  __device__ __forceinline__ void load_to(const T* row, int v, int hi, uint32_t rest) {
    if (v + N <= hi) {
      load(row + v);
    } else {
      fill(rest);
      if constexpr (kVec) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (v + i < hi) {
            if constexpr (sizeof(T) == 4) {
              w[i] = __ldg(reinterpret_cast<const uint32_t*>(row + v + i));
            } else {
              const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(row + v + i));
              w[i >> 1] = i & 1 ? (w[i >> 1] & 0xFFFFu) | (h << 16) : (w[i >> 1] & 0xFFFF0000u) | h;
            }
          }
        }
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[i]);
    } else {
      const uint16_t h = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
      return to_f32(*reinterpret_cast<const T*>(&h));
    }
  }
};

// The weight of a token in steps of 2^-44 (NaN and negative values: 0), as
// its upper and lower 22 bits plus the constant kMagic each.  A sum that is
// rounded towards zero onto 2^23 has its whole part in the last 23 bits:
// w 2^22 is split without the slow conversions to integers (and what is left
// of it is exact).
constexpr uint32_t kMagic = 0x4B000000u;  // the bits of 2^23
__device__ __forceinline__ void weight_parts(float p, float q, uint32_t& hi, uint32_t& lo) {
  const float w = __saturatef(p - q);
  const float t = __fmaf_rz(w, 4194304.f, 8388608.f);
  const float rest = fmaf(w, 4194304.f, 8388608.f - t);
  hi = __float_as_uint(t);
  lo = __float_as_uint(__fmaf_rz(rest, 4194304.f, 8388608.f));
}
__device__ __forceinline__ uint64_t weight(float p, float q) {
  uint32_t hi, lo;
  weight_parts(p, q, hi, lo);
  return ((uint64_t)(hi - kMagic) << 22) + (lo - kMagic);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// floor(u * total), exactly: u is a whole number of at most 24 bits times a
// power of two, and total is below 2^63.  In [0, total) for total > 0; 0 for
// NaN and for u <= 0, and for u >= 1, which is no uniform, that of the largest
// 31-bit number below 1.
__device__ __forceinline__ uint64_t threshold(float u, uint64_t total) {
  if (!(u > 0.f)) return 0;
  const uint32_t bits = __float_as_uint(u);
  const int e = max(1, (int)(bits >> 23));  // u = k 2^(e - 150)
  uint64_t k = (bits & 0x7FFFFFu) | (bits >> 23 ? 0x800000u : 0u);
  int shift = 150 - e;  // 24 .. 149
  if (u >= 1.f) k = 0x7FFFFFFFu, shift = 31;
  const uint64_t hi = __umul64hi(k, total), lo = k * total;
  return shift < 64 ? (hi << (64 - shift)) | (lo >> shift) : shift < 128 ? hi >> (shift - 64) : 0;
}

// N consecutive weights a lane: 32 * N a warp step.  A warp takes kBatch steps
// at a time, and the next kBatch are loaded before these are used.  Their sums
// are kept, so that the threshold is placed by reading one batch again.
template <typename T, int N>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kVThreads, 4)
verify_kernel(const VerifyArgs a, int seg) {
  constexpr int kBatch = N == 1 ? 8 : 2;
  constexpr int kSpan = kBatch * 32 * N;  // elements of a batch
  // batches of a warp: V < 2^19 over the cluster's warps
  constexpr int kMaxBatches = MSA_VERIFY_MAX_VOCAB / (kCluster * kVWarps * kSpan) + 2;
  __shared__ uint64_t batch_tot[kVWarps][kMaxBatches];
  __shared__ uint64_t warp_tot[kVWarps];
  __shared__ uint64_t cta_tot[kCluster];
  __shared__ int s_acc;
  __shared__ int s_used;
  cg::cluster_group cluster = cg::this_cluster();
  // A CTA's shared memory may be written from outside only once the CTA has
  // started: each says so here, and all are waited for just before the totals
  // are exchanged, by when that costs nothing.
  auto started = cluster.barrier_arrive();
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cluster.block_rank();
  const int64_t b = blockIdx.x / kCluster;
  const int n = a.n, V = (int)a.V;
  const T* target = static_cast<const T*>(a.target) + b * a.t_req;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + b * a.d_req : nullptr;
  const float u = __ldg(a.u + b * n + n - 1);

  // which drafts stand: lane i decides draft i (every CTA for itself)
  const int drafts = a.counts ? min(max(__ldg(a.counts + b), 0), n - 1) : n - 1;
  if (warp == 0) {
    bool ok = false;
    int x = -1;
    if (lane < n - 1) {
      // a draft behind this request's last changes nothing, and its token
      // need not be waited for
      x = __ldg(a.tokens_in + b * (n - 1) + lane);
      if (x >= 0 && x < V) {
        const double p = to_f32(target[lane * a.t_row + x]);
        const double q = draft ? (double)to_f32(draft[lane * a.d_row + x]) : 1.0;
        ok = lane < drafts && (double)__ldg(a.u + b * n + lane) * q < p;
      }
    }
    const uint32_t fell = ~__ballot_sync(0xffffffffu, ok);
    const int acc = fell ? __ffs(fell) - 1 : 32;
    const int used = __shfl_sync(0xffffffffu, x, acc & 31);
    if (lane == 0) {
      s_acc = min(acc, drafts);
      s_used = acc < drafts && used < V ? max(used, -1) : -1;  // -1: not a token
    }
    if (rank == 0) {  // the drafts that stand, and -1 behind the next token
      if (lane < n && lane != min(acc, drafts))
        a.tokens[b * n + lane] = lane < acc ? x : -1;
    }
  }
  __syncthreads();
  const int acc = s_acc;
  const bool refused = acc < drafts;
  const T* prow = target + acc * a.t_row;
  const T* qrow = refused && draft ? draft + acc * a.d_row : nullptr;
  // a certain draft (no draft probabilities) that fell is left out
  int skip = refused && !draft ? s_used : -1;

  // this CTA's part of the row, cut among its warps in whole batches
  const int lo = min(V, rank * seg), hi = min(V, lo + seg);
  const int batches = ((hi - lo + kSpan - 1) / kSpan + kVWarps - 1) / kVWarps;
  const int wlo = min(hi, lo + warp * batches * kSpan);
  const int whi = min(hi, wlo + batches * kSpan);

  for (int pass = 0; pass < 2; ++pass) {
    // pass 1 only where p <= q everywhere and yet a draft fell (distributions
    // that do not add up to one): the token is drawn from p itself
    const T* q = pass == 0 ? qrow : nullptr;
    if (pass == 1) skip = -1;
    uint64_t sum = 0;
    Raw<T, N> rp[2][kBatch], rq[2][kBatch];
    auto load = [&](int buf, int v0) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) rp[buf][k].load_to(prow, v0 + (k * 32 + lane) * N, whi, 0u);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (q) rq[buf][k].load_to(q, v0 + (k * 32 + lane) * N, whi, 0u); else rq[buf][k].fill(0u);
    };
    auto add = [&](int buf, int v0, int i) {
      // at most 16 weights: their parts' sums stay in 32 bits
      uint32_t h = 0u - kBatch * N * kMagic, l = h;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          uint32_t x, y;
          weight_parts(rp[buf][k].at(e), rq[buf][k].at(e), x, y);
          h += x, l += y;
        }
      uint64_t own = ((uint64_t)h << 22) + l;
      const int o = skip - v0 - lane * N;  // the token left out, from this lane's first
      if (o >= 0 && o < kSpan && o % (32 * N) < N && skip < whi) own -= weight(to_f32(prow[skip]), 0.f);
      own = warp_sum(own);
      if (lane == 0) batch_tot[warp][i] = own;
      sum += own;
    };
    if (wlo < whi) load(0, wlo);
    for (int i = 0, v0 = wlo; v0 < whi; i += 2, v0 += 2 * kSpan) {
      if (v0 + kSpan < whi) load(1, v0 + kSpan);
      add(0, v0, i);
      if (v0 + kSpan < whi) {
        if (v0 + 2 * kSpan < whi) load(0, v0 + 2 * kSpan);
        add(1, v0 + kSpan, i + 1);
      }
    }
    if (lane == 0) warp_tot[warp] = sum;
    __syncthreads();
    if (pass == 0) cluster.barrier_wait(std::move(started));
    if (threadIdx.x < kCluster) {
      uint64_t t = 0;
#pragma unroll
      for (int i = 0; i < kVWarps; ++i) t += warp_tot[i];
      *cluster.map_shared_rank(&cta_tot[rank], threadIdx.x) = t;
    }
    cluster.sync();
    // only now has every CTA read the request's number of drafts, which
    // `accepted` may replace
    if (pass == 0 && rank == 0 && threadIdx.x == 0) a.accepted[b] = s_acc;
    uint64_t total = 0, before = 0;
#pragma unroll
    for (int i = 0; i < kCluster; ++i) {
      if (i < rank) before += cta_tot[i];
      total += cta_tot[i];
    }
    if (total == 0) {
      if (pass == 0) {
        cluster.sync();  // the totals are read before they are written again
        continue;
      }
      if (rank == 0 && threadIdx.x == 0) a.tokens[b * n + s_acc] = -1;  // no probability at all
      return;
    }
    uint64_t t = threshold(u, total);
    if (t < before || t - before >= cta_tot[rank]) return;  // another CTA's
    t -= before;
    for (int i = 0; i < warp; ++i) {
      if (t < warp_tot[i]) return;  // an earlier warp's
      t -= warp_tot[i];
    }
    if (t >= warp_tot[warp]) return;
    // this warp's: the batch that passes the threshold once more, its steps'
    // sums, then the step that does
    int i = 0;
    while (t >= batch_tot[warp][i]) t -= batch_tot[warp][i++];
    const int v0 = wlo + i * kSpan;
    load(0, v0);
    for (int k = 0; k < kBatch; ++k) {
      uint64_t w[N], own = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (j == k) x = rp[0][j].at(e), y = rq[0][j].at(e);
        w[e] = v0 + (k * 32 + lane) * N + e == skip ? 0 : weight(x, y);
        own += w[e];
      }
      uint64_t incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, incl > t);
      if (past) {
        if (lane == __ffs(past) - 1) {
          uint64_t sofar = incl - own;
          int e = 0;
          while (e < N - 1 && sofar + w[e] <= t) sofar += w[e++];
          a.tokens[b * n + s_acc] = v0 + (k * 32 + lane) * N + e;
        }
        return;
      }
      t -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return;
  }
}

// A value and its place as one integer whose order is that of the value, and
// among equal values (+0 and -0 are equal) that of the lower place.
__device__ __forceinline__ uint64_t best_key(float x, uint32_t place) {
  uint32_t f = __float_as_uint(x == 0.f ? 0.f : x);
  f = (f >> 31) ? ~f : f | 0x80000000u;
  return ((uint64_t)f << 32) | (0xFFFFFFFFu - place);
}

template <typename T, int N>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kVThreads, 4)
greedy_kernel(const VerifyArgs a, int seg) {
  constexpr int kBatch = N == 1 ? 16 : 4;
  constexpr int kSpan = kBatch * 32 * N;
  __shared__ uint64_t warp_best[kMaxVerify][kVWarps];
  __shared__ uint64_t draft_key[kMaxVerify];
  __shared__ uint64_t cta_best[kCluster];  // rank 0's is complete
  __shared__ int beaten;  // a row known to end the accepted drafts
  cg::cluster_group cluster = cg::this_cluster();
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cluster.block_rank();
  const int64_t b = blockIdx.x / kCluster;
  const int n = a.n, V = (int)a.V;
  const T* target = static_cast<const T*>(a.target) + b * a.t_req;
  const int drafts = a.counts ? min(max(__ldg(a.counts + b), 0), n - 1) : n - 1;
  // this CTA's part of every row, cut among its warps in whole batches
  const int lo = min(V, rank * seg), hi = min(V, lo + seg);
  const int batches = max(1, ((hi - lo + kSpan - 1) / kSpan + kVWarps - 1) / kVWarps);
  const int wlo = min(hi, lo + warp * batches * kSpan);
  const int whi = min(hi, wlo + batches * kSpan);
  // batch j of this warp: of row j / batches; a place past the part is NaN,
  // which is never the best
  Raw<T, N> r[2][kBatch];
  const uint32_t nan = sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
  auto load = [&](int buf, int row, int part) {
    const T* p = target + row * a.t_row;
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      r[buf][k].load_to(p, wlo + part * kSpan + (k * 32 + lane) * N, whi, nan);
  };
  load(0, 0, 0);
  if (warp == 0) {
    // the keys to beat; 0, which any value beats, for what is no token or NaN
    uint64_t key = ~0ull;
    if (lane < n - 1) {
      const int x = __ldg(a.tokens_in + b * (n - 1) + lane);
      const float mine = x >= 0 && x < V ? to_f32(target[lane * a.t_row + x]) : NAN;
      key = mine == mine ? best_key(mine, (uint32_t)x) : 0;
    }
    // the first draft that cannot stand, or the end of them
    const uint32_t bad = __ballot_sync(0xffffffffu, lane < drafts && key == 0);
    draft_key[lane] = key;
    if (lane == 0) beaten = bad ? __ffs(bad) - 1 : drafts;
  }
  cluster.sync();  // every CTA's `beaten` is set before another lowers it

  // The rows in order, each warp by itself, the next batch (of this row or
  // the next) in flight while one is looked through.  A warp that sees a
  // draft beaten lowers every CTA's `beaten`; rows behind that one are not
  // looked through.
  float best = -INFINITY;
  uint32_t place = 0xFFFFFFFFu;
  int row = 0, part = 0;
  auto look = [&](int buf) {  // false: done
    if (part == 0) {
      if (row > __shfl_sync(0xffffffffu, *(volatile int*)&beaten, 0)) return false;
      best = -INFINITY, place = 0xFFFFFFFFu;
    }
    const bool last = part + 1 == batches;
    const int next_row = last ? row + 1 : row, next_part = last ? 0 : part + 1;
    if (next_row <= drafts) load(buf ^ 1, next_row, next_part);
    // a thread's places ascend, so the first of equal values stays
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float x = r[buf][k].at(e);
        if (x > best || (x == best && place == 0xFFFFFFFFu))
          best = x, place = (uint32_t)(wlo + part * kSpan + (k * 32 + lane) * N + e);
      }
    if (last) {
      uint64_t key = place == 0xFFFFFFFFu ? 0 : best_key(best, place);  // 0: nothing but NaN
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
        key = other > key ? other : key;
      }
      if (lane == 0) warp_best[row][warp] = key;
      if (row < drafts && key > draft_key[row] && lane < kCluster)
        atomicMin(cluster.map_shared_rank(&beaten, lane), row);
    }
    row = next_row, part = next_part;
    return row <= drafts;
  };
  while (look(0) && look(1)) {
  }
  cluster.sync();
  // every warp has scanned row `beaten`, and no draft before it is beaten:
  // that row's best is the next token
  const int acc = beaten;
  if (warp == 0) {
    uint64_t key = lane < kVWarps ? warp_best[acc][lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
      key = other > key ? other : key;
    }
    if (lane == 0) *cluster.map_shared_rank(&cta_best[rank], 0) = key;
  }
  cluster.sync();
  if (rank != 0 || warp != 0) return;
  uint64_t key = 0;
  for (int c = 0; c < kCluster; ++c) key = cta_best[c] > key ? cta_best[c] : key;
  const int next = key ? (int)(0xFFFFFFFFu - (uint32_t)key) : -1;
  if (lane < n)
    a.tokens[b * n + lane] =
        lane < acc ? __ldg(a.tokens_in + b * (n - 1) + lane) : lane == acc ? next : -1;
  if (lane == 0) a.accepted[b] = acc;
}

template <typename T>
bool vector_rows(const void* p, int64_t req, int64_t row) {
  constexpr int64_t n = 16 / sizeof(T);
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && req % n == 0 && row % n == 0;
}

template <typename T>
cudaError_t launch_verify_type(const VerifyArgs& a, bool greedy, cudaStream_t stream) {
  constexpr int N = 16 / sizeof(T);
  // 16-byte loads where every row starts on 16 bytes; else one value a load
  // (an odd vocabulary's rows start anywhere).  Greedy, 64 x 8 bf16 rows of
  // 131072: 25 us, by single values 48; 64 rows of 200000 fp32 drawn from:
  // 21.3 us and 25.2, one row of 32000 4.3 either way
  const bool vec = vector_rows<T>(a.target, a.t_req, a.t_row) &&
                   (greedy || !a.draft || vector_rows<T>(a.draft, a.d_req, a.d_row));
  const int seg = (int)(ceil_div(ceil_div(a.V, kCluster), 32 * N) * (32 * N));
  const dim3 grid((unsigned)(a.B * kCluster));
  auto run = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(kVThreads), 0, stream, a, seg);
  };
  if (greedy) return vec ? run(greedy_kernel<T, N>) : run(greedy_kernel<T, 1>);
  return vec ? run(verify_kernel<T, N>) : run(verify_kernel<T, 1>);
}

cudaError_t launch_any(const VerifyArgs& a, bool greedy, cudaStream_t stream) {
  if (a.B <= 0) return cudaSuccess;
  switch (a.dtype) {
    case MSA_DTYPE_F32: return launch_verify_type<float>(a, greedy, stream);
    case MSA_DTYPE_BF16: return launch_verify_type<__nv_bfloat16>(a, greedy, stream);
    default: return launch_verify_type<__half>(a, greedy, stream);
  }
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream) {
  return launch_any(a, false, stream);
}

cudaError_t launch_verify_greedy(const VerifyArgs& a, cudaStream_t stream) {
  return launch_any(a, true, stream);
}

}  // namespace msa
