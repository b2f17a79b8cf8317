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
//
// Greedy: draft i stands iff it is the first of the largest values of its
// row.  The same cluster scans the request's rows in order, each CTA its
// eighth; a CTA that has seen a draft beaten tells the others (a plain
// shared-memory minimum in each CTA, no barrier), who then leave out the
// rows behind it: those rows cannot matter.
#include <algorithm>
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kCluster = 8;
constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kMaxVerify = 32;  // rows of one request

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

template <typename T, int N>
struct Vec {
  T v[N];
};
template <typename T, int N>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[N]) {
  if constexpr (N * sizeof(T) == 16) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
    const Vec<T, N>& t = reinterpret_cast<const Vec<T, N>&>(w);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(t.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(p[i]);
  }
}

// The weight of a token in steps of 2^-44 (NaN and negative values: 0).
__device__ __forceinline__ uint64_t weight(float p, float q) {
  return __float2ull_rz(fminf(fmaxf(p - q, 0.f), 1.f) * 17592186044416.f);
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// floor(u * total) for u rounded down to 31 bits, in [0, total) for total > 0
__device__ __forceinline__ uint64_t threshold(float u, uint64_t total) {
  const double x = (double)u * 2147483648.0;
  const uint64_t k = x > 0.0 ? (uint64_t)fmin(x, 2147483647.0) : 0;  // NaN: 0
  return k * (total >> 31) + ((k * (total & 0x7FFFFFFFu)) >> 31);
}

// N consecutive weights a lane: 32 * N a warp step.
template <typename T, int N>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kVThreads)
verify_kernel(const VerifyArgs a, int64_t seg) {
  __shared__ uint64_t warp_tot[kVWarps];
  __shared__ uint64_t cta_tot[kCluster];
  __shared__ int s_acc;
  __shared__ int s_used;
  cg::cluster_group cluster = cg::this_cluster();
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cluster.block_rank();
  const int64_t b = blockIdx.x / kCluster;
  const int n = a.n;
  const T* target = static_cast<const T*>(a.target) + b * a.t_req;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + b * a.d_req : nullptr;

  // which drafts stand: lane i decides draft i (every CTA for itself)
  const int drafts = a.counts ? min(max(__ldg(a.counts + b), 0), n - 1) : n - 1;
  if (warp == 0) {
    bool ok = false;
    int x = -1;
    if (lane < drafts) {
      x = __ldg(a.tokens_in + b * (n - 1) + lane);
      if (x >= 0 && x < a.V) {
        const double p = to_f32(target[lane * a.t_row + x]);
        const double q = draft ? (double)to_f32(draft[lane * a.d_row + x]) : 1.0;
        ok = (double)__ldg(a.u + b * n + lane) * q < p;
      }
    }
    const uint32_t fell = ~__ballot_sync(0xffffffffu, ok);
    const int acc = fell ? __ffs(fell) - 1 : 32;
    const int used = __shfl_sync(0xffffffffu, x, acc & 31);
    if (lane == 0) {
      s_acc = min(acc, drafts);
      s_used = acc < drafts ? used : -1;
    }
    if (rank == 0) {  // the drafts that stand, and -1 behind the next token
      if (lane < n && lane != min(acc, drafts))
        a.tokens[b * n + lane] = lane < acc ? x : -1;
      if (lane == 0) a.accepted[b] = min(acc, drafts);
    }
  }
  __syncthreads();
  const int acc = s_acc;
  const bool refused = acc < drafts;
  const T* prow = target + acc * a.t_row;
  const T* qrow = refused && draft ? draft + acc * a.d_row : nullptr;
  // a certain draft (no draft probabilities) that fell is left out
  const int64_t skip = refused && !draft ? s_used : -1;

  // this CTA's part of the row, cut among its warps in whole warp steps
  const int64_t lo = min(a.V, rank * seg), hi = min(a.V, lo + seg);
  const int64_t steps = (hi - lo + 32 * N - 1) / (32 * N);
  const int64_t wsteps = (steps + kVWarps - 1) / kVWarps;
  const int64_t wlo = min(hi, lo + warp * wsteps * (32 * N));
  const int64_t whi = min(hi, wlo + wsteps * (32 * N));

  auto weights_at = [&](int64_t v, const T* q, uint64_t (&w)[N]) {
    if (N == 1 || v + N <= whi) {
      float p[N], d[N];
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = d[i] = 0.f;
      if (v < whi) {
        load_vec<T, N>(prow + v, p);
        if (q) load_vec<T, N>(q + v, d);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = v + i == skip ? 0 : weight(p[i], d[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        w[i] = v + i < whi && v + i != skip
                   ? weight(to_f32(prow[v + i]), q ? to_f32(q[v + i]) : 0.f)
                   : 0;
    }
  };

  const float u = __ldg(a.u + b * n + n - 1);
  for (int pass = 0; pass < 2; ++pass) {
    // pass 1 only where p <= q everywhere and yet a draft fell (distributions
    // that do not add up to one): the token is drawn from p itself
    const T* q = pass == 0 ? qrow : nullptr;
    uint64_t sum = 0;
#pragma unroll 4
    for (int64_t v = wlo + lane * N; v < whi; v += 32 * N) {
      uint64_t w[N];
      weights_at(v, q, w);
#pragma unroll
      for (int i = 0; i < N; ++i) sum += w[i];
    }
    sum = warp_sum(sum);
    if (lane == 0) warp_tot[warp] = sum;
    __syncthreads();
    if (threadIdx.x < kCluster) {
      uint64_t t = 0;
#pragma unroll
      for (int i = 0; i < kVWarps; ++i) t += warp_tot[i];
      *cluster.map_shared_rank(&cta_tot[rank], threadIdx.x) = t;
    }
    cluster.sync();
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
      if (rank == 0 && threadIdx.x == 0) a.tokens[b * n + acc] = -1;  // no probability at all
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
    for (int64_t v0 = wlo; v0 < whi; v0 += 32 * N) {
      uint64_t w[N], own = 0;
      weights_at(v0 + lane * N, q, w);
#pragma unroll
      for (int i = 0; i < N; ++i) own += w[i];
      uint64_t incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, incl > t);
      if (past) {
        if (lane == __ffs(past) - 1) {
          uint64_t at = incl - own;
          int i = 0;
          while (i < N - 1 && at + w[i] <= t) at += w[i++];
          a.tokens[b * n + acc] = (int32_t)(v0 + lane * N + i);
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
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kVThreads)
greedy_kernel(const VerifyArgs a, int64_t seg) {
  __shared__ uint64_t warp_best[kVWarps];
  __shared__ uint64_t row_best[kCluster][kMaxVerify];  // rank 0's is complete
  __shared__ int beaten;  // a row known to end the accepted drafts
  cg::cluster_group cluster = cg::this_cluster();
  if (threadIdx.x == 0) beaten = a.n;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cluster.block_rank();
  const int64_t b = blockIdx.x / kCluster;
  const int n = a.n;
  const T* target = static_cast<const T*>(a.target) + b * a.t_req;
  const int drafts = a.counts ? min(max(__ldg(a.counts + b), 0), n - 1) : n - 1;
  const int64_t lo = min(a.V, rank * seg), hi = min(a.V, lo + seg);
  cluster.sync();  // every CTA's `beaten` is set before another lowers it

  for (int i = 0; i <= drafts; ++i) {
    // the row's best in this CTA's part: a thread's places ascend, so the
    // first of equal values stays
    float best = -INFINITY;
    uint32_t place = 0xFFFFFFFFu;
    const T* row = target + i * a.t_row;
#pragma unroll 4
    for (int64_t v = lo + threadIdx.x * N; v < hi; v += kVThreads * N) {
      if (v + N <= hi) {
        float x[N];
        load_vec<T, N>(row + v, x);
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (x[k] > best || (x[k] == best && place == 0xFFFFFFFFu))
            best = x[k], place = (uint32_t)(v + k);
      } else {
        for (int k = 0; v + k < hi; ++k) {
          const float x = to_f32(row[v + k]);
          if (x > best || (x == best && place == 0xFFFFFFFFu)) best = x, place = (uint32_t)(v + k);
        }
      }
    }
    uint64_t key = place == 0xFFFFFFFFu ? 0 : best_key(best, place);  // 0: nothing but NaN
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
      key = other > key ? other : key;
    }
    if (lane == 0) warp_best[warp] = key;
    __syncthreads();
    if (warp == 0) {
      key = lane < kVWarps ? warp_best[lane] : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
        key = other > key ? other : key;
      }
      if (lane == 0) *cluster.map_shared_rank(&row_best[rank][i], 0) = key;
      if (i < drafts) {
        const int x = __ldg(a.tokens_in + b * (n - 1) + i);
        const float mine = x >= 0 && x < a.V ? to_f32(row[x]) : NAN;
        if (!(mine == mine) || key > best_key(mine, (uint32_t)x))
          if (lane < kCluster) atomicMin(cluster.map_shared_rank(&beaten, lane), i);
      }
    }
    // one decision for the whole CTA: other CTAs lower `beaten` at any time
    if (__syncthreads_or(*(volatile int*)&beaten <= i)) break;
  }
  cluster.sync();
  if (rank != 0 || warp != 0) return;
  // rows up to the first whose draft is beaten were scanned by every CTA
  uint64_t key = 0;
  int x = -1;
  if (lane <= drafts) {
    if (lane <= beaten)
      for (int c = 0; c < kCluster; ++c) key = row_best[c][lane] > key ? row_best[c][lane] : key;
    if (lane < drafts) x = __ldg(a.tokens_in + b * (n - 1) + lane);
  }
  const int first = key ? (int)(0xFFFFFFFFu - (uint32_t)key) : -1;
  const bool ok = lane < drafts && lane <= beaten && x == first && x >= 0;
  const uint32_t fell = ~__ballot_sync(0xffffffffu, ok);
  const int acc = min(fell ? __ffs(fell) - 1 : 32, drafts);
  if (lane < n) a.tokens[b * n + lane] = lane < acc ? x : lane == acc ? first : -1;
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
  // (an odd vocabulary's rows start anywhere)
  const bool vec = vector_rows<T>(a.target, a.t_req, a.t_row) &&
                   (greedy || !a.draft || vector_rows<T>(a.draft, a.d_req, a.d_row));
  const int64_t seg = ceil_div(ceil_div(a.V, kCluster), 32 * N) * (32 * N);
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
