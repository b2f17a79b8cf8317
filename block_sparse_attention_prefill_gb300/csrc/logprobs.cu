// Log probabilities of given tokens, their ranks, the entropies of the rows and
// each row's best alternatives, from logits, in one pass over them.
//
// With m near the row's maximum, l = sum e^(x - m) and s = sum e^(x - m) (x - m):
//   log p(t) = (x_t - m) - log l,   H = log l - s / l
// m, l and s are kept by each thread in fp32, m raised when a larger value is
// met, and merged at the end by their m.  x - m is taken before it is multiplied
// by log2 e, so that large logits cost no accuracy.
//
// The k best are found without a list kept on the way: the pass notes the
// largest value of every chunk of 512 bytes (a warp's load).  The k best values
// lie in the k chunks whose largest come first (of equal ones those with lower
// indices): any other chunk has k values before all of its own.  These chunks
// are read again, from L2, and the k-th best of their values is found by
// bisection on keys (value, index) that are all different, so that the work
// is bounded whatever the row holds (all equal, ascending, masked).  Bisection
// ends as soon as few enough keys are left; they are put in order by counting.
//
// A cluster of 1 to 8 CTAs takes a row (as many as fill the GPU when there are
// few rows): each finds its own k best, and the first merges them through
// distributed shared memory.  Rows may start anywhere: whole 16-byte vectors
// are loaded, the first and last of a row value by value.
#include <algorithm>
#include <cfloat>
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "common.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kTop = MSA_LOGPROBS_MAX_TOP;
constexpr int kBatch = 4;        // chunks of a warp in flight
constexpr int kVocabBits = 19;   // V < 2^19
constexpr int kChunkBits = 13;   // chunks of a row: at most 4097
constexpr int kMaxChunks = (MSA_VERIFY_MAX_VOCAB * 4) / 512 + 1;
constexpr int kMostChunks = 48;  // chunks that are read again (at least k)
constexpr int kFew = 64;         // keys that are put in order by counting
static_assert(MSA_VERIFY_MAX_VOCAB == 1 << kVocabBits && kMaxChunks < 1 << kChunkBits, "keys");
static_assert(kMostChunks % kWarps == 0 && kTop <= kMostChunks && kTop <= kFew, "selection");
constexpr float kLowest = -FLT_MAX;  // m before any value (finite: x - m is no NaN)
constexpr float kFar = -200.f;       // e^d is 0 in fp32 at and below this, and 0 times it 0
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// An integer whose order is that of the values; +0 and -0 are equal, NaN is
// below all (0).
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t f = __float_as_uint(x == 0.f ? 0.f : x);
  return x != x ? 0u : (f >> 31) ? ~f : f | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ float max_or_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// A row whose first value is `shift` values behind `base`, which lies on 16
// bytes.
template <typename T>
struct Row {
  const T* base;
  int shift, V;
};

// 16 bytes of a row: vector v holds places v N - shift .. + N - 1.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  uint32_t w[4];
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[i]);
    } else {
      const uint16_t h = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
      return to_f32(*reinterpret_cast<const T*>(&h));
    }
  }
  // -inf in places outside the row
  __device__ __forceinline__ void load(const Row<T>& r, int v) {
    const int first = v * N - r.shift;
    if (first >= 0 && first + N <= r.V) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(r.base) + v);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
      const uint32_t inf = sizeof(T) == 4 ? 0xFF800000u
                           : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = inf;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (first + i >= 0 && first + i < r.V) {
          if constexpr (sizeof(T) == 4) {
            w[i] = __ldg(reinterpret_cast<const uint32_t*>(r.base) + v * N + i);
          } else {
            const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(r.base) + v * N + i);
            w[i >> 1] = i & 1 ? (w[i >> 1] & 0xFFFFu) | (h << 16) : (w[i >> 1] & 0xFFFF0000u) | h;
          }
        }
      }
    }
  }
  // the order of its largest value in the row
  __device__ __forceinline__ uint32_t top(const Row<T>& r, int v) const {
    const int first = v * N - r.shift;
    float x = __uint_as_float(0x7FFFFFFFu);  // fmaxf leaves NaN out
    if (first >= 0 && first + N <= r.V) {
#pragma unroll
      for (int i = 0; i < N; ++i) x = fmaxf(x, at(i));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (first + i >= 0 && first + i < r.V) x = fmaxf(x, at(i));
    }
    return order_of(x);
  }
};

// A key whose number of keys at or above it, over all threads of the CTA, is
// k .. most.  `count` gives a thread's number for a key.  There are at least k
// at or above `lo` (n_lo of them), fewer than k at or above `hi`; all keys are
// different, so that there is such a key.  Steps down from hi first, a step
// four times the last, since the k largest often lie close together.
template <typename F>
__device__ __forceinline__ uint64_t pick(uint64_t lo, uint64_t hi, int n_lo, int k, int most,
                                         uint64_t step, F count) {
  __shared__ int s_sum[2][kWarps];
  for (int turn = 0; n_lo > most && hi - lo > 1; turn ^= 1) {
    const uint64_t half = (hi - lo) / 2;
    const uint64_t mid = hi - (step < half ? step : half);
    const int n = __reduce_add_sync(0xffffffffu, count(mid));
    if ((threadIdx.x & 31) == 0) s_sum[turn][threadIdx.x >> 5] = n;
    __syncthreads();  // the other buffer is free: it was read before this
    int all = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) all += s_sum[turn][i];
    if (all >= k) lo = mid, n_lo = all, step = ~0ull; else hi = mid, step = step > ~0ull / 4 ? ~0ull : 4 * step;
  }
  __syncthreads();
  return lo;
}

struct Part {  // of a warp
  float m, l, s;
  int before;  // values that come before the token
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) logprobs_kernel(const LogprobsArgs a, int cluster_size) {
  constexpr int N = Vec<T>::N;
  __shared__ uint32_t s_key[kMaxChunks];
  __shared__ uint32_t s_top[kWarps];
  __shared__ Part s_part[kMaxCluster * kWarps];            // rank 0's is complete
  __shared__ uint64_t s_all[kMaxCluster][kTop];            // likewise
  __shared__ uint64_t s_cand[kFew], s_best[kTop];
  __shared__ int s_list[kMostChunks];
  __shared__ int s_n[2];
  cg::cluster_group cluster = cg::this_cluster();
  // a CTA's shared memory may be written from outside once it has started
  if (cluster_size > 1) cluster.barrier_arrive();
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_size > 1 ? (int)cluster.block_rank() : 0;
  const int64_t t = blockIdx.x / cluster_size;
  const int V = a.V;
  Row<T> row;
  {
    const T* first = static_cast<const T*>(a.logits) + t * a.row;
    row.shift = (int)(reinterpret_cast<uintptr_t>(first) % 16 / sizeof(T));
    row.base = first - row.shift;
    row.V = V;
  }
  const int chunks = (row.shift + V + 32 * N - 1) / (32 * N);
  const int per = (chunks + cluster_size - 1) / cluster_size;
  const int c0 = min(chunks, rank * per), nch = min(chunks, c0 + per) - c0;  // this CTA's
  Vec<T> x[2][kBatch];
  auto load = [&](Vec<T> (&to)[kBatch], int i) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      // a chunk behind the CTA's last is one behind the row
      const int c = i + k * kWarps < nch ? c0 + i + k * kWarps : chunks;
      to[k].load(row, c * 32 + lane);
    }
  };
  load(x[0], warp);
  const int token = a.tokens ? __ldg(a.tokens + t) : -1;
  const bool is_token = token >= 0 && token < V;
  const float mine = is_token ? to_f32(row.base[row.shift + token]) : __uint_as_float(0x7FFFFFFFu);
  const uint32_t mine_key = order_of(mine);  // 0: none

  Part p = {kLowest, 0.f, 0.f, 0};
  float2 l2 = make_float2(0.f, 0.f), s2 = l2;
  uint32_t warp_top = 0;
  auto add = [&](const Vec<T> (&v)[kBatch], int i) {
    uint32_t key[kBatch], top = 0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int c = i + k * kWarps < nch ? c0 + i + k * kWarps : chunks;
      key[k] = __reduce_max_sync(0xffffffffu, v[k].top(row, c * 32 + lane));
      top = max(top, key[k]);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (lane == k && i + k * kWarps < nch) s_key[i + k * kWarps] = key[k];
    if (top > warp_top) {
      warp_top = top;
      const float m = value_of(top);
      if (m > p.m) {
        const float d = max_or_nan(p.m - m, kFar), f = ex2_approx(d * kLog2e);
        s2 = make_float2(f * fmaf(l2.x, d, s2.x), f * fmaf(l2.y, d, s2.y));
        l2 = make_float2(l2.x * f, l2.y * f);
        p.m = m;
      }
    }
    const float2 m2 = make_float2(-p.m, -p.m), c2 = make_float2(kLog2e, kLog2e);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        float2 d = add2(make_float2(v[k].at(e), v[k].at(e + 1)), m2);
        d.x = max_or_nan(d.x, kFar), d.y = max_or_nan(d.y, kFar);
        float2 w = mul2(d, c2);
        w.x = ex2_approx(w.x), w.y = ex2_approx(w.y);
        l2 = add2(l2, w);
        s2 = fma2(w, d, s2);
      }
      if (key[k] >= mine_key && mine_key) {
        const int first = ((c0 + i + k * kWarps) * 32 + lane) * N - row.shift;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float y = v[k].at(e);
          p.before += y > mine || (y == mine && first + e >= 0 && first + e < token);
        }
      }
    }
  };
  for (int i = warp; i < nch; i += 2 * kBatch * kWarps) {
    load(x[1], i + kBatch * kWarps);
    add(x[0], i);
    if (i + kBatch * kWarps >= nch) break;
    load(x[0], i + 2 * kBatch * kWarps);
    add(x[1], i + kBatch * kWarps);
  }
  p.l = l2.x + l2.y, p.s = s2.x + s2.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    p.l += __shfl_xor_sync(0xffffffffu, p.l, o);
    p.s += __shfl_xor_sync(0xffffffffu, p.s, o);
    p.before += __shfl_xor_sync(0xffffffffu, p.before, o);
  }
  if (lane == 0) s_top[warp] = warp_top;
  if (tid < 2) s_n[tid] = 0;
  if (tid < kTop) s_best[tid] = 0;
  __syncthreads();

  const int k = a.top;
  if (k > 0 && nch > 0) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = max(top, s_top[i]);
    // the chunks that the k best lie in
    auto chunk_key = [&](int c) {
      return ((uint64_t)s_key[c] << kChunkBits) | (uint32_t)((1 << kChunkBits) - 1 - c);
    };
    const uint64_t from = pick(0, (uint64_t)(top + 1ull) << kChunkBits, nch, min(k, nch), kMostChunks,
                               1ull << (20 + kChunkBits), [&](uint64_t key) {
                                 int n = 0;
                                 for (int c = tid; c < nch; c += kThreads) n += chunk_key(c) >= key;
                                 return n;
                               });
    for (int c = tid; c < nch; c += kThreads)
      if (chunk_key(c) >= from) s_list[atomicAdd(&s_n[0], 1)] = c0 + c;
    __syncthreads();
    const int listed = s_n[0];
    constexpr int kMine = kMostChunks / kWarps;
    Vec<T> y[kMine];
    int at[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int c = j * kWarps + warp < listed ? s_list[j * kWarps + warp] : chunks;
      at[j] = c * 32 + lane;
      y[j].load(row, at[j]);
    }
    auto value_key = [&](int j, int e) {
      const int i = at[j] * N - row.shift + e;
      const uint32_t o = i >= 0 && i < V ? order_of(y[j].at(e)) : 0u;
      return o ? ((uint64_t)o << kVocabBits) | (uint32_t)((1 << kVocabBits) - 1 - i) : 0ull;
    };
    auto count = [&](uint64_t key) {
      int n = 0;
#pragma unroll
      for (int j = 0; j < kMine; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e) n += value_key(j, e) >= key;
      return n;
    };
    // every listed chunk has a value at or above the least of their largest
    const uint64_t least = max((uint64_t)1, (from >> kChunkBits) << kVocabBits);
    const int some = __reduce_add_sync(0xffffffffu, count(least));
    if (lane == 0 && some) atomicAdd(&s_n[1], some);
    __syncthreads();
    const int n = s_n[1];
    if (tid == 0) s_n[0] = 0;
    const uint64_t low = pick(least, (uint64_t)(top + 1ull) << kVocabBits, n, min(k, n), kFew,
                              1ull << (20 + kVocabBits), count);
    // (pick's last barrier stands behind s_n[0] = 0)
#pragma unroll
    for (int j = 0; j < kMine; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint64_t key = value_key(j, e);
        if (key >= low) s_cand[atomicAdd(&s_n[0], 1)] = key;
      }
    __syncthreads();
    const int cands = s_n[0];
    if (tid < cands) {
      const uint64_t key = s_cand[tid];
      int place = 0;
      for (int i = 0; i < cands; ++i) place += s_cand[i] > key;
      if (place < k) s_best[place] = key;
    }
    __syncthreads();
  }

  // to rank 0
  if (cluster_size > 1) cluster.barrier_wait();
  if (lane == 0)
    *(cluster_size > 1 ? cluster.map_shared_rank(&s_part[rank * kWarps + warp], 0)
                       : &s_part[warp]) = p;
  if (cluster_size > 1 && tid < k) *cluster.map_shared_rank(&s_all[rank][tid], 0) = s_best[tid];
  if (cluster_size > 1) cluster.sync(); else __syncthreads();
  if (rank != 0) return;
  // every warp merges the sums for itself
  const int parts = cluster_size * kWarps;  // at most 64
  const Part none = {kLowest, 0.f, 0.f, 0};
  const Part u = lane < parts ? s_part[lane] : none, v = lane + 32 < parts ? s_part[lane + 32] : none;
  float m = fmaxf(u.m, v.m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f, s = 0.f;
  int before = u.before + v.before;
  auto join = [&](const Part& q) {
    const float d = max_or_nan(q.m - m, kFar), f = exp2f(d * kLog2e);
    l += f * q.l;
    s += f * fmaf(q.l, d, q.s);
  };
  join(u), join(v);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, o);
    s += __shfl_xor_sync(0xffffffffu, s, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  const float norm = logf(l);
  auto logprob = [&](float value) { return l == 0.f ? -INFINITY : (value - m) - norm; };
  if (tid == 0) {
    if (a.logprobs) a.logprobs[t] = is_token ? logprob(mine) : -INFINITY;
    if (a.ranks) a.ranks[t] = mine_key ? before : -1;
    if (a.entropy) a.entropy[t] = l == 0.f ? 0.f : norm - s / l;
  }
  if (k == 0) return;
  auto put = [&](int place, uint64_t key) {
    a.top_tokens[t * k + place] = key ? (int)((1 << kVocabBits) - 1 - (uint32_t)(key & ((1 << kVocabBits) - 1))) : -1;
    a.top_logprobs[t * k + place] = key ? logprob(value_of((uint32_t)(key >> kVocabBits))) : -INFINITY;
  };
  if (cluster_size == 1) {
    if (tid < k) put(tid, s_best[tid]);
    return;
  }
  // one candidate a thread: its place among all
  const int of = tid / kTop, pos = tid % kTop;
  uint64_t key = of < cluster_size && pos < k ? s_all[of][pos] : 0;
  int place = 0, some = 0;
  for (int r = 0; r < cluster_size; ++r)
    for (int i = 0; i < k; ++i) {
      const uint64_t other = s_all[r][i];
      place += other > key;
      some += other != 0;
    }
  if (key && place < k) put(place, key);
  if (tid >= some && tid < k) put(tid, 0);  // fewer than k values
}

template <typename T>
cudaError_t launch_type(const LogprobsArgs& a, cudaStream_t stream) {
  // CTAs of a row: as many as keep about four an SM, each with 16 chunks or more
  const int64_t chunks = ceil_div((int64_t)a.V * sizeof(T), 512);
  int c = kMaxCluster;
  while (c > 1 && (a.T * c > (int64_t)num_sms() * 4 || chunks < 16 * c)) c /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.T * c));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)c;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, a, c);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs& a, cudaStream_t stream) {
  if (a.T <= 0) return cudaSuccess;
  switch (a.dtype) {
    case MSA_DTYPE_F32: return launch_type<float>(a, stream);
    case MSA_DTYPE_BF16: return launch_type<__nv_bfloat16>(a, stream);
    default: return launch_type<__half>(a, stream);
  }
}

}  // namespace msa
