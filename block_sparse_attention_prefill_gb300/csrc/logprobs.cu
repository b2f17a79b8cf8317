// Log probabilities of given tokens, their ranks, the entropies of the rows and
// each row's best alternatives, from logits, in one pass over them.
//
// With m near the row's maximum, l = sum e^(x - m) and s = sum e^(x - m) (x - m):
//   log p(t) = (x_t - m) - log l,   H = log l - s / l
// m, l and s are kept by each thread in fp32 (as powers of 2), m raised for a
// whole warp when a larger value is met, and merged at the end by their m.
//
// The k best are found without a list kept on the way: the pass notes the
// largest value of every chunk of 512 bytes (a warp's load), and of each lane.
// The k-th largest of 64 groups of lanes' is a bound that k values pass, and few
// more (24 for k = 20, were they in random order); the chunks whose largest pass
// it are read again, from L2, and their values that do, 512 at most, are put in
// order by counting.  Where more than that pass (rows that are all equal,
// ascending, masked) bounds are found by bisection on keys (value, index) that
// are all different: the k best lie in the k chunks whose largest come first (of
// equal ones those with lower indices, as any other chunk has k values before
// all of its own), and in the k of their vectors for which the same holds.  So
// the work is bounded whatever the row holds.
//
// Bounds and what was measured (GPU time, replayed from a graph): 2048 rows of
// 131072 bf16, 5 best: 111 us, 4.8 TB/s; without tokens and best 87 (6.2 TB/s).
// Ranks cost a packed comparison and a sum for every two values (14 us), the
// selection about 4 us a row and CTA, in which its warps load little (12 us).
// 16 rows of 200003 fp32, 20 best: 10.1 us, latency (the pass 5, bound and
// selection 2.5, exchange and merge of the cluster 2.5).
//
// A cluster of 1 to 8 CTAs takes a row (as many as fill the GPU when there are
// few rows): each finds its own k best and hands them to the first through
// distributed shared memory, whose warps merge them by twos (bitonic merges).
// Rows may start anywhere: whole 16-byte vectors are loaded, the first and last
// of a row value by value.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "common.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace msa {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kTop = MSA_LOGPROBS_MAX_TOP;
constexpr int kVocabBits = 19;   // V < 2^19
constexpr int kChunkBits = 13;   // chunks of a row: at most 4097
constexpr int kVecBits = 18;     // vectors of a row: at most 2^17 + 1
constexpr int kMaxChunks = (MSA_VERIFY_MAX_VOCAB * 4) / 512 + 1;
constexpr int kMostChunks = 64;  // chunks that are read again
constexpr int kRound = 4;        // of a thread's vectors among them, in flight
constexpr int kMostVecs = 64;    // vectors whose values are looked at
constexpr int kFew = kMostVecs * 8;
constexpr int kBuckets = 64;     // of a CTA's lanes
static_assert(MSA_VERIFY_MAX_VOCAB == 1 << kVocabBits && kMaxChunks < 1 << kChunkBits, "keys");
static_assert(kTop == 32 && kTop <= kMostChunks && kTop <= kMostVecs, "selection");
constexpr float kLowest = -FLT_MAX;  // m before any value (finite: x - m is no NaN)
constexpr float kFar = -200.f;       // 2^t is 0 in fp32 at and below this, and 0 times it 0
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same<T, __half>::value) return __float2half(x);
  else return __float2bfloat16(x);
}
// The next larger number of the type (NaN above infinity).
template <typename T>
__device__ __forceinline__ T next_above(T x) {
  using U = typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type;
  constexpr U kSign = (U)1 << (8 * sizeof(T) - 1);
  U u = *reinterpret_cast<const U*>(&x);
  u = (U)(u << 1) == 0 ? (U)1 : u & kSign ? (U)(u - 1) : (U)(u + 1);
  return *reinterpret_cast<const T*>(&u);
}

// An integer whose order is that of the values; +0 and -0 are equal, NaN is
// below all (0).
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t f = __float_as_uint(x == 0.f ? 0.f : x);
  return x != x ? 0u : (f >> 31) ? ~f : f | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}
// A value and its place; keys of one row are all different.
__device__ __forceinline__ uint64_t value_key(float x, int place) {
  const uint32_t o = order_of(x);
  return o ? ((uint64_t)o << kVocabBits) | (uint32_t)((1 << kVocabBits) - 1 - place) : 0ull;
}

__device__ __forceinline__ float max_or_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float largest(float a, float b) { return fmaxf(a, b); }  // leaves NaN out
// The largest of the warp's values, NaN left out.
__device__ __forceinline__ float warp_max(float x) {
  float d;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(x));
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
  static constexpr bool k16 = sizeof(T) == 2;
  using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
  uint32_t w[4];
  __device__ __forceinline__ T2 two(int i) const { return *reinterpret_cast<const T2*>(&w[i]); }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (!k16) {
      return __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    } else {
      return i & 1 ? __high2float(two(i >> 1)) : __low2float(two(i >> 1));
    }
  }
  __device__ __forceinline__ void load(const Row<T>& r, int v) {  // wholly inside the row
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(r.base) + v);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  }
  // -inf in places outside the row
  __device__ __forceinline__ void load_edge(const Row<T>& r, int v) {
    const int first = v * N - r.shift;
    if (first >= 0 && first + N <= r.V) return load(r, v);
    const uint32_t inf = !k16 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = inf;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (first + i >= 0 && first + i < r.V) {
        if constexpr (!k16) {
          w[i] = __ldg(reinterpret_cast<const uint32_t*>(r.base) + v * N + i);
        } else {
          const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(r.base) + v * N + i);
          w[i >> 1] = i & 1 ? (w[i >> 1] & 0xFFFFu) | (h << 16) : (w[i >> 1] & 0xFFFF0000u) | h;
        }
      }
    }
  }
  // its largest value, NaN if it has none
  __device__ __forceinline__ float top() const {
    if constexpr (k16) {
      const T2 x = __hmax2(__hmax2(two(0), two(1)), __hmax2(two(2), two(3)));
      return largest(__low2float(x), __high2float(x));
    } else {
      return largest(largest(at(0), at(1)), largest(at(2), at(3)));
    }
  }
  // the same of a vector that may reach over the row's ends
  __device__ __forceinline__ float top_edge(const Row<T>& r, int v) const {
    float x = __uint_as_float(0x7FFFFFFFu);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int place = v * N - r.shift + i;
      if (place >= 0 && place < r.V) x = largest(x, at(i));
    }
    return x;
  }
};

// A reference m has sums in powers of 2 of one of two kinds.  Near 0, of x log2 e
// - r with r = m log2 e rounded to fp32, whose rounding, at most 2^-4 here, is the
// same in all terms.  Far from 0 that rounding would grow (to 64 at 1e9: powers
// out of fp32's range), and they are of (x - m) log2 e, two operations.  (m =
// -FLT_MAX: no value yet.)
__device__ __forceinline__ bool is_far(float m) { return !(fabsf(m) < 1e6f); }
enum { kPlain, kBounded, kFarM };
// r of m: a rounded product, wherever it is used (never fused with a sum: the terms
// and what they are joined by would then not be by the same r)
__device__ __forceinline__ float ref_of(float m) { return __fmul_rn(m, kLog2e); }

// What sums by the reference (m, r) have to be multiplied by, as a power of 2, to
// be by (m2, r2); kFar and less count as kFar.
__device__ __forceinline__ float shift_of(float m, float r, float m2, float r2) {
  const float d = !is_far(m2) ? (!is_far(m) ? r - r2 : fmaf(m, kLog2e, -r2))
                  : !is_far(m) ? -fmaf(m2, kLog2e, -r) : (m - m2) * kLog2e;
  return max_or_nan(d, kFar);
}

// What a thread gathers on its way, in powers of 2: l = sum 2^t and s = sum 2^t t
// of t = x log2 e - r, a fused operation (far from 0: of (x - m) log2 e, two).
// What log2 e and r lack of exactness is the same in all terms and in the token's
// own t, so that large logits cost no accuracy.
template <typename T>
struct Sums {
  using V = Vec<T>;
  float m, r;
  float2 l, s;  // (of the even and the odd values)
  int before;   // values that come before the token
  // What is far below m counts as that far: -inf would give 0 times -inf.  Of 16
  // bits two values at once before they are widened, by a number `low` that lies
  // at least 200 below m whichever way it is rounded; where the type has none,
  // and of fp32, t is bounded.
  typename V::T2 low;
  int mode;

  __device__ __forceinline__ void raise(float to) {
    const float r2 = ref_of(to);
    const float d = shift_of(m, r, to, r2), f = ex2_approx(d);
    s = make_float2(f * fmaf(l.x, d, s.x), f * fmaf(l.y, d, s.y));
    l = make_float2(l.x * f, l.y * f);
    m = to, r = r2;
    mode = is_far(to) ? kFarM : kBounded;
    if constexpr (V::k16) {
      constexpr bool kHalf = std::is_same<T, __half>::value;
      const float least = m + kFar - fabsf(m) * 0.015625f;
      if (least > (kHalf ? -64000.f : -3.3e38f) && mode == kBounded) mode = kPlain;
      if constexpr (kHalf) low = __float2half2_rn(least);
      else low = __float2bfloat162_rn(least);
    }
  }
  template <int kMode>
  __device__ __forceinline__ void add_as(const V& v) {
    const float2 r2 = make_float2(-r, -r), c2 = make_float2(kLog2e, kLog2e);
#pragma unroll
    for (int i = 0; i < 4; i += V::k16 ? 1 : 2) {
      float2 t;
      if constexpr (V::k16) {
        V x = v;
        if constexpr (kMode == kPlain) {
          const typename V::T2 y = __hmax2_nan(v.two(i), low);
          x.w[i] = *reinterpret_cast<const uint32_t*>(&y);
        }
        t = make_float2(x.at(2 * i), x.at(2 * i + 1));
      } else {
        t = make_float2(v.at(i), v.at(i + 1));
      }
      if constexpr (kMode == kFarM)
        t = mul2(add2(t, make_float2(-m, -m)), c2);
      else
        t = fma2(t, c2, r2);
      if constexpr (kMode != kPlain) t.x = max_or_nan(t.x, kFar), t.y = max_or_nan(t.y, kFar);
      const float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
      l = add2(l, p);
      s = fma2(p, t, s);
    }
  }
};

// A key whose number of keys at or above it, over all threads of the CTA, is
// k .. most.  `count` gives a thread's number for a key.  There are at least k
// at or above `lo` (n_lo of them), fewer than k at or above `hi`; all keys are
// different, so that there is such a key.  Steps down from hi first, a step
// four times the last, since the k largest often lie close together.
template <int kWarps, typename F>
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
    if (all >= k) lo = mid, n_lo = all, step = ~0ull;
    else hi = mid, step = step > ~0ull / 4 ? ~0ull : 4 * step;
  }
  __syncthreads();
  return lo;
}

struct Part {  // of a warp, its sums of 2^t with t = (x - m) log2 e
  float m, l, s;
  int before;
};

// kBatch: chunks of a warp that are worked on together, with as many more in
// flight: 4 with 24 warps an SM (80 registers a thread), 2 with 32.
constexpr int warps_of_sm(int batch) { return batch == 4 ? 24 : 32; }
constexpr int ctas_of_sm(int warps, int batch) { return warps_of_sm(batch) / warps; }

template <typename T, int kWarps, int kBatch>
__global__ void __launch_bounds__(kWarps * 32, ctas_of_sm(kWarps, kBatch))
logprobs_kernel(const LogprobsArgs a, int cluster_size) {
  using V = Vec<T>;
  constexpr int N = V::N, kThreads = kWarps * 32;
  constexpr int kMine = kMostChunks / kWarps;  // vectors of a thread among the chunks read again
  static_assert(kMine % kRound == 0 && kThreads % kBuckets == 0, "selection");
  extern __shared__ float s_max[];  // the largest value of each chunk
  __shared__ float s_top[kWarps], s_bound;
  __shared__ __align__(16) float s_bucket[kBuckets];
  __shared__ Part s_part[kMaxCluster * kWarps];  // rank 0's is complete
  __shared__ uint64_t s_all[kMaxCluster][kTop];  // likewise; in order, 0 behind the last
  __shared__ uint64_t s_cand[kFew], s_best[kTop];
  __shared__ int s_list[kMostChunks];
  __shared__ int s_n[2];  // chunks listed, values gathered
  cg::cluster_group cluster = cg::this_cluster();
  // a CTA's shared memory may be written from outside once it has started
  if (cluster_size > 1) cluster.barrier_arrive();
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = cluster_size > 1 ? (int)cluster.block_rank() : 0;
  const int64_t t = blockIdx.x / cluster_size;
  Row<T> row;
  {
    const T* first = static_cast<const T*>(a.logits) + t * a.row;
    row.shift = (int)(reinterpret_cast<uintptr_t>(first) % 16 / sizeof(T));
    row.base = first - row.shift;
    row.V = a.V;
  }
  const int chunks = (row.shift + a.V + 32 * N - 1) / (32 * N);
  const int per = (chunks + cluster_size - 1) / cluster_size;
  const int c0 = min(chunks, rank * per), nch = min(chunks, c0 + per) - c0;  // this CTA's
  // its chunks that lie wholly inside the row: in0 .. in1 - 1
  const int in0 = c0 == 0 && row.shift > 0 ? 1 : 0;
  const int in1 = min(nch, (row.shift + a.V) / (32 * N) - c0);
  V x[2][kBatch];
  auto load = [&](V (&to)[kBatch], int c) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (c + k * kWarps < in1) to[k].load(row, (c0 + c + k * kWarps) * 32 + lane);
  };
  load(x[0], in0 + warp);
  const int token = a.tokens ? __ldg(a.tokens + t) : -1;
  const bool is_token = token >= 0 && token < a.V;
  const float mine = is_token ? to_f32(row.base[row.shift + token]) : __uint_as_float(0x7FFFFFFFu);
  const int token_chunk = is_token ? (row.shift + token) / (32 * N) - c0 : -1;

  Sums<T> sum;
  sum.m = sum.r = kLowest;
  sum.l = sum.s = make_float2(0.f, 0.f);
  sum.before = 0;
  sum.mode = kFarM;
  // values before the token in a chunk that it lies in, or at an end of the row
  auto count_places = [&](const V& v, int c) {
    const int first = ((c0 + c) * 32 + lane) * N - row.shift;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float y = v.at(e);
      sum.before += y > mine || (y == mine && first + e >= 0 && first + e < token);
    }
  };
  // the chunks that the row ends in
  auto edge = [&](int c) {
    V v;
    const int at = (c0 + c) * 32 + lane;
    v.load_edge(row, at);
    const float top = warp_max(v.top_edge(row, at));
    if (lane == 0) s_max[c] = top;
    if (top > sum.m) sum.raise(top);
    if (sum.mode == kFarM) sum.template add_as<kFarM>(v); else sum.template add_as<kBounded>(v);
    count_places(v, c);
  };
  // In the chunks before the token's values as large come before it, in those
  // behind it larger ones: values at or above the next larger number.
  const T mine1 = from_f32<T>(mine), above1 = next_above(mine1);
  const float above_mine = to_f32(above1);
  const typename V::T2 mine2 = {mine1, mine1}, above2 = {above1, above1};
  float bucket = -INFINITY;  // the lane's largest value
  auto add_some = [&](auto full, const V (&v)[kBatch], int c) {
    float top[kBatch], most = kLowest;
    auto there = [&](int k) { return decltype(full)::value || c + k * kWarps < in1; };
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (!there(k)) continue;
      const float own = v[k].top();
      bucket = largest(bucket, own);
      top[k] = warp_max(own);
      most = largest(most, top[k]);
    }
    float kept = -INFINITY;
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (there(k) && lane == k) kept = top[k];
    if (lane < kBatch && (decltype(full)::value || c + lane * kWarps < in1)) s_max[c + lane * kWarps] = kept;
    if (most > sum.m) sum.raise(most);
    constexpr int kUsual = V::k16 ? kPlain : kBounded;
    if (sum.mode == kUsual) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (there(k)) sum.template add_as<kUsual>(v[k]);
    } else {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (!there(k)) continue;
        if (sum.mode == kFarM) sum.template add_as<kFarM>(v[k]); else sum.template add_as<kBounded>(v[k]);
      }
    }
    if (!(most >= mine)) return;  // (no token: mine is NaN)
    if (token_chunk >= c && token_chunk <= c + (kBatch - 1) * kWarps && (token_chunk - c) % kWarps == 0) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (there(k)) count_places(v[k], c + k * kWarps);
      return;
    }
    using T2 = typename V::T2;
    T2 n2 = T2{T(0.f), T(0.f)};
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (!there(k)) continue;
      const bool before = c + k * kWarps < token_chunk;
      if constexpr (V::k16) {
        const T2 bound = before ? mine2 : above2;
#pragma unroll
        for (int i = 0; i < 4; ++i) n2 = __hadd2(n2, __hge2(v[k].two(i), bound));
      } else {
        const float bound = before ? mine : above_mine;
#pragma unroll
        for (int e = 0; e < N; ++e) sum.before += v[k].at(e) >= bound;
      }
    }
    if constexpr (V::k16) sum.before += (int)(__low2float(n2) + __high2float(n2));  // at most 32
  };
  auto add = [&](const V (&v)[kBatch], int c) {
    if (c + (kBatch - 1) * kWarps < in1) add_some(std::true_type(), v, c);
    else add_some(std::false_type(), v, c);
  };
  constexpr int kStep = kBatch * kWarps;
  if (in0 > 0 && warp == kWarps - 1) edge(0);
  for (int c = max(in1, in0) + warp; c < nch; c += kWarps) edge(c);
  for (int c = in0 + warp; c < in1; c += 2 * kStep) {
    load(x[1], c + kStep);
    add(x[0], c);
    if (c + kStep >= in1) break;
    load(x[0], c + 2 * kStep);
    add(x[1], c + kStep);
  }
  Part p = {sum.m, sum.l.x + sum.l.y, sum.s.x + sum.s.y, sum.before};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    p.l += __shfl_xor_sync(0xffffffffu, p.l, o);
    p.s += __shfl_xor_sync(0xffffffffu, p.s, o);
    p.before += __shfl_xor_sync(0xffffffffu, p.before, o);
  }
  if (!is_far(p.m)) {  // r's rounding out of the sums: from here on they are by m itself
    const float o = fmaf(p.m, kLog2e, -ref_of(p.m)), f = ex2_approx(-o);
    p.s = f * fmaf(p.l, -o, p.s);
    p.l *= f;
  }
  if (lane == 0) s_top[warp] = sum.m;
  // 64 buckets of the CTA: its lanes by as many together as make 64
  constexpr int kOfWarp = kBuckets / kWarps;
#pragma unroll
  for (int o = 16; o >= kOfWarp; o >>= 1) bucket = largest(bucket, __shfl_xor_sync(0xffffffffu, bucket, o));
  if (lane < kOfWarp) s_bucket[warp * kOfWarp + lane] = bucket;
  if (tid < 2) s_n[tid] = 0;
  if (tid < kTop) s_best[tid] = 0;
  __syncthreads();

  const int k = a.top;
  if (k > 0 && nch > 0) {
    // this thread's vectors of the listed chunks from the j0-th on, -1: none
    auto read = [&](V (&y)[kRound], int (&at)[kRound], int j0, int listed) {
#pragma unroll
      for (int j = 0; j < kRound; ++j) {
        const int of = (j0 + j) * kWarps + warp;
        at[j] = of < listed ? s_list[of] * 32 + lane : -1;
        if (at[j] >= 0) y[j].load_edge(row, at[j]);
      }
    };
    // A bound that k values pass: the k-th largest of the buckets' largest values,
    // whose place is the number of those before it (some threads a value)
    {
      constexpr int kShare = kThreads / kBuckets;
      const int j = tid / kShare, i0 = tid % kShare * (kBuckets / kShare);
      const float u = s_bucket[j];
      int place = 0;
#pragma unroll
      for (int i = 0; i < kBuckets / kShare; i += 4) {
        const float4 other = *reinterpret_cast<const float4*>(s_bucket + i0 + i);
        place += other.x > u || (other.x == u && i0 + i < j);
        place += other.y > u || (other.y == u && i0 + i + 1 < j);
        place += other.z > u || (other.z == u && i0 + i + 2 < j);
        place += other.w > u || (other.w == u && i0 + i + 3 < j);
      }
#pragma unroll
      for (int o = 1; o < kShare; o <<= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
      if (place == k - 1) s_bound = u;
    }
    __syncthreads();
    const float bound = s_bound;
    if (bound > -INFINITY) {
      for (int c = tid; c < nch; c += kThreads) {
        if (s_max[c] >= bound) {
          const int to = atomicAdd(&s_n[0], 1);
          if (to < kMostChunks) s_list[to] = c0 + c;
        }
      }
    } else if (tid == 0) {
      s_n[0] = kMostChunks + 1;
    }
    __syncthreads();
    const int passed = s_n[0];
    if (passed <= kMostChunks) {
      // the places of the values that pass the bound (above -inf); few lanes have any
#pragma unroll 1
      for (int j0 = 0; j0 * kWarps < passed; j0 += kRound) {
        V y[kRound];
        int at[kRound];
        read(y, at, j0, passed);
        uint32_t hits[kRound];
        int n = 0;
#pragma unroll
        for (int j = 0; j < kRound; ++j) {
          hits[j] = 0;
#pragma unroll
          for (int e = 0; e < N; ++e) hits[j] |= y[j].at(e) >= bound ? 1u << e : 0u;
          if (at[j] < 0) hits[j] = 0;
          n += __popc(hits[j]);
        }
        if (n > 0) {
          int to = atomicAdd(&s_n[1], n);
#pragma unroll
          for (int j = 0; j < kRound; ++j)
            for (uint32_t h = hits[j]; h; h &= h - 1, ++to)
              if (to < kFew) s_cand[to] = (uint64_t)(at[j] * N - row.shift + __ffs(h) - 1);
        }
      }
    }
    __syncthreads();
    int cands = s_n[1];
    if (passed > kMostChunks || cands > kFew) {
      // Too many pass (values that are alike, few chunks): bounds by bisection,
      // of the chunks first, then of their vectors, on keys that are all different
      __syncthreads();
      if (tid < 2) s_n[tid] = 0;
      float most = s_top[0];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) most = largest(most, s_top[i]);
      const uint64_t above = (uint64_t)order_of(most) + 1;
      auto chunk_key = [&](int c) {
        return ((uint64_t)order_of(s_max[c]) << kChunkBits) | (uint32_t)((1 << kChunkBits) - 1 - c);
      };
      const uint64_t from = pick<kWarps>(0, above << kChunkBits, nch, min(k, nch), min(kMostChunks, max(2 * k, 8)),
                                 1ull << (20 + kChunkBits), [&](uint64_t key) {
                                   int n = 0;
                                   for (int c = tid; c < nch; c += kThreads) n += chunk_key(c) >= key;
                                   return n;
                                 });
      // (pick ends with a barrier)
      for (int c = tid; c < nch; c += kThreads)
        if (chunk_key(c) >= from) s_list[atomicAdd(&s_n[0], 1)] = c0 + c;
      __syncthreads();
      const int listed = s_n[0];
      uint64_t key[kMine];
#pragma unroll
      for (int j0 = 0; j0 < kMine; j0 += kRound) {
        V y[kRound];
        int at[kRound];
        read(y, at, j0, listed);
#pragma unroll
        for (int j = 0; j < kRound; ++j) {
          const uint32_t o = at[j] < 0 ? 0u : order_of(y[j].top_edge(row, at[j]));
          key[j0 + j] = o ? ((uint64_t)o << kVecBits) | (uint32_t)((1 << kVecBits) - 1 - at[j]) : 0ull;
        }
      }
      auto count = [&](uint64_t of) {
        int n = 0;
#pragma unroll
        for (int j = 0; j < kMine; ++j) n += key[j] >= of;
        return n;
      };
      const int some = __reduce_add_sync(0xffffffffu, count(1));
      if (lane == 0) atomicAdd(&s_n[1], some);
      __syncthreads();
      const int n = s_n[1];
      __syncthreads();
      if (tid == 0) s_n[1] = 0;
      const uint64_t low = pick<kWarps>(1, above << kVecBits, n, min(k, n), min(kMostVecs, max(2 * k, 16)),
                                1ull << (20 + kVecBits), count);
      // (here -inf may be among the best: places outside the row are told apart)
      const uint32_t least = max(1u, (uint32_t)(low >> kVecBits));
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        if (key[j] < low) continue;
        const int first = ((1 << kVecBits) - 1 - (int)(key[j] & ((1 << kVecBits) - 1))) * N - row.shift;
        for (int i = max(first, 0); i < min(first + N, a.V); ++i)
          if (order_of(to_f32(row.base[row.shift + i])) >= least) s_cand[atomicAdd(&s_n[1], 1)] = (uint64_t)i;
      }
      __syncthreads();
      cands = s_n[1];
    }
    // the values at these places, and their order
    for (int c = tid; c < cands; c += kThreads) {
      const int place = (int)s_cand[c];
      s_cand[c] = value_key(to_f32(row.base[row.shift + place]), place);
    }
    __syncthreads();
    for (int c = tid; c < cands; c += kThreads) {
      const uint64_t one = s_cand[c];
      int place = 0;
#pragma unroll 4
      for (int i = 0; i < cands; ++i) place += s_cand[i] > one;
      if (place < k) s_best[place] = one;
    }
    __syncthreads();
  }

  // to rank 0
  if (cluster_size > 1) {
    cluster.barrier_wait();
    if (lane == 0) *cluster.map_shared_rank(&s_part[rank * kWarps + warp], 0) = p;
    if (tid < kTop) *cluster.map_shared_rank(&s_all[rank][tid], 0) = s_best[tid];
    cluster.sync();
    if (rank != 0) return;
  } else {
    if (lane == 0) s_part[warp] = p;
    __syncthreads();
  }
  // every warp merges the sums for itself
  const int parts = cluster_size * kWarps;
  constexpr int kParts = kMaxCluster * kWarps / 32;  // of a lane
  Part part[kParts];
  float m = kLowest;
  int before = 0;
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    part[i] = {kLowest, 0.f, 0.f, 0};
    if (lane + 32 * i < parts) part[i] = s_part[lane + 32 * i];
    m = largest(m, part[i].m);
    before += part[i].before;
  }
  m = warp_max(m);
  float l = 0.f, s = 0.f;
  auto join = [&](const Part& q) {
    const float d = max_or_nan((q.m - m) * kLog2e, kFar), f = ex2_approx(d);
    l += f * q.l;
    s += f * fmaf(q.l, d, q.s);
  };
#pragma unroll
  for (int i = 0; i < kParts; ++i) join(part[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, o);
    s += __shfl_xor_sync(0xffffffffu, s, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  const float norm = log2f(l);
  auto logprob = [&](float value) { return l == 0.f ? -INFINITY : (value - m) - kLn2 * norm; };
  if (tid == 0) {
    if (a.logprobs) a.logprobs[t] = is_token ? logprob(mine) : -INFINITY;
    if (a.ranks) a.ranks[t] = mine == mine ? before : -1;
    if (a.entropy) a.entropy[t] = l == 0.f ? 0.f : kLn2 * (norm - s / l);
  }
  if (k == 0) return;
  auto put = [&](int place, uint64_t key) {
    a.top_tokens[t * k + place] = key ? (1 << kVocabBits) - 1 - (int)(key & ((1 << kVocabBits) - 1)) : -1;
    a.top_logprobs[t * k + place] = key ? logprob(value_of((uint32_t)(key >> kVocabBits))) : -INFINITY;
  };
  if (cluster_size == 1) {
    if (tid < k) put(tid, s_best[tid]);
    return;
  }
  // Two lists in order at a time into one, by a warp: of the first's i-th and the
  // second's i-th from the end the larger ones are the 32 best, first ascending
  // or descending and then the other way, and five exchanges put them in order.
  for (int lists = cluster_size / 2; lists > 0; lists /= 2) {
    if (warp < lists) {
      const uint64_t one = s_all[warp][lane], other = s_all[warp + lists][kTop - 1 - lane];
      uint64_t key = one > other ? one : other;
#pragma unroll
      for (int o = kTop / 2; o > 0; o /= 2) {
        const uint64_t far = __shfl_xor_sync(0xffffffffu, key, o);
        key = ((lane & o) == 0) == (key > far) ? key : far;
      }
      s_all[warp][lane] = key;
      if (lists == 1 && lane < k) put(lane, key);
    }
    __syncthreads();
  }
}

template <typename T, int kWarps, int kBatch>
cudaError_t launch_as(const LogprobsArgs& a, int cluster, int64_t chunks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.T * cluster));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = (size_t)ceil_div(chunks, cluster) * sizeof(float);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, kWarps, kBatch>, a, cluster);
}

template <typename T>
cudaError_t launch_type(const LogprobsArgs& a, cudaStream_t stream) {
  // Which CTAs and how many a row: the least of an estimate in microseconds.  A
  // round of CTAs takes what is fixed (launch, selection, outputs: 6, half a one
  // more in clusters, up to `crowd` more where an SM has all its CTAs; later
  // rounds' half overlaps the rows still read) and its share of the bytes at
  // 6 TB/s, of a round that is not full at least `least`.
  // 10 best, measured (and estimated), with 16, 8 or 4 warps a CTA x CTAs a row:
  //   131072 bf16:   64 rows 16x2 9.9 (10), 8x4 10.5 (11), 4x8 10.9
  //     190 rows 8x2 17.0 (17), 8x1 18.8 (19); 304 rows 8x1 19.7 (23), 16x1 23.1
  //     512 rows 4x2 35.2 (34), 8x1 40.6 (40), 4x1 45.7 (42)
  //     912 rows 8x1 53.8 (51), 4x1 55.0 (54); 1024 rows 4x1 60.0 (58), 8x1 64.1 (65)
  //    1500 rows 8x1 86.6 (90), 4x1 95.8 (94); 2048 rows 4x1 111 (110), 8x1 115 (116)
  //   32000 bf16: 152 rows 16x1 7.9 (8), 8x1 8.4 (9); 512 rows 4x1 13.7 (16), 8x1 16.8 (18)
  //   200003 fp32: 12 rows 16x8 7.9 (11), 8x8 9.2 (11); 16 rows 8x8 9.8 (11), 16x8, whose
  //     clusters do not all find room at once, 13.2; 100 rows 8x4 18.6 (22), 16x1 19.4 (25)
  const int64_t chunks = ceil_div((int64_t)a.V * sizeof(T), 512) + 1;
  const double sms = num_sms();
  constexpr double kFixed = 6.0, kCluster = 0.5, kChunk = 0.013;  // (512 bytes on every SM)
  struct Kind {
    int warps, ctas;  // of a CTA, of an SM
    double crowd, least;
    int chunks, most; // of a CTA at least, where a row has several; of a row's CTAs
  };
  static_assert(kMaxCluster == 8, "kinds");
  constexpr Kind kinds[] = {{16, 1, 0.5, 0.88, 64, 8}, {8, 3, 1.5, 0.35, 12, 8}, {4, 8, 4.0, 0.32, 64, 2}};
  static_assert(ctas_of_sm(16, 4) == 1 && ctas_of_sm(8, 4) == 3 && ctas_of_sm(4, 2) == 8, "kinds");
  int warps = 8, cluster = 1;
  double best = DBL_MAX;
  for (const Kind& kind : kinds) {
    for (int c = 1; c <= kind.most && (c == 1 || chunks >= (int64_t)kind.chunks * c); c *= 2) {
      const double rounds = (double)a.T * c / (sms * kind.ctas);
      // one CTA an SM: clusters have to find room in what is left of a GPC
      if (kind.ctas == 1 && (chunks < kind.chunks || rounds > (c == 8 ? 0.66 : c == 4 ? 0.85 : 1.0))) continue;
      const double whole = std::floor(rounds), rest = rounds - whole;
      const double fixed = kFixed + (c > 1 ? kCluster : 0.0) + kind.crowd * std::min(rounds, 1.0);
      const double t = fixed * (std::ceil(rounds) + 1.0) / 2.0 +
                       kChunk * kind.ctas * (double)chunks / c *
                           (whole + (rest > 0 ? kind.least + (1.0 - kind.least) * rest : 0.0));
      if (t < best) best = t, warps = kind.warps, cluster = c;
    }
  }
  switch (warps) {
    case 16: return launch_as<T, 16, 4>(a, cluster, chunks, stream);
    case 8: return launch_as<T, 8, 4>(a, cluster, chunks, stream);
    default: return launch_as<T, 4, 2>(a, cluster, chunks, stream);
  }
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
