// Trees of drafted tokens, given by each token's parent: the ancestor masks and
// positions that attention and rotation need, and, after the target has run,
// the path that its own tokens follow, whose rows of the cache are moved to
// their place in the sequence.
//
// A request's new tokens are its tree's nodes, parents before their children.
//
//   mask     anc(i) = {i} + anc(parent(i)); position = context + |anc(i)| - 1
//   accept   path = node 0, then the first child whose token is the target's
//            choice after the node before it, and so on; row context + path[j]
//            becomes row context + j, in every layer
//
// Both are bound by latency: a few dependent loads and a few rounds in shared
// memory (GPU time, replayed from a graph: masks of one tree of 16 2.3 us, of 256
// of up to 255 4.5; acceptance of one tree in 4 layers 1.9 us, of 64 in 32 3.4).  A CTA takes a request.  Ancestors are found by doubling: every round
// a node takes over what its farthest known ancestor knows, so that a chain of
// 256 takes 8 rounds and not 255.  An accepting CTA finds the path for itself
// and then moves rows of some (layer, head)s: 16 lanes a row, 16 bytes each.
// A lane only ever reads and writes its own 16 bytes of the rows, in order of
// the path, and a row's new place is never behind its old one: no row is written
// before it has been read.
#include <algorithm>

#include "common.cuh"
#include "lookup.cuh"
#include "nvfp4.cuh"

namespace msa {
namespace {

constexpr int kNodes = MSA_TREE_MAX_TOKENS;
constexpr int kWords = kNodes / 32;

// A request's tokens, or false where the lengths do not fit.
struct Request {
  int first;  // of the batch's tokens
  int n;
  int64_t context;  // tokens before them
};
__device__ __forceinline__ bool request_at(const int32_t* cu_q, const int32_t* cu_k, int b,
                                           int64_t T, int max_q, Request* r) {
  const int q0 = __ldg(cu_q + b), q1 = __ldg(cu_q + b + 1);
  const int64_t seq = (int64_t)__ldg(cu_k + b + 1) - __ldg(cu_k + b);
  const int64_t n = (int64_t)q1 - q0;
  r->first = q0;
  r->n = (int)n;
  r->context = seq - n;
  return q0 >= 0 && n >= 0 && q1 <= T && n <= max_q && seq >= n;
}

__global__ void __launch_bounds__(kNodes) tree_mask_kernel(const TreeMaskArgs a) {
  __shared__ uint32_t s_mask[2][kNodes][kWords + 1];  // (a word apart: no bank twice)
  __shared__ int s_up[2][kNodes];
  pdl_wait();
  pdl_trigger();
  const int i = threadIdx.x, b = blockIdx.x, W = a.words;
  Request r;
  if (!request_at(a.cu_q, a.cu_k, b, a.T, a.max_q, &r)) {
    if (i == 0 && a.status) atomicOr(a.status, (unsigned)MSA_STATUS_BAD_SEQLENS);
    return;
  }
  int up = -1;
  if (i < r.n) {
    up = __ldg(a.parents + r.first + i);
    if (up < -1 || up >= i) {
      if (a.status) atomicOr(a.status, (unsigned)MSA_STATUS_BAD_TREE);
      up = -1;
    }
    for (int w = 0; w < W; ++w) s_mask[0][i][w] = w == i >> 5 ? 1u << (i & 31) : 0u;
    s_up[0][i] = up;
  }
  int cur = 0;
  while (__syncthreads_or(up >= 0)) {
    if (i < r.n) {
      for (int w = 0; w < W; ++w)
        s_mask[cur ^ 1][i][w] = s_mask[cur][i][w] | (up >= 0 ? s_mask[cur][up][w] : 0u);
      up = up >= 0 ? s_up[cur][up] : -1;
      s_up[cur ^ 1][i] = up;
    }
    cur ^= 1;
  }
  // (the loop's last barrier stands behind all writes)
  if (i < r.n && a.positions) {
    int depth = -1;
    for (int w = 0; w < W; ++w) depth += __popc(s_mask[cur][i][w]);
    a.positions[r.first + i] = (int)(r.context + depth);
  }
  if (a.mask) {
    uint32_t* out = a.mask + (int64_t)r.first * W;
    for (int e = i; e < r.n * W; e += blockDim.x) out[e] = s_mask[cur][e / W][e % W];
  }
}

constexpr int kAcceptThreads = 256;
constexpr int kRowLanes = 16;
constexpr int kSlots = kAcceptThreads / kRowLanes;
constexpr int kRowsInFlight = 4;

template <bool kFp4>
__global__ void __launch_bounds__(kAcceptThreads)
tree_accept_kernel(const __grid_constant__ TreeAcceptArgs a) {
  __shared__ int s_chosen[kNodes], s_next[kNodes], s_path[kNodes], s_draft[kNodes];
  __shared__ int64_t s_src[kNodes], s_dst[kNodes];  // rows of the pool, or -1
  __shared__ int s_count;
  pdl_wait();
  pdl_trigger();
  const int i = threadIdx.x, b = blockIdx.x;
  Request r;
  const bool ok = request_at(a.cu_q, a.cu_k, b, a.T, a.max_q, &r);
  if (!ok) r.n = 0;
  int up = -1;
  if (i < r.n) {
    up = __ldg(a.parents + r.first + i);
    s_chosen[i] = __ldg(a.chosen + r.first + i);
    s_draft[i] = __ldg(a.drafts + r.first + i);
    s_next[i] = kNodes;
  }
  __syncthreads();
  uint32_t bad = ok ? 0 : (uint32_t)MSA_STATUS_BAD_SEQLENS;
  if (i > 0 && i < r.n) {
    if (up >= 0 && up < i) {
      // (-1, msa_logprobs' best of a row of NaN, is no token)
      if (s_draft[i] >= 0 && s_draft[i] == s_chosen[up]) atomicMin(&s_next[up], i);
    } else if (up != -1) {
      bad |= MSA_STATUS_BAD_TREE;
    }
  }
  __syncthreads();
  if (i == 0) {
    int n = 0;
    for (int at = 0; at < r.n; at = s_next[at]) s_path[n++] = at;
    s_count = n;
  }
  __syncthreads();
  const int count = s_count;  // nodes of the path, the root with them
  if (blockIdx.y == 0) {
    if (i < a.max_q) {
      const int64_t o = (int64_t)b * a.max_q + i;
      a.tokens[o] = i + 1 < count ? s_draft[s_path[i + 1]] : i + 1 == count ? s_chosen[s_path[i]] : -1;
      if (a.path) a.path[o] = i < count ? s_path[i] : -1;
    }
    if (i == 0) a.accepted[b] = max(count - 1, 0);
  }
  if (a.layers > 0 && i < count && s_path[i] != i) {
    s_src[i] = pool_row(a.block_table, a.bt_stride, a.num_pages, b, r.context + s_path[i], &bad);
    s_dst[i] = pool_row(a.block_table, a.bt_stride, a.num_pages, b, r.context + i, &bad);
  } else if (i < count) {
    s_src[i] = s_dst[i] = -1;
  }
  if (bad && a.status && blockIdx.y == 0) atomicOr(a.status, bad);
  if (a.layers == 0 || count < 2) return;
  __syncthreads();
  // the first nodes of a path are often in their place already
  int j0 = 1;
  while (j0 < count && s_path[j0] == j0) ++j0;
  const int lane = i % kRowLanes;
  if (kFp4 && lane >= 10) return;  // 2 x (4 lanes of codes, one of scales)
  const int units = a.layers * a.Hkv;
  for (int u = blockIdx.y * kSlots + i / kRowLanes; u < units; u += gridDim.y * kSlots) {
    const int layer = u / a.Hkv, h = u - layer * a.Hkv;
    uint8_t* base = a.pools[layer];
    auto place = [&](int64_t row) {
      const int64_t head = row / kPage * a.Hkv + h;
      const int in = (int)(row % kPage);
      if constexpr (kFp4) {
        uint8_t* slot = base + head * kFp4PageHead + (lane >= 5 ? kFp4Slot : 0);
        const int piece = lane >= 5 ? lane - 5 : lane;
        return piece < 4 ? slot + in * (kD / 2) + piece * 16 : slot + kFp4Codes + in * 8;
      } else {
        return base + (head * kPage + in) * (2 * kD) + lane * 16;
      }
    };
    const bool scales = kFp4 && lane % 5 == 4;  // 8 bytes
    for (int j = j0; j < count; j += kRowsInFlight) {
      uint4 x[kRowsInFlight];
      uint8_t* dst[kRowsInFlight];
#pragma unroll
      for (int k = 0; k < kRowsInFlight; ++k) {
        const int64_t s = j + k < count ? s_src[j + k] : -1, d = j + k < count ? s_dst[j + k] : -1;
        dst[k] = nullptr;
        if (s >= 0 && d >= 0) {
          const uint8_t* src = place(s);
          dst[k] = place(d);
          if (scales) {
            const uint2 y = *reinterpret_cast<const uint2*>(src);
            x[k] = make_uint4(y.x, y.y, 0u, 0u);
          } else {
            x[k] = *reinterpret_cast<const uint4*>(src);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kRowsInFlight; ++k) {
        if (dst[k]) {
          if (scales)
            *reinterpret_cast<uint2*>(dst[k]) = make_uint2(x[k].x, x[k].y);
          else
            *reinterpret_cast<uint4*>(dst[k]) = x[k];
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_tree_mask(const TreeMaskArgs& a, cudaStream_t stream) {
  if (a.B <= 0 || a.T <= 0) return cudaSuccess;
  const int threads = (int)ceil_div(std::max(a.max_q, 1), 32) * 32;
  return launch_pdl(tree_mask_kernel, dim3((unsigned)a.B), dim3(threads), 0, stream, a);
}

cudaError_t launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t stream) {
  if (a.B <= 0) return cudaSuccess;
  // CTAs of a request: a (layer, head) a slot, up to about four CTAs an SM
  const int64_t most = std::max<int64_t>(1, (int64_t)num_sms() * 4 / a.B);
  const int64_t y = std::max<int64_t>(1, std::min(most, ceil_div((int64_t)a.layers * a.Hkv, kSlots)));
  const dim3 grid((unsigned)a.B, (unsigned)y);
  return a.fp4 ? launch_pdl(tree_accept_kernel<true>, grid, dim3(kAcceptThreads), 0, stream, a)
               : launch_pdl(tree_accept_kernel<false>, grid, dim3(kAcceptThreads), 0, stream, a);
}

}  // namespace msa
