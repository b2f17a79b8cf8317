// Q, K and V of new tokens on their way from the projection to the attention:
// Q and K are normalised by head (where weights are given) and rotated to
// their positions, Q is quantised to E4M3 (or rounded to bf16), K and V are
// quantised and written into their pages.
//
//   y = x / sqrt(mean x^2 + eps) * w
//   pair j of a head is turned by pos f_j:  (a, b) -> (a c - b s, a s + b c)
//   Q: E4M3(y / q_scale) or bf16(y);  K, V: as msa_kv_write writes them
//
// all in fp32, with one rounding at the end.  The angle: f_j is kept as a
// fraction of a turn in steps of 2^-64, and its product with the whole number
// pos, modulo 2^64, is the fraction of the turn at that position with an error
// of pos 2^-65 turns.  So positions of any size cost no accuracy, no table of
// cosines is read (4 bytes a value and position, as many as a row of bf16 has)
// and no fp64 arithmetic is needed.
//
// One pass over the data, bound by HBM for long chunks and by latency for
// decode steps.  A slot of 8 lanes (16 for fp32: 32 bytes a lane) takes a token
// and a run of its heads, Q's then K's then V's: a lane's places in the row stay
// the same, so its cosines and sines are found once for all of them and stay in
// registers.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kv_codec.cuh"
#include "lookup.cuh"
#include "nvfp4.cuh"
#include "ptx.cuh"

namespace msa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kStaged = 512;  // requests whose lengths a CTA keeps in shared memory
constexpr int kInFlight = 2;  // rows of a slot loaded together

// Which values make a pair: neighbours; values half of the rotated part apart,
// in whole lanes; the same where the half is no whole number of lanes.
enum { kNeighbours = 0, kHalvesByLane = 1, kHalves = 2 };

struct RopeParams {
  Recip q, k, v;
  float k6, v6;   // 6 g, NVFP4
  int chunks;     // of a token's rows
  int run;        // rows of a chunk
  bool q_wide, kv_wide;  // rows lie on 32 bytes
};

// 16-byte chunks of 8 kept apart by rows of 8, so that lanes that read chunks
// a power of two apart meet in no bank.
__device__ __forceinline__ int spread(int chunk) { return chunk ^ ((chunk >> 3) & 7); }

template <typename T, bool kFp4, int kPairing>
__global__ void __launch_bounds__(kRopeThreads, 2)
rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeParams p) {
  constexpr int kV = kVals<T>;               // values of a lane
  constexpr int N = kV / 2;
  constexpr int kLanes = kD / kV;            // of a slot
  constexpr int kSlots = kRopeThreads / kLanes;
  constexpr int kAngles = kPairing == kNeighbours ? N : kV;
  __shared__ uint64_t s_turns[MSA_ROPE_MAX_PAIRS];
  __shared__ uint8_t s_axis[MSA_ROPE_MAX_PAIRS];
  __shared__ __align__(16) float s_norm[2][kD];
  __shared__ int64_t s_page[32];
  __shared__ int s_off[32], s_pos[32];
  __shared__ int s_cu[kStaged + 1], s_cuk[kStaged + 1];
  __shared__ float s_row[kPairing == kHalves ? kSlots : 1][kD + 4];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t unit0 = (int64_t)blockIdx.x * kSlots;
  const int64_t t0 = unit0 / p.chunks;
  const int slot = tid / kLanes, cc = tid % kLanes;
  const uint32_t peers = (kLanes == 32 ? 0xffffffffu : (1u << kLanes) - 1u) << (lane & ~(kLanes - 1));
  const int64_t unit = unit0 + slot;
  const int64_t t = unit / p.chunks;
  const int i = (int)(t - t0);  // the token within the CTA's
  const int rows = a.Hq + 2 * a.Hkv;
  const int r_first = (int)(unit - t * p.chunks) * p.run;
  const int r_end = t < a.T ? min(rows, r_first + p.run) : r_first;
  // a row's first byte of this lane
  auto source = [&](int r) {
    const T* x = static_cast<const T*>(r < a.Hq ? a.q : r < a.Hq + a.Hkv ? a.k : a.v);
    const int64_t token = r < a.Hq ? a.q_token : r < a.Hq + a.Hkv ? a.k_token : a.v_token;
    const int64_t head = r < a.Hq ? a.q_head : r < a.Hq + a.Hkv ? a.k_head : a.v_head;
    const int h = r < a.Hq ? r : r < a.Hq + a.Hkv ? r - a.Hq : r - a.Hq - a.Hkv;
    return x + t * token + h * head + cc * kV;
  };
  uint32_t w[kInFlight][8];
  auto load = [&](int r0) {
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      if (r0 + k < r_end) {
        load32(source(r0 + k), r0 + k < a.Hq ? p.q_wide : p.kv_wide, w[k]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[k][e] = 0u;
      }
    }
  };
  load(r_first);  // does not wait for the look-up
  for (int j = tid; j < a.pairs; j += kRopeThreads) {
    s_turns[j] = a.turns[j];
    s_axis[j] = a.axis[j];
  }
  if (tid < 2 * kD / 4) {
    const float* n = tid < kD / 4 ? a.q_norm : a.k_norm;
    const int c = tid % (kD / 4);
    if (n)
      reinterpret_cast<float4*>(s_norm[tid / (kD / 4)])[spread(c)] =
          make_float4(__ldg(n + 4 * c), __ldg(n + 4 * c + 1), __ldg(n + 4 * c + 2), __ldg(n + 4 * c + 3));
  }
  const bool staged = a.B <= kStaged;
  if (staged) {
    for (int b = tid; b <= a.B; b += kRopeThreads) {
      s_cu[b] = __ldg(a.cu + b);
      s_cuk[b] = __ldg(a.cu_k + b);
    }
    __syncthreads();
  }
  // the CTA's tokens (at most one a slot): their places in the pool
  if (tid < 32) {
    const int64_t tt = t0 + lane;
    const bool used = lane < kSlots && tt < a.T;
    int b;
    if (staged) {
      int lo = 0, hi = a.B;  // the number of requests that end at or before tt
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (s_cu[mid + 1] <= tt) lo = mid + 1; else hi = mid;
      }
      b = lo;
    } else {
      b = lane_request_of(a.cu, a.B, (int)t0);
    }
    int64_t row = -1, pos = 0;
    if (used && b < a.B) {
      const int* cu = staged ? s_cu : a.cu;
      const int* cu_k = staged ? s_cuk : a.cu_k;
      const int first = cu[b];
      const int64_t q_len = (int64_t)cu[b + 1] - first, seq = (int64_t)cu_k[b + 1] - cu_k[b];
      pos = seq - q_len + (tt - first);
      uint32_t bad = q_len > seq || first > tt ? MSA_STATUS_BAD_SEQLENS : 0;
      if (!bad) row = pool_row(a.block_table, a.bt_stride, a.num_pages, b, pos, &bad);
      if (bad && a.status) atomicOr(a.status, bad);
    }
    s_page[lane] = row < 0 ? 0 : row / kPage * ((int64_t)a.Hkv * (kFp4 ? kFp4PageHead : kPage * 2 * kD));
    s_off[lane] = row < 0 ? -1 : (int)(row % kPage);
    s_pos[lane] = (int)pos;
  }
  __syncthreads();
  if (r_first >= r_end) return;
  const int off = s_off[i];
  if (off < 0) return;

  // cosines and sines of this lane's pairs (or of its values' pairs)
  float cs[kAngles], sn[kAngles];
  if (r_first < a.Hq + a.Hkv) {
    int pos = a.positions && a.axes == 1 ? __ldg(a.positions + t) : s_pos[i];
#pragma unroll
    for (int e = 0; e < kAngles; ++e) {
      const int at = cc * kAngles + e;
      const int j = kPairing == kNeighbours || at < a.pairs ? at : at - a.pairs;
      cs[e] = 1.f, sn[e] = 0.f;
      if (j < a.pairs) {
        if (a.axes > 1 && a.positions) pos = __ldg(a.positions + s_axis[j] * a.T + t);
        const uint64_t turn = s_turns[j] * (uint64_t)(int64_t)pos;
        const int32_t signed_turn = (int32_t)(uint32_t)((turn + 0x80000000u) >> 32);
        sincospif((float)signed_turn * 0x1p-31f, &sn[e], &cs[e]);
        if (kPairing != kNeighbours && at < a.pairs) sn[e] = -sn[e];
      }
    }
  }

  auto handle = [&](int r, const uint32_t (&raw)[8]) {
    float2 x[N];
    unpack<T>(raw, x);
    const bool is_q = r < a.Hq, turned = r < a.Hq + a.Hkv;
    if (turned) {
      if (is_q ? a.q_norm != nullptr : a.k_norm != nullptr) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < N; ++e) ss = fma2(x[e], x[e], ss);
        float sum = ss.x + ss.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(peers, sum, o);
        const float f = 1.f / sqrtf(sum * (1.f / kD) + a.eps);
        const float4* weight = reinterpret_cast<const float4*>(s_norm[is_q ? 0 : 1]);
#pragma unroll
        for (int c = 0; c < kV / 4; ++c) {
          const float4 g = weight[spread(cc * (kV / 4) + c)];
          x[2 * c] = mul2(mul2(x[2 * c], make_float2(f, f)), make_float2(g.x, g.y));
          x[2 * c + 1] = mul2(mul2(x[2 * c + 1], make_float2(f, f)), make_float2(g.z, g.w));
        }
      }
      if constexpr (kPairing == kNeighbours) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float2 y = make_float2(fmaf(x[e].x, cs[e], -x[e].y * sn[e]),
                                       fmaf(x[e].x, sn[e], x[e].y * cs[e]));
          if (cc * N + e < a.pairs) x[e] = y;
        }
      } else if constexpr (kPairing == kHalvesByLane) {
        const int step = a.pairs / kV;  // lanes of a half
        const int other = cc < step ? cc + step : cc < 2 * step ? cc - step : cc;
        const int from = (lane & ~(kLanes - 1)) + other;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float2 y = make_float2(__shfl_sync(peers, x[e].x, from),
                                       __shfl_sync(peers, x[e].y, from));
          if (cc < 2 * step)
            x[e] = make_float2(fmaf(x[e].x, cs[2 * e], y.x * sn[2 * e]),
                               fmaf(x[e].y, cs[2 * e + 1], y.y * sn[2 * e + 1]));
        }
      } else {
        float* row = s_row[slot];
#pragma unroll
        for (int e = 0; e < N; ++e)
          *reinterpret_cast<float2*>(row + cc * kV + 2 * e) = x[e];
        __syncwarp(peers);
#pragma unroll
        for (int e = 0; e < kV; ++e) {
          const int d = cc * kV + e;
          if (d < 2 * a.pairs) {
            const float y = row[d < a.pairs ? d + a.pairs : d - a.pairs];
            float& mine = e & 1 ? x[e / 2].y : x[e / 2].x;
            mine = fmaf(mine, cs[e], y * sn[e]);
          }
        }
        __syncwarp(peers);
      }
    }
    if (is_q) {
      uint8_t* out = static_cast<uint8_t*>(a.q_out) +
                     ((t * a.Hq + r) * kD + cc * kV) * (a.q_bf16 ? 2 : 1);
      if (a.q_bf16) {
        uint32_t o[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[e].x, x[e].y);
          o[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
#pragma unroll
        for (int e = 0; e < N; e += 4)
          reinterpret_cast<uint4*>(out)[e / 4] = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      } else {
        uint32_t code[N / 2];
        encode_e4m3<N>(x, p.q, code);
        store_words<N / 2>(out, code);
      }
      return;
    }
    const int half = turned ? 0 : 1;
    const int h = r - a.Hq - half * a.Hkv;
    if constexpr (kFp4) {
      uint8_t* base = a.pool + s_page[i] + (int64_t)h * kFp4PageHead + half * kFp4Slot;
      uint32_t code[N / 4], s;
      encode_nvfp4<N>(x, half ? a.v_scale : a.k_scale, half ? p.v6 : p.k6, code, &s, peers);
      store_words<N / 4>(base + off * (kD / 2) + cc * N, code);
      if (N == 8 || (cc & 1) == 0) base[kFp4Codes + off * 8 + cc * N / 8] = (uint8_t)s;
    } else {
      uint32_t code[N / 2];
      encode_e4m3<N>(x, half ? p.v : p.k, code);
      store_words<N / 2>(a.pool + s_page[i] + ((int64_t)h * kPage + off) * (2 * kD) + half * kD + cc * kV,
                         code);
    }
  };
  for (int r = r_first; r < r_end; r += kInFlight) {
#pragma unroll
    for (int k = 0; k < kInFlight; ++k)
      if (r + k < r_end) handle(r + k, w[k]);
    load(r + kInFlight);
  }
}

template <typename T, bool kFp4>
cudaError_t launch_type(const RopeArgs& a, cudaStream_t stream) {
  constexpr int kSlots = kRopeThreads * kVals<T> / kD;
  const int64_t rows = a.Hq + 2 * a.Hkv;
  RopeParams p;
  p.q = recip_of(a.q_bf16 ? 1.f : a.q_scale), p.k = recip_of(a.k_scale), p.v = recip_of(a.v_scale);
  p.k6 = 6.f * a.k_scale, p.v6 = 6.f * a.v_scale;
  // rows of a slot: all of a token's where there are tokens for two CTAs an SM
  const int64_t slots = (int64_t)num_sms() * 2 * kSlots;
  const int64_t run = std::min<int64_t>(rows, ceil_div(ceil_div(a.T * rows, slots), kInFlight) * kInFlight);
  p.chunks = (int)ceil_div(rows, run);
  p.run = (int)ceil_div(rows, p.chunks);
  const int64_t es = sizeof(T);
  auto on32 = [&](const void* x, int64_t token, int64_t head) {
    return reinterpret_cast<uintptr_t>(x) % 32 == 0 && token * es % 32 == 0 && head * es % 32 == 0;
  };
  p.q_wide = on32(a.q, a.q_token, a.q_head);
  p.kv_wide = on32(a.k, a.k_token, a.k_head) && on32(a.v, a.v_token, a.v_head);
  const int64_t grid = ceil_div(a.T * p.chunks, kSlots);
  auto run_it = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kRopeThreads), 0, stream, a, p);
  };
  if (a.interleaved || a.pairs == 0) return run_it(rope_kernel<T, kFp4, kNeighbours>);
  if (a.pairs % kVals<T> == 0) return run_it(rope_kernel<T, kFp4, kHalvesByLane>);
  return run_it(rope_kernel<T, kFp4, kHalves>);
}

}  // namespace

cudaError_t launch_rope_write(const RopeArgs& a, cudaStream_t stream) {
  if (a.T <= 0 || a.B <= 0) return cudaSuccess;
  switch (a.dtype) {
    case MSA_DTYPE_F32: return a.fp4 ? launch_type<float, true>(a, stream) : launch_type<float, false>(a, stream);
    case MSA_DTYPE_BF16:
      return a.fp4 ? launch_type<__nv_bfloat16, true>(a, stream) : launch_type<__nv_bfloat16, false>(a, stream);
    default: return a.fp4 ? launch_type<__half, true>(a, stream) : launch_type<__half, false>(a, stream);
  }
}

}  // namespace msa
