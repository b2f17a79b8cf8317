// Writing new K/V tokens into the pages of the pool, quantised, and reading
// cached tokens back, dequantised (the two page formats of msa.h).
//
//   write E4M3   code = E4M3(x / scale), nearest even, saturating at 448
//   write NVFP4  per 16 values: s = E4M3(min(amax / (6 g), 448)),
//                code = E2M1(x / (s g)), nearest even, saturating at 6, and
//                0 where s g is 0 or x is NaN (E2M1 has no NaN)
//   read         E4M3 code x scale, or E4M3(code x s) x g (what the NVFP4
//                attention reads): the product in fp32, rounded to the
//                output's type
//
// (kv_codec.cuh has the quantisation.)
//
// Both directions are one pass over the data, bound by HBM for long chunks
// and by the latency of the look-up (token -> request -> position -> page)
// for decode steps.  A CTA takes a run of consecutive tokens with all their
// heads: its warps first find the tokens' places in the pool into shared
// memory, 32 tokens a warp at once, then every thread moves 32 bytes of K or
// V at a time, four of them in flight, the lanes of a warp side by side in
// either array.  A thread's head, half and place in the row stay the same, so
// that an address costs one addition.
//
// Measured: 59 k tokens x 8 heads bf16 -> E4M3 60.8 us, 6.0 TB/s; 1 M tokens x
// 2 heads E4M3 -> bf16 238 us, 6.8 TB/s (a plain copy's rate); 71 k tokens
// NVFP4 -> fp32 31 us, 5.3 TB/s; 512 tokens x 2 heads 4.0 us, of which the
// launch and the look-up's three dependent loads are most.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv_codec.cuh"
#include "lookup.cuh"
#include "nvfp4.cuh"
#include "ptx.cuh"

namespace msa {
namespace {

constexpr int kCacheThreads = 256;
constexpr int kMaxTokens = 128;  // tokens of one CTA
constexpr int kStaged = 512;     // requests whose lengths a CTA keeps in shared memory
// 32-byte pieces in flight per thread (an NVFP4 write needs its registers)
template <bool kFp4, bool kWrite>
constexpr int kBatch = kFp4 && kWrite ? 2 : 4;

__device__ __forceinline__ float2 half2_times(uint32_t h, float scale) {
  return mul2(__half22float2(*reinterpret_cast<const __half2*>(&h)), make_float2(scale, scale));
}

template <int N>
__device__ __forceinline__ void decode_e4m3(const uint32_t (&w)[N / 2], float scale,
                                            float2 (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    x[i] = half2_times(*reinterpret_cast<const uint32_t*>(&h), scale);
  }
}

// E4M3(code x block scale): the product of an E2M1 and an E4M3 value (a 6-bit
// significand, magnitude 0 or 2^-10 .. 2688) is exact in f16; the rounding to
// E4M3 and back is the conversion the attention reads through.
template <int N>
__device__ __forceinline__ void decode_nvfp4(const uint32_t (&w)[N / 4], uint32_t scale8, float g,
                                             float2 (&x)[N]) {
  const __half2 s = __half2half2(
      __half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)scale8, __NV_E4M3)));
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t two = (w[i >> 2] >> (8 * (i & 3))) & 0xFFu;
    const __half2 v = __hmul2(
        __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)two, __NV_E2M1)), s);
    const __nv_fp8x2_storage_t e =
        __nv_cvt_halfraw2_to_fp8x2(__half2_raw(v), __NV_SATFINITE, __NV_E4M3);
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(e, __NV_E4M3);
    x[i] = half2_times(*reinterpret_cast<const uint32_t*>(&h), g);
  }
}

// NW consecutive words of the pool.
template <int NW>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[NW]) {
  if constexpr (NW == 4) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (NW == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
}
struct CacheScales {
  Recip k, v;        // E4M3 writes
  float k6, v6;      // 6 g, NVFP4 writes
  int tokens;        // of a CTA
  bool wide;         // K and V rows lie on 32 bytes
};

// kWrite: k / v -> pool; else pool -> k / v.
template <typename T, bool kFp4, bool kWrite>
__global__ void __launch_bounds__(kCacheThreads, kWrite && !kFp4 ? 3 : 4)
kv_cache_kernel(const KvCacheArgs a, const CacheScales sc) {
  constexpr int N = kVals<T> / 2;                 // pairs of a piece
  constexpr int kPieces = 2 * kD / kVals<T>;      // of a token's K and V of one head
  constexpr int kSlots = kCacheThreads / kPieces; // (token, head)s at a time
  constexpr int NW = kFp4 ? N / 4 : N / 2;        // words of codes of a piece
  constexpr int kB = kBatch<kFp4, kWrite>;
  // a token's place: its page's first byte, and its row in the page
  __shared__ int64_t s_page[kMaxTokens];
  __shared__ int s_off[kMaxTokens];
  __shared__ int s_cu[kStaged + 1], s_cuk[kWrite ? kStaged + 1 : 1];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * sc.tokens;
  const int n = (int)min((int64_t)sc.tokens, a.T - t0);
  const int64_t page_bytes = (int64_t)a.Hkv * (kFp4 ? kFp4PageHead : kPage * 2 * kD);
  // up to kStaged requests: one load brings all lengths into shared memory,
  // where the search costs no round trip to L2 (decode step of 64 requests:
  // 4.0 us, searched in L2 4.7)
  const bool staged = a.B <= kStaged;
  if (staged) {
    for (int i = threadIdx.x; i <= a.B; i += kCacheThreads) {
      s_cu[i] = __ldg(a.cu + i);
      if (kWrite) s_cuk[i] = __ldg(a.cu_k + i);
    }
    __syncthreads();
  }
  if (warp * 32 < n) {
    const int i = warp * 32 + lane, t = (int)(t0 + i);
    int b;
    if (staged) {
      int lo = 0, hi = a.B;  // the number of requests that end at or before t
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (s_cu[mid + 1] <= t) lo = mid + 1; else hi = mid;
      }
      b = lo;
    } else {
      b = lane_request_of(a.cu, a.B, (int)(t0 + warp * 32));
    }
    int64_t row = -1;
    if (i < n && b < a.B) {
      const int* cu = staged ? s_cu : a.cu;
      const int first = cu[b];
      int64_t pos;
      uint32_t bad = 0;
      if (kWrite) {
        const int* cu_k = staged ? s_cuk : a.cu_k;
        const int64_t q_len = (int64_t)cu[b + 1] - first;
        const int64_t seq = (int64_t)cu_k[b + 1] - cu_k[b];
        pos = seq - q_len + (t - first);
        if (q_len > seq) bad = MSA_STATUS_BAD_SEQLENS;
      } else {
        pos = (int64_t)(a.starts ? __ldg(a.starts + b) : 0) + (t - first);
      }
      if (first > t) bad = MSA_STATUS_BAD_SEQLENS;
      if (!bad) row = pool_row(a.block_table, a.bt_stride, a.num_pages, b, pos, &bad);
      if (bad && a.status) atomicOr(a.status, bad);
    }
    if (i < n) {
      s_page[i] = row < 0 ? -1 : row / kPage * page_bytes;
      s_off[i] = row < 0 ? -1 : (int)(row % kPage);
    }
  }
  const int slot = threadIdx.x / kPieces, c = threadIdx.x % kPieces;
  const int half = c / (kPieces / 2), cc = c % (kPieces / 2);
  const float scale = half ? a.v_scale : a.k_scale;
  const Recip r = half ? sc.v : sc.k;
  // few heads: several tokens at a time; many: several heads of a token
  const int H = a.Hkv;
  const int step = H <= kSlots ? kSlots / H : 1;
  const int i0 = H <= kSlots ? slot / H : 0;
  const int h0 = H <= kSlots ? slot % H : slot, h_step = H <= kSlots ? H : kSlots;
  const int64_t token = half ? a.v_token : a.k_token, head = half ? a.v_head : a.k_head;
  T* x0 = static_cast<T*>(half ? a.v : a.k) + t0 * token + cc * kVals<T>;
  // the piece's codes from its page-head's first byte; rows of 256 or 64 bytes
  const int code0 = kFp4 ? half * kFp4Slot + cc * (NW * 4) : half * kD + cc * (NW * 4);
  constexpr int kRow = kFp4 ? kD / 2 : 2 * kD;
  const int64_t head_bytes = kFp4 ? kFp4PageHead : kPage * 2 * kD;
  // whole warps walk the loops together (the block scales are shared between
  // lanes); a slot past the last token or head has nothing to do
  const bool slot_used = i0 < step;
  const int h_rounds = (H + h_step - 1) / h_step;
  uint32_t w[kB][kWrite ? 8 : NW];
  // a write's input does not wait for the look-up
  auto load_input = [&](int h, int ib) {
#pragma unroll
    for (int k = 0; k < kB; ++k) {
      const int i = ib + k * step + i0;
      if (slot_used && h < H && i < n)
        load32(x0 + h * head + i * token, sc.wide, w[k]);
      else
#pragma unroll
        for (int e = 0; e < (kWrite ? 8 : 0); ++e) w[k][e] = 0u;
    }
  };
  if constexpr (kWrite) load_input(h0, 0);
  __syncthreads();
  for (int hr = 0; hr < h_rounds; ++hr) {
    const int h = h0 + hr * h_step;
    const bool on = slot_used && h < H;
    T* xh = x0 + (on ? h : 0) * head;
    uint8_t* ph = a.pool + (on ? h : 0) * head_bytes;
    for (int ib = 0; ib < n; ib += kB * step) {
      int off[kB];
      uint8_t* page[kB];
      uint32_t s8[kB];
#pragma unroll
      for (int k = 0; k < kB; ++k) {
        const int i = ib + k * step + i0;
        off[k] = on && i < n ? s_off[i] : -1;
        page[k] = ph + (off[k] >= 0 ? s_page[i] : 0);
        if (!kWrite && off[k] >= 0) {
          load_words<NW>(page[k] + code0 + off[k] * kRow,
                         reinterpret_cast<uint32_t(&)[NW]>(w[k]));
          if (kFp4) s8[k] = __ldg(page[k] + half * kFp4Slot + kFp4Codes + off[k] * 8 + cc * N / 8);
        }
      }
#pragma unroll
      for (int k = 0; k < kB; ++k) {
        float2 x[N];
        if constexpr (kWrite) {
          unpack<T>(w[k], x);
          uint32_t code[NW];
          if constexpr (kFp4) {
            uint32_t s;
            encode_nvfp4<N>(x, scale, half ? sc.v6 : sc.k6, code, &s);
            if (off[k] >= 0 && (N == 8 || (cc & 1) == 0))
              page[k][half * kFp4Slot + kFp4Codes + off[k] * 8 + cc * N / 8] = (uint8_t)s;
          } else {
            encode_e4m3<N, false>(x, r, code);
          }
          if (off[k] >= 0) store_words<NW>(page[k] + code0 + off[k] * kRow, code);
        } else if (off[k] >= 0) {
          if constexpr (kFp4) decode_nvfp4<N>(w[k], s8[k], scale, x);
          else decode_e4m3<N>(w[k], scale, x);
          uint32_t o[8];
          pack<T>(x, o);
          store32(xh + (int64_t)(ib + k * step + i0) * token, sc.wide, o);
        }
      }
      if constexpr (kWrite) {
        const int next = ib + kB * step;
        if (next < n) load_input(h, next);
        else if (hr + 1 < h_rounds) load_input(h + h_step, 0);
      }
    }
  }
}

template <typename T>
cudaError_t launch_type(const KvCacheArgs& a, cudaStream_t stream) {
  constexpr int kSlots = kCacheThreads * kVals<T> / (2 * kD);
  const int64_t step = std::max<int64_t>(1, kSlots / a.Hkv);
  // tokens per CTA: as many as make one wave of four CTAs an SM, up to eight
  // pieces a thread.  512 tokens x 2 heads: one piece 4.0 us, eight 5.5 (few
  // CTAs); 59 k x 8 heads: eight 60.8 us, four 68, one 208 (the look-ups);
  // NVFP4, 17 k x 2 heads: one wave 14.8 us, a wave and a half 17.4
  const int64_t rounds = std::min<int64_t>(8, ceil_div(a.T, step * num_sms() * 4));
  const int64_t tokens = std::min<int64_t>(kMaxTokens, rounds * step);
  CacheScales sc;
  sc.k = recip_of(a.k_scale), sc.v = recip_of(a.v_scale);
  sc.k6 = 6.f * a.k_scale, sc.v6 = 6.f * a.v_scale;
  sc.tokens = (int)tokens;
  const int64_t es = sizeof(T);
  auto on32 = [&](const void* p, int64_t token, int64_t head) {
    return reinterpret_cast<uintptr_t>(p) % 32 == 0 && token * es % 32 == 0 && head * es % 32 == 0;
  };
  // 32-byte accesses where all rows allow them: NVFP4 read to fp32 31 us, by
  // 16 bytes 40; 1M tokens to bf16 238 us, by 16 bytes 246
  sc.wide = on32(a.k, a.k_token, a.k_head) && on32(a.v, a.v_token, a.v_head);
  const int64_t grid = ceil_div(a.T, tokens);
  auto run = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kCacheThreads), 0, stream, a, sc);
  };
  if (a.fp4) return a.write ? run(kv_cache_kernel<T, true, true>) : run(kv_cache_kernel<T, true, false>);
  return a.write ? run(kv_cache_kernel<T, false, true>) : run(kv_cache_kernel<T, false, false>);
}

}  // namespace

cudaError_t launch_kv_cache(const KvCacheArgs& a, cudaStream_t stream) {
  if (a.T <= 0 || a.B <= 0) return cudaSuccess;
  switch (a.dtype) {
    case MSA_DTYPE_F32: return launch_type<float>(a, stream);
    case MSA_DTYPE_BF16: return launch_type<__nv_bfloat16>(a, stream);
    default: return launch_type<__half>(a, stream);
  }
}

}  // namespace msa
