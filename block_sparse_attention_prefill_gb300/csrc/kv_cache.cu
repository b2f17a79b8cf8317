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
// All arithmetic is fp32 with true divisions, so that a code is the nearest
// one to the quotient and not to a product with a rounded reciprocal.
//
// Both are one pass over the data, bound by HBM for long chunks and by the
// latency of the look-up (token -> request -> position -> page) for decode
// steps.  A CTA takes a run of consecutive tokens with all their heads.  Its
// warps first find the tokens' rows of the pool into shared memory (a 32-way
// search of cu_seqlens, one or two steps, instead of a binary one), then
// every thread handles blocks of 16 values: 16 threads to a (token, head),
// 8 for K and 8 for V, whose accesses cover the whole 256-byte row of an E4M3
// page (or the 64 code bytes of each NVFP4 slot).
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "lookup.cuh"
#include "nvfp4.cuh"
#include "ptx.cuh"

namespace msa {
namespace {

constexpr int kCacheThreads = 256;
constexpr int kMaxTokens = 64;  // tokens of one CTA

// 16 consecutive values in fp32.
__device__ __forceinline__ void load16(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
    x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
      x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void load16(const __half* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      x[8 * i + 2 * k] = f.x, x[8 * i + 2 * k + 1] = f.y;
    }
  }
}

__device__ __forceinline__ void store16(float* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(p)[i] =
        make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void store16(__half* p, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

__device__ __forceinline__ uint4 encode_e4m3(const float (&x)[16], float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(x[4 * i] / scale, x[4 * i + 1] / scale), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(x[4 * i + 2] / scale, x[4 * i + 3] / scale), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 values -> 8 code bytes (the first value in the low nibble) and the
// block's E4M3 scale.
__device__ __forceinline__ uint2 encode_nvfp4(const float (&x)[16], float g, float g6,
                                              uint32_t* scale) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));  // ignores NaN
  const __nv_fp8_storage_t s8 =
      __nv_cvt_float_to_fp8(amax / g6, __NV_SATFINITE, __NV_E4M3);
  *scale = s8;
  const float den = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3))) * g;
  uint32_t w[2] = {0u, 0u};
  if (den > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a = x[2 * i] / den, b = x[2 * i + 1] / den;
      a = isnan(a) ? 0.f : a;
      b = isnan(b) ? 0.f : b;
      const uint32_t two =
          __nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest);
      w[i >> 2] |= two << (8 * (i & 3));
    }
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void decode_e4m3(uint4 c, float scale, float (&x)[16]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3));
    const float2 f = __half22float2(h);
    x[2 * i] = f.x * scale, x[2 * i + 1] = f.y * scale;
  }
}

// E4M3(code x block scale): the product of an E2M1 and an E4M3 value (a 6-bit
// significand, magnitude 0 or 2^-10 .. 2688) is exact in f16; the rounding to
// E4M3 and back is the conversion the attention reads through.
__device__ __forceinline__ void decode_nvfp4(uint2 codes, uint32_t scale8, float g,
                                             float (&x)[16]) {
  const __half2 s = __half2half2(
      __half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)scale8, __NV_E4M3)));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t two = ((i < 4 ? codes.x : codes.y) >> (8 * (i & 3))) & 0xFFu;
    const __half2 v = __hmul2(
        __half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)two, __NV_E2M1)), s);
    const __nv_fp8x2_storage_t e =
        __nv_cvt_halfraw2_to_fp8x2(__half2_raw(v), __NV_SATFINITE, __NV_E4M3);
    const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(e, __NV_E4M3)));
    x[2 * i] = f.x * g, x[2 * i + 1] = f.y * g;
  }
}

// kWrite: k / v -> pool; else pool -> k / v.
template <typename T, bool kFp4, bool kWrite>
__global__ void __launch_bounds__(kCacheThreads)
kv_cache_kernel(const KvCacheArgs a, int tokens, float k_scale6, float v_scale6) {
  __shared__ int64_t rows[kMaxTokens];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const int n = (int)min((int64_t)tokens, a.T - t0);
  for (int i = warp; i < n; i += kCacheThreads / 32) {
    const int t = (int)(t0 + i);
    const int b = warp_request_of(a.cu, a.B, t);
    int64_t row = -1;
    if (b < a.B) {
      const int first = __ldg(a.cu + b);
      int64_t pos;
      uint32_t bad = 0;
      if (kWrite) {
        const int64_t q_len = (int64_t)__ldg(a.cu + b + 1) - first;
        const int64_t seq = (int64_t)__ldg(a.cu_k + b + 1) - __ldg(a.cu_k + b);
        pos = seq - q_len + (t - first);
        if (q_len > seq) bad = MSA_STATUS_BAD_SEQLENS;
      } else {
        pos = (int64_t)(a.starts ? __ldg(a.starts + b) : 0) + (t - first);
      }
      if (first > t) bad = MSA_STATUS_BAD_SEQLENS;
      if (!bad) row = pool_row(a.block_table, a.bt_stride, a.num_pages, b, pos, &bad);
      if (bad && lane == 0 && a.status) atomicOr(a.status, bad);
    }
    if (lane == 0) rows[i] = row;
  }
  __syncthreads();
  const int units = n * a.Hkv * 16;
#pragma unroll 2
  for (int u = threadIdx.x; u < units; u += kCacheThreads) {
    const int c = u & 7, half = (u >> 3) & 1, th = u >> 4;
    const int i = th / a.Hkv, h = th - i * a.Hkv;
    const int64_t row = rows[i];
    if (row < 0) continue;
    const int64_t page = row / kPage;
    const int off = (int)(row % kPage);
    const int64_t head = page * a.Hkv + h;
    T* x = reinterpret_cast<T*>(half ? a.v : a.k) +
           (t0 + i) * (half ? a.v_token : a.k_token) + h * (half ? a.v_head : a.k_head) + c * 16;
    const float scale = half ? a.v_scale : a.k_scale;
    float f[16];
    if (!kFp4) {
      uint4* p = reinterpret_cast<uint4*>(a.pool + (head * kPage + off) * (2 * kD) + half * kD +
                                          c * 16);
      if (kWrite) {
        load16(x, f);
        *p = encode_e4m3(f, scale);
      } else {
        decode_e4m3(__ldg(p), scale, f);
        store16(x, f);
      }
    } else {
      uint8_t* slot = a.pool + head * kFp4PageHead + half * kFp4Slot;
      uint2* p = reinterpret_cast<uint2*>(slot + off * 64 + c * 8);
      uint8_t* ps = slot + kFp4Codes + off * 8 + c;
      if (kWrite) {
        load16(x, f);
        uint32_t s;
        *p = encode_nvfp4(f, scale, half ? v_scale6 : k_scale6, &s);
        *ps = (uint8_t)s;
      } else {
        decode_nvfp4(__ldg(p), __ldg(ps), scale, f);
        store16(x, f);
      }
    }
  }
}

template <typename T>
cudaError_t launch_type(const KvCacheArgs& a, cudaStream_t stream) {
  // tokens per CTA: one block of 16 values a thread while that fills the GPU
  // (decode steps), up to four a thread for long chunks
  const int per_token = (int)a.Hkv * 16;
  int64_t tokens = std::max<int64_t>(1, kCacheThreads / per_token);
  const int64_t many = std::min<int64_t>(kMaxTokens, std::max<int64_t>(1, 4 * kCacheThreads / per_token));
  if (a.T >= many * num_sms() * 8) tokens = many;
  const int64_t grid = ceil_div(a.T, tokens);
  auto run = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kCacheThreads), 0, stream, a,
                      (int)tokens, 6.f * a.k_scale, 6.f * a.v_scale);
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
