// Pieces of 32 bytes of K, V or Q, and their quantisation to the two page
// formats, shared by the kernels that write the cache.
//
// A code is the one nearest to the fp32 quotient, not to a product with a
// rounded reciprocal.  Where it can be told without dividing it is: x times
// a reciprocal made a little too small, and a little too large, enclose the
// quotient; if both round to the same code, so does the quotient.  The few
// values near the middle of two codes are divided (a scale that is a power
// of two, whose ties are many, has an exact reciprocal).
//
// Scales like 0.01 bring many bf16 values there (its powers of 2).  Residuals
// make their division cheap: with the correctly rounded reciprocal y, q = x y and
// twice q += (x - s q) y, whose residuals are exact; the last gives the rounded
// quotient (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  The rotation's V takes them (59 k tokens x 40
// rows, 4 of them V's, by 0.01: 167 us, by division 180; by 0.0127 163 both
// ways), the plain write does not (59 k tokens x 16 rows by 0.01: 88 instead of
// 101, but 75 instead of 59 by 0.0127: the code of a path that is hardly taken
// costs it more than its division).
#pragma once

#include <cmath>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <type_traits>

#include "ptx.cuh"

namespace msa {

// 32 bytes of K or V as fp32: 8 fp32 values or 16 of the 2-byte types.
template <typename T>
constexpr int kVals = 32 / sizeof(T);

__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t* w) {
  if (wide) {
    ldg_nc_v8(p, reinterpret_cast<uint32_t(&)[8]>(*w));
  } else {
    const uint4 a = __ldg(static_cast<const uint4*>(p)), b = __ldg(static_cast<const uint4*>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t (&w)[8]) {
  if (wide) {
    st_global_v8(p, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Words of T -> pairs of fp32 values, and back.
template <typename T>
__device__ __forceinline__ void unpack(const uint32_t (&w)[8], float2 (&x)[kVals<T> / 2]) {
#pragma unroll
  for (int i = 0; i < kVals<T> / 2; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    } else {
      x[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    }
  }
}
template <typename T>
__device__ __forceinline__ void pack(const float2 (&x)[kVals<T> / 2], uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < kVals<T> / 2; ++i) {
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(x[i].x), w[2 * i + 1] = __float_as_uint(x[i].y);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(x[i].x, x[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}

// How codes are found for a scale (see the top): 1 / scale rounded down and
// up by more than the errors of the reciprocal, the product and the quotient
// together (3 * 2^-24 of it); equal for a power of two; not used where the
// scale is so small or large that these, or a residual's last bit (2^-47 of the
// value, 2^-11 scales at least where codes differ), could leave fp32's range.
struct Recip {
  float scale, inverse, lo, hi;
  bool use;
};
__host__ __device__ inline Recip recip_of(float scale) {
  Recip r;
  r.scale = scale;
  r.use = scale > 1e-25f && scale < 1e25f;
  const float inv = 1.f / scale;
  r.inverse = inv;
#ifdef __CUDA_ARCH__
  const bool two = (__float_as_uint(scale) & 0x7FFFFFu) == 0;
#else
  int e;
  const bool two = std::frexp(scale, &e) == 0.5f;
#endif
  r.lo = two ? inv : inv * (1.f - 4.76837158203125e-7f);  // 2^-21
  r.hi = two ? inv : inv * (1.f + 4.76837158203125e-7f);
  return r;
}

// N pairs -> N / 2 words of four E4M3 codes.
template <int N, bool kResiduals>
__device__ __forceinline__ void encode_e4m3(const float2 (&x)[N], const Recip& r,
                                            uint32_t (&w)[N / 2]) {
  uint32_t differ = r.use ? 0u : 1u;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    uint32_t lo[2], hi[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      lo[k] = __nv_cvt_float2_to_fp8x2(mul2(x[2 * i + k], make_float2(r.lo, r.lo)), __NV_SATFINITE,
                                       __NV_E4M3);
      hi[k] = __nv_cvt_float2_to_fp8x2(mul2(x[2 * i + k], make_float2(r.hi, r.hi)), __NV_SATFINITE,
                                       __NV_E4M3);
    }
    w[i] = lo[0] | (lo[1] << 16);
    differ |= w[i] ^ (hi[0] | (hi[1] << 16));
  }
  if (kResiduals && r.use && differ) {
    const float2 y = make_float2(r.inverse, r.inverse), minus = make_float2(-r.scale, -r.scale);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      uint32_t hi[2], code[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 v = x[2 * i + k];
        hi[k] = __nv_cvt_float2_to_fp8x2(mul2(v, make_float2(r.hi, r.hi)), __NV_SATFINITE, __NV_E4M3);
        float2 q = mul2(v, y);
        q = fma2(fma2(q, minus, v), y, q);
        q = fma2(fma2(q, minus, v), y, q);
        code[k] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
      }
      // only codes that differ (the others' quotients may be infinite)
      const uint32_t those = __vcmpne4(w[i], hi[0] | (hi[1] << 16));
      w[i] = (w[i] & ~those) | ((code[0] | (code[1] << 16)) & those);
    }
  } else if (differ) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint32_t a = __nv_cvt_float2_to_fp8x2(
          make_float2(x[2 * i].x / r.scale, x[2 * i].y / r.scale), __NV_SATFINITE, __NV_E4M3);
      const uint32_t b = __nv_cvt_float2_to_fp8x2(
          make_float2(x[2 * i + 1].x / r.scale, x[2 * i + 1].y / r.scale), __NV_SATFINITE,
          __NV_E4M3);
      w[i] = a | (b << 16);
    }
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// N pairs (a block of 16 values; or a half or a quarter of one, N = 4 or 2, with
// the next lane's, or the next three's) -> words of eight E2M1 codes, the first
// in the low nibble (N = 2: half a word), and the block's E4M3 scale.  Called by
// whole warps.
template <int N>
__device__ __forceinline__ void encode_nvfp4(const float2 (&x)[N], float g, float g6,
                                             uint32_t (&w)[(N + 3) / 4], uint32_t* scale) {
  float amax = 0.f, sick = 0.f;  // sick: NaN if one of the values is
#pragma unroll
  for (int i = 0; i < N; ++i) {
    amax = fmaxf(amax, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));  // ignores NaN
    sick = max_nan(sick, max_nan(x[i].x, x[i].y));
  }
  if constexpr (N <= 4) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  if constexpr (N == 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const __nv_fp8_storage_t s8 =
      __nv_cvt_float_to_fp8(amax / g6, __NV_SATFINITE, __NV_E4M3);
  *scale = s8;
  const float den = __half2float(__half(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3))) * g;
#pragma unroll
  for (int i = 0; i < (N + 3) / 4; ++i) w[i] = 0u;
  if (!(den > 0.f)) return;
  const Recip r = recip_of(den);
  uint32_t differ = r.use && sick == sick ? 0u : 1u;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp4x2(mul2(x[i], make_float2(r.lo, r.lo)), __NV_E2M1,
                                                 cudaRoundNearest);
    const uint32_t hi = __nv_cvt_float2_to_fp4x2(mul2(x[i], make_float2(r.hi, r.hi)), __NV_E2M1,
                                                 cudaRoundNearest);
    differ |= lo ^ hi;
    w[i >> 2] |= lo << (8 * (i & 3));
  }
  if (differ) {
#pragma unroll
    for (int i = 0; i < (N + 3) / 4; ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float a = x[i].x / den, b = x[i].y / den;
      a = isnan(a) ? 0.f : a;
      b = isnan(b) ? 0.f : b;
      w[i >> 2] |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1,
                                                      cudaRoundNearest)
                   << (8 * (i & 3));
    }
  }
}

// NW consecutive words to the pool.
template <int NW>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t (&w)[NW]) {
  if constexpr (NW == 4) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if constexpr (NW == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint32_t*>(p) = w[0];
  }
}

}  // namespace msa
