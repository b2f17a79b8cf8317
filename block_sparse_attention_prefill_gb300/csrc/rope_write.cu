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
// of pos 2^-65 turns; its first 32 bits, from -1/2 to 1/2, become an fp32 number
// (off by 2^-26 turns at most, by less near 0).  So positions of any size cost no accuracy, no table of
// cosines is read (4 bytes a value and position, as many as a row of bf16 has)
// and no fp64 arithmetic is needed.
//
// One pass over the data, bound by HBM for long chunks and by latency for
// decode steps.  A slot of 8 lanes (16 for fp32: 32 bytes a lane) takes a token
// and a run of its heads, Q's then K's then V's, with the same heads in all of a
// warp's slots: a lane's places in the row stay the same, so its cosines and
// sines are found once for all heads and stay in registers, and no branch divides
// a warp.  Where pairs are half of the rotated part apart a lane takes two pieces
// of 16 bytes that are, so that it has both values of its pairs (32 contiguous
// bytes and exchanges between lanes: 243 us instead of 180).
//
// Measured (GPU time, replayed from a graph): 59 k tokens x (32 + 2 x 4) heads
// bf16 -> E4M3 163 us, 5.6 TB/s; 512 tokens x (16 + 2 x 2) heads 6.1 us, of which
// the launch, the look-up's dependent loads and the angles are most.
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

constexpr int kRopeThreads = 128, kRopeWarps = kRopeThreads / 32;
constexpr int kStaged = 512;  // requests whose lengths a CTA keeps in shared memory
// Rows of a slot in flight, and CTAs an SM, by the registers that a format needs
// (before rounds were told apart, see launch_type: 8 chunks of 8k tokens to E4M3
// 162 us, by 4 and 4: 170; 8 k tokens to NVFP4 and back 28.9 us, by 3 and 5: 30.3)
constexpr int in_flight(bool fp4) { return fp4 ? 4 : 3; }
constexpr int ctas_of_sm(bool fp4) { return fp4 ? 4 : 5; }

// Where a lane's two pieces of 16 bytes lie and how its pairs are formed.
//   kNeighbours  side by side; pairs of neighbouring values
//   kSplit       half of the rotated part apart (or, behind it, half of the
//                rest): a lane has both values of its pairs
//   kHalves      side by side; a pair's other value comes through shared memory
//                (a half that is no whole number of pieces)
enum { kNeighbours, kSplit, kHalves };

struct RopeParams {
  float q_inverse, k_inverse;
  Recip v;
  float k6, v6;   // 6 g, NVFP4
  struct Part {   // CTAs of one kind, from the first on
    int cta, group;  // first CTA and group of a warp's tokens
    int chunks;      // of a token's rows
    int run;         // rows of a chunk
  } part[2];
  bool q_wide, kv_wide;  // rows lie on 32 bytes
};

// Four E4M3 codes, nearest even, saturating.
__device__ __forceinline__ uint32_t four_e4m3(float2 a, float2 b) {
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}\n"
      : "=r"(w)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return w;
}

template <typename T, bool kFp4, int kPairing>
__global__ void __launch_bounds__(kRopeThreads, ctas_of_sm(kFp4))
rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeParams p) {
  constexpr int kInFlight = in_flight(kFp4);
  constexpr int kV = kVals<T>, kPiece = kV / 2;  // values of a lane, and of a piece
  constexpr int N = kV / 2, H = N / 2;           // pairs of values: of a lane, of a piece
  constexpr int kLanes = kD / kV;                // of a slot
  constexpr int kTokens = 32 / kLanes;           // of a warp
  constexpr int kCtaTokens = kRopeWarps * kTokens;
  constexpr bool kIsSplit = kPairing == kSplit;
  static_assert(kCtaTokens <= 32, "looked up by one warp");
  __shared__ uint64_t s_turns[MSA_ROPE_MAX_PAIRS];
  __shared__ uint8_t s_axis[MSA_ROPE_MAX_PAIRS];
  __shared__ __align__(16) float s_norm[2][kD];
  __shared__ int64_t s_page[32];
  __shared__ int s_off[32], s_pos[32];
  __shared__ int s_cu[kStaged + 1], s_cuk[kStaged + 1];
  __shared__ float s_row[kPairing == kHalves ? kCtaTokens : 1][kD + 4];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (the same for all lanes)
  // a warp takes kTokens tokens and a run of their heads: its rows are all of Q,
  // all of K or all of V at a time
  const RopeParams::Part& m = p.part[(int)blockIdx.x >= p.part[1].cta];
  const int64_t unit0 = (int64_t)((int)blockIdx.x - m.cta) * kRopeWarps, unit = unit0 + warp;
  const int64_t t0 = (m.group + unit0 / m.chunks) * kTokens, group = m.group + unit / m.chunks;
  const int slot = lane / kLanes, cc = lane % kLanes;
  const int64_t t = group * kTokens + slot;
  const int i = (int)(t - t0);  // the token within the CTA's
  const int k0 = a.Hq, v0 = a.Hq + a.Hkv, rows = v0 + a.Hkv;  // first rows of K and V
  const int r_first = (int)(unit - (group - m.group) * m.chunks) * m.run;
  const int r_end = group * kTokens < a.T ? min(rows, r_first + m.run) : r_first;
  const bool in_batch = t < a.T;
  // the first values of the lane's pieces
  const int turned = a.pairs / kPiece;  // (kSplit) lanes with pairs
  const int d0 = !kIsSplit ? cc * kV : cc < turned ? cc * kPiece : a.pairs + cc * kPiece;
  const int d1 = !kIsSplit ? d0 + kPiece : cc < turned ? d0 + a.pairs : kD / 2 + cc * kPiece;
  // Rows in order, Q's, K's, V's: the next one to load, its kind's next.
  struct Walk {
    const T* at;
    int64_t head;
    int row;
  } next;
  auto enter = [&](Walk& x, int r) {  // row r is the first of a kind, or of the run
    const bool q = r < k0, k = r < v0;
    x.head = q ? a.q_head : k ? a.k_head : a.v_head;
    x.at = static_cast<const T*>(q ? a.q : k ? a.k : a.v) +
           t * (q ? a.q_token : k ? a.k_token : a.v_token) + (r - (q ? 0 : k ? k0 : v0)) * x.head + d0;
    x.row = r;
  };
  enter(next, r_first);
  uint32_t w[kInFlight][8];
  auto load = [&](uint32_t (&to)[8]) {  // the next row, zeros behind the last
    if (next.row < r_end && in_batch) {
      if constexpr (kIsSplit) {
        const uint4 lo = __ldg(reinterpret_cast<const uint4*>(next.at));
        const uint4 hi = __ldg(reinterpret_cast<const uint4*>(next.at + (d1 - d0)));
        to[0] = lo.x, to[1] = lo.y, to[2] = lo.z, to[3] = lo.w;
        to[4] = hi.x, to[5] = hi.y, to[6] = hi.z, to[7] = hi.w;
      } else {
        load32(next.at, next.row < k0 ? p.q_wide : p.kv_wide, to);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) to[e] = 0u;
    }
    next.at += next.head;
    if (++next.row == k0 || next.row == v0) enter(next, next.row);
  };
#pragma unroll
  for (int k = 0; k < kInFlight; ++k) load(w[k]);  // does not wait for the look-up
  int pos = a.positions && a.axes == 1 && in_batch ? __ldg(a.positions + t) : 0;
  for (int j = tid; j < a.pairs; j += kRopeThreads) {
    s_turns[j] = a.turns[j];
    s_axis[j] = a.axis[j];
  }
  if (tid < 2 * kD / 4) {
    const float* n = tid < kD / 4 ? a.q_norm : a.k_norm;
    const int c = tid % (kD / 4);
    if (n)
      reinterpret_cast<float4*>(s_norm[tid / (kD / 4)])[c] =
          make_float4(__ldg(n + 4 * c), __ldg(n + 4 * c + 1), __ldg(n + 4 * c + 2), __ldg(n + 4 * c + 3));
  }
  const bool staged = a.B <= kStaged;
  if (staged) {
    for (int b = tid; b <= a.B; b += kRopeThreads) {
      s_cu[b] = __ldg(a.cu + b);
      s_cuk[b] = __ldg(a.cu_k + b);
    }
  }
  __syncthreads();
  // the CTA's tokens: their places in the pool, found by warp 0; the page's number
  // is on its way while the angles are found
  int64_t place = -1;
  int page = 0;
  uint32_t bad = 0;
  if (warp == 0) {
    const int64_t tt = t0 + lane;
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
    if (lane < kCtaTokens && tt < a.T && b < a.B) {
      const int* cu = staged ? s_cu : a.cu;
      const int* cu_k = staged ? s_cuk : a.cu_k;
      const int first = cu[b];
      const int64_t q_len = (int64_t)cu[b + 1] - first, seq = (int64_t)cu_k[b + 1] - cu_k[b];
      place = seq - q_len + (tt - first);
      if (q_len > seq || first > tt || place < 0 || place / kPage >= a.bt_stride) {
        bad = MSA_STATUS_BAD_SEQLENS;
        place = -1;
      } else {
        page = __ldg(a.block_table + b * a.bt_stride + place / kPage);
      }
    }
  }
  auto finish = [&] {
    if (warp == 0) {
      if (place >= 0 && (page < 0 || page >= a.num_pages)) bad = MSA_STATUS_BAD_BLOCK;
      if (bad && a.status) atomicOr(a.status, bad);
      const bool there = place >= 0 && !bad;
      s_page[lane] = there ? (int64_t)page * a.Hkv * (kFp4 ? kFp4PageHead : kPage * 2 * kD) : 0;
      s_off[lane] = there ? (int)(place % kPage) : -1;
      s_pos[lane] = (int)place;
    }
    __syncthreads();
  };
  if (!a.positions) finish();
  // Cosines and sines of the lane's pairs (kHalves: of its values' pairs, the
  // sine with its sign), 1 and 0 where there is none.
  constexpr int kAngles = kPairing == kHalves ? kV : kPiece;
  float cs[kAngles], sn[kAngles], ms[kIsSplit ? kAngles : 1];
  auto pair_of = [&](int e) {  // -1: none
    if (kPairing == kNeighbours) return cc * N + e < a.pairs ? cc * N + e : -1;
    if (kIsSplit) return cc < turned ? d0 + e : -1;
    return d0 + e < a.pairs ? d0 + e : d0 + e < 2 * a.pairs ? d0 + e - a.pairs : -1;
  };
  if (r_first < min(v0, r_end)) {
    if (!a.positions) pos = s_pos[i];
#pragma unroll
    for (int e = 0; e < kAngles; ++e) {
      const int j = pair_of(e);
      cs[e] = 1.f, sn[e] = 0.f;
      if (j >= 0) {
        if (a.axes > 1 && a.positions && in_batch) pos = __ldg(a.positions + s_axis[j] * a.T + t);
        const uint64_t turn = s_turns[j] * (uint64_t)(int64_t)pos;
        const int32_t signed_turn = (int32_t)(uint32_t)((turn + 0x80000000u) >> 32);
        sincospif((float)signed_turn * 0x1p-31f, &sn[e], &cs[e]);
        if (kPairing == kHalves && d0 + e < a.pairs) sn[e] = -sn[e];
      }
      if (kIsSplit) ms[e] = -sn[e];  // (a packed product takes no sign)
    }
  }
  if (a.positions) finish();
  if (r_first >= r_end) return;  // (whole warps)
  const int off = s_off[i];
  const bool live = off >= 0;  // what is written of this slot's token
  // the norm's weights, of Q and then of K
  float2 g[N];
  auto weights = [&](const float* of) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float4 y = *reinterpret_cast<const float4*>(of + (e < H ? d0 + 2 * e : d1 + 2 * (e - H)));
      g[e] = make_float2(y.x, y.y), g[e + 1] = make_float2(y.z, y.w);
    }
  };
  if (a.q_norm && r_first < k0) weights(s_norm[0]);
  if (a.k_norm && r_first >= k0) weights(s_norm[1]);

  // x normalised and turned
  auto turn = [&](float2 (&x)[N], bool normed) {
    if (normed) {
      float2 ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < N; ++e) ss = fma2(x[e], x[e], ss);
      float sum = ss.x + ss.y;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      const float f = rsqrtf(sum * (1.f / kD) + a.eps);
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = mul2(mul2(x[e], make_float2(f, f)), g[e]);
    }
    if constexpr (kPairing == kNeighbours) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float2 y = make_float2(fmaf(x[e].x, cs[e], -x[e].y * sn[e]), fmaf(x[e].x, sn[e], x[e].y * cs[e]));
        if (pair_of(e) >= 0) x[e] = y;
      }
    } else if constexpr (kIsSplit) {
      if (cc < turned) {
#pragma unroll
        for (int e = 0; e < H; ++e) {
          const float2 c = make_float2(cs[2 * e], cs[2 * e + 1]), s = make_float2(sn[2 * e], sn[2 * e + 1]);
          const float2 minus = make_float2(ms[2 * e], ms[2 * e + 1]);
          const float2 lo = x[e], hi = x[e + H];
          x[e] = fma2(lo, c, mul2(hi, minus));
          x[e + H] = fma2(lo, s, mul2(hi, c));
        }
      }
    } else {
      float* row = s_row[warp * kTokens + slot];
#pragma unroll
      for (int e = 0; e < N; ++e) *reinterpret_cast<float2*>(row + d0 + 2 * e) = x[e];
      __syncwarp();
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        const int d = d0 + e;
        if (d < 2 * a.pairs) {
          float& mine = e & 1 ? x[e / 2].y : x[e / 2].x;
          mine = fmaf(mine, cs[e], row[d < a.pairs ? d + a.pairs : d - a.pairs] * sn[e]);
        }
      }
      __syncwarp();
    }
  };
  // one byte a value, at the row's first byte
  auto store8 = [&](uint8_t* to, const uint32_t (&code)[N / 2]) {
    if constexpr (!kIsSplit) {
      store_words<N / 2>(to + d0, code);
    } else {
      uint32_t lo[N / 4], hi[N / 4];
#pragma unroll
      for (int e = 0; e < N / 4; ++e) lo[e] = code[e], hi[e] = code[N / 4 + e];
      store_words<N / 4>(to + d0, lo);
      store_words<N / 4>(to + d1, hi);
    }
  };
  // NVFP4 codes and scales of a row, from its slot's first byte
  auto store4 = [&](uint8_t* to, const float2 (&x)[N], float scale, float scale6) {
    if constexpr (!kIsSplit) {
      uint32_t code[N / 4], s;
      encode_nvfp4<N>(x, scale, scale6, code, &s);
      if (live) {
        store_words<N / 4>(to + off * (kD / 2) + d0 / 2, code);
        if (d0 % 16 == 0) to[kFp4Codes + off * 8 + d0 / 16] = (uint8_t)s;
      }
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float2 y[H];
#pragma unroll
        for (int e = 0; e < H; ++e) y[e] = x[half * H + e];
        const int d = half ? d1 : d0;
        uint32_t code[1], s;
        encode_nvfp4<H>(y, scale, scale6, code, &s);
        if (live) {
          if constexpr (H == 4) *reinterpret_cast<uint32_t*>(to + off * (kD / 2) + d / 2) = code[0];
          else *reinterpret_cast<uint16_t*>(to + off * (kD / 2) + d / 2) = (uint16_t)code[0];
          if (d % 16 == 0) to[kFp4Codes + off * 8 + d / 16] = (uint8_t)s;
        }
      }
    }
  };
  uint8_t* const q_to = static_cast<uint8_t*>(a.q_out) + t * a.Hq * (a.q_bf16 ? 2 * kD : kD);
  uint8_t* const k_page = a.pool + s_page[i] + (kFp4 ? 0 : off * (2 * kD));
  const int64_t head_bytes = kFp4 ? kFp4PageHead : kPage * 2 * kD;
  auto handle = [&](int r, const uint32_t (&raw)[8]) {
    float2 x[N];
    unpack<T>(raw, x);
    if (r >= v0) {
      uint8_t* to = k_page + (r - v0) * head_bytes;
      if constexpr (kFp4) {
        store4(to + kFp4Slot, x, a.v_scale, p.v6);
      } else {
        uint32_t code[N / 2];
        encode_e4m3<N, true>(x, p.v, code);
        if (live) store8(to + kD, code);
      }
      return;
    }
    const bool is_q = r < k0;
    if (r == k0 && a.k_norm) weights(s_norm[1]);
    turn(x, (is_q ? a.q_norm : a.k_norm) != nullptr);
    if ((is_q && a.q_bf16) || (!is_q && kFp4)) {
      if (!is_q) {
        store4(k_page + (r - k0) * head_bytes, x, a.k_scale, p.k6);
      } else {
        uint32_t o[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[e].x, x[e].y);
          o[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        uint16_t* to = reinterpret_cast<uint16_t*>(q_to) + r * kD;
        if (live) {
#pragma unroll
          for (int e = 0; e < N; e += H) {
            uint32_t* at = reinterpret_cast<uint32_t*>(to + (e ? d1 : d0));
            if constexpr (H == 4) *reinterpret_cast<uint4*>(at) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            else *reinterpret_cast<uint2*>(at) = make_uint2(o[e], o[e + 1]);
          }
        }
      }
      return;
    }
    // E4M3 of Q, or of K: of a product with the reciprocal, off by 2^-23 of itself
    // at most.  Where a value was normalised or turned that is one rounding more
    // among its others; where it was not, it is the only one, and its code can be
    // the neighbour of the true quotient's where that lies this near to the middle
    // of two (of bf16 and fp16 values, by ten usual scales, none does).
    const float m = is_q ? p.q_inverse : p.k_inverse;
    uint32_t code[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e)
      code[e] = four_e4m3(mul2(x[2 * e], make_float2(m, m)), mul2(x[2 * e + 1], make_float2(m, m)));
    if (live) store8(is_q ? q_to + r * kD : k_page + (r - k0) * head_bytes, code);
  };
  for (int r = r_first; r < r_end; r += kInFlight) {
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      if (r + k < r_end) handle(r + k, w[k]);
      load(w[k]);
    }
  }
}

template <typename T, bool kFp4>
cudaError_t launch_type(const RopeArgs& a, cudaStream_t stream) {
  constexpr int kTokens = 32 * kVals<T> / kD;  // of a warp
  const int64_t rows = a.Hq + 2 * a.Hkv, groups = ceil_div(a.T, kTokens);
  RopeParams p;
  p.q_inverse = 1.f / a.q_scale, p.k_inverse = 1.f / a.k_scale;
  p.v = recip_of(a.v_scale);
  p.k6 = 6.f * a.k_scale, p.v6 = 6.f * a.v_scale;
  // Whole rounds of the GPU's places take all rows of their tokens; the tokens of
  // the last round share its places, so that it is one round (16 k tokens x (32 +
  // 2 x 8) heads to E4M3, 1.35 rounds: 78 us, by one chunk a token 89; 4096
  // tokens, 0.34: 28, by chunks that come to just over one round 34).
  const int64_t places = (int64_t)num_sms() * ctas_of_sm(kFp4) * kRopeWarps;
  const int64_t whole = groups / places * places, rest = groups - whole;
  const int run = (int)ceil_div(rows, std::min(rows, rest > 0 ? places / rest : 1));
  p.part[0] = {0, 0, 1, (int)rows};
  p.part[1] = {(int)(whole / kRopeWarps), (int)whole, (int)ceil_div(rows, run), run};
  const int64_t es = sizeof(T);
  auto on32 = [&](const void* x, int64_t token, int64_t head) {
    return reinterpret_cast<uintptr_t>(x) % 32 == 0 && token * es % 32 == 0 && head * es % 32 == 0;
  };
  p.q_wide = on32(a.q, a.q_token, a.q_head);
  p.kv_wide = on32(a.k, a.k_token, a.k_head) && on32(a.v, a.v_token, a.v_head);
  const int64_t grid = p.part[1].cta + ceil_div(rest * p.part[1].chunks, kRopeWarps);
  auto run_it = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kRopeThreads), 0, stream, a, p);
  };
  if (a.interleaved || a.pairs == 0) return run_it(rope_kernel<T, kFp4, kNeighbours>);
  // whole pieces, and for NVFP4 whole blocks of 16 in a lane and its neighbours
  if (a.pairs % std::max<int>(kVals<T> / 2, kFp4 ? 16 : 0) == 0) return run_it(rope_kernel<T, kFp4, kSplit>);
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
