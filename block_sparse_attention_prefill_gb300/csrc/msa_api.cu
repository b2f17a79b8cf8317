// The C ABI of libmsa (declared in include/msa.h): host-side argument
// checks, workspace layout and the launch sequence of each call.  Nothing
// here allocates device memory or synchronises, except msa_read_status /
// msa_read_counters, which are documented to synchronise.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <mutex>

#include "common.cuh"

namespace msa {

namespace {
std::atomic<uint64_t> g_test_wait_ns{0};
}  // namespace

uint64_t pipeline_wait_limit_ns() {
  const uint64_t t = g_test_wait_ns.load(std::memory_order_relaxed);
  return t ? t : kWaitLimitNs;
}

int num_sms() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev < 0 || dev >= 64) dev = 0;
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) !=
            cudaSuccess || n <= 0)
      n = 1;
    cached[dev] = n;
  }
  return cached[dev];
}

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kI32Max = 2147483647;
constexpr int64_t kFp4PageBytes = MSA_NVFP4_PAGE_HEAD_BYTES;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// Carves one workspace into 256-byte aligned pieces (or just measures).
struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  template <typename T>
  T* take(int64_t count) {
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off = align_up(off + (size_t)count * sizeof(T));
    return p;
  }
};

struct PlanShape {
  int64_t B, T, Hq, Hkv, R, max_q, G, C, W, rows, ntiles, max_nnz, max_work;
};

int plan_shape(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t R,
               int64_t max_q, PlanShape* s) {
  if (B < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || R < 0 || max_q < 0)
    return MSA_ERR_SHAPE;
  if (Hq % Hkv != 0) return MSA_ERR_UNSUPPORTED;
  const int64_t G = Hq / Hkv;
  if (G < 1 || G > kTileM || Hkv > 127) return MSA_ERR_UNSUPPORTED;
  s->B = B;
  s->T = T;
  s->Hq = Hq;
  s->Hkv = Hkv;
  s->R = R;
  s->max_q = max_q;
  s->G = G;
  s->C = kTileM / G;
  s->W = 4 * ceil_div(max_q, 128);  // 32-bit words, a multiple of 4
  s->rows = Hkv * R;
  s->ntiles = ceil_div(s->rows, plan_tile_rows(s->rows, s->W));
  s->max_nnz = T * Hkv * kTopK;
  s->max_work = ceil_div(s->max_nnz, s->C) + std::min(s->rows, s->max_nnz);
  // every index the kernels form must fit in int32
  if (s->rows >= kI32Max || s->max_nnz >= kI32Max || s->max_work >= kI32Max ||
      T * Hq >= kI32Max / kTopK || B >= kI32Max / 2 ||
      (double)s->rows * (double)s->W * 4.0 > 9.0e15)
    return MSA_ERR_SHAPE;
  return MSA_OK;
}

// One work record: an int4 header plus one int4 per token of the chunk.
int64_t record_bytes(const PlanShape& s) { return 16 * (1 + s.C); }

// Lays out the plan workspace; with base == nullptr only the size counts.
size_t plan_layout(const PlanShape& s, void* base, msa_plan_t* pl) {
  Carver c(base);
  int32_t* req_off = c.take<int32_t>(s.B + 1);
  uint32_t* bitmap = c.take<uint32_t>(s.rows * s.W);
  int32_t* word_pre = c.take<int32_t>(s.rows * s.W);
  int32_t* row_cnt = c.take<int32_t>(s.rows);
  int32_t* row_loc = c.take<int32_t>(2 * s.rows);
  uint64_t* tile_state = c.take<uint64_t>(s.ntiles);
  int32_t* row_ptr = c.take<int32_t>(s.rows + 1);
  int32_t* q_idx = c.take<int32_t>(s.max_nnz);
  uint8_t* slot = c.take<uint8_t>(s.max_nnz);
  int32_t* work = c.take<int32_t>(4 * s.max_work);
  char* records = c.take<char>(s.max_work * record_bytes(s));
  int32_t* counters = c.take<int32_t>(4);
  uint16_t* slot_mask = c.take<uint16_t>(s.T * s.Hkv);
  uint32_t* status = c.take<uint32_t>(1);
  if (pl) {
    pl->req_off = req_off;
    pl->bitmap = bitmap;
    pl->word_pre = word_pre;
    pl->row_cnt = row_cnt;
    pl->row_loc = row_loc;
    pl->tile_state = tile_state;
    pl->records = records;
    pl->record_bytes = record_bytes(s);
    pl->row_ptr = row_ptr;
    pl->q_idx = q_idx;
    pl->slot = slot;
    pl->work = work;
    pl->counters = counters;
    pl->slot_mask = slot_mask;
    pl->status = status;
  }
  return c.off;
}

struct PartialBufs {
  uint8_t* o = nullptr;
  uint8_t* big = nullptr;
  float* lse = nullptr;
  float* vscale = nullptr;
};

// The prefill workspace: v_scale, then per (token, query head, top-k slot)
// a 128-byte E4M3 partial row, its lse, and a 256-byte bf16 overflow row
// (written only for halves of large magnitude).
size_t prefill_layout(int64_t T, int64_t Hq, void* base, PartialBufs* b) {
  Carver c(base);
  float* vs = c.take<float>(1);
  uint8_t* po = c.take<uint8_t>(T * Hq * kTopK * kD);
  float* pl = c.take<float>(T * Hq * kTopK);
  uint8_t* pb = c.take<uint8_t>(T * Hq * kTopK * 2 * kD);
  if (b) {
    b->o = po;
    b->big = pb;
    b->lse = pl;
    b->vscale = vs;
  }
  return c.off;
}

bool aligned(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

int cuda_rc(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }

// topk_hkv / h_begin: the KV heads of topk's layout and the first of this
// call's Hkv among them (a head shard; topk_hkv == Hkv, h_begin == 0 else).
int plan_impl(const int32_t* topk, const int32_t* cu_q, const int32_t* cu_k,
              const int32_t* block_table, int64_t bt_stride, int64_t num_pages,
              int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t R,
              int64_t max_q, int64_t max_k, void* ws, size_t ws_bytes,
              msa_plan_t* plan, cudaStream_t stream, int64_t topk_hkv = -1,
              int64_t h_begin = 0) {
  if (!plan) return MSA_ERR_NULL;
  PlanShape s;
  int rc = plan_shape(B, T, Hq, Hkv, R, max_q, &s);
  if (rc) return rc;
  if (topk_hkv < 0) topk_hkv = Hkv;
  if (h_begin < 0 || h_begin + Hkv > topk_hkv || topk_hkv > 127 ||
      T * topk_hkv >= kI32Max / kTopK)
    return MSA_ERR_SHAPE;
  if (max_k < 0 || max_k > kI32Max || num_pages < 0 || bt_stride < 0 ||
      max_q > max_k)
    return MSA_ERR_SHAPE;
  if (ceil_div(max_k, kPage) > (1 << 24)) return MSA_ERR_SHAPE;
  if (!cu_q || !cu_k) return MSA_ERR_NULL;
  if (T > 0 && (!topk || !block_table)) return MSA_ERR_NULL;
  if (B > 0 && R > 0 && bt_stride < 1) return MSA_ERR_SHAPE;
  // a request of max_k keys has ceil(max_k / 128) logical pages: its
  // block_table row must hold them
  if (B > 0 && bt_stride < ceil_div(max_k, kPage)) return MSA_ERR_SHAPE;
  if (!aligned(topk, 4) || !aligned(cu_q, 4) || !aligned(cu_k, 4) ||
      !aligned(block_table, 4))
    return MSA_ERR_ALIGN;
  const size_t need = plan_layout(s, nullptr, nullptr);
  if (!ws || ws_bytes < need) return MSA_ERR_WORKSPACE;
  if (!aligned(ws, kAlign)) return MSA_ERR_ALIGN;
  std::memset(plan, 0, sizeof(*plan));
  plan->B = B;
  plan->T = T;
  plan->Hq = Hq;
  plan->Hkv = Hkv;
  plan->total_rows = R;
  plan->max_seqlen_q = max_q;
  plan->max_seqlen_k = max_k;
  plan->num_pages = num_pages;
  plan->bt_stride = bt_stride;
  plan->bitmap_words = s.W;
  plan->chunk_tokens = s.C;
  plan->max_nnz = s.max_nnz;
  plan->max_work = s.max_work;
  plan->rows = s.rows;
  plan->cu_seqlens_q = cu_q;
  plan->cu_seqlens_k = cu_k;
  plan_layout(s, ws, plan);
  return cuda_rc(launch_plan(*plan, topk, block_table, stream, (int)topk_hkv, (int)h_begin));
}

int attention_impl(const uint8_t* q, const uint8_t* kv, int64_t num_pages,
                   float q_scale, float k_scale, float v_scale,
                   float softmax_scale, const int32_t* block_table,
                   int64_t bt_stride, const msa_plan_t* plan, void* ws,
                   size_t ws_bytes, cudaStream_t stream,
                   int kv_format = MSA_KV_E4M3, bool q_bf16 = false) {
  if (!plan) return MSA_ERR_NULL;
  const int64_t T = plan->T, Hq = plan->Hq;
  if (T == 0) return MSA_OK;
  if (!q || !kv || !block_table) return MSA_ERR_NULL;
  if (num_pages != plan->num_pages || bt_stride != plan->bt_stride)
    return MSA_ERR_SHAPE;
  if (num_pages * plan->Hkv * kPage >= kI32Max) return MSA_ERR_SHAPE;
  if (!(q_scale > 0.f) || !(k_scale > 0.f) || !(v_scale > 0.f) ||
      !(softmax_scale > 0.f) || !std::isfinite(q_scale * k_scale * softmax_scale))
    return MSA_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(kv, 16)) return MSA_ERR_ALIGN;
  const size_t need = prefill_layout(T, Hq, nullptr, nullptr);
  if (!ws || ws_bytes < need) return MSA_ERR_WORKSPACE;
  if (!aligned(ws, kAlign)) return MSA_ERR_ALIGN;
  AttnArgs a;
  a.q = q;
  a.kv = kv;
  a.num_pages = num_pages;
  a.score_log2 = (float)((double)q_scale * (double)k_scale *
                         (double)softmax_scale * 1.4426950408889634074);
  a.v_scale = v_scale;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.plan = plan;
  a.kv_format = kv_format;
  a.q_bf16 = q_bf16 ? 1 : 0;
  PartialBufs pb;
  prefill_layout(T, Hq, ws, &pb);
  a.part_o = pb.o;
  a.part_big = pb.big;
  a.part_lse = pb.lse;
  a.part_vscale = pb.vscale;
  if (num_pages == 0) return MSA_OK;
  return cuda_rc(launch_attention(a, stream));
}

int prefill_combine_impl(const msa_plan_t* plan, void* ws, size_t ws_bytes,
                         uint16_t* out, float* lse, cudaStream_t stream) {
  if (!plan) return MSA_ERR_NULL;
  const int64_t T = plan->T, Hq = plan->Hq;
  if (T == 0) return MSA_OK;
  if (!out) return MSA_ERR_NULL;
  if (!aligned(out, 8) || !aligned(lse, 4)) return MSA_ERR_ALIGN;
  const size_t need = prefill_layout(T, Hq, nullptr, nullptr);
  if (!ws || ws_bytes < need) return MSA_ERR_WORKSPACE;
  if (!aligned(ws, kAlign)) return MSA_ERR_ALIGN;
  PartialBufs pb;
  prefill_layout(T, Hq, ws, &pb);
  return cuda_rc(launch_combine_attn(pb.o, pb.big, pb.lse, pb.vscale, plan->slot_mask,
                                     Hq / plan->Hkv, T * Hq, out, lse, stream));
}

int prefill_impl(const uint8_t* q, const uint8_t* kv, int64_t num_pages,
                 float q_scale, float k_scale, float v_scale,
                 float softmax_scale, const int32_t* block_table,
                 int64_t bt_stride, const msa_plan_t* plan, void* ws,
                 size_t ws_bytes, uint16_t* out, float* lse,
                 cudaStream_t stream, int kv_format = MSA_KV_E4M3,
                 bool q_bf16 = false) {
  if (!plan) return MSA_ERR_NULL;
  if (plan->T == 0) return MSA_OK;
  if (!out) return MSA_ERR_NULL;
  if (!aligned(out, 8) || !aligned(lse, 4)) return MSA_ERR_ALIGN;
  int rc = attention_impl(q, kv, num_pages, q_scale, k_scale, v_scale,
                          softmax_scale, block_table, bt_stride, plan, ws,
                          ws_bytes, stream, kv_format, q_bf16);
  if (rc) return rc;
  return prefill_combine_impl(plan, ws, ws_bytes, out, lse, stream);
}

// k and v of a cache write or read: 16-byte aligned rows of 128 values with
// token and head strides (in elements) that keep them aligned.
int check_rows(const void* p, int64_t token, int64_t head, int64_t T, int64_t Hkv, int64_t es) {
  if (!p) return MSA_ERR_NULL;
  if (token < 0 || head < 0) return MSA_ERR_SHAPE;
  if (!aligned(p, 16) || (T > 1 && token * es % 16) || (Hkv > 1 && head * es % 16))
    return MSA_ERR_ALIGN;
  return MSA_OK;
}

int kv_cache_impl(KvCacheArgs a, int64_t B, int64_t Hkv, const void* lens, cudaStream_t st) {
  if (a.dtype != MSA_DTYPE_F32 && a.dtype != MSA_DTYPE_BF16 && a.dtype != MSA_DTYPE_F16)
    return MSA_ERR_UNSUPPORTED;
  if (B < 0 || B >= kI32Max / 2 || a.T < 0 || a.T >= kI32Max || Hkv < 1 || Hkv > 127 ||
      a.num_pages < 0 || a.num_pages >= kI32Max || a.bt_stride < 0 || a.bt_stride > (1 << 24))
    return MSA_ERR_SHAPE;
  if (!(a.k_scale > 0.f) || !(a.v_scale > 0.f) || !std::isfinite(a.k_scale) ||
      !std::isfinite(a.v_scale))
    return MSA_ERR_SHAPE;
  if (a.write && a.fp4 && (!std::isfinite(6.f * a.k_scale) || !std::isfinite(6.f * a.v_scale)))
    return MSA_ERR_SHAPE;
  if (B == 0 || a.T == 0) return MSA_OK;
  if (!a.pool || !a.block_table || !a.cu || (a.write && !lens)) return MSA_ERR_NULL;
  const int64_t es = a.dtype == MSA_DTYPE_F32 ? 4 : 2;
  int rc = check_rows(a.k, a.k_token, a.k_head, a.T, Hkv, es);
  if (rc) return rc;
  rc = check_rows(a.v, a.v_token, a.v_head, a.T, Hkv, es);
  if (rc) return rc;
  if (!aligned(a.pool, 16) || !aligned(a.block_table, 4) || !aligned(a.cu, 4) ||
      !aligned(a.cu_k, 4) || !aligned(a.starts, 4) || !aligned(a.status, 4))
    return MSA_ERR_ALIGN;
  a.B = (int)B;
  a.Hkv = (int)Hkv;
  return cuda_rc(launch_kv_cache(a, st));
}

int kv_write_impl(const void* k, int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                  int64_t v_head, int dtype, uint8_t* pool, int64_t num_pages, float k_scale,
                  float v_scale, const int32_t* block_table, int64_t bt_stride,
                  const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t T, int64_t Hkv,
                  uint32_t* status, void* stream, bool fp4) {
  KvCacheArgs a = {};
  a.k = const_cast<void*>(k);
  a.v = const_cast<void*>(v);
  a.k_token = k_token, a.k_head = k_head, a.v_token = v_token, a.v_head = v_head;
  a.dtype = dtype;
  a.pool = pool;
  a.num_pages = num_pages;
  a.k_scale = k_scale, a.v_scale = v_scale;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.cu = cu_q;
  a.cu_k = cu_k;
  a.T = T;
  a.status = status;
  a.fp4 = fp4;
  a.write = true;
  return kv_cache_impl(a, B, Hkv, cu_k, static_cast<cudaStream_t>(stream));
}

int kv_read_impl(const uint8_t* pool, int64_t num_pages, float k_scale, float v_scale,
                 const int32_t* block_table, int64_t bt_stride, const int32_t* cu,
                 const int32_t* starts, int64_t B, int64_t T, int64_t Hkv, void* k,
                 int64_t k_token, int64_t k_head, void* v, int64_t v_token, int64_t v_head,
                 int dtype, uint32_t* status, void* stream, bool fp4) {
  KvCacheArgs a = {};
  a.k = k;
  a.v = v;
  a.k_token = k_token, a.k_head = k_head, a.v_token = v_token, a.v_head = v_head;
  a.dtype = dtype;
  a.pool = const_cast<uint8_t*>(pool);
  a.num_pages = num_pages;
  a.k_scale = k_scale, a.v_scale = v_scale;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.cu = cu;
  a.starts = starts;
  a.T = T;
  a.status = status;
  a.fp4 = fp4;
  a.write = false;
  return kv_cache_impl(a, B, Hkv, nullptr, static_cast<cudaStream_t>(stream));
}

// 1 / (2 pi) modulo 2^-128 as two words of 64 bits behind the point, and the
// next 64 bits: 1 / 2 pi = 0.28BE60DB9391054A 7F09D5F47D4D3770 36D8A5664F10E410 ...
// (hexadecimal).
constexpr uint64_t kTurn[3] = {0x28BE60DB9391054Aull, 0x7F09D5F47D4D3770ull,
                               0x36D8A5664F10E410ull};

// f / 2 pi modulo 1 in steps of 2^-64, rounded to nearest: f = m 2^e with a
// whole number m of 53 bits, times the 192 bits above in whole numbers.  The
// product's error, m 2^(e - 192), is below 2^-100 for |f| < 2^32.
bool turns_of(double f, uint64_t* out) {
  if (!std::isfinite(f) || std::fabs(f) >= 4294967296.0) return false;
  int e;
  const double frac = std::frexp(std::fabs(f), &e);
  const uint64_t m = (uint64_t)std::ldexp(frac, 53);
  e -= 53;  // at most -21
  // w[0]: whole turns (m's upper part), w[1 .. 3] behind the point
  uint64_t w[4];
  unsigned __int128 carry = 0;
  for (int i = 2; i >= 0; --i) {
    carry += (unsigned __int128)m * kTurn[i];
    w[i + 1] = (uint64_t)carry;
    carry >>= 64;
  }
  w[0] = (uint64_t)carry;
  // shift right by -e bits; what falls off below 2^-64 turns decides the rounding
  int s = -e;
  while (s >= 64) {
    for (int i = 3; i > 0; --i) w[i] = w[i - 1];
    w[0] = 0;
    s -= 64;
    if (-e - s >= 256) break;
  }
  if (-e - s >= 256) {
    for (uint64_t& x : w) x = 0;
    s = 0;
  }
  if (s > 0)
    for (int i = 3; i >= 0; --i) w[i] = (w[i] >> s) | (i > 0 ? w[i - 1] << (64 - s) : 0);
  const uint64_t turn = w[1] + (w[2] >> 63);
  *out = f < 0 ? 0 - turn : turn;
  return true;
}

int rope_write_impl(const msa_rope_t* rope, RopeArgs a, int64_t B, int64_t Hq, int64_t Hkv,
                    cudaStream_t st) {
  if (!rope) return MSA_ERR_NULL;
  if (a.dtype != MSA_DTYPE_F32 && a.dtype != MSA_DTYPE_BF16 && a.dtype != MSA_DTYPE_F16)
    return MSA_ERR_UNSUPPORTED;
  if (rope->pairs < 0 || rope->pairs > MSA_ROPE_MAX_PAIRS || rope->axes < 1 ||
      rope->axes > MSA_ROPE_MAX_AXES || !(rope->eps >= 0.0) || !std::isfinite((float)rope->eps))
    return MSA_ERR_SHAPE;
  for (int64_t j = 0; j < rope->pairs; ++j)
    if (rope->axis[j] >= rope->axes) return MSA_ERR_SHAPE;
  if (B < 0 || B >= kI32Max / 2 || a.T < 0 || a.T >= kI32Max || Hkv < 1 || Hkv > 127 || Hq < 0 ||
      Hq > 127 * kTileM || a.num_pages < 0 || a.num_pages >= kI32Max || a.bt_stride < 0 ||
      a.bt_stride > (1 << 24))
    return MSA_ERR_SHAPE;
  if (!(a.k_scale > 0.f) || !(a.v_scale > 0.f) || !std::isfinite(a.k_scale) ||
      !std::isfinite(a.v_scale))
    return MSA_ERR_SHAPE;
  if (Hq > 0 && !a.q_bf16 && (!(a.q_scale > 0.f) || !std::isfinite(a.q_scale)))
    return MSA_ERR_SHAPE;
  if (a.fp4 && (!std::isfinite(6.f * a.k_scale) || !std::isfinite(6.f * a.v_scale)))
    return MSA_ERR_SHAPE;
  // E4M3 codes of Q and K are of products with these
  if ((Hq > 0 && !a.q_bf16 && !std::isfinite(1.f / a.q_scale)) ||
      (!a.fp4 && !std::isfinite(1.f / a.k_scale)))
    return MSA_ERR_SHAPE;
  if (B == 0 || a.T == 0) return MSA_OK;
  if (!a.pool || !a.block_table || !a.cu || !a.cu_k || (Hq > 0 && !a.q_out)) return MSA_ERR_NULL;
  const int64_t es = a.dtype == MSA_DTYPE_F32 ? 4 : 2;
  int rc = Hq > 0 ? check_rows(a.q, a.q_token, a.q_head, a.T, Hq, es) : MSA_OK;
  if (!rc) rc = check_rows(a.k, a.k_token, a.k_head, a.T, Hkv, es);
  if (!rc) rc = check_rows(a.v, a.v_token, a.v_head, a.T, Hkv, es);
  if (rc) return rc;
  if (!aligned(a.pool, 16) || !aligned(a.q_out, 16) || !aligned(a.block_table, 4) ||
      !aligned(a.cu, 4) || !aligned(a.cu_k, 4) || !aligned(a.positions, 4) ||
      !aligned(a.status, 4) || !aligned(rope->q_norm, 4) || !aligned(rope->k_norm, 4))
    return MSA_ERR_ALIGN;
  a.B = (int)B;
  a.Hq = (int)Hq;
  a.Hkv = (int)Hkv;
  a.q_norm = rope->q_norm;
  a.k_norm = rope->k_norm;
  a.eps = (float)rope->eps;
  a.pairs = (int)rope->pairs;
  a.axes = (int)rope->axes;
  a.interleaved = rope->interleaved != 0;
  std::copy_n(rope->turns, MSA_ROPE_MAX_PAIRS, a.turns);
  std::copy_n(rope->axis, MSA_ROPE_MAX_PAIRS, a.axis);
  return cuda_rc(launch_rope_write(a, st));
}

int verify_impl(const VerifyArgs& a, bool greedy, cudaStream_t st) {
  if (a.dtype != MSA_DTYPE_F32 && a.dtype != MSA_DTYPE_BF16 && a.dtype != MSA_DTYPE_F16)
    return MSA_ERR_UNSUPPORTED;
  if (a.B < 0 || a.B > kI32Max / 64 || a.n < 1 || a.n > MSA_VERIFY_MAX_TOKENS || a.V < 1 ||
      a.V >= MSA_VERIFY_MAX_VOCAB || a.t_req < 0 || a.t_row < 0 || a.d_req < 0 || a.d_row < 0)
    return MSA_ERR_SHAPE;
  if (a.B == 0) return MSA_OK;
  if (!a.target || !a.tokens || !a.accepted || (a.n > 1 && !a.tokens_in) || (!greedy && !a.u))
    return MSA_ERR_NULL;
  const size_t es = a.dtype == MSA_DTYPE_F32 ? 4 : 2;
  if (!aligned(a.target, es) || !aligned(a.draft, es) || !aligned(a.tokens_in, 4) ||
      !aligned(a.u, 4) || !aligned(a.counts, 4) || !aligned(a.tokens, 4) ||
      !aligned(a.accepted, 4))
    return MSA_ERR_ALIGN;
  return cuda_rc(greedy ? launch_verify_greedy(a, st) : launch_verify(a, st));
}

// Host-side checks of the shared-prefix attention's sizes.
int prefix_shape(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t prefix, int64_t max_q,
                 int64_t max_k, size_t* bytes) {
  if (B < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || prefix < 0 || max_q < 0 || max_k < max_q ||
      max_k > (1 << 30) || prefix > max_k / kPage || B >= kI32Max / 2)
    return MSA_ERR_SHAPE;
  if (Hq % Hkv != 0 || Hq / Hkv > kTileM || Hkv > 127) return MSA_ERR_UNSUPPORTED;
  if (T >= kI32Max / kTopK || T * Hq >= kI32Max / kTopK) return MSA_ERR_SHAPE;
  *bytes = prefix_workspace(B, T, Hq, Hkv, prefix, max_k);
  return *bytes ? MSA_OK : MSA_ERR_SHAPE;
}

// The calls of the shared-prefix attention, causal or (mask) of trees.
int prefix_attention_impl(PrefixArgs a, float q_scale, float k_scale, float softmax_scale,
                          void* workspace, size_t workspace_bytes, cudaStream_t st) {
  size_t need = 0;
  int rc = prefix_shape(a.B, a.T, a.Hq, a.Hkv, a.prefix_pages, a.max_q, a.max_k, &need);
  if (rc) return rc;
  if (a.num_pages < 0 || a.num_pages >= kI32Max || a.num_pages * a.Hkv * kPage >= kI32Max ||
      a.bt_stride < ceil_div(a.max_k, kPage) || a.bt_stride > (1 << 24))
    return MSA_ERR_SHAPE;
  // the largest score of E4M3 codes, 128 * 448^2 products, has to be finite
  const double score = (double)q_scale * (double)k_scale * (double)softmax_scale *
                       1.4426950408889634074;
  if (!(q_scale > 0.f) || !(k_scale > 0.f) || !(a.v_scale > 0.f) || !(softmax_scale > 0.f) ||
      !(score * kD * 448.0 * 448.0 < FLT_MAX) || !std::isfinite(a.v_scale))
    return MSA_ERR_SHAPE;
  if (a.B == 0 || a.T == 0) return MSA_OK;
  if (!a.q || !a.kv || !a.block_table || !a.cu_q || !a.cu_k || !a.out) return MSA_ERR_NULL;
  if (!aligned(a.q, 16) || !aligned(a.kv, 16) || !aligned(a.block_table, 4) ||
      !aligned(a.cu_q, 4) || !aligned(a.cu_k, 4) || !aligned(a.out, 8) || !aligned(a.lse, 4) ||
      !aligned(a.mask, 4) || !aligned(a.status, 4))
    return MSA_ERR_ALIGN;
  if (!workspace || workspace_bytes < need) return MSA_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return MSA_ERR_ALIGN;
  // never 0, by which a masked score of -inf would become NaN
  a.score_log2 = std::max((float)score, FLT_MIN);
  return cuda_rc(launch_prefix_attention(a, workspace, st));
}

int tree_lengths(int64_t B, int64_t T, int64_t max_q) {
  return B < 0 || B >= kI32Max / 2 || T < 0 || T >= kI32Max / kTopK || max_q < 0 ||
                 max_q > MSA_TREE_MAX_TOKENS
             ? MSA_ERR_SHAPE
             : MSA_OK;
}

int tree_accept_impl(TreeAcceptArgs a, uint8_t* const* pools, int64_t layers, int64_t Hkv,
                     int64_t B, int64_t max_q, cudaStream_t st) {
  int rc = tree_lengths(B, a.T, max_q);
  if (rc) return rc;
  if (layers < 0 || layers > MSA_TREE_MAX_LAYERS || (layers > 0 && (Hkv < 1 || Hkv > 127)) ||
      a.num_pages < 0 || a.num_pages >= kI32Max || a.bt_stride < 0 || a.bt_stride > (1 << 24))
    return MSA_ERR_SHAPE;
  if (B == 0) return MSA_OK;
  if (!a.accepted || (max_q > 0 && !a.tokens) || !a.cu_q || !a.cu_k) return MSA_ERR_NULL;
  if (a.T > 0 && (!a.drafts || !a.parents || !a.chosen)) return MSA_ERR_NULL;
  if (layers > 0 && (!pools || !a.block_table)) return MSA_ERR_NULL;
  if (!aligned(a.drafts, 4) || !aligned(a.parents, 4) || !aligned(a.chosen, 4) ||
      !aligned(a.cu_q, 4) || !aligned(a.cu_k, 4) || !aligned(a.block_table, 4) ||
      !aligned(a.tokens, 4) || !aligned(a.accepted, 4) || !aligned(a.path, 4) ||
      !aligned(a.status, 4))
    return MSA_ERR_ALIGN;
  uintptr_t at[MSA_TREE_MAX_LAYERS];
  for (int64_t i = 0; i < layers; ++i) {
    if (!pools[i]) return MSA_ERR_NULL;
    if (!aligned(pools[i], 16)) return MSA_ERR_ALIGN;
    a.pools[i] = pools[i];
    at[i] = reinterpret_cast<uintptr_t>(pools[i]);
  }
  // rows of a pool given twice would be moved by two at once
  std::sort(at, at + layers);
  const uint64_t bytes = (uint64_t)a.num_pages * (uint64_t)Hkv *
                         (a.fp4 ? kFp4PageBytes : kPage * 2 * kD);
  for (int64_t i = 1; i < layers; ++i)
    if (at[i] - at[i - 1] < std::max<uint64_t>(bytes, 1)) return MSA_ERR_SHAPE;
  a.B = (int)B;
  a.max_q = (int)max_q;
  a.Hkv = (int)Hkv;
  a.layers = (int)layers;
  return cuda_rc(launch_tree_accept(a, st));
}

struct DecodeLayout {
  int64_t R;
  size_t cu_bytes, plan_bytes, prefill_bytes, total;
};

int decode_layout(int64_t B, int64_t n, int64_t Hq, int64_t Hkv,
                  int64_t max_k, DecodeLayout* d) {
  if (B < 0 || n < 1 || n > 8 || max_k < n || max_k > kI32Max)
    return MSA_ERR_SHAPE;
  if (B > kI32Max / 8) return MSA_ERR_SHAPE;
  d->R = B * ceil_div(max_k, kPage);
  PlanShape s;
  int rc = plan_shape(B, B * n, Hq, Hkv, d->R, n, &s);
  if (rc) return rc;
  d->cu_bytes = align_up(2 * (size_t)(B + 1) * sizeof(int32_t));
  d->plan_bytes = plan_layout(s, nullptr, nullptr);
  d->prefill_bytes = prefill_layout(B * n, Hq, nullptr, nullptr);
  d->total = d->cu_bytes + d->plan_bytes + d->prefill_bytes;
  return MSA_OK;
}

int decode_impl(const uint8_t* q, const uint8_t* kv, int64_t num_pages,
                float q_scale, float k_scale, float v_scale,
                float softmax_scale, const int32_t* topk,
                const int32_t* block_table, int64_t bt_stride,
                const int32_t* seq_lens, int64_t B, int64_t n, int64_t Hq,
                int64_t Hkv, int64_t max_seqlen_k, void* workspace,
                size_t workspace_bytes, uint16_t* out, float* lse,
                msa_plan_t* plan_out, cudaStream_t st, int kv_format) {
  DecodeLayout d;
  int rc = decode_layout(B, n, Hq, Hkv, max_seqlen_k, &d);
  if (rc) return rc;
  if (B == 0) return MSA_OK;
  if (!seq_lens) return MSA_ERR_NULL;
  if (!workspace || workspace_bytes < d.total) return MSA_ERR_WORKSPACE;
  if (!aligned(workspace, kAlign)) return MSA_ERR_ALIGN;
  char* ws = static_cast<char*>(workspace);
  int32_t* cu_q = reinterpret_cast<int32_t*>(ws);
  int32_t* cu_k = cu_q + (B + 1);
  msa_plan_t local;
  msa_plan_t* plan = plan_out ? plan_out : &local;
  // validate everything the plan checks before launching anything
  PlanShape s;
  rc = plan_shape(B, B * n, Hq, Hkv, d.R, n, &s);
  if (rc) return rc;
  if (!q || !kv || !out || !topk || !block_table) return MSA_ERR_NULL;
  if (bt_stride < 1 || bt_stride < ceil_div(max_seqlen_k, kPage) || num_pages < 0 ||
      num_pages * Hkv * kPage >= kI32Max)
    return MSA_ERR_SHAPE;
  if (!(q_scale > 0.f) || !(k_scale > 0.f) || !(v_scale > 0.f) ||
      !(softmax_scale > 0.f))
    return MSA_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(out, 8) ||
      !aligned(lse, 4) || !aligned(topk, 4) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4))
    return MSA_ERR_ALIGN;
  if (launch_decode_seqlens(seq_lens, B, n, cu_q, cu_k, st) != cudaSuccess)
    return MSA_ERR_CUDA;
  rc = plan_impl(topk, cu_q, cu_k, block_table, bt_stride, num_pages, B, B * n,
                 Hq, Hkv, d.R, n, max_seqlen_k, ws + d.cu_bytes, d.plan_bytes,
                 plan, st);
  if (rc) return rc;
  return prefill_impl(q, kv, num_pages, q_scale, k_scale, v_scale,
                      softmax_scale, block_table, bt_stride, plan,
                      ws + d.cu_bytes + d.plan_bytes, d.prefill_bytes, out,
                      lse, st, kv_format);
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

int msa_version(void) { return 100; }

const char* msa_status_string(int code) {
  switch (code) {
    case MSA_OK: return "ok";
    case MSA_ERR_SHAPE: return "a size, count or stride is out of range";
    case MSA_ERR_UNSUPPORTED: return "unsupported configuration";
    case MSA_ERR_ALIGN: return "pointer not aligned as required";
    case MSA_ERR_WORKSPACE: return "workspace missing or too small";
    case MSA_ERR_CUDA: return "a CUDA call failed";
    case MSA_ERR_NULL: return "a required pointer is NULL";
    case MSA_ERR_TOO_LARGE:
      return "problem needs more scratch than msa_decode_noalloc's fixed array";
    case MSA_ERR_BUSY:
      return "msa_decode_noalloc is already being called from another thread";
    default: return "unknown status";
  }
}

int msa_plan_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv,
                             int64_t total_rows, int64_t max_seqlen_q,
                             size_t* bytes) {
  if (!bytes) return MSA_ERR_NULL;
  PlanShape s;
  int rc = plan_shape(B, T, Hq, Hkv, total_rows, max_seqlen_q, &s);
  if (rc) return rc;
  *bytes = plan_layout(s, nullptr, nullptr);
  return MSA_OK;
}

int msa_plan(const int32_t* topk, const int32_t* cu_seqlens_q,
             const int32_t* cu_seqlens_k, const int32_t* block_table,
             int64_t bt_stride, int64_t num_pages, int64_t B, int64_t T,
             int64_t Hq, int64_t Hkv, int64_t total_rows,
             int64_t max_seqlen_q, int64_t max_seqlen_k, void* workspace,
             size_t workspace_bytes, msa_plan_t* plan, void* stream) {
  return plan_impl(topk, cu_seqlens_q, cu_seqlens_k, block_table, bt_stride,
                   num_pages, B, T, Hq, Hkv, total_rows, max_seqlen_q,
                   max_seqlen_k, workspace, workspace_bytes, plan,
                   static_cast<cudaStream_t>(stream));
}

int msa_plan_heads(const int32_t* topk, int64_t topk_hkv, int64_t h_begin,
                   const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                   const int32_t* block_table, int64_t bt_stride, int64_t num_pages,
                   int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t total_rows,
                   int64_t max_seqlen_q, int64_t max_seqlen_k, void* workspace,
                   size_t workspace_bytes, msa_plan_t* plan, void* stream) {
  return plan_impl(topk, cu_seqlens_q, cu_seqlens_k, block_table, bt_stride,
                   num_pages, B, T, Hq, Hkv, total_rows, max_seqlen_q,
                   max_seqlen_k, workspace, workspace_bytes, plan,
                   static_cast<cudaStream_t>(stream), topk_hkv, h_begin);
}

int msa_prefill_workspace_bytes(int64_t T, int64_t Hq, size_t* bytes) {
  if (!bytes) return MSA_ERR_NULL;
  if (T < 0 || Hq <= 0 || T * Hq >= kI32Max / kTopK) return MSA_ERR_SHAPE;
  *bytes = prefill_layout(T, Hq, nullptr, nullptr);
  return MSA_OK;
}

int msa_prefill(const uint8_t* q, const uint8_t* kv, int64_t num_pages,
                float q_scale, float k_scale, float v_scale,
                float softmax_scale, const int32_t* block_table,
                int64_t bt_stride, const msa_plan_t* plan, void* workspace,
                size_t workspace_bytes, uint16_t* out, float* lse,
                void* stream) {
  return prefill_impl(q, kv, num_pages, q_scale, k_scale, v_scale,
                      softmax_scale, block_table, bt_stride, plan, workspace,
                      workspace_bytes, out, lse,
                      static_cast<cudaStream_t>(stream));
}

int msa_prefill_nvfp4(const uint8_t* q, const uint8_t* kv4, int64_t num_pages,
                      float q_scale, float k_scale, float v_scale,
                      float softmax_scale, const int32_t* block_table,
                      int64_t bt_stride, const msa_plan_t* plan,
                      void* workspace, size_t workspace_bytes, uint16_t* out,
                      float* lse, void* stream) {
  return prefill_impl(q, kv4, num_pages, q_scale, k_scale, v_scale,
                      softmax_scale, block_table, bt_stride, plan, workspace,
                      workspace_bytes, out, lse,
                      static_cast<cudaStream_t>(stream), MSA_KV_NVFP4);
}

int msa_nvfp4_to_e4m3(const uint8_t* kv4, int64_t page_heads, uint8_t* kv8,
                      void* stream) {
  if (page_heads < 0 || page_heads > (int64_t(1) << 40) / kFp4PageBytes)
    return MSA_ERR_SHAPE;
  if (page_heads == 0) return MSA_OK;
  if (!kv4 || !kv8) return MSA_ERR_NULL;
  if (!aligned(kv4, 16) || !aligned(kv8, 16)) return MSA_ERR_ALIGN;
  return cuda_rc(launch_nvfp4_to_e4m3(kv4, page_heads, kv8,
                                      static_cast<cudaStream_t>(stream)));
}

int msa_prefill_attention(const uint8_t* q, const uint8_t* kv,
                          int64_t num_pages, float q_scale, float k_scale,
                          float v_scale, float softmax_scale,
                          const int32_t* block_table, int64_t bt_stride,
                          const msa_plan_t* plan, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return attention_impl(q, kv, num_pages, q_scale, k_scale, v_scale,
                        softmax_scale, block_table, bt_stride, plan, workspace,
                        workspace_bytes, static_cast<cudaStream_t>(stream));
}

int msa_prefill_attention_nvfp4(const uint8_t* q, const uint8_t* kv4,
                                int64_t num_pages, float q_scale, float k_scale,
                                float v_scale, float softmax_scale,
                                const int32_t* block_table, int64_t bt_stride,
                                const msa_plan_t* plan, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return attention_impl(q, kv4, num_pages, q_scale, k_scale, v_scale,
                        softmax_scale, block_table, bt_stride, plan, workspace,
                        workspace_bytes, static_cast<cudaStream_t>(stream),
                        MSA_KV_NVFP4);
}

int msa_prefill_bf16q(const uint16_t* q16, const uint8_t* kv, int64_t num_pages,
                      float q_scale, float k_scale, float v_scale,
                      float softmax_scale, const int32_t* block_table,
                      int64_t bt_stride, const msa_plan_t* plan,
                      void* workspace, size_t workspace_bytes, uint16_t* out,
                      float* lse, void* stream) {
  return prefill_impl(reinterpret_cast<const uint8_t*>(q16), kv, num_pages, q_scale,
                      k_scale, v_scale, softmax_scale, block_table, bt_stride, plan,
                      workspace, workspace_bytes, out, lse,
                      static_cast<cudaStream_t>(stream), MSA_KV_E4M3, true);
}

int msa_prefill_attention_bf16q(const uint16_t* q16, const uint8_t* kv,
                                int64_t num_pages, float q_scale, float k_scale,
                                float v_scale, float softmax_scale,
                                const int32_t* block_table, int64_t bt_stride,
                                const msa_plan_t* plan, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return attention_impl(reinterpret_cast<const uint8_t*>(q16), kv, num_pages, q_scale,
                        k_scale, v_scale, softmax_scale, block_table, bt_stride, plan,
                        workspace, workspace_bytes, static_cast<cudaStream_t>(stream),
                        MSA_KV_E4M3, true);
}

int msa_prefill_combine(const msa_plan_t* plan, void* workspace,
                        size_t workspace_bytes, uint16_t* out, float* lse,
                        void* stream) {
  return prefill_combine_impl(plan, workspace, workspace_bytes, out, lse,
                              static_cast<cudaStream_t>(stream));
}

int msa_combine(const void* part_o, int part_dtype, const float* part_lse,
                int64_t rows, int64_t splits, uint16_t* out, float* lse_out,
                void* stream) {
  if (rows < 0 || splits < 1 || splits > 64 || rows >= kI32Max)
    return MSA_ERR_SHAPE;
  if (part_dtype != MSA_DTYPE_F32 && part_dtype != MSA_DTYPE_BF16)
    return MSA_ERR_UNSUPPORTED;
  if (rows == 0) return MSA_OK;
  if (!part_o || !part_lse || !out) return MSA_ERR_NULL;
  if (!aligned(part_o, part_dtype == MSA_DTYPE_F32 ? 16 : 8) ||
      !aligned(part_lse, 4) || !aligned(out, 8) || !aligned(lse_out, 4))
    return MSA_ERR_ALIGN;
  return cuda_rc(launch_combine(part_o, part_dtype, part_lse, rows,
                                splits, out, lse_out,
                                static_cast<cudaStream_t>(stream)));
}

int msa_kv_write(const void* k, int64_t k_token, int64_t k_head, const void* v, int64_t v_token,
                 int64_t v_head, int dtype, uint8_t* kv, int64_t num_pages, float k_scale,
                 float v_scale, const int32_t* block_table, int64_t bt_stride,
                 const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int64_t B, int64_t T,
                 int64_t Hkv, uint32_t* status, void* stream) {
  return kv_write_impl(k, k_token, k_head, v, v_token, v_head, dtype, kv, num_pages, k_scale,
                       v_scale, block_table, bt_stride, cu_seqlens_q, cu_seqlens_k, B, T, Hkv,
                       status, stream, false);
}

int msa_kv_write_nvfp4(const void* k, int64_t k_token, int64_t k_head, const void* v,
                       int64_t v_token, int64_t v_head, int dtype, uint8_t* kv4,
                       int64_t num_pages, float k_scale, float v_scale,
                       const int32_t* block_table, int64_t bt_stride,
                       const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int64_t B,
                       int64_t T, int64_t Hkv, uint32_t* status, void* stream) {
  return kv_write_impl(k, k_token, k_head, v, v_token, v_head, dtype, kv4, num_pages, k_scale,
                       v_scale, block_table, bt_stride, cu_seqlens_q, cu_seqlens_k, B, T, Hkv,
                       status, stream, true);
}

int msa_kv_read(const uint8_t* kv, int64_t num_pages, float k_scale, float v_scale,
                const int32_t* block_table, int64_t bt_stride, const int32_t* cu_tokens,
                const int32_t* starts, int64_t B, int64_t T, int64_t Hkv, void* k,
                int64_t k_token, int64_t k_head, void* v, int64_t v_token, int64_t v_head,
                int dtype, uint32_t* status, void* stream) {
  return kv_read_impl(kv, num_pages, k_scale, v_scale, block_table, bt_stride, cu_tokens, starts,
                      B, T, Hkv, k, k_token, k_head, v, v_token, v_head, dtype, status, stream,
                      false);
}

int msa_kv_read_nvfp4(const uint8_t* kv4, int64_t num_pages, float k_scale, float v_scale,
                      const int32_t* block_table, int64_t bt_stride, const int32_t* cu_tokens,
                      const int32_t* starts, int64_t B, int64_t T, int64_t Hkv, void* k,
                      int64_t k_token, int64_t k_head, void* v, int64_t v_token, int64_t v_head,
                      int dtype, uint32_t* status, void* stream) {
  return kv_read_impl(kv4, num_pages, k_scale, v_scale, block_table, bt_stride, cu_tokens, starts,
                      B, T, Hkv, k, k_token, k_head, v, v_token, v_head, dtype, status, stream,
                      true);
}

int msa_rope_turns(const double* inv_freq, int64_t n, uint64_t* turns) {
  if (n < 0) return MSA_ERR_SHAPE;
  if (n > 0 && (!inv_freq || !turns)) return MSA_ERR_NULL;
  for (int64_t j = 0; j < n; ++j)
    if (!turns_of(inv_freq[j], turns + j)) return MSA_ERR_SHAPE;
  return MSA_OK;
}

int msa_rope_write(const msa_rope_t* rope, const int32_t* positions, const void* q,
                   int64_t q_token, int64_t q_head, const void* k, int64_t k_token,
                   int64_t k_head, const void* v, int64_t v_token, int64_t v_head, int dtype,
                   void* q_out, int q_bf16, float q_scale, uint8_t* kv, int64_t num_pages,
                   float k_scale, float v_scale, const int32_t* block_table, int64_t bt_stride,
                   const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int64_t B,
                   int64_t T, int64_t Hq, int64_t Hkv, uint32_t* status, void* stream) {
  RopeArgs a = {};
  a.q = q, a.k = k, a.v = v;
  a.q_token = q_token, a.q_head = q_head, a.k_token = k_token, a.k_head = k_head;
  a.v_token = v_token, a.v_head = v_head;
  a.dtype = dtype;
  a.q_out = q_out;
  a.q_bf16 = q_bf16 != 0;
  a.q_scale = q_scale, a.k_scale = k_scale, a.v_scale = v_scale;
  a.pool = kv;
  a.num_pages = num_pages;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.cu = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.positions = positions;
  a.T = T;
  a.status = status;
  a.fp4 = false;
  return rope_write_impl(rope, a, B, Hq, Hkv, static_cast<cudaStream_t>(stream));
}

int msa_rope_write_nvfp4(const msa_rope_t* rope, const int32_t* positions, const void* q,
                         int64_t q_token, int64_t q_head, const void* k, int64_t k_token,
                         int64_t k_head, const void* v, int64_t v_token, int64_t v_head, int dtype,
                         void* q_out, int q_bf16, float q_scale, uint8_t* kv4, int64_t num_pages,
                         float k_scale, float v_scale, const int32_t* block_table, int64_t bt_stride,
                         const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int64_t B,
                         int64_t T, int64_t Hq, int64_t Hkv, uint32_t* status, void* stream) {
  RopeArgs a = {};
  a.q = q, a.k = k, a.v = v;
  a.q_token = q_token, a.q_head = q_head, a.k_token = k_token, a.k_head = k_head;
  a.v_token = v_token, a.v_head = v_head;
  a.dtype = dtype;
  a.q_out = q_out;
  a.q_bf16 = q_bf16 != 0;
  a.q_scale = q_scale, a.k_scale = k_scale, a.v_scale = v_scale;
  a.pool = kv4;
  a.num_pages = num_pages;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.cu = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.positions = positions;
  a.T = T;
  a.status = status;
  a.fp4 = true;
  return rope_write_impl(rope, a, B, Hq, Hkv, static_cast<cudaStream_t>(stream));
}

int msa_prefix_attention_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv,
                                         int64_t prefix_pages, int64_t max_seqlen_q,
                                         int64_t max_seqlen_k, size_t* bytes) {
  if (!bytes) return MSA_ERR_NULL;
  return prefix_shape(B, T, Hq, Hkv, prefix_pages, max_seqlen_q, max_seqlen_k, bytes);
}

int msa_prefix_attention(const uint8_t* q, const uint8_t* kv, int64_t num_pages, float q_scale,
                         float k_scale, float v_scale, float softmax_scale,
                         const int32_t* block_table, int64_t bt_stride,
                         const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int64_t B,
                         int64_t T, int64_t Hq, int64_t Hkv, int64_t prefix_pages,
                         int64_t max_seqlen_q, int64_t max_seqlen_k, void* workspace,
                         size_t workspace_bytes, uint16_t* out, float* lse, uint32_t* status,
                         void* stream) {
  PrefixArgs a = {};
  a.q = q;
  a.kv = kv;
  a.num_pages = num_pages;
  a.v_scale = v_scale;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.B = B, a.T = T, a.Hq = Hq, a.Hkv = Hkv;
  a.prefix_pages = prefix_pages;
  a.max_q = max_seqlen_q, a.max_k = max_seqlen_k;
  a.out = out;
  a.lse = lse;
  a.status = status;
  return prefix_attention_impl(a, q_scale, k_scale, softmax_scale, workspace, workspace_bytes,
                               static_cast<cudaStream_t>(stream));
}

int msa_tree_mask(const int32_t* parents, const int32_t* cu_seqlens_q,
                  const int32_t* cu_seqlens_k, int64_t B, int64_t T, int64_t max_seqlen_q,
                  uint32_t* mask, int32_t* positions, uint32_t* status, void* stream) {
  int rc = tree_lengths(B, T, max_seqlen_q);
  if (rc) return rc;
  if (B == 0 || T == 0) return MSA_OK;
  if (!parents || !cu_seqlens_q || !cu_seqlens_k) return MSA_ERR_NULL;
  if (!aligned(parents, 4) || !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4) ||
      !aligned(mask, 4) || !aligned(positions, 4) || !aligned(status, 4))
    return MSA_ERR_ALIGN;
  const TreeMaskArgs a = {parents, cu_seqlens_q, cu_seqlens_k, (int)B, T, (int)max_seqlen_q,
                          (int)ceil_div(max_seqlen_q, 32), mask, positions, status};
  return cuda_rc(launch_tree_mask(a, static_cast<cudaStream_t>(stream)));
}

int msa_tree_attention(const uint8_t* q, const uint8_t* kv, int64_t num_pages, float q_scale,
                       float k_scale, float v_scale, float softmax_scale,
                       const int32_t* block_table, int64_t bt_stride,
                       const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                       const uint32_t* mask, int64_t mask_words, int64_t B, int64_t T,
                       int64_t Hq, int64_t Hkv, int64_t prefix_pages, int64_t max_seqlen_q,
                       int64_t max_seqlen_k, void* workspace, size_t workspace_bytes,
                       uint16_t* out, float* lse, uint32_t* status, void* stream) {
  int rc = tree_lengths(B, T, max_seqlen_q);
  if (rc) return rc;
  if (mask_words < ceil_div(max_seqlen_q, 32) || mask_words > (1 << 20)) return MSA_ERR_SHAPE;
  if (B > 0 && T > 0 && max_seqlen_q > 0 && !mask) return MSA_ERR_NULL;
  PrefixArgs a = {};
  a.q = q;
  a.kv = kv;
  a.num_pages = num_pages;
  a.v_scale = v_scale;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.cu_q = cu_seqlens_q;
  a.cu_k = cu_seqlens_k;
  a.B = B, a.T = T, a.Hq = Hq, a.Hkv = Hkv;
  a.prefix_pages = prefix_pages;
  a.max_q = max_seqlen_q, a.max_k = max_seqlen_k;
  a.out = out;
  a.lse = lse;
  a.status = status;
  a.mask = mask;
  a.mask_words = (int)mask_words;
  return prefix_attention_impl(a, q_scale, k_scale, softmax_scale, workspace, workspace_bytes,
                               static_cast<cudaStream_t>(stream));
}

int msa_verify(const void* target_probs, int64_t target_req, int64_t target_row,
               const void* draft_probs, int64_t draft_req, int64_t draft_row, int dtype,
               const int32_t* draft_tokens, const float* uniforms, const int32_t* num_drafts,
               int64_t B, int64_t n, int64_t V, int32_t* tokens, int32_t* accepted,
               void* stream) {
  if (n < 1 || n > MSA_VERIFY_MAX_TOKENS) return MSA_ERR_SHAPE;
  VerifyArgs a = {target_probs, target_req, target_row, n > 1 ? draft_probs : nullptr, draft_req,
                  draft_row, dtype, draft_tokens, uniforms, num_drafts, B, (int)n, V, tokens,
                  accepted};
  return verify_impl(a, false, static_cast<cudaStream_t>(stream));
}

int msa_verify_greedy(const void* target, int64_t target_req, int64_t target_row, int dtype,
                      const int32_t* draft_tokens, const int32_t* num_drafts, int64_t B,
                      int64_t n, int64_t V, int32_t* tokens, int32_t* accepted, void* stream) {
  if (n < 1 || n > MSA_VERIFY_MAX_TOKENS) return MSA_ERR_SHAPE;
  VerifyArgs a = {target, target_req, target_row, nullptr, 0, 0, dtype, draft_tokens, nullptr,
                  num_drafts, B, (int)n, V, tokens, accepted};
  return verify_impl(a, true, static_cast<cudaStream_t>(stream));
}

int msa_tree_accept(const int32_t* draft_tokens, const int32_t* parents,
                    const int32_t* chosen, const int32_t* cu_seqlens_q,
                    const int32_t* cu_seqlens_k, int64_t B, int64_t T, int64_t max_seqlen_q,
                    uint8_t* const* kv, int64_t layers, int64_t num_pages, int64_t Hkv,
                    const int32_t* block_table, int64_t bt_stride, int32_t* tokens,
                    int32_t* accepted, int32_t* path, uint32_t* status, void* stream) {
  TreeAcceptArgs a = {};
  a.drafts = draft_tokens, a.parents = parents, a.chosen = chosen;
  a.cu_q = cu_seqlens_q, a.cu_k = cu_seqlens_k;
  a.T = T;
  a.block_table = block_table;
  a.bt_stride = bt_stride, a.num_pages = num_pages;
  a.fp4 = false;
  a.tokens = tokens, a.accepted = accepted, a.path = path;
  a.status = status;
  return tree_accept_impl(a, kv, layers, Hkv, B, max_seqlen_q, static_cast<cudaStream_t>(stream));
}

int msa_tree_accept_nvfp4(const int32_t* draft_tokens, const int32_t* parents,
                          const int32_t* chosen, const int32_t* cu_seqlens_q,
                          const int32_t* cu_seqlens_k, int64_t B, int64_t T, int64_t max_seqlen_q,
                          uint8_t* const* kv4, int64_t layers, int64_t num_pages, int64_t Hkv,
                          const int32_t* block_table, int64_t bt_stride, int32_t* tokens,
                          int32_t* accepted, int32_t* path, uint32_t* status, void* stream) {
  TreeAcceptArgs a = {};
  a.drafts = draft_tokens, a.parents = parents, a.chosen = chosen;
  a.cu_q = cu_seqlens_q, a.cu_k = cu_seqlens_k;
  a.T = T;
  a.block_table = block_table;
  a.bt_stride = bt_stride, a.num_pages = num_pages;
  a.fp4 = true;
  a.tokens = tokens, a.accepted = accepted, a.path = path;
  a.status = status;
  return tree_accept_impl(a, kv4, layers, Hkv, B, max_seqlen_q, static_cast<cudaStream_t>(stream));
}

int msa_logprobs(const void* logits, int64_t row_stride, int dtype, const int32_t* tokens,
                 int64_t T, int64_t V, int64_t top, float* logprobs, int32_t* ranks,
                 float* entropy, int32_t* top_tokens, float* top_logprobs, void* stream) {
  if (dtype != MSA_DTYPE_F32 && dtype != MSA_DTYPE_BF16 && dtype != MSA_DTYPE_F16)
    return MSA_ERR_UNSUPPORTED;
  if (T < 0 || T > kI32Max / 64 || V < 1 || V >= MSA_VERIFY_MAX_VOCAB || row_stride < 0 ||
      top < 0 || top > MSA_LOGPROBS_MAX_TOP)
    return MSA_ERR_SHAPE;
  if (T == 0) return MSA_OK;
  if (!logits || (top > 0 && (!top_tokens || !top_logprobs)) || (!tokens && (logprobs || ranks)))
    return MSA_ERR_NULL;
  if (!aligned(logits, dtype == MSA_DTYPE_F32 ? 4 : 2) || !aligned(tokens, 4) ||
      !aligned(logprobs, 4) || !aligned(ranks, 4) || !aligned(entropy, 4) ||
      !aligned(top_tokens, 4) || !aligned(top_logprobs, 4))
    return MSA_ERR_ALIGN;
  const LogprobsArgs a = {logits, row_stride, dtype, tokens, T, (int)V, (int)top, logprobs, ranks,
                          entropy, top_tokens, top_logprobs};
  return cuda_rc(launch_logprobs(a, static_cast<cudaStream_t>(stream)));
}

int msa_decode_workspace_bytes(int64_t B, int64_t n, int64_t Hq, int64_t Hkv,
                               int64_t max_seqlen_k, size_t* bytes) {
  if (!bytes) return MSA_ERR_NULL;
  DecodeLayout d;
  int rc = decode_layout(B, n, Hq, Hkv, max_seqlen_k, &d);
  if (rc) return rc;
  *bytes = d.total;
  return MSA_OK;
}

int msa_decode(const uint8_t* q, const uint8_t* kv, int64_t num_pages,
               float q_scale, float k_scale, float v_scale,
               float softmax_scale, const int32_t* topk,
               const int32_t* block_table, int64_t bt_stride,
               const int32_t* seq_lens, int64_t B, int64_t n, int64_t Hq,
               int64_t Hkv, int64_t max_seqlen_k, void* workspace,
               size_t workspace_bytes, uint16_t* out, float* lse,
               msa_plan_t* plan_out, void* stream) {
  return decode_impl(q, kv, num_pages, q_scale, k_scale, v_scale,
                     softmax_scale, topk, block_table, bt_stride, seq_lens, B,
                     n, Hq, Hkv, max_seqlen_k, workspace, workspace_bytes, out,
                     lse, plan_out, static_cast<cudaStream_t>(stream),
                     MSA_KV_E4M3);
}

int msa_decode_nvfp4(const uint8_t* q, const uint8_t* kv4, int64_t num_pages,
                     float q_scale, float k_scale, float v_scale,
                     float softmax_scale, const int32_t* topk,
                     const int32_t* block_table, int64_t bt_stride,
                     const int32_t* seq_lens, int64_t B, int64_t n, int64_t Hq,
                     int64_t Hkv, int64_t max_seqlen_k, void* workspace,
                     size_t workspace_bytes, uint16_t* out, float* lse,
                     msa_plan_t* plan_out, void* stream) {
  return decode_impl(q, kv4, num_pages, q_scale, k_scale, v_scale,
                     softmax_scale, topk, block_table, bt_stride, seq_lens, B,
                     n, Hq, Hkv, max_seqlen_k, workspace, workspace_bytes, out,
                     lse, plan_out, static_cast<cudaStream_t>(stream),
                     MSA_KV_NVFP4);
}

}  // extern "C"

namespace {

// Scratch of msa_decode_noalloc: one fixed array on every GPU that loads this
// library, kept until the process exits.  Host code must not use its name
// as a device address; it asks the runtime for the address instead.
static __device__ __align__(256) unsigned char
    g_decode_scratch[MSA_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};
std::atomic<int> g_noalloc_busy{0};

// The array's device address in the current device's context.  Outside
// stream capture it is looked up on every call (the runtime call is cheap
// once the module is loaded, and a fresh lookup stays right after a context
// is torn down and rebuilt); under capture, where the first lookup's module
// load must not happen, the address from this device's last call outside
// capture is used.
int decode_scratch(cudaStream_t stream, void** ptr) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MSA_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return MSA_ERR_UNSUPPORTED;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess) return MSA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (cs == cudaStreamCaptureStatusNone) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_decode_scratch) != cudaSuccess || p == nullptr)
      return MSA_ERR_CUDA;
    g_scratch_ptr[dev] = p;
  } else if (g_scratch_ptr[dev] == nullptr) {
    return MSA_ERR_CUDA;  // no call outside capture on this device yet
  }
  *ptr = g_scratch_ptr[dev];
  return MSA_OK;
}

}  // namespace

extern "C" {

int msa_decode_noalloc(const uint8_t* q, const uint8_t* kv, int64_t num_pages,
                       float q_scale, float k_scale, float v_scale,
                       float softmax_scale, const int32_t* topk,
                       const int32_t* block_table, int64_t bt_stride,
                       const int32_t* seq_lens, int64_t B, int64_t n,
                       int64_t Hq, int64_t Hkv, int64_t max_seqlen_k,
                       uint16_t* out, float* lse, void* stream) {
  size_t need = 0;
  int rc = msa_decode_workspace_bytes(B, n, Hq, Hkv, max_seqlen_k, &need);
  if (rc) return rc;
  if (need > (size_t)MSA_NOALLOC_SCRATCH_BYTES) return MSA_ERR_TOO_LARGE;
  if (B == 0) return MSA_OK;
  // a second host thread entering while one is enqueueing would share the
  // array: refuse it instead of letting the two overwrite each other
  int expected = 0;
  if (!g_noalloc_busy.compare_exchange_strong(expected, 1)) return MSA_ERR_BUSY;
  void* scratch = nullptr;
  rc = decode_scratch(static_cast<cudaStream_t>(stream), &scratch);
  if (rc == MSA_OK)
    rc = msa_decode(q, kv, num_pages, q_scale, k_scale, v_scale, softmax_scale,
                    topk, block_table, bt_stride, seq_lens, B, n, Hq, Hkv,
                    max_seqlen_k, scratch, MSA_NOALLOC_SCRATCH_BYTES, out, lse,
                    nullptr, stream);
  g_noalloc_busy.store(0);
  return rc;
}

int msa_test_set_wait_limit_ns(uint64_t ns) {
  g_test_wait_ns.store(ns, std::memory_order_relaxed);
  return MSA_OK;
}

int msa_read_status(const msa_plan_t* plan, uint32_t* status) {
  if (!plan || !status || !plan->status) return MSA_ERR_NULL;
  return cuda_rc(cudaMemcpy(status, plan->status, sizeof(uint32_t),
                            cudaMemcpyDeviceToHost));
}

int msa_read_counters(const msa_plan_t* plan, int64_t* nnz,
                      int64_t* num_work) {
  if (!plan || !plan->counters) return MSA_ERR_NULL;
  int32_t c[4] = {0, 0, 0, 0};
  cudaError_t e =
      cudaMemcpy(c, plan->counters, sizeof(c), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return MSA_ERR_CUDA;
  if (nnz) *nnz = c[0];
  if (num_work) *num_work = c[1];
  return MSA_OK;
}

}  // extern "C"
