// C ABI of the attention operators: argument checks and launches.
#include <math.h>

#include "attn.cuh"
#include "pipeline.cuh"

using namespace exl3;

namespace {

// Rows of a sequence and kv head up to which attn_rows is taken.  8 kv heads of
// 128, us against attn_tiles at 16 and 32 rows.  bf16: 16 sequences of 4000
// 54 / 60, 67 / 60; 256 of 1000 174 / 198, 326 / 200; one of 500 12 / 15,
// 12 / 15.  E4M3 (which attn_tiles has to widen): 40 / 59, 54 / 59; 123 / 205,
// 222 / 205; 13 / 16, 13 / 16; at 48 rows 77 / 60, 319 / 207.
constexpr int kRowsMost = 16, kRowsMostE4m3 = 32;
constexpr size_t kHead = EXL3_ATTENTION_HEAD_BYTES;  // status word, counters
static_assert(256 + kRowsCounters * 4 <= kHead, "counters");

// The bounded waits of attn_tiles (exl3_test_set_attention_wait_fault).
struct Waits {
  long long budget = kWaitBudgetCycles;
  int stuck_barrier = -1;
};
Waits g_waits;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool good(const void* p) { return p && aligned16(p); }

exl3_status check_cache(const exl3_kv_cache* c, exl3_dtype dt, int max_dim) {
  if (!c) return EXL3_ERR_ARG;
  if (c->dtype != (int)dt && c->dtype != EXL3_E4M3) return EXL3_ERR_ARG;
  if (c->dtype != EXL3_E4M3 && (c->k_scale || c->v_scale)) return EXL3_ERR_ARG;
  if (c->num_pages < 0 || c->page_size < 16 || c->page_size > kMaxPageSize ||
      c->page_size % 16 || c->kv_heads < 1 || c->head_dim < 8 || c->head_dim % 8 ||
      c->head_dim > max_dim)
    return EXL3_ERR_SHAPE;
  if (c->num_pages > 0 && (!good(c->k) || !good(c->v))) return EXL3_ERR_ARG;
  const int64_t step = c->dtype == EXL3_E4M3 ? 16 : 8;
  for (const int64_t s : {c->page_stride, c->token_stride, c->head_stride})
    if (s < 0 || s % step) return EXL3_ERR_ARG;
  return EXL3_OK;
}

// Block scales of an E4M3 cache (none: s null).
exl3_status check_scales(const exl3_kv_cache* c, const exl3_kv_scales* s) {
  if (!s) return EXL3_OK;
  if (c->dtype != EXL3_E4M3 || c->k_scale || c->v_scale || s->page_stride < c->kv_heads)
    return EXL3_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(s->k) | reinterpret_cast<uintptr_t>(s->v)) & 3)
    return EXL3_ERR_ARG;
  if (c->num_pages > 0 && (!s->k || !s->v)) return EXL3_ERR_ARG;
  return EXL3_OK;
}

exl3_status check_batch(const exl3_kv_batch* b) {
  if (!b) return EXL3_ERR_ARG;
  if (b->num_seqs < 0 || b->num_seqs > kMaxSeqs || b->max_pages < 0 || b->max_q < 0 ||
      b->table_stride < 0)
    return EXL3_ERR_SHAPE;
  if (b->num_seqs > 0 && (!b->cu_q || !b->seq_lens || (b->max_pages > 0 && !b->block_table)))
    return EXL3_ERR_ARG;
  return EXL3_OK;
}

exl3_status check_heads(const exl3_heads* h, int T, int need_out) {
  if (h->heads < 1) return EXL3_ERR_SHAPE;
  if (T > 0 && (!good(h->x) || (need_out && !good(h->out)))) return EXL3_ERR_ARG;
  if (h->weight && !aligned16(h->weight)) return EXL3_ERR_ARG;
  if (h->token_stride % 8 || h->head_stride % 8 || h->token_stride < 0 || h->head_stride < 0)
    return EXL3_ERR_ARG;
  if (need_out && (h->out_token_stride % 8 || h->out_head_stride % 8 || h->out_token_stride < 0 ||
                   h->out_head_stride < 0))
    return EXL3_ERR_ARG;
  return EXL3_OK;
}

exl3_status check_rope(const exl3_rope* r, int head_dim) {
  if (!r) return EXL3_OK;
  if (r->rotary_dim < 16 || r->rotary_dim % 16 || r->rotary_dim > head_dim) return EXL3_ERR_SHAPE;
  if (!r->inv_freq || (r->interleaved != 0 && r->interleaved != 1)) return EXL3_ERR_ARG;
  return EXL3_OK;
}

HeadSet head_set(const exl3_heads* h) {
  HeadSet s{};
  s.x = static_cast<const uint16_t*>(h->x);
  s.out = static_cast<uint16_t*>(h->out);
  s.weight = static_cast<const uint16_t*>(h->weight);
  s.heads = h->heads;
  s.ts = h->token_stride;
  s.hs = h->head_stride;
  s.ots = h->out_token_stride;
  s.ohs = h->out_head_stride;
  return s;
}

Cache cache_of(const exl3_kv_cache* c, const exl3_kv_scales* s) {
  const int64_t e = c->dtype == EXL3_E4M3 ? 1 : 2;
  Cache o{};
  o.k = static_cast<const uint8_t*>(c->k);
  o.v = static_cast<const uint8_t*>(c->v);
  o.num_pages = c->num_pages;
  o.page_size = c->page_size;
  o.page_shift = c->page_size & (c->page_size - 1) ? -1 : __builtin_ctz(c->page_size);
  o.page_bytes = c->page_stride * e;
  o.token_bytes = c->token_stride * e;
  o.head_bytes = c->head_stride * e;
  o.k_scale = s ? s->k : c->k_scale;
  o.v_scale = s ? s->v : c->v_scale;
  o.scale_stride = s ? s->page_stride : 0;
  return o;
}

Batch batch_of(const exl3_kv_batch* b, int T, int page_size) {
  return Batch{b->num_seqs, b->max_q,    b->max_pages, T,
               page_size,   b->table_stride, b->cu_q,  b->seq_lens, b->block_table};
}

bool bad_dtype(exl3_dtype dt) { return dt != EXL3_F16 && dt != EXL3_BF16; }

exl3_status kv_append(const exl3_kv_cache* cache, const exl3_kv_scales* scales,
                      const exl3_kv_batch* batch, const exl3_heads* q, const exl3_heads* k,
                      const exl3_heads* v, exl3_dtype dt, int T, const exl3_rope* rope,
                      const int32_t* positions, float eps, int32_t* status, void* stream) {
  if (!k || !v || !status || bad_dtype(dt) || !(eps >= 0.0f)) return EXL3_ERR_ARG;
  if (T < 0) return EXL3_ERR_SHAPE;
  exl3_status e;
  if ((e = check_cache(cache, dt, 256)) != EXL3_OK) return e;
  if ((e = check_scales(cache, scales)) != EXL3_OK) return e;
  if ((e = check_batch(batch)) != EXL3_OK) return e;
  if (q && (e = check_heads(q, T, 1)) != EXL3_OK) return e;
  if ((e = check_heads(k, T, 0)) != EXL3_OK) return e;
  if ((e = check_heads(v, T, 0)) != EXL3_OK) return e;
  if (k->heads != cache->kv_heads || v->heads != cache->kv_heads) return EXL3_ERR_SHAPE;
  if ((e = check_rope(rope, cache->head_dim)) != EXL3_OK) return e;
  if (T == 0 || batch->num_seqs == 0) return EXL3_OK;
  NormRopeParams p{};
  if (q) p.set[0] = head_set(q);
  p.set[1] = head_set(k);
  p.set[2] = head_set(v);
  p.set[2].weight = nullptr;
  p.append = 1;
  p.bf16 = dt == EXL3_BF16;
  p.e4m3 = cache->dtype == EXL3_E4M3;
  p.T = T;
  p.dim = cache->head_dim;
  p.inv_dim = 1.0f / (float)p.dim;
  p.positions = positions;
  if (rope) {
    p.inv_freq = rope->inv_freq;
    p.rot = rope->rotary_dim;
    p.inter = rope->interleaved;
  }
  p.eps = eps;
  p.cache = cache_of(cache, scales);
  p.batch = batch_of(batch, T, cache->page_size);
  p.status = status;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return (scales ? launch_append_blocks(p, st) : launch_norm_rope(p, st)) == cudaSuccess
             ? EXL3_OK
             : EXL3_ERR_CUDA;
}


exl3_status attend(const exl3_kv_cache* cache, const exl3_kv_scales* scales,
                   const exl3_kv_batch* batch, const void* q, int64_t q_token_stride,
                   int64_t q_head_stride, exl3_dtype dt, int T, int heads, float scale, int causal,
                   int window, void* out, float* lse, int path, void* ws, size_t ws_bytes,
                   void* stream) {
  if (bad_dtype(dt) || !(scale > 0.0f) || !isfinite(scale) || (causal != 0 && causal != 1) ||
      window < 0 || (window > 0 && !causal) || path < EXL3_PATH_AUTO || path > EXL3_PATH_GEMM)
    return EXL3_ERR_ARG;
  if (T < 0 || heads < 1) return EXL3_ERR_SHAPE;
  exl3_status e;
  if ((e = check_cache(cache, dt, 128)) != EXL3_OK) return e;
  if (cache->head_dim != 64 && cache->head_dim != 128) return EXL3_ERR_SHAPE;
  if (heads % cache->kv_heads) return EXL3_ERR_SHAPE;
  if ((e = check_scales(cache, scales)) != EXL3_OK) return e;
  if ((e = check_batch(batch)) != EXL3_OK) return e;
  if ((long long)T * (heads / cache->kv_heads) > (1ll << 30)) return EXL3_ERR_SHAPE;
  if (q_token_stride % 8 || q_head_stride % 8 || q_token_stride < 0 || q_head_stride < 0)
    return EXL3_ERR_ARG;
  if (T == 0 || batch->num_seqs == 0) return EXL3_OK;
  if (!good(q) || !out || (reinterpret_cast<uintptr_t>(out) & 31) ||
      (reinterpret_cast<uintptr_t>(lse) & 3))
    return EXL3_ERR_ARG;
  if (!good(ws) || ws_bytes < exl3_paged_attention_workspace_size(T, heads, cache->kv_heads,
                                                                  cache->head_dim, batch->num_seqs))
    return EXL3_ERR_WORKSPACE;
  AttnParams p{};
  p.cache = cache_of(cache, scales);
  p.batch = batch_of(batch, T, cache->page_size);
  p.q = static_cast<const uint16_t*>(q);
  p.q_ts = q_token_stride;
  p.q_hs = q_head_stride;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.heads = heads;
  p.kv_heads = cache->kv_heads;
  p.group = heads / cache->kv_heads;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.causal = causal;
  p.window = window < kMaxLen ? window : kMaxLen;  // (either sees every earlier key)
  p.bf16 = dt == EXL3_BF16;
  p.e4m3 = cache->dtype == EXL3_E4M3;
  p.dim = cache->head_dim;
  p.blocks = scales != nullptr;
  p.status = static_cast<int32_t*>(ws);
  p.counters = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + 256);
  p.scratch = static_cast<uint8_t*>(ws) + kHead;
  p.wait_budget = g_waits.budget;
  p.wait_looks = (uint32_t)(g_waits.budget / 500);  // of up to 1 us, 2000 cycles
  p.stuck_barrier = g_waits.stuck_barrier;
  // Few rows per sequence and kv head: the cache's bytes bound the step.
  bool tiles = (long long)batch->max_q * p.group > (p.e4m3 ? kRowsMostE4m3 : kRowsMost);
  if (path != EXL3_PATH_AUTO) tiles = path == EXL3_PATH_GEMM;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t err = cudaErrorNotSupported;  // a cache that cannot be a TMA source
  if (tiles) err = launch_attn_tiles(p, st);
  if (err == cudaErrorNotSupported) err = launch_attn_rows(p, st);
  return err == cudaSuccess ? EXL3_OK : EXL3_ERR_CUDA;
}

}  // namespace

extern "C" {

exl3_status exl3_qk_norm_rope(const exl3_heads* q, const exl3_heads* k, exl3_dtype dt, int T,
                              int head_dim, const int32_t* positions, const exl3_rope* rope,
                              float eps, void* stream) {
  if (!q || bad_dtype(dt) || !(eps >= 0.0f)) return EXL3_ERR_ARG;
  if (T < 0 || head_dim < 8 || head_dim % 8 || head_dim > 256) return EXL3_ERR_SHAPE;
  exl3_status e;
  if ((e = check_heads(q, T, 1)) != EXL3_OK) return e;
  if (k && (e = check_heads(k, T, 1)) != EXL3_OK) return e;
  if ((e = check_rope(rope, head_dim)) != EXL3_OK) return e;
  if (T == 0) return EXL3_OK;
  if (rope && !positions) return EXL3_ERR_ARG;
  NormRopeParams p{};
  p.set[0] = head_set(q);
  if (k) p.set[1] = head_set(k);
  p.bf16 = dt == EXL3_BF16;
  p.T = T;
  p.dim = head_dim;
  p.inv_dim = 1.0f / (float)p.dim;
  p.positions = positions;
  if (rope) {
    p.inv_freq = rope->inv_freq;
    p.rot = rope->rotary_dim;
    p.inter = rope->interleaved;
  }
  p.eps = eps;
  return launch_norm_rope(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? EXL3_OK
                                                                              : EXL3_ERR_CUDA;
}

exl3_status exl3_kv_append(const exl3_kv_cache* cache, const exl3_kv_batch* batch,
                           const exl3_heads* q, const exl3_heads* k, const exl3_heads* v,
                           exl3_dtype dt, int T, const exl3_rope* rope, const int32_t* positions,
                           float eps, int32_t* status, void* stream) {
  return kv_append(cache, nullptr, batch, q, k, v, dt, T, rope, positions, eps, status, stream);
}

exl3_status exl3_kv_append_blocks(const exl3_kv_cache* cache, const exl3_kv_scales* scales,
                                  const exl3_kv_batch* batch, const exl3_heads* q,
                                  const exl3_heads* k, const exl3_heads* v, exl3_dtype dt, int T,
                                  const exl3_rope* rope, const int32_t* positions, float eps,
                                  int32_t* status, void* stream) {
  if (!scales) return EXL3_ERR_ARG;
  return kv_append(cache, scales, batch, q, k, v, dt, T, rope, positions, eps, status, stream);
}

size_t exl3_paged_attention_workspace_size(int T, int heads, int kv_heads, int head_dim,
                                           int num_seqs) {
  if (T < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads ||
      (head_dim != 64 && head_dim != 128) || num_seqs < 0 || num_seqs > kMaxSeqs)
    return 0;
  const size_t a = attn_rows_scratch_bytes(head_dim);
  const size_t b = attn_tiles_scratch_bytes((long long)T * (heads / kv_heads), num_seqs, head_dim);
  return kHead + (a > b ? a : b);
}

exl3_status exl3_paged_attention(const exl3_kv_cache* cache, const exl3_kv_batch* batch,
                                 const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                 exl3_dtype dt, int T, int heads, float scale, int causal,
                                 int window, void* out, float* lse, int path, void* ws,
                                 size_t ws_bytes, void* stream) {
  return attend(cache, nullptr, batch, q, q_token_stride, q_head_stride, dt, T, heads, scale,
                causal, window, out, lse, path, ws, ws_bytes, stream);
}

exl3_status exl3_paged_attention_blocks(const exl3_kv_cache* cache, const exl3_kv_scales* scales,
                                        const exl3_kv_batch* batch, const void* q,
                                        int64_t q_token_stride, int64_t q_head_stride,
                                        exl3_dtype dt, int T, int heads, float scale, int causal,
                                        int window, void* out, float* lse, int path, void* ws,
                                        size_t ws_bytes, void* stream) {
  if (!scales) return EXL3_ERR_ARG;
  return attend(cache, scales, batch, q, q_token_stride, q_head_stride, dt, T, heads, scale, causal,
                window, out, lse, path, ws, ws_bytes, stream);
}

exl3_status exl3_test_set_attention_wait_fault(int barrier, long long budget_cycles) {
  if (barrier == -1) {
    g_waits = Waits{};
    return EXL3_OK;
  }
  if (barrier < 0 || budget_cycles < 1000000 || budget_cycles > kWaitBudgetCycles)
    return EXL3_ERR_ARG;
  g_waits.stuck_barrier = barrier;
  g_waits.budget = budget_cycles;
  return EXL3_OK;
}

}  // extern "C"
