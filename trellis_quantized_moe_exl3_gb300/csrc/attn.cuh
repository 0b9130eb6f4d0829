// What the kernels of attention over a paged cache share: the step's batch,
// the cache's addressing, and the launch interface between them and the C ABI
// (attention.cu).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/exl3.h"
#include "internal.h"

namespace exl3 {

// Device status bits of these kernels (sticky word).
enum : int32_t { kStatusBadPage = 1, kStatusBadBatch = 2 };

constexpr int kMaxSeqs = 65535;
constexpr int kMaxPageSize = 4096;
constexpr int kMaxLen = 1 << 30;  // of a sequence: sums of two positions fit 32 bits
constexpr int kSms = 152;
constexpr int kRowsCounters = 640;  // parts counters of attn_rows

struct Batch {
  int num_seqs, max_q, max_pages, T;
  int page_size;
  int64_t table_stride;
  const int32_t* cu_q;
  const int32_t* seq_lens;
  const int32_t* table;
};

// One sequence of the step, as the kernels see it: new tokens q0 .. q0+n-1,
// len tokens in all.  An inconsistent cu_q leaves the sequence out (n = 0); a
// length out of range is clamped; both set kStatusBadBatch.
struct Seq {
  int q0, n, len;
};
__device__ __forceinline__ Seq load_seq(const Batch& bt, int b, int32_t* bad) {
  Seq s;
  s.q0 = __ldg(bt.cu_q + b);
  const int q1 = __ldg(bt.cu_q + b + 1);
  s.len = __ldg(bt.seq_lens + b);
  s.n = q1 - s.q0;
  if (s.q0 < 0 || q1 > bt.T || s.n < 0) {
    *bad |= kStatusBadBatch;
    s.n = 0;
    s.q0 = 0;
  }
  const long long pages = (long long)bt.max_pages * bt.page_size;
  const long long most = pages < kMaxLen ? pages : kMaxLen;
  if (s.len < 0 || (long long)s.len > most) {
    *bad |= kStatusBadBatch;
    s.len = s.len < 0 ? 0 : (int)most;
  }
  return s;
}

struct Cache {
  const uint8_t* k;
  const uint8_t* v;
  int num_pages, page_size;
  int page_shift;  // log2 of page_size, -1 if it is no power of two
  int64_t page_bytes, token_bytes, head_bytes;  // strides
  const float* k_scale;
  const float* v_scale;
};

// ---- norm, rotation, append (norm_rope.cu)
struct HeadSet {
  const uint16_t* x;
  uint16_t* out;
  const uint16_t* weight;
  int heads;
  int64_t ts, hs, ots, ohs;
};
struct NormRopeParams {
  HeadSet set[3];  // q, k, v (heads = 0: absent); append: k and v go to the cache
  int append, bf16, e4m3;
  int T, dim;
  const int32_t* positions;
  const double* inv_freq;
  int rot, inter;
  float eps, inv_dim;
  Cache cache;  // append
  Batch batch;
  int32_t* status;
};
cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t st);

// ---- attention
struct AttnParams {
  Cache cache;
  Batch batch;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  uint16_t* out;
  float* lse;  // may be null
  int heads, kv_heads, group;
  float scale_log2;  // scale * log2(e)
  int causal, window;
  int bf16, e4m3, dim;
  int32_t* status;
  int32_t* counters;  // [kRowsCounters], zero between calls
  void* scratch;
  // the bounded waits of attn_tiles: the MMA warp's in looks (its status bit
  // ends the other warps'), the drains' in cycles; the barrier that never
  // completes (-1: none; a test of the waits)
  uint32_t wait_looks;
  int stuck_barrier;
  long long wait_budget;
};
size_t attn_rows_scratch_bytes(int dim);
cudaError_t launch_attn_rows(const AttnParams& p, cudaStream_t st);
// rows: new tokens times group
size_t attn_tiles_scratch_bytes(long long rows, int seqs, int dim);
// cudaErrorNotSupported, before any launch, where the cache cannot be a TMA
// source (it has no pages, the driver does not take its strides)
cudaError_t launch_attn_tiles(const AttnParams& p, cudaStream_t st);

}  // namespace exl3
