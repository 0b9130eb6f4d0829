// A pool of cache pages on the GPU: block tables, positions and slots of a
// step from its sequences' lengths, without the host.
//
//   need_b = ceil((L_b + n_b) / P) - ceil(L_b / P), e_b = need_0 + .. + need_(b-1)
//   k-th new page of b = free[count - 1 - e_b - k]
//
// and the way back for tokens that are taken off again, which leaves the stack
// of free pages as it was before they came.
//
// A scan over the sequences, then a copy of their table rows.  Small steps are a
// chain of loads (indices, lengths, pages): one launch, a cluster whose first CTA
// scans and whose CTAs then write rows with it.  Where the rows are many, eight
// SMs are too few to write them: the scan and the rows are two launches.
#include "attn.cuh"
#include "common.cuh"
#include "pipeline.cuh"

namespace exl3 {
namespace {

constexpr int kThreads = 512, kCtas = 8;
// Words a step writes up to which it is one launch: a step and its way back, us in
// one / two launches of extend, 8 sequences of 128 pages 7.9 / 8.7, 64 of 256 8.7 /
// 9.1, 128 of 512 (65536 words) 9.2 / 9.1, 256 of 2048 17.1 / 10.3.
constexpr long long kFused = 65536;
constexpr int kOwners = 8192;  // rows of a pool whose claims fit shared memory

enum : int32_t { kPoolBadRequest = 1, kPoolNoPages = 2, kPoolTooLong = 4 };

// What the first CTA says of a sequence of the step.
struct Rec {
  int row;    // of the pool, -1: left out
  int len;    // tokens before
  int len2;   // tokens after
  int first;  // pages of the step's sequences before this one, taken or given back
};

struct PoolParams {
  int num_pages, page_size, page_shift, max_seqs, max_pages;
  int32_t* table;
  int32_t* lens;
  int32_t* free;
  int32_t* count;
  int num;  // sequences of the step
  const int32_t* seqs;
  const int32_t* n;  // new tokens; tokens to drop (null: all)
  const int32_t* step_lens;  // trim: 0 for sequences that the step did not serve (null: all served)
  int max_tokens;
  int32_t* cu_q;
  int32_t* seq_lens;
  int32_t* block_table;
  int32_t* positions;
  int64_t* slots;
  int32_t* status;
  int32_t* owner;  // [max_seqs], zero between calls
  Rec* rec;        // [num]
};

// (a page size is a multiple of 16, most often a power of two)
struct Page {
  int size, shift;  // shift: log2 of the size, -1 if it is no power of two
  __device__ int of(int pos) const { return shift >= 0 ? pos >> shift : pos / size; }
};
__device__ __forceinline__ int pages_of(int len, Page page) { return page.of(len + page.size - 1); }

// Inclusive scan of two values over the CTA; *total receives the sums.
__device__ __forceinline__ longlong2 scan2(longlong2 v, longlong2* total) {
  __shared__ longlong2 sums[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v.x, m), y = __shfl_up_sync(0xffffffffu, v.y, m);
    if (lane >= m) {
      v.x += x;
      v.y += y;
    }
  }
  __syncthreads();
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  longlong2 t = lane < kThreads / 32 ? sums[lane] : make_longlong2(0, 0);
#pragma unroll
  for (int m = 1; m < kThreads / 32; m <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, t.x, m), y = __shfl_up_sync(0xffffffffu, t.y, m);
    if (lane >= m) {
      t.x += x;
      t.y += y;
    }
  }
  const int last = kThreads / 32 - 1;
  *total = make_longlong2(__shfl_sync(0xffffffffu, t.x, last), __shfl_sync(0xffffffffu, t.y, last));
  const long long x = __shfl_sync(0xffffffffu, t.x, max(warp - 1, 0));
  const long long y = __shfl_sync(0xffffffffu, t.y, max(warp - 1, 0));
  if (warp > 0) {
    v.x += x;
    v.y += y;
  }
  return v;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Claims: sequence i of the step may use its row if the row exists and no earlier
// one names it.  A row's owner is the greatest num - i (0: none).
struct Claims {
  int32_t* owner;
  int num, max_seqs;
  __device__ Claims(const PoolParams& p, int32_t* shared) : num(p.num), max_seqs(p.max_seqs) {
    owner = max_seqs <= kOwners ? shared : p.owner;
    if (owner == shared) {
      for (int s = threadIdx.x; s < max_seqs; s += kThreads) owner[s] = 0;
      __syncthreads();
    }
    for (int i = threadIdx.x; i < num; i += kThreads) {
      const int s = __ldg(p.seqs + i);
      if (s >= 0 && s < max_seqs) atomicMax(owner + s, num - i);
    }
    __threadfence_block();
    __syncthreads();
  }
  __device__ bool holds(int i, int s) const {
    return s >= 0 && s < max_seqs && *static_cast<volatile int32_t*>(owner + s) == num - i;
  }
  // (the workspace's are left at zero)
  __device__ void end(const PoolParams& p) const {
    if (owner != p.owner) return;
    __syncthreads();
    for (int i = threadIdx.x; i < num; i += kThreads) {
      const int s = __ldg(p.seqs + i);
      if (s >= 0 && s < max_seqs) owner[s] = 0;
    }
  }
};
__device__ __forceinline__ int length_of(const PoolParams& p, int s) {
  return min(max(p.lens[s], 0), (int)min((long long)p.max_pages * p.page_size, (long long)kMaxLen));
}
__device__ __forceinline__ Rec load_rec(const PoolParams& p, int i) {
  const int4 v = __ldcg(reinterpret_cast<const int4*>(p.rec + i));
  return Rec{v.x, v.y, v.z, v.w};
}

// The scan (one CTA): lengths, records, the pool's new state.
__device__ __forceinline__ void plan_extend(const PoolParams& p, int32_t* shared) {
  const Page P{p.page_size, p.page_shift};
  const int count = min(max(*p.count, 0), p.num_pages);
  const long long most = min((long long)p.max_pages * P.size, (long long)kMaxLen);
  __shared__ int s_taken, s_bad;
  if (threadIdx.x == 0) s_taken = s_bad = 0;
  const Claims claims(p, shared);
  int32_t bad = 0;
  longlong2 run = make_longlong2(0, 0), total;
  int taken = 0;
  for (int i0 = 0; i0 < p.num; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    int s = -1, len = 0, n = 0;
    bool ok = false;
    if (i < p.num) {
      s = __ldg(p.seqs + i);
      n = __ldg(p.n + i);
      ok = claims.holds(i, s) && n >= 0;
      if (!ok) bad |= kPoolBadRequest;
      n = max(n, 0);
      if (ok) {
        len = length_of(p, s);
        if (len + (long long)n > most) {
          ok = false;
          bad |= kPoolTooLong;
        }
      }
    }
    const long long need = ok ? pages_of(len + n, P) - pages_of(len, P) : 0;
    const longlong2 inc = scan2(make_longlong2(n, need), &total);
    const long long q1 = run.x + inc.x, e = run.y + inc.y - need;
    if (i < p.num) {
      if (ok && n > 0 && q1 > p.max_tokens) {
        ok = false;
        bad |= kPoolTooLong;
      }
      if (ok && need > 0 && e + need > count) {
        ok = false;
        bad |= kPoolNoPages;
      }
      p.cu_q[i + 1] = (int)min(q1, (long long)p.max_tokens);
      p.seq_lens[i] = ok ? len + n : 0;
      p.rec[i] = Rec{ok ? s : -1, len, len + n, (int)min(e, (long long)p.num_pages)};
      if (ok) {
        p.lens[s] = len + n;
        if (need > 0) taken = max(taken, (int)(e + need));
      }
    }
    run.x += total.x;
    run.y += total.y;
  }
  if (taken) atomicMax(&s_taken, taken);
  if (bad) atomicOr(&s_bad, bad);
  claims.end(p);
  __syncthreads();
  if (threadIdx.x == 0) {
    p.cu_q[0] = 0;
    // (the pages are read from the stack after its count falls: they stay there)
    *p.count = count - s_taken;
    p.status[1] = count;
    if (s_bad) atomicOr(p.status, s_bad);
  }
}

// Table rows, positions and slots, by `threads` threads of which this is `me`.
template <int VEC>
__device__ __forceinline__ void fill_rows(const PoolParams& p, int count, int me, int threads) {
  constexpr int U = 4, kItem = 32 * U * VEC;  // entries that a warp writes at a time
  const Page P{p.page_size, p.page_shift};
  const int lane = me & 31;
  const long long per_row = (p.max_pages + kItem - 1) / kItem, items = per_row * p.num;
  for (long long it = me >> 5; it < items; it += threads >> 5) {
    const int i = (int)(it / per_row), k0 = (int)(it % per_row) * kItem + lane * VEC;
    const Rec r = load_rec(p, i);
    const int have = r.row < 0 ? 0 : pages_of(r.len, P), want = r.row < 0 ? 0 : pages_of(r.len2, P);
    int32_t* mine = p.table + (int64_t)max(r.row, 0) * p.max_pages;
    int32_t* out = p.block_table + (int64_t)i * p.max_pages;
    int id[U][VEC];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int k = k0 + u * 32 * VEC;
#pragma unroll
      for (int v = 0; v < VEC; v++) id[u][v] = -1;
      if (k < have && k < p.max_pages) {
        if (VEC == 4) {
          const int4 w = *reinterpret_cast<const int4*>(mine + k);
          id[u][0] = w.x;
          id[u][VEC > 1 ? 1 : 0] = w.y;
          id[u][VEC > 1 ? 2 : 0] = w.z;
          id[u][VEC > 1 ? 3 : 0] = w.w;
        } else {
          id[u][0] = mine[k];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int k = k0 + u * 32 * VEC;
      if (k + VEC > have && k < want) {
#pragma unroll
        for (int v = 0; v < VEC; v++)
          if (k + v >= have && k + v < want) {
            id[u][v] = p.free[count - 1 - r.first - (k + v - have)];
            mine[k + v] = id[u][v];
          }
      }
#pragma unroll
      for (int v = 0; v < VEC; v++)
        if (k + v >= want) id[u][v] = -1;
      if (k < p.max_pages) {
        if (VEC == 4)
          *reinterpret_cast<int4*>(out + k) =
              make_int4(id[u][0], id[u][VEC > 1 ? 1 : 0], id[u][VEC > 1 ? 2 : 0], id[u][VEC > 1 ? 3 : 0]);
        else
          out[k] = id[u][0];
      }
    }
  }
}
__device__ __forceinline__ void fill(const PoolParams& p, int me, int threads) {
  const Page P{p.page_size, p.page_shift};
  const int count = __ldcg(p.status + 1);
  // 16 bytes at a time where rows begin on 16 bytes
  if (p.max_pages % 4 == 0 &&
      ((reinterpret_cast<uintptr_t>(p.table) | reinterpret_cast<uintptr_t>(p.block_table)) & 15) == 0)
    fill_rows<4>(p, count, me, threads);
  else
    fill_rows<1>(p, count, me, threads);
  // place j of sequence i, in row t
  auto put = [&](int t, int j, const Rec& r) {
    int pos = -1;
    int64_t slot = -1;
    if (r.row >= 0) {
      pos = r.len + j;
      const int k = P.of(pos), have = pages_of(r.len, P);
      const int id = k < have ? p.table[(int64_t)r.row * p.max_pages + k]
                              : p.free[count - 1 - r.first - (k - have)];
      if (id >= 0) slot = (int64_t)id * P.size + (pos - k * P.size);
    }
    p.positions[t] = pos;
    p.slots[t] = slot;
  };
  // (from the last warps on, while the first ones write table rows)
  const int from = threads - 1 - me;
  int all = p.num > 0 ? __ldcg(p.cu_q + p.num) : 0;  // rows that are some sequence's
  if (p.max_tokens <= 64 * p.num) {
    // few tokens each: a warp per sequence
    for (int i = from >> 5; i < p.num; i += threads >> 5) {
      const Rec r = load_rec(p, i);
      const int t0 = __ldcg(p.cu_q + i), n = __ldcg(p.cu_q + i + 1) - t0;
      for (int j = from & 31; j < n; j += 32) put(t0 + j, j, r);
    }
  } else {
    for (int t = from; t < all; t += threads) {
      int lo = 0, hi = p.num;  // the last sequence that begins at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldcg(p.cu_q + mid) <= t)
          lo = mid;
        else
          hi = mid;
      }
      put(t, t - __ldcg(p.cu_q + lo), load_rec(p, lo));
    }
  }
  for (int t = all + from; t < p.max_tokens; t += threads) {
    p.positions[t] = -1;
    p.slots[t] = -1;
  }
}

// One cluster: the scan, then the rows.
__global__ void __launch_bounds__(kThreads) extend_kernel(PoolParams p) {
  __shared__ int32_t owners[kOwners];
  pdl_wait();
  if (blockIdx.x == 0) plan_extend(p, owners);
  cluster_sync();  // (releases what the first CTA wrote to the others)
  fill(p, blockIdx.x * kThreads + threadIdx.x, kCtas * kThreads);
}
// The same in two launches.
__global__ void __launch_bounds__(kThreads) extend_plan_kernel(PoolParams p) {
  __shared__ int32_t owners[kOwners];
  pdl_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  plan_extend(p, owners);
}
__global__ void __launch_bounds__(kThreads) extend_fill_kernel(PoolParams p) {
  pdl_wait();
  fill(p, blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads);
}

__global__ void __launch_bounds__(kThreads) trim_kernel(PoolParams p) {
  __shared__ int32_t owners[kOwners];
  pdl_wait();
  const int rank = blockIdx.x;
  const Page P{p.page_size, p.page_shift};
  if (rank == 0) {
    const Claims claims(p, owners);
    const int count = min(max(*p.count, 0), p.num_pages);
    int32_t bad = 0;
    longlong2 run = make_longlong2(0, 0), total;
    for (int i0 = 0; i0 < p.num; i0 += kThreads) {
      const int i = i0 + threadIdx.x;
      int s = -1, len = 0, n = 0;
      bool ok = false;
      if (i < p.num) {
        s = __ldg(p.seqs + i);
        ok = claims.holds(i, s);
        if (ok && p.step_lens && __ldg(p.step_lens + i) <= 0) {
          ok = false;  // it got no tokens: what its row holds is older
        } else if (ok) {
          len = length_of(p, s);
          n = p.n ? __ldg(p.n + i) : len;
          if (n < 0 || n > len) bad |= kPoolBadRequest;
          n = min(max(n, 0), len);
        } else {
          bad |= kPoolBadRequest;
        }
      }
      const long long back = ok ? pages_of(len, P) - pages_of(len - n, P) : 0;
      const longlong2 inc = scan2(make_longlong2(0, back), &total);
      if (i < p.num) {
        const long long e = run.y + inc.y - back;
        p.rec[i] = Rec{ok ? s : -1, len, len - n, (int)min(e, (long long)kMaxLen)};
        if (ok) p.lens[s] = len - n;
      }
      run.y += total.y;
    }
    claims.end(p);
    if (run.y > p.num_pages - count) {  // more than there are: the pool was tampered with
      bad |= kPoolBadRequest;
      run.y = p.num_pages - count;
    }
    if (bad) atomicOr(p.status, bad);
    if (threadIdx.x == 0) {
      *p.count = count + (int)run.y;
      p.status[1] = count + (int)run.y;
      p.status[2] = count;
    }
  }
  cluster_sync();
  // the first page of the first sequence goes on top
  const int top = __ldcg(p.status + 1) - 1, bottom = __ldcg(p.status + 2);
  const int warp = (rank * kThreads + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  constexpr int kWarps = kCtas * kThreads / 32;
  for (int i = warp; i < p.num; i += kWarps) {
    const int4 r = __ldcg(reinterpret_cast<const int4*>(p.rec + i));
    if (r.x < 0) continue;
    int32_t* mine = p.table + (int64_t)r.x * p.max_pages;
    const int keep = pages_of(r.z, P), had = pages_of(r.y, P);
    for (int k = keep + lane; k < had; k += 32) {
      const int64_t at = (int64_t)top - r.w - (k - keep);
      if (at >= bottom) p.free[at] = mine[k];
      mine[k] = -1;
    }
  }
}

cudaError_t launch(void (*kernel)(PoolParams), const PoolParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  note_launches(1);
  return e;
}

// workspace: status word and two for the count, the owners, the records
size_t owners_at() { return 256; }
size_t records_at(int max_seqs) { return (owners_at() + (size_t)max_seqs * 4 + 255) & ~(size_t)255; }

exl3_status check(const exl3_page_pool* o, int num, const int32_t* seqs, const void* ws,
                  size_t ws_bytes) {
  if (!o) return EXL3_ERR_ARG;
  if (o->num_pages < 0 || o->page_size < 16 || o->page_size > kMaxPageSize || o->page_size % 16 ||
      o->max_seqs < 1 || o->max_seqs > kMaxSeqs || o->max_pages < 1 || num < 0 || num > kMaxSeqs ||
      (long long)o->max_pages * o->page_size > kMaxLen)
    return EXL3_ERR_SHAPE;
  if (!o->table || !o->lens || !o->count || (o->num_pages > 0 && !o->free) || (num > 0 && !seqs))
    return EXL3_ERR_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15) ||
      ws_bytes < exl3_pages_workspace_size(o->max_seqs, num))
    return EXL3_ERR_WORKSPACE;
  return EXL3_OK;
}

PoolParams params_of(const exl3_page_pool* o, int num, const int32_t* seqs, const int32_t* n,
                     void* ws) {
  PoolParams p{};
  p.num_pages = o->num_pages;
  p.page_size = o->page_size;
  p.page_shift = o->page_size & (o->page_size - 1) ? -1 : __builtin_ctz(o->page_size);
  p.max_seqs = o->max_seqs;
  p.max_pages = o->max_pages;
  p.table = o->table;
  p.lens = o->lens;
  p.free = o->free;
  p.count = o->count;
  p.num = num;
  p.seqs = seqs;
  p.n = n;
  p.status = static_cast<int32_t*>(ws);
  p.owner = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + owners_at());
  p.rec = reinterpret_cast<Rec*>(static_cast<uint8_t*>(ws) + records_at(o->max_seqs));
  return p;
}

}  // namespace
}  // namespace exl3

using namespace exl3;

extern "C" {

size_t exl3_pages_workspace_size(int max_seqs, int num) {
  if (max_seqs < 1 || max_seqs > kMaxSeqs || num < 0 || num > kMaxSeqs) return 0;
  return records_at(max_seqs) + (size_t)num * sizeof(Rec);
}

exl3_status exl3_pages_extend(const exl3_page_pool* pool, int num, const int32_t* seqs,
                              const int32_t* q_lens, int max_tokens, int32_t* cu_q,
                              int32_t* seq_lens, int32_t* block_table, int32_t* positions,
                              int64_t* slots, void* ws, size_t ws_bytes, void* stream) {
  const exl3_status e = check(pool, num, seqs, ws, ws_bytes);
  if (e != EXL3_OK) return e;
  if (max_tokens < 0 || max_tokens > (1 << 30)) return EXL3_ERR_SHAPE;
  if (!cu_q || (num > 0 && (!q_lens || !seq_lens || !block_table)) ||
      (max_tokens > 0 && (!positions || !slots)) || (reinterpret_cast<uintptr_t>(slots) & 7))
    return EXL3_ERR_ARG;
  PoolParams p = params_of(pool, num, seqs, q_lens, ws);
  p.max_tokens = max_tokens;
  p.cu_q = cu_q;
  p.seq_lens = seq_lens;
  p.block_table = block_table;
  p.positions = positions;
  p.slots = slots;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  if ((long long)num * pool->max_pages + 3ll * max_tokens <= kFused) {
    err = launch(extend_kernel, p, st);
  } else {
    err = launch_pdl(extend_plan_kernel, dim3(1), dim3(kThreads), 0, st, p);
    if (err == cudaSuccess) err = launch_pdl(extend_fill_kernel, dim3(2 * kSms), dim3(kThreads), 0, st, p);
    note_launches(2);
  }
  return err == cudaSuccess ? EXL3_OK : EXL3_ERR_CUDA;
}

exl3_status exl3_pages_trim_step(const exl3_page_pool* pool, int num, const int32_t* seqs,
                                 const int32_t* drop, const int32_t* step_lens, void* ws,
                                 size_t ws_bytes, void* stream) {
  const exl3_status e = check(pool, num, seqs, ws, ws_bytes);
  if (e != EXL3_OK) return e;
  if (num == 0) return EXL3_OK;
  PoolParams p = params_of(pool, num, seqs, drop, ws);
  p.step_lens = step_lens;
  return launch(trim_kernel, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? EXL3_OK
                                                                                  : EXL3_ERR_CUDA;
}

exl3_status exl3_pages_trim(const exl3_page_pool* pool, int num, const int32_t* seqs,
                            const int32_t* drop, void* ws, size_t ws_bytes, void* stream) {
  return exl3_pages_trim_step(pool, num, seqs, drop, nullptr, ws, ws_bytes, stream);
}

}  // extern "C"
