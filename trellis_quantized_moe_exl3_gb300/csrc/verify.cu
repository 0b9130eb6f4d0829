// Verification of drafted tokens against the target's probabilities.
//
// Draft j of a sequence (token x) is accepted while u_j q_j(x) < p_j(x).  At
// the first refusal a the next token is drawn from max(p_a - q_a, 0), after
// the last accepted draft from p_d, in either case as the first v whose
// cumulative weight exceeds sample_u times the total.
//
// Both decisions are exact.  u q is a product of two 24-bit values, formed in
// 64 bits; weights are summed as 64-bit integers in units of 2^-56 (what is
// above 2^-32 is held whole, a row of 2^18 tokens loses at most 2^-38), so the
// order of a sum does not matter, and no border between two tokens moves with
// the split of a row over threads.
//
// One row of p (and of q) per sequence is all that has to be read: memory
// bounds large batches, the chain of loads (bounds, drafts, their
// probabilities, the row, the chosen piece again) the small ones.  A cluster
// of CTAs takes a sequence, so that the pieces' sums meet in distributed
// shared memory: one launch, no workspace, nothing to zero.
#include "attn.cuh"
#include "common.cuh"
#include "pipeline.cuh"

namespace exl3 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kUnroll = 8;  // loads of a row in flight per thread

struct VerifyParams {
  const void* p;
  const void* q;  // null: the drafts are certain
  int64_t p_stride, q_stride;
  int vocab, num_seqs, drafts;
  const int32_t* cu;
  const int32_t* draft;
  const float* accept_u;
  const float* sample_u;
  int32_t* tokens;
  int32_t* accepted;
  int32_t* dropped;
};

template <int DT>
__device__ __forceinline__ float value(const void* x, int64_t i) {
  if (DT == EXL3_F32) return __ldg(static_cast<const float*>(x) + i);
  return load_act(x, DT == EXL3_BF16, (size_t)i);
}

// A probability in units of 2^-56; NaN and what is negative count as 0.
__device__ __forceinline__ unsigned long long fixed(float x) {
  return x > 0.0f ? __float2ull_rz(fminf(x, 1.0f) * 0x1p56f) : 0ull;
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// The weights of one row: p, or max(p - q, 0), or p without one token.
template <int DT>
struct Row {
  const void* p;
  const void* q;
  int64_t p0, q0;
  int skip;  // -1: none
  __device__ __forceinline__ unsigned long long at(int v) const {
    unsigned long long w = fixed(value<DT>(p, p0 + v));
    if (q) {
      const unsigned long long x = fixed(value<DT>(q, q0 + v));
      w = w > x ? w - x : 0;
    }
    return v == skip ? 0 : w;
  }
};

__device__ __forceinline__ unsigned long long load_remote(unsigned long long* at, int rank) {
  uint32_t a;
  unsigned long long v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

template <int DT>
__global__ void __launch_bounds__(kThreads) verify_kernel(VerifyParams p, int ctas) {
  __shared__ unsigned long long total[2];         // of this CTA, by pass
  __shared__ unsigned long long warp_total[kWarps];
  __shared__ int s_accepted;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  pdl_wait();
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1);
  const bool good = c0 >= 0 && c1 >= c0 && c1 <= p.drafts;
  const int d = good ? c1 - c0 : 0;
  // ---- the first refusal (every CTA for itself)
  if (warp == 0) {
    int a = d;
    for (int j0 = 0; j0 < d; j0 += 32) {
      const int j = j0 + lane;
      bool no = false;
      if (j < d) {
        const int x = __ldg(p.draft + c0 + j);
        no = true;
        if (x >= 0 && x < p.vocab) {
          const double u = __ldg(p.accept_u + c0 + j);
          const float pp = value<DT>(p.p, (int64_t)(c0 + j + b) * p.p_stride + x);
          const float qq = p.q ? value<DT>(p.q, (int64_t)(c0 + j) * p.q_stride + x) : 1.0f;
          no = !(u * (double)qq < (double)pp);
        }
      }
      const uint32_t m = __ballot_sync(0xffffffffu, no);
      if (m) {
        a = j0 + __ffs(m) - 1;
        break;
      }
    }
    if (lane == 0) s_accepted = a;
  }
  __syncthreads();
  const int a = s_accepted;
  if (rank == 0) {
    // accepted drafts, then -1 (the drawn token's place too, until it is known);
    // rows that belong to no sequence as well
    if (good)
      for (int j = threadIdx.x; j <= d; j += kThreads)
        p.tokens[c0 + b + j] = j < a ? __ldg(p.draft + c0 + j) : -1;
    if (b == p.num_seqs - 1 && good)
      for (int64_t j = (int64_t)c1 + b + 1 + threadIdx.x; j < (int64_t)p.drafts + p.num_seqs;
           j += kThreads)
        p.tokens[j] = -1;
    if (threadIdx.x == 0) {
      p.accepted[b] = a;
      p.dropped[b] = d - a;
    }
  }
  if (!good) return;  // (the whole cluster: it waits for no one)

  // ---- the row's weights: this CTA's piece, a run of it per warp
  Row<DT> row;
  row.p = p.p;
  row.p0 = (int64_t)(c0 + a + b) * p.p_stride;
  row.q = a < d ? p.q : nullptr;
  row.q0 = (int64_t)(c0 + a) * p.q_stride;
  row.skip = a < d && !p.q ? __ldg(p.draft + c0 + a) : -1;
  const int run = ((p.vocab + ctas * kWarps - 1) / (ctas * kWarps) + 31) & ~31;
  const int v0 = min((rank * kWarps + warp) * run, p.vocab), v1 = min(v0 + run, p.vocab);
  unsigned long long all = 0, before = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; pass++) {
    unsigned long long sum = 0;
#pragma unroll kUnroll
    for (int v = v0 + lane; v < v1; v += 32) sum += row.at(v);
    sum = warp_sum(sum);
    if (lane == 0) warp_total[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned long long t = 0;
      for (int w = 0; w < kWarps; w++) t += warp_total[w];
      total[pass] = t;
    }
    cluster_sync();
    all = before = 0;
    for (int r = 0; r < ctas; r++) {
      const unsigned long long t = load_remote(&total[pass], r);
      if (r < rank) before += t;
      all += t;
    }
    // nothing is left of p without q: the target's own probabilities
    if (all > 0 || (!row.q && row.skip < 0)) break;
    row.q = nullptr;
    row.skip = -1;
  }
  // no CTA leaves while another may read its sums
  cluster_sync();

  // ---- the token: the first v with a cumulative weight above u * all
  const float u = fminf(fmaxf(__ldg(p.sample_u + b), 0.0f), 1.0f - 0x1p-24f);
  const unsigned long long want = __umul64hi(__float2ull_rz(u * 0x1p64f), all);
  if (all == 0) return;
  for (int w = 0; w < warp; w++) before += warp_total[w];
  if (want < before || want - before >= warp_total[warp]) return;
  for (int v = v0; v < v1; v += 32) {
    unsigned long long inc = v + lane < v1 ? row.at(v + lane) : 0;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const unsigned long long o = __shfl_up_sync(0xffffffffu, inc, m);
      if (lane >= m) inc += o;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, before + inc > want);
    if (m) {
      if (lane == 0) p.tokens[c0 + b + a] = v + __ffs(m) - 1;
      return;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
}

template <int DT>
cudaError_t launch(const VerifyParams& p, cudaStream_t st) {
  constexpr int ctas = 8;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.num_seqs * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<DT>, p, ctas);
  note_launches(1);
  return e;
}

}  // namespace
}  // namespace exl3

using namespace exl3;

extern "C" exl3_status exl3_verify_drafts(const void* p, int64_t p_stride, const void* q,
                                          int64_t q_stride, exl3_dtype dt, int vocab, int num_seqs,
                                          int drafts, const int32_t* cu_draft, const int32_t* draft,
                                          const float* accept_u, const float* sample_u,
                                          int32_t* tokens, int32_t* accepted, int32_t* dropped,
                                          void* stream) {
  if (dt != EXL3_F16 && dt != EXL3_BF16 && dt != EXL3_F32) return EXL3_ERR_ARG;
  if (vocab < 1 || vocab > (1 << 24) || num_seqs < 0 || num_seqs > kMaxSeqs || drafts < 0 ||
      drafts > (1 << 30))
    return EXL3_ERR_SHAPE;
  if (p_stride < vocab || (q && q_stride < vocab)) return EXL3_ERR_ARG;
  if (num_seqs == 0) return EXL3_OK;
  const uintptr_t size = dt == EXL3_F32 ? 4 : 2;
  if (!p || reinterpret_cast<uintptr_t>(p) % size || reinterpret_cast<uintptr_t>(q) % size ||
      !cu_draft || !sample_u || !tokens || !accepted || !dropped ||
      (drafts > 0 && (!draft || !accept_u)))
    return EXL3_ERR_ARG;
  const VerifyParams a{p,        q,     p_stride, q_stride, vocab,  num_seqs, drafts,
                       cu_draft, draft, accept_u, sample_u, tokens, accepted, dropped};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dt == EXL3_F32    ? launch<EXL3_F32>(a, st)
                        : dt == EXL3_BF16 ? launch<EXL3_BF16>(a, st)
                                          : launch<EXL3_F16>(a, st);
  return e == cudaSuccess ? EXL3_OK : EXL3_ERR_CUDA;
}
