// Verification of drafted tokens against the target's probabilities.
//
// Draft j of a sequence (token x) is accepted while u_j q_j(x) < p_j(x).  At
// the first refusal a the next token is drawn from max(p_a - q_a, 0), after
// the last accepted draft from p_d, in either case as the first v whose
// cumulative weight exceeds sample_u times the total.
//
// Both decisions are exact.  u q is a product of two 24-bit values, formed in
// 64 bits; weights are summed as 64-bit integers in units of 2^-46, so the order
// of a sum does not matter, and no border between two tokens moves with the split
// of a row over threads.  (What is above 2^-22 is held whole; over a row of 2^17
// tokens the roundings of the others come to about 2^-38 of it.)
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

constexpr int kThreads = 256, kWarps = kThreads / 32, kPerSm = 1024 / kThreads;
// of a cluster, one cluster per sequence.  64 pairs of rows of 131072 fp32 (floor 10
// us): 16.6 us; 16 CTAs of 128 threads as fast, 16 of 256 and 8 of 128 slower
constexpr int kCtas = 8;
constexpr int kGroups = 8;  // parts of a warp's run whose sums are kept (draw: four lanes each)
constexpr int kUnroll = 4;  // 16-byte loads of p (and of q) in flight per thread

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
  const int32_t* step_lens;  // 0: the step did not serve the sequence (null: all served)
};

template <int DT>
__device__ __forceinline__ float value(const void* x, int64_t i) {
  if (DT == EXL3_F32) return __ldg(static_cast<const float*>(x) + i);
  return load_act(x, DT == EXL3_BF16, (size_t)i);
}

// A probability x rounded to units of 2^-46, h 2^23 + l, as the low bits of two
// floats: each a sum with a power of two (and a half, for signed ones) that leaves
// a step of 1; what the first leaves over is exact.  NaN and what is negative
// count as 0.  (Conversions to integers issue at an eighth of the rate.)
struct Limbs {
  uint32_t h, l;
};
constexpr float kH = 0x1p23f, kL = 0x1.8p23f;
__device__ __forceinline__ Limbs limbs(float x) {
  const float y = __saturatef(x);
  const float h = fmaf(y, 0x1p23f, kH);
  const float r = fmaf(y, 0x1p23f, -(h - kH));
  return Limbs{__float_as_uint(h), __float_as_uint(fmaf(r, 0x1p23f, kL))};
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// The weights of one row: p, or max(p - q, 0), or p without one token.  Chunks
// are the 16-byte pieces of p's memory: token v is element v + shift of them.
template <int DT>
struct Row {
  static constexpr int kSize = DT == EXL3_F32 ? 4 : 2, VEC = 16 / kSize;
  const uint8_t* p;  // the first chunk
  const uint8_t* q;  // the same tokens of q, or null
  int shift, vocab;
  int skip;          // a token without weight, -1: none
  int inner0, inner_n;  // the chunks that are the row's whole
  bool q_aligned;
  struct Chunk {
    uint4 p, q;
  };
  // element i of a chunk's 16 bytes
  static __device__ __forceinline__ float element(const uint4& w, int i) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    if (DT == EXL3_F32) return __uint_as_float(x[i]);
    if (DT == EXL3_BF16)
      return __uint_as_float(i & 1 ? x[i >> 1] & 0xFFFF0000u : x[i >> 1] << 16);
    return __half2float(__ushort_as_half((unsigned short)(x[i >> 1] >> (16 * (i & 1)))));
  }
  // the elements [lo, hi) of 16 bytes that need not be aligned, 0 for the others
  static __device__ __forceinline__ uint4 pieces(const uint8_t* at, int lo, int hi) {
    uint32_t x[4] = {};
#pragma unroll
    for (int i = 0; i < VEC; i++)
      if (i >= lo && i < hi) {
        if (DT == EXL3_F32)
          x[i] = __ldg(reinterpret_cast<const uint32_t*>(at) + i);
        else
          x[i >> 1] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(at) + i) << (16 * (i & 1));
      }
    return make_uint4(x[0], x[1], x[2], x[3]);
  }
  template <bool Q>
  __device__ __forceinline__ Chunk load(int c, int end) const {
    Chunk x;
    x.p = x.q = make_uint4(0, 0, 0, 0);
    if (c >= end) return x;
    const int64_t at = (int64_t)c * 16;
    const bool inner = (unsigned)(c - inner0) < (unsigned)inner_n;
    const int lo = inner ? 0 : shift - c * VEC, hi = inner ? VEC : lo + vocab;
    if (inner)
      x.p = __ldg(reinterpret_cast<const uint4*>(p + at));
    else
      x.p = pieces(p + at, lo, hi);
    if (Q) {
      if (inner && q_aligned)
        x.q = __ldg(reinterpret_cast<const uint4*>(q + at));
      else
        x.q = pieces(q + at, lo, hi);
    }
    return x;
  }
  // adds the weight of element i of chunk c, limb by limb
  template <bool Q>
  __device__ __forceinline__ void add(const Chunk& x, int c, int i, Limbs& sum) const {
    const float a = element(x.p, i);
    const Limbs w = limbs(a);
    Limbs minus{__float_as_uint(kH), __float_as_uint(kL)};
    bool some = c * VEC + i != skip + shift;
    if (Q) {
      const float b = element(x.q, i);
      minus = limbs(b);
      some = __saturatef(a) > __saturatef(b);
    }
    if (some) {
      sum.h += w.h - minus.h;
      sum.l += w.l - minus.l;
    }
  }
  static __device__ __forceinline__ long long whole(const Limbs& x) {
    return ((long long)(int)x.h << 23) + (int)x.l;
  }
  // the weight of a chunk
  template <bool Q>
  __device__ __forceinline__ long long weigh(const Chunk& x, int c) const {
    Limbs sum{0, 0};
#pragma unroll
    for (int i = 0; i < VEC; i++) add<Q>(x, c, i, sum);
    return whole(sum);
  }
  // the sums of a warp's groups of `per` loads by lane, to `sums`, and of all
  // `loads` of them
  template <bool Q>
  __device__ __forceinline__ long long sum(int c0, int loads, int per, int end, int lane,
                                           long long (*sums)[32]) const {
    long long all = 0, s = 0;
    int left = per, g = 0;
    // the loads whose chunks are all the row's whole, and aligned
    const int lo = c0 < inner0 ? 1 : 0;
    const int hi = Q && !q_aligned ? 0 : (min(inner0 + inner_n, end) - c0) / 32;
    const uint8_t* pl = p + (int64_t)(c0 + lane) * 16;
    const int64_t to_q = q - p;
#pragma unroll 1
    for (int it = 0; it < loads; it += kUnroll, pl += kUnroll * 512) {
      Chunk x[kUnroll];
      if (it >= lo && it + kUnroll <= hi) {
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
          x[u].p = __ldg(reinterpret_cast<const uint4*>(pl + u * 512));
          if (Q) x[u].q = __ldg(reinterpret_cast<const uint4*>(pl + to_q + u * 512));
        }
      } else {
#pragma unroll
        for (int u = 0; u < kUnroll; u++)  // (nothing past the run: `end` is its end)
          x[u] = load<Q>(c0 + (it + u) * 32 + lane, end);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; u++) {
        s += weigh<Q>(x[u], c0 + (it + u) * 32 + lane);
        if (--left == 0) {
          if (g < kGroups) sums[g][lane] = s;
          g++;
          all += s;
          s = 0;
          left = per;
        }
      }
    }
    for (int x = g; x < kGroups; x++) sums[x][lane] = x == g ? s : 0;
    return all + s;
  }
  // the first token of the chunks c0 .. whose cumulative weight is above want
  // (less than what they weigh), in every lane that finds it; -1 in the others
  template <bool Q>
  __device__ __forceinline__ int find(int c0, int per, int end, int lane, long long want) const {
#pragma unroll 1
    for (int it = 0; it < per; it++) {
      const int c = c0 + it * 32 + lane;
      const Chunk x = load<Q>(c, end);
      const long long mine = weigh<Q>(x, c);
      long long inc = mine;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, m);
        if (lane >= m) inc += o;
      }
      if (__any_sync(0xffffffffu, inc > want)) {
        if (!(inc > want && inc - mine <= want)) return -1;
        long long s = inc - mine;
        int v = -1;
#pragma unroll
        for (int i = 0; i < VEC; i++) {
          Limbs w{0, 0};
          add<Q>(x, c, i, w);
          s += whole(w);
          if (v < 0 && s > want) v = c * VEC + i - shift;
        }
        return v;
      }
      want -= __shfl_sync(0xffffffffu, inc, 31);
    }
    return -1;
  }
};

__device__ __forceinline__ long long load_remote(long long* at, int rank) {
  uint32_t a;
  long long v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// The token of a row that weighs `all` (`before` of it in the CTAs before this
// one): the first v with a cumulative weight above u * all.  The one warp whose
// run holds it writes it to place `at`.
template <int DT>
__device__ __forceinline__ void draw(const VerifyParams& p, const Row<DT>& row, int at, int b,
                                     int first, int per, int last, long long all, long long before,
                                     const long long* warp_total, const long long (*sums)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float u = fminf(fmaxf(__ldg(p.sample_u + b), 0.0f), 1.0f - 0x1p-24f);
  long long want =
      (long long)__umul64hi(__float2ull_rz(u * 0x1p64f), (unsigned long long)all) - before;
#pragma unroll
  for (int w = 0; w < kWarps; w++) want -= w < warp ? warp_total[w] : 0;
  if (want < 0 || want >= warp_total[warp]) return;
  // the group: four lanes sum one, then the sums before it (one after the other,
  // each over the warp, they took 1 us)
  long long mine = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) mine += sums[lane >> 2][(lane & 3) + 4 * i];
  mine += __shfl_xor_sync(0xffffffffu, mine, 1);
  mine += __shfl_xor_sync(0xffffffffu, mine, 2);
  long long inc = mine;
#pragma unroll
  for (int m = 4; m < 32; m <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, m);
    if (lane >= m) inc += o;
  }
  const int g = (__ffs(__ballot_sync(0xffffffffu, inc > want)) - 1) >> 2;
  want -= __shfl_sync(0xffffffffu, inc - mine, 4 * g);
  const int c = first + g * per * 32;
  const int v = row.q ? row.template find<true>(c, per, last, lane, want)
                      : row.template find<false>(c, per, last, lane, want);
  if (v >= 0) p.tokens[at] = v;
}

template <int DT>
__global__ void __launch_bounds__(kThreads, kPerSm) verify_kernel(VerifyParams p) {
  __shared__ long long total[2];  // of this CTA, by pass
  __shared__ long long warp_total[kWarps];
  __shared__ long long sums[kWarps][kGroups][32];
  __shared__ int s_accepted;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / kCtas, rank = blockIdx.x % kCtas;
  pdl_wait();
  const int c0 = __ldg(p.cu + b), c1 = __ldg(p.cu + b + 1);
  // the drafts that belong to sequences, and whether the step served this one (asked
  // for now, looked at once the drafts have been decided on: 0.1 us less than at once)
  int lo = __ldg(p.cu), hi = __ldg(p.cu + p.num_seqs);
  const int len = p.step_lens ? __ldg(p.step_lens + b) : 1;
  const int d = c0 >= 0 && c1 >= c0 && c1 <= p.drafts ? c1 - c0 : 0;
  // ---- the first refusal (every CTA for itself)
  const bool few = d < 32;  // (the drafts then stay in the lanes of the first warp)
  int mine = -1;
  if (warp == 0) {
    int a = d, x = 0;
    for (int j0 = 0; j0 < d; j0 += 32) {
      const int j = j0 + lane;
      bool no = false;
      if (j < d) {
        x = __ldg(p.draft + c0 + j);
        no = true;
        if (x >= 0 && x < p.vocab) {
          const double u = __ldg(p.accept_u + c0 + j);
          // (held to 0 .. 1, NaN as 0, as the weights are)
          const float pp = __saturatef(value<DT>(p.p, (int64_t)(c0 + j + b) * p.p_stride + x));
          const float qq =
              p.q ? __saturatef(value<DT>(p.q, (int64_t)(c0 + j) * p.q_stride + x)) : 1.0f;
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
    mine = lane < a ? x : -1;
  }
  // (a bound out of range says nothing)
  if (lo < 0 || lo > p.drafts) lo = 0;
  if (hi < 0 || hi > p.drafts) hi = p.drafts;
  const bool good = c0 >= lo && c1 >= c0 && c1 <= hi && len > 0;
  auto none = [&](int64_t from, int64_t to) {  // places of no token
#pragma unroll 1
    for (int64_t j = from + threadIdx.x; j < to; j += kThreads) p.tokens[j] = -1;
  };
  if (rank == 1) {  // (the first CTA has the tokens to write)
    if (b == 0) none(0, lo);
    if (b == p.num_seqs - 1) none((int64_t)hi + p.num_seqs, (int64_t)p.drafts + p.num_seqs);
  }
  // Left out: bounds that do not ascend, or a sequence that the step did not
  // serve, whose rows of p are those of no token: nothing is drawn, nothing came
  // that could be dropped.  (The bounds, held to lo .. hi, lead from the first
  // place to the last in steps up and down, and every place lies in a step up: of
  // a sequence that writes its own, or of one that is left out.)
  if (!good) {
    if (rank == 0) {
      const int from = b == 0 ? lo : min(max(c0, lo), hi);
      const int to = b == p.num_seqs - 1 ? hi : min(max(c1, lo), hi);
      none((int64_t)from + b, (int64_t)to + b + 1);
      if (threadIdx.x == 0) p.accepted[b] = p.dropped[b] = 0;
    }
    return;  // (the whole cluster: it waits for no one)
  }
  if (rank == 0 && warp == 0 && few && lane <= d) p.tokens[c0 + b + lane] = mine;
  __syncthreads();
  const int a = s_accepted;
  if (rank == 0) {
    // accepted drafts, then -1 (the drawn token's place too, until it is known)
    if (!few)
      for (int j = threadIdx.x; j <= d; j += kThreads)
        p.tokens[c0 + b + j] = j < a ? __ldg(p.draft + c0 + j) : -1;
    if (threadIdx.x == 0) {
      p.accepted[b] = a;
      p.dropped[b] = d - a;
    }
  }

  // ---- the row's weights: a run of chunks per warp
  Row<DT> row;
  row.vocab = p.vocab;
  row.skip = a < d && !p.q ? __ldg(p.draft + c0 + a) : -1;
  row.p = static_cast<const uint8_t*>(p.p) + (int64_t)(c0 + a + b) * p.p_stride * row.kSize;
  row.shift = (int)(reinterpret_cast<uintptr_t>(row.p) & 15) / row.kSize;
  row.p -= row.shift * row.kSize;
  row.q = nullptr;
  row.q_aligned = false;
  if (a < d && p.q) {
    row.q = static_cast<const uint8_t*>(p.q) + (int64_t)(c0 + a) * p.q_stride * row.kSize -
            row.shift * row.kSize;
    row.q_aligned = (reinterpret_cast<uintptr_t>(row.q) & 15) == 0;
  }
  const int end = (row.shift + p.vocab + row.VEC - 1) / row.VEC;  // chunks
  row.inner0 = row.shift > 0;
  row.inner_n = max((row.shift + p.vocab) / row.VEC - row.inner0, 0);
  // `per` of a run's loads are a group (short rows have fewer groups)
  constexpr int kAll = kCtas * kWarps;
  const int loads = (end + kAll * 32 - 1) / (kAll * 32);
  const int per = (loads + kGroups - 1) / kGroups;
  const int run = loads * 32;
  const int first = (rank * kWarps + warp) * run, last = min(first + run, end);
  long long all = 0, before = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; pass++) {
    const long long sum =
        warp_sum(row.q ? row.template sum<true>(first, loads, per, last, lane, sums[warp])
                       : row.template sum<false>(first, loads, per, last, lane, sums[warp]));
    if (lane == 0) warp_total[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
      long long t = 0;
#pragma unroll
      for (int w = 0; w < kWarps; w++) t += warp_total[w];
      total[pass] = t;
    }
    cluster_sync();
    all = before = 0;
#pragma unroll
    for (int r = 0; r < kCtas; r++) {
      const long long t = load_remote(&total[pass], r);
      if (r < rank) before += t;
      all += t;
    }
    // nothing is left of p without q: the target's own probabilities
    if (all > 0 || (!row.q && row.skip < 0)) break;
    row.q = nullptr;
    row.skip = -1;
  }
  // (no CTA leaves while another may read its sums: waited for at the end)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (all > 0) draw(p, row, c0 + b + a, b, first, per, last, all, before, warp_total, sums[warp]);
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int DT>
cudaError_t launch(const VerifyParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.num_seqs * kCtas);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_kernel<DT>, p);
  note_launches(1);
  return e;
}

}  // namespace
}  // namespace exl3

using namespace exl3;

extern "C" {

exl3_status exl3_verify_drafts_step(const void* p, int64_t p_stride, const void* q, int64_t q_stride,
                                    exl3_dtype dt, int vocab, int num_seqs, int drafts,
                                    const int32_t* cu_draft, const int32_t* draft,
                                    const float* accept_u, const float* sample_u,
                                    const int32_t* step_lens, int32_t* tokens, int32_t* accepted,
                                    int32_t* dropped, void* stream) {
  if (dt != EXL3_F16 && dt != EXL3_BF16 && dt != EXL3_F32) return EXL3_ERR_ARG;
  if (vocab < 1 || vocab > (1 << 24) || num_seqs < 0 || num_seqs > kMaxSeqs || drafts < 0 ||
      drafts > (1 << 30))
    return EXL3_ERR_SHAPE;
  if (p_stride < vocab || (q && q_stride < vocab)) return EXL3_ERR_ARG;
  if (num_seqs == 0) {
    if (drafts == 0) return EXL3_OK;
    if (!tokens) return EXL3_ERR_ARG;
    return cudaMemsetAsync(tokens, 0xFF, (size_t)drafts * 4, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? EXL3_OK
               : EXL3_ERR_CUDA;
  }
  const uintptr_t size = dt == EXL3_F32 ? 4 : 2;
  if (!p || reinterpret_cast<uintptr_t>(p) % size || reinterpret_cast<uintptr_t>(q) % size ||
      !cu_draft || !sample_u || !tokens || !accepted || !dropped ||
      (drafts > 0 && (!draft || !accept_u)))
    return EXL3_ERR_ARG;
  const VerifyParams a{p,     q,        p_stride, q_stride, vocab,    num_seqs, drafts,   cu_draft,
                       draft, accept_u, sample_u, tokens,   accepted, dropped,  step_lens};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dt == EXL3_F32    ? launch<EXL3_F32>(a, st)
                        : dt == EXL3_BF16 ? launch<EXL3_BF16>(a, st)
                                          : launch<EXL3_F16>(a, st);
  return e == cudaSuccess ? EXL3_OK : EXL3_ERR_CUDA;
}

exl3_status exl3_verify_drafts(const void* p, int64_t p_stride, const void* q, int64_t q_stride,
                               exl3_dtype dt, int vocab, int num_seqs, int drafts,
                               const int32_t* cu_draft, const int32_t* draft, const float* accept_u,
                               const float* sample_u, int32_t* tokens, int32_t* accepted,
                               int32_t* dropped, void* stream) {
  return exl3_verify_drafts_step(p, p_stride, q, q_stride, dt, vocab, num_seqs, drafts, cu_draft,
                                 draft, accept_u, sample_u, nullptr, tokens, accepted, dropped, stream);
}

}  // extern "C"
