// RMS norm of every query and key head, the position rotation, and the append
// of keys and values to a paged cache, in one pass over the projections'
// output.
//
//   y = x / sqrt(mean(x^2) + eps) * w                       (weight given)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = position * inv_freq[i]
//
// The pass reads and writes every element once and computes ~10 operations on
// it, so memory is what it cannot do without; small calls are bounded by
// latency.  7168 tokens of 40 heads take 28.3 us, 77 % of the memory's rate,
// with 63 % of the issue slots taken and no unit saturated.
//
// A row (one head vector) belongs to LPR lanes of 8 channels.  A lane's
// channels are two runs of 4 that hold the two sides of 4 rotation pairs
// (halves rot/2 apart, or 8 neighbours when interleaved), so the rotation
// needs no other lane and the sum of squares is the only shuffle.  A lane
// group takes head j of all TOK tokens of the block, with the loads of its
// next head in flight; cos and sin of a token are computed once for all heads
// (in shared memory, 4 + 4 floats per lane and row).
//
// The angle never exists as a number of radians: inv_freq is turned into a
// 64-bit fixed-point fraction of a turn per position (integer arithmetic),
// its product with the position wraps modulo one turn exactly, and the top
// bits go to sincospi.  A position of 2^31 loses no more than position 1.
#include "norm_rope.cuh"

namespace exl3 {
namespace {

// small blocks: the two barriers of a block stall few warps (7168 tokens of 40
// heads, 28.4 us; 35.3 us with 256 threads, 30.4 us with registers for one more
// block per SM, 31.5 us as a persistent loop that prefetches across groups)
constexpr int kThreads = 128;

// LPR lanes hold a row of up to 8 LPR channels; TOK tokens per block, heads
// blockIdx.y * slice .. + slice - 1 of q, k and v counted through.
template <int LPR, int TOK, int BF16, int INTER>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(NormRopeParams p, int slice) {
  constexpr int NG = kThreads / LPR;
  __shared__ float4 cs[2][TOK][32];   // cos, sin of pairs 4 i .. 4 i + 3
  __shared__ int64_t dst_k[TOK];      // byte offset of the token in the cache, -1: none
  __shared__ int32_t s_pos[TOK];
  pdl_wait();
  const int t0 = blockIdx.x * TOK;
  const int nt = min(TOK, p.T - t0);
  const int all = p.set[0].heads + p.set[1].heads + p.set[2].heads;
  const int jend = min((int)(blockIdx.y + 1) * slice, all);
  const int grp = threadIdx.x / LPR, lane = threadIdx.x % LPR;
  const bool in_row = lane * 8 < p.dim;
  const int rot_lanes = p.rot / 8;
  // first channels of the lane's two runs
  int ca = lane * 8, cb = ca + 4;
  if (!INTER && lane < rot_lanes) {
    ca = lane * 4;
    cb = ca + p.rot / 2;
  }

  auto set_of = [&](int j, int* h) {
    int s = 0;
    if (j >= p.set[0].heads) {
      j -= p.set[0].heads;
      s = 1;
      if (j >= p.set[1].heads) {
        j -= p.set[1].heads;
        s = 2;
      }
    }
    *h = j;
    return s;
  };
  struct Raw {
    uint2 a[TOK], b[TOK];
  };
  auto load = [&](int j, Raw& r) {
    int h;
    const int s = set_of(j, &h);
    const HeadSet& hs = p.set[s];
    const uint16_t* x = hs.x + (int64_t)t0 * hs.ts + h * hs.hs;
#pragma unroll
    for (int t = 0; t < TOK; t++) {
      r.a[t] = r.b[t] = make_uint2(0, 0);
      if (j < jend && in_row && t < nt) {
        r.a[t] = *reinterpret_cast<const uint2*>(x + t * hs.ts + ca);
        r.b[t] = *reinterpret_cast<const uint2*>(x + t * hs.ts + cb);
      }
    }
  };
  // the first rows are in flight while positions, pages and angles are found
  int j = blockIdx.y * slice + grp;
  Raw nxt;
  load(j, nxt);

  const int w = threadIdx.x >> 5, wl = threadIdx.x & 31;
  if (p.append) {
    if (w < nt) {  // warp w: the sequence and the place of token w
      const int t = t0 + w;
      int below = 0;  // sequences that end at or before t
      for (int b = wl; b < p.batch.num_seqs; b += 32) below += __ldg(p.batch.cu_q + b + 1) <= t;
      const int b = __reduce_add_sync(0xffffffffu, below);
      int64_t off = -1;
      int pos = 0;
      int32_t bad = 0;
      if (b < p.batch.num_seqs) {
        const Seq s = load_seq(p.batch, b, &bad);
        pos = s.len - s.n + (t - s.q0);
        // (where cu_q does not ascend, the sequence found need not hold t)
        if (t < s.q0 || t - s.q0 >= s.n || pos < 0) {
          bad |= kStatusBadBatch;
        } else {
          const int pi = pos / p.cache.page_size;
          const int page = __ldg(p.batch.table + (int64_t)b * p.batch.table_stride + pi);
          if (page < 0 || page >= p.cache.num_pages)
            bad |= kStatusBadPage;
          else
            off = page * p.cache.page_bytes +
                  (int64_t)(pos - pi * p.cache.page_size) * p.cache.token_bytes;
        }
      } else {
        off = -2;  // padding: nothing is written for this token
      }
      if (wl == 0) {
        dst_k[w] = off;
        s_pos[w] = p.positions ? __ldg(p.positions + t) : pos;
        if (bad && blockIdx.y == 0) atomicOr(p.status, bad);
      }
    }
  } else if (threadIdx.x < nt && p.positions) {
    s_pos[threadIdx.x] = __ldg(p.positions + t0 + threadIdx.x);
  }
  __syncthreads();
  if (p.inv_freq) {
    const int half = p.rot / 2;
    for (int i = threadIdx.x; i < TOK * 128; i += kThreads) {
      const int t = i >> 7, f = i & 127;
      if (t < nt && f < half) {
        const float2 v = cos_sin(s_pos[t], __ldg(p.inv_freq + f));
        reinterpret_cast<float*>(&cs[0][t][0])[f] = v.x;
        reinterpret_cast<float*>(&cs[1][t][0])[f] = v.y;
      }
    }
    __syncthreads();
  }

  for (int jb = blockIdx.y * slice; jb < jend; jb += NG, j += NG) {
    Raw raw = nxt;
    load(j + NG, nxt);
    int h;
    const int s = set_of(j, &h);  // (past the end: computes on zeros, stores nothing)
    const HeadSet& hs = p.set[s];
    const bool turn = p.inv_freq && s < 2 && lane < rot_lanes;
    float wt[8];
    if (hs.weight && in_row) {
      unpack4(__ldg(reinterpret_cast<const uint2*>(hs.weight + ca)), BF16, wt);
      unpack4(__ldg(reinterpret_cast<const uint2*>(hs.weight + cb)), BF16, wt + 4);
    }
    const bool to_cache = p.append && s > 0;
    float scale = 1.0f;
    if (to_cache && p.e4m3 && j < jend) {
      const float* sc = s == 1 ? p.cache.k_scale : p.cache.v_scale;
      if (sc) scale = __ldg(sc + h);
    }
    uint16_t* out = to_cache ? nullptr : hs.out + (int64_t)t0 * hs.ots + h * hs.ohs;
#pragma unroll
    for (int t = 0; t < TOK; t++) {
      float v[8];
      unpack4(raw.a[t], BF16, v);
      unpack4(raw.b[t], BF16, v + 4);
      float2* v2 = reinterpret_cast<float2*>(v);
      if (hs.weight) {  // (one set per lane group, the shuffle stays inside it)
        float2 q2 = mul2(v2[0], v2[0]);
#pragma unroll
        for (int e = 1; e < 4; e++) q2 = fma2(v2[e], v2[e], q2);
        float sq = q2.x + q2.y;
        const uint32_t mask = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1) << (wl / LPR * LPR);
#pragma unroll
        for (int m = LPR / 2; m > 0; m >>= 1) sq += __shfl_xor_sync(mask, sq, m, LPR);
        const float r = rsqrtf(fmaf(sq, p.inv_dim, p.eps));
#pragma unroll
        for (int e = 0; e < 4; e++)
          v2[e] = mul2(mul2(v2[e], make_float2(r, r)), make_float2(wt[2 * e], wt[2 * e + 1]));
      }
      if (turn) {
        const float4 c = cs[0][t][lane], sn = cs[1][t][lane];
        if (INTER) {
          // (a, b) of a pair share a register pair: a' = a c - b s, b' = a s + b c
          const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
          for (int e = 0; e < 4; e++)
            v2[e] = fma2(v2[e], make_float2(cc[e], cc[e]),
                         mul2(make_float2(v2[e].y, v2[e].x), make_float2(-ss[e], ss[e])));
        } else {
          const float2 c2[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
          const float2 s2[2] = {make_float2(sn.x, sn.y), make_float2(sn.z, sn.w)};
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const float2 a = v2[e], b = v2[2 + e];
            v2[e] = fma2(a, c2[e], mul2(b, make_float2(-s2[e].x, -s2[e].y)));
            v2[2 + e] = fma2(b, c2[e], mul2(a, s2[e]));
          }
        }
      }
      if (j < jend && in_row && t < nt) {
        if (!to_cache) {
          if (!p.append || dst_k[t] != -2) {
            uint16_t* o = out + t * hs.ots;
            *reinterpret_cast<uint2*>(o + ca) = pack4(v, BF16);
            *reinterpret_cast<uint2*>(o + cb) = pack4(v + 4, BF16);
          }
        } else if (dst_k[t] >= 0) {
          uint8_t* base = const_cast<uint8_t*>(s == 1 ? p.cache.k : p.cache.v) + dst_k[t] +
                          h * p.cache.head_bytes;
          if (p.e4m3) {
            if (scale == 0.0f) {  // (whatever is stored stands for 0; a NaN stays one)
#pragma unroll
              for (int e = 0; e < 8; e++) v[e] = v[e] != v[e] ? v[e] : 0.0f;
            } else if (scale != 1.0f) {
#pragma unroll
              for (int e = 0; e < 8; e++) v[e] = __fdiv_rn(v[e], scale);
            }
            *reinterpret_cast<uint32_t*>(base + ca) =
                e4m3_pack2(v[0], v[1]) | (e4m3_pack2(v[2], v[3]) << 16);
            *reinterpret_cast<uint32_t*>(base + cb) =
                e4m3_pack2(v[4], v[5]) | (e4m3_pack2(v[6], v[7]) << 16);
          } else {
            *reinterpret_cast<uint2*>(base + ca * 2) = pack4(v, BF16);
            *reinterpret_cast<uint2*>(base + cb * 2) = pack4(v + 4, BF16);
          }
        }
      }
    }
  }
}

template <int LPR, int TOK>
cudaError_t launch_cfg(const NormRopeParams& p, cudaStream_t st) {
  const int all = p.set[0].heads + p.set[1].heads + p.set[2].heads;
  const int nx = (p.T + TOK - 1) / TOK;
  constexpr int groups = kThreads / LPR;
  // few tokens: the heads are spread over several blocks as well, so that the
  // GPU is filled
  int slices = (2 * kSms + nx - 1) / nx;
  const int most = (all + groups - 1) / groups;
  if (slices > most) slices = most;
  const int slice = (all + slices - 1) / slices;
  const dim3 grid((unsigned)nx, (unsigned)((all + slice - 1) / slice));
  const dim3 block(kThreads);
  cudaError_t err;
  if (p.inter)
    err = p.bf16 ? launch_pdl(norm_rope_kernel<LPR, TOK, 1, 1>, grid, block, 0, st, p, slice)
                 : launch_pdl(norm_rope_kernel<LPR, TOK, 0, 1>, grid, block, 0, st, p, slice);
  else
    err = p.bf16 ? launch_pdl(norm_rope_kernel<LPR, TOK, 1, 0>, grid, block, 0, st, p, slice)
                 : launch_pdl(norm_rope_kernel<LPR, TOK, 0, 0>, grid, block, 0, st, p, slice);
  note_launches(1);
  return err;
}

template <int LPR>
cudaError_t launch_lpr(const NormRopeParams& p, cudaStream_t st) {
  // four tokens per block (four rows of a lane group in flight) once that
  // still gives every SM a few blocks
  return p.T >= 4 * 4 * kSms ? launch_cfg<LPR, 4>(p, st) : launch_cfg<LPR, 1>(p, st);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t st) {
  return p.dim <= 64 ? launch_lpr<8>(p, st) : p.dim <= 128 ? launch_lpr<16>(p, st)
                                                           : launch_lpr<32>(p, st);
}

}  // namespace exl3
