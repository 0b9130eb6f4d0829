// RMS norm of every query and key head, the position rotation, and the append
// of keys and values to a paged cache, in one pass over the projections'
// output.
//
//   y = x / sqrt(mean(x^2) + eps) * w                       (weight given)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = position * inv_freq[i]
//
// The pass reads and writes every element once and computes ~10 operations on
// it, so memory bounds it; small calls are bounded by latency.  A row (one
// head vector) belongs to LPR lanes holding 8 channels (16 bytes) each: the
// sum of squares is a shuffle reduction, the half-split pair's partner sits in
// a lane rotary_dim/16 away, the interleaved one in the same lane.  A block
// takes a few tokens with all their heads, so each token's cos and sin are
// computed once (into shared memory) for all of them.
//
// The angle never exists as a number of radians: inv_freq is turned into a
// 64-bit fixed-point fraction of a turn per position (integer arithmetic),
// its product with the position wraps modulo one turn exactly, and the top
// bits go to sincospi.  A position of 2^31 loses no more than position 1.
#include <math.h>

#include "attn.cuh"
#include "common.cuh"

namespace exl3 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 4;
constexpr int kUnroll = 4;   // rows of a lane group in flight

// 2^64 * f / (2 pi) modulo 2^64 for 0 <= f < 64.  f = M 2^(e-1086) with M the
// 53-bit mantissa shifted to the top of 64 bits; C = floor(2^66 / (2 pi)), so
// the result is hi64(M C) 2^(e-1024), with a relative error below 2^-62.
__device__ __forceinline__ uint64_t turns_of(double f) {
  const uint64_t u = (uint64_t)__double_as_longlong(f);
  const int e = (int)(u >> 52) & 0x7FF;
  if (e == 0) return 0;
  const uint64_t m = ((u & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull) << 11;
  const uint64_t p = __umul64hi(m, 0xA2F9836E4E441529ull);
  const int s = 1024 - e;
  if (s >= 64 || s < -5) return 0;
  const uint64_t t = s >= 0 ? p >> s : p << -s;
  return (u >> 63) ? 0 - t : t;
}

__device__ __forceinline__ float2 cos_sin(int32_t pos, double inv_freq) {
  const uint64_t phase = turns_of(inv_freq) * (uint64_t)(int64_t)pos;
  float s, c;
  sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ void unpack8(const uint4& r, int bf16, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if (bf16) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8], int bf16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if (bf16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// LPR lanes hold a row of up to 8 LPR channels.
template <int LPR>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(NormRopeParams p, int tok, int slice) {
  constexpr int NG = kThreads / LPR;
  __shared__ float2 cs[kMaxTok][128];
  __shared__ int64_t dst_k[kMaxTok];  // byte offset of the token in the cache, -1: none
  __shared__ int32_t s_pos[kMaxTok];
  pdl_wait();
  const int t0 = blockIdx.x * tok;
  const int nt = min(tok, p.T - t0);
  const int all = p.set[0].heads + p.set[1].heads + p.set[2].heads;
  const int j0 = blockIdx.y * slice;
  const int nj = min(slice, all - j0);
  const int rows = nt * nj;
  const int grp = threadIdx.x / LPR, lane = threadIdx.x % LPR;
  const int c0 = lane * 8;
  const bool in_row = c0 < p.dim;

  // row i of the block: token, set (0 q, 1 k, 2 v) and head
  auto locate = [&](int i, int* t, int* set, int* h) {
    *t = i / nj;
    int j = j0 + i - *t * nj;
    int s = 0;
    if (j >= p.set[0].heads) {
      j -= p.set[0].heads;
      s = 1;
      if (j >= p.set[1].heads) {
        j -= p.set[1].heads;
        s = 2;
      }
    }
    *set = s;
    *h = j;
  };
  auto load = [&](int i) -> uint4 {
    if (i >= rows || !in_row) return make_uint4(0, 0, 0, 0);
    int t, s, h;
    locate(i, &t, &s, &h);
    const HeadSet& hs = p.set[s];
    return *reinterpret_cast<const uint4*>(hs.x + (int64_t)(t0 + t) * hs.ts + h * hs.hs + c0);
  };
  // the first rows are in flight while positions, pages and angles are found
  uint4 raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; u++) raw[u] = load(grp + u * NG);

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
        if (s.n <= 0 || t < s.q0 || pos < 0) {
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
        if (bad && j0 == 0) atomicOr(p.status, bad);
      }
    }
  } else if (threadIdx.x < nt && p.positions) {
    s_pos[threadIdx.x] = __ldg(p.positions + t0 + threadIdx.x);
  }
  __syncthreads();
  if (p.inv_freq) {
    const int half = p.rot / 2;
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int t = i / half, f = i - t * half;
      cs[t][f] = cos_sin(s_pos[t], __ldg(p.inv_freq + f));
    }
    __syncthreads();
  }

  const int rot_half = p.rot / 2, rot_lanes = p.rot / 8, half_lanes = p.rot / 16;
  for (int i0 = grp; i0 < rows; i0 += NG * kUnroll) {
    uint4 nxt[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; u++) nxt[u] = load(i0 + (kUnroll + u) * NG);
#pragma unroll
    for (int u = 0; u < kUnroll; u++) {
      // (a group past the last row computes on zeros: its lanes take part in
      // the shuffles)
      const int i = min(i0 + u * NG, rows - 1);
      const bool live = i0 + u * NG < rows;
      int t, s, h;
      locate(i, &t, &s, &h);
      const HeadSet& hs = p.set[s];
      float v[8];
      unpack8(raw[u], p.bf16, v);
      float sq = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; e++) sq = fmaf(v[e], v[e], sq);
#pragma unroll
      for (int m = LPR / 2; m > 0; m >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, m, LPR);
      if (hs.weight && in_row) {
        const float r = 1.0f / sqrtf(sq / (float)p.dim + p.eps);
        float wv[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(hs.weight + c0)), p.bf16, wv);
#pragma unroll
        for (int e = 0; e < 8; e++) v[e] = v[e] * r * wv[e];
      }
      if (p.inv_freq) {
        if (p.inter) {
          if (lane < rot_lanes && s < 2) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const float2 a = cs[t][4 * lane + e];
              const float x0 = v[2 * e], x1 = v[2 * e + 1];
              v[2 * e] = x0 * a.x - x1 * a.y;
              v[2 * e + 1] = x0 * a.y + x1 * a.x;
            }
          }
        } else {
          const bool lo = lane < half_lanes;
          const int src = lo ? lane + half_lanes : lane - half_lanes;
#pragma unroll
          for (int e = 0; e < 8; e++) {
            const float o = __shfl_sync(0xffffffffu, v[e], src, LPR);
            if (lane < rot_lanes && s < 2) {
              const float2 a = cs[t][lo ? c0 + e : c0 + e - rot_half];
              v[e] = lo ? v[e] * a.x - o * a.y : o * a.y + v[e] * a.x;
            }
          }
        }
      }
      if (live && in_row) {
        if (s == 0 || !p.append) {
          if (!p.append || dst_k[t] != -2)
            *reinterpret_cast<uint4*>(hs.out + (int64_t)(t0 + t) * hs.ots + h * hs.ohs + c0) =
                pack8(v, p.bf16);
        } else if (dst_k[t] >= 0) {
          uint8_t* base = const_cast<uint8_t*>(s == 1 ? p.cache.k : p.cache.v) + dst_k[t] +
                          h * p.cache.head_bytes;
          if (p.e4m3) {
            const float* sc = s == 1 ? p.cache.k_scale : p.cache.v_scale;
            if (sc) {
              const float f = __ldg(sc + h);
#pragma unroll
              for (int e = 0; e < 8; e++) v[e] = __fdiv_rn(v[e], f);
            }
            uint2 b;
            b.x = e4m3_pack2(v[0], v[1]) | (e4m3_pack2(v[2], v[3]) << 16);
            b.y = e4m3_pack2(v[4], v[5]) | (e4m3_pack2(v[6], v[7]) << 16);
            *reinterpret_cast<uint2*>(base + c0) = b;
          } else {
            *reinterpret_cast<uint4*>(base + c0 * 2) = pack8(v, p.bf16);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; u++) raw[u] = nxt[u];
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t st) {
  const int all = p.set[0].heads + p.set[1].heads + p.set[2].heads;
  // many tokens: blocks of kMaxTok tokens with all heads; few: one token per
  // block and its heads over several blocks, so that the GPU is filled
  const int tok = p.T >= kSms * 8 * kMaxTok ? kMaxTok : p.T >= kSms * 16 ? 2 : 1;
  const int nx = (p.T + tok - 1) / tok;
  const int lpr = p.dim <= 64 ? 8 : p.dim <= 128 ? 16 : 32;
  const int groups = kThreads / lpr;
  int slices = (2 * kSms + nx - 1) / nx;
  const int most = (all + groups - 1) / groups;
  if (slices > most) slices = most;
  const int slice = (all + slices - 1) / slices;
  const dim3 grid((unsigned)nx, (unsigned)((all + slice - 1) / slice));
  cudaError_t err;
  if (lpr == 8)
    err = launch_pdl(norm_rope_kernel<8>, grid, dim3(kThreads), 0, st, p, tok, slice);
  else if (lpr == 16)
    err = launch_pdl(norm_rope_kernel<16>, grid, dim3(kThreads), 0, st, p, tok, slice);
  else
    err = launch_pdl(norm_rope_kernel<32>, grid, dim3(kThreads), 0, st, p, tok, slice);
  note_launches(1);
  return err;
}

}  // namespace exl3
