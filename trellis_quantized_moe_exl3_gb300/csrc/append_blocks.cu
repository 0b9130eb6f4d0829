// The append of keys and values to a paged E4M3 cache with a scale per block
// (page) and kv head.
//
//   scale = the least 2^e with max |x| <= 448 * 2^e over the block's tokens
//   byte  = E4M3_RNE(x / scale)
//
// Tokens come to a block a few at a time, so its scale only grows: where new
// tokens need more than it covers, the older tokens' bytes are brought to the
// new one.  Scales are powers of two so that this is exact (but for values
// that leave E4M3's normal range, below 2^-6 of the scale): however often a
// block has grown, its tokens have been rounded once, and E4M3 loses nothing
// by it, being a floating type.  A block that begins with a new token starts
// anew.
//
// A unit (block, kv head, keys or values) belongs to a team of lane groups (a
// head vector's lanes, as in norm_rope_kernel): one group where a step brings
// a few tokens per sequence, a whole CTA for prompts.  The first kHold rows of
// a group stay in registers between the maximum and the rounding, later ones
// (long blocks) are formed twice.
#include "norm_rope.cuh"

namespace exl3 {
namespace {

constexpr int kThreads = 128;

// the least 2^e >= top / 448, within the range of scales
__device__ __forceinline__ float scale_for(float top) {
  const uint32_t u = __float_as_uint(fmaxf(top, 448.0f * kLeastScale));
  // top = m 2^x, 1 <= m < 2, against 448 = 1.75 * 2^8
  const uint32_t e = (u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
  return fminf(__uint_as_float(e << 23), kMostScale);
}

template <int LPR, int TEAM, int BF16, int INTER>
__global__ void __launch_bounds__(kThreads) append_blocks_kernel(NormRopeParams p) {
  constexpr int NG = kThreads / LPR, NT = NG / TEAM;
  constexpr int kHold = TEAM == 1 ? 4 : 8;
  static_assert(TEAM == 1 || TEAM == NG, "a team is a lane group or the CTA");
  __shared__ float tops[NG];
  const int wl = threadIdx.x & 31;
  const int grp = threadIdx.x / LPR, lane = threadIdx.x % LPR;
  const uint32_t mask = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1) << (wl / LPR * LPR);
  const int P = p.cache.page_size;
  pdl_wait();

  // ---- the block: sequence b has the slots cu_q[b] / P + 2 b .. of the grid,
  // as many as it can touch blocks (every warp for itself)
  const int slot = blockIdx.x;
  int below = 0;
  for (int b = wl; b < p.batch.num_seqs; b += 32)
    below += __ldg(p.batch.cu_q + b + 1) / P + 2 * (b + 1) <= slot;
  const int b = __reduce_add_sync(0xffffffffu, below);
  if (b >= p.batch.num_seqs) return;
  int32_t bad = 0;
  const Seq s = load_seq(p.batch, b, &bad);
  const int start = s.len - s.n;  // position of the first new token
  if (s.n > 0 && start < 0) bad |= kStatusBadBatch;
  const int from = max(start, 0);
  const int blk = from / P + slot - (s.q0 / P + 2 * b);
  const int lo = max(from, blk * P), hi = (int)min((long long)s.len, ((long long)blk + 1) * P);
  int page = -1;
  if (s.n > 0 && blk >= from / P && lo < hi) {
    page = __ldg(p.batch.table + (int64_t)b * p.batch.table_stride + blk);
    if (page < 0 || page >= p.cache.num_pages) {
      bad |= kStatusBadPage;
      page = -1;
    }
  }
  if (bad && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(p.status, bad);
  if (page < 0) return;

  // ---- the unit
  const int unit = blockIdx.y * NT + (TEAM == 1 ? grp : 0);
  if (unit >= 2 * p.set[1].heads) return;  // (whole groups; no barrier below unless TEAM = NG)
  const int kv = unit & 1, h = unit >> 1, me = TEAM == 1 ? 0 : grp;
  const HeadSet& hs = p.set[1 + kv];
  const bool in_row = lane * 8 < p.dim;
  const bool turn = !kv && p.inv_freq && lane < p.rot / 8;
  int ca = lane * 8, cb = ca + 4;  // first channels of the lane's two runs
  if (!INTER && lane < p.rot / 8) {
    ca = lane * 4;
    cb = ca + p.rot / 2;
  }
  float* const scale_at = const_cast<float*>(kv ? p.cache.v_scale : p.cache.k_scale) +
                          page * p.cache.scale_stride + h;
  const int older = lo - blk * P, rows = hi - lo;
  const float held = older > 0 ? *scale_at : 0.0f;
  uint64_t turns[4];
  if (turn) {
#pragma unroll
    for (int e = 0; e < 4; e++) turns[e] = turns_of(__ldg(p.inv_freq + 4 * lane + e));
  }
  float wt[8] = {};
  if (hs.weight && in_row) {
    unpack4(__ldg(reinterpret_cast<const uint2*>(hs.weight + ca)), BF16, wt);
    unpack4(__ldg(reinterpret_cast<const uint2*>(hs.weight + cb)), BF16, wt + 4);
  }
  const int t0 = s.q0 + lo - start;  // row of the block's first new token
  const uint16_t* const x0 = hs.x + (int64_t)t0 * hs.ts + h * hs.hs;

  struct Raw {
    uint2 a, b;
  };
  auto load = [&](int r) {
    Raw w{make_uint2(0, 0), make_uint2(0, 0)};
    if (in_row && r < rows) {
      w.a = *reinterpret_cast<const uint2*>(x0 + r * hs.ts + ca);
      w.b = *reinterpret_cast<const uint2*>(x0 + r * hs.ts + cb);
    }
    return w;
  };
  // new token r of the block, normed and rotated
  auto form = [&](const Raw& w, int r, float* v) {
    unpack4(w.a, BF16, v);
    unpack4(w.b, BF16, v + 4);
    if (hs.weight) {
      float sq = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; e++) sq = fmaf(v[e], v[e], sq);
#pragma unroll
      for (int m = LPR / 2; m > 0; m >>= 1) sq += __shfl_xor_sync(mask, sq, m, LPR);
      const float f = rsqrtf(fmaf(sq, p.inv_dim, p.eps));
#pragma unroll
      for (int e = 0; e < 8; e++) v[e] = v[e] * f * wt[e];
    }
    if (turn) {
      const int pos = p.positions ? __ldg(p.positions + min(t0 + r, p.T - 1)) : lo + r;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        float sn, c;
        sincospif((float)(int32_t)((turns[e] * (uint64_t)(int64_t)pos) >> 32) * 0x1p-31f, &sn, &c);
        float& x = v[INTER ? 2 * e : e];
        float& y = v[INTER ? 2 * e + 1 : 4 + e];
        const float x1 = fmaf(x, c, -(y * sn)), y1 = fmaf(y, c, x * sn);
        x = x1;
        y = y1;
      }
    }
  };

  // ---- the largest value
  float top = 0.0f;
  float keep[kHold][8];
  {
    Raw raw[kHold];
#pragma unroll
    for (int i = 0; i < kHold; i++) raw[i] = load(me + i * TEAM);
#pragma unroll
    for (int i = 0; i < kHold; i++) {
      if (TEAM == 1 && i * TEAM >= rows) break;  // (the same in the whole group)
      form(raw[i], me + i * TEAM, keep[i]);
#pragma unroll
      for (int e = 0; e < 8; e++) top = fmaxf(top, fabsf(keep[i][e]));
    }
  }
  for (int r0 = kHold * TEAM; r0 < rows; r0 += TEAM) {
    float v[8];
    form(load(r0 + me), r0 + me, v);
#pragma unroll
    for (int e = 0; e < 8; e++) top = fmaxf(top, fabsf(v[e]));
  }
#pragma unroll
  for (int m = LPR / 2; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, m, LPR));
  if (TEAM > 1) {
    if (lane == 0) tops[grp] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NG; i++) top = fmaxf(top, tops[i]);
  }

  // ---- the scale
  if (!(held >= 0.0f && held <= kMostScale)) {  // no scale: the block is left alone
    if (lane == 0 && me == 0) atomicOr(p.status, kStatusBadScale);
    return;
  }
  const float old = fmaxf(held, kLeastScale);
  const float scale = top <= 448.0f * old ? old : scale_for(top);
  if (lane == 0 && me == 0) *scale_at = scale;
  uint8_t* const dst = const_cast<uint8_t*>(kv ? p.cache.v : p.cache.k) +
                       page * p.cache.page_bytes + h * p.cache.head_bytes;

  // ---- older tokens, where it has grown
  if (older > 0 && scale != old && in_row) {
    const float ratio = old / scale;
    for (int r = me; r < older; r += TEAM) {
      uint2* at = reinterpret_cast<uint2*>(dst + r * p.cache.token_bytes + lane * 8);
      const uint2 w = *at;
      uint32_t o[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const uint32_t x = i ? w.y : w.x;
        const float2 a = e4m3_float2(x), c = e4m3_float2(x >> 16);
        o[i] = e4m3_pack2(a.x * ratio, a.y * ratio) |
               (e4m3_pack2(c.x * ratio, c.y * ratio) << 16);
      }
      *at = make_uint2(o[0], o[1]);
    }
  }

  // ---- new tokens
  const bool exact = (__float_as_uint(scale) & 0x7FFFFFu) == 0;  // (its inverse is a float)
  const float inv = 1.0f / scale;
  auto store = [&](int r, float* v) {
    if (!in_row || r >= rows) return;
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = exact ? v[e] * inv : __fdiv_rn(v[e], scale);
    uint8_t* at = dst + (int64_t)(older + r) * p.cache.token_bytes;
    *reinterpret_cast<uint32_t*>(at + ca) = e4m3_pack2(v[0], v[1]) | (e4m3_pack2(v[2], v[3]) << 16);
    *reinterpret_cast<uint32_t*>(at + cb) = e4m3_pack2(v[4], v[5]) | (e4m3_pack2(v[6], v[7]) << 16);
  };
#pragma unroll
  for (int i = 0; i < kHold; i++) store(me + i * TEAM, keep[i]);
  for (int r0 = kHold * TEAM; r0 < rows; r0 += TEAM) {
    float v[8];
    form(load(r0 + me), r0 + me, v);
    store(r0 + me, v);
  }
}

template <int LPR, int TEAM>
cudaError_t launch_team(const NormRopeParams& p, cudaStream_t st) {
  constexpr int NT = kThreads / LPR / TEAM;
  const dim3 grid((unsigned)(p.T / p.cache.page_size + 2 * p.batch.num_seqs),
                  (unsigned)((2 * p.set[1].heads + NT - 1) / NT));
  const dim3 block(kThreads);
  note_launches(1);
  if (p.inter)
    return p.bf16 ? launch_pdl(append_blocks_kernel<LPR, TEAM, 1, 1>, grid, block, 0, st, p)
                  : launch_pdl(append_blocks_kernel<LPR, TEAM, 0, 1>, grid, block, 0, st, p);
  return p.bf16 ? launch_pdl(append_blocks_kernel<LPR, TEAM, 1, 0>, grid, block, 0, st, p)
                : launch_pdl(append_blocks_kernel<LPR, TEAM, 0, 0>, grid, block, 0, st, p);
}

template <int LPR>
cudaError_t launch_lpr(const NormRopeParams& p, cudaStream_t st) {
  return p.batch.max_q <= 4 ? launch_team<LPR, 1>(p, st) : launch_team<LPR, kThreads / LPR>(p, st);
}

}  // namespace

cudaError_t launch_append_blocks(const NormRopeParams& p, cudaStream_t st) {
  if (p.set[0].heads > 0) {
    NormRopeParams q = p;  // the queries alone
    q.set[1] = q.set[2] = HeadSet{};
    const cudaError_t e = launch_norm_rope(q, st);
    if (e != cudaSuccess) return e;
  }
  return p.dim <= 64 ? launch_lpr<8>(p, st) : p.dim <= 128 ? launch_lpr<16>(p, st)
                                                           : launch_lpr<32>(p, st);
}

}  // namespace exl3
