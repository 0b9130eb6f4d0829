// The append of keys and values to a paged E4M3 cache with a scale per block
// (page) and kv head, queries normed and rotated in the same launch.
//
//   scale = the least 2^e with max |x| <= 448 * 2^e over the block's tokens
//   byte  = E4M3_RNE(x * (1 / scale))
//
// Tokens come to a block a few at a time, so its scale only grows: where new
// tokens need more than it covers, the older tokens' bytes are brought to the
// new one.  Scales are powers of two so that this is exact (but for values
// that leave E4M3's normal range, below 2^-6 of the scale): however often a
// block has grown, its tokens have been rounded once, and E4M3 loses nothing
// by it, being a floating type.  A block that begins with a new token starts
// anew.
//
// A head vector belongs to LPR lanes of 16 channels: two runs of 8 that hold both
// sides of 8 rotation pairs.  (With 8 channels per lane the addresses, shuffles
// and loops around them were most of what was issued: 7000 tokens of 48 heads
// took 48 us.)  Keys and values: a unit (block, kv head, keys or values) belongs to
// a team of such lane groups, one group where a step brings a few tokens per
// sequence, a whole CTA for prompts; the first kHold rows of a group stay in
// registers between the maximum and the rounding, later ones (long blocks) are
// formed twice.  Queries: a lane group takes some heads of one token, whose
// cosines and sines it keeps.
#include "norm_rope.cuh"

namespace exl3 {
namespace {

// three CTAs of 80 registers on an SM (7000 tokens 40.5 us; four of 64 44.6, two 47)
constexpr int kThreads = 256, kPerSm = 3;

// the least 2^e >= top / 448, within the range of scales
__device__ __forceinline__ float scale_for(float top) {
  const uint32_t u = __float_as_uint(fmaxf(top, 448.0f * kLeastScale));
  // top = m 2^x, 1 <= m < 2, against 448 = 1.75 * 2^8
  const uint32_t e = (u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
  return fminf(__uint_as_float(e << 23), kMostScale);
}

// A lane's share of a head vector.
struct Raw {
  uint4 a, b;
};
template <int BF16>
__device__ __forceinline__ void unpack8(const uint4& r, float2* v) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; i++)
    v[i] = BF16 ? make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u))
                : __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
}
template <int BF16>
__device__ __forceinline__ uint4 pack8(const float2* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if (BF16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[i].x, v[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 h = __floats2half2_rn(v[i].x, v[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int LPR, int BF16, int INTER>
struct Lane {
  int lane, ca, cb;  // its place in the row, the first channels of its two runs
  bool in_a, in_b;   // whether they are there
  bool pairs;        // it has rotation pairs
  uint32_t mask;
  __device__ __forceinline__ Lane(const NormRopeParams& p) {
    lane = threadIdx.x % LPR;
    mask = ((1u << LPR) - 1) << ((threadIdx.x & 31) / LPR * LPR);
    pairs = p.inv_freq && lane < p.rot / 16;
    ca = lane * 16;
    cb = ca + 8;
    if (!INTER && lane < p.rot / 16) {
      ca = lane * 8;
      cb = ca + p.rot / 2;
    }
    in_a = ca < p.dim;
    in_b = cb < p.dim;
  }
  __device__ __forceinline__ Raw load(const uint16_t* x, bool some) const {
    Raw w{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (some && in_a) w.a = *reinterpret_cast<const uint4*>(x + ca);
    if (some && in_b) w.b = *reinterpret_cast<const uint4*>(x + cb);
    return w;
  }
  static __device__ __forceinline__ void unpack(const Raw& w, float2* v) {
    unpack8<BF16>(w.a, v);
    unpack8<BF16>(w.b, v + 4);
  }
  // cosines and sines of its pairs 2 e, 2 e + 1 at a position.  The fraction of a
  // turn is exact; the fast functions of it are off by 2^-21, a row's values, keys and
  // queries alike, by 1e-6 of its largest (a cache with a scale per head has exact
  // ones, 1e-7).  An 8-bit key cannot tell; a 16-bit query can where it is below a
  // 500th of its row's largest in fp16, a 4000th in bf16, and no score, a sum over the
  // row, can.  (A fifth of the instructions of the exact ones.)
  __device__ __forceinline__ void angles(const uint64_t* turns, int pos, int e, float2* c,
                                         float2* s) const {
    float x[2];
#pragma unroll
    for (int i = 0; i < 2; i++)
      x[i] = (float)(int32_t)((turns[8 * lane + 2 * e + i] * (uint64_t)(int64_t)pos) >> 32) *
             (0x1p-31f * 3.14159265358979f);
    *c = make_float2(__cosf(x[0]), __cosf(x[1]));
    *s = make_float2(__sinf(x[0]), __sinf(x[1]));
  }
  __device__ __forceinline__ void norm(float2* v, const Raw& weight, const NormRopeParams& p) const {
    float2 q2 = mul2(v[0], v[0]);
#pragma unroll
    for (int e = 1; e < 8; e++) q2 = fma2(v[e], v[e], q2);
    float sq = q2.x + q2.y;
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) sq += __shfl_xor_sync(mask, sq, m, LPR);
    const float f = rsqrtf(fmaf(sq, p.inv_dim, p.eps));
    float2 wt[8];
    unpack(weight, wt);
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = mul2(mul2(v[e], make_float2(f, f)), wt[e]);
  }
  // turns pairs 2 e, 2 e + 1
  static __device__ __forceinline__ void rotate(float2* v, int e, float2 c, float2 s) {
    if (INTER) {  // (a, b) of a pair share a register pair: a' = a c - b s, b' = a s + b c
      const float cc[2] = {c.x, c.y}, ss[2] = {s.x, s.y};
#pragma unroll
      for (int i = 0; i < 2; i++) {
        float2& x = v[2 * e + i];
        x = fma2(x, make_float2(cc[i], cc[i]),
                 mul2(make_float2(x.y, x.x), make_float2(-ss[i], ss[i])));
      }
    } else {
      const float2 a = v[e], b = v[4 + e];
      v[e] = fma2(a, c, mul2(b, make_float2(-s.x, -s.y)));
      v[4 + e] = fma2(b, c, mul2(a, s));
    }
  }
  __device__ __forceinline__ int sum(int x) const {
#pragma unroll
    for (int m = LPR / 2; m > 0; m >>= 1) x += __shfl_xor_sync(mask, x, m, LPR);
    return x;
  }
};

// Queries: lane group `item` of the launch takes heads of one token.
template <int LPR, int BF16, int INTER>
__device__ __forceinline__ void do_queries(const NormRopeParams& p, const uint64_t* turns,
                                           int64_t item, int slices, int per) {
  const Lane<LPR, BF16, INTER> ln(p);
  const int64_t ti = item / slices;
  if (ti >= p.T) return;
  const int t = (int)ti, j0 = (int)(item % slices) * per, j1 = min(j0 + per, p.set[0].heads);
  const HeadSet& hs = p.set[0];
  const uint16_t* x = hs.x + (int64_t)t * hs.ts + j0 * hs.hs;
  Raw raw = ln.load(x, j0 < j1);
  const Raw weight = ln.load(hs.weight, hs.weight != nullptr);
  int below = 0;  // sequences that end at or before t
  for (int b = ln.lane; b < p.batch.num_seqs; b += LPR) below += __ldg(p.batch.cu_q + b + 1) <= t;
  const int b = ln.sum(below);
  if (b >= p.batch.num_seqs) return;  // padding: left as it is
  float2 c[4], s[4];
  if (p.inv_freq) {
    int32_t ignored = 0;
    const Seq q = load_seq(p.batch, b, &ignored);
    const int pos = p.positions ? __ldg(p.positions + t) : q.len - q.n + (t - q.q0);
    if (ln.pairs) {
#pragma unroll
      for (int e = 0; e < 4; e++) ln.angles(turns, pos, e, &c[e], &s[e]);
    }
  }
  uint16_t* out = hs.out + (int64_t)t * hs.ots + j0 * hs.ohs;
#pragma unroll 1
  for (int j = j0; j < j1; j++, out += hs.ohs) {
    float2 v[8];
    ln.unpack(raw, v);
    x += hs.hs;
    raw = ln.load(x, j + 1 < j1);
    if (hs.weight) ln.norm(v, weight, p);
    if (ln.pairs) {
#pragma unroll
      for (int e = 0; e < 4; e++) ln.rotate(v, e, c[e], s[e]);
    }
    if (ln.in_a) *reinterpret_cast<uint4*>(out + ln.ca) = pack8<BF16>(v);
    if (ln.in_b) *reinterpret_cast<uint4*>(out + ln.cb) = pack8<BF16>(v + 4);
  }
}

// The new tokens of one block.
struct Job {
  int rows;         // how many; 0: nothing to do
  int lo;           // position of the first one
  int older;        // tokens before them in the block
  int t0;           // their first row
  int64_t entry;    // of the block table, the block's page
};
// Block slot `slot` of the launch (one warp): sequence b has the slots
// cu_q[b] / P + 2 b .., as many as it can touch blocks.  The page is not looked
// up here: its load and the rows' go out together.
__device__ __forceinline__ Job find_job(const NormRopeParams& p, int slot, bool report) {
  const int P = p.cache.page_size, shift = p.cache.page_shift, lane = threadIdx.x & 31;
  auto pages = [&](int x) { return shift >= 0 ? x >> shift : x / P; };  // (x >= 0 where it counts)
  int32_t bad = 0;
  Seq mine{};  // of sequence `lane`, loaded beside the bounds
  const int few = p.batch.num_seqs <= 32;
  if (few && lane < p.batch.num_seqs) mine = load_seq(p.batch, lane, &bad);
  int below = 0;
  for (int b = lane; b < p.batch.num_seqs; b += 32)
    below += pages(__ldg(p.batch.cu_q + b + 1)) + 2 * (b + 1) <= slot;
  const int b = __reduce_add_sync(0xffffffffu, below);
  Job j{};
  if (b >= p.batch.num_seqs) return j;
  Seq s;
  if (few) {
    s.q0 = __shfl_sync(0xffffffffu, mine.q0, b);
    s.n = __shfl_sync(0xffffffffu, mine.n, b);
    s.len = __shfl_sync(0xffffffffu, mine.len, b);
    bad = __shfl_sync(0xffffffffu, bad, b);
  } else {
    s = load_seq(p.batch, b, &bad);
  }
  const int start = s.len - s.n;  // position of the first new token
  if (s.n > 0 && start < 0) bad |= kStatusBadBatch;
  const int from = max(start, 0), first = pages(from);
  const int blk = first + slot - (pages(s.q0) + 2 * b);
  if (s.n > 0 && blk >= first && (long long)blk * P < s.len) {
    j.lo = max(from, blk * P);
    j.rows = min(s.len, blk * P + P) - j.lo;  // (lengths are at most 2^30)
    j.older = j.lo - blk * P;
    j.t0 = s.q0 + j.lo - start;
    j.entry = (int64_t)b * p.batch.table_stride + blk;
  }
  if (bad && report && lane == 0) atomicOr(p.status, bad);
  return j;
}

// Keys and values of a block: the units unit0 + 0, 1, .., one per team.  A team is
// `team` (a power of two) lane groups.
template <int LPR, int kHold, int BF16, int INTER>
__device__ __forceinline__ void do_block(const NormRopeParams& p, const uint64_t* turns,
                                         const Job& job, int unit0, int team, bool report) {
  using L = Lane<LPR, BF16, INTER>;
  constexpr int GW = 32 / LPR, kWarps = kThreads / 32;
  __shared__ uint32_t tops[kWarps];
  const int grp = threadIdx.x / LPR, wl = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const L ln(p);
  const int me = grp & (team - 1), unit = unit0 + grp / team;
  const uint32_t mask = team >= GW ? 0xffffffffu
                                   : ((1u << (team * LPR)) - 1) << (wl & ~(team * LPR - 1));
  const bool live = unit < 2 * p.set[1].heads;
  const int kv = unit & 1, h = live ? unit >> 1 : 0;
  const int rows = live ? job.rows : 0, lo = job.lo, older = job.older, t0 = job.t0;
  const HeadSet& hs = p.set[1 + kv];
  const uint16_t* const x0 = hs.x + (int64_t)t0 * hs.ts + h * hs.hs;
  Raw raw[kHold];
#pragma unroll
  for (int i = 0; i < kHold; i++)
    raw[i] = ln.load(x0 + (me + i * team) * hs.ts, me + i * team < rows);
  const int page = __ldg(p.batch.table + job.entry);
  if (page < 0 || page >= p.cache.num_pages) {  // (the whole CTA)
    if (report && threadIdx.x == 0) atomicOr(p.status, kStatusBadPage);
    return;
  }
  const bool turn = !kv && ln.pairs;
  float* const scale_at = const_cast<float*>(kv ? p.cache.v_scale : p.cache.k_scale) +
                          page * p.cache.scale_stride + h;
  const float held = older > 0 ? *scale_at : 0.0f;
  // new token r of the block, normed and rotated
  auto form = [&](const Raw& w, int r, float2* v) {
    ln.unpack(w, v);
    if (hs.weight) ln.norm(v, ln.load(hs.weight, true), p);
    if (turn) {
      const int pos = p.positions ? __ldg(p.positions + min(t0 + r, p.T - 1)) : lo + r;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        float2 c, sn;
        ln.angles(turns, pos, e, &c, &sn);
        ln.rotate(v, e, c, sn);
      }
    }
  };
  auto raise = [](float top, const float2* v) {
#pragma unroll
    for (int e = 0; e < 8; e++)  // (a NaN counts for nothing)
      asm("max.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(fabsf(v[e].x)), "f"(fabsf(v[e].y)));
    return top;
  };

  // ---- the largest value
  float top = 0.0f;
  float2 keep[kHold][8];
#pragma unroll
  for (int i = 0; i < kHold; i++) {
    form(raw[i], me + i * team, keep[i]);
    top = raise(top, keep[i]);
  }
#pragma unroll 1
  for (int r0 = kHold * team; r0 < rows; r0 += team) {
    float2 v[8];
    form(ln.load(x0 + (r0 + me) * hs.ts, r0 + me < rows), r0 + me, v);
    top = raise(top, v);
  }
  // (as whole numbers: it is no NaN and not negative)
  uint32_t most = __reduce_max_sync(mask, __float_as_uint(top));
  if (team > GW) {
    const int w0 = warp & ~(team / GW - 1);
    if (wl == 0) tops[warp] = most;
    __syncthreads();
    most = __reduce_max_sync(0xffffffffu, tops[w0 + (wl & (team / GW - 1))]);
  }
  top = __uint_as_float(most);

  // ---- the scale
  if (!live) return;
  if (!good_scale(held)) {  // no scale: the block is left alone
    if (ln.lane == 0 && me == 0) atomicOr(p.status, kStatusBadScale);
    return;
  }
  const float old = fmaxf(held, kLeastScale);
  const float scale = top <= 448.0f * old ? old : scale_for(top);
  if (ln.lane == 0 && me == 0) *scale_at = scale;
  uint8_t* const dst = const_cast<uint8_t*>(kv ? p.cache.v : p.cache.k) +
                       page * p.cache.page_bytes + h * p.cache.head_bytes;

  // ---- older tokens, where it has grown
  if (older > 0 && scale != old) {
    const float ratio = old / scale;
#pragma unroll 1
    for (int r = me; r < older; r += team)
#pragma unroll
      for (int half = 0; half < 2; half++) {
        if (!(half ? ln.in_b : ln.in_a)) continue;
        uint2* at =
            reinterpret_cast<uint2*>(dst + r * p.cache.token_bytes + (half ? ln.cb : ln.ca));
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
  const float inv = 1.0f / scale;  // (exact for a power of two)
  uint8_t* const dst_new = dst + (int64_t)older * p.cache.token_bytes;
  auto store = [&](int r, const float2* v) {
    if (r >= rows) return;
    uint8_t* at = dst_new + r * p.cache.token_bytes;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 a = mul2(v[2 * i], make_float2(inv, inv));
      const float2 b = mul2(v[2 * i + 1], make_float2(inv, inv));
      w[i] = e4m3_pack2(a.x, a.y) | (e4m3_pack2(b.x, b.y) << 16);
    }
    if (ln.in_a) *reinterpret_cast<uint2*>(at + ln.ca) = make_uint2(w[0], w[1]);
    if (ln.in_b) *reinterpret_cast<uint2*>(at + ln.cb) = make_uint2(w[2], w[3]);
  };
#pragma unroll
  for (int i = 0; i < kHold; i++) store(me + i * team, keep[i]);
#pragma unroll 1
  for (int r0 = kHold * team; r0 < rows; r0 += team) {
    float2 v[8];
    form(ln.load(x0 + (r0 + me) * hs.ts, r0 + me < rows), r0 + me, v);
    store(r0 + me, v);
  }
}

// `blocks` block slots of `groups` CTAs each; the other CTAs: queries, `slices`
// lane groups to a token, `per` heads to a lane group.
struct Split {
  int blocks, groups, team, slices, per;
};
template <int LPR, int kHold, int BF16, int INTER>
__global__ void __launch_bounds__(kThreads, kPerSm) append_blocks_kernel(NormRopeParams p, Split c) {
  constexpr int NG = kThreads / LPR;
  __shared__ uint64_t turns[128];  // of the pairs, per position
  __shared__ Job s_job;
  // (keys and values first; in turn with the queries they took as long)
  const int64_t cta = blockIdx.x, first = (int64_t)c.blocks * c.groups;
  const bool block = cta < first;
  pdl_wait();
  // the first warp finds the block, others the angles
  if (block && threadIdx.x < 32) {
    const Job j = find_job(p, (int)(cta / c.groups), cta % c.groups == 0);
    if (threadIdx.x == 0) s_job = j;
  }
  const int i = threadIdx.x - 32;
  if (p.inv_freq && i >= 0 && i < p.rot / 2) turns[i] = turns_of(__ldg(p.inv_freq + i));
  __syncthreads();
  if (!block) {
    do_queries<LPR, BF16, INTER>(p, turns, (cta - first) * NG + threadIdx.x / LPR, c.slices, c.per);
  } else {
    const Job job = s_job;
    if (job.rows > 0)
      do_block<LPR, kHold, BF16, INTER>(p, turns, job, (int)(cta % c.groups) * (NG / c.team), c.team,
                                        cta % c.groups == 0);
  }
}

template <int LPR, int kHold>
cudaError_t launch_hold(const NormRopeParams& p, cudaStream_t st) {
  constexpr int NG = kThreads / LPR;
  Split c{};
  c.blocks = p.T / p.cache.page_size + 2 * p.batch.num_seqs;
  // a team's lane groups hold the most rows that a step can bring to a block
  const int rows = p.batch.max_q < p.cache.page_size ? p.batch.max_q : p.cache.page_size;
  for (c.team = 1; c.team < NG && c.team * kHold < rows;) c.team *= 2;
  const int teams = NG / c.team;
  c.groups = (2 * p.set[1].heads + teams - 1) / teams;
  long long ctas = (long long)c.blocks * c.groups;
  // a token's query heads are spread over lane groups until those fill the GPU
  if (p.set[0].heads > 0) {
    const long long want = (4ll * kSms * kPerSm * NG + p.T - 1) / p.T;
    c.slices = (int)(want < p.set[0].heads ? want : p.set[0].heads);
    c.per = (p.set[0].heads + c.slices - 1) / c.slices;
    c.slices = (p.set[0].heads + c.per - 1) / c.per;
    ctas += ((long long)p.T * c.slices + NG - 1) / NG;
  }
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)ctas), block(kThreads);
  note_launches(1);
  if (p.inter)
    return p.bf16 ? launch_pdl(append_blocks_kernel<LPR, kHold, 1, 1>, grid, block, 0, st, p, c)
                  : launch_pdl(append_blocks_kernel<LPR, kHold, 0, 1>, grid, block, 0, st, p, c);
  return p.bf16 ? launch_pdl(append_blocks_kernel<LPR, kHold, 1, 0>, grid, block, 0, st, p, c)
                : launch_pdl(append_blocks_kernel<LPR, kHold, 0, 0>, grid, block, 0, st, p, c);
}

template <int LPR>
cudaError_t launch_lpr(const NormRopeParams& p, cudaStream_t st) {
  // one row per lane group keeps a step of a few tokens short (64 of one token 3.6 us,
  // with two 4.3), two keep a block of 64 tokens in registers (7000 tokens 40.5 us,
  // with one, formed twice, 42.7)
  return p.batch.max_q <= 8 ? launch_hold<LPR, 1>(p, st) : launch_hold<LPR, 2>(p, st);
}

}  // namespace

cudaError_t launch_append_blocks(const NormRopeParams& p, cudaStream_t st) {
  return p.dim <= 64 ? launch_lpr<4>(p, st) : p.dim <= 128 ? launch_lpr<8>(p, st)
                                                           : launch_lpr<16>(p, st);
}

}  // namespace exl3
