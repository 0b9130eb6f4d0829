// Attention of few new tokens over a paged cache (decode and verify steps):
// warp-level MMA, bounded by the cache's bytes.
//
//   out = sum_p softmax_p(scale q.k_p) v_p, one pass: every warp keeps the
//   running maximum m and sum l of its keys and an unnormalised O, rescaled
//   when m grows; parts are joined by m and l.
//
// Rows.  The group = heads / kv_heads query heads of a kv head and the new
// tokens are the rows of one matrix (row = token * group + head), 16 or 32 of
// them per work unit, so a key is read once for all of them.
//
// Work.  A unit is (sequence, kv head, row chunk); its keys are counted in
// granules of 64.  All units' granules form one line that is cut into equal
// pieces, one per CTA, from the device-side lengths alone: ragged batches
// balance, one long sequence fills the GPU, and nothing is planned on the
// host.  A CTA whose piece holds a whole unit writes the output; parts of a
// unit go to scratch (at most two per CTA) and attn_rows_join_kernel sums
// them in order, so results do not depend on timing.
//
// Inside a CTA the 4 warps take key tiles in turn, each with its own ring of
// asynchronous copies, and meet only at the end of a unit.  Keys outside
// [first, last visible] and keys of absent pages are zero-filled, never read.
//
// E4M3 caches are multiplied as fp16 (every E4M3 value is exact there):
// bf16 queries are brought to fp16 with a power of two per row that goes back
// into the score's scale.  Channels of the K product are permuted so that a
// lane's operands are 16 consecutive bytes; V goes through ldmatrix.trans,
// where an 8-bit pair of channels travels as one 16-bit element.
#include <math.h>

#include "attn.cuh"
#include "common.cuh"
#include "pipeline.cuh"

namespace exl3 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
constexpr int kGran = 64;            // keys per granule
constexpr int kCtasPerSm = 2;
constexpr int kGrid = kSms * kCtasPerSm;
constexpr float kLn2 = 0.69314718055994531f;

template <int D_, int NQ_, int E8_, int BF_>
struct Cfg {
  static constexpr int D = D_, NQ = NQ_, E8 = E8_, BF = BF_;
  static constexpr int RB = D * (E8 ? 1 : 2);       // bytes of a key row
  static constexpr int CPR = RB / 16;               // 16-byte chunks of it
  static constexpr int KT = 4096 / RB;              // keys per tile: 4 KB of K, 4 KB of V
  static constexpr int NT = KT / 8;                 // score tiles of 8 keys
  static constexpr int SUB = KT / 16;               // 16-key groups (one page each)
  static constexpr int RPI = 32 / CPR;              // rows per copy instruction
  static constexpr int RT = 16 * NQ;                // rows of a unit
  static constexpr int kStageBytes = 8192;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int OS = D + 4;                  // floats per row of the join buffer
  static constexpr int kSmem = kWarps * kWarpBytes + kWarps * RT * 8 + kWarps * kStages * 4 + 64;
};
static_assert(16 * 2 * (128 + 4) * 4 <= kStages * 8192, "join buffer fits a warp's ring");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
template <int BF>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}
template <int BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two E4M3 bytes (the low half of w) to fp16
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}

// Byte offset of 16-byte chunk j of key row r in a K tile (read as 16 bytes
// per lane: 2 rows x 4 chunks per wavefront) and in a V tile (ldmatrix: 8
// rows x 1 chunk), both free of bank conflicts.
template <class C>
__device__ __forceinline__ uint32_t k_off(int r, int j) {
  return r * C::RB + ((C::CPR >= 8 ? j ^ ((r & 1) << 2) : j) << 4);
}
template <class C>
__device__ __forceinline__ uint32_t v_off(int r, int j) {
  return r * C::RB + ((C::CPR >= 8 ? j ^ (r & 7) : j ^ ((r >> 1) & 3)) << 4);
}

// Whether this lane's eighth of a V tile holds an infinity or a NaN.
template <class C>
__device__ __forceinline__ bool not_finite(uint32_t vd, int lane) {
  constexpr uint32_t E = C::E8 ? 0x7F7F7F7Fu : C::BF ? 0x7F807F80u : 0x7C007C00u;
  bool r = false;
  for (int i = 0; i < 8; i++) {
    const uint4 v = lds16(vd + (i * 32 + lane) * 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; j++)
      r |= (C::E8 ? __vcmpeq4(w[j] & E, E) : __vcmpeq2(w[j] & E, E)) != 0;
  }
  return r;
}

// o += p v key by key for the rows that see the key.
template <class C>
__device__ __forceinline__ void add_seen(float (&o)[C::NQ][C::D / 8][4],
                                         const float (&s)[C::NQ][C::NT][4], uint32_t vd, int key0,
                                         uint32_t gone, const int (&hi)[C::NQ][2],
                                         const int (&lo)[C::NQ][2], int g, int c) {
#pragma unroll 1
  for (int k = 0; k < C::KT; k++) {
    float pr[C::NQ][2];
#pragma unroll
    for (int q = 0; q < C::NQ; q++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float x = 0.0f;
#pragma unroll
        for (int n = 0; n < C::NT; n++)
          if (n == k >> 3) x = k & 1 ? s[q][n][2 * e + 1] : s[q][n][2 * e];
        pr[q][e] = __shfl_sync(0xffffffffu, x, 4 * g + (k >> 1 & 3));
      }
    const int key = key0 + k;
    if (gone >> (k >> 4) & 1) continue;
#pragma unroll
    for (int j = 0; j < C::CPR; j++) {
      uint32_t w;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(vd + v_off<C>(k, j) + 4 * c));
      float v[4];
      if (C::E8) {
        const uint32_t a = e4m3_to_f16x2(w), b = e4m3_to_f16x2(w >> 16);
        const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
        const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
        v[0] = fa.x;  // tile 2j: channels 4c, 4c + 2
        v[1] = fb.x;
        v[2] = fa.y;  // tile 2j + 1: channels 4c + 1, 4c + 3
        v[3] = fb.y;
      } else if (C::BF) {
        v[0] = __uint_as_float(w << 16);
        v[1] = __uint_as_float(w & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        v[0] = f.x;
        v[1] = f.y;
      }
      constexpr int TP = C::E8 ? 2 : 1;  // score-column tiles of 8 channels per chunk
#pragma unroll
      for (int q = 0; q < C::NQ; q++)
#pragma unroll
        for (int e = 0; e < 2; e++)
          if (key <= hi[q][e] && key >= lo[q][e]) {
#pragma unroll
            for (int t = 0; t < TP; t++) {
              float(&d)[4] = o[q][TP * j + t];
              d[2 * e] = fmaf(pr[q][e], v[2 * t], d[2 * e]);
              d[2 * e + 1] = fmaf(pr[q][e], v[2 * t + 1], d[2 * e + 1]);
            }
          }
    }
  }
}

// ---- the line of granules

struct SeqWork {
  Seq s;
  int rc;       // row chunks
  int first;    // first granule of keys any new token sees
  int n;        // granules per unit
  long long w;  // granules of the sequence over all its units
};
__device__ __forceinline__ SeqWork seq_work(const AttnParams& p, int rt, int b, int32_t* bad) {
  SeqWork o;
  o.s = load_seq(p.batch, b, bad);
  o.rc = (int)(((long long)o.s.n * p.group + rt - 1) / rt);
  int lo = 0;
  if (p.window > 0) {
    lo = o.s.len - o.s.n - p.window + 1;
    if (lo < 0) lo = 0;
  }
  o.first = lo / kGran;
  o.n = (o.s.len + kGran - 1) / kGran - o.first;
  if (o.n < 1) o.n = 1;  // a unit without keys still has an output
  o.w = (long long)o.rc * p.kv_heads * o.n;
  return o;
}

// All granules (return value) and the sequence b whose granules [base,
// base + w) hold point at(total), by one pass over the lengths: every thread
// takes consecutive sequences, a block scan joins them.
struct Place {
  int b;
  long long base;
};
template <class At>
__device__ __forceinline__ long long scan_line(const AttnParams& p, int rt, At at, Place* place,
                                               int32_t* bad) {
  __shared__ long long warp_sum[kWarps];
  __shared__ Place found;
  const int per = (p.batch.num_seqs + kThreads - 1) / kThreads;
  const int b0 = threadIdx.x * per, b1 = min(b0 + per, p.batch.num_seqs);
  long long mine = 0;
  for (int b = b0; b < b1; b++) mine += seq_work(p, rt, b, bad).w;
  long long inc = mine;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, m);
    if (lane >= m) inc += o;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const long long pos = at(total);
  long long base = before + inc - mine;
  if (pos >= base && pos < base + mine) {
    int b = b0;
    for (;; b++) {
      const long long w = seq_work(p, rt, b, bad).w;
      if (pos < base + w) break;
      base += w;
    }
    found.b = b;
    found.base = base;
  }
  __syncthreads();
  *place = found;
  return total;
}

// The CTAs in use for a line of `total` granules, and where piece c starts.
__device__ __forceinline__ int pieces_of(long long total) {
  return total < kGrid ? (int)total : kGrid;
}
__device__ __forceinline__ long long piece_start(long long total, int pieces, int c) {
  return total * c / pieces;
}

// scratch: [kGrid][2] parts of RT rows: fp32 O rows, then (m, l) pairs
__host__ __device__ constexpr size_t part_floats(int rt, int d) { return (size_t)rt * (d + 2); }

template <class C>
__device__ __forceinline__ void store_out4(const AttnParams& p, int token, int head, int d0,
                                           const float (&o)[4], int bf) {
  uint2 w;
  if (bf) {
    w.x = pack2<1>(o[0], o[1]);
    w.y = pack2<1>(o[2], o[3]);
  } else {
    w.x = pack2<0>(o[0], o[1]);
    w.y = pack2<0>(o[2], o[3]);
  }
  *reinterpret_cast<uint2*>(p.out + ((int64_t)token * p.heads + head) * C::D + d0) = w;
}

// Final value of a row: o / l (0 where nothing was seen) and the natural log.
__device__ __forceinline__ float row_inverse(float l, float vs) { return l > 0.0f || l != l ? vs / l : 0.0f; }
__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.0f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <class C>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attn_rows_kernel(AttnParams p) {
  constexpr int D = C::D, NQ = C::NQ, KT = C::KT, NT = C::NT, RT = C::RT;
  constexpr int MBF = C::BF && !C::E8;  // type of the products
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * C::kWarpBytes;
  const uint32_t ring_s = smem_u32(ring);
  float2* ml = reinterpret_cast<float2*>(smem + kWarps * C::kWarpBytes);  // [warp][RT]
  uint32_t* absent = reinterpret_cast<uint32_t*>(ml + kWarps * RT) + warp * kStages;

  pdl_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int32_t bad = 0;
  Place place;
  const long long total = scan_line(
      p, RT,
      [&](long long t) {
        const int n = pieces_of(t);
        return (int)blockIdx.x < n ? piece_start(t, n, blockIdx.x) : -1LL;
      },
      &place, &bad);
  if (bad && blockIdx.x == 0) atomicOr(p.status, bad);
  const int pieces = pieces_of(total);
  if ((int)blockIdx.x >= pieces) return;
  long long pos = piece_start(total, pieces, blockIdx.x);
  const long long end = piece_start(total, pieces, blockIdx.x + 1);
  int b = place.b;
  long long base = place.base;
  bool first_part = true;

  while (pos < end && b < p.batch.num_seqs) {
    const SeqWork sw = seq_work(p, RT, b, &bad);
    if (pos >= base + sw.w) {
      base += sw.w;
      b++;
      continue;
    }
    const int u = (int)((pos - base) / sw.n), g0 = (int)((pos - base) % sw.n);
    const int cnt = (int)min((long long)(sw.n - g0), end - pos);
    const int h = u / sw.rc, rc = u % sw.rc;
    pos += cnt;

    // ---- rows: token of row r, its visible keys [lo, hi]
    const int nrows = min(RT, sw.s.n * p.group - rc * RT);
    const int tok0 = rc * RT / p.group, tok1 = (rc * RT + nrows - 1) / p.group;
    const int pos0 = sw.s.len - sw.s.n;
    auto vis_hi = [&](int tok) { return p.causal ? pos0 + tok : sw.s.len - 1; };
    auto vis_lo = [&](int tok) { return p.window > 0 ? max(0, pos0 + tok - p.window + 1) : 0; };
    int hi[NQ][2], lo[NQ][2];
#pragma unroll
    for (int q = 0; q < NQ; q++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int tok = min(rc * RT + 16 * q + 8 * e + g, rc * RT + nrows - 1) / p.group;
        hi[q][e] = vis_hi(tok);
        lo[q][e] = vis_lo(tok);
      }
    // keys any row sees, and keys every row sees
    const int any0 = vis_lo(tok0), any1 = vis_hi(tok1) + 1;
    const int all0 = vis_lo(tok1), all1 = vis_hi(tok0) + 1;
    const int kbeg = max((sw.first + g0) * kGran, any0 / KT * KT);
    const int kend = min((sw.first + g0 + cnt) * kGran, any1);
    const int t_first = kbeg / KT;
    const int ntile = kend > kbeg ? (kend + KT - 1) / KT - t_first : 0;
    const int mine = ntile > warp ? (ntile - warp + kWarps - 1) / kWarps : 0;

    const int32_t* table = p.batch.table + (int64_t)b * p.batch.table_stride;
    const int ps = p.cache.page_size;
    // page of 16-key group j of this warp's tile i (-1 past the end)
    auto page_of = [&](int i, int j) {
      const int key = (t_first + warp + i * kWarps) * KT + 16 * j;
      return i < mine && key < any1 ? __ldg(table + key / ps) : -1;
    };
    int pg[C::SUB];
#pragma unroll
    for (int j = 0; j < C::SUB; j++) pg[j] = page_of(0, j);
    auto issue = [&](int i) {
      if (i < mine) {
        const int st = i % kStages;
        const int key0 = (t_first + warp + i * kWarps) * KT;
        const uint32_t kd = ring_s + st * C::kStageBytes, vd = kd + 4096;
        const int ch = lane % C::CPR;
        uint32_t gone = 0;
#pragma unroll
        for (int j = 0; j < C::SUB; j++) {
          const int keyj = key0 + 16 * j;
          const bool ok = pg[j] >= 0 && pg[j] < p.cache.num_pages;
          if (!ok) {
            gone |= 1u << j;
            if (keyj < any1 && keyj + 16 > any0) bad |= kStatusBadPage;
          }
          const int64_t at = (int64_t)(ok ? pg[j] : 0) * p.cache.page_bytes +
                             (int64_t)(keyj % ps) * p.cache.token_bytes + h * p.cache.head_bytes +
                             ch * 16;
#pragma unroll
          for (int it = 0; it < 16 / C::RPI; it++) {
            const int r = it * C::RPI + lane / C::CPR;  // row inside the group
            const int key = keyj + r;
            const int64_t off = at + (int64_t)r * p.cache.token_bytes;
            const bool in = ok && key >= any0 && key < any1;
            const int64_t o = in ? off : 0;
            cp_async16(kd + k_off<C>(16 * j + r, ch), p.cache.k + o, in ? 16 : 0);
            cp_async16(vd + v_off<C>(16 * j + r, ch), p.cache.v + o, in ? 16 : 0);
          }
        }
        if (lane == 0) absent[st] = gone;
#pragma unroll
        for (int j = 0; j < C::SUB; j++) pg[j] = page_of(i + 1, j);
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; i++) issue(i);

    // ---- queries to registers, in the channel order of the K operand
    uint32_t qf[NQ][D / 16][4];
    float cs[NQ][2];  // row factor of the scores, log2 units
    const float cbase = p.scale_log2 * (C::E8 && p.cache.k_scale ? __ldg(p.cache.k_scale + h) : 1.0f);
#pragma unroll
    for (int q = 0; q < NQ; q++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int r = 16 * q + 8 * e + g;
        const bool in = r < nrows;
        const int row = rc * RT + (in ? r : 0);
        const uint16_t* src = p.q + (int64_t)(sw.s.q0 + row / p.group) * p.q_ts +
                              (int64_t)(h * p.group + row % p.group) * p.q_hs;
        // chunk i: 16 bytes of K, 8 channels (16-bit) or 16 (E4M3)
        uint32_t w[D / 8];  // this lane's words: 2 per MMA step
        constexpr int PC = C::E8 ? 2 : 1;
#pragma unroll
        for (int i = 0; i < C::CPR / 4; i++)
#pragma unroll
          for (int x = 0; x < PC; x++) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in)
              v = *reinterpret_cast<const uint4*>(src + (c + 4 * i) * (8 * PC) + 8 * x);
            w[(i * PC + x) * 4] = v.x;
            w[(i * PC + x) * 4 + 1] = v.y;
            w[(i * PC + x) * 4 + 2] = v.z;
            w[(i * PC + x) * 4 + 3] = v.w;
          }
        cs[q][e] = cbase;
        if (C::E8 && C::BF) {
          // bf16 to fp16: 2^s brings the row's largest value to [2^14, 2^15);
          // values below 2^-38 of it lose bits
          float am = 0.0f;
#pragma unroll
          for (int i = 0; i < D / 8; i++)
            am = fmaxf(am, fmaxf(fabsf(__uint_as_float(w[i] << 16)),
                                 fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
          am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
          am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
          const int sh = fp16_scale_exp(am);
          const float f = exp2f((float)sh);
          cs[q][e] = cbase * exp2f((float)-sh);
#pragma unroll
          for (int i = 0; i < D / 8; i++)
            w[i] = pack2<0>(__uint_as_float(w[i] << 16) * f,
                            __uint_as_float(w[i] & 0xFFFF0000u) * f);
        }
#pragma unroll
        for (int s = 0; s < D / 16; s++) {
          qf[q][s][e] = w[2 * s];
          qf[q][s][2 + e] = w[2 * s + 1];
        }
      }

    float o[NQ][D / 8][4];
    float m[NQ][2], l[NQ][2];
#pragma unroll
    for (int q = 0; q < NQ; q++) {
#pragma unroll
      for (int j = 0; j < D / 8; j++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[q][j][e] = 0.0f;
      m[q][0] = m[q][1] = -INFINITY;
      l[q][0] = l[q][1] = 0.0f;
    }

    for (int i = 0; i < mine; i++) {
      cp_wait<kStages - 2>();
      __syncwarp();
      issue(i + kStages - 1);
      const int st = i % kStages;
      const int key0 = (t_first + warp + i * kWarps) * KT;
      const uint32_t kd = ring_s + st * C::kStageBytes, vd = kd + 4096;
      const uint32_t gone = absent[st];

      // ---- scores
      float s[NQ][NT][4];
#pragma unroll
      for (int n = 0; n < NT; n++) {
#pragma unroll
        for (int q = 0; q < NQ; q++)
#pragma unroll
          for (int e = 0; e < 4; e++) s[q][n][e] = 0.0f;
#pragma unroll
        for (int x = 0; x < C::CPR / 4; x++) {
          const uint4 kv = lds16(kd + k_off<C>(8 * n + g, c + 4 * x));
          const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w};
          if (C::E8) {
#pragma unroll
            for (int y = 0; y < 4; y++) {
              const uint32_t b0 = e4m3_to_f16x2(kw[y]), b1 = e4m3_to_f16x2(kw[y] >> 16);
#pragma unroll
              for (int q = 0; q < NQ; q++) mma16<MBF>(s[q][n], qf[q][4 * x + y], b0, b1);
            }
          } else {
#pragma unroll
            for (int y = 0; y < 2; y++)
#pragma unroll
              for (int q = 0; q < NQ; q++)
                mma16<MBF>(s[q][n], qf[q][2 * x + y], kw[2 * y], kw[2 * y + 1]);
          }
        }
      }
      const bool part = key0 < all0 || key0 + KT > all1 || gone;
      if (part) {
#pragma unroll
        for (int q = 0; q < NQ; q++)
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const int key = key0 + 8 * n + 2 * c + (e & 1);
              if (key > hi[q][e >> 1] || key < lo[q][e >> 1] || (gone >> (n >> 1) & 1))
                s[q][n][e] = -INFINITY;
            }
      }
      // ---- running maximum, terms, sum
#pragma unroll
      for (int q = 0; q < NQ; q++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          float mx = s[q][0][2 * e];
#pragma unroll
          for (int n = 0; n < NT; n++) mx = fmaxf(mx, fmaxf(s[q][n][2 * e], s[q][n][2 * e + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          mx *= cs[q][e];
          const float mn = fmaxf(m[q][e], mx);
          const float ms = mn == -INFINITY ? 0.0f : mn;
          if (mn > m[q][e]) {
            const float f = ex2(m[q][e] - ms);
            l[q][e] *= f;
#pragma unroll
            for (int j = 0; j < D / 8; j++) {
              o[q][j][2 * e] *= f;
              o[q][j][2 * e + 1] *= f;
            }
            m[q][e] = mn;
          }
          float sum = 0.0f;
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int x = 0; x < 2; x++) {
              const float t = ex2(fmaf(s[q][n][2 * e + x], cs[q][e], -ms));
              s[q][n][2 * e + x] = t;
              sum += t;
            }
          l[q][e] += sum;
        }
      // ---- values
      // a tile with keys that only some rows see: a value there that is not
      // finite would reach the other rows as 0 * inf, so such a tile (looked
      // for here only) goes key by key
      if ((max(key0, any0) < all0 || min(key0 + KT, any1) > all1) &&
          __any_sync(0xffffffffu, not_finite<C>(vd, lane))) {
        add_seen<C>(o, s, vd, key0, gone, hi, lo, g, c);
        continue;
      }
#pragma unroll
      for (int j = 0; j < KT / 16; j++) {
        uint32_t pf[NQ][4];
#pragma unroll
        for (int q = 0; q < NQ; q++) {
          pf[q][0] = pack2<MBF>(s[q][2 * j][0], s[q][2 * j][1]);
          pf[q][1] = pack2<MBF>(s[q][2 * j][2], s[q][2 * j][3]);
          pf[q][2] = pack2<MBF>(s[q][2 * j + 1][0], s[q][2 * j + 1][1]);
          pf[q][3] = pack2<MBF>(s[q][2 * j + 1][2], s[q][2 * j + 1][3]);
        }
#pragma unroll
        for (int x = 0; x < C::CPR / 2; x++) {
          uint32_t v[4];
          ldsm4t(vd + v_off<C>(16 * j + (lane & 15), 2 * x + (lane >> 4)), v);
          if (C::E8) {
#pragma unroll
            for (int y = 0; y < 2; y++) {
              const uint32_t a0 = e4m3_to_f16x2(v[2 * y]), a1 = e4m3_to_f16x2(v[2 * y] >> 16);
              const uint32_t b0 = e4m3_to_f16x2(v[2 * y + 1]),
                             b1 = e4m3_to_f16x2(v[2 * y + 1] >> 16);
#pragma unroll
              for (int q = 0; q < NQ; q++) {
                mma16<MBF>(o[q][4 * x + 2 * y], pf[q], __byte_perm(a0, a1, 0x5410),
                           __byte_perm(b0, b1, 0x5410));
                mma16<MBF>(o[q][4 * x + 2 * y + 1], pf[q], __byte_perm(a0, a1, 0x7632),
                           __byte_perm(b0, b1, 0x7632));
              }
            }
          } else {
#pragma unroll
            for (int y = 0; y < 2; y++)
#pragma unroll
              for (int q = 0; q < NQ; q++)
                mma16<MBF>(o[q][2 * x + y], pf[q], v[2 * y], v[2 * y + 1]);
          }
        }
      }
    }
    cp_wait<0>();
    __syncwarp();

    // ---- join the warps: the ring is idle
    float* buf = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int q = 0; q < NQ; q++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int r = 16 * q + 8 * e + g;
        float sum = l[q][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (c == 0) ml[warp * RT + r] = make_float2(m[q][e], sum);
        if (C::E8) {
          // even tiles hold channels 4c, 4c+2 of a 16-channel chunk, odd ones
          // 4c+1, 4c+3
#pragma unroll
          for (int j = 0; j < D / 16; j++)
            *reinterpret_cast<float4*>(buf + r * C::OS + 16 * j + 4 * c) =
                make_float4(o[q][2 * j][2 * e], o[q][2 * j + 1][2 * e], o[q][2 * j][2 * e + 1],
                            o[q][2 * j + 1][2 * e + 1]);
        } else {
#pragma unroll
          for (int j = 0; j < D / 8; j++)
            *reinterpret_cast<float2*>(buf + r * C::OS + 8 * j + 2 * c) =
                make_float2(o[q][j][2 * e], o[q][j][2 * e + 1]);
        }
      }
    __syncthreads();
    const bool whole = cnt == sw.n;
    float* part = reinterpret_cast<float*>(p.scratch) +
                  ((size_t)blockIdx.x * 2 + (first_part ? 0 : 1)) * part_floats(RT, D);
    const float vs = C::E8 && p.cache.v_scale ? __ldg(p.cache.v_scale + h) : 1.0f;
    for (int i = threadIdx.x; i < nrows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d0 = (i % (D / 4)) * 4;
      float2 st[kWarps];
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        st[w] = ml[w * RT + r];
        mm = fmaxf(mm, st[w].x);
      }
      const float ms = mm == -INFINITY ? 0.0f : mm;
      float ll = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        const float f = ex2(st[w].x - ms);
        ll += st[w].y * f;
        const float4 x = *reinterpret_cast<const float4*>(
            smem + w * C::kWarpBytes + (r * C::OS + d0) * 4);
        acc[0] = fmaf(x.x, f, acc[0]);
        acc[1] = fmaf(x.y, f, acc[1]);
        acc[2] = fmaf(x.z, f, acc[2]);
        acc[3] = fmaf(x.w, f, acc[3]);
      }
      if (whole) {
        const int row = rc * RT + r;
        const int token = sw.s.q0 + row / p.group, head = h * p.group + row % p.group;
        const float inv = row_inverse(ll, vs);
#pragma unroll
        for (int e = 0; e < 4; e++) acc[e] *= inv;
        store_out4<C>(p, token, head, d0, acc, C::BF);
        if (p.lse && d0 == 0) p.lse[(int64_t)token * p.heads + head] = row_lse(mm, ll);
      } else {
        *reinterpret_cast<float4*>(part + r * D + d0) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (d0 == 0) *reinterpret_cast<float2*>(part + RT * D + 2 * r) = make_float2(mm, ll);
      }
    }
    first_part = false;
    __syncthreads();  // the buffers are refilled by the next unit
  }
  if (bad) atomicOr(p.status, bad);
}

// Sums the parts of every unit that a cut of the line goes through.  Block
// (x, y): cut x + 1; the block of a unit's first cut does the unit.  Rows are
// spread over the warps and over y.
template <class C>
__global__ void __launch_bounds__(kThreads) attn_rows_join_kernel(AttnParams p) {
  constexpr int D = C::D, RT = C::RT;
  const int cut = blockIdx.x + 1;
  int32_t bad = 0;
  Place place;
  const long long total = scan_line(
      p, RT,
      [&](long long t) {
        const int n = pieces_of(t);
        return cut < n ? piece_start(t, n, cut) : -1LL;
      },
      &place, &bad);
  const int pieces = pieces_of(total);
  const bool live = cut < pieces;
  const SeqWork sw = live ? seq_work(p, RT, place.b, &bad) : SeqWork{};
  const long long at = live ? piece_start(total, pieces, cut) : 0;
  pdl_wait();
  if (!live) return;
  const int u = (int)((at - place.base) / sw.n);
  const long long u0 = place.base + (long long)u * sw.n, u1 = u0 + sw.n;
  if (at == u0 || piece_start(total, pieces, cut - 1) > u0) return;
  // pieces first .. last hold the unit's parts
  const int first = cut - 1;
  int last = cut;
  while (last + 1 < pieces && piece_start(total, pieces, last + 1) < u1) last++;
  const int h = u / sw.rc, rc = u % sw.rc;
  const int nrows = min(RT, sw.s.n * p.group - rc * RT);
  const float vs = C::E8 && p.cache.v_scale ? __ldg(p.cache.v_scale + h) : 1.0f;
  constexpr int LR = D / 4;  // threads of a row
  const int d0 = (threadIdx.x % LR) * 4;
  const float* parts = reinterpret_cast<const float*>(p.scratch);
  // the first piece's part is its second one, unless the unit starts it
  const size_t slot0 = (size_t)first * 2 + (piece_start(total, pieces, first) < u0 ? 1 : 0);
  for (int r = blockIdx.y * (kThreads / LR) + threadIdx.x / LR; r < nrows;
       r += gridDim.y * (kThreads / LR)) {
    float mm = -INFINITY, ll = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int c = first; c <= last; c++) {
      const float* part = parts + (c == first ? slot0 : (size_t)c * 2) * part_floats(RT, D);
      const float2 st = *reinterpret_cast<const float2*>(part + RT * D + 2 * r);
      const float4 x = *reinterpret_cast<const float4*>(part + r * D + d0);
      const float mn = fmaxf(mm, st.x);
      const float ms = mn == -INFINITY ? 0.0f : mn;
      const float f0 = ex2(mm - ms), f1 = ex2(st.x - ms);
      mm = mn;
      ll = ll * f0 + st.y * f1;
      acc[0] = acc[0] * f0 + x.x * f1;
      acc[1] = acc[1] * f0 + x.y * f1;
      acc[2] = acc[2] * f0 + x.z * f1;
      acc[3] = acc[3] * f0 + x.w * f1;
    }
    const int row = rc * RT + r;
    const int token = sw.s.q0 + row / p.group, head = h * p.group + row % p.group;
    const float inv = row_inverse(ll, vs);
#pragma unroll
    for (int e = 0; e < 4; e++) acc[e] *= inv;
    store_out4<C>(p, token, head, d0, acc, C::BF);
    if (p.lse && d0 == 0) p.lse[(int64_t)token * p.heads + head] = row_lse(mm, ll);
  }
}

template <class C>
cudaError_t launch_cfg(const AttnParams& p, cudaStream_t st) {
  static bool init = false;
  if (!init) {
    const cudaError_t e = cudaFuncSetAttribute(
        attn_rows_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    init = true;
  }
  cudaError_t err =
      launch_pdl(attn_rows_kernel<C>, dim3(kGrid), dim3(kThreads), C::kSmem, st, p);
  note_launches(1);
  if (err != cudaSuccess) return err;
  err = launch_pdl(attn_rows_join_kernel<C>, dim3(kGrid - 1, 1), dim3(kThreads), 0, st, p);
  note_launches(1);
  return err;
}

template <int D, int NQ>
cudaError_t launch_types(const AttnParams& p, cudaStream_t st) {
  if (p.e4m3)
    return p.bf16 ? launch_cfg<Cfg<D, NQ, 1, 1>>(p, st) : launch_cfg<Cfg<D, NQ, 1, 0>>(p, st);
  return p.bf16 ? launch_cfg<Cfg<D, NQ, 0, 1>>(p, st) : launch_cfg<Cfg<D, NQ, 0, 0>>(p, st);
}

}  // namespace

size_t attn_rows_scratch_bytes(int dim) { return (size_t)kGrid * 2 * part_floats(32, dim) * 4; }

cudaError_t launch_attn_rows(const AttnParams& p, cudaStream_t st) {
  // 16 rows per unit while one sequence's new tokens fit them, 32 otherwise
  // (half the reads of the cache per row)
  const bool wide = (long long)p.batch.max_q * p.group > 16;
  if (p.dim == 64) return wide ? launch_types<64, 2>(p, st) : launch_types<64, 1>(p, st);
  return wide ? launch_types<128, 2>(p, st) : launch_types<128, 1>(p, st);
}

}  // namespace exl3
