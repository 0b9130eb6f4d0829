// Attention of few new tokens over a paged cache (decode and verify steps):
// warp-level MMA, bounded by the cache's bytes.
//
//   out = sum_p softmax_p(scale q.k_p) v_p, one pass: every warp keeps the
//   running maximum m and sum l of its keys and an unnormalised O, rescaled
//   when m grows; parts are joined by m and l.
//
// Rows.  The group = heads / kv_heads query heads of a kv head and the new
// tokens are the rows of one matrix (row = token * group + head), 8 or 16
// of them per work unit, so a key is read once for all of them.  Both products
// are formed transposed, S^T = K Q^T and O^T = V^T P^T: the rows are then the
// MMA's N (8), not its M (16), so that 4 to 8 rows, the common case of
// single-token steps, cost half the products and half the registers (32 fp32
// of O per thread at head_dim 128), which leaves room for the warps that hide
// the loads.
//
// Work.  A unit is (sequence, kv head, row chunk); its keys are counted in
// granules of 64.  All units' granules form one line that is cut into equal
// pieces, one per CTA, from the device-side lengths alone: ragged batches
// balance, one long sequence fills the GPU, and nothing is planned on the
// host.  A CTA whose piece holds a whole unit writes the output; parts of a
// unit go to scratch (at most two per CTA), and the CTA that finishes the
// unit's last part joins them in their order on the line, so that results do
// not depend on timing.
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
constexpr int kGran = 64;            // keys per granule
constexpr float kRescale = 8.0f;     // log2 growth of the maximum that rescales O
constexpr float kLn2 = 0.69314718055994531f;

template <int D_, int NB_, int E8_, int BF_>
struct Cfg {
  static constexpr int D = D_, NB = NB_, E8 = E8_, BF = BF_;
  static constexpr int MBF = BF && !E8;             // type of the products
  // Softmax terms meet V as 16-bit values (an fp32 product would have to be
  // split in two and take twice the MMAs): bf16 rounds a term by 2^-9 of it at
  // most; fp16 by 2^-12 while it is above 2^-14, so there the terms are 2^7
  // times as large (below 2^15 with kRescale), and what is lost of a small one
  // is below 2^-32 of the largest.  The sum is of the unrounded terms.
  static constexpr float kLift = MBF ? 0.0f : 7.0f;
  static constexpr int RB = D * (E8 ? 1 : 2);       // bytes of a key row
  static constexpr int CPR = RB / 16;               // 16-byte chunks of it
  // bytes of K (and of V) in a tile: 2 KB at 64 channels let 4 CTAs share an
  // SM; E4M3 tiles of 128 channels took 89 us with 2 KB (16 keys) where they
  // take 83 with 4 KB (one token over 4 x 110,000 keys)
  static constexpr int kHalf = D == 128 ? 4096 : 2048;
  static constexpr int KT = kHalf / RB;             // keys per tile, 16 or 32
  static constexpr int MT = KT / 16;                // 16-key groups (one page each)
  static constexpr int RPI = 32 / CPR;              // rows per copy instruction
  static constexpr int RT = 8 * NB;                 // rows of a unit
  static constexpr int kStages = 3;
  static constexpr int kStageBytes = 2 * kHalf;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int OS = D + 4;                  // floats per row of the join buffer
  static constexpr int kJoinBytes = RT * OS * 4;
  static constexpr int kRing = kWarps * (kWarpBytes > kJoinBytes ? kWarpBytes : kJoinBytes);
  static constexpr int kSmem = kRing + kWarps * RT * 8 + kWarps * kStages * 4 + 64;
  static constexpr int kCtasPerSm = D == 128 ? 2 : 4;
  static constexpr int kGrid = kSms * kCtasPerSm;
  static constexpr int kFlat = D == 128 ? 40 : 24;  // most parts that are joined in one step
};

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
// 8x8 transpose of 16-bit pairs over the warp
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
template <int BF>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
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

// Whether this lane's share of a V tile holds an infinity or a NaN.
template <class C>
__device__ __forceinline__ bool not_finite(uint32_t vd, int lane) {
  constexpr uint32_t E = C::E8 ? 0x7F7F7F7Fu : C::BF ? 0x7F807F80u : 0x7C007C00u;
  bool r = false;
  for (int i = 0; i < C::kHalf / 512; i++) {
    const uint4 v = lds16(vd + (i * 32 + lane) * 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; j++)
      r |= (C::E8 ? __vcmpeq4(w[j] & E, E) : __vcmpeq2(w[j] & E, E)) != 0;
  }
  return r;
}

// Value of channel d of key k in a V tile.
template <class C>
__device__ __forceinline__ float v_at(uint32_t vd, int k, int d) {
  const int byte = d * (C::E8 ? 1 : 2);
  uint32_t w;
  asm volatile("ld.shared.u32 %0, [%1];"
               : "=r"(w)
               : "r"(vd + v_off<C>(k, byte >> 4) + (byte & 12)));
  w >>= (byte & 3) * 8;
  if (C::E8) {
    const uint32_t h = e4m3_to_f16x2(w & 0xFFu);
    return __low2float(*reinterpret_cast<const __half2*>(&h));
  }
  if (C::BF) return __uint_as_float(w << 16);
  return __half2float(__ushort_as_half((unsigned short)w));
}

// Channel of accumulator row half hf (rows g, g + 8 of the MMA) in channel
// tile x: 16-bit tiles hold 16 channels in order, E4M3 tiles even channels in
// rows 0-7 and odd ones in rows 8-15.
template <class C>
__device__ __forceinline__ int o_channel(int x, int hf, int g) {
  return C::E8 ? 16 * x + 2 * g + hf : 16 * x + 8 * hf + g;
}

// o += p v key by key for the rows that see the key.
template <class C>
__device__ __forceinline__ void add_seen(float (&o)[C::NB][C::D / 16][4],
                                         const float (&s)[C::NB][C::MT][4], uint32_t vd, int key0,
                                         uint32_t gone, const int (&hi)[C::NB][2],
                                         const int (&lo)[C::NB][2], int g, int c) {
#pragma unroll
  for (int t = 0; t < C::MT; t++) {
    if (gone >> t & 1) continue;
#pragma unroll 1
    for (int k = 0; k < 16; k++) {
      const int key = key0 + 16 * t + k;
      float pr[C::NB][2];
#pragma unroll
      for (int b = 0; b < C::NB; b++)
#pragma unroll
        for (int e = 0; e < 2; e++)
          pr[b][e] = __shfl_sync(0xffffffffu, k & 8 ? s[b][t][2 + e] : s[b][t][e], 4 * (k & 7) + c);
#pragma unroll
      for (int x = 0; x < C::D / 16; x++)
#pragma unroll
        for (int hf = 0; hf < 2; hf++) {
          const float v = v_at<C>(vd, 16 * t + k, o_channel<C>(x, hf, g));
#pragma unroll
          for (int b = 0; b < C::NB; b++)
#pragma unroll
            for (int e = 0; e < 2; e++)
              if (key <= hi[b][e] && key >= lo[b][e])
                o[b][x][2 * hf + e] = fmaf(pr[b][e], v, o[b][x][2 * hf + e]);
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

// The CTAs in use for a line of `total` granules, where piece c starts, and
// the piece that holds granule x.
template <class C>
__device__ __forceinline__ int pieces_of(long long total) {
  return total < C::kGrid ? (int)total : C::kGrid;
}
__device__ __forceinline__ long long piece_start(long long total, int pieces, int c) {
  return total * c / pieces;
}
__device__ __forceinline__ int piece_with(long long total, int pieces, long long x) {
  return (int)(((x + 1) * pieces + total - 1) / total) - 1;
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
__device__ __forceinline__ float row_lse(float m, float l, float lift) {
  return l > 0.0f || l != l ? (m + (log2f(l) - lift)) * kLn2 : -INFINITY;
}

template <class C>
__global__ void __launch_bounds__(kThreads, C::kCtasPerSm) attn_rows_kernel(AttnParams p) {
  constexpr int D = C::D, NB = C::NB, KT = C::KT, MT = C::MT, RT = C::RT;
  constexpr int MBF = C::MBF;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t ring_s = smem_u32(smem + warp * C::kWarpBytes);
  float2* ml = reinterpret_cast<float2*>(smem + C::kRing);  // [warp][RT]
  uint32_t* absent = reinterpret_cast<uint32_t*>(ml + kWarps * RT) + warp * C::kStages;

  pdl_wait();
  int32_t bad = 0;
  Place place;
  const long long total = scan_line(
      p, RT,
      [&](long long t) {
        const int n = pieces_of<C>(t);
        return (int)blockIdx.x < n ? piece_start(t, n, blockIdx.x) : -1LL;
      },
      &place, &bad);
  if (bad && blockIdx.x == 0) atomicOr(p.status, bad);
  const int pieces = pieces_of<C>(total);
  if ((int)blockIdx.x >= pieces) return;
  long long pos = piece_start(total, pieces, blockIdx.x);
  const long long end = piece_start(total, pieces, blockIdx.x + 1);
  int b = place.b;
  long long base = place.base;
  bool first_part = true;
  int done = 0;  // granules of the piece so far

  const int ps = p.cache.page_size, ps_shift = p.cache.page_shift;
  const int64_t tb = p.cache.token_bytes;
  // this lane's place in a group of rows that one copy instruction fetches
  const int lrow = lane / C::CPR, lch = lane % C::CPR;
  const int64_t lane_off = lrow * tb + lch * 16;
  const int64_t it_off = C::RPI * tb;

  while (pos < end && b < p.batch.num_seqs) {
    const SeqWork sw = seq_work(p, RT, b, &bad);
    if (pos >= base + sw.w) {
      base += sw.w;
      b++;
      continue;
    }
    const int u = (int)((pos - base) / sw.n), g0 = (int)((pos - base) % sw.n);
    const long long u0 = base + (long long)u * sw.n;  // the unit's place on the line
    const int cnt = (int)min((long long)(sw.n - g0), end - pos);
    const int h = u / sw.rc, rc = u % sw.rc;
    pos += cnt;

    // ---- rows: token of row r, its visible keys [lo, hi]
    const int nrows = min(RT, sw.s.n * p.group - rc * RT);
    const int tok0 = rc * RT / p.group, tok1 = (rc * RT + nrows - 1) / p.group;
    const int pos0 = sw.s.len - sw.s.n;
    auto vis_hi = [&](int tok) { return p.causal ? pos0 + tok : sw.s.len - 1; };
    auto vis_lo = [&](int tok) { return p.window > 0 ? max(0, pos0 + tok - p.window + 1) : 0; };
    // keys any row sees, and keys every row sees
    const int any0 = vis_lo(tok0), any1 = vis_hi(tok1) + 1;
    const int all0 = vis_lo(tok1), all1 = vis_hi(tok0) + 1;
    const int kbeg = max((sw.first + g0) * kGran, any0 / KT * KT);
    const int kend = min((sw.first + g0 + cnt) * kGran, any1);
    const int t_first = kbeg / KT;
    const int ntile = kend > kbeg ? (kend + KT - 1) / KT - t_first : 0;
    const int mine = ntile > warp ? (ntile - warp + kWarps - 1) / kWarps : 0;
    // The tiles are taken in a circle that begins where the piece would be by
    // now if all pieces had begun at multiples of their length: pieces of a
    // sequence's other heads then read the same tokens at about the same time,
    // neighbours in memory.
    int turn;
    {
      const float len = (float)total / pieces, e = (float)done;
      const int x0 = (int)(ceilf((g0 - e) / len) * len + e) - g0;
      turn = x0 * (kGran / KT);
      if (x0 < 0 || turn >= ntile) turn = 0;
      done += cnt;
      turn += warp;
    }
    auto key_of = [&](int i) {  // first key of this warp's tile i
      const int x = turn + i * kWarps;
      return (t_first + (x < ntile ? x : x - ntile)) * KT;
    };

    const int32_t* table = p.batch.table + (int64_t)b * p.batch.table_stride;
    // page of 16-key group j of this warp's tile i (-1 past the end)
    auto page_of = [&](int i, int j) {
      const int key = key_of(i) + 16 * j;
      if (i >= mine || key >= any1) return -1;
      return __ldg(table + (ps_shift >= 0 ? key >> ps_shift : key / ps));
    };
    int pg[MT];
#pragma unroll
    for (int j = 0; j < MT; j++) pg[j] = page_of(0, j);
    const uint8_t* const kh = p.cache.k + h * p.cache.head_bytes + lane_off;
    const uint8_t* const vh = p.cache.v + h * p.cache.head_bytes + lane_off;
    int ist = 0;  // stage of the next issue
    auto issue = [&](int i) {
      if (i < mine) {
        const int key0 = key_of(i);
        const uint32_t kd = ring_s + ist * C::kStageBytes, vd = kd + C::kHalf;
        uint32_t gone = 0;
#pragma unroll
        for (int j = 0; j < MT; j++) {
          const int keyj = key0 + 16 * j;
          const bool ok = (unsigned)pg[j] < (unsigned)p.cache.num_pages;
          if (!ok) {
            gone |= 1u << j;
            if (keyj < any1 && keyj + 16 > any0) bad |= kStatusBadPage;
          }
          const int in_page = ps_shift >= 0 ? keyj & (ps - 1) : keyj % ps;
          int64_t at = (int64_t)pg[j] * p.cache.page_bytes + in_page * tb;
          if (ok && keyj >= any0 && keyj + 16 <= any1) {
#pragma unroll
            for (int it = 0; it < 16 / C::RPI; it++, at += it_off) {
              const int r = 16 * j + it * C::RPI + lrow;
              cp_async16(kd + k_off<C>(r, lch), kh + at, 16);
              cp_async16(vd + v_off<C>(r, lch), vh + at, 16);
            }
          } else {
#pragma unroll
            for (int it = 0; it < 16 / C::RPI; it++, at += it_off) {
              const int r = 16 * j + it * C::RPI + lrow;
              const bool in = ok && key0 + r >= any0 && key0 + r < any1;
              cp_async16(kd + k_off<C>(r, lch), in ? kh + at : p.cache.k, in ? 16 : 0);
              cp_async16(vd + v_off<C>(r, lch), in ? vh + at : p.cache.v, in ? 16 : 0);
            }
          }
        }
        if (lane == 0) absent[ist] = gone;
#pragma unroll
        for (int j = 0; j < MT; j++) pg[j] = page_of(i + 1, j);
      }
      cp_commit();
      ist = ist == C::kStages - 1 ? 0 : ist + 1;
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; i++) issue(i);

    // ---- queries to registers (B operand: lane g holds row g), in the
    // channel order of the K operand
    uint32_t qf[NB][D / 8];
    float cs[NB][2];        // factor of the scores of rows 8 b + 2 c + e, log2 units
    int hi[NB][2], lo[NB][2];
    const float cbase = p.scale_log2 * (C::E8 && p.cache.k_scale ? __ldg(p.cache.k_scale + h) : 1.0f);
#pragma unroll
    for (int nb = 0; nb < NB; nb++) {
      const int r = 8 * nb + g;
      const int row = rc * RT + min(r, nrows - 1);
      const uint16_t* src = p.q + (int64_t)(sw.s.q0 + row / p.group) * p.q_ts +
                            (int64_t)(h * p.group + row % p.group) * p.q_hs;
      // a 16-byte chunk of K holds 8 channels (16-bit) or 16 (E4M3)
      constexpr int PC = C::E8 ? 2 : 1;
#pragma unroll
      for (int i = 0; i < C::CPR / 4; i++)
#pragma unroll
        for (int x = 0; x < PC; x++) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (r < nrows) v = *reinterpret_cast<const uint4*>(src + (c + 4 * i) * (8 * PC) + 8 * x);
          qf[nb][(i * PC + x) * 4] = v.x;
          qf[nb][(i * PC + x) * 4 + 1] = v.y;
          qf[nb][(i * PC + x) * 4 + 2] = v.z;
          qf[nb][(i * PC + x) * 4 + 3] = v.w;
        }
      float f_row = cbase;
      if (C::E8 && C::BF) {
        // bf16 to fp16: 2^s brings the row's largest value to [2^14, 2^15);
        // values below 2^-31 of it lose bits, those below 2^-39 vanish
        float am = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 8; i++)
          am = fmaxf(am, fmaxf(fabsf(__uint_as_float(qf[nb][i] << 16)),
                               fabsf(__uint_as_float(qf[nb][i] & 0xFFFF0000u))));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
        const int sh = fp16_scale_exp(am);
        const float f = exp2f((float)sh);
        f_row = cbase * exp2f((float)-sh);
#pragma unroll
        for (int i = 0; i < D / 8; i++)
          qf[nb][i] = pack2<0>(__uint_as_float(qf[nb][i] << 16) * f,
                               __uint_as_float(qf[nb][i] & 0xFFFF0000u) * f);
      }
      if (C::E8 && !(f_row > 0.0f)) {
        // a factor that is not positive (a k_scale of 0 or below) would turn
        // the -inf of masked scores: its sign, or its 0, goes to the queries
        const __half2 x = __float2half2_rn(f_row < 0.0f ? -1.0f : f_row == 0.0f ? 0.0f : NAN);
#pragma unroll
        for (int i = 0; i < D / 8; i++) {
          const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&qf[nb][i]), x);
          qf[nb][i] = *reinterpret_cast<const uint32_t*>(&y);
        }
        f_row = f_row < 0.0f ? -f_row : 1.0f;
      }
#pragma unroll
      for (int e = 0; e < 2; e++) {
        cs[nb][e] = __shfl_sync(0xffffffffu, f_row, 4 * (2 * c + e));
        const int tok = (rc * RT + min(8 * nb + 2 * c + e, nrows - 1)) / p.group;
        hi[nb][e] = vis_hi(tok);
        lo[nb][e] = vis_lo(tok);
      }
    }

    float o[NB][D / 16][4];
    float m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; nb++) {
#pragma unroll
      for (int x = 0; x < D / 16; x++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[nb][x][e] = 0.0f;
      m[nb][0] = m[nb][1] = -INFINITY;
      l[nb][0] = l[nb][1] = 0.0f;
    }

    int st = 0;
    for (int i = 0; i < mine; i++) {
      cp_wait<C::kStages - 2>();
      __syncwarp();
      issue(i + C::kStages - 1);
      const int key0 = key_of(i);
      const uint32_t kd = ring_s + st * C::kStageBytes, vd = kd + C::kHalf;
      const uint32_t gone = absent[st];
      st = st == C::kStages - 1 ? 0 : st + 1;

      // ---- scores
      float s[NB][MT][4];
#pragma unroll
      for (int t = 0; t < MT; t++) {
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
          for (int e = 0; e < 4; e++) s[nb][t][e] = 0.0f;
#pragma unroll
        for (int x = 0; x < C::CPR / 4; x++) {
          const uint4 k0 = lds16(kd + k_off<C>(16 * t + g, c + 4 * x));
          const uint4 k1 = lds16(kd + k_off<C>(16 * t + 8 + g, c + 4 * x));
          const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
          if (C::E8) {
#pragma unroll
            for (int y = 0; y < 4; y++) {
              const uint32_t a0 = e4m3_to_f16x2(w0[y]), a2 = e4m3_to_f16x2(w0[y] >> 16);
              const uint32_t a1 = e4m3_to_f16x2(w1[y]), a3 = e4m3_to_f16x2(w1[y] >> 16);
#pragma unroll
              for (int nb = 0; nb < NB; nb++)
                mma16<MBF>(s[nb][t], a0, a1, a2, a3, qf[nb][8 * x + 2 * y], qf[nb][8 * x + 2 * y + 1]);
            }
          } else {
#pragma unroll
            for (int y = 0; y < 2; y++)
#pragma unroll
              for (int nb = 0; nb < NB; nb++)
                mma16<MBF>(s[nb][t], w0[2 * y], w1[2 * y], w0[2 * y + 1], w1[2 * y + 1],
                           qf[nb][4 * x + 2 * y], qf[nb][4 * x + 2 * y + 1]);
          }
        }
      }
      if (key0 < all0 || key0 + KT > all1 || gone) {
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
          for (int t = 0; t < MT; t++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const int key = key0 + 16 * t + 8 * (e >> 1) + g;
              if (key > hi[nb][e & 1] || key < lo[nb][e & 1] || (gone >> t & 1))
                s[nb][t][e] = -INFINITY;
            }
      }
      // ---- terms, sum (a row's keys lie over the 8 lanes g).  m is brought
      // up to the maximum only when some row's has grown past 2^8 of it (terms
      // stay in range of both 16-bit types, and m goes out with l), so that
      // most tiles need one vote and no shuffles.
      float mx[NB][2];
      bool grow = false;
#pragma unroll
      for (int nb = 0; nb < NB; nb++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          mx[nb][e] = fmaxf(s[nb][0][e], s[nb][0][2 + e]);
#pragma unroll
          for (int t = 1; t < MT; t++)
            mx[nb][e] = fmaxf(mx[nb][e], fmaxf(s[nb][t][e], s[nb][t][2 + e]));
          mx[nb][e] *= cs[nb][e];
          grow |= mx[nb][e] > m[nb][e] + kRescale;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nb = 0; nb < NB; nb++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float x = mx[nb][e];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            if (x > m[nb][e]) {
              const float f = ex2(m[nb][e] - x);
              l[nb][e] *= f;
#pragma unroll
              for (int y = 0; y < D / 16; y++) {
                o[nb][y][e] *= f;
                o[nb][y][2 + e] *= f;
              }
              m[nb][e] = x;
            }
          }
      }
#pragma unroll
      for (int nb = 0; nb < NB; nb++)
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const float ms = (m[nb][e] == -INFINITY ? 0.0f : m[nb][e]) - C::kLift;
#pragma unroll
          for (int t = 0; t < MT; t++)
#pragma unroll
            for (int y = 0; y < 2; y++) {
              const float v = ex2(fmaf(s[nb][t][2 * y + e], cs[nb][e], -ms));
              s[nb][t][2 * y + e] = v;
              l[nb][e] += v;
            }
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
      for (int t = 0; t < MT; t++) {
        uint32_t pf[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; nb++) {
          pf[nb][0] = movm_t(pack2<MBF>(s[nb][t][0], s[nb][t][1]));
          pf[nb][1] = movm_t(pack2<MBF>(s[nb][t][2], s[nb][t][3]));
        }
#pragma unroll
        for (int x = 0; x < C::CPR / 2; x++) {
          uint32_t v[4];  // keys 0-7 and 8-15 of chunks 2 x and 2 x + 1
          ldsm4t(vd + v_off<C>(16 * t + (lane & 7) + (lane >> 4) * 8, 2 * x + (lane >> 3 & 1)), v);
          if (C::E8) {
#pragma unroll
            for (int y = 0; y < 2; y++) {
              // bytes (key 0: even, odd channel; key 1: even, odd) to pairs of keys
              const uint32_t w0 = __byte_perm(v[y], 0, 0x3120), w1 = __byte_perm(v[2 + y], 0, 0x3120);
              const uint32_t a0 = e4m3_to_f16x2(w0), a1 = e4m3_to_f16x2(w0 >> 16);
              const uint32_t a2 = e4m3_to_f16x2(w1), a3 = e4m3_to_f16x2(w1 >> 16);
#pragma unroll
              for (int nb = 0; nb < NB; nb++)
                mma16<MBF>(o[nb][2 * x + y], a0, a1, a2, a3, pf[nb][0], pf[nb][1]);
            }
          } else {
#pragma unroll
            for (int nb = 0; nb < NB; nb++)
              mma16<MBF>(o[nb][x], v[0], v[1], v[2], v[3], pf[nb][0], pf[nb][1]);
          }
        }
      }
    }
    cp_wait<0>();
    __syncthreads();  // every warp's ring is idle: the join buffers may cover it

    // ---- join the warps
    float* buf = reinterpret_cast<float*>(smem) + warp * (RT * C::OS);
#pragma unroll
    for (int nb = 0; nb < NB; nb++)
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const int r = 8 * nb + 2 * c + e;
        float sum = l[nb][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        if (g == 0) ml[warp * RT + r] = make_float2(m[nb][e], sum);
#pragma unroll
        for (int x = 0; x < D / 16; x++)
#pragma unroll
          for (int hf = 0; hf < 2; hf++)
            buf[r * C::OS + o_channel<C>(x, hf, g)] = o[nb][x][2 * hf + e];
      }
    __syncthreads();
    const bool whole = cnt == sw.n;
    float* part = reinterpret_cast<float*>(p.scratch) +
                  ((size_t)blockIdx.x * 2 + (first_part ? 0 : 1)) * part_floats(RT, D);
    const float vs = C::E8 && p.cache.v_scale ? __ldg(p.cache.v_scale + h) : 1.0f;
    for (int i = threadIdx.x; i < nrows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), d0 = (i % (D / 4)) * 4;
      float2 sl[kWarps];
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        sl[w] = ml[w * RT + r];
        mm = fmaxf(mm, sl[w].x);
      }
      const float ms = mm == -INFINITY ? 0.0f : mm;
      float ll = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kWarps; w++) {
        const float f = ex2(sl[w].x - ms);
        ll += sl[w].y * f;
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem) +
                                                          (w * RT + r) * C::OS + d0);
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
        if (p.lse && d0 == 0) p.lse[(int64_t)token * p.heads + head] = row_lse(mm, ll, C::kLift);
      } else {
        *reinterpret_cast<float4*>(part + r * D + d0) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (d0 == 0) *reinterpret_cast<float2*>(part + RT * D + 2 * r) = make_float2(mm, ll);
      }
    }
    first_part = false;
    if (!whole) {
      // ---- the CTA that brings a unit's last part joins them all.  Many
      // parts are joined in two steps, groups of about sqrt(parts) first, so
      // that no CTA reads them all.  One token of 16 heads per kv head over
      // 8000 keys (2 units of 125 parts of 16 x 128): 33.5 us with one step,
      // 20.2 with two; but 38 parts of 4 rows 15.6 and 17.0, and units of 19
      // parts of 16 x 64 18.0 and 25.0.
      const int c0 = piece_with(total, pieces, u0), c1 = piece_with(total, pieces, u0 + sw.n - 1);
      const float* parts = reinterpret_cast<const float*>(p.scratch);
      // piece c0 holds the unit's first part as its second, unless the unit
      // starts the piece; every other piece as its first
      const size_t slot0 = (size_t)c0 * 2 + (piece_start(total, pieces, c0) < u0 ? 1 : 0);
      auto part_of = [&](int i) {
        return parts + (i == 0 ? slot0 : (size_t)(c0 + i) * 2) * part_floats(RT, D);
      };
      const int np = c1 - c0 + 1;
      const int per = np <= C::kFlat ? np : (int)ceilf(sqrtf((float)np));  // parts of a group
      const int ng = (np + per - 1) / per;
      const int lead = ((int)blockIdx.x - c0) / per * per;  // first part of this one's group
      const int members = min(per, np - lead);

      // Joins the n parts from + y * step into the output, or in place into
      // the first of them (every thread writes what it alone reads).
      auto join = [&](int from, int step, int n, bool to_out) {
        // weights of the parts, a warp per row: w = 2^(m - max m)
        float* wt = reinterpret_cast<float*>(smem);  // [RT][n]
        for (int r = warp; r < nrows; r += kWarps) {
          auto at = [&](int y) {
            return reinterpret_cast<const float2*>(part_of(from + y * step) + RT * D + 2 * r);
          };
          float mm = -INFINITY;
          for (int y = lane; y < n; y += 32) mm = fmaxf(mm, __ldcg(at(y)).x);
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
          const float ms = mm == -INFINITY ? 0.0f : mm;
          float ll = 0.0f;
          for (int y = lane; y < n; y += 32) {
            const float2 x = __ldcg(at(y));
            const float f = ex2(x.x - ms);
            wt[r * n + y] = f;
            ll = fmaf(x.y, f, ll);
          }
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, x);
          if (lane == 0) ml[r] = make_float2(mm, ll);
        }
        __syncthreads();
        constexpr int IPT = RT * (D / 4) / kThreads;  // 16-byte columns per thread
        constexpr int U = 16 / IPT;                   // loads in flight
        float acc[IPT][4] = {};
        const int d0 = threadIdx.x % (D / 4) * 4, r0 = threadIdx.x / (D / 4);
        constexpr int RS = kThreads / (D / 4);
#pragma unroll U
        for (int y = 0; y < n; y++) {
          const float* src = part_of(from + y * step) + d0;
#pragma unroll
          for (int k = 0; k < IPT; k++) {
            const int r = r0 + k * RS;
            if (r < nrows) {
              const float4 x = __ldcg(reinterpret_cast<const float4*>(src + r * D));
              const float f = wt[r * n + y];
              acc[k][0] = fmaf(x.x, f, acc[k][0]);
              acc[k][1] = fmaf(x.y, f, acc[k][1]);
              acc[k][2] = fmaf(x.z, f, acc[k][2]);
              acc[k][3] = fmaf(x.w, f, acc[k][3]);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < IPT; k++) {
          const int r = r0 + k * RS;
          if (r >= nrows) break;
          const float2 sl = ml[r];
          if (to_out) {
            const int row = rc * RT + r;
            const int token = sw.s.q0 + row / p.group, head = h * p.group + row % p.group;
            const float inv = row_inverse(sl.y, vs);
#pragma unroll
            for (int e = 0; e < 4; e++) acc[k][e] *= inv;
            store_out4<C>(p, token, head, d0, acc[k], C::BF);
            if (p.lse && d0 == 0) p.lse[(int64_t)token * p.heads + head] = row_lse(sl.x, sl.y, C::kLift);
          } else {
            float* dst = const_cast<float*>(part_of(from));
            *reinterpret_cast<float4*>(dst + r * D + d0) =
                make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
            if (d0 == 0) *reinterpret_cast<float2*>(dst + RT * D + 2 * r) = sl;
          }
        }
      };
      // Counts one arrival; true in every thread for the last of `all`.  A
      // piece's word has three counts of 10 bits: the first group (0) and the
      // groups (10) of the unit that begins in it, and the later group (20)
      // of the unit that reaches into it.
      auto arrive = [&](int piece, int shift, int all) {
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
          const int was = atomicAdd(p.counters + piece, 1 << shift) >> shift & 1023;
          s_last = was == all - 1;
          if (s_last) atomicSub(p.counters + piece, all << shift);  // for the next call
        }
        __syncthreads();
        if (s_last) __threadfence();
        return s_last != 0;
      };
      if (arrive(c0 + lead, lead ? 20 : 0, members)) {
        join(lead, 1, members, ng == 1);
        if (ng > 1 && arrive(c0, 10, ng)) join(0, per, ng, true);
      }
    }
    __syncthreads();  // the buffers are refilled by the next unit
  }
  if (bad) atomicOr(p.status, bad);
}

template <class C>
cudaError_t launch_cfg(const AttnParams& p, cudaStream_t st) {
  // the join's weights, and the resident CTAs, fit the shared memory
  static_assert(C::RT * C::kGrid * 4 <= C::kRing, "join weights");
  static_assert(C::kCtasPerSm * (C::kSmem + 1200) <= 227 * 1024, "resident CTAs");
  static_assert(C::kGrid <= kRowsCounters, "counters");
  static bool init = false;
  if (!init) {
    const cudaError_t e = cudaFuncSetAttribute(
        attn_rows_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    init = true;
  }
  const cudaError_t err =
      launch_pdl(attn_rows_kernel<C>, dim3(C::kGrid), dim3(kThreads), C::kSmem, st, p);
  note_launches(1);
  return err;
}

template <int D, int NB>
cudaError_t launch_types(const AttnParams& p, cudaStream_t st) {
  if (p.e4m3)
    return p.bf16 ? launch_cfg<Cfg<D, NB, 1, 1>>(p, st) : launch_cfg<Cfg<D, NB, 1, 0>>(p, st);
  return p.bf16 ? launch_cfg<Cfg<D, NB, 0, 1>>(p, st) : launch_cfg<Cfg<D, NB, 0, 0>>(p, st);
}

template <int D>
cudaError_t launch_dim(const AttnParams& p, cudaStream_t st) {
  // the fewest rows per unit that hold one sequence's new tokens; 16 where
  // neither does (units of 32, whose registers leave no room for the warps
  // that hide the loads, took as long as two of 16)
  return (long long)p.batch.max_q * p.group <= 8 ? launch_types<D, 1>(p, st)
                                                 : launch_types<D, 2>(p, st);
}

}  // namespace

size_t attn_rows_scratch_bytes(int dim) {
  return (size_t)kSms * 4 * 2 * part_floats(16, dim) * 4;  // 4 CTAs of 16 rows at most
}

cudaError_t launch_attn_rows(const AttnParams& p, cudaStream_t st) {
  return p.dim == 64 ? launch_dim<64>(p, st) : launch_dim<128>(p, st);
}

}  // namespace exl3
