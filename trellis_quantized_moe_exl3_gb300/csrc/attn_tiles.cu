// Attention of many new tokens over a paged cache (chunks and prompts):
// tcgen05 tensor cores, operands by TMA, accumulators and softmax terms in
// TMEM.
//
//   out = sum_p softmax_p(scale q.k_p) v_p, one pass over the keys with a
//   running maximum m and sum l per row.
//
// Rows and tiles.  The group = heads / kv_heads query heads of a kv head and
// the new tokens are the rows of one matrix (row = token * group + head).  A
// unit of work is (sequence, kv head, 256 rows): two row tiles of 128 against
// key tiles of 128, so one loaded K or V tile serves two products and the
// tensor core works on one row tile while the other's softmax runs.
//
// Roles of a CTA (one per SM, persistent): two softmax warpgroups (one row
// tile each, one thread per row: no shuffles), one warp that issues the MMAs,
// one that issues the TMA loads, and for E4M3 caches four warps that widen
// the 8-bit tiles to fp16 (exact) in shared memory.
//   S = Q K^T   A, B from shared memory, S (128 fp32 columns) in TMEM
//   P           written over S as 16-bit pairs, the A operand of
//   O += P V    B = V as it lies in memory (keys are the K dimension, so V is
//               the MN-major operand), O (head_dim fp32 columns) in TMEM
// A row's O is rescaled only when its maximum has grown by more than 2^8
// since the last time (P stays below 2^8, in range for both 16-bit types, and
// the final division removes the common factor), which leaves almost no
// rescales after a row's first tiles.
//
// Work.  All units' key tiles form one line (heads outermost) that
// plan_kernel measures from the device-side lengths and cuts into equal
// pieces, one per CTA.  Parts of a unit that a cut goes through go to scratch,
// at most two per CTA, and attn_tiles_join_kernel sums them in order.
//
// A page of the cache is fetched as boxes of the largest power of two of
// tokens that divides the page size; keys past the last visible one and pages
// that do not exist are out-of-range coordinates, which TMA fills with zeros.
// Rows of V that a box brings in beyond the visible range (a page's stale end)
// are zeroed before they meet P = 0.
#include <cuda.h>
#include <math.h>

#include "attn.cuh"
#include "common.cuh"
#include "umma.cuh"

namespace exl3 {
namespace {

constexpr int kTile = 128;          // rows of a row tile, keys of a key tile
constexpr int kUnitRows = 256;
constexpr int kGrid = kSms;
constexpr int kMinSteps = 4;        // key tiles per piece, where there are enough
constexpr float kRescale = 8.0f;    // log2 growth of the maximum that rescales O
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kGone = 16;           // ring of absent-page masks (steps)

template <int D_, int E8_, int BF_>
struct Cfg {
  static constexpr int D = D_, E8 = E8_, BF = BF_;
  static constexpr int MBF = BF && !E8;                  // type of the products
  static constexpr int kOp = kTile * D * 2;              // bytes of a 16-bit operand tile
  static constexpr int kRaw = kTile * D;                 // bytes of an E4M3 tile
  static constexpr int kStages = E8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);
  static constexpr int kRawStages = E8 ? 4 : 0;
  static constexpr int kOffKV = 2 * kOp;
  static constexpr int kOffRaw = kOffKV + kStages * kOp;
  static constexpr int kOffBar = kOffRaw + kRawStages * kRaw;
  static constexpr int kBars = 2 * kStages + 2 * kRawStages + 9;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kSmem = kOffMisc + kGone * 4 + 32 + 1024;
  static constexpr int kThreads = E8 ? 512 : 384;
  // registers of a softmax thread and of the others (their sum over the CTA
  // is what the launch holds: 128 or 168 a thread)
  static constexpr int kRegsSoft = E8 ? 192 : 216, kRegsRest = E8 ? 64 : 72;
  static constexpr int kTmemCols = 512;
};

// ------------------------------------------------------------ PTX helpers
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a));
}
// the wait, tied to the registers of a load, so that no use moves before it
__device__ __forceinline__ void tmem_ld32_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(a)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int c0, int c1, int c2,
                                            int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 lanes at once
__device__ __forceinline__ void fma2(float& x, float& y, float c, float d) {
  asm("{\n\t.reg .b64 a, b, e;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\t"
      "mov.b64 e, {%3, %3};\n\tfma.rn.f32x2 a, a, b, e;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float& x, float& y, float u, float v) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(u), "f"(v));
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
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}

// ------------------------------------------------------------ work
// A unit: 256 packed rows of one sequence (for every kv head alike).
struct Unit {
  Seq s;
  int b, row0, nrows;
  int any0, any1;     // keys some row sees: [any0, any1)
  int all0, all1;     // keys every row sees
  int first, n;       // first key tile, key tiles (at least 1)
  int a0, e0, a1, e1; // key tiles [a, e) that row tile 0, 1 needs
};
__device__ __forceinline__ int vis_hi(const AttnParams& p, const Seq& s, int tok) {
  return p.causal ? s.len - s.n + tok : s.len - 1;
}
__device__ __forceinline__ int vis_lo(const AttnParams& p, const Seq& s, int tok) {
  return p.window > 0 ? max(0, s.len - s.n + tok - p.window + 1) : 0;
}
__device__ __forceinline__ Unit make_unit(const AttnParams& p, int b, const Seq& s, int idx) {
  Unit u;
  u.s = s;
  u.b = b;
  u.row0 = idx * kUnitRows;
  u.nrows = min(kUnitRows, s.n * p.group - u.row0);
  const int tok0 = u.row0 / p.group, tok1 = (u.row0 + u.nrows - 1) / p.group;
  u.any0 = vis_lo(p, s, tok0);
  u.any1 = max(vis_hi(p, s, tok1) + 1, u.any0);
  u.all0 = vis_lo(p, s, tok1);
  u.all1 = vis_hi(p, s, tok0) + 1;
  u.first = u.any0 / kTile;
  u.n = max(1, (u.any1 + kTile - 1) / kTile - u.first);
  auto range = [&](int t, int* a, int* e) {
    const int r0 = u.row0 + t * kTile, r1 = min(r0 + kTile, u.row0 + u.nrows) - 1;
    *a = *e = 0;
    if (r1 >= r0) {
      const int lo = vis_lo(p, s, r0 / p.group), hi = vis_hi(p, s, r1 / p.group) + 1;
      if (hi > lo) {
        *a = lo / kTile;
        *e = (hi + kTile - 1) / kTile;
      }
    }
  };
  range(0, &u.a0, &u.e0);
  range(1, &u.a1, &u.e1);
  return u;
}

// scratch: header, piece starts, unit records, first units of sequences,
// prefix sums of key tiles over units, then the parts.
struct PlanHead {
  long long line;   // key tiles of one kv head
  int units, pieces;
};
struct Start {
  int unit, head, off, pad;
};
struct Plan {
  PlanHead* head;
  Start* start;     // [kGrid]
  int2* rec;        // [units] {sequence, index of the unit in it}
  int* seq_unit;    // [num_seqs + 1]
  long long* pre;   // [units + 1]
  float* parts;     // [kGrid][2][part]
};
__host__ __device__ inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
__host__ __device__ inline size_t max_units(long long rows, int seqs) {
  return (size_t)(rows / kUnitRows + 1 + seqs);
}
__host__ __device__ inline size_t carve(void* base, long long rows, int seqs, Plan* o) {
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t at = 0;
  const size_t mu = max_units(rows, seqs);
  Plan p;
  p.head = reinterpret_cast<PlanHead*>(b + at);
  at += 256;
  p.start = reinterpret_cast<Start*>(b + at);
  at += align256(sizeof(Start) * kGrid);
  p.rec = reinterpret_cast<int2*>(b + at);
  at += align256(sizeof(int2) * mu);
  p.seq_unit = reinterpret_cast<int*>(b + at);
  at += align256(sizeof(int) * ((size_t)seqs + 1));
  p.pre = reinterpret_cast<long long*>(b + at);
  at += align256(sizeof(long long) * (mu + 1));
  p.parts = reinterpret_cast<float*>(b + at);
  if (o) *o = p;
  return at;
}
__host__ __device__ constexpr size_t part_floats(int d) { return (size_t)kUnitRows * (d + 2); }

__device__ __forceinline__ long long piece_start(long long total, int pieces, int c) {
  return total * c / pieces;
}

constexpr int kPlanThreads = 1024;

// Inclusive scan over the block; *total receives the sum.
__device__ __forceinline__ long long block_scan(long long v, long long* total) {
  __shared__ long long sums[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v += o;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  long long w = lane < kPlanThreads / 32 ? sums[lane] : 0;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, w, m);
    if (lane >= m) w += o;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return warp > 0 ? v + before : v;
}

// The line of key tiles from the device-side lengths (one block).
__global__ void __launch_bounds__(kPlanThreads) attn_plan_kernel(AttnParams p, Plan pl,
                                                                int max_unit) {
  constexpr int kCache = 2048;
  __shared__ long long pre_s[kCache + 1];
  __shared__ int unit_s[kCache + 1];
  pdl_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int B = p.batch.num_seqs;
  int32_t bad = 0;
  long long run = 0, total;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    long long n = 0;
    if (b < B) {
      const Seq s = load_seq(p.batch, b, &bad);
      n = ((long long)s.n * p.group + kUnitRows - 1) / kUnitRows;
    }
    const long long inc = block_scan(n, &total);
    if (b < B) {
      pl.seq_unit[b] = (int)(run + inc - n);
      if (b < kCache) unit_s[b] = (int)(run + inc - n);
    }
    run += total;
  }
  // (sequences that overlap, an inconsistent batch, could claim more units
  // than the rows make: the rest is left out)
  if (run > max_unit) {
    bad |= kStatusBadBatch;
    run = max_unit;
  }
  const int units = (int)run;
  if (bad) atomicOr(p.status, bad);
  __syncthreads();
  const bool cached = B <= kCache, pre_cached = units <= kCache;
  run = 0;
  for (int i0 = 0; i0 < units; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    long long n = 0;
    if (i < units) {
      int lo = 0, hi = B;  // the last sequence whose first unit is <= i
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((cached ? unit_s[mid] : pl.seq_unit[mid]) <= i)
          lo = mid;
        else
          hi = mid;
      }
      const int idx = i - (cached ? unit_s[lo] : pl.seq_unit[lo]);
      pl.rec[i] = make_int2(lo, idx);
      int32_t ignored = 0;
      n = make_unit(p, lo, load_seq(p.batch, lo, &ignored), idx).n;
    }
    const long long inc = block_scan(n, &total);
    if (i < units) {
      pl.pre[i] = run + inc - n;
      if (pre_cached) pre_s[i] = run + inc - n;
    }
    run += total;
  }
  __syncthreads();
  const long long all = run * p.kv_heads;
  const long long want = (all + kMinSteps - 1) / kMinSteps;
  const int pieces = want < kGrid ? (int)want : kGrid;
  if (threadIdx.x == 0) *pl.head = PlanHead{run, units, pieces};
  if (threadIdx.x < pieces) {
    const long long at = piece_start(all, pieces, threadIdx.x);
    const long long s = at % run;
    int lo = 0, hi = units;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((pre_cached ? pre_s[mid] : pl.pre[mid]) <= s)
        lo = mid;
      else
        hi = mid;
    }
    pl.start[threadIdx.x] =
        Start{lo, (int)(at / run), (int)(s - (pre_cached ? pre_s[lo] : pl.pre[lo])), 0};
  }
}

// The pieces of one CTA, unit by unit.  Every role walks them by itself.
struct Walk {
  const AttnParams& p;
  const Plan& pl;
  int unit, head, off, units;
  long long left;
  bool first;
  // the current part
  Unit u;
  int h, s0, s1;   // kv head, key tiles [s0, s1) counted from u.first
  int j0, j1;      // those of them that a row tile needs (a row tile's are a
                   // run, and the two runs meet)
  bool whole;
  int slot;        // 0: the first part of the piece
  __device__ Walk(const AttnParams& p_, const Plan& pl_) : p(p_), pl(pl_) {
    const PlanHead hd = *pl.head;
    const int c = blockIdx.x;
    left = 0;
    units = hd.units;
    first = true;
    if (c < hd.pieces) {
      const long long all = hd.line * p.kv_heads;
      left = piece_start(all, hd.pieces, c + 1) - piece_start(all, hd.pieces, c);
      const Start st = pl.start[c];
      unit = st.unit;
      head = st.head;
      off = st.off;
    }
  }
  __device__ bool next() {
    if (left <= 0) return false;
    const int2 r = pl.rec[unit];
    int32_t ignored = 0;
    u = make_unit(p, r.x, load_seq(p.batch, r.x, &ignored), r.y);
    h = head;
    s0 = off;
    s1 = (int)min((long long)u.n, off + left);
    if (s1 <= s0) return false;
    whole = s0 == 0 && s1 == u.n;
    const bool has0 = u.e0 > u.a0, has1 = u.e1 > u.a1;
    j0 = max(s0, (has0 ? u.a0 : u.a1) - u.first);
    j1 = min(s1, (has1 ? u.e1 : u.e0) - u.first);
    if (j1 < j0) j1 = j0;
    slot = first ? 0 : 1;
    first = false;
    left -= s1 - s0;
    off = 0;
    if (++unit == units) {
      unit = 0;
      head++;
    }
    return true;
  }
  // whether row tile t needs key tile j (counted from u.first)
  __device__ __forceinline__ bool act(int t, int j) const {
    return u.first + j >= (t ? u.a1 : u.a0) && u.first + j < (t ? u.e1 : u.e0);
  }
  // keys of tile j that only some rows see, some of them held
  __device__ __forceinline__ bool mixed(int j) const {
    const int k0 = (u.first + j) * kTile, k1 = k0 + kTile;
    return max(k0, u.any0) < u.all0 || min(k1, u.any1) > u.all1;
  }
  __device__ __forceinline__ bool ragged(int j) const {
    const int k0 = (u.first + j) * kTile;
    return k0 < u.any0 || k0 + kTile > u.any1;
  }
};

// 16-byte chunk of operand row r, channels 8 ch .. 8 ch + 7
template <int D>
__device__ __forceinline__ uint32_t op_off(int r, int ch) {
  return (ch >> 3) * (kTile * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

// Zeroes the rows of a V tile outside [r0, r1) and, where `mixed`, replaces
// values that are not finite by zero; returns whether there were any.  The
// rows that see them get them back at the end (add_poison).
template <class C>
__device__ __forceinline__ bool clean_v(uint32_t v, int r0, int r1, bool mixed, int lane) {
  constexpr uint32_t E = C::BF ? 0x7F807F80u : 0x7C007C00u;
  bool hit = false;
  for (int i = lane; i < kTile * (C::D / 8); i += 32) {
    const int r = i / (C::D / 8), ch = i % (C::D / 8);
    const uint32_t a = v + op_off<C::D>(r, ch);
    if (r < r0 || r >= r1) {
      sts16(a, 0, 0, 0, 0);
    } else if (mixed) {
      uint4 x = lds16(a);
      const uint32_t m0 = __vcmpeq2(x.x & E, E), m1 = __vcmpeq2(x.y & E, E),
                     m2 = __vcmpeq2(x.z & E, E), m3 = __vcmpeq2(x.w & E, E);
      if (m0 | m1 | m2 | m3) {
        hit = true;
        sts16(a, x.x & ~m0, x.y & ~m1, x.z & ~m2, x.w & ~m3);
      }
    }
  }
  return hit;
}

// Adds the values that are not finite, in the mixed tiles of a part, of the
// keys a row sees, to channels d0 .. d0 + 31 of its O.  keys0, keys1: the
// part's keys; all0, all1: those every row sees.
template <class C>
__device__ __noinline__ void add_poison(const Cache c, const int32_t* table, int h, int keys0,
                                        int keys1, int any0, int any1, int all0, int all1, int lo,
                                        int hi, int d0, float* o) {
  for (int k0 = keys0; k0 < keys1; k0 += kTile) {
    if (!(max(k0, any0) < all0 || min(k0 + kTile, any1) > all1)) continue;
    for (int key = max(k0, lo); key <= min(k0 + kTile - 1, hi); key++) {
      const int page = __ldg(table + key / c.page_size);
      if (page < 0 || page >= c.num_pages) continue;
      const uint8_t* v = c.v + page * c.page_bytes + (int64_t)(key % c.page_size) * c.token_bytes +
                         h * c.head_bytes;
      for (int i = 0; i < 32; i++) {
        float x;
        if (C::E8) {
          x = (v[d0 + i] & 0x7F) == 0x7F ? NAN : 0.0f;
        } else {
          x = load_act(v, C::BF, d0 + i);
          if (isfinite(x)) x = 0.0f;
        }
        o[i] += x;
      }
    }
  }
}

__device__ __forceinline__ float row_inverse(float l, float vs) { return l > 0.0f || l != l ? vs / l : 0.0f; }
__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.0f || l != l ? (m + log2f(l)) * kLn2 : -INFINITY;
}

struct Maps {
  CUtensorMap k, v;
  int box;          // tokens of a box
  int heads_first;  // dimension 1 is the heads (else the tokens of a page)
};

// ------------------------------------------------------------ main kernel
template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    attn_tiles_kernel(const __grid_constant__ Maps maps, AttnParams p, Plan pl) {
  constexpr int D = C::D;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* kv_empty = kv_full + C::kStages;
  uint64_t* raw_full = kv_empty + C::kStages;
  uint64_t* raw_empty = raw_full + C::kRawStages;
  uint64_t* q_full = raw_empty + C::kRawStages;  // [2] each from here on
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* all_done = o_full + 2;
  volatile uint32_t* gone = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc) + kGone;
  volatile uint32_t* poison = tmem_slot + 1;  // a count of cleaned values' parts

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; i++) {
      mbar_init(&kv_full[i], C::E8 ? 4 : 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < C::kRawStages; i++) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int t = 0; t < 2; t++) {
      mbar_init(&q_full[t], 4);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_full[t], 1);
    }
    mbar_init(all_done, 1);
    *poison = 0;
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_or_abort(bar, parity, p.status)) != 0;
  };

  if (warp < 8) {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoft));
    const int t = warp >> 2, q4 = warp & 3;
    const int row = 32 * q4 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const uint32_t s_col = tmem + lane_base + t * kTile;
    const uint32_t o_col = tmem + lane_base + 2 * kTile + t * D;
    const uint32_t q_s = sbase + t * C::kOp;
    uint32_t steps = 0;  // key tiles this row tile has gone through
    uint32_t base = 0;   // key tiles the CTA has loaded before this unit
    bool ok = true;
    Walk w(p, pl);
    while (ok && w.next()) {
      const int nt = min(kTile, w.u.nrows - t * kTile);  // rows of the tile
      const int j0 = max(w.s0, (t ? w.u.a1 : w.u.a0) - w.u.first);
      const int j1 = min(w.s1, (t ? w.u.e1 : w.u.e0) - w.u.first);
      const int prow = w.u.row0 + t * kTile + min(row, max(nt, 1) - 1);
      const int tok = min(prow, w.u.row0 + w.u.nrows - 1) / p.group;
      const int token = w.u.s.q0 + tok;
      const int head = w.h * p.group + min(prow, w.u.row0 + w.u.nrows - 1) % p.group;
      const int hi = vis_hi(p, w.u.s, tok), lo = vis_lo(p, w.u.s, tok);
      float c = p.scale_log2 * (C::E8 && p.cache.k_scale ? __ldg(p.cache.k_scale + w.h) : 1.0f);
      if (j0 < j1) {
        // ---- queries to shared memory (the last product that read the
        // previous ones is done: its scores were seen)
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)token * p.q_ts +
                                                          (int64_t)head * p.q_hs);
        uint4 v[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; i++) v[i] = row < nt ? src[i] : make_uint4(0, 0, 0, 0);
        if (C::E8 && C::BF) {
          // bf16 to fp16 by a power of two per row
          float am = 0.0f;
#pragma unroll
          for (int i = 0; i < D / 8; i++) {
            const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int y = 0; y < 4; y++)
              am = fmaxf(am, fmaxf(fabsf(__uint_as_float(x[y] << 16)),
                                   fabsf(__uint_as_float(x[y] & 0xFFFF0000u))));
          }
          const int sh = fp16_scale_exp(am);
          const float f = exp2f((float)sh);
          c *= exp2f((float)-sh);
          auto cv = [&](uint32_t x) {
            return pack2<0>(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xFFFF0000u) * f);
          };
#pragma unroll
          for (int i = 0; i < D / 8; i++)
            v[i] = make_uint4(cv(v[i].x), cv(v[i].y), cv(v[i].z), cv(v[i].w));
        }
#pragma unroll
        for (int i = 0; i < D / 8; i++)
          sts16(q_s + op_off<D>(row, i), v[i].x, v[i].y, v[i].z, v[i].w);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
      }
      float m = -INFINITY, l = 0.0f;
      for (int j = j0; j < j1; j++, steps++) {
        if (!(ok = wait(&s_full[t], steps & 1))) break;
        tc_fence_after();
        float s[kTile];
        uint32_t* sr = reinterpret_cast<uint32_t*>(s);
#pragma unroll
        for (int i = 0; i < 4; i++) tmem_ld32(s_col + 32 * i, sr + 32 * i);
#pragma unroll
        for (int i = 0; i < 4; i++) tmem_ld32_wait(sr + 32 * i);
        const int k0 = (w.u.first + j) * kTile;
        const uint32_t gm = gone[(base + j - w.j0) % kGone];
        if (k0 < w.u.all0 || k0 + kTile > w.u.all1 || gm) {
          const int h0 = hi - k0, l0 = lo - k0;
#pragma unroll
          for (int i = 0; i < kTile; i++)
            if (i > h0 || i < l0 || (gm >> (i >> 4) & 1)) s[i] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < kTile; i += 4)
#pragma unroll
          for (int e = 0; e < 4; e++) mx[e] = fmaxf(mx[e], s[i + e]);
        const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c);
        if (j == j0) {
          m = mn;
        } else {
          const bool grow = mn > m + kRescale || (m == -INFINITY && mn > m);
          if (__any_sync(0xffffffffu, grow)) {
            const float f = grow ? ex2(m - mn) : 1.0f;
            if (grow) m = mn;
            l *= f;
            // the product that last added to O is done
            if (!(ok = wait(&o_full[t], (steps - 1) & 1))) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < D / 32; i++) {
              uint32_t o[32];
              tmem_ld32(o_col + 32 * i, o);
              tmem_ld32_wait(o);
#pragma unroll
              for (int e = 0; e < 32; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(o_col + 32 * i, o);
            }
          }
        }
        const float ms = m == -INFINITY ? 0.0f : m;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int half = 0; half < 2; half++) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; i++) {
            float &x = s[64 * half + 2 * i], &y = s[64 * half + 2 * i + 1];
            fma2(x, y, c, -ms);
            x = ex2(x);
            y = ex2(y);
            add2(sum[(i & 1) * 2], sum[(i & 1) * 2 + 1], x, y);
            pk[i] = pack2<C::MBF>(x, y);
          }
          tmem_st32(s_col + 32 * half, pk);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      // ---- output
      if (j0 < j1) {
        if (!(ok = wait(&o_full[t], (steps - 1) & 1))) break;
        tc_fence_after();
      }
      const float vs = C::E8 && p.cache.v_scale ? __ldg(p.cache.v_scale + w.h) : 1.0f;
      const float inv = w.whole ? row_inverse(l, vs) : 1.0f;
      const bool bad_v = *poison != 0;
      float* part = pl.parts + ((size_t)blockIdx.x * 2 + w.slot) * part_floats(D);
      const int prt = t * kTile + row;
#pragma unroll 1
      for (int i = 0; i < D / 32; i++) {
        float o[32];
        uint32_t* orr = reinterpret_cast<uint32_t*>(o);
        __syncwarp();
        if (j0 < j1) {
          tmem_ld32(o_col + 32 * i, orr);
          tmem_ld32_wait(orr);
        } else {
#pragma unroll
          for (int e = 0; e < 32; e++) o[e] = 0.0f;
        }
        if (row < nt) {
          if (bad_v) {
            float tmp[32];
#pragma unroll
            for (int e = 0; e < 32; e++) tmp[e] = o[e];
            add_poison<C>(p.cache, p.batch.table + (int64_t)w.u.b * p.batch.table_stride, w.h,
                          (w.u.first + w.s0) * kTile, (w.u.first + w.s1) * kTile, w.u.any0, w.u.any1,
                          w.u.all0, w.u.all1, lo, hi, 32 * i, tmp);
#pragma unroll
            for (int e = 0; e < 32; e++) o[e] = tmp[e];
          }
          if (w.whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.out + ((int64_t)token * p.heads + head) * D + 32 * i);
#pragma unroll
            for (int e = 0; e < 4; e++)
              dst[e] = make_uint4(pack2<C::BF>(o[8 * e] * inv, o[8 * e + 1] * inv),
                                  pack2<C::BF>(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                  pack2<C::BF>(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                                  pack2<C::BF>(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
          } else {
            float4* dst = reinterpret_cast<float4*>(part + (size_t)prt * D + 32 * i);
#pragma unroll
            for (int e = 0; e < 8; e++)
              dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
      }
      tc_fence_before();  // O is read before the next unit's first product writes it
      if (row < nt) {
        if (!w.whole)
          *reinterpret_cast<float2*>(part + (size_t)kUnitRows * D + 2 * prt) = make_float2(m, l);
        else if (p.lse)
          p.lse[(int64_t)token * p.heads + head] = row_lse(m, l);
      }
      base += w.j1 - w.j0;
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------------ MMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    const uint32_t bf = C::MBF ? (1u << 7) | (1u << 10) : 0u;
    const uint32_t id_qk = umma_idesc_f16(kTile, kTile, 0, 0) | bf;
    const uint32_t id_pv = umma_idesc_f16(kTile, D, 0, 1) | bf;
    uint64_t qd[2];
    for (int t = 0; t < 2; t++) qd[t] = umma_desc(sbase + t * C::kOp, 16, 1024);
    // V: rows of 128 bytes hold 64 channels of one key; 8 keys 1024 B, the
    // second 64 channels kTile * 128 B on
    const uint64_t kd0 = umma_desc(sbase + C::kOffKV, 16, 1024);
    const uint64_t vd0 = umma_desc(sbase + C::kOffKV, kTile * 128, 1024);
    uint32_t n_q[2] = {0, 0}, n_p[2] = {0, 0};
    uint32_t load = 0;  // loads of the steps so far (K then V of each)
    bool ok = true;
    Walk w(p, pl);
    while (ok && w.next()) {
      uint32_t lk = 0, lk_prev = 0;    // load index of K of step j, j - 1
      bool started[2] = {false, false};
      bool any_prev = false;
      for (int j = w.j0; ok && j <= w.j1; j++) {
        const bool any = j < w.j1;
        if (any) {
          lk = load;
          load += 2;
        }
        const uint32_t kst = lk % C::kStages, vst = (lk_prev + 1) % C::kStages;
        if (any_prev) {
          if (!(ok = wait(&kv_full[vst], ((lk_prev + 1) / C::kStages) & 1))) break;
          if (!C::E8) {
            const bool mix = w.mixed(j - 1);
            if (mix || w.ragged(j - 1)) {
              const int k0 = (w.u.first + j - 1) * kTile;
              const bool hit = clean_v<C>(sbase + C::kOffKV + vst * C::kOp, w.u.any0 - k0,
                                          w.u.any1 - k0, mix, lane);
              if (__any_sync(0xffffffffu, hit) && lane == 0) *poison = 1;
              __threadfence_block();
              fence_async_smem();
              __syncwarp();
            }
          }
        }
        bool k_here = false;
#pragma unroll
        for (int t = 0; t < 2; t++) {
          if (any_prev && w.act(t, j - 1)) {
            if (!(ok = wait(&p_full[t], n_p[t] & 1))) break;
            n_p[t]++;
            tc_fence_after();
            if (lane == 0) {
              const uint32_t o = tmem + 2 * kTile + t * D, a = tmem + t * kTile;
              const uint64_t vd = vd0 + (uint64_t)(vst * (C::kOp >> 4));
#pragma unroll
              for (int k = 0; k < kTile / 16; k++)
                umma_ts(o, a + 8 * k, vd + k * (2048 >> 4), id_pv, started[t] || k > 0);
              umma_commit(&o_full[t]);
            }
            started[t] = true;
            __syncwarp();
          }
          if (any && w.act(t, j)) {
            if (!k_here) {
              if (!(ok = wait(&kv_full[kst], (lk / C::kStages) & 1))) break;
              k_here = true;
            }
            if (j == max(w.s0, (t ? w.u.a1 : w.u.a0) - w.u.first)) {
              if (!(ok = wait(&q_full[t], n_q[t] & 1))) break;
              n_q[t]++;
            }
            tc_fence_after();
            if (lane == 0) {
              const uint64_t kd = kd0 + (uint64_t)(kst * (C::kOp >> 4));
#pragma unroll
              for (int k = 0; k < D / 16; k++) {
                const uint64_t off = (uint64_t)(((k >> 2) * (kTile * 128) + (k & 3) * 32) >> 4);
                umma_f16(tmem + t * kTile, qd[t] + off, kd + off, id_qk, k > 0);
              }
              umma_commit(&s_full[t]);
            }
            __syncwarp();
          }
        }
        if (!ok) break;
        if (lane == 0) {
          if (any_prev) umma_commit(&kv_empty[vst]);
          if (any) umma_commit(&kv_empty[kst]);
        }
        __syncwarp();
        any_prev = any;
        lk_prev = lk;
      }
    }
    if (lane == 0) umma_commit(all_done);
  } else if (warp == 9) {
    // ------------------------------------------------------------------ TMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    constexpr int ST = C::E8 ? C::kRawStages : C::kStages;
    constexpr int HALF = C::E8 ? 1 : D / 64;      // boxes across the channels
    constexpr uint32_t BYTES = C::E8 ? C::kRaw : C::kOp;
    uint64_t* full = C::E8 ? raw_full : kv_full;
    uint64_t* empty = C::E8 ? raw_empty : kv_empty;
    const uint32_t ring = sbase + (C::E8 ? C::kOffRaw : C::kOffKV);
    const int nbox = kTile / maps.box;
    const int bx = lane / HALF, half = lane % HALF;
    const bool mine = bx < nbox;
    uint32_t load = 0;
    int32_t bad = 0;
    bool ok = true;
    Walk w(p, pl);
    while (ok && w.next()) {
      const int32_t* table = p.batch.table + (int64_t)w.u.b * p.batch.table_stride;
      for (int j = w.j0; ok && j < w.j1; j++) {
        const int key = (w.u.first + j) * kTile + bx * maps.box;
        int page = p.cache.num_pages;  // out of range: zeros
        bool absent = false;
        if (mine && key < w.u.any1 && key + maps.box > w.u.any0) {
          const int id = __ldg(table + key / p.cache.page_size);
          absent = id < 0 || id >= p.cache.num_pages;
          if (!absent) page = id;
        }
        // 16-key groups of absent pages
        uint32_t g = absent ? ((1u << (maps.box / 16)) - 1) << (bx * (maps.box / 16)) : 0u;
        g = __reduce_or_sync(0xffffffffu, g);
        if (g) bad |= kStatusBadPage;
        const int at = key % p.cache.page_size;
        for (int x = 0; x < 2; x++) {  // K, V
          const uint32_t st = load % ST;
          if (!(ok = wait(&empty[st], ((load / ST) & 1) ^ 1))) break;
          if (lane == 0) {
            if (x == 0) gone[(load >> 1) % kGone] = g;
            mbar_arrive_expect_tx(&full[st], BYTES);
          }
          __syncwarp();
          if (mine) {
            const uint32_t dst = ring + st * BYTES + half * (kTile * 128) +
                                 bx * maps.box * (C::E8 ? D : 128);
            const CUtensorMap* m = x == 0 ? &maps.k : &maps.v;
            if (maps.heads_first)
              tma_load_4d(dst, m, half * 64, w.h, at, page, &full[st]);
            else
              tma_load_4d(dst, m, half * 64, at, w.h, page, &full[st]);
          }
          load++;
        }
      }
    }
    if (bad && lane == 0) atomicOr(p.status, bad);
    // every box this warp requested has landed before the CTA may exit
    for (uint32_t i = load < ST ? 0 : load - ST; i < load; i++)
      mbar_drain(&full[i % ST], (i / ST) & 1, kWaitBudgetCycles);
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
  } else if constexpr (C::E8) {
    // -------------------------------------------------- widen E4M3 to fp16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    const int tid = threadIdx.x - 12 * 32;
    uint32_t load = 0;
    bool ok = true;
    Walk w(p, pl);
    while (ok && w.next()) {
      for (int j = w.j0; ok && j < w.j1; j++) {
        const int k0 = (w.u.first + j) * kTile;
        const int r0 = w.u.any0 - k0, r1 = w.u.any1 - k0;
        const bool mix = w.mixed(j);
        for (int x = 0; x < 2; x++) {
          const uint32_t rs = load % C::kRawStages, cs = load % C::kStages;
          if (!(ok = wait(&raw_full[rs], (load / C::kRawStages) & 1) &&
                     wait(&kv_empty[cs], ((load / C::kStages) & 1) ^ 1)))
            break;
          const uint32_t src = sbase + C::kOffRaw + rs * C::kRaw;
          const uint32_t dst = sbase + C::kOffKV + cs * C::kOp;
          bool hit = false;
#pragma unroll 4
          for (int i = tid; i < C::kRaw / 16; i += 128) {
            const int r = i / (D / 16), ch = i % (D / 16);
            uint4 v = lds16(src + i * 16);
            if (x == 1) {
              if (r < r0 || r >= r1) v = make_uint4(0, 0, 0, 0);
              if (mix) {
                constexpr uint32_t E = 0x7F7F7F7Fu;
                const uint32_t m0 = __vcmpeq4(v.x & E, E), m1 = __vcmpeq4(v.y & E, E),
                               m2 = __vcmpeq4(v.z & E, E), m3 = __vcmpeq4(v.w & E, E);
                hit |= (m0 | m1 | m2 | m3) != 0;
                v = make_uint4(v.x & ~m0, v.y & ~m1, v.z & ~m2, v.w & ~m3);
              }
            }
            const uint32_t y[8] = {e4m3_to_f16x2(v.x), e4m3_to_f16x2(v.x >> 16),
                                   e4m3_to_f16x2(v.y), e4m3_to_f16x2(v.y >> 16),
                                   e4m3_to_f16x2(v.z), e4m3_to_f16x2(v.z >> 16),
                                   e4m3_to_f16x2(v.w), e4m3_to_f16x2(v.w >> 16)};
            // lanes of the upper channels store their second chunk first: 8
            // lanes then cover all banks
            const uint32_t a0 = dst + op_off<D>(r, 2 * ch), a1 = dst + op_off<D>(r, 2 * ch + 1);
            if (ch & (D / 32)) {
              sts16(a1, y[4], y[5], y[6], y[7]);
              sts16(a0, y[0], y[1], y[2], y[3]);
            } else {
              sts16(a0, y[0], y[1], y[2], y[3]);
              sts16(a1, y[4], y[5], y[6], y[7]);
            }
          }
          if (hit) *poison = 1;
          __threadfence_block();
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&raw_empty[rs]);
            mbar_arrive(&kv_full[cs]);
          }
          load++;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    mbar_drain(all_done, 0, kWaitBudgetCycles);
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Sums the parts of every unit that a cut goes through: block (x, y) takes
// cut x + 1 (if it is its unit's first) and rows 8 y .. of every 8 gridDim.y.
template <class C>
__global__ void __launch_bounds__(256) attn_tiles_join_kernel(AttnParams p, Plan pl) {
  constexpr int D = C::D;
  pdl_wait();
  const PlanHead hd = *pl.head;
  const int cut = blockIdx.x + 1;
  if (cut >= hd.pieces) return;
  const long long all = hd.line * p.kv_heads;
  const Start st = pl.start[cut];
  if (st.off == 0) return;
  const long long u0 = piece_start(all, hd.pieces, cut) - st.off;
  if (piece_start(all, hd.pieces, cut - 1) > u0) return;
  const int2 rec = pl.rec[st.unit];
  int32_t ignored = 0;
  const Unit u = make_unit(p, rec.x, load_seq(p.batch, rec.x, &ignored), rec.y);
  const int first = cut - 1;
  int last = cut;
  while (last + 1 < hd.pieces && piece_start(all, hd.pieces, last + 1) < u0 + u.n) last++;
  const size_t slot0 = (size_t)first * 2 + (piece_start(all, hd.pieces, first) < u0 ? 1 : 0);
  const float vs = C::E8 && p.cache.v_scale ? __ldg(p.cache.v_scale + st.head) : 1.0f;
  constexpr int LR = D / 4;
  const int d0 = (threadIdx.x % LR) * 4;
  for (int r = blockIdx.y * (256 / LR) + threadIdx.x / LR; r < u.nrows;
       r += gridDim.y * (256 / LR)) {
    float mm = -INFINITY, ll = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int c = first; c <= last; c++) {
      const float* part = pl.parts + (c == first ? slot0 : (size_t)c * 2) * part_floats(D);
      const float2 s = *reinterpret_cast<const float2*>(part + (size_t)kUnitRows * D + 2 * r);
      const float4 x = *reinterpret_cast<const float4*>(part + (size_t)r * D + d0);
      const float mn = fmaxf(mm, s.x);
      const float ms = mn == -INFINITY ? 0.0f : mn;
      const float f0 = ex2(mm - ms), f1 = ex2(s.x - ms);
      mm = mn;
      ll = ll * f0 + s.y * f1;
      acc[0] = acc[0] * f0 + x.x * f1;
      acc[1] = acc[1] * f0 + x.y * f1;
      acc[2] = acc[2] * f0 + x.z * f1;
      acc[3] = acc[3] * f0 + x.w * f1;
    }
    const int prow = u.row0 + r;
    const int token = u.s.q0 + prow / p.group, head = st.head * p.group + prow % p.group;
    const float inv = row_inverse(ll, vs);
    uint2 o;
    o.x = pack2<C::BF>(acc[0] * inv, acc[1] * inv);
    o.y = pack2<C::BF>(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2*>(p.out + ((int64_t)token * p.heads + head) * D + d0) = o;
    if (p.lse && d0 == 0) p.lse[(int64_t)token * p.heads + head] = row_lse(mm, ll);
  }
}

// ------------------------------------------------------------ host
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<EncodeTiledFn>(ptr);
  }();
  return fn;
}

// The cache as a 4-D TMA source: channels, then heads and tokens of a page
// (the nearer in memory first), pages; a box is up to 128 tokens of one head.
bool make_maps(const AttnParams& p, Maps* m) {
  EncodeTiledFn fn = encode_fn();
  const Cache& c = p.cache;
  if (!fn || c.num_pages < 1) return false;
  m->box = c.page_size & -c.page_size;
  if (m->box > kTile) m->box = kTile;
  // (a dimension of one has no stride of its own)
  const int64_t row = (int64_t)p.dim * (p.e4m3 ? 1 : 2);
  const int64_t hb = p.kv_heads > 1 ? c.head_bytes : row, tb = c.token_bytes;
  const int64_t pb = c.num_pages > 1 ? c.page_bytes : row;
  m->heads_first = hb <= tb;
  const cuuint64_t dims[4] = {(cuuint64_t)p.dim,
                              (cuuint64_t)(m->heads_first ? p.kv_heads : c.page_size),
                              (cuuint64_t)(m->heads_first ? c.page_size : p.kv_heads),
                              (cuuint64_t)c.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)(m->heads_first ? hb : tb),
                                 (cuuint64_t)(m->heads_first ? tb : hb), (cuuint64_t)pb};
  const cuuint32_t inner = p.e4m3 ? (cuuint32_t)p.dim : 64u;
  const cuuint32_t box[4] = {inner, m->heads_first ? 1u : (cuuint32_t)m->box,
                             m->heads_first ? (cuuint32_t)m->box : 1u, 1u};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  for (int i = 0; i < 2; i++)
    if (fn(i ? &m->v : &m->k,
           p.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 4,
           const_cast<uint8_t*>(i ? c.v : c.k), dims, strides, box, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE,
           p.e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}

template <class C>
cudaError_t launch_cfg(const AttnParams& p, const Maps& maps, const Plan& pl, int max_unit,
                       cudaStream_t st) {
  static_assert(C::kSmem <= 227 * 1024, "shared memory");
  static bool init = false;
  if (!init) {
    const cudaError_t e = cudaFuncSetAttribute(
        attn_tiles_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    init = true;
  }
  cudaError_t e = launch_pdl(attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, p, pl, max_unit);
  note_launches(1);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_tiles_kernel<C>, dim3(kGrid), dim3(C::kThreads), C::kSmem, st, maps, p, pl);
  note_launches(1);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_tiles_join_kernel<C>, dim3(kGrid - 1, 8), dim3(256), 0, st, p, pl);
  note_launches(1);
  return e;
}

template <int D>
cudaError_t launch_types(const AttnParams& p, const Maps& m, const Plan& pl, int mu,
                         cudaStream_t st) {
  if (p.e4m3)
    return p.bf16 ? launch_cfg<Cfg<D, 1, 1>>(p, m, pl, mu, st)
                  : launch_cfg<Cfg<D, 1, 0>>(p, m, pl, mu, st);
  return p.bf16 ? launch_cfg<Cfg<D, 0, 1>>(p, m, pl, mu, st)
                : launch_cfg<Cfg<D, 0, 0>>(p, m, pl, mu, st);
}

}  // namespace

size_t attn_tiles_scratch_bytes(long long rows, int seqs, int dim) {
  return carve(nullptr, rows, seqs, nullptr) + (size_t)kGrid * 2 * part_floats(dim) * 4;
}

bool attn_tiles_can(const AttnParams& p) {
  Maps m;
  return make_maps(p, &m);
}

cudaError_t launch_attn_tiles(const AttnParams& p, cudaStream_t st) {
  Maps m;
  if (!make_maps(p, &m)) return cudaErrorNotSupported;
  const long long rows = (long long)p.batch.T * p.group;
  Plan pl;
  carve(p.scratch, rows, p.batch.num_seqs, &pl);
  const int mu = (int)max_units(rows, p.batch.num_seqs);
  return p.dim == 64 ? launch_types<64>(p, m, pl, mu, st) : launch_types<128>(p, m, pl, mu, st);
}

}  // namespace exl3
