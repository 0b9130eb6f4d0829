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
// tile each, one thread per row: no shuffles); a warp that issues the MMAs and
// nothing else, since the tensor core idles whenever it is late (one warp, not
// one per row tile: it keeps the row tiles in turn, and two free-running ones
// fall into step, both in softmax, then both in products, 1.5 times slower); a
// warp that walks the work, publishes each unit to the others and issues the
// TMA loads; a warp that brings in the next unit's queries; and a warp that
// cleans the few V tiles that need it, or, for E4M3 caches, four warps that
// widen the 8-bit tiles to fp16 (exact) in shared memory and clean them on the
// way.
//   S = Q K^T   A, B from shared memory, S (128 fp32 columns) in TMEM
//   P           written over S as 16-bit pairs, the A operand of
//   O += P V    B = V as it lies in memory (keys are the K dimension, so V is
//               the MN-major operand), O (head_dim fp32 columns) in TMEM
// P is handed over in two halves of 64 keys, so that the product starts while
// the second half's exponentials are taken.
// A row's O is rescaled only when its maximum has grown by more than 2^8
// since the last time (P stays in range for both 16-bit types, and the final
// division removes the common factor), which leaves almost no rescales after a
// row's first tiles.  P is 16 bits because that is what the tensor core
// multiplies: bf16 rounds a term by 2^-9 of it, fp16 by 2^-12; the sum is of
// the unrounded terms.
// What a step takes the longest for is not the products (2048 cycles of the
// tensor core at head_dim 128) but this code around them, and first of all the
// fetching of it: the MMA warp waited for almost nothing and still took 3000
// cycles a step (chunks of 512 at 16384 keys, 205 us), 2450 with the steps in
// the middle of a unit written out from uniform registers (190 us; over a whole
// call, start, unit changes and end included, 2950 to 3030).  So there
// is one copy of everything (terms against the maximum of the tiles before,
// which need a second one for the first tile and for rescales, were as fast
// over long units and 20 % slower over short ones).
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
//
// Block scales (a scale per page and kv head, E4M3) go from the TMA warp, which
// knows the pages, to the softmax warps in a ring beside that of absent pages,
// one entry per 16 keys.  With S the product of the queries and the stored keys
//   x = S scale ks + log2 vs,  w = 2^(x - m),  O += w v,  l += w / vs,
// so that the 16-bit terms w are largest where a key's share of the output is,
// whatever the scales of other blocks.  ks > 0: a group's maximum of x is that
// of S, and a term costs one fma as without block scales.
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
constexpr int kScaleSteps = 8;      // ring of block scales (at most stages + 3 in use)
constexpr int kUnits = 4;           // ring of published units
constexpr int kRecInts = 24;

template <int D_, int E8_, int BF_, int BS_ = 0>
struct Cfg {
  static constexpr int D = D_, E8 = E8_, BF = BF_;
  // block scales: 16-key groups that share one (1 or 4; 0: a scale per head)
  static constexpr int BS = BS_;
  static constexpr int MBF = BF && !E8;                  // type of the products
  // log2 of a factor of the terms: fp16 holds what is below 2^-14 in fewer
  // bits, so there they are 2^7 times as large (below 2^15 with kRescale)
  static constexpr float kLift = MBF ? 0.0f : 7.0f;
  static constexpr int kOp = kTile * D * 2;              // bytes of a 16-bit operand tile
  static constexpr int kRaw = kTile * D;                 // bytes of an E4M3 tile
  // stages of K and of V
  static constexpr int kStages = D == 64 ? 4 : 2, kStageBits = D == 64 ? 2 : 1;
  static constexpr int kOffK = 2 * kOp;
  static constexpr int kOffV = kOffK + kStages * kOp;
  static constexpr int kOffRaw = kOffV + kStages * kOp;  // E4M3: one K and one V tile
  static constexpr int kOffBar = kOffRaw + (E8 ? 2 * kRaw : 0);
  static constexpr int kBars = 5 * kStages + 4 + 15 + 2 * kUnits;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kOffUnits = kOffMisc + kGone * 4 + 16;
  static constexpr int kOffScales = (kOffUnits + kUnits * kRecInts * 4 + 15) & ~15;
  static constexpr int kSmem = kOffScales + (BS ? kScaleSteps * (kTile / 16) * 32 : 0);
  static_assert(kStages + 3 <= kScaleSteps, "ring");
  static constexpr int kCvtQ = E8 && BF;   // queries are brought to fp16
  static constexpr int kThreads = E8 ? 512 : 384;
  // registers of a softmax thread and of the others (their sum over the CTA
  // is what the launch holds: 128 or 168 a thread)
  static constexpr int kRegsSoft = E8 ? 192 : 216, kRegsRest = E8 ? 64 : 72;
  static constexpr int kTmemCols = 512;
};

// ------------------------------------------------------------ PTX helpers
// MMAs and commits are issued by a converged warp, one elected lane each (the
// same one for the same mask): the operands then stay in uniform registers.
// From a one-lane branch the issue of 8 MMAs takes 370 cycles, this way 90, of
// the 512 they run.  What comes from memory passes through a warp reduction and
// every branch hangs on a vote, so that all of it is uniform.
// (a, b: low words of the operands' descriptors, whose high word is kDescHi)
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
// Four products over 16 channels each, both operands 32 bytes on per product.
__device__ __forceinline__ void umma_ss4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 x<3>, y<3>;\n\t.reg .b64 a<4>, b<4>;\n\t"
      "add.u32 x0, %1, 2;\n\tadd.u32 x1, %1, 4;\n\tadd.u32 x2, %1, 6;\n\t"
      "add.u32 y0, %2, 2;\n\tadd.u32 y1, %2, 4;\n\tadd.u32 y2, %2, 6;\n\t"
      "mov.b64 a0, {%1, %5};\n\tmov.b64 a1, {x0, %5};\n\t"
      "mov.b64 a2, {x1, %5};\n\tmov.b64 a3, {x2, %5};\n\t"
      "mov.b64 b0, {%2, %5};\n\tmov.b64 b1, {y0, %5};\n\t"
      "mov.b64 b2, {y1, %5};\n\tmov.b64 b3, {y2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a0, b0, %3, p;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, 1;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// Four products over 16 keys each: A 8 columns of TMEM on per product, B 16
// rows of 128 bytes.
__device__ __forceinline__ void umma_ts4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 x<3>, y<3>;\n\t.reg .b64 b<4>;\n\t"
      "add.u32 x0, %1, 8;\n\tadd.u32 x1, %1, 16;\n\tadd.u32 x2, %1, 24;\n\t"
      "add.u32 y0, %2, 128;\n\tadd.u32 y1, %2, 256;\n\tadd.u32 y2, %2, 384;\n\t"
      "mov.b64 b0, {%2, %5};\n\tmov.b64 b1, {y0, %5};\n\t"
      "mov.b64 b2, {y1, %5};\n\tmov.b64 b3, {y2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b0, %3, p;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x0], b1, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x1], b2, %3, 1;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x2], b3, %3, 1;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar))
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
__device__ __forceinline__ void tmem_st16(uint32_t a, const float* v) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; i++) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
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
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int c0, int c1, int c2,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
// A whole warp waits for a phase of a barrier: the lanes' answers are voted
// on, so that the warp never diverges and a ready barrier costs a few
// instructions (the MMA warp's waits are on the critical path of every tile).
// False once a wait ran out of budget, here or (status word) anywhere.
__device__ __forceinline__ bool wait_some(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n\tmov.u32 %0, 1;\n\t"
      "WAIT:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "vote.sync.all.pred p, p, 0xffffffff;\n\t"
      "@p bra.uni END;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.lt.u32 p, n, 64;\n\t"
      "@p bra.uni WAIT;\n\t"
      "mov.u32 %0, 0;\n\t"
      "END:\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, int32_t* status) {
  const long long t0 = clock64();
  while (!wait_some(bar, parity)) {
    bool stop = *reinterpret_cast<volatile int32_t*>(status) & kStatusTimeout;
    if (clock64() - t0 > kWaitBudgetCycles) {
      atomicOr(status, kStatusTimeout);
      stop = true;
    }
    if (__any_sync(0xffffffffu, stop)) return false;
  }
  return true;
}
// As wait_warp, written so that the compiler sees the warp stay together (the
// MMA warp's loops and operands then live in uniform registers) and short: at
// most `limit` looks of up to 1 us each, after which the limit is 1.
__device__ __forceinline__ bool wait_uniform(uint32_t bar, uint32_t parity, uint32_t& limit) {
  uint32_t looks = 0;
  do {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (__all_sync(0xffffffffu, ok)) return true;
  } while (++looks < limit);
  limit = 1;
  return false;
}
// The long wait out of line (the roles' code has to stay in the instruction
// caches): not for the softmax warps, whose registers a call would have to save.
__device__ __noinline__ bool wait_long_call(uint32_t bar, uint32_t parity, int32_t* status) {
  return wait_long(bar, parity, status);
}
template <bool CALL>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int32_t* status) {
  const uint32_t a = smem_u32(bar);
  if (__builtin_expect(wait_some(a, parity), 1)) return true;
  return CALL ? wait_long_call(a, parity, status) : wait_long(a, parity, status);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 operations at once
__device__ __forceinline__ uint64_t both(float x) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void fma2(float& x, float& y, uint64_t c, uint64_t d) {
  asm("{\n\t.reg .b64 a;\n\tmov.b64 a, {%0, %1};\n\tfma.rn.f32x2 a, a, %2, %3;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "l"(c), "l"(d));
}
__device__ __forceinline__ void mul2(float& x, float& y, uint64_t c) {
  asm("{\n\t.reg .b64 a;\n\tmov.b64 a, {%0, %1};\n\tmul.rn.f32x2 a, a, %2;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "l"(c));
}
__device__ __forceinline__ void add2(uint64_t& acc, float u, float v) {
  asm("{\n\t.reg .b64 b;\n\tmov.b64 b, {%1, %2};\n\tadd.rn.f32x2 %0, %0, b;\n\t}"
      : "+l"(acc)
      : "f"(u), "f"(v));
}
__device__ __forceinline__ float sum2(uint64_t a) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
  return x + y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 32 bytes, one sector
__device__ __forceinline__ void stg32(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                      uint32_t e, uint32_t f, uint32_t g, uint32_t h) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b),
               "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(bytes)
               : "memory");
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
  int splits;       // units that cuts go through
  int split_rows;   // the most rows of one
};
struct Start {
  int unit, head, off, pad;
};
// A unit that cuts go through: its parts are in the first part slots of the
// pieces first .. last, but for the first one's, slot0.
struct Split {
  int first, last, slot0;
  int row0, nrows, q0, head, pad;
};
struct Plan {
  PlanHead* head;
  Start* start;     // [kGrid]
  Split* split;     // [kGrid], in no particular order
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
  p.split = reinterpret_cast<Split*>(b + at);
  at += align256(sizeof(Split) * kGrid);
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
      // (no further than max_unit, whose overlapping sequences could count past
      // 32 bits: the search below needs ascending numbers)
      const int first = (int)min(run + inc - n, (long long)max_unit);
      pl.seq_unit[b] = first;
      if (b < kCache) unit_s[b] = first;
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
  __shared__ int splits, split_rows;
  if (threadIdx.x == 0) splits = split_rows = 0;
  __syncthreads();
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
    const int off = (int)(s - (pre_cached ? pre_s[lo] : pl.pre[lo]));
    pl.start[threadIdx.x] = Start{lo, (int)(at / run), off, 0};
    const long long u0 = at - off;  // the unit's place on the line
    if (off > 0 && piece_start(all, pieces, threadIdx.x - 1) <= u0) {
      // the first cut inside its unit
      const int2 rec = pl.rec[lo];
      int32_t ignored = 0;
      const Unit u = make_unit(p, rec.x, load_seq(p.batch, rec.x, &ignored), rec.y);
      const int first = threadIdx.x - 1;
      // the piece that holds the unit's last key tile
      const int last = (int)(((u0 + u.n) * pieces + all - 1) / all) - 1;
      const int slot0 = 2 * first + (piece_start(all, pieces, first) < u0 ? 1 : 0);
      pl.split[atomicAdd(&splits, 1)] =
          Split{first, last, slot0, u.row0, u.nrows, u.s.q0, (int)(at / run), 0};
      atomicMax(&split_rows, u.nrows);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) *pl.head = PlanHead{run, units, pieces, splits, split_rows};
}

// A part of a unit as the TMA warp publishes it (in shared memory).
struct Rec {
  int live;           // 0: no more
  int b, h;           // sequence, kv head
  int q0, n, len;     // its new tokens and length
  int row0, nrows;    // packed rows
  int any0, any1, all0, all1;
  int first;          // key tile that j counts from
  int s0, s1;         // the part's key tiles
  int j0, j1;         // those that some row needs
  int t0a, t0e, t1a, t1e;  // those that row tile 0, 1 needs (empty: a >= e)
  int c0, c1;         // key tiles that every row sees whole
  int flags;          // 1: the whole unit, 2: not the first part of the piece
};
static_assert(sizeof(Rec) == kRecInts * 4, "record");

// The piece of this CTA, part by part.
struct Walk {
  const AttnParams& p;
  const Plan& pl;
  int unit, head, off, units;
  long long left;
  bool first;
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
  __device__ Rec next() {
    Rec r{};
    if (left <= 0) return r;
    const int2 id = pl.rec[unit];
    int32_t ignored = 0;
    const Unit u = make_unit(p, id.x, load_seq(p.batch, id.x, &ignored), id.y);
    r.s0 = off;
    r.s1 = (int)min((long long)u.n, off + left);
    if (r.s1 <= r.s0) return r;
    r.live = 1;
    r.b = u.b;
    r.h = head;
    r.q0 = u.s.q0;
    r.n = u.s.n;
    r.len = u.s.len;
    r.row0 = u.row0;
    r.nrows = u.nrows;
    r.any0 = u.any0;
    r.any1 = u.any1;
    r.all0 = u.all0;
    r.all1 = u.all1;
    r.first = u.first;
    r.t0a = max(r.s0, u.a0 - u.first);
    r.t0e = min(r.s1, u.e0 - u.first);
    r.t1a = max(r.s0, u.a1 - u.first);
    r.t1e = min(r.s1, u.e1 - u.first);
    // (the two runs meet: row tile 1 starts no later than one past tile 0's end)
    const bool has0 = r.t0e > r.t0a, has1 = r.t1e > r.t1a;
    r.j0 = has0 ? r.t0a : r.t1a;
    r.j1 = has1 ? r.t1e : r.t0e;
    if (!has0 && !has1) r.j0 = r.j1 = 0;
    r.c0 = (u.all0 + kTile - 1) / kTile - u.first;
    r.c1 = min(u.all1, u.any1) / kTile - u.first;
    r.flags = (r.s0 == 0 && r.s1 == u.n ? 1 : 0) | (first ? 0 : 2);
    first = false;
    left -= r.s1 - r.s0;
    off = 0;
    if (++unit == units) {
      unit = 0;
      head++;
    }
    return r;
  }
};
// A V tile that needs cleaning, scores that need masking: not every row sees
// all of the tile's keys.
__device__ __forceinline__ bool edge(const Rec& r, int j) { return j < r.c0 || j >= r.c1; }
// The rows [m0, m1) of the V tile from key k0 on that every row sees.  Their
// values stay as they are, whatever they are: add_poison gives back only what
// some rows see and others do not.
__device__ __forceinline__ void seen_by_all(const Rec& r, int k0, int* m0, int* m1) {
  *m0 = min(max(r.all0 - k0, 0), kTile);
  *m1 = min(max(r.all1 - k0, *m0), kTile);
}

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

// Top bits of the 16-bit values of w (of the bytes, E4M3) that are infinite or
// NaN: adding one to an exponent of all ones carries into the sign's place.
template <class C>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  if (C::E8) return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  return C::BF ? ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u
               : ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
}
// The same values as a mask of all their bits.
template <class C>
__device__ __forceinline__ uint32_t whole_mask(uint32_t top) {
  return C::E8 ? (top >> 7) * 0xFFu : (top >> 15) * 0xFFFFu;
}

// Rows ra .. rb - 1 of a V tile: those outside [r0, r1) are zeroed, values in
// the others that are not finite replaced by zero; returns whether there were
// any.  The rows that see them get them back at the end (add_poison).
template <class C>
__device__ __forceinline__ bool clean_v(uint32_t v, int ra, int rb, int r0, int r1, int lane) {
  constexpr int CH = C::D / 8, RI = 32 / CH, UN = 4;
  bool hit = false;
  const int ch = lane % CH;
#pragma unroll 1
  for (int r = ra + lane / CH; r < rb; r += UN * RI) {
    uint4 x[UN];
#pragma unroll
    for (int k = 0; k < UN; k++) x[k] = lds16(v + op_off<C::D>(min(r + k * RI, rb - 1), ch));
#pragma unroll
    for (int k = 0; k < UN; k++) {
      const int rk = min(r + k * RI, rb - 1);  // (the last row more than once)
      const uint32_t m0 = not_finite<C>(x[k].x), m1 = not_finite<C>(x[k].y),
               m2 = not_finite<C>(x[k].z), m3 = not_finite<C>(x[k].w);
      const bool in = rk >= r0 && rk < r1;
      if (in && !(m0 | m1 | m2 | m3)) continue;
      hit |= in;
      sts16(v + op_off<C::D>(rk, ch), in ? x[k].x & ~whole_mask<C>(m0) : 0u,
            in ? x[k].y & ~whole_mask<C>(m1) : 0u, in ? x[k].z & ~whole_mask<C>(m2) : 0u,
            in ? x[k].w & ~whole_mask<C>(m3) : 0u);
    }
  }
  return hit;
}

// Adds the values that are not finite, in the mixed tiles of a part, of the
// keys a row sees, to its O as written: fp32 part, or out.  keys0, keys1: the
// part's keys; all0, all1: those every row sees.
template <class C>
__device__ __noinline__ void add_poison(const Cache c, const int32_t* table, int h, int keys0,
                                        int keys1, int any0, int any1, int all0, int all1, int lo,
                                        int hi, float* part, uint16_t* out) {
  for (int k0 = keys0; k0 < keys1; k0 += kTile) {
    if (!(max(k0, any0) < all0 || min(k0 + kTile, any1) > all1)) continue;
    for (int key = max(k0, lo); key <= min(k0 + kTile - 1, hi); key++) {
      const int page = __ldg(table + key / c.page_size);
      if (page < 0 || page >= c.num_pages) continue;
      if (C::BS) {  // a block without a scale counts as absent
        const int64_t at = page * c.scale_stride + h;
        if (!good_scale(c.k_scale[at]) || !good_scale(c.v_scale[at])) continue;
      }
      const uint8_t* v = c.v + page * c.page_bytes + (int64_t)(key % c.page_size) * c.token_bytes +
                         h * c.head_bytes;
      for (int d = 0; d < C::D; d++) {
        float x;
        if (C::E8)
          x = (v[d] & 0x7F) == 0x7F ? NAN : 0.0f;
        else
          x = load_act(v, C::BF, d);
        if (isfinite(x)) continue;
        if (part)
          part[d] += x;
        else
          out[d] = (uint16_t)pack2<C::BF>(load_act(out, C::BF, d) + x, 0.0f);
      }
    }
  }
}

__device__ __forceinline__ float row_inverse(float l, float vs) { return l > 0.0f || l != l ? vs / l : 0.0f; }
__device__ __forceinline__ float row_lse(float m, float l, float lift) {
  return l > 0.0f || l != l ? (m + (log2f(l) - lift)) * kLn2 : -INFINITY;
}

// Scores of keys that the row does not see (before l0, after h0, in absent
// pages) to -inf.
__device__ __forceinline__ void mask_scores(float* s, int h0, int l0, uint32_t gm) {
#pragma unroll
  for (int w = 0; w < kTile / 32; w++) {
    const int a = min(max(l0 - 32 * w, 0), 32), b = min(max(h0 + 1 - 32 * w, 0), 32);
    uint32_t seen = a < b ? (0xffffffffu << a) & (0xffffffffu >> (32 - b)) : 0u;
    seen &= ~((gm >> (2 * w) & 1 ? 0x0000ffffu : 0u) | (gm >> (2 * w) & 2 ? 0xffff0000u : 0u));
#pragma unroll
    for (int i = 0; i < 32; i++)
      if (!(seen >> i & 1)) s[32 * w + i] = -INFINITY;
  }
}

// The block scales of 16 keys, twice each for packed arithmetic: of the keys, log2
// of the values' and its inverse.
struct __align__(16) GroupScales {
  float ks[2], lv[2], iv[2], pad[2];
};
// As take_terms, for the four groups of 16 keys from g on, BS of which share a
// factor and an offset, and sums divided by their value scales.
template <int MBF, int BS>
__device__ __forceinline__ void take_block_terms(const float* s, uint32_t* pk, uint64_t& sum,
                                                 uint64_t c, uint64_t n, const GroupScales* g) {
  uint64_t part[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 4; k += BS) {
    const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(g + k);
    const uint64_t iv = *reinterpret_cast<const uint64_t*>(g[k].iv);
    uint64_t ck, nk;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(ck) : "l"(f.x), "l"(c));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(nk) : "l"(f.y), "l"(n));
#pragma unroll
    for (int i = 0; i < 8 * BS; i++) {
      float x = s[16 * k + 2 * i], y = s[16 * k + 2 * i + 1];
      fma2(x, y, ck, nk);
      x = ex2(x);
      y = ex2(y);
      asm("{\n\t.reg .b64 b;\n\tmov.b64 b, {%1, %2};\n\tfma.rn.f32x2 %0, b, %3, %0;\n\t}"
          : "+l"(part[i & 1])
          : "f"(x), "f"(y), "l"(iv));
      pk[8 * k + i] = pack2<MBF>(x, y);
    }
  }
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(part[0]) : "l"(part[1]));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum) : "l"(part[0]));
}

// 64 softmax terms 2^(s c + n), their sum, and their 16-bit pairs.
template <int MBF>
__device__ __forceinline__ void take_terms(const float* s, uint32_t* pk, uint64_t& sum, uint64_t c,
                                           uint64_t n) {
  uint64_t part[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 32; i++) {
    float x = s[2 * i], y = s[2 * i + 1];
    fma2(x, y, c, n);
    x = ex2(x);
    y = ex2(y);
    add2(part[i & 1], x, y);
    pk[i] = pack2<MBF>(x, y);
  }
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(part[0]) : "l"(part[1]));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum) : "l"(part[0]));
}

struct Maps {
  CUtensorMap k, v;
  int box;          // tokens of a box
  int heads_first;  // dimension 1 is the heads (else the tokens of a page)
  CUtensorMap q;    // channels, heads, tokens; boxes of a row tile
  int q_boxes;      // 0: the group does not divide a row tile, no such boxes
};

// ------------------------------------------------------------ main kernel
template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    attn_tiles_kernel(const __grid_constant__ Maps maps, AttnParams p, Plan pl) {
  constexpr int D = C::D;
  // (aligned by its declaration, not by arithmetic, so that operand addresses
  // are known to be uniform; checked below)
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // [kStages] each
  uint64_t* k_empty = k_full + C::kStages;
  uint64_t* v_full = k_empty + C::kStages;
  uint64_t* v_empty = v_full + C::kStages;
  uint64_t* edge_full = v_empty + C::kStages;    // V tiles on their way to the cleaner
  uint64_t* raw_full = edge_full + C::kStages;   // E4M3 tiles: K, V
  uint64_t* raw_empty = raw_full + 2;
  uint64_t* q_full = raw_empty + 2;              // [2] each: row tiles
  uint64_t* q_raw = q_full + 2;                  // queries still in bf16
  uint64_t* q_free = q_raw + 2;
  uint64_t* s_full = q_free + 2;
  uint64_t* o_full = s_full + 2;
  uint64_t* p_full = o_full + 2;                 // [row tile][half]
  uint64_t* u_full = p_full + 4;
  uint64_t* u_empty = u_full + kUnits;
  uint64_t* all_done = u_empty + kUnits;
  volatile uint32_t* gone = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc) + kGone;
  volatile uint32_t* poison = tmem_slot + 1;     // a V tile held an infinity or a NaN
  Rec* recs = reinterpret_cast<Rec*>(smem + C::kOffUnits);
  GroupScales* const ring =  // [kScaleSteps][kTile / 16]
      reinterpret_cast<GroupScales*>(smem + C::kOffScales);

  // (the same in all lanes, known to the compiler as such)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; i++) {
      mbar_init(&k_full[i], C::E8 ? 4 : 1);
      mbar_init(&v_full[i], C::E8 ? 4 : 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&edge_full[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int t = 0; t < 2; t++) {
      mbar_init(&q_full[t], C::kCvtQ ? 4 : 1);
      mbar_init(&q_raw[t], 1);
      mbar_init(&q_free[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&o_full[t], 1);
      mbar_init(&p_full[2 * t], 4);
      mbar_init(&p_full[2 * t + 1], 4);
    }
    for (int i = 0; i < kUnits; i++) {
      mbar_init(&u_full[i], 1);
      // softmax warps, MMA, queries, cleaner or converters
      mbar_init(&u_empty[i], 8 + 1 + 1 + (C::E8 ? 4 : 1));
    }
    mbar_init(all_done, 1);
    if (p.stuck_barrier >= 0 && p.stuck_barrier < C::kBars) {  // a test of the waits
      asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(k_full + p.stuck_barrier))
                   : "memory");
      mbar_init(k_full + p.stuck_barrier, 1 << 16);
    }
    *poison = 0;
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // all 512 columns are this CTA's, so its TMEM addresses are constants
  constexpr uint32_t tmem = 0;
  if (*tmem_slot != 0 || (sbase & 1023)) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  pdl_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_warp<true>(bar, parity, p.status); };
  // the next published part, for a whole warp; live = 0 at the end or on abort
  auto next_rec = [&](uint32_t& n, auto wait) {
    const uint32_t i = n % kUnits;
    if (!wait(&u_full[i], (n / kUnits) & 1)) return Rec{};
    const Rec r = recs[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(&u_empty[i]);
    n++;
    return r;
  };

  if (warp < 8) {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoft));
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return wait_warp<false>(bar, parity, p.status);
    };
    const int t = warp >> 2, q4 = warp & 3;
    const int row = 32 * q4 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const uint32_t s_col = tmem + lane_base + t * kTile;
    const uint32_t o_col = tmem + lane_base + 2 * kTile + t * D;
    uint32_t steps = 0;  // key tiles this row tile has gone through
    uint32_t base = 0;   // key tiles the CTA has loaded before this unit
    uint32_t nrec = 0;   // parts seen
    uint32_t uses = 0;   // those of them with keys for this tile
    bool ok = true;
    // the part before, whose O is written once the next part's first products
    // are under way: its row, statistics, and place in the record ring
    bool owed = false, o_keys = false;
    float o_m = 0.0f, o_l = 0.0f;
    int o_row = 0, o_hi = 0, o_lo = 0;
    auto put_out = [&]() {
      const Rec& r = recs[(nrec - 1) % kUnits];
      if (o_keys) {
        if (!(ok = wait(&o_full[t], (uses - 1) & 1))) return;
        tc_fence_after();
      }
      const bool whole = r.flags & 1, in = row < r.nrows - t * kTile;
      const int tok = o_row / p.group;
      const int64_t at = (int64_t)(r.q0 + tok) * p.heads + r.h * p.group + (o_row - tok * p.group);
      const float vs = C::E8 && !C::BS && p.cache.v_scale ? __ldg(p.cache.v_scale + r.h) : 1.0f;
      const uint64_t inv2 = both(whole ? row_inverse(o_l, vs) : 1.0f);
      const int prt = t * kTile + row;
      float* part = pl.parts + ((size_t)blockIdx.x * 2 + (r.flags >> 1)) * part_floats(D);
      uint16_t* out = p.out + at * D;
#pragma unroll 1
      for (int i = 0; i < D / 32; i++) {
        float o[32];
        uint32_t* orr = reinterpret_cast<uint32_t*>(o);
        __syncwarp();
        if (o_keys) {
          tmem_ld32(o_col + 32 * i, orr);
          tmem_ld32_wait(orr);
        } else {
#pragma unroll
          for (int e = 0; e < 32; e++) o[e] = 0.0f;
        }
        if (!in) continue;
        if (whole) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; e++) {
            mul2(o[2 * e], o[2 * e + 1], inv2);
            w[e] = pack2<C::BF>(o[2 * e], o[2 * e + 1]);
          }
#pragma unroll
          for (int e = 0; e < 16; e += 8)
            stg32(out + 32 * i + 2 * e, w[e], w[e + 1], w[e + 2], w[e + 3], w[e + 4], w[e + 5],
                  w[e + 6], w[e + 7]);
        } else {
          float* dst = part + (size_t)prt * D + 32 * i;
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            stg32(dst + e, orr[e], orr[e + 1], orr[e + 2], orr[e + 3], orr[e + 4], orr[e + 5],
                  orr[e + 6], orr[e + 7]);
        }
      }
      tc_fence_before();  // O is read before the next unit's first product writes it
      if (in) {
        if (*poison != 0)
          add_poison<C>(p.cache, p.batch.table + (int64_t)r.b * p.batch.table_stride, r.h,
                        (r.first + r.s0) * kTile, (r.first + r.s1) * kTile, r.any0, r.any1, r.all0,
                        r.all1, o_lo, o_hi, whole ? nullptr : part + (size_t)prt * D, out);
        if (!whole)
          *reinterpret_cast<float2*>(part + (size_t)kUnitRows * D + 2 * prt) = make_float2(o_m, o_l);
        else if (p.lse)
          p.lse[at] = row_lse(o_m, o_l, C::kLift);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&u_empty[(nrec - 1) % kUnits]);
    };
    while (ok) {
      const uint32_t slot = nrec % kUnits;
      if (!(ok = wait(&u_full[slot], (nrec / kUnits) & 1))) break;
      const Rec r = recs[slot];
      const int nt = min(kTile, r.nrows - t * kTile);  // rows of the tile
      const int j0 = t ? r.t1a : r.t0a, j1 = t ? r.t1e : r.t0e;
      const int prow = min(r.row0 + t * kTile + row, r.row0 + r.nrows - 1);
      const int pos = r.len - r.n + prow / p.group;
      const int hi = p.causal ? pos : r.len - 1;
      const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
      float c = p.scale_log2 *
                (C::E8 && !C::BS && p.cache.k_scale ? __ldg(p.cache.k_scale + r.h) : 1.0f);
      if (C::kCvtQ && r.live && j0 < j1) {
        // bf16 queries to fp16, in place, by a power of two per row: 2^s
        // brings the row's largest value to [2^14, 2^15); values below 2^-31
        // of it lose bits, those below 2^-39 vanish
        if (!(ok = wait(&q_raw[t], uses & 1))) break;
        const uint32_t q = sbase + t * C::kOp;
        float am = 0.0f;
#pragma unroll 8
        for (int i = 0; i < D / 8; i++) {
          const uint4 v = lds16(q + op_off<D>(row, i));
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int y = 0; y < 4; y++)
            am = max3(am, fabsf(__uint_as_float(x[y] << 16)),
                      fabsf(__uint_as_float(x[y] & 0xFFFF0000u)));
        }
        const int sh = fp16_scale_exp(am);
        const float f = exp2f((float)sh);
        c *= exp2f((float)-sh);
#pragma unroll 4
        for (int i = 0; i < D / 8; i++) {
          const uint4 v = lds16(q + op_off<D>(row, i));
          uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int y = 0; y < 4; y++)
            x[y] = pack2<0>(__uint_as_float(x[y] << 16) * f,
                            __uint_as_float(x[y] & 0xFFFF0000u) * f);
          sts16(q + op_off<D>(row, i), x[0], x[1], x[2], x[3]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[t]);
      }
      // a factor that is not positive (a k_scale of 0 or below) would turn the
      // -inf of masked scores: it is applied before the mask then
      const float pre = c;
      const bool odd = C::E8 && !C::BS && __any_sync(0xffffffffu, !(c > 0.0f));
      if (odd) c = 1.0f;
      if (C::BS) c = fmaxf(c, 0x1p-86f);  // (times a scale it stays positive)
      if (owed) {
        put_out();
        if (!ok) break;
      }
      if (!r.live) break;
      nrec++;
      float m = -INFINITY, l = 0.0f;
      for (int j = j0; j < j1; j++, steps++) {
        if (!(ok = wait(&s_full[t], steps & 1))) break;
        tc_fence_after();
        float s[kTile];
        uint32_t* sr = reinterpret_cast<uint32_t*>(s);
#pragma unroll
        for (int i = 0; i < 4; i++) tmem_ld32(s_col + 32 * i, sr + 32 * i);
        const uint32_t gm = gone[(base + j - r.j0) % kGone];
#pragma unroll
        for (int i = 0; i < 4; i++) tmem_ld32_wait(sr + 32 * i);
        const int k0 = (r.first + j) * kTile;
        const int h0 = hi - k0, l0 = lo - k0;
        if (odd) {
          const uint64_t pre2 = both(pre);
#pragma unroll
          for (int i = 0; i < kTile / 2; i++) mul2(s[2 * i], s[2 * i + 1], pre2);
        }
        const bool masked = edge(r, j) || gm;
        if (masked) mask_scores(s, h0, l0, gm);
        const GroupScales* const gs = ring + (base + j - r.j0) % kScaleSteps * (kTile / 16);
        float mn = m;
        if constexpr (C::BS) {
#pragma unroll
          for (int g = 0; g < kTile / 16; g += C::BS) {
            const float4 f = *reinterpret_cast<const float4*>(gs + g);
            const float* t = s + 16 * g;
            constexpr int N = 16 * C::BS;
            float mx[2] = {t[0], t[1]};
#pragma unroll
            for (int i = 2; i + 4 <= N; i += 4)
#pragma unroll
              for (int e = 0; e < 2; e++) mx[e] = max3(mx[e], t[i + 2 * e], t[i + 2 * e + 1]);
            const float x = max3(fmaxf(mx[0], mx[1]), t[N - 2], t[N - 1]);
            mn = fmaxf(mn, fmaf(x, c * f.x, f.z));
          }
        } else {
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 4; i + 8 <= kTile; i += 8)
#pragma unroll
            for (int e = 0; e < 4; e++) mx[e] = max3(mx[e], s[i + 2 * e], s[i + 2 * e + 1]);
#pragma unroll
          for (int e = 0; e < 4; e++) mx[e] = fmaxf(mx[e], s[kTile - 4 + e]);
          mn = fmaxf(m, max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * c);
        }
        const bool grow = mn > m + kRescale || (m == -INFINITY && mn > m);
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2(m - mn) : 1.0f;
          if (grow) m = mn;
          l *= f;
          if (j > j0) {
            // (the scores of this tile are complete, so the product before
            // them, the last that added to O, is too)
            const uint64_t f2 = both(f);
#pragma unroll 1
            for (int i = 0; i < D / 16; i++) {
              float o[16];
              tmem_ld16(o_col + 16 * i, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int e = 0; e < 8; e++) mul2(o[2 * e], o[2 * e + 1], f2);
              tmem_st16(o_col + 16 * i, o);
            }
          }
        }
        uint32_t pk[32];
        uint64_t sum = 0;
        const uint64_t c2 = both(c), n2 = both(C::kLift - (m == -INFINITY ? 0.0f : m));
        if constexpr (C::BS > 0)
          take_block_terms<C::MBF, C::BS>(s, pk, sum, c2, n2, gs);
        else
          take_terms<C::MBF>(s, pk, sum, c2, n2);
        auto hand_over = [&](int half) {
          tmem_st32(s_col + 32 * half, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * t + half]);
        };
        hand_over(0);
        if constexpr (C::BS > 0)
          take_block_terms<C::MBF, C::BS>(s + 64, pk, sum, c2, n2, gs + 4);
        else
          take_terms<C::MBF>(s + 64, pk, sum, c2, n2);
        l += sum2(sum);
        hand_over(1);
      }
      if (!ok) break;
      base += r.j1 - r.j0;
      owed = true;
      o_keys = j0 < j1;
      uses += o_keys;
      o_m = m;
      o_l = l;
      o_row = prow;
      o_hi = hi;
      o_lo = lo;
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------------ MMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    // (no call in this role: a call would cost the operands their uniform
    // registers)
    uint32_t looks = p.wait_looks;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return wait_uniform(smem_u32(bar), parity, looks);
    };
    constexpr uint32_t bf = C::MBF ? (1u << 7) | (1u << 10) : 0u;
    const uint32_t id_qk = umma_idesc_f16(kTile, kTile, 0, 0) | bf;
    const uint32_t id_pv = umma_idesc_f16(kTile, D, 0, 1) | bf;
    uint32_t nq = 0, np = 0;        // bit t: parity of row tile t's next queries, P
    uint32_t n = 0, nrec = 0;       // steps so far: K and V of step n are in stage n % kStages
    bool ok = true;
    const uint64_t qd0 = umma_desc(sbase, 16, 1024);
    auto uni = [](uint32_t x) { return __reduce_max_sync(0xffffffffu, x); };
    const uint32_t q_lo = (uint32_t)qd0;
    const uint32_t k_lo = q_lo + (C::kOffK >> 4);
    // V: rows of 128 bytes hold 64 channels of one key; 8 keys 1024 B, the
    // second 64 channels kTile * 128 B on
    const uint32_t v_lo = (uint32_t)umma_desc(sbase + C::kOffV, kTile * 128, 1024);
    auto wait_kv = [&](uint64_t* full, uint32_t i) {
      return wait(&full[i % C::kStages], (i >> C::kStageBits) & 1);
    };
    // Step by step: the scores of key tile j (S) and the product with the
    // values of the tile before (V).  A unit's last product goes with the next
    // unit's first scores.
    int t0a = 0, t0e = 0, t1a = 0, t1e = 0;
    int j = 0, j1 = 0;              // the unit's steps to come
    uint32_t due = 0;               // bit t: row tile t's product is due,
    uint32_t add = 0, last = 0;     // adds to O, is its unit's last
    bool v_due = false, end = false;
    while (ok) {
      if (j >= j1 && !end) {
        const uint32_t slot = nrec % kUnits;
        ok = wait(&u_full[slot], (nrec / kUnits) & 1);
        const Rec& r = recs[slot];
        end = !ok || !uni(r.live);
        j = end ? 0 : uni(r.j0);
        j1 = end ? 0 : uni(r.j1);
        t0a = uni(r.t0a);
        t0e = uni(r.t0e);
        t1a = uni(r.t1a);
        t1e = uni(r.t1e);
        __syncwarp();
        if (lane == 0) mbar_arrive(&u_empty[slot]);
        __syncwarp();
        nrec++;
        if (j < j1) ok = wait_kv(k_full, n);
      }
      const bool has_k = j < j1;
      if (!has_k && !v_due) {
        if (end) break;
        continue;
      }
      // The run of steps in the middle of a unit, written out: both row tiles
      // take part in all of it.  (This warp's instructions, not the products,
      // are what a step takes the longest for.)
      const int mid = min(t0e, t1e) - 1;
      if (j >= max(t0a, t1a) + 2 && j < mid) {
#pragma unroll 1
        for (; ok && j < mid; j++) {
          const uint32_t kd = k_lo + n % C::kStages * (C::kOp >> 4);
          const uint32_t vd = v_lo + (n - 1) % C::kStages * (C::kOp >> 4);
          const uint32_t np0 = np & 1, np1 = np >> 1;
          auto scores = [&](int t, int y) {
            umma_ss4(t * kTile, q_lo + t * (C::kOp >> 4) + y * (kTile * 128 >> 4),
                     kd + y * (kTile * 128 >> 4), id_qk, y > 0);
          };
          auto values = [&](int t, int half) {
            umma_ts4(2 * kTile + t * D, t * kTile + 32 * half, vd + half * (4 * 2048 >> 4), id_pv, 1);
          };
          ok &= wait_kv(v_full, n - 1);
          ok &= wait(&p_full[0], np0);
          tc_fence_after();
          values(0, 0);
          ok &= wait(&p_full[1], np0);
          tc_fence_after();
          values(0, 1);
          ok &= wait_kv(k_full, n);
#pragma unroll
          for (int y = 0; y < D / 64; y++) scores(0, y);
          commit(&s_full[0]);
          ok &= wait(&p_full[2], np1);
          tc_fence_after();
          values(1, 0);
          ok &= wait(&p_full[3], np1);
          tc_fence_after();
          values(1, 1);
          commit(&v_empty[(n - 1) % C::kStages]);
#pragma unroll
          for (int y = 0; y < D / 64; y++) scores(1, y);
          commit(&s_full[1]);
          commit(&k_empty[n % C::kStages]);
          np ^= 3;
          n++;
        }
        ok = ok && wait_kv(v_full, n - 1) && wait_kv(k_full, n);
        if (!ok) break;
      }
      const uint32_t now = (has_k && j >= t0a && j < t0e ? 1u : 0u) |
                           (has_k && j >= t1a && j < t1e ? 2u : 0u);
      const uint32_t vd = v_lo + (n - 1) % C::kStages * (C::kOp >> 4);
      const uint32_t kd = k_lo + n % C::kStages * (C::kOp >> 4);
      // The issue of MMAs blocks while the tensor core is busy and leaves it a
      // few MMAs ahead at most: the next step's waits go between MMAs.
      auto wait_next = [&]() {
        if (has_k) ok = ok && wait_kv(v_full, n) && (j + 1 >= j1 || wait_kv(k_full, n + 1));
      };
      // (scores overwrite P, so they go after its product)
#pragma unroll 1
      for (int x = 0; x < 4; x++) {
        const int t = x >> 1;
        if (!(x & 1)) {
          if (due >> t & 1) {
            // O += P V; P comes in two halves of the keys
            uint32_t acc = add >> t & 1;
            const uint32_t o = 2 * kTile + t * D;
#pragma unroll 1
            for (int half = 0; half < 2; half++) {
              const uint32_t pa = t * kTile + 32 * half;
              const uint32_t v = vd + half * (4 * 2048 >> 4);
              ok &= wait(&p_full[2 * t + half], np >> t & 1);
              tc_fence_after();
              umma_ts4(o, pa, v, id_pv, acc);
              acc = 1;
            }
            np ^= 1u << t;
            if (last >> t & 1) commit(&o_full[t]);
          }
          if (t == 1 && v_due) commit(&v_empty[(n - 1) % C::kStages]);
        } else if (now >> t & 1) {
          if (j == (t ? t1a : t0a)) {
            ok &= wait(&q_full[t], nq >> t & 1);
            nq ^= 1u << t;
          }
          // S = Q K^T, 64 channels at a time
          tc_fence_after();
#pragma unroll 1
          for (int y = 0; y < D / 64; y++) {
            const uint32_t off = y * (kTile * 128 >> 4);
            const uint32_t qd = q_lo + t * (C::kOp >> 4) + off, kx = kd + off;
            const uint32_t sc = t * kTile;
            umma_ss4(sc, qd, kx, id_qk, y > 0);
            if (y == 0 && t == 1) wait_next();
          }
          commit(&s_full[t]);
          if (j == (t ? t1e : t0e) - 1) commit(&q_free[t]);
        } else if (t == 1) {
          wait_next();
        }
      }
      add = (j > t0a ? 1u : 0u) | (j > t1a ? 2u : 0u);
      last = (j == t0e - 1 ? 1u : 0u) | (j == t1e - 1 ? 2u : 0u);
      due = now;
      v_due = has_k;
      if (has_k) {
        commit(&k_empty[n % C::kStages]);
        n++;
        j++;
      }
    }
    if (looks != p.wait_looks && lane == 0) atomicOr(p.status, kStatusTimeout);
    commit(all_done);
  } else if (warp == 9) {
    // ------------------------------------------------------------ work, TMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    constexpr int HALF = C::E8 ? 1 : D / 64;      // boxes across the channels
    constexpr uint32_t BYTES = C::E8 ? C::kRaw : C::kOp;
    const int nbox = kTile / maps.box;
    const int bx = lane / HALF, half = lane % HALF;
    const bool mine = bx < nbox;
    const int ps = p.cache.page_size, ps_shift = p.cache.page_shift;
    uint32_t n = 0, nrec = 0;            // steps so far
    uint32_t to_edge = 0, edge_par = 0;  // per V stage: its last load went to the cleaner; its parity
    int32_t bad = 0;
    bool ok = true;
    Walk w(p, pl);
    while (ok) {
      const Rec r = w.next();
      const uint32_t slot = nrec % kUnits;
      if (!(ok = wait(&u_empty[slot], ((nrec / kUnits) & 1) ^ 1))) break;
      if (lane == 0) {
        recs[slot] = r;
        mbar_arrive(&u_full[slot]);
      }
      __syncwarp();
      nrec++;
      if (!r.live) break;
      const int32_t* table = p.batch.table + (int64_t)r.b * p.batch.table_stride;
      // page of this lane's box of key tile j; num_pages, out of range, reads zeros
      auto page_of = [&](int j) {
        const int key = (r.first + j) * kTile + bx * maps.box;
        if (!mine || j >= r.j1 || key >= r.any1 || key + maps.box <= r.any0) return p.cache.num_pages;
        return __ldg(table + (ps_shift >= 0 ? key >> ps_shift : key / ps));
      };
      // block scales of a page (none where there is no page: 0)
      auto scales_of = [&](int id) {
        float2 x = make_float2(0.0f, 0.0f);
        if (C::BS && (unsigned)id < (unsigned)p.cache.num_pages) {
          x.x = __ldg(p.cache.k_scale + id * p.cache.scale_stride + r.h);
          x.y = __ldg(p.cache.v_scale + id * p.cache.scale_stride + r.h);
        }
        return x;
      };
      int nxt = page_of(r.j0), nxt2 = C::BS ? page_of(r.j0 + 1) : 0;
      float2 snxt = scales_of(nxt);
      for (int j = r.j0; ok && j < r.j1; j++) {
        const int key = (r.first + j) * kTile + bx * maps.box;
        int id = nxt;
        float2 sc = snxt;
        bool no_scale = false;
        if (C::BS) {
          nxt = nxt2;
          snxt = scales_of(nxt);
          nxt2 = page_of(j + 2);
          if (!good_scale(sc.x) || !good_scale(sc.y)) {
            // (such a page is one that is needed: its keys count as absent)
            no_scale = true;
            bad |= kStatusBadScale;
            sc = make_float2(0.0f, 0.0f);
            id = -1;
          }
        } else {
          nxt = page_of(j + 1);
        }
        const bool absent = (unsigned)id > (unsigned)p.cache.num_pages ||
                            (id == p.cache.num_pages && mine && key < r.any1 &&
                             key + maps.box > r.any0);
        const int page = absent ? p.cache.num_pages : id;
        // 16-key groups of absent pages
        uint32_t g = absent ? ((1u << (maps.box / 16)) - 1) << (bx * (maps.box / 16)) : 0u;
        g = __reduce_or_sync(0xffffffffu, g);
        if (absent && !no_scale) bad |= kStatusBadPage;
        const int at = ps_shift >= 0 ? key & (ps - 1) : key % ps;
        const uint32_t st = n % C::kStages, par = (n >> C::kStageBits) & 1;
        if (C::BS) {
          // 16-key group `lane`, from the lane of its box (before the waits: nothing
          // stands between a free stage and its load.  The entry's last readers are
          // kScaleSteps steps back.)
          const int from = lane * 16 / maps.box;
          const float k = fmaxf(__shfl_sync(0xffffffffu, sc.x, from), kLeastScale);
          const float v = fmaxf(__shfl_sync(0xffffffffu, sc.y, from), kLeastScale);
          float l, i;
          asm("lg2.approx.f32 %0, %1;" : "=f"(l) : "f"(v));
          asm("rcp.approx.f32 %0, %1;" : "=f"(i) : "f"(v));
          if (lane < kTile / 16) {
            GroupScales* at = ring + n % kScaleSteps * (kTile / 16) + lane;
            *reinterpret_cast<float4*>(at->ks) = make_float4(k, k, l, l);
            *reinterpret_cast<float2*>(at->iv) = make_float2(i, i);
          }
        }
        if (C::BS) __syncwarp();
#pragma unroll 1
        for (int x = 0; x < 2; x++) {  // K, V
          uint64_t* const full = C::E8 ? &raw_full[x] : x ? &v_full[st] : &k_full[st];
          uint64_t* const empty = C::E8 ? &raw_empty[x] : x ? &v_empty[st] : &k_empty[st];
          if (!(ok = wait(empty, (C::E8 ? n & 1 : par) ^ 1))) break;
          uint64_t* bar = full;
          if (!C::E8 && x == 1) {
            to_edge &= ~(1u << st);
            if (edge(r, j)) {
              bar = &edge_full[st];
              to_edge |= 1u << st;
              edge_par ^= 1u << st;
            }
          }
          if (lane == 0) {
            if (x == 0) gone[n % kGone] = g;
            mbar_arrive_expect_tx(bar, BYTES);
          }
          __syncwarp();
          if (mine) {
            const uint32_t stage = sbase + (C::E8 ? C::kOffRaw + x * C::kRaw
                                                 : (x ? C::kOffV : C::kOffK) + st * C::kOp);
            const uint32_t dst = stage + half * (kTile * 128) + bx * maps.box * (C::E8 ? D : 128);
            const CUtensorMap* m = x == 0 ? &maps.k : &maps.v;
            if (maps.heads_first)
              tma_load_4d(dst, m, half * 64, r.h, at, page, bar);
            else
              tma_load_4d(dst, m, half * 64, at, r.h, page, bar);
          }
        }
        if (!ok) break;
        n++;
      }
    }
    bad = (int32_t)__reduce_or_sync(0xffffffffu, (uint32_t)bad);
    if (bad && lane == 0) atomicOr(p.status, bad);
    // every box this warp requested has landed before the CTA may exit (after
    // a wait that ran out, a step's K may be under way without its V)
    constexpr uint32_t kBack = C::E8 ? 1 : C::kStages;
#pragma unroll 1
    for (uint32_t i = n < kBack ? 0 : n - kBack; i < n + (ok ? 0 : 1); i++) {
      const uint32_t st = i % C::kStages, par = (i >> C::kStageBits) & 1;
      const long long budget = i < n ? p.wait_budget : 100000;
      mbar_drain(C::E8 ? &raw_full[0] : &k_full[st], C::E8 ? i & 1 : par, budget);
      if (i == n) break;
      const bool e = to_edge >> st & 1;
      mbar_drain(C::E8 ? &raw_full[1] : e ? &edge_full[st] : &v_full[st],
                 C::E8 ? i & 1 : e ? (edge_par >> st & 1) ^ 1 : par, budget);
    }
  } else if (warp == 11) {
    // -------------------------------------------------------------- queries
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    uint32_t nrec = 0, n[2] = {0, 0};
    bool ok = true;
    while (ok) {
      const Rec r = next_rec(nrec, wait);
      if (!r.live) break;
#pragma unroll
      for (int t = 0; t < 2; t++) {
        if (!ok || (t ? r.t1e <= r.t1a : r.t0e <= r.t0a)) continue;
        const int nt = min(kTile, r.nrows - t * kTile);
        // the last product that reads this tile's previous queries is done
        if (n[t] > 0 && !(ok = wait(&q_free[t], (n[t] - 1) & 1))) continue;
        const uint32_t dst = sbase + t * C::kOp;
        uint64_t* const bar = C::kCvtQ ? &q_raw[t] : &q_full[t];
        if (maps.q_boxes) {
          // rows past the sequence's end are other tokens' (or zeros): they
          // are computed and dropped
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, C::kOp);
            const int tok = r.q0 + (r.row0 + t * kTile) / p.group;
#pragma unroll
            for (int x = 0; x < D / 64; x++)
              tma_load_3d(dst + x * (kTile * 128), &maps.q, 64 * x, r.h * p.group, tok, bar);
          }
          __syncwarp();
        } else {
          constexpr int LR = D / 8, RI = 32 / LR;  // lanes of a row, rows at a time
          const int ch = lane % LR;
          int row = lane / LR;
          const int first = r.row0 + t * kTile + row;
          int tok = first / p.group, hd = first - tok * p.group;
          const uint16_t* q = p.q + (int64_t)(r.q0 + tok) * p.q_ts +
                              (int64_t)(r.h * p.group + hd) * p.q_hs + ch * 8;
          const int64_t wrap = p.q_ts - p.group * p.q_hs;
#pragma unroll 4
          for (; row < kTile; row += RI) {
            cp_async16(dst + op_off<D>(row, ch), row < nt ? q : p.q, row < nt ? 16 : 0);
            q += RI * p.q_hs;
            hd += RI;
            while (hd >= p.group) {
              hd -= p.group;
              q += wrap;
            }
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar);
        }
        n[t]++;
      }
    }
    // the last queries requested have landed before the CTA may exit
    if (maps.q_boxes) {
#pragma unroll
      for (int t = 0; t < 2; t++)
        if (n[t] > 0)
          mbar_drain(C::kCvtQ ? &q_raw[t] : &q_full[t], (n[t] - 1) & 1, p.wait_budget);
    }
  } else if (warp == 10) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    if constexpr (!C::E8) {
      // ---------------------------------------------------- clean V tiles
      uint32_t nrec = 0, n = 0, par = 0;
      bool ok = true;
      while (ok) {
        const Rec r = next_rec(nrec, wait);
        if (!r.live) break;
        for (int j = r.j0; ok && j < r.j1; j++, n++) {
          if (!edge(r, j)) continue;
          const uint32_t st = n % C::kStages;
          if (!(ok = wait(&edge_full[st], par >> st & 1))) break;
          par ^= 1u << st;
          // keys that every row sees need no look
          const int k0 = (r.first + j) * kTile;
          int m0, m1;
          seen_by_all(r, k0, &m0, &m1);
          bool hit = false;
#pragma unroll 1
          for (int x = 0; x < 2; x++)
            hit |= clean_v<C>(sbase + C::kOffV + st * C::kOp, x ? m1 : 0, x ? kTile : m0,
                              r.any0 - k0, r.any1 - k0, lane);
          if (__any_sync(0xffffffffu, hit) && lane == 0) *poison = 1;
          __threadfence_block();
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_full[st]);
        }
      }
    }
  } else if constexpr (C::E8) {
    // -------------------------------------------------- widen E4M3 to fp16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    const int tid = threadIdx.x - 12 * 32;
    uint32_t n = 0, nrec = 0;
    bool ok = true;
    while (ok) {
      const Rec rc = next_rec(nrec, wait);
      if (!rc.live) break;
      for (int j = rc.j0; ok && j < rc.j1; j++, n++) {
        const int k0 = (rc.first + j) * kTile;
        const int r0 = rc.any0 - k0, r1 = rc.any1 - k0;
        for (int x = 0; x < 2; x++) {
          const uint32_t st = n % C::kStages;
          uint64_t* const full = x ? &v_full[st] : &k_full[st];
          if (!(ok = wait(&raw_full[x], n & 1) &&
                     wait(x ? &v_empty[st] : &k_empty[st], ((n >> C::kStageBits) & 1) ^ 1)))
            break;
          const uint32_t src = sbase + C::kOffRaw + x * C::kRaw;
          const uint32_t dst = sbase + (x ? C::kOffV : C::kOffK) + st * C::kOp;
          const bool clean = x == 1 && edge(rc, j);
          int m0, m1;
          seen_by_all(rc, k0, &m0, &m1);
          bool hit = false;
          // 8 lanes take 4 chunks of a row and 4 of the next one, of the other
          // half of the channels where there are two, so that their loads and
          // their stores cover all banks
          constexpr int HALVES = D / 64, UN = 2;
          const int r8 = 2 * (tid >> 3) + (tid >> 2 & 1);
#pragma unroll 1
          for (int i0 = 0; i0 < 4 * HALVES; i0 += UN) {
            uint4 v[UN];
#pragma unroll
            for (int k = 0; k < UN; k++) {
              const int r = r8 + 32 * ((i0 + k) / HALVES);
              const int ch = (tid & 3) + (HALVES == 2 ? 4 * ((r ^ k) & 1) : 0);
              v[k] = lds16(src + r * D + ch * 16);
            }
#pragma unroll
            for (int k = 0; k < UN; k++) {
              const int r = r8 + 32 * ((i0 + k) / HALVES);
              const int ch = (tid & 3) + (HALVES == 2 ? 4 * ((r ^ k) & 1) : 0);
              if (clean) {
                if (r < r0 || r >= r1) v[k] = make_uint4(0, 0, 0, 0);
                const uint32_t some = r < m0 || r >= m1 ? 0xffffffffu : 0u;
                const uint32_t f0 = not_finite<C>(v[k].x) & some, f1 = not_finite<C>(v[k].y) & some,
                               f2 = not_finite<C>(v[k].z) & some, f3 = not_finite<C>(v[k].w) & some;
                hit |= (f0 | f1 | f2 | f3) != 0;
                v[k] = make_uint4(v[k].x & ~whole_mask<C>(f0), v[k].y & ~whole_mask<C>(f1),
                                  v[k].z & ~whole_mask<C>(f2), v[k].w & ~whole_mask<C>(f3));
              }
              sts16(dst + op_off<D>(r, 2 * ch), e4m3_to_f16x2(v[k].x), e4m3_to_f16x2(v[k].x >> 16),
                    e4m3_to_f16x2(v[k].y), e4m3_to_f16x2(v[k].y >> 16));
              sts16(dst + op_off<D>(r, 2 * ch + 1), e4m3_to_f16x2(v[k].z),
                    e4m3_to_f16x2(v[k].z >> 16), e4m3_to_f16x2(v[k].w), e4m3_to_f16x2(v[k].w >> 16));
            }
          }
          if (hit) *poison = 1;
          __threadfence_block();
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&raw_empty[x]);
            mbar_arrive(full);
          }
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    mbar_drain(all_done, 0, p.wait_budget);
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Sums the parts of the units that cuts go through, 256 / (head_dim / 4) rows
// of a unit at a time.
constexpr int kJoinBlocks = 8 * kSms;
template <class C>
__global__ void __launch_bounds__(256) attn_tiles_join_kernel(AttnParams p, Plan pl) {
  constexpr int D = C::D, LR = D / 4, kRows = 256 / LR;
  pdl_wait();
  const int splits = pl.head->splits, groups = (pl.head->split_rows + kRows - 1) / kRows;
  const int d0 = (threadIdx.x % LR) * 4;
  for (int i = blockIdx.x; i < splits * groups; i += gridDim.x) {
    const Split u = pl.split[i % splits];
    const int r = i / splits * kRows + threadIdx.x / LR;
    if (r >= u.nrows) continue;
    const float vs = C::E8 && !C::BS && p.cache.v_scale ? __ldg(p.cache.v_scale + u.head) : 1.0f;
    float mm = -INFINITY, ll = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int c = u.first; c <= u.last; c++) {
      const float* part = pl.parts + (size_t)(c == u.first ? u.slot0 : 2 * c) * part_floats(D);
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
    const int token = u.q0 + prow / p.group, head = u.head * p.group + prow % p.group;
    const float inv = row_inverse(ll, vs);
    uint2 o;
    o.x = pack2<C::BF>(acc[0] * inv, acc[1] * inv);
    o.y = pack2<C::BF>(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2*>(p.out + ((int64_t)token * p.heads + head) * D + d0) = o;
    if (p.lse && d0 == 0) p.lse[(int64_t)token * p.heads + head] = row_lse(mm, ll, C::kLift);
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
  // queries: a row tile is a box of group heads x 128 / group tokens, where
  // the group divides it
  m->q_boxes = 0;
  if (kTile % p.group == 0) {
    const int64_t qh = p.heads > 1 ? p.q_hs * 2 : (int64_t)p.dim * 2;
    const int64_t qt = p.batch.T > 1 ? p.q_ts * 2 : (int64_t)p.dim * 2;
    const cuuint64_t qdims[3] = {(cuuint64_t)p.dim, (cuuint64_t)p.heads, (cuuint64_t)p.batch.T};
    const cuuint64_t qstr[2] = {(cuuint64_t)qh, (cuuint64_t)qt};
    const cuuint32_t qbox[3] = {64u, (cuuint32_t)p.group, (cuuint32_t)(kTile / p.group)};
    m->q_boxes = fn(&m->q, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<uint16_t*>(p.q), qdims,
                    qstr, qbox, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  return true;
}

template <class C>
cudaError_t launch_cfg(const AttnParams& p, const Maps& maps, const Plan& pl, int max_unit,
                       cudaStream_t st) {
  static_assert(C::kSmem <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(attn_tiles_kernel<C>, C::kSmem, &done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, p, pl, max_unit);
  note_launches(1);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_tiles_kernel<C>, dim3(kGrid), dim3(C::kThreads), C::kSmem, st, maps, p, pl);
  note_launches(1);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_tiles_join_kernel<C>, dim3(kJoinBlocks), dim3(256), 0, st, p, pl);
  note_launches(1);
  return e;
}

template <int D>
cudaError_t launch_types(const AttnParams& p, const Maps& m, const Plan& pl, int mu,
                         cudaStream_t st) {
  if (p.blocks && m.box >= 64)  // a box, and so 64 keys, in one block
    return p.bf16 ? launch_cfg<Cfg<D, 1, 1, 4>>(p, m, pl, mu, st)
                  : launch_cfg<Cfg<D, 1, 0, 4>>(p, m, pl, mu, st);
  if (p.blocks)
    return p.bf16 ? launch_cfg<Cfg<D, 1, 1, 1>>(p, m, pl, mu, st)
                  : launch_cfg<Cfg<D, 1, 0, 1>>(p, m, pl, mu, st);
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
