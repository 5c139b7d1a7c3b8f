// Conditioning attention on the sm_100a tensor cores (tcgen05 + TMEM + TMA).
//
//   O = softmax(Q K^T * scale) V over the keys of up to two segments (prefix,
//   own keys), each of its own length, with lengths, packed sets and key
//   masks read on the device.
//
// What bounds it.  The keys of a text prompt are few, so an item is short: at
// head dim 72 a 128 x 80 step is about 400 cycles of tensor work (S with
// both operands in shared memory, PV with P in TMEM) against 640 cycles of
// special-function unit for its exponentials, of which a quarter go to the FMA
// pipe, and below about 190 keys reading Q and writing O takes longer than
// either.  The chain S -> softmax -> PV -> S of one tile leaves every unit idle
// most of the time, so several row tiles run side by side, each with its own
// chain; what is left is the latency of the hand-overs between them (tensor
// pipe 32%, special-function unit 39% busy at 320 keys).  Second comes the
// instruction cache: all roles together are 60 to 85 KB of code, and every
// variant that shortened them got faster (16 heads x 72, 65,536 rows, 320 keys:
// 176 us at 84 KB, 161 us at 71 KB, where it still is).
//
// Design (one persistent CTA per SM, warp-specialised):
//   * A work item is up to NT tiles of 128 rows of one (unit, head): three for
//     head dims up to 96, whose S (64 to 96 keys) and O fit three times into
//     the 512 TMEM columns, two (128 keys per step) for 128.
//   * Each tile has one issuer warp; S(j + 1) follows PV(j) in program order
//     into the same TMEM columns (MMAs of one thread execute in order), so the
//     chain has two hand-overs a step: S ready, P ready.  One issuer for all
//     tiles was bound by its own instructions (60 cycles an MMA).
//   * The softmax warps (one thread per row) also divide O by the row sum and
//     write it out: through the item's own Q tile, dead by then, with bulk tensor
//     stores, or row by row (fp32 results, partials, heads packed into rows).
//     Warps of their own for this were slower by 5% (more code, a hand-over).
//   * The running maximum is raised (and O rescaled in TMEM) only when it grows
//     by more than 2^8.
//   * When every key tile of a launch fits the K/V stages, a CTA walks
//     consecutive items and keeps K and V in shared memory until the set or the
//     head changes; otherwise they stream through the stages (65,536 rows, 16
//     heads x 72, 300 keys: 165 us kept, 200 us streamed through three stages).
//   * Split keys and one row tile (a token per sample): the tiles of a CTA take
//     the same rows and every NT-th step, one part each, so that NT chains run
//     (64 samples of one token, 16 heads x 72, 16,384 shared keys: 93 us with one
//     chain, 62 us with three; the combine kernel's share is in both).
//   * V helpers clear the rows of keys that do not count (which may hold NaN:
//     0 * NaN would reach O) and, where the head dim is padded, set column D to 1
//     so that PV adds up the rounded weights.
//   * Every wait is bounded; a wait that runs out sets an error word and an
//     abort epoch, in-flight copies are drained, TMEM is freed.
//
// Measured (device time of short runs at 1.9 GHz, 65,536 rows, 16 heads; the spatial
// kernel of this library beside it needs 213 us for 256 keys of 72 channels; under
// the power cap, at 1.7 to 1.85 GHz, the long ones take 5 to 15% more):
//   72 channels:  64 keys 87 us, 128 107 us, 320 160 us (604 TF/s), 1024 480 us
//                 (644 TF/s), 4096 1631 us (758 TF/s)
//   128 channels: 64 keys 137 us, 128 129 us, 320 290 us (592 TF/s), 1024 560 us
//                 (981 TF/s), 4096 1928 us (1140 TF/s)
#include <cuda.h>
#include <math.h>
#include <string.h>

#include <atomic>
#include <mutex>
#include <type_traits>

#include "cond.cuh"

namespace {

using st::Geom;
using st::pdl_trigger;
using st::pdl_wait;

__device__ unsigned int g_cond_error;        // bit of each role whose wait ran out first
__device__ unsigned int g_cond_abort_epoch;  // launch epoch that must abort

constexpr int BLOCK_M = 128;
constexpr unsigned long long WAIT_NS = 2000000000ull;  // a drain's limit: 2 s
constexpr uint32_t WAIT_CLOCKS = 3800000000u;          // a wait's: 2 s at 1.9 GHz
constexpr float NO_KEY = -3.0e38f;           // running max of a row no key counted for yet

template <int D, bool MIX = false> struct Cfg {
  static constexpr int NT = D <= 96 ? 3 : 2;           // row tiles in flight
  static constexpr int BN = D <= 64 ? 96 : (D <= 80 ? 80 : (D <= 96 ? 64 : 128));   // keys per step
  static constexpr int CH = BN / 16;                   // chunks of 16 keys (a K slice of PV)
  static constexpr int C0 = D >= 64 ? 64 : 32;
  static constexpr int R1 = D > 64 ? D - 64 : 0;
  static constexpr int C1 = R1 == 0 ? 0 : (R1 <= 16 ? 16 : (R1 <= 32 ? 32 : 64));
  static constexpr int C1X = C1 ? C1 : 16;
  static constexpr int SW0 = C0 * 2, SW1 = C1 * 2, SW1X = C1X * 2;
  static constexpr int QT0 = BLOCK_M * SW0;
  static constexpr int QTILE = QT0 + BLOCK_M * SW1;
  static constexpr int KT0 = BN * SW0;
  static constexpr int KBYTES = KT0 + BN * SW1, KTILE = (KBYTES + 1023) / 1024 * 1024;   // a 128B swizzle starts at 1 KB
  // V as VA column atoms of VW elements (MN-major), PV one MMA of N = DPV per 16
  // keys.  MIX (spread items of 72 to 96 channels, whose V is read by one tile
  // only and so bound by the rows of its boxes): an atom of 64 and one of VR, two
  // MMAs.  (16,384 keys, 64 rows, 16 heads x 72: 35 us so, 42 us in atoms of 16;
  // 65,536 rows, 4096 keys: 1669 us so, 1607 us in atoms of 16.)
  static constexpr int VW = MIX ? 64 : (D == 72 || D == 80) ? 16 : ((D == 96 || D == 32) ? 32 : 64);
  static constexpr int VA = MIX ? 1 : (D + VW - 1) / VW, NV0 = VA * VW;
  static constexpr int VR = MIX ? (D - 64 + 15) / 16 * 16 : 0, VRX = VR ? VR : 16, DPV = NV0 + VR;
  static constexpr int VSW = VW * 2, VAT = BN * VSW, VSWR = VRX * 2, VT0 = VA * VAT;
  static constexpr int VBYTES = VT0 + BN * VR * 2, VTILE = MIX ? (VBYTES + 1023) / 1024 * 1024 : VBYTES;
  static_assert(QTILE % 1024 == 0 && VT0 % (8 * VSW) == 0, "swizzle atoms");
  // where column D of a row lies: the ones
  static constexpr int ONE_AT = MIX ? VT0 : D / VW * VAT, ONE_SW = MIX ? VSWR : VSW, ONE_X = (D - (MIX ? 64 : D / VW * VW)) * 2;
  static constexpr bool ONES = DPV > D;
  static constexpr int TW = BN + DPV;                  // TMEM columns of a tile: S (P over it), O
  static_assert(NT * TW <= 512, "TMEM");
  // Q tiles: two items' worth, used in turn.  An item's O is staged over its Q
  // (dead by then) and stored from there, while the next item's Q is already in
  // the others: rows of 144 and 160 bytes as they are (16-byte stores of 8
  // lanes then meet at most 2 to a bank), the other widths in the layout of Q.
  // At head dim 128 one of the four gives way to a fourth K/V tile where the
  // keys take more than one step (TIGHT): row tile 1 then runs a step behind
  // row tile 0, in whose place its next Q goes, and stays there, which keeps the
  // two chains out of step.  (TF/s over 4096 and 300 keys: 1078 and 522 so; 2 K and
  // 1 V 955 and 532; K and V in turn in three tiles 874 and 556; O staged apart
  // from one Q tile each, the chains in step, 886 and 528, with row tile 1 held
  // back by 2 steps 924 and 505.  With a barrier per Q slot the kept form is at 1140
  // and 544.)
  static constexpr int NQ = 2 * NT;
  static constexpr bool TIGHT = D == 128;
  static constexpr bool DENSE = D == 72 || D == 80;
  static_assert(!DENSE || BLOCK_M * 2 * D <= QTILE, "O over Q");
  static constexpr int TABLE = D == 128 ? 32 : 64;     // key ranges of a segment held in shared memory
  static constexpr int TAIL = 2 * TABLE * 8 + 384 + 512;    // key ranges, items, barriers and the TMEM slot
  // K and V stages: as many of both as fit behind the Q tiles, at most NB.  Of
  // the items of a spread launch (below) only one is in flight: NT Q tiles, and
  // more stages.  The barriers of a step are counted apart from its stage, NB of
  // them: a multiple of NT, so that with the steps dealt out to the tiles a
  // barrier belongs to one tile, which sees every phase of it.
  static constexpr int NB = TIGHT ? 2 : 6;
  static constexpr int SMEM = 232448, ROOM = SMEM - 1024 - TAIL;
  __host__ __device__ static constexpr int stages(int nq) {
    const int n = (ROOM - nq * QTILE) / (KTILE + VTILE);
    return n < NB ? n : NB;
  }
  static_assert(NB % NT == 0 && stages(NQ - TIGHT) >= 2 && (TIGHT || stages(NT) >= NT), "stages");
  // warps: softmax and epilogue of the tiles, then loader, issuers, V helper;
  // the rest of the last two warpgroups idles
  static constexpr int W_LOAD = 4 * NT, W_MMA = W_LOAD + 1, W_FIX = W_MMA + NT;
  static constexpr int NF = NT == 3 ? 3 : 1;           // V helpers (as many as stay on whole barriers: NB % NF == 0)
  static constexpr int MISC = NT == 3 ? 8 : 4;
  static_assert(8 * (2 * NQ + 5 * NB + 4 * NT + 8) + 4 <= 512, "barriers");
  static_assert(NB % NF == 0 && 1 + NT + NF <= MISC, "helpers");
  static constexpr int THREADS = 32 * (W_LOAD + MISC);
  // registers: granted at launch, then moved to the softmax (setmaxnreg)
  static constexpr int R_LAUNCH = NT == 3 ? 96 : 168;
  static constexpr int R_SOFT = NT == 3 ? 128 : 208, R_MISC = NT == 3 ? 48 : 88;
  static_assert(128 * NT * R_SOFT + 32 * MISC * R_MISC <= THREADS * R_LAUNCH, "register split");
};

// ---------------------------------------------------------------- exp2
__device__ __forceinline__ float ex2_mufu(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^x on the FMA pipe for x <= 8: the degree-3 polynomial of the spatial
// kernel (fit_exp2_poly.py; max relative error 7.5e-5), clamped at 2^-125.  NaN
// gives some finite number: the row's maximum carries it instead.
constexpr float kP0 = 0.9999280571937561f, kP1 = 0.6932609677314758f;
constexpr float kP2 = 0.2426111251115799f, kP3 = 0.0551716685295105f;
constexpr int kPolyPairs = 2;                // of every 8 pairs of scores

// Packed fp32 pairs in 64-bit registers: constants stay in their pair.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float x, float y) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ f32x2 pair(uint32_t x, uint32_t y) { return pair(__uint_as_float(x), __uint_as_float(y)); }
__device__ __forceinline__ float2 unpair(f32x2 a) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
  return d;
}
__device__ __forceinline__ f32x2 ffma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 fadd2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fmul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Maxima that keep NaN (fmaxf drops it).
__device__ __forceinline__ float fmax2(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 ex2_poly2(f32x2 xx) {
  float2 x = unpair(xx);
  const f32x2 c = pair(fmaxf(x.x, -125.0f), fmaxf(x.y, -125.0f));
  const f32x2 t = fadd2(c, pair(12582912.0f, 12582912.0f));
  const f32x2 j = fadd2(t, pair(-12582912.0f, -12582912.0f));
  const f32x2 f = ffma2(j, pair(-1.0f, -1.0f), c);
  f32x2 q = ffma2(pair(kP3, kP3), f, pair(kP2, kP2));
  q = ffma2(q, f, pair(kP1, kP1));
  q = ffma2(q, f, pair(kP0, kP0));
  const float2 y = unpair(q), tt = unpair(t);
  return make_float2(__int_as_float(__float_as_int(y.x) + (__float_as_int(tt.x) << 23)),
                     __int_as_float(__float_as_int(y.y) + (__float_as_int(tt.y) << 23)));
}

// ---------------------------------------------------------------- PTX helpers
__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ unsigned long long globaltimer() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// try_wait that suspends the thread until the phase completes or about
// `hint_ns` nanoseconds pass.
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity, uint32_t hint_ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(hint_ns)
      : "memory");
  return ok != 0;
}
// Bounded wait for a phase: the thread sleeps in the barrier; the clock and the
// abort epoch are only looked at after a sleep that ended without the phase.
// A warp that waits does so with all lanes on one barrier, which answers them
// together.  (Polling before the sleep, and a vote on the answer, each cost the
// other warps more issue slots than the earlier wake-up gained: 10% and 15% of
// a launch.)  The limit is counted in SM clocks, WAIT_CLOCKS of them, and what
// ended is recorded by the caller, once per role: a wait is a few instructions.
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, uint32_t epoch) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait(b, parity, 100000u)) return true;
  const uint32_t t0 = uint32_t(clock());
  while (!mbar_try_wait(b, parity, 100000u))
    if (*reinterpret_cast<volatile unsigned int *>(&g_cond_abort_epoch) == epoch || uint32_t(clock()) - t0 > WAIT_CLOCKS)
      return false;
  return true;
}
// A wait of this role gave up: the first one of a launch is recorded, and the
// launch's other waits end.
__device__ __forceinline__ void gave_up(uint32_t epoch, int role) {
  if (atomicExch(&g_cond_abort_epoch, epoch) != epoch) atomicOr(&g_cond_error, 1u << role);
}
// The same for the end of work already issued, whatever the abort epoch.
__device__ __forceinline__ void mbar_drain(uint64_t *bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer();
  while (!mbar_try_wait(smem_u32(bar), parity, 100000u) && globaltimer() - t0 < WAIT_NS) {
  }
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1,
                                            int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1),
        "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1,
                                            int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1),
        "r"(c2), "r"(c3)
      : "memory");
}
// Tiled bulk store shared -> global (out-of-range rows and columns are dropped).
__device__ __forceinline__ void tma_store_5d(const CUtensorMap *map, const void *src, int c0, int c1, int c2, int c3,
                                             int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5, %6}], [%1];"
      ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The MMA and commit instructions are issued by the lane whose `lead` is set,
// by predicate instead of a branch: the control flow around them stays
// uniform, so descriptors are computed on the uniform datapath.
__device__ __forceinline__ void tc_commit(uint32_t lead, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}
// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
#define COND_LD16(taddr, r)                                                                                          \
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];" \
               : "=r"((r)[0]), "=r"((r)[1]), "=r"((r)[2]), "=r"((r)[3]), "=r"((r)[4]), "=r"((r)[5]), "=r"((r)[6]),    \
                 "=r"((r)[7]), "=r"((r)[8]), "=r"((r)[9]), "=r"((r)[10]), "=r"((r)[11]), "=r"((r)[12]),               \
                 "=r"((r)[13]), "=r"((r)[14]), "=r"((r)[15])                                                          \
               : "r"(taddr))
#define COND_ST16(taddr, r)                                                                                           \
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" \
               ::"r"(taddr), "r"((r)[0]), "r"((r)[1]), "r"((r)[2]), "r"((r)[3]), "r"((r)[4]), "r"((r)[5]),            \
                 "r"((r)[6]), "r"((r)[7]), "r"((r)[8]), "r"((r)[9]), "r"((r)[10]), "r"((r)[11]), "r"((r)[12]),        \
                 "r"((r)[13]), "r"((r)[14]), "r"((r)[15])                                                             \
               : "memory")
#define COND_LD8(taddr, r)                                                                                            \
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"                                \
               : "=r"((r)[0]), "=r"((r)[1]), "=r"((r)[2]), "=r"((r)[3]), "=r"((r)[4]), "=r"((r)[5]), "=r"((r)[6]),    \
                 "=r"((r)[7])                                                                                         \
               : "r"(taddr))
#define COND_ST8(taddr, r)                                                                                            \
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"((r)[0]),      \
               "r"((r)[1]), "r"((r)[2]), "r"((r)[3]), "r"((r)[4]), "r"((r)[5]), "r"((r)[6]), "r"((r)[7])              \
               : "memory")
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor: start address, leading and stride byte
// offsets, version 1, swizzle layout 2 = 128B, 4 = 64B, 6 = 32B.  The low word
// is the start address in 16-byte units (14 bits hold all of shared memory)
// and the leading offset, so later operands of a tile are an addition away.
template <uint32_t LBO> __device__ __forceinline__ uint32_t sdesc_lo(uint32_t saddr) {
  return (saddr >> 4) | (((LBO >> 4) & 0x3FFFu) << 16);
}
template <uint32_t SBO, uint32_t LAYOUT> __device__ __forceinline__ uint64_t sdesc(uint32_t lo) {
  constexpr uint32_t hi = ((SBO >> 4) & 0x3FFFu) | (1u << 14) | (LAYOUT << 29);
  return ((uint64_t)hi << 32) | lo;
}
__host__ __device__ constexpr uint32_t layout_of(int swizzle_bytes) {
  return swizzle_bytes == 128 ? 2u : (swizzle_bytes == 64 ? 4u : 6u);
}
// Instruction descriptor, kind::f16: fp32 accumulate, bf16 A and B.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Lane 0's value, known to the compiler to be the same in the whole warp.
template <typename T> __device__ __forceinline__ T uniform(T v) { return T(__shfl_sync(0xffffffffu, v, 0)); }
// True in one lane of the converged warp, always the same one.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok));
  return ok;
}
// 16-byte chunk f of row r of a swizzled tile with rows of `bytes`.
template <int BYTES> __device__ __forceinline__ int swz(int r, int f) {
  return f ^ (BYTES == 128 ? (r & 7) : (BYTES == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1)));
}

// ---------------------------------------------------------------- work items
struct Maps {
  CUtensorMap q0, q1;          // the head's first C0 channels, the rest
  CUtensorMap k0[2], k1[2], v[2], vr[2];      // K alike; V's atoms, the rest of V
  CUtensorMap o0, o1;
};

struct Args {
  st::CondParams c;
  st::FastDiv dqb, dsplit, dhw, dkv, dt, dtblk, dper[2];
  int n_tblk;                  // frame blocks of a batch
  int q_blocks, tile_rows;     // row blocks of a unit, rows of a tile (128, or whole groups of heads)
  // Resident: the row blocks are cut into bands of `band` (the last one
  // `band_last`), and items run through all heads and units within a band
  int band, band_last, cols, n_bands;
  st::FastDiv dband, dband_last, dbandcols;
  int n_items;
  int weighed;                 // resident, sets of different lengths: items are cut by cost
  int resident;                // every key tile of an item fits the ring: K and V stay from item to item
  int max_steps;
  int spread;                  // the tiles of a CTA take the same rows and every NT-th step
  int nq, ns;                  // Q slots, K and V stages
  st::FastDiv dns;
  int n_split;                 // parts of an item's keys (each NT of the call's parts with spread)
  int tma_out;                 // bf16 rows go out as tiles
  float scale_log2;
  uint32_t epoch;
};

// One item, written by the scheduler warp and read by every other.
struct alignas(16) Item {
  int n_qt;                    // row tiles; 0: no more items
  int n_kv;                    // steps of this item
  int n0, n1;                  // keys of the segments
  int s0, j0;                  // steps of segment 0; first step
  int set0, set1;              // the segments' sets
  int row0, row1;              // first rows of their key ranges (packed)
  int r0, w, unit, split;      // first row, walked head, unit, part of the keys
  int c3, c4;                  // the unit's frame coordinates in the Q and O maps
  int kvh;
  int fresh;                   // its keys are not those of the item before
  int release;                 // nor those of the item after
  int qb, qb_end;              // row block of the unit; end of its band
};
constexpr int ITEMS = 4;       // items in flight between the scheduler and the others
static_assert(ITEMS * sizeof(Item) <= 384, "item ring");

struct Step {
  int seg, key, valid;         // segment, first key in its range, keys that exist
  int set, row;                // set, and the row of the key range's start (packed)
};

template <int BN> __device__ __forceinline__ Step step_of(const Item &it, int j) {
  Step s;
  j += it.j0;
  s.seg = j < it.s0 ? 0 : 1;
  s.key = (s.seg ? j - it.s0 : j) * BN;
  s.valid = (s.seg ? it.n1 : it.n0) - s.key;
  s.set = s.seg ? it.set1 : it.set0;
  s.row = s.seg ? it.row1 : it.row0;
  return s;
}

template <int D> __device__ __forceinline__ void rows_of(const Args &a, Item &it) {
  it.r0 = it.qb * Cfg<D>::NT * a.tile_rows;
  const int left = a.c.R - it.r0;
  it.n_qt = a.spread ? Cfg<D>::NT : left > 2 * a.tile_rows && Cfg<D>::NT > 2 ? 3 : (left > a.tile_rows ? 2 : 1);
}

// The keys of segment g that batch b attends.  table: the segments' ranges.
template <int D>
__device__ __forceinline__ void set_range(const Args &a, const int2 *table, int g, int b, int &set, int &row, int &n) {
  set = row = n = 0;
  if (g >= a.c.n_seg) return;
  set = int(st::fdiv(uint32_t(b), a.dper[g]));
  if (a.c.seg[g].n_sets <= Cfg<D>::TABLE) {
    const int2 r = table[g * Cfg<D>::TABLE + set];
    row = r.x;
    n = r.y;
  } else {
    st::KvSeg sg = a.c.seg[g];
    sg.len = st::after_wait(sg.len);
    sg.offsets = st::after_wait(sg.offsets);
    const st::KvRange r = st::kv_range(sg, b);
    row = r.row0;
    n = r.n;
  }
}

// Streaming: q block fastest, then split, head, unit.  Resident: q block of a
// band, head and unit, band.
template <int D>
__device__ __forceinline__ Item decode(const Args &a, const int2 *table, int x) {
  using K = Cfg<D>;
  Item it;
  uint32_t z;                                  // unit * HW + walked head
  if (a.resident) {
    const int band = int(st::fdiv(uint32_t(x), a.dbandcols));
    const bool last = band + 1 >= a.n_bands;
    const int len = last ? a.band_last : a.band;
    x -= band * a.band * a.cols;
    z = st::fdiv(uint32_t(x), last ? a.dband_last : a.dband);
    it.qb = band * a.band + x - int(z) * len;
    it.qb_end = band * a.band + len;
    it.split = 0;
  } else {
    const uint32_t y = st::fdiv(uint32_t(x), a.dqb);
    it.qb = x - int(y) * a.q_blocks;
    it.qb_end = a.q_blocks;
    z = st::fdiv(y, a.dsplit);
    it.split = int(y) - int(z) * a.n_split;
  }
  it.unit = int(st::fdiv(z, a.dhw));
  it.w = int(z) - it.unit * a.c.HW;
  it.kvh = int(st::fdiv(uint32_t(it.w), a.dkv));
  rows_of<D>(a, it);
  const int ub = int(st::fdiv(uint32_t(it.unit), a.dt)), t = it.unit - ub * a.c.g.T;
  if (a.c.g.tblk != a.c.g.T) {
    const int tb = int(st::fdiv(uint32_t(t), a.dtblk));
    it.c3 = t - tb * a.c.g.tblk;
    it.c4 = ub * a.n_tblk + tb;
  } else {
    it.c3 = t;
    it.c4 = ub;
  }
  const int b = ub * a.c.bm;
  set_range<D>(a, table, 0, b, it.set0, it.row0, it.n0);
  set_range<D>(a, table, 1, b, it.set1, it.row1, it.n1);
  it.s0 = (it.n0 + K::BN - 1) / K::BN;
  const int total = it.s0 + (it.n1 + K::BN - 1) / K::BN;
  if (a.n_split == 1) {
    it.j0 = 0;
    it.n_kv = total;
  } else {
    it.j0 = int(st::fdiv(uint32_t(total) * uint32_t(it.split), a.dsplit));
    it.n_kv = int(st::fdiv(uint32_t(total) * uint32_t(it.split + 1), a.dsplit)) - it.j0;
  }
  return it;
}
// Whether two items attend the same key tiles (and so share resident stages).
__device__ __forceinline__ bool same_keys(const Item &a, const Item &b) {
  return a.kvh == b.kvh && a.set0 == b.set0 && a.set1 == b.set1;
}

// The items of a CTA.  Streaming: every gridDim-th, so that the CTAs that run
// together share K/V tiles in L2.  Resident: consecutive ones, a band of row
// blocks of one head; the next row block needs no division.  The CTAs beside
// work on the same rows of the other heads, whose channels lie next to these
// in Q and O: sectors that two heads share, and DRAM pages, are then touched
// at about the same time.  (Heads at different rows at a time: Q and O of
// 65,536 x 16 heads x 72 ran at 2.3 TB/s.)  Where the sets differ in length
// the cut is by cost: an item without keys costs about as much as ITEM_STEPS
// steps.  Finding the cut takes 5 us for 8 units (serial code, read for the
// first time), so it pays from about four items per CTA on.
constexpr int ITEM_STEPS = 2, WEIGHED = 16;      // units up to which the cut is by cost
template <int D> struct Walk {
  int x, end, inc;
  static __device__ __forceinline__ int cost(const Args &a, const int2 *table, int unit) {
    const int b = int(st::fdiv(uint32_t(unit), a.dt)) * a.c.bm;
    int set, row, n0, n1;
    set_range<D>(a, table, 0, b, set, row, n0);
    set_range<D>(a, table, 1, b, set, row, n1);
    return ITEM_STEPS + (n0 + Cfg<D>::BN - 1) / Cfg<D>::BN + (n1 + Cfg<D>::BN - 1) / Cfg<D>::BN;
  }
  // first item of CTA `cta`
  static __device__ int cut(const Args &a, const int2 *table, int units, uint32_t sum, int cta) {
    const unsigned long long col = (unsigned long long)sum * a.c.HW;   // a row block of all heads
    unsigned long long rest = col * a.q_blocks * cta / gridDim.x;
    const int band = min(int(rest / (col * a.band)), a.n_bands - 1);
    rest -= col * a.band * band;
    const int len = band + 1 < a.n_bands ? a.band : a.band_last;
    int z = 0;
    for (int u = 0; u < units; ++u) {
      const uint32_t c = cost(a, table, u);
      const unsigned long long all = (unsigned long long)c * a.c.HW * len;
      if (rest < all) return band * a.band * a.cols + z * len + int(rest / c);
      rest -= all;
      z += a.c.HW;
    }
    return band * a.band * a.cols + z * len;
  }
  __device__ __forceinline__ explicit Walk(const Args &a, const int2 *table) {
    if (a.resident) {
      inc = 1;
      if (a.weighed) {
        const int units = a.c.g.B * a.c.g.T;
        uint32_t sum = 0;
        for (int u = 0; u < units; ++u) sum += cost(a, table, u);
        x = cut(a, table, units, sum, blockIdx.x);
        end = cut(a, table, units, sum, blockIdx.x + 1);
      } else if (int(gridDim.x) >= a.n_bands * a.cols) {   // a band of a head per CTA
        const int band = int(blockIdx.x) / a.cols, col = int(blockIdx.x) - band * a.cols;
        const int len = band + 1 < a.n_bands ? a.band : a.band_last;
        x = band * a.band * a.cols + col * len;
        end = band < a.n_bands ? x + len : x;
      } else {
        x = int((long long)a.n_items * blockIdx.x / gridDim.x);
        end = int((long long)a.n_items * (blockIdx.x + 1) / gridDim.x);
      }
    } else {
      x = blockIdx.x;
      end = a.n_items;
      inc = gridDim.x;
    }
  }
};

// A reader's place in the ring of items.
struct Reader {
  uint32_t i = 0;
  // The next item, once it is there: the caller reads what it needs, then the
  // warp hands it back.
  __device__ __forceinline__ const Item *get(const Item *items, uint64_t *full, uint32_t epoch) const {
    return mbar_wait(full + i % ITEMS, (i / ITEMS) & 1, epoch) ? items + i % ITEMS : nullptr;
  }
  __device__ __forceinline__ void done(uint64_t *empty, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + i % ITEMS);
    ++i;
  }
};

// Position of the K/V ring: streaming, steps follow one another; resident,
// step j is in stage j and `run` counts the loads of each.
template <int NB> struct Ring {
  uint32_t pos = 0, run = 0;
  // barriers and their phase
  __device__ __forceinline__ int bar(bool resident, int j) const { return resident ? j : int((pos + j) % NB); }
  __device__ __forceinline__ uint32_t phase(bool resident, int j) const {
    return (resident ? run : (pos + j) / NB) & 1;
  }
  __device__ __forceinline__ int stage(const Args &a, bool resident, int j) const {
    const uint32_t x = pos + j;
    return resident ? j : int(x - st::fdiv(x, a.dns) * uint32_t(a.ns));
  }
};

// The steps of an item a tile takes: all, or (keys spread over the tiles) every
// NT-th, by the position in the ring: step j of an item that began at `pos`
// belongs to tile (pos + j) % NT.
template <int NT> __device__ __forceinline__ int first_step(bool spread, uint32_t pos, int X) {
  if (!spread) return 0;
  const int f = X - int(pos % NT);
  return f < 0 ? f + NT : f;
}
// Its place among the item's Q tiles.
__device__ __forceinline__ int q_index(bool spread, int first, int X) { return spread ? first : X; }
// Q tiles of an item: of every tile that has a step of it.
__device__ __forceinline__ int q_tiles(bool spread, int n_qt, int n_kv) {
  return spread ? min(n_qt, n_kv) : (n_kv > 0 ? n_qt : 0);
}
// Its n-th Q tile's slot where each tile has its own.
__device__ __forceinline__ int own_slot(bool spread, int X, uint32_t n) { return spread ? X : 2 * X + int(n & 1); }
// TIGHT: the next slot of the Q tiles, which take the slots in turn, and the
// parity of its turn.  A slot has its own barrier then: it cannot be filled again
// before its tile has been released, so no waiter falls behind by two phases (a
// tile's barriers in turn could, where others' rows left it one tile in a slot
// after another).
struct QTurn {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ QTurn ahead(int i, int nq) const {
    QTurn t;
    const bool wrap = slot + i >= nq;
    t.slot = slot + i - (wrap ? nq : 0);
    t.parity = parity ^ (wrap ? 1 : 0);
    return t;
  }
};

template <int D, bool MIX>
__global__ void __launch_bounds__(Cfg<D, MIX>::THREADS, 1)
    cond_attn_sm100(const __grid_constant__ Maps mp, const __grid_constant__ Args a) {
  using K = Cfg<D, MIX>;
  constexpr int NT = K::NT, NB = K::NB, NQ = K::NQ, BN = K::BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sQ = base;
  const int nq = a.nq;
  uint8_t *sK = sQ + nq * K::QTILE;
  uint8_t *sV = sK + a.ns * K::KTILE;
  int2 *sSet = reinterpret_cast<int2 *>(sQ + K::ROOM);
  Item *sItem = reinterpret_cast<Item *>(sSet + 2 * K::TABLE);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sItem + ITEMS);
  uint64_t *q_full = bars, *q_empty = q_full + NQ;   // q_empty: by slot; q_full: the same (TIGHT), or two per tile, its Q tiles in turn
  uint64_t *k_full = q_empty + NQ, *k_empty = k_full + NB;      // k_empty, v_empty: one arrival per tile that reads the stage
  uint64_t *v_full = k_empty + NB, *v_empty = v_full + NB, *v_ready = v_empty + NB;
  // per tile: S ready; P written; O of an item complete
  uint64_t *s_full = v_ready + NB, *p_full = s_full + NT, *o_full = p_full + NT;
  uint64_t *mma_done = o_full + NT;
  uint64_t *item_full = mma_done + NT, *item_empty = item_full + ITEMS;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(item_empty + ITEMS);

  const bool resident = a.resident != 0, spread = a.spread != 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NQ; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 4);             // the softmax warps, once O is out of it
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, spread ? 1 : NT);
      mbar_init(v_full + i, 1);
      mbar_init(v_empty + i, spread ? 1 : NT);
      mbar_init(v_ready + i, 1);
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, BLOCK_M);
      mbar_init(o_full + i, 1);
      mbar_init(mma_done + i, 1);
    }
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(item_full + i, 1);
      mbar_init(item_empty + i, 5 * NT + K::NF);   // softmax warps, issuers, helpers
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == K::W_LOAD) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 32 * (K::W_LOAD + 1)) {   // (maps are parameters: nothing to wait for)
    prefetch_map(&mp.q0);
    if (K::C1) prefetch_map(&mp.q1);
    if (a.c.seg[0].L) {
      prefetch_map(&mp.k0[0]);
      if (K::C1) prefetch_map(&mp.k1[0]);
      prefetch_map(&mp.v[0]);
    }
  }
  // the rows behind the whole groups of a tile are 0, and their scores as tame as
  // the others' (left as they were they could be NaN and have O rescaled in every step)
  if (a.tile_rows < BLOCK_M) {
    for (int i = a.tile_rows * K::SW0 + 16 * int(threadIdx.x); i < K::QT0; i += 16 * K::THREADS)
      for (int n = 0; n < nq; ++n) *reinterpret_cast<uint4 *>(sQ + n * K::QTILE + i) = make_uint4(0, 0, 0, 0);
    for (int i = K::QT0 + a.tile_rows * K::SW1 + 16 * int(threadIdx.x); i < K::QTILE; i += 16 * K::THREADS)
      for (int n = 0; n < nq; ++n) *reinterpret_cast<uint4 *>(sQ + n * K::QTILE + i) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
  }
  // barriers and TMEM are set up: let the next kernel of the stream be
  // scheduled, then wait for the previous one before any global access
  pdl_trigger();
  pdl_wait();
  // the sets' key ranges; a warp per set looks where a mask's last key is, so that
  // the padding behind a prompt costs nothing
#pragma unroll 1
  for (int g = 0; g < a.c.n_seg; ++g) {
    st::KvSeg sg = a.c.seg[g];
    if (sg.n_sets > K::TABLE) continue;
    sg.len = st::after_wait(sg.len);
    sg.offsets = st::after_wait(sg.offsets);
    if (!sg.mask) {
      if (int(threadIdx.x) < sg.n_sets) {
        const st::KvRange r = st::kv_range(sg, int(threadIdx.x) * sg.per);
        sSet[g * K::TABLE + threadIdx.x] = make_int2(r.row0, r.n);
      }
      continue;
    }
#pragma unroll 1
    for (int set = warp; set < sg.n_sets; set += K::THREADS / 32) {
      const int n = st::last_key(st::after_wait(sg.mask) + (long long)set * sg.L, st::kv_range(sg, set * sg.per).n, lane);
      if (lane == 0) sSet[g * K::TABLE + set] = make_int2(0, n);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t epoch = a.epoch;

  if (warp >= K::W_LOAD) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(K::R_MISC));
    if (warp == K::W_LOAD) {
      // ================= scheduler and TMA producer =================
      // An item is handed out once the next one is known, then loaded.
      if (lane == 0) {
        bool ok = true;
        Ring<NB> ring;
        uint32_t qn = 0;                              // 2 bits per tile: its Q tiles so far (barrier, phase)
        int last_kv = -1;                             // streaming: ring position of the last K/V issued
        int loaded = 0;                               // resident: stages loaded in this run
        bool first = true;
        Walk<D> wk(a, sSet);
        const bool tight = K::TIGHT && nq < NQ;
        QTurn qt;                                     // TIGHT: next Q slot
        // the item's Q tiles [i0, i1)
        auto load_q = [&](const Item &it, int i0, int i1) -> bool {
          i1 = min(i1, q_tiles(spread, it.n_qt, it.n_kv));
#pragma unroll 1
          for (int i = i0; i < i1; ++i) {
            const int X = spread ? int((ring.pos + i) % NT) : i;
            const uint32_t n = qn >> 2 * X & 3;
            const int slot = K::TIGHT ? qt.slot : own_slot(spread, X, n);
            uint64_t *full = q_full + (K::TIGHT ? slot : 2 * X + int(n & 1));
            const uint32_t ph = (K::TIGHT ? qt.parity : (spread ? n : n >> 1) & 1) ^ 1;
            if (!(ok = mbar_wait(q_empty + slot, ph, epoch))) return false;
            qn ^= (n ^ ((n + 1) & 3)) << 2 * X;
            uint8_t *dst = sQ + slot * K::QTILE;
            if (K::TIGHT) qt = qt.ahead(1, nq);
            const int row = it.r0 + (spread ? 0 : X * a.tile_rows);
            mbar_expect_tx(full, a.tile_rows * (K::SW0 + K::SW1));
            if (a.c.G > 1) {
              tma_load_5d(dst, &mp.q0, full, 0, 0, it.w, row / a.c.G, it.unit);
              if (K::C1) tma_load_5d(dst + K::QT0, &mp.q1, full, 64, 0, it.w, row / a.c.G, it.unit);
            } else {
              tma_load_5d(dst, &mp.q0, full, 0, it.w, row, it.c3, it.c4);
              if (K::C1) tma_load_5d(dst + K::QT0, &mp.q1, full, 64, it.w, row, it.c3, it.c4);
            }
          }
          return true;
        };
        Item sch;                                     // the item to publish
        sch.n_qt = 1;
        sch.qb = sch.qb_end = 0;
        sch.set0 = -1;
        for (uint32_t i = 0; ok; ++i) {
          // item i, and whether it has other keys than its neighbours
          if (sch.n_qt > 0) {
            const Item prev = sch;
            if (wk.x >= wk.end) {
              sch.n_qt = 0;
            } else if (wk.inc == 1 && sch.qb + 1 < sch.qb_end) {
              ++sch.qb;
              rows_of<D>(a, sch);
            } else {
              sch = decode<D>(a, sSet, wk.x);
            }
            wk.x += wk.inc;
            sch.fresh = !same_keys(prev, sch);
            // the item before is complete now: hand it out
            if (i > 0) {
              sItem[(i - 1) % ITEMS].release = sch.n_qt == 0 || sch.fresh;
              mbar_arrive(item_full + (i - 1) % ITEMS);
            }
            if (!(ok = mbar_wait(item_empty + i % ITEMS, ((i / ITEMS) & 1) ^ 1, epoch))) break;
            sItem[i % ITEMS] = sch;
            if (sch.n_qt == 0) mbar_arrive(item_full + i % ITEMS);
          }
          if (i == 0) continue;
          const Item &it = sItem[(i - 1) % ITEMS];    // its slot is not written again before the next but two
          if (it.n_qt == 0) break;
          const bool load_kv = !resident || it.fresh;
          if (resident && load_kv && !first) ++ring.run;
          first = false;
          const int n = resident ? (load_kv ? a.max_steps : 1) : it.n_kv;
          for (int j = 0; j < n && ok; ++j) {
            const int bar = ring.bar(resident, j), st = ring.stage(a, resident, j);
            // the stage is free once the step before it there has been read
            const uint32_t before = ring.pos + j - a.ns;
            const int was = resident ? j : int(before % NB);
            const uint32_t ph = resident ? (ring.run & 1) ^ 1 : before / NB & 1;
            const bool wait = resident || int(ring.pos + j) >= a.ns;
            const Step sp = step_of<BN>(it, j);
            const int g = sp.seg;
            const int set = a.c.seg[g].offsets ? 0 : sp.set;   // packed: rows of one long sequence
            const bool real = j < it.n_kv;            // resident: stages past the item's steps only change phase
            if (load_kv) {
              if (wait && !(ok = mbar_wait(k_empty + was, ph, epoch))) break;
              if (real) {
                mbar_expect_tx(k_full + bar, K::KBYTES);
                uint8_t *dk = sK + st * K::KTILE;
                tma_load_4d(dk, &mp.k0[g], k_full + bar, 0, it.kvh, sp.row + sp.key, set);
                if (K::C1) tma_load_4d(dk + K::KT0, &mp.k1[g], k_full + bar, 64, it.kvh, sp.row + sp.key, set);
                if (!resident) last_kv = int(ring.pos) + j;
                else loaded = j + 1;
              } else {
                mbar_arrive(k_full + bar);
              }
            }
            if (j == 0 && !load_q(it, 0, tight ? 1 : NT)) break;
            if (load_kv) {
              if (wait && !(ok = mbar_wait(v_empty + was, ph, epoch))) break;
              if (real) {
                mbar_expect_tx(v_full + bar, K::VBYTES);
                uint8_t *dv = sV + st * K::VTILE;
#pragma unroll 1
                for (int t = 0; t < K::VA; ++t)
                  tma_load_4d(dv + t * K::VAT, &mp.v[g], v_full + bar, t * K::VW, it.kvh, sp.row + sp.key, set);
                if (MIX) tma_load_4d(dv + K::VT0, &mp.vr[g], v_full + bar, K::NV0, it.kvh, sp.row + sp.key, set);
              } else {
                mbar_arrive(v_full + bar);
              }
            }
            if (tight && j == (n > 1 ? 1 : 0) && !load_q(it, 1, NT)) break;
          }
          if (!resident) ring.pos += it.n_kv;
        }
        if (!ok) {
          gave_up(epoch, 0);
          // the last load issued into every stage and Q slot (a wait for one
          // that was not issued runs into its limit)
          if (resident) {
            for (int j = 0; j < loaded; ++j) {
              mbar_drain(k_full + j, ring.run & 1);
              mbar_drain(v_full + j, ring.run & 1);
            }
          } else {
            for (int i = last_kv; i >= 0 && i > last_kv - NB; --i) mbar_drain(k_full + i % NB, (i / NB) & 1);
            for (int i = last_kv; i >= 0 && i > last_kv - NB; --i) mbar_drain(v_full + i % NB, (i / NB) & 1);
          }
          // (a barrier never used answers at once)
          if (K::TIGHT) {
            for (int i = 0; i < nq; ++i) mbar_drain(q_full + i, qt.parity ^ (i < qt.slot ? 0 : 1));
          } else {
            for (int X = 0; X < NT; ++X)
              for (uint32_t k = 1; k <= 2; ++k) {
                const uint32_t n = ((qn >> 2 * X) - k) & 3;
                mbar_drain(q_full + 2 * X + (n & 1), n >> 1);
              }
          }
        }
      }
      __syncwarp();
    } else if (warp >= K::W_MMA && warp < K::W_MMA + NT) {
      // ================= issuer of tile X =================
      // P of a step ready -> its PV, then S of the next step (of the next item
      // after the last) into the same columns: MMAs of one thread execute in
      // order.  The whole warp walks the loop.
      const int X = uniform(warp) - K::W_MMA;
      const uint32_t aQ = smem_u32(sQ), aK = smem_u32(sK), aV = smem_u32(sV);
      const uint32_t dS = uniform(tmem) + X * K::TW, dO = dS + BN;
      const uint32_t lead = elect_one();
      bool ok = true;
      Ring<NB> ring;
      Reader rd;
      uint32_t qc = 0, steps = 0;                      // Q tiles and steps of this tile so far
      QTurn qt;                                        // TIGHT: first Q slot of the item
      // This tile has waited for the stages it now holds (resident: those of its
      // run).  The run's first item may have no rows for it, so a later one waits;
      // the stages' phases stay until this tile, too, has handed them back.
      bool landed = false;
      struct Work {                                    // what the issuer needs of an item
        int n_qt, n, n0, n1, s0, j0;
        bool release;
        // chunks of 16 keys of step j
        __device__ __forceinline__ int chunks(int j) const {
          j += j0;
          const int left = j < s0 ? n0 - j * BN : n1 - (j - s0) * BN;
          return left >= BN ? K::CH : (left + 15) >> 4;
        }
      };
      Work wk;
      auto fetch = [&]() -> bool {
        const Item *ip = rd.get(sItem, item_full, epoch);
        if (!ip) return false;
        wk.n_qt = uniform(ip->n_qt);
        wk.n = uniform(ip->n_kv);
        wk.n0 = uniform(ip->n0);
        wk.n1 = uniform(ip->n1);
        wk.s0 = uniform(ip->s0);
        wk.j0 = uniform(ip->j0);
        wk.release = !resident || uniform(ip->release);
        rd.done(item_empty, lane);
        return true;
      };
      ok = fetch();
      while (ok && wk.n_qt > 0) {
        const Work cur = wk;
        const int j0 = first_step<NT>(spread, ring.pos, X), inc = spread ? NT : 1;
        const bool here = X < cur.n_qt && j0 < cur.n;
        if (here) {
          const QTurn mine = qt.ahead(q_index(spread, j0, X), nq);
          const int slot = K::TIGHT ? mine.slot : own_slot(spread, X, qc);
          const uint32_t qa = sdesc_lo<16>(aQ + slot * K::QTILE);
          if (!(ok = mbar_wait(q_full + (K::TIGHT ? slot : 2 * X + int(qc & 1)), K::TIGHT ? mine.parity : (qc >> 1) & 1, epoch)))
            break;
          ++qc;
          for (int j = j0; j < cur.n; j += inc, ++steps) {
            // S(j), over P(j - 1), which PV(j - 1) has read by then; only as many
            // keys as there are (whole chunks)
            const int bar = ring.bar(resident, j), st = ring.stage(a, resident, j);
            const uint32_t ph = ring.phase(resident, j);
            if (!landed && !(ok = mbar_wait(k_full + bar, ph, epoch))) break;
            tc_fence_after();
            const int nk = cur.chunks(j);
            const uint32_t ids = idesc_bf16(BLOCK_M, 0, 0, 0) | uint32_t(nk * 2) << 17;
            const uint32_t ka = sdesc_lo<16>(aK + st * K::KTILE);
#pragma unroll
            for (int kk = 0; kk < K::C0 / 16; ++kk)
              mma_ss(lead, dS, sdesc<8 * K::SW0, layout_of(K::SW0)>(qa + kk * 2),
                     sdesc<8 * K::SW0, layout_of(K::SW0)>(ka + kk * 2), ids, kk > 0);
            if (K::C1) {
#pragma unroll
              for (int kk = 0; kk < K::C1X / 16; ++kk)
                mma_ss(lead, dS, sdesc<8 * K::SW1X, layout_of(K::SW1X)>(qa + K::QT0 / 16 + kk * 2),
                       sdesc<8 * K::SW1X, layout_of(K::SW1X)>(ka + K::KT0 / 16 + kk * 2), ids, 1);
            }
            tc_commit(lead, s_full + X);
            if (cur.release) tc_commit(lead, k_empty + bar);  // handed back at the last item that reads it
            // PV(j)
            if (!landed && !(ok = mbar_wait(v_ready + bar, ph, epoch))) break;
            const bool last = j + inc >= cur.n;
            if (last && !(ok = fetch())) break;              // wk: now the next item
            const uint32_t va = sdesc_lo<K::VAT>(aV + st * K::VTILE);
            if (!(ok = mbar_wait(p_full + X, steps & 1, epoch))) break;
            tc_fence_after();
            constexpr uint32_t IDPV = idesc_bf16(BLOCK_M, K::NV0, 0, 1), IDVR = idesc_bf16(BLOCK_M, K::VRX, 0, 1);
            const uint32_t vr = sdesc_lo<16>(aV + st * K::VTILE + K::VT0);
#pragma unroll
            for (int kk = 0; kk < K::CH; ++kk)
              if (kk < nk) {
                const uint32_t acc = (j > j0 || kk > 0) ? 1u : 0u;
                mma_ts(lead, dO, dS + kk * 8, sdesc<8 * K::VSW, layout_of(K::VSW)>(va + kk * K::VSW), IDPV, acc);
                if (MIX)
                  mma_ts(lead, dO + K::NV0, dS + kk * 8, sdesc<8 * K::VSWR, layout_of(K::VSWR)>(vr + kk * K::VSWR), IDVR, acc);
              }
            if (last) tc_commit(lead, o_full + X);
            if (cur.release) tc_commit(lead, v_empty + bar);
          }
          if (!ok) break;
          landed = resident;
        }
        if (cur.release) landed = false;
        // stages this tile did not use in this item: hand them back once they
        // were filled (a commit: earlier items of the run may still read them)
        if (cur.release && !spread) {
          const int last = resident ? a.max_steps : cur.n;
          for (int j = here ? cur.n : 0; j < last && ok; ++j) {
            const int bar = ring.bar(resident, j);
            const uint32_t ph = ring.phase(resident, j);
            if (!(ok = mbar_wait(k_full + bar, ph, epoch))) break;
            tc_commit(lead, k_empty + bar);
            if (!(ok = mbar_wait(v_ready + bar, ph, epoch))) break;
            tc_commit(lead, v_empty + bar);
          }
        }
        if (K::TIGHT) qt = qt.ahead(q_tiles(spread, cur.n_qt, cur.n), nq);
        if (resident) ring.run += cur.release;
        else ring.pos += cur.n;
        if (!here && ok) ok = fetch();
      }
      if (!ok && lane == 0) gave_up(epoch, 1 + X);
      // every MMA issued completes before TMEM is released
      __syncwarp();
      tc_commit(lead, mma_done + X);
      mbar_drain(mma_done + X, 0);
      __syncwarp();
    } else if (warp >= K::W_FIX && warp < K::W_FIX + K::NF) {
      // ================= V rows of keys that do not count; ones column =================
      bool ok = true;
      Ring<NB> ring;
      Reader rd;
      bool first = true;
      while (ok) {
        const Item *ip = rd.get(sItem, item_full, epoch);
        if (!(ok = ip != nullptr)) break;
        const Item it = *ip;
        rd.done(item_empty, lane);
        if (it.n_qt == 0) break;
        if (resident && !it.fresh) continue;
        if (resident && !first) ++ring.run;
        first = false;
        const int n = resident ? a.max_steps : it.n_kv;
        // its steps: those whose barrier is one of its own
        int j = warp - K::W_FIX - (resident ? 0 : int(ring.pos % K::NF));
        if (j < 0) j += K::NF;
        for (; j < n; j += K::NF) {
          const int bar = ring.bar(resident, j), st = ring.stage(a, resident, j);
          const uint32_t ph = ring.phase(resident, j);
          const Step sp = step_of<BN>(it, j);
          const unsigned char *mk = a.c.seg[sp.seg].mask;
          const bool real = j < it.n_kv;
          bool keep[(BN + 31) / 32];
          bool dead = false;                   // the tile has rows to clear
          if (real) {                          // before the wait: the mask bytes are on their way
            if (mk) mk += (long long)sp.set * a.c.seg[sp.seg].L + sp.key;
#pragma unroll
            for (int i = 0; i < (BN + 31) / 32; ++i) {
              const int r = lane + 32 * i;
              keep[i] = r < sp.valid && (!mk || st::after_wait(mk)[r]);
              dead |= !keep[i] && (BN % 32 == 0 || r < BN);
            }
          }
          const bool work = real && (K::ONES || __any_sync(0xffffffffu, dead));
          if (lane == 0) ok = mbar_wait(v_full + bar, ph, epoch);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          if (work) {
            uint8_t *vt = sV + st * K::VTILE;
#pragma unroll
            for (int i = 0; i < (BN + 31) / 32; ++i) {
              const int r = lane + 32 * i;
              if (BN % 32 && r >= BN) continue;
              if (!keep[i]) {
                for (int t = 0; t < K::VA; ++t)
#pragma unroll
                  for (int f = 0; f < K::VSW / 16; ++f)
                    *reinterpret_cast<uint4 *>(vt + t * K::VAT + r * K::VSW + f * 16) = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int f = 0; f < K::VR / 8; ++f)
                  *reinterpret_cast<uint4 *>(vt + K::VT0 + r * K::VSWR + f * 16) = make_uint4(0, 0, 0, 0);
              } else if (K::ONES) {
                *reinterpret_cast<uint16_t *>(vt + K::ONE_AT + r * K::ONE_SW + (swz<K::ONE_SW>(r, K::ONE_X >> 4) << 4) + (K::ONE_X & 15)) =
                    0x3F80;                    // bf16 1.0
              }
            }
            fence_async_smem();                // visible to the tensor core
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(v_ready + bar);
        }
        if (!resident) ring.pos += it.n_kv;
      }
      if (!ok && lane == 0) gave_up(epoch, 1 + NT);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(K::R_SOFT));
    // ================= softmax and epilogue of tile X, one thread per row =================
    const int X = warp >> 2;
    const int r = ((warp & 3) << 5) + lane;    // row in tile == TMEM lane
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + X * K::TW;
    const uint32_t tO = tS + BN;
    const float sl2 = a.scale_log2;
    const f32x2 scale2 = pair(sl2, sl2);
    uint32_t gs = 0, oc = 0, pos = 0;          // steps and items of this tile; steps of all
    const int inc = spread ? NT : 1;
    QTurn qt;                                  // TIGHT: the item's first Q slot
    int slot = 0;                              // this tile's last
    bool pending = false;                      // O of the item before is on its way out of its Q slot
    // Hands that slot to the loader once the store has read it.
    auto release_slot = [&]() {
      if (lane == 0 && pending) {
        bulk_wait_read();
        mbar_arrive(q_empty + (K::TIGHT ? slot : own_slot(false, X, oc - 1)));
      }
      pending = false;
    };
    bool ok = true;
    Reader rd;
    while (ok) {
      const Item *ip = rd.get(sItem, item_full, epoch);
      if (!(ok = ip != nullptr)) break;
      const Item &it = *ip;                    // handed back at the end
      const int n_kv = it.n_kv, n0 = it.n0, n1 = it.n1, s0 = it.s0, j0 = it.j0;
      if (it.n_qt == 0) break;
      const int first = first_step<NT>(spread, pos, X);
      const int mine = K::TIGHT ? qt.ahead(q_index(spread, first, X), nq).slot : own_slot(spread, X, oc);
      if (K::TIGHT) qt = qt.ahead(q_tiles(spread, it.n_qt, n_kv), nq);
      pos += n_kv;
      if (X >= it.n_qt || first >= n_kv) release_slot();   // (no first step to do it at)
      if (X >= it.n_qt) {
        rd.done(item_empty, lane);
        continue;
      }
      float m = NO_KEY, l = 0.f;
      for (int j = first; j < n_kv; j += inc, ++gs) {
        const int g = j0 + j < s0 ? 0 : 1, key0 = (g ? j0 + j - s0 : j0 + j) * BN;
        const int valid = (g ? n1 : n0) - key0;
        const unsigned char *mk = a.c.seg[g].mask;
        const bool part = valid < BN || mk;    // some of its keys do not count: `live` has a bit for each that does
        uint32_t live[(BN + 31) / 32];
        if (part) {
          if (mk) mk += (long long)(g ? it.set1 : it.set0) * a.c.seg[g].L + key0;
#pragma unroll
          for (int i = 0; i < (BN + 31) / 32; ++i)
            live[i] = __ballot_sync(0xffffffffu, 32 * i + lane < valid && (!mk || st::after_wait(mk)[32 * i + lane]));
        }
        if (!(ok = mbar_wait(s_full + X, gs & 1, epoch))) break;
        tc_fence_after();
        uint32_t sr[K::CH][16];
#pragma unroll
        for (int c = 0; c < K::CH; ++c) COND_LD16(tS + c * 16, sr[c]);   // (chunks past the keys hold anything)
        tmem_wait_ld();
        if (part) {
#pragma unroll
          for (int c = 0; c < K::CH; ++c) {
            const uint32_t keep = live[c >> 1] >> ((c & 1) * 16) & 0xffffu;
            if (keep != 0xffffu) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (!(keep >> e & 1)) sr[c][e] = __float_as_uint(-INFINITY);
            }
          }
        }
        float mxp[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mxp[e] = fmax2(__uint_as_float(sr[0][2 * e]), __uint_as_float(sr[0][2 * e + 1]));
#pragma unroll
        for (int c = 1; c < 2 * K::CH; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mxp[e] = fmax3(mxp[e], __uint_as_float(sr[c >> 1][(c & 1) * 8 + 2 * e]),
                           __uint_as_float(sr[c >> 1][(c & 1) * 8 + 2 * e + 1]));
        // A step without any key leaves the row at NO_KEY: its weights are 0.  A NaN
        // score makes the maximum NaN from here on; one of +inf stays the maximum.
        // Either makes the row NaN where O is written.
        const float mx = fmax2(fmax2(fmax3(mxp[0], mxp[1], mxp[2]), mxp[3]) * sl2, NO_KEY);
        if (j == first) {
          m = mx;
        } else {
          const bool need = !(mx <= m + 8.0f);         // (in every step of a NaN row; the test of m for it cost 1.5%)
          if (__any_sync(0xffffffffu, need)) {
            // S(j) complete means PV(j - 1) is (one thread issued both): rescale O in TMEM
            const float corr = need ? ex2_mufu(m - mx) : 1.0f;
            if (need) {
              if (!K::ONES) l *= corr;         // with the ones column the sum is rescaled with O
              m = mx;
            }
#pragma unroll 1
            for (int c = 0; c < K::DPV / 8; ++c) {
              uint32_t ov[8];
              COND_LD8(tO + c * 8, ov);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * corr);
              COND_ST8(tO + c * 8, ov);
            }
            tmem_wait_st();
          }
        }
        const f32x2 negm = pair(-m, -m);
        f32x2 acc[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < K::CH; ++c) {
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const f32x2 xx = ffma2(pair(sr[c][2 * e], sr[c][2 * e + 1]), scale2, negm);
            float2 w;
            if (e < kPolyPairs) {
              w = ex2_poly2(xx);
            } else {
              w = unpair(xx);
              w.x = ex2_mufu(w.x);
              w.y = ex2_mufu(w.y);
            }
            if (!K::ONES) acc[e & 1] = fadd2(acc[e & 1], pair(w.x, w.y));
            // rounded to bf16, the operand of PV (tf32 would halve its rate and double P
            // in TMEM): at most 2^-8 relative, so O is off by at most 2^-8 of the weighted
            // mean of |V| (measured, with O's own rounding: 0.0023 relative, 0.0017 without)
            pk[e] = st::pack_bf16x2(w.x, w.y);
          }
          COND_ST8(tS + c * 8, pk);
        }
        if (!K::ONES) {
          const float2 t = unpair(fadd2(acc[0], acc[1]));
          l += t.x + t.y;
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full + X);
        if (j == first) release_slot();
      }
      if (!ok) break;
      // O of the item: divided by the row sum, written out.  P of the next item
      // follows in this warp, so its PV cannot overwrite O before it is read.
      const bool some = first < n_kv;
      const bool tma = a.tma_out && some;      // (an item without keys has no slot)
      const int row = it.r0 + (spread ? 0 : X * a.tile_rows) + r;   // row of the unit
      const bool valid = r < a.tile_rows && row < a.c.R;
      const int part = spread ? it.split * NT + first : it.split;   // by its steps, whichever tile took them
      float inv = 0.f, lse = -INFINITY;
      uint8_t *stg = sQ + mine * K::QTILE;
      if (some) {
        if (!(ok = mbar_wait(o_full + X, oc & 1, epoch))) break;
        ++oc;
        tc_fence_after();
      }
      // where the row goes without the tiled store
      char *out = nullptr;
      bool f32 = false;
      if (!tma && valid) {
        const long long prow = (long long)part * a.c.part_rows + ((long long)it.unit * a.c.HW + it.w) * a.c.R + row;
        f32 = a.c.part_o || a.c.o_f32;
        out = a.c.part_o ? reinterpret_cast<char *>(a.c.part_o + prow * D)
                         : static_cast<char *>(a.c.o) + st::cond_row<false>(a.c, it.unit, it.w, row) * (f32 ? 4 : 2);
      }
      // O leaves TMEM in groups of chunks of 16 columns, from the last ones
      // (which may hold the row sum)
      constexpr int NCH = (D + 15) / 16, GRP = NCH <= 5 ? NCH : NCH / 2;
      if (some && K::ONES) {
        uint32_t sum[8];                       // the sum of the bf16 weights
        COND_LD8(tO + D, sum);
        tmem_wait_ld();
        l = __uint_as_float(sum[0]);
      }
      if (some && m != NO_KEY) {               // else no key counted: o = 0, lse = -inf
        const float bad = m - m;               // NaN for a maximum of NaN or +inf, else 0
        // (the fast forms: l is at least 1 and below 2^39, where they are off by 2 units and
        // by 2 units or 2^-21.4, far below the weights' rounding)
        inv = __fdividef(1.0f, l) + bad;
        lse = (m + __log2f(l)) * 0.6931471805599453f + bad;
      }
      const f32x2 inv2 = pair(inv, inv);
      if (tma) {
#pragma unroll
        for (int k0 = 0; k0 < NCH; k0 += GRP) {
          uint32_t ov[GRP][16];
#pragma unroll
          for (int i = 0; i < GRP; ++i) COND_LD16(tO + (k0 + i) * 16, ov[i]);
          tmem_wait_ld();
          if (inv == 0.f) {                    // (O of such a row may hold anything)
#pragma unroll
            for (int i = 0; i < GRP; ++i)
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[i][e] = 0;
          }
#pragma unroll
          for (int i = 0; i < 2 * GRP; ++i) {  // 8 columns
            const int f = 2 * k0 + i;
            if (8 * f >= D) continue;
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = (i & 1) * 8 + 2 * e;
              const float2 y = unpair(fmul2(pair(ov[i >> 1][c], ov[i >> 1][c + 1]), inv2));
              v[e] = st::pack_bf16x2(y.x, y.y);
            }
            uint8_t *dst;
            if constexpr (K::DENSE) dst = stg + r * (2 * D) + 16 * f;
            else if (8 * f < K::C0) dst = stg + r * K::SW0 + (swz<K::SW0>(r, f) << 4);
            else dst = stg + K::QT0 + r * K::SW1X + (swz<K::SW1X>(r, f - K::C0 / 8) << 4);
            *reinterpret_cast<uint4 *>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      } else {
#pragma unroll 1
        for (int f = 0; f < D / 8; ++f) {      // fp32 results, parts and packed heads: row by row
          uint32_t ov[8];
          COND_LD8(tO + 8 * f, ov);
          tmem_wait_ld();
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = inv == 0.f ? 0.f : __uint_as_float(ov[e]) * inv;
          if (out && f32) {
            *reinterpret_cast<float4 *>(out + 32 * f) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4 *>(out + 32 * f + 16) = make_float4(y[4], y[5], y[6], y[7]);
          } else if (out) {
            *reinterpret_cast<uint4 *>(out + 16 * f) = make_uint4(st::pack_bf16x2(y[0], y[1]), st::pack_bf16x2(y[2], y[3]),
                                                                  st::pack_bf16x2(y[4], y[5]), st::pack_bf16x2(y[6], y[7]));
          }
        }
      }
      if (some) {
        if (tma) {
          pending = true;
          slot = mine;
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int row0 = it.r0 + X * a.tile_rows + (warp & 3) * 32;
            if (row0 < a.c.R) {
              tma_store_5d(&mp.o0, stg + (warp & 3) * 32 * (K::DENSE ? 2 * D : K::SW0), 0, it.w, row0, it.c3, it.c4);
              if (K::C1 && !K::DENSE) tma_store_5d(&mp.o1, stg + K::QT0 + (warp & 3) * 32 * K::SW1X, 64, it.w, row0, it.c3, it.c4);
            }
            bulk_commit();
          }
        } else if (lane == 0) {
          mbar_arrive(q_empty + mine);         // Q was read, nothing is staged over it
        }
      }
      if (valid) {
        if (a.c.part_o)
          a.c.part_lse[(long long)part * a.c.part_rows + ((long long)it.unit * a.c.HW + it.w) * a.c.R + row] = lse;
        else if (a.c.lse) a.c.lse[st::cond_lse(a.c, it.unit, it.w, row)] = lse;
      }
      rd.done(item_empty, lane);
    }
    if (!ok && lane == 0) gave_up(epoch, 8 + X);
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == K::W_LOAD) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ---------------------------------------------------------------- host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

bool encode(CUtensorMap *m, const void *ptr, int rank, const long long *dims, const long long *strides,
            const int *box, int swizzle_bytes) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t d[5], s[4];
  cuuint32_t b[5], one[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = (cuuint64_t)dims[i];
    b[i] = (cuuint32_t)box[i];
    one[i] = 1;
    if (i) s[i - 1] = (cuuint64_t)strides[i] * 2;
  }
  const CUtensorMapSwizzle sw = swizzle_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                : swizzle_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                : swizzle_bytes == 32 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_NONE;
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(ptr), d, s, b, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Q and O: (d, head, row, frame, block), or with packed heads (d, head of the
// group, group, row, unit).
bool map_q(CUtensorMap *m, const void *ptr, const st::CondParams &p, int box_d, int swizzle, int rows) {
  const Geom &g = p.g;
  const bool blocks = g.tblk != g.T;
  if (p.G > 1) {
    const long long dims[5] = {g.D, p.G, p.HW, p.R0, g.B};
    const long long strides[5] = {1, g.D, (long long)p.G * g.D, g.ss, g.sb};
    const int box[5] = {box_d, p.G, 1, rows / p.G, 1};
    return encode(m, ptr, 5, dims, strides, box, swizzle);
  }
  const long long dims[5] = {g.D, g.H, p.R0, blocks ? g.tblk : g.T, blocks ? (long long)g.B * (g.T / g.tblk) : g.B};
  const long long strides[5] = {1, g.D, g.ss, g.st, blocks ? g.stb : g.sb};
  const int box[5] = {box_d, 1, rows, 1, 1};
  return encode(m, ptr, 5, dims, strides, box, swizzle);
}
bool map_kv(CUtensorMap *m, const void *ptr, const st::CondParams &p, const st::KvSeg &s, int box_d, int swizzle,
            int rows) {
  const int hkv = p.HW / p.hdiv;
  const bool packed = s.offsets != nullptr;
  const long long dims[4] = {p.g.D, hkv, packed ? s.n_rows : s.L, packed ? 1 : s.n_sets};
  const long long strides[4] = {1, p.g.D, s.stride_l, packed ? s.stride_l : s.stride_set};
  const int box[4] = {box_d, 1, rows, 1};
  return encode(m, ptr, 4, dims, strides, box, swizzle);
}

std::atomic<uint32_t> g_epoch{0};

template <int D, bool MIX = false> st_status launch(const st::CondParams &p, cudaStream_t s) {
  using K = Cfg<D, MIX>;
  Args a = {};
  a.c = p;
  a.tile_rows = BLOCK_M / p.G * p.G;
  a.spread = p.spread > 1 ? 1 : 0;
  a.n_split = p.n_split / p.spread;
  a.q_blocks = (p.R + K::NT * a.tile_rows - 1) / (K::NT * a.tile_rows);
  const long long items = (long long)st::cond_units(p) * p.HW * a.n_split * a.q_blocks;
  if (items > 0x3fffffffLL) return ST_ERR_SHAPE;
  a.n_items = int(items);
  a.dqb = st::make_fastdiv(uint32_t(a.q_blocks));
  a.dsplit = st::make_fastdiv(uint32_t(a.n_split));
  a.dhw = st::make_fastdiv(uint32_t(p.HW));
  a.dkv = st::make_fastdiv(uint32_t(p.hdiv));
  a.dt = st::make_fastdiv(uint32_t(p.g.T));
  a.dtblk = st::make_fastdiv(uint32_t(p.g.tblk));
  a.n_tblk = p.g.T / p.g.tblk;
  long long steps = 0;
  Maps m;
  memset(&m, 0, sizeof(m));
  for (int g = 0; g < p.n_seg; ++g) {
    const st::KvSeg &sg = p.seg[g];
    a.dper[g] = st::make_fastdiv(uint32_t(sg.per));
    steps += (sg.L + K::BN - 1) / K::BN;
    if (!sg.L) continue;                       // no keys: never loaded
    if (!map_kv(&m.k0[g], sg.k, p, sg, K::C0, K::SW0, K::BN) ||
        (K::C1 && !map_kv(&m.k1[g], sg.k, p, sg, K::C1X, K::SW1X, K::BN)) ||
        !map_kv(&m.v[g], sg.v, p, sg, K::VW, K::VSW, K::BN) ||
        (MIX && !map_kv(&m.vr[g], sg.v, p, sg, K::VRX, K::VSWR, K::BN)))
      return ST_ERR_CUDA;
  }
  if (steps * (a.n_split + 1) >= (1LL << 31)) return ST_ERR_SHAPE;
  a.max_steps = int(steps);
  a.nq = K::TIGHT ? K::NQ - (steps > 1) : (a.spread ? K::NT : K::NQ);
  a.ns = K::stages(a.nq);
  a.dns = st::make_fastdiv(uint32_t(a.ns));
  a.resident = p.n_split == 1 && steps <= a.ns ? 1 : 0;
  a.tma_out = !p.part_o && !p.o_f32 && p.G == 1 ? 1 : 0;
  if (!map_q(&m.q0, p.q, p, K::C0, K::SW0, a.tile_rows) ||
      (K::C1 && !map_q(&m.q1, p.q, p, K::C1X, K::SW1X, a.tile_rows)) ||
      (a.tma_out && (!map_q(&m.o0, p.o, p, K::DENSE ? D : K::C0, K::DENSE ? 0 : K::SW0, 32) ||
                     (K::C1 && !K::DENSE && !map_q(&m.o1, p.o, p, K::C1X, K::SW1X, 32)))))
    return ST_ERR_CUDA;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.epoch = g_epoch.fetch_add(1) + 1;
  const int ctas = int(items < st::num_sms() ? items : st::num_sms());
  if (a.resident) {
    // bands of one CTA each if that keeps the longest CTA as short as an even
    // share of the items does, else bands of about that share, which a CTA may
    // begin or end within
    a.cols = st::cond_units(p) * p.HW;
    const int share = (a.n_items + ctas - 1) / ctas;
    for (int g = 0; g < p.n_seg; ++g) a.weighed |= p.seg[g].n_sets > 1 && (p.seg[g].len || p.seg[g].offsets);
    a.weighed = a.weighed && st::cond_units(p) <= WEIGHED && a.n_items >= 4 * ctas;
    const int whole = a.cols <= ctas && !a.weighed ? (a.q_blocks + ctas / a.cols - 1) / (ctas / a.cols) : a.q_blocks + 1;
    a.band = whole <= share ? whole : (share < a.q_blocks ? share : a.q_blocks);
    a.n_bands = (a.q_blocks + a.band - 1) / a.band;
    a.band_last = a.q_blocks - (a.n_bands - 1) * a.band;
    a.dband = st::make_fastdiv(uint32_t(a.band));
    a.dband_last = st::make_fastdiv(uint32_t(a.band_last));
    a.dbandcols = st::make_fastdiv(uint32_t(a.band) * uint32_t(a.cols));
  }
  auto kern = cond_attn_sm100<D, MIX>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, K::SMEM) != cudaSuccess)
    return ST_ERR_CUDA;
  // A build that grants fewer registers than the split assumes would wait in
  // setmaxnreg forever: refuse it.
  static int regs_ok = -1;
  if (regs_ok < 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return ST_ERR_CUDA;
    regs_ok = fa.numRegs * K::THREADS >= 128 * K::NT * K::R_SOFT + 32 * K::MISC * K::R_MISC ? 1 : 0;
  }
  if (!regs_ok) return ST_ERR_UNSUPPORTED;
  return st::launch_pdl(kern, dim3(ctas), dim3(K::THREADS), K::SMEM, s, m, a);
}

template <int D> st::CondTile tile_of() { return {BLOCK_M, Cfg<D>::NT, Cfg<D>::BN}; }

}  // namespace

namespace st {

unsigned int read_and_clear_cond_error(cudaStream_t stream, cudaError_t *err) {
  unsigned int word = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&word, g_cond_error, sizeof(word), 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(g_cond_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(g_cond_abort_epoch, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (err) *err = e;
  return word;
}

CondTile cond_tile(int D) {
  switch (D) {
    case 32: return tile_of<32>();
    case 64: return tile_of<64>();
    case 72: return tile_of<72>();
    case 80: return tile_of<80>();
    case 96: return tile_of<96>();
    default: return tile_of<128>();
  }
}

st_status cond_sm100(const CondParams &p, cudaStream_t s) {
  switch (p.g.D) {
    case 32: return launch<32>(p, s);
    case 64: return launch<64>(p, s);
    case 72: return p.spread > 1 ? launch<72, true>(p, s) : launch<72>(p, s);
    case 80: return p.spread > 1 ? launch<80, true>(p, s) : launch<80>(p, s);
    case 96: return p.spread > 1 ? launch<96, true>(p, s) : launch<96>(p, s);
    case 128: return launch<128>(p, s);
  }
  return ST_ERR_UNSUPPORTED;
}

}  // namespace st
