// Conditioning attention on the sm_100a tensor cores (tcgen05 + TMEM + TMA).
//
//   O = softmax(Q K^T * scale) V over the keys of up to two segments (prefix,
//   own keys), each of its own length, with lengths, packed sets and key
//   masks read on the device.
//
// What bounds it.  The keys of a text prompt are few, so an item is short: at
// head dim 72 a 128 x 64 step is about 420 cycles of tensor work (S with
// both operands in shared memory, PV with P in TMEM) against 512 cycles of
// special-function unit for its exponentials, and below about 190 keys reading
// Q and writing O takes longer than either.  The chain S -> softmax -> PV -> S
// of one tile leaves every unit idle most of the time, so several row tiles run
// side by side, each with its own chain.
//
// Design (one persistent CTA per SM, warp-specialised):
//   * A work item is up to NT tiles of 128 rows of one (unit, head): three for
//     head dims up to 96, whose S (64 keys) and O fit three times into the 512
//     TMEM columns, two (128 keys per step) for 128.  A spatial kernel of two
//     tiles with S double-buffered has the same number of scores in flight
//     but two softmax warps per sub-partition; three warps hide more of each
//     other's TMEM loads and barrier waits.
//   * Each tile has one issuer thread.  S(j + 1) follows PV(j) in program order
//     into the same TMEM columns (MMAs of one thread execute in order), so the
//     chain has two hand-overs a step: S ready, P ready.
//   * When every key tile of a launch fits the K/V ring, a CTA walks
//     consecutive items and keeps K and V in shared memory until the set or the
//     head changes; otherwise they stream through the ring.
//   * One warp per V stage clears the rows of keys that do not count (which may
//     hold NaN: 0 * NaN would reach O) and, where the head dim is padded, sets
//     column D to 1 so that PV adds up the rounded weights.
//   * Softmax: one thread per row, running max raised (and O rescaled in TMEM)
//     only when it grows by more than 2^8; exponentials on the special-function
//     unit with every fourth pair on the FMA pipe.
//   * The epilogue warps divide O by the row sum and write it with bulk tensor
//     stores, or row by row (fp32 partials, heads packed into rows).
//   * Every wait is bounded; a wait that runs out sets an error word and an
//     abort epoch, in-flight copies are drained, TMEM is freed.
#include <cuda.h>
#include <math.h>
#include <string.h>

#include <atomic>
#include <mutex>

#include "cond.cuh"

namespace {

using st::Geom;
using st::pdl_trigger;
using st::pdl_wait;

__device__ unsigned int g_cond_error;        // sites of waits that ran out
__device__ unsigned int g_cond_abort_epoch;  // launch epoch that must abort

constexpr int BLOCK_M = 128;
constexpr unsigned long long WAIT_NS = 2000000000ull;  // 2 s per wait
constexpr int SET_TABLE = 64;                // key ranges of a segment held in shared memory
constexpr float NO_KEY = -3.0e38f;           // running max of a row no key counted for yet

template <int D> struct Cfg {
  static constexpr int NT = D <= 96 ? 3 : 2;           // row tiles in flight
  static constexpr int BN = D <= 96 ? 64 : 128;        // keys per step
  static constexpr int C0 = D >= 64 ? 64 : 32;
  static constexpr int R1 = D > 64 ? D - 64 : 0;
  static constexpr int C1 = R1 == 0 ? 0 : (R1 <= 16 ? 16 : (R1 <= 32 ? 32 : 64));
  static constexpr int C1X = C1 ? C1 : 16;
  static constexpr int SW0 = C0 * 2, SW1 = C1 * 2, SW1X = C1X * 2;
  static constexpr int QT0 = BLOCK_M * SW0;
  static constexpr int QTILE = QT0 + BLOCK_M * SW1;
  static constexpr int KT0 = BN * SW0;
  static constexpr int KTILE = KT0 + BN * SW1;
  // V as column atoms of VW elements (MN-major), PV one MMA of N = DPV per 16 keys
  static constexpr int VW = (D == 72 || D == 80) ? 16 : ((D == 96 || D == 32) ? 32 : 64);
  static constexpr int DPV = ((D + VW - 1) / VW) * VW;
  static constexpr int VA = DPV / VW, VSW = VW * 2, VAT = BN * VSW, VTILE = VA * VAT;
  static constexpr bool ONES = DPV > D;
  static constexpr int TW = BN + DPV;                  // TMEM columns of a tile: S (P over it), O
  static_assert(NT * TW <= 512, "TMEM");
  // Q tiles: QB slots per row tile, its own so that its issuer sees every phase
  static constexpr int QB = D == 32 ? 2 : 1, NQ = NT * QB;
  // staging of a warp's 32 rows of O, a 128-byte chunk at a time for head dim 128
  static constexpr int STG = 32 * (D == 128 ? SW0 : SW0 + SW1);
  static constexpr int NSTG = NT;                      // one per tile
  static constexpr int TAIL = 4 * NSTG * STG + 2 * SET_TABLE * 8 + 512 + (NT == 3 ? 1024 : 512);   // + items, barriers
  static constexpr int NS_RAW = (232448 - 1024 - TAIL - NQ * QTILE) / (KTILE + VTILE);
  static constexpr int NS = NS_RAW > 8 ? 8 : NS_RAW;   // K/V stages
  static constexpr int SMEM = 1024 + NQ * QTILE + NS * (KTILE + VTILE) + TAIL;
  static_assert(SMEM <= 232448 && NS >= 2, "shared memory");
  // warps: softmax and epilogue of the tiles (4 each), then loader, issuers, V
  // helper, scheduler; the rest of the last two warpgroups idles
  static constexpr int W_LOAD = 4 * NT, W_MMA = W_LOAD + 1, W_FIX = W_MMA + NT, W_SCHED = W_FIX + 1;
  static constexpr int THREADS = 32 * (W_LOAD + 8);
  // registers: granted at launch, then moved to the softmax (setmaxnreg)
  static constexpr int R_LAUNCH = NT == 3 ? 96 : 128;
  static constexpr int R_SOFT = NT == 3 ? 120 : 200, R_MISC = 56;
  static_assert(128 * NT * R_SOFT + 256 * R_MISC <= THREADS * R_LAUNCH, "register split");
};

// ---------------------------------------------------------------- exp2
__device__ __forceinline__ float ex2_mufu(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^x on the FMA pipe for x <= 8: the degree-3 polynomial of the spatial
// kernel (fit_exp2_poly.py; max relative error 7.5e-5), clamped at 2^-125.
constexpr float kP0 = 0.9999280571937561f, kP1 = 0.6932609677314758f;
constexpr float kP2 = 0.2426111251115799f, kP3 = 0.0551716685295105f;
constexpr int kPolyPairs = 2;                // of every 8 pairs of scores

__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float2 ex2_poly2(float2 x) {
  x.x = fmaxf(x.x, -125.0f);
  x.y = fmaxf(x.y, -125.0f);
  const float2 t = fadd2(x, make_float2(12582912.0f, 12582912.0f));
  const float2 j = fadd2(t, make_float2(-12582912.0f, -12582912.0f));
  const float2 f = ffma2(j, make_float2(-1.0f, -1.0f), x);
  float2 q = ffma2(make_float2(kP3, kP3), f, make_float2(kP2, kP2));
  q = ffma2(q, f, make_float2(kP1, kP1));
  q = ffma2(q, f, make_float2(kP0, kP0));
  return make_float2(__int_as_float(__float_as_int(q.x) + (__float_as_int(t.x) << 23)),
                     __int_as_float(__float_as_int(q.y) + (__float_as_int(t.y) << 23)));
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
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// try_wait that suspends the thread until the phase completes or about
// `hint_ns` nanoseconds pass.
__device__ __forceinline__ bool mbar_try_wait(uint64_t *bar, uint32_t parity, uint32_t hint_ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(hint_ns)
      : "memory");
  return ok != 0;
}
// Bounded wait for a phase by one thread: it sleeps in the barrier; the clock
// and the abort epoch are only consulted after a sleep of ~0.1 ms that ended
// without the phase.
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, uint32_t epoch, int site) {
  if (mbar_test(bar, parity)) return true;
  const unsigned long long t0 = globaltimer();
  while (true) {
    if (mbar_try_wait(bar, parity, 100000u)) return true;
    if (*reinterpret_cast<volatile unsigned int *>(&g_cond_abort_epoch) == epoch) return false;
    if (globaltimer() - t0 > WAIT_NS) {
      atomicOr(&g_cond_error, 1u << (site & 31));
      atomicExch(&g_cond_abort_epoch, epoch);
      return false;
    }
  }
}
// The same by a whole warp, whose lanes agree on the answer (a warp that
// gives up does so in all lanes).  SPIN polls come first: a polling warp
// resumes sooner than a suspended one, which the MMA chain notices.
template <int SPIN = 0>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint32_t epoch, int site) {
  for (int i = 0; i <= SPIN; ++i)
    if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  const unsigned long long t0 = globaltimer();
  while (true) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity, 100000u))) return true;
    bool stop = *reinterpret_cast<volatile unsigned int *>(&g_cond_abort_epoch) == epoch;
    if (globaltimer() - t0 > WAIT_NS) {
      atomicOr(&g_cond_error, 1u << (site & 31));
      atomicExch(&g_cond_abort_epoch, epoch);
      stop = true;
    }
    if (__any_sync(0xffffffffu, stop)) return false;
  }
}
// The same for the end of work already issued, whatever the abort epoch.
__device__ __forceinline__ void mbar_drain(uint64_t *bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer();
  while (!mbar_try_wait(bar, parity, 100000u) && globaltimer() - t0 < WAIT_NS) {
  }
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
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}
// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
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
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor: start address, leading and stride byte
// offsets, version 1, swizzle layout 2 = 128B, 4 = 64B, 6 = 32B.
template <uint32_t LBO, uint32_t SBO, uint32_t LAYOUT>
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr) {
  constexpr uint32_t hi = ((SBO >> 4) & 0x3FFFu) | (1u << 14) | (LAYOUT << 29);
  constexpr uint32_t lo = ((LBO >> 4) & 0x3FFFu) << 16;
  return ((uint64_t)hi << 32) | (uint64_t)(((saddr >> 4) & 0x3FFFu) | lo);
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
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok));
  return ok != 0;
}
// 16-byte chunk f of row r of a swizzled tile with rows of `bytes`.
template <int BYTES> __device__ __forceinline__ int swz(int r, int f) {
  return f ^ (BYTES == 128 ? (r & 7) : (BYTES == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1)));
}

// ---------------------------------------------------------------- work items
struct Maps {
  CUtensorMap q0, q1;          // the head's first C0 channels, the rest
  CUtensorMap k0[2], k1[2], v[2];
  CUtensorMap o0, o1;
};

struct Args {
  st::CondParams c;
  st::FastDiv dqb, dsplit, dhw, dkv, dt, dper[2];
  int q_blocks, tile_rows;     // row blocks of a unit, rows of a tile (128, or whole groups of heads)
  int n_items;
  int resident;                // every key tile of an item fits the ring: K and V stay from item to item
  int max_steps;
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
  int qb;                      // row block of the unit
  int pad[4];
};
constexpr int ITEMS = 4;       // items in flight between the scheduler and the others
static_assert(ITEMS * sizeof(Item) <= 512, "item ring");

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
  it.n_qt = left > 2 * a.tile_rows && Cfg<D>::NT > 2 ? 3 : (left > a.tile_rows ? 2 : 1);
}

// q block fastest, then split, head, unit.  table: the segments' key ranges (row, n).
template <int D>
__device__ __forceinline__ Item decode(const Args &a, const int2 *table, int x) {
  using K = Cfg<D>;
  Item it;
  const uint32_t y = st::fdiv(uint32_t(x), a.dqb);
  it.qb = x - int(y) * a.q_blocks;
  const uint32_t z = st::fdiv(y, a.dsplit);
  it.split = int(y) - int(z) * a.c.n_split;
  it.unit = int(st::fdiv(z, a.dhw));
  it.w = int(z) - it.unit * a.c.HW;
  it.kvh = int(st::fdiv(uint32_t(it.w), a.dkv));
  rows_of<D>(a, it);
  const int ub = int(st::fdiv(uint32_t(it.unit), a.dt)), t = it.unit - ub * a.c.g.T;
  if (a.c.g.tblk != a.c.g.T) {
    it.c3 = t % a.c.g.tblk;
    it.c4 = ub * (a.c.g.T / a.c.g.tblk) + t / a.c.g.tblk;
  } else {
    it.c3 = t;
    it.c4 = ub;
  }
  const int b = ub * a.c.bm;
  auto range = [&](int g, int &set, int &row, int &n) {
    set = row = n = 0;
    if (g >= a.c.n_seg) return;
    set = int(st::fdiv(uint32_t(b), a.dper[g]));
    if (a.c.seg[g].n_sets <= SET_TABLE) {
      const int2 r = table[g * SET_TABLE + set];
      row = r.x;
      n = r.y;
    } else {
      const st::KvRange r = st::kv_range(a.c.seg[g], b);
      row = r.row0;
      n = r.n;
    }
  };
  range(0, it.set0, it.row0, it.n0);
  range(1, it.set1, it.row1, it.n1);
  it.s0 = (it.n0 + K::BN - 1) / K::BN;
  const int total = it.s0 + (it.n1 + K::BN - 1) / K::BN;
  if (a.c.n_split == 1) {
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

// The items of a CTA: consecutive ones when K and V stay resident, else every
// gridDim-th, so that the CTAs that run together share K/V tiles in L2.  The
// next row block of the same keys needs no division.
template <int D> struct Walk {
  int x, end, inc;
  __device__ __forceinline__ explicit Walk(const Args &a) {
    if (a.resident) {
      x = int((long long)a.n_items * blockIdx.x / gridDim.x);
      end = int((long long)a.n_items * (blockIdx.x + 1) / gridDim.x);
      inc = 1;
    } else {
      x = blockIdx.x;
      end = a.n_items;
      inc = gridDim.x;
    }
  }
  __device__ __forceinline__ Item after(const Args &a, const int2 *table, const Item &it) const {
    Item nx = it;
    if (x + inc >= end) {
      nx.n_qt = 0;
    } else if (inc == 1 && it.qb + 1 < a.q_blocks) {
      ++nx.qb;
      rows_of<D>(a, nx);
    } else {
      nx = decode<D>(a, table, x + inc);
    }
    nx.fresh = !same_keys(it, nx);
    return nx;
  }
};

// A reader's place in the ring of items.
struct Reader {
  uint32_t i = 0;
  // The next item, once it is there: the caller reads what it needs, then the
  // warp hands it back.
  template <int SPIN>
  __device__ __forceinline__ const Item *get(const Item *items, uint64_t *full, uint32_t epoch, int site) const {
    return warp_wait<SPIN>(full + i % ITEMS, (i / ITEMS) & 1, epoch, site) ? items + i % ITEMS : nullptr;
  }
  __device__ __forceinline__ void done(uint64_t *empty, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + i % ITEMS);
    ++i;
  }
};

// Position of the K/V ring: streaming, steps follow one another; resident,
// step j is in stage j and `run` counts the loads of each.
template <int NS> struct Ring {
  uint32_t pos = 0, run = 0;
  __device__ __forceinline__ int stage(bool resident, int j) const { return resident ? j : int((pos + j) % NS); }
  __device__ __forceinline__ uint32_t phase(bool resident, int j) const {
    return (resident ? run : (pos + j) / NS) & 1;
  }
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::THREADS, 1)
    cond_attn_sm100(const __grid_constant__ Maps mp, const __grid_constant__ Args a) {
  using K = Cfg<D>;
  constexpr int NT = K::NT, NS = K::NS, NQ = K::NQ, QB = K::QB, BN = K::BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sQ = base;
  uint8_t *sK = sQ + NQ * K::QTILE;
  uint8_t *sV = sK + NS * K::KTILE;
  uint8_t *sStg = sV + NS * K::VTILE;
  int2 *sSet = reinterpret_cast<int2 *>(sStg + 4 * K::NSTG * K::STG);
  Item *sItem = reinterpret_cast<Item *>(sSet + 2 * SET_TABLE);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sItem + ITEMS);
  uint64_t *q_full = bars, *q_empty = q_full + NQ;
  uint64_t *k_full = q_empty + NQ, *k_empty = k_full + NS;       // k_empty, v_empty: one arrival per tile
  uint64_t *v_full = k_empty + NS, *v_empty = v_full + NS, *v_ready = v_empty + NS;
  uint64_t *s_full = v_ready + NS, *p_full = s_full + NT;
  uint64_t *o_full = p_full + NT, *mma_done = o_full + NT;
  uint64_t *item_full = mma_done + NT, *item_empty = item_full + ITEMS;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(item_empty + ITEMS);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NQ; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, NT);
      mbar_init(v_full + i, 1);
      mbar_init(v_empty + i, NT);
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
      mbar_init(item_empty + i, 5 * NT + 2);   // softmax warps, issuers, loader, helper
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == K::W_LOAD) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // barriers and TMEM are set up: let the next kernel of the stream be
  // scheduled, then wait for the previous one before any global access
  pdl_trigger();
  pdl_wait();
#pragma unroll
  for (int g = 0; g < 2; ++g)
    if (g < a.c.n_seg && a.c.seg[g].n_sets <= SET_TABLE && int(threadIdx.x) < a.c.seg[g].n_sets) {
      st::KvSeg sg = a.c.seg[g];
      sg.len = st::after_wait(sg.len);
      sg.offsets = st::after_wait(sg.offsets);
      const st::KvRange r = st::kv_range(sg, int(threadIdx.x) * sg.per);
      sSet[g * SET_TABLE + threadIdx.x] = make_int2(r.row0, r.n);
    }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t epoch = a.epoch;
  const bool resident = a.resident != 0;

  if (warp >= K::W_LOAD) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(K::R_MISC));
    if (warp == K::W_LOAD) {
      // ================= TMA producer =================
      bool ok = true;
      Ring<NS> ring;
      Reader rd;
      uint32_t qc[NT];                                // Q tiles so far
#pragma unroll
      for (int X = 0; X < NT; ++X) qc[X] = 0;
      int last_kv = -1;                               // streaming: ring position of the last K/V issued
      int loaded = 0;                                 // resident: stages loaded in this run
      bool first = true;
      while (ok) {
        const Item *ip = rd.get<0>(sItem, item_full, epoch, 15);
        if (!(ok = ip != nullptr)) break;
        const Item it = *ip;
        rd.done(item_empty, lane);
        if (it.n_qt == 0) break;
        if (lane == 0) {
          const bool load_kv = !resident || it.fresh;
          if (resident && load_kv && !first) ++ring.run;
          first = false;
          const int n = resident ? (load_kv ? a.max_steps : 1) : it.n_kv;
          for (int j = 0; j < n && ok; ++j) {
            const int st = ring.stage(resident, j);
            const uint32_t ph = ring.phase(resident, j);
            const Step sp = step_of<BN>(it, j);
            const int g = sp.seg;
            const int set = a.c.seg[g].offsets ? 0 : sp.set;   // packed: rows of one long sequence
            const bool real = j < it.n_kv;            // resident: stages past the item's steps only change phase
            if (load_kv) {
              if (!(ok = mbar_wait(k_empty + st, ph ^ 1, epoch, 1))) break;
              if (real) {
                mbar_expect_tx(k_full + st, K::KTILE);
                uint8_t *dk = sK + st * K::KTILE;
                tma_load_4d(dk, &mp.k0[g], k_full + st, 0, it.kvh, sp.row + sp.key, set);
                if (K::C1) tma_load_4d(dk + K::KT0, &mp.k1[g], k_full + st, 64, it.kvh, sp.row + sp.key, set);
                if (!resident) last_kv = int(ring.pos) + j;
                else loaded = j + 1;
              } else {
                mbar_arrive(k_full + st);
              }
            }
            if (j == 0 && it.n_kv > 0) {
#pragma unroll
              for (int X = 0; X < NT; ++X) {
                if (X >= it.n_qt || !ok) continue;
                const int qs = X * QB + qc[X] % QB;
                if (!(ok = mbar_wait(q_empty + qs, ((qc[X] / QB) & 1) ^ 1, epoch, 0))) continue;
                ++qc[X];
                uint8_t *dst = sQ + qs * K::QTILE;
                const int row = it.r0 + X * a.tile_rows;
                mbar_expect_tx(q_full + qs, a.tile_rows * (K::SW0 + K::SW1));
                if (a.c.G > 1) {
                  tma_load_5d(dst, &mp.q0, q_full + qs, 0, 0, it.w, row / a.c.G, it.unit);
                  if (K::C1) tma_load_5d(dst + K::QT0, &mp.q1, q_full + qs, 64, 0, it.w, row / a.c.G, it.unit);
                } else {
                  tma_load_5d(dst, &mp.q0, q_full + qs, 0, it.w, row, it.c3, it.c4);
                  if (K::C1) tma_load_5d(dst + K::QT0, &mp.q1, q_full + qs, 64, it.w, row, it.c3, it.c4);
                }
              }
              if (!ok) break;
            }
            if (load_kv) {
              if (!(ok = mbar_wait(v_empty + st, ph ^ 1, epoch, 2))) break;
              if (real) {
                mbar_expect_tx(v_full + st, K::VTILE);
                uint8_t *dv = sV + st * K::VTILE;
#pragma unroll
                for (int t = 0; t < K::VA; ++t)
                  tma_load_4d(dv + t * K::VAT, &mp.v[g], v_full + st, t * K::VW, it.kvh, sp.row + sp.key, set);
              } else {
                mbar_arrive(v_full + st);
              }
            }
          }
          if (!resident) ring.pos += it.n_kv;
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      if (!ok && lane == 0) {
        // the last load issued into every stage and Q slot (a wait for one
        // that was not issued runs into its limit)
        if (resident) {
          for (int j = 0; j < loaded; ++j) {
            mbar_drain(k_full + j, ring.run & 1);
            mbar_drain(v_full + j, ring.run & 1);
          }
        } else {
          for (int i = (last_kv - NS + 1 > 0 ? last_kv - NS + 1 : 0); i <= last_kv; ++i) {
            mbar_drain(k_full + i % NS, (i / NS) & 1);
            mbar_drain(v_full + i % NS, (i / NS) & 1);
          }
        }
#pragma unroll
        for (int X = 0; X < NT; ++X)
          for (int i = (int(qc[X]) > QB ? int(qc[X]) - QB : 0); i < int(qc[X]); ++i)
            mbar_drain(q_full + X * QB + i % QB, (i / QB) & 1);
      }
      __syncwarp();
    } else if (warp >= K::W_MMA && warp < K::W_MMA + NT) {
      // ================= issuer of tile X =================
      // P of a step ready -> its PV, then S of the next step (of the next item
      // after the last) into the same columns.  The whole warp walks the loop
      // and one elected lane issues, so addresses and descriptors stay in
      // uniform registers: computed by one diverged lane, an MMA took about 200
      // cycles to issue.
      const int X = uniform(warp) - K::W_MMA;
      constexpr uint32_t IDS = idesc_bf16(BLOCK_M, BN, 0, 0), IDPV = idesc_bf16(BLOCK_M, K::DPV, 0, 1);
      const uint32_t aQ = smem_u32(sQ), aK = smem_u32(sK), aV = smem_u32(sV);
      const uint32_t dS = uniform(tmem) + X * K::TW, dO = dS + BN;
      const bool leader = elect_one();
      bool ok = true;
      Ring<NS> ring;
      Reader rd;
      uint32_t qc = 0, steps = 0;                      // items and steps of this tile
      auto issue_s = [&](uint32_t qs, int st) {        // Q in slot qs, K in stage st
        const uint32_t qa = aQ + qs * K::QTILE, ka = aK + st * K::KTILE;
#pragma unroll
        for (int kk = 0; kk < K::C0 / 16; ++kk)
          mma_ss(dS, sdesc<16, 8 * K::SW0, layout_of(K::SW0)>(qa + kk * 32),
                 sdesc<16, 8 * K::SW0, layout_of(K::SW0)>(ka + kk * 32), IDS, kk > 0);
        if (K::C1) {
#pragma unroll
          for (int kk = 0; kk < K::C1X / 16; ++kk)
            mma_ss(dS, sdesc<16, 8 * K::SW1X, layout_of(K::SW1X)>(qa + K::QT0 + kk * 32),
                   sdesc<16, 8 * K::SW1X, layout_of(K::SW1X)>(ka + K::KT0 + kk * 32), IDS, 1);
        }
        tc_commit(s_full + X);
      };
      int n = 0, n_qt = 0;
      bool fresh = false, release = false;
      auto fetch = [&]() -> bool {                     // the next item into n, n_qt, fresh, release
        const Item *ip = rd.get<32>(sItem, item_full, epoch, 15);
        if (!ip) return false;
        n_qt = uniform(ip->n_qt);
        n = uniform(ip->n_kv);
        fresh = !resident || uniform(ip->fresh);
        release = !resident || uniform(ip->release);
        rd.done(item_empty, lane);
        return true;
      };
      // S of an item's first step: waits for its Q, and its K if new
      auto first_s = [&](const Ring<NS> &rg) -> bool {
        const uint32_t qs = X * QB + qc % QB;
        const int st = rg.stage(resident, 0);
        if (!warp_wait<32>(q_full + qs, (qc / QB) & 1, epoch, 3)) return false;
        if (fresh && !warp_wait<32>(k_full + st, rg.phase(resident, 0), epoch, 4)) return false;
        tc_fence_after();
        if (leader) {
          issue_s(qs, st);
          // the stage is handed back at the last item that reads it
          if (release) tc_commit(k_empty + st);
          if (n == 1) tc_commit(q_empty + qs);
        }
        __syncwarp();
        return true;
      };
      bool primed = false;                             // S of the item's first step is issued
      ok = fetch();
      while (ok && n_qt > 0) {
        const int cn = n;
        const bool cfresh = fresh, crel = release, here = X < n_qt && n > 0;
        if (here && !primed && !(ok = first_s(ring))) break;
        primed = false;
        const uint32_t qs = X * QB + qc % QB;
        if (here) ++qc;
        Ring<NS> next_ring = ring;                     // position of the next item
        if (resident) next_ring.run += crel;
        else next_ring.pos += cn;
        if (here) {
          for (int j = 0; j < cn; ++j, ++steps) {
            const bool more = j + 1 < cn;
            const int st = ring.stage(resident, j), st1 = ring.stage(resident, j + 1);
            if (cfresh) {
              if (!(ok = warp_wait<32>(v_ready + st, ring.phase(resident, j), epoch, 5))) break;
              if (more && !(ok = warp_wait<32>(k_full + st1, ring.phase(resident, j + 1), epoch, 4))) break;
            }
            if (!more && !(ok = fetch())) break;       // n, n_qt, fresh, release: now the next item's
            if (!(ok = warp_wait<32>(p_full + X, steps & 1, epoch, 7))) break;
            tc_fence_after();
            if (leader) {
              const uint32_t va = aV + st * K::VTILE;
#pragma unroll
              for (int kk = 0; kk < BN / 16; ++kk)
                mma_ts(dO, dS + kk * 8, sdesc<K::VAT, 8 * K::VSW, layout_of(K::VSW)>(va + kk * 16 * K::VSW), IDPV,
                       (j > 0 || kk > 0) ? 1u : 0u);
              if (more) {
                issue_s(qs, st1);                      // over P(j), which PV(j) has read by then
                if (crel) {
                  tc_commit(v_empty + st);
                  tc_commit(k_empty + st1);
                }
                if (j + 2 == cn) tc_commit(q_empty + qs);
              } else {
                tc_commit(o_full + X);
                if (crel) tc_commit(v_empty + st);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          // straight on to the next item
          if (X < n_qt && n > 0) {
            if (!(ok = first_s(next_ring))) break;
            primed = true;
          }
        }
        // stages this tile did not use in this item: hand them back once they
        // were filled (a commit: earlier items of the run may still read them)
        if (crel) {
          const int last = resident ? a.max_steps : cn;
          for (int j = here ? cn : 0; j < last && ok; ++j) {
            const int st = ring.stage(resident, j);
            const uint32_t ph = ring.phase(resident, j);
            if (!(ok = warp_wait(k_full + st, ph, epoch, 8))) break;
            if (!(ok = warp_wait(v_ready + st, ph, epoch, 9))) break;
            if (leader) {
              tc_commit(k_empty + st);
              tc_commit(v_empty + st);
            }
            __syncwarp();
          }
        }
        if (!here && ok) ok = fetch();
        ring = next_ring;
      }
      // every MMA issued completes before TMEM is released
      __syncwarp();
      if (leader) {
        tc_commit(mma_done + X);
        mbar_drain(mma_done + X, 0);
      }
      __syncwarp();
    } else if (warp == K::W_SCHED) {
      // ================= scheduler =================
      if (lane == 0) {
        Walk<D> wk(a);
        Item it;
        if (wk.x < wk.end) it = decode<D>(a, sSet, wk.x);
        else it.n_qt = 0;
        it.fresh = 1;
        for (uint32_t i = 0;; ++i) {
          Item nx = it;
          if (it.n_qt > 0) nx = wk.after(a, sSet, it);
          it.release = it.n_qt > 0 && (nx.n_qt == 0 || nx.fresh);
          if (!mbar_wait(item_empty + i % ITEMS, ((i / ITEMS) & 1) ^ 1, epoch, 16)) break;
          sItem[i % ITEMS] = it;
          mbar_arrive(item_full + i % ITEMS);
          if (it.n_qt == 0) break;
          it = nx;
          wk.x += wk.inc;
        }
      }
      __syncwarp();
    } else if (warp == K::W_FIX) {
      // ================= V rows of keys that do not count; ones column =================
      constexpr int A1 = K::ONES ? D / K::VW : 0, XB = (D % K::VW) * 2;
      bool ok = true;
      Ring<NS> ring;
      Reader rd;
      bool first = true;
      while (ok) {
        const Item *ip = rd.get<0>(sItem, item_full, epoch, 15);
        if (!ip) break;
        const Item it = *ip;
        rd.done(item_empty, lane);
        if (it.n_qt == 0) break;
        if (resident && !it.fresh) continue;
        if (resident && !first) ++ring.run;
        first = false;
        const int n = resident ? a.max_steps : it.n_kv;
        for (int j = 0; j < n; ++j) {
          const int st = ring.stage(resident, j);
          const uint32_t ph = ring.phase(resident, j);
          const Step sp = step_of<BN>(it, j);
          const unsigned char *mk = a.c.seg[sp.seg].mask;
          const bool work = j < it.n_kv && (K::ONES || sp.valid < BN || mk);
          bool keep[BN / 32];
          if (work) {                          // before the wait: the mask bytes are on their way
            if (mk) mk += (long long)sp.set * a.c.seg[sp.seg].L + sp.key;
#pragma unroll
            for (int i = 0; i < BN / 32; ++i) {
              const int r = lane + 32 * i;
              keep[i] = r < sp.valid && (!mk || st::after_wait(mk)[r]);
            }
          }
          if (lane == 0) ok = mbar_wait(v_full + st, ph, epoch, 10);
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          if (work) {
            uint8_t *vt = sV + st * K::VTILE;
#pragma unroll
            for (int i = 0; i < BN / 32; ++i) {
              const int r = lane + 32 * i;
              if (!keep[i]) {
                for (int t = 0; t < K::VA; ++t)
#pragma unroll
                  for (int f = 0; f < K::VSW / 16; ++f)
                    *reinterpret_cast<uint4 *>(vt + t * K::VAT + r * K::VSW + f * 16) = make_uint4(0, 0, 0, 0);
              } else if (K::ONES) {
                *reinterpret_cast<uint16_t *>(vt + A1 * K::VAT + r * K::VSW + (swz<K::VSW>(r, XB >> 4) << 4) + (XB & 15)) =
                    0x3F80;                    // bf16 1.0
              }
            }
            fence_async_smem();                // visible to the tensor core
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(v_ready + st);
        }
        if (!resident) ring.pos += it.n_kv;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(K::R_SOFT));
    // ================= softmax and epilogue of tile X =================
    const int X = warp >> 2;                   // tile
    const int r = ((warp & 3) << 5) + lane;    // row in tile == TMEM lane
    const uint32_t tS = tmem + ((uint32_t)((warp & 3) * 32) << 16) + X * K::TW;
    const uint32_t tO = tS + BN;
    const float sl2 = a.scale_log2;
    const float2 scale2 = make_float2(sl2, sl2);
    uint8_t *stg = sStg + warp * K::STG;
    uint32_t gs = 0, oc = 0;                   // steps and items of this tile
    bool ok = true;
    Reader rd;
    while (ok) {
      const Item *ip = rd.get<8>(sItem, item_full, epoch, 15);
      if (!ip) break;
      const Item it = *ip;
      rd.done(item_empty, lane);
      if (it.n_qt == 0) break;
      if (X >= it.n_qt) continue;
      float m = NO_KEY, l = 0.f;
      for (int j = 0; j < it.n_kv; ++j, ++gs) {
        const Step sp = step_of<BN>(it, j);
        const unsigned char *mk = a.c.seg[sp.seg].mask;
        uint32_t live[BN / 32];                // keys of the step that count, when some do not
        const bool partial = sp.valid < BN || mk;
        if (partial) {
          if (mk) mk += (long long)sp.set * a.c.seg[sp.seg].L + sp.key;
#pragma unroll
          for (int i = 0; i < BN / 32; ++i)
            live[i] = __ballot_sync(0xffffffffu, 32 * i + lane < sp.valid && (!mk || st::after_wait(mk)[32 * i + lane]));
        }
        if (!(ok = warp_wait<8>(s_full + X, gs & 1, epoch, 11))) break;
        tc_fence_after();
        uint32_t sr[BN];
#pragma unroll
        for (int c = 0; c < BN / 16; ++c) COND_LD16(tS + c * 16, sr + c * 16);
        tmem_wait_ld();
        if (partial) {
#pragma unroll
          for (int c = 0; c < BN; ++c)
            if (!(live[c >> 5] >> (c & 31) & 1)) sr[c] = __float_as_uint(-INFINITY);
        }
        float mxp[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) mxp[e] = __uint_as_float(sr[e]);
#pragma unroll
        for (int c = 4; c + 8 <= BN; c += 8) {
          mxp[0] = fmax3(mxp[0], __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
          mxp[1] = fmax3(mxp[1], __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
          mxp[2] = fmax3(mxp[2], __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
          mxp[3] = fmax3(mxp[3], __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
        }
        mxp[0] = fmax3(mxp[0], __uint_as_float(sr[BN - 4]), __uint_as_float(sr[BN - 3]));
        mxp[1] = fmax3(mxp[1], __uint_as_float(sr[BN - 2]), __uint_as_float(sr[BN - 1]));
        // a step without any key leaves the row at NO_KEY: its weights are 0
        const float mx = fmaxf(fmaxf(fmax3(mxp[0], mxp[1], mxp[2]), mxp[3]) * sl2, NO_KEY);
        if (j == 0) {
          m = mx;
        } else {
          const bool need = mx > m + 8.0f;
          if (__any_sync(0xffffffffu, need)) {
            // S(j) complete means PV(j - 1) is (one thread issued both): rescale O in TMEM
            const float corr = need ? ex2_mufu(m - mx) : 1.0f;
            if (need) {
              if (!K::ONES) l *= corr;         // with the ones column the sum is rescaled with O
              m = mx;
            }
#pragma unroll 1
            for (int c = 0; c < K::DPV / 16; ++c) {
              uint32_t ov[16];
              COND_LD16(tO + c * 16, ov);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * corr);
              COND_ST16(tO + c * 16, ov);
            }
            tmem_wait_st();
          }
        }
        const float2 negm = make_float2(-m, -m);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c0 = 0; c0 < BN; c0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 xx = ffma2(make_float2(__uint_as_float(sr[c0 + c]), __uint_as_float(sr[c0 + c + 1])),
                                    scale2, negm);
            float2 e;
            if (((c >> 1) & 7) < kPolyPairs) {
              e = ex2_poly2(xx);
            } else {
              e.x = ex2_mufu(xx.x);
              e.y = ex2_mufu(xx.y);
            }
            if (!K::ONES) acc[(c >> 1) & 3] = fadd2(acc[(c >> 1) & 3], e);
            pk[c >> 1] = st::pack_bf16x2(e.x, e.y);
          }
          COND_ST16(tS + (c0 >> 1), pk);
        }
        if (!K::ONES) {
          const float2 s01 = fadd2(acc[0], acc[1]), s23 = fadd2(acc[2], acc[3]);
          const float2 s = fadd2(s01, s23);
          l += s.x + s.y;
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full + X);
      }
      if (!ok) break;
      // O of the item: divided by the row sum, written out.  P of the next item
      // follows in this warp, so its PV cannot overwrite O before it is read.
      const int row = it.r0 + X * a.tile_rows + r;           // row of the unit
      const bool valid = r < a.tile_rows && row < a.c.R;
      const bool some = it.n_kv > 0;
      float inv = 0.f, lse = -INFINITY;
      if (some) {
        if (!(ok = warp_wait<8>(o_full + X, oc & 1, epoch, 13))) break;
        ++oc;
        tc_fence_after();
      }
      const long long prow = (long long)it.split * a.c.part_rows + ((long long)it.unit * a.c.HW + it.w) * a.c.R + row;
      const long long off = a.tma_out || !valid ? 0 : (a.c.part_o ? prow * D : st::cond_row(a.c, it.unit, it.w, row));
      const int row0 = it.r0 + X * a.tile_rows + (warp & 3) * 32;
      // O leaves TMEM from its last columns (which may hold the row sum), GRP
      // chunks of 16 at a time
      constexpr int NCH = (D + 15) / 16, GRP = D == 128 ? 4 : (D == 96 ? 3 : NCH);
#pragma unroll
      for (int c0 = NCH; c0 > 0; c0 -= GRP) {
        uint32_t ov[GRP][16];
#pragma unroll
        for (int i = 0; i < GRP; ++i)
          if (c0 - 1 - i >= 0) {
            if (some) COND_LD16(tO + (c0 - 1 - i) * 16, ov[i]);
            else
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[i][e] = 0u;
          }
        if (some) {
          tmem_wait_ld();
          if (c0 == NCH) {
            if constexpr (K::ONES) l = __uint_as_float(ov[0][D % 16]);   // the sum of the bf16 weights
            if (m > NO_KEY || l != l) {      // else no key counted: o = 0, lse = -inf
              inv = __fdividef(1.0f, l);
              lse = (m + __log2f(l)) * 0.6931471805599453f;
            }
          }
        }
        if (a.tma_out) {
          if (c0 == NCH) {
            if (lane == 0) bulk_wait_read(); // the previous tile's store has read the staging rows
            __syncwarp();
          }
          if (D == 128 && c0 == 4) {         // one 128-byte chunk of staging: the upper half goes out first
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (row0 < a.c.R) tma_store_5d(&mp.o1, stg, 64, it.w, row0, it.c3, it.c4);
              bulk_commit();
              bulk_wait_read();
            }
            __syncwarp();
          }
        }
#pragma unroll
        for (int i = 0; i < GRP; ++i) {
          const int c = (c0 - 1 - i) * 16;
          if (c < 0) continue;
          float y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = __uint_as_float(ov[i][e]) * inv;
          if (!a.tma_out && valid && (a.c.part_o || a.c.o_f32)) {
            // a part without keys is not read by the combine kernel
            float *dst = (a.c.part_o ? a.c.part_o : static_cast<float *>(a.c.o)) + off + c;
#pragma unroll
            for (int f = 0; f < 4; ++f)
              if (c + 4 * f < D)
                *reinterpret_cast<float4 *>(dst + 4 * f) = make_float4(y[4 * f], y[4 * f + 1], y[4 * f + 2], y[4 * f + 3]);
          }
          if (a.tma_out || (valid && !a.c.part_o && !a.c.o_f32)) {
            // staged in the swizzle of the store's part of the head, or straight to the row
            const bool lo = D == 128 || c < K::C0;
            const int f0 = (c < K::C0 ? c : c - K::C0) / 8;
            uint8_t *rowp = lo ? stg + lane * K::SW0 : stg + 32 * K::SW0 + lane * K::SW1X;
            uint16_t *dst = static_cast<uint16_t *>(a.c.o) + off + c;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const int at = lo ? swz<K::SW0>(lane, f0 + f) : swz<K::SW1X>(lane, f0 + f);
              const uint4 v = make_uint4(st::pack_bf16x2(y[8 * f], y[8 * f + 1]), st::pack_bf16x2(y[8 * f + 2], y[8 * f + 3]),
                                         st::pack_bf16x2(y[8 * f + 4], y[8 * f + 5]), st::pack_bf16x2(y[8 * f + 6], y[8 * f + 7]));
              if (a.tma_out) *reinterpret_cast<uint4 *>(rowp + (at << 4)) = v;
              else if (c + 8 * f < D) *reinterpret_cast<uint4 *>(dst + 8 * f) = v;
            }
          }
        }
      }
      if (a.tma_out) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && row0 < a.c.R) {
          tma_store_5d(&mp.o0, stg, 0, it.w, row0, it.c3, it.c4);
          if (K::C1 && D != 128) tma_store_5d(&mp.o1, stg + 32 * K::SW0, 64, it.w, row0, it.c3, it.c4);
          bulk_commit();
        }
      }
      if (valid) {
        if (a.c.part_o) a.c.part_lse[prow] = lse;
        else if (a.c.lse) a.c.lse[st::cond_lse(a.c, it.unit, it.w, row)] = lse;
      }
    }
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
                                : swizzle_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B;
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(ptr), d, s, b, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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

template <int D> st_status launch(const st::CondParams &p, cudaStream_t s) {
  using K = Cfg<D>;
  Args a = {};
  a.c = p;
  a.tile_rows = BLOCK_M / p.G * p.G;
  a.q_blocks = (p.R + K::NT * a.tile_rows - 1) / (K::NT * a.tile_rows);
  const long long items = (long long)st::cond_units(p) * p.HW * p.n_split * a.q_blocks;
  if (items > 0x3fffffffLL) return ST_ERR_SHAPE;
  a.n_items = int(items);
  a.dqb = st::make_fastdiv(uint32_t(a.q_blocks));
  a.dsplit = st::make_fastdiv(uint32_t(p.n_split));
  a.dhw = st::make_fastdiv(uint32_t(p.HW));
  a.dkv = st::make_fastdiv(uint32_t(p.hdiv));
  a.dt = st::make_fastdiv(uint32_t(p.g.T));
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
        !map_kv(&m.v[g], sg.v, p, sg, K::VW, K::VSW, K::BN))
      return ST_ERR_CUDA;
  }
  if (steps * (p.n_split + 1) >= (1LL << 31)) return ST_ERR_SHAPE;
  a.max_steps = int(steps);
  a.resident = p.n_split == 1 && steps <= K::NS ? 1 : 0;
  a.tma_out = !p.part_o && !p.o_f32 && p.G == 1 ? 1 : 0;
  if (!map_q(&m.q0, p.q, p, K::C0, K::SW0, a.tile_rows) ||
      (K::C1 && !map_q(&m.q1, p.q, p, K::C1X, K::SW1X, a.tile_rows)) ||
      (a.tma_out && (!map_q(&m.o0, p.o, p, K::C0, K::SW0, 32) || (K::C1 && !map_q(&m.o1, p.o, p, K::C1X, K::SW1X, 32)))))
    return ST_ERR_CUDA;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.epoch = g_epoch.fetch_add(1) + 1;
  const int ctas = int(items < st::num_sms() ? items : st::num_sms());
  auto kern = cond_attn_sm100<D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, K::SMEM) != cudaSuccess)
    return ST_ERR_CUDA;
  // A build that grants fewer registers than the split assumes would wait in
  // setmaxnreg forever: refuse it.
  static int regs_ok = -1;
  if (regs_ok < 0) {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return ST_ERR_CUDA;
    regs_ok = fa.numRegs * K::THREADS >= 128 * K::NT * K::R_SOFT + 256 * K::R_MISC ? 1 : 0;
  }
  if (!regs_ok) return ST_ERR_UNSUPPORTED;
  return st::launch_pdl(kern, dim3(ctas), dim3(K::THREADS), K::SMEM, s, m, a);
}

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

CondTile cond_tile(int D) { return D <= 96 ? CondTile{3 * 128, 64} : CondTile{2 * 128, 128}; }

st_status cond_sm100(const CondParams &p, cudaStream_t s) {
  switch (p.g.D) {
    case 32: return launch<32>(p, s);
    case 64: return launch<64>(p, s);
    case 72: return launch<72>(p, s);
    case 80: return launch<80>(p, s);
    case 96: return launch<96>(p, s);
    case 128: return launch<128>(p, s);
  }
  return ST_ERR_UNSUPPORTED;
}

}  // namespace st
