// st_attn_cross and st_attn_prefix: validation, the plan of a launch, and the
// kernel that combines split parts.
//
// The plan, from sizes and strides alone:
//   * Frames and tokens with one stride between rows are one unit of T * S
//     rows, and batches that share their only set of keys and follow one
//     another in memory are one unit too: full row tiles, one walk over the
//     shared keys.
//   * Grouped heads (H > H_kv) of units below one 128-row tile become rows, so
//     a K/V tile is read once for its whole group.
//   * Few work items: the keys are split into parts whose fp32 partials go to
//     the workspace and are combined by a second kernel, as attn_chunk_merge
//     does (same formula), so that one query over long states still uses every SM
//     (2 x 24 heads of 128 channels on 8 KV heads, 20,736 keys: 41 us of 26 us
//     that reading the states takes).
//   * Samples of at most PACK_ROWS rows that share a prefix attend to it in
//     packed tiles; the combine kernel attends each row's own keys.
#include <math.h>

#include "cond.cuh"

namespace {

using st::CondParams;
using st::Geom;
using st::KvSeg;

// Samples of a prefix are packed up to this many rows each (heads of a group
// included), and only where the prefix is longer than rows x own keys: the
// combine kernel reads a sample's own keys once per row.  64 samples, 16 heads
// x 72, 64 own keys, packed and not: prefix of 4096, 1 row 31 and 461 us, 8 rows
// 86 and 461, 32 rows 275 and 461; prefix of 512, 32 rows 194 and 87.
constexpr int PACK_ROWS = 32;
// Parts of split keys: at most MAX_SPLIT (two per lane of the combine kernel),
// of MIN_KEYS keys at least, from SPLIT_KEYS keys on, or fewer where there is
// little to combine.  16 heads x 72, split and not: 1 row of 4 batches, 600
// keys 15.5 and 15.8 us, 1200 keys 19.6 and 23.8; 64 rows of 2 batches, 600 keys
// 20.4 and 15.6; 200 rows, 1200 keys 23 and 30.
constexpr int MAX_SPLIT = 64, MIN_KEYS = 256, SPLIT_KEYS = 1024;
constexpr int FEW_ROWS = 1024, SPLIT_KEYS_FEW = 640;

bool d_supported(int D) { return D == 32 || D == 64 || D == 72 || D == 80 || D == 96 || D == 128; }

st_status make_seg(const st_kv_desc *d, const Geom &g, KvSeg &s, int &H_kv) {
  if (!d) return ST_ERR_NULL;
  if (d->size != (int)sizeof(st_kv_desc)) return ST_ERR_SHAPE;
  if (d->n_sets <= 0 || d->L < 0 || d->H_kv < 0 || d->stride_set < 0 || d->stride_l < 0 || d->n_rows < 0)
    return ST_ERR_SHAPE;
  if (d->L == 0 && (d->len || d->offsets || d->mask)) return ST_ERR_SHAPE;
  if (d->offsets && (d->len || d->mask || d->n_rows > 0x7fffffffLL)) return ST_ERR_SHAPE;
  if (!d->offsets && d->n_rows) return ST_ERR_SHAPE;
  if (g.B % d->n_sets) return ST_ERR_DIVISIBILITY;
  H_kv = d->H_kv ? d->H_kv : g.H;
  if (g.H % H_kv) return ST_ERR_DIVISIBILITY;
  s = KvSeg{};
  s.L = d->L;
  s.n_sets = d->n_sets;
  s.per = g.B / d->n_sets;
  s.len = d->len;
  s.offsets = d->offsets;
  s.mask = d->mask;
  s.n_rows = int(d->n_rows);
  const long long row = (long long)H_kv * g.D;
  s.stride_l = d->stride_l ? d->stride_l : row;
  s.stride_set = d->stride_set ? d->stride_set : (long long)d->L * s.stride_l;
  if (s.stride_l < row) return ST_ERR_SHAPE;
  // packed sets of no rows at all: no keys
  if (d->offsets && d->n_rows == 0) s.L = 0;
  return ST_OK;
}

bool seg_aligned(const KvSeg &s, int esize) {
  return s.stride_l % (16 / esize) == 0 && s.stride_set % (16 / esize) == 0;
}

struct Plan {
  CondParams p;
  st_dtype dtype;
  size_t workspace;            // bytes asked for; 0: none
};

int ceil_div(long long a, long long b) { return int((a + b - 1) / b); }

// with_ws = false: the plan of a call without workspace.
st_status make_plan(const st_attn_desc *desc, const st_kv_desc *d0, const st_kv_desc *d1, bool with_ws, Plan &pl) {
  Geom g;
  int lo, hi;
  st_status s = st::make_geom(desc, false, g, lo, hi);
  if (s != ST_OK) return s;
  if (desc->kv_begin != 0 || desc->kv_end != 0) return ST_ERR_SHAPE;
  if (lo != 0 || hi != g.T) return ST_ERR_UNSUPPORTED;
  const bool bf16 = desc->dtype == ST_BF16;
  if (bf16 ? !d_supported(g.D) : g.D > 128) return ST_ERR_UNSUPPORTED;
  // the tensor maps take tokens at one stride and batches of whole frame blocks
  // (as st_attn_spatial); the fp32 kernel finds each row by itself
  const bool tokens = g.sblk == g.S || g.ssb == (long long)g.sblk * g.ss;
  if (bf16 && !tokens) return ST_ERR_UNSUPPORTED;
  if (bf16 && g.tblk != g.T && g.sb != (long long)(g.T / g.tblk) * g.stb) return ST_ERR_UNSUPPORTED;
  if (g.ss < (long long)g.H * g.D) return ST_ERR_SHAPE;
  if (bf16 && (g.ss % 8 || g.st % 8 || g.stb % 8 || g.sb % 8)) return ST_ERR_ALIGN;
  CondParams &p = pl.p;
  p = CondParams{};
  int hk0, hk1;
  KvSeg seg0, seg1;
  if ((s = make_seg(d0, g, seg0, hk0)) != ST_OK) return s;
  if (bf16 && !seg_aligned(seg0, 2)) return ST_ERR_ALIGN;
  p.seg[0] = seg0;
  p.n_seg = 1;
  if (d1) {
    if ((s = make_seg(d1, g, seg1, hk1)) != ST_OK) return s;
    if (bf16 && !seg_aligned(seg1, 2)) return ST_ERR_ALIGN;
    if (hk1 != hk0) return ST_ERR_SHAPE;
    p.seg[1] = seg1;
    p.n_seg = 2;
  }
  const long long all_rows = (long long)g.B * g.T * g.S;
  if (all_rows * g.H >= (1LL << 31) || (long long)seg0.L + (d1 ? seg1.L : 0) >= (1LL << 30)) return ST_ERR_SHAPE;
  // One query per frame: no token stride is used, so the one between frames (or,
  // with one frame, batches) takes its place, and queries at any distance (columns
  // of a fused projection, say) become rows as dense ones do.
  if (g.S == 1) {
    const long long step = g.T > 1 ? g.st : g.sb;
    if (step >= (long long)g.H * g.D) g.ss = step;
  }
  p.T0 = g.T;
  p.S0 = g.S;
  p.bm = 1;
  // one stride between all rows of a batch
  const bool flat = tokens && (g.T == 1 || (g.st == (long long)g.S * g.ss &&
                                            (g.tblk == g.T || g.stb == (long long)g.tblk * g.st)));
  if (flat) {
    g.S *= g.T;
    g.T = 1;
  }
  if (tokens) {
    g.sblk = g.S;
    g.ssb = (long long)g.S * g.ss;
  }
  if (flat) {
    g.tblk = 1;
    g.st = g.stb = g.ssb;
  }
  const int grp = g.H / hk0;
  // batches that share every key they attend, or (few rows) their prefix
  const bool follow = flat && g.sb == (long long)g.S * g.ss;
  const bool share = !d1 && seg0.per > 1 && follow;
  const bool pack = with_ws && d1 && seg0.per > 1 && follow && (long long)g.S * grp <= PACK_ROWS &&
                    seg0.L > (long long)g.S * grp * seg1.L;
  if (share || pack) {
    p.bm = seg0.per;
    if (pack) {
      p.own = seg1;
      p.n_seg = 1;
    }
    g.B /= p.bm;
    g.sb *= p.bm;
    g.S *= p.bm;
    g.sblk = g.S;
    g.st = g.stb = g.ssb = (long long)g.S * g.ss;
  }
  const bool pack_heads = flat && grp > 1 && g.S < 128 && grp <= 128;
  p.G = pack_heads ? grp : 1;
  p.HW = g.H / p.G;
  p.hdiv = pack_heads ? 1 : grp;
  p.g = g;
  p.R0 = g.S;
  p.R = g.S * p.G;
  p.part_rows = all_rows * g.H;
  p.scale = desc->scale > 0.f ? desc->scale : 1.0f / sqrtf((float)g.D);
  p.o_f32 = desc->o_fp32 || !bf16;
  pl.dtype = desc->dtype;
  // split long keys when the items leave more than half of the GPU idle; items
  // of one row tile then take one part of their keys with each of their tiles
  const st::CondTile t = bf16 ? st::cond_tile(g.D) : st::CondTile{64, 1, 64};
  long long steps = 0, keys = 0;
  for (int i = 0; i < p.n_seg; ++i) {
    steps += ceil_div(p.seg[i].L, t.keys);
    keys += p.seg[i].L;
  }
  const int tile_rows = bf16 ? t.rows / p.G * p.G : t.rows;
  const long long items = (long long)st::cond_units(p) * p.HW * ceil_div(p.R, tile_rows * t.tiles);
  const long long cap = (long long)st::device_sms() * (bf16 ? 1 : 2);
  p.n_split = p.spread = 1;
  const long long min_steps = ceil_div(MIN_KEYS, t.keys);
  if (with_ws && items * 2 <= cap && keys >= (p.part_rows <= FEW_ROWS ? SPLIT_KEYS_FEW : SPLIT_KEYS)) {
    if (p.R <= tile_rows) p.spread = t.tiles;
    long long n = cap / items;
    if (n > steps / min_steps) n = steps / min_steps;
    if (n > MAX_SPLIT / p.spread) n = MAX_SPLIT / p.spread;
    p.n_split = int(n) * p.spread;
  }
  pl.workspace = p.n_split > 1 || pack ? size_t(p.n_split) * size_t(p.part_rows) * size_t(g.D + 1) * 4 : 0;
  return ST_OK;
}

// ---------------------------------------------------------------- combine
// The parts' weights exp(lse_c - M) (M the largest), the weighted rows, and
// with OWN the row's own keys in the same softmax.  Parts whose LSE is -inf (no
// key) are not read.  Bound by the latency of its chains of loads more than by
// the bytes (64 rows x 16 heads, 27 parts and 64 own keys each: 14 us): WPR warps
// take a row (every WPR-th part and 16 keys), a lane holds
// 4 consecutive channels, and the warps join over shared memory.
__device__ __forceinline__ float4 load4(const uint16_t *p, int) {
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ float4 load4(const float *p, int n) {   // n: channels that exist; rows 4-byte aligned
  return make_float4(p[0], n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
}
__device__ __forceinline__ void axpy4(float4 &a, float w, const float4 &x) {
  a.x = fmaf(w, x.x, a.x);
  a.y = fmaf(w, x.y, a.y);
  a.z = fmaf(w, x.z, a.z);
  a.w = fmaf(w, x.w, a.w);
}

constexpr int BATCH = 8;       // loads of a lane in flight

// LOOP: a block takes row after row (under a budget; with the loop the bf16 kernel
// spills, one token behind a prefix 54 for 48 us).
template <typename T, bool OWN, int WPR, bool LOOP>
__global__ void __launch_bounds__(128, WPR == 4 && sizeof(T) == 2 ? 8 : 4) cond_combine(const __grid_constant__ CondParams p) {
  __shared__ __align__(16) float sq[4][128];
  __shared__ float sm[4], sl[4];
  constexpr float L2E = 1.4426950408889634f;
  st::pdl_trigger();
  st::pdl_wait();
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int sub = wp % WPR;                    // this warp's share of the row
  const int D = p.g.D, d0 = 4 * lane, nd = D - d0;
  // (rows of a call: below 2^31; WPR = 4: the rows of a block's warps are the same)
#pragma unroll 1
  for (uint32_t row = blockIdx.x * (4 / WPR) + wp / WPR; row < p.part_rows; row += gridDim.x * (4 / WPR)) {
    const uint32_t col = row / uint32_t(p.R);
    const int r = int(row - col * uint32_t(p.R)), unit = int(col / uint32_t(p.HW)), w = int(col) - unit * p.HW;
    const long long off = st::cond_row<sizeof(T) == 4>(p, unit, w, r);
    const float *part_lse = st::after_wait(p.part_lse), *part_o = st::after_wait(p.part_o);
    // the parts of this warp: sub, sub + WPR, ... (at most 64 in all)
    const int n = p.n_split;
    const int c0 = sub + WPR * lane, c1 = c0 + 32 * WPR;
    const float l0 = c0 < n ? part_lse[(long long)c0 * p.part_rows + row] : -INFINITY;
    const float l1 = c1 < n ? part_lse[(long long)c1 * p.part_rows + row] : -INFINITY;
    float m = -INFINITY, l = 0.f;                // running max (log2 units) and sum; the same in all lanes
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (OWN) {
      const T *q = static_cast<const T *>(st::after_wait(p.q)) + off;
      const float sl2 = p.scale * L2E;
      if (nd > 0) {
        const float4 x = load4(q + d0, nd);
        *reinterpret_cast<float4 *>(&sq[wp][d0]) = make_float4(x.x * sl2, x.y * sl2, x.z * sl2, x.w * sl2);
      }
      __syncwarp();
      const int b = cond_batch(p, unit) + r / p.G / (p.T0 * p.S0);
      st::KvSeg sg = p.own;
      sg.len = st::after_wait(sg.len);
      sg.offsets = st::after_wait(sg.offsets);
      const st::KvRange kr = st::kv_range(sg, b);
      const long long base = (long long)kr.set * (sg.offsets ? 0 : sg.stride_set) + (long long)kr.row0 * sg.stride_l +
                             (long long)((w * p.G + r % p.G) / (p.G * p.hdiv)) * D;
      const T *K = static_cast<const T *>(st::after_wait(sg.k)) + base;
      const T *V = static_cast<const T *>(st::after_wait(sg.v)) + base;
      const unsigned char *mk = sg.mask ? st::after_wait(sg.mask) + (long long)kr.set * sg.L : nullptr;
      for (int k0 = 16 * sub; k0 < kr.n; k0 += 16 * WPR) {
        const int key = k0 + (lane >> 1), half = lane & 1;     // two lanes per key, every other 8 channels each
        float x = 0.f;
        const bool on = key < kr.n && (!mk || mk[key]);
        // V of the first keys is on its way with K (a key that does not count is not read)
        const unsigned counts = __ballot_sync(0xffffffffu, on);
        const T *vp = V + (long long)k0 * sg.stride_l + d0;
        float4 x4[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          x4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (nd > 0 && (counts >> 2 * i & 1)) x4[i] = load4(vp + i * sg.stride_l, nd);
        }
        if (on) {
          const T *kp = K + (long long)key * sg.stride_l;
          if constexpr (sizeof(T) == 2) {
            uint4 v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
              if (16 * c + 8 * half < D) v[c] = *reinterpret_cast<const uint4 *>(kp + 16 * c + 8 * half);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int d = 16 * c + 8 * half;
              if (d >= D) break;
              const uint32_t u[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                x = fmaf(sq[wp][d + 2 * i], __uint_as_float(u[i] << 16), x);
                x = fmaf(sq[wp][d + 2 * i + 1], __uint_as_float(u[i] & 0xffff0000u), x);
              }
            }
          } else {
#pragma unroll 8
            for (int d = half; d < D; d += 2) x = fmaf(sq[wp][d], kp[d], x);
          }
        }
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        if (!on) x = -INFINITY;
        float mx = x;
#pragma unroll
        for (int y = 16; y > 0; y >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
        const float mn = fmaxf(m, mx);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float corr = exp2f(m - ref), e = exp2f(x - ref);
        float sum = e;
#pragma unroll
        for (int y = 16; y > 1; y >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
        l = l * corr + sum;
        m = mn;
        acc = make_float4(acc.x * corr, acc.y * corr, acc.z * corr, acc.w * corr);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) axpy4(acc, __shfl_sync(0xffffffffu, e, 2 * i), x4[i]);
        if (counts >> 2 * BATCH) {
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            x4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (nd > 0 && (counts >> 2 * (BATCH + i) & 1)) x4[i] = load4(vp + (BATCH + i) * sg.stride_l, nd);
          }
#pragma unroll
          for (int i = 0; i < BATCH; ++i) axpy4(acc, __shfl_sync(0xffffffffu, e, 2 * (BATCH + i)), x4[i]);
        }
      }
    }
    // the parts
    float M = fmaxf(l0, l1) * L2E;
#pragma unroll
    for (int y = 16; y > 0; y >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, y));
    M = fmaxf(M, m);
    const float ref = M == -INFINITY ? 0.f : M;
    const float own = exp2f(m - ref);            // 0 without own keys
    const float w0 = exp2f(l0 * L2E - ref), w1 = exp2f(l1 * L2E - ref);
    float sum = w0 + w1;
#pragma unroll
    for (int y = 16; y > 0; y >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
    sum += l * own;
    acc = make_float4(acc.x * own, acc.y * own, acc.z * own, acc.w * own);
    for (int b = 0; sub + WPR * b < n; b += BATCH) {
      float4 x4[BATCH];
      float wc[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int c = b + i;                     // (c <= 63; a part past the last has weight 0)
        wc[i] = __shfl_sync(0xffffffffu, c < 32 ? w0 : w1, c & 31);
        x4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (wc[i] != 0.f && nd > 0) {
          const float *src = part_o + ((long long)(sub + WPR * c) * p.part_rows + row) * D + d0;
          if constexpr (sizeof(T) == 2) x4[i] = *reinterpret_cast<const float4 *>(src);
          else x4[i] = load4(src, nd);
        }
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) axpy4(acc, wc[i], x4[i]);
    }
    if constexpr (WPR > 1) {                     // join the warps of the row
      if (lane == 0) {
        sm[wp] = M;
        sl[wp] = sum;
      }
      __syncthreads();
      const float all = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
      const float base = all == -INFINITY ? 0.f : all;
      const float scale = exp2f(M - base);       // 0 for a warp without a key
      *reinterpret_cast<float4 *>(&sq[wp][d0]) = make_float4(acc.x * scale, acc.y * scale, acc.z * scale, acc.w * scale);
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum = fmaf(sl[i], exp2f(sm[i] - base), sum);
      M = all;
      __syncthreads();
      if (!LOOP && sub) return;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) axpy4(acc, 1.f, *reinterpret_cast<const float4 *>(&sq[i][d0]));
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const float y[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
    if (sub == 0 && nd > 0) {
      if (p.o_f32) {
        float *o = static_cast<float *>(p.o) + off + d0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < nd) o[i] = y[i];
      } else {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + off + d0) =
            make_uint2(st::pack_bf16x2(y[0], y[1]), st::pack_bf16x2(y[2], y[3]));
      }
    }
    if (sub == 0 && p.lse && lane == 0)
      p.lse[st::cond_lse(p, unit, w, r)] = sum == 0.f ? -INFINITY : (M + log2f(sum)) / L2E;
    if constexpr (!LOOP) return;
    // the next row's Q goes where this one's sums (WPR > 1) or Q are still read
    if constexpr (WPR > 1) __syncthreads();
    else __syncwarp();
  }
}

// Four warps per row up to 8 rows per SM, else a warp.  So many bf16 blocks run at
// once; of fp32 4 fit an SM with own keys and 7 without, and their second round
// still pays.  Whole calls behind one prefix, 64 own keys, four warps and one: bf16,
// 72 channels, 1024 rows of 27 parts 47.6 and 54.0 us from HBM (37.2 and 35.0 where
// all of it stays in L2), 2048 rows of 12 parts 50.7 and 36.2; fp32, 592 rows of 16
// parts 90 and 113, 1024 rows 104 and 117 (128 channels 141 and 164), 1536 rows of 9
// parts 193 both.
template <typename T, bool OWN> st_status combine_own(const CondParams &p, cudaStream_t s) {
  const bool four = p.part_rows <= (long long)st::device_sms() * 8;
  const long long blocks = four ? p.part_rows : (p.part_rows + 3) / 4;
  const int sms = st::num_sms();
  if (sms < st::device_sms() && blocks > sms * 8LL) {      // a budget: as many blocks as run at once
    const auto kern = four ? cond_combine<T, OWN, 4, true> : cond_combine<T, OWN, 1, true>;
    return st::launch_pdl(kern, dim3(unsigned(sms * 8)), dim3(128), 0, s, p);
  }
  const auto kern = four ? cond_combine<T, OWN, 4, false> : cond_combine<T, OWN, 1, false>;
  return st::launch_pdl(kern, dim3(unsigned(blocks)), dim3(128), 0, s, p);
}
template <typename T> st_status combine(const CondParams &p, cudaStream_t s) {
  return p.own.k ? combine_own<T, true>(p, s) : combine_own<T, false>(p, s);
}

st_status run(const st_attn_desc *desc, const st_kv_desc *d0, const st_kv_desc *d1, const void *q, const void *k0,
              const void *v0, const void *k1, const void *v1, void *o, float *lse, void *ws, size_t ws_bytes,
              st_stream_t stream) {
  if (!desc || !d0 || !q || !o) return ST_ERR_NULL;
  Plan pl;
  st_status s = make_plan(desc, d0, d1, ws != nullptr, pl);
  if (s != ST_OK) return s;
  CondParams &p = pl.p;
  // pointers of a set without keys may be NULL
  if ((p.seg[0].L && (!k0 || !v0)) || (d1 && p.seg[1].L && (!k1 || !v1))) return ST_ERR_NULL;
  if (ws && ws_bytes < pl.workspace) return ST_ERR_SHAPE;
  const bool bf16 = pl.dtype == ST_BF16;
  const size_t al = bf16 ? 16 : 4;
  if (!st::is_aligned(q, al) || !st::is_aligned(o, al) || !st::is_aligned(k0, al) || !st::is_aligned(v0, al) ||
      !st::is_aligned(k1, al) || !st::is_aligned(v1, al) || !st::is_aligned(lse, 4) || !st::is_aligned(ws, 16))
    return ST_ERR_ALIGN;
  for (const KvSeg &sg : p.seg)
    if (!st::is_aligned(sg.len, 4) || !st::is_aligned(sg.offsets, 4)) return ST_ERR_ALIGN;
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.seg[0].k = k0;
  p.seg[0].v = v0;
  p.seg[1].k = k1;
  p.seg[1].v = v1;
  const bool own = d1 && p.n_seg == 1;
  p.own = own ? p.seg[1] : KvSeg{};
  if (own && !p.own.L) p.own.k = p.own.v = q;  // no keys: never read
  if (pl.workspace) {
    p.part_o = static_cast<float *>(ws);
    p.part_lse = p.part_o + (long long)p.n_split * p.part_rows * p.g.D;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  s = bf16 ? st::cond_sm100(p, st) : st::cond_simt(p, st);
  if (s != ST_OK || !pl.workspace) return s;
  return bf16 ? combine<uint16_t>(p, st) : combine<float>(p, st);
}

size_t ws_bytes(const st_attn_desc *desc, const st_kv_desc *d0, const st_kv_desc *d1) {
  Plan pl;
  if (!desc || !d0 || make_plan(desc, d0, d1, true, pl) != ST_OK) return 0;
  return pl.workspace;
}

}  // namespace

ST_API st_status st_attn_cross(const st_attn_desc *desc, const st_kv_desc *kv, const void *q, const void *k,
                               const void *v, void *o, float *lse, void *workspace, size_t workspace_bytes,
                               st_stream_t stream) {
  return run(desc, kv, nullptr, q, k, v, nullptr, nullptr, o, lse, workspace, workspace_bytes, stream);
}

ST_API size_t st_attn_cross_workspace_bytes(const st_attn_desc *desc, const st_kv_desc *kv) {
  return ws_bytes(desc, kv, nullptr);
}

ST_API st_status st_attn_prefix(const st_attn_desc *desc, const st_kv_desc *prefix, const st_kv_desc *own,
                                const void *q, const void *k_prefix, const void *v_prefix, const void *k,
                                const void *v, void *o, float *lse, void *workspace, size_t workspace_bytes,
                                st_stream_t stream) {
  if (!own) return ST_ERR_NULL;
  return run(desc, prefix, own, q, k_prefix, v_prefix, k, v, o, lse, workspace, workspace_bytes, stream);
}

ST_API size_t st_attn_prefix_workspace_bytes(const st_attn_desc *desc, const st_kv_desc *prefix,
                                             const st_kv_desc *own) {
  return own ? ws_bytes(desc, prefix, own) : 0;
}
