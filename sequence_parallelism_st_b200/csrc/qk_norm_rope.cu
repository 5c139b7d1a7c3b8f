// st_qk_norm_rope: per-head RMSNorm of Q and K and their rotary embedding in
// one pass, where no relayout moves them.
//
//   y = x / sqrt(mean(x^2) + eps) * gamma;  (a, b) -> (a c - b s, a s + b c)
//
// Bound by HBM: every element is read once and written once.  A lane owns 8
// channels of a head (one 16-byte vector of bf16; with the halves pairing 4
// channels and their 4 partners, two 8-byte vectors), so a pair never crosses
// lanes; a head is D / 8 consecutive lanes and a warp holds floor(32 / (D / 8))
// heads of one token at a time.  The sum of squares runs over a head's lanes
// with shuffles.  The heads of Q and K of a token are one list, cut into tasks
// of two to four such groups; a warp has the loads of its next task in flight while
// it works on one, and the sums of a task's groups run side by side.  Gains lie
// in shared memory; the arithmetic is in pairs, since issue slots are what is
// short next (75% used).  bf16: 24 + 24 heads of 128 channels, 65,536 tokens 299 us
// in short runs (5.5 TB/s; 334 us under the power cap at 1.78 GHz; 394 us without the
// loads ahead and the pairs), 16 + 16 heads of 72 (27 of 32 lanes at work), 19,200
// tokens 42 us (4.2 TB/s; 69 us).  fp32: 535 to 545 us (6.0 TB/s) and 64 to 67 us
// (5.4 TB/s).
#include "common.cuh"

namespace {

// Pairs of fp32 in 64-bit registers: one instruction for two products.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float x, float y) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
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
__device__ __forceinline__ f32x2 fmul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 1 / sqrt(x): the hardware's estimate and one Newton step, which 0, infinity and
// NaN go without.
__device__ __forceinline__ float inv_sqrt(float x) {
  const float y = rsqrtf(x);
  const float z = fmaf(0.5f * y, fmaf(-x * y, y, 1.f), y);
  return x > 0.f && x < INFINITY ? z : y;
}

struct QkArgs {
  const void *q, *k;
  void *qo, *ko;
  long long sq, sk, sqo, sko;
  const float *gq, *gk;
  const float4 *table;
  const int *positions;
  int n_pos, period, n_tokens, hq, heads, D;   // heads: of Q and K
  float eps;
  int chunks;                  // tasks of a token
  st::FastDiv dchunk, dperiod;
};

template <typename T, bool HALVES> struct Lane8;   // a lane's 8 channels in memory
template <bool HALVES> struct Lane8<uint16_t, HALVES> {
  uint2 a, b;
  __device__ __forceinline__ void load(const uint16_t *p, int j, int half) {
    if constexpr (HALVES) {
      a = *reinterpret_cast<const uint2 *>(p + 4 * j);
      b = *reinterpret_cast<const uint2 *>(p + half + 4 * j);
    } else {
      const uint4 v = *reinterpret_cast<const uint4 *>(p + 8 * j);
      a = make_uint2(v.x, v.y);
      b = make_uint2(v.z, v.w);
    }
  }
  __device__ __forceinline__ void get(f32x2 *x) const {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ static void store(uint16_t *p, int j, int half, const float *x) {
    const uint32_t w0 = st::pack_bf16x2(x[0], x[1]), w1 = st::pack_bf16x2(x[2], x[3]);
    const uint32_t w2 = st::pack_bf16x2(x[4], x[5]), w3 = st::pack_bf16x2(x[6], x[7]);
    if constexpr (HALVES) {
      *reinterpret_cast<uint2 *>(p + 4 * j) = make_uint2(w0, w1);
      *reinterpret_cast<uint2 *>(p + half + 4 * j) = make_uint2(w2, w3);
    } else {
      *reinterpret_cast<uint4 *>(p + 8 * j) = make_uint4(w0, w1, w2, w3);
    }
  }
};
template <bool HALVES> struct Lane8<float, HALVES> {
  float4 a, b;
  __device__ __forceinline__ static int second(int j, int half) { return HALVES ? half + 4 * j : 8 * j + 4; }
  __device__ __forceinline__ static int first(int j) { return HALVES ? 4 * j : 8 * j; }
  __device__ __forceinline__ void load(const float *p, int j, int half) {
    a = *reinterpret_cast<const float4 *>(p + first(j));
    b = *reinterpret_cast<const float4 *>(p + second(j, half));
  }
  __device__ __forceinline__ void get(f32x2 *x) const {
    x[0] = pair(a.x, a.y);
    x[1] = pair(a.z, a.w);
    x[2] = pair(b.x, b.y);
    x[3] = pair(b.z, b.w);
  }
  __device__ __forceinline__ static void store(float *p, int j, int half, const float *x) {
    *reinterpret_cast<float4 *>(p + first(j)) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + second(j, half)) = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// LPH: lanes of a head (D / 8), or 0 for any.  UNROLL: groups of a task.
template <typename T, bool HALVES, bool ROPE, int LPH, int UNROLL>
__global__ void __launch_bounds__(256, 3) qk_norm_rope(const __grid_constant__ QkArgs a) {
  __shared__ __align__(16) float gains[2][256];
  const int lane = threadIdx.x & 31;
  const int lph = LPH ? LPH : a.D >> 3, hpw = 32 / lph, D = 8 * lph;
  const int hs = lane / lph, j = lane - hs * lph;
  const bool live = hs < hpw;
  const int half = D >> 1;
  const uint32_t tasks = uint32_t(a.n_tokens) * uint32_t(a.chunks);
  const uint32_t warps = gridDim.x * (blockDim.x >> 5);
  st::pdl_trigger();
  st::pdl_wait();
  const T *q = static_cast<const T *>(st::after_wait(a.q)), *k = static_cast<const T *>(st::after_wait(a.k));
  const float4 *table = st::after_wait(a.table);
  const int *positions = st::after_wait(a.positions);
  if (int(threadIdx.x) < D) {
    const float *gq = st::after_wait(a.gq), *gk = st::after_wait(a.gk);
    gains[0][threadIdx.x] = gq ? gq[threadIdx.x] : 1.f;
    gains[1][threadIdx.x] = gk ? gk[threadIdx.x] : 1.f;
  }
  __syncthreads();
  const float inv_d = 1.f / float(D);
  const int d0 = HALVES ? 4 * j : 8 * j, d1 = HALVES ? half + 4 * j : 8 * j + 4;

  struct Task {
    uint32_t token;
    int h0, pos;               // the lane's first head, the token's row of the table
  };
  Lane8<T, HALVES> next[UNROLL];
  auto fetch = [&](uint32_t t, Task &task) {
    task.token = st::fdiv(t, a.dchunk);
    task.h0 = int(t - task.token * uint32_t(a.chunks)) * UNROLL * hpw + hs;
    const T *rq = q + (long long)task.token * a.sq, *rk = k + (long long)task.token * a.sk - a.hq * D;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int h = task.h0 + u * hpw;
      if (live && h < a.heads) next[u].load((h < a.hq ? rq : rk) + h * D, j, half);
    }
    if constexpr (ROPE) {
      if (positions) task.pos = positions[task.token];
      else task.pos = int(task.token - st::fdiv(task.token, a.dperiod) * uint32_t(a.period));
    }
  };
  uint32_t t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  Task task;
  if (t < tasks) fetch(t, task);
  for (; t < tasks; t += warps) {
    const Task cur = task;
    Lane8<T, HALVES> v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) v[u] = next[u];
    float4 cs0 = make_float4(1.f, 0.f, 1.f, 0.f), cs1 = cs0;
    if constexpr (ROPE) {
      if (cur.pos >= 0 && cur.pos < a.n_pos && live) {       // a position outside the table turns nothing
        const float4 *row = table + (long long)cur.pos * (D >> 2) + 2 * j;
        cs0 = row[0];
        cs1 = row[1];
      }
    }
    if (t + warps < tasks) fetch(t + warps, task);
    float ss[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      f32x2 x[4];
      v[u].get(x);             // (lanes past the heads: registers of no row, whose sums no one uses)
      f32x2 s = fmul2(x[0], x[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) s = ffma2(x[i], x[i], s);
      ss[u] = unpair(s).x + unpair(s).y;
    }
    // sums over the lanes of a head, in the order of a fixed tree
    if constexpr (LPH != 0 && (LPH & (LPH - 1)) == 0) {
#pragma unroll
      for (int o = 1; o < LPH; o <<= 1)
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], o);
    } else {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        if (o >= lph) break;
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
          const float y = __shfl_down_sync(0xffffffffu, ss[u], o);
          if (j + o < lph) ss[u] += y;
        }
      }
#pragma unroll
      for (int u = 0; u < UNROLL; ++u) ss[u] = __shfl_sync(0xffffffffu, ss[u], (live ? hs : 0) * lph);
    }
    f32x2 co[2], si[2], nsi[2];
    if constexpr (ROPE && HALVES) {
      co[0] = pair(cs0.x, cs0.z);
      co[1] = pair(cs1.x, cs1.z);
      si[0] = pair(cs0.y, cs0.w);
      si[1] = pair(cs1.y, cs1.w);
      nsi[0] = pair(-cs0.y, -cs0.w);
      nsi[1] = pair(-cs1.y, -cs1.w);
    }
    T *wq = static_cast<T *>(a.qo) + (long long)cur.token * a.sqo, *wk = static_cast<T *>(a.ko) + (long long)cur.token * a.sko - a.hq * D;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int h = cur.h0 + u * hpw;
      if (!live || h >= a.heads) continue;
      f32x2 x[4];              // the lane's channels d0 .. d0 + 3, d1 .. d1 + 3
      v[u].get(x);
      const float inv = inv_sqrt(fmaf(ss[u], inv_d, a.eps));
      const float *g = gains[h < a.hq ? 0 : 1];
      const ulonglong2 g0 = *reinterpret_cast<const ulonglong2 *>(g + d0), g1 = *reinterpret_cast<const ulonglong2 *>(g + d1);
      const f32x2 gx[4] = {g0.x, g0.y, g1.x, g1.y}, inv2 = pair(inv, inv);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = fmul2(fmul2(x[i], inv2), gx[i]);
      if constexpr (ROPE && HALVES) {          // (x[0], x[1]) with (x[2], x[3])
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const f32x2 p0 = x[i], p1 = x[2 + i];
          x[i] = ffma2(p1, nsi[i], fmul2(p0, co[i]));
          x[2 + i] = ffma2(p0, si[i], fmul2(p1, co[i]));
        }
      } else if constexpr (ROPE) {             // the two of each pair
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 p = unpair(x[i]);
          const float4 cs = i < 2 ? cs0 : cs1;
          const float c = i & 1 ? cs.z : cs.x, sn = i & 1 ? cs.w : cs.y;
          x[i] = ffma2(pair(p.y, p.x), pair(-sn, sn), fmul2(x[i], pair(c, c)));
        }
      }
      float y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = unpair(x[i]).x;
        y[2 * i + 1] = unpair(x[i]).y;
      }
      Lane8<T, HALVES>::store((h < a.hq ? wq : wk) + h * D, j, half, y);
    }
  }
}

template <typename T, bool HALVES, bool ROPE, int UNROLL> st_status launch_groups(const QkArgs &a, cudaStream_t s) {
  const long long tasks = (long long)a.n_tokens * a.chunks;
  const long long want = (tasks + 7) / 8, cap = (long long)st::num_sms() * 3;
  const dim3 grid(unsigned(want < cap ? want : cap));
  switch (a.D) {
    case 32: return st::launch_pdl(qk_norm_rope<T, HALVES, ROPE, 4, UNROLL>, grid, 256, 0, s, a);
    case 64: return st::launch_pdl(qk_norm_rope<T, HALVES, ROPE, 8, UNROLL>, grid, 256, 0, s, a);
    case 72: return st::launch_pdl(qk_norm_rope<T, HALVES, ROPE, 9, UNROLL>, grid, 256, 0, s, a);
    case 80: return st::launch_pdl(qk_norm_rope<T, HALVES, ROPE, 10, UNROLL>, grid, 256, 0, s, a);
    case 96: return st::launch_pdl(qk_norm_rope<T, HALVES, ROPE, 12, UNROLL>, grid, 256, 0, s, a);
    case 128: return st::launch_pdl(qk_norm_rope<T, HALVES, ROPE, 16, UNROLL>, grid, 256, 0, s, a);
    default: return st::launch_pdl(qk_norm_rope<T, HALVES, ROPE, 0, UNROLL>, grid, 256, 0, s, a);
  }
}
// Four groups of bf16 a task, or three where that leaves fewer places empty
// (65,536 tokens, 48 heads of 128 channels: 289 us with four, 309 with three, in one run; 20 heads of 64,
// five groups: 77 and 67); two of fp32 (four spill).
template <typename T, bool HALVES, bool ROPE> st_status launch_pairing(QkArgs a, cudaStream_t s) {
  const int hpw = 32 / (a.D / 8), groups = (a.heads + hpw - 1) / hpw;
  const bool three = (groups + 2) / 3 * 3 < (groups + 3) / 4 * 4;
  const int unroll = sizeof(T) == 4 ? 2 : (three ? 3 : 4);
  a.chunks = (groups + unroll - 1) / unroll;
  if ((long long)a.n_tokens * a.chunks >= (1LL << 31) - (1LL << 24)) return ST_ERR_SHAPE;
  a.dchunk = st::make_fastdiv(uint32_t(a.chunks));
  if constexpr (sizeof(T) == 4) return launch_groups<T, HALVES, ROPE, 2>(a, s);
  else return three ? launch_groups<T, HALVES, ROPE, 3>(a, s) : launch_groups<T, HALVES, ROPE, 4>(a, s);
}
template <typename T> st_status launch(const QkArgs &a, int pairing, cudaStream_t s) {
  if (!a.table) return launch_pairing<T, false, false>(a, s);
  return pairing == ST_ROPE_HALVES ? launch_pairing<T, true, true>(a, s) : launch_pairing<T, false, true>(a, s);
}

struct Rows {
  const char *p;
  long long stride, width;     // bytes
};
// Whether n rows of a and of b share no byte.  Rows of one stride may
// interleave (columns of the same matrix).
bool disjoint(const Rows &a, const Rows &b, long long n) {
  if (!a.p || !b.p) return true;
  if (a.p + (n - 1) * a.stride + a.width <= b.p || b.p + (n - 1) * b.stride + b.width <= a.p) return true;
  if (a.stride != b.stride) return false;
  long long d = (b.p - a.p) % a.stride;
  if (d < 0) d += a.stride;
  return d >= a.width && d + b.width <= a.stride;
}
bool same(const Rows &a, const Rows &b) { return a.p == b.p && a.stride == b.stride; }

}  // namespace

ST_API st_status st_qk_norm_rope(const st_qk_desc *d, const void *q, const void *k, void *q_out, void *k_out,
                                 const float *q_gamma, const float *k_gamma, const float *rope_table,
                                 int rope_positions, const int *positions, st_stream_t stream) {
  if (!d) return ST_ERR_NULL;
  if (d->size != (int)sizeof(st_qk_desc)) return ST_ERR_SHAPE;
  if (d->n_tokens <= 0 || d->h_q < 0 || d->h_k < 0 || d->h_q + (long long)d->h_k <= 0 || d->D <= 0 || d->pos_period < 0)
    return ST_ERR_SHAPE;
  if (!(d->eps >= 0.f)) return ST_ERR_SHAPE;
  if (((long long)d->h_q + d->h_k) * d->D > (1LL << 30)) return ST_ERR_SHAPE;
  if (d->dtype != ST_F32 && d->dtype != ST_BF16) return ST_ERR_DTYPE;
  if (d->pairing != ST_ROPE_INTERLEAVED && d->pairing != ST_ROPE_HALVES) return ST_ERR_SHAPE;
  if (d->D % 8 || d->D > 256) return ST_ERR_UNSUPPORTED;
  if ((d->h_q && (!q || !q_out)) || (d->h_k && (!k || !k_out))) return ST_ERR_NULL;
  const int e = d->dtype == ST_BF16 ? 2 : 4;
  QkArgs a = {};
  const long long wq = (long long)d->h_q * d->D, wk = (long long)d->h_k * d->D;
  a.sq = d->stride_q ? d->stride_q : wq;
  a.sk = d->stride_k ? d->stride_k : wk;
  a.sqo = d->stride_q_out ? d->stride_q_out : wq;
  a.sko = d->stride_k_out ? d->stride_k_out : wk;
  if ((d->h_q && (a.sq < wq || a.sqo < wq)) || (d->h_k && (a.sk < wk || a.sko < wk))) return ST_ERR_SHAPE;
  const long long v = 16 / e;
  if (d->h_q && (a.sq % v || a.sqo % v || !st::is_aligned(q, 16) || !st::is_aligned(q_out, 16))) return ST_ERR_ALIGN;
  if (d->h_k && (a.sk % v || a.sko % v || !st::is_aligned(k, 16) || !st::is_aligned(k_out, 16))) return ST_ERR_ALIGN;
  if (!st::is_aligned(q_gamma, 4) || !st::is_aligned(k_gamma, 4) || !st::is_aligned(positions, 4)) return ST_ERR_ALIGN;
  if (rope_table) {
    if (!st::is_aligned(rope_table, 16)) return ST_ERR_ALIGN;
    if (rope_positions <= 0) return ST_ERR_SHAPE;
    const int need = d->pos_period && d->pos_period < d->n_tokens ? d->pos_period : d->n_tokens;
    if (!positions && rope_positions < need) return ST_ERR_SHAPE;
  }
  const Rows rq{d->h_q ? static_cast<const char *>(q) : nullptr, a.sq * e, wq * e};
  const Rows rk{d->h_k ? static_cast<const char *>(k) : nullptr, a.sk * e, wk * e};
  const Rows rqo{d->h_q ? static_cast<const char *>(q_out) : nullptr, a.sqo * e, wq * e};
  const Rows rko{d->h_k ? static_cast<const char *>(k_out) : nullptr, a.sko * e, wk * e};
  const long long n = d->n_tokens;
  if ((!same(rq, rqo) && !disjoint(rq, rqo, n)) || (!same(rk, rko) && !disjoint(rk, rko, n)) ||
      !disjoint(rq, rko, n) || !disjoint(rk, rqo, n) || !disjoint(rqo, rko, n))
    return ST_ERR_SHAPE;
  a.q = q;
  a.k = k;
  a.qo = q_out;
  a.ko = k_out;
  a.gq = q_gamma;
  a.gk = k_gamma;
  a.table = reinterpret_cast<const float4 *>(rope_table);
  a.positions = positions;
  a.n_pos = rope_positions;
  a.period = d->pos_period ? d->pos_period : d->n_tokens;
  a.n_tokens = d->n_tokens;
  a.hq = d->h_q;
  a.heads = d->h_q + d->h_k;
  a.D = d->D;
  a.eps = d->eps;
  a.dperiod = st::make_fastdiv(uint32_t(a.period));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return d->dtype == ST_BF16 ? launch<uint16_t>(a, d->pairing, s) : launch<float>(a, d->pairing, s);
}
