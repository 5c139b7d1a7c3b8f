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
// with shuffles.  A warp task is UNROLL such groups of heads of one token,
// loaded before any is used; the task's row of the table is read once for all
// of them.  One token is spread over as many warps as it has groups, so a
// single token costs one trip to memory.
#include "common.cuh"

namespace {

constexpr int UNROLL = 4;

struct QkArgs {
  const void *q, *k;
  void *qo, *ko;
  long long sq, sk, sqo, sko;
  const float *gq, *gk;
  const float4 *table;
  const int *positions;
  int n_pos, period, n_tokens, hq, hk, D;
  float eps;
  int chunks_q, chunks;        // tasks of a token: of Q, in all
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
  __device__ __forceinline__ void get(float *x) const {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
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
  __device__ __forceinline__ void get(float *x) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ static void store(float *p, int j, int half, const float *x) {
    *reinterpret_cast<float4 *>(p + first(j)) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + second(j, half)) = make_float4(x[4], x[5], x[6], x[7]);
  }
};

template <typename T, bool HALVES, bool ROPE>
__global__ void __launch_bounds__(256) qk_norm_rope(const __grid_constant__ QkArgs a) {
  const int lane = threadIdx.x & 31;
  const int lph = a.D >> 3, hpw = 32 / lph;    // lanes of a head, heads of a warp
  const int hs = lane / lph, j = lane - hs * lph;
  const bool live = hs < hpw;
  const int half = a.D >> 1;
  const uint32_t tasks = uint32_t(a.n_tokens) * uint32_t(a.chunks);
  const uint32_t warps = gridDim.x * (blockDim.x >> 5);
  st::pdl_trigger();
  st::pdl_wait();
  const T *q = static_cast<const T *>(st::after_wait(a.q)), *k = static_cast<const T *>(st::after_wait(a.k));
  const float *gq = st::after_wait(a.gq), *gk = st::after_wait(a.gk);
  const float4 *table = st::after_wait(a.table);
  const int *positions = st::after_wait(a.positions);
  // the lane's gains of Q and of K
  float gains[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = HALVES ? (i < 4 ? 4 * j + i : half + 4 * j + i - 4) : 8 * j + i;
    gains[0][i] = gq && live ? gq[d] : 1.f;
    gains[1][i] = gk && live ? gk[d] : 1.f;
  }
  const float inv_d = 1.f / float(a.D);
  for (uint32_t t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); t < tasks; t += warps) {
    const uint32_t token = st::fdiv(t, a.dchunk);
    int c = int(t - token * uint32_t(a.chunks));
    const bool is_k = c >= a.chunks_q;
    if (is_k) c -= a.chunks_q;
    const int H = is_k ? a.hk : a.hq;
    const T *src = is_k ? k + (long long)token * a.sk : q + (long long)token * a.sq;
    T *dst = is_k ? static_cast<T *>(a.ko) + (long long)token * a.sko : static_cast<T *>(a.qo) + (long long)token * a.sqo;
    const int h0 = c * UNROLL * hpw + hs;
    Lane8<T, HALVES> v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (live && h0 + u * hpw < H) v[u].load(src + (long long)(h0 + u * hpw) * a.D, j, half);
    float4 cs0 = make_float4(1.f, 0.f, 1.f, 0.f), cs1 = cs0;
    if constexpr (ROPE) {
      const int pos = positions ? positions[token] : int(token - st::fdiv(token, a.dperiod) * uint32_t(a.period));
      if (pos >= 0 && pos < a.n_pos && live) {   // a position outside the table turns nothing
        const float4 *row = table + (long long)pos * (a.D >> 2) + 2 * j;
        cs0 = row[0];
        cs1 = row[1];
      }
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int h = h0 + u * hpw;
      if (c * UNROLL * hpw + u * hpw >= H) break;   // the same for the whole warp
      const bool on = live && h < H;
      float x[8];
      float ss = 0.f;
      if (on) {
        v[u].get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
      }
      // sum over the lph lanes of the head, in the order of a fixed tree
      for (int o = 1; o < lph; o <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, ss, o);
        if (j + o < lph) ss += y;
      }
      ss = __shfl_sync(0xffffffffu, ss, (hs < hpw ? hs : 0) * lph);
      if (!on) continue;
      const float inv = 1.f / sqrtf(fmaf(ss, inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * (is_k ? gains[1][i] : gains[0][i]);
      if constexpr (ROPE) {
        const float co[4] = {cs0.x, cs0.z, cs1.x, cs1.z}, si[4] = {cs0.y, cs0.w, cs1.y, cs1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float &p0 = HALVES ? x[i] : x[2 * i], &p1 = HALVES ? x[4 + i] : x[2 * i + 1];
          const float y0 = p0 * co[i] - p1 * si[i];
          p1 = p0 * si[i] + p1 * co[i];
          p0 = y0;
        }
      }
      Lane8<T, HALVES>::store(dst + (long long)h * a.D, j, half, x);
    }
  }
}

template <typename T> st_status launch(const QkArgs &a, int pairing, cudaStream_t s) {
  const long long tasks = (long long)a.n_tokens * a.chunks;
  const long long want = (tasks + 7) / 8, cap = (long long)st::num_sms() * 8;
  const int grid = int(want < cap ? want : cap);
  if (a.table)
    return pairing == ST_ROPE_HALVES ? st::launch_pdl(qk_norm_rope<T, true, true>, grid, 256, 0, s, a)
                                     : st::launch_pdl(qk_norm_rope<T, false, true>, grid, 256, 0, s, a);
  return st::launch_pdl(qk_norm_rope<T, false, false>, grid, 256, 0, s, a);
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
  a.hk = d->h_k;
  a.D = d->D;
  a.eps = d->eps;
  const int heads = 32 / (d->D / 8) * UNROLL;  // heads of a task
  a.chunks_q = (d->h_q + heads - 1) / heads;
  a.chunks = a.chunks_q + (d->h_k + heads - 1) / heads;
  if ((long long)a.n_tokens * a.chunks >= (1LL << 31) - (1LL << 24)) return ST_ERR_SHAPE;
  a.dchunk = st::make_fastdiv(uint32_t(a.chunks));
  a.dperiod = st::make_fastdiv(uint32_t(a.period));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return d->dtype == ST_BF16 ? launch<uint16_t>(a, d->pairing, s) : launch<float>(a, d->pairing, s);
}
