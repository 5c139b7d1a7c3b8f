// Conditioning attention on the fp32 FMA pipes.
//
// fp32 workloads ask for 1e-4 or better, which rules out single tf32 or bf16
// products.  A CTA of 256 threads owns 64 query rows of one (unit, head): Q
// stays in shared memory, keys come in tiles of 64, thread (ty, tx) holds a
// 4 x 4 piece of the scores (rows 4 ty .. 4 ty + 3, keys tx + 16 j) and 4
// rows x 4 columns per 64 channels of the output.  The softmax is the online
// form (running max and sum per row in fp32); the probabilities replace the K
// tile in shared memory, so two CTAs fit an SM at head dim 128 and one loads
// while the other multiplies.
//
// Bound by the pieces of shared memory that feed 4 x 4 products a thread (72
// channels: issue slots 61%, shared memory 44%, FMA pipe 40%): 16,384 rows x 16
// heads, 512 keys of 128 channels 2531 us (27 TFLOP/s), 300 of 72 channels 1293 us
// (17.5; a second 64-channel piece holds 8).  Asynchronous copies of the next K and
// V tile under the products were no faster.  A tile of fewer rows costs what 64 do:
// one query of 24 heads on 8, 2 x 20,736 keys of 128 channels 439 us, of 52 us that
// reading K and V takes.
#include <math.h>

#include "cond.cuh"

namespace {

constexpr int BM = 64, BN = 64, NT = 256;

// Channels c .. c + 3 of a row (n of them exist); rows of 16-byte vectors where
// the head dim, the strides and the pointers allow.
__device__ __forceinline__ float4 load4(const float *p, int n, bool vec) {
  if (vec) return *reinterpret_cast<const float4 *>(p);
  return make_float4(p[0], n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
}

// Products of the thread's 4 rows with NE of its keys (16 apart); the others of
// a short tile hold no key.
template <int NE>
__device__ __forceinline__ void scores(float (&s)[4][4], const float *q, const float *k, int pitch, int DP) {
#pragma unroll 2
  for (int d = 0; d < DP; d += 4) {
    float4 a[4], b[NE];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4 *>(q + i * pitch + d);
#pragma unroll
    for (int e = 0; e < NE; ++e) b[e] = *reinterpret_cast<const float4 *>(k + 16 * e * pitch + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < NE; ++e) {
        s[i][e] = fmaf(a[i].x, b[e].x, s[i][e]);
        s[i][e] = fmaf(a[i].y, b[e].y, s[i][e]);
        s[i][e] = fmaf(a[i].z, b[e].z, s[i][e]);
        s[i][e] = fmaf(a[i].w, b[e].w, s[i][e]);
      }
  }
}

// NC: 64-channel chunks of the head (D <= 64 * NC).  ANY: tokens may lie at a
// two-level stride, and a block may take item after item (under a budget); apart
// because the divisions and the loop cost every other call (a tiny one 8.4 for
// 8.0 us, 16,384 rows x 16 heads, 512 keys of 128 channels 2548 for 2534).
template <int NC, bool ANY>
__global__ void __launch_bounds__(NT) cond_simt_kernel(const __grid_constant__ st::CondParams p, uint32_t row_blocks, uint32_t items, bool vec) {
  extern __shared__ float sm[];
  const int D = p.g.D, DP = (D + 3) / 4 * 4, PQ = DP + 4;
  float *sQ = sm, *sK = sQ + BM * PQ, *sV = sK + (BM * (PQ > BN + 4 ? PQ : BN + 4));
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  // (an item's Q replaces the last one's once every thread has passed the barrier
  // behind its scores, its keys behind the next)
#pragma unroll 1
  for (uint32_t item = blockIdx.x; !ANY || item < items; item += gridDim.x) {
    uint32_t x = item;
    const int rb = int(x % row_blocks);
    x /= row_blocks;
    const int sp = int(x % uint32_t(p.n_split));
    x /= uint32_t(p.n_split);
    const int w = int(x % uint32_t(p.HW)), unit = int(x / uint32_t(p.HW));
    const int rows = p.R, r0 = rb * BM;
    const int kvh = w / p.hdiv;
    st::pdl_trigger();
    st::pdl_wait();
    const float *Q = static_cast<const float *>(st::after_wait(p.q));
    const int vpr = DP / 4;                    // vectors of a row
    for (int i = tid; i < BM * vpr; i += NT) {
      const int r = i / vpr, c = (i - r * vpr) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r0 + r < rows) v = load4(Q + st::cond_row<ANY>(p, unit, w, r0 + r) + c, D - c, vec);
      *reinterpret_cast<float4 *>(sQ + r * PQ + c) = v;
    }
    float m[4], l[4], acc[4][NC][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][c][e] = 0.f;
    }
    const float sl2 = p.scale * 1.4426950408889634f;
    st::KvRange kr[2];
    int steps[2] = {0, 0};
    for (int g = 0; g < p.n_seg; ++g) {
      st::KvSeg sg = p.seg[g];
      sg.len = st::after_wait(sg.len);
      sg.offsets = st::after_wait(sg.offsets);
      kr[g] = st::kv_range(sg, st::cond_batch(p, unit));
      // (every warp looks for itself: the padding behind a prompt costs nothing)
      if (sg.mask) kr[g].n = st::last_key(st::after_wait(sg.mask) + (long long)kr[g].set * sg.L, kr[g].n, tid & 31);
      steps[g] = (kr[g].n + BN - 1) / BN;
    }
    const long long total = (long long)steps[0] + steps[1];
    const int j0 = int(total * sp / p.n_split), j1 = int(total * (sp + 1) / p.n_split);
    for (int j = j0; j < j1; ++j) {
      const int g = j < steps[0] ? 0 : 1;
      const int key0 = (g ? j - steps[0] : j) * BN;
      const st::KvSeg &sg = p.seg[g];
      const int nv = min(BN, kr[g].n - key0);
      const long long base = (long long)kr[g].set * (sg.offsets ? 0 : sg.stride_set) +
                             (long long)(kr[g].row0 + key0) * sg.stride_l + (long long)kvh * D;
      const float *Kp = static_cast<const float *>(st::after_wait(sg.k)) + base;
      const float *Vp = static_cast<const float *>(st::after_wait(sg.v)) + base;
      const unsigned char *mk = sg.mask ? st::after_wait(sg.mask) + (long long)kr[g].set * sg.L + key0 : nullptr;
      __syncthreads();
      for (int i = tid; i < BN * vpr; i += NT) {
        const int r = i / vpr, c = (i - r * vpr) * 4;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        // a key that does not count is never read, so its V cannot reach the sum
        if (r < nv && (!mk || mk[r])) {
          const long long off = (long long)r * sg.stride_l + c;
          a = load4(Kp + off, D - c, vec);
          b = load4(Vp + off, D - c, vec);
        }
        *reinterpret_cast<float4 *>(sK + r * PQ + c) = a;
        *reinterpret_cast<float4 *>(sV + r * DP + c) = b;
      }
      __syncthreads();
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
      if (nv > BN / 2) scores<4>(s, sQ + 4 * ty * PQ, sK + tx * PQ, PQ, DP);
      else if (nv > BN / 4) scores<2>(s, sQ + 4 * ty * PQ, sK + tx * PQ, PQ, DP);
      else scores<1>(s, sQ + 4 * ty * PQ, sK + tx * PQ, PQ, DP);
      bool keep[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = tx + 16 * e;
        keep[e] = c < nv && (!mk || mk[c]);
      }
      __syncthreads();                           // every thread has read the K tile
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][e] = keep[e] ? s[i][e] * sl2 : -INFINITY;
          mx = fmaxf(mx, s[i][e]);
        }
#pragma unroll
        for (int y = 8; y > 0; y >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
        const float mn = fmaxf(m[i], mx);
        const float ref = mn == -INFINITY ? 0.f : mn;   // nothing counted yet: every weight is 0
        const float corr = exp2f(m[i] - ref);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][e] = exp2f(s[i][e] - ref);
          sum += s[i][e];
          sK[(4 * ty + i) * (BN + 4) + tx + 16 * e] = s[i][e];
        }
#pragma unroll
        for (int y = 8; y > 0; y >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, y);
        l[i] = l[i] * corr + sum;
        m[i] = mn;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][c][e] *= corr;
      }
      __syncthreads();
      for (int k = 0; k < nv; k += 4) {          // (weights past nv are 0)
        float4 pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pr[i] = *reinterpret_cast<const float4 *>(sK + (4 * ty + i) * (BN + 4) + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int col = c * 64 + tx * 4;
            if (col < DP) {
              const float4 v = *reinterpret_cast<const float4 *>(sV + (k + kk) * DP + col);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float pv = kk == 0 ? pr[i].x : kk == 1 ? pr[i].y : kk == 2 ? pr[i].z : pr[i].w;
                acc[i][c][0] = fmaf(pv, v.x, acc[i][c][0]);
                acc[i][c][1] = fmaf(pv, v.y, acc[i][c][1]);
                acc[i][c][2] = fmaf(pv, v.z, acc[i][c][2]);
                acc[i][c][3] = fmaf(pv, v.w, acc[i][c][3]);
              }
            }
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 4 * ty + i;
      if (r >= rows) continue;
      const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);   // NaN scores stay NaN
      const float lse = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.6931471805599453f;
      const long long prow = (long long)sp * p.part_rows + ((long long)unit * p.HW + w) * rows + r;
      const long long off = p.part_o ? prow * D : st::cond_row<ANY>(p, unit, w, r);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = c * 64 + tx * 4 + e;
          if (d >= D) continue;
          const float y = acc[i][c][e] * inv;
          if (p.part_o) p.part_o[off + d] = y;
          else static_cast<float *>(p.o)[off + d] = y;
        }
      if (tx == 0) {
        if (p.part_o) p.part_lse[prow] = lse;
        else if (p.lse) p.lse[st::cond_lse(p, unit, w, r)] = lse;
      }
    }
    if constexpr (!ANY) return;
  }
}

template <int NC> st_status launch(const st::CondParams &p, cudaStream_t s) {
  const int DP = (p.g.D + 3) / 4 * 4, PQ = DP + 4;
  const size_t smem = size_t(BM * PQ + BM * (PQ > BN + 4 ? PQ : BN + 4) + BN * DP) * 4;
  const int row_blocks = (p.R + BM - 1) / BM;
  const long long grid = (long long)row_blocks * p.n_split * p.HW * st::cond_units(p);
  if (grid > 0x7fffffffLL) return ST_ERR_SHAPE;
  const st::Geom &g = p.g;
  bool vec = g.D % 4 == 0 && st::is_aligned(p.q, 16) && g.ss % 4 == 0 && g.st % 4 == 0 && g.stb % 4 == 0 && g.sb % 4 == 0 &&
             g.ssb % 4 == 0;
  for (int i = 0; i < p.n_seg; ++i)
    vec = vec && st::is_aligned(p.seg[i].k, 16) && st::is_aligned(p.seg[i].v, 16) && p.seg[i].stride_l % 4 == 0 &&
          p.seg[i].stride_set % 4 == 0;
  const int sms = st::num_sms();
  const bool few = sms < st::device_sms() && grid > sms * 2LL;       // a budget: the two blocks per SM that run at once
  const bool any = few || g.sblk < g.S;
  const auto kern = any ? cond_simt_kernel<NC, true> : cond_simt_kernel<NC, false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
    return ST_ERR_CUDA;
  return st::launch_pdl(kern, dim3(unsigned(few ? sms * 2 : grid)), dim3(NT), smem, s, p, uint32_t(row_blocks), uint32_t(grid), vec);
}

}  // namespace

namespace st {

st_status cond_simt(const CondParams &p, cudaStream_t s) {
  if (p.g.D > 128) return ST_ERR_UNSUPPORTED;
  return p.g.D <= 64 ? launch<1>(p, s) : launch<2>(p, s);
}

}  // namespace st
