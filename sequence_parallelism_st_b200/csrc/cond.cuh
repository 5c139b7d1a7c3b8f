// Conditioning attention (st_attn_cross, st_attn_prefix): what the host plans
// for a launch and what its kernels share.
//
// Queries come in units of R rows that attend to the same keys: a unit is one
// (batch, frame), or a whole batch when its frames and tokens are uniformly
// strided, or the batches that share a prefix when few rows are packed
// together.  Keys come in up to two segments (the prefix, then the own keys),
// each the sets of one st_kv_desc.
#pragma once

#include "attn_geom.cuh"

namespace st {

struct KvSeg {
  const void *k, *v;
  const int *len, *offsets;
  const unsigned char *mask;
  long long stride_set, stride_l;
  int L, n_sets, per;          // per: batches that share a set
  int n_rows;                  // packed: rows in all (0: padded sets)
};

// First row (packed; 0 otherwise) and number of keys of a set.
struct KvRange {
  int set, row0, n;
};
__device__ __forceinline__ KvRange kv_range(const KvSeg &g, int b) {
  KvRange r;
  r.set = b / g.per;
  r.row0 = 0;
  r.n = g.L;
  if (g.offsets) {
    int a = g.offsets[r.set], z = g.offsets[r.set + 1];
    a = min(max(a, 0), g.n_rows);
    z = min(max(z, a), g.n_rows);
    r.row0 = a;
    r.n = min(z - a, g.L);
  } else if (g.len) {
    r.n = min(max(g.len[r.set], 0), g.L);
  }
  return r;
}

// Keys up to the last of the first n that the mask lets count (a warp's answer,
// looked for from the end, 256 at a time).
__device__ __forceinline__ int last_key(const unsigned char *mask, int n, int lane) {
#pragma unroll 1
  while (n > 0) {
    int last = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = n - 1 - lane - 32 * i;
      if (k >= 0 && mask[k]) last = max(last, k + 1);
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (last) return last;
    n -= 256;
  }
  return 0;
}

struct CondParams {
  Geom g;                      // Q and O by unit: g.B batches (or groups of batches) of g.T frames of R0 rows
  int R0;                      // query rows of a unit (g.S)
  int R;                       // R0 * G: rows once the heads of a group are packed into them
  int bm;                      // batches a unit packs (their rows follow one another)
  int G;                       // heads packed into the rows (H / H_kv), or 1
  int HW;                      // heads walked: H / G
  int hdiv;                    // kv head = walked head / hdiv
  int T0, S0;                  // frames and queries of the call
  KvSeg seg[2];
  int n_seg;
  KvSeg own;                   // attended by the combine kernel (packed batches); own.k NULL: none
  int n_split;                 // parts the keys of a unit are split into
  int spread;                  // parts that one work item takes side by side (1, or the tiles of an item)
  float scale;
  const void *q;
  void *o;
  float *lse;
  int o_f32;
  // Partials (n_split > 1, or own keys left to the combine kernel): normalised
  // fp32 rows [part][row][D] and their natural-log LSE [part][row], with
  // row = (unit * HW + walked head) * R + packed row; NULL: written to o.
  float *part_o, *part_lse;
  long long part_rows;
};

__host__ __device__ __forceinline__ int cond_units(const CondParams &p) { return p.g.B * p.g.T; }
// First batch of a unit.
__device__ __forceinline__ int cond_batch(const CondParams &p, int unit) { return unit / p.g.T * p.bm; }
// Packed row r of walked head w: element offset in Q and O.  BLOCKS: tokens may
// lie at a two-level stride (fp32; the tensor maps of bf16 take one).
template <bool BLOCKS>
__device__ __forceinline__ long long cond_row(const CondParams &p, int unit, int w, int r) {
  const int s = r / p.G, g = r - s * p.G;
  const int b = unit / p.g.T, t = unit - b * p.g.T;
  const long long token = BLOCKS ? p.g.token(s) : (long long)s * p.g.ss;
  return p.g.frame(b, t) + token + (long long)(w * p.G + g) * p.g.D;
}
// Its index in the caller's LSE [B, T, H, S].
__device__ __forceinline__ long long cond_lse(const CondParams &p, int unit, int w, int r) {
  const int s = r / p.G, g = r - s * p.G;
  long long f = unit;                          // frame of the call, b * T + t
  int s0 = s;
  if (p.g.T == 1) {                            // the unit's rows run over bm * T frames
    const int t = s / p.S0;
    s0 = s - t * p.S0;
    f = (long long)unit * p.bm * p.T0 + t;
  }
  return (f * p.g.H + (w * p.G + g)) * p.S0 + s0;
}

// SMs of the current device, whatever the thread's budget.
int device_sms();

st_status cond_simt(const CondParams &p, cudaStream_t s);
// What a kernel walks: rows of a tile, tiles of a work item, keys per step.
struct CondTile {
  int rows, tiles, keys;
};
CondTile cond_tile(int D);
st_status cond_sm100(const CondParams &p, cudaStream_t s);
unsigned int read_and_clear_cond_error(cudaStream_t stream, cudaError_t *err);

}  // namespace st
