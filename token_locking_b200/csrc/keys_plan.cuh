// Work plan of the key-set kernels (attention over a key set per sequence, and
// the weight each key receives), computed on the device from the caller's
// offsets and lengths, so that a captured graph follows them as they change.
//
// A job is a run of query rows against one list of key tiles; it is cut into
// units (a block of rows, or of keys for the weight kernel) of T inner tiles
// each.  All units laid end to end, each as OV + T virtual tiles (OV: its
// start-up and epilogue in tile times), make W virtual tiles, and CTA c of nC
// takes [c chunk, (c + 1) chunk) of them: equal shares whatever the lengths,
// with a unit cut where a share ends.  A cut unit leaves partial results in
// slots (at most two per CTA: the piece a share starts in the middle of, and
// the one it leaves unfinished) that a second kernel joins in the order of the
// CTAs, so no result depends on which CTA finished first.
#pragma once
#include "common.cuh"
#include "internal.h"

namespace sl {

constexpr int KP_JOBS = SL_MAX_BATCH + 1;

struct KeyPlan {
  int q0[SL_MAX_BATCH + 1];   // first row of each sequence (clamped, ascending); [batch] = end
  int kl[SL_MAX_BATCH];       // keys of each sequence's set, in [0, n_ctx]
  int wbase[KP_JOBS + 1];     // first virtual tile of each job; [njobs] = W
  int T[KP_JOBS];             // inner tiles of a unit of the job
  int njobs, stacked, chunk, empty;   // empty: some sequence has rows and no keys
};

// One piece of a unit, as one CTA computes it.
struct KeyPiece {
  int job, unit, hk;          // row (or key) block and K/V head of the unit
  int t0, t1, T;              // inner tiles [t0, t1) of T
  int w_unit;                 // the unit's first virtual tile
};

__device__ __forceinline__ int kp_tiles(int n, int tile) { return (n + tile - 1) / tile; }

__device__ __forceinline__ int warp_incl_sum(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// Built by warp 0 (all 32 lanes); the caller synchronises the block after it.
// weight = false: attention, units of uq rows, T = prefix and own key tiles of
// kt keys, one unit per K/V head.  weight = true: units of kt keys, T = the
// row blocks of uq rows of every K/V head.
__device__ inline void key_plan_build(KeyPlan &pl, const KeyArgs &a, int uq, int kt, int n_ctas,
                                      bool weight, int lane) {
  const int B = a.batch;
  // row offsets, clamped into [0, M] and made ascending: a bad offset can only
  // shorten a sequence, never send a row index out of range
  int carry = 0;
  for (int c = 0; c <= B; c += 32) {
    const int i = c + lane;
    int v = i <= B ? min(max(a.seq_off[i], 0), a.M) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) v = max(v, __shfl_up_sync(0xffffffffu, v, o));
    v = max(v, carry);
    if (i <= B) pl.q0[i] = v;
    carry = __shfl_sync(0xffffffffu, v, 31);
  }
  __syncwarp();
  const int tp = weight ? 0 : kp_tiles(a.prefix_len, kt);
  // tiles of both layouts: the prefix in every sequence's list, or once for
  // the rows of all sequences together
  int cat = 0, own = 0, emp = 0;
  for (int b = lane; b < B; b += 32) {
    const int n = a.key_len ? min(max(a.key_len[b], 0), a.n_ctx) : a.n_ctx;
    pl.kl[b] = n;
    const int qn = pl.q0[b + 1] - pl.q0[b], nu = kp_tiles(qn, uq), to = kp_tiles(n, kt);
    cat += tp + to > 0 ? nu * (tp + to + KP_OV) : 0;
    own += to > 0 ? nu * (to + KP_OV) : 0;
    emp |= qn > 0 && tp + to == 0;
  }
  __syncwarp();
  cat = warp_sum_i(cat);
  own = warp_sum_i(own);
  emp = __any_sync(0xffffffffu, emp);
  const int rows = pl.q0[B] - pl.q0[0];
  bool stacked = false;
  if (a.stack && tp > 0) {
    // the joined layout reads the prefix once per block of rows of any
    // sequence, but each row's two partial results pass through memory
    const int once = kp_tiles(rows, uq) * (tp + KP_OV) + own;
    const int join = (int)((long long)rows * a.G * KP_JOIN_NUM / KP_JOIN_DEN);
    stacked = once + join < cat;
  }
  // jobs and their first virtual tiles
  const int njobs = B + (stacked ? 1 : 0);
  int base = 0;
  for (int c = 0; c < njobs; c += 32) {
    const int j = c + lane;
    int T = 0, cost = 0;
    if (j < njobs) {
      int nu;
      if (stacked && j == 0) {
        T = tp;
        nu = kp_tiles(rows, uq);
      } else {
        const int b = stacked ? j - 1 : j;
        const int qn = pl.q0[b + 1] - pl.q0[b];
        if (weight) {
          T = kp_tiles(qn, uq) * a.Hkv;
          nu = kp_tiles(pl.kl[b], kt);
        } else {
          T = (stacked ? 0 : tp) + kp_tiles(pl.kl[b], kt);
          nu = kp_tiles(qn, uq) * a.Hkv;
        }
      }
      if (stacked && j == 0) nu *= a.Hkv;
      cost = T > 0 ? nu * (T + KP_OV) : 0;
    }
    const int inc = warp_incl_sum(cost, lane);
    if (j < njobs) {
      pl.T[j] = T;
      pl.wbase[j] = base + inc - cost;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) {
    pl.wbase[njobs] = base;
    pl.njobs = njobs;
    pl.stacked = stacked;
    pl.empty = emp;
    const int share = (base + n_ctas - 1) / n_ctas;
    pl.chunk = max(share, KP_MIN_CHUNK);
  }
  __syncwarp();
}

// Sequence of job j, or -1 for the shared prefix's job.
__device__ __forceinline__ int kp_seq(const KeyPlan &pl, int j) { return pl.stacked ? j - 1 : j; }

// The piece of the unit at virtual tile w that ends at or before w_end; w moves
// to its end.  False once nothing is left; pieces without inner tiles (a cut
// inside the start-up share) are passed over.
__device__ __forceinline__ bool key_next(const KeyPlan &pl, int heads, int &w, int w_end, int &job,
                                         KeyPiece &p) {
  w_end = min(w_end, pl.wbase[pl.njobs]);
  while (w < w_end) {
    while (w >= pl.wbase[job + 1]) ++job;
    const int T = pl.T[job], cu = T + KP_OV;
    const int rel = w - pl.wbase[job];
    const int u = rel / cu, v0 = rel - u * cu;
    const int v1 = min(cu, v0 + (w_end - w));
    p.job = job;
    p.unit = u / heads;
    p.hk = u - p.unit * heads;
    p.T = T;
    p.t0 = max(0, v0 - KP_OV);
    p.t1 = v1 - KP_OV;
    p.w_unit = w - v0;
    w += v1 - v0;
    if (p.t1 > p.t0) return true;
  }
  return false;
}

// Slot of a CTA's piece that does not cover its unit.
__device__ __forceinline__ int kp_slot(int cta, int t0) { return 2 * cta + (t0 > 0 ? 0 : 1); }

// The CTAs whose shares meet a unit, and the tiles of CTA c's piece of it.
__device__ __forceinline__ void kp_piece_of(const KeyPlan &pl, int w_unit, int T, int c, int &t0,
                                            int &t1) {
  const int v0 = max(c * pl.chunk, w_unit) - w_unit;
  const int v1 = min((long long)(c + 1) * pl.chunk, (long long)w_unit + T + KP_OV) - w_unit;
  t0 = max(0, v0 - KP_OV);
  t1 = v1 - KP_OV;
}

}  // namespace sl
