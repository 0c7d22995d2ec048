// Work plan of the key-set kernels (attention over a key set per sequence, and
// the weight each key receives), computed on the device from the caller's
// offsets and lengths, so that a captured graph follows them as they change.
//
// A job is a run of query rows against one list of key tiles; it is cut into
// units (a block of rows, or of keys for the weight kernel) of T inner tiles
// each.  All units laid end to end, each as ov + T virtual tiles (ov: its
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
  int q0[SL_MAX_BATCH + 1];   // first row of each sequence (clamped, ascending); from [batch] the end
  int kl[SL_MAX_BATCH];       // keys of each sequence's set, in [0, n_ctx]
  int wbase[KP_JOBS + 1];     // first virtual tile of each job; from [njobs] W
  int T[KP_JOBS];             // inner tiles of a unit of the job
  int nu[KP_JOBS];            // units of the job per K/V head
  int ubase[KP_JOBS + 1];     // first unit of each job, counted over all; from [njobs] their number
  int njobs, stacked, chunk, per, ov, heads, empty;   // empty: some sequence has rows and no keys
};

// One piece of a unit, as one CTA computes it.
struct KeyPiece {
  int job, unit, hk;          // row (or key) block and K/V head of the unit
  int t0, t1, T;              // inner tiles [t0, t1) of T
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

// Built by one warp (all 32 lanes); the caller synchronises the block after it.
// weight = false: attention, units of uq rows, T = prefix and own key tiles of
// kt keys, one unit per K/V head.  weight = true: units of kt keys, T = the
// row blocks of uq rows of every K/V head.  A lane holds sequences `lane` and
// `32 + lane`: every operand is loaded at once and the rest is registers, since
// all other warps of the launch wait for it.
__device__ inline void key_plan_build(KeyPlan &pl, const KeyArgs &a, int uq, int kt, int n_ctas,
                                      bool weight, int lane) {
  static_assert(SL_MAX_BATCH == 64, "two sequences per lane");
  const int ov = a.ov;
  const int B = a.batch, b0 = lane, b1 = lane + 32;
  int v0 = a.seq_off[min(b0, B)], v1 = a.seq_off[min(b1, B)], ve = a.seq_off[B];
  int k0 = a.n_ctx, k1 = a.n_ctx;
  if (a.key_len) {
    k0 = a.key_len[min(b0, B - 1)];
    k1 = a.key_len[min(b1, B - 1)];
  }
  // row offsets, clamped into [0, M] and made ascending: a bad offset can only
  // shorten a sequence, never send a row index out of range; sequences behind
  // the last have no rows
  v0 = min(max(v0, 0), a.M);
  v1 = min(max(v1, 0), a.M);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    v0 = max(v0, __shfl_up_sync(0xffffffffu, v0, o));
    v1 = max(v1, __shfl_up_sync(0xffffffffu, v1, o));
  }
  v1 = max(v1, __shfl_sync(0xffffffffu, v0, 31));
  ve = max(min(max(ve, 0), a.M), __shfl_sync(0xffffffffu, v1, 31));
  k0 = b0 < B ? min(max(k0, 0), a.n_ctx) : 0;
  k1 = b1 < B ? min(max(k1, 0), a.n_ctx) : 0;
  const int first = __shfl_sync(0xffffffffu, v0, 0);
  int e0 = __shfl_down_sync(0xffffffffu, v0, 1), e1 = __shfl_down_sync(0xffffffffu, v1, 1);
  const int v1_0 = __shfl_sync(0xffffffffu, v1, 0);
  if (lane == 31) {
    e0 = v1_0;
    e1 = ve;
  }
  pl.q0[b0] = v0;
  pl.q0[b1] = v1;
  pl.kl[b0] = k0;
  pl.kl[b1] = k1;
  const int rows = ve - first;
  const int tp = weight ? 0 : kp_tiles(a.prefix_len, kt);
  const int u0 = kp_tiles(e0 - v0, uq), u1 = kp_tiles(e1 - v1, uq);   // row blocks
  const int t0 = kp_tiles(k0, kt), t1 = kp_tiles(k1, kt);             // own key tiles
  // tiles of both layouts: the prefix in every sequence's list, or once for
  // the rows of all sequences together
  bool stacked = false;
  const bool empty = __any_sync(0xffffffffu, (u0 > 0 && tp + t0 == 0) || (u1 > 0 && tp + t1 == 0));
  const int nu_p = kp_tiles(rows, uq);
  if (a.stack && tp > 0) {
    const int cat = __reduce_add_sync(0xffffffffu, u0 * (tp + t0 + ov) + u1 * (tp + t1 + ov));
    const int own = __reduce_add_sync(
        0xffffffffu, (t0 > 0 ? u0 * (t0 + ov) : 0) + (t1 > 0 ? u1 * (t1 + ov) : 0));
    // the joined layout reads the prefix once per block of rows of any
    // sequence, but each row's two partial results pass through memory
    const int once = nu_p * (tp + ov) + own;
    const int join = (int)((long long)rows * a.G * KP_JOIN_NUM / KP_JOIN_DEN);
    stacked = once + join < cat;
  }
  // jobs (the shared prefix first, where it is one) and their first virtual tiles
  const int sh = stacked ? 1 : 0;
  const int T0 = weight ? u0 * a.Hkv : (stacked ? 0 : tp) + t0;
  const int T1 = weight ? u1 * a.Hkv : (stacked ? 0 : tp) + t1;
  const int x0 = T0 > 0 ? (weight ? t0 : u0 * a.Hkv) : 0, c0 = x0 * (T0 + ov);
  const int x1 = T1 > 0 ? (weight ? t1 : u1 * a.Hkv) : 0, c1 = x1 * (T1 + ov);
  const int xp = stacked ? nu_p * a.Hkv : 0, cp = xp * (tp + ov);
  pl.T[b0 + sh] = T0;
  pl.T[b1 + sh] = T1;
  pl.nu[b0 + sh] = max(weight ? t0 : u0, 1);
  pl.nu[b1 + sh] = max(weight ? t1 : u1, 1);
  const int total = cp + __reduce_add_sync(0xffffffffu, c0 + c1);
  int share = (total + n_ctas - 1) / n_ctas;
  // the same in units, and the longest of them
  const int y0 = warp_incl_sum(x0, lane), y1 = warp_incl_sum(x1, lane);
  const int uhalf = xp + __shfl_sync(0xffffffffu, y0, 31);
  const int U = uhalf + __shfl_sync(0xffffffffu, y1, 31);
  const int longest = ov + __reduce_max_sync(
      0xffffffffu, max(stacked ? tp : 0, max(x0 > 0 ? T0 : 0, x1 > 0 ? T1 : 0)));
  int per = (U + n_ctas - 1) / n_ctas;
  // (a joint prefix passes every row through memory either way)
  if ((long long)per * longest > share + (stacked ? 0 : a.join_cost)) per = 0;
  share = max(share, a.min_chunk);
  // A prefix that every sequence's list begins with is read by all of them: where
  // that costs little, each sequence's units begin with a share, so that CTAs of
  // different sequences run through it together and it comes from memory once
  // (four sequences over 16384 keys, 8 tiles apart: 1.1 GB of 0.27 read).
  int d0 = c0, d1 = c1;
  if (!per && !stacked && tp > 0) {
    const int most = share + share / 32;
    for (int ch = share; ch <= most; ch += share / 64 + 1) {
      const int n0 = kp_tiles(c0, ch), n1 = kp_tiles(c1, ch);
      if ((int)__reduce_add_sync(0xffffffffu, n0 + n1) > n_ctas) continue;
      share = ch;
      d0 = n0 * ch;
      d1 = n1 * ch;
      break;
    }
  }
  const int i0 = warp_incl_sum(d0, lane), i1 = warp_incl_sum(d1, lane);
  const int half = cp + __shfl_sync(0xffffffffu, i0, 31);
  const int W = half + __shfl_sync(0xffffffffu, i1, 31);
  pl.ubase[b0 + sh] = xp + y0 - x0;
  pl.ubase[b1 + sh] = uhalf + y1 - x1;
  pl.wbase[b0 + sh] = cp + i0 - d0;
  pl.wbase[b1 + sh] = half + i1 - d1;
  if (lane == 0) {
    if (stacked) {
      pl.T[0] = tp;
      pl.nu[0] = max(nu_p, 1);
      pl.wbase[0] = pl.ubase[0] = 0;
    }
    pl.q0[64] = ve;
    pl.wbase[64 + sh] = W;
    pl.ubase[64 + sh] = U;
    pl.njobs = B + sh;
    pl.stacked = stacked;
    pl.ov = ov;
    pl.heads = a.Hkv;
    pl.empty = empty;
    pl.chunk = share;
    pl.per = per;
  }
  __syncwarp();
}

// The plan of a launch, for the kernel that follows it: written by one block
// (`n` threads, the plan complete and synchronised), read by all of the next.
constexpr int KP_WORDS = sizeof(KeyPlan) / 4;
static_assert(KP_WORDS <= KEY_PLAN_WORDS, "the workspace holds the plan");
__device__ __forceinline__ void key_plan_publish(const KeyPlan &pl, int *to, int tid, int n) {
  for (int i = tid; i < KP_WORDS; i += n) to[i] = reinterpret_cast<const int *>(&pl)[i];
}
__device__ __forceinline__ void key_plan_fetch(KeyPlan &pl, const int *from, int tid, int n) {
  for (int i = tid; i < KP_WORDS; i += n) reinterpret_cast<int *>(&pl)[i] = __ldcg(from + i);
}

// Sequence of job j, or -1 for the shared prefix's job.
__device__ __forceinline__ int kp_seq(const KeyPlan &pl, int j) { return pl.stacked ? j - 1 : j; }

// The job whose virtual tiles (or units) hold `at` (all lanes of a warp).
__device__ __forceinline__ int kp_job_at(const KeyPlan &pl, const int *base, int at, int lane) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < KP_JOBS; i += 32)
    n += __popc(__ballot_sync(0xffffffffu, i + lane < pl.njobs && at >= base[min(i + lane + 1, KP_JOBS)]));
  return min(n, pl.njobs - 1);
}

// CTA c's share: virtual tiles [w, w_end), or where shares are whole units, units
// w, w + n_ctas, ... below w_end, so that the CTAs work on neighbouring units at a
// time and a head's keys come from memory once (a run of neighbouring units per
// CTA read 714 MB for 168 at 4 x 2048 rows over 1536 keys, in 1.18 times the time).
__device__ __forceinline__ void key_begin(const KeyPlan &pl, int c, int lane, int &w, int &w_end,
                                          int &job) {
  const int W = pl.wbase[pl.njobs];
  if (pl.per) {
    w = c;
    w_end = pl.ubase[pl.njobs];
  } else {
    w = (int)min((long long)c * pl.chunk, (long long)W);
    w_end = (int)min((long long)(c + 1) * pl.chunk, (long long)W);
  }
  job = kp_job_at(pl, pl.per ? pl.ubase : pl.wbase, w, lane);
}

// Units follow one another head by head, so that the row blocks of a head meet its
// keys together (1 to 3 % of the time); of a joint prefix's job, block by block
// (head by head took 3 % more at two blocks of 256 rows over 8192 keys).
__device__ __forceinline__ void kp_unit_of(const KeyPlan &pl, int job, int u, int &unit, int &hk) {
  const bool by_block = pl.stacked && job == 0;
  const int d = by_block ? pl.heads : pl.nu[job], q = u / d, r = u - q * d;
  unit = by_block ? q : r;
  hk = by_block ? r : q;
}

// The piece of the unit at virtual tile w that ends at or before w_end (or the
// whole unit w); w moves behind it.  False once nothing is left; pieces without
// inner tiles (a cut inside the start-up share) are passed over.
__device__ __forceinline__ bool key_next(const KeyPlan &pl, int &w, int w_end, int &job,
                                         KeyPiece &p) {
  if (pl.per) {
    if (w >= w_end) return false;
    while (w >= pl.ubase[job + 1]) ++job;
    p.job = job;
    kp_unit_of(pl, job, w - pl.ubase[job], p.unit, p.hk);
    p.T = p.t1 = pl.T[job];
    p.t0 = 0;
    w += gridDim.x;
    return true;
  }
  while (w < w_end) {
    while (w >= pl.wbase[job + 1]) ++job;
    const int T = pl.T[job], cu = T + pl.ov;
    const int rel = w - pl.wbase[job];
    const int u = rel / cu, v0 = rel - u * cu;
    if (u >= pl.ubase[job + 1] - pl.ubase[job]) {   // behind the job's last unit
      w = pl.wbase[job + 1];
      continue;
    }
    const int v1 = min(cu, v0 + (w_end - w));
    p.job = job;
    kp_unit_of(pl, job, u, p.unit, p.hk);
    p.T = T;
    p.t0 = max(0, v0 - pl.ov);
    p.t1 = v1 - pl.ov;
    w += v1 - v0;
    if (p.t1 > p.t0) return true;
  }
  return false;
}

// Slot of a CTA's piece that does not cover its unit.
__device__ __forceinline__ int kp_slot(int cta, int t0) { return 2 * cta + (t0 > 0 ? 0 : 1); }

// Division by a number that is known before many of them: n / d for 0 <= n < 2^31.
// With s = ceil(log2 d) - 1 and m = ceil(2^(32 + s) / d) < 2^32, m d exceeds
// 2^(32 + s) by less than d <= 2^(s + 1), so n m / 2^(32 + s) is too large by less
// than n / 2^31 / d < 1 / d, and its whole part is that of n / d.
struct FastDiv {
  uint32_t m;
  int s;                      // -1: d = 1
  __host__ __device__ static FastDiv of(int d) {
    FastDiv f{0u, -1};
    while ((2ll << f.s + 1) < 2ll * d) ++f.s;
    if (f.s >= 0) f.m = (uint32_t)(((1ull << (32 + f.s)) + d - 1) / d);
    return f;
  }
  __device__ __forceinline__ int div(int n) const {
    return s < 0 ? n : (int)(__umulhi((uint32_t)n, m) >> s);
  }
};

// The shares that meet a unit of T tiles: the first, the last, and CTA c's tiles
// of it.
__device__ __forceinline__ int kp_first(const KeyPlan &pl, FastDiv chunk, int w_unit) {
  return pl.per ? 0 : chunk.div(w_unit);
}
__device__ __forceinline__ int kp_last(const KeyPlan &pl, FastDiv chunk, int w_unit, int T) {
  return pl.per ? 0 : chunk.div(w_unit + T + pl.ov - 1);
}
__device__ __forceinline__ void kp_piece_of(const KeyPlan &pl, int w_unit, int T, int c, int &t0,
                                            int &t1) {
  if (pl.per) {
    t0 = 0;
    t1 = T;
    return;
  }
  const int v0 = max(c * pl.chunk, w_unit) - w_unit;
  const int v1 = min((long long)(c + 1) * pl.chunk, (long long)w_unit + T + pl.ov) - w_unit;
  t0 = max(0, v0 - pl.ov);
  t1 = v1 - pl.ov;
}

}  // namespace sl
