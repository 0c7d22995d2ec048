// Attention of the active rows over a key set per sequence: the first key_len
// cache entries or a list of kept positions (what an eviction leaves), and a
// prefix shared by the whole batch.
//
// The pages keep the keys and values of every locked position and let each
// active row attend to all N of them, O(M N d) a step (Paper-Notes, "permanent
// locking"; gist.science/nl section 2, "Complexiteitsvermindering").  A row's
// key set here is what the caller kept of them:
//   z_jhn = scale q_jh . k_n,  lse_jh = log sum_n exp(z_jhn),
//   o_jh = sum_n exp(z_jhn - lse_jh) v_n   over the prefix and the sequence's set,
// in one pass over the keys with a running maximum and sum.  The G = H / Hkv
// query heads of a K/V head share its tiles: a tile's rows are (query row,
// head of the group) pairs.  A row without keys has o = 0, lse = -inf.
//
// This file holds the fp32-arithmetic kernel (fp32 models, and bf16 heads the
// tensor-core kernel does not take) and the kernel that joins partial rows.
#include "common.cuh"
#include "keys_common.cuh"
#include "keys_plan.cuh"

namespace sl {

namespace {
constexpr int KS_T = 64;              // packed rows and keys of a tile
constexpr int KS_THREADS = 256;
}  // namespace

// Rows (qr, g) packed as qr * G + g; 64 packed rows against 64 keys at a time,
// 256 threads as 16 x 16: thread (ty, tx) holds scores of rows 4 ty + i and
// keys tx + 16 j, and of the output rows 4 ty + i the columns 4 tx + 64 c.
// Operands are staged in shared memory as fp32 with rows padded by four floats
// (16 rows read at a time then fall into distinct banks), four threads a row, a
// key's position read a tile ahead.  Bound by shared memory reads (8 16-byte reads
// per 64 multiply-adds), and in small calls by latency: 200 and 159 rows of 8 heads
// of 64 over 192 and 130 keys take 24 us with shares of one tile, 36 us of two.
template <typename T>
__global__ void __launch_bounds__(KS_THREADS) key_attn_simt_kernel(const KeyArgs a) {
  extern __shared__ float4 ks_smem4[];
  __shared__ KeyPlan pl;
  float *smem = reinterpret_cast<float *>(ks_smem4);
  const int D = a.D, ld = D + 4;
  float *sq = smem, *sk = sq + KS_T * ld, *sv = sk + KS_T * ld, *sp = sv + KS_T * ld;
  constexpr int LP = KS_T + 4;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, lane = tid & 31;
  const int QR = KS_T / a.G;                        // query rows of a unit
  pdl_wait();
  if (tid < 32) key_plan_build(pl, a, QR, KS_T, gridDim.x, false, lane);
  __syncthreads();
  if (blockIdx.x == 0) key_plan_publish(pl, a.plan, tid, KS_THREADS);
  pdl_trigger();
  const int tp = kp_tiles(a.prefix_len, KS_T);
  const int lr = tid >> 2, lc = (tid & 3) * 4;      // row and first column this thread stages
  const float c2 = a.scale * KEY_LOG2E;

  int w, w_end, job;
  key_begin(pl, blockIdx.x, lane, w, w_end, job);
  KeyPiece pc;
  while (key_next(pl, w, w_end, job, pc)) {
    const int b = kp_seq(pl, pc.job);
    const int r0 = (b < 0 ? pl.q0[0] : pl.q0[b]) + pc.unit * QR;
    const int rn = min(QR, (b < 0 ? pl.q0[a.batch] : pl.q0[b + 1]) - r0) * a.G;   // packed rows
    __syncthreads();
    {
      const int g = lr / a.G;
      const T *src = (const T *)a.q + (r0 + g) * a.ld_q + (pc.hk * a.G + lr - g * a.G) * D;
#pragma unroll 4
      for (int c = lc; c < D; c += 16)
        *reinterpret_cast<float4 *>(sq + lr * ld + c) =
            lr < rn ? load4(src + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // cache position of this thread's key of tile t, -1 where there is none
    auto entry = [&](int t) {
      const bool pre = b < 0 || (!pl.stacked && t < tp);
      const int i = (pre || pl.stacked ? t : t - tp) * KS_T + lr;
      if (t >= pc.t1 || i >= (pre ? a.prefix_len : pl.kl[b])) return -1;
      return pre ? i : key_pos(a, b, i);
    };
    int nxt = entry(pc.t0);
    float m[4], l[4];
    float4 acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      acc[i][0] = acc[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int t = pc.t0; t < pc.t1; ++t) {
      // the tile's keys: of the prefix, then of the sequence's own set
      const bool pre = b < 0 || (!pl.stacked && t < tp);
      const int i0 = (pre || pl.stacked ? t : t - tp) * KS_T;
      const int nv = min(KS_T, (pre ? a.prefix_len : pl.kl[b]) - i0);
      const int pos = nxt;
      const long long off = pre ? pos * a.ld_p + pc.hk * D
                                : ((long long)b * a.n_ctx + pos) * a.ld_kv + pc.hk * D;
      const T *kr = (const T *)(pre ? a.kp : a.k) + off, *vr = (const T *)(pre ? a.vp : a.v) + off;
      __syncthreads();
#pragma unroll 4
      for (int c = lc; c < D; c += 16) {
        float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
        if (pos >= 0) {
          kv = load4(kr + c);
          vv = load4(vr + c);
        }
        *reinterpret_cast<float4 *>(sk + lr * ld + c) = kv;
        *reinterpret_cast<float4 *>(sv + lr * ld + c) = vv;
      }
      nxt = entry(t + 1);
      __syncthreads();
      float s[4][4] = {};
      for (int c = 0; c < D; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(sq + (4 * ty + i) * ld + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * j) * ld + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
            s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
            s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
            s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mt = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = tx + 16 * j < nv ? s[i][j] * c2 : -INFINITY;
          mt = fmaxf(mt, s[i][j]);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        const float mn = fmaxf(m[i], mt);
        const float ms = mn == -INFINITY ? 0.f : mn;      // no finite score yet: all p = 0
        const float al = exp2f(m[i] - ms);                // 2^-inf = 0 at the first tile
        float rs = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = exp2f(s[i][j] - ms);
          sp[(4 * ty + i) * LP + tx + 16 * j] = p;
          rs += p;
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, o);
        l[i] = l[i] * al + rs;
        m[i] = mn;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          acc[i][c].x *= al;
          acc[i][c].y *= al;
          acc[i][c].z *= al;
          acc[i][c].w *= al;
        }
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 4 * tx + 64 * c;
        if (col >= D) continue;
        for (int n = 0; n < KS_T; n += 4) {
          float4 p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4 *>(sp + (4 * ty + i) * LP + n);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 v = *reinterpret_cast<const float4 *>(sv + (n + e) * ld + col);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float pe = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
              acc[i][c].x = fmaf(pe, v.x, acc[i][c].x);
              acc[i][c].y = fmaf(pe, v.y, acc[i][c].y);
              acc[i][c].z = fmaf(pe, v.z, acc[i][c].z);
              acc[i][c].w = fmaf(pe, v.w, acc[i][c].w);
            }
          }
        }
      }
    }
    // whole unit of a sequence's full key list: final rows; else partial ones
    const bool whole = pc.t0 == 0 && pc.t1 == pc.T;
    const KeyRecs recs(a, KS_T);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * ty + i;
      if (r >= rn) continue;
      const int row = r0 + r / a.G, h = pc.hk * a.G + r % a.G;
      if (whole && !pl.stacked) {
        const float inv = key_inv(l[i]);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (4 * tx + 64 * c < D)
            store4((T *)a.o + row * a.ld_o + h * D + 4 * tx + 64 * c,
                   key_mean(acc[i][c], l[i], inv));
        if (a.lse && tx == 0)
          a.lse[(size_t)row * a.H + h] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * KEY_LN2;
        continue;
      }
      const size_t rec = whole ? key_rec_row(a, KS_T, b < 0 ? 0 : 1, row, h)
                               : key_rec_slot(kp_slot(blockIdx.x, pc.t0), KS_T, r);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (4 * tx + 64 * c < D) store4(recs.o + rec * D + 4 * tx + 64 * c, acc[i][c]);
      if (tx == 0) recs.ml[rec] = make_float2(m[i], l[i]);
    }
  }
}

// ------------------------------------------------------------------- joining --
// Partial rows (max m in base 2, sum l, unnormalised o) of one (row, head)
// joined in the order of the CTAs that left them: o = sum_i 2^(m_i - m) o_i / L,
// L = sum_i 2^(m_i - m) l_i.  Lanes over the columns.  Bound by the latency of
// the loads, so several are in flight per warp: of four rows at a time, or of
// four pieces; where there are few rows, nw warps of a block share one row's
// pieces and their sums are joined in warp order.  Without a joint prefix only
// units that a CTA's share cut have partial rows: blockIdx.x = c looks at the
// cut at the start of CTA c's share, and the first cut of a unit joins it,
// blockIdx.y sharing its rows.  With one, every row does (one part from the
// prefix, one from its sequence's own keys).  After a launch of one CTA per SM all
// blocks fit the GPU at once (twice as many took 16 us of 48 at 300 rows and 32
// heads a sequence); after one of two per SM (fp32 arithmetic, heads up to 64) they
// come in two rounds.  64 registers let four blocks share an SM and spill 164 bytes
// a thread.
constexpr int KJ_WARPS = 8, KJ_Y = 4;         // warps of a block, blocks per cut
struct JoinAcc {
  float m, l;
  float4 o;
};

__device__ __forceinline__ void join_rec(JoinAcc &x, float2 ml, float4 u) {
  const float mn = fmaxf(x.m, ml.x);
  const float ms = mn == -INFINITY ? 0.f : mn;
  const float ca = exp2f(x.m - ms), cb = exp2f(ml.x - ms);
  x.l = x.l * ca + ml.y * cb;
  x.m = mn;
  x.o.x = x.o.x * ca + u.x * cb;
  x.o.y = x.o.y * ca + u.y * cb;
  x.o.z = x.o.z * ca + u.z * cb;
  x.o.w = x.o.w * ca + u.w * cb;
}

template <typename T>
__device__ __forceinline__ void join_store(const KeyArgs &a, const JoinAcc &x, int row, int h,
                                           int lane) {
  if (4 * lane < a.D)
    store4((T *)a.o + row * a.ld_o + h * a.D + 4 * lane, key_mean(x.o, x.l, key_inv(x.l)));
  if (a.lse && lane == 0)
    a.lse[(size_t)row * a.H + h] = x.l == 0.f ? -INFINITY : (x.m + log2f(x.l)) * KEY_LN2;
}

// A unit of job j, the CTAs c0 .. c0 + n - 1 whose shares meet it.
struct JoinUnit {
  int j, wu, c0, n;
  __device__ __forceinline__ JoinUnit(const KeyPlan &pl, FastDiv chunk, int job, int w_unit) {
    j = job;
    wu = w_unit;
    c0 = kp_first(pl, chunk, wu);
    n = pl.T[j] > 0 ? kp_last(pl, chunk, wu, pl.T[j]) - c0 + 1 : 0;
  }
  // Record of packed row r in the e-th of them, or -1 if it holds none of its
  // tiles; row_rec: where a piece that is the whole unit left the row.
  __device__ __forceinline__ long long rec(const KeyPlan &pl, int e, int rt, int r,
                                           size_t row_rec) const {
    int t0, t1;
    kp_piece_of(pl, wu, pl.T[j], c0 + e, t0, t1);
    if (t1 <= t0) return -1;
    return t0 == 0 && t1 == pl.T[j] ? (long long)row_rec
                                    : (long long)key_rec_slot(kp_slot(c0 + e, t0), rt, r);
  }
};

// Warps per row: as many as leave every row a place at once.
__device__ __forceinline__ int join_warps(long long rows, long long warps) {
  return rows * 8 <= warps ? 8 : rows * 4 <= warps ? 4 : rows * 2 <= warps ? 2 : 1;
}

template <typename T>
__global__ void __launch_bounds__(32 * KJ_WARPS, 4) key_join_kernel(const KeyArgs a, int rt, int uq,
                                                                     FastDiv by_h, FastDiv by_g,
                                                                     FastDiv by_uq) {
  __shared__ KeyPlan pl;
  __shared__ JoinAcc part[KJ_WARPS][32];
  __shared__ FastDiv by_chunk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  key_plan_fetch(pl, a.plan, threadIdx.x, 32 * KJ_WARPS);
  if (threadIdx.x == 0)
    by_chunk = FastDiv::of(__ldcg(reinterpret_cast<const int *>(
        &reinterpret_cast<const KeyPlan *>(a.plan)->chunk)));
  __syncthreads();
  const FastDiv chunk = by_chunk;
  const KeyRecs recs(a, rt);
  const JoinAcc none{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  const float4 *ro = reinterpret_cast<const float4 *>(recs.o + 4 * lane);
  const bool col = 4 * lane < a.D;
  const int d4 = a.D >> 2;
  // the block's warps that share a row join their sums and write it
  auto finish = [&](JoinAcc &x, int nw, int sub, bool there, int row, int h) {
    if (nw > 1) {
      part[warp][lane] = x;
      __syncthreads();
      if (there && sub == 0)
        for (int e = 1; e < nw; ++e) {
          const JoinAcc &y = part[warp + e][lane];
          join_rec(x, make_float2(y.m, y.l), y.o);
        }
    }
    if (there && sub == 0) join_store<T>(a, x, row, h, lane);
    if (nw > 1) __syncthreads();
  };
  // pieces sub, sub + nw, ... of n, four in flight; rec(e) gives a record or -1
  auto gather = [&](JoinAcc &x, int n, int sub, int nw, auto rec) {
    for (int e = sub; e < n; e += 4 * nw) {
      float2 ml[4];
      float4 u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const long long i = e + k * nw < n ? rec(e + k * nw) : -1;
        ml[k] = make_float2(-INFINITY, 0.f);
        u[k] = none.o;
        if (i >= 0) {
          ml[k] = __ldcg(recs.ml + i);
          if (col) u[k] = __ldcg(ro + i * d4);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) join_rec(x, ml[k], u[k]);
    }
  };
  // the pieces of four rows whose packed rows are `step` apart in one unit, n of
  // them there; row, h: the first's, where the unit may be whole (part 0 or 1)
  auto gather4 = [&](JoinAcc (&x)[4], const JoinUnit &un, int r, int step, int n, int part, int row,
                     int h) {
    for (int e = 0; e < un.n; ++e) {
      int t0, t1;
      kp_piece_of(pl, un.wu, pl.T[un.j], un.c0 + e, t0, t1);
      if (t1 <= t0) continue;
      const bool whole = t0 == 0 && t1 == pl.T[un.j];
      const size_t i = whole ? key_rec_row(a, rt, part, row, h)
                             : key_rec_slot(kp_slot(un.c0 + e, t0), rt, r);
      const size_t st = whole ? a.H : step;
      float2 ml[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        v[k] = none.o;
        if (k < n) {
          ml[k] = __ldcg(recs.ml + i + k * st);
          if (col) v[k] = __ldcg(ro + (i + k * st) * d4);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) join_rec(x[k], ml[k], v[k]);
    }
  };
  const int W = pl.wbase[pl.njobs];
  const int blk = blockIdx.y * gridDim.x + blockIdx.x, n_blks = gridDim.x * gridDim.y;
  if (pl.stacked) {
    const int items = (pl.q0[a.batch] - pl.q0[0]) * a.H;   // below 2^31: the joint rows are few
    const int nw = join_warps(items, (long long)n_blks * KJ_WARPS);
    if (nw == 1) {
      // four rows of a head at a time, in runs that share both units: finding a
      // row's units and pieces cost more than its loads
      const int rows = pl.q0[a.batch] - pl.q0[0], groups = (rows + 3) / 4 * a.H;
      int b = 0;
      for (int i = blk * KJ_WARPS + warp; i < groups; i += n_blks * KJ_WARPS) {
        const int grp = by_h.div(i), h = i - grp * a.H;
        const int hk = by_g.div(h), g = h - hk * a.G;
        const int end = min(4 * grp + 4, rows);
        for (int rp = 4 * grp; rp < end;) {
          const int row = pl.q0[0] + rp;
          while (pl.q0[b + 1] <= row) ++b;
          const int rb = row - pl.q0[b], up = by_uq.div(rp), ub = by_uq.div(rb);
          const JoinUnit p(pl, chunk, 0, pl.wbase[0] + (up * a.Hkv + hk) * (pl.T[0] + pl.ov));
          const JoinUnit o(pl, chunk, b + 1,
                           pl.wbase[b + 1] + (hk * pl.nu[b + 1] + ub) * (pl.T[b + 1] + pl.ov));
          const int n = min(min(end, (up + 1) * uq) - rp, min(pl.q0[b + 1], pl.q0[b] + (ub + 1) * uq) - row);
          JoinAcc x[4] = {none, none, none, none};
          gather4(x, p, (rp - up * uq) * a.G + g, a.G, n, 0, row, h);
          gather4(x, o, (rb - ub * uq) * a.G + g, a.G, n, 1, row, h);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < n) join_store<T>(a, x[k], row + k, h, lane);
          rp += n;
        }
      }
      return;
    }
    const int sub = warp % nw, per = KJ_WARPS / nw;
    int b = 0;
    for (int i0 = blk * per; i0 < items; i0 += n_blks * per) {
      const int i = i0 + warp / nw;
      const bool there = i < items;
      JoinAcc x = none;
      int row = 0, h = 0;
      if (there) {
        const int rp = by_h.div(i);
        h = i - rp * a.H;
        row = pl.q0[0] + rp;
        const int hk = by_g.div(h), g = h - hk * a.G;
        while (pl.q0[b + 1] <= row) ++b;
        const int rb = row - pl.q0[b], up = by_uq.div(rp), ub = by_uq.div(rb);
        const JoinUnit p(pl, chunk, 0, pl.wbase[0] + (up * a.Hkv + hk) * (pl.T[0] + pl.ov));
        const JoinUnit o(pl, chunk, b + 1, pl.wbase[b + 1] + (hk * pl.nu[b + 1] + ub) * (pl.T[b + 1] + pl.ov));
        const int r_p = (rp - up * uq) * a.G + g, r_o = (rb - ub * uq) * a.G + g;
        gather(x, p.n + o.n, sub, nw, [&](int e) {
          return e < p.n ? p.rec(pl, e, rt, r_p, key_rec_row(a, rt, 0, row, h))
                         : o.rec(pl, e - p.n, rt, r_o, key_rec_row(a, rt, 1, row, h));
        });
      }
      finish(x, nw, sub, there, row, h);
    }
    return;
  }
  if (pl.empty) {
    for (int b = 0; b < a.batch; ++b) {
      if (pl.T[b] > 0) continue;
      const long long n = (long long)(pl.q0[b + 1] - pl.q0[b]) * a.H;
      for (long long i = (long long)blk * KJ_WARPS + warp; i < n; i += (long long)n_blks * KJ_WARPS)
        join_store<T>(a, none, pl.q0[b] + (int)(i / a.H), (int)(i % a.H), lane);
    }
  }
  const int c = blockIdx.x;
  const long long cut = (long long)c * pl.chunk;
  if (c == 0 || cut >= W || pl.per) return;
  const int j = kp_job_at(pl, pl.wbase, (int)cut, lane);
  const int cu = pl.T[j] + pl.ov, u = ((int)cut - pl.wbase[j]) / cu;
  const int wu = pl.wbase[j] + u * cu;
  // between two units, or behind a job's last one
  if (cut == wu || u >= pl.ubase[j + 1] - pl.ubase[j]) return;
  // its cuts share the rows: this is the k-th of n_cuts; none of them where all
  // its tiles lie in one share, which then wrote the rows
  const JoinUnit un(pl, chunk, j, wu);
  const int n_cuts = un.n - 1, k = c - un.c0 - 1;
  for (int e = 0, t0 = 0, t1 = 0; e < un.n && t1 == 0; ++e) {
    kp_piece_of(pl, wu, pl.T[j], un.c0 + e, t0, t1);
    if (t0 == 0 && t1 == pl.T[j]) return;
    t1 = max(t1, 0);
  }
  int unit, hk;
  kp_unit_of(pl, j, u, unit, hk);
  const int r0 = pl.q0[j] + unit * uq;
  const int rn = min(uq, pl.q0[j + 1] - r0) * a.G;
  const int y = k * gridDim.y + blockIdx.y, n_y = n_cuts * gridDim.y;   // this block of the unit's
  const int nw = join_warps(rn, (long long)KJ_WARPS * n_y), sub = warp % nw, per = KJ_WARPS / nw;
  if (nw > 1 || rn <= 2 * KJ_WARPS * n_y) {   // few rows a warp: four pieces in flight
    for (int i0 = y * per; i0 < rn; i0 += n_y * per) {
      const int r = i0 + warp / nw;
      const bool there = r < rn;
      JoinAcc x = none;
      const int rq = by_g.div(r);
      if (there) gather(x, un.n, sub, nw, [&](int e) { return un.rec(pl, e, rt, r, 0); });
      finish(x, nw, sub, there, r0 + rq, hk * a.G + r - rq * a.G);
    }
    return;
  }
  const int step = n_y * KJ_WARPS;
  for (int ra = y * KJ_WARPS + warp; ra < rn; ra += 4 * step) {
    JoinAcc x[4] = {none, none, none, none};
    gather4(x, un, ra, step, (rn - ra + step - 1) / step, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = ra + k * step, rq = by_g.div(r);
      if (r < rn) join_store<T>(a, x[k], r0 + rq, hk * a.G + r - rq * a.G, lane);
    }
  }
}

// ---------------------------------------------------------------------- host --
namespace {
size_t simt_smem(int D) { return ((size_t)3 * KS_T * (D + 4) + KS_T * (KS_T + 4)) * 4; }

template <typename T> cudaError_t run_simt(const KeyArgs &a, cudaStream_t s) {
  const cudaError_t e =
      launch_k(key_attn_simt_kernel<T>, a.n_ctas, KS_THREADS, simt_smem(a.D), s, a);
  if (e != cudaSuccess) return e;
  return launch_key_join(a, KS_T, KS_T / a.G, s);
}
}  // namespace

cudaError_t key_attn_setup(int dtype, int D) {
  if (key_attn_tc_takes(dtype, D)) return key_attn_tc_setup(D);
  const int smem = (int)simt_smem(D);
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  return dtype == SL_BF16 ? cudaFuncSetAttribute(key_attn_simt_kernel<bf16>, attr, smem)
                          : cudaFuncSetAttribute(key_attn_simt_kernel<float>, attr, smem);
}

int key_attn_ctas(int dtype, int D, int num_sms) {
  if (key_attn_tc_takes(dtype, D)) return num_sms;
  return num_sms * (D <= 64 ? 2 : 1);
}

size_t key_attn_ws_floats(int dtype, int D, int H, int n_ctas, int stack_rows) {
  const size_t slot_rows = key_attn_tc_takes(dtype, D) ? 256 : KS_T;
  return 2 * (size_t)n_ctas * slot_rows * (D + 2) + 2 * (size_t)stack_rows * H * (D + 2);
}

cudaError_t launch_key_join(const KeyArgs &a, int rt, int uq, cudaStream_t s) {
  const dim3 grid(a.n_ctas, KJ_Y);
  const FastDiv by_h = FastDiv::of(a.H), by_g = FastDiv::of(a.G), by_uq = FastDiv::of(uq);
  return a.dtype == SL_BF16
             ? launch_k(key_join_kernel<bf16>, grid, 32 * KJ_WARPS, 0, s, a, rt, uq, by_h, by_g, by_uq)
             : launch_k(key_join_kernel<float>, grid, 32 * KJ_WARPS, 0, s, a, rt, uq, by_h, by_g,
                        by_uq);
}

// Shares of one tile: see the kernel (24 us against 36 with two).
cudaError_t launch_key_attn(KeyArgs a, cudaStream_t s) {
  if (key_attn_tc_takes(a.dtype, a.D)) return launch_key_attn_tc(a, s);
  a.ov = 1;
  a.min_chunk = 1;
  a.join_cost = 0;
  return a.dtype == SL_BF16 ? run_simt<bf16>(a, s) : run_simt<float>(a, s);
}

}  // namespace sl
