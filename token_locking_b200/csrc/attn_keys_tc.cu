// Attention over a key set per sequence (see attn_keys.cu for the operator) on
// the 5th-generation tensor cores, for bf16 heads of 64 and 128.
//
// A unit is two tiles of 128 packed rows (query row, head of the group) of one
// K/V head against a list of tiles of BN keys; a CTA takes whole units or an equal
// share of all their tiles (keys_plan.cuh) and runs through them without a break:
//   warps 0,3    producers.  Warp 0 copies Q by TMA in boxes [QR query rows]
//                [G heads][64], so that packed rows land in order whatever G,
//                and every full tile of the prefix or of an unlisted cache.
//                Listed keys, and the tile a key set ends in, are copied row by
//                row by both warps (16-byte asynchronous copies, two tiles
//                in flight), zeros for entries that are not there: what lies
//                behind a key set never reaches shared memory.  (Four-row TMA
//                gathers instead took 17 clocks a row of 128 bytes, 7200 clocks
//                a tile.)
//   warps 1,2    one lane each issues S_j = Q_j K^T and O_j += P_j V of row tile
//                j (warp 1 owns TMEM).  One issuing warp for both tiles took
//                some 2500 clocks a tile of keys, in waits and issue alone.
//   warps 4..19  softmax: two warpgroups per row tile, a row per thread in
//                each and half of the tile's keys; the halves exchange their
//                maxima through TMEM.  (One warpgroup per tile, all keys: 2300
//                clocks per 80 keys, with two warps per scheduler too few to keep
//                the exponentials running through the waits.  Both halves taking
//                the maximum over all keys: 2 % more time.)  The maximum is
//                raised only when a tile exceeds it by 2^8 (O is rescaled then);
//                p is rounded to bf16 for the product (half a step), its sum taken
//                in fp32 before.
// The two row tiles are two independent chains (scores, softmax, P V) that
// share K and V, so that the tensor cores work on one while the other's
// exponentials are taken.
// Key tiles of 80 (heads of 128) or 96 (64): S, P and O of both row tiles then
// fill TMEM without sharing columns, so that scores of the next tile are issued
// as soon as the last ones have been read.
//
// What bounds it: a tile of 80 keys takes 2135 clocks for both row tiles, of
// which the products need 1470 (416 + 320 each, measured alone) and the
// exponentials 1280; the rest is the softmax warps' way from one barrier to the
// next.  Long calls run at 1.4 GHz (clocks over nanoseconds) under the power
// limit, where a third fewer instructions or a shift of the two chains against
// each other changed nothing, but less memory traffic did: 4 x 256 rows of 32
// heads over a shared prefix of 16384 take 305 to 314 us back to back (two cards)
// with the prefix read from memory once, 341 us with four times.  Short calls are
// bound by starting: 0.9 us for the plan, 2.5 us to the first scores.
#include <string.h>

#include <algorithm>

#include "common.cuh"
#include "keys_common.cuh"
#include "keys_plan.cuh"
#include "keys_tc.cuh"

namespace sl {

namespace {
constexpr int KC_ROWS = 128;                  // packed rows of a tile (TMEM lanes)
constexpr int KC_THREADS = 128 + 4 * 128;
constexpr float KC_RESCALE = 8.f;

template <int D, int BN> struct KcCfg {
  static constexpr int NB = D / 64;                     // 128-byte boxes of a row
  static constexpr int QBOX = KC_ROWS * 128, KBOX = BN * 128;
  static constexpr int SLOT = NB * KBOX;                // a K or V tile
  static constexpr int KV_OFF = 2 * NB * QBOX;
  static constexpr int TAIL = 2048;                     // barriers and plan
  // ring of NP stages, a K and a V tile each
  static constexpr int NP = (232448 - 1024 - TAIL - KV_OFF) / (2 * SLOT);
  static constexpr int BAR_OFF = KV_OFF + 2 * NP * SLOT;
  static constexpr int SMEM = BAR_OFF + TAIL + 1024;    // + alignment
  // barriers: Q full, Q free; per stage full, free; per row tile four; drain
  static constexpr int B_QF = 0, B_QE = 1, B_F = 2, B_E = 2 + NP, B_TILE = 2 + 2 * NP;
  static constexpr int B_DRAIN = B_TILE + 8, B_COUNT = B_DRAIN + 2;
  // row copies: 16-byte chunks of a row, rows of a warp instruction, instructions
  // of each of the two warps, tiles in flight
  static constexpr int CH = D / 8, RPI = 32 / CH, NI = BN / RPI / 2, LAG = 2;
  static constexpr int PLAN_OFF = BAR_OFF + 256;
  // TMEM columns: per row tile S, then P (two bf16 keys a column), from a
  // multiple of 64; then O of both
  static constexpr uint32_t T_COLS = (BN + BN / 2 + 63) / 64 * 64;
  static constexpr uint32_t O_COL = 2 * T_COLS;
  static constexpr uint32_t X_COL = BN + BN / 2;        // the two halves' row maxima, twice
  static constexpr uint32_t L_COL = X_COL + 4;          // and row sums
  static_assert(O_COL + 2 * D <= 512 && L_COL + 2 <= T_COLS, "TMEM columns");
  static constexpr int HB = BN / 2;                     // keys of a softmax warpgroup
  static_assert(8 * B_COUNT + 20 <= 256 && sizeof(KeyPlan) <= TAIL - 256, "barriers and plan");
  static_assert(BN % (2 * RPI) == 0 && NI * RPI <= 64, "two rows a lane of a warp's share");
  static_assert(LAG < NP, "row copies in flight");
  static_assert(SMEM <= 232448 && BN % 16 == 0, "shared memory, key tile");
};
}  // namespace

struct KcParams {
  CUtensorMap q, k, v, kp, vp;
  KeyArgs a;
};

__device__ __forceinline__ uint32_t kc_pack(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

template <int D, int BN>
__global__ void __launch_bounds__(KC_THREADS, 1) key_attn_tc_kernel(
    const __grid_constant__ KcParams p) {
  using C = KcCfg<D, BN>;
  extern __shared__ uint8_t kc_smem[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)kc_smem + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = s_addr(smem);
  const uint32_t bar0 = sbase + C::BAR_OFF;
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  // per row tile: 0 scores ready, 1 scores read, 2 P written, 3 P V done
  auto tbar = [&](int j, int k) { return bar0 + 8u * (uint32_t)(C::B_TILE + 4 * j + k); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::BAR_OFF + 8 * C::B_COUNT);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  KeyFills *fills = reinterpret_cast<KeyFills *>(tmem_slot + 2);
  KeyPlan &pl = *reinterpret_cast<KeyPlan *>(smem + C::PLAN_OFF);
  const KeyArgs &a = p.a;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const unsigned long long lim = a.wait_ns;
  const int QR = KC_ROWS / a.G;               // query rows of a tile

  if (threadIdx.x == 0) {
    mbar_init(bar(C::B_QF), 1);
    mbar_init(bar(C::B_QE), 2);               // both issuing warps
    for (int s = 0; s < C::NP; ++s) {
      mbar_init(bar(C::B_F + s), 2);          // both producers
      mbar_init(bar(C::B_E + s), 2);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(tbar(j, 0), 1);               // MMA commit
      mbar_init(tbar(j, 1), 8);               // the tile's eight softmax warps
      mbar_init(tbar(j, 2), 8);
      mbar_init(tbar(j, 3), 1);
    }
    mbar_init(bar(C::B_DRAIN), 1);
    mbar_init(bar(C::B_DRAIN + 1), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&p.q);
    tma_prefetch_desc(&p.k);
    tma_prefetch_desc(&p.v);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     s_addr(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  if (warp == 0) key_plan_build(pl, a, 2 * QR, BN, gridDim.x, false, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  if (blockIdx.x == 0) key_plan_publish(pl, a.plan, threadIdx.x, KC_THREADS);
  const uint32_t tmem_base = *tmem_slot;
  const int tp = kp_tiles(a.prefix_len, BN);

  // every role walks the same pieces
  int w, w_end, job;
  key_begin(pl, blockIdx.x, lane, w, w_end, job);
  KeyPiece pc{};
  // first query row and query rows of a piece's unit; row tiles it fills
  auto rows_of = [&](int &r0, int &rn) {
    const int b = kp_seq(pl, pc.job);
    r0 = (b < 0 ? pl.q0[0] : pl.q0[b]) + pc.unit * 2 * QR;
    rn = min(2 * QR, (b < 0 ? pl.q0[a.batch] : pl.q0[b + 1]) - r0);
    return rn > QR ? 2 : 1;
  };

  if (warp == 0 || warp == 3) {
    // --------------------------------------------------------- producers
    const int pw = warp == 0 ? 0 : 1;
    const int g0 = lane / C::CH, ch = lane % C::CH;
    // instruction i of this warp copies rows (2 i + pw) RPI + g0; lane l holds
    // the cache positions of the l-th and (32 + l)-th row of the warp's share
    const int my_row = (2 * (lane / C::RPI) + pw) * C::RPI + lane % C::RPI;
    const int my_row2 = my_row + 64;          // 32 rows of the share later
    // where this lane's chunk goes: rows advance by 2 RPI, a multiple of 4
    const uint32_t off = (ch >> 3) * C::KBOX + (pw * C::RPI + g0) * 128;
    const uint32_t sw0 = ((ch ^ (pw * C::RPI + g0)) & 7) << 4, sw1 = sw0 ^ (4 << 4);
    int st = 0, np = 0;                       // stage, pieces
    uint32_t ph = 0;
    bool ok = true;
    bool lost = a.lost && blockIdx.x == 0 && pw == 0;   // test hook: the first tile is left out
    while (ok && key_next(pl, w, w_end, job, pc)) {
      int r0, rn;
      const int nj = rows_of(r0, rn), b = kp_seq(pl, pc.job);
      // position of row r of tile t, -1 where there is none
      auto entry = [&](int t, int r) {
        const bool pre = b < 0 || (!pl.stacked && t < tp);
        const int i = (pl.stacked ? t : t - tp) * BN + r;
        return pre || t >= pc.t1 || r >= BN || i >= pl.kl[b] ? -1 : key_pos(a, b, i);
      };
      int nxt = entry(pc.t0, my_row), nxt2 = entry(pc.t0, my_row2);
      if (pw == 0) {
        if (!key_wait(bar(C::B_QE), (uint32_t)(np & 1) ^ 1u, abort_flag, lim)) { ok = false; break; }
        if (lane == 0) {
          mbar_expect_tx(bar(C::B_QF), (uint32_t)(nj * C::NB * 128 * a.G * QR));
          for (int j = 0; j < nj; ++j)
            for (int c = 0; c < C::NB; ++c)
              tma_load_3d(sbase + (j * C::NB + c) * C::QBOX, &p.q, 64 * c, pc.hk * a.G,
                          r0 + j * QR, bar(C::B_QF));
        }
      }
      ++np;
      // tiles whose copies this warp has issued but not yet handed over, and
      // the stage of the first of them
      int pend = 0, pst = st;
      auto hand_over = [&]() {
        fence_proxy_async_smem();             // written by copies, read by the tensor cores
        __syncwarp();
        if (lane == 0 && !lost) mbar_arrive(bar(C::B_F + pst));
        lost = false;
        pst = pst + 1 == C::NP ? 0 : pst + 1;
        --pend;
      };
      for (int t = pc.t0; t < pc.t1; ++t) {
        const bool pre = b < 0 || (!pl.stacked && t < tp);
        const int i0 = (pre || pl.stacked ? t : t - tp) * BN;
        const bool by_row = !pre && (a.keys || i0 + BN > pl.kl[b]);
        const int pos = nxt, pos2 = nxt2;
        nxt = entry(t + 1, my_row);
        nxt2 = entry(t + 1, my_row2);
        const uint32_t dst = sbase + C::KV_OFF + 2 * st * C::SLOT;
        if (!by_row && pend > 0) {
          key_copy_wait<0>();
          while (pend > 0) hand_over();
        }
        if (!key_wait(bar(C::B_E + st), ph ^ 1u, abort_flag, lim)) { ok = false; break; }
        if (by_row) {
          // one position serves K and V: src_k + d_kv is V's row
          const bf16 *src_k = (const bf16 *)a.k + (long long)b * a.n_ctx * a.ld_kv + pc.hk * D + ch * 8;
          const ptrdiff_t d_kv = (const bf16 *)a.v - (const bf16 *)a.k;
          const uint32_t d0 = dst + off;
#pragma unroll
          for (int i = 0; i < C::NI; ++i) {
            const int ps = i * C::RPI < 32
                               ? __shfl_sync(0xffffffffu, pos, (i * C::RPI + g0) & 31)
                               : __shfl_sync(0xffffffffu, pos2, (i * C::RPI + g0) & 31);
            const bf16 *src = src_k + max(ps, 0) * a.ld_kv;
            const uint32_t to = d0 + i * 2 * C::RPI * 128 + ((i * 2 * C::RPI) & 4 ? sw1 : sw0);
            key_copy16(to, src, ps >= 0);
            key_copy16(to + C::SLOT, src + d_kv, ps >= 0);
          }
          key_copy_commit();
          if (++pend == C::LAG) {
            key_copy_wait<C::LAG - 1>();
            hand_over();
          }
        } else {
          if (lane == 0 && !lost) {
            if (pw == 0) {
              const int y = pre ? i0 : b * a.n_ctx + i0;
              mbar_expect_tx(bar(C::B_F + st), 2 * C::SLOT);
#pragma unroll
              for (int kv = 0; kv < 2; ++kv) {
                const CUtensorMap *m = pre ? (kv ? &p.vp : &p.kp) : (kv ? &p.v : &p.k);
#pragma unroll
                for (int c = 0; c < C::NB; ++c)
                  tma_load_2d(dst + kv * C::SLOT + c * C::KBOX, m, pc.hk * D + 64 * c, y,
                              bar(C::B_F + st));
              }
            } else {
              mbar_arrive(bar(C::B_F + st));
            }
          }
          lost = false;
          pst = st + 1 == C::NP ? 0 : st + 1;
        }
        if (++st == C::NP) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
      if (pend > 0) {
        key_copy_wait<0>();
        while (pend > 0) hand_over();
      }
    }
    key_copy_wait<0>();
    if (!ok && lane == 0) {
      atomicExch(a.err, DEV_TIMEOUT_PRODUCER);
      *abort_flag = 1;
    }
    if (pw == 0 && lane == 0) *fills = KeyFills{st, (int)ph, np};
  } else if (warp < 3) {
    // ------------------------------------------------------------- MMA
    const int j = warp - 1;                   // row tile
    constexpr uint32_t id_s = idesc_bf16_f32<BN>();
    constexpr uint32_t id_o = idesc_bf16_f32_bmn<D>();
    const bool leader = key_elect();
    const uint64_t dq = smem_desc_sw128(sbase + j * C::NB * C::QBOX);
    const uint64_t dk = smem_desc_sw128(sbase + C::KV_OFF);
    const uint64_t dv = smem_desc_sw128_mn(sbase + C::KV_OFF + C::SLOT, C::KBOX, 1024);
    const uint32_t t_s = tmem_base + j * C::T_COLS, t_o = tmem_base + C::O_COL + j * D;
    int np = 0;
    int ks = 0, vs = 0;                       // stages of the next scores and P V product
    uint32_t kph = 0;
    uint32_t cs = 0, cv = 0;                  // scores and P V products issued, parities
    bool ok = true;
    while (ok && key_next(pl, w, w_end, job, pc)) {
      int r0, rn;
      const bool mine = j < rows_of(r0, rn);
      const int nt = pc.t1 - pc.t0;
      ok = key_wait(bar(C::B_QF), (uint32_t)(np & 1), abort_flag, lim);
      ++np;
      // scores of tile t are issued one tile ahead of its P V product
      for (int t = -1; ok && t < nt; ++t) {
        if (t + 1 < nt) {
          ok = key_wait(bar(C::B_F + ks), kph, abort_flag, lim);
          if (!ok) break;
          if (mine) {
            // the buffer's last scores have been read
            ok = key_wait(tbar(j, 1), cs ^ 1u, abort_flag, lim);
            if (!ok) break;
            tc_fence_after();
            const uint64_t bk = dk + (uint64_t)(uint32_t)(ks * (2 * C::SLOT >> 4));
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc_mma(t_s, dq + ((kk >> 2) * C::QBOX >> 4) + 2 * (kk & 3),
                       bk + ((kk >> 2) * C::KBOX >> 4) + 2 * (kk & 3), id_s, kk > 0 ? 1u : 0u);
              tc_commit(tbar(j, 0));
            }
            cs ^= 1u;
          }
          if (t + 2 == nt && leader) tc_commit(bar(C::B_QE));
          __syncwarp();
          if (++ks == C::NP) {
            ks = 0;
            kph ^= 1u;
          }
        }
        if (t < 0) continue;
        if (mine) {
          ok = key_wait(tbar(j, 2), cv, abort_flag, lim);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bv = dv + (uint64_t)(uint32_t)(vs * (2 * C::SLOT >> 4));
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              tc_mma_ts(t_o, t_s + BN + kk * 8, bv + kk * (2048 >> 4), id_o,
                        (t > 0 || kk > 0) ? 1u : 0u);
            tc_commit(tbar(j, 3));
          }
          cv ^= 1u;
        }
        if (leader) tc_commit(bar(C::B_E + vs));   // done with the stage
        __syncwarp();
        if (++vs == C::NP) vs = 0;
      }
    }
    if (!ok && lane == 0) {
      atomicExch(a.err, DEV_TIMEOUT_MMA);
      *abort_flag = 1;
    }
    if (leader) {
      tc_commit(bar(C::B_DRAIN + j));
      volatile int never = 0;
      mbar_wait(bar(C::B_DRAIN + j), 0, &never, lim);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- softmax
    constexpr int HB = C::HB;
    const int j = (warp - 4) >> 3;            // row tile
    const int half = (warp - 4) >> 2 & 1;     // keys half HB .. half HB + HB of a tile
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;        // packed row (TMEM lane)
    const int rq = r / a.G, rg = r - rq * a.G;
    const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16) + j * C::T_COLS;
    const uint32_t t_s = t_row + half * HB;
    const uint32_t t_p = t_row + BN + half * (HB / 2);
    const uint32_t t_o = tmem_base + ((uint32_t)(quarter * 32) << 16) + C::O_COL + j * D +
                         half * (D / 2);      // this warpgroup's columns of O
    const float c2 = a.scale * KEY_LOG2E;
    const int rt = 2 * QR * a.G;              // packed rows of a unit
    const KeyRecs recs(a, rt);
    const bool o32 = ((uintptr_t)a.o & 31) == 0 && a.ld_o % 16 == 0;
    uint32_t cs = 0;                          // score tiles taken
    // After a wait that ran out the loops go on without waiting (the abort flag
    // ends later waits at once), so that both halves of a tile meet below.
    bool ok = true;
    auto wait = [&](int k, uint32_t parity) {
      if (!ok) return;
      ok = key_wait(tbar(j, k), parity, abort_flag, lim);
      if (!ok && lane == 0) {
        atomicExch(a.err, DEV_TIMEOUT_EPI);
        *abort_flag = 1;
      }
    };
    while (key_next(pl, w, w_end, job, pc)) {
      int r0, rn;
      if (rows_of(r0, rn) <= j) continue;
      const int b = kp_seq(pl, pc.job);
      // the tiles that end the prefix and the sequence's own keys, and their keys
      const int t_pre = b < 0 || !pl.stacked ? tp - 1 : -1, n_pre = a.prefix_len - (tp - 1) * BN;
      const int t_own = b < 0 ? -1 : pc.T - 1;
      const int n_own = b < 0 ? 0 : pl.kl[b] - (pl.stacked ? t_own : t_own - tp) * BN;
      float m = -INFINITY, l = 0.f;
      for (int t = pc.t0; t < pc.t1; ++t, ++cs) {
        const int nv = t == t_pre ? n_pre : t == t_own ? n_own : BN;
        wait(0, cs & 1u);
        tc_fence_after();
        float s[HB];
        tmem_ld_cols<HB>(t_s, s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tbar(j, 1));
        if (nv < BN) {
          key_cold();
#pragma unroll
          for (int i = 0; i < HB; ++i) s[i] = half * HB + i < nv ? s[i] : -INFINITY;
        }
        // the row's maximum over both halves, through two columns of TMEM (the
        // other two of four next time: the barrier orders the rest)
        float mt = max_of<HB>(s);
        const uint32_t t_x = t_row + C::X_COL + 2 * (cs & 1u);
        tmem_st1_u(t_x + half, __float_as_uint(mt));
        tmem_wait_st();
        tc_fence_before();
        named_bar_sync(1 + j * 4 + quarter, 64);
        tc_fence_after();
        mt = c2 * fmaxf(mt, __uint_as_float(tmem_ld1_u(t_x + (half ^ 1))));
        const bool first = t == pc.t0;
        const float m_new = fmaxf(m, mt);
        const bool resc = !first && m_new > m + KC_RESCALE;
        const float m_use = (first || resc) ? m_new : m;
        const float alpha = resc ? (m == -INFINITY ? 0.f : ex2_approx(m - m_new)) : 1.f;
        const float m_sub = m_use == -INFINITY ? 0.f : -m_use;  // all scores -inf: p = 0
        f32x2 sa[2] = {0ull, 0ull};
        const f32x2 cc = pack2(c2, c2), mm = pack2(m_sub, m_sub);
        uint32_t pk[HB / 2];
#pragma unroll
        for (int i = 0; i < HB; i += 2) {
          float x, y;
          unpack2(fma2(pack2(s[i], s[i + 1]), cc, mm), x, y);
          x = ex2_approx(x);
          y = ex2_approx(y);
          sa[i >> 1 & 1] = add2(sa[i >> 1 & 1], pack2(x, y));
          pk[i / 2] = kc_pack(x, y);
        }
        float l0, l1;
        unpack2(add2(sa[0], sa[1]), l0, l1);
        l = l * alpha + (l0 + l1);
        m = m_use;
        // the last P V product has read P and written O
        if (!first) wait(3, (cs & 1u) ^ 1u);
        tc_fence_after();
        if (__any_sync(0xffffffffu, resc)) {
#pragma unroll 1
          for (int c = 0; c < D / 2; c += 32) {
            float o[32];
            tmem_ld32_nw(t_o + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tmem_st32(t_o + c, o);
          }
        }
        tmem_st_cols<HB / 2>(t_p, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tbar(j, 2));
      }
      // the row's sum: both halves' through TMEM
      wait(3, (cs - 1u) & 1u);
      tc_fence_after();
      tmem_st1_u(t_row + C::L_COL + half, __float_as_uint(l));
      tmem_wait_st();
      tc_fence_before();
      named_bar_sync(1 + j * 4 + quarter, 64);
      tc_fence_after();
      l += __uint_as_float(tmem_ld1_u(t_row + C::L_COL + (half ^ 1)));
      if (!ok) continue;
      // O leaves in 32-column parts: final rows of a whole unit, else partial ones
      const bool live = rq < QR && j * QR + rq < rn;
      const int row = r0 + j * QR + rq, h = pc.hk * a.G + rg;
      const bool whole = pc.t0 == 0 && pc.t1 == pc.T;
      float o[32];
      if (whole && !pl.stacked) {
        const float inv = key_inv(l);
        bf16 *orow = (bf16 *)a.o + row * a.ld_o + h * D + half * (D / 2);
#pragma unroll 1
        for (int c0 = 0; c0 < D / 2; c0 += 32) {
          tmem_ld_cols<32>(t_o + c0, o);
          if (live) {
            uint32_t u[16];
#pragma unroll
            for (int c = 0; c < 16; ++c)
              u[c] = l == 0.f ? 0u : kc_pack(o[2 * c] * inv, o[2 * c + 1] * inv);
            if (o32) {
              st_global_v8(orow + c0, u);
              st_global_v8(orow + c0 + 16, u + 8);
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                reinterpret_cast<uint4 *>(orow + c0)[c] =
                    make_uint4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
            }
          }
        }
        if (live && a.lse && half == 0)
          a.lse[(size_t)row * a.H + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * KEY_LN2;
      } else {
        const size_t rec = whole ? key_rec_row(a, rt, b < 0 ? 0 : 1, row, h)
                                 : key_rec_slot(kp_slot(blockIdx.x, pc.t0), rt, j * QR * a.G + r);
        float *dst = recs.o + rec * D + half * (D / 2);
#pragma unroll 1
        for (int c0 = 0; c0 < D / 2; c0 += 32) {
          tmem_ld_cols<32>(t_o + c0, o);
          if (live) {
#pragma unroll
            for (int c = 0; c < 32; c += 8)
              st_global_v8(dst + c0 + c, reinterpret_cast<const uint32_t *>(o + c));
          }
        }
        if (live && half == 0) recs.ml[rec] = make_float2(m, l);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // no role can raise the flag any more
  if (threadIdx.x == 0 && *abort_flag) key_drain(*fills, bar(C::B_F), C::NP, bar(C::B_QF), lim);
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(512)
                 : "memory");
  }
}

// ---------------------------------------------------------------------- host --
namespace {
template <int D> struct KcBn;                 // key tile: S, P and O of two row tiles fill TMEM
template <> struct KcBn<128> { static constexpr int v = 80; };
template <> struct KcBn<64> { static constexpr int v = 96; };

template <int D> cudaError_t run_tc(const KeyArgs &a, cudaStream_t s) {
  constexpr int BN = KcBn<D>::v;
  using C = KcCfg<D, BN>;
  KcParams p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  const int QR = KC_ROWS / a.G;
  const long long rows = (long long)a.batch * a.n_ctx;
  bool ok = tma_encode_heads(&p.q, a.q, a.M, a.H, D, a.ld_q, a.G, QR) &&
            tma_encode_rows(&p.k, a.k, rows, a.Hkv * D, a.ld_kv, BN) &&
            tma_encode_rows(&p.v, a.v, rows, a.Hkv * D, a.ld_kv, BN);
  if (ok && a.prefix_len > 0)
    ok = tma_encode_rows(&p.kp, a.kp, a.prefix_len, a.Hkv * D, a.ld_p, BN) &&
         tma_encode_rows(&p.vp, a.vp, a.prefix_len, a.Hkv * D, a.ld_p, BN);
  if (!ok) return cudaErrorInvalidValue;
  const cudaError_t e = launch_k(key_attn_tc_kernel<D, BN>, a.n_ctas, KC_THREADS, C::SMEM, s, p);
  if (e != cudaSuccess) return e;
  return launch_key_join(a, 2 * QR * a.G, 2 * QR, s);
}
}  // namespace

cudaError_t key_attn_tc_setup(int D) {
  return D == 128 ? cudaFuncSetAttribute(key_attn_tc_kernel<128, KcBn<128>::v>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         KcCfg<128, KcBn<128>::v>::SMEM)
                  : cudaFuncSetAttribute(key_attn_tc_kernel<64, KcBn<64>::v>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         KcCfg<64, KcBn<64>::v>::SMEM);
}

bool key_attn_tc_takes(int dtype, int D) { return dtype == SL_BF16 && (D == 64 || D == 128); }

// The plan's costs in tile times.  A unit's start-up and epilogue, ov: with 1 / 2 / 4
// one row per sequence over a prefix of 2048 takes 16.1 / 15.8 / 16.5 us, 16 x 32
// rows over 8192 120 / 122 / 127, five ragged sequences over 4097 49.7 / 48.2 / 46.0.
// Least share: with 1 / 3 / 6 the first of these takes 15.7 / 15.8 / 17.7, the others
// the same.  A join, beside which whole units may be uneven: with 0 / 7 / 20 windows
// over 1024 kept keys take 51.2 / 34.6 / 34.6, the others the same.
cudaError_t launch_key_attn_tc(KeyArgs a, cudaStream_t s) {
  a.ov = 2;
  a.min_chunk = 3;
  a.join_cost = 7;
  return a.D == 128 ? run_tc<128>(a, s) : run_tc<64>(a, s);
}

}  // namespace sl
