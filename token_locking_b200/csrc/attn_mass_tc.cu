// The attention weight each cached key receives (see attn_mass.cu for the
// operator) on the 5th-generation tensor cores, for bf16 heads of 64 and 128.
//
// Keys are the rows of the product, S_j = K_j Q^T, so that a key is a TMEM lane
// and the sum over heads and query rows stays in one thread's register.  A unit
// is two tiles of 128 keys; its inner tiles are the blocks of 128 packed rows
// (query row, head of the group) of every K/V head:
//   warp 0       TMA producer: the two K tiles once per K/V head, the Q blocks
//                (boxes [QR query rows][G heads][64]) through a ring
//   warp 3       -lse log2(e) of a block's rows into the ring, and a mark where
//                some of them weigh nothing; with warp 0, rows of listed keys
//                (16-byte asynchronous copies)
//   warps 1,2    one lane each issues the products of key tile j, into one of
//                two score buffers
//   warps 4..19  two warpgroups per key tile: a thread sums
//                2^(s scale log2(e) - lse log2(e)) over half of a block's rows
// A product takes 512 clocks and its 128 x 128 exponentials 1024, so the
// exponentials bound the kernel: 4 sequences of 2048 rows, keys and 32 heads take
// 184 to 190 us (two cards), the special-function unit busy 78 % of the time.  (A
// quarter of the exponentials by a polynomial on the FMA pipe: 5 % more, under the
// power limit.)  They are the unit's own 2^x (2^-22 relative error), four times the
// plain form's error and far below the scores' rounding.  With a list the rows of a
// head's keys are copied one by one into the one K buffer: 201 us, and 112 against
// 99 for 1024 keys.
// The K tiles need one buffer only: when a head's products are done, the score
// buffers hold work for longer than the next head's copy takes.
#include <string.h>

#include <algorithm>

#include "common.cuh"
#include "keys_common.cuh"
#include "keys_plan.cuh"
#include "keys_tc.cuh"

namespace sl {

namespace {
constexpr int KM_THREADS = 128 + 4 * 128;
constexpr int KM_KEYS = 256;                  // keys of a unit
constexpr int KM_HALF = 64;                   // rows of a block that a thread sums
// In place of the first -lse log2(e) of a half block: some of its rows weigh
// nothing.  (A NaN; a half block that begins with this very one takes the marked
// path too.  The bits read for every half block instead: 1.4 % of the long call's
// time, in the queue that the exponentials wait in; the mark 0.5 %.)
constexpr uint32_t KM_MARK = 0x7fc0a5a5u;

template <int D> struct KmCfg {
  static constexpr int NB = D / 64;                     // 128-byte boxes of a row
  static constexpr int BOX = 128 * 128, TILE = NB * BOX;
  static constexpr int TAIL = 2048;
  // a stage: Q block, lse of its 128 rows with marks, the same without, a bit for
  // each row that weighs nothing; aligned
  static constexpr int K_OFF = 0, Q_OFF = 2 * TILE, LSE = TILE, PLAIN = 512, OUT = TILE + 1024;
  static constexpr int STAGE = TILE + 2048;
  static constexpr int NS = D == 128 ? 4 : 6;           // Q blocks in flight
  static constexpr int BAR_OFF = Q_OFF + NS * STAGE, SMEM = BAR_OFF + TAIL + 1024;
  // barriers: K full, K free; per Q stage full, free; per key tile and score
  // buffer full, free; drain
  static constexpr int B_KF = 0, B_KE = 1, B_F = 2, B_E = 2 + NS, B_TILE = 2 + 2 * NS;
  static constexpr int B_DRAIN = B_TILE + 8, B_COUNT = B_DRAIN + 2;
  static constexpr int PLAN_OFF = BAR_OFF + 256;
  static constexpr int CH = D / 8, RPI = 32 / CH;       // row copies: see the attention kernel
  static constexpr int NI = KM_KEYS / RPI / 2;          // instructions of each of two warps
  static_assert(8 * B_COUNT + 20 <= 256 && sizeof(KeyPlan) <= TAIL - 256, "barriers and plan");
  static_assert(SMEM <= 232448, "shared memory");
};
}  // namespace

struct KmParams {
  CUtensorMap q, k;
  KeyArgs a;
};

template <int D>
__global__ void __launch_bounds__(KM_THREADS, 1) key_mass_tc_kernel(
    const __grid_constant__ KmParams p) {
  using C = KmCfg<D>;
  extern __shared__ uint8_t km_smem[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)km_smem + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = s_addr(smem);
  const uint32_t bar0 = sbase + C::BAR_OFF;
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  auto tfull = [&](int j, int u) { return bar0 + 8u * (uint32_t)(C::B_TILE + 4 * j + u); };
  auto tfree = [&](int j, int u) { return bar0 + 8u * (uint32_t)(C::B_TILE + 4 * j + 2 + u); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::BAR_OFF + 8 * C::B_COUNT);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  KeyFills *fills = reinterpret_cast<KeyFills *>(tmem_slot + 2);
  KeyPlan &pl = *reinterpret_cast<KeyPlan *>(smem + C::PLAN_OFF);
  const KeyArgs &a = p.a;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const unsigned long long lim = a.wait_ns;
  const int QR = 128 / a.G;                   // query rows of a block

  if (threadIdx.x == 0) {
    mbar_init(bar(C::B_KF), 2);               // warps 0 and 3
    mbar_init(bar(C::B_KE), 2);               // both issuing warps
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(bar(C::B_F + s), 2);
      mbar_init(bar(C::B_E + s), 2 + 16);     // issuing warps, and readers of the lse
    }
    for (int j = 0; j < 2; ++j)
      for (int u = 0; u < 2; ++u) {
        mbar_init(tfull(j, u), 1);
        mbar_init(tfree(j, u), 8);
      }
    mbar_init(bar(C::B_DRAIN), 1);
    mbar_init(bar(C::B_DRAIN + 1), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (a.M > 0) {                            // no rows: the maps are not made
      tma_prefetch_desc(&p.q);
      tma_prefetch_desc(&p.k);
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     s_addr(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  if (warp == 0) key_plan_build(pl, a, QR, KM_KEYS, gridDim.x, true, lane);
  key_mass_start(a, blockIdx.x * KM_THREADS + threadIdx.x, gridDim.x * KM_THREADS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  if (blockIdx.x == 0) key_plan_publish(pl, a.plan, threadIdx.x, KM_THREADS);
  const uint32_t tmem_base = *tmem_slot;

  // every role walks the same pieces, and in them the same (K/V head, block)s
  int w, w_end, job;
  key_begin(pl, blockIdx.x, lane, w, w_end, job);
  KeyPiece pc{};
  int st = 0;                                 // Q stage
  uint32_t ph = 0;
  auto next_stage = [&]() {
    if (++st == C::NS) {
      st = 0;
      ph ^= 1u;
    }
  };
  bool ok = true;

  if (warp == 0 || warp == 3) {
    // --------------------------------------------------------- producers
    const int pw = warp == 0 ? 0 : 1;
    const int g0 = lane / C::CH, ch = lane % C::CH;
    const uint32_t off = (ch >> 3) * C::BOX + (pw * C::RPI + g0) * 128;
    const uint32_t sw0 = ((ch ^ (pw * C::RPI + g0)) & 7) << 4, sw1 = sw0 ^ (4 << 4);
    int nk = 0;                               // K tiles copied
    // test hook: the first of them (nk = 1) is left out
    const int skip = a.lost && blockIdx.x == 0 && pw == 0 ? 1 : 0;
    while (ok && key_next(pl, w, w_end, job, pc)) {
      const int b = pc.job, i0 = pc.unit * KM_KEYS;
      const int nj = pl.kl[b] - i0 > 128 ? 2 : 1;
      const int q0 = pl.q0[b], qn = pl.q0[b + 1] - q0, nqt = kp_tiles(qn, QR);
      int hk = pc.t0 / nqt, blk = pc.t0 - hk * nqt;
      // -lse log2(e) of this lane's four rows of a block (warp 3); +inf: rows that
      // are not there, or saw no key, weigh nothing
      float nl[4];
      auto lse_of = [&](int h, int bk) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 32 * e + lane, rq = r / a.G;
          nl[e] = rq < QR && bk * QR + rq < qn
                      ? -a.lse[(size_t)(q0 + bk * QR + rq) * a.H + h * a.G + r - rq * a.G] * KEY_LOG2E
                      : INFINITY;
        }
      };
      if (pw == 1) lse_of(hk, blk);
      for (int t = pc.t0; t < pc.t1; ++t) {
        const bool new_k = t == pc.t0 || blk == 0;
        if (new_k) {
          ok = key_wait(bar(C::B_KE), (uint32_t)(nk & 1) ^ 1u, abort_flag, lim);
          if (!ok) break;
          ++nk;
          if (a.keys) {
            const bf16 *src = (const bf16 *)a.k + (long long)b * a.n_ctx * a.ld_kv + hk * D + ch * 8;
            int pos = 0;
#pragma unroll 4
            for (int i = 0; i < C::NI; ++i) {
              // positions of the next 32 rows of this warp's share, one a lane
              if (i * C::RPI % 32 == 0) {
                const int l = i * C::RPI + lane;
                const int e = i0 + (2 * (l / C::RPI) + pw) * C::RPI + l % C::RPI;
                pos = e < pl.kl[b] ? key_pos(a, b, e) : -1;
              }
              const int ps = __shfl_sync(0xffffffffu, pos, (i * C::RPI + g0) & 31);
              key_copy16(sbase + C::K_OFF + (i * 2 * C::RPI >> 7) * C::TILE + off +
                             (i * 2 * C::RPI & 127) * 128 + ((i * 2 * C::RPI) & 4 ? sw1 : sw0),
                         src + (ps < 0 ? 0 : ps) * a.ld_kv, ps >= 0);
            }
            key_copy_commit();
          } else if (lane == 0 && nk != skip) {
            if (pw == 0) {
              mbar_expect_tx(bar(C::B_KF), nj * C::TILE);
              for (int j = 0; j < nj; ++j)
                for (int c = 0; c < C::NB; ++c)
                  tma_load_2d(sbase + C::K_OFF + j * C::TILE + c * C::BOX, &p.k, hk * D + 64 * c,
                              b * a.n_ctx + i0 + j * 128, bar(C::B_KF));
            } else {
              mbar_arrive(bar(C::B_KF));
            }
          }
        }
        ok = key_wait(bar(C::B_E + st), ph ^ 1u, abort_flag, lim);
        if (!ok) break;
        const uint32_t stage = sbase + C::Q_OFF + st * C::STAGE;
        if (pw == 0) {
          if (lane == 0) {
            mbar_expect_tx(bar(C::B_F + st), (uint32_t)(C::NB * 128 * a.G * QR));
            for (int c = 0; c < C::NB; ++c)
              tma_load_3d(stage + c * C::BOX, &p.q, 64 * c, hk * a.G, q0 + blk * QR,
                          bar(C::B_F + st));
          }
        } else {
          uint8_t *dst = smem + C::Q_OFF + st * C::STAGE;
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const uint32_t lo = __ballot_sync(0xffffffffu, nl[e] == INFINITY);
            const uint32_t hi = __ballot_sync(0xffffffffu, nl[e + 1] == INFINITY);
            const float x = nl[e] == INFINITY ? 0.f : nl[e];
            const float y = nl[e + 1] == INFINITY ? 0.f : nl[e + 1];
            const bool mark =
                __any_sync(0xffffffffu, (lo | hi) != 0 || __float_as_uint(x) == KM_MARK);
            float *to = reinterpret_cast<float *>(dst + C::LSE) + 32 * e + lane;
            to[0] = mark && lane == 0 ? __uint_as_float(KM_MARK) : x;
            to[32] = y;
            if (mark) {
              to[C::PLAIN / 4] = x;
              to[C::PLAIN / 4 + 32] = y;
              if (lane == 0) reinterpret_cast<uint2 *>(dst + C::OUT)[e / 2] = make_uint2(lo, hi);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_F + st));
        }
        if (new_k && a.keys) {
          key_copy_wait<0>();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && nk != skip) mbar_arrive(bar(C::B_KF));
        }
        if (++blk == nqt) {
          blk = 0;
          ++hk;
        }
        if (pw == 1 && t + 1 < pc.t1) lse_of(hk, blk);
        next_stage();
      }
    }
    key_copy_wait<0>();
    if (!ok && lane == 0) {
      atomicExch(a.err, DEV_TIMEOUT_PRODUCER);
      *abort_flag = 1;
    }
    if (pw == 0 && lane == 0) *fills = KeyFills{st, (int)ph, nk};
  } else if (warp < 3) {
    // ------------------------------------------------------------- MMA
    const int j = warp - 1;                   // key tile
    constexpr uint32_t id = idesc_bf16_f32<128>();
    const bool leader = key_elect();
    const uint64_t dk = smem_desc_sw128(sbase + C::K_OFF + j * C::TILE);
    const uint64_t dq = smem_desc_sw128(sbase + C::Q_OFF);
    int nk = 0;
    uint32_t cs = 0;                          // products issued
    while (ok && key_next(pl, w, w_end, job, pc)) {
      const int b = pc.job;
      const bool mine = j == 0 || pl.kl[b] - pc.unit * KM_KEYS > 128;
      const int nqt = kp_tiles(pl.q0[b + 1] - pl.q0[b], QR);
      int blk = pc.t0 % nqt;
      for (int t = pc.t0; t < pc.t1; ++t) {
        if (t == pc.t0 || blk == 0) {
          ok = key_wait(bar(C::B_KF), (uint32_t)(nk & 1), abort_flag, lim);
          if (!ok) break;
          ++nk;
        }
        ok = key_wait(bar(C::B_F + st), ph, abort_flag, lim);
        if (!ok) break;
        if (mine) {
          const uint32_t u = cs & 1u;
          ok = key_wait(tfree(j, u), ((cs >> 1) & 1u) ^ 1u, abort_flag, lim);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bq = dq + (uint64_t)(uint32_t)(st * (C::STAGE >> 4));
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc_mma(tmem_base + (2 * j + u) * 128,
                     dk + ((kk >> 2) * C::BOX >> 4) + 2 * (kk & 3),
                     bq + ((kk >> 2) * C::BOX >> 4) + 2 * (kk & 3), id, kk > 0 ? 1u : 0u);
            tc_commit(tfull(j, u));
          }
          ++cs;
        }
        if (++blk == nqt) blk = 0;
        if (leader) {
          tc_commit(bar(C::B_E + st));
          if (blk == 0 || t + 1 == pc.t1) tc_commit(bar(C::B_KE));
        }
        __syncwarp();
        next_stage();
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
    // ----------------------------------------------------- exponentials
    const int j = (warp - 4) >> 3;            // key tile
    const int half = (warp - 4) >> 2 & 1;     // rows 64 half .. 64 half + 64 of a block
    const int quarter = warp & 3;
    const uint32_t t_s = tmem_base + ((uint32_t)(quarter * 32) << 16) + 2 * j * 128 + half * KM_HALF;
    const float c2 = a.scale * KEY_LOG2E;
    const f32x2 cc = pack2(c2, c2);
    uint32_t cs = 0;
    while (ok && key_next(pl, w, w_end, job, pc)) {
      const int b = pc.job, i0 = pc.unit * KM_KEYS + j * 128 + quarter * 32 + lane;
      const bool mine = j == 0 || pl.kl[b] - pc.unit * KM_KEYS > 128;
      f32x2 sum[2] = {0ull, 0ull};
      for (int t = pc.t0; t < pc.t1; ++t) {
        ok = key_wait(bar(C::B_F + st), ph, abort_flag, lim);
        if (!ok) break;
        if (mine) {
          const uint32_t u = cs & 1u;
          ok = key_wait(tfull(j, u), (cs >> 1) & 1u, abort_flag, lim);
          if (!ok) break;
          tc_fence_after();
          const uint8_t *stage = smem + C::Q_OFF + st * C::STAGE;
          const ulonglong2 *nl =
              reinterpret_cast<const ulonglong2 *>(stage + C::LSE) + half * (KM_HALF / 4);
          ulonglong2 x = nl[0];
          uint2 out = make_uint2(0u, 0u);
          if ((uint32_t)x.x == KM_MARK) {
            key_cold();
            out = reinterpret_cast<const uint2 *>(stage + C::OUT)[half];
            nl += C::PLAIN / 16;
            x = nl[0];
          }
#pragma unroll
          for (int c = 0; c < KM_HALF; c += 32) {
            float s[32];
            tmem_ld_cols<32>(t_s + u * 128 + c, s);
            if (c + 32 == KM_HALF) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(tfree(j, u));
            }
            // rows that weigh nothing may hold anything, NaN among it
            if (const uint32_t bits = c == 0 ? out.x : out.y) {
              key_cold();
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] = bits >> i & 1 ? -INFINITY : s[i];
            }
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              if (c + i > 0) x = nl[(c + i) / 4];
              float p[4];
              unpack2(fma2(pack2(s[i], s[i + 1]), cc, x.x), p[0], p[1]);
              unpack2(fma2(pack2(s[i + 2], s[i + 3]), cc, x.y), p[2], p[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) p[e] = ex2_approx(p[e]);
              sum[0] = add2(sum[0], pack2(p[0], p[1]));
              sum[1] = add2(sum[1], pack2(p[2], p[3]));
            }
          }
          ++cs;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::B_E + st));
        next_stage();
      }
      if (ok && mine && i0 < pl.kl[b]) {
        float v0, v1;
        unpack2(add2(sum[0], sum[1]), v0, v1);
        const float v = v0 + v1;
        const bool whole = pc.t0 == 0 && pc.t1 == pc.T;
        const size_t n_slots = 2 * (size_t)a.n_ctas * 2 * KM_KEYS;
        a.ws[whole ? n_slots + (size_t)half * a.batch * a.n_ctx + (size_t)b * a.n_ctx + i0
                   : ((size_t)kp_slot(blockIdx.x, pc.t0) * 2 + half) * KM_KEYS + j * 128 +
                         quarter * 32 + lane] = v;
      }
    }
    if (!ok && lane == 0) {
      atomicExch(a.err, DEV_TIMEOUT_EPI);
      *abort_flag = 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // no role can raise the flag any more
  if (threadIdx.x == 0 && *abort_flag) key_drain(*fills, bar(C::B_F), C::NS, bar(C::B_KF), lim);
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(512)
                 : "memory");
  }
}

// ---------------------------------------------------------------------- host --
namespace {
template <int D> cudaError_t run_mass_tc(const KeyArgs &a, cudaStream_t s) {
  KmParams p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  const int QR = 128 / a.G;
  if (a.M > 0 &&
      !(tma_encode_heads(&p.q, a.q, a.M, a.H, D, a.ld_q, a.G, QR) &&
        tma_encode_rows(&p.k, a.k, (long long)a.batch * a.n_ctx, a.Hkv * D, a.ld_kv, 128)))
    return cudaErrorInvalidValue;
  const cudaError_t e =
      launch_k(key_mass_tc_kernel<D>, a.n_ctas, KM_THREADS, KmCfg<D>::SMEM, s, p);
  if (e != cudaSuccess) return e;
  return launch_key_mass_add(a, KM_KEYS, 2, s);
}
}  // namespace

cudaError_t key_mass_tc_setup(int D) {
  return D == 128 ? cudaFuncSetAttribute(key_mass_tc_kernel<128>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         KmCfg<128>::SMEM)
                  : cudaFuncSetAttribute(key_mass_tc_kernel<64>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         KmCfg<64>::SMEM);
}

// Least share of a CTA, in tile times: with 1 / 2 / 4 the weights of a window of 200
// rows over 384 keys take 17.9 / 15.3 / 16.4 us, longer calls the same.
cudaError_t launch_key_mass_tc(KeyArgs a, cudaStream_t s) {
  a.ov = 1;
  a.min_chunk = 2;
  a.join_cost = 0;
  return a.D == 128 ? run_mass_tc<128>(a, s) : run_mass_tc<64>(a, s);
}

}  // namespace sl
