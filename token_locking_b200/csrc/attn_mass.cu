// The attention weight each cached key receives from the active rows:
//   w_bn = sum_h sum_{j in b} exp(scale q_jh . k_n - lse_jh)
// with the log partition lse the attention left, so that the weights are those
// of the attention over its whole key set, accumulated over layers and steps
// as mass = decay mass_prev + w.  A locked position's K/V stay in the cache
// for the rest of the decode (Paper-Notes, "permanent locking"); the weight
// says which of them the active rows still look at.
//
// A unit is a tile of keys, its inner tiles the row blocks of every K/V head,
// so the sum over heads and rows stays in registers; units that a CTA's share
// cut leave one partial sum per key, joined in CTA order by the second kernel.
#include <algorithm>

#include "common.cuh"
#include "keys_common.cuh"
#include "keys_plan.cuh"

namespace sl {

namespace {
constexpr int MS_T = 64;
constexpr int MS_THREADS = 256;
}  // namespace

// 64 keys against 64 packed rows (qr, g) at a time in fp32 arithmetic; thread
// (ty, tx) of 16 x 16 holds the scores of rows 4 ty + i and keys tx + 16 j.
template <typename T>
__global__ void __launch_bounds__(MS_THREADS) key_mass_simt_kernel(const KeyArgs a) {
  extern __shared__ float4 ms_smem4[];
  __shared__ KeyPlan pl;
  __shared__ float sL[MS_T], red[MS_THREADS / 16][MS_T];
  float *smem = reinterpret_cast<float *>(ms_smem4);
  const int D = a.D, ld = D + 4;
  float *sq = smem, *sk = sq + MS_T * ld;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, lane = tid & 31;
  const int lr = tid >> 2, lc = (tid & 3) * 4;      // row and first column this thread stages
  const int QR = MS_T / a.G;
  pdl_wait();
  if (tid < 32) key_plan_build(pl, a, QR, MS_T, gridDim.x, true, lane);
  key_mass_start(a, blockIdx.x * MS_THREADS + tid, gridDim.x * MS_THREADS);
  __syncthreads();
  if (blockIdx.x == 0) key_plan_publish(pl, a.plan, tid, MS_THREADS);
  pdl_trigger();
  const float c2 = a.scale * KEY_LOG2E;
  int w, w_end, job;
  key_begin(pl, blockIdx.x, lane, w, w_end, job);
  KeyPiece pc;
  while (key_next(pl, w, w_end, job, pc)) {
    const int b = pc.job;
    const int i0 = pc.unit * MS_T, nv = min(MS_T, pl.kl[b] - i0);
    const int qn = pl.q0[b + 1] - pl.q0[b], nqt = kp_tiles(qn, QR);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    int hk_staged = -1;
    const int pos = lr < nv ? key_pos(a, b, i0 + lr) : -1;   // of the key this thread stages
    for (int t = pc.t0; t < pc.t1; ++t) {
      const int hk = t / nqt, r0 = pl.q0[b] + (t - hk * nqt) * QR;
      const int rn = min(QR, pl.q0[b + 1] - r0) * a.G;
      __syncthreads();
      if (hk != hk_staged) {
        hk_staged = hk;
        const T *src = (const T *)a.k + ((long long)b * a.n_ctx + pos) * a.ld_kv + hk * D;
#pragma unroll 4
        for (int c = lc; c < D; c += 16)
          *reinterpret_cast<float4 *>(sk + lr * ld + c) =
              pos >= 0 ? load4(src + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      {
        const int g = lr / a.G;
        const T *src = (const T *)a.q + (r0 + g) * a.ld_q + (hk * a.G + lr - g * a.G) * D;
#pragma unroll 4
        for (int c = lc; c < D; c += 16)
          *reinterpret_cast<float4 *>(sq + lr * ld + c) =
              lr < rn ? load4(src + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (tid < MS_T) {
        // -inf: rows that are not there, or saw no key, weigh nothing
        float L = -INFINITY;
        if (tid < rn) L = a.lse[(size_t)(r0 + tid / a.G) * a.H + hk * a.G + tid % a.G] * KEY_LOG2E;
        sL[tid] = L;
      }
      __syncthreads();
      float s[4][4] = {};
#pragma unroll 4
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
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float L = sL[4 * ty + i];
          // a select: the score may be anything where L is -inf
          acc[j] += L == -INFINITY ? 0.f : exp2f(fmaf(s[i][j], c2, -L));
        }
    }
    // the key's sum over the 16 row groups
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) red[ty][tx + 16 * j] = acc[j];
    __syncthreads();
    if (tid < nv) {
      float v = 0.f;
#pragma unroll
      for (int y = 0; y < MS_THREADS / 16; ++y) v += red[y][tid];
      const bool whole = pc.t0 == 0 && pc.t1 == pc.T;
      float *dst = whole ? a.ws + 2 * (size_t)gridDim.x * MS_T + (size_t)b * a.n_ctx + i0
                         : a.ws + (size_t)kp_slot(blockIdx.x, pc.t0) * MS_T;
      dst[tid] = v;
    }
  }
}

// Adds each key's weight (`parts` sums of it): one thread per entry of a key
// set.  An entry that a list names twice counts twice, so the additions are
// atomic; a position that is named once receives one addition, and its result
// does not depend on any order.
// A block takes 32 entries at a time, its warps a unit's pieces in turn; the
// warps' sums are added in warp order.
__global__ void __launch_bounds__(256) key_mass_add_kernel(const KeyArgs a, int kt, int parts) {
  __shared__ KeyPlan pl;
  __shared__ float sum[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  key_plan_fetch(pl, a.plan, threadIdx.x, 256);
  __syncthreads();
  const int b = blockIdx.y;
  const int T = pl.T[b];
  if (T == 0) return;
  for (int i0 = blockIdx.x * 32; i0 < pl.kl[b]; i0 += gridDim.x * 32) {
    const int i = i0 + lane;                  // 32 entries lie in one unit
    const int wu = pl.wbase[b] + i0 / kt * (T + pl.ov);
    const int c0 = pl.per ? 0 : wu / pl.chunk, c1 = pl.per ? 0 : (wu + T + pl.ov - 1) / pl.chunk;
    float v = 0.f;
    for (int c = c0 + warp; c <= c1; c += 8) {
      int t0, t1;
      kp_piece_of(pl, wu, T, c, t0, t1);
      if (t1 <= t0) continue;
      const bool whole = t0 == 0 && t1 == T;
      if (whole && i >= pl.kl[b]) continue;
      const float *src = whole ? a.ws + 2 * (size_t)a.n_ctas * parts * kt + (size_t)b * a.n_ctx + i
                               : a.ws + (size_t)kp_slot(c, t0) * parts * kt + i % kt;
      const size_t step = whole ? (size_t)a.batch * a.n_ctx : kt;
      for (int q = 0; q < parts; ++q) v += __ldcg(src + q * step);
    }
    sum[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && i < pl.kl[b]) {
#pragma unroll
      for (int e = 1; e < 8; ++e) v += sum[e][lane];
      const int pos = key_pos(a, b, i);
      if (pos >= 0) atomicAdd(a.mass + (size_t)b * a.n_ctx + pos, v);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------- host --
namespace {
size_t mass_simt_smem(int D) { return (size_t)2 * MS_T * (D + 4) * 4; }

template <typename T> cudaError_t run_mass_simt(const KeyArgs &a, cudaStream_t s) {
  const cudaError_t e =
      launch_k(key_mass_simt_kernel<T>, a.n_ctas, MS_THREADS, mass_simt_smem(a.D), s, a);
  if (e != cudaSuccess) return e;
  return launch_key_mass_add(a, MS_T, 1, s);
}
}  // namespace

cudaError_t key_mass_setup(int dtype, int D) {
  if (key_attn_tc_takes(dtype, D)) return key_mass_tc_setup(D);
  const int smem = (int)mass_simt_smem(D);
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  return dtype == SL_BF16 ? cudaFuncSetAttribute(key_mass_simt_kernel<bf16>, attr, smem)
                          : cudaFuncSetAttribute(key_mass_simt_kernel<float>, attr, smem);
}

int key_mass_ctas(int dtype, int D, int num_sms) {
  return num_sms * (key_attn_tc_takes(dtype, D) ? 1 : 2);
}

size_t key_mass_ws_floats(int dtype, int D, int batch, int n_ctx, int n_ctas) {
  const bool tc = key_attn_tc_takes(dtype, D);
  const size_t slot = tc ? 2 * 256 : MS_T, parts = tc ? 2 : 1;
  return 2 * (size_t)n_ctas * slot + parts * batch * n_ctx;
}

cudaError_t launch_key_mass_add(const KeyArgs &a, int kt, int parts, cudaStream_t s) {
  const dim3 grid(std::min((a.n_ctx + 31) / 32, 1024), a.batch);
  return launch_k(key_mass_add_kernel, grid, 256, 0, s, a, kt, parts);
}

cudaError_t launch_key_mass(KeyArgs a, cudaStream_t s) {
  if (key_attn_tc_takes(a.dtype, a.D)) return launch_key_mass_tc(a, s);
  a.ov = 1;
  a.min_chunk = 1;
  a.join_cost = 0;
  return a.dtype == SL_BF16 ? run_mass_simt<bf16>(a, s) : run_mass_simt<float>(a, s);
}

}  // namespace sl
