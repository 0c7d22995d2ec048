// Eviction from the cache by accumulated attention weight: each sequence keeps
// its protected entries (the active rows, whose K/V are rewritten every step)
// and the heaviest of the others up to a budget.
//
//   here    = present,  fixed = here && protect,  cand = here && !protect
//   r       = max(0, budget - |fixed|)
//   kept    = fixed or one of the r heaviest candidates (ties to the lower
//             position; NaN weighs as little as -inf)
//   keys    = the kept positions in ascending order, key_len their number
//
// One CTA per sequence: an exact order statistic by radix selection on the
// weights' order-preserving bits, then a stable write of the list.
#include "common.cuh"
#include "internal.h"

namespace sl {

namespace {
constexpr int EV_THREADS = 1024;
constexpr uint32_t EV_FIXED = 0xffffffffu;   // above every weight's bits
constexpr uint32_t EV_ABSENT = 0u;           // below every weight's bits

// Order-preserving bits of a weight: -inf maps to 0x007fffff, +inf to
// 0xff800000; -0 counts as 0 and NaN as -inf.
__device__ __forceinline__ uint32_t ev_bits(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
}  // namespace

__global__ void __launch_bounds__(EV_THREADS) evict_kernel(
    int n_ctx, int budget, const float *__restrict__ mass, const uint8_t *protect,
    const uint8_t *present, int32_t *__restrict__ keys, int32_t *__restrict__ key_len,
    uint8_t *present_out) {
  __shared__ unsigned int hist[256];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_rank, sh_fixed, sh_cand, wsum[32], wsum2[32], tot, tot2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t base = (size_t)blockIdx.x * n_ctx;
  pdl_wait();
  pdl_trigger();
  auto key = [&](int i) -> uint32_t {
    if (present && !present[base + i]) return EV_ABSENT;
    if (protect && protect[base + i]) return EV_FIXED;
    return ev_bits(mass[base + i]);
  };
  if (tid == 0) sh_fixed = sh_cand = 0;
  __syncthreads();
  int nf = 0, nc = 0;
  for (int i = tid; i < n_ctx; i += EV_THREADS) {
    const uint32_t k = key(i);
    nf += k == EV_FIXED;
    nc += k != EV_FIXED && k != EV_ABSENT;
  }
  nf = warp_sum_i(nf);
  nc = warp_sum_i(nc);
  if (lane == 0) {
    atomicAdd(&sh_fixed, nf);
    atomicAdd(&sh_cand, nc);
  }
  __syncthreads();
  const int room = min(max(0, budget - sh_fixed), sh_cand);
  // the room-th heaviest candidate: thr, of which `ties` are kept
  uint32_t thr = EV_FIXED, pmask = 0;
  int ties = 0;
  if (room == sh_cand) {
    thr = EV_ABSENT;
  } else if (room > 0) {
    uint32_t prefix = 0;
    int rank = room - 1;                       // from the heaviest, 0-based
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += EV_THREADS) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n_ctx; i += EV_THREADS) {
        const uint32_t k = key(i);
        if (k != EV_FIXED && k != EV_ABSENT && (k & pmask) == prefix)
          atomicAdd(&hist[(k >> shift) & 0xff], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        int r = rank, d = 255;
        while (d > 0 && r >= (int)hist[d]) r -= (int)hist[d--];
        sh_prefix = prefix | ((uint32_t)d << shift);
        sh_rank = r;
      }
      __syncthreads();
      prefix = sh_prefix;
      rank = sh_rank;
      pmask |= 0xffu << shift;
      __syncthreads();
    }
    thr = prefix;
    ties = rank + 1;
  }
  // stable write: entries above thr, and the first `ties` equal to it
  int out = 0, seen = 0;
  for (int i0 = 0; i0 < n_ctx; i0 += EV_THREADS) {
    const int i = i0 + tid;
    const uint32_t k = i < n_ctx ? key(i) : EV_ABSENT;
    const bool eq = k == thr && thr != EV_ABSENT && thr != EV_FIXED;
    const unsigned int be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) wsum2[warp] = __popc(be);
    __syncthreads();
    if (warp == 0) {
      int v = wsum2[lane], inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      wsum2[lane] = inc - v;
      if (lane == 31) tot2 = inc;
    }
    __syncthreads();
    const int nth = seen + wsum2[warp] + __popc(be & ((1u << lane) - 1u));
    const bool keep = k != EV_ABSENT && (k == EV_FIXED || k > thr || (eq && nth < ties));
    const unsigned int bk = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) wsum[warp] = __popc(bk);
    __syncthreads();
    if (warp == 0) {
      int v = wsum[lane], inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      wsum[lane] = inc - v;
      if (lane == 31) tot = inc;
    }
    __syncthreads();
    if (keep) keys[base + out + wsum[warp] + __popc(bk & ((1u << lane) - 1u))] = i;
    if (present_out && i < n_ctx) present_out[base + i] = keep;
    out += tot;
    seen += tot2;
    __syncthreads();
  }
  if (tid == 0) key_len[blockIdx.x] = out;
}

int evict_max_ctx() { return 1 << 20; }

cudaError_t launch_evict(int batch, int n_ctx, int budget, const float *mass,
                         const uint8_t *protect, const uint8_t *present, int32_t *keys,
                         int32_t *key_len, uint8_t *present_out, cudaStream_t s) {
  return launch_k(evict_kernel, batch, EV_THREADS, 0, s, n_ctx, budget, mass, protect, present,
                  keys, key_len, present_out);
}

}  // namespace sl
