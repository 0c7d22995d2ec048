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
// An exact order statistic by radix selection on the weights' order-preserving
// bits (11, 11 and 10 at a time), then a stable write of the list.  A cluster
// of CTAs takes one sequence, each a run of its entries: histograms and counts
// are summed over the cluster through distributed shared memory, whole numbers
// in a fixed order, so the result is exact and the same every time.
//
// Bound by latency: 4 x 2048 entries take 9.2 us, 4 x 131072 take 22 us (their
// bytes 0.6 us), of which 5 us are the second and third pass and about 6 us the
// first pass's loads and histogram.  Eight loads in flight a thread instead of
// four, ahead of the histogram: 0.7 us more.
#include "common.cuh"
#include "internal.h"

namespace sl {

namespace {
constexpr int EV_THREADS = 1024, EV_WARPS = EV_THREADS / 32;
constexpr int EV_BINS = 2048, EV_CLUSTER = 8;
constexpr int EV_CACHE = 48 * 1024;          // entries of a CTA kept in shared memory
constexpr uint32_t EV_FIXED = 0xffffffffu;   // above every weight's bits
constexpr uint32_t EV_ABSENT = 0u;           // below every weight's bits

// Order-preserving bits of a weight: -inf maps to 0x007fffff, +inf to
// 0xff800000; -0 counts as 0 and NaN as -inf.
__device__ __forceinline__ uint32_t ev_bits(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// A word of shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ int cluster_ld(const void *p, int rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p);
  int v;
  asm volatile("{\n .reg .u32 r;\n mapa.shared::cluster.u32 r, %1, %2;\n"
               " ld.shared::cluster.u32 %0, [r];\n}\n"
               : "=r"(v)
               : "r"(a), "r"(rank)
               : "memory");
  return v;
}

// The sum over the cluster of a word at the same place in every CTA.
__device__ __forceinline__ int cluster_total(const void *p, int n_c) {
  int v[EV_CLUSTER], t = 0;
#pragma unroll
  for (int r = 0; r < EV_CLUSTER; ++r) v[r] = r < n_c ? cluster_ld(p, r) : 0;
#pragma unroll
  for (int r = 0; r < EV_CLUSTER; ++r) t += v[r];
  return t;
}

struct EvShared {
  unsigned int hist[3][EV_BINS];
  int coarse[3][EV_WARPS];                   // sums of EV_BINS / 32 bins
  int wsum[EV_WARPS], wsum2[EV_WARPS];
  int fixed, cand;                           // of this CTA's entries
  int above, equal;                          // of this CTA's: kept for certain, at the threshold
  int digit, rank, count;                    // of the bin that holds the threshold
};
}  // namespace

__device__ __forceinline__ int ev_warp_sum(int v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

__global__ void __launch_bounds__(EV_THREADS) evict_kernel(
    int n_ctx, int budget, int seg, int cached, const float *__restrict__ mass,
    const uint8_t *protect, const uint8_t *present, int32_t *__restrict__ keys,
    int32_t *__restrict__ key_len, uint8_t *present_out) {
  extern __shared__ uint32_t ev_keys[];
  __shared__ EvShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int rank_c, n_c;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank_c));
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n_c));
  const size_t base = (size_t)(blockIdx.x / n_c) * n_ctx;
  // this CTA's entries: [e0, e0 + n)
  const int e0 = min(rank_c * seg, n_ctx), n = min(seg, n_ctx - e0);
  for (int i = tid; i < 3 * EV_BINS; i += EV_THREADS) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) sh.fixed = sh.cand = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  auto fetch = [&](int i) -> uint32_t {
    const size_t e = base + e0 + i;
    const float x = mass[e];                 // all three loads in flight together
    const bool here = !present || present[e], fixed = protect && protect[e];
    return !here ? EV_ABSENT : fixed ? EV_FIXED : ev_bits(x);
  };
  auto key = [&](int i) -> uint32_t { return cached ? ev_keys[i] : fetch(i); };
  auto candidate = [](uint32_t k) { return k != EV_FIXED && k != EV_ABSENT; };

  // counts, and the first histogram
  int nf = 0, nc = 0;
#pragma unroll 4
  for (int i = tid; i < n; i += EV_THREADS) {
    const uint32_t k = fetch(i);
    if (cached) ev_keys[i] = k;
    nf += k == EV_FIXED;
    if (candidate(k)) {
      ++nc;
      atomicAdd(&sh.hist[0][k >> 21], 1u);
    }
  }
  nf = warp_sum_i(nf);
  nc = warp_sum_i(nc);
  if (lane == 0) {
    atomicAdd(&sh.fixed, nf);
    atomicAdd(&sh.cand, nc);
  }
  auto coarse = [&](int pass) {               // a warp per 64 bins
    __syncthreads();
    const unsigned int *h = sh.hist[pass] + 64 * warp;
    const int v = warp_sum_i((int)(h[lane] + h[32 + lane]));
    if (lane == 0) sh.coarse[pass][warp] = v;
  };
  coarse(0);
  cluster_sync();
  const int fixed = cluster_total(&sh.fixed, n_c), cand = cluster_total(&sh.cand, n_c);
  const int room = min(max(0, budget - fixed), cand);
  // the room-th heaviest candidate: thr, of which `ties` are kept
  uint32_t thr = EV_FIXED;
  int ties = 0;
  if (room == cand) {
    thr = EV_ABSENT;
  } else if (room > 0) {
    uint32_t prefix = 0;
    int rank = room - 1;                     // from the heaviest, 0-based
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      if (pass > 0) {
        const uint32_t pmask = pass == 1 ? 0xffe00000u : 0xfffffc00u;
        const uint32_t dmask = pass == 1 ? 0x7ffu : 0x3ffu;
#pragma unroll 4
        for (int i = tid; i < n; i += EV_THREADS) {
          const uint32_t k = key(i);
          if (candidate(k) && (k & pmask) == prefix)
            atomicAdd(&sh.hist[pass][(k >> shift) & dmask], 1u);
        }
        coarse(pass);
        cluster_sync();
      }
      // One warp finds the digit, from the heaviest bin: the 64 bins that hold
      // it by the coarse sums, then the bin.  (All bins read from every CTA took
      // 9 us of 27 at 4 x 131072 entries.)
      if (warp == 0) {
        const int c = cluster_total(&sh.coarse[pass][31 - lane], n_c);
        const int ci = ev_warp_sum(c, lane);
        const unsigned int at = __ballot_sync(0xffffffffu, ci - c <= rank && rank < ci);
        const int src = __ffs(at) - 1;       // some bins hold it: at is not zero
        const int rest = rank - __shfl_sync(0xffffffffu, ci - c, src);
        const int d = 64 * (31 - src) + 63 - 2 * lane;
        const int h1 = cluster_total(&sh.hist[pass][d], n_c);
        const int h0 = cluster_total(&sh.hist[pass][d - 1], n_c);
        const int hi = ev_warp_sum(h1 + h0, lane), excl = hi - h1 - h0;
        if (excl <= rest && rest < hi) {
          const bool low = rest >= excl + h1;
          sh.digit = low ? d - 1 : d;
          sh.rank = rest - excl - (low ? h1 : 0);
          sh.count = low ? h0 : h1;
        }
      }
      __syncthreads();
      prefix |= (uint32_t)sh.digit << shift;
      rank = sh.rank;
      const bool all = rank + 1 == sh.count;
      __syncthreads();
      if (all) {
        // the whole bin stays: everything from its first weight on, no ties
        // left to settle (mostly so after two passes)
        thr = prefix - 1;
        break;
      }
      thr = prefix;
      ties = pass == 2 ? rank + 1 : 0;
    }
  }
  // a warp's run of this CTA's entries: how many are kept for certain, and how
  // many equal the threshold
  const int run = (n + EV_WARPS - 1) / EV_WARPS;
  const int i0 = min(warp * run, n), i1 = min(i0 + run, n);
  auto above = [&](uint32_t k) { return k != EV_ABSENT && (k == EV_FIXED || k > thr); };
  auto equal = [&](uint32_t k) { return k == thr && candidate(k); };
  int ca = 0, ce = 0;
#pragma unroll 4
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t k = key(i);
    ca += above(k);
    ce += equal(k);
  }
  ca = warp_sum_i(ca);
  ce = warp_sum_i(ce);
  if (lane == 0) {
    sh.wsum[warp] = ca;
    sh.wsum2[warp] = ce;
  }
  __syncthreads();
  // lanes as warps: entries of the earlier warps of this CTA
  int wa = lane < warp ? sh.wsum[lane] : 0, we = lane < warp ? sh.wsum2[lane] : 0;
  wa = warp_sum_i(wa);
  we = warp_sum_i(we);
  if (warp == EV_WARPS - 1 && lane == 0) {
    sh.above = wa + ca;
    sh.equal = we + ce;
  }
  cluster_sync();
  int out = wa, seen = we, ta = 0, te = 0;   // before this warp; of the sequence
  int xa[EV_CLUSTER], xe[EV_CLUSTER];
#pragma unroll
  for (int r = 0; r < EV_CLUSTER; ++r) {
    xa[r] = r < n_c ? cluster_ld(&sh.above, r) : 0;
    xe[r] = r < n_c ? cluster_ld(&sh.equal, r) : 0;
  }
#pragma unroll
  for (int r = 0; r < EV_CLUSTER; ++r) {
    ta += xa[r];
    te += xe[r];
    out += r < rank_c ? xa[r] : 0;
    seen += r < rank_c ? xe[r] : 0;
  }
  out += min(seen, ties);
  // stable write: entries above thr, and the first `ties` equal to it
  const unsigned int below = (1u << lane) - 1u;
#pragma unroll 4
  for (int i = i0; i < i1; i += 32) {
    const uint32_t k = i + lane < i1 ? key(i + lane) : EV_ABSENT;
    const bool eq = equal(k);
    const unsigned int be = __ballot_sync(0xffffffffu, eq);
    const bool keep = above(k) || (eq && seen + __popc(be & below) < ties);
    const unsigned int bk = __ballot_sync(0xffffffffu, keep);
    if (keep) keys[base + out + __popc(bk & below)] = e0 + i + lane;
    if (present_out && i + lane < i1) present_out[base + e0 + i + lane] = keep;
    out += __popc(bk);
    seen += __popc(be);
  }
  if (rank_c == 0 && tid == 0) key_len[blockIdx.x / n_c] = ta + min(te, ties);
  cluster_sync();                            // no CTA leaves while another reads its counts
}

// The longest that is offered: its eight CTAs read 2^17 entries each in every pass.
int evict_max_ctx() { return 1 << 20; }

cudaError_t launch_evict(int batch, int n_ctx, int budget, const float *mass,
                         const uint8_t *protect, const uint8_t *present, int32_t *keys,
                         int32_t *key_len, uint8_t *present_out, cudaStream_t s) {
  // CTAs a sequence by entries a thread: a cluster's exchanges cost about what it
  // shares out at four (4 sequences, with 1 / 2 / 4 / 8 CTAs each: 2048 entries 9.2 /
  // 8.9 / 8.9 / 9.7 us, 4096 10.3 / 9.7 / 9.1 / 9.9, 8192 12.7 / 10.7 / 9.8 / 10.1,
  // 12000 12.7 / 9.4 / 7.9 / 8.4, 16384 14.7 / 10.3 / 8.1 / 8.0, 24000 19.6 / 12.9 /
  // 9.5 / 8.7); beyond that the largest portable cluster
  const int cs = n_ctx <= 4 * EV_THREADS ? 1 : n_ctx <= 8 * EV_THREADS ? 2
                 : n_ctx <= 16 * EV_THREADS ? 4 : EV_CLUSTER;
  const int seg = (n_ctx + cs - 1) / cs, cached = seg <= EV_CACHE;
  const size_t smem = cached ? (size_t)seg * 4 : 0;
  if (smem > 16 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, EV_CACHE * 4);
    if (e != cudaSuccess) return e;
  }
  return launch_k_cluster(cs, evict_kernel, dim3(batch * cs), EV_THREADS, smem, s, n_ctx, budget,
                          seg, cached, mass, protect, present, keys, key_len, present_out);
}

}  // namespace sl
