// Helpers shared by the key-set kernels on the tensor cores.
#pragma once
#include "tc_ptx.cuh"

namespace sl {

// N fp32 columns of this thread's TMEM lane (N a multiple of 8), one wait.
template <int N> __device__ __forceinline__ void tmem_ld_cols(uint32_t t, float *s) {
#pragma unroll
  for (int c = 0; c + 32 <= N; c += 32) tmem_ld32_nw(t + c, s + c);
  if constexpr (N % 32 >= 16) tmem_ld16_nw(t + N / 32 * 32, s + N / 32 * 32);
  if constexpr (N % 16 == 8) tmem_ld8_nw(t + N - 8, s + N - 8);
  tmem_wait_ld();
}
// N columns of it (N a multiple of 4), without a wait.
template <int N> __device__ __forceinline__ void tmem_st_cols(uint32_t t, const uint32_t *r) {
  static_assert(N < 32 && N % 4 == 0, "columns");
  if constexpr (N >= 16) tmem_st16_u(t, r);
  if constexpr (N % 16 >= 8) tmem_st8_u(t + N / 16 * 16, r + N / 16 * 16);
  if constexpr (N % 8 == 4) tmem_st4_u(t + N - 4, r + N - 4);
}
// The largest of s[0..N) (N even).
template <int N> __device__ __forceinline__ float max_of(const float *s) {
  float a = s[0], b = s[1];
#pragma unroll
  for (int i = 2; i + 3 < N; i += 4) {
    a = max3(a, s[i], s[i + 1]);
    b = max3(b, s[i + 2], s[i + 3]);
  }
  if constexpr (N % 4 == 0) a = max3(a, s[N - 2], s[N - 1]);
  return fmaxf(a, b);
}

// All lanes wait; the outcome is the same for all.  The waiting loop is kept out
// of line: the roles' code competes for the instruction caches.
static __device__ __noinline__ bool key_wait_long(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                          unsigned long long lim) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, lim));
}
__device__ __forceinline__ bool key_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                        unsigned long long lim) {
  if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
  return key_wait_long(bar, parity, abort_flag, lim);
}

// Parity of the last fill of stage s of a ring whose next fill goes to stage st in
// the phase of parity ph.  (For a stage never filled: parity 1, for which a new
// barrier lets its waiter pass.)
__host__ __device__ __forceinline__ uint32_t key_ring_parity(int s, int st, uint32_t ph) {
  return s < st ? ph : ph ^ 1u;
}

// Where warp 0's copies ended, for whoever waits for them.
struct KeyFills {
  int st, ph;                 // the ring's next stage and its parity
  int n;                      // fills of the other operand's barrier
};
// Waits, within the limit, for the last fills of a ring of `stages` barriers and of
// the other operand's: those of a CTA that gave up, which must land before it exits
// (otherwise the issuing warps have waited for each).  A fill that was not handed
// over costs its share of the limit.
static __device__ __noinline__ void key_drain(const KeyFills &f, uint32_t ring, int stages,
                                              uint32_t other, unsigned long long lim) {
  volatile int never = 0;
  if (f.n > 0) mbar_wait(other, (uint32_t)(f.n - 1) & 1u, &never, lim / 2);
  for (int s = 0; s < stages; ++s)
    mbar_wait(ring + 8u * (uint32_t)s, key_ring_parity(s, f.st, (uint32_t)f.ph), &never,
              lim / (2 * stages));
}

// Keeps a branch a branch: masks turned into selects cost two instructions a
// score in every tile, a third of the softmax's.
__device__ __forceinline__ void key_cold() { asm volatile("" ::: "memory"); }
// One lane of the warp (the same every time).
__device__ __forceinline__ bool key_elect() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok));
  return ok != 0;
}
// 16 bytes to shared memory, zeros where the source is not there.
__device__ __forceinline__ void key_copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void key_copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N> __device__ __forceinline__ void key_copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace sl
