// Helpers shared by the key-set kernels.
#pragma once
#include "common.cuh"
#include "internal.h"

namespace sl {

constexpr float KEY_LOG2E = 1.4426950408889634f;
constexpr float KEY_LN2 = 0.6931471805599453f;

// 4 consecutive elements as fp32, and back
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const bf16 *p) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(bf16 *p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t *>(&a);
  u.y = *reinterpret_cast<uint32_t *>(&b);
  *reinterpret_cast<uint2 *>(p) = u;
}

// 1 / l for a row's sum of weights l: a NaN stays one.
__device__ __forceinline__ float key_inv(float l) { return l > 0.f ? 1.f / l : l; }
// o / l; 0 for a row without weight, whose o may be 0 times an infinite v.
__device__ __forceinline__ float4 key_mean(float4 o, float l, float inv) {
  if (l == 0.f) return make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

// Position of entry i of sequence b's key set; -1 for a list entry outside
// [0, n_ctx), which stands for a key and value of zeros and is reported.
__device__ __forceinline__ int key_pos(const KeyArgs &a, int b, int i) {
  if (!a.keys) return i;
  const int n = a.keys[(size_t)b * a.n_ctx + i];
  if ((unsigned)n < (unsigned)a.n_ctx) return n;
  atomicCAS(a.err, DEV_OK, DEV_BAD_INDEX);    // an earlier report stays
  return -1;
}

// mass = decay mass_prev at every position, before the weights are added.
__device__ __forceinline__ void key_mass_start(const KeyArgs &a, int i, int n_threads) {
  const long long n = (long long)a.batch * a.n_ctx;
  for (long long e = i; e < n; e += n_threads)
    a.mass[e] = a.decay == 0.f ? 0.f : a.decay * a.mass_prev[e];
}

// Partial rows (maximum in base 2, sum, unnormalised o): two slots of rt packed
// rows per CTA for units that a share cut, then (with a joint prefix) one per
// row, head and part.  All o rows come first, then all (maximum, sum) pairs.
struct KeyRecs {
  float *o;
  float2 *ml;
  int D;
  __device__ __forceinline__ KeyRecs(const KeyArgs &a, int rt) {
    const size_t n = 2 * (size_t)a.n_ctas * rt + (a.stack ? 2 * (size_t)a.M * a.H : 0);
    o = a.ws;
    ml = reinterpret_cast<float2 *>(a.ws + n * a.D);
    D = a.D;
  }
};
__device__ __forceinline__ size_t key_rec_slot(int slot, int rt, int r) {
  return (size_t)slot * rt + r;
}
__device__ __forceinline__ size_t key_rec_row(const KeyArgs &a, int rt, int part, int row, int h) {
  return 2 * (size_t)a.n_ctas * rt + ((size_t)part * a.M + row) * a.H + h;
}

}  // namespace sl
