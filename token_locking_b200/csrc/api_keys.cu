// Host side of the key-set operators: attention over a key set per sequence,
// the attention weight each key receives, and eviction by that weight.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <new>

#include "common.cuh"
#include "internal.h"

using namespace sl;

struct sl_key_attn {
  sl_key_attn_config cfg;
  int device, num_sms, group;
  int attn_ctas, mass_ctas, stack_rows;
  float scale;
  float *ws = nullptr;
  int *err = nullptr;
};

namespace {
size_t elem_size(int dtype) { return dtype == SL_BF16 ? 2 : 4; }

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// A row-major operand of `cols` columns with 16-byte aligned rows.
bool rows_ok(const void *p, long long ld, int cols, size_t es) {
  return p && aligned16(p) && ld >= cols && (ld * es) % 16 == 0 && ld <= (long long)INT_MAX;
}

sl_status fill_args(const sl_key_attn *a, const char *fn, int rows, const void *d_q,
                    int64_t ld_q, const void *d_k, int64_t ld_kv, const sl_key_set *set,
                    int prefix_len, KeyArgs *x) {
  if (!a) return fail(SL_ERR_INVALID, "%s: null object", fn);
  const sl_key_attn_config &c = a->cfg;
  if (prefix_len < 0 || prefix_len > KEY_MAX_ROWS)
    return fail(SL_ERR_INVALID, "%s: prefix_len %d outside [0, 2^31 - 2^16]", fn, prefix_len);
  int dev = -1;
  SL_CUDA(cudaGetDevice(&dev));
  if (dev != a->device)
    return fail(SL_ERR_INVALID, "%s: the object belongs to device %d, the current one is %d", fn,
                a->device, dev);
  if (rows < 0 || rows > c.max_rows)
    return fail(SL_ERR_INVALID, "%s: rows %d outside [0, max_rows = %d]", fn, rows, c.max_rows);
  if (!set || !set->d_seq_off) return fail(SL_ERR_INVALID, "%s: null key set or offsets", fn);
  const size_t es = elem_size(c.dtype);
  if (rows > 0 && !rows_ok(d_q, ld_q, c.n_heads * c.head_dim, es))
    return fail(SL_ERR_INVALID, "%s: q needs 16-byte aligned rows of at least %d columns", fn,
                c.n_heads * c.head_dim);
  if (!rows_ok(d_k, ld_kv, c.n_kv_heads * c.head_dim, es))
    return fail(SL_ERR_INVALID, "%s: k/v need 16-byte aligned rows of at least %d columns", fn,
                c.n_kv_heads * c.head_dim);
  // the work plan counts (row block, head, key tile) triples in 32 bits
  const double tiles = (double)(prefix_len + (double)c.n_ctx) / 64.0 + 4;
  const double blocks = c.n_kv_heads * ((double)rows * a->group / 32.0 + 2.0 * c.batch);
  if (tiles * (blocks + 2.0 * c.batch) > 1e9)
    return fail(SL_ERR_UNSUPPORTED, "%s: rows x keys x heads too large for one call", fn);
  *x = KeyArgs{};
  x->dtype = c.dtype;
  x->batch = c.batch;
  x->n_ctx = c.n_ctx;
  x->M = rows;
  x->H = c.n_heads;
  x->Hkv = c.n_kv_heads;
  x->G = a->group;
  x->D = c.head_dim;
  x->prefix_len = prefix_len;
  x->stack = prefix_len > 0 && rows <= a->stack_rows;
  x->scale = a->scale;
  x->q = d_q;
  x->k = d_k;
  x->ld_q = ld_q;
  x->ld_kv = ld_kv;
  x->seq_off = set->d_seq_off;
  x->key_len = set->d_key_len;
  x->keys = set->d_keys;
  x->plan = reinterpret_cast<int *>(a->ws);
  x->ws = a->ws + KEY_PLAN_WORDS;
  x->err = a->err;
  x->wait_ns = wait_limit_ns() ? wait_limit_ns() : WAIT_LIMIT_NS;
  return SL_OK;
}
}  // namespace

extern "C" sl_status sl_key_attn_create(const sl_key_attn_config *cfg, sl_key_attn **out) {
  if (!cfg || !out) return fail(SL_ERR_INVALID, "sl_key_attn_create: null argument");
  *out = nullptr;
  if (cfg->dtype != SL_F32 && cfg->dtype != SL_BF16)
    return fail(SL_ERR_INVALID, "sl_key_attn_create: dtype %d", cfg->dtype);
  if (cfg->batch < 1 || cfg->batch > SL_MAX_BATCH || cfg->n_ctx < 1 ||
      (long long)cfg->batch * cfg->n_ctx > KEY_MAX_ROWS)
    return fail(SL_ERR_INVALID, "sl_key_attn_create: batch in [1, %d], n_ctx > 0 and batch * n_ctx "
                "up to 2^31 - 2^16 required", SL_MAX_BATCH);
  if (cfg->max_rows < 1 || cfg->max_rows > KEY_MAX_ROWS)
    return fail(SL_ERR_INVALID, "sl_key_attn_create: max_rows %d outside [1, 2^31 - 2^16]",
                cfg->max_rows);
  if (cfg->n_heads < 1 || cfg->n_kv_heads < 1 || cfg->n_heads % cfg->n_kv_heads != 0)
    return fail(SL_ERR_INVALID, "sl_key_attn_create: n_kv_heads %d does not divide n_heads %d",
                cfg->n_kv_heads, cfg->n_heads);
  const int group = cfg->n_heads / cfg->n_kv_heads;
  if (group > 64)
    return fail(SL_ERR_UNSUPPORTED, "sl_key_attn_create: %d query heads per K/V head (64 at most)",
                group);
  const size_t es = elem_size(cfg->dtype);
  if (cfg->head_dim < 1 || cfg->head_dim > 128 || (cfg->head_dim * es) % 16 != 0)
    return fail(SL_ERR_UNSUPPORTED, "sl_key_attn_create: head_dim %d (16-byte multiples up to 128 "
                "elements)", cfg->head_dim);
  if (cfg->n_heads > (1 << 20) / cfg->head_dim)
    return fail(SL_ERR_UNSUPPORTED, "sl_key_attn_create: n_heads * head_dim above 2^20");
  if (!(cfg->scale >= 0.f) || !isfinite(cfg->scale))
    return fail(SL_ERR_INVALID, "sl_key_attn_create: scale must be positive and finite (0 = default)");
  sl_key_attn *a = new (std::nothrow) sl_key_attn();
  if (!a) return fail(SL_ERR_OOM, "sl_key_attn_create: host allocation failed");
  a->cfg = *cfg;
  a->group = group;
  a->scale = cfg->scale > 0.f ? cfg->scale : 1.f / sqrtf((float)cfg->head_dim);
  cudaError_t e = cudaGetDevice(&a->device);
  if (e == cudaSuccess)
    e = cudaDeviceGetAttribute(&a->num_sms, cudaDevAttrMultiProcessorCount, a->device);
  if (e == cudaSuccess) e = key_attn_setup(cfg->dtype, cfg->head_dim);
  if (e == cudaSuccess) e = key_mass_setup(cfg->dtype, cfg->head_dim);
  if (e != cudaSuccess) {
    delete a;
    return cuda_fail(e, "sl_key_attn_create");
  }
  a->attn_ctas = key_attn_ctas(cfg->dtype, cfg->head_dim, a->num_sms);
  a->mass_ctas = key_mass_ctas(cfg->dtype, cfg->head_dim, a->num_sms);
  // a joint pass over the prefix pays while a sequence's rows leave much of a
  // unit's 256 empty, and takes 1 KB of workspace a row and head (heads of 128): up to
  // 96 packed rows a sequence.  (32 heads over a prefix of 8192: 16 x 64 rows 194 us,
  // 437 without; 16 x 112 rows 445 us, 319 if the workspace reached that far.)
  a->stack_rows =
      cfg->prefix ? (int)std::min<long long>(cfg->max_rows, (long long)96 * cfg->batch / group) : 0;
  const size_t floats = std::max(
      key_attn_ws_floats(cfg->dtype, cfg->head_dim, cfg->n_heads, a->attn_ctas, a->stack_rows),
      key_mass_ws_floats(cfg->dtype, cfg->head_dim, cfg->batch, cfg->n_ctx, a->mass_ctas));
  a->err = device_error_word();
  if (!a->err || cudaMalloc((void **)&a->ws, (floats + KEY_PLAN_WORDS) * sizeof(float)) != cudaSuccess) {
    cudaGetLastError();
    sl_key_attn_destroy(a);
    return fail(SL_ERR_OOM, "sl_key_attn_create: device allocation failed");
  }
  *out = a;
  return SL_OK;
}

extern "C" void sl_key_attn_destroy(sl_key_attn *a) {
  if (!a) return;
  if (a->ws) cudaFree(a->ws);
  delete a;
}

extern "C" sl_status sl_key_attention(sl_key_attn *a, int rows, const void *d_q, int64_t ld_q,
                                      const void *d_k, const void *d_v, int64_t ld_kv,
                                      const sl_key_set *set, const void *d_k_prefix,
                                      const void *d_v_prefix, int64_t ld_prefix, int prefix_len,
                                      void *d_o, int64_t ld_o, float *d_lse, void *stream) {
  KeyArgs x;
  sl_status st = fill_args(a, "sl_key_attention", rows, d_q, ld_q, d_k, ld_kv, set, prefix_len, &x);
  if (st != SL_OK) return st;
  const sl_key_attn_config &c = a->cfg;
  const size_t es = elem_size(c.dtype);
  const int hd = c.n_heads * c.head_dim, hkd = c.n_kv_heads * c.head_dim;
  if (!d_v || !aligned16(d_v))
    return fail(SL_ERR_INVALID, "sl_key_attention: v must be 16-byte aligned and not null");
  if (prefix_len > 0) {
    if (!c.prefix)
      return fail(SL_ERR_INVALID, "sl_key_attention: the object was created without a prefix");
    if (!rows_ok(d_k_prefix, ld_prefix, hkd, es) || !rows_ok(d_v_prefix, ld_prefix, hkd, es))
      return fail(SL_ERR_INVALID, "sl_key_attention: the prefix needs 16-byte aligned rows of at "
                  "least %d columns", hkd);
  }
  if (rows == 0) return SL_OK;
  if (!rows_ok(d_o, ld_o, hd, es))
    return fail(SL_ERR_INVALID, "sl_key_attention: o needs 16-byte aligned rows of at least %d "
                "columns", hd);
  x.v = d_v;
  x.kp = d_k_prefix;
  x.vp = d_v_prefix;
  x.ld_p = ld_prefix;
  x.o = d_o;
  x.ld_o = ld_o;
  x.lse = d_lse;
  x.n_ctas = a->attn_ctas;
  x.lost = key_attn_tc_takes(c.dtype, c.head_dim) ? take_lost_load() : 0;
  SL_CUDA(launch_key_attn(x, (cudaStream_t)stream));
  return SL_OK;
}

extern "C" sl_status sl_key_mass(sl_key_attn *a, int rows, const void *d_q, int64_t ld_q,
                                 const void *d_k, int64_t ld_kv, const sl_key_set *set,
                                 const float *d_lse, float decay, const float *d_mass_prev,
                                 float *d_mass, void *stream) {
  KeyArgs x;
  sl_status st = fill_args(a, "sl_key_mass", rows, d_q, ld_q, d_k, ld_kv, set, 0, &x);
  if (st != SL_OK) return st;
  if (!d_mass || (rows > 0 && !d_lse))
    return fail(SL_ERR_INVALID, "sl_key_mass: null lse or mass");
  if (!isfinite(decay)) return fail(SL_ERR_INVALID, "sl_key_mass: decay must be finite");
  if (decay != 0.f && !d_mass_prev)
    return fail(SL_ERR_INVALID, "sl_key_mass: decay %g needs the previous weights", decay);
  x.lse = const_cast<float *>(d_lse);
  x.decay = decay;
  x.mass_prev = d_mass_prev;
  x.mass = d_mass;
  x.n_ctas = a->mass_ctas;
  x.lost = rows > 0 && key_attn_tc_takes(x.dtype, x.D) ? take_lost_load() : 0;
  SL_CUDA(launch_key_mass(x, (cudaStream_t)stream));
  return SL_OK;
}

extern "C" sl_status sl_kv_evict(int batch, int n_ctx, int budget, const float *d_mass,
                                 const uint8_t *d_protect, const uint8_t *d_present,
                                 int32_t *d_keys, int32_t *d_key_len, uint8_t *d_present_out,
                                 void *stream) {
  if (batch < 1 || batch > SL_MAX_BATCH || n_ctx < 1 || (long long)batch * n_ctx > INT_MAX)
    return fail(SL_ERR_INVALID, "sl_kv_evict: batch in [1, %d], n_ctx > 0 and batch * n_ctx below "
                "2^31 required", SL_MAX_BATCH);
  if (n_ctx > evict_max_ctx())
    return fail(SL_ERR_UNSUPPORTED, "sl_kv_evict: n_ctx %d above %d", n_ctx, evict_max_ctx());
  if (budget < 0) return fail(SL_ERR_INVALID, "sl_kv_evict: budget %d < 0", budget);
  if (!d_mass || !d_keys || !d_key_len) return fail(SL_ERR_INVALID, "sl_kv_evict: null argument");
  SL_CUDA(launch_evict(batch, n_ctx, budget, d_mass, d_protect, d_present, d_keys, d_key_len,
                       d_present_out, (cudaStream_t)stream));
  return SL_OK;
}
