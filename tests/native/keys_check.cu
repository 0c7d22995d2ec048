// Host-only checks of the key-set operators (no GPU needed): sizes whose tile
// arithmetic would pass 32 bits are refused before anything is launched, and a
// kernel that gives up waits for the last fill of every stage of its ring.  It
// includes the host side's source so that it sees objects as the library makes
// them.
#include "api_keys.cu"
#include "keys_tc.cuh"

#include <cstdio>

static int g_fail = 0;
static long g_checked = 0;

#define CHECK(cond, ...)                                              \
  do {                                                                \
    ++g_checked;                                                      \
    if (!(cond)) {                                                    \
      if (++g_fail <= 25) {                                           \
        printf("FAIL (%s) ", #cond);                                  \
        printf(__VA_ARGS__);                                          \
        printf("\n");                                                 \
      }                                                               \
    }                                                                 \
  } while (0)

static void check_sizes() {
  // the last tile and the last grid stride of the largest sizes stay in range
  for (long long past : {255ll, 2 * 96ll, 1024 * 32ll})
    CHECK(KEY_MAX_ROWS + past <= INT_MAX, "%lld past the last row", past);
  CHECK(KEY_MAX_ROWS == 2147418112, "2^31 - 2^16");
  const sl_key_attn_config good{SL_BF16, 1, 64, 8, 2, 2, 64, 1, 0.f};
  sl_key_attn *out = nullptr;
  for (int n : {KEY_MAX_ROWS + 1, INT_MAX - 300, INT_MAX}) {
    sl_key_attn_config c = good;
    c.n_ctx = n;
    CHECK(sl_key_attn_create(&c, &out) == SL_ERR_INVALID && !out, "n_ctx %d", n);
    c = good;
    c.max_rows = n;
    CHECK(sl_key_attn_create(&c, &out) == SL_ERR_INVALID && !out, "max_rows %d", n);
    sl_key_attn a{};
    a.cfg = good;
    a.group = 1;
    const int32_t *off = reinterpret_cast<const int32_t *>(16);
    const sl_key_set set{off, nullptr, nullptr};
    const void *p = reinterpret_cast<const void *>(16);
    CHECK(sl_key_attention(&a, 1, p, 128, p, p, 128, &set, p, p, 128, n, const_cast<void *>(p), 128,
                           nullptr, nullptr) == SL_ERR_INVALID,
          "prefix_len %d", n);
  }
  sl_key_attn_config c = good;
  c.batch = 64;
  c.n_ctx = 1 << 25;
  CHECK(sl_key_attn_create(&c, &out) == SL_ERR_INVALID && !out, "64 x 2^25");
}

// A barrier that has completed n phases lets a waiter for parity p pass if the
// phase under way has the other one.
static bool passes(int n, uint32_t p) { return ((uint32_t)n & 1u) != p; }

static void check_rings() {
  for (int stages = 1; stages <= 9; ++stages)
    for (int fills = 0; fills <= 4 * stages + 1; ++fills) {
      const int st = fills % stages;
      const uint32_t ph = (uint32_t)(fills / stages) & 1u;
      for (int s = 0; s < stages; ++s) {
        const int own = fills / stages + (s < st);   // fills of this stage
        const uint32_t p = key_ring_parity(s, st, ph);
        CHECK(passes(own, p), "stage %d of %d after %d fills, all landed", s, stages, fills);
        CHECK(own == 0 || !passes(own - 1, p), "stage %d of %d after %d fills, one in flight", s,
              stages, fills);
      }
    }
}

int main() {
  check_sizes();
  check_rings();
  printf("%ld checks, %d failures\n", g_checked, g_fail);
  return g_fail != 0;
}
