// Host-only checks of the key-set operators (no GPU needed): sizes whose tile
// arithmetic would pass 32 bits are refused before anything is launched.  It
// includes the host side's source so that it sees objects as the library makes
// them.
#include "api_keys.cu"

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

int main() {
  check_sizes();
  printf("%ld checks, %d failures\n", g_checked, g_fail);
  return g_fail != 0;
}
