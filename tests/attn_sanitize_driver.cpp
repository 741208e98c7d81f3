// Drives the host code of the attention-side entry points -- argument
// validation and workspace sizes, with sizes at the ends of their types --
// under AddressSanitizer and UndefinedBehaviorSanitizer (host code only; no
// call here reaches a launch).  Built and run by tests/test_attn_sanitizers.py.
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "bitlinear.h"

#define CHECK(c)                                                       \
  do {                                                                 \
    if (!(c)) {                                                        \
      std::fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); \
      return 1;                                                        \
    }                                                                  \
  } while (0)

int main() {
  alignas(256) static unsigned char stand_in[4096];  // only its address is used
  unsigned char* A = stand_in;
  uint16_t* B = (uint16_t*)A;
  float* F = (float*)A;
  int32_t* I = (int32_t*)A;
  const int64_t ends[] = {INT64_MIN, -(1ll << 32), -1, 0, 1, 2, 63, 64, 65, 128, 4096, 4097, (1ll << 22) - 8, 1ll << 22,
                          (1ll << 26) - 3, (1ll << 31) - 1025, (1ll << 31) - 1024, (1ll << 31) - 1, 1ll << 31, 1ll << 32,
                          1ll << 62, INT64_MAX};
  // every argument in turn at the ends of its type, with no buffers: refused,
  // or nothing to do
  int refused = 0;
  auto no = [&](int status) {
    refused += status != BL_OK;
    return status == BL_EINVAL || status == BL_ESHAPE || status == BL_EWORKSPACE || status == BL_OK;
  };
  for (int64_t x : ends)
    for (int at = 0; at < 9; ++at) {
      int64_t n[9] = {2, 100, 200, 4, 2, 128, 512, 256, 256};  // batch, rows, keys, hq, hkv, d, strides
      n[at] = x;
      bitlinear_qk_rope_bwd_workspace_bytes(n[5]);
      bitlinear_attn_fwd_workspace_bytes(n[0], n[1], n[2], n[3], n[4], n[5]);
      bitlinear_attn_bwd_workspace_bytes(n[0], n[1], n[2], n[3], n[4], n[5]);
      bitlinear_attn_cache_workspace_bytes(n[0], n[1], n[3], n[4], n[5]);
      CHECK(no(bitlinear_rope_table(n[1], n[5], 1e4, nullptr, nullptr)));
      CHECK(no(bitlinear_qk_rope(nullptr, B, B, BL_TYPE_BF16, n[6], n[7], n[8], n[1], n[3], n[4], n[5], F, F, 1e-6f, F, n[2],
                                 I, nullptr, n[1], B, B, B, nullptr)));
      CHECK(no(bitlinear_qk_rope_bwd(nullptr, B, BL_TYPE_F32, n[6], n[7], n[1], n[3], n[4], n[5], F, F, 1e-6f, F, n[2], I, B, B,
                                     B, B, nullptr, F, A, 1 << 30, nullptr)));
      CHECK(no(bitlinear_attn_fwd(B, B, B, n[6], n[7], n[8], I, I, n[0], n[1], n[2], n[3], n[4], n[5], 0.1f, nullptr, F, A,
                                  (size_t)1 << 40, nullptr)));
      CHECK(no(bitlinear_attn_bwd(B, B, B, n[6], n[7], n[8], B, F, B, BL_TYPE_BF16, I, I, n[0], n[1], n[2], n[3], n[4], n[5],
                                  0.1f, nullptr, nullptr, B, A, (size_t)1 << 40, nullptr)));
      CHECK(no(bitlinear_attn_cache(B, n[6], B, B, n[2], I, n[7], n[8], I, nullptr, n[0], n[1], n[3], n[4], n[5], 0.1f, nullptr,
                                    A, (size_t)1 << 40, nullptr)));
      CHECK(no(bitlinear_attn_cache(B, 512, B, B, n[2], I, n[1], n[6], I, nullptr, n[0], 1, n[3], n[4], n[5], 0.1f, nullptr, A,
                                    (size_t)1 << 40, nullptr)));
    }
  CHECK(refused > 900);
  // sizes over many shapes: never less for more rows of one shape
  for (int64_t d : {64, 128})
    for (int64_t hkv : {1, 2, 5})
      for (int64_t group : {1, 4, 7})
        for (int64_t rows = 1; rows < (1 << 20); rows = rows * 3 + 1) {
          CHECK(bitlinear_attn_bwd_workspace_bytes(3, rows, rows, hkv * group, hkv, d) >=
                (size_t)rows * hkv * group * (8 + 2 * d));
          bitlinear_attn_fwd_workspace_bytes(3, rows / 9 + 1, rows, hkv * group, hkv, d);
        }
  for (int64_t draft = 1; draft <= 64; ++draft) CHECK(bitlinear_attn_cache_workspace_bytes(7, draft, 20, 5, 128) > 0);
  std::puts("attention host code ran clean");
  return 0;
}
