// Drives the host code of the feed-forward side's entry points -- argument
// validation and workspace sizes, with sizes at the ends of their types --
// under AddressSanitizer and UndefinedBehaviorSanitizer (host code only; no
// call here reaches a launch).  Built and run by tests/test_ffn_sanitizers.py.
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
  int8_t* Q = (int8_t*)A;
  float* F = (float*)A;
  double* D = (double*)A;
  const int64_t ends[] = {INT64_MIN, -(1ll << 32), -1, 0, 1, 2, 8, 16, 63, 64, 65, 128, 4096, 4097, 16384, (1ll << 22) - 128,
                          1ll << 22, (1ll << 23) - 1, 1ll << 23, (1ll << 29) - 32, (1ll << 31) - 128, (1ll << 31) - 1,
                          1ll << 31, 1ll << 32, 1ll << 62, INT64_MAX};
  // every size in turn, and every pair, at the ends of its type, with the last
  // buffer missing: refused, or nothing to do
  int refused = 0;
  auto no = [&](int status) {
    refused += status != BL_OK;
    return status == BL_EINVAL || status == BL_ESHAPE || status == BL_EWORKSPACE || status == BL_OK;
  };
  for (int64_t x : ends)
    for (int64_t y : ends)
      for (int at = 0; at < 3; ++at) {
        int64_t n[3] = {100, 256, 128};  // rows or tokens, width or k, n_out or stride
        n[at] = x;
        n[(at + 1) % 3] = y;
        for (int type : {BL_TYPE_F32, BL_TYPE_BF16}) {
          CHECK(no(bitlinear_ckpt_pack(A, type, n[2], n[0], n[1], Q, nullptr, nullptr)));
          CHECK(no(bitlinear_ckpt_unpack(Q, F, n[0], n[1], nullptr, type, nullptr)));
          CHECK(no(bitlinear_layernorm(A, type, n[2], n[0], n[1], F, F, 1e-6f, 1, nullptr, type, F, F, Q, F, nullptr)));
          CHECK(no(bitlinear_layernorm_bwd(A, type, nullptr, n[2], n[0], n[1], F, F, F, A, type, A, nullptr, type, nullptr,
                                           nullptr, A, (size_t)1 << 40, nullptr)));
        }
        CHECK(no(bitlinear_layernorm_bwd(Q, BL_TYPE_Q8, F, n[1], n[0], n[1], F, F, F, A, BL_TYPE_F32, A, nullptr, BL_TYPE_F32,
                                         nullptr, nullptr, A, (size_t)1 << 40, nullptr)));
        bitlinear_layernorm_bwd_workspace_bytes(n[1]);
        const size_t f = bitlinear_glu_workspace_bytes(n[0], n[1], n[2]), b = bitlinear_glu_bwd_workspace_bytes(n[0], n[1], n[2]);
        CHECK(f < (size_t)1 << 36 && b < (size_t)1 << 40);
        CHECK(no(bitlinear_glu(Q, F, n[0], n[1], A, D, A, D, n[2], 6, 8, BL_ACT_SILU, nullptr, BL_TYPE_Q8, Q, F, Q, F, A,
                               (size_t)1 << 40, nullptr)));
        if (n[0] != 0)  // (without tokens the gradients are cleared)
          CHECK(no(bitlinear_glu_bwd(nullptr, BL_TYPE_F32, BL_TYPE_Q8, Q, F, Q, F, Q, F, A, D, A, D, n[0], n[1], n[2], 6, 8,
                                     BL_ACT_RELU2, BL_TYPE_BF16, B, B, B, A, (size_t)1 << 40, nullptr)));
      }
  CHECK(refused > 10000);
  // the backward's workspace over many shapes: never less than its operands, and any
  // number of parts fits it
  for (int64_t k : {128, 896, 2560, 8960})
    for (int64_t n_out : {128, 4864, 6912, 11008})
      for (int64_t tokens = 1; tokens < 20000; tokens = tokens * 3 / 2 + 1) {
        const size_t ws = bitlinear_glu_bwd_workspace_bytes(tokens, k, n_out);
        CHECK(ws >= (size_t)(4 * tokens * n_out * 2 + 2 * tokens * k + 4 * n_out * k));
        CHECK(ws <= (size_t)(10 * (tokens + 64) * n_out + 2 * (tokens + 64) * k + 4 * n_out * k) +
                        (size_t)(4 * 32 * tokens * k + 2 * 4 * 4 * n_out * k + 4096));
      }
  std::puts("feed-forward host code ran clean");
  return 0;
}
