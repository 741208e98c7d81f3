// glu.h -- the gated feed-forward's launchers (internal to the library) and
// the layout of its backward's workspace.
#pragma once

#include "launch.h"

namespace bl {

enum GluAct { kActRelu2 = 0, kActSilu = 1 };
constexpr int kSaveNone = -1;  // otherwise a RowType: what G and U are kept as

struct GluArgs {
  const int8_t* xq;
  const float* x_scale;
  int64_t tokens, k, n_out;
  const void *gate, *up;  // packed codes
  const double *gate_gamma, *up_gamma;
  int act;
  uint16_t* H;
  int save;
  void *G, *U;
  float *Gs, *Us;
};
hipError_t launch_glu(const GluArgs& a, int S, void* ws, hipStream_t s);
size_t glu_ws_bytes(int64_t tokens, int64_t k, int64_t n_out);

struct GluBwdArgs {
  const void* dH;
  int dh_type, save, act;
  const void *G, *U;
  const float *Gs, *Us;
  const int8_t* xq;
  const float* x_scale;
  const void *gate, *up;
  const double *gate_gamma, *up_gamma;
  int64_t tokens, k, n_out;
  int grad_type;
  void *dX, *dWg, *dWu;
  char* ws;
};

// Workspace of the backward: bf16 operands of its three products (each region
// 256-byte aligned) and the planes of products that are split along k.
//   dgu    [tokens][2 n_out]: dG gate_gamma beside dU up_gamma
//   dgs_t, dus_t  [n_out][tp]: (dG s_t)^T, (dU s_t)^T, tp = tokens rounded up to 64
//   xq_t   [k][tp];  codes_t  [k][2 n_out]: both layers' codes, transposed
// The operands of a product that is not split lie in tiles (rows rounded up to 16).
struct GluBwdLayout {
  size_t dgu, dgs_t, dus_t, xq_t, codes_t, partials, bytes;
  bool dx_tiled, dw_tiled;
};
inline GluBwdLayout glu_bwd_layout(int64_t tokens, int64_t k, int64_t n_out) {
  const int64_t tp = bwd_tokens_padded(tokens);
  GluBwdLayout l;
  l.dgu = 0;
  l.dgs_t = l.dgu + bwd_align((size_t)tp * 2 * n_out * 2);
  l.dus_t = l.dgs_t + bwd_align((size_t)n_out * tp * 2);
  l.xq_t = l.dus_t + bwd_align((size_t)n_out * tp * 2);
  l.codes_t = l.xq_t + bwd_align((size_t)k * tp * 2);
  l.partials = l.codes_t + bwd_align((size_t)k * 2 * n_out * 2);
  const int sx = bwd_splits(tokens, k, 2 * n_out), sw = bwd_splits(n_out, k, tp);
  l.dx_tiled = sx == 1;
  l.dw_tiled = sw == 1;
  const size_t px = sx > 1 ? (size_t)sx * tokens * k * 4 : 0, pw = sw > 1 ? (size_t)sw * n_out * k * 4 : 0;
  l.bytes = l.partials + bwd_align(px > pw ? px : pw);
  return l;
}
hipError_t launch_glu_bwd(const GluBwdArgs& a, int S, hipStream_t s);
// the rest of the backward once dgu, dgs_t and dus_t are written: the other
// operands, then the products
hipError_t launch_glu_products(const GluBwdArgs& a, int S, hipStream_t s);
hipError_t launch_zero(float* p, int64_t n, hipStream_t s);

}  // namespace bl
