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
size_t glu_ws_bytes(int64_t tokens, int64_t k, int64_t n_out, bool q8);  // q8: G and U are kept in 8 bits

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

// Workspace of the backward: bf16 operands of its three products, in tiles
// (tiled_at; each region 256-byte aligned), and the planes of products that are
// split along their depth.
//   dgu    [tp][2 n_out]: dG gate_gamma, then dU up_gamma; tp = tokens rounded up to 64
//   dgs_t, dus_t  [n_out][tp]: (dG s_t)^T, (dU s_t)^T
//   xq_t   [k][tp];  codes_t  [k][2 n_out]: both layers' codes, transposed
struct GluBwdLayout {
  size_t dgu, dgs_t, dus_t, xq_t, codes_t, planes_x, planes_g, planes_u, bytes;
  int split_x, split_w;  // parts of dX's depth, of each weight gradient's
  bool narrow;           // tiles of 256 x 128, else 256 x 256
};
// All products run in one launch of 256 x 256 tiles, one on a CU.  A product is cut
// along its depth where it is deeper than a CU's share of all the work, but no
// part shallower than kGluPart: a part costs a binary32 plane of the output to
// write and to read.  Where one round of such tiles does not fill the CUs, dX, the
// deepest, is cut into as many parts as do, and the launch takes twice as many tiles of
// 256 x 128, two on a CU (547 tokens, 896 x 4864, binary32 gradients: 42.7 us in place of
// 46.9; 32 tokens: 30.9 and 32.7).  Up to 256 tokens, where the weight gradients' tiles are
// little more than their stores, it takes those too (32 tokens, 1536 x 8960: 58 us in place of
// 66, 256 tokens: 64 and 75; 300: 73 and 74; 4096 tokens, 2560 x 6912: 560 in place of 477).
constexpr int64_t kGluPart = 1024;
inline int glu_parts(int64_t depth, int64_t share, int most) {
  const int64_t per = share > kGluPart ? share : kGluPart, parts = (depth + per - 1) / per;
  return parts > most ? most : (int)parts;
}
inline GluBwdLayout glu_bwd_layout(int64_t tokens, int64_t k, int64_t n_out) {
  const int64_t tp = bwd_tokens_padded(tokens);
  const int64_t cols = (k + 255) / 256, tiles_x = (tokens + 255) / 256 * cols, tiles_w = (n_out + 255) / 256 * cols;
  const int64_t share = (tiles_x * 2 * n_out + 2 * tiles_w * tp) / 256;
  GluBwdLayout l;
  l.split_x = glu_parts(2 * n_out, share, 8);
  l.split_w = glu_parts(tp, share, 4);
  const int64_t all_w = 2 * tiles_w * l.split_w;
  const bool one_round = tiles_x * l.split_x + all_w <= 256;
  if (one_round && tiles_x > 0) {
    const int64_t room = (256 - all_w) / tiles_x, most = 2 * n_out / 512, parts = room < most ? room : most;
    l.split_x = (int)(parts > 32 ? 32 : parts > l.split_x ? parts : l.split_x);
  }
  l.narrow = one_round || tp <= 256;
  l.dgu = 0;
  l.dgs_t = l.dgu + bwd_align((size_t)tp * 2 * n_out * 2);
  l.dus_t = l.dgs_t + bwd_align((size_t)n_out * tp * 2);
  l.xq_t = l.dus_t + bwd_align((size_t)n_out * tp * 2);
  l.codes_t = l.xq_t + bwd_align((size_t)k * tp * 2);
  l.planes_x = l.codes_t + bwd_align((size_t)k * 2 * n_out * 2);
  l.planes_g = l.planes_x + (l.split_x > 1 ? bwd_align((size_t)l.split_x * tokens * k * 4) : 0);
  const size_t w = l.split_w > 1 ? bwd_align((size_t)l.split_w * n_out * k * 4) : 0;
  l.planes_u = l.planes_g + w;
  l.bytes = l.planes_u + w;
  return l;
}
hipError_t launch_glu_bwd(const GluBwdArgs& a, int S, hipStream_t s);
hipError_t launch_zero(float* p, int64_t n, hipStream_t s);

}  // namespace bl
