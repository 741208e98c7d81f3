// glu_gate.h -- the gated feed-forward's activations and the gating part of its
// backward: device pieces of the forward's kernels and of the backward's
// preparation.
#pragma once

#include "ckpt.h"
#include "common.h"
#include "glu.h"

namespace bl {

// ---------------------------------------------------------------- the gating
// exp(-g) is v_exp_f32 (1 ulp) of RN(-g log2 e), whose rounding and constant cost it
// 1.5 |g| 2^-24 of its value; v_rcp_f32 adds 1 ulp, so for g > 0 the sigmoid is good to
// some 2 ulp and for g < 0 to (1.5 |g| + 7) 2^-24.  Where 1 + exp(-g) passes 2^126 it is 0 in
// place of less than 2^-126.  (With a correctly rounded division 6001 tokens, 2048 x
// 11008 took 226 us, now 216.)
__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.f + __expf(-g)); }
// max(g, 0) that keeps a NaN: where a scale or a checkpoint's block is NaN, the outputs show it
__device__ __forceinline__ float relu(float g) { return g <= 0.f ? 0.f : g; }
template <int kAct>
__device__ __forceinline__ float act_value(float g) {
  if constexpr (kAct == kActRelu2) {
    const float r = relu(g);
    return r * r;
  } else {
    return g * sigmoid(g);
  }
}
// act(g) and its derivative
template <int kAct>
__device__ __forceinline__ void act_both(float g, float& value, float& slope) {
  if constexpr (kAct == kActRelu2) {
    const float r = relu(g);
    value = r * r;
    slope = 2.f * r;
  } else {
    const float z = sigmoid(g);
    value = g * z;
    slope = z * fmaf(g, 1.f - z, 1.f);
  }
}

// ------------------------------------------------------- backward, the gating
// dU = dh act(g) and dG = dh u act'(g) of a 64 x 64 tile (tokens x columns) in
// binary32, and from them the four bf16 operands of the products, each rounded
// once: dG gate_gamma and dU up_gamma by rows (for dX), dG s_t and dU s_t
// transposed through LDS (for the weights' gradients, whose contraction runs over
// tokens; tokens past the last give zeros).  bf16 is what the matrix instructions
// take, whatever the types of dH and the gradients: 2.3e-3 of the exact gradients where
// results rounded once to bf16 have 1.7e-3.  A second part for each (codes and x_q are
// exact) would take twice the products.
constexpr int kGatePitch = 66;  // LDS pitch (bf16) of a transposed tile

// 16 consecutive values of a row
template <int T>
__device__ __forceinline__ void load_run16(const void* p, int64_t e, float scale, float* x) {
  Raw8<T> a, b;
  a.load(p, e);
  b.load(p, e + 8);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = a.get(i, scale);
    x[8 + i] = b.get(i, scale);
  }
}

// by 256 threads; tg, tu: 64 rows of kGatePitch each
template <int kSave, int kAct>
__device__ __forceinline__ void glu_gate_tile(const GluBwdArgs& a, const GluBwdLayout& l, int job, int tid, uint16_t* tg,
                                              uint16_t* tu) {
  const int64_t tp = bwd_tokens_padded(a.tokens), bx = tp / 64;
  const int64_t t0 = 64 * (job % bx), c0 = 64 * (job / bx);
  {
    const int t = tid >> 2, c16 = 16 * (tid & 3);
    const int64_t token = t0 + t, col = c0 + c16;
    float dg[16], du[16], s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) dg[i] = du[i] = 0.f;
    if (token < a.tokens) {
      const int64_t e = token * a.n_out + col;
      float dh[16], g[16], u[16], gs = 0.f, us = 0.f;
      if (a.dh_type == kRowF32) load_run16<kRowF32>(a.dH, e, 0.f, dh);
      else load_run16<kRowBf16>(a.dH, e, 0.f, dh);
      if (kSave == kRowQ8) {
        gs = ld_global(a.Gs + e / kCkptBlock);
        us = ld_global(a.Us + e / kCkptBlock);
      }
      load_run16<kSave>(a.G, e, gs, g);
      load_run16<kSave>(a.U, e, us, u);
      s = ld_global(a.x_scale + token);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float value, slope;
        act_both<kAct>(g[i], value, slope);
        du[i] = dh[i] * value;
        dg[i] = dh[i] * u[i] * slope;
      }
      if (a.dX) {
        const float gg = (float)ld_global(a.gate_gamma), gu = (float)ld_global(a.up_gamma);
        float y[16], z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          y[i] = dg[i] * gg;
          z[i] = du[i] * gu;
        }
        uint16_t* dgu = reinterpret_cast<uint16_t*>(a.ws + l.dgu);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          store_row8(dgu, kRowBf16, tiled_at(token, col + 8 * h, 2 * a.n_out), y + 8 * h);
          store_row8(dgu, kRowBf16, tiled_at(token, a.n_out + col + 8 * h, 2 * a.n_out), z + 8 * h);
        }
      }
    }
    if (!a.dWg) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      tg[t * kGatePitch + c16 + i] = one_bf16(dg[i] * s);
      tu[t * kGatePitch + c16 + i] = one_bf16(du[i] * s);
    }
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int q = (tid + 256 * p) & 511, r = q >> 3, t8 = 8 * (q & 7);
    const uint16_t* tile = p < 2 ? tg : tu;
    uint16_t* out = reinterpret_cast<uint16_t*>(a.ws + (p < 2 ? l.dgs_t : l.dus_t));
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = (uint32_t)tile[(t8 + 2 * e) * kGatePitch + r] | ((uint32_t)tile[(t8 + 2 * e + 1) * kGatePitch + r] << 16);
    st_global(reinterpret_cast<u32x4*>(out + tiled_at(c0 + r, t0 + t8, tp)), u32x4{o[0], o[1], o[2], o[3]});
  }
}

}  // namespace bl
