// glu.hip -- the gated feed-forward's first half in one kernel (two ternary x
// int8 projections, the activation and the product) and the gating part of its
// backward.
#include "ckpt.h"
#include "common.h"
#include "glu.h"
#include "launch.h"

namespace bl {

// ---------------------------------------------------------------- the gating
template <int kAct>
__device__ __forceinline__ float act_value(float g) {
  if constexpr (kAct == kActRelu2) {
    const float r = g > 0.f ? g : 0.f;
    return r * r;
  } else {
    return g / (1.f + __expf(-g));  // an infinite exp gives -0, the limit
  }
}
// act(g) and its derivative
template <int kAct>
__device__ __forceinline__ void act_both(float g, float& value, float& slope) {
  if constexpr (kAct == kActRelu2) {
    const float r = g > 0.f ? g : 0.f;
    value = r * r;
    slope = 2.f * r;
  } else {
    const float z = 1.f / (1.f + __expf(-g));
    value = g * z;
    slope = z * fmaf(g, 1.f - z, 1.f);
  }
}

// ------------------------------------------------------- forward, few tokens
// A workgroup computes 64 outputs (one packed strip of each layer) of 16 kTT
// tokens: eight wavefronts take the gate strip's k blocks and eight the up
// strip's, each every eighth.  A lane's chunk of a superblock holds the A
// operands it needs (rows along the matrix instruction's rows), the activations
// are the B operands; the sixteen partial sums meet in LDS over the code tables,
// where each thread then owns one output: a wavefront holds one token's 64
// outputs, which is one checkpoint block.
constexpr int kSmallCopies = 32;  // code table copies: lane l reads copy l % 32
constexpr int kSmallPitch = 68;   // int32 of a token's 64 sums, padded
constexpr uint32_t kGluOOB = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t glu_rsrc(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

template <int S>
__device__ __forceinline__ void load_chunk_at(__amdgpu_buffer_rsrc_t r, uint32_t o, uint32_t* w) {
  constexpr int kW = block_bytes(S) / 4;
  const u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0);
  w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  if constexpr (kW == 8) {
    const u32x4 b = __builtin_amdgcn_raw_buffer_load_b128(r, o + 16, 0, 0);
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  } else if constexpr (kW == 7) {
    const u32x3 b = __builtin_amdgcn_raw_buffer_load_b96(r, o + 16, 0, 0);
    w[4] = b.x; w[5] = b.y; w[6] = b.z;
  } else if constexpr (kW == 6) {
    const u32x2 b = __builtin_amdgcn_raw_buffer_load_b64(r, o + 16, 0, 0);
    w[4] = b.x; w[5] = b.y;
  } else {
    static_assert(kW == 5, "chunk size");
    w[4] = __builtin_amdgcn_raw_buffer_load_b32(r, o + 16, 0, 0);
  }
}
// A operand of matrix instruction m = 2i + h (row tile i, k half h): the codes
// of fields 2m and 2m + 1 of the chunk
template <int S>
__device__ __forceinline__ v4i chunk_operand(const uint32_t* w, int m, const uint32_t* lut_lane) {
  constexpr int kW = block_bytes(S) / 4, kField = 8 + S;
  v4i a;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int off = (2 * m + q) * kField, offh = off + S;
    const uint32_t lo_next = (off >> 5) + 1 < kW ? w[(off >> 5) + 1] : 0u;
    const uint32_t hi_next = (offh >> 5) + 1 < kW ? w[(offh >> 5) + 1] : 0u;
    const uint32_t klo = funnel(lo_next, w[off >> 5], off & 31) & 0xffu;
    const uint32_t khi = funnel(hi_next, w[offh >> 5], offh & 31) & 0xffu;
    a[2 * q] = (int)lut_lane[(klo * 2 + 0) * kSmallCopies];
    a[2 * q + 1] = (int)lut_lane[(khi * 2 + 1) * kSmallCopies];
  }
  return a;
}
__device__ __forceinline__ v4i mfma_i8(v4i a, v4i b, v4i c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ v4i load_b128(__amdgpu_buffer_rsrc_t r, uint32_t o) {
  return (v4i)__builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0);
}

// one output: h, and g and u where they are kept; the 64 lanes of a wavefront
// hold one token's values of one block
template <int kAct>
__device__ __forceinline__ void glu_output(const GluArgs& a, float g, float u, int64_t token, int64_t col, int lane) {
  const int64_t e = token * a.n_out + col;
  st_global(a.H + e, f32_to_bf16_rne(act_value<kAct>(g) * u));
  if (a.save == kSaveNone) return;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const float x = s ? u : g;
    void* out = s ? a.U : a.G;
    if (a.save == kRowF32) {
      st_global(static_cast<float*>(out) + e, x);
    } else if (a.save == kRowBf16) {
      st_global(static_cast<uint16_t*>(out) + e, f32_to_bf16_rne(x));
    } else {
      uint32_t top = abs_bits(x);
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) top = max_u(top, (uint32_t)__shfl_xor((int)top, o, 64));
      const CkptScale c = ckpt_scale(top);
      st_global(static_cast<int8_t*>(out) + e, (int8_t)ckpt_code(x, c.inv));
      if (lane == 0) st_global((s ? a.Us : a.Gs) + e / kCkptBlock, c.scale);
    }
  }
}

template <int S, int kAct, int kTT>
__global__ __launch_bounds__(1024) void glu_small_kernel(GluArgs a) {
  __shared__ __attribute__((aligned(16))) int lds[16 * 16 * kSmallPitch];
  static_assert(16 * 16 * kSmallPitch >= 512 * kSmallCopies, "the tables fit where the sums meet");
  uint32_t* lut = reinterpret_cast<uint32_t*>(lds);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int side = wave >> 3, first = wave & 7;  // gate or up; first k block
  const int64_t strip = blockIdx.x, t0 = (int64_t)blockIdx.y * (16 * kTT);
  const int nkb = (int)(a.k / kBlockK);
#pragma unroll
  for (int r = 0; r < 512 * kSmallCopies / 4 / 1024; ++r) {
    const uint32_t v = ld_global(&kHalfCodeTable.v[(tid + 1024 * r) / (kSmallCopies / 4)]);
    reinterpret_cast<u32x4*>(lut)[tid + 1024 * r] = u32x4{v, v, v, v};
  }
  const uint32_t* lut_lane = lut + (lane & (kSmallCopies - 1));
  constexpr int kSb = kStripRows * block_bytes(S);  // bytes of a superblock
  const char* base = static_cast<const char*>(side ? a.up : a.gate) + strip * nkb * (int64_t)kSb;
  const __amdgpu_buffer_rsrc_t pr = glu_rsrc(base, (int64_t)nkb * kSb), xr = glu_rsrc(a.xq, a.tokens * a.k);
  uint32_t xo[kTT];
#pragma unroll
  for (int j = 0; j < kTT; ++j) {
    const int64_t t = t0 + 16 * j + (lane & 15);
    xo[j] = t < a.tokens ? (uint32_t)(t * a.k + 16 * (lane >> 4)) : kGluOOB;
  }
  v4i c[kTT][4];
#pragma unroll
  for (int j = 0; j < kTT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) c[j][i] = v4i{0, 0, 0, 0};
  __syncthreads();
  for (int kb = first; kb < nkb; kb += 8) {
    uint32_t w[block_bytes(S) / 4];
    load_chunk_at<S>(pr, (uint32_t)(kb * kSb + lane * block_bytes(S)), w);
    v4i b[kTT][2];
#pragma unroll
    for (int j = 0; j < kTT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        b[j][h] = load_b128(xr, xo[j] == kGluOOB ? kGluOOB : xo[j] + (uint32_t)(kb * kBlockK + 64 * h));
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v4i op = chunk_operand<S>(w, 2 * i + h, lut_lane);
#pragma unroll
        for (int j = 0; j < kTT; ++j) c[j][i] = mfma_i8(op, b[j][h], c[j][i]);
      }
  }
  const double gg = ld_global(a.gate_gamma), gu = ld_global(a.up_gamma);
#pragma unroll
  for (int j = 0; j < kTT; ++j) {
    __syncthreads();  // tables, or the sums of the tile before, are read
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<v4i*>(&lds[(wave * 16 + (lane & 15)) * kSmallPitch + 16 * i + 4 * (lane >> 4)]) = c[j][i];
    __syncthreads();
    const int64_t token = t0 + 16 * j + wave;
    int sums[2] = {0, 0};
#pragma unroll
    for (int z = 0; z < 16; ++z) sums[z >> 3] += lds[(z * 16 + wave) * kSmallPitch + lane];
    if (token < a.tokens) {
      const float s = ld_global(a.x_scale + token);
      glu_output<kAct>(a, out_value(sums[0], out_scale(gg, s)), out_value(sums[1], out_scale(gu, s)), token,
                       strip * kStripRows + lane, lane);
    }
  }
}

// ------------------------------------------------------- backward, the gating
// dU = dh act(g) and dG = dh u act'(g) of a 64 x 64 tile (tokens x columns) in
// binary32, and from them the four bf16 operands of the products, each rounded
// once: dG gate_gamma and dU up_gamma by rows (for dX), dG s_t and dU s_t
// transposed through LDS (for the weights' gradients, whose contraction runs over
// tokens; tokens past the last give zeros).
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

template <int kSave, int kAct>
__global__ __launch_bounds__(256) void glu_gate_bwd_kernel(GluBwdArgs a, GluBwdLayout l) {
  __shared__ uint16_t tg[64 * kGatePitch], tu[64 * kGatePitch];
  const int tid = threadIdx.x;
  const int64_t tp = bwd_tokens_padded(a.tokens), bx = tp / 64;
  const int64_t t0 = 64 * (blockIdx.x % bx), c0 = 64 * (blockIdx.x / bx);
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
        uint16_t* row = reinterpret_cast<uint16_t*>(a.ws + l.dgu) + token * 2 * a.n_out + col;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          store_row8(row, kRowBf16, 8 * h, y + 8 * h);
          store_row8(row, kRowBf16, a.n_out + 8 * h, z + 8 * h);
        }
      }
    }
    if (!a.dWg) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      tg[t * kGatePitch + c16 + i] = f32_to_bf16_rne(dg[i] * s);
      tu[t * kGatePitch + c16 + i] = f32_to_bf16_rne(du[i] * s);
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
    st_global(reinterpret_cast<u32x4*>(out + (c0 + r) * tp + t0 + t8), u32x4{o[0], o[1], o[2], o[3]});
  }
}

// ------------------------------------------------------------------ host
size_t glu_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

template <int S, int kAct>
static hipError_t glu_launch(const GluArgs& a, hipStream_t s) {
  const unsigned strips = (unsigned)(a.n_out / kStripRows);
  const int tiles = a.tokens <= 16 ? 1 : a.tokens <= 32 ? 2 : 4;
  const dim3 grid(strips, (unsigned)((a.tokens + 16 * tiles - 1) / (16 * tiles)));
  if (tiles == 1) glu_small_kernel<S, kAct, 1><<<grid, 1024, 0, s>>>(a);
  else if (tiles == 2) glu_small_kernel<S, kAct, 2><<<grid, 1024, 0, s>>>(a);
  else glu_small_kernel<S, kAct, 4><<<grid, 1024, 0, s>>>(a);
  return hipGetLastError();
}
template <int S>
static hipError_t glu_launch_s(const GluArgs& a, hipStream_t s) {
  return a.act == kActRelu2 ? glu_launch<S, kActRelu2>(a, s) : glu_launch<S, kActSilu>(a, s);
}
hipError_t launch_glu(const GluArgs& a, int S, void*, hipStream_t s) {
  if (S == 8) return glu_launch_s<8>(a, s);
  if (S == 6) return glu_launch_s<6>(a, s);
  if (S == 2) return glu_launch_s<2>(a, s);
  return glu_launch_s<4>(a, s);
}

template <int kSave>
static hipError_t gate_bwd_launch(const GluBwdArgs& a, const GluBwdLayout& l, hipStream_t s) {
  const unsigned grid = (unsigned)(bwd_tokens_padded(a.tokens) / 64 * (a.n_out / 64));
  if (a.act == kActRelu2) glu_gate_bwd_kernel<kSave, kActRelu2><<<grid, 256, 0, s>>>(a, l);
  else glu_gate_bwd_kernel<kSave, kActSilu><<<grid, 256, 0, s>>>(a, l);
  return hipGetLastError();
}
hipError_t launch_glu_bwd(const GluBwdArgs& a, int S, hipStream_t s) {
  const GluBwdLayout l = glu_bwd_layout(a.tokens, a.k, a.n_out);
  const hipError_t e = a.save == kRowF32 ? gate_bwd_launch<kRowF32>(a, l, s)
                     : a.save == kRowBf16 ? gate_bwd_launch<kRowBf16>(a, l, s) : gate_bwd_launch<kRowQ8>(a, l, s);
  return e != hipSuccess ? e : launch_glu_products(a, S, s);
}

}  // namespace bl
