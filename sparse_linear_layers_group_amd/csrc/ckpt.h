// ckpt.h -- 8-bit checkpoints of activations, and rows of the types they
// come in: device pieces that the norm, gating and checkpoint kernels share.
#pragma once

#include "common.h"
#include "launch.h"

namespace bl {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

// A block is kCkptBlock consecutive values of a row (the last of a row may
// be shorter).  With a = max |x| of the block, in binary32:
//   code = the integer nearest to x inv (ties to even), inv = RN(127 / a),
//   scale = RN(a / 127),  and a value comes back as RN(code scale).
// The fused multiply-add below rounds the exact product x inv once, to an
// integer: 1.5 * 2^23 is added, where binary32 holds integers only, and the
// code is the low byte of the result.  |x inv| <= 127 (1 + 2^-24), so codes
// stay in -127..127.  Eight bits keep a value within half a step, 1/254 of its
// block's largest: of a block of normal values some 0.6% of their size, a
// fifth of what an 8-bit floating-point format with 3 fraction bits loses.
// Blocks below 2^-100 come back as zeros (127 / a would leave binary32); one
// with an infinity or a NaN comes back as NaN, so it shows.
struct CkptScale {
  float inv, scale;
};
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }
// `top`: the largest abs_bits of the block (as integers, so that a NaN wins)
__device__ __forceinline__ CkptScale ckpt_scale(uint32_t top) {
  const float a = __uint_as_float(top);
  if (top >= 0x7f800000u) return CkptScale{0.f, __builtin_nanf("")};
  if (a < 0x1p-100f) return CkptScale{0.f, 0.f};
  return CkptScale{127.f / a, a / 127.f};
}
__device__ __forceinline__ uint32_t ckpt_code(float x, float inv) {
  return __float_as_uint(fmaf(x, inv, 0x1.8p23f)) & 0xffu;
}
__device__ __forceinline__ float ckpt_value(uint32_t word, int byte, float scale) {
  return (float)(int8_t)(word >> (8 * byte)) * scale;
}

// the two bf16 nearest to a and b (ties to even)
__device__ __forceinline__ uint32_t pair_bf16(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}
// one of them (a NaN stays one, whatever its bits)
__device__ __forceinline__ uint16_t one_bf16(float a) { return (uint16_t)pair_bf16(a, a); }

// Eight consecutive values of a row as they lie in memory
enum RowType { kRowF32 = 0, kRowBf16 = 1, kRowQ8 = 2 };
template <int T>
struct Raw8;
template <>
struct Raw8<kRowF32> {
  f32x4_t a, b;
  __device__ __forceinline__ void load(const void* p, int64_t e) {
    const f32x4_t* q = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + e);
    a = ld_global(q);
    b = ld_global(q + 1);
  }
  __device__ __forceinline__ void zero() { a = b = f32x4_t{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ float get(int i, float) const { return i < 4 ? a[i & 3] : b[i & 3]; }
};
template <>
struct Raw8<kRowBf16> {
  u32x4 a;
  __device__ __forceinline__ void load(const void* p, int64_t e) {
    a = ld_global(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + e));
  }
  __device__ __forceinline__ void zero() { a = u32x4{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ float get(int i, float) const {
    return (i & 1) ? bf16_hi(a[(i >> 1) & 3]) : bf16_lo(a[(i >> 1) & 3]);
  }
};
template <>
struct Raw8<kRowQ8> {
  u32x2 a;
  __device__ __forceinline__ void load(const void* p, int64_t e) {
    a = ld_global(reinterpret_cast<const u32x2*>(static_cast<const int8_t*>(p) + e));
  }
  __device__ __forceinline__ void zero() { a = u32x2{0u, 0u}; }
  __device__ __forceinline__ float get(int i, float scale) const { return ckpt_value(a[i >> 2], i & 3, scale); }
};

// eight values as binary32 or (rounded once) bf16
__device__ __forceinline__ void store_row8(void* p, int type, int64_t e, const float* y) {
  if (type == kRowF32) {
    f32x4_t* q = reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + e);
    st_global(q, f32x4_t{y[0], y[1], y[2], y[3]});
    st_global(q + 1, f32x4_t{y[4], y[5], y[6], y[7]});
  } else {
    st_global(reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + e),
              u32x4{pair_bf16(y[0], y[1]), pair_bf16(y[2], y[3]), pair_bf16(y[4], y[5]), pair_bf16(y[6], y[7])});
  }
}

// The codes of eight values of a block that eight neighbouring lanes hold
// (lane % 8 = place in the block); the block's first lane stores its scale.
// All 64 lanes call it; `in`: this lane's values are part of the row.
__device__ __forceinline__ void ckpt_store8(const float* x, bool in, int lane, int8_t* codes, float* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_u(top, abs_bits(x[i]));
  if (!in) top = 0;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max_u(top, (uint32_t)__shfl_xor((int)top, o, 64));
  const CkptScale c = ckpt_scale(top);
  if (!in) return;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i >> 2] |= ckpt_code(x[i], c.inv) << (8 * (i & 3));
  st_global(reinterpret_cast<u32x2*>(codes), u32x2{w[0], w[1]});
  if ((lane & 7) == 0) st_global(scale, c.scale);
}

}  // namespace bl
