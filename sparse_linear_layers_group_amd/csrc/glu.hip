// glu.hip -- the gated feed-forward's first half: two ternary x int8 projections
// with the activation and the product in their epilogue, in one kernel up to some
// hundred tokens, behind a launch that decodes the codes once for many.
#include "ckpt.h"
#include "common.h"
#include "glu.h"
#include "glu_gate.h"
#include "launch.h"

#include <type_traits>

namespace bl {

// ------------------------------------------------------- forward, few tokens
// A workgroup computes 64 outputs (one packed strip of each layer) of 16
// tokens: eight wavefronts take the gate strip's k blocks and eight the up
// strip's, each every eighth.  A lane's chunk of a superblock holds the A
// operands it needs (rows along the matrix instruction's rows), the activations
// are the B operands; the sixteen partial sums meet in LDS over the code tables,
// where each thread then owns one output: a wavefront holds one token's 64
// outputs, which is one checkpoint block.
// Bound by latency (launch, tables, one chunk's loads after another, the join): one
// token, 896 x 4864 6:8, 4.1 us; 16 tokens, 2560 x 6912, 6.0 us for 8 MB.
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
  st_global(a.H + e, one_bf16(act_value<kAct>(g) * u));
  if (a.save == kSaveNone) return;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const float x = s ? u : g;
    void* out = s ? a.U : a.G;
    if (a.save == kRowF32) {
      st_global(static_cast<float*>(out) + e, x);
    } else if (a.save == kRowBf16) {
      st_global(static_cast<uint16_t*>(out) + e, one_bf16(x));
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

template <int S, int kAct>
__global__ __launch_bounds__(1024) void glu_small_kernel(GluArgs a) {
  __shared__ __attribute__((aligned(16))) int lds[16 * 16 * kSmallPitch];
  static_assert(16 * 16 * kSmallPitch >= 512 * kSmallCopies, "the tables fit where the sums meet");
  uint32_t* lut = reinterpret_cast<uint32_t*>(lds);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int side = wave >> 3, first = wave & 7;  // gate or up; first k block
  const int64_t strip = blockIdx.x, t0 = 16 * (int64_t)blockIdx.y;
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
  const int64_t t = t0 + (lane & 15);
  const uint32_t xo = t < a.tokens ? (uint32_t)(t * a.k + 16 * (lane >> 4)) : kGluOOB;
  v4i c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = v4i{0, 0, 0, 0};
  __syncthreads();
  for (int kb = first; kb < nkb; kb += 8) {
    uint32_t w[block_bytes(S) / 4];
    load_chunk_at<S>(pr, (uint32_t)(kb * kSb + lane * block_bytes(S)), w);
    v4i b[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) b[h] = load_b128(xr, xo == kGluOOB ? kGluOOB : xo + (uint32_t)(kb * kBlockK + 64 * h));
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) c[i] = mfma_i8(chunk_operand<S>(w, 2 * i + h, lut_lane), b[h], c[i]);
  }
  const double gg = ld_global(a.gate_gamma), gu = ld_global(a.up_gamma);
  __syncthreads();  // the tables are read
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<v4i*>(&lds[(wave * 16 + (lane & 15)) * kSmallPitch + 16 * i + 4 * (lane >> 4)]) = c[i];
  __syncthreads();
  const int64_t token = t0 + wave;
  int sums[2] = {0, 0};
#pragma unroll
  for (int z = 0; z < 16; ++z) sums[z >> 3] += lds[(z * 16 + wave) * kSmallPitch + lane];
  if (token < a.tokens) {
    const float s = ld_global(a.x_scale + token);
    glu_output<kAct>(a, out_value(sums[0], out_scale(gg, s)), out_value(sums[1], out_scale(gu, s)), token,
                     strip * kStripRows + lane, lane);
  }
}

typedef __attribute__((address_space(3))) char glu_lds_char;
typedef __attribute__((address_space(3))) void glu_lds_void;
__device__ __forceinline__ void glu_dma16(__amdgpu_buffer_rsrc_t r, glu_lds_char* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (glu_lds_void*)dst, 16, off, 0, 0, 0);
}
template <int N, bool kLds = false>
__device__ __forceinline__ void glu_wait() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | ((kLds ? 0 : 15) << 8));
}

// Workgroup barrier behind which LDS writes are seen; loads into registers stay in
// flight
__device__ __forceinline__ void glu_barrier() {
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8));  // lgkmcnt(0) only
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ------------------------------------------------------ forward, some tokens
// A workgroup computes 16 kRT outputs (of both layers) of kTokens tokens.  Each
// wavefront decodes an equal share of a k block's A operands, once for all tokens,
// into LDS, where all read them.  The activations come to LDS by DMA in whole 128-byte
// lines, eight rows an instruction (as operands, 16 rows of 64 bytes, straight from
// memory they bound the kernel: 24.4 us in place of 19.4 at 256 tokens, 2560 x 6912;
// 16.4 now).  One k block (128 k) per barrier: while its products run, the next
// block's operands are decoded, and the activations and the codes two blocks on are on
// their way.  Bound by the way from the codes through LDS to the products between two
// barriers; fragments read a block ahead, codes by DMA, or a fifth fewer operand reads
// (one row tile and two token tiles a wavefront) gave nothing, codes three blocks
// ahead cost 10 %.  Half a strip (kRT = 2) makes
// enough workgroups for the CUs; a checkpoint's block of 64 outputs needs a whole one
// (kRT = 4), whose row tiles two wavefronts share.
constexpr int kMidThreads = 512;
// place of 16-byte piece `piece` (0..7) of activation row `row` in its 128 bytes: reads
// of 16 rows' pieces as operands are free of bank conflicts (see row64_place)
__device__ __forceinline__ int row128_place(int row, int piece) { return piece ^ ((row >> 1) & 7); }
// the stages of the activations, kTokens rows of 128 bytes
__shared__ __attribute__((aligned(1024))) char g_mid64_st0[64 * 128], g_mid64_st1[64 * 128], g_mid64_st2[64 * 128];
__shared__ __attribute__((aligned(1024))) char g_mid128_st0[128 * 128], g_mid128_st1[128 * 128], g_mid128_st2[128 * 128];
__shared__ __attribute__((aligned(1024))) char g_mid256_st0[256 * 128], g_mid256_st1[256 * 128], g_mid256_st2[256 * 128];
template <int kTokens, int P>
__device__ __forceinline__ char* mid_stage() {
  static_assert(kTokens == 64 || kTokens == 128 || kTokens == 256, "the stages above");
  if constexpr (kTokens == 64) return P == 0 ? g_mid64_st0 : P == 1 ? g_mid64_st1 : g_mid64_st2;
  else if constexpr (kTokens == 128) return P == 0 ? g_mid128_st0 : P == 1 ? g_mid128_st1 : g_mid128_st2;
  else return P == 0 ? g_mid256_st0 : P == 1 ? g_mid256_st1 : g_mid256_st2;
}

template <int S, int kAct, int kRT, int kTokens>
__global__ __launch_bounds__(kMidThreads, 2) void glu_mid_kernel(GluArgs a) {
  constexpr int kOps = 4 * kRT;       // A operands of a k block: (layer, row tile, k half)
  constexpr int kShare = kOps / 8;    // of one wavefront
  constexpr int kRW = 2;              // row tiles of a wavefront's products
  constexpr int kGroups = 8 * kRW / kRT;       // wavefronts side by side along the tokens
  constexpr int kTG = kTokens / 16 / kGroups;  // token tiles of a wavefront
  // code table copies (8: two workgroups of 128 tokens fit a CU, 14.2 us in place of 17.1
  // at 128 tokens, 1536 x 8960, where there are more workgroups than CUs; 4% slower
  // where there are not)
  constexpr int kMidCopies = kTG == 1 ? 8 : 16;
  constexpr int kX = kTokens / 64;    // DMA instructions of a wavefront and block
  __shared__ __attribute__((aligned(16))) uint32_t lut[512 * kMidCopies];
  __shared__ __attribute__((aligned(16))) v4i A[2][kOps * 64];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int kPer = 4 / kRT;  // workgroups of a strip
  const int64_t strip = blockIdx.x / kPer;
  const int part = blockIdx.x % kPer;  // which kRT row tiles of it
  const int64_t t0 = (int64_t)blockIdx.y * kTokens;
  const int group = wave % kGroups, row0 = wave / kGroups * kRW;  // of the wavefront: its tokens, its first row tile
  const int nkb = (int)(a.k / kBlockK);
  constexpr int kSb = kStripRows * block_bytes(S);
  const int64_t at = strip * nkb * (int64_t)kSb;
  const __amdgpu_buffer_rsrc_t xr = glu_rsrc(a.xq, a.tokens * a.k);
  // A operand `op`: layer op / (2 kRT), row tile part kRT + op / 2 % kRT, k half op % 2.
  // Its two fields of a lane's chunk start at bit 2 m (8 + S), m = 2 (row tile) + half: at
  // most 32 bits, in two words (a word behind the chunk is never used)
  constexpr int kField = 8 + S;
  auto field_bit = [&](int op) { return 2 * (2 * (part * kRT + (op >> 1) % kRT) + (op & 1)) * kField; };
  const __amdgpu_buffer_rsrc_t pr[2] = {glu_rsrc(static_cast<const char*>(a.gate) + at, (int64_t)nkb * kSb),
                                        glu_rsrc(static_cast<const char*>(a.up) + at, (int64_t)nkb * kSb)};
  uint32_t w[2][kShare][2];  // codes: block kb's in w[kb % 2], until they are decoded
  auto load_codes = [&](int kb, uint32_t (&dst)[kShare][2]) {
#pragma unroll
    for (int s = 0; s < kShare; ++s) {
      const int op = wave * kShare + s;
      const uint32_t o = (uint32_t)(kb * kSb + lane * block_bytes(S) + (field_bit(op) >> 5) * 4);
      const __amdgpu_buffer_rsrc_t r = op >= 2 * kRT ? pr[1] : pr[0];
      dst[s][0] = __builtin_amdgcn_raw_buffer_load_b32(r, kb < nkb ? o : kGluOOB, 0, 0);
      dst[s][1] = __builtin_amdgcn_raw_buffer_load_b32(r, kb < nkb ? o + 4 : kGluOOB, 0, 0);
    }
  };
  const uint32_t* lut_lane = lut + (lane & (kMidCopies - 1));
  auto look_up = [&](const uint32_t (&src)[kShare][2], v4i (&v)[kShare]) {
#pragma unroll
    for (int s = 0; s < kShare; ++s) {
      const uint32_t f = funnel(src[s][1], src[s][0], field_bit(wave * kShare + s) & 31);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t x = f >> (e * kField);
        v[s][2 * e] = (int)lut_lane[((x & 0xffu) * 2 + 0) * kMidCopies];
        v[s][2 * e + 1] = (int)lut_lane[((x >> S & 0xffu) * 2 + 1) * kMidCopies];
      }
    }
  };
  auto put = [&](const v4i (&v)[kShare], v4i* to) {
#pragma unroll
    for (int s = 0; s < kShare; ++s) to[(wave * kShare + s) * 64 + lane] = v[s];
  };
  uint32_t xo[kX];
#pragma unroll
  for (int q = 0; q < kX; ++q) {
    const int row = 8 * (wave * kX + q) + (lane >> 3);
    const int64_t t = t0 + row;
    xo[q] = t < a.tokens ? (uint32_t)(t * a.k + 16 * row128_place(row, lane & 7)) : kGluOOB;
  }
  auto load_x = [&](auto stage, int kb) {
    glu_lds_char* st = (glu_lds_char*)mid_stage<kTokens, decltype(stage)::value>();
#pragma unroll
    for (int q = 0; q < kX; ++q)
      glu_dma16(xr, st + 1024 * (wave * kX + q), xo[q] == kGluOOB || kb >= nkb ? kGluOOB : xo[q] + (uint32_t)(kb * kBlockK));
  };
  uint32_t tv[512 * kMidCopies / 4 / kMidThreads];
#pragma unroll
  for (int r = 0; r < 512 * kMidCopies / 4 / kMidThreads; ++r)
    tv[r] = ld_global(&kHalfCodeTable.v[(tid + kMidThreads * r) / (kMidCopies / 4)]);
  load_x(std::integral_constant<int, 0>{}, 0);
  load_codes(0, w[0]);
  load_x(std::integral_constant<int, 1>{}, 1);
  load_codes(1, w[1]);
#pragma unroll
  for (int r = 0; r < 512 * kMidCopies / 4 / kMidThreads; ++r)
    reinterpret_cast<u32x4*>(lut)[tid + kMidThreads * r] = u32x4{tv[r], tv[r], tv[r], tv[r]};
  v4i c[2 * kRW][kTG];  // gate's row tiles, then up's
#pragma unroll
  for (int i = 0; i < 2 * kRW; ++i)
#pragma unroll
    for (int j = 0; j < kTG; ++j) c[i][j] = v4i{0, 0, 0, 0};
  __syncthreads();
  v4i next[kShare];
  look_up(w[0], next);
  put(next, A[0]);
  glu_wait<0>();  // the first two blocks' activations
  glu_barrier();
  // block kb: its operands are in A[kb % 2], its activations in stage kb % 3; blocks past
  // the last read zeros and are not used
  const uint32_t x_at = (uint32_t)((16 * group * kTG + l16) * 128);
  auto block = [&](auto number, int kb) {
    constexpr int U = decltype(number)::value, P = U & 1;
    load_x(std::integral_constant<int, (U + 2) % 3>{}, kb + 2);
    // (fences: left alone the compiler moved the loads to where they are used and
    // read each operand after the products of the one before)
    __builtin_amdgcn_sched_barrier(0);
    const glu_lds_char* st = (const glu_lds_char*)mid_stage<kTokens, U % 3>() + x_at;
    v4i op[2 * kRW][2], b[kTG][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < kTG; ++j)
        b[j][h] = *reinterpret_cast<const __attribute__((address_space(3))) v4i*>(
            st + 2048 * j + 16 * row128_place(l16, 4 * h + lg));
#pragma unroll
      for (int i = 0; i < 2 * kRW; ++i) op[i][h] = A[P][(2 * (i / kRW * kRT + row0 + i % kRW) + h) * 64 + lane];
    }
    // The next block's activations and codes are there once no more than the kX loads
    // above, the last that were asked for, are in flight (loads return in order; those of
    // codes are not counted, as the compiler joins some of them).  Behind the barrier
    // below that holds for all wavefronts.
    glu_wait<kX>();
    look_up(w[(U + 1) % 2], next);
    load_codes(kb + 2, w[U % 2]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2 * kRW; ++i)
#pragma unroll
        for (int j = 0; j < kTG; ++j) c[i][j] = mfma_i8(op[i][h], b[j][h], c[i][j]);
    put(next, A[P ^ 1]);
    __builtin_amdgcn_sched_barrier(0);
    glu_barrier();
  };
  int kb = 0;
  for (; kb + 5 < nkb; kb += 6) {
    block(std::integral_constant<int, 0>{}, kb);
    block(std::integral_constant<int, 1>{}, kb + 1);
    block(std::integral_constant<int, 2>{}, kb + 2);
    block(std::integral_constant<int, 3>{}, kb + 3);
    block(std::integral_constant<int, 4>{}, kb + 4);
    block(std::integral_constant<int, 5>{}, kb + 5);
  }
  if (kb < nkb) block(std::integral_constant<int, 0>{}, kb);
  if (kb + 1 < nkb) block(std::integral_constant<int, 1>{}, kb + 1);
  if (kb + 2 < nkb) block(std::integral_constant<int, 2>{}, kb + 2);
  if (kb + 3 < nkb) block(std::integral_constant<int, 3>{}, kb + 3);
  if (kb + 4 < nkb) block(std::integral_constant<int, 4>{}, kb + 4);
  glu_wait<0>();  // no DMA outlives the workgroup
  // lane: outputs n0 + 16 i + 4 lg + q (i < kRW: gate, i + kRW: up) of token 16 j + l16 of the
  // wavefront's
  const double gg = ld_global(a.gate_gamma), gu = ld_global(a.up_gamma);
  const int64_t n0 = strip * kStripRows + 16 * (kRT * part + row0);
#pragma unroll
  for (int j = 0; j < kTG; ++j) {
    const int64_t token = t0 + 16 * (group * kTG + j) + l16;
    const bool in = token < a.tokens;
    const float s = in ? ld_global(a.x_scale + token) : 0.f;
    const float sg = out_scale(gg, s), su = out_scale(gu, s);
    const int64_t e = token * a.n_out + n0 + 4 * lg;
    float g[4 * kRW], u[4 * kRW];
#pragma unroll
    for (int i = 0; i < kRW; ++i) {
      float h[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        g[4 * i + q] = out_value(c[i][j][q], sg);
        u[4 * i + q] = out_value(c[i + kRW][j][q], su);
        h[q] = act_value<kAct>(g[4 * i + q]) * u[4 * i + q];
      }
      if (in) st_global(reinterpret_cast<u32x2*>(a.H + e + 16 * i), u32x2{pair_bf16(h[0], h[1]), pair_bf16(h[2], h[3])});
    }
    if constexpr (kRT == 4) {
      // 8-bit G and U (the only use of whole strips): a block's largest lies in two wavefronts
      __shared__ uint32_t tops[2][2][kTokens];  // [row half][layer][token]
      uint32_t top[2] = {0u, 0u};
#pragma unroll
      for (int z = 0; z < 2; ++z) {
#pragma unroll
        for (int i = 0; i < 4 * kRW; ++i) top[z] = max_u(top[z], abs_bits(z ? u[i] : g[i]));
        top[z] = max_u(top[z], (uint32_t)__shfl_xor((int)top[z], 16, 64));
        top[z] = max_u(top[z], (uint32_t)__shfl_xor((int)top[z], 32, 64));
        if (lg == 0) tops[row0 / kRW][z][16 * (group * kTG + j) + l16] = top[z];
      }
      __syncthreads();
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        if (!in) break;
        const CkptScale cs = ckpt_scale(max_u(top[z], tops[1 - row0 / kRW][z][16 * (group * kTG + j) + l16]));
#pragma unroll
        for (int i = 0; i < kRW; ++i) {
          uint32_t word = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) word |= ckpt_code(z ? u[4 * i + q] : g[4 * i + q], cs.inv) << (8 * q);
          st_global(reinterpret_cast<uint32_t*>(static_cast<int8_t*>(z ? a.U : a.G) + e + 16 * i), word);
        }
        if (lg == 0 && row0 == 0) st_global((z ? a.Us : a.Gs) + (token * a.n_out + n0) / kCkptBlock, cs.scale);
      }
    } else if (in && a.save != kSaveNone) {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float* x = z ? u : g;
        void* out = z ? a.U : a.G;
#pragma unroll
        for (int i = 0; i < kRW; ++i) {
          if (a.save == kRowF32)
            st_global(reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + e + 16 * i),
                      f32x4_t{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]});
          else
            st_global(reinterpret_cast<u32x2*>(static_cast<uint16_t*>(out) + e + 16 * i),
                      u32x2{pair_bf16(x[4 * i], x[4 * i + 1]), pair_bf16(x[4 * i + 2], x[4 * i + 3])});
        }
      }
    }
  }
}

// ------------------------------------------------------ forward, many tokens
// Both layers' codes are decoded once into int8 (a pass over the weights, some 6%
// of the products' time at 4096 tokens), and an int8 product runs on tiles of
// 128 outputs (256 rows: for each 64 outputs their gate rows, then their up
// rows) x 128 tokens, two workgroups on a CU, so that one's outputs are written under
// the other's products (6001 tokens, 2048 x 11008: 214 us, then 234 as the clock
// falls, 2.3 POPS; one workgroup of 256 tokens took 13 % more; 64 tokens, twice the
// workgroups, 10 % less at 391 tokens, 1536 x 8960, and up to 28 % more elsewhere).
// Bound by the way through LDS beside the products: 4096 tokens, 2560 x 6912, 127 us,
// matrix units busy 54 % of the time.  A wavefront computes 64 outputs of both layers
// (128 rows) x 64 tokens, so a lane holds g and u of the same outputs and the
// gating needs no exchange.  Tiles stream through three LDS stages of 64 k
// filled by LDS DMA; a step's fragments are read from LDS while the matrix
// instructions of the step before run, so a stage is refilled as soon as its
// fragments are in registers.
//
// A row's 64 bytes of a stage are four 16-byte pieces in the order of row64_place,
// which keeps the fragment reads free of bank conflicts.  The decoded codes lie in
// memory in that order: 8 KiB for each (64 outputs, 64 k), a wavefront's DMA
// instruction a whole KiB of it.
constexpr int kGluRows = 256;                 // rows of a tile: 128 outputs
constexpr int kGluK = 64;                     // k of a stage
constexpr int kGluABytes = kGluRows * kGluK;  // 16 KiB
constexpr int kPairBytes = 128 * kGluK;       // decoded codes of 64 outputs, 64 k

// One packed superblock (64 rows x 128 k) per wavefront: lane c = r + 16 q holds, as
// the operand (i, h), the codes of row 16 i + r at k = 64 h + 16 q .. + 15, one piece.
// The activations are laid out likewise: 16 tokens x 64 k a KiB, all of 16 tokens one
// after another (in rows every DMA instruction would read half a line of each of 16
// tokens, see tiled_at: the product took 137 us in place of 125 at 4096 tokens,
// 2560 x 6912, 8-bit G and U kept).
// Bound by memory; a wavefront's first chunk is on its way while the tables are
// filled, and sixteen wavefronts share one set of them (four, loading after the
// fill: 15.4 us at 391 tokens, 1536 x 8960 4:8, now 12.8).
constexpr int kDecodeThreads = 1024;
template <int S>
__global__ __launch_bounds__(kDecodeThreads) void glu_decode_kernel(const char* __restrict__ gate,
                                                                   const char* __restrict__ up, int64_t superblocks,
                                                                   int nkb, char* __restrict__ out,
                                                                   const int8_t* __restrict__ xq, int64_t tokens,
                                                                   int64_t x_jobs, char* __restrict__ x_out) {
  __shared__ __attribute__((aligned(16))) uint32_t lut[512 * kSmallCopies];
  constexpr int kBytes = block_bytes(S), kRuns = 512 * kSmallCopies / 4 / kDecodeThreads;
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t stride = (int64_t)gridDim.x * (kDecodeThreads / 64);
  // jobs of a wavefront: superblocks, gate's of all strips, then up's; then 16 tokens x 128 k
  int64_t j = (int64_t)blockIdx.x * (kDecodeThreads / 64) + (tid >> 6);
  uint32_t w[kBytes / 4], tv[kRuns];
  const auto load = [&](int64_t job) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(
        (job >= superblocks ? up + (job - superblocks) * kStripRows * kBytes : gate + job * kStripRows * kBytes) + lane * kBytes);
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i) w[i] = ld_global(src + i);
  };
#pragma unroll
  for (int r = 0; r < kRuns; ++r) tv[r] = ld_global(&kHalfCodeTable.v[(tid + kDecodeThreads * r) / (kSmallCopies / 4)]);
  if (j < 2 * superblocks) load(j);
#pragma unroll
  for (int r = 0; r < kRuns; ++r)
    reinterpret_cast<u32x4*>(lut)[tid + kDecodeThreads * r] = u32x4{tv[r], tv[r], tv[r], tv[r]};
  const uint32_t* lut_lane = lut + (lane & (kSmallCopies - 1));
  __syncthreads();
  for (; j < 2 * superblocks; j += stride) {
    const int side = j >= superblocks;
    const int64_t sb = side ? j - superblocks : j, strip = sb / nkb, kb = sb - strip * nkb;
    v4i c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = chunk_operand<S>(w, i, lut_lane);
    if (j + stride < 2 * superblocks) load(j + stride);
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // operand 2 (row tile) + (k half)
      const int row = 64 * side + 16 * (i >> 1) + (lane & 15);
      char* dst = out + (strip * (2 * nkb) + 2 * kb + (i & 1)) * kPairBytes + row * kGluK + 16 * row64_place(row, lane >> 4);
      st_global(reinterpret_cast<v4i*>(dst), c[i]);
    }
  }
  for (; j < 2 * superblocks + x_jobs; j += stride) {
    const int64_t x = j - 2 * superblocks, tb = x / nkb, kb = x - tb * nkb;
    const int row = lane >> 2;
    const int64_t token = 16 * tb + row < tokens ? 16 * tb + row : tokens - 1;  // rows past the last are not used
    const v4i* src = reinterpret_cast<const v4i*>(xq + token * nkb * kBlockK + kb * kBlockK) + row64_place(row, lane & 3);
    v4i* dst = reinterpret_cast<v4i*>(x_out + (tb * nkb + kb) * 2048) + lane;
    const v4i v0 = ld_global(src), v1 = ld_global(src + 4);
    st_global(dst, v0);
    st_global(dst + 64, v1);
  }
}

// LDS of the stages: separate objects, so that the compiler sees that reads of one
// stage and DMA into the others touch different memory (namespace scope: a
// __shared__ array inside a template made the host pass drop the kernel's stub)
constexpr int kGluTokens = 128;                              // of a tile
constexpr int kGluStageBytes = kGluABytes + kGluTokens * kGluK;
constexpr int kGluPerStep = 6;                               // DMA instructions of a wavefront and step: four of A, two of B
__shared__ __attribute__((aligned(1024))) char g_glu_st0[kGluStageBytes];
__shared__ __attribute__((aligned(1024))) char g_glu_st1[kGluStageBytes];
__shared__ __attribute__((aligned(1024))) char g_glu_st2[kGluStageBytes];
template <int P>
__device__ __forceinline__ char* glu_stage() {
  return P == 0 ? g_glu_st0 : P == 1 ? g_glu_st1 : g_glu_st2;
}

struct GluFrags {
  v4i a[8], b[4];
};

// A wavefront's 32 tokens x 64 outputs of one result, kBytes a token, from LDS (rows
// kBytes + 16 apart) to memory in whole 16-byte pieces: a token's outputs are one
// or half a 128-byte line
template <int kBytes>
__device__ __forceinline__ void glu_flush(const glu_lds_char* rows, void* out, int64_t token, int64_t tokens, int64_t row_bytes,
                                          int64_t col_bytes, int lane) {
  constexpr int kPieces = kBytes / 16, kAtOnce = 64 / kPieces;
  asm volatile("" ::: "memory");
#pragma unroll
  for (int p = 0; p < 32 / kAtOnce; ++p) {
    const int t = p * kAtOnce + lane / kPieces, c = 16 * (lane % kPieces);
    const v4i v = *reinterpret_cast<const __attribute__((address_space(3))) v4i*>(rows + t * (kBytes + 16) + c);
    if (token + t < tokens) st_global(reinterpret_cast<v4i*>(static_cast<char*>(out) + (token + t) * row_bytes + col_bytes + c), v);
  }
  asm volatile("" ::: "memory");
}

template <int kAct>
__global__ __launch_bounds__(256, 2) void glu_gemm_kernel(GluArgs a, const char* __restrict__ codes,
                                                          const char* __restrict__ x, int row_tiles, int token_tiles) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l16 = lane & 15, lg = lane >> 4;
  // Workgroup (XCD x, slot) takes the slot-th tile of XCD x's contiguous eighth of
  // an order in groups of four token tiles, row tiles within a group: an XCD's
  // workgroups run a compact block and share its operands in their L2.
  int rt, tt;
  {
    const int tiles = row_tiles * token_tiles, per = (tiles + 7) / 8, full = tiles - (per - 1) * 8;
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    if (slot >= (xcd < full ? per : per - 1)) return;
    const int t = xcd < full ? xcd * per + slot : full * per + (xcd - full) * (per - 1) + slot;
    const int g = t / (4 * row_tiles), r = t - g * 4 * row_tiles;
    const int gm = token_tiles - 4 * g < 4 ? token_tiles - 4 * g : 4;
    tt = 4 * g + r % gm;
    rt = r / gm;
  }
  const int64_t t0 = (int64_t)tt * kGluTokens;
  const int nks = (int)(a.k / kGluK);
  // A: two pairs of 64 outputs, each nks pieces of 8 KiB, in order
  const __amdgpu_buffer_rsrc_t ar = glu_rsrc(codes + (int64_t)rt * 2 * nks * kPairBytes, (int64_t)2 * nks * kPairBytes);
  const __amdgpu_buffer_rsrc_t br = glu_rsrc(x, (a.tokens + 15) / 16 * 16 * a.k);
  uint32_t a_off[4], b_off[2];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int at = 4 * wave + q;  // KiB of the stage's 16
    a_off[q] = (uint32_t)((at >> 3) * nks * kPairBytes + (at & 7) * 1024 + 16 * lane);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int64_t t = t0 + 32 * wave + 16 * q;
    b_off[q] = t < a.tokens ? (uint32_t)(t * a.k + 16 * lane) : kGluOOB;
  }
  // past the last step the same instructions read zeros into a stage that nobody
  // reads, so the waits can count them
  auto dma = [&](auto stage, int ks) {
    constexpr int P = decltype(stage)::value;
    glu_lds_char* st = (glu_lds_char*)glu_stage<P>();
    const bool in = ks < nks;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      glu_dma16(ar, st + 1024 * (4 * wave + q), in ? a_off[q] + (uint32_t)(ks * kPairBytes) : kGluOOB);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      glu_dma16(br, st + kGluABytes + 1024 * (2 * wave + q),
                in && b_off[q] != kGluOOB ? b_off[q] + (uint32_t)(ks * 1024) : kGluOOB);
  };
  v4i c[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = v4i{0, 0, 0, 0};
  const uint32_t frag = (uint32_t)(l16 * kGluK + 16 * row64_place(l16, lg));
  const uint32_t a_base = (uint32_t)(wm * 128 * kGluK) + frag, b_base = (uint32_t)(kGluABytes + wn * 64 * kGluK) + frag;
  auto read = [&](auto stage, GluFrags& f) {
    constexpr int P = decltype(stage)::value;
    const glu_lds_char* st = (const glu_lds_char*)glu_stage<P>();
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f.b[j] = *reinterpret_cast<const __attribute__((address_space(3))) v4i*>(st + b_base + j * 16 * kGluK);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f.a[i] = *reinterpret_cast<const __attribute__((address_space(3))) v4i*>(st + a_base + i * 16 * kGluK);
  };
  // Step ks: its fragments are in `now` (read in step ks - 1).  Once every wavefront
  // is here, stage ks % 3 is free and takes step ks + 3; step ks + 1, whose DMA has
  // landed for all, is read into `next`.
  auto step = [&](auto stage, int ks, GluFrags& now, GluFrags& next) {
    constexpr int P = decltype(stage)::value;
    glu_wait<kGluPerStep, true>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    dma(std::integral_constant<int, P>{}, ks + 3);
    read(std::integral_constant<int, (P + 1) % 3>{}, next);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[i][j] = mfma_i8(now.a[i], now.b[j], c[i][j]);
    // order of issue: the reads for the next step first, a product after each (left
    // alone, the compiler put them last and every step waited for them), then
    // the DMA, then the rest
#pragma unroll
    for (int r = 0; r < 12; ++r) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix instruction
    }
#pragma unroll
    for (int r = 0; r < kGluPerStep; ++r) {
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // load
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 20 - kGluPerStep, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  using S2 = std::integral_constant<int, 2>;
  GluFrags f0, f1;
  dma(S0{}, 0);
  dma(S1{}, 1);
  dma(S2{}, 2);
  glu_wait<2 * kGluPerStep>();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  read(S0{}, f0);
  int ks = 0;
  for (; ks + 5 < nks; ks += 6) {  // three stages x two fragment sets
    step(S0{}, ks, f0, f1);
    step(S1{}, ks + 1, f1, f0);
    step(S2{}, ks + 2, f0, f1);
    step(S0{}, ks + 3, f1, f0);
    step(S1{}, ks + 4, f0, f1);
    step(S2{}, ks + 5, f1, f0);
  }
  if (ks < nks) step(S0{}, ks, f0, f1);
  if (ks + 1 < nks) step(S1{}, ks + 1, f1, f0);
  if (ks + 2 < nks) step(S2{}, ks + 2, f0, f1);
  if (ks + 3 < nks) step(S0{}, ks + 3, f1, f0);
  if (ks + 4 < nks) step(S1{}, ks + 4, f0, f1);
  glu_wait<0, true>();  // no DMA outlives the workgroup, no read its stage

  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");

  // Lane: outputs n0 + 16 i + 4 lg + q (i < 4: gate, i + 4: up) of token
  // t0 + 64 wn + 16 j + l16.  Results pass through LDS, 32 tokens at a time, in a part
  // of the stages that is the wavefront's own, so that they are stored in whole lines.
  constexpr int kPart = kGluStageBytes / 2;
  static_assert(32 * (128 + 16) <= kPart, "32 rows of 64 bf16");
  glu_lds_char* part = (glu_lds_char*)(wave < 2 ? g_glu_st0 : g_glu_st1) + (wave & 1) * kPart;
  const double gg = ld_global(a.gate_gamma), gu = ld_global(a.up_gamma);
  const int64_t n0 = (int64_t)rt * 128 + wm * 64;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int64_t first = t0 + 64 * wn + 32 * half;
    float g[2][16], u[2][16];
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      const int j = 2 * half + jj;
      const int64_t token = first + 16 * jj + l16;
      const float s = token < a.tokens ? ld_global(a.x_scale + token) : 0.f;
      const float sg = out_scale(gg, s), su = out_scale(gu, s);
      glu_lds_char* row = part + (16 * jj + l16) * (128 + 16) + 8 * lg;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          g[jj][4 * i + q] = out_value(c[i][j][q], sg);
          u[jj][4 * i + q] = out_value(c[i + 4][j][q], su);
          h[q] = act_value<kAct>(g[jj][4 * i + q]) * u[jj][4 * i + q];
        }
        *reinterpret_cast<__attribute__((address_space(3))) u32x2*>(row + 32 * i) =
            u32x2{pair_bf16(h[0], h[1]), pair_bf16(h[2], h[3])};
      }
    }
    glu_flush<128>(part, a.H, first, a.tokens, 2 * a.n_out, 2 * n0, lane);
    if (a.save == kSaveNone) continue;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      void* out = z ? a.U : a.G;
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        const float* x = z ? u[jj] : g[jj];
        const int64_t token = first + 16 * jj + l16;
        if (a.save == kRowQ8) {
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) top = max_u(top, abs_bits(x[i]));
          top = max_u(top, (uint32_t)__shfl_xor((int)top, 16, 64));
          top = max_u(top, (uint32_t)__shfl_xor((int)top, 32, 64));
          const CkptScale cs = ckpt_scale(top);
          glu_lds_char* row = part + (16 * jj + l16) * (64 + 16) + 4 * lg;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) w |= ckpt_code(x[4 * i + q], cs.inv) << (8 * q);
            *reinterpret_cast<__attribute__((address_space(3))) uint32_t*>(row + 16 * i) = w;
          }
          if (lg == 0 && token < a.tokens) st_global((z ? a.Us : a.Gs) + (token * a.n_out + n0) / kCkptBlock, cs.scale);
        } else if (a.save == kRowBf16) {
          glu_lds_char* row = part + (16 * jj + l16) * (128 + 16) + 8 * lg;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<__attribute__((address_space(3))) u32x2*>(row + 32 * i) =
                u32x2{pair_bf16(x[4 * i], x[4 * i + 1]), pair_bf16(x[4 * i + 2], x[4 * i + 3])};
        } else if (token < a.tokens) {  // binary32: a lane's four outputs are 16 bytes already
          float* row = static_cast<float*>(out) + token * a.n_out + n0 + 4 * lg;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            st_global(reinterpret_cast<f32x4_t*>(row + 16 * i), f32x4_t{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]});
        }
      }
      if (a.save == kRowQ8) glu_flush<64>(part, out, first, a.tokens, a.n_out, n0, lane);
      else if (a.save == kRowBf16) glu_flush<128>(part, out, first, a.tokens, 2 * a.n_out, 2 * n0, lane);
    }
  }
}

// ------------------------------------------------------------------ host
// Up to kGluFewTokens tokens every 16 have workgroups of their own (calls, 6:8; 96 tokens
// of 896 x 4864, 1536 x 8960, 2560 x 6912: 7.6, 12.0, 12.7 us, by the kernel for some
// tokens 7.8, 12.6, 11.5; 64 tokens: 7.7, 9.8, 9.5 and 7.7, 12.7, 11.6; 128 tokens: 8.3,
// 14.9, 15.8 and 7.8, 13.0, 11.8).
// Beyond, tiles of 32 outputs that decode for themselves, for 256 tokens at a time, one
// on a CU, or for 128, of which a CU holds two and runs one in some half of the
// time: whichever gives a CU less to do (256 tokens of 2560 x 6912, 1 or 2 of them on a
// CU: 16.8 us, of 128 tokens 18.7; of 1536 x 8960, 2 or 3: 21.5 and 18.2).  With more
// than kGluMidRounds of the smaller on a CU the codes are decoded once for all (300
// tokens of 2048 x 11008, 5: 34.2 us, decoded once 41.7; 512 tokens of 1536 x 8960, 5:
// 27.9 and 33.6; 768 tokens of 2560 x 6912, 6: 46.2 and 42.7).  8-bit G and U need tiles
// of 64 outputs, of 64 or 128 tokens (192 tokens of 1536 x 8960, 2 or 2 on a CU: 18.6 us,
// of 128 tokens 25.2; 300 tokens of 2048 x 4096, 2 or 1: 22.0 and 17.3), which win up to
// kGluMidRoundsQ8 (768 tokens, 896 x 4864, 4: 22.5 us, decoded once 27.9; 391 tokens,
// 1536 x 8960, 4: 32.3 and 38.5; 512 tokens, 2560 x 6912, 4: 37.7 and 36.9; 1280 tokens,
// 896 x 4864, 5: 32.9 and 34.0).
constexpr int64_t kGluFewTokens = 96, kGluMidRounds = 5, kGluMidRoundsQ8 = 4;
// tokens of a tile that decodes for itself; 0: the codes are decoded once
static int glu_mid_tokens(int64_t tokens, int64_t n_out, bool q8) {
  const int64_t outputs = q8 ? 64 : 32, t = q8 ? 64 : 128;
  const auto on_a_cu = [&](int64_t t) { return (n_out / outputs * ((tokens + t - 1) / t) + 255) / 256; };
  const int64_t small = on_a_cu(t), large = 2 * on_a_cu(2 * t);
  if ((small < large ? small : large) > (q8 ? kGluMidRoundsQ8 : kGluMidRounds)) return 0;
  return (int)(small < large ? t : 2 * t);
}
size_t glu_ws_bytes(int64_t tokens, int64_t k, int64_t n_out, bool q8) {
  if (tokens <= kGluFewTokens || glu_mid_tokens(tokens, n_out, q8)) return 0;
  return (size_t)(2 * n_out * k + (tokens + 15) / 16 * 16 * k);
}

template <int S, int kAct>
static hipError_t glu_launch(const GluArgs& a, void* ws, hipStream_t s) {
  const unsigned strips = (unsigned)(a.n_out / kStripRows);
  const auto blocks_of = [&](int tokens) { return (unsigned)((a.tokens + tokens - 1) / tokens); };
  if (a.tokens <= kGluFewTokens) {
    glu_small_kernel<S, kAct><<<dim3(strips, blocks_of(16)), 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  if (const int tile = glu_mid_tokens(a.tokens, a.n_out, a.save == kRowQ8)) {
    if (tile == 64) glu_mid_kernel<S, kAct, 4, 64><<<dim3(strips, blocks_of(64)), kMidThreads, 0, s>>>(a);
    else if (a.save == kRowQ8) glu_mid_kernel<S, kAct, 4, 128><<<dim3(strips, blocks_of(128)), kMidThreads, 0, s>>>(a);
    else if (tile == 128) glu_mid_kernel<S, kAct, 2, 128><<<dim3(2 * strips, blocks_of(128)), kMidThreads, 0, s>>>(a);
    else glu_mid_kernel<S, kAct, 2, 256><<<dim3(2 * strips, blocks_of(256)), kMidThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  const int nkb = (int)(a.k / kBlockK);
  const int64_t superblocks = a.n_out / kStripRows * nkb;
  const int64_t x_jobs = (a.tokens + 15) / 16 * nkb, blocks = (2 * superblocks + x_jobs + kDecodeThreads / 64 - 1) / (kDecodeThreads / 64);
  char* const codes = static_cast<char*>(ws);
  char* const x = codes + 2 * a.n_out * a.k;
  glu_decode_kernel<S><<<(unsigned)(blocks < 512 ? blocks : 512), kDecodeThreads, 0, s>>>(
      static_cast<const char*>(a.gate), static_cast<const char*>(a.up), superblocks, nkb, codes, a.xq, a.tokens, x_jobs, x);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int row_tiles = (int)(a.n_out / 128);
  const int token_tiles = (int)((a.tokens + kGluTokens - 1) / kGluTokens);
  const int64_t tiles = (int64_t)row_tiles * token_tiles;
  glu_gemm_kernel<kAct><<<(unsigned)((tiles + 7) / 8 * 8), 256, 0, s>>>(a, codes, x, row_tiles, token_tiles);
  return hipGetLastError();
}
template <int S>
static hipError_t glu_launch_s(const GluArgs& a, void* ws, hipStream_t s) {
  return a.act == kActRelu2 ? glu_launch<S, kActRelu2>(a, ws, s) : glu_launch<S, kActSilu>(a, ws, s);
}
hipError_t launch_glu(const GluArgs& a, int S, void* ws, hipStream_t s) {
  if (S == 8) return glu_launch_s<8>(a, ws, s);
  if (S == 6) return glu_launch_s<6>(a, ws, s);
  if (S == 2) return glu_launch_s<2>(a, ws, s);
  return glu_launch_s<4>(a, ws, s);
}

}  // namespace bl
