// rope.hip -- head norms and rotary positions of a block's queries and keys
// in one pass (with the copy of K and V rows into a cache), its backward,
// and the cosine / sine table both read.
#include "common.h"
#include "launch.h"

namespace bl {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------
// A lane owns 16 elements of a head row: e = 8l .. 8l+7 of the first half
// and the same of the second half, so both members of every rotated pair
// (i, i + d/2) sit in one lane and every access is 16 bytes.  D/16 lanes
// (8 or 4) share a row; sums over a row are two or three lane exchanges.
// A wavefront takes one token and kRowsHeld rows per lane group of its
// heads, all loads issued before the first use: the token's table slice is
// read once for them.
// ---------------------------------------------------------------------
constexpr int kRowsHeld = 2;
template <int D>
struct RopeMap {
  static constexpr int kLanes = D / 16;          // lanes of a row
  static constexpr int kGroups = 64 / kLanes;    // rows of a wavefront at a time
  static constexpr int kUnit = kGroups * kRowsHeld;  // head rows of a wavefront's unit
};

__device__ __forceinline__ float rsq(float x) { return __builtin_amdgcn_rsqf(x); }

// sum over the D/16 lanes that share a row
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < RopeMap<D>::kLanes; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 y = __builtin_convertvector(f32x2{a, b}, bf16x2);  // nearest, ties to even
  return __builtin_bit_cast(uint32_t, y);
}

// 8 elements from binary32 or bf16 memory
template <bool F32>
struct Vec8;
template <>
struct Vec8<true> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t e) {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + e);
    a = ld_global(q);
    b = ld_global(q + 1);
  }
  __device__ __forceinline__ void zero() { a = b = f32x4{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
  __device__ __forceinline__ void scale(float k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] *= k;
      b[i] *= k;
    }
  }
};
template <>
struct Vec8<false> {
  u32x4 a;
  __device__ __forceinline__ void load(const void* p, int64_t e) {
    a = ld_global(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + e));
  }
  __device__ __forceinline__ void zero() { a = u32x4{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ float get(int i) const {
    return (i & 1) ? bf16_hi(a[(i >> 1) & 3]) : bf16_lo(a[(i >> 1) & 3]);
  }
  __device__ __forceinline__ void scale(float k) {  // by a power of two
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = pack_bf16(bf16_lo(a[i]) * k, bf16_hi(a[i]) * k);
  }
};

// 1 / sqrt(mean(x^2) + eps) of the row that D/16 lanes hold.  Where the squares
// leave binary32 (from some 1e18 on: an infinite mean made the row zeros; below
// 2^-50 with an eps as small) the row is first scaled by a power of two, in
// place: the result is then that of the scaled row, and `by` the scale.  The
// branch is taken for a whole wavefront and no ordinary row takes it.
template <int D, bool F32>
__device__ __forceinline__ float row_scale(Vec8<F32>& lo, Vec8<F32>& hi, float eps, float& by) {
  auto mean = [&](float e) {
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(lo.get(i), lo.get(i), fmaf(hi.get(i), hi.get(i), sq));
    return fmaf(row_sum<D>(sq), 1.f / D, e);
  };
  float m = mean(eps);
  by = 1.f;
  if (__ballot(!(m >= 0x1p-100f && m <= 0x1p127f))) {
    by = m > 0x1p127f ? 0x1p-70f : m < 0x1p-100f ? 0x1p96f : 1.f;
    lo.scale(by);
    hi.scale(by);
    m = mean(eps * by * by);
  }
  return rsq(m);
}

// cosines and sines of a lane's 8 pairs at one position; a position outside
// the table gives NaN, so a wrong one shows in the outputs
struct Turn {
  float c[8], s[8];
  __device__ __forceinline__ void load(const float* table, int64_t max_pos, int half, int32_t p, int i0) {
    const bool in = p >= 0 && p < max_pos;
    const f32x4* t = reinterpret_cast<const f32x4*>(table + ((int64_t)(in ? p : 0) * half + i0) * 2);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 v = ld_global(t + q);
      c[2 * q] = in ? v[0] : __builtin_nanf("");
      s[2 * q] = in ? v[1] : __builtin_nanf("");
      c[2 * q + 1] = in ? v[2] : __builtin_nanf("");
      s[2 * q + 1] = in ? v[3] : __builtin_nanf("");
    }
  }
};

__device__ __forceinline__ void store8(uint16_t* p, const float* y) {
  st_global(reinterpret_cast<u32x4*>(p), u32x4{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                               pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7])});
}

// y = R(pos) (w * x / rms(x)) for rows of q and k, V rows copied; all
// rounded once to bf16.  Bound by HBM where there is much to move (6001 tokens,
// 14 + 2 + 2 heads of 64, bf16: 28 MB in 9.0 us, 3.1 TB/s of which 2 us are the
// launch), by three loads one after another (position, table, weights) in a
// serving step (64 tokens: 4.1 us).
template <int D, bool F32, bool NORM>
__global__ __launch_bounds__(256) void qk_rope_kernel(RopeArgs a) {
  typedef RopeMap<D> M;
  const int lane = threadIdx.x & 63;
  const int heads = a.hq + a.hkv + (a.V ? a.hkv : 0);
  const int chunks = (heads + M::kUnit - 1) / M::kUnit;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t = unit / chunks;
  if (t >= a.tokens) return;
  const int h0 = (int)(unit - t * chunks) * M::kUnit + lane / M::kLanes;
  const int i0 = 8 * (lane % M::kLanes);  // first pair of this lane
  Vec8<F32> lo[kRowsHeld], hi[kRowsHeld];
#pragma unroll
  for (int r = 0; r < kRowsHeld; ++r) {
    const int h = h0 + r * M::kGroups;
    const void* base = h < a.hq ? a.Q : h < a.hq + a.hkv ? a.K : a.V;
    const int64_t e = h < a.hq ? t * a.q_stride + (int64_t)h * D
                    : h < a.hq + a.hkv ? t * a.k_stride + (int64_t)(h - a.hq) * D
                                       : t * a.v_stride + (int64_t)(h - a.hq - a.hkv) * D;
    lo[r].zero();
    hi[r].zero();
    if (h < heads) {
      lo[r].load(base, e + i0);
      hi[r].load(base, e + i0 + D / 2);
    }
  }
  Turn turn;
  turn.load(a.table, a.max_pos, D / 2, ld_global(a.pos + t), i0);
  // the row of K and V: this token's, or the cache row its slot names
  const int64_t row = a.slots ? ld_global(a.slots + t) : t;
  const bool kept = row >= 0 && row < a.kv_rows;
#pragma unroll
  for (int r = 0; r < kRowsHeld; ++r) {
    const int h = h0 + r * M::kGroups;
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
    float x[8], y[8], rs = 1.f, by;
    Vec8<F32> xl = lo[r], xh = hi[r];
    if (NORM) rs = row_scale<D>(xl, xh, a.eps, by);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = is_v ? lo[r].get(i) : xl.get(i);
      y[i] = is_v ? hi[r].get(i) : xh.get(i);
    }
    if (NORM) {
      if (!is_v) {
        const float* w = is_q ? a.qw : a.kw;
        Vec8<true> wl, wh;
        wl.load(w, i0);
        wh.load(w, i0 + D / 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = x[i] * rs * wl.get(i);
          y[i] = y[i] * rs * wh.get(i);
        }
      }
    }
    if (!is_v) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = x[i], q = y[i];
        x[i] = fmaf(p, turn.c[i], -(q * turn.s[i]));
        y[i] = fmaf(q, turn.c[i], p * turn.s[i]);
      }
    }
    if (h >= heads || (!is_q && !kept)) continue;
    uint16_t* out = is_q ? a.Qr + (t * a.hq + h) * D
                  : is_v ? a.Vr + (row * a.hkv + h - a.hq - a.hkv) * D
                         : a.Kr + (row * a.hkv + h - a.hq) * D;
    store8(out + i0, x);
    store8(out + i0 + D / 2, y);
  }
}

// Backward of one row, with g = R(pos)^T dy and n = x / rms(x):
//   dw += g n,   a = w g,   dx = (a - n mean(a n)) / rms(x)
// (without norms dx = g).  With norms each workgroup walks over units and
// keeps its share of dw in registers (a binary32 sum per lane and element, over
// one unit of every 4 kRopeDwRows of a large call), joins them in LDS in a fixed order and
// writes one row of partial sums; rope_dw_kernel adds those in binary64.
// No atomics: reruns give the same bits.
// Bound by HBM: x and dy are read and dx is written once.  The sums take the
// registers to 162 - 168, so three workgroups fit a CU and kRopeDwRows of them are
// launched, which walk side by side to the end (1024, a third more than fit:
// 64.6 us in place of 52.1 at 8192 tokens of 20 + 5 heads of 128 in binary32;
// 512: 54.9 us; now 51.3 us for 210 MB, 4.1 TB/s).
template <int D, bool F32, bool NORM>
__global__ __launch_bounds__(256, NORM ? 3 : 4) void qk_rope_bwd_kernel(RopeBwdArgs a) {
  typedef RopeMap<D> M;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int heads = a.hq + a.hkv;
  const int chunks = (heads + M::kUnit - 1) / M::kUnit;
  const int64_t units = a.tokens * chunks;
  const int i0 = 8 * (lane % M::kLanes);
  float gw[2][16];  // [q or k][element]
#pragma unroll
  for (int i = 0; i < 16; ++i) gw[0][i] = gw[1][i] = 0.f;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + wave; unit < units; unit += (int64_t)gridDim.x * 4) {
    const int64_t t = unit / chunks;
    const int h0 = (int)(unit - t * chunks) * M::kUnit + lane / M::kLanes;
    Vec8<F32> xl[kRowsHeld], xh[kRowsHeld];
    Vec8<false> gl[kRowsHeld], gh[kRowsHeld];
#pragma unroll
    for (int r = 0; r < kRowsHeld; ++r) {
      const int h = h0 + r * M::kGroups;
      const bool is_q = h < a.hq;
      gl[r].zero();
      gh[r].zero();
      xl[r].zero();
      xh[r].zero();
      if (h < heads) {
        const uint16_t* dy = is_q ? a.dQr + (t * a.hq + h) * D : a.dKr + (t * a.hkv + h - a.hq) * D;
        gl[r].load(dy, i0);
        gh[r].load(dy, i0 + D / 2);
        if (NORM) {
          const void* x = is_q ? a.Q : a.K;
          const int64_t e = is_q ? t * a.q_stride + (int64_t)h * D : t * a.k_stride + (int64_t)(h - a.hq) * D;
          xl[r].load(x, e + i0);
          xh[r].load(x, e + i0 + D / 2);
        }
      }
    }
    Turn turn;
    turn.load(a.table, a.max_pos, D / 2, ld_global(a.pos + t), i0);
#pragma unroll
    for (int r = 0; r < kRowsHeld; ++r) {
      const int h = h0 + r * M::kGroups;
      const bool is_q = h < a.hq;
      float p[8], q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = gl[r].get(i), v = gh[r].get(i);
        p[i] = fmaf(u, turn.c[i], v * turn.s[i]);
        q[i] = fmaf(v, turn.c[i], -(u * turn.s[i]));
      }
      if (NORM) {
        float by;
        const float rs = row_scale<D>(xl[r], xh[r], a.eps, by);
        const float* w = is_q ? a.qw : a.kw;
        Vec8<true> wl, wh;
        wl.load(w, i0);
        wh.load(w, i0 + D / 2);
        const bool add = h < heads;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float nl = xl[r].get(i) * rs, nh = xh[r].get(i) * rs;
          const float ul = add ? p[i] * nl : 0.f, uh = add ? q[i] * nh : 0.f;
          gw[0][i] += is_q ? ul : 0.f;
          gw[0][8 + i] += is_q ? uh : 0.f;
          gw[1][i] += is_q ? 0.f : ul;
          gw[1][8 + i] += is_q ? 0.f : uh;
          p[i] *= wl.get(i);
          q[i] *= wh.get(i);
          dot = fmaf(p[i], nl, fmaf(q[i], nh, dot));
        }
        dot = row_sum<D>(dot) * (1.f / D);
        const float rx = rs * by;  // of the row as it was
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[i] = rx * fmaf(-(xl[r].get(i) * rs), dot, p[i]);
          q[i] = rx * fmaf(-(xh[r].get(i) * rs), dot, q[i]);
        }
      }
      if (h >= heads) continue;
      uint16_t* out = is_q ? a.dQ + (t * a.hq + h) * D : a.dK + (t * a.hkv + h - a.hq) * D;
      store8(out + i0, p);
      store8(out + i0 + D / 2, q);
    }
  }
  if (!NORM) return;
  // lane groups, then wavefronts, then this workgroup's row of partials
  __shared__ float part[4][2][D];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = gw[s][i];
#pragma unroll
      for (int o = M::kLanes; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
      if (lane < M::kLanes) part[wave][s][(i < 8 ? 0 : D / 2) + i0 + (i & 7)] = v;
    }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * D; e += 256)
    st_global(a.part + (int64_t)blockIdx.x * 2 * D + e,
              (part[0][e / D][e % D] + part[1][e / D][e % D]) + (part[2][e / D][e % D] + part[3][e / D][e % D]));
}

// dw[e] = sum of the workgroups' partials: 4 columns of 2D per workgroup, its
// threads along the rows, joined in LDS, all in binary64 and in a fixed order
// (768 rows of 256 columns: 4.6 us, latency)
__global__ __launch_bounds__(256) void rope_dw_kernel(const float* __restrict__ part, int rows, int d,
                                                     float* __restrict__ gq, float* __restrict__ gk) {
  __shared__ double red[4][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 4;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int u = 0; u < kRopeDwRows / 256; ++u) {
    const int i = threadIdx.x + 256 * u;
    if (i < rows) {
      const f32x4 x = ld_global(reinterpret_cast<const f32x4*>(part + (int64_t)i * 2 * d + e));
#pragma unroll
      for (int c = 0; c < 4; ++c) s[c] += (double)x[c];
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s[c] += __shfl_xor(s[c], o, 64);
    if (lane == 0) red[wave][c] = s[c];
  }
  __syncthreads();
  if (threadIdx.x < 4) {
    const int c = threadIdx.x;
    const float v = (float)((red[0][c] + red[1][c]) + (red[2][c] + red[3][c]));
    if (e + c < d) gq[e + c] = v;
    else gk[e + c - d] = v;
  }
}

// cos and sin of p * base^(-2i/d), formed in binary64 (a binary32 product
// would lose the angle of far positions) and rounded once.  Made once for a
// model; bound by the binary64 power and sine.
__global__ __launch_bounds__(256) void rope_table_kernel(float* __restrict__ table, int64_t pairs, int half,
                                                        double base) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= pairs) return;
  const int64_t p = e / half, i = e - p * half;
  const double angle = (double)p * pow(base, -(double)i / (double)half);
  double s, c;
  sincos(angle, &s, &c);
  st_global(reinterpret_cast<f32x2*>(table) + e, f32x2{(float)c, (float)s});
}

// ------------------------------------------------------------------ host
template <int D, bool F32>
static hipError_t rope_launch(const RopeArgs& a, hipStream_t s) {
  const int64_t heads = a.hq + a.hkv + (a.V ? a.hkv : 0);
  const int64_t units = a.tokens * ((heads + RopeMap<D>::kUnit - 1) / RopeMap<D>::kUnit);
  const dim3 grid((unsigned)((units + 3) / 4));
  if (a.qw) qk_rope_kernel<D, F32, true><<<grid, 256, 0, s>>>(a);
  else qk_rope_kernel<D, F32, false><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_qk_rope(const RopeArgs& a, int64_t d, bool f32, hipStream_t s) {
  if (d == 128) return f32 ? rope_launch<128, true>(a, s) : rope_launch<128, false>(a, s);
  return f32 ? rope_launch<64, true>(a, s) : rope_launch<64, false>(a, s);
}

template <int D, bool F32>
static hipError_t rope_bwd_launch(const RopeBwdArgs& a, hipStream_t s) {
  const int64_t heads = a.hq + a.hkv;
  const int64_t units = a.tokens * ((heads + RopeMap<D>::kUnit - 1) / RopeMap<D>::kUnit);
  int64_t blocks = (units + 3) / 4;
  if (a.qw) {
    if (blocks > kRopeDwRows) blocks = kRopeDwRows;
    if (blocks > 0) qk_rope_bwd_kernel<D, F32, true><<<dim3((unsigned)blocks), 256, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    rope_dw_kernel<<<dim3(2 * D / 4), 256, 0, s>>>(a.part, (int)blocks, D, a.gqw, a.gkw);
  } else {
    qk_rope_bwd_kernel<D, F32, false><<<dim3((unsigned)blocks), 256, 0, s>>>(a);
  }
  return hipGetLastError();
}
hipError_t launch_qk_rope_bwd(const RopeBwdArgs& a, int64_t d, bool f32, hipStream_t s) {
  if (d == 128) return f32 ? rope_bwd_launch<128, true>(a, s) : rope_bwd_launch<128, false>(a, s);
  return f32 ? rope_bwd_launch<64, true>(a, s) : rope_bwd_launch<64, false>(a, s);
}

hipError_t launch_rope_table(float* table, int64_t max_pos, int64_t d, double base, hipStream_t s) {
  const int64_t pairs = max_pos * (d / 2);
  rope_table_kernel<<<dim3((unsigned)((pairs + 255) / 256)), 256, 0, s>>>(table, pairs, (int)(d / 2), base);
  return hipGetLastError();
}

}  // namespace bl
