// attn.hip -- causal attention of packed sequences with grouped heads:
// forward and backward.
#include <type_traits>

#include "attn.h"
#include "launch.h"

namespace bl {

namespace {
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kQRows = 128;  // query rows of a forward / dQ workgroup: 32 per wavefront
constexpr int kKRows = 64;   // key rows of a tile in LDS
constexpr int kExactTiles = 2;  // dQ workgroups with at most this many key tiles form delta from P dP
constexpr float kMostLse = 65536.f;  // largest |lse| of a row with gradients
constexpr int kBKeys = 64;   // key rows of a dK / dV workgroup: two blocks of 32, four wavefronts each
constexpr int kBRows = 128;  // query rows of its stages: 32 per wavefront
constexpr int kMaxSplits = 8;  // (16 made every join 1 - 2 us longer and saved 2 us in a few calls)
constexpr float kInf = __builtin_huge_valf();
}  // namespace

// One LDS array per stage, the stage a compile-time choice: the compiler
// then sees that reads of one stage and DMA into the other touch different
// objects and does not wait for the DMA in flight.
template <int D>
struct PairBytes {  // two tiles of 64 rows
  static constexpr int kTile = kKRows * 2 * D;
  static constexpr int kAll = 2 * kTile;
};
__shared__ __attribute__((aligned(1024))) char g_a128_st0[PairBytes<128>::kAll];
__shared__ __attribute__((aligned(1024))) char g_a128_st1[PairBytes<128>::kAll];
__shared__ __attribute__((aligned(1024))) char g_a64_st0[PairBytes<64>::kAll];
__shared__ __attribute__((aligned(1024))) char g_a64_st1[PairBytes<64>::kAll];
template <int D, int P>
__device__ __forceinline__ lds_char* pair_stage() {
  static_assert(D == 64 || D == 128, "head sizes");
  if constexpr (D == 128) return (lds_char*)(P == 0 ? g_a128_st0 : g_a128_st1);
  else return (lds_char*)(P == 0 ? g_a64_st0 : g_a64_st1);
}
// the forward's stages: tiles of K and of V apart
__shared__ __attribute__((aligned(1024))) char g_f128_k0[PairBytes<128>::kTile];
__shared__ __attribute__((aligned(1024))) char g_f128_k1[PairBytes<128>::kTile];
__shared__ __attribute__((aligned(1024))) char g_f128_v0[PairBytes<128>::kTile];
__shared__ __attribute__((aligned(1024))) char g_f128_v1[PairBytes<128>::kTile];
__shared__ __attribute__((aligned(1024))) char g_f64_k0[PairBytes<64>::kTile];
__shared__ __attribute__((aligned(1024))) char g_f64_k1[PairBytes<64>::kTile];
__shared__ __attribute__((aligned(1024))) char g_f64_v0[PairBytes<64>::kTile];
__shared__ __attribute__((aligned(1024))) char g_f64_v1[PairBytes<64>::kTile];
template <int D, int P>
__device__ __forceinline__ lds_char* k_stage() {
  if constexpr (D == 128) return (lds_char*)(P == 0 ? g_f128_k0 : g_f128_k1);
  else return (lds_char*)(P == 0 ? g_f64_k0 : g_f64_k1);
}
template <int D, int P>
__device__ __forceinline__ lds_char* v_stage() {
  if constexpr (D == 128) return (lds_char*)(P == 0 ? g_f128_v0 : g_f128_v1);
  else return (lds_char*)(P == 0 ? g_f64_v0 : g_f64_v1);
}

// stages of the dK / dV kernel: 128 rows of Q and dO, their lse and delta
template <int D>
struct WideBytes {
  static constexpr int kTile = kBRows * 2 * D;
  static constexpr int kAll = 2 * kTile + 2 * 4 * kBRows;
};
__shared__ __attribute__((aligned(1024))) char g_w128_st0[WideBytes<128>::kAll];
__shared__ __attribute__((aligned(1024))) char g_w128_st1[WideBytes<128>::kAll];
__shared__ __attribute__((aligned(1024))) char g_w64_st0[WideBytes<64>::kAll];
__shared__ __attribute__((aligned(1024))) char g_w64_st1[WideBytes<64>::kAll];
template <int D, int P>
__device__ __forceinline__ lds_char* wide_stage() {
  if constexpr (D == 128) return (lds_char*)(P == 0 ? g_w128_st0 : g_w128_st1);
  else return (lds_char*)(P == 0 ? g_w64_st0 : g_w64_st1);
}

// the dK / dV kernel's rows of V, and the operands of K that are not kept in
// registers: two of D = 128's eight for both blocks of 32 keys
__shared__ __attribute__((aligned(1024))) char g_v128[kBKeys * 2 * 128];
__shared__ __attribute__((aligned(1024))) char g_v64[kBKeys * 2 * 64];
__shared__ __attribute__((aligned(1024))) char g_k128[2 * 2 * 1024];
template <int D>
__device__ __forceinline__ lds_char* v_rows() {
  if constexpr (D == 128) return (lds_char*)g_v128;
  else return (lds_char*)g_v64;
}

// DMA of R rows of a row-major array into a tile: wavefront w takes kDma
// consecutive instructions.  Rows past `rows` read zeros (the buffer ends
// there), so what lies behind a sequence, whatever it holds, never reaches a
// product.
template <int D, int R = kKRows, int W = 4>
struct TileDma {
  typedef Tile<D> T;
  static constexpr int kDma = R / T::kDmaRows / W;
  static_assert(kDma % T::kVariants == 0 || T::kVariants % kDma == 0, "compile-time permutations");
  uint32_t off[kDma];
  int wave;
  int64_t stride;
  __device__ __forceinline__ TileDma(int lane, int w, int64_t st) : wave(w), stride(st) {
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      const int ins = w * kDma + i;
      off[i] = dma_offset<D>(lane, ins % T::kVariants, st) + (uint32_t)(ins * T::kDmaRows * (int)st * 2);
    }
  }
  // p: first row's elements; rows >= 1 of them are the sequence's
  __device__ __forceinline__ void issue(lds_char* to, const uint16_t* p, int rows) const {
    const int n = rows < R ? rows : R;
    const __amdgpu_buffer_rsrc_t r = rows_rsrc(p, (uint32_t)((n - 1) * (int)stride * 2 + 2 * D));
#pragma unroll
    for (int i = 0; i < kDma; ++i) lds_load16(r, to + 1024 * (wave * kDma + i), off[i]);
  }
};
template <int D, int R = kKRows, int W = 4>
struct PairDma {  // two arrays, one tile after the other
  TileDma<D, R, W> a, b;
  __device__ __forceinline__ PairDma(int lane, int w, int64_t sa, int64_t sb) : a(lane, w, sa), b(lane, w, sb) {}
  __device__ __forceinline__ void issue(lds_char* st, const uint16_t* x, const uint16_t* y, int rows) const {
    a.issue(st, x, rows);
    b.issue(st + R * Tile<D>::kRowBytes, y, rows);
  }
};

// a row's elements as B operands: 16s + 8(l/32) .. +7 for s = 0 .. D/16-1.
// Lanes past the last row take that row's (their results are not stored): a
// condition around the loads would make each wait for the one before it.
template <int D>
__device__ __forceinline__ void load_row_operand(v8bf* f, const uint16_t* row, int lane) {
#pragma unroll
  for (int s = 0; s < D / 16; ++s)
    f[s] = __builtin_bit_cast(v8bf, ld_global(reinterpret_cast<const u32x4*>(row + 16 * s + 8 * (lane >> 5))));
}

template <int N>
__device__ __forceinline__ void clear(v16f* acc) {
#pragma unroll
  for (int t = 0; t < N; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[t][i] = 0.f;
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// ---------------------------------------------------------------- forward
// O = softmax(scale Q K^T) V in one pass over the keys: per 64-key tile
//   S^T = K Q^T,  m' = max(m, max S),  P = 2^((S - m') scale log2 e),
//   l = l 2^((m - m') ..) + sum P,  O^T = O^T 2^(..) + V^T P^T
// with m, l, O in binary32; P is rounded to bf16 (half a step, at most 2^-8
// relative; its sign differs from key to key) for the second product, the sum
// l is of the unrounded P.  m' only moves when a score passes it by 8 in the
// exponent of 2: P then stays below 2^8 and the 64 accumulators are
// rescaled a few times per row instead of once per tile.
//
// The exponent is one fma, S scale log2 e - ms with ms = m scale log2 e rounded:
// the rounding of ms (2^-24 of it) turns up in every P of the row alike, and
// differs only between tiles of different m.  Where |ms| passes kSteep that is no
// longer small (at 2^31 it leaves the range of P altogether), and the tile's
// scores are made differences S - m before their exponents are taken.
//
// Bound by the matrix unit and, beside it, the exponentials: one tile of a
// wavefront is 32 matrix instructions (1024 clocks) and about 200 others, which
// two wavefronts per SIMD overlap in part.  128 rows a workgroup (32 in each
// wavefront: their O, scores and Q take 250 registers) and two workgroups per
// CU; K and V in two stages each, so a load has a whole tile's time.  16384
// tokens, 16 + 2 heads of 128: 1049 us, 1048 TFLOP/s of the products below the
// diagonal, the matrix unit busy 53 % of the clocks; without the exponentials
// 750 us.  8192 tokens in seven sequences, 20 + 5 heads: 127 us, 39 % busy (the
// longest rows of one sequence are as long as a CU's mean share).
// Tried without gain: two heads of a group in a workgroup of eight wavefronts
// (half the loads, 5 % slower at 16384 tokens), priorities by length.
//
// Where there are few tiles of rows, `splits` workgroups are launched for
// each, and as many as its keys make parts of about `target` key tiles share
// them: each leaves its binary32 O, m and l in `part` ([split][hq][total_q]
// rows of D, then [split][hq][total_q] pairs), and attn_fwd_join_kernel adds
// them in order.
__device__ __forceinline__ int parts_of(int tiles, int splits, int target) {
  const int n = (tiles + target - 1) / target;
  return n < 1 ? 1 : n < splits ? n : splits;
}
__device__ __forceinline__ int key_tiles(const Rows& qr, const Rows& kr, int q0) {  // that rows q0 .. q0 + 127 see
  const int last = q0 + kQRows < qr.len ? q0 + kQRows : qr.len;
  return (clampi(last + kr.len - qr.len, 0, kr.len) + kKRows - 1) / kKRows;
}
template <int D>
__global__ __launch_bounds__(256, 2) void attn_fwd_kernel(AttnArgs a, int items, int splits, int target,
                                                         float* __restrict__ part) {
  typedef Tile<D> T;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.hq / a.hkv;
  const Place pl = place_of(blockIdx.x, items, a.hkv, group * splits);
  const Item it = find_item(a.cu_q, a.total_q, a.cu_k, a.total_k, a.batch, kQRows, pl.rank);
  if (it.seq < 0) return;
  const int split = pl.part / group, kvh = pl.pair, head = kvh * group + pl.part - split * group;
  const Rows qr = it.mine, kr = it.other;
  const int q0 = it.level * kQRows;
  const int off = kr.len - qr.len;
  const int w0 = q0 + 32 * wave, r = w0 + (lane & 31);
  const bool in = r < qr.len;
  // key tiles that the workgroup's and this wavefront's last rows see
  const int wlast = w0 + 32 < qr.len ? w0 + 32 : qr.len;
  const int all = key_tiles(qr, kr, q0);
  const int wall = w0 < qr.len ? (clampi(wlast + off, 0, kr.len) + kKRows - 1) / kKRows : 0;
  // this workgroup's tiles [first, tiles) of them
  const int parts = parts_of(all, splits, target);
  if (split >= parts) return;
  const int first = (int)((int64_t)all * split / parts), tiles = (int)((int64_t)all * (split + 1) / parts);
  const int wtiles = wall < tiles ? wall : tiles;

  v8bf qf[D / 16];
  load_row_operand<D>(qf, a.Q + (int64_t)(qr.start + (in ? r : qr.len - 1)) * a.q_stride + (int64_t)head * D, lane);
  const TileDma<D> kd(lane, wave, a.k_stride), vd(lane, wave, a.v_stride);
  const uint16_t* kp = a.K + (int64_t)kr.start * a.k_stride + (int64_t)kvh * D;
  const uint16_t* vp = a.V + (int64_t)kr.start * a.v_stride + (int64_t)kvh * D;
  // LDS addresses: pieces 2s and columns 32t are address bits of their own
  // (5.. and 6..), so one exclusive or makes each from the first.  They are
  // made again for every tile: kept, they would cost 13 registers.
  uint32_t ka = a_addr<D>(lane, 0);
  TrAddr va = tr_addrs<D>(lane, 0, 0);

  const float sl = a.scale * kLog2e;
  const int seen = r + off - 4 * (lane >> 5);  // last visible key, minus this lane's row offset
  v16f o[D / 32], s[2][2];  // scores of the tiles in stage 0 and 1
  clear<D / 32>(o);
  float m = -kInf, ms = 0.f, l = 0.f;  // ms: m scale log2 e, 0 while m is -inf, and while steep
  bool steep = false;                  // some row's |m scale log2 e| > kSteep (the same in all lanes)

  auto issue_k = [&](lds_char* to, int t) {
    if (t < tiles) kd.issue(to, kp + (int64_t)t * kKRows * a.k_stride, kr.len - t * kKRows);
  };
  auto issue_v = [&](lds_char* to, int t) {
    if (t < tiles) vd.issue(to, vp + (int64_t)t * kKRows * a.v_stride, kr.len - t * kKRows);
  };
  auto scores = [&](const lds_char* st, v16f* x) {
    clear<2>(x);
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) x[i] = mfma32(lds_read8(st + (ka ^ (32 * k)) + i * 32 * T::kRowBytes), qf[k], x[i]);
  };
  auto mask = [&](v16f* x, int t) {
    if (t * kKRows + kKRows > w0 + off + 1) {  // the diagonal
      const int y = seen - t * kKRows;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) x[i][j] = 32 * i + 8 * (j >> 2) + (j & 3) <= y ? x[i][j] : -kInf;
    }
  };
  auto most = [&](const v16f* x) {
    float mx = x[0][0];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) mx = fmaxf(mx, x[i][j]);
    return half_join(mx, [](float u, float v) { return fmaxf(u, v); });
  };
  auto raise = [&](float mx, v16f* x) {
    if (__ballot((mx - m) * sl > 8.f)) {  // (NaN where both are -inf: a row that sees no key yet)
      const float mn = fmaxf(m, mx), z = mn == -kInf ? 0.f : mn;
      const float f = exp2_hw((m - z) * sl);
      m = mn;
      ms = z * sl;
      steep = __ballot(fabsf(ms) > kSteep) != 0;
      if (steep) ms = 0.f;
      l *= f;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[d][j] *= f;
    }
    if (steep) {
      const float z = m == -kInf ? 0.f : m;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) x[i][j] -= z;
    }
  };
  // P of a tile's scores as operands; its sum goes to l
  auto weights = [&](v16f* x, v8bf* p) {
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 8 * (i & 1); j < 8 * (i & 1) + 8; ++j) {
        x[i >> 1][j] = exp2_hw(fmaf(x[i >> 1][j], sl, -ms));
        sum[j & 1] += x[i >> 1][j];
      }
      p[i] = operand_of(x[i >> 1], i & 1);
    }
    l += sum[0] + sum[1];
  };
  auto values = [&](const lds_char* st, const v8bf* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int d = 0; d < D / 32; ++d) o[d] = mfma32(tr_operand<D>(st, TrAddr{va.near ^ (64 * d), va.far ^ (64 * d)}, 16 * i), p[i], o[d]);
  };
  // K of tile t + 1 and V of tile t have landed; K of t + 2 and V of t + 1
  // start on their way, into the places of K of t and V of t - 1
  auto arrive = [&, &ka = ka, &va = va](auto stage, int t) {
    constexpr int P = decltype(stage)::value;
    wait_dma<0>();
    lds_barrier();
    issue_k(k_stage<D, P>(), t + 2);
    issue_v(v_stage<D, P ^ 1>(), t + 1);
    asm volatile("" : "+v"(ka), "+v"(va.near), "+v"(va.far));
  };
  // Tile t, its scores in the s of its stage: the next tile's scores are computed among
  // the exponentials of this one, the next maximum among the products with
  // V, so that the matrix unit has work throughout.  (The empty statements
  // keep the compiler from moving the exponentials out of that block.)
  auto step = [&](auto stage, int t) {
    constexpr int P = decltype(stage)::value;
    arrive(stage, t);
    v8bf p[4];
    asm volatile("" : "+v"(s[P][0]), "+v"(s[P][1]));
    scores(k_stage<D, P ^ 1>(), s[P ^ 1]);
    weights(s[P], p);
    asm volatile("" : "+v"(p[0]), "+v"(p[1]), "+v"(p[2]), "+v"(p[3]), "+v"(l));
    __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x402, 1024 / D, 0);
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x402, 1024 / D, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
    mask(s[P ^ 1], t + 1);
    const float mx = most(s[P ^ 1]);
    values(v_stage<D, P>(), p);
    __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
    for (int i = 0; i < D / 8 - 3; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x2, 2, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x8, 3, 0);
    __builtin_amdgcn_sched_barrier(0);
    raise(mx, s[P ^ 1]);
  };
  auto end = [&](auto stage, int t) {  // this wavefront's last tile
    constexpr int P = decltype(stage)::value;
    arrive(stage, t);
    v8bf p[4];
    weights(s[P], p);
    values(v_stage<D, P>(), p);
  };

  typedef std::integral_constant<int, 0> S0;
  typedef std::integral_constant<int, 1> S1;
  // The two workgroups of a CU (256 apart when the chip fills up) at different
  // priorities: their wavefronts drift apart and meet less often in the same
  // phase (16384 tokens: 1041 -> 1020 us).
  if (blockIdx.x >> 8 & 1) __builtin_amdgcn_s_setprio(1);
  int t = first;  // (stages alternate from the first tile on: S0 is its stage)
  if (first < tiles) {
    issue_k(k_stage<D, 0>(), first);
    issue_v(v_stage<D, 0>(), first);
    issue_k(k_stage<D, 1>(), first + 1);
    // the first K has landed; the rest may be on its way
    if (first + 1 < tiles) wait_dma<2 * TileDma<D>::kDma>();
    else wait_dma<TileDma<D>::kDma>();
    lds_barrier();
  }
  if (first < wtiles) {
    scores(k_stage<D, 0>(), s[0]);
    mask(s[0], first);
    raise(most(s[0]), s[0]);
    for (; t + 2 < wtiles; t += 2) {
      step(S0{}, t);
      step(S1{}, t + 1);
    }
    if (t + 1 < wtiles) {
      step(S0{}, t);
      end(S1{}, t + 1);
      t += 2;
    } else {
      end(S0{}, t);
      t += 1;
    }
  }
  for (; t < tiles; ++t) {  // the other wavefronts' tiles
    if ((t - first) & 1) arrive(S1{}, t);
    else arrive(S0{}, t);
  }

  l = half_join(l, [](float u, float v) { return u + v; });
  if (parts > 1) {
    if (in) {
      const int64_t rows = (int64_t)a.hq * a.total_q, at = ((int64_t)split * a.hq + head) * a.total_q + qr.start + r;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          st_global(reinterpret_cast<v4f*>(part + at * D + 32 * d + 8 * q + 4 * (lane >> 5)),
                    v4f{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]});
      if (lane < 32) st_global(reinterpret_cast<v2f*>(part + splits * rows * D) + at, v2f{m, l});
    }
    return;
  }
  // a row that sees no key: zeros, and -inf as the logarithm of its sum (NaN
  // scores make l NaN, and lse with it)
  store_row<D>(a.O + ((int64_t)(qr.start + r) * a.hq + head) * D, o, l > 0.f ? 1.f / l : 0.f, lane, in);
  if (a.lse && in && lane < 32)
    st_global(a.lse + (int64_t)head * a.total_q + qr.start + r, l == 0.f ? -kInf : fmaf(m, sl, log2_hw(l)) * kLn2);
}

// O and lse of rows whose keys were split: 8 (D = 128) or 16 rows of a tile and
// head per workgroup, 4 elements a thread, all parts loaded before the first is
// used.  Bound by the binary32 parts: 480 of 128 rows (31 MB) take 7.9 us.
template <int D>
__global__ __launch_bounds__(256) void attn_fwd_join_kernel(AttnArgs a, int splits, int target,
                                                           const float* __restrict__ part) {
  constexpr int kRows = 256 / (D / 4);  // rows of a workgroup
  constexpr int kParts = kQRows / kRows;
  const int tile = blockIdx.x / kParts, head = tile % a.hq;
  const Item it = find_item(a.cu_q, a.total_q, a.cu_k, a.total_k, a.batch, kQRows, tile / a.hq);
  if (it.seq < 0) return;
  const Rows qr = it.mine;
  const int parts = parts_of(key_tiles(qr, it.other, it.level * kQRows), splits, target);
  if (parts == 1) return;  // its workgroup wrote the rows
  const int r = it.level * kQRows + blockIdx.x % kParts * kRows + threadIdx.x / (D / 4), c = threadIdx.x % (D / 4);
  if (r >= qr.len) return;
  const int64_t plane = (int64_t)a.hq * a.total_q, at = (int64_t)head * a.total_q + qr.start + r;
  const float sl = a.scale * kLog2e;
  v4f x[kMaxSplits];
  v2f ml[kMaxSplits];
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s) {
    const int64_t i = (s < parts ? s : 0) * plane + at;
    x[s] = ld_global(reinterpret_cast<const v4f*>(part + i * D) + c);
    ml[s] = ld_global(reinterpret_cast<const v2f*>(part + splits * plane * D) + i);
  }
  float m = -kInf;
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s) m = fmaxf(m, ml[s][0]);
  const float z = m == -kInf ? 0.f : m;
  v4f y = v4f{0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s) {
    const float w = s < parts ? exp2_hw((ml[s][0] - z) * sl) : 0.f;
    l = fmaf(ml[s][1], w, l);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = fmaf(x[s][e], w, y[e]);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  st_global(reinterpret_cast<u32x2*>(a.O + ((int64_t)(qr.start + r) * a.hq + head) * D) + c,
            u32x2{pk_bf16(y[0] * inv, y[1] * inv), pk_bf16(y[2] * inv, y[3] * inv)});
  if (a.lse && c == 0) st_global(a.lse + at, l == 0.f ? -kInf : fmaf(m, sl, log2_hw(l)) * kLn2);
}

// --------------------------------------------------------------- backward
// With P = exp(S - lse) recomputed from the forward's lse:
//   delta = rowsum(dO O),  dV = P^T dO,  dP = dO V^T,  dS = P (dP - delta),
//   dQ = scale dS K,  dK = scale dS^T Q
// in two passes without atomics: one workgroup per 128 query rows walks the
// keys for dQ, one per 64 keys walks the rows of all query heads of its
// group for dK and dV.  S and dP are computed in both, 7 products in place
// of 5; the alternative, dQ added up in memory by the workgroups of all key
// tiles, writes and reads binary32 dQ once per tile of keys and leaves the
// order of the sums to chance.  P and dS are rounded to bf16 for the products,
// every sum is binary32.
//
// delta from the bf16 O carries O's rounding into every dS of its row.  Over
// many keys that is small against the rounding of dS itself, but rows that
// see few keys make up most of the gradients' norm: there it raised the
// relative error of dQ and dK from 2.4e-3 to 2.7e-3 (bf16 outputs alone:
// 1.7e-3).  Workgroups of at most kExactTiles key tiles therefore form
// delta = sum P dP in binary32 in a sweep of their own over tiles that stay
// in LDS, and leave it in memory for the dK / dV pass (four tiles instead of
// two gain another 1 % of the error and double the time of small calls).
//
// lse is binary32, and so is -lse / scale that S is added to: P carries their
// rounding, two to five half steps of lse (measured with exact scores: 0.4 % at |lse|
// = 1e4, 1 - 2 % at 1e5, 27 % at 2.5e6).  Rows beyond kMostLse, where that passes the
// rounding of P to bf16 several times over, get NaN in place of wrong gradients.

// The dQ pass comes first and leaves for the other what it adds to its
// products as the accumulators' first values, -lse / scale to S (-inf where
// a row sees no key, so P becomes 0) and -delta to dP, and dO rounded to
// bf16 where it comes in binary32.
//
// Bound by the matrix unit with LDS beside it (every operand from LDS, 1 KiB
// per instruction, serves one product): 8192 tokens in four sequences, 20 + 5
// heads of 128: 196 us (average of 20 runs; the shortest 181), 924 TFLOP/s of
// its three products, the matrix unit busy 51 % of the clocks.  Two workgroups
// per CU (224 registers), K and V tiles in two stages.  Small calls are a chain of latencies (finding the item,
// the rows, the tiles, the exact sums): 512 tokens, 14 + 2 heads of 64: 11 us.
//
// Keys are shared out as in the forward: parts leave binary32 sums in `part`
// ([split][hq][total_q] rows of D), which attn_dq_join_kernel adds in order (2452
// tokens, 12 heads: 70 us unsplit, 50 and 11 to join; 300 rows behind 3000 keys,
// 16 heads: 79 us, 26 and 6).
template <int D>
__global__ __launch_bounds__(256, 2) void attn_dq_kernel(AttnBwdArgs a, int items, int splits, int target,
                                                        uint16_t* __restrict__ copy, float* __restrict__ ndelta,
                                                        float* __restrict__ shift, float* __restrict__ part) {
  typedef Tile<D> T;
  constexpr int kTile = PairBytes<D>::kTile;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.hq / a.hkv;
  const Place pl = place_of(blockIdx.x, items, a.hkv, group * splits);
  const Item it = find_item(a.cu_q, a.total_q, a.cu_k, a.total_k, a.batch, kQRows, pl.rank);
  if (it.seq < 0) return;
  const int split = pl.part / group, kvh = pl.pair, head = kvh * group + pl.part - split * group;
  const Rows qr = it.mine, kr = it.other;
  const int q0 = it.level * kQRows;
  const int off = kr.len - qr.len;
  const int w0 = q0 + 32 * wave, r = w0 + (lane & 31);
  const bool in = r < qr.len;
  const int wlast = w0 + 32 < qr.len ? w0 + 32 : qr.len;
  const int all = key_tiles(qr, kr, q0);
  const int wall = w0 < qr.len ? (clampi(wlast + off, 0, kr.len) + kKRows - 1) / kKRows : 0;
  // this workgroup's tiles [first, tiles) of them
  const int parts = parts_of(all, splits, target);
  if (split >= parts) return;
  const int first = (int)((int64_t)all * split / parts), tiles = (int)((int64_t)all * (split + 1) / parts);
  const int wtiles = wall < tiles ? wall : tiles;

  // the first tiles are on their way before anything is waited for; few keys
  // (less than a part): both of them, and they stay
  const bool few = all <= kExactTiles;
  const PairDma<D> dma(lane, wave, a.k_stride, a.v_stride);
  const uint16_t* kp = a.K + (int64_t)kr.start * a.k_stride + (int64_t)kvh * D;
  const uint16_t* vp = a.V + (int64_t)kr.start * a.v_stride + (int64_t)kvh * D;
  auto issue = [&](lds_char* st, int t) {
    if (t < tiles)
      dma.issue(st, kp + (int64_t)t * kKRows * a.k_stride, vp + (int64_t)t * kKRows * a.v_stride, kr.len - t * kKRows);
  };
  issue(pair_stage<D, 0>(), first);
  if (few) issue(pair_stage<D, 1>(), 1);

  const int64_t row = qr.start + (in ? r : qr.len - 1), at = (row * a.hq + head) * D;
  const int64_t sum_at = (int64_t)head * a.total_q + row;
  v8bf qf[D / 16], gf[D / 16], of[D / 16];
  load_row_operand<D>(qf, a.Q + row * a.q_stride + (int64_t)head * D, lane);
  load_row_operand<D>(of, a.O + at, lane);
  const float given = ld_global(a.lse + sum_at);
  const bool wild = given != -kInf && !(fabsf(given) <= kMostLse);
  const float lse = wild ? __builtin_nanf("") : given;
  if (a.do_f32) {
    const v4f* p = reinterpret_cast<const v4f*>(static_cast<const float*>(a.dO) + at + 8 * (lane >> 5));
    v4f x[D / 16][2];
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) x[s][i] = ld_global(p + 4 * s + i);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const v4f y = x[s][0], z = x[s][1];
      const u32x4 g = u32x4{pk_bf16(y[0], y[1]), pk_bf16(y[2], y[3]), pk_bf16(z[0], z[1]), pk_bf16(z[2], z[3])};
      if (in && split == 0) st_global(reinterpret_cast<u32x4*>(copy + at + 16 * s + 8 * (lane >> 5)), g);
      gf[s] = __builtin_bit_cast(v8bf, g);
    }
  } else {
    load_row_operand<D>(gf, static_cast<const uint16_t*>(a.dO) + at, lane);
  }
  float nd = 0.f;  // -delta, from the row's O
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    const u32x4 o = __builtin_bit_cast(u32x4, of[s]), g = __builtin_bit_cast(u32x4, gf[s]);
#pragma unroll
    for (int i = 0; i < 4; ++i) nd = fmaf(-bf16_lo(o[i]), bf16_lo(g[i]), fmaf(-bf16_hi(o[i]), bf16_hi(g[i]), nd));
  }
  nd = half_join(nd, [](float u, float v) { return u + v; });
  if (in && split == 0 && lane < 32) {
    st_global(ndelta + sum_at, nd);
    st_global(shift + sum_at, lse == -kInf ? -kInf : -lse / a.scale);
  }
  const float le = lse == -kInf ? -kInf : -lse * kLog2e;
  uint32_t ka[D / 16];
  TrAddr kt[D / 32];
#pragma unroll
  for (int s = 0; s < D / 16; ++s) ka[s] = a_addr<D>(lane, s);
#pragma unroll
  for (int t = 0; t < D / 32; ++t) kt[t] = tr_addrs<D>(lane, t, 0);
  const float sl = a.scale * kLog2e;
  const int seen = r + off - 4 * (lane >> 5);
  v16f dq[D / 32];
  clear<D / 32>(dq);

  // P and dP of 32 keys
  auto probs = [&](const lds_char* st, int t, int i, v16f* s, v16f* g) {
    clear<1>(s);
    clear<1>(g);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      s[0] = mfma32(lds_read8(st + ka[k] + i * 32 * T::kRowBytes), qf[k], s[0]);
      g[0] = mfma32(lds_read8(st + kTile + ka[k] + i * 32 * T::kRowBytes), gf[k], g[0]);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) s[0][j] = exp2_hw(fmaf(s[0][j], sl, le));
    if (t * kKRows + kKRows > w0 + off + 1) {  // the diagonal
      const int x = seen - t * kKRows;
#pragma unroll
      for (int j = 0; j < 16; ++j) s[0][j] = 32 * i + 8 * (j >> 2) + (j & 3) <= x ? s[0][j] : 0.f;
    }
  };
  auto grads = [&](auto stage, int t) {
    const lds_char* st = pair_stage<D, decltype(stage)::value>();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v16f s[1], g[1];
      probs(st, t, i, s, g);
#pragma unroll
      for (int j = 0; j < 16; ++j) s[0][j] *= g[0][j] + nd;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const v8bf p = operand_of(s[0], k);
#pragma unroll
        for (int d = 0; d < D / 32; ++d) dq[d] = mfma32(tr_operand<D>(st, kt[d], 32 * i + 16 * k), p, dq[d]);
      }
    }
  };
  typedef std::integral_constant<int, 0> S0;
  typedef std::integral_constant<int, 1> S1;
  if (few) {
    wait_dma<0>();
    lds_barrier();
    float exact = 0.f;  // this lane's share of sum P dP
    auto sums = [&](auto stage, int t) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v16f s[1], g[1];
        probs(pair_stage<D, decltype(stage)::value>(), t, i, s, g);
#pragma unroll
        for (int j = 0; j < 16; ++j) exact = fmaf(s[0][j], g[0][j], exact);
      }
    };
    if (wtiles > 0) sums(S0{}, 0);
    if (wtiles > 1) sums(S1{}, 1);
    nd = -half_join(exact, [](float u, float v) { return u + v; });
    // (a row of NaN keeps its finite delta there: 0 times that is 0 at the keys it does not see)
    if (in && lane < 32 && !wild) st_global(ndelta + sum_at, nd);
  }
  auto step = [&](auto stage, int t) {
    if (!few) {  // (few: both tiles are there)
      wait_dma<0>();
      lds_barrier();
      issue(pair_stage<D, decltype(stage)::value ^ 1>(), t + 1);
    }
    if (t < wtiles) grads(stage, t);
  };
  int t = first;
  for (; t + 1 < tiles; t += 2) {
    step(S0{}, t);
    step(S1{}, t + 1);
  }
  if (t < tiles) step(S0{}, t);
  if (parts == 1) {
    store_row<D>(a.dQ + at, dq, a.scale, lane, in);
  } else if (in) {
    float* p = part + ((int64_t)split * a.hq * a.total_q + sum_at) * D;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        st_global(reinterpret_cast<v4f*>(p + 32 * d + 8 * q + 4 * (lane >> 5)),
                  v4f{dq[d][4 * q], dq[d][4 * q + 1], dq[d][4 * q + 2], dq[d][4 * q + 3]});
  }
}

// dQ of rows whose keys were split: the parts' sums in order, 4 elements a
// thread (see attn_fwd_join_kernel)
template <int D>
__global__ __launch_bounds__(256) void attn_dq_join_kernel(AttnBwdArgs a, int splits, int target,
                                                          const float* __restrict__ part) {
  constexpr int kRows = 256 / (D / 4);  // rows of a workgroup
  constexpr int kParts = kQRows / kRows;
  const int tile = blockIdx.x / kParts, head = tile % a.hq;
  const Item it = find_item(a.cu_q, a.total_q, a.cu_k, a.total_k, a.batch, kQRows, tile / a.hq);
  if (it.seq < 0) return;
  const Rows qr = it.mine;
  const int parts = parts_of(key_tiles(qr, it.other, it.level * kQRows), splits, target);
  if (parts == 1) return;  // its workgroup wrote the rows
  const int r = it.level * kQRows + blockIdx.x % kParts * kRows + threadIdx.x / (D / 4), c = threadIdx.x % (D / 4);
  if (r >= qr.len) return;
  const int64_t plane = (int64_t)a.hq * a.total_q, at = (int64_t)head * a.total_q + qr.start + r;
  v4f x[kMaxSplits];
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s)
    x[s] = ld_global(reinterpret_cast<const v4f*>(part + ((s < parts ? s : 0) * plane + at) * D) + c);
  v4f y = x[0];
#pragma unroll
  for (int s = 1; s < kMaxSplits; ++s)
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] += s < parts ? x[s][e] : 0.f;
  st_global(reinterpret_cast<u32x2*>(a.dQ + ((int64_t)(qr.start + r) * a.hq + head) * D) + c,
            u32x2{pk_bf16(y[0] * a.scale, y[1] * a.scale), pk_bf16(y[2] * a.scale, y[3] * a.scale)});
}

// dK and dV of 64 keys.  Lanes run over keys here: S = Q K^T has a key per
// column, so P and dS are again B operands as they stand, of the products
// over query rows.  Q and dO stream through LDS in stages of 128 rows, for
// all query heads of the group; K stays in registers, V in LDS (with V in
// registers too a wavefront needs more than half of them, and one per SIMD
// has nothing to run while it waits).  Of the eight wavefronts four share a
// block of 32 keys, each with 32 rows of the stage; their sums meet through
// LDS at the end.  (128 keys a workgroup read each stage for twice the keys,
// but make half as many workgroups, each twice as long: with 8192 tokens in
// four sequences and 5 key/value heads the longest was 2.3 times the average
// load of a CU.  Four wavefronts with both blocks of keys each, which read an
// operand from LDS for two products, need 512 registers: 382 us in place of
// 300, one wavefront per SIMD and moves between the two register files.)
//
// Bound by the matrix unit with LDS beside it: 8192 tokens in four sequences,
// 20 + 5 heads of 128: 336 us (average of 20 runs; the shortest 306), 718
// TFLOP/s of its four products, the matrix unit busy 40 % of the clocks, LDS
// 32 %; each CU runs 15 % of the time with one
// wavefront per SIMD or none (the tile of a sequence's first keys is as long as
// a CU's mean share).  512 tokens, 14 + 2 heads of 64: 11 us and 3.8 us to join.
//
// `splits` workgroups share a tile where there are few: each takes a part of
// the (stage, head) steps and leaves binary32 sums in `part`
// ([split][dK, dV][total_k][hkv][D]), which attn_dkv_join_kernel adds in
// order.
template <int D>
__global__ __launch_bounds__(512, 2) void attn_dkv_kernel(AttnBwdArgs a, int items, const uint16_t* __restrict__ dO,
                                                         const float* __restrict__ ndelta,
                                                         const float* __restrict__ shift, int splits,
                                                         float* __restrict__ part) {
  typedef Tile<D> T;
  constexpr int kTile = WideBytes<D>::kTile;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = wave & 1, rq = wave >> 1;
  const Place pl = place_of(blockIdx.x, items, a.hkv, splits);
  const Item it = find_item(a.cu_k, a.total_k, a.cu_q, a.total_q, a.batch, kBKeys, pl.rank);
  if (it.seq < 0) return;
  const int kvh = pl.pair, split = pl.part, group = a.hq / a.hkv;
  const Rows qr = it.other, kr = it.mine;
  // the first keys are seen by the most rows: highest level first
  const int k0 = ((kr.len + kBKeys - 1) / kBKeys - 1 - it.level) * kBKeys;
  const int off = kr.len - qr.len;
  const int w0 = k0 + 32 * kw, j = w0 + (lane & 31);
  const bool in = j < kr.len;
  const int first = (k0 - off > 0 ? k0 - off : 0) / kBRows;  // first stage with a row that sees a key of these
  const int n = (qr.len + kBRows - 1) / kBRows - first;      // stages per head
  const int steps = n > 0 ? n * group : 0;
  const int i0 = (int)((int64_t)steps * split / splits), i1 = (int)((int64_t)steps * (split + 1) / splits);

  {  // V rows k0 .. k0 + 63
    constexpr int kDma = kBKeys / T::kDmaRows / 8;
    const int rows = kr.len - k0 < kBKeys ? kr.len - k0 : kBKeys;
    const __amdgpu_buffer_rsrc_t r = rows_rsrc(a.V + (int64_t)(kr.start + k0) * a.v_stride + (int64_t)kvh * D,
                                               (uint32_t)((rows - 1) * (int)a.v_stride * 2 + 2 * D));
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      const int ins = wave * kDma + i;
      lds_load16(r, v_rows<D>() + 1024 * ins,
                 dma_offset<D>(lane, ins % T::kVariants, a.v_stride) + (uint32_t)(ins * T::kDmaRows * (int)a.v_stride * 2));
    }
  }
  const int64_t g_stride = (int64_t)a.hq * D;
  const PairDma<D, kBRows, 8> dma(lane, wave, a.q_stride, g_stride);
  auto issue = [&](lds_char* st, int h, int t) {
    const int64_t row = qr.start + t * kBRows;
    const int rows = qr.len - t * kBRows;
    const int64_t head = (int64_t)kvh * group + h;
    dma.issue(st, a.Q + row * a.q_stride + head * D, dO + row * g_stride + head * D, rows);
    if (rq < 2) {  // the rows' first values, 64 rows a wavefront; zeros past the sequence (dO is 0 there)
      const float* p = (rq ? ndelta : shift) + head * a.total_q + row;
      lds_load4(rows_rsrc(p, (uint32_t)((rows < kBRows ? rows : kBRows) * 4)),
                st + 2 * kTile + 4 * kBRows * rq + 256 * kw, (uint32_t)(lane + 64 * kw) * 4);
    }
  };
  // The last rows first, all heads of the group for each stage: workgroups of
  // different keys that start together then read the same stages together.
  int t = first + n - 1 - i0 / group, h = i0 % group;  // of the step being computed
  if (i0 < i1) issue(wide_stage<D, 0>(), h, t);
  constexpr int kHeld = D == 128 ? 6 : 4;  // (all eight: 256 registers and spills)
  typedef __attribute__((address_space(3))) v8bf lds_v8bf;
  lds_char* const kx = (lds_char*)g_k128 + 2048 * kw + 16 * lane;
  v8bf kf[kHeld];
  {
    v8bf k[D / 16];
    load_row_operand<D>(k, a.K + (int64_t)(kr.start + (in ? j : kr.len - 1)) * a.k_stride + (int64_t)kvh * D, lane);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) kf[i] = k[i];
    if constexpr (kHeld < D / 16) {
      if (rq == 0) {
#pragma unroll
        for (int i = kHeld; i < D / 16; ++i) *reinterpret_cast<lds_v8bf*>(kx + 1024 * (i - kHeld)) = k[i];
      }
    }
  }
  // LDS addresses: pieces 2s and columns 32t are address bits of their own
  // (5.. and 6..), so one exclusive or makes each from the first.  They are
  // made again in every step: kept, they would cost 13 registers.
  uint32_t qa = a_addr<D>(lane, 0);
  TrAddr qt = tr_addrs<D>(lane, 0, 32 * rq * T::kRowBytes);
  const lds_char* const vr = v_rows<D>() + 32 * kw * T::kRowBytes;
  const float sl = a.scale * kLog2e;
  v16f dk[D / 32], dv[D / 32];
  clear<D / 32>(dk);
  clear<D / 32>(dv);

  auto step = [&](auto stage, int i) {
    constexpr int P = decltype(stage)::value;
    wait_dma<0>();
    lds_barrier();
    const int nh = h + 1 < group ? h + 1 : 0, nt = nh ? t : t - 1;
    if (i + 1 < i1) issue(wide_stage<D, P ^ 1>(), nh, nt);
    const lds_char* st = wide_stage<D, P>();
    const int r0 = t * kBRows + 32 * rq;  // this wavefront's rows r0 .. r0 + 31
    t = nt;
    h = nh;
    // (Rows that see none of these keys are computed too, as zeros: the other
    // wavefronts of the step take as long, and accumulators that pass through
    // a branch are copied around it.)
    const lds_char* const sq = st + 32 * rq * T::kRowBytes;
    asm volatile("" : "+v"(qa), "+v"(qt.near), "+v"(qt.far));
    v16f s, g;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const lds_char* p = st + 2 * kTile + (32 * rq + 8 * u + 4 * (lane >> 5)) * 4;
      const v4f x = *reinterpret_cast<const __attribute__((address_space(3))) v4f*>(p);
      const v4f y = *reinterpret_cast<const __attribute__((address_space(3))) v4f*>(p + 4 * kBRows);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[4 * u + e] = x[e];
        g[4 * u + e] = y[e];
      }
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      s = mfma32(lds_read8(sq + (qa ^ (32 * k))), k < kHeld ? kf[k % kHeld] : lds_read8(kx + 1024 * (k - kHeld)), s);
    if (r0 + off < w0 + 31) {  // the diagonal
      const int x = j - off - r0 - 4 * (lane >> 5);  // first row that sees this lane's key
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = 8 * (e >> 2) + (e & 3) >= x ? s[e] : -kInf;
    }
    // dP among the exponentials, dV among the products P dP, then dK
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" : "+v"(s));
    v8bf p[2], w[2];
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      g = mfma32(lds_read8(sq + kTile + (qa ^ (32 * k))), lds_read8(vr + (qa ^ (32 * k))), g);
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = exp2_hw(s[e] * sl);
#pragma unroll
    for (int k = 0; k < 2; ++k) p[k] = operand_of(s, k);
    asm volatile("" : "+v"(p[0]), "+v"(p[1]), "+v"(s));
    __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x402, 640 / D, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
        dv[d] = mfma32(tr_operand<D>(st + kTile, TrAddr{qt.near ^ (64 * d), qt.far ^ (64 * d)}, 16 * k), p[k], dv[d]);
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] *= g[e];
#pragma unroll
    for (int k = 0; k < 2; ++k) w[k] = operand_of(s, k);
    asm volatile("" : "+v"(w[0]), "+v"(w[1]));
    __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x2, 384 / D, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
        dk[d] = mfma32(tr_operand<D>(st, TrAddr{qt.near ^ (64 * d), qt.far ^ (64 * d)}, 16 * k), w[k], dk[d]);
    __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
  };

  int i = i0;
  for (; i + 1 < i1; i += 2) {
    step(std::integral_constant<int, 0>{}, i);
    step(std::integral_constant<int, 1>{}, i + 1);
  }
  if (i < i1) step(std::integral_constant<int, 0>{}, i);

  // Join the four wavefronts of a block, ((0 + 2) + (1 + 3)): quarters 2 and 3
  // leave their sums for 0 and 1, then 0 takes dK and 1 dV from the other.
  // A box holds D/32 accumulators, 16 bytes per lane and quad of registers.
  typedef __attribute__((address_space(3))) v4f lds_v4f;
  constexpr int kBox = D / 32 * 4096;
  auto box = [&](int at) {  // eight of them, four to a stage
    return (at < 4 ? wide_stage<D, 0>() : wide_stage<D, 1>()) + kBox * (at & 3);
  };
  auto leave = [&](lds_char* to, const v16f* x) {
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<lds_v4f*>(to + 1024 * (4 * d + q) + 16 * lane) =
            v4f{x[d][4 * q], x[d][4 * q + 1], x[d][4 * q + 2], x[d][4 * q + 3]};
  };
  auto add = [&](const lds_char* from, v16f* x) {
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const v4f z = *reinterpret_cast<const lds_v4f*>(from + 1024 * (4 * d + q) + 16 * lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[d][4 * q + e] += z[e];
      }
  };
  const int64_t out = ((int64_t)(kr.start + j) * a.hkv + kvh) * D;
  auto finish = [&](const v16f* x, uint16_t* y, float mul) {
    if (splits == 1) {
      store_row<D>(y + out, x, mul, lane, in);
    } else if (in) {
      float* p = part + (int64_t)(2 * split + rq) * a.total_k * a.hkv * D + out;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          st_global(reinterpret_cast<v4f*>(p + 32 * d + 8 * q + 4 * (lane >> 5)),
                    v4f{x[d][4 * q], x[d][4 * q + 1], x[d][4 * q + 2], x[d][4 * q + 3]});
    }
  };
  wait_dma<0>();    // no DMA is in flight (V's, where there were no steps)
  __syncthreads();  // the stages are free
  if (rq >= 2) {
    leave(box(2 * (rq - 2) + kw), dk);
    leave(box(4 + 2 * (rq - 2) + kw), dv);
  }
  __syncthreads();
  if (rq < 2) {
    add(box(2 * rq + kw), dk);
    add(box(4 + 2 * rq + kw), dv);
  }
  __syncthreads();
  if (rq == 0) leave(box(kw), dv);
  if (rq == 1) leave(box(2 + kw), dk);
  __syncthreads();
  if (rq == 0) {
    add(box(2 + kw), dk);
    finish(dk, a.dK, a.scale);
  } else if (rq == 1) {
    add(box(kw), dv);
    finish(dv, a.dV, 1.f);
  }
}

// dK and dV of split tiles: the splits' sums in order, 8 elements a thread,
// all loaded before the first is used (bound by latency: 3.8 us)
template <int D>
__global__ __launch_bounds__(256) void attn_dkv_join_kernel(AttnBwdArgs a, int splits,
                                                           const float* __restrict__ part) {
  constexpr int kParts = 2 * kBKeys * (D / 8) / 256;  // workgroups of a tile
  const int tile = blockIdx.x / kParts, which = blockIdx.x % kParts / (kParts / 2);
  const Item it = find_item(a.cu_k, a.total_k, a.cu_q, a.total_q, a.batch, kBKeys, tile / a.hkv);
  if (it.seq < 0) return;
  const Rows kr = it.mine;
  const int f = blockIdx.x % (kParts / 2) * 256 + threadIdx.x;
  const int row = it.level * kBKeys + f / (D / 8);
  if (row >= kr.len) return;
  const int64_t plane = a.total_k * a.hkv * D;
  const int64_t at = ((int64_t)(kr.start + row) * a.hkv + tile % a.hkv) * D + 8 * (f % (D / 8));
  v4f u[kMaxSplits], v[kMaxSplits];
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s) {
    const v4f* p = reinterpret_cast<const v4f*>(part + (2 * (s < splits ? s : 0) + which) * plane + at);
    u[s] = ld_global(p);
    v[s] = ld_global(p + 1);
  }
  v4f x = u[0], y = v[0];
#pragma unroll
  for (int s = 1; s < kMaxSplits; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] += s < splits ? u[s][i] : 0.f;
      y[i] += s < splits ? v[s][i] : 0.f;
    }
  const float mul = which ? 1.f : a.scale;
  st_global(reinterpret_cast<u32x4*>((which ? a.dV : a.dK) + at),
            u32x4{pk_bf16(x[0] * mul, x[1] * mul), pk_bf16(x[2] * mul, x[3] * mul),
                  pk_bf16(y[0] * mul, y[1] * mul), pk_bf16(y[2] * mul, y[3] * mul)});
}

// ------------------------------------------------------------------- host
namespace {
int64_t most_tiles(int64_t rows, int64_t batch, int64_t tile) {
  // every sequence adds at most one partly filled tile
  return rows / tile + (batch < rows ? batch : rows);
}
size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t bwd_row_bytes(int64_t total_q, int64_t hq) { return align256((size_t)total_q * hq * 4); }
}  // namespace

// How a forward with few tiles of rows shares out the keys: into parts as
// long as they can be for all of them to run at once, two workgroups per CU
// (one more than 512 would start when the others are done: 903 rows behind
// 11779 keys, 12 heads: 73 us with 528 parts, 54 us with 480, 166 us unsplit),
// by the mean length (the kernels see the true ones), and not shorter than
// is worth a join: four tiles for rows behind a longer context (16 rows, 2048
// keys, 16 heads: 43.6 us unsplit, 18.7 with parts of eight tiles, 13.5 of four,
// 13.8 of two), six for whole prompts, whose rows see half of the keys on
// average (1900 tokens, 8 heads: 45.3 us unsplit, 32.7 with eight, 32.3 with six,
// 35.7 with four).  splits = 1: not at all.
struct FwdSplit {
  int splits, target;
};
static FwdSplit fwd_split(int64_t batch, int64_t total_q, int64_t total_k, int64_t hq) {
  // (every sequence has a tile of its own, however short: 64 tokens of as many
  // sequences of 1500 keys, 16 heads: 126 us counted as one tile and split, 74 us)
  const int64_t full = (total_q + kQRows - 1) / kQRows, each = batch < total_q ? batch : total_q;
  const int64_t tiles = (full > each ? full : each) * hq;
  const int64_t keys = total_k / (batch > 0 ? batch : 1) / kKRows;
  const bool prompts = total_q >= total_k;
  const int64_t least = prompts ? 6 : 4;
  if (tiles > 256 || keys < 2 * least) return FwdSplit{1, 1};
  const int64_t mean = prompts ? (keys + 1) / 2 : keys;
  const int64_t room = 512 - tiles / 2, target = (tiles * mean + room - 1) / room;  // (a tile ends in half a part)
  const int64_t t = target < least ? least : target;
  const int64_t most = (2 * mean + t - 1) / t;  // parts of a sequence of twice the mean length
  if (most < 2) return FwdSplit{1, 1};
  return FwdSplit{most > kMaxSplits ? kMaxSplits : (int)most, (int)t};
}

// workspace: partial O, m and l of split tiles
size_t attn_fwd_ws_bytes(int64_t batch, int64_t total_q, int64_t total_k, int64_t hq, int64_t, int64_t d) {
  const int splits = fwd_split(batch, total_q, total_k, hq).splits;
  return splits > 1 ? (size_t)splits * hq * total_q * (d + 2) * 4 : 0;
}

template <int D>
static hipError_t fwd_launch(const AttnArgs& a, float* part, hipStream_t s) {
  const FwdSplit p = fwd_split(a.batch, a.total_q, a.total_k, a.hq);
  const int64_t items = most_tiles(a.total_q, a.batch, kQRows);
  attn_fwd_kernel<D><<<dim3((unsigned)placed_blocks(items, a.hkv, a.hq / a.hkv * p.splits)), 256, 0, s>>>(
      a, (int)items, p.splits, p.target, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  attn_fwd_join_kernel<D><<<dim3((unsigned)(items * a.hq * (kQRows / (256 / (D / 4))))), 256, 0, s>>>(
      a, p.splits, p.target, part);
  return hipGetLastError();
}
hipError_t launch_attn_fwd(const AttnArgs& a, int64_t d, void* ws, hipStream_t s) {
  return d == 128 ? fwd_launch<128>(a, static_cast<float*>(ws), s) : fwd_launch<64>(a, static_cast<float*>(ws), s);
}

// Workgroups that share a dK / dV tile: as many as the chip runs at once (one
// per CU, at D = 64 two).  At D = 128 twice as many for whole prompts whose parts
// stay long: with one workgroup per CU and tiles of unequal length a second
// round evens them out (3945 tokens in six sequences, 12 + 2 heads: 113 us unsplit, 66 with
// two, 51 with three, 55 with four, joins 7 - 8 more; 8192 in four, 16 + 2 heads:
// 252 and 169; but 1259 in six, 20 + 5 heads, steps that are few: 36 unsplit, 26
// with two, 28 with three and four; 300 rows behind 3000 keys, 16 + 2 heads, tiles
// of equal length: 35 with two, 41 with five).  D = 64: 512 tokens in three sequences, 14 +
// 2 heads: 27 unsplit, 11 with eight; 4136 in three, 8 + 8 heads, as many tiles
// as places: 32 unsplit, 46 with two.
static int dkv_splits(int64_t batch, int64_t total_q, int64_t total_k, int64_t hq, int64_t hkv, int64_t d) {
  const int64_t full = (total_k + kBKeys - 1) / kBKeys, each = batch < total_k ? batch : total_k;
  const int64_t tiles = (full > each ? full : each) * hkv, group = hq / hkv;
  if (tiles == 0) return 1;
  const int64_t places = d == 128 ? 256 : 512;
  int64_t s = places / tiles;
  // steps of a tile of the mean prompt, whose rows see half of the keys
  const int64_t mean = (total_q / (batch > 0 ? batch : 1) + kBRows - 1) / kBRows * group / 2;
  if (d == 128 && total_q >= total_k && mean / 3 * tiles >= 2 * places) s = 2 * places / tiles;
  const int64_t steps = group * ((total_q + kBRows - 1) / kBRows);
  s = s > kMaxSplits ? kMaxSplits : s;
  s = s > steps ? steps : s;
  return s < 1 ? 1 : (int)s;
}

// workspace: -delta, -lse / scale ([hq][total_q] each), dO in bf16, and the
// partial sums of one pass after the other: dQ, then dK and dV
static size_t bwd_part_bytes(int64_t batch, int64_t total_q, int64_t total_k, int64_t hq, int64_t hkv, int64_t d) {
  const int q = fwd_split(batch, total_q, total_k, hq).splits, k = dkv_splits(batch, total_q, total_k, hq, hkv, d);
  const size_t nq = q > 1 ? (size_t)q * total_q * hq * d * 4 : 0, nk = k > 1 ? (size_t)k * 2 * total_k * hkv * d * 4 : 0;
  return nq > nk ? nq : nk;
}
size_t attn_bwd_ws_bytes(int64_t batch, int64_t total_q, int64_t total_k, int64_t hq, int64_t hkv, int64_t d) {
  return 2 * bwd_row_bytes(total_q, hq) + align256((size_t)total_q * hq * d * 2) +
         bwd_part_bytes(batch, total_q, total_k, hq, hkv, d);
}

template <int D>
static hipError_t bwd_launch(const AttnBwdArgs& a, hipStream_t s) {
  char* ws = static_cast<char*>(a.ws);
  float* delta = reinterpret_cast<float*>(ws);
  float* shift = reinterpret_cast<float*>(ws + bwd_row_bytes(a.total_q, a.hq));
  uint16_t* copy = reinterpret_cast<uint16_t*>(ws + 2 * bwd_row_bytes(a.total_q, a.hq));
  float* part = reinterpret_cast<float*>(ws + 2 * bwd_row_bytes(a.total_q, a.hq) +
                                         align256((size_t)a.total_q * a.hq * D * 2));
  const uint16_t* dO = a.do_f32 ? copy : static_cast<const uint16_t*>(a.dO);
  if (a.total_q > 0) {
    const int64_t items = most_tiles(a.total_q, a.batch, kQRows);
    const FwdSplit p = fwd_split(a.batch, a.total_q, a.total_k, a.hq);
    attn_dq_kernel<D><<<dim3((unsigned)placed_blocks(items, a.hkv, a.hq / a.hkv * p.splits)), 256, 0, s>>>(
        a, (int)items, p.splits, p.target, copy, delta, shift, part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.splits > 1) {
      attn_dq_join_kernel<D><<<dim3((unsigned)(items * a.hq * (kQRows / (256 / (D / 4))))), 256, 0, s>>>(
          a, p.splits, p.target, part);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  if (a.total_k > 0) {
    const int splits = dkv_splits(a.batch, a.total_q, a.total_k, a.hq, a.hkv, D);
    const int64_t items = most_tiles(a.total_k, a.batch, kBKeys);
    attn_dkv_kernel<D><<<dim3((unsigned)placed_blocks(items, a.hkv, splits)), 512, 0, s>>>(a, (int)items, dO, delta, shift,
                                                                                       splits, part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (splits > 1) attn_dkv_join_kernel<D><<<dim3((unsigned)(items * a.hkv * (2 * kBKeys * (D / 8) / 256))), 256, 0, s>>>(a, splits, part);
  }
  return hipGetLastError();
}
hipError_t launch_attn_bwd(const AttnBwdArgs& a, int64_t d, hipStream_t s) {
  return d == 128 ? bwd_launch<128>(a, s) : bwd_launch<64>(a, s);
}

}  // namespace bl
