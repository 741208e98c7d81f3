// attn_cache.hip -- attention of new or drafted tokens over a paged cache.
#include <type_traits>

#include "attn.h"
#include "launch.h"

namespace bl {

namespace {
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInf = __builtin_huge_valf();
constexpr int kCols = 32;     // rows of Q (drafted tokens x heads of a group) in a matrix operand
constexpr int kGranule = 16;  // rows that share a page
}  // namespace

// ---------------------------------------------------------------------
// The call is bound by reading K and V once.  A unit is one sequence's
// key/value head with the rows of Q of its group's heads and all drafted
// tokens, which share the tiles that are read; its keys are cut into tiles.
// All units' tiles in a row are dealt in equal contiguous ranges to as many
// workgroups as fill the chip, whatever the lengths: a unit that is cut
// between workgroups leaves partial results (O, max, sum) in the workspace,
// which the second kernel joins in a fixed order.  The ranges follow from
// the lengths in device memory, so a captured graph may be replayed with
// others.  Starting on a unit (its pages, the first loads, the join) takes as
// long as several tiles, so each counts as kStart tiles more than it has:
// otherwise a workgroup with a handful of short sequences ends last (eight
// sequences of 50 - 400 rows: 15.6 us without, 11.7 with six; eight drafted trees
// behind 24 - 9001 rows: 66 and 42 us).
//
// Up to 32 rows (decoding): each of the four wavefronts takes a quarter of a
// unit's tiles of 32 keys and streams them through two LDS stages of its
// own; no barriers, one tile in flight while one is computed (64 KiB per CU).
// The wavefronts meet in LDS at the end of the unit or the range.  64
// sequences of 1024 - 8192 rows, 16 + 2 heads of 128 (301 MB): 64.5 us with the
// join, 4.7 TB/s, as fast as a large copy; one of 32768 rows, 20 + 5 heads
// (84 MB): 22.6 us, of which the join takes 4.5 and the first loads 3.
//
// More rows (drafted trees): up to 128 in a unit, 32 for each wavefront, on
// common tiles of 64 keys in four stages, three of them in flight.  One
// workgroup per CU with deep prefetch rather than two with less: a range that
// is half as long leaves twice as many partial results, which at 96 rows are
// a quarter of the bytes of K and V already.  (The first form with several
// blocks of 32 rows per wavefront ran out of registers; with units of 32 rows
// it read K and V once for each: 24 tokens of 4 heads behind 38,000 rows took
// 113 us, with two stages and two workgroups per CU 41 us of this kernel, now
// 35.)  Those 38,000 rows in eight sequences, 5 key/value heads (99 MB), are
// 40 us with the join: 3 to find the ranges, 7 to start on one or two units
// each, 14 for a workgroup's 12 tiles (their loads alone 10), 6 to write 13 MB
// of partial results and 6.5 to join them.  (The next tile's scores among the
// exponentials, as in the forward, gained nothing here.)
// ---------------------------------------------------------------------
template <int D, bool WIDE>
struct CacheForm {
  static constexpr int kRows = WIDE ? 64 : 32;           // keys of a tile
  static constexpr int kBytes = kRows * 2 * D;           // K or V of a tile
  static constexpr int kStage = WIDE ? 2 * kBytes : 8 * kBytes;  // of the workgroup
  static constexpr int kBlocks = D == 128 ? 256 : 512;   // workgroups: 1 or 2 per CU by LDS
  static constexpr int kUnitBlocks = WIDE ? 4 : 1;       // blocks of 32 rows of Q in a unit, at most
  static constexpr int kStart = 6;                       // tiles that starting on a unit counts as
  static constexpr int kRowF32 = D + 4;                  // padded row when wavefronts are joined
};
template <int D>
constexpr int kPart = kCols * D + 2 * kCols;  // floats of a partial result of one block

__shared__ __attribute__((aligned(1024))) char g_c128_st0[CacheForm<128, false>::kStage];
__shared__ __attribute__((aligned(1024))) char g_c128_st1[CacheForm<128, false>::kStage];
__shared__ __attribute__((aligned(1024))) char g_c64_st0[CacheForm<64, false>::kStage];
__shared__ __attribute__((aligned(1024))) char g_c64_st1[CacheForm<64, false>::kStage];
__shared__ float g_cred[9 * 32];  // [4][32] maxima, [4][32] sums, [32] joined sums
__shared__ __attribute__((aligned(1024))) char g_d128_st0[CacheForm<128, true>::kStage];
__shared__ __attribute__((aligned(1024))) char g_d128_st1[CacheForm<128, true>::kStage];
__shared__ __attribute__((aligned(1024))) char g_d128_st2[CacheForm<128, true>::kStage];
__shared__ __attribute__((aligned(1024))) char g_d128_st3[CacheForm<128, true>::kStage];
__shared__ __attribute__((aligned(1024))) char g_d64_st0[CacheForm<64, true>::kStage];
__shared__ __attribute__((aligned(1024))) char g_d64_st1[CacheForm<64, true>::kStage];
__shared__ __attribute__((aligned(1024))) char g_d64_st2[CacheForm<64, true>::kStage];
__shared__ __attribute__((aligned(1024))) char g_d64_st3[CacheForm<64, true>::kStage];
template <int D, bool WIDE, int P>
__device__ __forceinline__ lds_char* cache_stage() {
  if constexpr (WIDE) {
    if constexpr (D == 128) return (lds_char*)(P == 0 ? g_d128_st0 : P == 1 ? g_d128_st1 : P == 2 ? g_d128_st2 : g_d128_st3);
    else return (lds_char*)(P == 0 ? g_d64_st0 : P == 1 ? g_d64_st1 : P == 2 ? g_d64_st2 : g_d64_st3);
  } else {
    if constexpr (D == 128) return (lds_char*)(P == 0 ? g_c128_st0 : g_c128_st1);
    else return (lds_char*)(P == 0 ? g_c64_st0 : g_c64_st1);
  }
}

__device__ __forceinline__ int cache_len(const AttnCacheArgs& a, int b) {
  const int64_t most = a.max_pages * a.page;
  const int n = ld_global(a.lens + b);
  return n < 0 ? 0 : n > most ? (int)most : n;
}
template <class F>
__device__ __forceinline__ int cache_tiles(int len) {
  return (len + F::kRows - 1) / F::kRows;
}
template <class F>
__device__ __forceinline__ int unit_places(int tiles) {  // in the row of all units' tiles
  return tiles > 0 ? tiles + F::kStart : 0;
}
// blocks of 32 rows of Q, and those of a unit: as few units as possible,
// then equal ones
__host__ __device__ inline int col_blocks(int rows) { return (rows + kCols - 1) / kCols; }
template <class F>
__host__ __device__ inline int unit_blocks(int blocks) {
  const int units = (blocks + F::kUnitBlocks - 1) / F::kUnitBlocks;
  return (blocks + units - 1) / units;
}
template <class F>
__device__ __forceinline__ int range_tiles(int all) {
  return (all + F::kBlocks - 1) / F::kBlocks;
}

// This workgroup's range [g0, g1) of tiles, and the sequence that holds g0
// with the tiles before it; b = batch if there is nothing to do.
struct CacheRange {
  int g0, g1, b, before;
};
template <class F>
__device__ __forceinline__ CacheRange cache_range(const AttnCacheArgs& a, int units) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int i = lane; i < a.batch; i += 64) n += unit_places<F>(cache_tiles<F>(cache_len(a, i)));
  const int all = wave_sum_i(n) * units;
  const int per = range_tiles<F>(all);
  CacheRange r{0, 0, a.batch, 0};
  if ((int64_t)blockIdx.x * per >= all) return r;
  r.g0 = blockIdx.x * per;
  r.g1 = per < all - r.g0 ? r.g0 + per : all;
  int before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const int c = b0 + lane < a.batch ? unit_places<F>(cache_tiles<F>(cache_len(a, b0 + lane))) * units : 0;
    const int incl = before + wave_scan_i(c);
    const unsigned long long hit = __ballot(incl > r.g0);
    if (hit) {
      const int l = __builtin_amdgcn_readfirstlane(__ffsll(hit) - 1);
      r.b = b0 + l;
      r.before = __builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(c, l);
      break;
    }
    before = __builtin_amdgcn_readlane(incl, 63);
  }
  return r;
}

// Where a sequence's granules lie: lane i holds granule base + i's place in
// the cache (in granules), or -1 where there are no rows
struct Lookup {
  int where, base;
  __device__ __forceinline__ void at(const AttnCacheArgs& a, int b, int len, int first, int lane) {
    const int gpp = (int)(a.page / kGranule), g = first + lane;
    base = first;
    where = -1;
    if ((int64_t)g * kGranule < len) {
      const int p = g / gpp;
      const int32_t page = ld_global(a.pages + (int64_t)b * a.max_pages + p);
      if (page >= 0 && page < a.pool) where = page * gpp + (g - p * gpp);
    }
  }
};

// A granule's rows of K and V into LDS; zeros past `left` rows and where
// there are none
template <int D>
struct GranuleDma {
  typedef Tile<D> T;
  static constexpr int kDma = kGranule / T::kDmaRows;  // instructions of K or V
  uint32_t off[kDma];
  int stride;
  __device__ __forceinline__ GranuleDma(int lane, int st) : stride(st) {
#pragma unroll
    for (int i = 0; i < kDma; ++i)
      off[i] = dma_offset<D>(lane, i % T::kVariants, st) + (uint32_t)(i * T::kDmaRows * st * 2);
  }
  __device__ __forceinline__ void issue(lds_char* k, lds_char* v, const uint16_t* kp, const uint16_t* vp, int at,
                                        int left) const {
    const int n = at < 0 ? 0 : left < kGranule ? left : kGranule;
    const int64_t row = (int64_t)(at < 0 ? 0 : at) * kGranule;
    const uint32_t bytes = n > 0 ? (uint32_t)((n - 1) * stride * 2 + 2 * D) : 0;
    const __amdgpu_buffer_rsrc_t rk = rows_rsrc(kp + row * stride, bytes), rv = rows_rsrc(vp + row * stride, bytes);
#pragma unroll
    for (int i = 0; i < kDma; ++i) lds_load16(rk, k + 1024 * i, off[i]);
#pragma unroll
    for (int i = 0; i < kDma; ++i) lds_load16(rv, v + 1024 * i, off[i]);
  }
};

// A lane's row of Q in a unit: drafted token i, head h of the group
template <int D>
struct QRow {
  int token, head;
  bool in;
  uint64_t seen;  // drafted tokens it sees
  // (rows past the last take that one's: a condition around the loads would
  // make each wait for the one before it)
  __device__ __forceinline__ void load(const AttnCacheArgs& a, v8bf* f, int b, int kvh, int c, int lane) {
    const int group = a.hq / a.hkv, rows = group * a.draft;
    in = c < rows;
    c = in ? c : rows - 1;
    token = c / group;
    head = c - token * group;
    const uint16_t* q = a.Q + ((int64_t)b * a.draft + token) * a.q_stride + (int64_t)(kvh * group + head) * D;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      f[s] = __builtin_bit_cast(v8bf, ld_global(reinterpret_cast<const u32x4*>(q + 16 * s + 8 * (lane >> 5))));
    seen = a.tree ? ld_global(a.tree + (int64_t)b * a.draft + token) : (2ull << token) - 1;
    if (a.draft < 64) seen &= (1ull << a.draft) - 1;
  }
  // scores of 32 keys: row0 is the first one's place behind the context
  // (below 0: in it), gone: which of the two granules hold no rows
  __device__ __forceinline__ void mask(v16f& s, int row0, int gone, int lane) const {
    uint32_t v = 0;  // bit r: key r is seen
    if (row0 <= -32) v = ~0u;
    else if (row0 < 0) v = (uint32_t)(seen << -row0) | ((1u << -row0) - 1);
    else if (row0 < 64) v = (uint32_t)(seen >> row0);
    v &= (gone & 1 ? 0u : 0xffffu) | (gone & 2 ? 0u : 0xffff0000u);
    v >>= 4 * (lane >> 5);
#pragma unroll
    for (int j = 0; j < 16; ++j) s[j] = v & (1u << (8 * (j >> 2) + (j & 3))) ? s[j] : -kInf;
  }
};

// running maximum, sum and O^T of 32 rows of Q; see attn_fwd_kernel
template <int D>
struct Running {
  v16f o[D / 32];
  float m, l;
  bool steep;  // some row's |m scale log2 e| > kSteep (the same in all lanes)
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[d][j] = 0.f;
    m = -kInf;
    l = 0.f;
    steep = false;
  }
  __device__ __forceinline__ void raise(float mx, float sl) {
    mx = half_join(mx, [](float p, float q) { return fmaxf(p, q); });
    if (__ballot((mx - m) * sl > 8.f)) {
      const float mn = fmaxf(m, mx);
      const float f = exp2_hw((m - (mn == -kInf ? 0.f : mn)) * sl);
      m = mn;
      steep = __ballot((mn == -kInf ? 0.f : fabsf(mn)) * sl > kSteep) != 0;
      l *= f;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[d][j] *= f;
    }
  }
  __device__ __forceinline__ void weigh(v16f& s, float sl) {
    const float z = m == -kInf ? 0.f : m, ms = steep ? 0.f : z * sl;
    if (steep) {
#pragma unroll
      for (int j = 0; j < 16; ++j) s[j] -= z;
    }
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      s[j] = exp2_hw(fmaf(s[j], sl, -ms));
      sum += s[j];
    }
    l += sum;
  }
};
__device__ __forceinline__ float most16(const v16f& s) {
  float mx = s[0];
#pragma unroll
  for (int j = 1; j < 16; ++j) mx = fmaxf(mx, s[j]);
  return mx;
}

template <int D>
__global__ __launch_bounds__(256, D == 128 ? 1 : 2) void attn_cache_kernel(AttnCacheArgs a) {
  typedef CacheForm<D, false> F;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.hq / a.hkv, rows = group * a.draft, units = a.hkv;
  const CacheRange range = cache_range<F>(a, units);
  int b = range.b, before = range.before;
  const int stride = a.hkv * D;
  const GranuleDma<D> dma(lane, stride);
  const uint32_t mine = wave * 2 * F::kBytes;  // this wavefront's part of a stage
  uint32_t ka[D / 16];
  TrAddr va[D / 32];
#pragma unroll
  for (int s = 0; s < D / 16; ++s) ka[s] = mine + a_addr<D>(lane, s);
#pragma unroll
  for (int t = 0; t < D / 32; ++t) va[t] = tr_addrs<D>(lane, t, mine + F::kBytes);
  const float sl = a.scale * kLog2e;

  for (int g = range.g0; g < range.g1 && b < a.batch;) {
    // key/value head kvh of sequence b, tiles [t0, t1) of it
    const int len = __builtin_amdgcn_readfirstlane(cache_len(a, b));
    const int nt = cache_tiles<F>(len), places = unit_places<F>(nt);
    if (g - before >= places * units) {  // next sequence (also past empty ones)
      before += places * units;
      ++b;
      continue;
    }
    const int kvh = (g - before) / places, t0 = (g - before) - kvh * places;
    const int end = g - t0 + places;  // where the next unit starts
    if (t0 >= nt) {
      g = end;
      continue;
    }
    const int t1 = nt - t0 < range.g1 - g ? nt : t0 + range.g1 - g;
    const int ctx = len - a.draft;  // rows before the drafted ones (may be below 0)
    const uint16_t* kp = a.K + (int64_t)kvh * D;
    const uint16_t* vp = a.V + (int64_t)kvh * D;
    // this wavefront's tiles [w0, w1)
    const int quarter = (t1 - t0 + 3) / 4;
    const int w0 = t0 + wave * quarter < t1 ? t0 + wave * quarter : t1;
    const int w1 = w0 + quarter < t1 ? w0 + quarter : t1;
    Lookup pages;
    // loads tile t; returns which of its two granules hold no rows
    auto issue = [&](lds_char* st, int t) {
      int missing = 0;
      __builtin_amdgcn_s_waitcnt(0xc07f);  // LDS reads of this stage have returned
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = __builtin_amdgcn_readlane(pages.where, 2 * t - pages.base + h);
        missing |= at < 0 ? 1 << h : 0;
        lds_char* to = st + mine + h * kGranule * Tile<D>::kRowBytes;
        dma.issue(to, to + F::kBytes, kp, vp, at, len - (t * F::kRows + h * kGranule));
      }
      return missing;
    };
    int gone = 0;  // granules of the tile being computed that hold no rows
    if (w0 < w1) {
      pages.at(a, b, len, 2 * w0, lane);
      gone = issue(cache_stage<D, false, 0>(), w0);
    }
    v8bf qf[D / 16];
    QRow<D> q;
    q.load(a, qf, b, kvh, lane & 31, lane);
    Running<D> acc;
    acc.clear();

    auto step = [&](auto stage, int t) {
      constexpr int P = decltype(stage)::value;
      int next = 0;
      if (t + 1 < w1) {
        if (2 * (t + 1) - pages.base >= 64) pages.at(a, b, len, 2 * (t + 1), lane);
        next = issue(cache_stage<D, false, P ^ 1>(), t + 1);
        wait_dma<4 * GranuleDma<D>::kDma>();
      } else {
        wait_dma<0>();
      }
      asm volatile("" ::: "memory");
      const lds_char* st = cache_stage<D, false, P>();
      v16f s;
#pragma unroll
      for (int j = 0; j < 16; ++j) s[j] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) s = mfma32(lds_read8(st + ka[k]), qf[k], s);
      if (gone | (t * F::kRows + F::kRows > ctx)) q.mask(s, t * F::kRows - ctx, gone, lane);
      acc.raise(most16(s), sl);
      acc.weigh(s, sl);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const v8bf p = operand_of(s, k);
#pragma unroll
        for (int d = 0; d < D / 32; ++d) acc.o[d] = mfma32(tr_operand<D>(st, va[d], 16 * k), p, acc.o[d]);
      }
      gone = next;
    };

    for (int t = w0; t < w1;) {
      step(std::integral_constant<int, 0>{}, t);
      if (++t == w1) break;
      step(std::integral_constant<int, 1>{}, t);
      ++t;
    }
    acc.l = half_join(acc.l, [](float x, float y) { return x + y; });

    // join the wavefronts: common maximum, then the scaled sums through LDS
    // (each wavefront's stages are its own until here), wavefronts 0, 1 in
    // stage 0 and 2, 3 in stage 1
    typedef __attribute__((address_space(3))) v4f lds_v4f;
    static_assert(2 * kCols * F::kRowF32 * 4 <= F::kStage, "two joined blocks in a stage");
    __syncthreads();
    if (lane < 32) {
      g_cred[32 * wave + lane] = acc.m;
      g_cred[128 + 32 * wave + lane] = acc.l;
    }
    __syncthreads();
    float mt = -kInf, lt = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) mt = fmaxf(mt, g_cred[32 * w + (lane & 31)]);
    const float mz = mt == -kInf ? 0.f : mt;
#pragma unroll
    for (int w = 0; w < 4; ++w) lt += g_cred[128 + 32 * w + (lane & 31)] * exp2_hw((g_cred[32 * w + (lane & 31)] - mz) * sl);
    const float f = exp2_hw((acc.m - mz) * sl);
    lds_char* const box =
        (wave < 2 ? cache_stage<D, false, 0>() : cache_stage<D, false, 1>()) + (wave & 1) * kCols * F::kRowF32 * 4;
    if (q.in) {
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<lds_v4f*>(box + ((lane & 31) * F::kRowF32 + 32 * d + 8 * e + 4 * (lane >> 5)) * 4) =
              v4f{acc.o[d][4 * e] * f, acc.o[d][4 * e + 1] * f, acc.o[d][4 * e + 2] * f, acc.o[d][4 * e + 3] * f};
    }
    const bool whole = t0 == 0 && t1 == nt;
    float* part = static_cast<float*>(a.ws) + ((int64_t)blockIdx.x * 2 + (g == range.g0 ? 0 : 1)) * kPart<D>;
    if (threadIdx.x < 32) {
      g_cred[256 + lane] = lt;
      if (!whole && q.in) {
        st_global(part + kCols * D + lane, mt);
        st_global(part + kCols * D + kCols + lane, lt);
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < rows * (D / 4); e += 256) {
      const int r = e / (D / 4), d = 4 * (e % (D / 4));
      const uint32_t at = (uint32_t)(r * F::kRowF32 + d) * 4, half = kCols * F::kRowF32 * 4;
      const v4f x0 = *reinterpret_cast<const lds_v4f*>(cache_stage<D, false, 0>() + at);
      const v4f x1 = *reinterpret_cast<const lds_v4f*>(cache_stage<D, false, 0>() + half + at);
      const v4f x2 = *reinterpret_cast<const lds_v4f*>(cache_stage<D, false, 1>() + at);
      const v4f x3 = *reinterpret_cast<const lds_v4f*>(cache_stage<D, false, 1>() + half + at);
      v4f y;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = (x0[i] + x1[i]) + (x2[i] + x3[i]);
      if (whole) {
        const float s = g_cred[256 + r];
        const float inv = s > 0.f ? 1.f / s : 0.f;
        const int i = r / group, h = r - i * group;
        st_global(reinterpret_cast<u32x2*>(a.O + (((int64_t)b * a.draft + i) * a.hq + kvh * group + h) * D + d),
                  u32x2{pk_bf16(y[0] * inv, y[1] * inv), pk_bf16(y[2] * inv, y[3] * inv)});
      } else {
        st_global(reinterpret_cast<v4f*>(part + r * D + d), y);
      }
    }
    __syncthreads();  // the stages are free again
    g = t1 == nt ? end : g + t1 - t0;
  }
}

template <int D>
__global__ __launch_bounds__(256, D == 128 ? 1 : 2) void attn_cache_wide_kernel(AttnCacheArgs a) {
  typedef CacheForm<D, true> F;
  typedef Tile<D> T;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.hq / a.hkv, blocks = col_blocks(group * a.draft), nc = unit_blocks<F>(blocks);
  const int cols = (blocks + nc - 1) / nc, units = a.hkv * cols;
  const CacheRange range = cache_range<F>(a, units);
  int b = range.b, before = range.before;
  const int stride = a.hkv * D;
  const GranuleDma<D> dma(lane, stride);
  uint32_t ka[D / 16];
  TrAddr va[D / 32];
#pragma unroll
  for (int s = 0; s < D / 16; ++s) ka[s] = a_addr<D>(lane, s);
#pragma unroll
  for (int t = 0; t < D / 32; ++t) va[t] = tr_addrs<D>(lane, t, F::kBytes);
  const float sl = a.scale * kLog2e;

  for (int g = range.g0; g < range.g1 && b < a.batch;) {
    // unit u of sequence b, tiles [t0, t1) of it
    const int len = __builtin_amdgcn_readfirstlane(cache_len(a, b));
    const int nt = cache_tiles<F>(len), places = unit_places<F>(nt);
    if (g - before >= places * units) {
      before += places * units;
      ++b;
      continue;
    }
    const int u = (g - before) / places, t0 = (g - before) - u * places;
    const int end = g - t0 + places;
    if (t0 >= nt) {
      g = end;
      continue;
    }
    const int t1 = nt - t0 < range.g1 - g ? nt : t0 + range.g1 - g;
    const int kvh = u / cols, block = (u - kvh * cols) * nc + wave;  // this wavefront's 32 rows of Q
    const bool busy = wave < nc && block < blocks;
    const int ctx = len - a.draft;
    const uint16_t* kp = a.K + (int64_t)kvh * D;
    const uint16_t* vp = a.V + (int64_t)kvh * D;
    Lookup pages;
    // this wavefront's granule of tile t (t1 and on: nothing is read, but as
    // many instructions are issued, so the waits below can count them);
    // returns which of the tile's four hold no rows
    auto issue = [&](auto stage, int t) {
      if (4 * t - pages.base >= 64) pages.at(a, b, len, 4 * t, lane);
      int missing = 0;
#pragma unroll
      for (int h = 0; h < 4; ++h)
        missing |= __builtin_amdgcn_readlane(pages.where, 4 * t - pages.base + h) < 0 ? 1 << h : 0;
      const int at = t < t1 ? __builtin_amdgcn_readlane(pages.where, 4 * t - pages.base + wave) : -1;
      lds_char* to = cache_stage<D, true, decltype(stage)::value>() + wave * kGranule * T::kRowBytes;
      dma.issue(to, to + F::kBytes, kp, vp, at, len - (t * F::kRows + wave * kGranule));
      return missing;
    };
    typedef std::integral_constant<int, 0> S0;
    typedef std::integral_constant<int, 1> S1;
    typedef std::integral_constant<int, 2> S2;
    typedef std::integral_constant<int, 3> S3;
    pages.at(a, b, len, 4 * t0, lane);
    // (before the tiles: loads return in order, and a wait for these rows would
    // be one for three tiles)
    v8bf qf[D / 16];
    QRow<D> q;
    q.load(a, qf, b, kvh, busy ? block * kCols + (lane & 31) : blocks * kCols, lane);
    int gone0 = issue(S0{}, t0), gone1 = issue(S1{}, t0 + 1), gone2 = issue(S2{}, t0 + 2);  // of the next three tiles
    Running<D> acc;
    acc.clear();

    auto step = [&](auto stage, auto last, int t) {
      constexpr int P = decltype(stage)::value;
      wait_dma<2 * 2 * GranuleDma<D>::kDma>();
      lds_barrier();
      const int now = gone0;
      gone0 = gone1;
      gone1 = gone2;
      gone2 = issue(last, t + 3);
      const lds_char* st = cache_stage<D, true, P>();
      v16f s[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) s[i][j] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) s[i] = mfma32(lds_read8(st + ka[k] + i * 32 * T::kRowBytes), qf[k], s[i]);
      if (now | (t * F::kRows + F::kRows > ctx)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) q.mask(s[i], t * F::kRows + 32 * i - ctx, now >> (2 * i), lane);
      }
      acc.raise(fmaxf(most16(s[0]), most16(s[1])), sl);
#pragma unroll
      for (int i = 0; i < 2; ++i) acc.weigh(s[i], sl);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const v8bf p = operand_of(s[k >> 1], k & 1);
#pragma unroll
        for (int d = 0; d < D / 32; ++d) acc.o[d] = mfma32(tr_operand<D>(st, va[d], 16 * k), p, acc.o[d]);
      }
    };
    // (leaving between the stages keeps one copy of each: with copies for the
    // last tiles the code no longer fitted the instruction cache)
    for (int t = t0;;) {
      step(S0{}, S3{}, t);
      if (++t == t1) break;
      step(S1{}, S0{}, t);
      if (++t == t1) break;
      step(S2{}, S1{}, t);
      if (++t == t1) break;
      step(S3{}, S2{}, t);
      if (++t == t1) break;
    }
    wait_dma<0>();
    acc.l = half_join(acc.l, [](float x, float y) { return x + y; });
    if (t0 == 0 && t1 == nt) {
      const float inv = acc.l > 0.f ? 1.f / acc.l : 0.f;
      uint16_t* out = a.O + (((int64_t)b * a.draft + q.token) * a.hq + kvh * group + q.head) * D;
      if (busy) store_row<D>(out, acc.o, inv, lane, q.in);
    } else if (q.in) {
      float* part = static_cast<float*>(a.ws) + (((int64_t)blockIdx.x * 2 + (g == range.g0 ? 0 : 1)) * nc + wave) * kPart<D>;
      if (lane < 32) {
        st_global(part + kCols * D + lane, acc.m);
        st_global(part + kCols * D + kCols + lane, acc.l);
      }
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          st_global(reinterpret_cast<v4f*>(part + (lane & 31) * D + 32 * d + 8 * e + 4 * (lane >> 5)),
                    v4f{acc.o[d][4 * e], acc.o[d][4 * e + 1], acc.o[d][4 * e + 2], acc.o[d][4 * e + 3]});
    }
    lds_barrier();  // the stages are free again (all reads have been used)
    g = t1 == nt ? end : g + t1 - t0;
  }
}

// Rows of units that were cut are joined from the partial results of their
// unit (weights 2^(m - max)) by groups of D/4 threads, each of which takes
// every so-manieth part with a running maximum; the groups then meet in a
// fixed order.  WIDE: one wavefront per row, 2 or 4 groups (many rows, few
// parts); otherwise one workgroup per row, 8 or 16 groups (few rows, many
// parts: one per workgroup that shared a long sequence).  Rows of empty
// sequences become zeros; rows that one workgroup had all of are written.
// Bound by latency (lengths, then parts, then the meeting): 4.4 - 6.4 us.
struct Joined {
  v4f acc;
  float m, l;
  __device__ __forceinline__ void add(const v4f& x, float mx, float lx, float sl) {
    const float mn = fmaxf(m, mx), z = mn == -kInf ? 0.f : mn;
    const float f = exp2_hw((m - z) * sl), w = exp2_hw((mx - z) * sl);
    m = mn;
    l = fmaf(lx, w, l * f);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(x[e], w, acc[e] * f);
  }
};
template <int D, bool WIDE>
__global__ __launch_bounds__(256) void attn_cache_join_kernel(AttnCacheArgs a) {
  typedef CacheForm<D, WIDE> F;
  constexpr int kGroups = (WIDE ? 64 : 256) / (D / 4);
  __shared__ v4f sum[WIDE ? 1 : kGroups][D / 4];
  __shared__ float msum[kGroups], lsum[kGroups];
  const int lane = threadIdx.x & 63, thread = WIDE ? lane : threadIdx.x;
  const int64_t row = WIDE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;  // (sequence, token, head)
  const int64_t bt = row / a.hq;
  const int head = (int)(row - bt * a.hq), b = (int)(bt / a.draft), i = (int)(bt - (int64_t)b * a.draft);
  if (b >= a.batch) return;
  const int group = a.hq / a.hkv, blocks = col_blocks(group * a.draft), nc = unit_blocks<F>(blocks);
  const int cols = (blocks + nc - 1) / nc, units = a.hkv * cols;
  const int kvh = head / group, c = i * group + head - kvh * group;
  const int nt = cache_tiles<F>(cache_len(a, b));
  int all = 0, before = 0;
  for (int s = lane; s < a.batch; s += 64) {
    const int n = unit_places<F>(cache_tiles<F>(cache_len(a, s)));
    all += n;
    before += s < b ? n : 0;
  }
  all = wave_sum_i(all) * units;
  before = wave_sum_i(before) * units;
  const int per = range_tiles<F>(all);
  const int s0 = before + (kvh * cols + c / (nc * kCols)) * unit_places<F>(nt), s1 = s0 + nt;  // the unit's tiles
  const int at = thread / (D / 4), d = thread % (D / 4);
  uint16_t* out = a.O + (bt * a.hq + head) * D;
  if (nt == 0) {
    if (at == 0) st_global(reinterpret_cast<u32x2*>(out) + d, u32x2{0u, 0u});
    return;
  }
  const int p0 = s0 / per, p1 = (s1 - 1) / per;
  if (p0 == p1) return;
  const float sl = a.scale * kLog2e;
  const int r = c % kCols;
  const float* ws = static_cast<const float*>(a.ws) + (int64_t)(c / kCols % nc) * kPart<D>;
  auto part = [&](int p) { return ws + ((int64_t)p * 2 + (p > p0 || s0 == p0 * per ? 0 : 1)) * nc * kPart<D>; };
  Joined y{v4f{0.f, 0.f, 0.f, 0.f}, -kInf, 0.f};
  for (int p = p0 + at; p <= p1; p += 4 * kGroups) {
    v4f x[4];
    float m[4], l[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool is = p + u * kGroups <= p1;
      const float* q = part(is ? p + u * kGroups : p);
      x[u] = ld_global(reinterpret_cast<const v4f*>(q + r * D) + d);
      m[u] = ld_global(q + kCols * D + r);
      l[u] = ld_global(q + kCols * D + kCols + r);
      m[u] = is ? m[u] : -kInf;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) y.add(x[u], m[u], l[u], sl);
  }
  if constexpr (WIDE) {
#pragma unroll
    for (int o = D / 4; o < 64; o <<= 1) {  // lower and upper halves, so every lane adds in the same order
      Joined x{v4f{__shfl_xor(y.acc[0], o, 64), __shfl_xor(y.acc[1], o, 64), __shfl_xor(y.acc[2], o, 64),
                   __shfl_xor(y.acc[3], o, 64)},
               __shfl_xor(y.m, o, 64), __shfl_xor(y.l, o, 64)};
      y.add(x.acc, x.m, x.l, sl);
    }
    if (at) return;
  } else {
    sum[at][d] = y.acc;
    if (d == 0) {
      msum[at] = y.m;
      lsum[at] = y.l;
    }
    __syncthreads();
    if (at) return;
#pragma unroll
    for (int g = 1; g < kGroups; ++g) y.add(sum[g][d], msum[g], lsum[g], sl);
  }
  const float inv = y.l > 0.f ? 1.f / y.l : 0.f;
  st_global(reinterpret_cast<u32x2*>(out) + d,
            u32x2{pk_bf16(y.acc[0] * inv, y.acc[1] * inv), pk_bf16(y.acc[2] * inv, y.acc[3] * inv)});
}

// ------------------------------------------------------------------- host
// workspace: two partial results per workgroup and block of the first kernel
template <int D>
static size_t cache_ws(int rows) {
  const int blocks = col_blocks(rows);
  if (blocks == 1) return (size_t)CacheForm<D, false>::kBlocks * 2 * kPart<D> * 4;
  return (size_t)CacheForm<D, true>::kBlocks * 2 * unit_blocks<CacheForm<D, true>>(blocks) * kPart<D> * 4;
}
size_t attn_cache_ws_bytes(int64_t, int64_t draft, int64_t hq, int64_t hkv, int64_t d) {
  const int rows = (int)(hq / hkv * draft);
  return d == 128 ? cache_ws<128>(rows) : cache_ws<64>(rows);
}

template <int D>
static hipError_t cache_launch(const AttnCacheArgs& a, hipStream_t s) {
  const int64_t rows = (int64_t)a.batch * a.draft * a.hq;
  const bool wide = a.hq / a.hkv * a.draft > kCols;
  if (wide) attn_cache_wide_kernel<D><<<dim3(CacheForm<D, true>::kBlocks), 256, 0, s>>>(a);
  else attn_cache_kernel<D><<<dim3(CacheForm<D, false>::kBlocks), 256, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (wide) attn_cache_join_kernel<D, true><<<dim3((unsigned)((rows + 3) / 4)), 256, 0, s>>>(a);
  else attn_cache_join_kernel<D, false><<<dim3((unsigned)rows), 256, 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_attn_cache(const AttnCacheArgs& a, int64_t d, hipStream_t s) {
  return d == 128 ? cache_launch<128>(a, s) : cache_launch<64>(a, s);
}

}  // namespace bl
