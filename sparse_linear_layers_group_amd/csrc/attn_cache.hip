// attn_cache.hip -- attention of new or drafted tokens over a paged cache.
#include <type_traits>

#include "attn.h"
#include "launch.h"

namespace bl {

namespace {
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInf = __builtin_huge_valf();
constexpr int kCols = 32;      // rows of Q (drafted tokens x heads of a group) of one unit
constexpr int kCRows = 32;     // key rows of a tile
constexpr int kGranule = 16;   // rows that share a page
constexpr int kMinTiles = 4;   // tiles of a workgroup's range, at least: one per wavefront
}  // namespace

// ---------------------------------------------------------------------
// The call is bound by reading K and V once.  A unit is one sequence's
// key/value head with up to 32 rows of Q (all heads of the group and all
// drafted tokens share the tiles that are read); its keys are cut into
// tiles of 32 rows.  All units' tiles in a row are dealt in equal
// contiguous ranges to as many workgroups as fill the chip, whatever the
// lengths: a unit that is cut between workgroups leaves partial results
// (O, max, sum) in the workspace, which the second kernel joins in a fixed
// order.  The ranges follow from the lengths in device memory, so a
// captured graph may be replayed with others.
//
// Within a range each of the four wavefronts takes a quarter of a unit's
// tiles and streams them through two LDS stages of its own: no barriers,
// one tile in flight while one is computed (64 KiB per CU).
// ---------------------------------------------------------------------
template <int D>
struct CacheTile {
  static constexpr int kBytes = kCRows * 2 * D;          // K or V of a tile
  static constexpr int kStage = 2 * kBytes;              // both
  static constexpr int kDma = 2 * kCRows / Tile<D>::kDmaRows;  // DMA instructions of a stage
  static constexpr int kRowF32 = D + 4;                  // padded row when wavefronts are joined
  static constexpr int kBlocks = D == 128 ? 256 : 512;   // workgroups: 1 or 2 per CU by LDS
  static constexpr int kPart = kCols * D + 2 * kCols;    // floats of a partial result
};
__shared__ __attribute__((aligned(1024))) char g_c128_st0[4 * CacheTile<128>::kStage + 2048];
__shared__ __attribute__((aligned(1024))) char g_c128_st1[4 * CacheTile<128>::kStage];
__shared__ __attribute__((aligned(1024))) char g_c64_st0[4 * CacheTile<64>::kStage + 2048];
__shared__ __attribute__((aligned(1024))) char g_c64_st1[4 * CacheTile<64>::kStage];
template <int D, int P>
__device__ __forceinline__ lds_char* cache_stage() {
  if constexpr (D == 128) return (lds_char*)(P == 0 ? g_c128_st0 : g_c128_st1);
  else return (lds_char*)(P == 0 ? g_c64_st0 : g_c64_st1);
}

__device__ __forceinline__ int cache_len(const AttnCacheArgs& a, int b) {
  const int64_t most = a.max_pages * a.page;
  const int n = ld_global(a.lens + b);
  return n < 0 ? 0 : n > most ? (int)most : n;
}
__device__ __forceinline__ int cache_tiles(int len) { return (len + kCRows - 1) / kCRows; }

// tiles of all units before sequence b (b = batch: all of them)
__device__ __forceinline__ int tiles_before(const AttnCacheArgs& a, int units, int b, int lane) {
  int n = 0;
  for (int i = lane; i < b; i += 64) n += cache_tiles(cache_len(a, i));
  return wave_sum_i(n) * units;
}
__device__ __forceinline__ int range_tiles(int all, int blocks) {
  const int per = (all + blocks - 1) / blocks;
  return per < kMinTiles ? kMinTiles : per;
}

template <int D>
__global__ __launch_bounds__(256, D == 128 ? 1 : 2) void attn_cache_kernel(AttnCacheArgs a) {
  typedef Tile<D> T;
  typedef CacheTile<D> C;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.hq / a.hkv, rows = group * a.draft;
  const int cols = (rows + kCols - 1) / kCols, units = a.hkv * cols;
  const int all = __builtin_amdgcn_readfirstlane(tiles_before(a, units, a.batch, lane));
  const int per = range_tiles(all, C::kBlocks);
  if ((int64_t)blockIdx.x * per >= all) return;
  const int g0 = blockIdx.x * per, g1 = g0 + per < all ? g0 + per : all;

  // the sequence that holds tile g0
  int b = a.batch, before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 64) {
    const int n = b0 + lane < a.batch ? cache_tiles(cache_len(a, b0 + lane)) * units : 0;
    const int incl = before + wave_scan_i(n, lane);
    const unsigned long long hit = __ballot(incl > g0);
    if (hit) {
      const int l = __ffsll(hit) - 1;
      b = b0 + l;
      before = __shfl(incl, l, 64) - __shfl(n, l, 64);
      break;
    }
    before = __shfl(incl, 63, 64);
  }
  b = __builtin_amdgcn_readfirstlane(b);
  before = __builtin_amdgcn_readfirstlane(before);

  const int stride = a.hkv * D;
  uint32_t off[4];  // of the granule's DMA instructions (D = 64 uses two)
  constexpr int kPerGranule = kGranule / T::kDmaRows;
#pragma unroll
  for (int i = 0; i < kPerGranule; ++i)
    off[i] = dma_offset<D>(lane, i % T::kVariants, stride) + (uint32_t)(i * T::kDmaRows * stride * 2);
  uint32_t ka[D / 16];
  TrAddr va[D / 32];
#pragma unroll
  for (int s = 0; s < D / 16; ++s) ka[s] = wave * C::kStage + a_addr<D>(lane, s);
#pragma unroll
  for (int t = 0; t < D / 32; ++t) va[t] = tr_addrs<D>(lane, t, wave * C::kStage + C::kBytes);
  const float sl = a.scale * kLog2e;
  const int gpp = (int)(a.page / kGranule);

  for (int g = g0; g < g1 && b < a.batch;) {
    // unit u of sequence b, tiles [t0, t1) of it
    const int len = __builtin_amdgcn_readfirstlane(cache_len(a, b));
    const int nt = cache_tiles(len);
    if (g - before >= nt * units) {  // next sequence (also past empty ones)
      before += nt * units;
      ++b;
      continue;
    }
    const int u = (g - before) / nt, t0 = (g - before) - u * nt;
    const int t1 = nt - t0 < g1 - g ? nt : t0 + g1 - g;
    const int kvh = u / cols, c0 = (u - kvh * cols) * kCols;
    // this lane's row of Q: drafted token i, head h of the group
    const int c = c0 + (lane & 31), ci = c / group, ch = c - ci * group;
    const bool in = c < rows;
    v8bf qf[D / 16];
    {
      const uint16_t* q = a.Q + ((int64_t)b * a.draft + ci) * a.q_stride + (int64_t)(kvh * group + ch) * D;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        u32x4 v = u32x4{0u, 0u, 0u, 0u};
        if (in) v = ld_global(reinterpret_cast<const u32x4*>(q + 16 * s + 8 * (lane >> 5)));
        qf[s] = __builtin_bit_cast(v8bf, v);
      }
    }
    const int ctx = len - a.draft;  // rows before the drafted ones (may be below 0)
    uint64_t seen = 0;              // drafted tokens this row sees
    if (in) seen = a.tree ? ld_global(a.tree + (int64_t)b * a.draft + ci) : (2ull << ci) - 1;
    if (a.draft < 64) seen &= (1ull << a.draft) - 1;

    const uint16_t* kp = a.K + (int64_t)kvh * D;
    const uint16_t* vp = a.V + (int64_t)kvh * D;
    // this wavefront's tiles [w0, w1); lane i holds where granule base + i
    // lies in the cache (in granules), or -1
    const int quarter = (t1 - t0 + 3) / 4;
    const int w0 = t0 + wave * quarter < t1 ? t0 + wave * quarter : t1;
    const int w1 = w0 + quarter < t1 ? w0 + quarter : t1;
    int where = -1, base = 0;
    auto look_up = [&](int t) {
      base = 2 * t;
      const int gi = base + lane;
      where = -1;
      if ((int64_t)gi * kGranule < len) {
        const int p = gi / gpp;
        const int32_t page = ld_global(a.pages + (int64_t)b * a.max_pages + p);
        if (page >= 0 && page < a.pool) where = page * gpp + (gi - p * gpp);
      }
    };
    // loads tile t; returns which of its two granules hold no rows
    auto issue = [&](lds_char* st, int t) {
      int missing = 0;
      __builtin_amdgcn_s_waitcnt(0xc07f);  // LDS reads of this stage have returned
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = __builtin_amdgcn_readlane(where, 2 * t - base + h);
        const int left = len - (t * kCRows + h * kGranule);
        const int n = at < 0 ? 0 : left < kGranule ? left : kGranule;
        missing |= at < 0 ? 1 << h : 0;
        const int64_t row = (int64_t)(at < 0 ? 0 : at) * kGranule;
        const uint32_t bytes = n > 0 ? (uint32_t)((n - 1) * stride * 2 + 2 * D) : 0;
        const __amdgpu_buffer_rsrc_t rk = rows_rsrc(kp + row * stride, bytes), rv = rows_rsrc(vp + row * stride, bytes);
        lds_char* dst = st + wave * C::kStage + h * kGranule * T::kRowBytes;
#pragma unroll
        for (int i = 0; i < kPerGranule; ++i) lds_load16(rk, dst + 1024 * i, off[i]);
#pragma unroll
        for (int i = 0; i < kPerGranule; ++i) lds_load16(rv, dst + C::kBytes + 1024 * i, off[i]);
      }
      return missing;
    };

    v16f o[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[d][j] = 0.f;
    float m = -kInf, l = 0.f;
    int gone = 0;  // granules of the tile being computed that hold no rows

    auto step = [&](auto stage, int t) {
      constexpr int P = decltype(stage)::value;
      int next = 0;
      if (t + 1 < w1) {
        if (2 * (t + 1) - base >= 64) look_up(t + 1);
        next = issue(cache_stage<D, P ^ 1>(), t + 1);
        wait_dma<C::kDma>();
      } else {
        wait_dma<0>();
      }
      asm volatile("" ::: "memory");
      const lds_char* st = cache_stage<D, P>();
      v16f s;
#pragma unroll
      for (int j = 0; j < 16; ++j) s[j] = 0.f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) s = mfma32(lds_read8(st + ka[k]), qf[k], s);
      if (gone | (t * kCRows + kCRows > ctx)) {
        const int x = 4 * (lane >> 5);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int r = 8 * (j >> 2) + (j & 3) + x;        // row of the tile
          const int e = t * kCRows + r - ctx;              // drafted token it is, below 0: context
          const bool v = (e < 0 || (e < 64 && (seen >> (e & 63) & 1))) && !(gone >> (j >> 3) & 1);
          s[j] = v ? s[j] : -kInf;
        }
      }
      float mx = s[0];
#pragma unroll
      for (int j = 1; j < 16; ++j) mx = fmaxf(mx, s[j]);
      mx = half_join(mx, [](float p, float q) { return fmaxf(p, q); });
      if (__ballot((mx - m) * sl > 8.f)) {
        const float mn = fmaxf(m, mx);
        const float f = exp2_hw((m - (mn == -kInf ? 0.f : mn)) * sl);
        m = mn;
        l *= f;
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
          for (int j = 0; j < 16; ++j) o[d][j] *= f;
      }
      const float ms = (m == -kInf ? 0.f : m) * sl;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        s[j] = exp2_hw(fmaf(s[j], sl, -ms));
        sum += s[j];
      }
      l += sum;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const v8bf p = operand_of(s, k);
#pragma unroll
        for (int d = 0; d < D / 32; ++d) o[d] = mfma32(tr_operand<D>(st, va[d], 16 * k), p, o[d]);
      }
      gone = next;
    };

    if (w0 < w1) {
      look_up(w0);
      gone = issue(cache_stage<D, 0>(), w0);
    }
    int t = w0;
    for (; t + 1 < w1; t += 2) {
      step(std::integral_constant<int, 0>{}, t);
      step(std::integral_constant<int, 1>{}, t + 1);
    }
    if (t < w1) step(std::integral_constant<int, 0>{}, t);
    l = half_join(l, [](float p, float q) { return p + q; });

    // join the wavefronts: common maximum, then the scaled sums through LDS
    // (each wavefront's stages are its own until here)
    lds_char* const red = cache_stage<D, 0>() + 4 * C::kStage;  // [4][32] maxima, [4][32] sums, [32] joined sums
    typedef __attribute__((address_space(3))) float lds_float;
    typedef __attribute__((address_space(3))) v4f lds_v4f;
    __syncthreads();
    if (lane < 32) {
      reinterpret_cast<lds_float*>(red)[32 * wave + lane] = m;
      reinterpret_cast<lds_float*>(red)[128 + 32 * wave + lane] = l;
    }
    __syncthreads();
    float mt = -kInf, lt = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) mt = fmaxf(mt, reinterpret_cast<const lds_float*>(red)[32 * w + (lane & 31)]);
    const float mz = mt == -kInf ? 0.f : mt;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      lt += reinterpret_cast<const lds_float*>(red)[128 + 32 * w + (lane & 31)] *
            exp2_hw((reinterpret_cast<const lds_float*>(red)[32 * w + (lane & 31)] - mz) * sl);
    const float f = exp2_hw((m - mz) * sl);
    // wavefronts 0, 1 in stage 0 and 2, 3 in stage 1 (a stage holds two
    // padded binary32 copies of a 32-row result)
    lds_char* const mine = (wave < 2 ? cache_stage<D, 0>() : cache_stage<D, 1>()) + (wave & 1) * kCols * C::kRowF32 * 4;
    if (in) {
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<lds_v4f*>(mine + ((lane & 31) * C::kRowF32 + 32 * d + 8 * q + 4 * (lane >> 5)) * 4) =
              v4f{o[d][4 * q] * f, o[d][4 * q + 1] * f, o[d][4 * q + 2] * f, o[d][4 * q + 3] * f};
    }
    const bool whole = t0 == 0 && t1 == nt;
    float* part = static_cast<float*>(a.ws) + ((int64_t)blockIdx.x * 2 + (g == g0 ? 0 : 1)) * C::kPart;
    if (threadIdx.x < 32) {
      reinterpret_cast<lds_float*>(red)[256 + lane] = lt;
      if (!whole && in) {
        st_global(part + kCols * D + lane, mt);
        st_global(part + kCols * D + kCols + lane, lt);
      }
    }
    __syncthreads();
    const int used = rows - c0 < kCols ? rows - c0 : kCols;
    for (int e = threadIdx.x; e < used * (D / 4); e += 256) {
      const int r = e / (D / 4), d = 4 * (e % (D / 4));
      const uint32_t at = (uint32_t)(r * C::kRowF32 + d) * 4;
      const uint32_t half = kCols * C::kRowF32 * 4;
      const v4f x0 = *reinterpret_cast<const lds_v4f*>(cache_stage<D, 0>() + at);
      const v4f x1 = *reinterpret_cast<const lds_v4f*>(cache_stage<D, 0>() + half + at);
      const v4f x2 = *reinterpret_cast<const lds_v4f*>(cache_stage<D, 1>() + at);
      const v4f x3 = *reinterpret_cast<const lds_v4f*>(cache_stage<D, 1>() + half + at);
      v4f y;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = (x0[i] + x1[i]) + (x2[i] + x3[i]);
      if (whole) {
        const float s = reinterpret_cast<const lds_float*>(red)[256 + r];
        const float inv = s > 0.f ? 1.f / s : 0.f;
        const int cc = c0 + r, i = cc / group, h = cc - i * group;
        st_global(reinterpret_cast<u32x2*>(a.O + (((int64_t)b * a.draft + i) * a.hq + kvh * group + h) * D + d),
                  u32x2{pk_bf16(y[0] * inv, y[1] * inv), pk_bf16(y[2] * inv, y[3] * inv)});
      } else {
        st_global(reinterpret_cast<v4f*>(part + r * D + d), y);
      }
    }
    __syncthreads();  // the stages are free again
    g += t1 - t0;
  }
}

// Rows of units that were cut: one wavefront per row of Q joins the partial
// results of its unit, workgroup after workgroup (weights 2^(m - max)), and
// writes the row; rows of empty sequences become zeros.
template <int D>
__global__ __launch_bounds__(256) void attn_cache_join_kernel(AttnCacheArgs a) {
  typedef CacheTile<D> C;
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);  // (sequence, drafted token, head)
  const int64_t bt = row / a.hq;
  const int head = (int)(row - bt * a.hq), b = (int)(bt / a.draft), i = (int)(bt - (int64_t)b * a.draft);
  if (b >= a.batch) return;
  const int group = a.hq / a.hkv, rows = group * a.draft;
  const int cols = (rows + kCols - 1) / kCols, units = a.hkv * cols;
  const int kvh = head / group, c = i * group + head - kvh * group;
  const int all = tiles_before(a, units, a.batch, lane), before = tiles_before(a, units, b, lane);
  const int per = range_tiles(all, C::kBlocks);
  const int nt = cache_tiles(cache_len(a, b));
  const int s0 = before + (kvh * cols + c / kCols) * nt, s1 = s0 + nt;  // the unit's tiles
  typedef float vec __attribute__((ext_vector_type(D / 64)));
  vec acc;
#pragma unroll
  for (int e = 0; e < D / 64; ++e) acc[e] = 0.f;
  float inv = 0.f;
  if (nt > 0) {
    const int p0 = s0 / per, p1 = (s1 - 1) / per;
    if (p0 == p1) return;  // one workgroup had all of it
    const float sl = a.scale * kLog2e;
    const float* ws = static_cast<const float*>(a.ws);
    const int r = c % kCols;
    auto part = [&](int p) { return ws + ((int64_t)p * 2 + (p > p0 || s0 == p0 * per ? 0 : 1)) * C::kPart; };
    float mt = -kInf;
    for (int p = p0 + lane; p <= p1; p += 64) mt = fmaxf(mt, ld_global(part(p) + kCols * D + r));
    mt = wave_max(mt);
    const float mz = mt == -kInf ? 0.f : mt;
    float lt = 0.f;
    for (int q = p0; q <= p1; q += 64) {
      float w = 0.f;
      if (q + lane <= p1) {
        w = exp2_hw((ld_global(part(q + lane) + kCols * D + r) - mz) * sl);
        lt = fmaf(ld_global(part(q + lane) + kCols * D + kCols + r), w, lt);
      }
      const int n = p1 - q + 1 < 64 ? p1 - q + 1 : 64;
      for (int p = 0; p < n; ++p) {
        const vec x = ld_global(reinterpret_cast<const vec*>(part(q + p) + r * D) + lane);
        const float f = __shfl(w, p, 64);
#pragma unroll
        for (int e = 0; e < D / 64; ++e) acc[e] = fmaf(x[e], f, acc[e]);
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) lt += __shfl_xor(lt, o, 64);
    inv = lt > 0.f ? 1.f / lt : 0.f;
  }
  uint16_t* out = a.O + (bt * a.hq + head) * D;
  if constexpr (D == 128) st_global(reinterpret_cast<uint32_t*>(out) + lane, pk_bf16(acc[0] * inv, acc[1] * inv));
  else st_global(out + lane, (uint16_t)pk_bf16(acc[0] * inv, 0.f));
}

// ------------------------------------------------------------------- host
// workspace: two partial results per workgroup of the first kernel
size_t attn_cache_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t d) {
  return d == 128 ? (size_t)CacheTile<128>::kBlocks * 2 * CacheTile<128>::kPart * 4
                  : (size_t)CacheTile<64>::kBlocks * 2 * CacheTile<64>::kPart * 4;
}

template <int D>
static hipError_t cache_launch(const AttnCacheArgs& a, hipStream_t s) {
  attn_cache_kernel<D><<<dim3(CacheTile<D>::kBlocks), 256, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t rows = (int64_t)a.batch * a.draft * a.hq;
  attn_cache_join_kernel<D><<<dim3((unsigned)((rows + 3) / 4)), 256, 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_attn_cache(const AttnCacheArgs& a, int64_t d, hipStream_t s) {
  return d == 128 ? cache_launch<128>(a, s) : cache_launch<64>(a, s);
}

}  // namespace bl
