// norm.hip -- layer norm of rows (with or without centring), forward and
// backward with the sums over rows of the parameters' gradients, and 8-bit
// checkpoints of rows, which both directions take part in.
#include "ckpt.h"
#include "common.h"
#include "launch.h"

namespace bl {

// A row of n values is held by kThreads threads, kV runs of eight consecutive
// values each: run i of thread t is run i * kThreads + t of the row, so
// neighbouring threads read neighbouring 16 or 32 bytes.  The whole row stays in
// registers between its sums and its outputs: every input is read once.
template <int kThreads>
struct RowSums {
  static constexpr int kWaves = kThreads / 64;
  // sum over the row's threads (`wave`: this one's in the workgroup); `slot`: a
  // different one for each sum between two barriers that all of the workgroup passes
  __device__ static __forceinline__ float sum(float v, float (*red)[8], int slot, int wave) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
    if constexpr (kWaves > 1) {
      if ((threadIdx.x & 63) == 0) red[slot][wave] = v;
      __syncthreads();
      const int first = wave & ~(kWaves - 1);
      v = red[slot][first];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += red[slot][first + w];
    }
    return v;
  }
};

// 1 / sqrt(v), v the variance + eps; one that leaves binary32 gives NaN, not rows of
// zeros
__device__ __forceinline__ float rstd_of(float v) {
  return v < __builtin_inff() ? __builtin_amdgcn_rsqf(v) : __builtin_nanf("");
}
// Below kTinyVar squares lose bits or vanish, and v_rsq_f32 takes what is below 2^-126 for
// 0: such rows (values of 1e-12 and less, eps no larger than their squares) are squared
// once more, scaled by kTinyScale.  The smallest value's square is then 2^-106, and rows
// of 16384 below the limit stay below 2^127.
constexpr float kTinyVar = 0x1p-80f, kTinyScale = 0x1p96f;

// Forward.  Up to 2560 values a row is a wavefront's, four rows a workgroup, and the
// weights come from L2 behind the sums (kept in registers from the start they
// cost wavefronts: 4096 x 2560 binary32 with a checkpoint 18.6 us, so 16.4 us for 74
// MB).  Longer rows are 256 threads'; from 4097 to 12288 values a workgroup walks over
// rows with the weights and bias in registers, as many workgroups as the CUs hold: 2049 x
// 8960 bf16 17.4 us for 73 MB, 4.2 TB/s (a workgroup for each row, which reads 72 KB of
// parameters for its 18 KB: 20.3).  8192 x 6144 binary32 47.5 us (56.0).  Shorter rows
// gain nothing by it (8192 x 4096 bf16 22.9 us either way), and longer ones leave too
// few wavefronts (2048 x 16384 bf16 29.2 us without, 35.3 with).
constexpr int norm_walkers(int threads, int values) {  // workgroups, or 0 for one a row
  return threads < 256 || values < 3 || values > 6 ? 0 : values < 5 ? 768 : 512;
}
template <int T, int kThreads, int kV>
__global__ __launch_bounds__(256) void layernorm_kernel(NormArgs a) {
  constexpr int kRows = 256 / kThreads;  // rows of a workgroup
  constexpr bool kWalk = norm_walkers(kThreads, kV) > 0;
  __shared__ float red[4][8];
  const int tid = kRows > 1 ? threadIdx.x % kThreads : threadIdx.x, lane = threadIdx.x & 63;
  int64_t row = (int64_t)blockIdx.x * kRows + (kRows > 1 ? threadIdx.x / kThreads : 0);
  if (row >= a.rows) return;  // whole wavefronts, and no barrier follows where a workgroup has several rows
  Raw8<T> raw[kV];
  bool in[kV];
  const auto load = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int64_t e = 8 * ((int64_t)i * kThreads + tid);
      in[i] = e < a.n;
      raw[i].zero();
      if (in[i] && r < a.rows) raw[i].load(a.X, r * a.x_stride + e);
    }
  };
  load(row);
  Raw8<kRowF32> w[kWalk ? kV : 1], b[kWalk ? kV : 1];
  if (kWalk) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      if (in[i] && a.weight) w[kWalk ? i : 0].load(a.weight, 8 * ((int64_t)i * kThreads + tid));
      if (in[i] && a.bias) b[kWalk ? i : 0].load(a.bias, 8 * ((int64_t)i * kThreads + tid));
    }
  }
  const float inv_n = 1.f / (float)a.n;
  int slot = 0;
  do {
    float mean = 0.f;
    if (a.center) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += raw[i].get(j, 0.f);
      mean = RowSums<kThreads>::sum(s, red, slot, threadIdx.x >> 6) * inv_n;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < kV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = raw[i].get(j, 0.f) - mean;
        q = in[i] ? fmaf(d, d, q) : q;
      }
    const float v = RowSums<kThreads>::sum(q, red, slot + 1, threadIdx.x >> 6) * inv_n + a.eps;
    float rstd = rstd_of(v);
    if (v < kTinyVar) {  // the same for all of the row's threads
      q = 0.f;
#pragma unroll
      for (int i = 0; i < kV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = (raw[i].get(j, 0.f) - mean) * kTinyScale;
          q = in[i] ? fmaf(d, d, q) : q;
        }
      // (the mean's slot: everyone has read it before the barrier of the sum above)
      q = RowSums<kThreads>::sum(q, red, slot, threadIdx.x >> 6) * inv_n;
      rstd = rstd_of(q + a.eps * kTinyScale * kTinyScale) * kTinyScale;
    }
    slot ^= 2;  // a row's sums are read before the barriers of the next row's, which use the other slots
    if (tid == 0) {
      if (a.mean) st_global(a.mean + row, mean);
      if (a.rstd) st_global(a.rstd + row, rstd);
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int64_t e = 8 * ((int64_t)i * kThreads + tid);
      float x[8], y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = raw[i].get(j, 0.f);
      if (a.codes)
        ckpt_store8(x, in[i], lane, a.codes + row * a.n + e,
                    a.scales + row * ((a.n + kCkptBlock - 1) / kCkptBlock) + e / kCkptBlock);
      if (!in[i]) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = (x[j] - mean) * rstd;
      if (a.weight) {
        if (!kWalk) w[0].load(a.weight, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= w[kWalk ? i : 0].get(j, 0.f);
      }
      if (a.bias) {
        if (!kWalk) b[0].load(a.bias, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] += b[kWalk ? i : 0].get(j, 0.f);
      }
      store_row8(a.Y, a.y_type, row * a.n + e, y);
    }
    if (!kWalk) return;
    row += gridDim.x;
    load(row);
  } while (row < a.rows);
}

// Backward of rows: with n = (x - mean) rstd and a = w dy,
//   dx = rstd (a - mean(a) - n mean(a n)) (+ dR),  dw = sum dy n,  db = sum dy
// (no mean(a) without centring).  Each group of kThreads walks over rows and
// keeps its share of dw and db in registers; a workgroup's groups are joined in
// LDS in a fixed order, and each workgroup writes one row of partial sums, which
// norm_dw_kernel adds in binary64.  No atomics: reruns give the same bits.
// Bound by memory.  The sums take so many registers that two wavefronts fit a SIMD,
// so each keeps the next row's x and dy on their way while it sums and writes
// its row (with 32 values a thread there are no registers left for that).  The weights
// lie in LDS (from L2 for each row: 27.4 and 38.0 us below).  4096 x 2560, 8-bit x,
// bf16 dy, binary32 dR and dX: 25.7 us for 115 MB, 4.5 TB/s (one wavefront a row, 40
// values a lane, nothing ahead: 42.0); 2049 x 8960 bf16 with binary32 dy and bias: 36.4
// us, 4.0 TB/s (45.4).
template <int T, int D, int kThreads, int kV, bool kBias>
__global__ __launch_bounds__(512) void layernorm_bwd_kernel(NormBwdArgs a) {
  constexpr int kRows = 512 / kThreads;  // rows of a workgroup at a time
  __shared__ float red[4][8];
  constexpr bool kAhead = kV < 4;
  __shared__ __attribute__((aligned(16))) f32x4_t weight[kThreads * kV * 2];
  for (int c = threadIdx.x; c < kThreads * kV * 2; c += 512) {
    f32x4_t v{1.f, 1.f, 1.f, 1.f};
    if (a.weight && 4 * c < a.n) v = ld_global(reinterpret_cast<const f32x4_t*>(a.weight) + c);
    weight[c] = v;
  }
  __syncthreads();
  const int tid = kRows > 1 ? threadIdx.x % kThreads : threadIdx.x;
  const int group = kRows > 1 ? threadIdx.x / kThreads : 0, wave = threadIdx.x >> 6;
  const float inv_n = 1.f / (float)a.n;
  const int64_t blocks = (a.n + kCkptBlock - 1) / kCkptBlock, stride = (int64_t)gridDim.x * kRows;
  float gw[kV][8], gb[kBias ? kV : 1][8];
#pragma unroll
  for (int i = 0; i < kV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) gw[i][j] = gb[kBias ? i : 0][j] = 0.f;
  Raw8<T> rx[kV];
  Raw8<D> rd[kV];
  float xs[kV], mean = 0.f, rstd = 0.f;
  // (a group without a row takes part in the barriers, with zeros)
  const auto load = [&](int64_t row) {
    const bool live = row < a.rows;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int64_t e = 8 * ((int64_t)i * kThreads + tid);
      rx[i].zero();
      rd[i].zero();
      xs[i] = 0.f;
      if (live && e < a.n) {
        rx[i].load(a.X, row * a.x_stride + e);
        rd[i].load(a.dY, row * a.n + e);
        if (T == kRowQ8) xs[i] = ld_global(a.x_scales + row * blocks + e / kCkptBlock);
      }
    }
    mean = live && a.mean ? ld_global(a.mean + row) : 0.f;
    rstd = live ? ld_global(a.rstd + row) : 0.f;
  };
  int slot = 0;
  if (kAhead) load((int64_t)blockIdx.x * kRows + group);
  for (int64_t base = (int64_t)blockIdx.x * kRows; base < a.rows; base += stride) {
    const int64_t row = base + group;
    const bool live = row < a.rows;
    if (!kAhead) load(row);
    Raw8<kRowF32> rr[kV];  // binary32 dR, or bf16 in the first half
    if (a.dR) {
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int64_t e = 8 * ((int64_t)i * kThreads + tid);
        if (!live || e >= a.n) continue;
        if (a.dx_type == kRowF32) {
          rr[i].load(a.dR, row * a.n + e);
        } else {
          Raw8<kRowBf16> h;
          h.load(a.dR, row * a.n + e);
          rr[i].a = __builtin_bit_cast(f32x4_t, h.a);
        }
      }
    }
    float sa = 0.f, sn = 0.f;
    float x[kV][8], d[kV][8];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int64_t e = 8 * ((int64_t)i * kThreads + tid);
      const Raw8<kRowF32> w{weight[e / 4], weight[e / 4 + 1]};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // threads past the row hold dy = 0, and n = 0
        const float n = e < a.n ? (rx[i].get(j, xs[i]) - mean) * rstd : 0.f;
        const float dy = rd[i].get(j, 0.f);
        gw[i][j] = fmaf(dy, n, gw[i][j]);
        if (kBias) gb[kBias ? i : 0][j] += dy;
        x[i][j] = n;
        d[i][j] = dy * w.get(j, 0.f);
        sa += d[i][j];
        sn = fmaf(d[i][j], n, sn);
      }
    }
    const float r = rstd;
    const bool centred = a.mean != nullptr;
    if (kAhead) load(row + stride);
    sn = RowSums<kThreads>::sum(sn, red, slot, wave) * inv_n;
    sa = centred ? RowSums<kThreads>::sum(sa, red, slot + 1, wave) * inv_n : 0.f;
    slot ^= 2;  // a row's sums are read before the barriers of the next row's, which use the other slots
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int64_t e = 8 * ((int64_t)i * kThreads + tid);
      if (!live || e >= a.n) continue;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = r * fmaf(-x[i][j], sn, d[i][j] - sa);
      if (a.dR) {
        const u32x4 h = __builtin_bit_cast(u32x4, rr[i].a);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          y[j] += a.dx_type == kRowF32 ? rr[i].get(j, 0.f) : (j & 1) ? bf16_hi(h[j >> 1]) : bf16_lo(h[j >> 1]);
      }
      store_row8(a.dX, a.dx_type, row * a.n + e, y);
    }
  }
  if (!a.part) return;
  // one row of partial sums for each workgroup: dw's n, and with kBias db's behind them
  float* out = a.part + (int64_t)blockIdx.x * (kBias ? 2 : 1) * a.n;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int64_t e = 8 * ((int64_t)i * kThreads + tid);
      if (e >= a.n) continue;
      store_row8(out, kRowF32, e, gw[i]);
      if (kBias) store_row8(out, kRowF32, a.n + e, gb[kBias ? i : 0]);
    }
  } else {
    // one run at a time: the groups' values beside each other, then summed in order
    __shared__ __attribute__((aligned(16))) float join[kRows][kThreads * 8];
#pragma unroll
    for (int s = 0; s < (kBias ? 2 : 1); ++s)
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<f32x4_t*>(&join[group][tid * 8 + 4 * h]) =
              s ? f32x4_t{gb[kBias ? i : 0][4 * h], gb[kBias ? i : 0][4 * h + 1], gb[kBias ? i : 0][4 * h + 2],
                          gb[kBias ? i : 0][4 * h + 3]}
                : f32x4_t{gw[i][4 * h], gw[i][4 * h + 1], gw[i][4 * h + 2], gw[i][4 * h + 3]};
        __syncthreads();
        for (int c = threadIdx.x; c < kThreads * 8; c += 512) {
          const int64_t e = 8 * (int64_t)i * kThreads + c;
          if (e >= a.n) continue;
          float v = join[0][c];
#pragma unroll
          for (int g = 1; g < kRows; ++g) v += join[g][c];
          st_global(out + s * a.n + e, v);
        }
      }
  }
}

// dw and db: sums of the workgroups' rows of partials.  A workgroup takes 32 columns,
// its 32 groups of 8 threads (4 columns each) every 32nd row, all of them asked
// for at once; joined in LDS, all in binary64 and in a fixed order (256 rows of
// 2560: 4.7 us, latency).
constexpr int kPartsEach = kNormParts / 32;
__global__ __launch_bounds__(256) void norm_dw_kernel(const float* __restrict__ part, int rows, int64_t n, int64_t cols,
                                                     float* __restrict__ dw, float* __restrict__ db) {
  __shared__ double red[32][33];
  const int c4 = 4 * (threadIdx.x & 7), g = threadIdx.x >> 3;
  const int64_t c = (int64_t)blockIdx.x * 32 + c4;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  if (c < cols) {
    f32x4_t v[kPartsEach];
#pragma unroll
    for (int u = 0; u < kPartsEach; ++u) {
      v[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (g + 32 * u < rows) v[u] = ld_global(reinterpret_cast<const f32x4_t*>(part + (int64_t)(g + 32 * u) * cols + c));
    }
#pragma unroll
    for (int u = 0; u < kPartsEach; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] += (double)v[u][q];
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) red[g][c4 + q] = s[q];
  __syncthreads();
  if (threadIdx.x < 32) {
    const int64_t e = (int64_t)blockIdx.x * 32 + threadIdx.x;
    double t = red[0][threadIdx.x];
#pragma unroll
    for (int h = 1; h < 32; ++h) t += red[h][threadIdx.x];
    float* out = e < n ? dw : db;
    if (e < cols && out) st_global(out + (e < n ? e : e - n), (float)t);
  }
}

__global__ void norm_zero_kernel(float* __restrict__ dw, float* __restrict__ db, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  if (dw) st_global(dw + i, 0.f);
  if (db) st_global(db + i, 0.f);
}

// ------------------------------------------------------- 8-bit checkpoints
// Eight lanes hold a block of 64 values, eight each, as the norm's rows do.  Bound by
// memory: 8192 x 6912 binary32, 286 MB each way, packed in 66 us, 4.3 TB/s, and
// unpacked in 56, 5.1 TB/s.
template <int T>
__global__ __launch_bounds__(256) void ckpt_pack_kernel(const void* __restrict__ X, int64_t x_stride, int64_t units,
                                                        int64_t n, int8_t* __restrict__ codes,
                                                        float* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int64_t blocks = (n + kCkptBlock - 1) / kCkptBlock;
  const int64_t u = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
  const int64_t row = u / blocks, b = u - row * blocks, e = b * kCkptBlock + 8 * (lane & 7);
  const bool in = u < units && e < n;
  Raw8<T> raw;
  raw.zero();
  if (in) raw.load(X, row * x_stride + e);
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = raw.get(j, 0.f);
  ckpt_store8(x, in, lane, codes + row * n + e, scales + u);
}

__global__ __launch_bounds__(256) void ckpt_unpack_kernel(const int8_t* __restrict__ codes,
                                                          const float* __restrict__ scales, int64_t units, int64_t n,
                                                          void* __restrict__ Y, int y_type) {
  const int64_t blocks = (n + kCkptBlock - 1) / kCkptBlock;
  const int64_t u = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
  const int64_t row = u / blocks, b = u - row * blocks, e = b * kCkptBlock + 8 * (threadIdx.x & 7);
  if (u >= units || e >= n) return;
  Raw8<kRowQ8> raw;
  raw.load(codes, row * n + e);
  const float s = ld_global(scales + u);
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = raw.get(j, s);
  store_row8(Y, y_type, row * n + e, y);
}

// ------------------------------------------------------------------ host
// Threads of a row, forward: one wavefront up to 2560 values (five runs of eight a
// lane, no barriers), then four.  Backward: as many as leave a thread 24 values,
// whose sums and whose next row's inputs fit its registers.
template <int T, int kThreads, int kV>
static hipError_t norm_launch(const NormArgs& a, hipStream_t s) {
  constexpr int kRows = 256 / kThreads;
  int64_t blocks = (a.rows + kRows - 1) / kRows;
  constexpr int kWalkers = norm_walkers(kThreads, kV);
  if (kWalkers && blocks > kWalkers) blocks = kWalkers;
  layernorm_kernel<T, kThreads, kV><<<(unsigned)blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <int T>
static hipError_t norm_pick(const NormArgs& a, hipStream_t s) {
  const int64_t runs = (a.n + 7) / 8;
  if (runs <= 64) return norm_launch<T, 64, 1>(a, s);
  if (runs <= 128) return norm_launch<T, 64, 2>(a, s);
  if (runs <= 192) return norm_launch<T, 64, 3>(a, s);
  if (runs <= 256) return norm_launch<T, 64, 4>(a, s);
  if (runs <= 320) return norm_launch<T, 64, 5>(a, s);
  if (runs <= 512) return norm_launch<T, 256, 2>(a, s);
  if (runs <= 768) return norm_launch<T, 256, 3>(a, s);
  if (runs <= 1024) return norm_launch<T, 256, 4>(a, s);
  if (runs <= 1280) return norm_launch<T, 256, 5>(a, s);
  if (runs <= 1536) return norm_launch<T, 256, 6>(a, s);
  return norm_launch<T, 256, 8>(a, s);
}
hipError_t launch_layernorm(const NormArgs& a, int x_type, hipStream_t s) {
  return x_type == kRowF32 ? norm_pick<kRowF32>(a, s) : norm_pick<kRowBf16>(a, s);
}

template <int T, int D, int kThreads, int kV>
static hipError_t norm_bwd_launch(const NormBwdArgs& a, hipStream_t s) {
  constexpr int kRows = 512 / kThreads;
  int64_t blocks = (a.rows + kRows - 1) / kRows;
  if (blocks > kNormParts) blocks = kNormParts;
  if (a.dbias) layernorm_bwd_kernel<T, D, kThreads, kV, true><<<(unsigned)blocks, 512, 0, s>>>(a);
  else layernorm_bwd_kernel<T, D, kThreads, kV, false><<<(unsigned)blocks, 512, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.part) return e;
  const int64_t cols = a.dbias ? 2 * a.n : a.n;
  norm_dw_kernel<<<(unsigned)((cols + 31) / 32), 256, 0, s>>>(a.part, (int)blocks, a.n, cols, a.dweight, a.dbias);
  return hipGetLastError();
}
template <int T, int D>
static hipError_t norm_bwd_pick(const NormBwdArgs& a, hipStream_t s) {
  const int64_t runs = (a.n + 7) / 8;
  if (runs <= 64) return norm_bwd_launch<T, D, 64, 1>(a, s);
  if (runs <= 128) return norm_bwd_launch<T, D, 64, 2>(a, s);
  if (runs <= 192) return norm_bwd_launch<T, D, 64, 3>(a, s);
  if (runs <= 384) return norm_bwd_launch<T, D, 128, 3>(a, s);
  if (runs <= 768) return norm_bwd_launch<T, D, 256, 3>(a, s);
  if (runs <= 1536) return norm_bwd_launch<T, D, 512, 3>(a, s);
  return norm_bwd_launch<T, D, 512, 4>(a, s);
}
template <int T>
static hipError_t norm_bwd_pick_dy(const NormBwdArgs& a, hipStream_t s) {
  return a.dy_type == kRowF32 ? norm_bwd_pick<T, kRowF32>(a, s) : norm_bwd_pick<T, kRowBf16>(a, s);
}
hipError_t launch_layernorm_bwd(const NormBwdArgs& a, int x_type, hipStream_t s) {
  if (a.rows == 0) {
    norm_zero_kernel<<<(unsigned)((a.n + 255) / 256), 256, 0, s>>>(a.dweight, a.dbias, a.n);
    return hipGetLastError();
  }
  if (x_type == kRowF32) return norm_bwd_pick_dy<kRowF32>(a, s);
  return x_type == kRowBf16 ? norm_bwd_pick_dy<kRowBf16>(a, s) : norm_bwd_pick_dy<kRowQ8>(a, s);
}

hipError_t launch_ckpt_pack(const void* X, int x_type, int64_t x_stride, int64_t rows, int64_t n, int8_t* codes,
                            float* scales, hipStream_t s) {
  const int64_t units = rows * ((n + kCkptBlock - 1) / kCkptBlock);
  const unsigned grid = (unsigned)((units + 31) / 32);
  if (x_type == kRowF32) ckpt_pack_kernel<kRowF32><<<grid, 256, 0, s>>>(X, x_stride, units, n, codes, scales);
  else ckpt_pack_kernel<kRowBf16><<<grid, 256, 0, s>>>(X, x_stride, units, n, codes, scales);
  return hipGetLastError();
}
hipError_t launch_ckpt_unpack(const int8_t* codes, const float* scales, int64_t rows, int64_t n, void* Y, int y_type,
                              hipStream_t s) {
  const int64_t units = rows * ((n + kCkptBlock - 1) / kCkptBlock);
  ckpt_unpack_kernel<<<(unsigned)((units + 31) / 32), 256, 0, s>>>(codes, scales, units, n, Y, y_type);
  return hipGetLastError();
}

}  // namespace bl
