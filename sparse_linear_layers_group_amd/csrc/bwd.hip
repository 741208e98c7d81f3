// bwd.hip -- dual straight-through backward of BitLinear on gfx950.
//
// Sparse-BitNet article §三 and §六: the gradient passes straight through
// the ternary rounding and the N:M sparsification, and a masked weight
// still receives its gradient.
//   dX[t, c] = gamma * sum_r dY[t, r] * code[r, c]     (through the masked
//              ternary weights the forward used)
//   dW[r, c] = sum_t dY[t, r] * s_t * x_q[t, c]        (dense)
// Both are one bf16 "NT" product C[m, n] = alpha * sum_k A[m, k] B[n, k]
// on v_mfma_f32_16x16x32_bf16 with binary32 accumulation, whose operands
// both run along the contraction index in memory:
//   dX: A = dY [tokens x n_out] as given, B = codes^T [k x n_out];
//   dW: A = (dY * s)^T [n_out x tokens], B = x_q^T [k x tokens].
// Prep kernels write the operands that are not in that form into the
// workspace: the codes decoded from the packed layout and transposed
// (exact in bf16), bf16(dY * s_t) transposed (rounded once), and x_q
// transposed (exact).  Every conversion happens once per element, so the
// product kernel is a plain copy-to-LDS and MFMA loop.
#include "bwd_group.h"
#include "bitlinear.h"
#include "common.h"
#include "glu.h"
#include "glu_gate.h"
#include "launch.h"

#include <algorithm>
#include <atomic>
#include <utility>
#include <vector>

#include <type_traits>

namespace bl {

// ------------------------------------------------------------- prep
// All operand conversions of one backward call run in one launch: a list
// of tasks (one matrix each), every workgroup of 256 threads takes one job
// of one task.  Jobs of a dY or x_q task are 64 x 64 transposes through
// LDS; jobs of a codes task are four packed superblocks, one per
// wavefront, transposed in registers.

// bf16 codes of one half-group from its 8-bit key: entry key * 2 + half
// holds positions 0..3 as two bf16 pairs (the int8 codes of half_codes
// with 0x01 -> +1.0 and 0xff -> -1.0, both exact)
struct HalfBf16Table {
  uint32_t v[1024];
};
constexpr uint32_t code_to_bf16(uint32_t byte) {
  return byte == 0u ? 0u : (byte == 1u ? 0x3f80u : 0xbf80u);
}
constexpr HalfBf16Table make_half_bf16_table() {
  HalfBf16Table t{};
  for (uint32_t e = 0; e < 512; ++e) {
    const uint32_t c = half_codes(e >> 1, e & 1u);
    t.v[2 * e] = code_to_bf16(c & 0xffu) | (code_to_bf16((c >> 8) & 0xffu) << 16);
    t.v[2 * e + 1] = code_to_bf16((c >> 16) & 0xffu) | (code_to_bf16(c >> 24) << 16);
  }
  return t;
}
__device__ constexpr HalfBf16Table kHalfBf16Table = make_half_bf16_table();
static_assert(make_half_bf16_table().v[2 * (2 * 0x1f + 0)] == 0x3f80bf80u,
              "low half, bitmap 1111, sign of nonzero 0: -1.0 then +1.0");

// the place of (row, c) in an operand that lies in tiles, or in rows `pitch` apart
__device__ __forceinline__ int64_t operand_at(int64_t row, int64_t c, int64_t pitch, bool tiled) {
  return tiled ? tiled_at(row, c, pitch) : row * pitch + c;
}

enum PrepKind : int32_t { kPrepCodes = 0, kPrepDys = 1, kPrepXq = 2 };

// One matrix of a prep launch.
//   codes: src = packed codes, rows = k blocks per strip, cols = strips,
//          pitch = np (rows of codes^T); jobs = ceil(superblocks / 4)
//   dys:   src = dY, scale = s_t, rows = tokens, cols = n_out, pitch = tp
//   xq:    src = x_q, rows = tokens, cols = k, pitch = tp
// dY and x_q jobs are (64-token block fastest, 64-column block) tiles.
struct PrepTask {
  const void* src;
  const float* scale;
  uint16_t* out;
  int64_t rows, cols, pitch;
  int32_t kind, jobs;
};
constexpr int kMaxPrep = 16;
struct PrepSet {
  PrepTask t[kMaxPrep];
  int32_t n;
};

// 64 x 64 transposes through LDS.  Source rows are the contraction index
// of the product (tokens); each thread loads 16 bytes of a source row and
// writes 16 bytes (8 consecutive source rows) of a destination row.
constexpr int kTP = 66;  // LDS pitch (bf16) of the 64 x 64 transpose tile

// dYsT[r][t] = bf16(dY[t][r] * s_t) for t < tokens, 0 for tokens <= t < tp
__device__ __forceinline__ void prep_dys_tile(const uint16_t* __restrict__ dY,
                                              const float* __restrict__ scale, int64_t tokens,
                                              int64_t n_out, int64_t tp, uint16_t* __restrict__ out,
                                              int64_t t0, int64_t r0, uint16_t* tile, int tid) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int q = tid + 256 * p, t = q >> 3, r8 = 8 * (q & 7);
    const int64_t tt = t0 + t;
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    float s = 0.f;
    if (tt < tokens && r0 + r8 < n_out) {  // n_out % 8 == 0: a run is all in or all out
      v = ld_global(reinterpret_cast<const u32x4*>(dY + tt * n_out + r0 + r8));
      s = scale[tt];
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
      tile[t * kTP + r8 + e] = f32_to_bf16_rne(x * s);
    }
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int q = tid + 256 * p, r = q >> 3, t8 = 8 * (q & 7);
    if (r0 + r >= n_out) continue;
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = (uint32_t)tile[(t8 + 2 * e) * kTP + r] | ((uint32_t)tile[(t8 + 2 * e + 1) * kTP + r] << 16);
    st_global(reinterpret_cast<u32x4*>(out + (r0 + r) * tp + t0 + t8), u32x4{o[0], o[1], o[2], o[3]});
  }
}

// xbT[c][t] = bf16(x_q[t][c]) (exact) for t < tokens, 0 up to tp
__device__ __forceinline__ void prep_xq_tile(const int8_t* __restrict__ xq, int64_t tokens, int64_t k,
                                             int64_t tp, uint16_t* __restrict__ out, int64_t t0,
                                             int64_t c0, uint16_t* tile, int tid, bool tiled) {
  {
    const int t = tid >> 2, c16 = 16 * (tid & 3);
    const int64_t tt = t0 + t;
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    if (tt < tokens) v = ld_global(reinterpret_cast<const u32x4*>(xq + tt * k + c0 + c16));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int8_t b = (int8_t)((w[e >> 2] >> (8 * (e & 3))) & 0xffu);
      tile[t * kTP + c16 + e] = f32_to_bf16_rne((float)b);
    }
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int q = tid + 256 * p, c = q >> 3, t8 = 8 * (q & 7);
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = (uint32_t)tile[(t8 + 2 * e) * kTP + c] | ((uint32_t)tile[(t8 + 2 * e + 1) * kTP + c] << 16);
    st_global(reinterpret_cast<u32x4*>(out + operand_at(c0 + c, t0 + t8, tp, tiled)), u32x4{o[0], o[1], o[2], o[3]});
  }
}

// Lane exchanges inside groups of 8 lanes (data-parallel primitives: the
// partner's register value, lane j reading lane j ^ 1, j ^ 2 or j ^ 4)
__device__ __forceinline__ uint32_t lane_xor1(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, false);  // quad_perm [1,0,3,2]
}
__device__ __forceinline__ uint32_t lane_xor2(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, false);  // quad_perm [2,3,0,1]
}
__device__ __forceinline__ uint32_t lane_xor4(uint32_t v) {
  // lanes 0-3 and 8-11 of each row of 16 read lane + 4 (row_shl:4), lanes
  // 4-7 and 12-15 read lane - 4 (row_shr:4)
  const int a = __builtin_amdgcn_update_dpp(0, (int)v, 0x104, 0xf, 0x5, false);
  return (uint32_t)__builtin_amdgcn_update_dpp(a, (int)v, 0x114, 0xf, 0xa, false);
}
__device__ __forceinline__ uint32_t byte_perm(uint32_t hi, uint32_t lo, uint32_t sel) {
  return __builtin_amdgcn_perm(hi, lo, sel);
}

// 8 x 8 transpose of bf16 values across the 8 lanes j = lane & 7 of a
// group: in d[m], lane j holds elements 2m, 2m+1 of row j; out o[m], lane
// j holds element j of rows 2m, 2m+1.  Three exchange stages, each with
// the partner at lane distance 1, 2, 4.
__device__ __forceinline__ void transpose8_bf16(const uint32_t (&d)[4], uint32_t (&o)[4], int lane) {
  const int j = lane & 7;
  // stage 1: lane j holds rows (j & ~1, +1) of elements 2m + (j & 1)
  const uint32_t sel = (j & 1) ? 0x03020706u : 0x05040100u;
  uint32_t x[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) x[m] = byte_perm(lane_xor1(d[m]), d[m], sel);
  // stage 2: lane j holds rows (j & ~3) .. +3 of elements 2m + (j & 1),
  // m = b and b + 2 with b = bit 1 of j
  const bool b = (j >> 1) & 1;
  const uint32_t r0 = lane_xor2(b ? x[0] : x[1]), r1 = lane_xor2(b ? x[2] : x[3]);
  const uint32_t k0 = b ? x[1] : x[0], k1 = b ? x[3] : x[2];
  const uint32_t y[4] = {b ? r0 : k0, b ? k0 : r0, b ? r1 : k1, b ? k1 : r1};
  // stage 3: lane j holds rows 0..7 of element 2(2t + b) + (j & 1) = j,
  // t = bit 2 of j
  const bool t = (j >> 2) & 1;
  const uint32_t q0 = lane_xor4(t ? y[0] : y[2]), q1 = lane_xor4(t ? y[1] : y[3]);
  const uint32_t h0 = t ? y[2] : y[0], h1 = t ? y[3] : y[1];
  o[0] = t ? q0 : h0;
  o[1] = t ? q1 : h1;
  o[2] = t ? h0 : q0;
  o[3] = t ? h1 : q1;
}

// codesT[c][r] = bf16(code[r][c]) for one packed superblock (64 rows x 128
// columns) per wavefront.  Lane c decodes chunk c: field f holds 8-group g
// = field_group(c, f) of row field_row(c, f), so the 8 lanes of a group
// hold 8 consecutive rows of one 8-group; after the transpose lane j holds
// column 8g + j of those rows, one 16-byte store.  Padding rows of the last
// strip are zero fields, so rows up to the strip end are written (the row
// pitch np = 64 * strips).
template <int S>
__device__ __forceinline__ void prep_codes_sb(const uint32_t* __restrict__ packed, int64_t sb,
                                              int64_t nkb, int64_t np, uint16_t* __restrict__ out,
                                              const u32x2* lut, int lane, bool tiled) {
  constexpr int kW = block_bytes(S) / 4;
  const int64_t strip = sb / nkb, kb = sb - strip * nkb;
  uint32_t w[kW + 1];
  const uint32_t* src = packed + (sb * kStripRows + lane) * kW;
#pragma unroll
  for (int i = 0; i < kW; ++i) w[i] = ld_global(src + i);
  w[kW] = 0;
  const int64_t row0 = kb * kBlockK + (lane & 7), col0 = strip * kStripRows + (lane & 8);
  auto lk = [&](uint32_t key, int half) { return lut[key * 2 + half]; };
  auto emit = [&](int f, u32x2 lo, u32x2 hi) {
    const uint32_t d[4] = {lo.x, lo.y, hi.x, hi.y};
    uint32_t o[4];
    transpose8_bf16(d, o, lane);
    st_global(reinterpret_cast<u32x4*>(out + operand_at(row0 + 8 * field_group(lane, f), col0 + 16 * (f >> 2), np, tiled)),
              u32x4{o[0], o[1], o[2], o[3]});
  };
  decode_groups<S, 0, 16>(w, lk, emit);
}

template <int S>
__global__ __launch_bounds__(256) void prep_group_kernel(PrepSet set) {
  __shared__ uint16_t tile[64 * kTP];
  __shared__ u32x2 lut[512];
  const int tid = threadIdx.x;
  int job = (int)blockIdx.x, ti = 0;
  while (ti + 1 < set.n && job >= set.t[ti].jobs) job -= set.t[ti].jobs, ++ti;
  const PrepTask& tk = set.t[ti];
  if (tk.kind == kPrepCodes) {
    reinterpret_cast<u32x4*>(lut)[tid] = ld_global(reinterpret_cast<const u32x4*>(kHalfBf16Table.v) + tid);
    __syncthreads();
    const int64_t sb = 4 * (int64_t)job + (tid >> 6);
    if (sb < tk.rows * tk.cols)
      prep_codes_sb<S>(reinterpret_cast<const uint32_t*>(tk.src), sb, tk.rows, tk.pitch, tk.out, lut,
                       tid & 63, false);
    return;
  }
  const int64_t bx = tk.pitch / 64, t0 = 64 * (job % bx), c0 = 64 * (job / bx);
  if (tk.kind == kPrepDys)
    prep_dys_tile(reinterpret_cast<const uint16_t*>(tk.src), tk.scale, tk.rows, tk.cols, tk.pitch, tk.out,
                  t0, c0, tile, tid);
  else
    prep_xq_tile(reinterpret_cast<const int8_t*>(tk.src), tk.rows, tk.cols, tk.pitch, tk.out, t0, c0,
                 tile, tid, false);
}

// Everything the products of the gated feed-forward's backward read, in one launch:
// the gating's 64 x 64 tiles, then the codes of both layers, then x_q^T.  Bound by
// memory: 4096 tokens, 2560 x 6912 6:8, 8-bit G and U, 89 us for 450 MB, 5.0 TB/s
// (the gating in a launch of its own: 71 + 28); 547 tokens, 896 x 4864: 13.4 (10.4 + 8.0).
struct GluPrepJobs {
  int32_t gate, codes, xq;  // codes: of one layer
};
template <int S, int kSave, int kAct>
__global__ __launch_bounds__(256) void glu_prep_kernel(GluBwdArgs a, GluBwdLayout l, GluPrepJobs jobs) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * 64 * kGatePitch];
  static_assert(sizeof(lds) >= sizeof(kHalfBf16Table) && kGatePitch >= kTP, "the table, or a tile of x_q");
  const int tid = threadIdx.x;
  int job = (int)blockIdx.x;
  if (job < jobs.gate) {
    glu_gate_tile<kSave, kAct>(a, l, job, tid, lds, lds + 64 * kGatePitch);
    return;
  }
  job -= jobs.gate;
  const int64_t nkb = a.k / kBlockK, n2 = 2 * a.n_out;
  if (job < 2 * jobs.codes) {
    const bool up = job >= jobs.codes;
    u32x2* lut = reinterpret_cast<u32x2*>(lds);
    reinterpret_cast<u32x4*>(lds)[tid] = ld_global(reinterpret_cast<const u32x4*>(kHalfBf16Table.v) + tid);
    __syncthreads();
    const int64_t sb = 4 * (int64_t)(up ? job - jobs.codes : job) + (tid >> 6);
    // (column n_out of a tiled operand: n_out / 32 blocks of 512 on)
    uint16_t* out = reinterpret_cast<uint16_t*>(a.ws + l.codes_t) + (up ? 16 * a.n_out : 0);
    if (sb < a.n_out / kStripRows * nkb)
      prep_codes_sb<S>(static_cast<const uint32_t*>(up ? a.up : a.gate), sb, nkb, n2, out, lut, tid & 63, true);
    return;
  }
  job -= 2 * jobs.codes;
  const int64_t tp = bwd_tokens_padded(a.tokens), bx = tp / 64;
  prep_xq_tile(a.xq, a.tokens, a.k, tp, reinterpret_cast<uint16_t*>(a.ws + l.xq_t), 64 * (job % bx), 64 * (job / bx), lds, tid,
               true);
}

// ------------------------------------------------------------- product
// C[m][n] = alpha * sum_k A[m][k] * B[n][k], A/B bf16 row-major with row
// pitches lda/ldb (elements, multiples of 8), C binary32 [M][ldc].
// Workgroup tile 128 x 128, four wavefronts of 64 x 64 (4 x 4 MFMA
// tiles); k advances 64 at a time through double-buffered LDS tiles
// (rows padded to 80 bf16; of the pitches 64, 68, 72 and 80 this one
// measured fastest on MI355X, 64 slowest).  Global loads run two steps
// ahead in a register ring; one barrier per step.  k positions at or past
// K read as zero.  The output goes out with streaming stores.
//
// Tile order: workgroups are dealt round-robin to the 8 XCDs, each with its
// own L2.  Workgroup b is mapped to the (b % 8)-th contiguous eighth of a
// grouped tile order (groups of kGroupM row tiles, column tiles within a
// group, row tiles fastest), so the workgroups an XCD runs at once cover a
// compact block of rows and columns and share their operand rows in that
// L2; with the plain row-major order every XCD read nearly all of both
// operands.
constexpr int kBP = 80;
constexpr int kGroupM = 8;

// One product of a launch: C[M][N] (row pitch ldc) = alpha * A B^T over a
// k range of klen (split launches: plane blockIdx.y of C).
struct NtProblem {
  const uint16_t* A;
  const uint16_t* B;
  float* C;
  const double* alpha;
  int64_t lda, ldb, ldc, M, N, K, klen;
  // gated epilogue (256-row kernel only; N a multiple of 4, as for every output of it): with G set, C is not written;
  // the squared-ReLU gating backward of C (as relu2_gate_bwd_kernel
  // computes it from a stored C) goes to dG and dU instead, G, U, dG, dU
  // laid out like C
  const float* G = nullptr;
  const float* U = nullptr;
  uint16_t* dG = nullptr;
  uint16_t* dU = nullptr;
  // with Cb set, C is not written but rounded to bf16 into Cb, laid out like C
  // (256-row kernel only)
  uint16_t* Cb = nullptr;
  // A and B in tiles of depth K (256-row kernel only)
  bool tiled = false;
  // cut along the depth into this many ranges of whole blocks of 32, range i to plane
  // i of C (256-row kernel, tiled).  The tiles of a range are neighbours in the
  // tile order, so an XCD runs most of a range and its L2 serves their common operands
  int32_t parts = 1;
};

// the products of one launch of the 256-row kernel (its tiles dealt over
// the XCDs problem by problem, in this order)
constexpr int kMaxNt = 16;
struct NtSet {
  NtProblem p[kMaxNt];
  int32_t n;
};

__host__ __device__ inline int64_t nt_tiles(const NtProblem& p) {
  return ((p.M + 127) / 128) * ((p.N + 127) / 128);
}

// XCD share of a problem's tiles: XCD x runs tiles [start, start + cnt)
__device__ __forceinline__ void xcd_share(int64_t T, int64_t x, int64_t& start, int64_t& cnt) {
  const int64_t per = (T + 7) / 8, full = T - (per - 1) * 8;  // XCDs that get `per` tiles
  cnt = T == 0 ? 0 : (x < full ? per : per - 1);
  start = T == 0 ? 0 : (x < full ? x * per : full * per + (x - full) * (per - 1));
}

// A launch runs one or two independent products (the dX and dW of a
// layer): the tiles of each are shared out over the 8 XCDs separately, so
// every XCD runs the same mix of the two (tiles of different k depth cost
// different times), the first problem's first within an XCD.  Two
// products in one launch fill the partly used last round of each with
// tiles of the other.
__global__ __launch_bounds__(256, 2) void gemm_nt_bf16_kernel(NtProblem p0, NtProblem p1) {
  __shared__ __attribute__((aligned(16))) uint16_t As[2][128 * kBP];
  __shared__ __attribute__((aligned(16))) uint16_t Bs[2][128 * kBP];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l16 = lane & 15, lg = lane >> 4;
  int64_t m0, n0, t;
  bool second;
  {
    const int64_t xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    int64_t s0, c0, s1, c1;
    xcd_share(nt_tiles(p0), xcd, s0, c0);
    xcd_share(nt_tiles(p1), xcd, s1, c1);
    if (slot >= c0 + c1) return;
    second = slot >= c0;
    t = second ? s1 + slot - c0 : s0 + slot;
  }
  const NtProblem& pr = second ? p1 : p0;
  const uint16_t* __restrict__ A = pr.A;
  const uint16_t* __restrict__ B = pr.B;
  float* __restrict__ C = pr.C;
  const double* __restrict__ alpha = pr.alpha;
  const int64_t lda = pr.lda, ldb = pr.ldb, ldc = pr.ldc, M = pr.M, N = pr.N, klen = pr.klen;
  int64_t K = pr.K;
  {
    const int64_t tiles_m = (M + 127) / 128, tiles_n = (N + 127) / 128;
    const int64_t g = t / (kGroupM * tiles_n), r = t - g * kGroupM * tiles_n;
    const int64_t gm = tiles_m - g * kGroupM < kGroupM ? tiles_m - g * kGroupM : kGroupM;
    m0 = (g * kGroupM + r % gm) * 128;
    n0 = (r / gm) * 128;
  }
  // k range of this workgroup's split (blockIdx.y): [k0, k0 + klen) of K;
  // a split writes its partial tile to plane blockIdx.y of C
  const int64_t k0 = (int64_t)blockIdx.y * klen;
  K = K - k0 < klen ? K - k0 : klen;
  C += (int64_t)blockIdx.y * M * ldc;
  const int64_t nks = (K + 63) / 64;

  // loads: piece q = tid + 256 p (p < 4) of each tile is row q/8, k
  // columns 8*(q%8) .. +8 of the step.  A register ring holds two steps in
  // flight, so a step's global loads have two steps of MFMAs to land.
  u32x4 ra[2][4], rb[2][4];
  // buffer loads: an offset past the range (kOOB) reads zeros, so rows
  // past M/N and k past K need no branches (operands stay below 2 GiB)
  const __amdgpu_buffer_rsrc_t ar =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(A), (short)0, (int)(M * lda * 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t br =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(B), (short)0, (int)(N * ldb * 2), 0x00020000);
  constexpr uint32_t kOOB = 0x80000000u;
  uint32_t a_off[4], b_off[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int q = tid + 256 * p, row = q >> 3, kc = 8 * (q & 7);
    a_off[p] = m0 + row < M ? (uint32_t)(((m0 + row) * lda + k0 + kc) * 2) : kOOB;
    b_off[p] = n0 + row < N ? (uint32_t)(((n0 + row) * ldb + k0 + kc) * 2) : kOOB;
  }
  auto load = [&](int64_t ks, u32x4* xa, u32x4* xb) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int kc = 8 * ((tid + 256 * p) & 7);
      const bool ka = ks * 64 + kc < K;
      const uint32_t ko = (uint32_t)(ks * 128);
      xa[p] = __builtin_amdgcn_raw_buffer_load_b128(ar, ka ? a_off[p] + ko : kOOB, 0, 0);
      xb[p] = __builtin_amdgcn_raw_buffer_load_b128(br, ka ? b_off[p] + ko : kOOB, 0, 0);
    }
  };
  auto store = [&](int st, const u32x4* xa, const u32x4* xb) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int q = tid + 256 * p, row = q >> 3, kc = 8 * (q & 7);
      *reinterpret_cast<u32x4*>(&As[st][row * kBP + kc]) = xa[p];
      *reinterpret_cast<u32x4*>(&Bs[st][row * kBP + kc]) = xb[p];
    }
  };

  v4f c[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  // step ks (parity P): MFMAs from LDS stage P; in between, step ks+1
  // (registers ra/rb[P^1], loaded two steps ago) goes to stage P^1 and
  // those registers take the loads of step ks+3.  Loads past the last step
  // read zeros (k >= K) and their stores are never read.
  auto step = [&](auto parity, int64_t ks) {
    constexpr int P = decltype(parity)::value;
    // fragments of both k halves are read up front, so the second half's
    // LDS latency hides behind the first half's MFMAs
    v8bf a[2][4], b[2][4];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        a[kk][i] = *reinterpret_cast<const v8bf*>(&As[P][(wm * 64 + i * 16 + l16) * kBP + kk * 32 + lg * 8]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[kk][j] = *reinterpret_cast<const v8bf*>(&Bs[P][(wn * 64 + j * 16 + l16) * kBP + kk * 32 + lg * 8]);
    }
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          c[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[kk][i], b[kk][j], c[i][j], 0, 0, 0);
      if (kk == 0) {
        store(P ^ 1, ra[P ^ 1], rb[P ^ 1]);
        load(ks + 3, ra[P ^ 1], rb[P ^ 1]);
      }
    }
    __syncthreads();
  };

  load(0, ra[0], rb[0]);
  load(1, ra[1], rb[1]);
  store(0, ra[0], rb[0]);
  load(2, ra[0], rb[0]);
  __syncthreads();
  int64_t ks = 0;
  for (; ks + 1 < nks; ks += 2) {
    step(std::integral_constant<int, 0>{}, ks);
    step(std::integral_constant<int, 1>{}, ks + 1);
  }
  if (ks < nks) step(std::integral_constant<int, 0>{}, ks);

  // lane holds C[m0 + 64wm + 16i + 4lg + q][n0 + 64wn + 16j + l16]
  const double g = alpha ? *alpha : 1.0;
  if (m0 + 128 <= M && n0 + 128 <= N) {  // whole tile in range: no checks
    float* cb = C + (m0 + wm * 64 + 4 * lg) * ldc + n0 + wn * 64 + l16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float* cr = cb + (int64_t)(i * 16 + q) * ldc;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          st_stream(cr + j * 16, alpha ? (float)((double)c[i][j][q] * g) : c[i][j][q]);
      }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t m = m0 + wm * 64 + i * 16 + 4 * lg + q;
      if (m >= M) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + wn * 64 + j * 16 + l16;
        if (n < N) C[m * ldc + n] = alpha ? (float)((double)c[i][j][q] * g) : c[i][j][q];
      }
    }
}

// ------------------------------------------- 256 x 128 and 256 x 256 tiles
// Large products run on 256-row tiles of wavefronts of 128 x 64 (8 x 4
// MFMA tiles each): 256 x 128 (four wavefronts, two workgroups per CU) or
// 256 x 256 (eight wavefronts, one per CU).  Each byte of an operand
// fragment read from LDS feeds 1.33 times the MFMA work of the 64 x 64
// wavefront tiles above, and each byte written into LDS 1.33 (256 x 128) or
// 2 (256 x 256) times: those tiles' fragment reads and tile writes need
// more LDS bandwidth than a CU has at the full MFMA rate.  (128 x 128
// wavefront tiles would read less still, but 256 accumulators per lane made
// the register allocator shuttle them between register files around every
// MFMA.)  The tiles stream through three LDS stages of 32 k filled by LDS
// DMA (buffer loads that write LDS directly, 16 bytes per lane, 1 KiB per
// wavefront instruction), issued three steps ahead.  In a stage each
// operand row's 64 bytes hold four 16-byte pieces, placed by row64_place
// so that fragment reads are free of bank conflicts, and a DMA instruction's
// 64 lanes still write 1 KiB in order (lane l writes row l / 4, position
// l % 4, and loads the piece that belongs there).
constexpr int kBigM = 256;
constexpr int kBigK = 32;                        // k per stage
constexpr int kBigABytes = kBigM * kBigK * 2;    // 16 KiB
template <int kWN>  // column wavefronts: tile N = 64 kWN, 2 kWN wavefronts
struct BigTile {
  static constexpr int N = 64 * kWN;
  static constexpr int kWaves = 2 * kWN;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kStageBytes = kBigABytes + N * kBigK * 2;
  static constexpr int kAInstr = 16 / kWaves;    // A DMA instructions per wavefront and step
  static constexpr int kPerStep = kAInstr + 2;   // + two of B
};

template <int kWN>
__host__ __device__ inline int64_t nt_tiles_big(const NtProblem& p) {
  return ((p.M + kBigM - 1) / kBigM) * ((p.N + BigTile<kWN>::N - 1) / BigTile<kWN>::N) * p.parts;
}

// gfx950-only builtins sit in plain (non-template) functions: used directly
// in the kernel template, the host pass (which checks template bodies
// against its own target) dropped the kernel's launch stub
__device__ __forceinline__ void lds_dma16(__amdgpu_buffer_rsrc_t r, __attribute__((address_space(3))) void* dst,
                                          uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 16, off, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma_bf16(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// wait until at most N vector memory operations of this wavefront are in
// flight (the waits below count LDS DMA themselves) and, with kLds, until
// its LDS reads have returned
template <int N, bool kLds = false>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | ((kLds ? 0 : 15) << 8));
}

// Order of issue within a step of 12 fragment reads, kLoads DMA instructions and 32
// products: the reads first, a product after each, then the DMA, then the rest.
// (Left alone, the compiler put the reads last, where the next step waits.)
template <int kLoads>
__device__ __forceinline__ void order_step() {
#pragma unroll
  for (int r = 0; r < 12; ++r) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix instruction
  }
#pragma unroll
  for (int r = 0; r < kLoads; ++r) {
    __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // load
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, 20 - kLoads, 0);
  __builtin_amdgcn_sched_barrier(0);
}

// the three stages are separate arrays, each step's stage a compile-time
// choice: the compiler then sees that a step's fragment reads and the DMA
// in flight into the other stages touch different objects, and waits only
// for the DMA of the stage being read (with one array it waited for every
// DMA in flight before each read)
// (namespace-scope arrays: a function-local __shared__ array in a template
// made the host pass drop the kernel's launch stub)
__shared__ __attribute__((aligned(1024))) char g_big2_st0[BigTile<2>::kStageBytes];
__shared__ __attribute__((aligned(1024))) char g_big2_st1[BigTile<2>::kStageBytes];
__shared__ __attribute__((aligned(1024))) char g_big2_st2[BigTile<2>::kStageBytes];
__shared__ __attribute__((aligned(1024))) char g_big4_st0[BigTile<4>::kStageBytes];
__shared__ __attribute__((aligned(1024))) char g_big4_st1[BigTile<4>::kStageBytes];
__shared__ __attribute__((aligned(1024))) char g_big4_st2[BigTile<4>::kStageBytes];
template <int kWN, int P>
__device__ __forceinline__ char* big_stage() {
  static_assert(kWN == 2 || kWN == 4, "tile widths");
  if constexpr (kWN == 2) return P == 0 ? g_big2_st0 : P == 1 ? g_big2_st1 : g_big2_st2;
  else return P == 0 ? g_big4_st0 : P == 1 ? g_big4_st1 : g_big4_st2;
}

// Lanes l and l ^ 1 hold four-column pieces 0..3 of rows r and r + 1 (l even: r) in p;
// in d the even lane gets pieces 0 and 2, the odd one 1 and 3, of both rows: d[e] is row
// r + e % 2
__device__ __forceinline__ void exchange_rows(const v4f (&p)[4], v4f (&d)[4], bool odd) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float own = odd ? p[2 * h + 1][q] : p[2 * h][q], other = odd ? p[2 * h][q] : p[2 * h + 1][q];
      const float got = __uint_as_float(lane_xor1(__float_as_uint(other)));
      d[2 * h][q] = odd ? got : own;
      d[2 * h + 1][q] = odd ? own : got;
    }
}

// (512 threads at most: two wavefronts per SIMD either way, so the
// register budget is the same; bounds that depend on kWN broke the host
// side's template deduction)
template <int kWN>
__global__ __launch_bounds__(512) void gemm_nt_bf16_big_kernel(NtSet set) {
  typedef BigTile<kWN> T;
  typedef __attribute__((address_space(3))) char lds_char;
  typedef __attribute__((address_space(3))) void lds_void;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / kWN, wn = wave % kWN;
  const int l16 = lane & 15, lg = lane >> 4;
  int64_t m0, n0, t = 0;
  int which = -1;
  {
    // workgroup (XCD x, slot) takes the slot-th tile of XCD x's run: the XCD
    // shares of the problems one after the other
    // (each problem's shares start where the ones before it left off, or the XCDs
    // that get a tile more would always be the same)
    const int64_t xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    int64_t before = 0, dealt = 0;
    for (int i = 0; i < set.n; ++i) {
      int64_t s0, c0;
      const int64_t tiles = nt_tiles_big<kWN>(set.p[i]);
      xcd_share(tiles, (xcd - dealt) & 7, s0, c0);
      dealt += tiles;
      if (which < 0 && slot < before + c0) {
        which = i;
        t = s0 + slot - before;
      }
      before += c0;
    }
    if (which < 0) return;
  }
  const NtProblem& pr = set.p[which];
  const uint16_t* __restrict__ A = pr.A;
  const uint16_t* __restrict__ B = pr.B;
  float* __restrict__ C = pr.C;
  const double* __restrict__ alpha = pr.alpha;
  const int64_t lda = pr.lda, ldb = pr.ldb, ldc = pr.ldc, M = pr.M, N = pr.N, klen = pr.klen;
  int K = (int)pr.K;
  int64_t k0 = (int64_t)blockIdx.y * klen;
  {
    const int64_t tiles_m = (M + kBigM - 1) / kBigM, tiles_n = (N + T::N - 1) / T::N;
    if (pr.parts > 1) {
      const int part = (int)(t / (tiles_m * tiles_n)), n32 = K / kBigK;
      t -= part * tiles_m * tiles_n;
      k0 = (int64_t)(n32 * part / pr.parts) * kBigK;
      K = (n32 * (part + 1) / pr.parts) * kBigK;
      C += part * M * ldc;
    }
    constexpr int64_t kG = 4;  // row tiles per group of the tile order
    const int64_t g = t / (kG * tiles_n), r = t - g * kG * tiles_n;
    const int64_t gm = tiles_m - g * kG < kG ? tiles_m - g * kG : kG;
    m0 = (g * kG + r % gm) * kBigM;
    n0 = (r / gm) * T::N;
  }
  K = (int)(K - k0 < klen ? K - k0 : klen);
  C += (int64_t)blockIdx.y * M * ldc;
  const int nks = (K + kBigK - 1) / kBigK;

  const int64_t ra = pr.tiled ? (M + 15) / 16 * 16 : M, rb = pr.tiled ? (N + 15) / 16 * 16 : N;
  const __amdgpu_buffer_rsrc_t ar = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(A), (short)0, (int)(ra * lda * 2), 0x00020000);
  const __amdgpu_buffer_rsrc_t br = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(B), (short)0, (int)(rb * ldb * 2), 0x00020000);
  constexpr uint32_t kOOB = 0x80000000u;
  // DMA: wavefront w fills A rows [16 kAInstr w, +16 kAInstr) and B rows
  // [32w, 32w + 32), 16 rows per instruction; lane l covers row l / 4 of
  // the instruction's 16 at position l % 4, i.e. logical piece kc / 8
  // below (the same for every instruction)
  const int kc = 8 * row64_place(lane >> 2, lane & 3);
  uint32_t a_off[T::kAInstr], b_off[2];
#pragma unroll
  for (int q = 0; q < T::kAInstr; ++q) {
    const int64_t row = 16 * (T::kAInstr * wave + q) + (lane >> 2);
    a_off[q] = m0 + row < M ? (uint32_t)((pr.tiled ? (m0 + row - (lane >> 2)) * lda + 16 * k0 + 8 * lane : (m0 + row) * lda + k0 + kc) * 2) : kOOB;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int64_t row = 32 * wave + 16 * q + (lane >> 2);
    b_off[q] = n0 + row < N ? (uint32_t)((pr.tiled ? (n0 + row - (lane >> 2)) * ldb + 16 * k0 + 8 * lane : (n0 + row) * ldb + k0 + kc) * 2) : kOOB;
  }
  const uint32_t step_bytes = pr.tiled ? 1024 : kBigK * 2;  // from a step's piece of a row (block) to the next
  // every step issues the same instructions per wavefront (past the last
  // step they read zeros into a stage nobody reads), so the waits below
  // can count them
  auto dma = [&](auto stage, int ks) {
    constexpr int P = decltype(stage)::value;
    const bool kv = ks * kBigK + kc < K;
    const uint32_t ko = (uint32_t)ks * step_bytes;
    lds_char* st = (lds_char*)big_stage<kWN, P>();
#pragma unroll
    for (int q = 0; q < T::kAInstr; ++q)
      lds_dma16(ar, (lds_void*)(st + 1024 * (T::kAInstr * wave + q)), kv ? a_off[q] + ko : kOOB);
#pragma unroll
    for (int q = 0; q < 2; ++q)
      lds_dma16(br, (lds_void*)(st + kBigABytes + 1024 * (2 * wave + q)), kv ? b_off[q] + ko : kOOB);
  };

  v4f c[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  // fragment of MFMA row tile i / column tile j: row (or column) 16i + l16
  // of the wavefront's range, logical k piece lg
  const uint32_t frag = (uint32_t)(l16 * 64 + 16 * row64_place(l16, lg));
  const uint32_t a_base = (uint32_t)(wm * 128 * 64) + frag;
  const uint32_t b_base = (uint32_t)kBigABytes + (uint32_t)(wn * 64 * 64) + frag;

  typedef std::integral_constant<int, 0> S0;
  typedef std::integral_constant<int, 1> S1;
  typedef std::integral_constant<int, 2> S2;
  // Step ks: its fragments were read in step ks - 1.  Once this wavefront's part of
  // step ks + 1 has landed, its fragment reads have returned and everyone is
  // here, stage ks % 3 is free and takes step ks + 3, and step ks + 1 is read from
  // its stage beside the products.  (Reading a step's fragments in the step itself
  // left the matrix units waiting for them: the three products of the gated
  // feed-forward's backward, 4096 tokens, 2560 x 6912, from rows: 493 us, then 476;
  // from tiles 391, and 380 with results in whole lines, 1.53 PFLOP/s, matrix units busy
  // 71 % of the time at 2.0 GHz.)
  struct Frags {
    v8bf a[8], b[4];
  };
  auto read = [&](auto stage, Frags& f) {
    constexpr int P = decltype(stage)::value;
    const lds_char* st = (const lds_char*)big_stage<kWN, P>();
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f.b[j] = *reinterpret_cast<const __attribute__((address_space(3))) v8bf*>(st + b_base + j * 16 * 64);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f.a[i] = *reinterpret_cast<const __attribute__((address_space(3))) v8bf*>(st + a_base + i * 16 * 64);
  };
  auto step = [&](auto stage, int ks, Frags& now, Frags& next) {
    constexpr int P = decltype(stage)::value;
    // A plain barrier with compiler-only fences: __syncthreads()'s workgroup
    // release would wait for every LDS DMA in flight (they write LDS)
    wait_vmcnt<T::kPerStep, true>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    dma(std::integral_constant<int, P>{}, ks + 3);
    read(std::integral_constant<int, (P + 1) % 3>{}, next);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c[i][j] = mfma_bf16(now.b[j], now.a[i], c[i][j]);
    order_step<T::kPerStep>();
  };

  Frags f0, f1;
  dma(S0{}, 0);
  dma(S1{}, 1);
  dma(S2{}, 2);
  wait_vmcnt<2 * T::kPerStep>();
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
  wait_vmcnt<0, true>();  // no LDS DMA outlives the workgroup

  // B's fragment is the instruction's first operand, so a lane holds four neighbouring
  // columns of a row: C[m0 + 128wm + 16i + l16][n0 + 64wn + 16j + 4lg + q], in q.  Lanes
  // l16 and l16 ^ 1 then exchange half of theirs (exchange_rows), and eight lanes hold 128
  // bytes of one row: entry e of d is row `row` + 16i + e % 2, columns `col` + 32 (e / 2) + q
  // (N is a multiple of 4: a lane's four are in range together).  Whole tiles take no
  // branch inside.  (With a branch to a store and four stores to a row's 128 bytes,
  // dX and dW of 64 tokens of 2560 x 2560 took 36.5 us, now 33.9; 2048 of 2560 x 640 50.0
  // and 44.3; 4096 of 6912 x 2560 284 and 263, with the gating 355 and 323; 8192 of
  // 11008 x 2048 786 and 705.  Streaming stores of quarter lines reached memory one by
  // one; of whole lines they are as fast as others at few tokens and up to 8 % faster
  // at many.)
  const double g = alpha ? *alpha : 1.0;
  const bool odd = (l16 & 1) != 0, whole_tile = m0 + kBigM <= M && n0 + T::N <= N;
  const int64_t row = m0 + wm * 128 + (l16 & ~1), col = n0 + wn * 64 + 4 * lg + (odd ? 16 : 0);
  const int64_t first = row * ldc + col;
  const auto at = [&](int i, int e) { return first + (16 * i + (e & 1)) * ldc + 32 * (e >> 1); };
  const auto out_of_range = [&](int i, int e) { return row + 16 * i + (e & 1) >= M || col + 32 * (e >> 1) >= N; };
  using Yes = std::true_type;
  using No = std::false_type;
  if (pr.G) {
    const float* __restrict__ G = pr.G;
    const float* __restrict__ U = pr.U;
    uint16_t* __restrict__ dG = pr.dG;
    uint16_t* __restrict__ dU = pr.dU;
    const auto gate = [&](auto whole) {
      // software-pipelined over the MFMA row tiles: row tile i + 1's loads issue
      // before row tile i's stores (stores could alias them as far as the compiler
      // knows, so a load written after a store waits)
      v4f gv[2][4], uv[2][4];
      const auto load = [&](int i, v4f (&gb)[4], v4f (&ub)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          gb[e] = ub[e] = v4f{0.f, 0.f, 0.f, 0.f};
          if (!decltype(whole)::value && out_of_range(i, e)) continue;
          gb[e] = ld_global(reinterpret_cast<const v4f*>(G + at(i, e)));
          ub[e] = ld_global(reinterpret_cast<const v4f*>(U + at(i, e)));
        }
      };
      load(0, gv[0], uv[0]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i + 1 < 8) load(i + 1, gv[(i + 1) & 1], uv[(i + 1) & 1]);
        v4f d[4];
        exchange_rows(c[i], d, odd);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v4f hu, hg;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float dh = (float)((double)d[e][q] * g);
            const float gq = gv[i & 1][e][q];
            const float r = gq > 0.f ? gq : 0.f;
            const float r2 = r * r;
            const float du = dh * uv[i & 1][e][q];
            hu[q] = dh * r2;
            hg[q] = du * (2.f * r);
          }
          if (!decltype(whole)::value && out_of_range(i, e)) continue;
          st_global(reinterpret_cast<u32x2*>(dU + at(i, e)), bf16x4(hu));
          st_global(reinterpret_cast<u32x2*>(dG + at(i, e)), bf16x4(hg));
        }
      }
    };
    if (whole_tile) gate(Yes{});
    else gate(No{});
    return;
  }
  const auto store = [&](auto whole, auto scaled, auto narrow) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v4f d[4];
      exchange_rows(c[i], d, odd);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!decltype(whole)::value && out_of_range(i, e)) continue;
        v4f y = d[e];
        if (decltype(scaled)::value)
#pragma unroll
          for (int q = 0; q < 4; ++q) y[q] = (float)((double)d[e][q] * g);
        if (decltype(narrow)::value) st_global(reinterpret_cast<u32x2*>(pr.Cb + at(i, e)), bf16x4(y));
        else st_stream(reinterpret_cast<v4f*>(C + at(i, e)), y);
      }
    }
  };
  // (bf16 results carry no factor)
  if (pr.Cb) whole_tile ? store(Yes{}, No{}, Yes{}) : store(No{}, No{}, Yes{});
  else if (alpha) whole_tile ? store(Yes{}, Yes{}, No{}) : store(No{}, Yes{}, No{});
  else whole_tile ? store(Yes{}, No{}, No{}) : store(No{}, No{}, No{});
}

// C = alpha * (sum of the split planes, in order), binary32 sums; to Cb in bf16
// where that is given
__global__ __launch_bounds__(256) void split_sum_kernel(const float* __restrict__ P, int splits,
                                                       int64_t n4, const double* __restrict__ alpha,
                                                       float* __restrict__ C, uint16_t* __restrict__ Cb) {
  const double g = alpha ? *alpha : 1.0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
    v4f acc = ld_global(reinterpret_cast<const v4f*>(P) + i);
    for (int s = 1; s < splits; s += 8) {  // eight planes' loads at a time
      v4f v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (s + u < splits) v[u] = ld_global(reinterpret_cast<const v4f*>(P) + (int64_t)(s + u) * n4 + i);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (s + u < splits)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] += v[u][e];
    }
    if (alpha) {
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = (float)((double)acc[e] * g);
    }
    if (Cb) st_global(reinterpret_cast<u32x2*>(Cb) + i, bf16x4(acc));
    else st_global(reinterpret_cast<v4f*>(C) + i, acc);
  }
}

// zero fill (dW when there are no tokens)
__global__ void zero_f32_kernel(float* __restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x)
    p[i] = 0.f;
}

// ------------------------------------------------------------- launchers
// A product with few tiles and a deep k range runs split along k: its
// planes go to `partials` (row pitch N, M * N floats each) and
// split_sum_kernel adds them in order into C.
static hipError_t gemm_nt_split(NtProblem p, float* partials, hipStream_t s) {
  const int splits = bwd_splits(p.M, p.N, p.K);
  const int64_t klen = bwd_split_len(p.K, splits);
  const int used = (int)((p.K + klen - 1) / klen);
  float* C = p.C;
  const double* alpha = p.alpha;
  p.C = partials;
  p.ldc = p.N;
  p.alpha = nullptr;
  p.klen = klen;
  NtProblem none = p;
  none.M = 0;  // no tiles
  const unsigned gx = (unsigned)((nt_tiles(p) + 7) / 8 * 8);
  gemm_nt_bf16_kernel<<<dim3(gx, (unsigned)used), 256, 0, s>>>(p, none);
  const int64_t n4 = p.M * p.N / 4;
  const int64_t blocks = (n4 + 255) / 256;
  split_sum_kernel<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, s>>>(partials, used, n4, alpha, C, nullptr);
  return hipGetLastError();
}

// Tiles of the products that are not split: 0 chooses per launch by the
// tile counts; 1, 2, 3 fix 128 x 128, 256 x 128 or 256 x 256
// (bitlinear_bwd_tiles).
static std::atomic<int> g_bwd_tiles{0};
int bwd_set_tiles(int tiles) {
  if (tiles < 0 || tiles > 3) return -1;
  g_bwd_tiles.store(tiles, std::memory_order_relaxed);
  return 0;
}
// The tile size with the shorter estimated time.  Each of an XCD's 32 CUs is given the
// next tile (the deepest products first, as they are launched) when it has least to do.
// A 256 x 256 tile, one on a CU, costs its depth; 256 x 128 tiles run two on a CU, both
// in 1.18 times a large one's time (they reach a lower rate), one alone in 0.6.  The
// choice is the faster one, or within 5% of it, for layers of 640 to 8960 at 512 to
// 8192 tokens.  (Counting rounds of tiles as if all were equally deep it was not: 1024
// tokens of 6912 x 2560, where 14 deep tiles and 34 shallow ones on an XCD are no
// longer than one deep tile and a half: 88 us with large tiles, 111 with small ones; 512
// tokens of 2560 x 6912 twice, the other way round: 174 and 143.)
static double big_time(const NtSet& set, bool wide) {
  struct Cu {
    double load;
    bool odd;
    int64_t last;  // depth of its last tile
  };
  Cu cu[32] = {};
  const auto later = [](const Cu& a, const Cu& b) { return a.load > b.load; };
  const double cost = wide ? 1.0 : 1.18 / 2;
  for (int i = 0; i < set.n; ++i) {
    int64_t tiles = ((wide ? nt_tiles_big<4>(set.p[i]) : nt_tiles_big<2>(set.p[i])) + 7) / 8;
    const int64_t depth = set.p[i].K;
    const double step = cost * (double)depth;
    // in one go, while there are enough tiles: those that bring every CU to within a tile
    // of the busiest, then rounds of one each
    double most = 0.0;
    for (const Cu& c : cu) most = c.load > most ? c.load : most;
    const auto lacks = [&](const Cu& c) { return (int64_t)((most - c.load) / step); };
    int64_t level = 0;
    for (const Cu& c : cu) level += lacks(c);
    if (level + 32 <= tiles) {
      const int64_t rounds = (tiles - level) / 32;
      for (Cu& c : cu) {
        const int64_t n = lacks(c) + rounds;
        if (n > 0) c = Cu{c.load + (double)n * step, c.odd != ((n & 1) != 0), depth};
      }
      tiles -= level + 32 * rounds;
      std::make_heap(cu, cu + 32, later);
    }
    for (; tiles > 0; --tiles) {
      std::pop_heap(cu, cu + 32, later);
      cu[31] = Cu{cu[31].load + step, !cu[31].odd, depth};
      std::push_heap(cu, cu + 32, later);
    }
  }
  double most = 0.0;
  for (const Cu& c : cu) {
    const double time = c.load + (!wide && c.odd ? (0.6 - cost) * (double)c.last : 0.0);
    most = time > most ? time : most;
  }
  return most;
}
static int big_kind(const NtSet& set) { return big_time(set, false) < big_time(set, true) ? 2 : 3; }
static int bwd_tile_kind(const NtSet& set) {
  const int f = g_bwd_tiles.load(std::memory_order_relaxed);
  return f ? f : big_kind(set);
}
static hipError_t launch_big(const NtSet& set, int kind, hipStream_t s) {
  int64_t per = 0;
  if (kind == 3) {
    for (int i = 0; i < set.n; ++i) per += (nt_tiles_big<4>(set.p[i]) + 7) / 8;
    gemm_nt_bf16_big_kernel<4><<<(unsigned)(8 * per), BigTile<4>::kThreads, 0, s>>>(set);
  } else {
    for (int i = 0; i < set.n; ++i) per += (nt_tiles_big<2>(set.p[i]) + 7) / 8;
    gemm_nt_bf16_big_kernel<2><<<(unsigned)(8 * per), BigTile<2>::kThreads, 0, s>>>(set);
  }
  return hipGetLastError();
}

// The products that are not split run in one launch (a null `b` is no
// second product); split ones follow, one after the other (they share the
// partial planes).
static hipError_t gemm_nt_run(const NtProblem* a, const NtProblem* b, float* partials, hipStream_t s) {
  const NtProblem* whole[2] = {nullptr, nullptr};
  const NtProblem* split[2] = {nullptr, nullptr};
  int nw = 0, ns = 0;
  for (const NtProblem* p : {a, b}) {
    if (!p) continue;
    if (bwd_splits(p->M, p->N, p->K) > 1) split[ns++] = p;
    else whole[nw++] = p;
  }
  if (nw) {
    NtProblem p0 = *whole[0], p1 = p0;
    if (nw == 2) {
      p1 = *whole[1];
      if (p1.K > p0.K) std::swap(p0, p1);  // the deeper product first within each XCD
    } else {
      p1.M = 0;  // no tiles
    }
    NtSet set{};
    set.p[0] = p0;
    set.p[1] = p1;
    set.n = nw;
    const int kind = bwd_tile_kind(set);
    if (kind >= 2) {
      hipError_t e = launch_big(set, kind, s);
      if (e != hipSuccess) return e;
    } else {
      const int64_t per = (nt_tiles(p0) + 7) / 8 + (nt_tiles(p1) + 7) / 8;
      gemm_nt_bf16_kernel<<<(unsigned)(8 * per), 256, 0, s>>>(p0, p1);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  for (int i = 0; i < ns; ++i) {
    hipError_t e = gemm_nt_split(*split[i], partials, s);
    if (e != hipSuccess) return e;
  }
  return hipGetLastError();
}

// the prep tasks of one call, launched together (in chunks of kMaxPrep)
struct PrepList {
  std::vector<PrepTask> t;
  hipError_t launch(int S, hipStream_t s) const {
    for (size_t first = 0; first < t.size(); first += kMaxPrep) {
      PrepSet set{};
      set.n = (int32_t)std::min<size_t>(kMaxPrep, t.size() - first);
      int64_t jobs = 0;
      for (int i = 0; i < set.n; ++i) {
        set.t[i] = t[first + (size_t)i];
        jobs += set.t[i].jobs;
      }
      if (jobs == 0) continue;
      if (S == 8) prep_group_kernel<8><<<(unsigned)jobs, 256, 0, s>>>(set);
      else if (S == 6) prep_group_kernel<6><<<(unsigned)jobs, 256, 0, s>>>(set);
      else if (S == 2) prep_group_kernel<2><<<(unsigned)jobs, 256, 0, s>>>(set);
      else prep_group_kernel<4><<<(unsigned)jobs, 256, 0, s>>>(set);
      hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
};

// dX operand: the codes decoded and transposed (codes^T [k x np])
static void prep_dx(PrepList& L, const void* packed, void* ws, int64_t tokens, int64_t k, int64_t n_out) {
  const int64_t nkb = k / kBlockK, strips = (n_out + kStripRows - 1) / kStripRows;
  uint16_t* codes_t = reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(ws) + bwd_codes_offset(tokens, k, n_out));
  L.t.push_back(PrepTask{packed, nullptr, codes_t, nkb, strips, strips * kStripRows, kPrepCodes,
                         (int32_t)((strips * nkb + 3) / 4)});
}

// dX [tokens x k] = gamma * dY [tokens x n_out] . codes^T [k x n_out]^T
static NtProblem dx_problem(const uint16_t* dY, const double* gamma, float* dX, void* ws, int64_t tokens,
                            int64_t k, int64_t n_out) {
  const int64_t np = (n_out + kStripRows - 1) / kStripRows * kStripRows;
  const uint16_t* codes_t =
      reinterpret_cast<const uint16_t*>(reinterpret_cast<char*>(ws) + bwd_codes_offset(tokens, k, n_out));
  return NtProblem{dY, codes_t, dX, gamma, n_out, np, k, tokens, k, n_out, n_out};
}

// dW operands: bf16(dY * s)^T unless with_dys is false, x_q^T unless
// with_xq is false (the grouped call reuses another item's x_q^T when two
// items share x_q, and its phases split the two)
static void prep_dw(PrepList& L, const uint16_t* dY, const int8_t* xq, const float* scale, void* ws,
                    int64_t tokens, int64_t k, int64_t n_out, bool with_xq = true, bool with_dys = true) {
  const int64_t tp = bwd_tokens_padded(tokens);
  char* w = reinterpret_cast<char*>(ws);
  uint16_t* dys_t = reinterpret_cast<uint16_t*>(w + bwd_dys_offset(tokens, k, n_out));
  uint16_t* xq_t = reinterpret_cast<uint16_t*>(w + bwd_xq_offset(tokens, k, n_out));
  if (with_dys)
    L.t.push_back(PrepTask{dY, scale, dys_t, tokens, n_out, tp, kPrepDys, (int32_t)((tp / 64) * ((n_out + 63) / 64))});
  if (with_xq) L.t.push_back(PrepTask{xq, nullptr, xq_t, tokens, k, tp, kPrepXq, (int32_t)((tp / 64) * (k / 64))});
}

// dW [n_out x k] = (dY s)^T [n_out x tp] . x_q^T [k x tp]^T
static NtProblem dw_problem(float* dW, void* ws, int64_t tokens, int64_t k, int64_t n_out) {
  const int64_t tp = bwd_tokens_padded(tokens);
  char* w = reinterpret_cast<char*>(ws);
  return NtProblem{reinterpret_cast<const uint16_t*>(w + bwd_dys_offset(tokens, k, n_out)),
                   reinterpret_cast<const uint16_t*>(w + bwd_xq_offset(tokens, k, n_out)),
                   dW, nullptr, tp, tp, k, n_out, k, tp, tp};
}

hipError_t launch_bwd(const uint16_t* dY, const int8_t* xq, const float* scale, const void* packed,
                      const double* gamma, float* dX, float* dW, void* ws, int64_t tokens, int64_t k,
                      int64_t n_out, int S, hipStream_t s) {
  if (tokens == 0) {  // dX is empty; dW is all zeros
    if (dW) zero_f32_kernel<<<1024, 256, 0, s>>>(dW, n_out * k);
    return hipGetLastError();
  }
  PrepList L;
  if (dX) prep_dx(L, packed, ws, tokens, k, n_out);
  if (dW) prep_dw(L, dY, xq, scale, ws, tokens, k, n_out);
  hipError_t e = L.launch(S, s);
  if (e != hipSuccess) return e;
  NtProblem px{}, pw{};
  if (dX) px = dx_problem(dY, gamma, dX, ws, tokens, k, n_out);
  if (dW) pw = dw_problem(dW, ws, tokens, k, n_out);
  float* partials = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + bwd_partial_offset(tokens, k, n_out));
  return gemm_nt_run(dX ? &px : nullptr, dW ? &pw : nullptr, partials, s);
}

// The down projection's backward with the gating backward fused into its
// dX product: the dX tiles never reach memory; their epilogue forms dG and
// dU (the squared-ReLU gating backward of dX, as relu2_gate_bwd_kernel
// computes it), so results equal bitlinear_bwd followed by the gating
// backward bit for bit.  dX runs unsplit on the 256-row kernel (its
// epilogue holds the gating); dW as in launch_bwd.  tokens > 0.
hipError_t launch_bwd_gate(const uint16_t* dY, const int8_t* xq, const float* scale, const void* packed,
                           const double* gamma, const float* G, const float* U, uint16_t* dG, uint16_t* dU,
                           float* dW, void* ws, int64_t tokens, int64_t k, int64_t n_out, int S,
                           hipStream_t s) {
  PrepList L;
  prep_dx(L, packed, ws, tokens, k, n_out);
  if (dW) prep_dw(L, dY, xq, scale, ws, tokens, k, n_out);
  hipError_t e = L.launch(S, s);
  if (e != hipSuccess) return e;
  NtProblem px = dx_problem(dY, gamma, nullptr, ws, tokens, k, n_out);
  px.G = G;
  px.U = U;
  px.dG = dG;
  px.dU = dU;
  NtSet set{};
  set.p[0] = px;
  set.n = 1;
  NtProblem pw{};
  bool dw_split = false;
  if (dW) {
    pw = dw_problem(dW, ws, tokens, k, n_out);
    dw_split = bwd_splits(pw.M, pw.N, pw.K) > 1;
    if (!dw_split) {
      set.p[1] = pw;
      set.n = 2;
      if (pw.K > px.K) std::swap(set.p[0], set.p[1]);  // the deeper product first within each XCD
    }
  }
  const int f = g_bwd_tiles.load(std::memory_order_relaxed);
  e = launch_big(set, f >= 2 ? f : big_kind(set), s);  // 128 x 128 tiles have no gated epilogue
  if (e != hipSuccess) return e;
  if (dw_split) {
    float* partials = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + bwd_partial_offset(tokens, k, n_out));
    e = gemm_nt_split(pw, partials, s);
    if (e != hipSuccess) return e;
  }
  return hipGetLastError();
}

hipError_t launch_zero(float* p, int64_t n, hipStream_t s) {
  zero_f32_kernel<<<1024, 256, 0, s>>>(p, n);
  return hipGetLastError();
}

template <int S>
static hipError_t glu_prep(const GluBwdArgs& a, const GluBwdLayout& l, hipStream_t s) {
  const int64_t tb = bwd_tokens_padded(a.tokens) / 64, superblocks = a.n_out / kStripRows * (a.k / kBlockK);
  GluPrepJobs jobs{};
  jobs.gate = (int32_t)(tb * (a.n_out / 64));
  if (a.dX) jobs.codes = (int32_t)((superblocks + 3) / 4);
  if (a.dWg) jobs.xq = (int32_t)(tb * (a.k / 64));
  const unsigned grid = (unsigned)(jobs.gate + 2 * jobs.codes + jobs.xq);
  const auto run = [&](auto save) {
    constexpr int kSave = decltype(save)::value;
    if (a.act == kActRelu2) glu_prep_kernel<S, kSave, kActRelu2><<<grid, 256, 0, s>>>(a, l, jobs);
    else glu_prep_kernel<S, kSave, kActSilu><<<grid, 256, 0, s>>>(a, l, jobs);
    return hipGetLastError();
  };
  if (a.save == kRowF32) return run(std::integral_constant<int, kRowF32>{});
  return a.save == kRowBf16 ? run(std::integral_constant<int, kRowBf16>{}) : run(std::integral_constant<int, kRowQ8>{});
}

// The products of the gated feed-forward's backward.  dX is one product of
// depth 2 n_out: dG gate_gamma and dU up_gamma stand side by side in dgu and so do the two
// layers' codes in codes_t, so it is written once.  The deepest products' tiles start
// first.
hipError_t launch_glu_bwd(const GluBwdArgs& a, int S, hipStream_t s) {
  const GluBwdLayout l = glu_bwd_layout(a.tokens, a.k, a.n_out);
  const int64_t tp = bwd_tokens_padded(a.tokens), n2 = 2 * a.n_out;
  const auto at = [&](size_t o) { return reinterpret_cast<uint16_t*>(a.ws + o); };
  hipError_t e = S == 8 ? glu_prep<8>(a, l, s) : S == 6 ? glu_prep<6>(a, l, s) : S == 2 ? glu_prep<2>(a, l, s) : glu_prep<4>(a, l, s);
  if (e != hipSuccess) return e;

  const bool b16 = a.grad_type == BL_TYPE_BF16;
  NtSet set{};
  // out [rows][k] = A [rows][depth] B [k][depth]^T
  const auto add = [&](size_t A, size_t B, void* out, size_t planes, int64_t rows, int64_t depth, int parts) {
    NtProblem p{at(A), at(B), nullptr, nullptr, depth, depth, a.k, rows, a.k, depth, depth};
    p.tiled = true;
    p.parts = parts;
    if (parts > 1) p.C = reinterpret_cast<float*>(a.ws + planes);
    else if (b16) p.Cb = static_cast<uint16_t*>(out);
    else p.C = static_cast<float*>(out);
    set.p[set.n++] = p;
  };
  if (a.dX) add(l.dgu, l.codes_t, a.dX, l.planes_x, a.tokens, n2, l.split_x);
  if (a.dWg) {
    add(l.dgs_t, l.xq_t, a.dWg, l.planes_g, a.n_out, tp, l.split_w);
    add(l.dus_t, l.xq_t, a.dWu, l.planes_u, a.n_out, tp, l.split_w);
  }
  std::stable_sort(set.p, set.p + set.n, [](const NtProblem& x, const NtProblem& y) { return x.K / x.parts > y.K / y.parts; });
  e = launch_big(set, l.narrow ? 2 : 3, s);
  const auto sum = [&](void* out, size_t planes, int64_t rows, int parts) {
    if (e != hipSuccess || !out || parts == 1) return;
    const int64_t n4 = rows * a.k / 4, blocks = (n4 + 255) / 256;
    split_sum_kernel<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, s>>>(
        reinterpret_cast<const float*>(a.ws + planes), parts, n4, nullptr, b16 ? nullptr : static_cast<float*>(out),
        b16 ? static_cast<uint16_t*>(out) : nullptr);
    e = hipGetLastError();
  };
  sum(a.dX, l.planes_x, a.tokens, l.split_x);
  sum(a.dWg, l.planes_g, a.n_out, l.split_w);
  sum(a.dWu, l.planes_u, a.n_out, l.split_w);
  return e;
}

hipError_t launch_bwd_group(const BwdItem* items, int count, int64_t tokens, int S, void* ws, int phase,
                            hipStream_t s) {
  // phase bit 0: the conversions that read only packed codes and x_q;
  // bit 1: the dY conversions and the products.  Both walk the items in
  // the same order, so every operand lands at the same place either way
  const bool first = (phase & 1) != 0, second = (phase & 2) != 0;
  std::vector<NtProblem> probs;
  // x_q^T already prepared in this call, by x_q pointer and k: layers fed
  // the same input (q, k, v; gate, up) share it
  struct XqT {
    const int8_t* xq;
    int64_t k;
    const uint16_t* t;
  };
  std::vector<XqT> done;
  PrepList L;
  char* w = reinterpret_cast<char*>(ws);
  for (int i = 0; i < count; ++i) {
    const BwdItem& it = items[i];
    if (it.dX) {
      if (first) prep_dx(L, it.packed, w, tokens, it.k, it.n_out);
      probs.push_back(dx_problem(it.dY, it.gamma, it.dX, w, tokens, it.k, it.n_out));
    }
    if (it.dW) {
      const XqT* seen = nullptr;
      for (const XqT& d : done)
        if (d.xq == it.xq && d.k == it.k) seen = &d;
      prep_dw(L, it.dY, it.xq, it.scale, w, tokens, it.k, it.n_out, first && seen == nullptr, second);
      NtProblem p = dw_problem(it.dW, w, tokens, it.k, it.n_out);
      if (seen) p.B = seen->t;
      else done.push_back(XqT{it.xq, it.k, p.B});
      probs.push_back(p);
    }
    w += bwd_group_item_bytes(tokens, it.k, it.n_out);
  }
  hipError_t pe = L.launch(S, s);
  if (pe != hipSuccess || !second) return pe;
  // deepest contraction first: within each XCD the longest tiles start
  // first and the short ones fill the end (a longest-first schedule)
  std::stable_sort(probs.begin(), probs.end(),
                   [](const NtProblem& a, const NtProblem& b) { return a.K > b.K; });
  for (size_t first = 0; first < probs.size(); first += kMaxNt) {
    NtSet set{};
    set.n = (int32_t)std::min<size_t>(kMaxNt, probs.size() - first);
    for (int i = 0; i < set.n; ++i) set.p[i] = probs[first + (size_t)i];
    const int f = g_bwd_tiles.load(std::memory_order_relaxed);
    hipError_t e = launch_big(set, f >= 2 ? f : big_kind(set), s);  // 128 x 128 tiles take two products only
    if (e != hipSuccess) return e;
  }
  return hipGetLastError();
}

}  // namespace bl
