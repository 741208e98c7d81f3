// attn.h -- device pieces the attention kernels share: matrix operands of
// the 32 x 32 x 16 bf16 instruction, LDS tiles filled by DMA, and the order
// of the work items.
#pragma once

#include "common.h"

namespace bl {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) void lds_void;

// v_mfma_f32_32x32x16_bf16: lane l holds A[l%32][8(l/32) .. +7] and
// B[8(l/32) .. +7][l%32]; register i of its result is element
// [8(i/4) + 4(l/32) + i%4][l%32].
//
// The forward, dQ and cache kernels keep the softmax's row along the lanes:
// with S^T = K Q^T a lane holds one query's scores (column l%32) and after exp
// two consecutive groups of four registers are, as they stand, the B operand
// of the product over keys: its slots 0-3 and 4-7 are then keys 4(l/32) + 0..3
// and 8 + 4(l/32) + 0..3 of 16, and A is read from LDS in the same order.
// (The dK / dV kernel does the same with keys along the lanes and sums over
// rows.)  The probabilities never leave the registers.
__device__ __forceinline__ v16f mfma32(v8bf a, v8bf b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
// transposing LDS read: of each 16 lanes, lanes 4j..4j+3 address 8 bytes
// each of row j (16 elements); lane i receives element i of rows 0..3
__device__ __forceinline__ v4s lds_read_tr(const lds_char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(p));
}
__device__ __forceinline__ v8bf lds_read8(const lds_char* p) {
  return *reinterpret_cast<const __attribute__((address_space(3))) v8bf*>(p);
}
__device__ __forceinline__ v8bf join(v4s a, v4s b) {
  return __builtin_bit_cast(v8bf, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {  // nearest, ties to even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, v2bf));
}
// registers 8s .. 8s+7 of a result as the B operand described above
__device__ __forceinline__ v8bf operand_of(const v16f& x, int s) {
  return __builtin_bit_cast(v8bf, u32x4{pk_bf16(x[8 * s], x[8 * s + 1]), pk_bf16(x[8 * s + 2], x[8 * s + 3]),
                                        pk_bf16(x[8 * s + 4], x[8 * s + 5]), pk_bf16(x[8 * s + 6], x[8 * s + 7])});
}
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_hw(float x) { return __builtin_amdgcn_logf(x); }
// Largest |m scale log2 e| whose rounding may stay in the exponents of a
// softmax: 2^-12 of an exponent, 2^-12 of P, a sixteenth of P's rounding to bf16
constexpr float kSteep = 4096.f;
// the other half wavefront's value of the same column, combined with `f`
template <class F>
__device__ __forceinline__ float half_join(float v, F f) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
// exchanges a's upper with b's lower half wavefront
__device__ __forceinline__ void half_swap(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ void lds_load16(__amdgpu_buffer_rsrc_t r, lds_char* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void lds_load4(__amdgpu_buffer_rsrc_t r, lds_char* dst, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 4, off, 0, 0, 0);
}
// wait until at most N of this wavefront's memory operations (LDS DMA
// included) are in flight, and until its LDS reads have returned
template <int N>
__device__ __forceinline__ void wait_dma() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (0 << 8));
}
// workgroup barrier that leaves LDS DMA in flight (a release would drain it)
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------
// A tile of rows of D bf16 in LDS, row after row, the 16-byte pieces of row
// r permuted: piece c at place c ^ swz(r).  LDS serves 256 bytes a clock to
// these reads, a 16-byte read 16 lanes at a time, an 8-byte transposing read
// 32 lanes at a time.  The permutation spreads both over all of a 256-byte
// bank line: 16 consecutive rows' reads of one piece (an A operand by rows),
// and a transposing read's four aligned rows of 64 bytes.  (A permutation by
// r % 8 within 128 bytes left both at half that rate: 128 of the 265 LDS
// clocks of a 64-key tile of the forward were bank conflicts.)
// ---------------------------------------------------------------------
template <int D>
struct Tile {
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kPieces = D / 8;            // 16-byte pieces of a row
  static constexpr int kDmaRows = 64 / kPieces;    // rows of one DMA instruction (4 or 8)
  static constexpr int kVariants = 16 / kDmaRows;  // row residues mod 16 an instruction can start at
  static constexpr uint32_t kFar = D == 128 ? 32 : 16;  // address bits that differ between rows r and r + 8
  __device__ static __forceinline__ constexpr int swz(int r) {
    return D == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : ((r & 2) << 1) | ((r >> 1) & 2) | ((r >> 3) & 1);
  }
};

// offset, from the first row of a DMA instruction's rows, that this lane
// loads; `var`: (first row / kDmaRows) % kVariants
template <int D>
__device__ __forceinline__ uint32_t dma_offset(int lane, int var, int64_t stride) {
  typedef Tile<D> T;
  const int r = lane / T::kPieces, c = (lane % T::kPieces) ^ T::swz(r + var * T::kDmaRows);
  return (uint32_t)(r * (int)stride * 2 + c * 16);
}
// address (from the tile's start) of the operand of rows l%32, elements
// 16s + 8(l/32) .. +7; 32 rows further on the permutation is the same
template <int D>
__device__ __forceinline__ uint32_t a_addr(int lane, int s) {
  const int r = lane & 31;
  return (uint32_t)(r * Tile<D>::kRowBytes + (((2 * s + (lane >> 5)) ^ Tile<D>::swz(r)) << 4));
}
// address of the transposing read that gives lane l column 32t + l%32 of
// rows 4(l/32) + 0..3; 16 rows further on the permutation is the same
template <int D>
__device__ __forceinline__ uint32_t tr_addr(int lane, int t) {
  const int r = 4 * (lane >> 5) + ((lane & 15) >> 2);
  const int c = 4 * t + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  return (uint32_t)(r * Tile<D>::kRowBytes + ((c ^ Tile<D>::swz(r)) << 4) + 8 * (lane & 1));
}
// the two addresses of an A operand [columns 32t..+31][16 rows]: rows
// 4(l/32) + 0..3 and the same 8 rows further on
struct TrAddr {
  uint32_t near, far;
};
template <int D>
__device__ __forceinline__ TrAddr tr_addrs(int lane, int t, uint32_t base) {
  const uint32_t a = tr_addr<D>(lane, t);
  return TrAddr{base + a, base + (a ^ Tile<D>::kFar) + 8 * Tile<D>::kRowBytes};
}
template <int D>
__device__ __forceinline__ v8bf tr_operand(const lds_char* tile, TrAddr a, int r0) {
  return join(lds_read_tr(tile + a.near + r0 * Tile<D>::kRowBytes), lds_read_tr(tile + a.far + r0 * Tile<D>::kRowBytes));
}

// acc^T (column = row of the output, registers = its D elements) times mul,
// as bf16: after an exchange between the half wavefronts every lane stores
// 16 bytes of its row at a time
template <int D>
__device__ __forceinline__ void store_row(uint16_t* row, const v16f* acc, float mul, int lane, bool in) {
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int e = 8 * u;
      uint32_t a0 = pk_bf16(acc[t][e] * mul, acc[t][e + 1] * mul);
      uint32_t a1 = pk_bf16(acc[t][e + 2] * mul, acc[t][e + 3] * mul);
      uint32_t b0 = pk_bf16(acc[t][e + 4] * mul, acc[t][e + 5] * mul);
      uint32_t b1 = pk_bf16(acc[t][e + 6] * mul, acc[t][e + 7] * mul);
      half_swap(a0, b0);
      half_swap(a1, b1);
      if (in) st_global(reinterpret_cast<u32x4*>(row + 32 * t + 16 * u + 8 * (lane >> 5)), u32x4{a0, a1, b0, b1});
    }
}

// ---------------------------------------------------------------------
// Work items are tiles of the sequences, every sequence cut into
// ceil(len / rows) of them, numbered so that those with the highest level
// (place in the sequence) come first: under a causal mask the longest work
// starts first and the short tiles fill up the end.  Every wavefront finds
// its item by itself: level by bisection over the sequences' tile counts
// held by the lanes.  Batches beyond kOrdered sequences are walked in order
// instead (one pass of prefix sums), where a bisection would read the
// lengths over and over.
// Lengths come from device memory: rows outside the buffers are cut off
// here, so wrong offsets cannot lead outside them.
// ---------------------------------------------------------------------
constexpr int kOrderedPerLane = 4;
constexpr int kOrdered = 64 * kOrderedPerLane;

// Sums over the lanes 0 .. lane by DPP moves within the vector unit (rows of
// 16, then the last lane of a row to the next rows): a tenth of the time of
// exchanges through LDS, of which finding an item takes dozens one after the
// other.
template <int kCtrl, int kRows>
__device__ __forceinline__ int dpp_from(int none, int v) {
  return __builtin_amdgcn_update_dpp(none, v, kCtrl, kRows, 0xf, false);
}
__device__ __forceinline__ int wave_scan_i(int v) {
  v += dpp_from<0x111, 0xf>(0, v);  // row_shr:1, 2, 4, 8
  v += dpp_from<0x112, 0xf>(0, v);
  v += dpp_from<0x114, 0xf>(0, v);
  v += dpp_from<0x118, 0xf>(0, v);
  v += dpp_from<0x142, 0xa>(0, v);  // row_bcast:15 into rows 1 and 3
  v += dpp_from<0x143, 0xc>(0, v);  // row_bcast:31 into rows 2 and 3
  return v;
}
__device__ __forceinline__ int wave_sum_i(int v) { return __builtin_amdgcn_readlane(wave_scan_i(v), 63); }
__device__ __forceinline__ int max_i(int a, int b) { return a > b ? a : b; }
__device__ __forceinline__ int wave_max_i(int v) {  // of values >= 0
  v = max_i(v, dpp_from<0x111, 0xf>(0, v));
  v = max_i(v, dpp_from<0x112, 0xf>(0, v));
  v = max_i(v, dpp_from<0x114, 0xf>(0, v));
  v = max_i(v, dpp_from<0x118, 0xf>(0, v));
  v = max_i(v, dpp_from<0x142, 0xa>(0, v));
  v = max_i(v, dpp_from<0x143, 0xc>(0, v));
  return __builtin_amdgcn_readlane(v, 63);
}

// rows [start, start + len) of sequence b
struct Rows {
  int start, len;
};
__device__ __forceinline__ Rows cut_rows(int lo, int hi, int64_t total) {
  lo = lo < 0 ? 0 : lo > total ? (int)total : lo;
  hi = hi < lo ? lo : hi > total ? (int)total : hi;
  return Rows{lo, hi - lo};
}
__device__ __forceinline__ Rows seq_rows(const int32_t* cu, int b, int64_t total) {
  return cut_rows(ld_global(cu + b), ld_global(cu + b + 1), total);
}
__device__ __forceinline__ Rows lane_rows(const Rows& r, int lane) {
  return Rows{__builtin_amdgcn_readlane(r.start, lane), __builtin_amdgcn_readlane(r.len, lane)};
}

// Item `rank` of the tiles of `rows` rows of the sequences in cu, with the
// sequence's rows there and in the other offsets (all the same in every lane)
struct Item {
  int seq, level;  // seq < 0: none
  Rows mine, other;
};
__device__ __forceinline__ Item find_item(const int32_t* cu, int64_t total, const int32_t* cu2, int64_t total2,
                                          int batch, int rows, int rank) {
  const int lane = threadIdx.x & 63;
  const Item none{-1, 0, {0, 0}, {0, 0}};
  if (batch > kOrdered) {
    int before = 0;
    for (int b0 = 0; b0 < batch; b0 += 64) {
      const int b = b0 + lane;
      const int n = b < batch ? (seq_rows(cu, b, total).len + rows - 1) / rows : 0;
      const int incl = before + wave_scan_i(n);
      const unsigned long long hit = __ballot(incl > rank);
      if (hit) {
        const int l = __builtin_amdgcn_readfirstlane(__ffsll(hit) - 1);
        const int level = rank - (__builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(n, l));
        const Rows r = seq_rows(cu, b0 + l, total), o = seq_rows(cu2, b0 + l, total2);
        return Item{b0 + l, level, lane_rows(r, 0), lane_rows(o, 0)};
      }
      before = __builtin_amdgcn_readlane(incl, 63);
    }
    return none;
  }
  Rows mine[kOrderedPerLane], other[kOrderedPerLane];
  int n[kOrderedPerLane], most = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kOrderedPerLane; ++i) {
    const int b = 64 * i + lane;
    mine[i] = other[i] = Rows{0, 0};
    if (b < batch) {
      mine[i] = seq_rows(cu, b, total);
      other[i] = seq_rows(cu2, b, total2);
    }
    n[i] = (mine[i].len + rows - 1) / rows;
    most = max_i(most, n[i]);
    all += n[i];
  }
  if (rank >= wave_sum_i(all)) return none;
  // at(L) = items of level L and above; the largest L with at(L) > rank
  const auto at = [&](int L) {
    int c = 0;
#pragma unroll
    for (int i = 0; i < kOrderedPerLane; ++i) c += n[i] > L ? n[i] - L : 0;
    return wave_sum_i(c);
  };
  int lo = 0, hi = wave_max_i(most);  // at(lo) > rank >= at(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at(mid) > rank) lo = mid;
    else hi = mid;
  }
  int skip = rank - at(lo + 1);  // among the sequences with more than lo tiles
#pragma unroll
  for (int i = 0; i < kOrderedPerLane; ++i) {
    const unsigned long long m = __ballot(n[i] > lo);
    const int c = __popcll(m);
    if (skip < c) {
      const bool mine_is = (m >> lane & 1) && __popcll(m & ((1ull << lane) - 1)) == skip;
      const int l = __builtin_amdgcn_readfirstlane(__ffsll(__ballot(mine_is)) - 1);
      return Item{64 * i + l, lo, lane_rows(mine[i], l), lane_rows(other[i], l)};
    }
    skip -= c;
  }
  return none;
}

// Workgroup id -> (item rank, head) for `items` ranks, `pairs` key/value
// heads and `per` workgroups of each.  Consecutive workgroups go to different
// XCDs, whose L2 caches are separate.  Eight ranks at a time are dealt so
// that an XCD's workgroups have the fewest possible key/value heads among
// them (8 * pairs (head, rank) pairs in that order, `pairs` to each XCD):
// they read the same rows at about the same time, and those reads meet in its
// L2.  Odd blocks of ranks run backwards, so no XCD always has the longer
// items.  Fewer than eight ranks are simply numbered: padded to eight, most
// workgroups of a small call would have nothing to do (two sequences of 64 and
// 100 tokens, 16 + 2 heads, forward and backward: 36.2 us padded, 35.1 us).
struct Place {
  int rank, pair, part;
};
__device__ __forceinline__ Place place_of(int id, int items, int pairs, int per) {
  if (items < 8) {
    const int s = id / per, rank = s / pairs;
    return Place{rank, s - rank * pairs, id - s * per};
  }
  const int xcd = id & 7, slot = id >> 3;
  const int s = slot / per, block = s / pairs;
  const int at = xcd * pairs + (s - block * pairs);
  const int r = at & 7;
  return Place{block * 8 + (block & 1 ? 7 - r : r), at >> 3, slot - s * per};
}
inline int64_t placed_items(int64_t items) { return items < 8 ? items : (items + 7) / 8 * 8; }
inline int64_t placed_blocks(int64_t items, int64_t pairs, int64_t per) { return placed_items(items) * pairs * per; }

}  // namespace bl
