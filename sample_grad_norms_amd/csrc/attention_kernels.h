// Causal softmax attention of packed sequences with grouped heads, and its
// gradients.
//
//   s_tu = a q_t . k_u,  u <= t in one sequence
//   o_t  = sum_u exp(s_tu - lse_t) v_u,   lse_t = log sum_u exp(s_tu)
//   with delta_t = do_t . o_t,  p_tu = exp(s_tu - lse_t),  ds_tu = p_tu (do_t . v_u - delta_t):
//   dv_u = sum_t p_tu do_t,   dk_u = a sum_t ds_tu q_t,   dq_t = a sum_u ds_tu k_u
//   (dk and dv sum over the query heads that share the key head).
//
// Nothing of size T x T is stored. Every product is an MFMA of 32 x 32 tiles
// whose result keeps the free index of the next product in its columns:
//   forward and dq:  S^T = K Q^T      (rows: keys, columns: queries)
//   dk and dv:       S   = Q K^T      (rows: queries, columns: keys)
// A lane then holds one column, 16 rows of it per tile, and those rows are the
// contraction index of the next product (O^T = V^T P^T, dQ^T = K^T dS^T,
// dV^T = dO^T P, dK^T = Q^T dS): the tile goes back into the matrix unit from
// the lane's own registers, rounded to the inputs' type, and the softmax
// statistics of a query are one value a lane. The other operand of that second
// product is the transpose of rows in LDS, read with the transposing LDS read.
//
// MFMA operands of the 32 x 32 tiles: lane l supplies row (or column) l % 32 and
// the K slots of half g = l / 32; of a result, lane l holds rows
// 8 (r / 4) + 4 g + r % 4, r = 0 .. 15, of column l % 32.
//
// Accumulators, statistics, delta and every sum are fp32. The weights p and ds
// are rounded to bf16 for bf16 inputs (half a step, up to 2^-8 relative, as the
// inputs themselves are); the sum of the weights takes them unrounded.
#pragma once
#include <type_traits>

#include "device_common.h"

namespace dpn {
namespace attn {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

struct Tensor {     // [token][head][D], strides in bytes
  char* p;
  int64_t st, sh;
};

struct Args {
  Tensor q, k, v, o, dO, dq, dk, dv;
  float* lse;         // [Hq][N]
  float* pairs;       // [Hq][N][2], backward: lse in units of log 2 and delta, of the first launch for the second
  const int32_t* cu;  // [S + 1], or null: S sequences of T tokens
  int32_t S, T, N;
  int32_t Hq, Hkv, D;
  float scale;        // a
  int32_t slots;      // tile slots per head
  int32_t slot0;      // first slot of the launch
  int32_t clear;      // set rows of no sequence to zero
  // Backward pass of small calls. dq where work groups share a tile's keys (the second
  // launch adds their sums):
  int32_t qsplits;    // work groups of 32 queries of one head, at most
  float* qparts;      // their sums, [slot][head][split][tile][1024]
  uint32_t* qcareful; // [slot][head][split], whether rows were cleaned
  // dk and dv where work groups share their keys' queries:
  int32_t splits;     // work groups of 32 keys of one key head, and
  int32_t groups;     // the number of such groups of 32 keys
  float* parts;       // their sums, [slot][key head][split][dk, dv][tile][1024]
  uint32_t* arrived;  // [slot][key head] of them have arrived (the launch before sets it to zero)
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kOutside = 0x80000000u;   // an offset past every buffer's range: reads as zero

// The sequence and tile of a slot. Slots count the tiles of the sequences one
// after another; a slot past the last tile has none (tiles is then the number of
// all). Offsets outside [0, N] or out of order are clamped, so no row outside the
// tensors is ever touched.
__device__ __forceinline__ bool find_tile(const Args& a, int32_t slot, int rows, int32_t& start, int32_t& len, int32_t& tile,
                                          int32_t& tiles) {
  if (!a.cu) {
    tiles = (a.T + rows - 1) / rows;
    const int32_t s = slot / tiles;
    start = s * a.T;
    len = a.T;
    tile = slot - s * tiles;
    return s < a.S;
  }
  const int lane = __lane_id();
  int32_t before = 0;
  for (int32_t s0 = 0; s0 < a.S; s0 += 64) {
    const int32_t s = s0 + lane;
    int32_t lo = 0, n = 0;
    if (s < a.S) {
      lo = min(max(a.cu[s], 0), a.N);
      n = min(max(a.cu[s + 1], lo), a.N) - lo;
    }
    const int32_t nt = (n + rows - 1) / rows;
    int32_t inc = nt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int32_t up = __shfl_up(inc, o);
      if (lane >= o) inc += up;
    }
    const int32_t total = __builtin_amdgcn_readlane(inc, 63);
    if (slot < before + total) {
      const int l = __builtin_ctzll(__ballot(before + inc > slot));
      start = __builtin_amdgcn_readlane(lo, l);
      len = __builtin_amdgcn_readlane(n, l);
      tiles = __builtin_amdgcn_readlane(nt, l);
      tile = slot - before - (__builtin_amdgcn_readlane(inc, l) - tiles);
      return true;
    }
    before += total;
  }
  tiles = before;
  return false;
}

// The slots without a tile share the rows of no sequence (before the first and
// behind the last) and set them to zero: row(r) is called by the whole block.
template <typename F>
__device__ __forceinline__ void clear_rest(const Args& a, int32_t slot, int32_t tiles, F row) {
  if (!a.clear || !a.cu) return;
  const int32_t first = min(max(a.cu[0], 0), a.N), last = min(max(a.cu[a.S], first), a.N);
  for (int64_t i = slot - tiles; i < (int64_t)first + a.N - last; i += a.slots - tiles)
    row(i < first ? (int32_t)i : (int32_t)(i - first + last));
}
__device__ __forceinline__ void clear_row(const Tensor& t, int32_t row, int32_t h, int32_t bytes) {
  char* p = t.p + row * t.st + h * t.sh;
  for (int32_t b = threadIdx.x * 16; b < bytes; b += blockDim.x * 16) *(uint4*)(p + b) = make_uint4(0, 0, 0, 0);
}

// DC: columns computed, 64, 96 or 128 (D filled up with zeros).
template <bool BF16, int DC>
struct Geo {
  static constexpr int kElem = BF16 ? 2 : 4;
  static constexpr int kPitch = (DC == 96 ? 128 : DC) * kElem;   // LDS bytes of a row
  static constexpr int kChunks = kPitch / 16;                    // 16-byte chunks of an LDS row
  static constexpr int kSwz = kChunks >= 16 ? 1 : 0;             // see swizzle
  static constexpr int kPairs = DC * kElem / 32;                 // chunk pairs: one chunk for each half of the wave
  static constexpr int kTiles = DC / 32;                         // 32-column tiles of a row
};

// Where row r keeps its chunk c: at c ^ (r & 7), and in rows of 256 bytes and
// more at c ^ 2 (r & 7). Eight rows' reads of one chunk, and the four rows x 32
// bytes of a transposing read, then fall on different banks.
template <bool BF16, int DC>
__device__ __forceinline__ int swizzle(int ch, int row) {
  return ch ^ ((row & 7) << Geo<BF16, DC>::kSwz);
}

// Buffer descriptor of the rows from p on (wave-uniform): raw, no stride, all
// that an offset below 2^31 reaches.
typedef int i32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4_t rows_of(const char* p) {
  const uint64_t u = (uint64_t)p;
  i32x4_t r;
  r.x = __builtin_amdgcn_readfirstlane((int)(uint32_t)u);
  r.y = __builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32) & 0xffff);
  r.z = 0x7fffffff;
  r.w = 0x00027000;
  return r;
}

// Pointer to row `row` of the tensor, head h (all wave-uniform).
__device__ __forceinline__ char* row_ptr(const Tensor& t, int64_t row, int32_t h) { return t.p + row * t.st + h * t.sh; }

// 16 or 4 bytes a lane from a buffer straight to LDS at lds + 16 (4) * lane.
// Written out so that the compiler adds no waits for them: `staged` waits.
__device__ __forceinline__ void dma_rows(i32x4_t rows, uint32_t off, int32_t more, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds" ::"v"(off), "s"(rows),
               "s"(__builtin_amdgcn_readfirstlane(lds)), "s"(more)
               : "memory");
}
__device__ __forceinline__ void dma_words(i32x4_t rows, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(off), "s"(rows),
               "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// Steps of ROWS rows of one head of a sequence into LDS by W waves, row-major
// with swizzled chunks. Rows past the sequence and columns past D read as zero.
template <bool BF16, int DC, int ROWS, int W>
struct Stream {
  using G = Geo<BF16, DC>;
  static constexpr int kLoads = ROWS * G::kChunks / (64 * W);    // of a wave
  static constexpr int kApart = 64 * W / G::kChunks;             // rows between a lane's loads
  static constexpr int kKinds = kApart >= 8 ? 1 : 8 / kApart;    // loads until the swizzle of a lane's row repeats
  static_assert(kLoads * 64 * W == ROWS * G::kChunks && kLoads % kKinds == 0, "whole loads");
  const char* p;      // the sequence's first row
  int64_t st;
  uint32_t off[kKinds];   // the lane's first loads: row, chunk
  int row;
  __device__ __forceinline__ Stream(const Tensor& t, int64_t start, int32_t h, int32_t D) {
    p = row_ptr(t, start, h);
    st = t.st;
    const int at = W == 1 ? threadIdx.x & 63 : threadIdx.x;
    row = at / G::kChunks;
#pragma unroll
    for (int j = 0; j < kKinds; ++j) {
      const int r = row + j * kApart, ch = swizzle<BF16, DC>(at % G::kChunks, r);
      off[j] = ch * 16 < D * G::kElem ? (uint32_t)(r * (int32_t)st + ch * 16) : kOutside;
    }
  }
  __device__ __forceinline__ void head(const Tensor& t, int64_t start, int32_t h) { p = row_ptr(t, start, h); }
  __device__ __forceinline__ void fetch(int32_t r0, int32_t len, uint32_t lds) const {
    const i32x4_t rows = rows_of(p + r0 * st);
    const uint32_t to = lds + (W == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024);
    const int32_t left = len - r0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t o = off[i % kKinds];
      const int32_t more = i / kKinds * kKinds * kApart * (int32_t)st;
      if (left >= ROWS) dma_rows(rows, o, more, to + i * W * 1024);
      else dma_rows(rows, row + i * kApart < left ? o : kOutside, more, to + i * W * 1024);
    }
  }
};

// This wave's direct loads have landed, and then every wave's; and every wave
// has read what it read from LDS before.
__device__ __forceinline__ void staged() {
  DPN_WAIT_VMCNT(0);
  __syncthreads();
}

// The same for rows that only this wave loads and reads.
__device__ __forceinline__ void own_staged() {
  __builtin_amdgcn_s_waitcnt(0x70);   // vmcnt(0) lgkmcnt(0)
  asm volatile("" ::: "memory");
}

// The wave's 32 stationary rows as an operand: lane l has row l % 32, chunk
// 2 i + l / 32 of pair i.
template <bool BF16, int DC>
__device__ __forceinline__ void load_operand(const Tensor& t, int64_t start, int32_t h, int32_t r0, int32_t len, int32_t D,
                                             uint4 (&f)[Geo<BF16, DC>::kPairs]) {
  using G = Geo<BF16, DC>;
  const __amdgpu_buffer_rsrc_t rs =
      __builtin_amdgcn_make_buffer_rsrc((void*)row_ptr(t, start + r0, h), 0, 0x7fffffff, 0x00027000);
  const int lane = threadIdx.x & 63, row = lane & 31, g = lane >> 5;
#pragma unroll
  for (int i = 0; i < G::kPairs; ++i) {
    const int ch = 2 * i + g;
    const bool in = r0 + row < len && ch * 16 < D * G::kElem;
    f[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                         rs, in ? (uint32_t)(row * (int32_t)t.st + ch * 16) : kOutside, 0, 0));
  }
}

template <bool BF16>
__device__ __forceinline__ f32x16_t mfma_chunk(const uint4& a, const uint4& b, f32x16_t c) {
  if constexpr (BF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(word(a, j)), __uint_as_float(word(b, j)), c, 0, 0, 0);
    return c;
  }
}

// 32 rows of LDS (at row r0, a multiple of 8) times the stationary operand: X f^T. A
// wave here yields to one in its softmax or second products (dq, dk and dv 2 % faster).
template <bool BF16, int DC>
__device__ __forceinline__ f32x16_t rows_times(const unsigned char* lds, int r0, const uint4 (&f)[Geo<BF16, DC>::kPairs]) {
  using G = Geo<BF16, DC>;
  const int lane = threadIdx.x & 63, row = lane & 31, g = lane >> 5;
  f32x16_t c = {};
  __builtin_amdgcn_s_setprio(0);
#pragma unroll
  for (int i = 0; i < G::kPairs; ++i) {
    const uint4 a = *(const uint4*)(lds + (row * G::kPitch + (swizzle<BF16, DC>(2 * i + g, row) << 4)) + r0 * G::kPitch);
    c = mfma_chunk<BF16>(a, f[i], c);
  }
  __builtin_amdgcn_s_setprio(1);
  return c;
}

// Eight weights of a column as an operand, rounded to bf16.
__device__ __forceinline__ uint4 pack_weights(const f32x16_t& w, int j) {
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){w[j + 2 * i], w[j + 2 * i + 1]}, bf16x2_t));
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// acc[tile] += (rows r0 .. r0 + 31 of LDS)^T w, where w's rows are those rows.
template <bool BF16, int DC>
__device__ __forceinline__ void columns_times(const unsigned char* lds, int r0, const f32x16_t& w,
                                              f32x16_t (&acc)[Geo<BF16, DC>::kTiles]) {
  using G = Geo<BF16, DC>;
  const int lane = threadIdx.x & 63, g = lane >> 5;
  if constexpr (BF16) {
    const int j = (lane >> 2) & 3, q = lane & 3, m0 = ((lane >> 4) & 1) * 16;
    const int row = 4 * g + j;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const uint4 b = pack_weights(w, ks * 8);
#pragma unroll
      for (int t = 0; t < G::kTiles; ++t) {
        const int ch = (t * 32 + m0 + 4 * q) >> 3;
        const unsigned char* p = lds + (row * G::kPitch + (swizzle<BF16, DC>(ch, row) << 4) + (q & 1) * 8) + (r0 + ks * 16) * G::kPitch;
        const uint2 lo = lds_read_tr16(p), hi = lds_read_tr16(p + 8 * G::kPitch);
        acc[t] = mfma_chunk<true>(make_uint4(lo.x, lo.y, hi.x, hi.y), b, acc[t]);
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = 4 * g + (r & 3);
#pragma unroll
      for (int t = 0; t < G::kTiles; ++t) {
        const int col = t * 32 + (lane & 31);
        const float x = *(const float*)(lds + (row * G::kPitch + (swizzle<BF16, DC>(col >> 2, row) << 4) + (col & 3) * 4) +
                                        (r0 + 8 * (r >> 2)) * G::kPitch);
        acc[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, w[r], acc[t], 0, 0, 0);
      }
    }
  }
}

// Keeps a uniform branch a branch: without it the compiler computes the masks
// of every step, of which one or two at the diagonal need them.
__device__ __forceinline__ void keep_branch() { asm volatile(""); }

// Halves (bf16) or words (fp32) of x that are infinities or NaN, as a mask.
template <bool BF16>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  if constexpr (BF16) {
    const uint32_t top = ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u;   // bit 15 of a half whose exponent is all ones
    return (top >> 15) * 0xffffu;
  } else {
    return (x & 0x7f800000u) == 0x7f800000u ? ~0u : 0u;
  }
}

// Whether some sum of the wave is an infinity or NaN (times zero, it is NaN).
template <int TILES>
__device__ __forceinline__ bool not_all_finite(const f32x16_t (&acc)[TILES]) {
  float z[2] = {0.f, 0.f};
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) z[r & 1] = fmaf(acc[t][r], 0.f, z[r & 1]);
  return __builtin_expect(__any(!(z[0] + z[1] == 0.f)), 0);
}

// Causality holds for infinities and NaN. A masked row has weights of zero, and as a
// product an infinity or NaN in it would still add NaN; only the 32 rows on a wave's
// diagonal are masked for some of its columns and not for others. There such entries
// are set to zero for the product, and added afterwards to the results of the rows
// that see them. The output and dq do so in a second pass of a wave whose sums come
// out not finite. dk and dv take each step on the diagonal so: a second pass would
// cost them registers (D 128, 4 x 1024: 257 us without the guard, 282 with it, 307
// with a second pass; D 64, 4 x 2048: 239, 252, 262). Before the first products, so
// that an infinity of dO there reaches dk through delta alone, as an infinity or NaN
// (after them 303; D 64 248).

// 32 rows in LDS, the wave's own: infinities and NaN become zero. Returns whether any were.
template <bool BF16, int DC>
__device__ __forceinline__ bool zero_not_finite(unsigned char* lds) {
  uint32_t any = 0;
#pragma unroll 1
  for (int i = 0; i < 32 * Geo<BF16, DC>::kChunks / 64; ++i) {
    uint4* p = (uint4*)(lds + (i * 64 + (threadIdx.x & 63)) * 16);
    const uint4 x = *p;
    const uint4 n = make_uint4(not_finite<BF16>(x.x), not_finite<BF16>(x.y), not_finite<BF16>(x.z), not_finite<BF16>(x.w));
    if (__builtin_expect(__any(n.x | n.y | n.z | n.w), 0)) {
      any = 1;
      *p = make_uint4(x.x & ~n.x, x.y & ~n.y, x.z & ~n.z, x.w & ~n.w);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return any;
}

// Adds the infinities and NaN of rows w0 .. w0 + 31 of head hs of src to the results
// of head ho that see them: those of the same and later rows (UP) or of the same and
// earlier ones; as they are, or as NaN (weights of either sign). By one wave.
template <bool BF16, bool UP, bool AS_NAN>
__device__ __forceinline__ void add_not_finite(const Tensor& src, int32_t hs, const Tensor& out, int32_t ho, int64_t start,
                                               int32_t len, int32_t w0, int32_t D) {
  constexpr int e = BF16 ? 2 : 4;
  for (int32_t d = threadIdx.x & 63; d < D; d += 64) {
    float bad = 0.f;
    for (int i = 0; i < 32; ++i) {
      const int32_t row = w0 + (UP ? i : 31 - i);
      if (row >= len) continue;
      const char* p = row_ptr(src, start + row, hs) + d * e;
      const uint32_t x = BF16 ? (uint32_t)*(const uint16_t*)p << 16 : *(const uint32_t*)p;
      if ((x & 0x7f800000u) == 0x7f800000u) bad += AS_NAN ? NAN : __uint_as_float(x);
      if (bad == 0.f) continue;
      char* q = row_ptr(out, start + row, ho) + d * e;
      if constexpr (BF16) *(uint16_t*)q = (uint16_t)f32_to_bf16_bits(bf16_bits_to_f32(*(const uint16_t*)q) + bad);
      else *(float*)q += bad;
    }
  }
}

// The value of the lane's column in the other half of the wave.
__device__ __forceinline__ float other_half(float x) {
  const auto y = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float((threadIdx.x & 32) ? y[0] : y[1]);
}

// Row r (0 .. 15) of a lane's half in a 32 x 32 result.
__device__ __forceinline__ int result_row(int r, int g) { return 8 * (r >> 2) + 4 * g + (r & 3); }

// Tile i (32 columns) of a row at p, from the transposed result acc, times f.
template <bool BF16>
__device__ __forceinline__ void store_tile(char* p, int i, int32_t D, const f32x16_t& acc, float f) {
  const int g = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int r4 = 0; r4 < 4; ++r4) {
    const int col = i * 32 + 8 * r4 + 4 * g;
    if (col >= D) continue;
    const float x[4] = {acc[4 * r4] * f, acc[4 * r4 + 1] * f, acc[4 * r4 + 2] * f, acc[4 * r4 + 3] * f};
    if constexpr (BF16) {
      uint2 y;
      y.x = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){x[0], x[1]}, bf16x2_t));
      y.y = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){x[2], x[3]}, bf16x2_t));
      *(uint2*)(p + col * 2) = y;
    } else {
      *(float4*)(p + col * 4) = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
}

// Columns of acc (transposed: rows are the D index) to row `row` of t, times f.
template <bool BF16, int DC>
__device__ __forceinline__ void store_rows(const Tensor& t, int64_t row, int32_t h, int32_t D,
                                           const f32x16_t (&acc)[Geo<BF16, DC>::kTiles], float f) {
  using G = Geo<BF16, DC>;
  char* p = t.p + row * t.st + h * t.sh;
#pragma unroll
  for (int i = 0; i < G::kTiles; ++i) store_tile<BF16>(p, i, D, acc[i], f);
}

// Blocks: x is the key head, y the query head of that key head, z the slot
// (from slot0 on). Blocks go to the 8 XCDs in turn, so the blocks that read one
// key head meet in one L2 when Hkv is a multiple or a divisor of 8.
__device__ __forceinline__ int32_t block_slot(const Args& a) { return a.slot0 + (int32_t)blockIdx.z; }

// Two forms of work groups.
//
// Tiles: 128 stationary rows, 32 a wave, whose four waves share 64 streamed rows
// a step in LDS. The least traffic and LDS writing a product.
//
// Rows: 32 stationary rows, whose NS waves take 32 streamed rows each in turn,
// from LDS of their own, so that no wave waits for another; their sums are joined
// at the end. Four times the work groups and shorter chains of steps.
template <bool BF16, int DC>
struct Tiles {
  using G = Geo<BF16, DC>;
  static constexpr int kWaves = 4, kThreads = 64 * kWaves, kRows = 128, kStep = 64;
  static constexpr int kStage = kStep * G::kPitch;   // bytes of one tensor's step
  using Rows = Stream<BF16, DC, kStep, kWaves>;      // double buffered
};

// Bytes of a wave's own step are kBuf, for two tensors and the kExtra of dk and
// dv. Two buffers where two work groups of them fit a CU: a second work group
// hides more of the loads' latency than a second buffer (dk and dv of
// B = 4, T = 2048, 16/4 heads, D = 128: 273 us with one buffer, 343 with two).
template <bool BF16, int DC, int NS, int EXTRA>
struct OwnRows {
  using G = Geo<BF16, DC>;
  static constexpr int kStage = 32 * G::kPitch, kBuf = 2 * kStage + EXTRA;
  static constexpr int kBuffers = NS * 2 * kBuf <= 80 * 1024 ? 2 : 1;
  static constexpr int kLds = NS * kBuffers * kBuf;
  using Rows = Stream<BF16, DC, 32, 1>;
};

// Adds the accumulators of the waves of a work group, in wave order, to the
// first one's. `lds` is free; every wave of the block calls it.
template <int NS, int TILES>
__device__ __forceinline__ void join(f32x16_t (&acc)[TILES], int split, unsigned char* lds) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    __syncthreads();
    if (split > 0) {
      f32x4_t* p = (f32x4_t*)(lds + (split - 1) * 4096) + lane;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        p[64 * j] = f32x4_t{acc[t][4 * j], acc[t][4 * j + 1], acc[t][4 * j + 2], acc[t][4 * j + 3]};
    }
    __syncthreads();
    if (split == 0) {
#pragma unroll
      for (int s = 1; s < NS; ++s) {
        const f32x4_t* p = (const f32x4_t*)(lds + (s - 1) * 4096) + lane;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4_t x = p[64 * j];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][4 * j + i] += x[i];
        }
      }
    }
  }
}

// The counters of a backward pass's second launch, set to zero by its first.
__device__ __forceinline__ void clear_arrived(const Args& a) {
  if (a.splits < 2) return;
  const int64_t block = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  const int64_t blocks = (int64_t)gridDim.x * gridDim.y * gridDim.z;
  for (int64_t i = block * blockDim.x + threadIdx.x; i < a.groups; i += blocks * blockDim.x) a.arrived[i] = 0;
}

// Largest growth of a score, in powers of two, that a wave lets pass without
// rescaling its sums: the weights stay below 2^8 and the sums far inside fp32.
constexpr float kGrowth = 8.f;

// One wave's pass over the keys k0, k0 + 32 NS, .. up to its 32 queries from w0 on,
// from LDS of its own. careful: without the infinities and NaN on the diagonal.
template <bool BF16, int DC, int NS, int BUFFERS>
__device__ __forceinline__ void forward_pass(bool careful, const Args& a, int32_t start, int32_t len, int32_t kh,
                                             int32_t w0, int32_t k0, unsigned char* mine, const uint4 (&q)[Geo<BF16, DC>::kPairs], float& m, float& l,
                                             f32x16_t (&acc)[Geo<BF16, DC>::kTiles]) {
  using G = Geo<BF16, DC>;
  using Rows = Stream<BF16, DC, 32, 1>;
  constexpr int kStage = 32 * G::kPitch, kBuf = 2 * kStage;
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int32_t query = w0 + (lane & 31);
  const float c = a.scale * kLog2e;
  const uint32_t base = lds_address(mine);
  const Rows ks(a.k, start, kh, a.D), vs(a.v, start, kh, a.D);
  const auto fetch = [&](int32_t r0, uint32_t to) {
    ks.fetch(r0, len, to);
    vs.fetch(r0, len, to + kStage);
  };
  if (k0 <= w0) fetch(k0, base);
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int t = 0; t < G::kTiles; ++t) acc[t] = f32x16_t{};
  int buf = 0;
  for (; k0 <= w0; k0 += 32 * NS) {
    own_staged();
    const bool more = k0 + 32 * NS <= w0;
    if (BUFFERS == 2 && more) fetch(k0 + 32 * NS, base + (buf ^ 1) * kBuf);
    unsigned char* lk = mine + buf * kBuf;
    unsigned char* lv = lk + kStage;
    f32x16_t s = rows_times<BF16, DC>(lk, 0, q);
    if (k0 == w0) {
      keep_branch();
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (k0 + result_row(r, g) > query) s[r] = -INFINITY;
    }
    float x[2] = {s[0], s[1]};
#pragma unroll
    for (int r = 2; r < 16; ++r) x[r & 1] = fmaxf(x[r & 1], s[r]);
    float top = fmaxf(x[0], x[1]);
    top = fmaxf(top, other_half(top));
    const bool grown = (top - m) * c > kGrowth;
    if (__any(grown)) {   // (each query by its own scores alone)
      keep_branch();
      const float f = grown ? __builtin_amdgcn_exp2f((m - top) * c) : 1.f;
      m = grown ? top : m;
      l *= f;
#pragma unroll
      for (int t = 0; t < G::kTiles; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[t][r] *= f;
    }
    // (queries that see none of a split's keys so far: every weight 0)
    const float mc = m == -INFINITY ? 0.f : m * c;
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -mc));
      sum[r & 1] += s[r];
    }
    l += sum[0] + sum[1];
    if (careful && k0 == w0) zero_not_finite<BF16, DC>(lv);
    columns_times<BF16, DC>(lv, 0, s, acc);
    if (BUFFERS == 2) {
      buf ^= 1;
    } else if (more) {
      own_staged();   // (the reads of this step are done)
      fetch(k0 + 32 * NS, base);
    }
  }
}

// The output by rows: 32 queries of one head, the keys split over NS waves, each with
// LDS and running softmax of its own and no barrier before the sums are joined. The
// chain of a work group is a quarter of the tiles' and its loads are used by 32 queries
// instead of 128: for few work groups, bound by the latency of a chain's steps (T = 1024,
// 16/4 heads, D = 64: 11.6 us against 18.7 by tiles; 4 sequences of 107 rows: 6 us).
template <bool BF16, int DC, int NS>
__global__ __launch_bounds__(64 * NS, BF16 ? 2 : 1) void k_forward_rows(Args a) {
  using G = Geo<BF16, DC>;
  using P = OwnRows<BF16, DC, NS, 0>;
  __shared__ __align__(1024) unsigned char lds[P::kLds];
  int32_t start, len, tile, tiles;
  if (!find_tile(a, block_slot(a), 32, start, len, tile, tiles)) {
    clear_rest(a, block_slot(a), tiles, [&](int32_t r) {
      clear_row(a.o, r, blockIdx.x * gridDim.y + blockIdx.y, a.D * G::kElem);
      if (threadIdx.x == 0) a.lse[(int64_t)(blockIdx.x * gridDim.y + blockIdx.y) * a.N + r] = 0.f;
    });
    return;
  }
  tile = tiles - 1 - tile;
  const int32_t kh = blockIdx.x, h = kh * gridDim.y + blockIdx.y;
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int split = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t w0 = tile * 32, query = w0 + (lane & 31);
  uint4 q[G::kPairs];
  load_operand<BF16, DC>(a.q, start, h, w0, len, a.D, q);
  const float c = a.scale * kLog2e;
  float m, l;
  f32x16_t acc[G::kTiles];
  unsigned char* mine = lds + split * P::kBuffers * P::kBuf;
  bool careful = false;
#pragma unroll 1
  for (;;) {
    forward_pass<BF16, DC, NS, P::kBuffers>(careful, a, start, len, kh, w0, 32 * split, mine, q, m, l, acc);
    if (careful || !not_all_finite(acc)) break;
    careful = true;
  }
  careful = __syncthreads_or(careful);
  l += other_half(l);
  if constexpr (NS > 1) {
    // the splits' sums on the scale of their common largest score
    float* st = (float*)lds;
    __syncthreads();
    st[split * 64 + lane] = m;
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < NS; ++i) top = fmaxf(top, st[i * 64 + lane]);
    const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f((m - top) * c);
    m = top;
    __syncthreads();
    st[split * 64 + lane] = l * f;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) l += st[i * 64 + lane];
#pragma unroll
    for (int t = 0; t < G::kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[t][r] *= f;
    join<NS, G::kTiles>(acc, split, lds);
    if (split > 0) return;
  }
  if (query < len) {
    store_rows<BF16, DC>(a.o, (int64_t)start + query, h, a.D, acc, 1.f / l);
    if (g == 0) a.lse[(int64_t)h * a.N + start + query] = fmaf(m, a.scale, logf(l));
  }
  if (careful) {
    __threadfence_block();
    add_not_finite<BF16, true, false>(a.v, kh, a.o, h, start, len, w0, a.D);
  }
}

// A step of 64 keys from r0 on by tiles, before its weights: masks the scores, raises
// the running maximum and rescales the sums. Returns the maximum in powers of two.
template <bool BF16, int DC>
__device__ __forceinline__ float raise_maximum(f32x16_t (&s)[2], int32_t r0, int32_t w0, int32_t query, float c, float& m, float& l,
                                               f32x16_t (&acc)[Geo<BF16, DC>::kTiles]) {
  using G = Geo<BF16, DC>;
  const int g = (threadIdx.x & 63) >> 5;
  if (r0 + 63 > w0) {
    keep_branch();
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (r0 + t * 32 + result_row(r, g) > query) s[t][r] = -INFINITY;
  }
  float x[4] = {s[0][0], s[0][1], s[0][2], s[0][3]};
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) x[r & 3] = fmaxf(x[r & 3], s[t][r]);
  float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  top = fmaxf(top, other_half(top));
  const bool grown = (top - m) * c > kGrowth;
  if (__any(grown)) {   // (each query by its own scores alone)
    keep_branch();
    const float f = grown ? __builtin_amdgcn_exp2f((m - top) * c) : 1.f;
    m = grown ? top : m;
    l *= f;
#pragma unroll
    for (int t = 0; t < G::kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[t][r] *= f;
  }
  return m == -INFINITY ? 0.f : m * c;   // (scores of -infinity alone have weights of zero)
}

// The step's scores become its weights, and join the sum.
__device__ __forceinline__ void weigh(f32x16_t (&s)[2], float c, float mc, float& l) {
  float sum[2] = {0.f, 0.f};
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[t][r] = __builtin_amdgcn_exp2f(fmaf(s[t][r], c, -mc));
      sum[r & 1] += s[t][r];
    }
  l += sum[0] + sum[1];
}

// A wave's queries of k_forward once more, without the infinities and NaN of values that
// some of them do not see. The same steps and operations, so that queries whose sums were
// finite keep their bits; keys and values in turn in the wave's quarter of the LDS.
template <bool BF16, int DC>
__device__ __forceinline__ void tile_again(const Args& a, int32_t start, int32_t len, int32_t kh, int32_t w0, unsigned char* mine,
                                           const uint4 (&q)[Geo<BF16, DC>::kPairs], float& m, float& l,
                                           f32x16_t (&acc)[Geo<BF16, DC>::kTiles]) {
  using G = Geo<BF16, DC>;
  const float c = a.scale * kLog2e;
  const int32_t query = w0 + (threadIdx.x & 31);
  const Stream<BF16, DC, 64, 1> ks(a.k, start, kh, a.D), vs(a.v, start, kh, a.D);
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int t = 0; t < G::kTiles; ++t) acc[t] = f32x16_t{};
#pragma unroll 1
  for (int32_t r0 = 0; r0 <= w0; r0 += 64) {
    own_staged();   // (the reads of the step before are done)
    ks.fetch(r0, len, lds_address(mine));
    own_staged();
    f32x16_t s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) s[t] = rows_times<BF16, DC>(mine, t * 32, q);
    own_staged();
    vs.fetch(r0, len, lds_address(mine));
    const float mc = raise_maximum<BF16, DC>(s, r0, w0, query, c, m, l, acc);
    weigh(s, c, mc, l);
    own_staged();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (r0 + t * 32 >= w0) zero_not_finite<BF16, DC>(mine + t * 32 * G::kPitch);
      columns_times<BF16, DC>(mine, t * 32, s[t], acc);
    }
  }
}

// The output by tiles: 128 queries of one head, 32 a wave, which share steps of 64 keys
// in two LDS buffers. Longest tiles first, so that the short ones fill the end. The scores
// of the next step are computed beside the weights of this one: what bounds it is a
// wave's exponentials, maxima and sums, about as long as its MFMAs, and two or three
// work groups a CU so that one wave's run beside another's. B = 4, T = 2048, 32/8 heads,
// D = 64: 104 us, 661 TF/s of the pairs u <= t; 12289 + 777 + 4100 rows, 16/2 heads,
// D = 128: 713 us, 968 TF/s. A large bf16 matrix product reaches 1241 TF/s.
template <bool BF16, int DC>
__global__ __launch_bounds__(256, BF16 ? 2 : 1) void k_forward(Args a) {
  using G = Geo<BF16, DC>;
  using P = Tiles<BF16, DC>;
  // keys are needed a step ahead of their values, whose scores they give
  __shared__ __align__(1024) unsigned char lds[4 * P::kStage];
  int32_t start, len, tile, tiles;
  if (!find_tile(a, block_slot(a), P::kRows, start, len, tile, tiles)) {
    clear_rest(a, block_slot(a), tiles, [&](int32_t r) {
      clear_row(a.o, r, blockIdx.x * gridDim.y + blockIdx.y, a.D * G::kElem);
      if (threadIdx.x == 0) a.lse[(int64_t)(blockIdx.x * gridDim.y + blockIdx.y) * a.N + r] = 0.f;
    });
    return;
  }
  tile = tiles - 1 - tile;   // the longest rows first
  const int32_t kh = blockIdx.x, h = kh * gridDim.y + blockIdx.y;
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t w0 = tile * P::kRows + wv * 32;   // the wave's first query
  const int32_t query = w0 + (lane & 31);
  const uint32_t base = lds_address(lds);
  const int32_t end = min(tile * P::kRows + P::kRows, len);   // keys that some query of the block sees
  const typename P::Rows ks(a.k, start, kh, a.D), vs(a.v, start, kh, a.D);
  ks.fetch(0, len, base);
  vs.fetch(0, len, base + 2 * P::kStage);
  if (P::kStep < end) ks.fetch(P::kStep, len, base + P::kStage);
  uint4 q[G::kPairs];
  load_operand<BF16, DC>(a.q, start, h, w0, len, a.D, q);
  const float c = a.scale * kLog2e;
  float m = -INFINITY, l = 0.f;
  f32x16_t acc[G::kTiles] = {};
  f32x16_t even[2], odd[2];   // scores of the even and the odd steps
  staged();
#pragma unroll
  for (int t = 0; t < 2; ++t) even[t] = rows_times<BF16, DC>(lds, t * 32, q);
  __syncthreads();
  const auto step = [&](int32_t r0, f32x16_t (&s)[2], f32x16_t (&next)[2], auto buffer) {
    constexpr int buf = buffer.value;
    if (r0 + P::kStep < end) vs.fetch(r0 + P::kStep, len, base + (2 + (buf ^ 1)) * P::kStage);
    if (r0 + 2 * P::kStep < end) ks.fetch(r0 + 2 * P::kStep, len, base + buf * P::kStage);
    if (r0 <= w0 + 31) {
      const float mc = raise_maximum<BF16, DC>(s, r0, w0, query, c, m, l, acc);
      // the next step's scores fill the matrix unit while this step's weights are computed
#pragma unroll
      for (int t = 0; t < 2; ++t) next[t] = rows_times<BF16, DC>(lds + (buf ^ 1) * P::kStage, t * 32, q);
      weigh(s, c, mc, l);
      const unsigned char* lv = lds + (2 + buf) * P::kStage;
#pragma unroll
      for (int t = 0; t < 2; ++t) columns_times<BF16, DC>(lv, t * 32, s[t], acc);
    }
    staged();
  };
  for (int32_t r0 = 0; r0 < end;) {
    step(r0, even, odd, std::integral_constant<int, 0>{});
    r0 += P::kStep;
    if (r0 >= end) break;
    step(r0, odd, even, std::integral_constant<int, 1>{});
    r0 += P::kStep;
  }
  // Masked values may have added NaN: the wave takes its queries once more, from its
  // quarter of the LDS (every wave is past the last step).
  const bool careful = not_all_finite(acc);
  if (careful) tile_again<BF16, DC>(a, start, len, kh, w0, lds + wv * P::kStage, q, m, l, acc);
  l += other_half(l);
  if (query < len) {
    store_rows<BF16, DC>(a.o, (int64_t)start + query, h, a.D, acc, 1.f / l);
    if (g == 0) a.lse[(int64_t)h * a.N + start + query] = fmaf(m, a.scale, logf(l));
  }
  if (careful) {
    __threadfence_block();
    add_not_finite<BF16, true, false>(a.v, kh, a.o, h, start, len, w0, a.D);
  }
}

// dot product of two 16-byte chunks
template <bool BF16>
__device__ __forceinline__ float dot_chunk(const uint4& x, const uint4& y, float s) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t u = word(x, j), v = word(y, j);
    if constexpr (BF16) {
      s = fmaf(__uint_as_float(u << 16), __uint_as_float(v << 16), s);
      s = fmaf(__uint_as_float(u & 0xffff0000u), __uint_as_float(v & 0xffff0000u), s);
    } else {
      s = fmaf(__uint_as_float(u), __uint_as_float(v), s);
    }
  }
  return s;
}

// lse in units of log 2. A query all of whose scores are -infinity has no weights: NaN,
// also against scores that are computed without the row's infinities.
__device__ __forceinline__ float scaled_lse(float lse) { return lse == -INFINITY ? NAN : lse * kLog2e; }

// One wave's pass for dq over the keys k0, k0 + 32 waves, .., as forward_pass.
template <bool BF16, int DC, int BUFFERS>
__device__ __forceinline__ void backward_q_pass(bool careful, const Args& a, int32_t start, int32_t len, int32_t kh,
                                                int32_t w0, int32_t k0, int32_t waves, unsigned char* mine, const uint4 (&q)[Geo<BF16, DC>::kPairs],
                                                const uint4 (&dO)[Geo<BF16, DC>::kPairs], float lse, float delta,
                                                f32x16_t (&acc)[Geo<BF16, DC>::kTiles]) {
  using G = Geo<BF16, DC>;
  using Rows = Stream<BF16, DC, 32, 1>;
  constexpr int kStage = 32 * G::kPitch, kBuf = 2 * kStage;
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int32_t query = w0 + (lane & 31);
  const float c = a.scale * kLog2e;
  const uint32_t base = lds_address(mine);
  const Rows ks(a.k, start, kh, a.D), vs(a.v, start, kh, a.D);
  const auto fetch = [&](int32_t r0, uint32_t to) {
    ks.fetch(r0, len, to);
    vs.fetch(r0, len, to + kStage);
  };
  if (k0 <= w0) fetch(k0, base);
#pragma unroll
  for (int t = 0; t < G::kTiles; ++t) acc[t] = f32x16_t{};
  int buf = 0;
  for (; k0 <= w0; k0 += 32 * waves) {
    own_staged();
    const bool more = k0 + 32 * waves <= w0;
    if (BUFFERS == 2 && more) fetch(k0 + 32 * waves, base + (buf ^ 1) * kBuf);
    unsigned char* lk = mine + buf * kBuf;
    unsigned char* lv = lk + kStage;
    f32x16_t s = rows_times<BF16, DC>(lk, 0, q);
    const f32x16_t dp = rows_times<BF16, DC>(lv, 0, dO);
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse)) * (dp[r] - delta);
    if (k0 == w0) {
      keep_branch();
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (k0 + result_row(r, g) > query) s[r] = 0.f;
      if (careful) zero_not_finite<BF16, DC>(lk);
    }
    columns_times<BF16, DC>(lk, 0, s, acc);
    if (BUFFERS == 2) {
      buf ^= 1;
    } else if (more) {
      own_staged();   // (the reads of this step are done)
      fetch(k0 + 32 * waves, base);
    }
  }
}

// dq, and the pairs for the second launch, by tiles as k_forward's. Three products a
// step (S, dP, dQ); bound by the MFMAs and the reads of K and V from LDS, each used by
// 32 queries a wave. B = 4, T = 2048, 32/8 heads, D = 64: 131 us, 787 TF/s.
template <bool BF16, int DC>
__global__ __launch_bounds__(256, !BF16 ? 1 : DC == 64 ? 3 : 2) void k_backward_q(Args a) {
  using G = Geo<BF16, DC>;
  using P = Tiles<BF16, DC>;
  __shared__ __align__(1024) unsigned char lds[4 * P::kStage];
  clear_arrived(a);
  int32_t start, len, tile, tiles;
  if (!find_tile(a, block_slot(a), P::kRows, start, len, tile, tiles)) {
    clear_rest(a, block_slot(a), tiles, [&](int32_t r) {
      clear_row(a.dq, r, blockIdx.x * gridDim.y + blockIdx.y, a.D * G::kElem);
    });
    return;
  }
  tile = tiles - 1 - tile;
  const int32_t kh = blockIdx.x, h = kh * gridDim.y + blockIdx.y;
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t w0 = tile * P::kRows + wv * 32;
  const int32_t query = w0 + (lane & 31);
  const uint32_t base = lds_address(lds);
  const int32_t end = min(tile * P::kRows + P::kRows, len);
  const typename P::Rows ks(a.k, start, kh, a.D), vs(a.v, start, kh, a.D);
  ks.fetch(0, len, base);
  vs.fetch(0, len, base + P::kStage);
  uint4 q[G::kPairs], dO[G::kPairs];
  float delta = 0.f;
  {
    uint4 o[G::kPairs];
    load_operand<BF16, DC>(a.dO, start, h, w0, len, a.D, dO);
    load_operand<BF16, DC>(a.o, start, h, w0, len, a.D, o);
    load_operand<BF16, DC>(a.q, start, h, w0, len, a.D, q);
#pragma unroll
    for (int i = 0; i < G::kPairs; ++i) delta = dot_chunk<BF16>(dO[i], o[i], delta);
    delta += other_half(delta);
  }
  float lse = 0.f;
  if (query < len) {
    const int64_t at = (int64_t)h * a.N + start + query;
    lse = scaled_lse(a.lse[at]);
    if (g == 0) {
      *(float2*)(a.pairs + 2 * at) = make_float2(lse, delta);
    }
  }
  const float c = a.scale * kLog2e;
  f32x16_t acc[G::kTiles] = {};
  staged();
  int buf = 0;
  for (int32_t r0 = 0; r0 < end; r0 += P::kStep) {
    if (r0 + P::kStep < end) {
      const uint32_t to = base + (buf ^ 1) * 2 * P::kStage;
      ks.fetch(r0 + P::kStep, len, to);
      vs.fetch(r0 + P::kStep, len, to + P::kStage);
    }
    if (r0 <= w0 + 31) {
      const unsigned char* lk = lds + buf * 2 * P::kStage;
      const unsigned char* lv = lk + P::kStage;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int32_t k0 = r0 + t * 32;
        if (k0 > w0) break;   // (all masked)
        f32x16_t s = rows_times<BF16, DC>(lk, t * 32, q);
        const f32x16_t dp = rows_times<BF16, DC>(lv, t * 32, dO);
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse)) * (dp[r] - delta);
        if (k0 == w0) {
          keep_branch();
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (k0 + result_row(r, g) > query) s[r] = 0.f;
        }
        columns_times<BF16, DC>(lk, t * 32, s, acc);
      }
    }
    staged();
    buf ^= 1;
  }
  const bool careful = not_all_finite(acc);   // see k_forward
  if (careful) backward_q_pass<BF16, DC, 1>(true, a, start, len, kh, w0, 0, 1, lds + wv * P::kStage, q, dO, lse, delta, acc);
  if (query < len) store_rows<BF16, DC>(a.dq, (int64_t)start + query, h, a.D, acc, a.scale);
  if (careful) {
    __threadfence_block();
    add_not_finite<BF16, true, true>(a.k, kh, a.dq, h, start, len, w0, a.D);
  }
}

// Work groups that share the keys of the 32 queries from w0 on, for kSteps steps a wave.
constexpr int kSteps = 2;
__device__ __forceinline__ int32_t query_splits(const Args& a, int32_t w0, int ns) {
  return min(a.qsplits, (w0 / 32 + kSteps * ns) / (kSteps * ns));
}

// The same by rows, as k_forward_rows. SPLIT: a few work groups share the keys, and the
// second launch adds their sums in order (join_queries): float32, 515 + 130 + 62 rows,
// 6/3 heads, D = 80 37 us alone, 22 shared; T = 1024, 8/4 heads, D = 64 39 either way;
// bf16, T = 1024, 16/4 heads, D = 64 16 alone. Bound by the chain of a wave's steps and,
// below 12 us, by its first loads.
template <bool BF16, int DC, int NS, bool SPLIT>
__global__ __launch_bounds__(64 * NS, BF16 ? 2 : 1) void k_backward_q_rows(Args a) {
  using G = Geo<BF16, DC>;
  using P = OwnRows<BF16, DC, NS, 0>;
  __shared__ __align__(1024) unsigned char lds[P::kLds];
  clear_arrived(a);
  const int32_t kh = blockIdx.x, rep = a.Hq / a.Hkv;
  const int32_t h = kh * rep + (SPLIT ? (int32_t)blockIdx.y % rep : (int32_t)blockIdx.y);
  const int32_t z = SPLIT ? (int32_t)blockIdx.y / rep : 0;
  int32_t start, len, tile, tiles;
  if (!find_tile(a, block_slot(a), 32, start, len, tile, tiles)) {
    if (z == 0) clear_rest(a, block_slot(a), tiles, [&](int32_t r) { clear_row(a.dq, r, h, a.D * G::kElem); });
    return;
  }
  tile = tiles - 1 - tile;
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int split = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t w0 = tile * 32, query = w0 + (lane & 31);
  const int32_t splits = SPLIT ? query_splits(a, w0, NS) : 1;
  if (SPLIT && z >= splits) return;
  uint4 q[G::kPairs], dO[G::kPairs];
  float delta = 0.f;
  {
    uint4 o[G::kPairs];
    load_operand<BF16, DC>(a.dO, start, h, w0, len, a.D, dO);
    load_operand<BF16, DC>(a.o, start, h, w0, len, a.D, o);
    load_operand<BF16, DC>(a.q, start, h, w0, len, a.D, q);
#pragma unroll
    for (int i = 0; i < G::kPairs; ++i) delta = dot_chunk<BF16>(dO[i], o[i], delta);
    delta += other_half(delta);
  }
  float lse = 0.f;
  if (query < len) {
    const int64_t at = (int64_t)h * a.N + start + query;
    lse = scaled_lse(a.lse[at]);
    if (g == 0 && split == 0 && z == 0) *(float2*)(a.pairs + 2 * at) = make_float2(lse, delta);
  }
  f32x16_t acc[G::kTiles];
  unsigned char* mine = lds + split * P::kBuffers * P::kBuf;
  bool careful = false;
#pragma unroll 1
  for (;;) {
    backward_q_pass<BF16, DC, P::kBuffers>(careful, a, start, len, kh, w0, 32 * (z * NS + split), splits * NS, mine, q, dO,
                                           lse, delta, acc);
    if (careful || !not_all_finite(acc)) break;
    careful = true;
  }
  careful = __syncthreads_or(careful);
  join<NS, G::kTiles>(acc, split, lds);
  if (split > 0) return;
  if (SPLIT && splits > 1) {
    const int64_t part = ((int64_t)blockIdx.z * a.Hq + h) * a.qsplits + z;
    f32x4_t* p = (f32x4_t*)a.qparts + part * (G::kTiles * 256) + lane;
#pragma unroll
    for (int t = 0; t < G::kTiles; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        p[t * 256 + 64 * j] = f32x4_t{acc[t][4 * j], acc[t][4 * j + 1], acc[t][4 * j + 2], acc[t][4 * j + 3]};
    if (lane == 0) a.qcareful[part] = careful;
    return;
  }
  if (query < len) store_rows<BF16, DC>(a.dq, (int64_t)start + query, h, a.D, acc, a.scale);
  if (careful) {
    __threadfence_block();
    add_not_finite<BF16, true, true>(a.k, kh, a.dq, h, start, len, w0, a.D);
  }
}

// The sums of k_backward_q_rows' work groups that shared the keys of 32 queries of one
// head, added in order: work groups behind the keys' own of the second launch.
template <bool BF16, int DC, int NS>
__device__ __forceinline__ void join_queries(const Args& a) {
  using G = Geo<BF16, DC>;
  const int64_t group = ((int64_t)((int32_t)blockIdx.z - a.slots) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  if (group >= (int64_t)a.slots * a.Hq) return;
  const int32_t slot = (int32_t)(group / a.Hq), h = (int32_t)(group % a.Hq);
  int32_t start, len, tile, tiles;
  if (!find_tile(a, slot, 32, start, len, tile, tiles)) return;
  const int32_t w0 = (tiles - 1 - tile) * 32;
  const int32_t splits = query_splits(a, w0, NS);
  if (splits < 2) return;
  const int lane = threadIdx.x & 63;
  const int split = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t query = w0 + (lane & 31);
  uint32_t careful = 0;
  for (int32_t z = 0; z < splits; ++z) careful |= a.qcareful[group * a.qsplits + z];
#pragma unroll 1
  for (int t = split; t < G::kTiles; t += NS) {
    f32x16_t x = {};
    for (int32_t z = 0; z < splits; ++z) {
      const f32x4_t* p = (const f32x4_t*)a.qparts + ((group * a.qsplits + z) * G::kTiles + t) * 256 + lane;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4_t y = p[64 * j];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * j + i] += y[i];
      }
    }
    if (query < len) store_tile<BF16>(row_ptr(a.dq, (int64_t)start + query, h), t, a.D, x, a.scale);
  }
  if (!careful) return;
  __syncthreads();
  if (split > 0) return;
  __threadfence_block();
  add_not_finite<BF16, true, true>(a.k, h / (a.Hq / a.Hkv), a.dq, h, start, len, w0, a.D);
}

// One wave's pass for dk and dv over the queries of the key head's query heads, from
// the keys w0 on: one step of 32 of `waves`, from the one `wave` on. Sets careful
// where the diagonal held others than finite numbers.
template <bool BF16, int DC, int NS>
__device__ __forceinline__ void backward_kv_pass(bool& careful, const Args& a, int32_t start, int32_t len, int32_t kh,
                                                 int32_t w0, int32_t wave, int32_t waves, unsigned char* mine, const uint4 (&k)[Geo<BF16, DC>::kPairs],
                                                 const uint4 (&v)[Geo<BF16, DC>::kPairs],
                                                 f32x16_t (&dk)[Geo<BF16, DC>::kTiles], f32x16_t (&dv)[Geo<BF16, DC>::kTiles]) {
  using P = OwnRows<BF16, DC, NS, 256>;
  using G = Geo<BF16, DC>;
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int32_t key = w0 + (lane & 31), rep = a.Hq / a.Hkv;
  const float c = a.scale * kLog2e;
  const uint32_t base = lds_address(mine);
  // 32 queries from q0 on of head h, with their lse and delta: zeros past the end
  // (whose weights are set to zero: against an infinity in a key they would be NaN)
  typename P::Rows qs(a.q, start, kh * rep, a.D), os(a.dO, start, kh * rep, a.D);
  const auto fetch = [&](int32_t h, int32_t q0, uint32_t to) {
    qs.head(a.q, start, h);
    os.head(a.dO, start, h);
    qs.fetch(q0, len, to);
    os.fetch(q0, len, to + P::kStage);
    const char* at = (const char*)(a.pairs + 2 * ((int64_t)h * a.N + start + q0));
    dma_words(rows_of(at), q0 + (lane >> 1) < len ? lane * 4 : kOutside, to + 2 * P::kStage);
  };
  // the steps of one head after another
  const int32_t hend = kh * rep + rep, end = w0 + (len - w0 + 31) / 32 * 32;
  const auto settle = [&](int32_t& h, int32_t& q0) {
    while (q0 >= end && h < hend) q0 -= end - w0, ++h;
  };
  int32_t h = kh * rep, q0 = w0 + 32 * wave;
  settle(h, q0);
  if (h < hend) fetch(h, q0, base);
#pragma unroll
  for (int t = 0; t < G::kTiles; ++t) dk[t] = f32x16_t{}, dv[t] = f32x16_t{};
  int buf = 0;
  while (h < hend) {
    int32_t nh = h, nq = q0 + 32 * waves;
    settle(nh, nq);
    own_staged();
    if (P::kBuffers == 2 && nh < hend) fetch(nh, nq, base + (buf ^ 1) * P::kBuf);
    unsigned char* lq = mine + buf * P::kBuf;
    unsigned char* lo = lq + P::kStage;
    const float* words = (const float*)(lq + 2 * P::kStage);
    if (q0 == w0) {   // (a query row that is not finite has lse or delta of NaN)
      careful |= zero_not_finite<BF16, DC>(lo);
      careful |= zero_not_finite<BF16, DC>(lq);
    }
    f32x16_t p = rows_times<BF16, DC>(lq, 0, k);
    f32x16_t ds = rows_times<BF16, DC>(lo, 0, v);
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const f32x4_t x = *(const f32x4_t*)(words + 2 * (8 * r4 + 4 * g + i));   // lse, delta of two queries
        const int r = 4 * r4 + i;
        p[r] = __builtin_amdgcn_exp2f(fmaf(p[r], c, -x[0]));
        ds[r] = p[r] * (ds[r] - x[1]);
        p[r + 1] = __builtin_amdgcn_exp2f(fmaf(p[r + 1], c, -x[2]));
        ds[r + 1] = p[r + 1] * (ds[r + 1] - x[3]);
      }
    }
    if (q0 == w0 || q0 + 32 > len) {
      keep_branch();
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int32_t query = q0 + result_row(r, g);
        if (query < key || query >= len) p[r] = 0.f, ds[r] = 0.f;
      }
    }
    columns_times<BF16, DC>(lo, 0, p, dv);
    columns_times<BF16, DC>(lq, 0, ds, dk);
    h = nh;
    q0 = nq;
    if (P::kBuffers == 2) {
      buf ^= 1;
    } else if (nh < hend) {
      own_staged();   // (the reads of this step are done)
      fetch(nh, nq, base);
    }
  }
}

// dk and dv by rows: 32 keys of one key head, all query heads of the key head and
// all queries from the diagonal on, by NS waves with LDS of their own: the keys stay in
// registers, and four products a step (S, dP, dV, dK) read 32 rows of q and dO. Bound by
// the chain of a step, reads, products, exponentials, products, of which the registers
// allow two waves a SIMD; the LDS is busy half of the time, and a fifth fewer reads (lse
// and delta as a column of the first products) gained 2 % at D = 64 and lost 5 % at 128.
// B = 4, T = 2048, 32/8 heads, D = 64: 229 us, 600 TF/s; 16/4 heads, D = 128: 285 us
// (where 12 registers spill).
// SPLIT: a few such work groups share
// the steps, as many as leave each wave kSteps of them, and the last to arrive adds
// their sums in a fixed order. The sums and the counter go past the L2 caches, which
// the XCDs do not share: fences, which write back and empty them, cost more than the
// split won (3/1 heads D = 64, 811 + 443 rows: 34 us with fences, 14 without, 26 unsplit).
template <bool BF16, int DC, int NS, bool SPLIT>
__global__ __launch_bounds__(64 * NS, BF16 || DC == 64 ? 2 : 1) void k_backward_kv(Args a) {
  using G = Geo<BF16, DC>;
  using P = OwnRows<BF16, DC, NS, 256>;
  __shared__ __align__(1024) unsigned char lds[P::kLds];
  if (SPLIT && (int32_t)blockIdx.z >= a.slots) return join_queries<BF16, DC, NS>(a);
  int32_t start, len, tile, tiles;
  const int32_t kh = blockIdx.x;
  if (!find_tile(a, block_slot(a), 32, start, len, tile, tiles)) {
    if (blockIdx.y == 0)
      clear_rest(a, block_slot(a), tiles, [&](int32_t r) {
        clear_row(a.dk, r, blockIdx.x, a.D * G::kElem);
        clear_row(a.dv, r, blockIdx.x, a.D * G::kElem);
      });
    return;
  }
  const int lane = threadIdx.x & 63;
  const int split = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t w0 = tile * 32, key = w0 + (lane & 31);
  // as many work groups as give each of their waves kSteps steps
  const int32_t steps = (len - w0 + 31) / 32 * (a.Hq / a.Hkv);
  const int32_t splits = SPLIT ? min(a.splits, (steps + kSteps * NS - 1) / (kSteps * NS)) : 1;
  if (SPLIT && (int32_t)blockIdx.y >= splits) return;
  unsigned char* mine = lds + split * P::kBuffers * P::kBuf;
  uint4 k[G::kPairs], v[G::kPairs];
  load_operand<BF16, DC>(a.k, start, kh, w0, len, a.D, k);
  load_operand<BF16, DC>(a.v, start, kh, w0, len, a.D, v);
  f32x16_t dk[G::kTiles], dv[G::kTiles];
  bool careful = false;
  backward_kv_pass<BF16, DC, NS>(careful, a, start, len, kh, w0, SPLIT ? blockIdx.y * NS + split : split, splits * NS,
                                 mine, k, v, dk, dv);
  careful = __syncthreads_or(careful);
  join<NS, G::kTiles>(dk, split, lds);
  join<NS, G::kTiles>(dv, split, lds);
  if constexpr (SPLIT) {
    // the last work group to arrive adds the sums of all, in their order
    const int64_t group = (int64_t)blockIdx.z * a.Hkv + kh;
    uint64_t* parts = (uint64_t*)a.parts + group * a.splits * (2 * G::kTiles * 512) + lane;
    if (split == 0) {
      uint64_t* p = parts + (int64_t)blockIdx.y * (2 * G::kTiles * 512);
#pragma unroll
      for (int t = 0; t < 2 * G::kTiles; ++t) {
        const f32x16_t& x = t < G::kTiles ? dk[t % G::kTiles] : dv[t % G::kTiles];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          __hip_atomic_store(p + (t * 8 + j) * 64, __builtin_bit_cast(uint64_t, (f32x2_t){x[2 * j], x[2 * j + 1]}),
                             __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (all have reached the memory)
      if (lane == 0) {
        const uint32_t me = careful ? 0x10001u : 1u;
        *(uint32_t*)lds = me + __hip_atomic_fetch_add(a.arrived + group, me, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    __syncthreads();
    const uint32_t arrived = *(const uint32_t*)lds;
    if ((int32_t)(arrived & 0xffff) != splits) return;
    careful = arrived >> 16;
#pragma unroll 1
    for (int t = split; t < 2 * G::kTiles; t += NS) {
      f32x16_t x = {};
      for (int32_t z = 0; z < splits; ++z) {
        const uint64_t* p = parts + (int64_t)(z * 2 * G::kTiles + t) * 512;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const f32x2_t y = __builtin_bit_cast(f32x2_t, __hip_atomic_load(p + 64 * j, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
          x[2 * j] += y[0];
          x[2 * j + 1] += y[1];
        }
      }
      const bool second = t >= G::kTiles;
      const Tensor& out = second ? a.dv : a.dk;
      if (key < len)
        store_tile<BF16>(row_ptr(out, (int64_t)start + key, kh), second ? t - G::kTiles : t, a.D, x, second ? 1.f : a.scale);
    }
    if (!careful) return;
    __syncthreads();
    if (split > 0) return;
  } else {
    if (split > 0) return;
    if (key < len) {
      store_rows<BF16, DC>(a.dk, (int64_t)start + key, kh, a.D, dk, a.scale);
      store_rows<BF16, DC>(a.dv, (int64_t)start + key, kh, a.D, dv, 1.f);
    }
  }
  if (careful) {
    __threadfence_block();
    const int32_t rep = a.Hq / a.Hkv;
    for (int32_t h = kh * rep; h < kh * rep + rep; ++h) {
      add_not_finite<BF16, false, true>(a.q, h, a.dk, kh, start, len, w0, a.D);
      add_not_finite<BF16, false, false>(a.dO, h, a.dv, kh, start, len, w0, a.D);   // (weights are not negative)
    }
  }
}

}  // namespace attn
}  // namespace dpn
