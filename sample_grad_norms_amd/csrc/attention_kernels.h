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
// are rounded to bf16 for bf16 inputs (half a step, 2^-9 relative, as the
// inputs themselves are); the sum of the weights takes them unrounded.
#pragma once
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
  float* delta;       // [Hq][N], backward
  const int32_t* cu;  // [S + 1], or null: S sequences of T tokens
  int32_t S, T, N;
  int32_t Hq, Hkv, D;
  float scale;        // a
  int32_t slots;      // tile slots per head
};

constexpr int kThreads = 256;
constexpr int kRows = 128;   // stationary rows of a work group: 32 a wave
constexpr int kStep = 64;    // streamed rows a step
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kOutside = 0x80000000u;   // an offset past every buffer's range: reads as zero

// The sequence and tile of a slot. Slots count the tiles of the sequences one
// after another; a slot past the last tile has none. Offsets outside [0, N] or
// out of order are clamped, so no row outside the tensors is ever touched.
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
  return false;
}

template <bool BF16, int DP>
struct Geo {
  static constexpr int kElem = BF16 ? 2 : 4;
  static constexpr int kChunks = DP * kElem / 16;    // 16-byte chunks of a row
  static constexpr int kPairs = kChunks / 2;         // chunk pairs: one chunk for each half of the wave
  static constexpr int kPitch = DP * kElem;          // LDS bytes of a row
  static constexpr int kTiles = DP / 32;             // 32-column tiles of a row
  static constexpr int kStage = kStep * kPitch;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const char* p) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, 0x7fffffff, 0x00027000);
}

// Pointer to row `row` of sequence start `start`, head h (all wave-uniform).
__device__ __forceinline__ char* row_ptr(const Tensor& t, int64_t row, int32_t h) { return t.p + row * t.st + h * t.sh; }

// Rows r0 .. r0 + 63 of a sequence into LDS, row-major with the 16-byte chunks
// of row r at chunk ^ (r & 7): reads of one chunk of eight rows then fall on
// different banks. Rows past `len` and columns past D read as zero.
template <bool BF16, int DP>
__device__ __forceinline__ void stage(const Tensor& t, int64_t start, int32_t h, int32_t r0, int32_t len, int32_t D,
                                      unsigned char* lds) {
  using G = Geo<BF16, DP>;
  const __amdgpu_buffer_rsrc_t rs = rows_of(row_ptr(t, start + r0, h));
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
  for (int i = 0; i < kStep * G::kChunks / kThreads; ++i) {
    const int at = i * kThreads + threadIdx.x;
    const int row = at / G::kChunks, ch = (at % G::kChunks) ^ (row & 7);
    const bool in = r0 + row < len && ch * 16 < D * G::kElem;
    const uint32_t off = in ? (uint32_t)(row * (int32_t)t.st + ch * 16) : kOutside;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rs, (__attribute__((address_space(3))) void*)(lds + (i * kThreads + wv * 64) * 16), 16, off, 0, 0, 0);
  }
}

// The wave's direct loads have landed, and then every wave's.
__device__ __forceinline__ void staged() {
  DPN_WAIT_VMCNT(0);
  __syncthreads();
}

__device__ __forceinline__ uint4 buffer16(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
}

// The wave's 32 stationary rows as an operand: lane l has row l % 32, chunk
// 2 i + l / 32 of pair i.
template <bool BF16, int DP>
__device__ __forceinline__ void load_operand(const Tensor& t, int64_t start, int32_t h, int32_t r0, int32_t len, int32_t D,
                                             uint4 (&f)[Geo<BF16, DP>::kPairs]) {
  using G = Geo<BF16, DP>;
  const __amdgpu_buffer_rsrc_t rs = rows_of(row_ptr(t, start + r0, h));
  const int lane = threadIdx.x & 63, row = lane & 31, g = lane >> 5;
#pragma unroll
  for (int i = 0; i < G::kPairs; ++i) {
    const int ch = 2 * i + g;
    const bool in = r0 + row < len && ch * 16 < D * G::kElem;
    f[i] = buffer16(rs, in ? (uint32_t)(row * (int32_t)t.st + ch * 16) : kOutside);
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

// 32 rows of LDS (at row r0) times the stationary operand: X f^T, 32 x 32.
template <bool BF16, int DP>
__device__ __forceinline__ f32x16_t rows_times(const unsigned char* lds, int r0, const uint4 (&f)[Geo<BF16, DP>::kPairs]) {
  using G = Geo<BF16, DP>;
  const int lane = threadIdx.x & 63, row = r0 + (lane & 31), g = lane >> 5;
  f32x16_t c = {};
#pragma unroll
  for (int i = 0; i < G::kPairs; ++i) {
    const uint4 a = *(const uint4*)(lds + row * G::kPitch + (((2 * i + g) ^ (row & 7)) << 4));
    c = mfma_chunk<BF16>(a, f[i], c);
  }
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
template <bool BF16, int DP>
__device__ __forceinline__ void columns_times(const unsigned char* lds, int r0, const f32x16_t& w,
                                              f32x16_t (&acc)[Geo<BF16, DP>::kTiles]) {
  using G = Geo<BF16, DP>;
  const int lane = threadIdx.x & 63, g = lane >> 5;
  if constexpr (BF16) {
    const int j = (lane >> 2) & 3, q = lane & 3, m0 = ((lane >> 4) & 1) * 16;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const uint4 b = pack_weights(w, ks * 8);
      const int ra = r0 + ks * 16 + 4 * g + j, rb = ra + 8;
#pragma unroll
      for (int t = 0; t < G::kTiles; ++t) {
        const int ch = (t * 32 + m0 + 4 * q) >> 3;
        const uint2 lo = lds_read_tr16(lds + ra * G::kPitch + ((ch ^ (ra & 7)) << 4) + (q & 1) * 8);
        const uint2 hi = lds_read_tr16(lds + rb * G::kPitch + ((ch ^ (rb & 7)) << 4) + (q & 1) * 8);
        acc[t] = mfma_chunk<true>(make_uint4(lo.x, lo.y, hi.x, hi.y), b, acc[t]);
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = r0 + 8 * (r >> 2) + 4 * g + (r & 3);
#pragma unroll
      for (int t = 0; t < G::kTiles; ++t) {
        const int col = t * 32 + (lane & 31);
        const float x = *(const float*)(lds + row * G::kPitch + (((col >> 2) ^ (row & 7)) << 4) + (col & 3) * 4);
        acc[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, w[r], acc[t], 0, 0, 0);
      }
    }
  }
}

__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

// Row r (0 .. 15) of a lane's half in a 32 x 32 result.
__device__ __forceinline__ int result_row(int r, int g) { return 8 * (r >> 2) + 4 * g + (r & 3); }

// Columns of acc (transposed: rows are the D index) to row `row` of t, times f.
template <bool BF16, int DP>
__device__ __forceinline__ void store_rows(const Tensor& t, int64_t row, int32_t h, int32_t D,
                                           const f32x16_t (&acc)[Geo<BF16, DP>::kTiles], float f) {
  using G = Geo<BF16, DP>;
  char* p = t.p + row * t.st + h * t.sh;
  const int g = (threadIdx.x & 63) >> 5;
#pragma unroll
  for (int i = 0; i < G::kTiles; ++i) {
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const int col = i * 32 + 8 * r4 + 4 * g;
      if (col >= D) continue;
      if constexpr (BF16) {
        uint2 x;
        x.x = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){acc[i][4 * r4] * f, acc[i][4 * r4 + 1] * f}, bf16x2_t));
        x.y = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){acc[i][4 * r4 + 2] * f, acc[i][4 * r4 + 3] * f}, bf16x2_t));
        *(uint2*)(p + col * 2) = x;
      } else {
        *(float4*)(p + col * 4) = make_float4(acc[i][4 * r4] * f, acc[i][4 * r4 + 1] * f, acc[i][4 * r4 + 2] * f, acc[i][4 * r4 + 3] * f);
      }
    }
  }
}

// Head and slot of a block. Blocks go to the 8 XCDs in turn; with the key head
// as the fastest index, the blocks that read one key head meet in one L2 when
// Hkv is a multiple or a divisor of 8.
__device__ __forceinline__ void block_head(const Args& a, int32_t& h, int32_t& slot) {
  const int32_t b = blockIdx.x, x = b % a.Hq, rep = a.Hq / a.Hkv;
  h = (x % a.Hkv) * rep + x / a.Hkv;
  slot = b / a.Hq;
}

template <bool BF16, int DP>
__global__ __launch_bounds__(kThreads) void k_forward(Args a) {
  using G = Geo<BF16, DP>;
  __shared__ __align__(16) unsigned char lk[G::kStage], lv[G::kStage];
  int32_t h, slot, start, len, tile, tiles;
  block_head(a, h, slot);
  if (!find_tile(a, slot, kRows, start, len, tile, tiles)) return;
  tile = tiles - 1 - tile;   // the longest rows first
  const int32_t kh = h / (a.Hq / a.Hkv);
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t w0 = tile * kRows + wv * 32;   // the wave's first query
  const int32_t query = w0 + (lane & 31);
  uint4 q[G::kPairs];
  load_operand<BF16, DP>(a.q, start, h, w0, len, a.D, q);
  const float c = a.scale * kLog2e;
  float m = -INFINITY, l = 0.f;
  f32x16_t acc[G::kTiles] = {};
  const int32_t end = min(tile * kRows + kRows, len);   // keys that some query of the block sees
  for (int32_t k0 = 0; k0 < end; k0 += kStep) {
    __syncthreads();
    stage<BF16, DP>(a.k, start, kh, k0, len, a.D, lk);
    stage<BF16, DP>(a.v, start, kh, k0, len, a.D, lv);
    staged();
    if (k0 > w0 + 31) continue;
    f32x16_t s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) s[t] = rows_times<BF16, DP>(lk, t * 32, q);
    if (k0 + kStep - 1 > w0) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (k0 + t * 32 + result_row(r, g) > query) s[t][r] = -INFINITY;
    }
    float top = s[0][0];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[t][r]);
    top = fmaxf(m, fmaxf(top, other_half(top)));
    const float f = __builtin_amdgcn_exp2f((m - top) * c);
    const float mc = top * c;
    m = top;
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[t][r] = __builtin_amdgcn_exp2f(fmaf(s[t][r], c, -mc));
        sum += s[t][r];
      }
    l = fmaf(l, f, sum);
#pragma unroll
    for (int t = 0; t < G::kTiles; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[t][r] *= f;
#pragma unroll
    for (int t = 0; t < 2; ++t) columns_times<BF16, DP>(lv, t * 32, s[t], acc);
  }
  l += other_half(l);
  if (query >= len) return;
  store_rows<BF16, DP>(a.o, (int64_t)start + query, h, a.D, acc, 1.f / l);
  if (g == 0) a.lse[(int64_t)h * a.N + start + query] = fmaf(m, a.scale, logf(l));
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

// dq, and delta for the second launch.
template <bool BF16, int DP>
__global__ __launch_bounds__(kThreads) void k_backward_q(Args a) {
  using G = Geo<BF16, DP>;
  __shared__ __align__(16) unsigned char lk[G::kStage], lv[G::kStage];
  int32_t h, slot, start, len, tile, tiles;
  block_head(a, h, slot);
  if (!find_tile(a, slot, kRows, start, len, tile, tiles)) return;
  tile = tiles - 1 - tile;
  const int32_t kh = h / (a.Hq / a.Hkv);
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t w0 = tile * kRows + wv * 32;
  const int32_t query = w0 + (lane & 31);
  uint4 q[G::kPairs], dO[G::kPairs];
  float delta = 0.f;
  {
    uint4 o[G::kPairs];
    load_operand<BF16, DP>(a.dO, start, h, w0, len, a.D, dO);
    load_operand<BF16, DP>(a.o, start, h, w0, len, a.D, o);
    load_operand<BF16, DP>(a.q, start, h, w0, len, a.D, q);
#pragma unroll
    for (int i = 0; i < G::kPairs; ++i) delta = dot_chunk<BF16>(dO[i], o[i], delta);
    delta += other_half(delta);
  }
  float lse = INFINITY;   // queries past the end: every weight 0
  if (query < len) {
    const int64_t at = (int64_t)h * a.N + start + query;
    lse = a.lse[at] * kLog2e;
    if (g == 0) a.delta[at] = delta;
  }
  const float c = a.scale * kLog2e;
  f32x16_t acc[G::kTiles] = {};
  const int32_t end = min(tile * kRows + kRows, len);
  for (int32_t k0 = 0; k0 < end; k0 += kStep) {
    __syncthreads();
    stage<BF16, DP>(a.k, start, kh, k0, len, a.D, lk);
    stage<BF16, DP>(a.v, start, kh, k0, len, a.D, lv);
    staged();
    if (k0 > w0 + 31) continue;
    const bool diag = k0 + kStep - 1 > w0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      f32x16_t s = rows_times<BF16, DP>(lk, t * 32, q);
      const f32x16_t dp = rows_times<BF16, DP>(lv, t * 32, dO);
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -lse)) * (dp[r] - delta);
      if (diag) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (k0 + t * 32 + result_row(r, g) > query) s[r] = 0.f;
      }
      columns_times<BF16, DP>(lk, t * 32, s, acc);
    }
  }
  if (query >= len) return;
  store_rows<BF16, DP>(a.dq, (int64_t)start + query, h, a.D, acc, a.scale);
}

// dk and dv of 128 keys of one key head: 32 keys a wave, all query heads of the
// key head and all queries from the diagonal on.
template <bool BF16, int DP>
__global__ __launch_bounds__(kThreads) void k_backward_kv(Args a) {
  using G = Geo<BF16, DP>;
  __shared__ __align__(16) unsigned char lq[G::kStage], lo[G::kStage];
  __shared__ __align__(16) float llse[kStep], ldelta[kStep];
  int32_t start, len, tile, tiles;
  const int32_t kh = blockIdx.x % a.Hkv, slot = blockIdx.x / a.Hkv, rep = a.Hq / a.Hkv;
  if (!find_tile(a, slot, kRows, start, len, tile, tiles)) return;
  const int lane = threadIdx.x & 63, g = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t w0 = tile * kRows + wv * 32;
  const int32_t key = w0 + (lane & 31);
  uint4 k[G::kPairs], v[G::kPairs];
  load_operand<BF16, DP>(a.k, start, kh, w0, len, a.D, k);
  load_operand<BF16, DP>(a.v, start, kh, w0, len, a.D, v);
  const float c = a.scale * kLog2e;
  f32x16_t dk[G::kTiles] = {}, dv[G::kTiles] = {};
  for (int32_t h = kh * rep; h < kh * rep + rep; ++h) {
    for (int32_t q0 = tile * kRows; q0 < len; q0 += kStep) {
      __syncthreads();
      stage<BF16, DP>(a.q, start, h, q0, len, a.D, lq);
      stage<BF16, DP>(a.dO, start, h, q0, len, a.D, lo);
      if (threadIdx.x < kStep) {
        const int32_t t = q0 + threadIdx.x;
        const int64_t at = (int64_t)h * a.N + start + t;
        llse[threadIdx.x] = t < len ? a.lse[at] * kLog2e : INFINITY;   // queries past the end: every weight 0
        ldelta[threadIdx.x] = t < len ? a.delta[at] : 0.f;
      }
      staged();
      if (q0 + kStep - 1 < w0) continue;
      const bool diag = q0 < w0 + 31;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x16_t p = rows_times<BF16, DP>(lq, t * 32, k);
        f32x16_t ds = rows_times<BF16, DP>(lo, t * 32, v);
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const float4 z = *(const float4*)(llse + t * 32 + 8 * r4 + 4 * g);
          const float4 e = *(const float4*)(ldelta + t * 32 + 8 * r4 + 4 * g);
          const float zz[4] = {z.x, z.y, z.z, z.w}, ee[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 4 * r4 + i;
            p[r] = __builtin_amdgcn_exp2f(fmaf(p[r], c, -zz[i]));
            ds[r] = p[r] * (ds[r] - ee[i]);
            if (diag && q0 + t * 32 + result_row(r, g) < key) p[r] = 0.f, ds[r] = 0.f;
          }
        }
        columns_times<BF16, DP>(lo, t * 32, p, dv);
        columns_times<BF16, DP>(lq, t * 32, ds, dk);
      }
    }
  }
  if (key >= len) return;
  store_rows<BF16, DP>(a.dk, (int64_t)start + key, kh, a.D, dk, a.scale);
  store_rows<BF16, DP>(a.dv, (int64_t)start + key, kh, a.D, dv, 1.f);
}

}  // namespace attn
}  // namespace dpn
