// Layer norm and RMS norm: forward, gradients, and the per-sample norm of the
// gradient of their gain and bias.
//
//   h = (x - mu) r,  r = (mean((x - mu)^2) + eps)^-1/2,  mu = mean(x) (0 for RMS norm)
//   forward   y = h w + b
//   backward  g = dy w,  dx = r (g - mean(g) - h mean(g h))   (RMS norm: no mean(g))
//             dw = sum_t c_t dy_t h_t,  db = sum_t c_t dy_t
//   norm      n_i = || sum_{t in i} G_t h_t ||^2 + || sum_{t in i} G_t ||^2
//
// All are bound by HBM: each row is read once, 16 bytes a lane, and stays in
// registers between its statistics and its results; the mean is known before the
// squares are summed. W waves hold a row (1 for up to 2048 bf16 columns, so that
// its sums are lane moves without a barrier; 4 and 16 for wider rows), NC chunks
// a lane, and a wave takes R rows at a time where its rows are short. Column sums
// stay in the registers of the lanes that hold the columns, over all rows of a
// block; blocks leave them in the workspace, and the second launch adds them in
// order, so that results are reproducible bit for bit. Everything is fp32, a
// sample's sum of squares over the columns fp64.
#pragma once
#include <type_traits>

#include "device_common.h"

namespace dpn {
namespace ln {

struct Args {
  const char* x;
  const char* dy;         // the output's gradient
  const char* w;
  const char* b;          // or null
  char* y;                // forward
  char* dx;               // or null
  char* dw;               // or null
  char* db;               // or null
  float* mean;            // [N]; forward: or null
  float* rstd;
  const float* c;         // [N / T] factors of the samples, or null
  float* part;            // [block][gain, bias][d], or null: one block, which writes dw and db
  uint32_t* arrived;      // [sample] work groups of the second launch of a norm that have arrived
  double* parts;          // [sample][work group]
  float* n;               // [sample]
  int32_t N, T, d;        // rows, rows of a sample
  int32_t blocks;         // backward: of the first launch; norm: of a sample
  int32_t columns;        // norm: d, or 2 d with the bias
  int32_t first;          // norm: 0, or d without the gain
  int32_t accumulate;
  float eps, inv;         // 1 / d
};

template <bool BF16>
struct Chunk {
  static constexpr int kN = BF16 ? 8 : 4, kElem = BF16 ? 2 : 4;   // elements of 16 bytes
  typedef float Floats[kN];
};

template <bool BF16>
__device__ __forceinline__ void widen(const uint4& u, typename Chunk<BF16>::Floats& f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = word(u, j);
    if constexpr (BF16) {
      f[2 * j] = __uint_as_float(x << 16);
      f[2 * j + 1] = __uint_as_float(x & 0xffff0000u);
    } else {
      f[j] = __uint_as_float(x);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow(const typename Chunk<BF16>::Floats& f) {
  if constexpr (BF16) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    uint32_t x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){f[2 * j], f[2 * j + 1]}, bf16x2));
    return make_uint4(x[0], x[1], x[2], x[3]);
  } else {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
}

template <bool BF16>
__device__ __forceinline__ void store_one(char* p, int64_t j, float v) {
  if constexpr (BF16) ((uint16_t*)p)[j] = (uint16_t)f32_to_bf16_bits(v);
  else ((float*)p)[j] = v;
}

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_f32(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROW_MASK, 0xf, true));
}

// Sums over the 64 lanes in the order of wave_sum, the same in every lane.
template <int M>
__device__ __forceinline__ void wave_sums(float (&v)[M]) {
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] += dpp_f32<0x111, 0xf>(v[m]);
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] += dpp_f32<0x112, 0xf>(v[m]);
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] += dpp_f32<0x114, 0xf>(v[m]);
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] += dpp_f32<0x118, 0xf>(v[m]);
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] += dpp_f32<0x142, 0xa>(v[m]);
#pragma unroll
  for (int m = 0; m < M; ++m) v[m] += dpp_f32<0x143, 0xc>(v[m]);
#pragma unroll
  for (int m = 0; m < M; ++m)
    v[m] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v[m]), 63));
}

// How a row lies on its lanes: lane l of W waves holds chunks l + 64 W i.
template <bool BF16, int NC, int W>
struct Row {
  static constexpr int kN = Chunk<BF16>::kN, kLanes = 64 * W;
  static constexpr int kColumns = kLanes * NC * kN;   // at most
  // Sums over the W waves of a row (lds: 4 W R floats of these waves). `turn` alternates, so
  // that one barrier is enough: what a call reads is written again two calls later.
  template <int M>
  static __device__ __forceinline__ void sums(float (&v)[M], float* lds, int& turn) {
    wave_sums(v);
    if constexpr (W > 1) {
      float* at = lds + turn * W * M;
      turn ^= 1;
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int m = 0; m < M; ++m) at[(threadIdx.x >> 6) % W * M + m] = v[m];
      __syncthreads();
#pragma unroll
      for (int m = 0; m < M; ++m) {
        v[m] = at[m];
#pragma unroll
        for (int w = 1; w < W; ++w) v[m] += at[w * M + m];
      }
    }
  }
};

// A row (wave-uniform) as a buffer of its own bytes: lanes past its end read zeros and
// store nothing, without a branch. No bytes for a row that is not there.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const char* p, int64_t row, int32_t bytes, bool there) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)(p + row * bytes), 0, there ? bytes : 0, 0x00027000);
}
__device__ __forceinline__ uint4 load_chunk(__amdgpu_buffer_rsrc_t row, int ch) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(row, ch * 16, 0, 0));
}
__device__ __forceinline__ void store_chunk(__amdgpu_buffer_rsrc_t row, int ch, const uint4& v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), row, ch * 16, 0, 0);
}

// R rows from `row` on into registers; rows from `end` on, and columns past d, are zeros.
template <bool BF16, int NC, int W, int R>
__device__ __forceinline__ void load_rows(const char* p, int64_t row, int64_t end, int32_t d, int lane, uint4 (&v)[R][NC]) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const __amdgpu_buffer_rsrc_t at = row_buffer(p, row + r, d * Chunk<BF16>::kElem, row + r < end);
#pragma unroll
    for (int i = 0; i < NC; ++i) v[r][i] = load_chunk(at, lane + 64 * W * i);
  }
}

// Keeps rows packed over a reduction: without it the compiler holds their floats, twice
// the registers, from one use to the next instead of widening them again.
template <int R, int NC>
__device__ __forceinline__ void keep_packed(uint4 (&v)[R][NC]) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < NC; ++i) asm volatile("" : "+v"(v[r][i].x), "+v"(v[r][i].y), "+v"(v[r][i].z), "+v"(v[r][i].w));
}

// Mean and reciprocal deviation of R rows.
template <bool BF16, bool RMS, int NC, int W, int R>
__device__ __forceinline__ void statistics(uint4 (&x)[R][NC], int32_t d, float eps, float inv, int lane, float* lds, int& turn,
                                           float (&mu)[R], float (&rs)[R]) {
  using C = Chunk<BF16>;
  float s[R];
  if constexpr (!RMS) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        typename C::Floats f;
        widen<BF16>(x[r][i], f);
#pragma unroll
        for (int e = 0; e < C::kN; ++e) s[r] += f[e];
      }
    }
    Row<BF16, NC, W>::sums(s, lds, turn);
    if constexpr (BF16) keep_packed(x);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    mu[r] = RMS ? 0.f : s[r] * inv;
    s[r] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const bool in = (lane + 64 * W * i) * C::kN < d;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      typename C::Floats f;
      widen<BF16>(x[r][i], f);
      const float m = in ? mu[r] : 0.f;   // (columns past d add nothing)
#pragma unroll
      for (int e = 0; e < C::kN; ++e) {
        const float u = RMS ? f[e] : f[e] - m;
        s[r] = fmaf(u, u, s[r]);
      }
    }
  }
  Row<BF16, NC, W>::sums(s, lds, turn);
  if constexpr (BF16) keep_packed(x);
#pragma unroll
  for (int r = 0; r < R; ++r) rs[r] = 1.f / sqrtf(fmaf(s[r], inv, eps));
}

// Forward. Gain and bias stay packed in registers over the rows of a work group; loads of
// eight work groups a CU hide each other. Bound by HBM: 4 x 4096 rows of 2048 bf16 in
// 22 us (RMS norm 21), 6.1 TB/s of what is read and written (a copy reaches 5.1: part comes
// from the last-level cache). W = 1: four
// rows' waves a work group; else one row's.
template <int W>
constexpr int kForwardThreads = W == 1 ? 256 : 64 * W;

template <bool BF16, bool RMS, int NC, int W, int R>
__global__ __launch_bounds__(kForwardThreads<W>) void k_forward(Args a) {
  using C = Chunk<BF16>;
  __shared__ float lds[W > 1 ? 2 * W * R : 1];
  int turn = 0;
  const int lane = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int32_t each = W == 1 ? 4 : 1;
  const int32_t wave = W == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  uint4 w[1][NC], b[1][NC];
  load_rows<BF16, NC, W, 1>(a.w, 0, 1, a.d, lane, w);
  if constexpr (!RMS) load_rows<BF16, NC, W, 1>(a.b, 0, a.b ? 1 : 0, a.d, lane, b);
  const int64_t step = (int64_t)gridDim.x * each * R;
  for (int64_t row = ((int64_t)blockIdx.x * each + wave) * R; row < a.N; row += step) {
    uint4 x[R][NC];
    load_rows<BF16, NC, W, R>(a.x, row, a.N, a.d, lane, x);
    if constexpr (BF16) {
      keep_packed(w);
      if constexpr (!RMS) keep_packed(b);
    }
    float mu[R], rs[R];
    statistics<BF16, RMS, NC, W, R>(x, a.d, a.eps, a.inv, lane, lds, turn, mu, rs);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row + r >= a.N) break;
      const __amdgpu_buffer_rsrc_t to = row_buffer(a.y, row + r, a.d * C::kElem, true);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        typename C::Floats f, g, o;
        widen<BF16>(x[r][i], f);
        widen<BF16>(w[0][i], g);
        if constexpr (!RMS) widen<BF16>(b[0][i], o);
#pragma unroll
        for (int e = 0; e < C::kN; ++e) {
          const float h = (RMS ? f[e] : f[e] - mu[r]) * rs[r];
          f[e] = RMS ? h * g[e] : fmaf(h, g[e], o[e]);
        }
        store_chunk(to, lane + 64 * W * i, narrow<BF16>(f));
      }
      if (lane == 0) {
        if (!RMS && a.mean) a.mean[row + r] = mu[r];
        if (a.rstd) a.rstd[row + r] = rs[r];
      }
    }
  }
}

// Rows of a round of a work group of the summing kernels, whose column sums it leaves as
// one: 8 of one wave, 2 of four (one of up to 2048 fp32 columns: gradients of 4 x 2048
// rows 39 us, 41 with two; but 8192 bf16 columns 60 us with one, 49 with two), one of sixteen.
template <bool BF16, int NC, int W>
constexpr int kSumRows = W == 1 ? 8 : W == 4 && (BF16 || NC > 2) ? 2 : 1;
template <bool BF16, int NC, int W>
constexpr int kSumWaves = W * kSumRows<BF16, NC, W>;
template <bool BF16, int NC, int W, int R>
constexpr int kSumLds = kSumRows<BF16, NC, W> > 1 && kSumRows<BF16, NC, W> * Row<BF16, NC, W>::kColumns > 4 * kSumWaves<BF16, NC, W> * R
                            ? kSumRows<BF16, NC, W> * Row<BF16, NC, W>::kColumns
                            : 4 * kSumWaves<BF16, NC, W> * R;

// Column sums of a work group: out(column, sum) for every column below d.
template <bool BF16, int NC, int W, typename F>
__device__ __forceinline__ void block_columns(const float (&acc)[NC][Chunk<BF16>::kN], int32_t d, float* lds, F out) {
  using C = Chunk<BF16>;
  constexpr int kRows = kSumRows<BF16, NC, W>;
  const int lane = threadIdx.x % (64 * W), mine = threadIdx.x / (64 * W);
  if constexpr (kRows > 1) {
    constexpr int kColumns = Row<BF16, NC, W>::kColumns;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < C::kN; e += 4)
        *(f32x4_t*)(lds + mine * kColumns + (lane + 64 * W * i) * C::kN + e) =
            f32x4_t{acc[i][e], acc[i][e + 1], acc[i][e + 2], acc[i][e + 3]};
    __syncthreads();
    for (int32_t j = threadIdx.x; j < d; j += 64 * kSumWaves<BF16, NC, W>) {
      float s = lds[j];
#pragma unroll
      for (int v = 1; v < kRows; ++v) s += lds[v * kColumns + j];
      out(j, s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int32_t j = (lane + 64 * W * i) * C::kN;
      if (j >= d) continue;
#pragma unroll
      for (int e = 0; e < C::kN; ++e) out(j + e, acc[i][e]);
    }
  }
}

// Gradients. A row's two sums (g and g h) are ready together, so dx costs one reduction; dw
// and db are summed in the registers of the lanes that hold their columns, 2 NC chunks of
// floats, which leaves two or three waves a SIMD. Bound by HBM: 4 x 4096 rows of 2048 bf16
// 35 to 36 us, 5.7 TB/s, and the columns 4 to 4.6 us.
template <bool BF16, bool RMS, int NC, int W, int R>
__global__ __launch_bounds__((64 * kSumWaves<BF16, NC, W>)) void k_backward(Args a) {
  using C = Chunk<BF16>;
  __shared__ __align__(16) float lds[kSumLds<BF16, NC, W, R>];
  int turn = 0;
  const int lane = threadIdx.x % (64 * W);
  const int32_t mine = __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * W));
  constexpr int32_t kStep = kSumRows<BF16, NC, W> * R;
  float* own = lds + mine * 4 * W * R;
  // the blocks' rounds in turn, so that rows of one time lie together
  const int64_t first = (int64_t)blockIdx.x * kStep, step = (int64_t)a.blocks * kStep;
  const int32_t end = a.N;
  uint4 w[1][NC];
  float aw[NC][C::kN] = {}, ab[NC][C::kN] = {};
  load_rows<BF16, NC, W, 1>(a.w, 0, 1, a.d, lane, w);
  for (int64_t at = first; at < end; at += step) {   // (all waves: they meet at the sums)
    const int64_t row = at + mine * R;
    uint4 x[R][NC], dy[R][NC];
    load_rows<BF16, NC, W, R>(a.dy, row, end, a.d, lane, dy);
    load_rows<BF16, NC, W, R>(a.x, row, end, a.d, lane, x);
    if constexpr (BF16) keep_packed(w);
    float mu[R], rs[R], cf[R], s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool in = row + r < end;
      mu[r] = !RMS && in ? a.mean[row + r] : 0.f;
      rs[r] = in ? a.rstd[row + r] : 0.f;
      cf[r] = in && a.c ? a.c[(uint32_t)(row + r) / (uint32_t)a.T] : 1.f;
      s[2 * r] = s[2 * r + 1] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      typename C::Floats wf;
      widen<BF16>(w[0][i], wf);
      const bool in = (lane + 64 * W * i) * C::kN < a.d;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        typename C::Floats f, g;
        widen<BF16>(x[r][i], f);
        widen<BF16>(dy[r][i], g);
        const float m = in ? mu[r] : 0.f;   // (0 times an h of infinity past d would be NaN in the row's sums)
#pragma unroll
        for (int e = 0; e < C::kN; ++e) {
          const float h = (RMS ? f[e] : f[e] - m) * rs[r];
          const float gw = g[e] * wf[e], gc = g[e] * cf[r];
          if constexpr (!RMS) s[2 * r] += gw;
          s[2 * r + 1] = fmaf(gw, h, s[2 * r + 1]);
          aw[i][e] = fmaf(gc, h, aw[i][e]);
          if constexpr (!RMS) ab[i][e] += gc;
        }
      }
      // (summed here: the compiler would do it behind the reduction and hold h and gc till then)
#pragma unroll
      for (int e = 0; e < C::kN; ++e) {
        asm volatile("" : "+v"(aw[i][e]));
        if constexpr (!RMS) asm volatile("" : "+v"(ab[i][e]));
      }
    }
    Row<BF16, NC, W>::sums(s, own, turn);
    if constexpr (BF16) {
      keep_packed(x);
      keep_packed(dy);
      keep_packed(w);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const __amdgpu_buffer_rsrc_t to = row_buffer(a.dx, row + r, a.d * C::kElem, a.dx && row + r < end);
      const float m1 = s[2 * r] * a.inv, m2 = s[2 * r + 1] * a.inv;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        typename C::Floats f, g, wf;
        widen<BF16>(x[r][i], f);
        widen<BF16>(dy[r][i], g);
        widen<BF16>(w[0][i], wf);
#pragma unroll
        for (int e = 0; e < C::kN; ++e) {
          const float h = (RMS ? f[e] : f[e] - mu[r]) * rs[r];
          f[e] = fmaf(-h, m2, RMS ? g[e] * wf[e] : fmaf(g[e], wf[e], -m1)) * rs[r];
        }
        store_chunk(to, lane + 64 * W * i, narrow<BF16>(f));
      }
    }
  }
  if (!a.dw && !a.db) return;
  float* part = a.part ? a.part + (int64_t)blockIdx.x * 2 * a.d : nullptr;
  block_columns<BF16, NC, W>(aw, a.d, lds, [&](int32_t j, float v) {
    if (part) part[j] = v;
    else if (a.dw) store_one<BF16>(a.dw, j, v);
  });
  if constexpr (!RMS)
    block_columns<BF16, NC, W>(ab, a.d, lds, [&](int32_t j, float v) {
      if (part) part[a.d + j] = v;
      else if (a.db) store_one<BF16>(a.db, j, v);
    });
}

// Columns of `rows` rows of partial sums, `pitch` apart, four to a thread: 1024 / slots
// threads lie along the columns, and `slots` (a power of two) share the rows, whose sums
// are added in a fixed order. The sums are those of the threads below 1024 / slots.
__device__ __forceinline__ f32x4_t add_rows(const float* p, int32_t rows, int64_t pitch, int32_t columns, int32_t slots, f32x4_t* lds) {
  const int32_t along = 1024 / slots, q = threadIdx.x & (along - 1), slot = threadIdx.x / along;
  f32x4_t s = {};
  if (4 * q < columns)
    for (int32_t r = slot; r < rows; r += 4 * slots) {   // (four loads in flight)
      f32x4_t v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = r + u * slots < rows ? *(const f32x4_t*)(p + (r + u * slots) * pitch + 4 * q) : f32x4_t{};
      s += (v[0] + v[1]) + (v[2] + v[3]);
    }
  for (int32_t h = slots >> 1; h > 0; h >>= 1) {
    if (slot >= h && slot < 2 * h) lds[threadIdx.x - h * along] = s;
    __syncthreads();
    if (slot < h) s += lds[threadIdx.x];
    __syncthreads();
  }
  return s;
}

// dw and db from the blocks' sums.
template <bool BF16>
__global__ __launch_bounds__(1024) void k_backward_columns(Args a, int32_t slots) {
  __shared__ __align__(16) f32x4_t lds[512];
  const int32_t j0 = blockIdx.x * (4096 / slots), j = j0 + 4 * threadIdx.x;
  char* out = blockIdx.y ? a.db : a.dw;
  if (!out) return;
  const f32x4_t s = add_rows(a.part + (int64_t)blockIdx.y * a.d + j0, a.blocks, 2 * (int64_t)a.d, a.d - j0, slots, lds);
  if (threadIdx.x * slots >= 1024 || j >= a.d) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) store_one<BF16>(out, j + e, s[e]);
}

// A sample's norm from the sum of its squares.
__device__ __forceinline__ void store_norm(const Args& a, int64_t i, double t) {
  a.n[i] = (float)(a.accumulate ? (double)a.n[i] + t : t);
}

// Column sums of G h and of G over a sample's rows (the y-th of a.blocks shares of
// them), and where a work group has them all the norm. The statistics are taken again
// from the rows, which are read anyway: two reductions, one behind the other, between the
// loads and the sums. Bound by HBM and that latency: 4 x 4096 rows of 2048 bf16 23 to 26 us,
// 5.2 to 5.7 TB/s, and the columns 5 to 5.6 us; 256 samples of 64 rows 27 us a call. (The
// next rows loaded ahead: 34.1 us a call against 33.7.)
template <bool BF16, bool RMS, int NC, int W, int R>
__global__ __launch_bounds__((64 * kSumWaves<BF16, NC, W>)) void k_norm(Args a) {
  using C = Chunk<BF16>;
  __shared__ __align__(16) float lds[kSumLds<BF16, NC, W, R>];
  __shared__ double total[kSumWaves<BF16, NC, W>];
  int turn = 0;
  const int lane = threadIdx.x % (64 * W);
  const int32_t mine = __builtin_amdgcn_readfirstlane(threadIdx.x / (64 * W));
  constexpr int32_t kStep = kSumRows<BF16, NC, W> * R;
  float* own = lds + mine * 4 * W * R;
  const int64_t item = blockIdx.x + (int64_t)blockIdx.y * gridDim.x, i = item / a.blocks;
  const int32_t share = (int32_t)(item - i * a.blocks);
  if (i * a.T >= a.N) return;
  const int64_t first = i * a.T + (int64_t)share * kStep, step = (int64_t)a.blocks * kStep;
  const int32_t end = (int32_t)((i + 1) * a.T);
  float aw[NC][C::kN] = {}, ab[NC][C::kN] = {};
  for (int64_t at = first; at < end; at += step) {
    const int64_t row = at + mine * R;
    uint4 x[R][NC], dy[R][NC];
    load_rows<BF16, NC, W, R>(a.x, row, end, a.d, lane, x);
    load_rows<BF16, NC, W, R>(a.dy, row, end, a.d, lane, dy);
    float mu[R], rs[R];
    statistics<BF16, RMS, NC, W, R>(x, a.d, a.eps, a.inv, lane, own, turn, mu, rs);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row + r >= end) break;
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        typename C::Floats f, g;
        widen<BF16>(x[r][k], f);
        widen<BF16>(dy[r][k], g);
#pragma unroll
        for (int e = 0; e < C::kN; ++e) {
          aw[k][e] = fmaf(g[e], (RMS ? f[e] : f[e] - mu[r]) * rs[r], aw[k][e]);
          if constexpr (!RMS) ab[k][e] += g[e];
        }
      }
    }
  }
  if (a.blocks > 1) {
    float* part = a.part + item * 2 * a.d;
    if (share == 0 && threadIdx.x == 0) a.arrived[i] = 0;   // (of the second launch)
    block_columns<BF16, NC, W>(aw, a.d, lds, [&](int32_t j, float v) { part[j] = v; });
    if constexpr (!RMS) block_columns<BF16, NC, W>(ab, a.d, lds, [&](int32_t j, float v) { part[a.d + j] = v; });
    return;
  }
  double s = 0.0;
  if (a.first == 0) block_columns<BF16, NC, W>(aw, a.d, lds, [&](int32_t, float v) { s += (double)v * v; });
  if constexpr (!RMS)
    if (a.first + a.columns > a.d) block_columns<BF16, NC, W>(ab, a.d, lds, [&](int32_t, float v) { s += (double)v * v; });
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) total[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  double t = 0.0;
#pragma unroll
  for (int v = 0; v < kSumWaves<BF16, NC, W>; ++v) t += total[v];
  store_norm(a, i, t);
}

// The norms from the work groups' column sums: 4096 / slots columns of a sample a work
// group; the last one of a sample to arrive adds their squares in order. The squares and
// the counter go past the L2 caches, which the XCDs do not share, and are waited for: a
// fence instead, which writes back and empties an L2, took 287 us for 256 samples of
// 2048 columns in 16384 work groups.
template <int UNUSED = 0>
__global__ __launch_bounds__(1024) void k_norm_columns(Args a, int64_t samples, int32_t groups, int32_t slots) {
  __shared__ __align__(16) f32x4_t lds[512];
  __shared__ double total[16];
  const int64_t item = blockIdx.x + (int64_t)blockIdx.y * gridDim.x, i = item / groups;
  const int32_t g = (int32_t)(item - i * groups), j0 = g * (4096 / slots);
  if (i >= samples) return;
  const f32x4_t v = add_rows(a.part + i * a.blocks * 2 * a.d + a.first + j0, a.blocks, 2 * (int64_t)a.d, a.columns - j0, slots, lds);
  double t = 0.0;
  if (threadIdx.x * slots < 1024)
#pragma unroll
    for (int e = 0; e < 4; ++e) t += (double)v[e] * v[e];
  t = wave_sum(t);
  if ((threadIdx.x & 63) == 0) total[threadIdx.x >> 6] = t;
  __syncthreads();
  if (threadIdx.x >= 64) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) t += total[w];
  if (groups > 1) {
    double* mine = a.parts + i * groups;
    uint32_t before = 0;
    if (threadIdx.x == 0) {
      __hip_atomic_store(mine + g, t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (it has reached the memory)
      before = __hip_atomic_fetch_add(a.arrived + i, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane((int)before) != groups - 1) return;
    t = 0.0;
    for (int32_t k = threadIdx.x; k < groups; k += 64) t += __hip_atomic_load(mine + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    t = wave_sum(t);
  }
  if (threadIdx.x == 0) store_norm(a, i, t);
}

}  // namespace ln
}  // namespace dpn
