// Embedding kernels: scaled lookup, the order of a batch's ids, and sums of
// gradient rows over runs of equal ids, for the per-sample norm and for the
// gradient of the table.
//
//   lookup  out[q] = s W[tok[q]]
//   norm    n_i = s^2 sum_v || sum_{q in sample i, tok[q] = v} G[q] ||^2
//   grad    dW[v] = s sum_q c_{sample(q)} [tok[q] = v] G[q]
//
// q = i T + t numbers the N = B T positions of a batch. Ids outside [0, V)
// have no row: they are given the key V, sort behind every row and are skipped.
//
// All three are bound by HBM: the rows are read once, sums are held in fp32
// registers, 16 bytes a lane and row, and there are no atomics, so every
// result is bitwise reproducible.
#pragma once
#include "device_common.h"

namespace dpn {
namespace embed {

// Block of a launch by its number: a dimension of a grid holds fewer than 2^32
// threads, so that many blocks lie along two (grid_of; the last ones may be past
// the end).
__device__ __forceinline__ uint32_t block_number() { return blockIdx.x + blockIdx.y * gridDim.x; }

// ---------------------------------------------------------------------------
// Order: the positions grouped by id, each group in position order. The groups
// are sorted by a mixed id, which spreads neighbouring ids (the frequent ones of
// a vocabulary) over the range; positions without a row come last.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kMaxDigits = 1024;
constexpr int kBucketBits = 8;
constexpr int kScanMost = 24 * kSortThreads;                 // positions of an order made in one launch
constexpr int kScanBits = kBucketBits + 10;                  // id bits of an order made in one launch
constexpr int kMaxSortBlocks = 64;

// Ids below 2^bits mixed one to one: a product with an odd number near 2^bits
// over the golden ratio, modulo 2^bits. Positions without a row get 2^bits.
__host__ __device__ __forceinline__ uint32_t mix_factor(int bits) { return (0x9e3779b1u >> (32 - bits)) | 1u; }
__device__ __forceinline__ uint32_t mixed(int32_t id, int32_t V, int bits) {
  return id < V ? ((uint32_t)id * mix_factor(bits)) & ((1u << bits) - 1u) : 1u << bits;
}

struct SortShared {
  uint32_t cnt[kSortWaves][kMaxDigits];
  uint32_t base[kMaxDigits];
  uint32_t scan[kSortWaves];
};

__device__ __forceinline__ int32_t id_key(const void* tok, int idx64, int64_t q, int32_t V) {
  const int64_t t = idx64 ? ((const int64_t*)tok)[q] : (int64_t)((const int32_t*)tok)[q];
  return (t >= 0 && t < (int64_t)V) ? (int32_t)t : V;
}

// Lanes of the wave (among `valid`) whose digit equals this lane's.
__device__ __forceinline__ uint64_t match_digit(uint32_t digit, int bits, uint64_t valid) {
  uint64_t m = valid;
  for (int b = 0; b < bits; ++b) {
    const uint64_t has = __ballot((digit >> b) & 1u);
    m &= ((digit >> b) & 1u) ? has : ~has;
  }
  return m;
}

// Counts one round of a wave's keys into its counters and returns the lane's
// rank among the wave's equal digits so far (stable: in position order).
__device__ __forceinline__ uint32_t count_round(uint32_t* cnt, uint32_t digit, int bits, bool valid) {
  const uint64_t m = match_digit(digit, bits, __ballot(valid));
  uint32_t rank = 0;
  if (valid) {
    const int lane = __lane_id();
    const uint32_t before = (uint32_t)__popcll(m & ((1ull << lane) - 1ull));
    const uint32_t old = cnt[digit];
    rank = old + before;
    if (before == 0) cnt[digit] = old + (uint32_t)__popcll(m);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the next round reads what this one counted
  __builtin_amdgcn_wave_barrier();
  return rank;
}

__device__ __forceinline__ void zero_counts(SortShared& sh, int bits) {
  for (int j = threadIdx.x; j < kSortWaves << bits; j += kSortThreads) sh.cnt[j >> bits][j & ((1 << bits) - 1)] = 0;
  __syncthreads();
}

// cnt[w][digit] becomes the wave's exclusive offset among the block's equal
// digits; returns the block's total of digit threadIdx.x (0 past the digits).
__device__ __forceinline__ uint32_t scan_waves(SortShared& sh, int digits) {
  __syncthreads();
  uint32_t run = 0;
  if ((int)threadIdx.x < digits) {
    uint32_t c[kSortWaves];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) c[w] = sh.cnt[w][threadIdx.x];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      sh.cnt[w][threadIdx.x] = run;
      run += c[w];
    }
  }
  return run;
}

// Exclusive sum of v over the threads of the block.
__device__ __forceinline__ uint32_t scan_block(SortShared& sh, uint32_t v) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = __shfl_up(inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 63) sh.scan[wv] = inc;
  __syncthreads();
  uint32_t all[kSortWaves], before = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) all[w] = sh.scan[w];
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) before += w < wv ? all[w] : 0u;
  return before + inc - v;
}

// An order in one launch: every block reads all ids, counts those of the buckets
// before its own (the leading bits of the mixed id), and sorts those of its own
// by the remaining bits; the last block places the positions without a row too.
// A bucket holds one part in 256 of the distinct ids, so that reading and mixing
// the ids is most of the work; the frequent ids' buckets take longest. A wave gathers
// its matches in LDS and ranks them 64 at a time. Bound by latency: 14 us for 16384
// positions of a vocabulary's frequencies (131072 ids), against 20 and three more
// launches by radix passes; 33000 positions (50257 ids) 26 against 21, hence kScanMost.
constexpr int kAhead = 8;                          // rounds whose ids a wave loads together
constexpr int kPending = (kAhead + 2) * kWave;     // matches that a wave holds

// A wave's segment of the positions, walked in order: seen(mixed id) for every
// position (2^bits: no row, all ones: none), take(mixed id, position, lanes) for the
// matches of bucket b, 64 at a time. Returns the number of matches where pend still
// holds all of them, else -1.
template <typename S, typename F>
__device__ __forceinline__ int walk(const void* tok, int idx64, int32_t N, int32_t V, int bits, int rem, uint32_t b, int seg0,
                                    int rounds, uint2 (&pend)[kPending], S seen, F take) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  bool whole = true;
  for (int r0 = 0; r0 < rounds; r0 += kAhead) {
    if (n > kPending - kAhead * kWave) {   // rank what does not leave room for the next rounds
      int at = 0;
      for (; at + 64 <= n; at += 64) take(pend[at + lane].x, pend[at + lane].y, 64);
      const uint2 x = pend[min(at + lane, kPending - 1)];
      __builtin_amdgcn_wave_barrier();
      pend[lane] = x;
      n -= at;
      whole = false;
    }
    uint32_t h[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int q = seg0 + (r0 + u) * kWave + lane;
      h[u] = r0 + u < rounds && q < N ? mixed(id_key(tok, idx64, q, V), V, bits) : ~0u;
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      seen(h[u], seg0 + (r0 + u) * kWave + lane);
      const bool match = h[u] >> rem == b;
      const uint64_t m = __ballot(match);
      if (match) pend[n + __popcll(m & ((1ull << lane) - 1ull))] = make_uint2(h[u], (uint32_t)(seg0 + (r0 + u) * kWave + lane));
      n += __popcll(m);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  for (int at = 0; at < n; at += 64) {
    const uint2 x = pend[min(at + lane, kPending - 1)];
    take(x.x, x.y, min(64, n - at));
  }
  return whole ? n : -1;
}

__global__ __launch_bounds__(kSortThreads) void k_order_scan(const void* tok, int idx64, int32_t N, int32_t V, int bits,
                                                             uint32_t inverse, int32_t* keys, int32_t* pos, int32_t* start) {
  __shared__ SortShared sh;
  __shared__ uint2 pend[kSortWaves][kPending];
  __shared__ uint32_t below[kSortWaves], none[kSortWaves];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t b = blockIdx.x;
  const bool last = b + 1 == gridDim.x;
  const int rem = bits > kBucketBits ? bits - kBucketBits : 0, digits = 1 << rem;
  const int rounds = (N + kSortThreads - 1) / kSortThreads;
  const int seg0 = wv * rounds * kWave;   // a contiguous segment a wave, so waves in order are positions in order
  zero_counts(sh, rem);
  uint32_t less = 0, without = 0;
  const int held = walk(tok, idx64, N, V, bits, rem, b, seg0, rounds, pend[wv],
                        [&](uint32_t h, int) {
                          less += h >> rem < b ? 1u : 0u;
                          without += h == 1u << bits ? 1u : 0u;
                        },
                        [&](uint32_t x, uint32_t, int n) { count_round(sh.cnt[wv], x & (digits - 1), rem, lane < n); });
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    less += __shfl_xor(less, o);
    without += __shfl_xor(without, o);
  }
  if (lane == 0) below[wv] = less, none[wv] = without;
  const uint32_t total = scan_waves(sh, digits);
  const uint32_t before = scan_block(sh, total);
  uint32_t offset = 0, ended = 0, tail = 0;   // positions below the bucket; without a row, in all and of the waves before
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    offset += below[w];
    ended += none[w];
    tail += w < wv ? none[w] : 0u;
  }
  if ((int)threadIdx.x < digits) sh.base[threadIdx.x] = offset + before;
  if (threadIdx.x == 0) start[b] = (int32_t)offset;
  if (last && threadIdx.x == 0) start[b + 1] = N - (int32_t)ended;
  __syncthreads();
  tail += (uint32_t)N - ended;
  const auto place = [&](uint32_t x, uint32_t q, int n) {
    const uint32_t dg = x & (digits - 1);
    const uint32_t rank = count_round(sh.cnt[wv], dg, rem, lane < n);
    if (lane < n) {
      const uint32_t to = sh.base[dg] + rank;
      keys[to] = (int32_t)((x * inverse) & ((1u << bits) - 1u));
      pos[to] = (int32_t)q;
    }
  };
  if (held >= 0 && !(last && ended > 0)) {
    for (int at = 0; at < held; at += 64) {
      const uint2 x = pend[wv][min(at + lane, kPending - 1)];
      place(x.x, x.y, min(64, held - at));
    }
    return;
  }
  walk(tok, idx64, N, V, bits, rem, b, seg0, rounds, pend[wv],
       [&](uint32_t h, int q) {
         if (!last) return;
         const bool mine = h == 1u << bits;
         const uint64_t m = __ballot(mine);
         if (mine) {
           const uint32_t to = tail + (uint32_t)__popcll(m & ((1ull << lane) - 1ull));
           keys[to] = V;
           pos[to] = q;
         }
         tail += (uint32_t)__popcll(m);
       },
       place);
}

// Larger batches and tables: radix passes over the mixed ids, `per` positions a block: digit counts of every
// block first (hist[block][digit]), then the stable scatter. src_keys is null
// in the first pass, which reads the ids.
__device__ __forceinline__ int32_t load_key(const void* tok, int idx64, const int32_t* src_keys, int64_t q, int32_t V) {
  return src_keys ? src_keys[q] : id_key(tok, idx64, q, V);
}

__global__ __launch_bounds__(kSortThreads) void k_order_count(const void* tok, int idx64, const int32_t* src_keys, int32_t N,
                                                              int32_t V, int id_bits, int shift, int bits, int per,
                                                              uint32_t* hist) {
  __shared__ uint32_t cnt[kMaxDigits];
  const int digits = 1 << bits;
  for (int j = threadIdx.x; j < digits; j += kSortThreads) cnt[j] = 0;
  __syncthreads();
  const int64_t lo = (int64_t)blockIdx.x * per, hi = lo + per < N ? lo + per : N;
  for (int64_t q = lo + threadIdx.x; q < hi; q += kSortThreads)
    atomicAdd(&cnt[(mixed(load_key(tok, idx64, src_keys, q, V), V, id_bits) >> shift) & (digits - 1)], 1u);
  __syncthreads();
  for (int j = threadIdx.x; j < digits; j += kSortThreads) hist[blockIdx.x * digits + j] = cnt[j];
}

constexpr int kHeldRounds = 4;   // rounds of a wave whose keys stay in registers between the two walks

__global__ __launch_bounds__(kSortThreads) void k_order_scatter(const void* tok, int idx64, const int32_t* src_keys,
                                                                const int32_t* src_pos, int32_t N, int32_t V, int id_bits,
                                                                int shift, int bits, int per, const uint32_t* hist, int32_t* keys,
                                                                int32_t* pos) {
  __shared__ SortShared sh;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int digits = 1 << bits, nb = gridDim.x;
  const int64_t lo = (int64_t)blockIdx.x * per, hi = lo + per < N ? lo + per : N;
  const int seg = (per + kSortWaves - 1) / kSortWaves;   // positions a wave walks, in order
  const int64_t wlo = lo + (int64_t)wv * seg < hi ? lo + (int64_t)wv * seg : hi;
  const int64_t whi = wlo + seg < hi ? wlo + seg : hi;
  const bool held = seg <= kHeldRounds * kWave;
  int32_t key[kHeldRounds], ps[kHeldRounds];
  if (held) {
#pragma unroll
    for (int r = 0; r < kHeldRounds; ++r) {
      const int64_t q = wlo + r * kWave + lane;
      key[r] = q < whi ? load_key(tok, idx64, src_keys, q, V) : 0;
      ps[r] = q < whi && src_pos ? src_pos[q] : (int32_t)q;
    }
  }
  // where this block's elements of each digit go
  uint32_t total = 0, before = 0;
  if ((int)threadIdx.x < digits) {
    for (int b0 = 0; b0 < nb; b0 += 16) {   // (16 loads in flight)
      uint32_t h[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) h[j] = b0 + j < nb ? hist[(b0 + j) * digits + threadIdx.x] : 0u;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (b0 + j < (int)blockIdx.x) before += h[j];
        total += h[j];
      }
    }
  }
  const uint32_t base = scan_block(sh, total) + before;
  if ((int)threadIdx.x < digits) sh.base[threadIdx.x] = base;
  zero_counts(sh, bits);
  if (held) {
    uint32_t rank[kHeldRounds];
#pragma unroll
    for (int r = 0; r < kHeldRounds; ++r) {
      if (wlo + r * kWave < whi)
        rank[r] = count_round(sh.cnt[wv], (mixed(key[r], V, id_bits) >> shift) & (digits - 1), bits, wlo + r * kWave + lane < whi);
    }
    scan_waves(sh, digits);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kHeldRounds; ++r) {
      if (wlo + r * kWave + lane < whi) {
        const uint32_t dg = (mixed(key[r], V, id_bits) >> shift) & (digits - 1);
        const uint32_t to = sh.base[dg] + sh.cnt[wv][dg] + rank[r];
        keys[to] = key[r];
        pos[to] = ps[r];
      }
    }
    return;
  }
  for (int64_t q0 = wlo; q0 < whi; q0 += kWave) {
    const int64_t q = q0 + lane;
    const bool in = q < whi;
    const uint32_t dg = in ? (mixed(load_key(tok, idx64, src_keys, q, V), V, id_bits) >> shift) & (digits - 1) : 0;
    count_round(sh.cnt[wv], dg, bits, in);
  }
  scan_waves(sh, digits);
  __syncthreads();
  // the same walk again, now from each wave's offsets
  for (int64_t q0 = wlo; q0 < whi; q0 += kWave) {
    const int64_t q = q0 + lane;
    const bool in = q < whi;
    const int32_t k = in ? load_key(tok, idx64, src_keys, q, V) : 0;
    const uint32_t dg = (mixed(k, V, id_bits) >> shift) & (digits - 1);
    const uint32_t rank = count_round(sh.cnt[wv], dg, bits, in);
    if (in) {
      const uint32_t to = sh.base[dg] + rank;
      keys[to] = k;
      pos[to] = src_pos ? src_pos[q] : (int32_t)q;
    }
  }
}

// ---------------------------------------------------------------------------
// Rows: 16 bytes a lane, 8 bf16 or 4 fp32 columns; a slice is one wave's width
// ---------------------------------------------------------------------------
template <bool BF16>
struct Row {
  static constexpr int kElems = BF16 ? 8 : 4;
  static constexpr int kSlice = kElems * kWave;
  static constexpr int kBytes = BF16 ? 2 : 4;
  __device__ static void add(float (&acc)[kElems], const uint4& v, float w) {
    if constexpr (BF16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = word(v, j);
        acc[2 * j] = fmaf(w, __uint_as_float(x << 16), acc[2 * j]);
        acc[2 * j + 1] = fmaf(w, __uint_as_float(x & 0xffff0000u), acc[2 * j + 1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = fmaf(w, __uint_as_float(word(v, j)), acc[j]);
    }
  }
  // rounded once to the element type (to nearest even)
  __device__ static uint4 pack(const float (&a)[kElems]) {
    if constexpr (BF16) {
      uint32_t b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = f32_to_bf16_bits(a[j]);
      return pack8(b);
    } else {
      return make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]), __float_as_uint(a[3]));
    }
  }
};

// Sum of v over the wave in a fixed order, the same in every lane.
__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// A wave copies kLookupRows rows at a time, 16 bytes a lane. Bound by HBM, which the
// distinct rows and the output cross once: 16384 rows of 2048 bf16 out of 131072 take
// 20 us, 134 MB at 6.6 TB/s; 37 rows of 1000 floats 3 us, the latency of two loads.
constexpr int kLookupRows = 4;   // rows a wave has in flight

template <bool BF16>
__global__ __launch_bounds__(256) void k_lookup(const void* tok, int idx64, const char* W, char* out, int64_t N, int32_t V,
                                                int32_t d, int32_t slices, float scale) {
  using R = Row<BF16>;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)block_number() * 4 + (threadIdx.x >> 6);
  const int64_t q0 = item / slices * kLookupRows;
  const int col = (int)(item % slices) * R::kSlice + lane * R::kElems;
  if (q0 >= N || col >= d) return;
  uint4 v[kLookupRows];
#pragma unroll
  for (int r = 0; r < kLookupRows; ++r) {
    v[r] = make_uint4(0, 0, 0, 0);
    if (q0 + r < N) {
      const int32_t id = id_key(tok, idx64, q0 + r, V);
      if (id < V) v[r] = ldg16(W + ((int64_t)id * d + col) * R::kBytes);
    }
  }
#pragma unroll
  for (int r = 0; r < kLookupRows; ++r) {
    if (q0 + r < N) {
      float a[R::kElems] = {};
      R::add(a, v[r], scale);
      stg16(out + ((q0 + r) * d + col) * R::kBytes, R::pack(a));
    }
  }
}

// ---------------------------------------------------------------------------
// Sums over runs of equal keys
//
// The sorted positions are cut into chunks of about R, one wave to a chunk and
// column slice. A chunk boundary at x = c R moves on to the next run start
// within R positions, so only runs of R positions and more are ever cut. The
// pieces of a cut run go to the workspace and a second launch joins them.
// Runs are of equal (id, sample) for the norm and of equal id for the gradient.
// ---------------------------------------------------------------------------
struct Runs {
  const int32_t* keys;   // grouped by id, V for positions without a row last
  const int32_t* pos;
  const int32_t* start;  // first position of each bucket, or null
  int bits;              // of the mixed ids
  int32_t N, T, V;
  double per;            // 1 / T
  int R;                 // at most 16, so that a wave's lanes see both ends of a chunk
  int32_t chunks;
};

enum { RUN_NORM = 0, RUN_GRAD = 1 };

__device__ __forceinline__ int32_t in_batch(const Runs& a, int32_t q) { return (int32_t)min((uint32_t)q, (uint32_t)a.N - 1u); }
__device__ __forceinline__ int32_t in_table(const Runs& a, int32_t key) { return (int32_t)min((uint32_t)key, (uint32_t)a.V); }

// Sample of position q, q / T: the fp64 quotient is off by less than one part in
// 2^51, so at most the last whole step of an exact multiple is missed.
__device__ __forceinline__ int32_t sample_of(const Runs& a, int32_t q) {
  const int32_t i = (int32_t)((double)q * a.per);
  return q - i * a.T >= a.T ? i + 1 : i;
}

// What a wave knows of chunk c: lane l describes sorted position c R - 1 + l, and
// the chunk reaches from x0 to x1. One round of loads covers both boundaries.
// (Values outside the batch or the table, which no order of this batch holds, are
// kept in bounds.)
struct Chunk {
  int32_t at;            // position of lane 0
  int32_t key, pos, smp;
  uint64_t starts;       // lanes whose position starts a run (positions past the end do)
  int32_t x0, x1;
  bool cut0, cut1;       // the boundary lies inside a run
};

template <int MODE>
__device__ __forceinline__ Chunk look_at(const Runs& a, int32_t c) {
  Chunk w;
  const int lane = __lane_id();
  w.at = (int32_t)((int64_t)c * a.R - 1);
  const int64_t j = (int64_t)w.at + lane;
  const bool in = j >= 0 && j < a.N;
  w.key = in ? in_table(a, a.keys[j]) : a.V;
  w.pos = in ? in_batch(a, a.pos[j]) : 0;
  w.smp = sample_of(a, w.pos);
  const int32_t key = __shfl_up(w.key, 1), smp = __shfl_up(w.smp, 1);
  w.starts = __ballot(!in || j == 0 || w.key != key || (MODE == RUN_NORM && w.smp != smp));
  const uint64_t window = (1ull << a.R) - 1;
  const uint64_t m0 = (w.starts >> 1) & window, m1 = (w.starts >> (1 + a.R)) & window;
  w.cut0 = m0 == 0;
  w.cut1 = m1 == 0;
  w.x0 = (int32_t)min((int64_t)w.at + 1 + (m0 ? __builtin_ctzll(m0) : 0), (int64_t)a.N);
  w.x1 = (int32_t)min((int64_t)w.at + 1 + a.R + (m1 ? __builtin_ctzll(m1) : 0), (int64_t)a.N);
  if (c == 0) w.x0 = 0, w.cut0 = false;
  return w;
}

// End of the run that holds sorted position j: a search by all 64 lanes.
template <int MODE>
__device__ __forceinline__ int32_t run_end(const Runs& a, int32_t j) {
  const int32_t key = a.keys[j], smp = MODE == RUN_NORM ? sample_of(a, a.pos[j]) : 0;
  const int lane = __lane_id();
  int64_t lo = j, hi = a.N;   // position lo is in the run, hi is not
  bool near = true;           // most runs end within 64 positions
  while (hi - lo > 1) {
    const int64_t step = near ? 1 : (hi - lo + 63) / 64;
    near = false;
    const int64_t p = lo + step * (lane + 1);
    const bool in = p < hi && a.keys[p] == key && (MODE != RUN_NORM || sample_of(a, a.pos[p]) == smp);
    const int cnt = __popcll(__ballot(in));   // the lanes inside are the first ones
    lo += step * cnt;
    if (cnt < 64) hi = min(hi, lo + step);
  }
  return (int32_t)hi;
}

// Whether id v occurs: a search in its bucket, or in the whole order.
__device__ __forceinline__ bool occurs(const Runs& a, int32_t v) {
  const uint32_t h = mixed(v, a.V, a.bits);
  int32_t lo = 0, hi = a.N;
  if (a.start) {
    const uint32_t b = h >> (a.bits > kBucketBits ? a.bits - kBucketBits : 0);
    lo = a.start[b];
    hi = a.start[b + 1];
  }
  lo = max(lo, 0);
  hi = min(hi, a.N);
  while (lo < hi) {
    const int32_t mid = lo + (hi - lo) / 2;
    const int32_t key = a.keys[mid];
    if (key == v) return true;
    if (mixed(key, a.V, a.bits) < h) lo = mid + 1;
    else hi = mid;
  }
  return false;
}

struct RunArgs {
  Runs runs;
  const char* G;        // [N][d]
  const float* c;       // per-sample weights or null (grad)
  float scale;          // grad
  char* out;            // grad: table [V][d]
  float* val;           // norm: [slices][N] squared sums, at the position that starts the run
  float* part;          // [chunks][2][d]: pieces of runs that started before the chunk / that go on after it
  int32_t d, slices;
  int accumulate;       // grad: add to the table's touched rows
  uint32_t* arrived;    // norm: counters to reset for the sum, or null
  int64_t items;        // chunks x slices
  int64_t fill_blocks;  // grad: blocks behind the items' that clear rows without an id
};

template <bool BF16>
__device__ __forceinline__ void put_row(const RunArgs& a, int32_t key, int col, const float (&acc)[Row<BF16>::kElems]) {
  using R = Row<BF16>;
  char* p = a.out + ((int64_t)key * a.d + col) * R::kBytes;
  if (a.accumulate) {
    float s[R::kElems];
#pragma unroll
    for (int j = 0; j < R::kElems; ++j) s[j] = acc[j];
    R::add(s, ldg16(p), 1.f);
    stg16(p, R::pack(s));
  } else {
    stg16(p, R::pack(acc));
  }
}

template <bool BF16>
__device__ __forceinline__ void put_part(const RunArgs& a, int32_t chunk, int slot, int col,
                                         const float (&acc)[Row<BF16>::kElems]) {
  float* p = a.part + ((int64_t)chunk * 2 + slot) * a.d + col;
#pragma unroll
  for (int j = 0; j < Row<BF16>::kElems; j += 4)
    stg16(p + j, make_uint4(__float_as_uint(acc[j]), __float_as_uint(acc[j + 1]), __float_as_uint(acc[j + 2]),
                            __float_as_uint(acc[j + 3])));
}

constexpr int kRowsAhead = 8;    // rows a wave loads ahead of adding them
constexpr int kFillRows = 64;    // table rows a clearing block looks at

// One wave an item: the rows of a chunk's positions in the groups' order, a slice of
// their columns, 16 bytes a lane and kRowsAhead rows in flight, added in registers
// until a run ends. Runs inside a chunk are finished here, so most rows of G are read
// once and leave nothing but a float (norm) or their table row (gradient); chunks of 32
// instead of 16 positions halve the pieces of cut runs but took longer, as one window of
// 64 lanes then no longer describes a chunk. The gradient clears the rows without an id
// in blocks behind the items', with stores that pass the caches. Bound by HBM: norm of
// 16384 positions of 2048 bf16 18 us (67 MB, 3.7 TB/s, of which 4 us are the latency of
// keys, positions and first rows), gradient into 131072 rows 110 us (604 MB, 5.5 TB/s).
template <bool BF16, int MODE>
__global__ __launch_bounds__(256) void k_run_sums(RunArgs a) {
  using R = Row<BF16>;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t item_blocks = (a.items + 3) / 4, block = block_number();
  if (MODE == RUN_GRAD && block >= item_blocks) {
    // clear the rows of ids that do not occur: lane r looks for row v0 + r
    const int64_t v0 = (block - item_blocks) * kFillRows;
    const int64_t v = v0 + lane;
    const bool absent = v < a.runs.V && !occurs(a.runs, (int32_t)v);
    uint64_t m = __ballot(absent);
    for (int j = 0; m; ++j) {
      const int r = __builtin_ctzll(m);
      m &= m - 1;
      if ((j & 3) != wv) continue;   // the block's waves take rows in turn
      char* p = a.out + (v0 + r) * a.d * R::kBytes;
      for (int col = lane * R::kElems; col < a.d; col += R::kSlice) __builtin_nontemporal_store(u32x4_t{0, 0, 0, 0}, (DPN_GLOBAL u32x4_t*)(p + (int64_t)col * R::kBytes));
    }
    return;
  }
  const int64_t item = block * 4 + wv;
  if (item >= a.items) return;
  const int32_t chunk = (int32_t)(item / a.slices);
  const int slice = (int)(item % a.slices);
  const int col = slice * R::kSlice + lane * R::kElems;
  const bool on = col < a.d;
  if (MODE == RUN_NORM && a.arrived && slice == 0 && lane == 0) {
    for (int64_t i = chunk; i * a.runs.T < a.runs.N; i += a.runs.chunks) a.arrived[i] = 0;
  }
  const Chunk w = look_at<MODE>(a.runs, chunk);
  const int off = w.x0 - w.at, len = w.x1 - w.x0;   // the chunk's first lane; at most 2 R - 1 rows
  const bool mine = lane >= off && lane < off + len;
  const int n = __popcll(__ballot(mine && w.key < a.runs.V));   // rows: the first ones, as V sorts last
  const uint64_t starts = w.starts >> off;
  if (MODE == RUN_NORM) {
    // every position's value is written once: 0 unless it starts a run
    if (mine && !(w.key < a.runs.V && ((w.starts >> lane) & 1))) a.val[(int64_t)slice * a.runs.N + w.pos] = 0.f;
  }
  if (n == 0) return;
  float wgt = 1.f;
  if (MODE == RUN_GRAD) wgt = a.c && mine ? a.scale * a.c[w.smp] : a.scale;
  float acc[R::kElems] = {};
  int first = 0;
  for (int j0 = 0; j0 < n; j0 += kRowsAhead) {
    uint4 v[kRowsAhead];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      v[u] = make_uint4(0, 0, 0, 0);
      if (j0 + u < n && on) {
        const int32_t q = __builtin_amdgcn_readlane(w.pos, off + j0 + u);
        v[u] = ldg16(a.G + ((int64_t)q * a.d + col) * R::kBytes);
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const int j = j0 + u;
      if (j < n) {
        float c = 1.f;
        if (MODE == RUN_GRAD) c = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wgt), off + j));
        R::add(acc, v[u], c);
        // the run ends here, or the chunk does
        if (j + 1 == n || ((starts >> (j + 1)) & 1)) {
          const bool head = first == 0 && w.cut0;                 // started before the chunk
          const bool tail = j + 1 == len && w.cut1;               // goes on after it
          if (head || tail) {
            if (on) put_part<BF16>(a, chunk, head ? 0 : 1, col, acc);
          } else if (MODE == RUN_NORM) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < R::kElems; ++e) s = fmaf(acc[e], acc[e], s);
            s = wave_sum_f32(s);
            if (lane == 0) a.val[(int64_t)slice * a.runs.N + __builtin_amdgcn_readlane(w.pos, off + first)] = s;
          } else if (on) {
            put_row<BF16>(a, __builtin_amdgcn_readlane(w.key, off + first), col, acc);
          }
          first = j + 1;
#pragma unroll
          for (int e = 0; e < R::kElems; ++e) acc[e] = 0.f;
        }
      }
    }
  }
}

// Joins the pieces of each cut run: the block of the chunk that the run starts
// in adds that chunk's tail and the heads of the chunks after it, four waves
// in turn, their sums added in wave order. Bound by latency: 7 us for 4096 items, most
// of which find no cut run.
template <bool BF16, int MODE>
__global__ __launch_bounds__(256) void k_run_join(RunArgs a) {
  using R = Row<BF16>;
  __shared__ float sums[3][R::kElems][kWave];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const uint32_t block = block_number();
  const int32_t chunk = (int32_t)(block / (uint32_t)a.slices);
  const int slice = (int)(block % (uint32_t)a.slices);
  if (chunk >= a.runs.chunks) return;
  const Chunk w = look_at<MODE>(a.runs, chunk);
  if (!w.cut1) return;
  // the run at x1 started in this chunk unless the chunk holds it whole, cut on both sides
  const int off = w.x0 - w.at;
  const uint64_t inner = (w.starts >> off) & ((1ull << (w.x1 - w.x0)) - 1);
  if (inner == 0) return;
  const int s = off + 63 - __builtin_clzll(inner);   // its first lane
  const int32_t key = __builtin_amdgcn_readlane(w.key, s), pos = __builtin_amdgcn_readlane(w.pos, s);
  if (key >= a.runs.V) return;
  const int32_t e = run_end<MODE>(a.runs, w.x1);
  const int32_t last = min(e / a.runs.R, a.runs.chunks) - 1;   // the last boundary with R positions of the run behind it
  const int col = slice * R::kSlice + lane * R::kElems;
  const bool on = col < a.d;
  float acc[R::kElems] = {};
  if (on) {
    for (int32_t ch = chunk + wv; ch <= last; ch += 32) {
      float4 f[8][R::kElems / 4];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int32_t c = ch + 4 * u;
        const float* p = a.part + ((int64_t)c * 2 + (c == chunk ? 1 : 0)) * a.d + col;
#pragma unroll
        for (int j = 0; j < R::kElems / 4; ++j) f[u][j] = c <= last ? ldg_f32x4(p + 4 * j) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int j = 0; j < R::kElems / 4; ++j) {
          acc[4 * j] += f[u][j].x;
          acc[4 * j + 1] += f[u][j].y;
          acc[4 * j + 2] += f[u][j].z;
          acc[4 * j + 3] += f[u][j].w;
        }
    }
  }
  if (wv > 0) {
#pragma unroll
    for (int j = 0; j < R::kElems; ++j) sums[wv - 1][j][lane] = acc[j];
  }
  __syncthreads();
  if (wv > 0) return;
#pragma unroll
  for (int w = 0; w < 3; ++w)
#pragma unroll
    for (int j = 0; j < R::kElems; ++j) acc[j] += sums[w][j][lane];
  if (MODE == RUN_NORM) {
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < R::kElems; ++j) t = fmaf(acc[j], acc[j], t);
    t = wave_sum_f32(t);
    if (lane == 0) a.val[(int64_t)slice * a.runs.N + pos] = t;
  } else if (on) {
    put_row<BF16>(a, key, col, acc);
  }
}

// n_i (+)= s^2 times the sum of the sample's values, in fp64. Long samples are
// summed by gridDim.x blocks; the last one to arrive adds their parts in order. Bound by
// latency: 4.4 us for 4 samples of 16384 values.
__global__ __launch_bounds__(1024) void k_norm_sum(const float* val, int64_t N, int32_t T, int32_t slices, double scale2,
                                                   float* n, int accumulate, double* parts, uint32_t* arrived) {
  __shared__ double part[16];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t i = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  if (i * T >= N) return;
  double s = 0.0;
  const float* p = val + i * T;
  const int32_t per = (T + gridDim.x - 1) / gridDim.x, t0 = blockIdx.x * per, t1 = min(t0 + per, T);
  for (int s0 = 0; s0 < slices; s0 += 4) {
    for (int t = t0 + threadIdx.x; t < t1; t += 4 * 1024) {   // (16 loads in flight)
      float x[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int sl = s0 + (u >> 2), tt = t + (u & 3) * 1024;
        x[u] = sl < slices && tt < t1 ? p[sl * N + tt] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < 16; ++u) s += (double)x[u];
    }
  }
  s = wave_sum(s);
  if (lane == 0) part[wv] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < 16; ++w) t += part[w];
  if (gridDim.x > 1) {
    double* mine = parts + i * gridDim.x;
    __hip_atomic_store(mine + blockIdx.x, t, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint32_t order = __hip_atomic_fetch_add(arrived + i, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    if (order != gridDim.x - 1) return;
    t = 0.0;
    for (uint32_t b = 0; b < gridDim.x; ++b) t += __hip_atomic_load(mine + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  t *= scale2;
  n[i] = (float)(accumulate ? (double)n[i] + t : t);
}

// ---------------------------------------------------------------------------
// Small batches in one launch, without an order: each wave looks for the equal
// ids itself among at most kSmallIds of them.
// ---------------------------------------------------------------------------
constexpr int kSmallIds = 256;

// Sum of the rows at the positions in `mask` of each 64 ids, weighted.
template <bool BF16, typename W>
__device__ __forceinline__ void add_rows(float (&acc)[Row<BF16>::kElems], const uint64_t (&mask)[kSmallIds / 64],
                                         const char* G, int64_t row_bytes, bool on, W weight) {
#pragma unroll
  for (int k = 0; k < kSmallIds / 64; ++k) {
    uint64_t m = mask[k];
    while (m) {
      int at[kRowsAhead];
      uint4 v[kRowsAhead];
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        at[u] = m ? 64 * k + __builtin_ctzll(m) : -1;
        if (m) m &= m - 1;
        v[u] = at[u] >= 0 && on ? ldg16(G + at[u] * row_bytes) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u)
        if (at[u] >= 0) Row<BF16>::add(acc, v[u], weight(at[u]));
    }
  }
}

// Norm of samples of at most kSmallIds positions, a block a sample. The first
// position of an id stands for its row. Bound by latency: 3 samples of 61 positions of
// 256 floats take 6.2 us, against four launches and 31 us with an order.
template <bool BF16>
__global__ __launch_bounds__(1024) void k_norm_small(const void* tok, int idx64, const char* G, int32_t B, int32_t T, int32_t V,
                                                     int32_t d, double scale2, float* n, int accumulate) {
  using R = Row<BF16>;
  __shared__ int32_t keys[kSmallIds];
  __shared__ double part[16];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t i = block_number();
  if (i >= (uint32_t)B) return;
  const int64_t q0 = (int64_t)i * T;
  if (threadIdx.x < kSmallIds) keys[threadIdx.x] = (int)threadIdx.x < T ? id_key(tok, idx64, q0 + threadIdx.x, V) : V;
  __syncthreads();
  int32_t mine[kSmallIds / 64];
#pragma unroll
  for (int k = 0; k < kSmallIds / 64; ++k) mine[k] = keys[64 * k + lane];
  double sum = 0.0;
  for (int t = wv; t < T; t += 16) {
    const int32_t key = __builtin_amdgcn_readfirstlane(keys[t]);
    if (key >= V) continue;
    uint64_t mask[kSmallIds / 64];
    bool first = true;
#pragma unroll
    for (int k = 0; k < kSmallIds / 64; ++k) {
      mask[k] = __ballot(mine[k] == key);
      if (64 * k + 63 < t) first = first && mask[k] == 0;
      else if (64 * k <= t) first = first && (mask[k] & ((1ull << (t & 63)) - 1ull)) == 0;
    }
    if (!first) continue;
    for (int c0 = 0; c0 < d; c0 += R::kSlice) {
      const int col = c0 + lane * R::kElems;
      float acc[R::kElems] = {};
      add_rows<BF16>(acc, mask, G + (q0 * d + col) * R::kBytes, (int64_t)d * R::kBytes, col < d, [](int) { return 1.f; });
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < R::kElems; ++e) s = fmaf(acc[e], acc[e], s);
      sum += (double)wave_sum_f32(s);
    }
  }
  if (lane == 0) part[wv] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < 16; ++w) t += part[w];
    t *= scale2;
    n[i] = (float)(accumulate ? (double)n[i] + t : t);
  }
}

constexpr int kSmallRows = 16;   // table rows of a block, four a wave

// Gradient of the table from at most kSmallIds positions in all: every block looks for
// its rows among all ids. Bound by latency: 183 positions into 2048 rows of 256 floats
// take 6.7 us.
template <bool BF16>
__global__ __launch_bounds__(256) void k_grad_small(const void* tok, int idx64, RunArgs a) {
  using R = Row<BF16>;
  __shared__ int32_t keys[kSmallIds];
  __shared__ float wgt[kSmallIds];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t v0 = (int32_t)block_number() * kSmallRows;
  {
    const int q = threadIdx.x;
    keys[q] = q < a.runs.N ? id_key(tok, idx64, q, a.runs.V) : a.runs.V;
    wgt[q] = a.c && q < a.runs.N ? a.scale * a.c[sample_of(a.runs, q)] : a.scale;
  }
  __syncthreads();
  int32_t mine[kSmallIds / 64];
#pragma unroll
  for (int k = 0; k < kSmallIds / 64; ++k) mine[k] = keys[64 * k + lane];
  for (int32_t v = v0 + wv; v < min(v0 + kSmallRows, a.runs.V); v += 4) {
    uint64_t mask[kSmallIds / 64], any = 0;
#pragma unroll
    for (int k = 0; k < kSmallIds / 64; ++k) {
      mask[k] = __ballot(mine[k] == v);
      any |= mask[k];
    }
    if (!any && a.accumulate) continue;
    for (int c0 = 0; c0 < a.d; c0 += R::kSlice) {
      const int col = c0 + lane * R::kElems;
      float acc[R::kElems] = {};
      if (any)
        add_rows<BF16>(acc, mask, a.G + (int64_t)col * R::kBytes, (int64_t)a.d * R::kBytes, col < a.d,
                       [&](int q) { return wgt[q]; });
      if (col < a.d) put_row<BF16>(a, v, col, acc);
    }
  }
}

}  // namespace embed
}  // namespace dpn
