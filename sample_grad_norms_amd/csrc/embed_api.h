// Host layer of the embedding calls: argument checks, workspace layout,
// launches. Included by dpnorm.cpp, whose helpers it uses.
#pragma once
#include "embed_kernels.h"

namespace {

constexpr int64_t kMaxPositions = (int64_t)1 << 30;

struct EmbedPlan {
  int32_t N = 0, T = 0, V = 0, d = 0;
  int slices = 0, R = 0;
  int64_t chunks = 0;
  // order
  bool scan = false;   // in one launch
  int id_bits = 0, passes = 0, bits = 0, blocks = 0, per = 0;
  size_t off_pos = 0, off_start = 0, order_bytes = 0, off_key2 = 0, off_pos2 = 0, off_hist = 0, order_ws = 0;
  // run sums: the order and its scratch where the call makes it, then the calls' own
  bool small_norm = false, small_grad = false;
  int sum_blocks = 1;  // of a sample
  size_t off_order = 0, off_order_ws = 0, off_val = 0, off_parts = 0, off_arrived = 0, off_part = 0, norm_ws = 0, off_part_grad = 0, grad_ws = 0;
};

dpnorm_status check_ids(int64_t B, int64_t T, int64_t V) {
  if (B < 1 || T < 1 || V < 1 || V > kMaxPositions || T > kMaxPositions || B > kMaxPositions / T) return DPNORM_ERR_SIZE;
  return DPNORM_OK;
}

dpnorm_status check_rows(dpnorm_dtype dt, int64_t rows, int64_t d) {
  if (dt != DPNORM_BF16 && dt != DPNORM_F32) return DPNORM_ERR_DTYPE;
  const int64_t g = dt == DPNORM_BF16 ? 8 : 4;
  if (d < 1 || d % g != 0 || d > ((int64_t)1 << 24)) return DPNORM_ERR_SIZE;
  if (rows > INT64_MAX / d / 16) return DPNORM_ERR_SIZE;
  return DPNORM_OK;
}

void plan_order(EmbedPlan& pl, int64_t B, int64_t T, int64_t V) {
  pl.N = (int32_t)(B * T);
  pl.T = (int32_t)T;
  pl.V = (int32_t)V;
  pl.id_bits = 1;
  while (((int64_t)1 << pl.id_bits) < V) ++pl.id_bits;
  pl.scan = pl.N <= embed::kScanMost && pl.id_bits <= embed::kScanBits;
  // radix passes of at most 9 bits over id_bits + 1 (the positions without a row)
  pl.passes = (pl.id_bits + 9) / 9;
  pl.bits = (pl.id_bits + pl.passes) / pl.passes;
  // a block for every 1024 positions, up to the 64 whose counts one thread adds up
  pl.blocks = (int)std::min<int64_t>(embed::kMaxSortBlocks, (pl.N + 1023) / 1024);
  pl.per = (pl.N + pl.blocks - 1) / pl.blocks;
  Bump o;
  o.take((size_t)pl.N * 4);
  pl.off_pos = o.take((size_t)pl.N * 4);
  pl.off_start = o.take((((size_t)1 << embed::kBucketBits) + 1) * 4);
  pl.order_bytes = align_up(o.off);
  Bump w;
  if (!pl.scan) {
    pl.off_key2 = w.take((size_t)pl.N * 4);
    pl.off_pos2 = w.take((size_t)pl.N * 4);
    pl.off_hist = w.take((size_t)pl.blocks * ((size_t)4 << pl.bits));
  }
  pl.order_ws = align_up(w.off);
}

// One launch without an order: up to 256 ids (of a sample for the norm, in all for
// the gradient) and, for the norm, samples that one CU reads in a few us
// (B = 3, T = 61, d = 256 fp32: 8 us against 31 with an order).
constexpr int64_t kSmallBytes = 256 * 1024;

void plan_runs(EmbedPlan& pl, dpnorm_dtype dt, int64_t d, bool ordered) {
  pl.d = (int32_t)d;
  pl.small_norm = !ordered && pl.T <= embed::kSmallIds && pl.T * d * (int64_t)esize(dt) <= kSmallBytes;
  pl.small_grad = !ordered && pl.N <= embed::kSmallIds;
  const int64_t width = dt == DPNORM_BF16 ? embed::Row<true>::kSlice : embed::Row<false>::kSlice;
  pl.slices = (int)((d + width - 1) / width);
  pl.R = 16;
  while (pl.R > 4 && (int64_t)pl.N * pl.slices / pl.R < 4096) pl.R >>= 1;
  pl.chunks = (pl.N + pl.R - 1) / pl.R;
  Bump n;
  if (!pl.small_norm) {
    if (!ordered) {
      pl.off_order = n.take(pl.order_bytes);
      pl.off_order_ws = n.take(pl.order_ws);
    }
    pl.off_val = n.take((size_t)pl.slices * (size_t)pl.N * 4);
    pl.off_part = n.take((size_t)pl.chunks * 2 * (size_t)d * 4);
    // blocks of at least 4096 values, where a sample has many
    pl.sum_blocks = (int)std::min<int64_t>(16, std::max<int64_t>(1, (int64_t)pl.T * pl.slices / 4096));
    if (pl.sum_blocks > 1) {
      const size_t samples = (size_t)(pl.N / pl.T);
      pl.off_parts = n.take(samples * pl.sum_blocks * 8);
      pl.off_arrived = n.take(samples * 4);
    }
  }
  pl.norm_ws = align_up(n.off);
  Bump g;
  if (!pl.small_grad) {
    if (!ordered) {   // (where the norm has them)
      pl.off_order = g.take(pl.order_bytes);
      pl.off_order_ws = g.take(pl.order_ws);
    }
    pl.off_part_grad = g.take((size_t)pl.chunks * 2 * (size_t)d * 4);
  }
  pl.grad_ws = align_up(g.off);
}

// A grid of `blocks` blocks (below 2^31), at most 2^20 along x: HIP takes fewer than
// 2^32 threads along a dimension, and 2^16 blocks along y.
dim3 grid_of(int64_t blocks) {
  const int64_t y = (blocks + (1 << 20) - 1) >> 20;
  return dim3((uint32_t)((blocks + y - 1) / y), (uint32_t)y);
}

// Blocks of one launch are numbered in 31 bits.
dpnorm_status check_grid(const EmbedPlan& pl) {
  const int64_t lim = 0x7fffffff;
  if (pl.chunks * pl.slices > lim) return DPNORM_ERR_SIZE;
  if ((pl.chunks * pl.slices + 3) / 4 + (pl.V + embed::kFillRows - 1) / embed::kFillRows > lim) return DPNORM_ERR_SIZE;
  return DPNORM_OK;
}

hipError_t launch_order(const EmbedPlan& pl, const void* tok, dpnorm_index it, void* order, void* ws, hipStream_t stream) {
  const int i64 = it == DPNORM_I64;
  int32_t* keys = (int32_t*)order;
  int32_t* pos = (int32_t*)((char*)order + pl.off_pos);
  if (pl.scan) {
    const uint32_t buckets = 1u << std::min(pl.id_bits, embed::kBucketBits);
    // the factor's inverse modulo 2^32 (each step doubles the bits that are right)
    uint32_t inverse = 1;
    for (int i = 0; i < 5; ++i) inverse *= 2u - embed::mix_factor(pl.id_bits) * inverse;
    embed::k_order_scan<<<buckets, embed::kSortThreads, 0, stream>>>(tok, i64, pl.N, pl.V, pl.id_bits, inverse, keys, pos,
                                                                    (int32_t*)((char*)order + pl.off_start));
    return hipGetLastError();
  }
  int32_t* key2 = (int32_t*)((char*)ws + pl.off_key2);
  int32_t* pos2 = (int32_t*)((char*)ws + pl.off_pos2);
  uint32_t* hist = (uint32_t*)((char*)ws + pl.off_hist);
  const int32_t *sk = nullptr, *sp = nullptr;
  for (int p = 0; p < pl.passes; ++p) {
    // the last pass writes the order; the ones before it alternate
    const bool to_order = (pl.passes - 1 - p) % 2 == 0;
    int32_t *dk = to_order ? keys : key2, *dp = to_order ? pos : pos2;
    embed::k_order_count<<<pl.blocks, embed::kSortThreads, 0, stream>>>(tok, i64, sk, pl.N, pl.V, pl.id_bits, p * pl.bits, pl.bits, pl.per,
                                                                       hist);
    embed::k_order_scatter<<<pl.blocks, embed::kSortThreads, 0, stream>>>(tok, i64, sk, sp, pl.N, pl.V, pl.id_bits, p * pl.bits, pl.bits,
                                                                         pl.per, hist, dk, dp);
    sk = dk;
    sp = dp;
  }
  return hipGetLastError();
}

embed::RunArgs run_args(const EmbedPlan& pl, const void* order, const void* G) {
  embed::RunArgs a{};
  a.runs.keys = (const int32_t*)order;
  a.runs.pos = order ? (const int32_t*)((const char*)order + pl.off_pos) : nullptr;   // (none: a small gradient)
  a.runs.start = order && pl.scan ? (const int32_t*)((const char*)order + pl.off_start) : nullptr;
  a.runs.bits = pl.id_bits;
  a.runs.N = pl.N;
  a.runs.T = pl.T;
  a.runs.V = pl.V;
  a.runs.per = 1.0 / pl.T;
  a.runs.R = pl.R;
  a.runs.chunks = (int32_t)pl.chunks;
  a.G = (const char*)G;
  a.d = pl.d;
  a.slices = pl.slices;
  a.items = pl.chunks * pl.slices;
  return a;
}

template <int MODE>
hipError_t launch_runs(const embed::RunArgs& a, bool bf16, hipStream_t stream) {
  const dim3 blocks = grid_of((a.items + 3) / 4 + a.fill_blocks), joins = grid_of(a.items);
  if (bf16) {
    embed::k_run_sums<true, MODE><<<blocks, 256, 0, stream>>>(a);
    embed::k_run_join<true, MODE><<<joins, 256, 0, stream>>>(a);
  } else {
    embed::k_run_sums<false, MODE><<<blocks, 256, 0, stream>>>(a);
    embed::k_run_join<false, MODE><<<joins, 256, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

extern "C" {

dpnorm_status dpnorm_embed_lookup(const void* tok, dpnorm_index it, const void* W, dpnorm_dtype dt, int64_t N, int64_t V,
                                  int64_t d, float scale, void* out, hipStream_t stream) {
  dpnorm_status st = check_ids(1, N, V);
  if (st == DPNORM_OK) st = check_rows(dt, std::max(N, V), d);
  if (st != DPNORM_OK) return st;
  if (it != DPNORM_I32 && it != DPNORM_I64) return DPNORM_ERR_DTYPE;
  if (!tok || !W || !out) return DPNORM_ERR_NULL;
  const size_t ib = it == DPNORM_I64 ? 8 : 4, e = esize(dt);
  if (!aligned(tok, ib) || !aligned(W, 16) || !aligned(out, 16)) return DPNORM_ERR_ALIGN;
  if (!std::isfinite(scale)) return DPNORM_ERR_VALUE;
  const size_t ob = (size_t)N * d * e;
  if (overlaps(out, ob, tok, (size_t)N * ib) || overlaps(out, ob, W, (size_t)V * d * e)) return DPNORM_ERR_VALUE;
  const bool bf16 = dt == DPNORM_BF16;
  const int64_t width = bf16 ? embed::Row<true>::kSlice : embed::Row<false>::kSlice;
  const int64_t slices = (d + width - 1) / width;
  const int64_t blocks = ((N + embed::kLookupRows - 1) / embed::kLookupRows * slices + 3) / 4;
  if (blocks > 0x7fffffff) return DPNORM_ERR_SIZE;
  if (bf16)
    embed::k_lookup<true><<<grid_of(blocks), 256, 0, stream>>>(tok, it == DPNORM_I64, (const char*)W, (char*)out, N, (int32_t)V,
                                                                (int32_t)d, (int32_t)slices, scale);
  else
    embed::k_lookup<false><<<grid_of(blocks), 256, 0, stream>>>(tok, it == DPNORM_I64, (const char*)W, (char*)out, N, (int32_t)V,
                                                                 (int32_t)d, (int32_t)slices, scale);
  return hip_status(hipGetLastError());
}

dpnorm_status dpnorm_embed_order_sizes(int64_t B, int64_t T, int64_t V, size_t* order_bytes, size_t* ws_bytes) {
  if (!order_bytes || !ws_bytes) return DPNORM_ERR_NULL;
  const dpnorm_status st = check_ids(B, T, V);
  if (st != DPNORM_OK) return st;
  EmbedPlan pl;
  plan_order(pl, B, T, V);
  *order_bytes = pl.order_bytes;
  *ws_bytes = pl.order_ws;
  return DPNORM_OK;
}

dpnorm_status dpnorm_embed_order(const void* tok, dpnorm_index it, int64_t B, int64_t T, int64_t V, void* order,
                                 size_t order_bytes, void* ws, size_t ws_bytes, hipStream_t stream) {
  const dpnorm_status st = check_ids(B, T, V);
  if (st != DPNORM_OK) return st;
  if (it != DPNORM_I32 && it != DPNORM_I64) return DPNORM_ERR_DTYPE;
  EmbedPlan pl;
  plan_order(pl, B, T, V);
  if (!tok || !order || (!ws && pl.order_ws)) return DPNORM_ERR_NULL;
  const size_t ib = it == DPNORM_I64 ? 8 : 4;
  if (!aligned(tok, ib) || !aligned(order, kAlign) || !aligned(ws, kAlign)) return DPNORM_ERR_ALIGN;
  if (order_bytes < pl.order_bytes || ws_bytes < pl.order_ws) return DPNORM_ERR_WORKSPACE;
  if (overlaps(order, pl.order_bytes, tok, (size_t)pl.N * ib) || overlaps(ws, pl.order_ws, tok, (size_t)pl.N * ib) ||
      overlaps(order, pl.order_bytes, ws, pl.order_ws))
    return DPNORM_ERR_VALUE;
  return hip_status(launch_order(pl, tok, it, order, ws, stream));
}

static dpnorm_status plan_embed(dpnorm_dtype dt, int64_t B, int64_t T, int64_t V, int64_t d, bool ordered, EmbedPlan& pl) {
  dpnorm_status st = check_ids(B, T, V);
  if (st == DPNORM_OK) st = check_rows(dt, std::max(B * T, V), d);
  if (st != DPNORM_OK) return st;
  plan_order(pl, B, T, V);
  plan_runs(pl, dt, d, ordered);
  return check_grid(pl);
}

// The checks that both calls share, and that the ids come from one place.
static dpnorm_status check_embed(const EmbedPlan& pl, const void* tok, dpnorm_index it, const void* order, const void* G,
                                 const void* out, const void* ws, size_t need, size_t ws_bytes, float scale, int accumulate) {
  if (!order && it != DPNORM_I32 && it != DPNORM_I64) return DPNORM_ERR_DTYPE;
  if ((!order && !tok) || !G || !out || (!ws && need)) return DPNORM_ERR_NULL;
  if (!aligned(order, kAlign) || (!order && !aligned(tok, it == DPNORM_I64 ? 8 : 4)) || !aligned(G, 16) || !aligned(ws, kAlign))
    return DPNORM_ERR_ALIGN;
  if (!std::isfinite(scale) || (accumulate != 0 && accumulate != 1)) return DPNORM_ERR_VALUE;
  if (ws_bytes < need) return DPNORM_ERR_WORKSPACE;
  return DPNORM_OK;
}

dpnorm_status dpnorm_embed_norm_workspace(dpnorm_dtype dt, int64_t B, int64_t T, int64_t V, int64_t d, int ordered,
                                          size_t* bytes) {
  if (!bytes) return DPNORM_ERR_NULL;
  if (ordered != 0 && ordered != 1) return DPNORM_ERR_VALUE;
  EmbedPlan pl;
  const dpnorm_status st = plan_embed(dt, B, T, V, d, ordered != 0, pl);
  if (st == DPNORM_OK) *bytes = pl.norm_ws;
  return st;
}

dpnorm_status dpnorm_embed_norm(const void* tok, dpnorm_index it, const void* order, const void* G, dpnorm_dtype dt, int64_t B,
                                int64_t T, int64_t V, int64_t d, float scale, float* n, int accumulate, void* ws,
                                size_t ws_bytes, hipStream_t stream) {
  EmbedPlan pl;
  dpnorm_status st = plan_embed(dt, B, T, V, d, order != nullptr, pl);
  if (st == DPNORM_OK) st = check_embed(pl, tok, it, order, G, n, ws, pl.norm_ws, ws_bytes, scale, accumulate);
  if (st != DPNORM_OK) return st;
  if (!aligned(n, 4)) return DPNORM_ERR_ALIGN;
  const size_t nb = (size_t)B * 4, gb = (size_t)pl.N * d * esize(dt);
  const void* ids = order ? order : tok;
  const size_t ib = order ? pl.order_bytes : (size_t)pl.N * (it == DPNORM_I64 ? 8 : 4);
  if (overlaps(n, nb, ids, ib) || overlaps(n, nb, G, gb) || overlaps(n, nb, ws, pl.norm_ws) ||
      overlaps(ws, pl.norm_ws, ids, ib) || overlaps(ws, pl.norm_ws, G, gb))
    return DPNORM_ERR_VALUE;
  const bool bf16 = dt == DPNORM_BF16;
  const double scale2 = (double)scale * (double)scale;
  if (pl.small_norm) {
    if (bf16)
      embed::k_norm_small<true><<<grid_of(B), 1024, 0, stream>>>(tok, it == DPNORM_I64, (const char*)G, (int32_t)B, pl.T, pl.V, pl.d,
                                                                 scale2, n, accumulate);
    else
      embed::k_norm_small<false><<<grid_of(B), 1024, 0, stream>>>(tok, it == DPNORM_I64, (const char*)G, (int32_t)B, pl.T, pl.V, pl.d,
                                                                  scale2, n, accumulate);
    return hip_status(hipGetLastError());
  }
  hipError_t he = hipSuccess;
  char* base = (char*)ws;
  if (!order) {
    he = launch_order(pl, tok, it, base + pl.off_order, base + pl.off_order_ws, stream);
    order = base + pl.off_order;
  }
  embed::RunArgs a = run_args(pl, order, G);
  a.val = (float*)(base + pl.off_val);
  a.part = (float*)(base + pl.off_part);
  double* parts = pl.sum_blocks > 1 ? (double*)(base + pl.off_parts) : nullptr;
  a.arrived = pl.sum_blocks > 1 ? (uint32_t*)(base + pl.off_arrived) : nullptr;
  if (he == hipSuccess) he = launch_runs<embed::RUN_NORM>(a, bf16, stream);
  if (he == hipSuccess) {
    const int64_t y = std::min<int64_t>(B, 65535);
    const dim3 grid((uint32_t)pl.sum_blocks, (uint32_t)y, (uint32_t)((B + y - 1) / y));
    embed::k_norm_sum<<<grid, 1024, 0, stream>>>(a.val, pl.N, pl.T, pl.slices, scale2, n, accumulate, parts, a.arrived);
    he = hipGetLastError();
  }
  return hip_status(he);
}

dpnorm_status dpnorm_embed_grad_workspace(dpnorm_dtype dt, int64_t B, int64_t T, int64_t V, int64_t d, int ordered,
                                          size_t* bytes) {
  if (!bytes) return DPNORM_ERR_NULL;
  if (ordered != 0 && ordered != 1) return DPNORM_ERR_VALUE;
  EmbedPlan pl;
  const dpnorm_status st = plan_embed(dt, B, T, V, d, ordered != 0, pl);
  if (st == DPNORM_OK) *bytes = pl.grad_ws;
  return st;
}

dpnorm_status dpnorm_embed_grad(const void* tok, dpnorm_index it, const void* order, const void* G, dpnorm_dtype dt, int64_t B,
                                int64_t T, int64_t V, int64_t d, float scale, const float* c, void* dW, int accumulate,
                                void* ws, size_t ws_bytes, hipStream_t stream) {
  EmbedPlan pl;
  dpnorm_status st = plan_embed(dt, B, T, V, d, order != nullptr, pl);
  if (st == DPNORM_OK) st = check_embed(pl, tok, it, order, G, dW, ws, pl.grad_ws, ws_bytes, scale, accumulate);
  if (st != DPNORM_OK) return st;
  if (!aligned(c, 4) || !aligned(dW, 16)) return DPNORM_ERR_ALIGN;
  const size_t e = esize(dt), wb = (size_t)V * d * e, gb = (size_t)pl.N * d * e, cb = (size_t)B * 4;
  const void* ids = order ? order : tok;
  const size_t ib = order ? pl.order_bytes : (size_t)pl.N * (it == DPNORM_I64 ? 8 : 4);
  if (overlaps(dW, wb, ids, ib) || overlaps(dW, wb, G, gb) || overlaps(dW, wb, c, cb) || overlaps(dW, wb, ws, pl.grad_ws) ||
      overlaps(ws, pl.grad_ws, ids, ib) || overlaps(ws, pl.grad_ws, G, gb) || overlaps(ws, pl.grad_ws, c, cb))
    return DPNORM_ERR_VALUE;
  const bool bf16 = dt == DPNORM_BF16;
  hipError_t he = hipSuccess;
  char* base = (char*)ws;
  if (!order && !pl.small_grad) {
    he = launch_order(pl, tok, it, base + pl.off_order, base + pl.off_order_ws, stream);
    order = base + pl.off_order;
  }
  embed::RunArgs a = run_args(pl, order, G);
  a.c = c;
  a.scale = scale;
  a.out = (char*)dW;
  a.accumulate = accumulate;
  if (pl.small_grad) {
    const dim3 blocks = grid_of((pl.V + embed::kSmallRows - 1) / embed::kSmallRows);
    if (bf16) embed::k_grad_small<true><<<blocks, 256, 0, stream>>>(tok, it == DPNORM_I64, a);
    else embed::k_grad_small<false><<<blocks, 256, 0, stream>>>(tok, it == DPNORM_I64, a);
    return hip_status(hipGetLastError());
  }
  a.part = (float*)(base + pl.off_part_grad);
  a.fill_blocks = accumulate ? 0 : (pl.V + embed::kFillRows - 1) / embed::kFillRows;
  if (he == hipSuccess) he = launch_runs<embed::RUN_GRAD>(a, bf16, stream);
  return hip_status(he);
}

}  // extern "C"
