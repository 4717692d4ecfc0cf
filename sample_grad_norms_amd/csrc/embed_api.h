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
  int passes = 0, bits = 0, blocks = 0, per = 0;
  size_t off_pos = 0, order_bytes = 0, off_key2 = 0, off_pos2 = 0, off_hist = 0, order_ws = 0;
  // run sums
  size_t off_val = 0, off_part = 0, norm_ws = 0, off_part_grad = 0, grad_ws = 0;
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
  int bits = 1;
  while (((int64_t)1 << bits) <= V) ++bits;   // keys 0 .. V
  pl.passes = (bits + 8) / 9;
  pl.bits = (bits + pl.passes - 1) / pl.passes;
  // a block for every 1024 positions, up to the 64 whose counts one thread adds up
  pl.blocks = (int)std::min<int64_t>(embed::kMaxSortBlocks, (pl.N + 1023) / 1024);
  pl.per = (pl.N + pl.blocks - 1) / pl.blocks;
  Bump o;
  o.take((size_t)pl.N * 4);
  pl.off_pos = o.take((size_t)pl.N * 4);
  pl.order_bytes = align_up(o.off);
  Bump w;
  if (pl.N > embed::kSmallSort) {
    pl.off_key2 = w.take((size_t)pl.N * 4);
    pl.off_pos2 = w.take((size_t)pl.N * 4);
    pl.off_hist = w.take((size_t)pl.blocks * ((size_t)4 << pl.bits));
  }
  pl.order_ws = align_up(w.off);
}

void plan_runs(EmbedPlan& pl, dpnorm_dtype dt, int64_t d) {
  pl.d = (int32_t)d;
  const int64_t width = dt == DPNORM_BF16 ? embed::Row<true>::kSlice : embed::Row<false>::kSlice;
  pl.slices = (int)((d + width - 1) / width);
  pl.R = 32;
  while (pl.R > 4 && (int64_t)pl.N * pl.slices / pl.R < 4096) pl.R >>= 1;
  pl.chunks = (pl.N + pl.R - 1) / pl.R;
  Bump n;
  pl.off_val = n.take((size_t)pl.slices * (size_t)pl.N * 4);
  pl.off_part = n.take((size_t)pl.chunks * 2 * (size_t)d * 4);
  pl.norm_ws = align_up(n.off);
  Bump g;
  pl.off_part_grad = g.take((size_t)pl.chunks * 2 * (size_t)d * 4);
  pl.grad_ws = align_up(g.off);
}

// Blocks of one launch fit the 2^31 - 1 of a grid's x dimension.
dpnorm_status check_grid(const EmbedPlan& pl) {
  const int64_t lim = 0x7fffffff;
  if (pl.chunks * pl.slices > lim) return DPNORM_ERR_SIZE;
  if ((pl.chunks * pl.slices + 3) / 4 + (pl.V + embed::kFillRows - 1) / embed::kFillRows > lim) return DPNORM_ERR_SIZE;
  return DPNORM_OK;
}

embed::RunArgs run_args(const EmbedPlan& pl, const void* order, const void* G) {
  embed::RunArgs a{};
  a.runs.keys = (const int32_t*)order;
  a.runs.pos = (const int32_t*)((const char*)order + pl.off_pos);
  a.runs.N = pl.N;
  a.runs.T = pl.T;
  a.runs.V = pl.V;
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
  const uint32_t blocks = (uint32_t)((a.items + 3) / 4 + a.fill_blocks);
  const uint32_t joins = (uint32_t)((int64_t)a.runs.chunks * a.slices);
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
    embed::k_lookup<true><<<(uint32_t)blocks, 256, 0, stream>>>(tok, it == DPNORM_I64, (const char*)W, (char*)out, N, (int32_t)V,
                                                                (int32_t)d, (int32_t)slices, scale);
  else
    embed::k_lookup<false><<<(uint32_t)blocks, 256, 0, stream>>>(tok, it == DPNORM_I64, (const char*)W, (char*)out, N, (int32_t)V,
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
  const int i64 = it == DPNORM_I64;
  int32_t* keys = (int32_t*)order;
  int32_t* pos = (int32_t*)((char*)order + pl.off_pos);
  if (pl.N <= embed::kSmallSort) {
    embed::k_order_small<<<1, embed::kSortThreads, 0, stream>>>(tok, i64, pl.N, pl.V, pl.passes, pl.bits, keys, pos);
    return hip_status(hipGetLastError());
  }
  int32_t* key2 = (int32_t*)((char*)ws + pl.off_key2);
  int32_t* pos2 = (int32_t*)((char*)ws + pl.off_pos2);
  uint32_t* hist = (uint32_t*)((char*)ws + pl.off_hist);
  const int32_t *sk = nullptr, *sp = nullptr;
  for (int p = 0; p < pl.passes; ++p) {
    // the last pass writes the order; the ones before it alternate
    const bool to_order = (pl.passes - 1 - p) % 2 == 0;
    int32_t *dk = to_order ? keys : key2, *dp = to_order ? pos : pos2;
    embed::k_order_count<<<pl.blocks, embed::kSortThreads, 0, stream>>>(tok, i64, sk, pl.N, pl.V, p * pl.bits, pl.bits, pl.per,
                                                                       hist);
    embed::k_order_scatter<<<pl.blocks, embed::kSortThreads, 0, stream>>>(tok, i64, sk, sp, pl.N, pl.V, p * pl.bits, pl.bits,
                                                                         pl.per, hist, dk, dp);
    sk = dk;
    sp = dp;
  }
  return hip_status(hipGetLastError());
}

dpnorm_status dpnorm_embed_norm_workspace(dpnorm_dtype dt, int64_t B, int64_t T, int64_t V, int64_t d, size_t* bytes) {
  if (!bytes) return DPNORM_ERR_NULL;
  dpnorm_status st = check_ids(B, T, V);
  if (st == DPNORM_OK) st = check_rows(dt, std::max(B * T, V), d);
  if (st != DPNORM_OK) return st;
  EmbedPlan pl;
  plan_order(pl, B, T, V);
  plan_runs(pl, dt, d);
  st = check_grid(pl);
  if (st != DPNORM_OK) return st;
  *bytes = pl.norm_ws;
  return DPNORM_OK;
}

dpnorm_status dpnorm_embed_norm(const void* order, const void* G, dpnorm_dtype dt, int64_t B, int64_t T, int64_t V, int64_t d,
                                float scale, float* n, int accumulate, void* ws, size_t ws_bytes, hipStream_t stream) {
  size_t bytes = 0;
  const dpnorm_status st = dpnorm_embed_norm_workspace(dt, B, T, V, d, &bytes);
  if (st != DPNORM_OK) return st;
  if (!order || !G || !n || !ws) return DPNORM_ERR_NULL;
  if (!aligned(order, kAlign) || !aligned(G, 16) || !aligned(n, 4) || !aligned(ws, kAlign)) return DPNORM_ERR_ALIGN;
  if (!std::isfinite(scale) || (accumulate != 0 && accumulate != 1)) return DPNORM_ERR_VALUE;
  if (ws_bytes < bytes) return DPNORM_ERR_WORKSPACE;
  EmbedPlan pl;
  plan_order(pl, B, T, V);
  plan_runs(pl, dt, d);
  const size_t nb = (size_t)B * 4, gb = (size_t)pl.N * d * esize(dt);
  if (overlaps(n, nb, order, pl.order_bytes) || overlaps(n, nb, G, gb) || overlaps(n, nb, ws, bytes) ||
      overlaps(ws, bytes, order, pl.order_bytes) || overlaps(ws, bytes, G, gb))
    return DPNORM_ERR_VALUE;
  embed::RunArgs a = run_args(pl, order, G);
  a.val = (float*)((char*)ws + pl.off_val);
  a.part = (float*)((char*)ws + pl.off_part);
  hipError_t he = launch_runs<embed::RUN_NORM>(a, dt == DPNORM_BF16, stream);
  if (he == hipSuccess) {
    embed::k_norm_sum<<<(uint32_t)B, 1024, 0, stream>>>(a.val, pl.N, pl.T, pl.slices, (double)scale * (double)scale, n, accumulate);
    he = hipGetLastError();
  }
  return hip_status(he);
}

dpnorm_status dpnorm_embed_grad_workspace(dpnorm_dtype dt, int64_t B, int64_t T, int64_t V, int64_t d, size_t* bytes) {
  if (!bytes) return DPNORM_ERR_NULL;
  dpnorm_status st = check_ids(B, T, V);
  if (st == DPNORM_OK) st = check_rows(dt, std::max(B * T, V), d);
  if (st != DPNORM_OK) return st;
  EmbedPlan pl;
  plan_order(pl, B, T, V);
  plan_runs(pl, dt, d);
  st = check_grid(pl);
  if (st != DPNORM_OK) return st;
  *bytes = pl.grad_ws;
  return DPNORM_OK;
}

dpnorm_status dpnorm_embed_grad(const void* order, const void* G, dpnorm_dtype dt, int64_t B, int64_t T, int64_t V, int64_t d,
                                float scale, const float* c, void* dW, int accumulate, void* ws, size_t ws_bytes,
                                hipStream_t stream) {
  size_t bytes = 0;
  const dpnorm_status st = dpnorm_embed_grad_workspace(dt, B, T, V, d, &bytes);
  if (st != DPNORM_OK) return st;
  if (!order || !G || !dW || !ws) return DPNORM_ERR_NULL;
  if (!aligned(order, kAlign) || !aligned(G, 16) || !aligned(c, 4) || !aligned(dW, 16) || !aligned(ws, kAlign))
    return DPNORM_ERR_ALIGN;
  if (!std::isfinite(scale) || (accumulate != 0 && accumulate != 1)) return DPNORM_ERR_VALUE;
  if (ws_bytes < bytes) return DPNORM_ERR_WORKSPACE;
  EmbedPlan pl;
  plan_order(pl, B, T, V);
  plan_runs(pl, dt, d);
  const size_t e = esize(dt), wb = (size_t)V * d * e, gb = (size_t)pl.N * d * e;
  if (overlaps(dW, wb, order, pl.order_bytes) || overlaps(dW, wb, G, gb) || overlaps(dW, wb, ws, bytes) ||
      (c && (overlaps(dW, wb, c, (size_t)B * 4) || overlaps(ws, bytes, c, (size_t)B * 4))) ||
      overlaps(ws, bytes, order, pl.order_bytes) || overlaps(ws, bytes, G, gb))
    return DPNORM_ERR_VALUE;
  embed::RunArgs a = run_args(pl, order, G);
  a.c = c;
  a.scale = scale;
  a.out = (char*)dW;
  a.accumulate = accumulate;
  a.part = (float*)((char*)ws + pl.off_part_grad);
  a.fill_blocks = accumulate ? 0 : (pl.V + embed::kFillRows - 1) / embed::kFillRows;
  return hip_status(launch_runs<embed::RUN_GRAD>(a, dt == DPNORM_BF16, stream));
}

}  // extern "C"
