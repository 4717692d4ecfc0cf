// Host layer of the layer-norm and RMS-norm calls: argument checks, workspace
// layout, launches. Included by dpnorm.cpp, whose helpers it uses.
#pragma once
#include "layernorm_kernels.h"

namespace {

constexpr int64_t kLnWidest = 32768, kLnRows = (int64_t)1 << 30;

dpnorm_status check_ln(dpnorm_dtype dt, dpnorm_ln_kind kind, int64_t B, int64_t T, int64_t d) {
  if (dt != DPNORM_BF16 && dt != DPNORM_F32) return DPNORM_ERR_DTYPE;
  if (kind != DPNORM_LN_LAYER && kind != DPNORM_LN_RMS) return DPNORM_ERR_DTYPE;
  const int64_t g = dt == DPNORM_BF16 ? 8 : 4;
  if (B < 1 || T < 1 || T > kLnRows || B > kLnRows / T || d < 1 || d % g != 0 || d > kLnWidest) return DPNORM_ERR_SIZE;
  return DPNORM_OK;
}

// Waves of a row, chunks a lane and rows at a time for d columns: a wave a row for up
// to 256 chunks, four for up to 1024, sixteen for more. f gets them as constants.
template <bool BF16, typename F>
hipError_t with_row(int64_t d, F f) {
  const auto is = [](auto v) { return v; };
  using std::integral_constant;
  const int64_t chunks = d / ln::Chunk<BF16>::kN;
  const auto go = [&](auto nc, auto w, auto r) { return f(is(nc), is(w), is(r)); };
  if (chunks <= 64) return go(integral_constant<int, 1>{}, integral_constant<int, 1>{}, integral_constant<int, 4>{});
  if (chunks <= 128) return go(integral_constant<int, 2>{}, integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (chunks <= 256) return go(integral_constant<int, 4>{}, integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (chunks <= 512) return go(integral_constant<int, 2>{}, integral_constant<int, 4>{}, integral_constant<int, BF16 ? 2 : 1>{});
  if (chunks <= 1024) return go(integral_constant<int, 4>{}, integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (chunks <= 2048) return go(integral_constant<int, 2>{}, integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if constexpr (BF16) {
    return go(integral_constant<int, 4>{}, integral_constant<int, 16>{}, integral_constant<int, 1>{});
  } else {
    if (chunks <= 4096) return go(integral_constant<int, 4>{}, integral_constant<int, 16>{}, integral_constant<int, 1>{});
    return go(integral_constant<int, 8>{}, integral_constant<int, 16>{}, integral_constant<int, 1>{});
  }
}

// The same with the type and kind: f(bf16, rms, nc, w, r).
template <typename F>
hipError_t with_ln(dpnorm_dtype dt, dpnorm_ln_kind kind, int64_t d, F f) {
  const auto kinds = [&](auto bf16) {
    return with_row<decltype(bf16)::value>(d, [&](auto nc, auto w, auto r) {
      return kind == DPNORM_LN_RMS ? f(bf16, std::true_type{}, nc, w, r) : f(bf16, std::false_type{}, nc, w, r);
    });
  };
  return dt == DPNORM_BF16 ? kinds(std::true_type{}) : kinds(std::false_type{});
}

// Work groups of the summing kernels that share `rows` rows (among `others` such sets of
// rows). One a CU, since each leaves 2 d sums for the second launch (4 x 4096 rows of 2048
// bf16: gradients 46 us with 256, 50 with 512); rows of four waves and two chunks, whose
// registers leave room, two a CU for the gradients (2 x 4096 rows of 4096 bf16: 46 us with
// 512, 51 with 256; norms 37 with 256, 41 with 512) and for fp32. Two rounds of rows each
// at least (four of rows of sixteen waves: 1024 rows of 16384 49 us, 73 with two). One work
// group, and one launch, for up to six rounds (gradients of 183 rows of 256 fp32, six
// rounds: 14 us, and 19 in two launches; 64 rows of 2048 bf16, eight: 22 and 19).
int64_t ln_blocks(dpnorm_dtype dt, int64_t d, int64_t rows, int64_t others, bool gradients) {
  const bool bf16 = dt == DPNORM_BF16;
  const int64_t chunks = d / (bf16 ? 8 : 4);
  const int64_t round = chunks <= 64 ? 32 : chunks <= 128 ? 16 : chunks <= 256 ? 8 : chunks <= 512 ? (bf16 ? 4 : 1) : chunks <= 1024 ? 2 : 1;
  if (rows <= 6 * round) return 1;
  const int64_t places = chunks > 256 && chunks <= 512 && (gradients || !bf16) ? 512 : 256;
  return std::max<int64_t>(1, std::min(places / others, rows / std::max<int64_t>(2 * round, 4)));
}

// Threads that share `rows` partial sums of a column (see add_rows): about four each.
int32_t ln_slots(int64_t rows) {
  int32_t s = 1;
  while (s < 64 && 4 * s < rows) s *= 2;
  return s;
}

ln::Args ln_args(int64_t B, int64_t T, int64_t d) {
  ln::Args a{};
  a.N = (int32_t)(B * T);
  a.T = (int32_t)T;
  a.d = (int32_t)d;
  a.inv = (float)(1.0 / (double)d);
  return a;
}

struct LnNormPlan {
  int64_t shares = 1, groups = 1;      // work groups of a sample in the two launches
  size_t off_arrived = 0, off_parts = 0, bytes = 0;
};
LnNormPlan plan_ln_norm(dpnorm_dtype dt, int64_t B, int64_t T, int64_t d, int32_t columns) {
  LnNormPlan p;
  p.shares = ln_blocks(dt, d, T, B, false);
  if (p.shares < 2) return p;
  const int64_t at_once = 4096 / ln_slots(p.shares);
  p.groups = (columns + at_once - 1) / at_once;
  Bump w;
  w.take((size_t)(B * p.shares) * 2 * d * 4);
  p.off_arrived = w.take((size_t)B * 4);
  p.off_parts = w.take((size_t)(B * p.groups) * 8);
  p.bytes = align_up(w.off);
  return p;
}

}  // namespace

extern "C" {

dpnorm_status dpnorm_layernorm_forward(const void* x, const void* w, const void* b, dpnorm_dtype dt, dpnorm_ln_kind kind,
                                       int64_t N, int64_t d, float eps, void* y, float* mean, float* rstd, hipStream_t stream) {
  const dpnorm_status st = check_ln(dt, kind, N, 1, d);
  if (st != DPNORM_OK) return st;
  if (!x || !w || !y) return DPNORM_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(b, 16) || !aligned(y, 16) || !aligned(mean, 4) || !aligned(rstd, 4))
    return DPNORM_ERR_ALIGN;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return DPNORM_ERR_VALUE;
  if (kind == DPNORM_LN_RMS && (b || mean)) return DPNORM_ERR_VALUE;
  const size_t e = esize(dt), xb = (size_t)N * d * e, wb = (size_t)d * e, sb = (size_t)N * 4;
  if (outputs_overlap({{x, xb}, {w, wb}, {b, wb}}, {{y, xb}, {mean, sb}, {rstd, sb}})) return DPNORM_ERR_VALUE;
  ln::Args a = ln_args(1, N, d);
  a.x = (const char*)x;
  a.w = (const char*)w;
  a.b = (const char*)b;
  a.y = (char*)y;
  a.mean = mean;
  a.rstd = rstd;
  a.eps = eps;
  return hip_status(with_ln(dt, kind, d, [&](auto bf16, auto rms, auto nc, auto wv, auto r) {
    constexpr int W = decltype(wv)::value, R = decltype(r)::value;
    const int64_t rows = (W == 1 ? 4 : 1) * R, places = W == 1 ? 2048 : W == 4 ? 2048 : 512;
    const uint32_t blocks = (uint32_t)std::min<int64_t>(places, (N + rows - 1) / rows);
    ln::k_forward<decltype(bf16)::value, decltype(rms)::value, decltype(nc)::value, W, R>
        <<<blocks, ln::kForwardThreads<W>, 0, stream>>>(a);
    return hipGetLastError();
  }));
}

dpnorm_status dpnorm_layernorm_backward_workspace(dpnorm_dtype dt, dpnorm_ln_kind kind, int64_t B, int64_t T, int64_t d,
                                                  size_t* bytes) {
  if (!bytes) return DPNORM_ERR_NULL;
  const dpnorm_status st = check_ln(dt, kind, B, T, d);
  if (st != DPNORM_OK) return st;
  const int64_t blocks = ln_blocks(dt, d, B * T, 1, true);
  *bytes = blocks > 1 ? align_up((size_t)blocks * 2 * d * 4) : 0;
  return DPNORM_OK;
}

dpnorm_status dpnorm_layernorm_backward(const void* dy, const void* x, const void* w, const float* mean, const float* rstd,
                                        dpnorm_dtype dt, dpnorm_ln_kind kind, int64_t B, int64_t T, int64_t d, const float* c,
                                        void* dx, void* dw, void* db, void* ws, size_t ws_bytes, hipStream_t stream) {
  size_t need = 0;
  const dpnorm_status st = dpnorm_layernorm_backward_workspace(dt, kind, B, T, d, &need);
  if (st != DPNORM_OK) return st;
  const bool layer = kind == DPNORM_LN_LAYER;
  if (!dw && !db) need = 0;
  if (!dy || !x || !w || !rstd || (layer && !mean) || (!dx && !dw && !db) || (need && !ws)) return DPNORM_ERR_NULL;
  for (const void* p : {dy, x, w, (const void*)dx, (const void*)dw, (const void*)db})
    if (!aligned(p, 16)) return DPNORM_ERR_ALIGN;
  if (!aligned(mean, 4) || !aligned(rstd, 4) || !aligned(c, 4) || (need && !aligned(ws, kAlign))) return DPNORM_ERR_ALIGN;
  if (!layer && (mean || db)) return DPNORM_ERR_VALUE;
  if (ws_bytes < need) return DPNORM_ERR_WORKSPACE;
  const size_t e = esize(dt), xb = (size_t)(B * T) * d * e, wb = (size_t)d * e, sb = (size_t)(B * T) * 4;
  if (outputs_overlap({{dy, xb}, {x, xb}, {w, wb}, {mean, sb}, {rstd, sb}, {c, (size_t)B * 4}},
                      {{dx, xb}, {dw, wb}, {db, wb}, {ws, need}}))
    return DPNORM_ERR_VALUE;
  ln::Args a = ln_args(B, T, d);
  a.dy = (const char*)dy;
  a.x = (const char*)x;
  a.w = (const char*)w;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.c = c;
  a.dx = (char*)dx;
  a.dw = (char*)dw;
  a.db = (char*)db;
  a.blocks = (int32_t)ln_blocks(dt, d, B * T, 1, true);
  a.part = a.blocks > 1 ? (float*)ws : nullptr;
  hipError_t he = with_ln(dt, kind, d, [&](auto bf16, auto rms, auto nc, auto wv, auto r) {
    constexpr bool BF16 = decltype(bf16)::value;
    constexpr int NC = decltype(nc)::value, W = decltype(wv)::value;
    ln::k_backward<BF16, decltype(rms)::value, NC, W, decltype(r)::value>
        <<<(uint32_t)a.blocks, 64 * ln::kSumWaves<BF16, NC, W>, 0, stream>>>(a);
    return hipGetLastError();
  });
  if (he == hipSuccess && a.part && (dw || db)) {
    const int32_t slots = ln_slots(a.blocks), at_once = 4096 / slots;
    const dim3 grid((uint32_t)((d + at_once - 1) / at_once), layer ? 2 : 1);
    if (dt == DPNORM_BF16) ln::k_backward_columns<true><<<grid, 1024, 0, stream>>>(a, slots);
    else ln::k_backward_columns<false><<<grid, 1024, 0, stream>>>(a, slots);
    he = hipGetLastError();
  }
  return hip_status(he);
}

dpnorm_status dpnorm_layernorm_norm_workspace(dpnorm_dtype dt, dpnorm_ln_kind kind, int64_t B, int64_t T, int64_t d, size_t* bytes) {
  if (!bytes) return DPNORM_ERR_NULL;
  const dpnorm_status st = check_ln(dt, kind, B, T, d);
  if (st != DPNORM_OK) return st;
  *bytes = plan_ln_norm(dt, B, T, d, (int32_t)(2 * d)).bytes;
  return DPNORM_OK;
}

dpnorm_status dpnorm_layernorm_norm(const void* x, const void* G, dpnorm_dtype dt, dpnorm_ln_kind kind, int64_t B, int64_t T,
                                    int64_t d, float eps, int parts, float* n, int accumulate, void* ws, size_t ws_bytes,
                                    hipStream_t stream) {
  const dpnorm_status st = check_ln(dt, kind, B, T, d);
  if (st != DPNORM_OK) return st;
  if (parts < 1 || parts > 3 || (kind == DPNORM_LN_RMS && parts != DPNORM_LN_GAIN)) return DPNORM_ERR_VALUE;
  const LnNormPlan p = plan_ln_norm(dt, B, T, d, (int32_t)(parts == 3 ? 2 * d : d));
  if (!x || !G || !n || (p.bytes && !ws)) return DPNORM_ERR_NULL;
  if (!aligned(x, 16) || !aligned(G, 16) || !aligned(n, 4) || (p.bytes && !aligned(ws, kAlign))) return DPNORM_ERR_ALIGN;
  if (!(eps >= 0.f) || !std::isfinite(eps) || (accumulate != 0 && accumulate != 1)) return DPNORM_ERR_VALUE;
  if (ws_bytes < p.bytes) return DPNORM_ERR_WORKSPACE;
  const size_t xb = (size_t)(B * T) * d * esize(dt);
  if (outputs_overlap({{x, xb}, {G, xb}}, {{n, (size_t)B * 4}, {ws, p.bytes}})) return DPNORM_ERR_VALUE;
  ln::Args a = ln_args(B, T, d);
  a.x = (const char*)x;
  a.dy = (const char*)G;
  a.eps = eps;
  a.n = n;
  a.accumulate = accumulate;
  a.blocks = (int32_t)p.shares;
  a.first = parts & DPNORM_LN_GAIN ? 0 : (int32_t)d;
  a.columns = (int32_t)(parts == 3 ? 2 * d : d);
  a.part = (float*)ws;
  a.arrived = (uint32_t*)((char*)ws + p.off_arrived);
  a.parts = (double*)((char*)ws + p.off_parts);
  hipError_t he = with_ln(dt, kind, d, [&](auto bf16, auto rms, auto nc, auto wv, auto r) {
    constexpr bool BF16 = decltype(bf16)::value;
    constexpr int NC = decltype(nc)::value, W = decltype(wv)::value;
    ln::k_norm<BF16, decltype(rms)::value, NC, W, decltype(r)::value>
        <<<grid_of(B * p.shares), 64 * ln::kSumWaves<BF16, NC, W>, 0, stream>>>(a);
    return hipGetLastError();
  });
  if (he == hipSuccess && p.shares > 1) {
    ln::k_norm_columns<><<<grid_of(B * p.groups), 1024, 0, stream>>>(a, B, (int32_t)p.groups, ln_slots(p.shares));
    he = hipGetLastError();
  }
  return hip_status(he);
}

}  // extern "C"
