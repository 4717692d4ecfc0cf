// Host layer of the attention calls: argument checks and launches. Included by
// dpnorm.cpp, whose helpers it uses.
#pragma once
#include "attention_kernels.h"

namespace {

struct AttnCheck {
  attn::Args a{};
  bool bf16 = true;
};

// The strides that are ever multiplied: 0 for a lone row or head, whatever the caller gives.
dpnorm_attn_tensor used_strides(const dpnorm_attn_tensor& t, int64_t N, int64_t H) {
  return {t.data, N > 1 ? t.stride_token : 0, H > 1 ? t.stride_head : 0};
}

// Bytes that a [N][H][D] tensor with the given element strides spans.
size_t span(const dpnorm_attn_tensor& x, int64_t N, int64_t H, int64_t D, size_t e) {
  const dpnorm_attn_tensor t = used_strides(x, N, H);
  return (size_t)((N - 1) * t.stride_token + (H - 1) * t.stride_head + D) * e;
}

// Whether the rows of an output are all apart (no element written twice).
bool rows_apart(const dpnorm_attn_tensor& t, int64_t N, int64_t H, int64_t D) {
  if (t.stride_token >= t.stride_head)
    return (H == 1 || t.stride_head >= D) && (N == 1 || t.stride_token >= (H - 1) * t.stride_head + D);
  return (N == 1 || t.stride_token >= D) && (H == 1 || t.stride_head >= (N - 1) * t.stride_token + D);
}

dpnorm_status check_shape(const dpnorm_attn_shape* s) {
  if (!s) return DPNORM_ERR_NULL;
  if (s->dtype != DPNORM_BF16 && s->dtype != DPNORM_F32) return DPNORM_ERR_DTYPE;
  const int64_t lim = (int64_t)1 << 30;
  if (s->N < 1 || s->N > lim || s->S < 1 || s->S > lim || s->Hq < 1 || s->Hkv < 1 || s->Hq > 65535 || s->Hq % s->Hkv != 0)
    return DPNORM_ERR_SIZE;
  const int64_t g = s->dtype == DPNORM_BF16 ? 8 : 4;
  if (s->D < 1 || s->D > 128 || s->D % g != 0) return DPNORM_ERR_SIZE;
  if (!s->cu_seqlens && s->N % s->S != 0) return DPNORM_ERR_SIZE;
  if (!aligned(s->cu_seqlens, 4)) return DPNORM_ERR_ALIGN;
  if (s->clear_rest != 0 && s->clear_rest != 1) return DPNORM_ERR_VALUE;
  if (!(s->scale > 0.f) || !std::isfinite(s->scale)) return DPNORM_ERR_VALUE;
  return DPNORM_OK;
}

dpnorm_status check_tensor(const dpnorm_attn_tensor* x, const dpnorm_attn_shape* s, int64_t H, bool output) {
  if (!x || !x->data) return DPNORM_ERR_NULL;
  if (!aligned(x->data, 16)) return DPNORM_ERR_ALIGN;
  const dpnorm_attn_tensor t = used_strides(*x, s->N, H);
  const int64_t g = s->dtype == DPNORM_BF16 ? 8 : 4;
  // the 64 rows of a step are addressed with 31-bit byte offsets
  const int64_t lim = (int64_t)1 << 22;
  if (t.stride_token < 0 || t.stride_head < 0 || t.stride_token >= lim || t.stride_head > ((int64_t)1 << 40) / H)
    return DPNORM_ERR_SIZE;
  if (t.stride_token % g != 0 || t.stride_head % g != 0) return DPNORM_ERR_ALIGN;
  if (output && !rows_apart(t, s->N, H, s->D)) return DPNORM_ERR_VALUE;
  return DPNORM_OK;
}

attn::Tensor tensor_of(const dpnorm_attn_tensor* x, int64_t N, int64_t H, size_t e) {
  const dpnorm_attn_tensor t = used_strides(*x, N, H);
  return attn::Tensor{(char*)t.data, t.stride_token * (int64_t)e, t.stride_head * (int64_t)e};
}

attn::Args attn_args(const dpnorm_attn_shape* s) {
  attn::Args a{};
  a.cu = s->cu_seqlens;
  a.S = (int32_t)s->S;
  a.N = (int32_t)s->N;
  a.T = (int32_t)(s->N / s->S);
  a.Hq = (int32_t)s->Hq;
  a.Hkv = (int32_t)s->Hkv;
  a.D = (int32_t)s->D;
  a.scale = s->scale;
  a.clear = s->cu_seqlens && s->clear_rest;
  return a;
}

// Every output apart from every input and from the other outputs.
struct Region {
  const void* p;
  size_t bytes;
};
bool outputs_overlap(const std::vector<Region>& in, const std::vector<Region>& out) {
  for (size_t j = 0; j < out.size(); ++j) {
    for (const Region& r : in)
      if (overlaps(out[j].p, out[j].bytes, r.p, r.bytes)) return true;
    for (size_t i = 0; i < j; ++i)
      if (overlaps(out[j].p, out[j].bytes, out[i].p, out[i].bytes)) return true;
  }
  return false;
}

// Slots of tiles of `rows` rows: sequences of any lengths have at most
// N / rows + S of them.
int64_t slots_of(const attn::Args& a, int rows) {
  return a.cu ? (int64_t)a.N / rows + a.S : (int64_t)a.S * ((a.T + rows - 1) / rows);
}

// Tiles or rows (see attention_kernels.h) for the forward pass and dq, by the
// work groups that rows give. Rows have the shorter chains and win while the
// work groups are few (us, rows against tiles: forward T = 1024, 16/4 heads,
// D = 64 11.6 against 18.7; T = 2048, 16 heads 26 against 33; T = 2048, 32 heads
// 48 against 37); float32 rows of up to 64 columns, where two of their work groups
// fit a CU, always (B = 2, T = 2048, 16/4 heads 190 against 275; 128 columns 410
// against 366).
constexpr int64_t kRowsMost = 1536;
template <bool BF16, int DC>
constexpr bool kRowsAlways = !BF16 && DC == 64;

// Never more work groups than leave the waves of the longest possible sequence kSteps steps.
int64_t most_splits(int64_t splits, int64_t steps) {
  return std::max<int64_t>(1, std::min(splits, (steps + 4 * attn::kSteps - 1) / (4 * attn::kSteps)));
}

// Groups of 32 keys of one key head, at most, and the steps of 32 queries of the first
// of a sequence of average length (the same with and without offsets).
int64_t key_groups(const attn::Args& a) { return ((int64_t)a.N / 32 + a.S) * a.Hkv; }
int64_t key_steps(const attn::Args& a) { return (int64_t)a.N / a.S / 32 * (a.Hq / a.Hkv); }

// dk and dv of bf16 rows of up to 64 columns: eight waves a work group instead of four
// while work groups that share keys would be too many and those of their own too few
// (below), if the chains are long. us, eight waves against four: B = 2, T = 2048, 32/4
// heads 125 against 168, 8/4 heads 38 against 44; 8 x 500 rows, 8/4 heads 28 against 19.
// Wider rows leave eight waves one work group a CU.
constexpr int64_t kKeysMost = 600;
bool keys_eight(const attn::Args& a) { return key_groups(a) <= kKeysMost && key_steps(a) >= 128; }

// dk and dv: the work groups that share the queries of 32 keys of one key head, at
// most (short ends take fewer, see k_backward_kv): about 1.5 for each place on the CUs,
// and three where places and keys are nearly as many but the chains are long. Odd, so
// that those without work do not fall to the same XCDs. us, shared against one work
// group: T = 2048, 32/4 heads D = 128 126 (3) against 283, 3/1 heads D = 64 of 811 + 443
// rows 14 (19) against 26; float32 T = 2048, 16/4 heads D = 64 171 (3) against 293, 8/2
// heads D = 128 of 1500 + 777 rows 176 (3) against 440; B = 2, T = 2048, 32/4 heads
// D = 128 232 (3) against 359, but 10/5 heads D = 64 57 (2) against 47; T = 1024, 16/4
// heads D = 64 22 (5), 30 (8).
template <bool BF16, int DC>
int32_t key_splits(const attn::Args& a) {
  const int64_t places = 256 * (attn::OwnRows<BF16, DC, 4, 256>::kLds <= 80 * 1024 ? 2 : 1);
  const int64_t groups = key_groups(a);
  const int64_t splits = most_splits(3 * places / (4 * groups) * 2 + 1, ((int64_t)a.N + 31) / 32 * (a.Hq / a.Hkv));
  if (splits > 1) return (int32_t)splits;
  // With a prefix every key in it has the whole sequence's queries, and those chains last
  // longest: three work groups share them where there are up to two for each place and the
  // chains are long by a sequence's average length (us of both launches at prefixes of 40 %,
  // three against one: 4 x 2048, 16/4 heads D = 64 239 against 280, D = 128 465 against 534;
  // 1501 + 900 + 33 + 1200 rows 174 against 223; 2 x (1300 + 700) 180 against 219; 4 x 900, of
  // 112 steps, 148 against 165; 8 x 1024 316 against 317; but 5 x 800, of 100 steps, 142
  // against 120, 4 x 800 124 against 116, and twice as many keys 917 against 904). The host
  // does not see how many rows a prefix has: of 90 % three win the same (5 x 900 255 against
  // 299), of 5 % they win or lose little where lengths differ (1501 + .. 167 against 185) and
  // lose where they do not (5 x 900 172 against 156, 8 x 480 174 against 162). Two where
  // chains are of 512 steps and more (two against three: 2 x 4096,
  // 16/4 heads D = 64 405 against 412, 96 593 against 607, 128 793 against 835; 8192, 16/2
  // heads 801 against 842, 1166 against 1219, 1571 against 1725; but 2 x 2048, 16/4 heads, of
  // 256 steps, 158 against 147, 221 against 203, 279 against 261).
  if (a.prefix && key_steps(a) > 104 && groups <= 1100) return key_steps(a) < 512 ? 3 : 2;
  if (BF16 && DC == 64) return (int32_t)splits;
  return key_steps(a) >= 256 && 4 * groups < 5 * places ? 3 : 1;
}

// dq: the same for the work groups that share the keys of 32 queries of one head. (Where
// there are any, there are such of dk and dv too, whose launch adds their sums.)
template <bool BF16, int DC>
int32_t query_splits(const attn::Args& a) {
  const int64_t places = 256 * (attn::OwnRows<BF16, DC, 4, 0>::kLds <= 80 * 1024 ? 2 : 1);
  return (int32_t)most_splits(3 * places / (4 * ((int64_t)a.N / 32 + a.S) * a.Hq) * 2 + 1, ((int64_t)a.N + 31) / 32);
}

template <bool BF16, int DC>
void set_splits(attn::Args& a) {
  a.splits = key_splits<BF16, DC>(a);
  a.qsplits = a.splits > 1 ? query_splits<BF16, DC>(a) : 1;
}
void set_splits(attn::Args& a, bool bf16) {
  if (bf16) a.D <= 64 ? set_splits<true, 64>(a) : a.D <= 96 ? set_splits<true, 96>(a) : set_splits<true, 128>(a);
  else a.D <= 64 ? set_splits<false, 64>(a) : a.D <= 96 ? set_splits<false, 96>(a) : set_splits<false, 128>(a);
}

// One launch, or more where a grid's z dimension does not hold the slots.
template <typename F>
hipError_t launch_slots(attn::Args a, int rows, int rep, F launch) {
  const int64_t slots = slots_of(a, rows) + (a.clear ? 1 : 0);   // one without a tile at least
  a.slots = (int32_t)slots;
  for (int64_t s = 0; s < slots; s += 65535) {
    a.slot0 = (int32_t)s;
    launch(a, dim3((uint32_t)a.Hkv, (uint32_t)rep, (uint32_t)std::min<int64_t>(65535, slots - s)));
  }
  return hipGetLastError();
}

template <bool BF16, int DC, int MOD>
hipError_t run_attn_forward(const attn::Args& a, hipStream_t stream) {
  const int rep = a.Hq / a.Hkv;
  if constexpr (!kRowsAlways<BF16, DC>) {
    if (slots_of(a, 32) * a.Hq > kRowsMost)
      return launch_slots(a, 128, rep, [&](const attn::Args& x, dim3 grid) {
        attn::k_forward<BF16, DC, MOD><<<grid, 256, 0, stream>>>(x);
      });
  }
  return launch_slots(a, 32, rep, [&](const attn::Args& x, dim3 grid) {
    attn::k_forward_rows<BF16, DC, 4, MOD><<<grid, 256, 0, stream>>>(x);
  });
}

template <bool BF16, int DC, int MOD>
hipError_t run_attn_backward_q(const attn::Args& a, hipStream_t stream) {
  const int rep = a.Hq / a.Hkv;
  if constexpr (!kRowsAlways<BF16, DC>) {
    if (slots_of(a, 32) * a.Hq > kRowsMost)
      return launch_slots(a, 128, rep, [&](const attn::Args& x, dim3 grid) {
        attn::k_backward_q<BF16, DC, MOD><<<grid, 256, 0, stream>>>(x);
      });
  }
  if (a.qsplits > 1)
    return launch_slots(a, 32, rep * a.qsplits, [&](const attn::Args& x, dim3 grid) {
      attn::k_backward_q_rows<BF16, DC, 4, true, MOD><<<grid, 256, 0, stream>>>(x);
    });
  return launch_slots(a, 32, rep, [&](const attn::Args& x, dim3 grid) {
    attn::k_backward_q_rows<BF16, DC, 4, false, MOD><<<grid, 256, 0, stream>>>(x);
  });
}

template <bool BF16, int DC, int MOD>
hipError_t run_attn_backward(const attn::Args& a, hipStream_t stream) {
  const hipError_t he = run_attn_backward_q<BF16, DC, MOD>(a, stream);
  if (he != hipSuccess) return he;
  if (a.splits > 1)
    return launch_slots(a, 32, a.splits, [&](const attn::Args& x, dim3 grid) {
      if (a.qsplits > 1) grid.z += (uint32_t)(((int64_t)x.slots * a.Hq + grid.x * grid.y - 1) / (grid.x * grid.y));
      attn::k_backward_kv<BF16, DC, 4, true, MOD><<<grid, 256, 0, stream>>>(x);
    });
  if constexpr (BF16 && DC == 64) {
    if (keys_eight(a))
      return launch_slots(a, 32, 1, [&](const attn::Args& x, dim3 grid) {
        attn::k_backward_kv<BF16, DC, 8, false, MOD><<<grid, 512, 0, stream>>>(x);
      });
  }
  return launch_slots(a, 32, 1, [&](const attn::Args& x, dim3 grid) {
    attn::k_backward_kv<BF16, DC, 4, false, MOD><<<grid, 256, 0, stream>>>(x);
  });
}

// f with the kernels' type, columns and set as constants.
template <int MOD, typename F>
hipError_t with_columns(bool bf16, int32_t D, F f) {
  using std::integral_constant;
  const auto go = [&](auto b) {
    constexpr bool B = decltype(b)::value;
    if (D <= 64) return f(b, integral_constant<int, 64>{}, integral_constant<int, MOD>{});
    if (D <= 96) return f(b, integral_constant<int, 96>{}, integral_constant<int, MOD>{});
    return f(integral_constant<bool, B>{}, integral_constant<int, 128>{}, integral_constant<int, MOD>{});
  };
  return bf16 ? go(integral_constant<bool, true>{}) : go(integral_constant<bool, false>{});
}
template <typename F>
hipError_t with_kernels(const attn::Args& a, bool bf16, F f) {
  if (a.cap > 0.f && a.slopes) return with_columns<attn::kCapped | attn::kBiased>(bf16, a.D, f);
  if (a.cap > 0.f) return with_columns<attn::kCapped>(bf16, a.D, f);
  if (a.slopes || a.prefix) return with_columns<attn::kBiased>(bf16, a.D, f);
  return with_columns<attn::kPlain>(bf16, a.D, f);
}

// Caps: a score's tanh has an absolute error of a few 2^-24, times the cap; past 1024 that
// would come near the rounding of bf16 weights. Slopes are added in units of the scale, and
// products squeezed by scale / cap.
dpnorm_status check_scores(const dpnorm_attn_shape* shape, const dpnorm_attn_scores* s) {
  if (!s) return DPNORM_OK;
  if (!(s->cap == 0.f || (s->cap >= 1.f / 1024 && s->cap <= 1024.f))) return DPNORM_ERR_VALUE;
  if (s->slopes && shape->scale < 0x1p-64f) return DPNORM_ERR_VALUE;
  if (s->cap > 0.f && shape->scale > 0x1p64f) return DPNORM_ERR_VALUE;
  if (!aligned(s->slopes, 4) || !aligned(s->prefix, 4)) return DPNORM_ERR_ALIGN;
  return DPNORM_OK;
}
void set_scores(attn::Args& a, const dpnorm_attn_scores* s) {
  if (!s) return;
  a.cap = s->cap;
  a.squeeze = s->cap > 0.f ? (float)(2.0 * 1.4426950408889634 * a.scale / s->cap) : 0.f;
  a.slopes = s->slopes;
  a.prefix = s->prefix;
}
// What the scores read, as inputs.
std::vector<Region> score_inputs(const dpnorm_attn_shape* shape, const dpnorm_attn_scores* s) {
  if (!s) return {};
  return {{s->slopes, (size_t)shape->Hq * 4}, {s->prefix, (size_t)shape->S * 4}};
}

// The workspace of a backward pass (its bytes; null to ask for them alone): the pairs,
// and where work groups share keys or queries their sums, counters and marks.
size_t backward_layout(attn::Args& a, bool bf16, void* ws) {
  set_splits(a, bf16);
  size_t bytes = 0;
  const auto take = [&](size_t n) {
    char* p = ws ? (char*)ws + bytes : nullptr;
    bytes += align_up(n);
    return p;
  };
  a.pairs = (float*)take((size_t)a.N * a.Hq * 8);
  if (a.splits < 2) return bytes;
  const size_t slots = (size_t)slots_of(a, 32) + 1, tile = 32 * 4 * (a.D <= 64 ? 64 : a.D <= 96 ? 96 : 128);
  a.groups = (int32_t)(slots * a.Hkv);
  a.arrived = (uint32_t*)take(slots * a.Hkv * 4);
  a.parts = (float*)take(slots * a.Hkv * a.splits * 2 * tile);
  if (a.qsplits < 2) return bytes;
  a.qcareful = (uint32_t*)take(slots * a.Hq * a.qsplits * 4);
  a.qparts = (float*)take(slots * a.Hq * a.qsplits * tile);
  return bytes;
}

}  // namespace

extern "C" {

dpnorm_status dpnorm_attention_scores_forward(const dpnorm_attn_shape* shape, const dpnorm_attn_scores* scores,
                                              const dpnorm_attn_tensor* q, const dpnorm_attn_tensor* k,
                                              const dpnorm_attn_tensor* v, const dpnorm_attn_tensor* o, float* lse,
                                              hipStream_t stream) {
  dpnorm_status st = check_shape(shape);
  if (st == DPNORM_OK) st = check_scores(shape, scores);
  if (st == DPNORM_OK) st = check_tensor(q, shape, shape->Hq, false);
  if (st == DPNORM_OK) st = check_tensor(k, shape, shape->Hkv, false);
  if (st == DPNORM_OK) st = check_tensor(v, shape, shape->Hkv, false);
  if (st == DPNORM_OK) st = check_tensor(o, shape, shape->Hq, true);
  if (st != DPNORM_OK) return st;
  if (!lse) return DPNORM_ERR_NULL;
  if (!aligned(lse, 4)) return DPNORM_ERR_ALIGN;
  const size_t e = esize(shape->dtype);
  const int64_t N = shape->N, Hq = shape->Hq, Hkv = shape->Hkv, D = shape->D;
  std::vector<Region> in = score_inputs(shape, scores);
  in.insert(in.end(), {{q->data, span(*q, N, Hq, D, e)}, {k->data, span(*k, N, Hkv, D, e)}, {v->data, span(*v, N, Hkv, D, e)},
                       {shape->cu_seqlens, (size_t)(shape->S + 1) * 4}});
  if (outputs_overlap(in, {{o->data, span(*o, N, Hq, D, e)}, {lse, (size_t)N * Hq * 4}})) return DPNORM_ERR_VALUE;
  attn::Args a = attn_args(shape);
  a.q = tensor_of(q, N, Hq, e);
  a.k = tensor_of(k, N, Hkv, e);
  a.v = tensor_of(v, N, Hkv, e);
  a.o = tensor_of(o, N, Hq, e);
  a.lse = lse;
  set_scores(a, scores);
  return hip_status(with_kernels(a, shape->dtype == DPNORM_BF16, [&](auto bf16, auto columns, auto mod) {
    return run_attn_forward<decltype(bf16)::value, decltype(columns)::value, decltype(mod)::value>(a, stream);
  }));
}

dpnorm_status dpnorm_attention_forward(const dpnorm_attn_shape* shape, const dpnorm_attn_tensor* q, const dpnorm_attn_tensor* k,
                                       const dpnorm_attn_tensor* v, const dpnorm_attn_tensor* o, float* lse,
                                       hipStream_t stream) {
  return dpnorm_attention_scores_forward(shape, nullptr, q, k, v, o, lse, stream);
}

dpnorm_status dpnorm_attention_scores_backward_workspace(const dpnorm_attn_shape* shape, const dpnorm_attn_scores* scores,
                                                         size_t* bytes) {
  if (!bytes) return DPNORM_ERR_NULL;
  dpnorm_status st = check_shape(shape);
  if (st == DPNORM_OK) st = check_scores(shape, scores);
  if (st != DPNORM_OK) return st;
  attn::Args a = attn_args(shape);
  set_scores(a, scores);
  *bytes = backward_layout(a, shape->dtype == DPNORM_BF16, nullptr);
  return DPNORM_OK;
}

dpnorm_status dpnorm_attention_backward_workspace(const dpnorm_attn_shape* shape, size_t* bytes) {
  return dpnorm_attention_scores_backward_workspace(shape, nullptr, bytes);
}

dpnorm_status dpnorm_attention_scores_backward(const dpnorm_attn_shape* shape, const dpnorm_attn_scores* scores,
                                               const dpnorm_attn_tensor* dO, const dpnorm_attn_tensor* q,
                                               const dpnorm_attn_tensor* k, const dpnorm_attn_tensor* v,
                                               const dpnorm_attn_tensor* o, const float* lse, const dpnorm_attn_tensor* dq,
                                               const dpnorm_attn_tensor* dk, const dpnorm_attn_tensor* dv, void* ws,
                                               size_t ws_bytes, hipStream_t stream) {
  size_t bytes = 0;
  dpnorm_status st = dpnorm_attention_scores_backward_workspace(shape, scores, &bytes);
  for (const dpnorm_attn_tensor* t : {dO, q, o})
    if (st == DPNORM_OK) st = check_tensor(t, shape, shape->Hq, false);
  for (const dpnorm_attn_tensor* t : {k, v})
    if (st == DPNORM_OK) st = check_tensor(t, shape, shape->Hkv, false);
  if (st == DPNORM_OK) st = check_tensor(dq, shape, shape->Hq, true);
  for (const dpnorm_attn_tensor* t : {dk, dv})
    if (st == DPNORM_OK) st = check_tensor(t, shape, shape->Hkv, true);
  if (st != DPNORM_OK) return st;
  if (!lse || !ws) return DPNORM_ERR_NULL;
  if (!aligned(lse, 4) || !aligned(ws, kAlign)) return DPNORM_ERR_ALIGN;
  if (ws_bytes < bytes) return DPNORM_ERR_WORKSPACE;
  const size_t e = esize(shape->dtype);
  const int64_t N = shape->N, Hq = shape->Hq, Hkv = shape->Hkv, D = shape->D;
  std::vector<Region> in = score_inputs(shape, scores);
  in.insert(in.end(), {{dO->data, span(*dO, N, Hq, D, e)}, {q->data, span(*q, N, Hq, D, e)}, {o->data, span(*o, N, Hq, D, e)},
                       {k->data, span(*k, N, Hkv, D, e)}, {v->data, span(*v, N, Hkv, D, e)}, {lse, (size_t)N * Hq * 4},
                       {shape->cu_seqlens, (size_t)(shape->S + 1) * 4}});
  if (outputs_overlap(in,
                      {{dq->data, span(*dq, N, Hq, D, e)}, {dk->data, span(*dk, N, Hkv, D, e)}, {dv->data, span(*dv, N, Hkv, D, e)},
                       {ws, bytes}}))
    return DPNORM_ERR_VALUE;
  attn::Args a = attn_args(shape);
  a.dO = tensor_of(dO, N, Hq, e);
  a.q = tensor_of(q, N, Hq, e);
  a.k = tensor_of(k, N, Hkv, e);
  a.v = tensor_of(v, N, Hkv, e);
  a.o = tensor_of(o, N, Hq, e);
  a.dq = tensor_of(dq, N, Hq, e);
  a.dk = tensor_of(dk, N, Hkv, e);
  a.dv = tensor_of(dv, N, Hkv, e);
  a.lse = const_cast<float*>(lse);
  set_scores(a, scores);
  backward_layout(a, shape->dtype == DPNORM_BF16, ws);
  return hip_status(with_kernels(a, shape->dtype == DPNORM_BF16, [&](auto bf16, auto columns, auto mod) {
    return run_attn_backward<decltype(bf16)::value, decltype(columns)::value, decltype(mod)::value>(a, stream);
  }));
}

dpnorm_status dpnorm_attention_backward(const dpnorm_attn_shape* shape, const dpnorm_attn_tensor* dO, const dpnorm_attn_tensor* q,
                                        const dpnorm_attn_tensor* k, const dpnorm_attn_tensor* v, const dpnorm_attn_tensor* o,
                                        const float* lse, const dpnorm_attn_tensor* dq, const dpnorm_attn_tensor* dk,
                                        const dpnorm_attn_tensor* dv, void* ws, size_t ws_bytes, hipStream_t stream) {
  return dpnorm_attention_scores_backward(shape, nullptr, dO, q, k, v, o, lse, dq, dk, dv, ws, ws_bytes, stream);
}

}  // extern "C"
