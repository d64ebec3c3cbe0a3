// C ABI of libbmoe.so, routing from logits and what a training step needs
// around the layer: host-side validation, workspace carving and the launches.
#include <algorithm>
#include <climits>
#include <cmath>
#include <vector>

#include "common.h"
#include "kernels.h"

namespace bmoe {
namespace {

constexpr int kMaxPicks = 64;

bool ok16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Shape and spec of a routing call; *out is filled on BMOE_OK.
bmoe_status check_route(bmoe_dtype dt, int T, int N, int k, const bmoe_route_spec* spec,
                        RouteSpec* out) {
  if (dt != BMOE_F32 && dt != BMOE_BF16) return BMOE_E_DTYPE;
  if (N < 1 || N > kMaxExperts || k < 1 || k > N || k > kMaxPicks || T < 0) return BMOE_E_SHAPE;
  if ((long long)T * k > INT_MAX) return BMOE_E_SHAPE;
  if (!spec) return BMOE_E_NULL;
  const bmoe_route_spec& s = *spec;
  if (s.score != BMOE_SCORE_SOFTMAX && s.score != BMOE_SCORE_SIGMOID) return BMOE_E_VALUE;
  if (s.group_score != BMOE_GROUP_MAX && s.group_score != BMOE_GROUP_TOP2) return BMOE_E_VALUE;
  if (!std::isfinite(s.scale)) return BMOE_E_VALUE;
  if (s.n_groups < 1 || s.n_groups > 64 || N % s.n_groups != 0) return BMOE_E_VALUE;
  if (s.topk_groups < 1 || s.topk_groups > s.n_groups) return BMOE_E_VALUE;
  if (s.topk_groups * (N / s.n_groups) < k) return BMOE_E_VALUE;
  out->score = s.score;
  out->renorm = s.renorm != 0;
  out->scale = s.scale;
  // keeping every group leaves every expert a candidate
  const bool grouped = s.topk_groups < s.n_groups;
  out->groups = grouped ? s.n_groups : 1;
  out->keep = grouped ? s.topk_groups : 1;
  out->group_score = s.group_score;
  return BMOE_OK;
}

bool pow2_d16(int d) { return d >= 16 && d <= 8192 && (d & (d - 1)) == 0; }

size_t elem(bmoe_dtype dt) { return dt == BMOE_BF16 ? 2 : 4; }

bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && a_bytes && b_bytes && x < y + b_bytes && y < x + a_bytes;
}

struct PairsLayout {
  size_t list, off, part, total;
  int tokens, ranges;
};
PairsLayout router_pairs_layout(int T, int d, int N, int k) {
  PairsLayout l;
  l.tokens = router_range_tokens(T, d, N);
  l.ranges = T > 0 ? (int)(((long long)T + l.tokens - 1) / l.tokens) : 1;
  const size_t list_bytes = up256((size_t)T * k * sizeof(int2));
  l.list = list_bytes;
  l.off = l.list + list_bytes;
  l.part = l.off + up256((size_t)l.ranges * (N + 1) * sizeof(int32_t));
  const int groups = (l.ranges + 3) / 4;
  l.total = l.part + (groups > 1 ? up256((size_t)groups * N * d * sizeof(float)) : 0);
  return l;
}

size_t dl_bytes(int T, int N) { return up256((size_t)T * N * sizeof(float)); }
size_t parts_bytes(int T, int N) {
  return up256(((size_t)T + 31) / 32 * 32 * 3 * router_parts_experts(N) * 2);
}

// The list of a gradient call: types, NULLs, alignment to the element, and
// (where it is written) no two written tensors, and no written and another
// read tensor, that share bytes. `out` may repeat `grads` entry by entry.
bmoe_status check_grads(int n, const bmoe_tensor* grads, const bmoe_tensor* out, bool writes) {
  if (n < 0) return BMOE_E_SHAPE;
  if (n == 0) return BMOE_OK;
  if (!grads) return BMOE_E_NULL;
  constexpr size_t kMostEntries = (size_t)1 << 40;  // a table's chunk numbers are 32 bits
  size_t entries = 0;
  for (int i = 0; i < n; ++i) {
    const bmoe_tensor& g = grads[i];
    if (g.dtype != BMOE_F32 && g.dtype != BMOE_BF16) return BMOE_E_DTYPE;
    if (g.count > kMostEntries - entries) return BMOE_E_SHAPE;
    entries += g.count;
    if (g.count && !g.data) return BMOE_E_NULL;
    if (reinterpret_cast<uintptr_t>(g.data) % elem((bmoe_dtype)g.dtype)) return BMOE_E_ALIGN;
    if (out) {
      if (out[i].dtype != g.dtype) return BMOE_E_DTYPE;
      if (out[i].count != g.count) return BMOE_E_SHAPE;
      if (g.count && !out[i].data) return BMOE_E_NULL;
      if (reinterpret_cast<uintptr_t>(out[i].data) % elem((bmoe_dtype)g.dtype)) return BMOE_E_ALIGN;
    }
  }
  if (!writes) return BMOE_OK;
  // Spans sorted by address: an overlap shows between a span and the furthest
  // end so far of the spans that it may not meet.
  struct Span {
    uintptr_t lo, hi;
    bool written;
  };
  try {
    std::vector<Span> v;
    v.reserve(out ? 2 * (size_t)n : (size_t)n);
    for (int i = 0; i < n; ++i) {
      if (!grads[i].count) continue;
      const size_t bytes = grads[i].count * elem((bmoe_dtype)grads[i].dtype);
      const uintptr_t a = reinterpret_cast<uintptr_t>(grads[i].data);
      const uintptr_t b = out ? reinterpret_cast<uintptr_t>(out[i].data) : a;
      if (a != b) v.push_back({a, a + bytes, false});
      v.push_back({b, b + bytes, true});
    }
    std::sort(v.begin(), v.end(), [](const Span& x, const Span& y) { return x.lo < y.lo; });
    uintptr_t end_w = 0, end_r = 0;  // furthest ends of written and of read spans
    for (const Span& x : v) {
      if (x.lo < end_w || (x.written && x.lo < end_r)) return BMOE_E_VALUE;
      if (x.written) end_w = std::max(end_w, x.hi);
      else end_r = std::max(end_r, x.hi);
    }
  } catch (...) {  // out of host memory: no exception leaves a C entry
    return BMOE_E_HIP;
  }
  return BMOE_OK;
}

// Runs f(table) over the list's non-empty tensors, kGradTab at a time.
template <typename F>
bmoe_status each_table(int n, const bmoe_tensor* grads, const bmoe_tensor* out, F f) {
  GradTable tab;
  tab.n = 0;
  tab.chunks = 0;
  for (int i = 0; i < n; ++i) {
    if (!grads[i].count) continue;
    const int bf16 = grads[i].dtype == BMOE_BF16;
    const uint32_t c = grad_chunks(grads[i].data, grads[i].count, bf16);
    if (tab.n == kGradTab) {
      if (f(tab) != hipSuccess) return BMOE_E_HIP;
      tab.n = 0;
      tab.chunks = 0;
    }
    tab.t[tab.n++] = {grads[i].data, out ? out[i].data : grads[i].data, grads[i].count, tab.chunks,
                      bf16};
    tab.chunks += c;
  }
  return !tab.n || f(tab) == hipSuccess ? BMOE_OK : BMOE_E_HIP;
}

// Partial sums of the whole list to part; their number to *used.
bmoe_status grad_sq_impl(int n, const bmoe_tensor* grads, double* part, int* used, hipStream_t s) {
  *used = 0;
  size_t chunks = 0;  // of the whole list: the scaling comes after all of its tables
  for (int i = 0; i < n; ++i)
    if (grads[i].count)
      chunks += grad_chunks(grads[i].data, grads[i].count, grads[i].dtype == BMOE_BF16);
  return each_table(n, grads, nullptr, [&](const GradTable& t) {
    int np = 0;
    const hipError_t e = launch_grad_sq(t, chunks, part + *used, &np, s);
    *used += np;
    return e;
  });
}

// part not NULL: the norm from its n_part sums, written to *norm.
bmoe_status grad_scale_impl(int n, const bmoe_tensor* grads, const bmoe_tensor* out,
                            const double* part, int n_part, float* norm, float max_norm,
                            hipStream_t s) {
  bool in_place = true;
  for (int i = 0; out && i < n; ++i) in_place &= out[i].data == grads[i].data || !grads[i].count;
  return each_table(n, grads, out, [&](const GradTable& t) {
    return launch_grad_scale(t, part, n_part, norm, max_norm, in_place, s);
  });
}

bool good_max_norm(float m) { return m > 0.f; }  // +inf: no clipping; NaN refused

}  // namespace
}  // namespace bmoe

using namespace bmoe;

extern "C" {

bmoe_status bmoe_router_logits(bmoe_dtype dt, int T, int d, int n_experts, const void* x,
                               const void* w_router, float* logits, void* stream) {
  if (dt != BMOE_F32 && dt != BMOE_BF16) return BMOE_E_DTYPE;
  if (!pow2_d16(d) || n_experts < 1 || n_experts > kMaxExperts || T < 0) return BMOE_E_SHAPE;
  if (T == 0) return BMOE_OK;
  if (!x || !w_router || !logits) return BMOE_E_NULL;
  if (!ok16(x) || !ok16(w_router) || !ok16(logits)) return BMOE_E_ALIGN;
  return launch_router_logits(dt, T, d, n_experts, x, w_router, logits,
                              static_cast<hipStream_t>(stream), KernelTiming{}) == hipSuccess
             ? BMOE_OK
             : BMOE_E_HIP;
}

bmoe_status bmoe_route(bmoe_dtype dt, int T, int n_experts, int k, const bmoe_route_spec* spec,
                       const void* logits, const float* bias, int32_t* ids, float* gates,
                       void* stream) {
  RouteSpec sp;
  const bmoe_status st = check_route(dt, T, n_experts, k, spec, &sp);
  if (st != BMOE_OK) return st;
  if (T == 0) return BMOE_OK;
  if (!logits || !ids || !gates) return BMOE_E_NULL;
  if (!ok16(logits) || !ok16(ids) || !ok16(gates) || (bias && !ok16(bias))) return BMOE_E_ALIGN;
  return launch_route(dt, T, n_experts, k, sp, logits, bias, ids, gates,
                      static_cast<hipStream_t>(stream)) == hipSuccess
             ? BMOE_OK
             : BMOE_E_HIP;
}

bmoe_status bmoe_route_backward(bmoe_dtype dt, int T, int n_experts, int k,
                                const bmoe_route_spec* spec, const void* logits,
                                const int32_t* ids, const float* dgates, float* dlogits,
                                void* stream) {
  RouteSpec sp;
  const bmoe_status st = check_route(dt, T, n_experts, k, spec, &sp);
  if (st != BMOE_OK) return st;
  if (T == 0) return BMOE_OK;
  if (!logits || !ids || !dgates || !dlogits) return BMOE_E_NULL;
  if (!ok16(logits) || !ok16(ids) || !ok16(dgates) || !ok16(dlogits)) return BMOE_E_ALIGN;
  return launch_route_bwd(dt, T, n_experts, k, sp, logits, ids, dgates, dlogits,
                          static_cast<hipStream_t>(stream)) == hipSuccess
             ? BMOE_OK
             : BMOE_E_HIP;
}

size_t bmoe_route_balance_workspace_bytes(int T, int n_experts, int k) {
  if (n_experts < 1 || n_experts > kMaxExperts || k < 1 || T < 0 || (long long)T * k > INT_MAX)
    return 0;
  return up256(balance_part_bytes((long long)T * k, n_experts)) + 256;
}

bmoe_status bmoe_route_balance(int T, int n_experts, int k, const int32_t* ids, int accumulate,
                               float rate, int32_t* load, float* bias, void* ws, size_t ws_bytes,
                               void* stream) {
  const size_t need = bmoe_route_balance_workspace_bytes(T, n_experts, k);
  if (!need) return BMOE_E_SHAPE;
  if (bias && !std::isfinite(rate)) return BMOE_E_VALUE;
  if (!load || (T > 0 && !ids)) return BMOE_E_NULL;
  if (!ws || ws_bytes < need) return BMOE_E_WORKSPACE;
  if (!ok16(ids) || !ok16(load) || !ok16(bias) || !ok16(ws)) return BMOE_E_ALIGN;
  return launch_balance((long long)T * k, n_experts, ids, accumulate, rate, load, bias,
                        static_cast<int*>(ws), static_cast<hipStream_t>(stream)) == hipSuccess
             ? BMOE_OK
             : BMOE_E_HIP;
}

size_t bmoe_router_backward_workspace_bytes(bmoe_dtype dt, int T, int d, int n_experts, int k) {
  if ((dt != BMOE_F32 && dt != BMOE_BF16) || !pow2_d16(d) || n_experts < 1 ||
      n_experts > kMaxExperts || k < 1 || k > n_experts || k > kMaxPicks || T < 0 ||
      (long long)T * k > INT_MAX)
    return 0;
  // dl [T][N] (its three parts for bf16) with the dW of the token ranges, or
  // the picks' pairs and lists with the dW of theirs
  const int S = dt == BMOE_BF16 ? router_dense_splits(T, d, n_experts)
                                : router_f32_splits(T, d, n_experts);
  const size_t dense =
      (dt == BMOE_BF16 ? parts_bytes(T, n_experts) : dl_bytes(T, n_experts)) +
      (S > 1 ? (size_t)S * n_experts * d * sizeof(float) : 0);
  const size_t sparse = router_pairs_layout(T, d, n_experts, k).total;
  return (dense > sparse ? dense : sparse) + 256;
}

bmoe_status bmoe_router_backward(bmoe_dtype dt, int T, int d, int n_experts, int k,
                                 const bmoe_route_spec* spec, const void* x, const void* w_router,
                                 const float* logits, const int32_t* ids, const float* dgates,
                                 const void* dx_add, void* dx, float* dw, void* ws,
                                 size_t ws_bytes, void* stream) {
  RouteSpec sp;
  const bmoe_status st = check_route(dt, T, n_experts, k, spec, &sp);
  if (st != BMOE_OK) return st;
  const size_t need = bmoe_router_backward_workspace_bytes(dt, T, d, n_experts, k);
  if (!need) return BMOE_E_SHAPE;
  if (!dw || (T > 0 && (!x || !w_router || !logits || !ids || !dgates || !dx)))
    return BMOE_E_NULL;
  if (!ws || ws_bytes < need) return BMOE_E_WORKSPACE;
  const void* ptrs[] = {x, w_router, logits, ids, dgates, dx_add, dx, dw, ws};
  for (const void* p : ptrs)
    if (!ok16(p)) return BMOE_E_ALIGN;
  // what is written while others are read shares no byte with them; dx_add is
  // read entry by entry before dx is written
  struct Span {
    const void* p;
    size_t bytes;
  };
  const size_t x_bytes = (size_t)T * d * elem(dt), w_entries = (size_t)n_experts * d;
  const Span written[] = {{dx, x_bytes}, {dw, w_entries * sizeof(float)}, {ws, need}};
  const Span read[] = {{x, x_bytes},
                       {w_router, w_entries * elem(dt)},
                       {logits, (size_t)T * n_experts * sizeof(float)},
                       {ids, (size_t)T * k * sizeof(int32_t)},
                       {dgates, (size_t)T * k * sizeof(float)},
                       {dx_add == dx ? nullptr : dx_add, x_bytes}};
  for (const Span& a : written) {
    for (const Span& b : read)
      if (overlap(a.p, a.bytes, b.p, b.bytes)) return BMOE_E_VALUE;
    for (const Span& b : written)
      if (&a != &b && overlap(a.p, a.bytes, b.p, b.bytes)) return BMOE_E_VALUE;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (T > 0 && !(sp.score == BMOE_SCORE_SOFTMAX && !sp.renorm)) {
    const PairsLayout l = router_pairs_layout(T, d, n_experts, k);
    char* base = static_cast<char*>(ws);
    RouterPairs rp;
    rp.pairs = reinterpret_cast<int2*>(base);
    rp.list = reinterpret_cast<int2*>(base + l.list);
    rp.off = reinterpret_cast<int32_t*>(base + l.off);
    rp.tokens = l.tokens;
    rp.ranges = l.ranges;
    if (launch_route_pairs(T, n_experts, k, sp, logits, ids, dgates, rp, s) != hipSuccess ||
        launch_router_bwd_sparse(dt, T, d, n_experts, k, x, w_router, rp, dx_add, dx, dw,
                                 reinterpret_cast<float*>(base + l.part), s) != hipSuccess)
      return BMOE_E_HIP;
    return BMOE_OK;
  }
  if (T > 0 && dt == BMOE_BF16) {
    uint16_t* parts = static_cast<uint16_t*>(ws);
    float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + parts_bytes(T, n_experts));
    if (launch_route_bwd_parts(T, n_experts, k, sp, logits, ids, dgates, parts, s) != hipSuccess ||
        launch_router_bwd_parts(T, d, n_experts, static_cast<const uint16_t*>(x),
                                static_cast<const uint16_t*>(w_router), parts,
                                static_cast<const uint16_t*>(dx_add), static_cast<uint16_t*>(dx),
                                dw, part, s) != hipSuccess)
      return BMOE_E_HIP;
    return BMOE_OK;
  }
  // fp32, or no tokens (dw = 0, whatever x's type)
  float* dl = static_cast<float*>(ws);
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + dl_bytes(T, n_experts));
  if (T > 0 &&
      launch_route_bwd(BMOE_F32, T, n_experts, k, sp, logits, ids, dgates, dl, s) != hipSuccess)
    return BMOE_E_HIP;
  return launch_router_bwd_f32(T, d, n_experts, static_cast<const float*>(x),
                               static_cast<const float*>(w_router), dl,
                               static_cast<const float*>(dx_add), static_cast<float*>(dx), dw,
                               part, s) == hipSuccess
             ? BMOE_OK
             : BMOE_E_HIP;
}

size_t bmoe_grad_workspace_bytes(int n) {
  if (n < 0) return 0;
  const size_t tables = ((size_t)n + kGradTab - 1) / kGradTab;
  return up256((tables ? tables : 1) * kGradParts * sizeof(double));
}

bmoe_status bmoe_grad_norm(int n, const bmoe_tensor* grads, float* norm, void* ws, size_t ws_bytes,
                           void* stream) {
  const bmoe_status st = check_grads(n, grads, nullptr, false);
  if (st != BMOE_OK) return st;
  if (!norm) return BMOE_E_NULL;
  if (!ws || ws_bytes < bmoe_grad_workspace_bytes(n)) return BMOE_E_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(norm) & 3u) || !ok16(ws)) return BMOE_E_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(ws);
  int used = 0;
  const bmoe_status rs = grad_sq_impl(n, grads, part, &used, s);
  if (rs != BMOE_OK) return rs;
  return launch_grad_norm(part, used, norm, s) == hipSuccess ? BMOE_OK : BMOE_E_HIP;
}

bmoe_status bmoe_grad_scale(int n, const bmoe_tensor* grads, const bmoe_tensor* out,
                            const float* norm, float max_norm, void* stream) {
  const bmoe_status st = check_grads(n, grads, out, true);
  if (st != BMOE_OK) return st;
  if (!good_max_norm(max_norm)) return BMOE_E_VALUE;
  if (!norm) return BMOE_E_NULL;
  if (reinterpret_cast<uintptr_t>(norm) & 3u) return BMOE_E_ALIGN;
  return grad_scale_impl(n, grads, out, nullptr, 0, const_cast<float*>(norm), max_norm,
                         static_cast<hipStream_t>(stream));
}

bmoe_status bmoe_grad_clip(int n, const bmoe_tensor* grads, const bmoe_tensor* out, float max_norm,
                           float* norm, void* ws, size_t ws_bytes, void* stream) {
  const bmoe_status st = check_grads(n, grads, out, true);
  if (st != BMOE_OK) return st;
  if (!good_max_norm(max_norm)) return BMOE_E_VALUE;
  if (!norm) return BMOE_E_NULL;
  if (!ws || ws_bytes < bmoe_grad_workspace_bytes(n)) return BMOE_E_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(norm) & 3u) || !ok16(ws)) return BMOE_E_ALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(ws);
  int used = 0;
  const bmoe_status rs = grad_sq_impl(n, grads, part, &used, s);
  if (rs != BMOE_OK) return rs;
  // One table's partial sums are added by every workgroup of the scaling (16
  // KB from L2, instead of a launch in between); more tables' once.
  const bool inside = used > 0 && used <= kGradParts;
  if (!inside && launch_grad_norm(part, used, norm, s) != hipSuccess) return BMOE_E_HIP;
  return grad_scale_impl(n, grads, out, inside ? part : nullptr, used, norm, max_norm, s);
}

}  // extern "C"
