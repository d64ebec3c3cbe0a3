// C ABI of libbmoe.so, what stands around an expert layer's block: dense
// experts, the norms around the block, orthogonalised updates. Host-side
// validation, workspace carving and the launches.
#include <climits>
#include <cmath>
#include <initializer_list>

#include "common.h"
#include "kernels.h"

namespace bmoe {
namespace {

constexpr int kMaxWidth = 65536;  // K and O of a dense expert
constexpr int kMaxNormWidth = 8192;
constexpr int kMaxOrtho = 16384;  // rows and columns of a matrix
constexpr int kMaxBatch = 65535;
constexpr int kMaxPicks = 64;

bool ok16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
bool ok_type(bmoe_dtype dt) { return dt == BMOE_F32 || dt == BMOE_BF16; }
size_t elem(bmoe_dtype dt) { return dt == BMOE_BF16 ? 2 : 4; }
bmoe_status status_of(hipError_t e) { return e == hipSuccess ? BMOE_OK : BMOE_E_HIP; }

struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
// No written span shares a byte with a read one or with another written one.
bool apart(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (const Span& a : written) {
    for (const Span& b : read)
      if (overlap(a, b)) return false;
    for (const Span& b : written)
      if (&a != &b && overlap(a, b)) return false;
  }
  return true;
}
bool all16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!ok16(p)) return false;
  return true;
}

bool grouped_shape(int M, int K, int O, int G, const void* perm, int k, int a_rows) {
  return M >= 0 && K >= 1 && K <= kMaxWidth && O >= 1 && O <= kMaxWidth && G >= 1 &&
         G <= kMaxExperts && (!perm || (k >= 1 && a_rows >= 1));
}

bmoe_status norm_spec(const bmoe_norm_spec* spec, NormCall* c) {
  if (!spec) return BMOE_E_NULL;
  if (!(spec->eps >= 0.f) || !std::isfinite(spec->eps) || !std::isfinite(spec->res_scale) ||
      !std::isfinite(spec->out_scale))
    return BMOE_E_VALUE;
  c->eps = spec->eps;
  c->res_scale = spec->res_scale;
  c->out_scale = spec->out_scale;
  return BMOE_OK;
}

// Rows of u are int32 numbers; M of them hold every pick unless inv says where.
bool norm_shape(int T, int d, int k, int M, const void* u, const void* inv) {
  if (T < 0 || d < 1 || d > kMaxNormWidth) return false;
  if (!u) return true;
  return k >= 1 && k <= kMaxPicks && (long long)T * k <= INT_MAX && M >= 0 &&
         (inv || M >= (long long)T * k);
}

// The range of the iteration under given coefficients: the singular values (all at
// most 1 at first) of X, whose squares are P's, and those of Q = a + b P + c P P,
// bounded through sigma^2 and a + b sigma^2 + c sigma^4 on a fine grid. No entry of
// a matrix passes its largest singular value.
struct OrthoRange {
  double x, q;
  bool ok;  // within what the products' fp16 parts hold: 16 with a scale of 2^12
};
OrthoRange ortho_range(const bmoe_ortho_spec& s) {
  double hi = 1.0, most_x = 1.0, most_q = 0.0;
  for (int i = 0; i < s.steps; ++i) {
    double next = 0.0;
    if (hi > most_x) most_x = hi;
    for (int j = 0; j <= 1024; ++j) {
      const double v = hi * j / 1024, v2 = v * v;
      const double q = std::fabs(s.a + (s.b + s.c * v2) * v2);
      if (!(q <= 15.0) || !(v2 <= 15.0)) return {0.0, 0.0, false};
      if (q > most_q) most_q = q;
      if (q * v > next) next = q * v;
    }
    hi = next * 1.01;  // (the last iterate is the result: no operand, so no bound)
  }
  return {most_x, most_q, true};
}
// The largest power of two up to 2^15 that leaves values of up to `most` within
// fp16 (65504, less what rounding and the grid may add).
float fp16_scale(double most) {
  int e = 15;
  while (std::ldexp(most, e) > 61440.0) --e;
  return (float)std::ldexp(1.0, e);
}

bmoe_status ortho_spec(const bmoe_ortho_spec* s, OrthoCall* c) {
  if (!s) return BMOE_E_NULL;
  if (s->steps < 1 || s->steps > 64 || !(s->eps >= 0.f) || !std::isfinite(s->eps) ||
      !std::isfinite(s->a) || !std::isfinite(s->b) || !std::isfinite(s->c))
    return BMOE_E_VALUE;
  const OrthoRange range = ortho_range(*s);
  if (!range.ok) return BMOE_E_VALUE;
  c->steps = s->steps;
  c->a = s->a;
  c->b = s->b;
  c->c = s->c;
  c->eps = s->eps;
  c->x_scale = fp16_scale(range.x * range.x);  // (range.x >= 1)
  c->q_scale = fp16_scale(range.q);
  return BMOE_OK;
}

// The calls that leave rows without a group or a pick as they were, or (fill) set
// them to 0.
bmoe_status grouped_product(bmoe_dtype dt, int M, int K, int O, int n_groups, const void* a,
                            int a_rows, const int32_t* perm, int k, const void* w,
                            const int32_t* offsets, void* c, bool fill, void* stream) {
  if (!ok_type(dt)) return BMOE_E_DTYPE;
  if (!grouped_shape(M, K, O, n_groups, perm, k, a_rows)) return BMOE_E_SHAPE;
  if (M == 0) return BMOE_OK;
  if (!a || !w || !offsets || !c) return BMOE_E_NULL;
  if (!all16({a, perm, w, offsets, c})) return BMOE_E_ALIGN;
  const size_t e = elem(dt);
  if (!apart({{c, (size_t)M * O * e}},
             {{a, (size_t)(perm ? a_rows : M) * K * e},
              {perm, (size_t)M * sizeof(int32_t)},
              {w, (size_t)n_groups * O * K * e},
              {offsets, (n_groups + 1) * sizeof(int32_t)}}))
    return BMOE_E_VALUE;
  return status_of(launch_grouped(dt, false, M, K, O, n_groups, a, perm, k, a_rows, w, offsets, c,
                                  fill, static_cast<hipStream_t>(stream)));
}

bmoe_status grouped_product_backward(bmoe_dtype dt, int M, int K, int O, int n_groups,
                                     const void* a, int a_rows, const int32_t* perm, int k,
                                     const void* w, const int32_t* offsets, const void* dc, void* da,
                                     float* dw, bool fill, void* ws, size_t ws_bytes, void* stream) {
  if (!ok_type(dt)) return BMOE_E_DTYPE;
  if (!grouped_shape(M, K, O, n_groups, perm, k, a_rows)) return BMOE_E_SHAPE;
  if (!offsets || (M > 0 && (!dc || (da && !w) || (dw && !a)))) return BMOE_E_NULL;
  const size_t need = bmoe_grouped_product_backward_workspace_bytes(dt, M, K, O, n_groups);
  if (!ws || ws_bytes < need) return BMOE_E_WORKSPACE;
  if (!all16({a, perm, w, offsets, dc, da, dw, ws})) return BMOE_E_ALIGN;
  const size_t e = elem(dt), w_entries = (size_t)n_groups * O * K;
  if (!apart({{da, (size_t)M * K * e}, {dw, w_entries * sizeof(float)}, {ws, need}},
             {{a, (size_t)(perm ? a_rows : M) * K * e},
              {perm, (size_t)M * sizeof(int32_t)},
              {w, w_entries * e},
              {offsets, (n_groups + 1) * sizeof(int32_t)},
              {dc, (size_t)M * O * e}}))
    return BMOE_E_VALUE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t h = hipSuccess;
  if (da && M > 0)
    h = launch_grouped(dt, true, M, O, K, n_groups, dc, nullptr, 1, M, w, offsets, da, fill, s);
  if (h == hipSuccess && dw)
    h = launch_grouped_dw(dt, M, O, K, n_groups, a, perm, k, perm ? a_rows : M, dc, offsets, dw,
                          static_cast<float*>(ws), s);
  return status_of(h);
}

bmoe_status norm_backward(bmoe_dtype dt, int T, int d, int k, const bmoe_norm_spec* spec,
                          const void* u, int u_rows, const int32_t* inv, const float* gates,
                          const void* r_out, const float* w_post, const float* w_pre,
                          const void* dr_out, const void* dn, void* du, float* dgates, void* dr,
                          float* dw_post, float* dw_pre, bool fill, void* ws, size_t ws_bytes,
                          void* stream) {
  if (!ok_type(dt)) return BMOE_E_DTYPE;
  if (!norm_shape(T, d, k, u_rows, u, inv)) return BMOE_E_SHAPE;
  NormCall c = {};
  const bmoe_status st = norm_spec(spec, &c);
  if (st != BMOE_OK) return st;
  // every gradient has what it is the gradient of, and dn what it came through
  // (arrays of no tokens may be NULL)
  if ((dw_post && !w_post) || (dw_pre && !w_pre) ||
      (T > 0 && ((!u && (du || dgates || w_post)) || (dgates && !gates) ||
                 (w_pre && (!r_out || !dn)) || (!w_pre && (dn || !dr_out)))))
    return BMOE_E_NULL;
  const size_t need = fill ? bmoe_residual_norm_backward_filled_workspace_bytes(dt, T, d, u_rows)
                           : bmoe_residual_norm_backward_workspace_bytes(dt, T, d);
  if (!need) return BMOE_E_SHAPE;  // (u_rows < 0 without u)
  if (!ws || ws_bytes < need) return BMOE_E_WORKSPACE;
  if (!all16({u, inv, gates, r_out, w_post, w_pre, dr_out, dn, du, dgates, dr, dw_post, dw_pre, ws}))
    return BMOE_E_ALIGN;
  const size_t rows = (size_t)T * d * elem(dt), picks = u ? (size_t)T * k * 4 : 0;
  const size_t u_bytes = (size_t)u_rows * d * elem(dt), w_bytes = d * sizeof(float);
  if (!apart({{du, u_bytes}, {dgates, picks}, {dr, rows}, {dw_post, w_bytes}, {dw_pre, w_bytes},
              {ws, need}},
             {{u, u_bytes},
              {inv, picks},
              {gates, picks},
              {r_out, rows},
              {w_post, w_bytes},
              {w_pre, w_bytes},
              {dr_out == dr ? nullptr : dr_out, rows},  // read row by row before it is written
              {dn, rows}}))
    return BMOE_E_VALUE;
  c.T = T;
  c.d = d;
  c.k = k;
  c.M = u_rows;
  c.u = u;
  c.inv = inv;
  c.gates = gates;
  c.w_post = w_post;
  c.w_pre = w_pre;
  c.x = r_out;
  c.dr_out = dr_out;
  c.dn = dn;
  c.du = du;
  c.dr = dr;
  c.dgates = dgates;
  c.dw_post = dw_post;
  c.dw_pre = dw_pre;
  if (fill && du) {
    c.fill = 1;
    c.marks = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + up256(norm_part_bytes(T, d)));
  }
  return status_of(launch_norm_bwd(dt, c, static_cast<float*>(ws), static_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace bmoe

using namespace bmoe;

extern "C" {

size_t bmoe_group_rows_workspace_bytes(int T, int n_experts, int k) {
  if (n_experts < 1 || n_experts > kMaxExperts || k < 1 || T < 0 || (long long)T * k > INT_MAX)
    return 0;
  return up256(group_count_bytes(T * k, n_experts)) + 256;
}

bmoe_status bmoe_group_rows(int T, int n_experts, int k, const int32_t* ids, int32_t* offsets,
                            int32_t* perm, int32_t* inv, void* ws, size_t ws_bytes, void* stream) {
  const size_t need = bmoe_group_rows_workspace_bytes(T, n_experts, k);
  if (!need) return BMOE_E_SHAPE;
  if (!offsets || (T > 0 && (!ids || !perm || !inv))) return BMOE_E_NULL;
  if (!ws || ws_bytes < need) return BMOE_E_WORKSPACE;
  if (!all16({ids, offsets, perm, inv, ws})) return BMOE_E_ALIGN;
  const size_t rows = (size_t)T * k * sizeof(int32_t);
  if (!apart({{offsets, (n_experts + 1) * sizeof(int32_t)}, {perm, rows}, {inv, rows}, {ws, need}},
             {{ids, rows}}))
    return BMOE_E_VALUE;
  return status_of(launch_group_rows(ids, T * k, n_experts, offsets, perm, inv,
                                     static_cast<int*>(ws), static_cast<hipStream_t>(stream)));
}

bmoe_status bmoe_grouped_product(bmoe_dtype dt, int M, int K, int O, int n_groups, const void* a,
                                 int a_rows, const int32_t* perm, int k, const void* w,
                                 const int32_t* offsets, void* c, void* stream) {
  return grouped_product(dt, M, K, O, n_groups, a, a_rows, perm, k, w, offsets, c, false, stream);
}

bmoe_status bmoe_grouped_product_filled(bmoe_dtype dt, int M, int K, int O, int n_groups,
                                        const void* a, int a_rows, const int32_t* perm, int k,
                                        const void* w, const int32_t* offsets, void* c,
                                        void* stream) {
  return grouped_product(dt, M, K, O, n_groups, a, a_rows, perm, k, w, offsets, c, true, stream);
}

size_t bmoe_grouped_product_backward_workspace_bytes(bmoe_dtype dt, int M, int K, int O,
                                                     int n_groups) {
  if (!ok_type(dt) || !grouped_shape(M, K, O, n_groups, nullptr, 1, 1)) return 0;
  const int splits = grouped_dw_splits(dt, M, O, K, n_groups);
  return (splits > 1 ? up256((size_t)splits * n_groups * O * K * sizeof(float)) : 0) + 256;
}

bmoe_status bmoe_grouped_product_backward(bmoe_dtype dt, int M, int K, int O, int n_groups,
                                          const void* a, int a_rows, const int32_t* perm, int k,
                                          const void* w, const int32_t* offsets, const void* dc,
                                          void* da, float* dw, void* ws, size_t ws_bytes,
                                          void* stream) {
  return grouped_product_backward(dt, M, K, O, n_groups, a, a_rows, perm, k, w, offsets, dc, da, dw,
                                  false, ws, ws_bytes, stream);
}

bmoe_status bmoe_grouped_product_backward_filled(bmoe_dtype dt, int M, int K, int O, int n_groups,
                                                 const void* a, int a_rows, const int32_t* perm,
                                                 int k, const void* w, const int32_t* offsets,
                                                 const void* dc, void* da, float* dw, void* ws,
                                                 size_t ws_bytes, void* stream) {
  return grouped_product_backward(dt, M, K, O, n_groups, a, a_rows, perm, k, w, offsets, dc, da, dw,
                                  true, ws, ws_bytes, stream);
}

bmoe_status bmoe_residual_norm(bmoe_dtype dt, int T, int d, int k, const bmoe_norm_spec* spec,
                               const void* u, int u_rows, const int32_t* inv, const float* gates,
                               const void* r, const float* w_post, const float* w_pre, void* r_out,
                               void* n, void* stream) {
  if (!ok_type(dt)) return BMOE_E_DTYPE;
  if (!norm_shape(T, d, k, u_rows, u, inv)) return BMOE_E_SHAPE;
  NormCall c = {};
  const bmoe_status st = norm_spec(spec, &c);
  if (st != BMOE_OK) return st;
  if (T == 0) return BMOE_OK;
  if ((!u && (!r || w_post)) || (w_pre && !n) || ((u || !w_pre) && !r_out)) return BMOE_E_NULL;
  if (!all16({u, inv, gates, r, w_post, w_pre, r_out, n})) return BMOE_E_ALIGN;
  const size_t rows = (size_t)T * d * elem(dt), picks = u ? (size_t)T * k * 4 : 0;
  if (!apart({{r_out, rows}, {w_pre ? n : nullptr, rows}},
             {{u, (size_t)u_rows * d * elem(dt)},
              {inv, picks},
              {gates, picks},
              {r == r_out ? nullptr : r, rows},  // read row by row before it is written
              {w_post, d * sizeof(float)},
              {w_pre, d * sizeof(float)}}) ||
      (r == r_out && w_pre && overlap({n, rows}, {r, rows})))
    return BMOE_E_VALUE;
  c.T = T;
  c.d = d;
  c.k = k;
  c.M = u_rows;
  c.u = u;
  c.inv = inv;
  c.gates = gates;
  c.r = r;
  c.w_post = w_post;
  c.w_pre = w_pre;
  c.r_out = r_out;
  c.n = n;
  return status_of(launch_norm(dt, c, static_cast<hipStream_t>(stream)));
}

size_t bmoe_residual_norm_backward_workspace_bytes(bmoe_dtype dt, int T, int d) {
  if (!ok_type(dt) || T < 0 || d < 1 || d > kMaxNormWidth) return 0;
  return up256(norm_part_bytes(T, d)) + 256;
}

size_t bmoe_residual_norm_backward_filled_workspace_bytes(bmoe_dtype dt, int T, int d, int u_rows) {
  const size_t n = bmoe_residual_norm_backward_workspace_bytes(dt, T, d);
  return n && u_rows >= 0 ? n + up256((size_t)u_rows * sizeof(int32_t)) : 0;
}

bmoe_status bmoe_residual_norm_backward(bmoe_dtype dt, int T, int d, int k,
                                        const bmoe_norm_spec* spec, const void* u, int u_rows,
                                        const int32_t* inv, const float* gates, const void* r_out,
                                        const float* w_post, const float* w_pre,
                                        const void* dr_out, const void* dn, void* du,
                                        float* dgates, void* dr, float* dw_post, float* dw_pre,
                                        void* ws, size_t ws_bytes, void* stream) {
  return norm_backward(dt, T, d, k, spec, u, u_rows, inv, gates, r_out, w_post, w_pre, dr_out, dn,
                       du, dgates, dr, dw_post, dw_pre, false, ws, ws_bytes, stream);
}

bmoe_status bmoe_residual_norm_backward_filled(
    bmoe_dtype dt, int T, int d, int k, const bmoe_norm_spec* spec, const void* u, int u_rows,
    const int32_t* inv, const float* gates, const void* r_out, const float* w_post,
    const float* w_pre, const void* dr_out, const void* dn, void* du, float* dgates, void* dr,
    float* dw_post, float* dw_pre, void* ws, size_t ws_bytes, void* stream) {
  return norm_backward(dt, T, d, k, spec, u, u_rows, inv, gates, r_out, w_post, w_pre, dr_out, dn,
                       du, dgates, dr, dw_post, dw_pre, true, ws, ws_bytes, stream);
}

size_t bmoe_orthogonalize_workspace_bytes(int batch, int rows, int cols) {
  if (batch < 0 || batch > kMaxBatch || rows < 1 || rows > kMaxOrtho || cols < 1 ||
      cols > kMaxOrtho)
    return 0;
  return ortho_workspace_bytes(batch, rows, cols) + 256;
}

bmoe_status bmoe_orthogonalize(bmoe_dtype dt, int batch, int rows, int cols,
                               const bmoe_ortho_spec* spec, const void* u, void* o, void* ws,
                               size_t ws_bytes, void* stream) {
  if (!ok_type(dt)) return BMOE_E_DTYPE;
  const size_t need = bmoe_orthogonalize_workspace_bytes(batch, rows, cols);
  if (!need) return BMOE_E_SHAPE;
  OrthoCall c = {};
  const bmoe_status st = ortho_spec(spec, &c);
  if (st != BMOE_OK) return st;
  if (batch == 0) return BMOE_OK;
  if (!u || !o) return BMOE_E_NULL;
  if (!ws || ws_bytes < need) return BMOE_E_WORKSPACE;
  if (!all16({u, o, ws})) return BMOE_E_ALIGN;
  const size_t bytes = (size_t)batch * rows * cols * elem(dt);
  // o may be u: it is written after u's last reading
  if (!apart({{o, bytes}, {ws, need}}, {{u == o ? nullptr : u, bytes}})) return BMOE_E_VALUE;
  c.batch = batch;
  c.rows = rows;
  c.cols = cols;
  c.u = u;
  c.u_bf16 = dt == BMOE_BF16;
  c.o = o;
  c.o_bf16 = dt == BMOE_BF16;
  return status_of(launch_ortho(c, ws, static_cast<hipStream_t>(stream)));
}

bmoe_status bmoe_orthogonal_step(bmoe_dtype w_dt, bmoe_dtype grad_dt, int batch, int rows, int cols,
                                 const bmoe_ortho_spec* spec, const bmoe_ortho_update* update,
                                 const void* grad, float* momentum, void* w, void* ws,
                                 size_t ws_bytes, void* stream) {
  if (!ok_type(w_dt) || !ok_type(grad_dt)) return BMOE_E_DTYPE;
  const size_t need = bmoe_orthogonalize_workspace_bytes(batch, rows, cols);
  if (!need) return BMOE_E_SHAPE;
  OrthoCall c = {};
  const bmoe_status st = ortho_spec(spec, &c);
  if (st != BMOE_OK) return st;
  if (!update) return BMOE_E_NULL;
  if (!(update->beta >= 0.f && update->beta < 1.f) || !std::isfinite(update->lr) ||
      !std::isfinite(update->weight_decay) || !std::isfinite(update->scale))
    return BMOE_E_VALUE;
  if (batch == 0) return BMOE_OK;
  if (!grad || !momentum || !w) return BMOE_E_NULL;
  if (!ws || ws_bytes < need) return BMOE_E_WORKSPACE;
  if (!all16({grad, momentum, w, ws})) return BMOE_E_ALIGN;
  const size_t n = (size_t)batch * rows * cols;
  if (!apart({{momentum, n * sizeof(float)}, {w, n * elem(w_dt)}, {ws, need}},
             {{grad, n * elem(grad_dt)}}))
    return BMOE_E_VALUE;
  c.batch = batch;
  c.rows = rows;
  c.cols = cols;
  c.u = grad;
  c.u_bf16 = grad_dt == BMOE_BF16;
  c.momentum = momentum;
  c.beta = update->beta;
  c.nesterov = update->nesterov != 0;
  c.o = w;
  c.o_bf16 = w_dt == BMOE_BF16;
  c.update = 1;
  c.keep = (float)(1.0 - (double)update->lr * update->weight_decay);
  c.rate = (float)((double)update->lr * update->scale);
  return status_of(launch_ortho(c, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
