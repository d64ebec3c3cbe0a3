// Norms around a block, fused with the sum of its expert rows, its gates and
// its scaled residual. For token t, all sums in fp32:
//   y = sum over j of g_tj u[row(t, j)]          (ascending j)
//   z = y * rsqrt(mean y^2 + eps) * w_post        (w_post NULL: z = y)
//   r' = res_scale r + out_scale z                (stored rounded)
//   n = r' * rsqrt(mean r'^2 + eps) * w_pre       (of the unrounded r')
// and its gradient from dr', dn, with r' as stored, q = rsqrt(mean v^2 + eps):
//   D(v, w, d) = q (w d - v q^2 mean(w d v)),   dw = sum over t of d v q
//   dr'' = dr' + D(r', w_pre, dn);  dr = res_scale dr'';  dz = out_scale dr''
//   dy = D(y, w_post, dz);  du = g dy;  dg = <dy, u>
//
// Bound by HBM: each array is read or written once (the gradient reads u a
// second time, out of L2, because dy needs sums over the row). A row belongs to
// TPR threads (a wave, or a whole workgroup), a thread to EPC * NV of its
// values, held in registers between the sums.
#include "common.h"
#include "kernels.h"

namespace bmoe {
namespace {

constexpr int kThreads = 256;

template <typename T_, int TPR_, int NV_, bool ALIGNED_>
struct NormCfg {
  using T = T_;
  static constexpr int TPR = TPR_, NV = NV_;     // threads per row, chunks per thread
  static constexpr bool ALIGNED = ALIGNED_;      // rows of whole 16-byte chunks
  static constexpr int EPC = 16 / sizeof(T);     // values per chunk
  static constexpr int VALS = EPC * NV;
  static constexpr int THREADS = TPR > kThreads ? TPR : kThreads;
  static constexpr int ROWS = THREADS / TPR;     // per workgroup
};

__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const uint16_t* p) { return bf16_lo(*p); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16_bits(v); }

// This thread's values of a row of d: chunks lane, lane + TPR, ... (zeros past d).
template <class C>
__device__ __forceinline__ void load_row(const typename C::T* row, int d, int lane,
                                         float (&v)[C::VALS]) {
#pragma unroll
  for (int i = 0; i < C::NV; ++i) {
    const int c = (i * C::TPR + lane) * C::EPC;
    if constexpr (C::ALIGNED) {
      if (c < d) {
        load16(row + c, v + i * C::EPC);
      } else {
#pragma unroll
        for (int e = 0; e < C::EPC; ++e) v[i * C::EPC + e] = 0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < C::EPC; ++e) v[i * C::EPC + e] = c + e < d ? get(row + c + e) : 0.f;
    }
  }
}
template <class C>
__device__ __forceinline__ void store_row(typename C::T* row, int d, int lane,
                                          const float (&v)[C::VALS], float scale) {
#pragma unroll
  for (int i = 0; i < C::NV; ++i) {
    const int c = (i * C::TPR + lane) * C::EPC;
    if constexpr (C::ALIGNED) {
      if (c < d) store16(v + i * C::EPC, row + c, scale);
    } else {
#pragma unroll
      for (int e = 0; e < C::EPC; ++e)
        if (c + e < d) put(row + c + e, v[i * C::EPC + e] * scale);
    }
  }
}
// fp32 weights, the same columns.
template <class C>
__device__ __forceinline__ void load_weight(const float* w, int d, int lane, float (&v)[C::VALS]) {
#pragma unroll
  for (int i = 0; i < C::NV; ++i) {
    const int c = (i * C::TPR + lane) * C::EPC;
#pragma unroll
    for (int e = 0; e < C::EPC; e += 4) {
      if (C::ALIGNED || c + e + 3 < d) {
        if (c < d) {
          load16(w + c + e, v + i * C::EPC + e);
          continue;
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) v[i * C::EPC + e + x] = c + e + x < d ? w[c + e + x] : 0.f;
    }
  }
}

// Sums of N values over the TPR threads of a row, the same in all of them.
// lds: N floats per wave.
template <class C, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* lds) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v[i] += __shfl_xor(v[i], o, 64);
  if constexpr (C::TPR > kWave) {
    constexpr int W = C::TPR / kWave;
    const int wave = threadIdx.x / kWave;
    __syncthreads();  // the last sums have been read
    if (threadIdx.x % kWave == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) lds[wave * N + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += lds[w * N + i];
      v[i] = s;
    }
  }
}

// Row of u that holds pick j of token t, or -1.
__device__ __forceinline__ long long u_row(const NormCall& p, int t, int j) {
  const long long at = (long long)t * p.k + j;
  const long long row = p.inv ? p.inv[at] : at;
  return row >= 0 && row < p.M ? row : -1;
}

// y of token t.
template <class C>
__device__ __forceinline__ void sum_picks(const NormCall& p, int t, int lane, float (&y)[C::VALS]) {
#pragma unroll
  for (int e = 0; e < C::VALS; ++e) y[e] = 0.f;
  const typename C::T* u = static_cast<const typename C::T*>(p.u);
  for (int j = 0; j < p.k; ++j) {
    const long long row = u_row(p, t, j);
    if (row < 0) continue;  // a padded pick, the same in the whole row
    const float g = p.gates ? p.gates[(long long)t * p.k + j] : 1.f;
    float v[C::VALS];
    load_row<C>(u + (size_t)row * p.d, p.d, lane, v);
#pragma unroll
    for (int e = 0; e < C::VALS; ++e) y[e] = fmaf(g, v[e], y[e]);
  }
}

__device__ __forceinline__ float rstd_of(float sum_sq, int d, float eps) {
  return 1.f / sqrtf(sum_sq / (float)d + eps);
}

template <class C>
__global__ __launch_bounds__(C::THREADS) void norm_kernel(NormCall p) {
  __shared__ float lds[C::THREADS / kWave];
  using T = typename C::T;
  const int lane = threadIdx.x % C::TPR;
  const long long t64 = (long long)blockIdx.x * C::ROWS + threadIdx.x / C::TPR;
  if (t64 >= p.T) return;  // a whole wave; whole workgroups where rows are theirs
  const int t = (int)t64;
  const size_t at = (size_t)t * p.d;
  float r[C::VALS];
  if (p.r) {
    load_row<C>(static_cast<const T*>(p.r) + at, p.d, lane, r);
#pragma unroll
    for (int e = 0; e < C::VALS; ++e) r[e] *= p.res_scale;
  } else {
#pragma unroll
    for (int e = 0; e < C::VALS; ++e) r[e] = 0.f;
  }
  if (p.u) {
    float y[C::VALS];
    sum_picks<C>(p, t, lane, y);
    if (p.w_post) {
      float w[C::VALS], s[1] = {0.f};
      load_weight<C>(p.w_post, p.d, lane, w);
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) s[0] = fmaf(y[e], y[e], s[0]);
      row_sum<C, 1>(s, lds);
      const float q = rstd_of(s[0], p.d, p.eps);
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) y[e] = y[e] * q * w[e];
    }
#pragma unroll
    for (int e = 0; e < C::VALS; ++e) r[e] = fmaf(p.out_scale, y[e], r[e]);
  }
  if (p.r_out) store_row<C>(static_cast<T*>(p.r_out) + at, p.d, lane, r, 1.f);
  if (p.w_pre) {
    float w[C::VALS], s[1] = {0.f};
    load_weight<C>(p.w_pre, p.d, lane, w);
#pragma unroll
    for (int e = 0; e < C::VALS; ++e) s[0] = fmaf(r[e], r[e], s[0]);
    row_sum<C, 1>(s, lds);
    const float q = rstd_of(s[0], p.d, p.eps);
#pragma unroll
    for (int e = 0; e < C::VALS; ++e) r[e] = r[e] * q * w[e];
    store_row<C>(static_cast<T*>(p.n) + at, p.d, lane, r, 1.f);
  }
}

// One workgroup takes ROWS tokens at a time, `gridDim.x` apart, and keeps the
// weights' gradients of its columns in registers; they end as partial sums
// part[side][workgroup][d], added in order by a second launch.
template <class C>
__global__ __launch_bounds__(C::THREADS) void norm_bwd_kernel(NormCall p, float* part) {
  __shared__ float lds[3 * (C::THREADS / kWave)];
  __shared__ float fold[C::ROWS > 1 ? C::ROWS * C::TPR * C::VALS : 1];
  using T = typename C::T;
  const int lane = threadIdx.x % C::TPR, sub = threadIdx.x / C::TPR;
  float dpre[C::VALS], dpost[C::VALS];
#pragma unroll
  for (int e = 0; e < C::VALS; ++e) dpre[e] = dpost[e] = 0.f;
  for (long long t0 = (long long)blockIdx.x * C::ROWS; t0 < p.T;
       t0 += (long long)gridDim.x * C::ROWS) {
    if (t0 + sub >= p.T) continue;  // whole waves (ROWS > 1 needs no barrier here)
    const int t = (int)(t0 + sub);
    const size_t at = (size_t)t * p.d;
    float dr[C::VALS], y[C::VALS];
    if (p.u) {
      sum_picks<C>(p, t, lane, y);
    } else {
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) y[e] = 0.f;
    }
    if (p.dr_out) {
      load_row<C>(static_cast<const T*>(p.dr_out) + at, p.d, lane, dr);
    } else {
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) dr[e] = 0.f;
    }
    float s[3] = {0.f, 0.f, 0.f};  // r'^2, w_pre dn r', y^2
#pragma unroll
    for (int e = 0; e < C::VALS; ++e) s[2] = fmaf(y[e], y[e], s[2]);
    if (p.w_pre) {
      float x[C::VALS], dn[C::VALS], w[C::VALS];
      load_row<C>(static_cast<const T*>(p.x) + at, p.d, lane, x);
      load_row<C>(static_cast<const T*>(p.dn) + at, p.d, lane, dn);
      load_weight<C>(p.w_pre, p.d, lane, w);
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) {
        s[0] = fmaf(x[e], x[e], s[0]);
        s[1] = fmaf(w[e] * dn[e], x[e], s[1]);
      }
      row_sum<C, 3>(s, lds);
      const float q = rstd_of(s[0], p.d, p.eps), m = s[1] / (float)p.d * q * q;
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) {
        dpre[e] = fmaf(dn[e], x[e] * q, dpre[e]);
        dr[e] = fmaf(q, w[e] * dn[e] - x[e] * m, dr[e]);
      }
    } else if (p.w_post) {
      row_sum<C, 3>(s, lds);
    }
    if (p.dr) store_row<C>(static_cast<T*>(p.dr) + at, p.d, lane, dr, p.res_scale);
    if (!p.u) continue;
    // dr becomes dz, then dy
#pragma unroll
    for (int e = 0; e < C::VALS; ++e) dr[e] *= p.out_scale;
    if (p.w_post) {
      float w[C::VALS], b[1] = {0.f};
      load_weight<C>(p.w_post, p.d, lane, w);
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) b[0] = fmaf(w[e] * dr[e], y[e], b[0]);
      row_sum<C, 1>(b, lds);
      const float q = rstd_of(s[2], p.d, p.eps), m = b[0] / (float)p.d * q * q;
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) {
        dpost[e] = fmaf(dr[e], y[e] * q, dpost[e]);
        dr[e] = q * (w[e] * dr[e] - y[e] * m);
      }
    }
    for (int j = 0; j < p.k; ++j) {
      const long long row = u_row(p, t, j), pick = (long long)t * p.k + j;
      float dg[1] = {0.f};
      if (row >= 0) {
        if (p.du)
          store_row<C>(static_cast<T*>(p.du) + (size_t)row * p.d, p.d, lane, dr,
                       p.gates ? p.gates[pick] : 1.f);
        if (p.dgates) {
          float v[C::VALS];
          load_row<C>(static_cast<const T*>(p.u) + (size_t)row * p.d, p.d, lane, v);
#pragma unroll
          for (int e = 0; e < C::VALS; ++e) dg[0] = fmaf(dr[e], v[e], dg[0]);
        }
      }
      if (p.dgates) {
        row_sum<C, 1>(dg, lds);
        if (lane == 0) p.dgates[pick] = dg[0];
      }
    }
  }
  // the partial sums of this workgroup, rows of it added in order
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (!(side ? p.dw_post : p.dw_pre)) continue;
    float* out = part + ((size_t)side * gridDim.x + blockIdx.x) * p.d;
    float(&v)[C::VALS] = side ? dpost : dpre;
    if constexpr (C::ROWS > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) fold[(sub * C::VALS + e) * C::TPR + lane] = v[e];
      __syncthreads();
      if (sub == 0) {
#pragma unroll
        for (int e = 0; e < C::VALS; ++e) {
          float s = v[e];
#pragma unroll
          for (int w = 1; w < C::ROWS; ++w) s += fold[(w * C::VALS + e) * C::TPR + lane];
          v[e] = s;
        }
      }
    }
    if (sub == 0) {
#pragma unroll
      for (int i = 0; i < C::NV; ++i) {
        const int c = (i * C::TPR + lane) * C::EPC;
#pragma unroll
        for (int e = 0; e < C::EPC; ++e)
          if (c + e < p.d) out[c + e] = v[i * C::EPC + e];
      }
    }
  }
}

// dw[c] = the partial sums of column c, in order: 64 columns a workgroup, four
// waves taking a quarter of the parts each.
__global__ __launch_bounds__(kThreads) void norm_weights_kernel(const float* part, int parts, int d,
                                                                float* dw_pre, float* dw_post) {
  __shared__ float lds[kThreads];
  float* dst = blockIdx.y ? dw_post : dw_pre;
  if (!dst) return;
  const int col = blockIdx.x * 64 + threadIdx.x % 64, q = threadIdx.x / 64;
  const int n = (parts + 3) / 4, lo = q * n, hi = min(parts, lo + n);
  float s = 0.f;
  if (col < d) {
    const float* src = part + (size_t)blockIdx.y * parts * d + col;
#pragma unroll 8
    for (int i = lo; i < hi; ++i) s += src[(size_t)i * d];
  }
  lds[threadIdx.x] = s;
  __syncthreads();
  if (q == 0 && col < d)
    dst[col] = ((s + lds[64 + threadIdx.x]) + lds[128 + threadIdx.x]) + lds[192 + threadIdx.x];
}

// Workgroups of the gradient: enough rows each that their partial sums stay few.
constexpr int kBwdGroups = 1024;

template <class C>
hipError_t launch_norm_cfg(const NormCall& c, hipStream_t s) {
  const size_t groups = ((size_t)c.T + C::ROWS - 1) / C::ROWS;
  return launch_kernel(norm_kernel<C>, dim3((unsigned)groups), dim3(C::THREADS), 0, s,
                       KernelTiming{}, c);
}
template <class C>
hipError_t launch_norm_bwd_cfg(const NormCall& c, float* part, hipStream_t s) {
  const size_t want = ((size_t)c.T + C::ROWS - 1) / C::ROWS;
  const int groups = (int)(want < kBwdGroups ? want : kBwdGroups);  // T = 0: no sums, dw = 0
  const hipError_t e = groups ? launch_kernel(norm_bwd_kernel<C>, dim3(groups), dim3(C::THREADS), 0,
                                              s, KernelTiming{}, c, part)
                              : hipSuccess;
  if (e != hipSuccess || (!c.dw_pre && !c.dw_post)) return e;
  return launch_kernel(norm_weights_kernel, dim3((c.d + 63) / 64, 2), dim3(kThreads), 0, s,
                       KernelTiming{}, (const float*)part, groups, c.d, c.dw_pre, c.dw_post);
}

// f(config) for rows of d values: a wave per row up to 1024 values (fp32: 512),
// 256 threads up to 4096 (2048), 1024 threads to 8192.
template <typename T, bool ALIGNED, typename F>
hipError_t with_width(int d, F f) {
  constexpr int EPC = 16 / sizeof(T);
  if (d <= 64 * EPC) return f(NormCfg<T, 64, 1, ALIGNED>{});
  if (d <= 128 * EPC) return f(NormCfg<T, 64, 2, ALIGNED>{});
  if (d <= 256 * EPC) return f(NormCfg<T, 256, 1, ALIGNED>{});
  if (d <= 512 * EPC) return f(NormCfg<T, 256, 2, ALIGNED>{});
  return f(NormCfg<T, 1024, sizeof(T) / 2, ALIGNED>{});
}
template <typename F>
hipError_t with_cfg(bmoe_dtype dt, int d, F f) {
  if (dt == BMOE_BF16)
    return d % 8 == 0 ? with_width<uint16_t, true>(d, f) : with_width<uint16_t, false>(d, f);
  return d % 4 == 0 ? with_width<float, true>(d, f) : with_width<float, false>(d, f);
}

}  // namespace

size_t norm_part_bytes(int T, int d) {
  const size_t groups = T < kBwdGroups ? T : kBwdGroups;
  return 2 * groups * d * sizeof(float);
}

hipError_t launch_norm(bmoe_dtype dt, const NormCall& c, hipStream_t s) {
  return with_cfg(dt, c.d, [&](auto cfg) { return launch_norm_cfg<decltype(cfg)>(c, s); });
}

hipError_t launch_norm_bwd(bmoe_dtype dt, const NormCall& c, float* part, hipStream_t s) {
  return with_cfg(dt, c.d, [&](auto cfg) { return launch_norm_bwd_cfg<decltype(cfg)>(c, part, s); });
}

}  // namespace bmoe
