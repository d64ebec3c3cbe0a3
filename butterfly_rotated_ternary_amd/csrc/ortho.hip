// Orthogonalisation of matrices by Newton-Schulz products, and the weight
// update that uses it:
//   X_0 = U / (|U|_F + eps),   P = X X^T,  Q = a I + b P + c P P,  X <- Q X
// `steps` times (P = X^T X and X <- X Q for matrices with more rows than
// columns, so P is always the smaller one). An odd polynomial of X moves its
// singular values and leaves its singular vectors.
//
// Numbers. Operands are kept as pairs of fp16, hi + lo, of the value times
// 2^12: 22 bits where a value is above 2^-14 of 1 after that scaling, an
// absolute error of 2^-37 below. The singular values stay below 16 (checked on
// the host for the given coefficients), so no scaled value passes 2^16. Three
// fp16 MFMAs (hi hi + hi lo + lo hi, fp32 sums) make one product of about fp32's
// accuracy at five times the rate that fp32 MFMAs have. The normalising sums are
// in 64 bits.
//
// P and Q are symmetric: only tiles on and below the diagonal are computed,
// each written twice. Rows are padded to whole 16-byte chunks (zeros).
#include "common.h"
#include "kernels.h"
#include "tile_product.h"

namespace bmoe {
namespace {

using namespace tile;

constexpr float kScale = 4096.f;  // of all fp16 operands

// What U is: u itself, or the momentum of a step (grad added to it).
struct Source {
  const void* u;       // or the gradient, [batch][rows][cols]
  float* momentum;     // NULL: u itself
  float beta;
  int nesterov, bf16;  // type of u
};

__device__ __forceinline__ float load_any(const void* p, int bf16, size_t i) {
  return bf16 ? bf16_lo(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}
// U's entry i once the momentum holds its new value m.
__device__ __forceinline__ float mixed(const Source& s, float g, float m) {
  return s.nesterov ? fmaf(s.beta, m, g) : m;
}

// ---- the norm (and the momentum's step) ----------------------------------------
constexpr int kSumThreads = 256;
constexpr int kSumParts = 256;  // workgroups per matrix, at most

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kSumThreads / 64; ++w) s += lds[w];
  return s;
}

__global__ __launch_bounds__(kSumThreads) void ortho_sum_kernel(Source src, size_t count,
                                                                double* part) {
  __shared__ double lds[kSumThreads / 64];
  const size_t first = (size_t)blockIdx.y * count;
  double acc = 0.0;
  for (size_t i = (size_t)blockIdx.x * kSumThreads + threadIdx.x; i < count;
       i += (size_t)gridDim.x * kSumThreads) {
    float u = load_any(src.u, src.bf16, first + i);
    if (src.momentum) {
      const float m = fmaf(src.beta, src.momentum[first + i], u);
      src.momentum[first + i] = m;
      u = mixed(src, u, m);
    }
    acc = fma((double)u, (double)u, acc);
  }
  const double s = block_sum(acc, lds);
  if (threadIdx.x == 0) part[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// A value times kScale as its two fp16 parts.
__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo) {
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
}

// ---- X_0 -----------------------------------------------------------------------
__global__ __launch_bounds__(kSumThreads) void ortho_split_kernel(Source src, int rows, int cols,
                                                                  int ld, float eps,
                                                                  const double* part, int parts,
                                                                  _Float16* hi, _Float16* lo) {
  __shared__ double lds[kSumThreads / 64];
  const double* mine = part + (size_t)blockIdx.y * parts;
  double acc = 0.0;
  for (int i = threadIdx.x; i < parts; i += kSumThreads) acc += mine[i];
  const float norm = (float)sqrt(block_sum(acc, lds)) + eps;
  const size_t in0 = (size_t)blockIdx.y * rows * cols, out0 = (size_t)blockIdx.y * rows * ld;
  const size_t n = (size_t)rows * ld;
  for (size_t i = (size_t)blockIdx.x * kSumThreads + threadIdx.x; i < n;
       i += (size_t)gridDim.x * kSumThreads) {
    const size_t row = i / ld;
    const int col = (int)(i % ld);
    float v = 0.f;
    if (col < cols) {
      const size_t at = in0 + row * cols + col;
      v = load_any(src.u, src.bf16, at);
      if (src.momentum) v = mixed(src, v, src.momentum[at]);
      v = v / norm * kScale;
    }
    split(v, hi[out0 + i], lo[out0 + i]);
  }
}

// ---- the products ----------------------------------------------------------------
enum Product { kGram, kPoly, kApply };

struct OrthoArgs {
  const _Float16 *x, *q;  // operands: hi parts, lo parts behind them
  size_t x_part, q_part;  // bytes between an operand's parts
  _Float16* out;          // hi part (kApply's last: NULL)
  size_t out_part;        // elements
  int rows, cols, ld, m, ldm;  // of X; of P and Q
  int batch, tiles, tiles_n;  // tiles per matrix
  float a, b, c;          // kPoly
  // the last product's epilogue
  void* o;                // [batch][rows][cols]: X, or w = keep w - rate X
  int o_bf16, update;
  float keep, rate;
};

__device__ __forceinline__ int2 triangle(int t) {
  int i = (int)((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  while (i * (i + 1) / 2 > t) --i;
  return make_int2(i, t - i * (i + 1) / 2);
}

template <class C, int PRODUCT, bool TALL>
__global__ __launch_bounds__(C::THREADS) void ortho_product_kernel(OrthoArgs p) {
  __shared__ __attribute__((aligned(1024))) char st0[C::STAGE];
  __shared__ __attribute__((aligned(1024))) char st1[C::STAGE];
  static_assert(C::NSTAGE == 2, "two stages");
  char* ring[2] = {st0, st1};
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int batch = grid_block() / p.tiles, t = grid_block() % p.tiles;
  if (batch >= p.batch) return;
  int2 tile;
  if constexpr (PRODUCT == kApply) tile = make_int2(t / p.tiles_n, t % p.tiles_n);
  else tile = triangle(t);
  const int r0 = tile.x * C::BM, c0 = tile.y * C::BN;
  const char* x = reinterpret_cast<const char*>(p.x) + (size_t)batch * p.rows * p.ld * 2;
  const char* q = reinterpret_cast<const char*>(p.q) + (size_t)batch * p.m * p.ldm * 2;
  const size_t x_ld = (size_t)p.ld * 2, q_ld = (size_t)p.ldm * 2;

  Acc<C> acc;
  clear<C>(acc);
  Reader<C, C::AMODE, C::BM, C::FM> ra;
  ra.init(wm * C::TM, lane);
  Reader<C, C::BMODE, C::BN, C::FN> rb;
  rb.init(wn * C::TN, lane);
  // chunks of a row beyond its values are zeros in memory up to ld (ldm)
  if constexpr (PRODUCT == kGram && TALL) {  // X^T X: down the rows of X
    RedRowsSource<C, C::BM, C::A_LOADS, SameRow> a;
    a.init(x, x_ld, r0, p.ld, p.rows, p.x_part, SameRow{}, lane, wave);
    RedRowsSource<C, C::BN, C::B_LOADS, SameRow> b;
    b.init(x, x_ld, c0, p.ld, p.rows, p.x_part, SameRow{}, lane, wave);
    run<C>(acc, ring, a, b, ra, rb, (p.rows + C::BK - 1) / C::BK, lane, wave);
  } else if constexpr (PRODUCT == kGram || PRODUCT == kPoly) {  // X X^T, P P = P P^T
    const char* src = PRODUCT == kGram ? x : q;
    const size_t ld = PRODUCT == kGram ? x_ld : q_ld;
    const int red = PRODUCT == kGram ? p.ld : p.ldm;
    const size_t part = PRODUCT == kGram ? p.x_part : p.q_part;
    OutRowsSource<C, C::BM, C::A_LOADS> a;
    a.init([&](int r) { return src + (size_t)min(r0 + r, p.m - 1) * ld; }, red, part, lane, wave);
    OutRowsSource<C, C::BN, C::B_LOADS> b;
    b.init([&](int r) { return src + (size_t)min(c0 + r, p.m - 1) * ld; }, red, part, lane, wave);
    run<C>(acc, ring, a, b, ra, rb, (red + C::BK - 1) / C::BK, lane, wave);
  } else if constexpr (TALL) {  // X Q: Q symmetric, its rows serve as columns
    OutRowsSource<C, C::BM, C::A_LOADS> a;
    a.init([&](int r) { return x + (size_t)min(r0 + r, p.rows - 1) * x_ld; }, p.ldm, p.x_part, lane,
           wave);
    OutRowsSource<C, C::BN, C::B_LOADS> b;
    b.init([&](int r) { return q + (size_t)min(c0 + r, p.m - 1) * q_ld; }, p.ldm, p.q_part, lane,
           wave);
    run<C>(acc, ring, a, b, ra, rb, (p.ldm + C::BK - 1) / C::BK, lane, wave);
  } else {  // Q X
    OutRowsSource<C, C::BM, C::A_LOADS> a;
    a.init([&](int r) { return q + (size_t)min(r0 + r, p.m - 1) * q_ld; }, p.m, p.q_part, lane,
           wave);
    RedRowsSource<C, C::BN, C::B_LOADS, SameRow> b;
    b.init(x, x_ld, c0, p.ld, p.m, p.x_part, SameRow{}, lane, wave);
    run<C>(acc, ring, a, b, ra, rb, (p.m + C::BK - 1) / C::BK, lane, wave);
  }

  const int out_rows = PRODUCT == kApply ? p.rows : p.m;
  const int out_cols = PRODUCT == kApply ? p.cols : p.m;
  const int out_ld = PRODUCT == kApply ? p.ld : p.ldm;
  _Float16* hi = p.out + (size_t)batch * out_rows * out_ld;
  _Float16* lo = hi + p.out_part;
  const _Float16* ph = reinterpret_cast<const _Float16*>(q);
  const _Float16* pl = reinterpret_cast<const _Float16*>(q + p.q_part);
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      const int col = c0 + wn * C::TN + 32 * j + acc_col(lane);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int row = r0 + wm * C::TM + 32 * i + acc_row(4 * g, lane);  // and three more
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = acc[i][j][4 * g + u] * (1.f / kScale);
        if constexpr (PRODUCT == kPoly) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float pv = 0.f;
            if (row + u < p.m && col < p.m) {
              const size_t at = (size_t)(row + u) * p.ldm + col;
              pv = (float)ph[at] + (float)pl[at];
            }
            v[u] = fmaf(p.c, v[u], p.b * pv) + (row + u == col ? p.a * kScale : 0.f);
          }
        }
        if (PRODUCT == kApply && p.o) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (row + u >= out_rows || col >= out_cols) continue;
            const size_t at = ((size_t)batch * out_rows + row + u) * out_cols + col;
            float o = v[u] * (1.f / kScale);
            if (p.update) o = fmaf(p.keep, load_any(p.o, p.o_bf16, at), -p.rate * o);
            if (p.o_bf16) static_cast<uint16_t*>(p.o)[at] = (uint16_t)f32_to_bf16_bits(o);
            else static_cast<float*>(p.o)[at] = o;
          }
          continue;
        }
        _Float16 h[4], l[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          split(col < out_cols ? v[u] : 0.f, h[u], l[u]);
          if (row + u < out_rows && col < out_ld) {
            const size_t at = (size_t)(row + u) * out_ld + col;
            hi[at] = h[u];
            lo[at] = l[u];
          }
        }
        if constexpr (PRODUCT != kApply) {
          // the mirrored tile: four consecutive columns of row `col`. (out_ld is
          // a multiple of 4, so four from a multiple of 4 are in or out whole;
          // their values past out_rows are the padding's zeros.)
          if (tile.x != tile.y && col < out_cols && row < out_ld) {
            typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
            f16x4 hv, lv;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              hv[u] = row + u < out_rows ? h[u] : (_Float16)0.f;
              lv[u] = row + u < out_rows ? l[u] : (_Float16)0.f;
            }
            const size_t at = (size_t)col * out_ld + row;
            *reinterpret_cast<f16x4*>(hi + at) = hv;
            *reinterpret_cast<f16x4*>(lo + at) = lv;
          }
        }
      }
    }
}

template <int AMODE, int BMODE>
using Tile = Cfg<kF16, 2, 128, 128, 2, 2, 2, AMODE, BMODE, true>;

template <int PRODUCT, bool TALL, int AMODE, int BMODE>
hipError_t launch_product_cfg(OrthoArgs p, hipStream_t s) {
  using C = Tile<AMODE, BMODE>;
  const int tm = ((PRODUCT == kApply ? p.rows : p.m) + C::BM - 1) / C::BM;
  p.tiles_n = ((PRODUCT == kApply ? p.cols : p.m) + C::BN - 1) / C::BN;
  p.tiles = PRODUCT == kApply ? tm * p.tiles_n : tm * (tm + 1) / 2;
  return launch_kernel(ortho_product_kernel<C, PRODUCT, TALL>,
                       grid_rows((size_t)p.tiles * p.batch), dim3(C::THREADS), 0, s, KernelTiming{},
                       p);
}

int padded(int n) { return (n + 7) / 8 * 8; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Layout {
  size_t part, x0, x1, p, q, total;  // byte offsets
  size_t x_part, p_part;             // bytes of one part
  int ld, m, ldm;
};
Layout layout(int batch, int rows, int cols) {
  Layout l;
  l.ld = padded(cols);
  l.m = rows < cols ? rows : cols;
  l.ldm = padded(l.m);
  l.x_part = up256((size_t)batch * rows * l.ld * 2);
  l.p_part = up256((size_t)batch * l.m * l.ldm * 2);
  l.part = 0;
  l.x0 = up256((size_t)batch * kSumParts * sizeof(double));
  l.x1 = l.x0 + 2 * l.x_part;
  l.p = l.x1 + 2 * l.x_part;
  l.q = l.p + 2 * l.p_part;
  l.total = l.q + 2 * l.p_part;
  return l;
}

}  // namespace

size_t ortho_workspace_bytes(int batch, int rows, int cols) {
  return layout(batch, rows, cols).total;
}

hipError_t launch_ortho(const OrthoCall& call, void* ws, hipStream_t s) {
  const int batch = call.batch, rows = call.rows, cols = call.cols;
  const Layout l = layout(batch, rows, cols);
  char* base = static_cast<char*>(ws);
  double* part = reinterpret_cast<double*>(base + l.part);
  Source src;
  src.u = call.u;
  src.momentum = call.momentum;
  src.beta = call.beta;
  src.nesterov = call.nesterov;
  src.bf16 = call.u_bf16;
  const size_t count = (size_t)rows * cols;
  const size_t want = (count + 4 * kSumThreads - 1) / (4 * kSumThreads);
  const int parts = (int)(want < kSumParts ? want : kSumParts);
  hipError_t e = launch_kernel(ortho_sum_kernel, dim3(parts, batch), dim3(kSumThreads), 0, s,
                               KernelTiming{}, src, count, part);
  if (e != hipSuccess) return e;
  _Float16* x[2] = {reinterpret_cast<_Float16*>(base + l.x0),
                    reinterpret_cast<_Float16*>(base + l.x1)};
  const size_t padded_count = (size_t)rows * l.ld;
  const size_t blocks = (padded_count + 4 * kSumThreads - 1) / (4 * kSumThreads);
  e = launch_kernel(ortho_split_kernel, dim3((unsigned)(blocks < 2048 ? blocks : 2048), batch),
                    dim3(kSumThreads), 0, s, KernelTiming{}, src, rows, cols, l.ld, call.eps,
                    (const double*)part, parts, x[0], x[0] + l.x_part / 2);
  if (e != hipSuccess) return e;

  _Float16* P = reinterpret_cast<_Float16*>(base + l.p);
  _Float16* Q = reinterpret_cast<_Float16*>(base + l.q);
  OrthoArgs p;
  p.batch = batch;
  p.rows = rows;
  p.cols = cols;
  p.ld = l.ld;
  p.m = l.m;
  p.ldm = l.ldm;
  p.x_part = l.x_part;
  p.q_part = l.p_part;
  p.a = call.a;
  p.b = call.b;
  p.c = call.c;
  p.o_bf16 = call.o_bf16;
  p.update = call.update;
  p.keep = call.keep;
  p.rate = call.rate;
  p.tiles = p.tiles_n = 0;
  const bool tall = rows > cols;
  for (int i = 0; i < call.steps; ++i) {
    p.x = x[i & 1];
    p.o = nullptr;
    p.q = nullptr;
    p.out = P;
    p.out_part = l.p_part / 2;
    e = tall ? launch_product_cfg<kGram, true, kRedRows, kRedRows>(p, s)
             : launch_product_cfg<kGram, false, kOutRows, kOutRows>(p, s);
    if (e != hipSuccess) return e;
    p.q = P;
    p.out = Q;
    e = launch_product_cfg<kPoly, false, kOutRows, kOutRows>(p, s);
    if (e != hipSuccess) return e;
    p.q = Q;
    p.out = x[(i + 1) & 1];
    p.out_part = l.x_part / 2;
    if (i + 1 == call.steps) p.o = call.o;
    e = tall ? launch_product_cfg<kApply, true, kOutRows, kOutRows>(p, s)
             : launch_product_cfg<kApply, false, kOutRows, kRedRows>(p, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace bmoe
