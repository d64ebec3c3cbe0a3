// Orthogonalisation of matrices by Newton-Schulz products, and the weight
// update that uses it:
//   X_0 = U / (|U|_F + eps),   P = X X^T,  Q = a I + b P + c P P,  X <- Q X
// `steps` times (P = X^T X and X <- X Q for matrices with more rows than
// columns, so P is always the smaller one). An odd polynomial of X moves its
// singular values and leaves its singular vectors.
//
// Numbers. Operands are kept as pairs of fp16, hi + lo, of the value times a power
// of two: the largest that leaves room for what X, P and Q can hold under the given
// coefficients (the host bounds their singular values; X and P share one; for 3.4445,
// -4.7750, 2.0315 2^15, and 2^14 for Q). That is 22 bits of a value above 2^-18, and an
// absolute error of 2^-40 (2^-39) below. Three fp16 MFMAs (hi hi + hi lo + lo hi,
// fp32 sums) make one product at five times the rate that fp32 MFMAs have. In the
// norm the result is as near to the exact one as an iteration in fp32 (64 x 512
// normal entries 1.5e-6 and 1.7e-6 off); a row or column far below the others meets
// the absolute error: with rows from 1 down to 1e-6 the smallest is 2e-5 (64 x 512) to
// 1e-4 (600 x 1500) off by itself, fp32 4e-6 to 2e-5. (One scale of 2^12 for all:
// 1.6e-4 to 8e-4.) The normalising sums are in 64 bits.
//
// P and Q are symmetric: only tiles on and below the diagonal are computed,
// each written twice. Rows are padded to whole 16-byte chunks (zeros).
//
// Bound by the matrix units where a side is long: 4096 x 4096, five steps, 3.6 to 3.8
// ms by the card (P 210, Q 200, X 320 us a step; 70, 70 and 81 % of the MFMA cycles).
// 64 matrices 1024 x 512, 1.31 to 1.43 ms: reductions of 512 and 1024 are 16 to 32
// steps, so each round of tiles spends as long filling its ring and storing as
// multiplying (P 97 to 101, Q 66 to 68, X 116 to 119 us; 51, 36 and 49 %).
#include "common.h"
#include "kernels.h"
#include "tile_product.h"

namespace bmoe {
namespace {

using namespace tile;

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

// Eight consecutive entries of U from i on, the momentum's step included (STEP).
template <bool STEP>
__device__ __forceinline__ void load8(const Source& s, size_t i, float (&v)[8]) {
  if (s.bf16) {
    load16(static_cast<const uint16_t*>(s.u) + i, v);
  } else {
    load16(static_cast<const float*>(s.u) + i, v);
    load16(static_cast<const float*>(s.u) + i + 4, v + 4);
  }
  if (!s.momentum) return;
  float m[8];
  load16(s.momentum + i, m);
  load16(s.momentum + i + 4, m + 4);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (STEP) m[e] = fmaf(s.beta, m[e], v[e]);
    v[e] = mixed(s, v[e], m[e]);
  }
  if (STEP) {
    store16(m, s.momentum + i, 1.f);
    store16(m + 4, s.momentum + i + 4, 1.f);
  }
}
template <bool STEP>
__device__ __forceinline__ float load1(const Source& s, size_t i) {
  const float u = load_any(s.u, s.bf16, i);
  if (!s.momentum) return u;
  float m = s.momentum[i];
  if (STEP) s.momentum[i] = m = fmaf(s.beta, m, u);
  return mixed(s, u, m);
}

// whole: matrices of whole chunks of eight.
__global__ __launch_bounds__(kSumThreads) void ortho_sum_kernel(Source src, size_t count, int whole,
                                                                double* part) {
  __shared__ double lds[kSumThreads / 64];
  const size_t first = (size_t)blockIdx.y * count, stride = (size_t)gridDim.x * kSumThreads;
  const size_t i0 = (size_t)blockIdx.x * kSumThreads + threadIdx.x;
  double acc = 0.0;
  if (whole) {
#pragma unroll 2
    for (size_t i = i0; i < count / 8; i += stride) {
      float v[8];
      load8<true>(src, first + 8 * i, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc = fma((double)v[e], (double)v[e], acc);
    }
  } else {
    for (size_t i = i0; i < count; i += stride) {
      const float v = load1<true>(src, first + i);
      acc = fma((double)v, (double)v, acc);
    }
  }
  const double s = block_sum(acc, lds);
  if (threadIdx.x == 0) part[(size_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// A scaled value as its two fp16 parts.
__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo) {
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
}

// ---- X_0 -----------------------------------------------------------------------
__global__ __launch_bounds__(kSumThreads) void ortho_split_kernel(Source src, int rows, int cols,
                                                                  int ld, float eps, float scale,
                                                                  const double* part, int parts,
                                                                  _Float16* hi, _Float16* lo) {
  __shared__ double lds[kSumThreads / 64];
  const double* mine = part + (size_t)blockIdx.y * parts;
  double acc = 0.0;
  for (int i = threadIdx.x; i < parts; i += kSumThreads) acc += mine[i];
  const float norm = (float)sqrt(block_sum(acc, lds)) + eps;
  const size_t in0 = (size_t)blockIdx.y * rows * cols, out0 = (size_t)blockIdx.y * rows * ld;
  const int chunks = ld / 8;
  const size_t n = (size_t)rows * chunks;
  for (size_t i = (size_t)blockIdx.x * kSumThreads + threadIdx.x; i < n;
       i += (size_t)gridDim.x * kSumThreads) {
    const size_t row = i / chunks;
    const int col = (int)(i - row * chunks) * 8;
    float v[8];
    if (cols == ld) {
      load8<false>(src, in0 + 8 * i, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = col + e < cols ? load1<false>(src, in0 + row * cols + col + e) : 0.f;
    }
    f16x8 h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      _Float16 a, b;
      split(v[e] / norm * scale, a, b);
      h[e] = a;
      l[e] = b;
    }
    *reinterpret_cast<f16x8*>(hi + out0 + 8 * i) = h;
    *reinterpret_cast<f16x8*>(lo + out0 + 8 * i) = l;
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
  int run_items;
  float unit;             // of the accumulators: to X's and P's scale
  float a, b, c;          // kPoly: to Q's scale
  // the last product's epilogue
  void* o;                // [batch][rows][cols]: X, or w = keep w - rate X
  int o_bf16, update;
  float keep, rate, unscale;  // 1 / the scale of X
};

// A 32 x 32 block of accumulators through LDS, so that a lane gets sixteen
// neighbours of a row, or of a column, and memory is read and written 16 bytes a
// lane. One wave's own LDS; its operations are in order.
struct Block {
  static constexpr int PITCH = 36;  // floats: rows stay 16-byte aligned, banks spread
  static constexpr int BYTES = 32 * PITCH * 4;
  __device__ __forceinline__ static void order() {
    __builtin_amdgcn_wave_barrier();
    __asm__ volatile("" ::: "memory");
  }
  __device__ __forceinline__ void stage(float* s, const f32x16& acc, int lane) const {
    order();  // the last block has been read
#pragma unroll
    for (int r = 0; r < 16; ++r) s[acc_row(r, lane) * PITCH + acc_col(lane)] = acc[r];
    order();
  }
  __device__ __forceinline__ void row(const float* s, int lane, float (&v)[16]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) load16(s + lane / 2 * PITCH + 16 * (lane & 1) + 4 * e, v + 4 * e);
  }
  __device__ __forceinline__ void put_row(float* s, int lane, const float (&v)[16]) const {
    order();
#pragma unroll
    for (int e = 0; e < 4; ++e)
      store16(v + 4 * e, s + lane / 2 * PITCH + 16 * (lane & 1) + 4 * e, 1.f);
    order();
  }
  __device__ __forceinline__ void column(const float* s, int lane, float (&v)[16]) const {
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = s[(16 * (lane & 1) + e) * PITCH + lane / 2];
  }
};

// v, sixteen entries of a row of P P at P's scale, to those of Q.
__device__ __forceinline__ void add_poly(const OrthoArgs& p, const char* q, int row, int col,
                                         float (&v)[16]) {
  const _Float16* hi = reinterpret_cast<const _Float16*>(q) + (size_t)row * p.ldm + col;
  const _Float16* lo = reinterpret_cast<const _Float16*>(
      reinterpret_cast<const char*>(hi) + p.q_part);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f16x8 a = {}, b = {};
    if (row < p.m && col + 8 * h < p.ldm) {
      a = *reinterpret_cast<const f16x8*>(hi + 8 * h);
      b = *reinterpret_cast<const f16x8*>(lo + 8 * h);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float pv = (float)a[e] + (float)b[e];
      v[8 * h + e] = fmaf(p.c, v[8 * h + e], p.b * pv);
      if (row == col + 8 * h + e) v[8 * h + e] += p.a;
    }
  }
}

// Sixteen entries of a row of an operand [rows][ld], cols of them values, the
// rest zeros.
__device__ __forceinline__ void store_parts(const OrthoArgs& p, int batch, int rows, int cols,
                                            int ld, int row, int col, const float (&v)[16]) {
  if (row >= rows) return;
  _Float16* hi = p.out + ((size_t)batch * rows + row) * ld + col;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (col + 8 * h >= ld) continue;
    f16x8 a, b;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      _Float16 x, y;
      split(col + 8 * h + e < cols ? v[8 * h + e] : 0.f, x, y);
      a[e] = x;
      b[e] = y;
    }
    *reinterpret_cast<f16x8*>(hi + 8 * h) = a;
    *reinterpret_cast<f16x8*>(hi + p.out_part + 8 * h) = b;
  }
}

// Sixteen entries of the last iterate (at X's scale) to the result or the weights.
__device__ __forceinline__ void store_result(const OrthoArgs& p, int batch, int row, int col,
                                             const float (&v)[16]) {
  if (row >= p.rows) return;
  const size_t at = ((size_t)batch * p.rows + row) * p.cols + col;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = p.cols - col - 8 * h;
    if (n <= 0) continue;
    float o[8];
    if (p.cols % 8 == 0) {
      if (p.update) {
        if (p.o_bf16) {
          load16(static_cast<const uint16_t*>(p.o) + at + 8 * h, o);
        } else {
          load16(static_cast<const float*>(p.o) + at + 8 * h, o);
          load16(static_cast<const float*>(p.o) + at + 8 * h + 4, o + 4);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = v[8 * h + e] * p.unscale;
        o[e] = p.update ? fmaf(p.keep, o[e], -p.rate * x) : x;
      }
      if (p.o_bf16) {
        store16(o, static_cast<uint16_t*>(p.o) + at + 8 * h, 1.f);
      } else {
        store16(o, static_cast<float*>(p.o) + at + 8 * h, 1.f);
        store16(o + 4, static_cast<float*>(p.o) + at + 8 * h + 4, 1.f);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= n) continue;
        float x = v[8 * h + e] * p.unscale;
        const size_t i = at + 8 * h + e;
        if (p.update) x = fmaf(p.keep, load_any(p.o, p.o_bf16, i), -p.rate * x);
        if (p.o_bf16) static_cast<uint16_t*>(p.o)[i] = (uint16_t)f32_to_bf16_bits(x);
        else static_cast<float*>(p.o)[i] = x;
      }
    }
  }
}

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
  __shared__ __attribute__((aligned(1024))) char st2[C::NSTAGE > 2 ? C::STAGE : 16];
  __shared__ __attribute__((aligned(1024))) char st3[C::NSTAGE > 3 ? C::STAGE : 16];
  char* all[4] = {st0, st1, st2, st3};
  char* ring[C::NSTAGE];
#pragma unroll
  for (int i = 0; i < C::NSTAGE; ++i) ring[i] = all[i];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const unsigned item = xcd_item(grid_block(), p.run_items);
  const int batch = item / p.tiles, t = item % p.tiles;
  if (batch >= p.batch) return;
  int2 tile;  // panels of four rows of tiles; of a symmetric matrix, rows of tiles
  if constexpr (PRODUCT == kApply) {
    const int panel = t / (4 * p.tiles_n), j = t - panel * 4 * p.tiles_n;
    const int high = min(4, p.tiles / p.tiles_n - 4 * panel);
    tile = make_int2(4 * panel + j % high, j / high);
  } else {
    tile = triangle(t);
  }
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
  // Chunks of a row beyond its values are zeros in memory, up to ld (ldm). P and
  // Q are symmetric: their rows, along the reduction, serve as rows and columns.
  const int red = PRODUCT == kGram && !TALL ? p.ld : PRODUCT == kGram ? p.rows : p.m;
  const int nsteps = (red + C::BK - 1) / C::BK;
  if constexpr (PRODUCT == kGram && !TALL) {  // X X^T
    OutRowsSource<C, C::BM, C::A_LOADS> a;
    a.init(
        x + r0 * x_ld, [&](int r) { return (uint32_t)(min(r, p.m - 1 - r0) * x_ld); }, red, p.x_part,
        lane, wave);
    OutRowsSource<C, C::BN, C::B_LOADS> b;
    b.init(
        x + c0 * x_ld, [&](int r) { return (uint32_t)(min(r, p.m - 1 - c0) * x_ld); }, red, p.x_part,
        lane, wave);
    run<C>(acc, ring, a, b, ra, rb, nsteps, lane, wave);
  } else if constexpr (PRODUCT == kApply && TALL) {  // X Q
    OutRowsSource<C, C::BM, C::A_LOADS> a;
    a.init(
        x + r0 * x_ld, [&](int r) { return (uint32_t)(min(r, p.rows - 1 - r0) * x_ld); }, red,
        p.x_part, lane, wave);
    RedRowsSource<C, C::BN, C::B_LOADS, SameRow> b;
    b.init(q, q_ld, c0, p.ldm, red, p.q_part, SameRow{}, lane, wave);
    run<C>(acc, ring, a, b, ra, rb, nsteps, lane, wave);
  } else {  // X^T X, P P, Q X
    const bool xa = PRODUCT == kGram, xb = PRODUCT != kPoly;
    RedRowsSource<C, C::BM, C::A_LOADS, SameRow> a;
    a.init(xa ? x : q, xa ? x_ld : q_ld, r0, xa ? p.ld : p.ldm, red, xa ? p.x_part : p.q_part,
           SameRow{}, lane, wave);
    RedRowsSource<C, C::BN, C::B_LOADS, SameRow> b;
    b.init(xb ? x : q, xb ? x_ld : q_ld, c0, xb ? p.ld : p.ldm, red, xb ? p.x_part : p.q_part,
           SameRow{}, lane, wave);
    run<C>(acc, ring, a, b, ra, rb, nsteps, lane, wave);
  }

  lds_barrier();  // every wave is done with the ring
  constexpr int PER = C::STAGE / Block::BYTES;  // waves' staging a stage holds
  static_assert(C::WAVES <= 2 * PER, "staging fits two stages");
  float* stg =
      reinterpret_cast<float*>((wave < PER ? st0 : st1) + (wave % PER) * Block::BYTES);
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      Block b;
      b.stage(stg, acc[i][j], lane);
      const int row0 = r0 + wm * C::TM + 32 * i, col0 = c0 + wn * C::TN + 32 * j;
      const int row = row0 + lane / 2, col = col0 + 16 * (lane & 1);
      float v[16];
      b.row(stg, lane, v);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= p.unit;
      if constexpr (PRODUCT == kPoly) add_poly(p, q, row, col, v);
      if constexpr (PRODUCT == kApply) {
        if (p.o) {
          store_result(p, batch, row, col, v);
        } else {
          store_parts(p, batch, p.rows, p.cols, p.ld, row, col, v);
        }
      } else {
        store_parts(p, batch, p.m, p.m, p.ldm, row, col, v);
        if (tile.x != tile.y) {  // the mirrored block
          if constexpr (PRODUCT == kPoly) b.put_row(stg, lane, v);
          b.column(stg, lane, v);
          if constexpr (PRODUCT == kGram) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] *= p.unit;
          }
          store_parts(p, batch, p.m, p.m, p.ldm, col0 + lane / 2, row0 + 16 * (lane & 1), v);
        }
      }
    }
}

// Tiles: of 128 x 128 (four waves, two workgroups per CU), 192 (four waves of 96)
// and 256 (eight waves of 128 x 64). With no more of them than CUs, where a
// launch lasts as long as its loads: 128 with eight waves and three steps ahead,
// and 64 (four waves, 128 bytes of reduction a step, three steps ahead). The tiles of
// 256 use all of a wave's 256 registers; four of their five kernels keep two to seven
// more in scratch memory.
enum TileKind { k64, k128Deep, k128, k192, k256 };
template <int KIND, int A, int B>
struct TileOf;
template <int A, int B>
struct TileOf<k64, A, B> {
  using type = Cfg<kF16, 2, 64, 64, 2, 2, 4, A, B, true, 128>;
};
template <int A, int B>
struct TileOf<k128Deep, A, B> {
  using type = Cfg<kF16, 2, 128, 128, 2, 4, 4, A, B, true>;
};
template <int A, int B>
struct TileOf<k128, A, B> {
  using type = Cfg<kF16, 2, 128, 128, 2, 2, 2, A, B, true>;
};
template <int A, int B>
struct TileOf<k192, A, B> {
  using type = Cfg<kF16, 2, 192, 192, 2, 2, 3, A, B, true>;
};
template <int A, int B>
struct TileOf<k256, A, B> {
  using type = Cfg<kF16, 2, 256, 256, 2, 4, 2, A, B, true>;
};

template <int PRODUCT>
int2 count_tiles(const OrthoArgs& p, int n) {  // of one matrix; per row of tiles
  const int tm = ((PRODUCT == kApply ? p.rows : p.m) + n - 1) / n;
  const int tn = ((PRODUCT == kApply ? p.cols : p.m) + n - 1) / n;
  return make_int2(PRODUCT == kApply ? tm * tn : tm * (tm + 1) / 2, tn);
}

template <int PRODUCT, bool TALL, int KIND>
hipError_t launch_tiles(OrthoArgs p, hipStream_t s) {
  constexpr int AMODE = (PRODUCT == kGram && !TALL) || (PRODUCT == kApply && TALL) ? kOutRows
                                                                                  : kRedRows;
  constexpr int BMODE = PRODUCT == kGram && !TALL ? kOutRows : kRedRows;
  using C = typename TileOf<KIND, AMODE, BMODE>::type;
  const int2 c = count_tiles<PRODUCT>(p, C::BM);
  p.tiles = c.x;
  p.tiles_n = c.y;
  const size_t items = (size_t)p.tiles * p.batch;
  p.run_items = items >= 256 ? 32 : 1;
  const size_t super = 8 * p.run_items;
  return launch_kernel(ortho_product_kernel<C, PRODUCT, TALL>,
                       grid_rows((items + super - 1) / super * super), dim3(C::THREADS), 0, s,
                       KernelTiming{}, p);
}

// The tile: the deep ones as long as each CU gets one at most (two of 64) - 1000
// x 1000 580 -> 230 us, 2048 x 2048 862 -> 687 us a call -, else by the time that
// the rounds of workgroups over 256 CUs take, in units of a round of two
// workgroups per CU of 128 x 128 (one per CU: 0.55). Measured at 4096 x 4096:
// whole products 351, 370 and 311 us, symmetric ones 296, 210 and 256 us with
// tiles of 128, 192 and 256; 64 matrices 1024 x 512: 150, 201, 136 and 111, 119,
// 110 us.
template <int PRODUCT, bool TALL>
hipError_t launch_product(const OrthoArgs& p, hipStream_t s) {
  const auto tiles = [&](int n) { return (long long)count_tiles<PRODUCT>(p, n).x * p.batch; };
  if (tiles(64) <= 512) return launch_tiles<PRODUCT, TALL, k64>(p, s);
  if (tiles(128) <= 256) return launch_tiles<PRODUCT, TALL, k128Deep>(p, s);
  const long long n128 = tiles(128), rest = n128 % 512;
  const double t128 = n128 / 512 + (rest > 256 ? 1.0 : rest > 0 ? 0.55 : 0.0);
  const double t192 = 1.1 * ((tiles(192) + 255) / 256);
  const double t256 = 1.75 * ((tiles(256) + 255) / 256);
  if (t128 <= t192 && t128 <= t256) return launch_tiles<PRODUCT, TALL, k128>(p, s);
  if (t192 <= t256) return launch_tiles<PRODUCT, TALL, k192>(p, s);
  return launch_tiles<PRODUCT, TALL, k256>(p, s);
}

// ---- small sides: the iteration with X in registers --------------------------------
// X [m][n] (transposed where rows > cols) with m <= 32 MB. A workgroup holds 256 NB
// columns of it in registers, wave w the columns 32 NB w .. as MFMA operands of
// two layouts:
//   x1: lane = row m, eight columns n a slice     (P = X X^T)
//   x2: lane = column n, eight rows m a slice     (Q X, X^T Q)
// Accumulators of X^T Q (lane = column m, rows n) are x1's next values and those
// of Q X (lane = column n, rows m) x2's, slice s of a block its registers 8 s ..
// 8 s + 7: computing both costs MFMAs instead of transposing. This fixes the
// order of the reduction inside a slice: element e of lane half h is index
// 8 (e / 4) + 4 h + e % 4; all operands follow it. P is added over the waves, in
// order, through LDS.
constexpr int kSmallWaves = 8, kSmallThreads = 64 * kSmallWaves;
constexpr int kPitch = 72;  // halves per row of P and Q in LDS

struct SmallArgs {
  Source src;
  int rows, cols, steps, tall;
  float a, b, c, eps;           // a, b, c: to Q's scale
  float scale;                  // of X and P
  float p_unit, x_unit;         // X X^T and P P, Q X: to that scale
  void* o;
  int o_bf16, update;
  float keep, rate, unscale;    // Q X to the result
  // matrices in slabs
  const double* part;  // [batch][parts]: sums of squares
  int parts;
  u32x4* x;            // [batch][slabs]: x2, as the lanes hold it
  const float* p_in;   // [batch][slabs]: sums of P over the slabs' columns
  float* p_out;
};

// Operands are kept as dwords of two values: the loop over the steps would carry
// single halves in a register each.
template <int MB, int NB>
struct Operands {
  u32x4 x1[MB][2 * NB][2], x2[NB][2 * MB][2];  // [..][slice][part]
};
template <int MB, int NB>
using Entries = f32x16[NB][MB];  // as accumulators of Q X

template <int MB>
struct SmallLds {
  static constexpr int BLOCKS = MB == 1 ? 1 : 3;  // of P on and above the diagonal
  static constexpr int RED = BLOCKS * 1024 > 1056 ? BLOCKS * 1024 : 1056;  // floats a wave
  __attribute__((aligned(16))) _Float16 P[2][32 * MB * kPitch], Q[2][32 * MB * kPitch];
  double dsum[kSmallWaves];
  float red[kSmallWaves][RED];
  __device__ __forceinline__ static void block_of(int i, int& r, int& c) {  // (0, 0), (0, 1), (1, 1)
    r = i == 2;
    c = i > 0;
  }
};

// This workgroup's matrix.
struct SmallMatrix {
  int m, n;
  Source src;
  void* out;
  __device__ __forceinline__ SmallMatrix(const SmallArgs& p, int batch) {
    m = p.tall ? p.cols : p.rows;
    n = p.tall ? p.rows : p.cols;
    const size_t first = (size_t)batch * p.rows * p.cols;
    src = p.src;
    src.u = static_cast<const char*>(src.u) + first * (src.bf16 ? 2 : 4);
    if (src.momentum) src.momentum += first;
    out = static_cast<char*>(p.o) + first * (p.o_bf16 ? 2 : 4);
  }
};

// The eight values of slice s in the order above, row `row` of P or Q.
__device__ __forceinline__ u32x4 read_symmetric(const _Float16* q, int row, int s, int lane) {
  const _Float16* p = q + row * kPitch + 16 * s + 4 * (lane >> 5);
  const u32x2 x = *reinterpret_cast<const u32x2*>(p), y = *reinterpret_cast<const u32x2*>(p + 8);
  return u32x4{x[0], x[1], y[0], y[1]};
}
__device__ __forceinline__ f32x16 mma3(const u32x4 (&a)[2], const u32x4 (&b)[2], f32x16 acc) {
  mma<kF16>(acc, a[0], b[1]);
  mma<kF16>(acc, a[1], b[0]);
  mma<kF16>(acc, a[0], b[0]);
  return acc;
}
__device__ __forceinline__ void split_slice(const f32x16& v, int s, float scale, u32x4 (&out)[2]) {
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const f32x2 x = {v[8 * s + 2 * e] * scale, v[8 * s + 2 * e + 1] * scale};
    const f16x2 hi = __builtin_convertvector(x, f16x2);
    const f32x2 back = __builtin_convertvector(hi, f32x2);
    const f32x2 rest = {x[0] - back[0], x[1] - back[1]};
    out[0][e] = __builtin_bit_cast(uint32_t, hi);
    out[1][e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, f16x2));
  }
}

// f(register, entry's number, whether it is one) for the lane's entries from
// column n0 on.
template <int MB, int NB, class F>
__device__ __forceinline__ void each_entry(const SmallArgs& p, const SmallMatrix& x, int n0, int lane,
                                           Entries<MB, NB>& v, F f) {
  // (a value of its own, or the entries' numbers would be kept from one use to
  // the next, in 32 MB NB registers)
  int n1 = n0;
  __asm__ volatile("" : "+v"(n1));
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int mi = 32 * mb + acc_row(r, lane), ni = n1 + 32 * nb;
        const bool in = mi < x.m && ni < x.n;
        const uint32_t at = p.tall ? (uint32_t)(ni * p.cols + mi) : (uint32_t)(mi * p.cols + ni);
        float e = v[nb][mb][r];
        f(e, in ? at : 0u, in);
        v[nb][mb][r] = e;
      }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// U's entries; STEP: the momentum's step with them. (Types are told apart outside
// of the loops, so that all loads are in flight together.)
template <int MB, int NB, bool STEP>
__device__ __forceinline__ void load_entries(const SmallArgs& p, const SmallMatrix& x, int n0,
                                             int lane, Entries<MB, NB>& v) {
  const Source& src = x.src;
  if (src.bf16)
    each_entry<MB, NB>(p, x, n0, lane, v, [&](float& e, uint32_t i, bool in) {
      const float u = bf16_lo(static_cast<const uint16_t*>(src.u)[i]);
      e = in ? u : 0.f;
    });
  else
    each_entry<MB, NB>(p, x, n0, lane, v, [&](float& e, uint32_t i, bool in) {
      const float u = static_cast<const float*>(src.u)[i];
      e = in ? u : 0.f;
    });
  if (src.momentum)
    each_entry<MB, NB>(p, x, n0, lane, v, [&](float& e, uint32_t i, bool in) {
      float mo = src.momentum[i];
      if (STEP) {
        mo = fmaf(src.beta, mo, e);
        if (in) src.momentum[i] = mo;
      }
      e = in ? mixed(src, e, mo) : 0.f;
    });
}

// The sum of v over the workgroup, in order.
__device__ __forceinline__ double small_sum(double v, double* dsum, int lane, int wave) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  if (lane == 0) dsum[wave] = v;
  __syncthreads();
  double total = 0.0;
#pragma unroll
  for (int w = 0; w < kSmallWaves; ++w) total += dsum[w];
  return total;
}

// X_0 in both layouts, the second through the wave's own LDS once (33 floats a
// row: no bank twice).
template <int MB, int NB>
__device__ __forceinline__ void first_operands(const Entries<MB, NB>& v, float norm, float scale,
                                               float* mine, int lane, Operands<MB, NB>& x) {
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      f32x16 y;
#pragma unroll
      for (int r = 0; r < 16; ++r) y[r] = v[nb][mb][r] / norm * scale;
#pragma unroll
      for (int s = 0; s < 2; ++s) split_slice(y, s, 1.f, x.x2[nb][2 * mb + s]);
      Block::order();
#pragma unroll
      for (int r = 0; r < 16; ++r) mine[acc_row(r, lane) * 33 + (lane & 31)] = y[r];
      Block::order();
      f32x16 t;
#pragma unroll
      for (int r = 0; r < 16; ++r) t[r] = mine[(lane & 31) * 33 + acc_row(r, lane)];
#pragma unroll
      for (int s = 0; s < 2; ++s) split_slice(t, s, 1.f, x.x1[mb][2 * nb + s]);
      __builtin_amdgcn_sched_barrier(0);  // (the next block's registers are this one's)
    }
}

// P of this wave's columns to its LDS, entry i * 1024 + 64 * register + lane of
// block i.
template <int MB, int NB>
__device__ __forceinline__ void wave_gram(const Operands<MB, NB>& x, float* mine, int lane) {
#pragma unroll
  for (int i = 0; i < SmallLds<MB>::BLOCKS; ++i) {
    int br, bc;
    SmallLds<MB>::block_of(i, br, bc);
    f32x16 acc = {};
#pragma unroll
    for (int s = 0; s < 2 * NB; ++s) acc = mma3(x.x1[br][s], x.x1[bc][s], acc);
#pragma unroll
    for (int r = 0; r < 16; ++r) mine[i * 1024 + r * 64 + lane] = acc[r];
  }
}
template <int MB>
__device__ __forceinline__ float waves_sum(const SmallLds<MB>& lds, int e) {
  float sum = lds.red[0][e];
#pragma unroll
  for (int w = 1; w < kSmallWaves; ++w) sum += lds.red[w][e];
  return sum;
}
// P's entry e (as above) from its sum, which has the scale twice.
template <int MB>
__device__ __forceinline__ void put_p(const SmallArgs& p, SmallLds<MB>& lds, int e, float sum) {
  const int i = e / 1024, r = e % 1024 / 64, l = e % 64;
  int br, bc;
  SmallLds<MB>::block_of(i, br, bc);
  const int row = 32 * br + acc_row(r, l), col = 32 * bc + (l & 31);
  _Float16 hi, lo;
  split(sum * p.p_unit, hi, lo);
  lds.P[0][row * kPitch + col] = hi;
  lds.P[1][row * kPitch + col] = lo;
  if (br != bc) {
    lds.P[0][col * kPitch + row] = hi;
    lds.P[1][col * kPitch + row] = lo;
  }
}
// Q = a I + b P + c P P, a block a wave.
template <int MB>
__device__ __forceinline__ void small_poly(const SmallArgs& p, SmallLds<MB>& lds, int lane, int wave) {
  if (wave >= SmallLds<MB>::BLOCKS) return;
  int br, bc;
  SmallLds<MB>::block_of(wave, br, bc);
  f32x16 acc = {};
#pragma unroll
  for (int s = 0; s < 2 * MB; ++s) {
    u32x4 fa[2], fb[2];
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      fa[part] = read_symmetric(lds.P[part], 32 * br + (lane & 31), s, lane);
      fb[part] = read_symmetric(lds.P[part], 32 * bc + (lane & 31), s, lane);
    }
    acc = mma3(fa, fb, acc);
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int row = 32 * br + acc_row(r, lane), col = 32 * bc + (lane & 31);
    const float pv = (float)lds.P[0][row * kPitch + col] + (float)lds.P[1][row * kPitch + col];
    float q = fmaf(p.c, acc[r] * p.p_unit, p.b * pv);
    if (row == col) q += p.a;
    _Float16 hi, lo;
    split(q, hi, lo);
    lds.Q[0][row * kPitch + col] = hi;
    lds.Q[1][row * kPitch + col] = lo;
    if (br != bc) {
      lds.Q[0][col * kPitch + row] = hi;
      lds.Q[1][col * kPitch + row] = lo;
    }
  }
}

template <int MB>
__device__ __forceinline__ void read_q(const SmallLds<MB>& lds, int mb, int lane,
                                       u32x4 (&q)[2 * MB][2]) {
#pragma unroll
  for (int s = 0; s < 2 * MB; ++s)
#pragma unroll
    for (int part = 0; part < 2; ++part)
      q[s][part] = read_symmetric(lds.Q[part], 32 * mb + (lane & 31), s, lane);
}
// X <- Q X, in both layouts.
template <int MB, int NB>
__device__ __forceinline__ void small_apply(const SmallArgs& p, const SmallLds<MB>& lds, int lane,
                                            Operands<MB, NB>& x) {
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    f32x16 next[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      u32x4 q[2 * MB][2];
      read_q<MB>(lds, mb, lane, q);
      next[mb] = f32x16{};  // Q X
      f32x16 t = {};        // X^T Q
#pragma unroll
      for (int s = 0; s < 2 * MB; ++s) {
        next[mb] = mma3(q[s], x.x2[nb][s], next[mb]);
        t = mma3(x.x2[nb][s], q[s], t);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) split_slice(t, s, p.x_unit, x.x1[mb][2 * nb + s]);
      __builtin_amdgcn_sched_barrier(0);  // (two blocks at a time would spill)
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int s = 0; s < 2; ++s) split_slice(next[mb], s, p.x_unit, x.x2[nb][2 * mb + s]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// A block of the last iterate (lane = column ni, rows mi ..) to the result.
template <typename T>
__device__ __forceinline__ void store_small_as(const SmallArgs& p, T* out, const f32x16& x, int m,
                                               int n, int mi, int ni, int lane) {
  float w[16];
  uint32_t at[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int row = mi + acc_row(r, lane);
    at[r] = row >= m || ni >= n ? 0u : (uint32_t)(p.tall ? ni * p.cols + row : row * p.cols + ni);
    w[r] = 0.f;
  }
  if (p.update) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      if constexpr (sizeof(T) == 2) w[r] = bf16_lo(out[at[r]]);
      else w[r] = out[at[r]];
    }
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    float o = x[r] * p.unscale;
    if (p.update) o = fmaf(p.keep, w[r], -p.rate * o);
    if (mi + acc_row(r, lane) < m && ni < n) {
      if constexpr (sizeof(T) == 2) out[at[r]] = (T)f32_to_bf16_bits(o);
      else out[at[r]] = o;
    }
  }
}
// The last Q X, from column n0 on.
template <int MB, int NB>
__device__ __forceinline__ void small_result(const SmallArgs& p, const SmallMatrix& x,
                                             const SmallLds<MB>& lds, int n0, int lane,
                                             const Operands<MB, NB>& ops) {
  int n1 = n0;  // (as in each_entry)
  __asm__ volatile("" : "+v"(n1));
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      u32x4 q[2 * MB][2];
      read_q<MB>(lds, mb, lane, q);
      f32x16 y = {};
#pragma unroll
      for (int s = 0; s < 2 * MB; ++s) y = mma3(q[s], ops.x2[nb][s], y);
      const int ni = n1 + 32 * nb;
      if (p.o_bf16)
        store_small_as(p, static_cast<uint16_t*>(x.out), y, x.m, x.n, 32 * mb, ni, lane);
      else
        store_small_as(p, static_cast<float*>(x.out), y, x.m, x.n, 32 * mb, ni, lane);
      __builtin_amdgcn_sched_barrier(0);
    }
}

// n <= 256 NB: the whole iteration in one workgroup, one launch for 17: 64 x 512
// fp32 141 -> 52 us, 64 of them 53 us. (MB = NB = 2, that size, keeps three of its
// registers in scratch memory.)
template <int MB, int NB>
__global__ __launch_bounds__(kSmallThreads) void ortho_small_kernel(SmallArgs p) {
  __shared__ SmallLds<MB> lds;
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const SmallMatrix x(p, blockIdx.x);
  const int n0 = 32 * NB * wave + (lane & 31);  // this lane's column of block 0
  Entries<MB, NB> v;
  load_entries<MB, NB, true>(p, x, n0, lane, v);
  double acc = 0.0;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc = fma((double)v[nb][mb][r], (double)v[nb][mb][r], acc);
  const float norm = (float)sqrt(small_sum(acc, lds.dsum, lane, wave)) + p.eps;
  Operands<MB, NB> ops;
  first_operands<MB, NB>(v, norm, p.scale, lds.red[wave], lane, ops);
  const auto make_q = [&]() {
    __syncthreads();  // red, P and Q have been read
    wave_gram<MB, NB>(ops, lds.red[wave], lane);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < SmallLds<MB>::BLOCKS * 2; ++j) {
      const int e = tid + j * kSmallThreads;
      put_p<MB>(p, lds, e, waves_sum<MB>(lds, e));
    }
    __syncthreads();
    small_poly<MB>(p, lds, lane, wave);
    __syncthreads();
  };
  for (int step = 1; step < p.steps; ++step) {
    make_q();
    small_apply<MB, NB>(p, lds, lane, ops);
  }
  make_q();
  small_result<MB, NB>(p, x, lds, n0, lane, ops);
}

// Longer n: slabs of 256 NB columns, a workgroup each. Only P needs all of them, so
// a launch takes a slab from one P to the next: it adds up the slabs' parts of P
// (in order, out of L2), forms Q, applies it and leaves its part of the next P
// and x2. The first launch has X_0 for X, the last one stores X: steps + 2 launches
// (one for the norm) instead of 3 steps + 2 of the products above: 64 x 2048 141 ->
// 57 us, 40 x 4096 195 -> 63 us, 64 matrices 64 x 2048 229 -> 170 us, 4096 of 8 x 2000
// 6.1 -> 2.6 ms. (Where one workgroup holds a matrix it is as fast for one, 52 and 52
// us at 64 x 512, and faster for many: 512 of them 135 and 269 us.)
enum SlabPhase { kFirst, kStep, kLast };
template <int MB, int NB, int PHASE>
__global__ __launch_bounds__(kSmallThreads) void ortho_slab_kernel(SmallArgs p) {
  __shared__ SmallLds<MB> lds;
  constexpr int SUMS = SmallLds<MB>::BLOCKS * 1024;  // entries of a part of P
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const SmallMatrix x(p, blockIdx.y);
  const int slabs = gridDim.x;
  const size_t slab = (size_t)blockIdx.y * slabs + blockIdx.x;
  const int n0 = 32 * NB * (blockIdx.x * kSmallWaves + wave) + (lane & 31);
  u32x4* kept = p.x + slab * (NB * 2 * MB * 2) * kSmallThreads + tid;
  Operands<MB, NB> ops;
  if constexpr (PHASE == kFirst) {
    Entries<MB, NB> v;
    load_entries<MB, NB, false>(p, x, n0, lane, v);
    double acc = 0.0;
    for (int i = tid; i < p.parts; i += kSmallThreads) acc += p.part[(size_t)blockIdx.y * p.parts + i];
    const float norm = (float)sqrt(small_sum(acc, lds.dsum, lane, wave)) + p.eps;
    first_operands<MB, NB>(v, norm, p.scale, lds.red[wave], lane, ops);
  } else {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int s = 0; s < 2 * MB; ++s)
#pragma unroll
        for (int part = 0; part < 2; ++part)
          ops.x2[nb][s][part] = kept[((nb * 2 * MB + s) * 2 + part) * kSmallThreads];
    const float* sums = p.p_in + (size_t)blockIdx.y * slabs * SUMS;
    constexpr int PAIRS = SUMS / 2 / kSmallThreads;  // of entries, a thread's
    f32x2 sum[PAIRS];
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) sum[j] = f32x2{0.f, 0.f};
    for (int g0 = 0; g0 < slabs; g0 += 8) {
      f32x2 part[8][PAIRS];
#pragma unroll
      for (int g = 0; g < 8; ++g)
#pragma unroll
        for (int j = 0; j < PAIRS; ++j)
          part[g][j] = g0 + g < slabs
                           ? *reinterpret_cast<const f32x2*>(sums + (size_t)(g0 + g) * SUMS +
                                                             2 * (tid + j * kSmallThreads))
                           : f32x2{0.f, 0.f};
#pragma unroll
      for (int g = 0; g < 8; ++g)
#pragma unroll
        for (int j = 0; j < PAIRS; ++j) {
          sum[j][0] += part[g][j][0];
          sum[j][1] += part[g][j][1];
        }
    }
#pragma unroll
    for (int j = 0; j < PAIRS; ++j) {
      put_p<MB>(p, lds, 2 * (tid + j * kSmallThreads), sum[j][0]);
      put_p<MB>(p, lds, 2 * (tid + j * kSmallThreads) + 1, sum[j][1]);
    }
    __syncthreads();
    small_poly<MB>(p, lds, lane, wave);
    __syncthreads();
    if constexpr (PHASE == kLast) {
      small_result<MB, NB>(p, x, lds, n0, lane, ops);
      return;
    } else {
      small_apply<MB, NB>(p, lds, lane, ops);
    }
  }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int s = 0; s < 2 * MB; ++s)
#pragma unroll
      for (int part = 0; part < 2; ++part)
        kept[((nb * 2 * MB + s) * 2 + part) * kSmallThreads] = ops.x2[nb][s][part];
  wave_gram<MB, NB>(ops, lds.red[wave], lane);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < SUMS / kSmallThreads; ++j) {
    const int e = tid + j * kSmallThreads;
    p.p_out[slab * SUMS + e] = waves_sum<MB>(lds, e);
  }
}

template <int MB, int NB>
hipError_t launch_small(const SmallArgs& p, int batch, hipStream_t s) {
  return launch_kernel(ortho_small_kernel<MB, NB>, dim3(batch), dim3(kSmallThreads), 0, s,
                       KernelTiming{}, p);
}
// p2: two buffers for the parts of P, taken in turn.
template <int MB, int NB>
hipError_t launch_slabs(SmallArgs p, int batch, int slabs, float* const (&p2)[2], hipStream_t s) {
  const dim3 grid(slabs, batch);
  for (int i = 0; i <= p.steps; ++i) {
    p.p_in = p2[(i + 1) & 1];
    p.p_out = p2[i & 1];
    const auto kernel = i == 0         ? ortho_slab_kernel<MB, NB, kFirst>
                        : i < p.steps ? ortho_slab_kernel<MB, NB, kStep>
                                      : ortho_slab_kernel<MB, NB, kLast>;
    const hipError_t e = launch_kernel(kernel, grid, dim3(kSmallThreads), 0, s, KernelTiming{}, p);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

int padded(int n) { return (n + 7) / 8 * 8; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Whether a matrix's smaller side fits the kernels that keep X in registers, and
// the blocks of 32 of each side that a wave of theirs holds.
struct SmallShape {
  int mb, nb, slabs;  // mb = 0: too large; slabs = 1: one workgroup
};
SmallShape small_shape(int rows, int cols) {
  const int low = rows < cols ? rows : cols, high = rows < cols ? cols : rows;
  if (low > 64) return {0, 0, 0};
  const int mb = low <= 32 ? 1 : 2, most = mb == 1 ? 4 : 2;
  if (high <= 256 * most) return {mb, high <= 256 ? 1 : high <= 512 ? 2 : 4, 1};
  return {mb, 1, (high + 255) / 256};
}

struct Layout {
  size_t part, x0, x1, p, q, total;  // byte offsets
  size_t x_part, p_part;             // bytes of one part
  int ld, m, ldm;
};
Layout layout(int batch, int rows, int cols) {
  Layout l = {};
  const SmallShape small = small_shape(rows, cols);
  if (small.slabs == 1) return l;
  if (small.mb) {  // x0: x2; p, q: the two buffers of the parts of P
    const size_t n = (size_t)batch * small.slabs;
    l.x0 = up256((size_t)batch * kSumParts * sizeof(double));
    l.p = l.x0 + n * (small.nb * 2 * small.mb * 2) * kSmallThreads * sizeof(u32x4);
    l.q = l.p + n * (small.mb == 1 ? 1 : 3) * 1024 * sizeof(float);
    l.total = l.q + (l.q - l.p);
    return l;
  }
  l.ld = padded(cols);
  l.m = rows < cols ? rows : cols;
  l.ldm = padded(l.m);
  l.x_part = up256((size_t)batch * rows * l.ld * 2);
  l.p_part = up256((size_t)batch * l.m * l.ldm * 2);
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
  const SmallShape small = small_shape(rows, cols);
  const Layout l = layout(batch, rows, cols);
  char* base = static_cast<char*>(ws);
  double* part = reinterpret_cast<double*>(base + l.part);
  Source src;
  src.u = call.u;
  src.momentum = call.momentum;
  src.beta = call.beta;
  src.nesterov = call.nesterov;
  src.bf16 = call.u_bf16;
  SmallArgs sp = {};
  sp.src = src;
  sp.rows = rows;
  sp.cols = cols;
  sp.steps = call.steps;
  sp.tall = rows > cols;
  // (powers of two: exact)
  sp.a = call.a * call.q_scale;
  sp.b = call.b * (call.q_scale / call.x_scale);
  sp.c = call.c * (call.q_scale / call.x_scale);
  sp.scale = call.x_scale;
  sp.p_unit = 1.f / call.x_scale;
  sp.x_unit = 1.f / call.q_scale;
  sp.unscale = sp.p_unit * sp.x_unit;
  sp.eps = call.eps;
  sp.o = call.o;
  sp.o_bf16 = call.o_bf16;
  sp.update = call.update;
  sp.keep = call.keep;
  sp.rate = call.rate;
  if (small.slabs == 1) {
    if (small.mb == 1)
      return small.nb == 1   ? launch_small<1, 1>(sp, batch, s)
             : small.nb == 2 ? launch_small<1, 2>(sp, batch, s)
                             : launch_small<1, 4>(sp, batch, s);
    return small.nb == 1 ? launch_small<2, 1>(sp, batch, s) : launch_small<2, 2>(sp, batch, s);
  }
  const size_t count = (size_t)rows * cols;
  // as many workgroups as fill the chip, at least a few rounds of entries each
  const size_t most = batch >= 32 ? 32 : kSumParts;
  const size_t want = (count + 16 * kSumThreads - 1) / (16 * kSumThreads);
  const int parts = (int)(want < most ? want : most);
  hipError_t e = launch_kernel(ortho_sum_kernel, dim3(parts, batch), dim3(kSumThreads), 0, s,
                               KernelTiming{}, src, count, (int)(count % 8 == 0), part);
  if (e != hipSuccess) return e;
  if (small.mb) {
    sp.part = part;
    sp.parts = parts;
    sp.x = reinterpret_cast<u32x4*>(base + l.x0);
    float* const p2[2] = {reinterpret_cast<float*>(base + l.p), reinterpret_cast<float*>(base + l.q)};
    return small.mb == 1 ? launch_slabs<1, 1>(sp, batch, small.slabs, p2, s)
                         : launch_slabs<2, 1>(sp, batch, small.slabs, p2, s);
  }
  _Float16* x[2] = {reinterpret_cast<_Float16*>(base + l.x0),
                    reinterpret_cast<_Float16*>(base + l.x1)};
  const size_t blocks = ((size_t)rows * l.ld / 8 + kSumThreads - 1) / kSumThreads;
  const size_t enough = batch >= 32 ? 64 : 2048;
  e = launch_kernel(ortho_split_kernel, dim3((unsigned)(blocks < enough ? blocks : enough), batch),
                    dim3(kSumThreads), 0, s, KernelTiming{}, src, rows, cols, l.ld, call.eps, call.x_scale,
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
  p.a = sp.a;
  p.b = sp.b;
  p.c = sp.c;
  p.unscale = sp.p_unit;
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
    p.unit = sp.p_unit;
    e = tall ? launch_product<kGram, true>(p, s) : launch_product<kGram, false>(p, s);
    if (e != hipSuccess) return e;
    p.q = P;
    p.out = Q;
    e = launch_product<kPoly, false>(p, s);
    if (e != hipSuccess) return e;
    p.q = Q;
    p.out = x[(i + 1) & 1];
    p.unit = sp.x_unit;
    p.out_part = l.x_part / 2;
    if (i + 1 == call.steps) p.o = call.o;
    e = tall ? launch_product<kApply, true>(p, s) : launch_product<kApply, false>(p, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace bmoe
