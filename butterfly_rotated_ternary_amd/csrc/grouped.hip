// Matrix products grouped by expert, ragged groups:
//   c[q]  = W_e a[row(q)]                  rows q of group e, e = 0 .. G - 1
//   da[q] = W_e^T dc[q]
//   dW_e  = sum over the rows q of e of dc[q] a[row(q)]^T      (fp32)
// with group e the rows offsets[e] .. offsets[e + 1] and row(q) = perm[q] / k
// (q itself without perm). The offsets live on the device: a workgroup finds
// its tile of a group from them, so the host never waits for the router.
//
// Large groups are bound by the matrix units together with the LDS and L2 that
// feed them: 131072 rows of 256 experts 4096 -> 1024, bf16, 1.24 ms (890 TFLOP/s; 57
// % of the MFMA cycles; 3.6 GB read, of them 2.1 GB weights and 1.1 GB rows, each
// of which four experts read); 32768 rows of 64 experts 2048 -> 2048: c and da 340 us,
// dW 400 to 470 (1.07 GB of fp32 results). One group of 4096 x 4096 x 4096: 113, 110
// and 117 us (1180 to 1250 TFLOP/s), fp32 1.0 to 1.1 ms (123 to 138). Few rows are
// bound by reading the weights: one token of 8 experts of 256, 46 MB, 11.4 us in a
// captured graph, 12 to 14 in the trace.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "tile_product.h"

namespace bmoe {
namespace {

using namespace tile;

// Rows of group e, whatever the offsets hold.
__device__ __forceinline__ int2 group_rows_of(const int32_t* offsets, int e, int M) {
  const int lo = min(max(offsets[e], 0), M), hi = min(max(offsets[e + 1], 0), M);
  return make_int2(lo, max(lo, hi));
}

struct GroupTile {
  int e, lo, hi;     // group (-1: no such tile) and its rows
  int tiles;         // rows of tiles in the group
  int i, col_tile;   // this tile's
};

// Work item t of all groups' tiles, groups ascending; a group has rows / MOST
// rows of tiles_n tiles, rounded up. They come in panels of four rows of tiles,
// so that the consecutive items that share an L2 are near square. Every wave
// looks its tile up for itself: 64 groups at a time, a prefix sum over the lanes;
// the loads of four times 64 groups' offsets come before the first sum, but the
// compiler waits for each. fill: the rows behind the last group are one more, G, those
// before the first another, G + 1 (behind the loop: as lanes of it they made one
// token of 8 experts 12.0 us instead of 11.4).
constexpr int kPanel = 4;
// Tile `at` of the `items` of group e.
__device__ __forceinline__ GroupTile tile_of(int e, int lo, int hi, int items, int tiles_n, int at) {
  // (offsets that do not ascend can overflow the sum: no tile then)
  if ((unsigned)at >= (unsigned)items) return {-1, 0, 0, 0, 0, 0};
  GroupTile g;
  g.e = e;
  g.lo = lo;
  g.hi = hi;
  g.tiles = items / tiles_n;
  const int panel = at / (kPanel * tiles_n), j = at - panel * kPanel * tiles_n;
  const int high = min(kPanel, g.tiles - panel * kPanel);
  g.i = panel * kPanel + j % high;
  g.col_tile = j / high;
  return g;
}
template <int MOST>
__device__ __forceinline__ GroupTile find_tile(const int32_t* offsets, int G, int M, int tiles_n,
                                               int fill, int t, int lane) {
  int before = 0;
  for (int e1 = 0; e1 < G; e1 += 4 * kWave) {
    int2 rows[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = e1 + u * kWave + lane;
      rows[u] = e < G ? group_rows_of(offsets, e, M) : make_int2(0, 0);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int2 r = rows[u];
      const int n = (int)(((unsigned)(r.y - r.x) + MOST - 1) / MOST) * tiles_n;
      const int incl = wave_incl_scan(n);
      const uint64_t past = __ballot(before + incl > t);
      if (past) {
        const int src = __ffsll((unsigned long long)past) - 1;
        const int items = __builtin_amdgcn_readlane(n, src);
        return tile_of(e1 + u * kWave + src, __builtin_amdgcn_readlane(r.x, src),
                       __builtin_amdgcn_readlane(r.y, src), items, tiles_n,
                       t - before - (__builtin_amdgcn_readlane(incl, src) - items));
      }
      before += __builtin_amdgcn_readlane(incl, kWave - 1);
    }
  }
  if (fill) {
    const int end = min(max(offsets[G], 0), M), begin = min(max(offsets[0], 0), M);
    const int behind = (int)(((unsigned)(M - end) + MOST - 1) / MOST) * tiles_n;
    const int ahead = (int)(((unsigned)begin + MOST - 1) / MOST) * tiles_n;
    if (t - before < behind) return tile_of(G, end, M, behind, tiles_n, t - before);
    if (t - before - behind < ahead)
      return tile_of(G + 1, 0, begin, ahead, tiles_n, t - before - behind);
  }
  return {-1, 0, 0, 0, 0, 0};
}

struct ProductArgs {
  const char* a;  // rows of the product's left operand, `red` values each
  const char* w;  // [G][O][K]
  char* c;        // [M][cols]
  const int32_t* offsets;
  const int32_t* perm;  // NULL: row q of a is row q of the product
  int k, a_rows, M, G, red, cols, tiles_n;
  int fill;  // whether rows of no group become 0
};

// Row q's row of a.
__device__ __forceinline__ int a_row(const ProductArgs& p, int q) {
  if (!p.perm) return q;
  const int t = p.perm[q] / p.k;
  return min(max(t, 0), p.a_rows - 1);
}

// A wave's accumulator blocks to bf16 rows of c, 16 rows at a time through its
// own LDS, so that stores are 16 bytes a lane over whole row segments.
template <class C>
__device__ __forceinline__ void store_bf16(const Acc<C>& acc, char* stg, char* c, size_t ld,
                                           int rows, int cols, int lane) {
  constexpr int PITCH = C::TN * 2, CHUNKS = C::TN / 8, RPQ = 64 / CHUNKS;
  static_assert((CHUNKS & (CHUNKS - 1)) == 0 && CHUNKS <= 64, "chunk swizzle");
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int r = 8 * h; r < 8 * h + 8; ++r) {
          const int row = acc_row(r, lane) - 16 * h, col = j * 32 + acc_col(lane);
          const int off = row * PITCH + 16 * ((col >> 3) ^ (row & (CHUNKS - 1))) + 2 * (col & 7);
          *reinterpret_cast<uint16_t*>(stg + off) = (uint16_t)f32_to_bf16_bits(acc[i][j][r]);
        }
#pragma unroll
      for (int q = 0; q < 16 / RPQ; ++q) {
        const int row = q * RPQ + lane / CHUNKS, ch = lane % CHUNKS;
        const uint4 v =
            *reinterpret_cast<const uint4*>(stg + row * PITCH + 16 * (ch ^ (row & (CHUNKS - 1))));
        const int at = i * 32 + 16 * h + row;
        if (at < rows && ch * 8 < cols)
          *reinterpret_cast<uint4*>(c + (size_t)at * ld + ch * 16) = v;
      }
    }
}

// The same value by value: fp32, and bf16 rows of odd lengths. STREAM: stores
// that leave the caches to the operands.
template <class C, typename T, bool STREAM = false>
__device__ __forceinline__ void store_plain(const Acc<C>& acc, char* c, size_t ld, int rows,
                                            int cols, int lane) {
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      const int col = j * 32 + acc_col(lane);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int row = i * 32 + acc_row(r, lane);
        if (row < rows && col < cols) {
          T* dst = reinterpret_cast<T*>(c + (size_t)row * ld) + col;
          if constexpr (sizeof(T) == 2) *dst = (T)f32_to_bf16_bits(acc[i][j][r]);
          else if constexpr (STREAM) __builtin_nontemporal_store(acc[i][j][r], dst);
          else *dst = acc[i][j][r];
        }
      }
    }
}

// One tile of c (BMODE kOutRows: W's rows are the output's columns) or of da
// (kRedRows: they are the reduction).
struct TileRows {
  int e, row0, rows;
  int red;  // 0 for rows of no group: nothing is read, the sums are 0
};
template <class C>
__device__ __forceinline__ void grouped_tile(const ProductArgs& p, const TileRows& t, int col0,
                                             char* const (&ring)[C::NSTAGE], int lane, int wave) {
  const size_t a_ld = (size_t)p.red * C::ES;
  OutRowsSource<C, C::AR, C::A_LOADS, true> a;
  a.init(
      nullptr, [&](int r) { return p.a + (size_t)a_row(p, t.row0 + min(r, t.rows - 1)) * a_ld; },
      t.red, 0, lane, wave);
  const char* w = p.w + (size_t)t.e * p.red * p.cols * C::ES;
  Acc<C> acc;
  clear<C>(acc);
  const int wm = wave / C::WN, wn = wave % C::WN;
  Reader<C, kOutRows, C::AR, C::FM> ra;
  ra.init(wm * C::TM, lane);
  Reader<C, C::BMODE, C::BN, C::FN> rb;
  rb.init(wn * C::TN, lane);
  const int nsteps = (t.red + C::BK - 1) / C::BK;
  if constexpr (C::BMODE == kOutRows) {
    OutRowsSource<C, C::BN, C::B_LOADS> b;
    b.init(
        w + (size_t)col0 * a_ld,
        [&](int r) { return (uint32_t)(min(r, p.cols - 1 - col0) * a_ld); }, t.red, 0, lane, wave);
    run<C>(acc, ring, a, b, ra, rb, nsteps, lane, wave);
  } else {
    RedRowsSource<C, C::BN, C::B_LOADS, SameRow> b;
    b.init(w, (size_t)p.cols * C::ES, col0, p.cols, t.red, 0, SameRow{}, lane, wave);
    run<C>(acc, ring, a, b, ra, rb, nsteps, lane, wave);
  }

  const size_t c_ld = (size_t)p.cols * C::ES;
  char* c = p.c + (size_t)(t.row0 + wm * C::TM) * c_ld + (size_t)(col0 + wn * C::TN) * C::ES;
  const int rl = t.rows - wm * C::TM, cl = p.cols - col0 - wn * C::TN;
  if constexpr (C::E == kF32) {
    store_plain<C, float>(acc, c, c_ld, rl, cl, lane);
  } else if (p.cols % 8 == 0) {
    static_assert(C::WAVES * 16 * C::TN * 2 <= C::STAGE, "staging fits a stage");
    lds_barrier();  // every wave is done with the ring
    store_bf16<C>(acc, ring[0] + wave * 16 * C::TN * 2, c, c_ld, rl, cl, lane);
  } else {
    store_plain<C, uint16_t>(acc, c, c_ld, rl, cl, lane);
  }
}

// Tiles of one width and heights of 64 to 64 FMAX rows (FMAX blocks of 32 for
// each of two waves). A group has the fewest rows of tiles that hold it, all
// equally high: 532 rows are three of 192, not two of 256 and one almost empty.
// One copy of the product for each height.
template <int E_, int FMAX_, int BN_, int WN_, int NSTAGE_, int BMODE_, bool ALIGNED_>
struct Family {
  static constexpr int NSTAGE = NSTAGE_;
  static constexpr int E = E_, FMAX = FMAX_, BN = BN_, WN = WN_, BMODE = BMODE_;
  static constexpr bool ALIGNED = ALIGNED_;
  template <int FM>
  using Height =
      Cfg<E, 1, 64 * FM, BN, 2, WN, NSTAGE, kOutRows, BMODE, ALIGNED, NSTAGE == 2 ? 128 : 64>;
  using Most = Height<FMAX>;
};

template <class F>
__global__ __launch_bounds__(F::Most::THREADS) void grouped_kernel(ProductArgs p, int run_items) {
  __shared__ __attribute__((aligned(1024))) char st0[F::Most::STAGE];
  __shared__ __attribute__((aligned(1024))) char st1[F::Most::STAGE];
  __shared__ __attribute__((aligned(1024))) char st2[F::NSTAGE > 2 ? F::Most::STAGE : 16];
  __shared__ __attribute__((aligned(1024))) char st3[F::NSTAGE > 3 ? F::Most::STAGE : 16];
  char* all[4] = {st0, st1, st2, st3};
  char* ring[F::NSTAGE];
#pragma unroll
  for (int s = 0; s < F::NSTAGE; ++s) ring[s] = all[s];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int item = xcd_item(grid_block(), run_items);
  const GroupTile g =
      find_tile<F::Most::BM>(p.offsets, p.G, p.M, p.tiles_n, p.fill, item, lane);
  if (g.e < 0) return;  // the whole workgroup
  const int height = (((unsigned)(g.hi - g.lo) + g.tiles - 1) / g.tiles + 63) / 64 * 64;
  TileRows t;
  t.e = g.e < p.G ? g.e : 0;
  t.red = g.e < p.G ? p.red : 0;
  t.row0 = g.lo + g.i * height;
  t.rows = min(height, g.hi - t.row0);
  if (t.rows <= 0) return;  // rounding up left the last tiles empty
  const int col0 = g.col_tile * F::BN;
  if (height == 64) {
    grouped_tile<typename F::template Height<1>>(p, t, col0, ring, lane, wave);
  } else if (F::FMAX <= 2 || height == 128) {
    grouped_tile<typename F::template Height<2>>(p, t, col0, ring, lane, wave);
  } else if constexpr (F::FMAX > 2) {
    if (height == 192) grouped_tile<typename F::template Height<3>>(p, t, col0, ring, lane, wave);
    else grouped_tile<typename F::template Height<4>>(p, t, col0, ring, lane, wave);
  }
}

// ---- groups of few rows (bf16): bound by reading W ------------------------------
// A workgroup computes 16 columns of c for up to 16 rows of a group: each of its
// four waves takes a quarter of K straight from memory into
// v_mfma_f32_16x16x32_bf16 (W's rows as the first operand, so a lane ends with
// four neighbours of a row of c); the quarters are added in order through LDS.
// Nothing is shared that LDS could keep: W is read once, and the rows of a come from
// L2. The source asks for eight loads of W at a time; the compiler turns the zeros of
// what is out of range into an address on the stack, so the loads are flat ones: six
// pairs are in flight together, the seventh and the eighth wait one by one, and none
// of the next eight is ahead. At K = 2048 that is six trips to memory in a row: one
// token of 8 experts 2048 -> 1408 takes 11.4 us, its bytes 9.1.
constexpr int kFewRows = 16, kFewCols = 16;
constexpr int kFewWaves = 4;

__global__ __launch_bounds__(64 * kFewWaves) void grouped_few_kernel(ProductArgs p) {
  constexpr int U = 8;  // slices of 32 in flight
  __shared__ f32x4 sums[kFewWaves][64];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const GroupTile g =
      find_tile<kFewRows>(p.offsets, p.G, p.M, p.tiles_n, p.fill, (int)grid_block(), lane);
  if (g.e < 0) return;  // the whole workgroup
  const int row0 = g.lo + g.i * kFewRows, rows = min(kFewRows, g.hi - row0);
  const int col0 = g.col_tile * kFewCols;
  const int e = g.e < p.G ? g.e : 0, red = g.e < p.G ? p.red : 0;  // (no group: sums of 0)
  const int slices = (red + 31) / 32, per = (slices + kFewWaves - 1) / kFewWaves;
  const int s0 = wave * per, s1 = min(slices, s0 + per);
  const int k0 = 8 * (lane >> 4);  // this lane's chunk of a slice
  const uint16_t* w = reinterpret_cast<const uint16_t*>(p.w) +
                      ((size_t)e * p.cols + min(col0 + (lane & 15), p.cols - 1)) * p.red + k0;
  const uint16_t* a = reinterpret_cast<const uint16_t*>(p.a) +
                      (size_t)a_row(p, row0 + min(lane & 15, rows - 1)) * p.red + k0;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int s = s0; s < s1; s += U) {
    uint4 wv[U], av[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = s + u < s1 && 32 * (s + u) + k0 < red;
      wv[u] = in ? *reinterpret_cast<const uint4*>(w + 32 * (s + u)) : zero;
      av[u] = in ? *reinterpret_cast<const uint4*>(a + 32 * (s + u)) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, wv[u]),
                                                    __builtin_bit_cast(bf16x8, av[u]), acc, 0, 0, 0);
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave) return;
  f32x4 c = sums[0][lane];
#pragma unroll
  for (int v = 1; v < kFewWaves; ++v) c += sums[v][lane];
  const int row = lane & 15, col = col0 + 4 * (lane >> 4);
  if (row < rows && col < p.cols)  // (cols is a multiple of 8)
    *reinterpret_cast<uint2*>(p.c + ((size_t)(row0 + row) * p.cols + col) * 2) =
        make_uint2(pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]));
}

// dW: one workgroup per expert, tile of its O x K entries and range of its rows
// (`splits` equal ranges, whose sums are added in order by a second launch, so
// that the result is the same each run). The rows are taken kListRows at a time,
// their rows of a listed in LDS first.
constexpr int kListRows = 1024;

struct DwArgs {
  const char* a;   // [a_rows][K]
  const char* dc;  // [M][O]
  float* dw;       // [splits][G][O][K]
  const int32_t* offsets;
  const int32_t* perm;
  int k, a_rows, M, G, O, K, tiles_o, tiles_k, splits;
};

template <class C>
__global__ __launch_bounds__(C::THREADS) void grouped_dw_kernel(DwArgs p, int run_items) {
  __shared__ __attribute__((aligned(1024))) char st0[C::STAGE];
  __shared__ __attribute__((aligned(1024))) char st1[C::STAGE];
  __shared__ __attribute__((aligned(1024))) char st2[C::NSTAGE > 2 ? C::STAGE : 16];
  __shared__ __attribute__((aligned(1024))) char st3[C::NSTAGE > 3 ? C::STAGE : 16];
  __shared__ int32_t list[kListRows];
  char* all[4] = {st0, st1, st2, st3};
  char* ring[C::NSTAGE];
#pragma unroll
  for (int s = 0; s < C::NSTAGE; ++s) ring[s] = all[s];

  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const unsigned item = xcd_item(grid_block(), run_items), tiles = p.tiles_o * p.tiles_k;
  const unsigned range = item / tiles;
  const int e = range / p.splits, split = range % p.splits;
  if (e >= p.G) return;
  const int t = item % tiles;
  const int o0 = t / p.tiles_k * C::BM, k0 = t % p.tiles_k * C::BN;
  int2 rows = group_rows_of(p.offsets, e, p.M);
  const unsigned all_rows = rows.y - rows.x, len = (all_rows + p.splits - 1) / p.splits;
  rows.x += (int)min(all_rows, split * len);
  const int count = (int)min((unsigned)(rows.y - rows.x), len);

  Acc<C> acc;
  clear<C>(acc);
  const int wm = wave / C::WN, wn = wave % C::WN;
  Reader<C, kRedRows, C::BM, C::FM> ra;
  ra.init(wm * C::TM, lane);
  Reader<C, kRedRows, C::BN, C::FN> rb;
  rb.init(wn * C::TN, lane);
  for (int done = 0, n; done < count; done += n) {
    const int q0 = rows.x + done;
    n = min(kListRows, count - done);
    __syncthreads();  // every wave is done with the list and the ring
    for (int i = threadIdx.x; i < n; i += C::THREADS) {
      const int q = q0 + i;
      list[i] = p.perm ? min(max(p.perm[q] / p.k, 0), p.a_rows - 1) : q;
    }
    __syncthreads();
    RedRowsSource<C, C::BM, C::A_LOADS, SameRow> a;
    a.init(p.dc + (size_t)q0 * p.O * C::ES, (size_t)p.O * C::ES, o0, p.O, n, 0, SameRow{}, lane,
           wave);
    RedRowsSource<C, C::BN, C::B_LOADS, ListedRow> b;
    b.init(p.a, (size_t)p.K * C::ES, k0, p.K, n, 0, ListedRow{list}, lane, wave);
    run<C>(acc, ring, a, b, ra, rb, (n + C::BK - 1) / C::BK, lane, wave);
  }
  const int ol = o0 + wm * C::TM, kl = k0 + wn * C::TN;
  char* dst = reinterpret_cast<char*>(p.dw + (((size_t)split * p.G + e) * p.O + ol) * p.K + kl);
  // whole 128-byte lines stream past the caches (64 experts of 2048 x 2048: 490 -> 450
  // us); others are put together in them
  if (p.K % 32 == 0)
    store_plain<C, float, true>(acc, dst, (size_t)p.K * 4, p.O - ol, p.K - kl, lane);
  else
    store_plain<C, float, false>(acc, dst, (size_t)p.K * 4, p.O - ol, p.K - kl, lane);
}

// dw = the sum of the ranges' parts, in order. n: entries of dw.
__global__ __launch_bounds__(256) void grouped_dw_sum_kernel(const float* part, int splits, size_t n,
                                                             float* dw) {
  const size_t i = ((size_t)grid_block() * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  if (i + 4 <= n && n % 4 == 0) {
    float4 s = *reinterpret_cast<const float4*>(part + i);
#pragma unroll 8
    for (int v = 1; v < splits; ++v) {
      const float4 x = *reinterpret_cast<const float4*>(part + v * n + i);
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    *reinterpret_cast<float4*>(dw + i) = s;
  } else {
    for (size_t j = i; j < n && j < i + 4; ++j) {
      float s = part[j];
      for (int v = 1; v < splits; ++v) s += part[v * n + j];
      dw[j] = s;
    }
  }
}

// Rows of tiles of up to `high` rows: a group's last may be short, so at most one more
// per group with rows, and per end with rows of no group; each holds a row.
size_t rows_of_tiles(const ProductArgs& p, int high) {
  return std::min((size_t)p.M / high + std::min(p.G, p.M) + 2 * p.fill, (size_t)p.M);
}

template <class F>
hipError_t launch_grouped_cfg(ProductArgs p, hipStream_t s) {
  p.tiles_n = (p.cols + F::BN - 1) / F::BN;
  const size_t tiles_m = rows_of_tiles(p, F::Most::BM);
  const size_t items = tiles_m * p.tiles_n;
  const int run_items = items >= 1024 ? 32 : 1;
  const size_t super = 8 * run_items;
  return launch_kernel(grouped_kernel<F>, grid_rows((items + super - 1) / super * super),
                       dim3(F::Most::THREADS), 0, s, KernelTiming{}, p, run_items);
}

hipError_t launch_few(ProductArgs p, hipStream_t s) {
  p.tiles_n = (p.cols + kFewCols - 1) / kFewCols;
  return launch_kernel(grouped_few_kernel, grid_rows(rows_of_tiles(p, kFewRows) * p.tiles_n),
                       dim3(64 * kFewWaves), 0, s, KernelTiming{}, p);
}

template <class C>
hipError_t launch_grouped_dw_cfg(DwArgs p, hipStream_t s) {
  p.tiles_o = (p.O + C::BM - 1) / C::BM;
  p.tiles_k = (p.K + C::BN - 1) / C::BN;
  const size_t items = (size_t)p.G * p.splits * p.tiles_o * p.tiles_k;
  const int run_items = items >= 1024 ? 32 : 1;
  const size_t super = 8 * run_items;
  return launch_kernel(grouped_dw_kernel<C>, grid_rows((items + super - 1) / super * super),
                       dim3(C::THREADS), 0, s, KernelTiming{}, p, run_items);
}

// (rows through registers: two stages of twice the reduction, 3 to 8 % faster)
template <int E, bool ALIGNED>
using DwTile128 =
    Cfg<E, 1, 128, 128, 2, 2, ALIGNED ? 4 : 2, kRedRows, kRedRows, ALIGNED, ALIGNED ? 64 : 128>;
template <int E>
using DwTile256 = Cfg<E, 1, 256, 256, 2, 4, 4, kRedRows, kRedRows, true>;
// The tile's width by the time of its rounds over the CUs: one workgroup of 256
// columns fits a CU, two of 128, three of 64; with fewer, a tile of 64 is done
// first. Rows x reduction x columns, groups, 256, 128, 64 wide: 8192 x 512 x 1024,
// 64: 21, 29, 29 us; 8192 x 1024 x 512, 64: 22, 30, -; 4096 x 1024 x 1024, 16: 26,
// 21, 22.5; 256 x 1024 x 1024, 16: 13.7, 13.2, 11.7; 2000 x 512 x 512, 8: 14.5, 8.9,
// 8.4.
template <int E, int BMODE>
hipError_t launch_grouped_type(const ProductArgs& p, hipStream_t s) {
  constexpr int EPC = E == kF32 ? 4 : 8;
  const long long used = p.G < p.M ? p.G : p.M;  // groups with rows, at most
  const auto items = [&](int high, int wide) {
    return (double)(used * (p.M / used / high + 1) * ((p.cols + wide - 1) / wide));
  };
  const double t256 = std::max(0.8, items(256, 256) * (0.8 / 256));
  const double t128 = std::max(0.62, items(128, 128) * (1.0 / 512));
  const double t64 = std::max(0.56, items(128, 64) * (1.0 / 1000));
  if (p.red % EPC != 0 || (BMODE == kRedRows && p.cols % EPC != 0))
    return t64 < t128 ? launch_grouped_cfg<Family<E, 2, 64, 2, 2, BMODE, false>>(p, s)
                      : launch_grouped_cfg<Family<E, 2, 128, 2, 2, BMODE, false>>(p, s);
  if constexpr (E == kBf16) {
    // Few rows per group and few tiles even of 64 columns: one token of 8 experts
    // of 256, 2048 x 1408, 11.4 us against 20 (memory 9.1); 72 rows of 13 experts,
    // 640 x 2640 (546 tiles), 18 against 11.
    if (BMODE == kOutRows && p.cols % 8 == 0 && p.M / used <= 16 && items(128, 64) < 256)
      return launch_few(p, s);
    if (t256 < t128 && t256 < t64)
      return launch_grouped_cfg<Family<E, 4, 256, 4, 4, BMODE, true>>(p, s);
  }
  return t64 < t128 ? launch_grouped_cfg<Family<E, 2, 64, 2, 2, BMODE, true>>(p, s)
                    : launch_grouped_cfg<Family<E, 2, 128, 2, 2, BMODE, true>>(p, s);
}

// Tiles of 256 x 256 where three quarters of the CUs get one: 32768 rows, 64
// experts of 2048 x 2048, 400 us against 540 with 128 x 128; 131072 rows, 256 of
// 512 x 512, 106 against 115.
bool dw_large(bmoe_dtype dt, int O, int K, int G) {
  return dt == BMOE_BF16 && O % 8 == 0 && K % 8 == 0 && O >= 256 && K >= 256 &&
         (long long)G * ((O + 255) / 256) * ((K + 255) / 256) >= 192;
}

template <int E>
hipError_t launch_dw_type(const DwArgs& p, hipStream_t s) {
  constexpr int EPC = E == kF32 ? 4 : 8;
  if (p.O % EPC != 0 || p.K % EPC != 0) return launch_grouped_dw_cfg<DwTile128<E, false>>(p, s);
  if constexpr (E == kBf16)
    if (dw_large(BMOE_BF16, p.O, p.K, p.G)) return launch_grouped_dw_cfg<DwTile256<E>>(p, s);
  return launch_grouped_dw_cfg<DwTile128<E, true>>(p, s);
}

}  // namespace

hipError_t launch_grouped(bmoe_dtype dt, bool back, int M, int red, int cols, int G, const void* a,
                          const int32_t* perm, int k, int a_rows, const void* w,
                          const int32_t* offsets, void* c, bool fill, hipStream_t s) {
  ProductArgs p;
  p.a = static_cast<const char*>(a);
  p.w = static_cast<const char*>(w);
  p.c = static_cast<char*>(c);
  p.offsets = offsets;
  p.perm = perm;
  p.k = k;
  p.a_rows = a_rows;
  p.M = M;
  p.G = G;
  p.red = red;
  p.cols = cols;
  p.tiles_n = 0;
  p.fill = fill;
  if (dt == BMOE_BF16)
    return back ? launch_grouped_type<kBf16, kRedRows>(p, s)
                : launch_grouped_type<kBf16, kOutRows>(p, s);
  return back ? launch_grouped_type<kF32, kRedRows>(p, s)
              : launch_grouped_type<kF32, kOutRows>(p, s);
}

// Ranges per group: enough that 128 x 128 tiles fill the CUs twice over, of at
// least 128 rows on average (parts cost 8 bytes an entry).
int grouped_dw_splits(bmoe_dtype dt, int M, int O, int K, int G) {
  if (dw_large(dt, O, K, G)) return 1;
  const long long tiles = (long long)G * ((O + 127) / 128) * ((K + 127) / 128);
  const long long most = M / G / 128;
  const long long want = 512 / tiles;
  return (int)std::max(1LL, std::min(std::min(want, most), 64LL));
}

hipError_t launch_grouped_dw(bmoe_dtype dt, int M, int O, int K, int G, const void* a,
                             const int32_t* perm, int k, int a_rows, const void* dc,
                             const int32_t* offsets, float* dw, float* part, hipStream_t s) {
  DwArgs p;
  p.a = static_cast<const char*>(a);
  p.dc = static_cast<const char*>(dc);
  p.splits = grouped_dw_splits(dt, M, O, K, G);
  p.dw = p.splits > 1 ? part : dw;
  p.offsets = offsets;
  p.perm = perm;
  p.k = k;
  p.a_rows = a_rows;
  p.M = M;
  p.G = G;
  p.O = O;
  p.K = K;
  p.tiles_o = p.tiles_k = 0;
  const hipError_t e = dt == BMOE_BF16 ? launch_dw_type<kBf16>(p, s) : launch_dw_type<kF32>(p, s);
  if (e != hipSuccess || p.splits == 1) return e;
  const size_t n = (size_t)G * O * K;
  return launch_kernel(grouped_dw_sum_kernel, grid_rows((n + 1023) / 1024), dim3(256), 0, s,
                       KernelTiming{}, (const float*)part, p.splits, n, dw);
}

}  // namespace bmoe
