// Matrix products grouped by expert, ragged groups:
//   c[q]  = W_e a[row(q)]                  rows q of group e, e = 0 .. G - 1
//   da[q] = W_e^T dc[q]
//   dW_e  = sum over the rows q of e of dc[q] a[row(q)]^T      (fp32)
// with group e the rows offsets[e] .. offsets[e + 1] and row(q) = perm[q] / k
// (q itself without perm). The offsets live on the device: a workgroup finds
// its tile of a group from them, so the host never waits for the router.
#include "common.h"
#include "kernels.h"
#include "tile_product.h"

namespace bmoe {
namespace {

using namespace tile;

struct GroupTile {
  int e, row0, rows;  // group, its tile's rows; e = -1: no such tile
  int height;         // 64, 128, ... MOST: the tile's rows rounded up
  int col_tile;
};

// Rows of group e, whatever the offsets hold.
__device__ __forceinline__ int2 group_rows_of(const int32_t* offsets, int e, int M) {
  const int lo = min(max(offsets[e], 0), M), hi = min(max(offsets[e + 1], 0), M);
  return make_int2(lo, max(lo, hi));
}

// Work item t of all groups' tiles, groups ascending. A group has the fewest
// rows of tiles of at most MOST rows that hold it, all equally high (in 64s): 532
// rows are three of 192, not two of 256 and one almost empty. Its tiles come in
// panels of four rows of tiles, so that the consecutive items that share an L2
// are near square. Every wave looks its tile up for itself: 64 groups at a time,
// a prefix sum over the lanes.
constexpr int kPanel = 4;
template <int MOST>
__device__ __forceinline__ GroupTile find_tile(const int32_t* offsets, int G, int M, int tiles_n,
                                               int t, int lane) {
  int before = 0;
  for (int e0 = 0; e0 < G; e0 += kWave) {
    int2 r = make_int2(0, 0);
    if (e0 + lane < G) r = group_rows_of(offsets, e0 + lane, M);
    const int n = (r.y - r.x + MOST - 1) / MOST * tiles_n;
    const int incl = wave_incl_scan(n);
    const uint64_t past = __ballot(before + incl > t);
    if (past) {
      const int src = __ffsll((unsigned long long)past) - 1;
      const int lo = __builtin_amdgcn_readlane(r.x, src), hi = __builtin_amdgcn_readlane(r.y, src);
      const int items = __builtin_amdgcn_readlane(n, src), tiles = items / tiles_n;
      const int i = t - before - (__builtin_amdgcn_readlane(incl, src) - items);
      const int panel = i / (kPanel * tiles_n), j = i - panel * kPanel * tiles_n;
      const int rows_of_tiles = min(kPanel, tiles - panel * kPanel);
      GroupTile g;
      g.e = e0 + src;
      g.height = ((hi - lo + tiles - 1) / tiles + 63) / 64 * 64;
      g.row0 = lo + (panel * kPanel + j % rows_of_tiles) * g.height;
      g.rows = min(g.height, hi - g.row0);  // none where rounding up left the last tiles empty
      g.col_tile = j / rows_of_tiles;
      return g;
    }
    before += __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  return {-1, 0, 0, 0, 0};
}

struct ProductArgs {
  const char* a;  // rows of the product's left operand, `red` values each
  const char* w;  // [G][O][K]
  char* c;        // [M][cols]
  const int32_t* offsets;
  const int32_t* perm;  // NULL: row q of a is row q of the product
  int k, a_rows, M, G, red, cols, tiles_n;
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

// The same value by value: fp32, and bf16 rows of odd lengths.
template <class C, typename T>
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
          else *dst = acc[i][j][r];
        }
      }
    }
}

// One tile of c (BMODE kOutRows: W's rows are the output's columns) or of da
// (kRedRows: they are the reduction).
template <class C>
__device__ __forceinline__ void grouped_tile(const ProductArgs& p, const GroupTile& t, int col0,
                                             char* const (&ring)[C::NSTAGE], int lane, int wave) {
  const size_t a_ld = (size_t)p.red * C::ES;
  OutRowsSource<C, C::AR, C::A_LOADS, true> a;
  a.init(
      nullptr, [&](int r) { return p.a + (size_t)a_row(p, t.row0 + min(r, t.rows - 1)) * a_ld; },
      p.red, 0, lane, wave);
  const char* w = p.w + (size_t)t.e * p.red * p.cols * C::ES;
  Acc<C> acc;
  clear<C>(acc);
  const int wm = wave / C::WN, wn = wave % C::WN;
  Reader<C, kOutRows, C::AR, C::FM> ra;
  ra.init(wm * C::TM, lane);
  Reader<C, C::BMODE, C::BN, C::FN> rb;
  rb.init(wn * C::TN, lane);
  const int nsteps = (p.red + C::BK - 1) / C::BK;
  if constexpr (C::BMODE == kOutRows) {
    OutRowsSource<C, C::BN, C::B_LOADS> b;
    b.init(
        w + (size_t)col0 * a_ld,
        [&](int r) { return (uint32_t)(min(r, p.cols - 1 - col0) * a_ld); }, p.red, 0, lane, wave);
    run<C>(acc, ring, a, b, ra, rb, nsteps, lane, wave);
  } else {
    RedRowsSource<C, C::BN, C::B_LOADS, SameRow> b;
    b.init(w, (size_t)p.cols * C::ES, col0, p.cols, p.red, 0, SameRow{}, lane, wave);
    run<C>(acc, ring, a, b, ra, rb, nsteps, lane, wave);
  }

  const size_t c_ld = (size_t)p.cols * C::ES;
  char* c = p.c + (size_t)(t.row0 + wm * C::TM) * c_ld + (size_t)(col0 + wn * C::TN) * C::ES;
  const int rl = t.rows - wm * C::TM, cl = p.cols - col0 - wn * C::TN;
  if constexpr (C::E == kBf16 && C::ALIGNED) {
    static_assert(C::WAVES * 16 * C::TN * 2 <= C::STAGE, "staging fits a stage");
    lds_barrier();  // every wave is done with the ring
    store_bf16<C>(acc, ring[0] + wave * 16 * C::TN * 2, c, c_ld, rl, cl, lane);
  } else if constexpr (C::E == kBf16) {
    store_plain<C, uint16_t>(acc, c, c_ld, rl, cl, lane);
  } else {
    store_plain<C, float>(acc, c, c_ld, rl, cl, lane);
  }
}

// Tiles of one width and heights of 64 to 64 FMAX rows (FMAX blocks of 32 for
// each of two waves), chosen per tile: one copy of the product for each.
template <int E_, int FMAX_, int BN_, int WN_, int NSTAGE_, int BMODE_, bool ALIGNED_>
struct Family {
  static constexpr int NSTAGE = NSTAGE_;
  static constexpr int E = E_, FMAX = FMAX_, BN = BN_, WN = WN_, BMODE = BMODE_;
  static constexpr bool ALIGNED = ALIGNED_;
  template <int FM>
  using Height = Cfg<E, 1, 64 * FM, BN, 2, WN, NSTAGE, kOutRows, BMODE, ALIGNED, NSTAGE == 2 ? 128 : 64>;
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
  const GroupTile t = find_tile<F::Most::BM>(p.offsets, p.G, p.M, p.tiles_n, item, lane);
  if (t.e < 0 || t.rows <= 0) return;  // the whole workgroup
  const int col0 = t.col_tile * F::BN;
  if (t.height == 64) {
    grouped_tile<typename F::template Height<1>>(p, t, col0, ring, lane, wave);
  } else if (F::FMAX <= 2 || t.height == 128) {
    grouped_tile<typename F::template Height<2>>(p, t, col0, ring, lane, wave);
  } else if constexpr (F::FMAX > 2) {
    if (t.height == 192) grouped_tile<typename F::template Height<3>>(p, t, col0, ring, lane, wave);
    else grouped_tile<typename F::template Height<4>>(p, t, col0, ring, lane, wave);
  }
}

// dW: one workgroup per expert and tile of its O x K entries. The rows of a
// group are taken kListRows at a time, their rows of a listed in LDS first.
constexpr int kListRows = 1024;

struct DwArgs {
  const char* a;   // [a_rows][K]
  const char* dc;  // [M][O]
  float* dw;       // [G][O][K]
  const int32_t* offsets;
  const int32_t* perm;
  int k, a_rows, M, G, O, K, tiles_o, tiles_k;
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
  const int e = item / tiles;
  if (e >= p.G) return;
  const int t = item % tiles;
  const int o0 = t / p.tiles_k * C::BM, k0 = t % p.tiles_k * C::BN;
  const int2 rows = group_rows_of(p.offsets, e, p.M);

  Acc<C> acc;
  clear<C>(acc);
  const int wm = wave / C::WN, wn = wave % C::WN;
  Reader<C, kRedRows, C::BM, C::FM> ra;
  ra.init(wm * C::TM, lane);
  Reader<C, kRedRows, C::BN, C::FN> rb;
  rb.init(wn * C::TN, lane);
  for (int q0 = rows.x; q0 < rows.y; q0 += kListRows) {
    const int n = min(kListRows, rows.y - q0);
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
  char* dst = reinterpret_cast<char*>(p.dw + ((size_t)e * p.O + ol) * p.K + kl);
  store_plain<C, float>(acc, dst, (size_t)p.K * 4, p.O - ol, p.K - kl, lane);
}

template <class F>
hipError_t launch_grouped_cfg(ProductArgs p, hipStream_t s) {
  p.tiles_n = (p.cols + F::BN - 1) / F::BN;
  // a group's last tile may be short: at most one more tile per group with rows
  const size_t tiles_m = (size_t)p.M / F::Most::BM + (p.G < p.M ? p.G : p.M);
  const size_t items = tiles_m * p.tiles_n;
  const int run_items = items >= 1024 ? 32 : 1;
  const size_t super = 8 * run_items;
  return launch_kernel(grouped_kernel<F>, grid_rows((items + super - 1) / super * super),
                       dim3(F::Most::THREADS), 0, s, KernelTiming{}, p, run_items);
}

template <class C>
hipError_t launch_grouped_dw_cfg(DwArgs p, hipStream_t s) {
  p.tiles_o = (p.O + C::BM - 1) / C::BM;
  p.tiles_k = (p.K + C::BN - 1) / C::BN;
  const size_t items = (size_t)p.G * p.tiles_o * p.tiles_k;
  const int run_items = items >= 1024 ? 32 : 1;
  const size_t super = 8 * run_items;
  return launch_kernel(grouped_dw_kernel<C>, grid_rows((items + super - 1) / super * super),
                       dim3(C::THREADS), 0, s, KernelTiming{}, p, run_items);
}

template <int E, bool ALIGNED>
using DwTile128 = Cfg<E, 1, 128, 128, 2, 2, 4, kRedRows, kRedRows, ALIGNED>;
template <int E>
using DwTile256 = Cfg<E, 1, 256, 256, 2, 4, 4, kRedRows, kRedRows, true>;

template <int E, int BMODE>
hipError_t launch_grouped_type(const ProductArgs& p, hipStream_t s) {
  constexpr int EPC = E == kF32 ? 4 : 8;
  if (p.red % EPC != 0 || p.cols % EPC != 0)
    return launch_grouped_cfg<Family<E, 2, 128, 2, 2, BMODE, false>>(p, s);
  if constexpr (E == kF32) return launch_grouped_cfg<Family<E, 2, 128, 2, 2, BMODE, true>>(p, s);
  else return launch_grouped_cfg<Family<E, 4, 256, 4, 4, BMODE, true>>(p, s);
}

template <int E>
hipError_t launch_dw_type(const DwArgs& p, hipStream_t s) {
  constexpr int EPC = E == kF32 ? 4 : 8;
  if (p.O % EPC == 0 && p.K % EPC == 0) {
    if constexpr (E == kBf16)
      if (p.O >= 256 && p.K >= 256) return launch_grouped_dw_cfg<DwTile256<E>>(p, s);
    return launch_grouped_dw_cfg<DwTile128<E, true>>(p, s);
  }
  return launch_grouped_dw_cfg<DwTile128<E, false>>(p, s);
}

}  // namespace

hipError_t launch_grouped(bmoe_dtype dt, bool back, int M, int red, int cols, int G, const void* a,
                          const int32_t* perm, int k, int a_rows, const void* w,
                          const int32_t* offsets, void* c, hipStream_t s) {
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
  if (dt == BMOE_BF16)
    return back ? launch_grouped_type<kBf16, kRedRows>(p, s)
                : launch_grouped_type<kBf16, kOutRows>(p, s);
  return back ? launch_grouped_type<kF32, kRedRows>(p, s)
              : launch_grouped_type<kF32, kOutRows>(p, s);
}

hipError_t launch_grouped_dw(bmoe_dtype dt, int M, int O, int K, int G, const void* a,
                             const int32_t* perm, int k, int a_rows, const void* dc,
                             const int32_t* offsets, float* dw, hipStream_t s) {
  DwArgs p;
  p.a = static_cast<const char*>(a);
  p.dc = static_cast<const char*>(dc);
  p.dw = dw;
  p.offsets = offsets;
  p.perm = perm;
  p.k = k;
  p.a_rows = a_rows;
  p.M = M;
  p.G = G;
  p.O = O;
  p.K = K;
  p.tiles_o = p.tiles_k = 0;
  return dt == BMOE_BF16 ? launch_dw_type<kBf16>(p, s) : launch_dw_type<kF32>(p, s);
}

}  // namespace bmoe
