// Gradient of the router's product l = x W_r^T, from the gradient of its
// logits dl [T][N] (fp32):
//   dx[t][c] = dx_add[t][c] + sum_e dl[t][e] W_r[e][c]
//   dW[e][c] = sum_t dl[t][e] x[t][c]
// Three ways: from the picks alone where only they move (sparse), on bf16 MFMA
// with dl in three bf16 parts (dense, bf16), on fp32 MFMA (dense, fp32).
#include "common.h"
#include "kernels.h"

namespace bmoe {
namespace {

// ---- sparse dl -------------------------------------------------------------------
// Where only the k picks of a token move (every spec but softmax without
// renorm), dl is k pairs (id, coefficient) per token: 4 T k d flops instead of
// 4 T N d, no rounding of dl, rows of W and of dW picked by id. The tokens are
// cut into ranges; within each the pairs are also listed by expert, in token
// order (launch_route_pairs). One launch does both products:
//
// dx: a thread takes 16 bytes of a row; the k rows of W come from L2.
// dW: a workgroup takes one expert, four consecutive ranges (one per wave) and
//     up to 64 V columns (V values per 16 bytes). Each lane keeps V sums in
//     registers while its wave walks the expert's list of its range (rows
//     narrower than a wave: several at once); the sums are added in order
//     through LDS, those of the groups of ranges by the join kernel, so the
//     order of every sum is fixed. The workgroups of a group of ranges run
//     together and walk the tokens upwards, so the k readers of a row of x
//     meet in the caches: in one L2 where a row has eight column chunks or
//     more (workgroups go to the eight XCDs in turn, so chunk c to XCD c % 8),
//     else in two to eight of them and the last-level cache.
// One launch, the dW workgroups first. Measured at T = 32768, d = 4096, 256
// experts, top 4 (bf16): dW 96 us and dx 117 us in launches of their own (dx
// moves 537 MB: 100 us at the rate of a large copy; dW gathers 1.07 GB of x
// through L2), the call 223 us so (235 us at six waves per SIMD instead of
// eight) and 237 us with two launches; T = 4096, d = 512, 64 experts, top 2
// 16.8 to 17.8 and 19.8 us. Alternating the roles' workgroups costs dW its hits
// in L2 (245 us with every third, 257 us with every fifth a dW one).
template <typename T>
struct SparseArgs {
  const int2* pairs;   // [T][k]
  const int2* list;    // (token, coefficient), by range and expert
  const int32_t* off;  // [ranges][N + 1] into list
  const T* x;
  const T* w;
  const T* dx_add;
  T* dx;
  float* dw;  // [groups of 4 ranges][N][d] (one group: the result itself)
  int T_, d, N, k, ranges;
  int chunks;     // column chunks of a row (a power of two, as d)
  unsigned n_dw;  // workgroups of the dW role
};

constexpr int kU = 8;  // rows of x in flight per lane

template <typename T, bool WIDE>
__device__ __forceinline__ void sparse_dw(const SparseArgs<T>& p, unsigned block, float* sums) {
  constexpr int V = 16 / sizeof(T);
  const int chunk = block & (p.chunks - 1), re = block >> __builtin_ctz(p.chunks);
  const int e = re % p.N, group = re / p.N;
  const int lpr = WIDE ? 64 : p.d / V;  // lanes per row
  const int slots = 64 / lpr;           // rows that a wave takes at once
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int slot = WIDE ? 0 : lane / lpr;
  const int col = lane % lpr * V;
  const int c = chunk * 64 * V + col;
  const int range = group * 4 + wave;
  int lo = 0, hi = 0;
  if (range < p.ranges) {
    const int32_t* off = p.off + (size_t)range * (p.N + 1) + e;
    lo = off[0];
    hi = off[1];
  }
  const T* x = p.x + c;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  if constexpr (WIDE) {
    // 64 list entries at a time, one per lane; their rows by readlane, so only
    // the rows' own loads wait on memory, kU of them in flight per lane
    for (int q0 = lo; q0 < hi; q0 += 64) {
      const int n = min(64, hi - q0);
      const int2 ent = p.list[q0 + min(lane, n - 1)];
      auto row = [&](int i) {
        return *reinterpret_cast<const u32x4*>(
            x + (size_t)__builtin_amdgcn_readlane(ent.x, i) * p.d);
      };
      auto add = [&](u32x4 v, int i) {
        const float f = __int_as_float(__builtin_amdgcn_readlane(ent.y, i));
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if constexpr (V == 8) {
            acc[2 * u] = fmaf(f, bf16_lo(v[u]), acc[2 * u]);
            acc[2 * u + 1] = fmaf(f, bf16_hi(v[u]), acc[2 * u + 1]);
          } else {
            acc[u] = fmaf(f, __uint_as_float(v[u]), acc[u]);
          }
        }
      };
      int i = 0;
      for (; i + kU <= n; i += kU) {
        u32x4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) v[u] = row(i + u);
#pragma unroll
        for (int u = 0; u < kU; ++u) add(v[u], i + u);
      }
      for (; i < n; ++i) add(row(i), i);
    }
  } else {
    for (int q = lo + slot; q < hi; q += slots) {
      const int2 ent = p.list[q];
      float v[V];
      load16(x + (size_t)ent.x * p.d, v);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(__int_as_float(ent.y), v[i], acc[i]);
    }
  }
  // sums[slot][col]
  const int cols = lpr * V;
#pragma unroll
  for (int i = 0; i < V; ++i) sums[(wave * slots + slot) * cols + col + i] = acc[i];
  __syncthreads();
  float* dst = p.dw + ((size_t)group * p.N + e) * p.d + chunk * 64 * V;
  for (int i = threadIdx.x; i < cols; i += 256) {
    float a = sums[i];
    for (int r = 1; r < 4 * slots; ++r) a += sums[r * cols + i];
    dst[i] = a;
  }
}

template <typename T, bool WIDE>
__device__ __forceinline__ void sparse_dx(const SparseArgs<T>& p, unsigned block) {
  constexpr int V = 16 / sizeof(T);
  const int per_row = p.d / V;
  const size_t u = (size_t)block * 256 + threadIdx.x;
  if (u >= (size_t)p.T_ * per_row) return;
  size_t t = u / per_row;
  // a wave's 64 threads share a row: its pairs come as scalars
  if (WIDE) t = (size_t)__builtin_amdgcn_readfirstlane((int)t);
  const int c = (int)(u % per_row) * V;
  float acc[V], v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  const int2* pr = p.pairs + t * p.k;
  const T* w = p.w + c;
  int j = 0;
  for (; j + 4 <= p.k; j += 4) {  // four rows of W in flight
    int2 q[4];
    bool all = true;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      q[u] = pr[j + u];
      all &= __int_as_float(q[u].y) != 0.f;
    }
    if (!all) break;
    float r[4][V];
#pragma unroll
    for (int u = 0; u < 4; ++u) load16(w + (size_t)q[u].x * p.d, r[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(__int_as_float(q[u].y), r[u][i], acc[i]);
  }
  for (; j < p.k; ++j) {  // the rest, and picks that add nothing
    const float f = __int_as_float(pr[j].y);
    if (f == 0.f) continue;
    load16(w + (size_t)pr[j].x * p.d, v);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = fmaf(f, v[i], acc[i]);
  }
  // (streamed, so that W and the dW role's rows of x keep the caches)
  if (p.dx_add) {
    const u32x4 a =
        __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p.dx_add + t * p.d + c));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (V == 8) {
        acc[2 * i] += bf16_lo(a[i]);
        acc[2 * i + 1] += bf16_hi(a[i]);
      } else {
        acc[i] += __uint_as_float(a[i]);
      }
    }
  }
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (V == 8) o[i] = pack_bf16x2(acc[2 * i], acc[2 * i + 1]);
    else o[i] = __float_as_uint(acc[i]);
  }
  __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(p.dx + t * p.d + c));
}

template <typename T, bool WIDE>
__global__ __launch_bounds__(256, 8) void router_sparse_kernel(SparseArgs<T> p) {
  __shared__ float sums[256 * (16 / sizeof(T))];
  const unsigned block = grid_block();
  if (block < p.n_dw) sparse_dw<T, WIDE>(p, block, sums);
  else sparse_dx<T, WIDE>(p, block - p.n_dw);
}

// dw = the ranges' sums, added in order.
__global__ __launch_bounds__(256) void router_dw_join_kernel(const float4* part, int S, size_t n4,
                                                             float4* dw) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  float4 a = part[i];
#pragma unroll 4
  for (int s = 1; s < S; ++s) {
    const float4 b = part[(size_t)s * n4 + i];
    a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
  }
  dw[i] = a;
}

template <typename T>
hipError_t sparse_t(int Tn, int d, int N, int k, const T* x, const T* w, const RouterPairs& rp,
                    const T* dx_add, T* dx, float* dw, float* part, hipStream_t s) {
  constexpr int V = 16 / sizeof(T);
  SparseArgs<T> p;
  p.pairs = rp.pairs;
  p.list = rp.list;
  p.off = rp.off;
  p.x = x;
  p.w = w;
  p.dx_add = dx_add;
  p.dx = dx;
  const int groups = (rp.ranges + 3) / 4;
  p.ranges = rp.ranges;
  p.dw = groups == 1 ? dw : part;
  p.T_ = Tn;
  p.d = d;
  p.N = N;
  p.k = k;
  p.chunks = (d + 64 * V - 1) / (64 * V);
  p.n_dw = (unsigned)p.chunks * N * groups;
  const dim3 grid = grid_rows(p.n_dw + ((size_t)Tn * (d / V) + 255) / 256);
  const hipError_t e = d >= 64 * V ? launch_kernel(router_sparse_kernel<T, true>, grid, dim3(256),
                                                   0, s, KernelTiming{}, p)
                                   : launch_kernel(router_sparse_kernel<T, false>, grid,
                                                   dim3(256), 0, s, KernelTiming{}, p);
  if (e != hipSuccess || groups == 1) return e;
  const size_t n4 = (size_t)N * d / 4;
  return launch_kernel(router_dw_join_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, s,
                       KernelTiming{}, reinterpret_cast<const float4*>(part), groups, n4,
                       reinterpret_cast<float4*>(dw));
}

// ---- dense dl, bf16: MFMA ----------------------------------------------------------
// dl as three bf16 parts (their products with bf16 x and W are exact, so only
// the fp32 sums round): three MFMAs per fragment into one accumulator.
// Operands whose reduction index is the row index of their matrix go through
// LDS tiles of padded rows and gfx950's transposing read: lane l gets column
// l % 32 and rows 8 (l / 32) + 0..7 of a 16-row slice from two reads. Rows are
// padded so that four neighbours start 64 bytes apart in the banks.
typedef short rb_v4s __attribute__((ext_vector_type(4)));
typedef uint64_t rb_u64x2 __attribute__((ext_vector_type(2)));

// Work item of this workgroup: XCD x (workgroups are dealt to the eight in turn)
// takes a run of consecutive items, the column tiles of the same tokens, so
// that those tokens' parts are fetched into one L2 only.
__device__ __forceinline__ unsigned xcd_item() {
  const unsigned b = blockIdx.x, n = gridDim.x;
  return n % 8 == 0 ? b % 8 * (n / 8) + b / 8 : b;
}

// Byte offset of this lane's first read for the 32 columns from col, slice 0.
template <int STRIDE>
__device__ __forceinline__ uint32_t tr_offset(int col, int lane) {
  const int gr = lane >> 4, L = lane & 15;
  return (uint32_t)((8 * (gr >> 1) + (L >> 2)) * STRIDE + (col + 16 * (gr & 1) + 4 * (L & 3)) * 2);
}
template <int STRIDE>
__device__ __forceinline__ bf16x8 tr_read(const char* p) {
  typedef __attribute__((address_space(3))) rb_v4s lds_v4s;
  const rb_v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p);
  const rb_v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * STRIDE));
  const rb_u64x2 x = {__builtin_bit_cast(uint64_t, lo), __builtin_bit_cast(uint64_t, hi)};
  return __builtin_bit_cast(bf16x8, x);
}

// dx: 64 tokens x 128 columns per workgroup, 4 waves of 32 x 64. W goes to LDS
// 64 experts at a time; the parts come straight from memory, stored in operand
// order (by token and expert the call took 73 us, 11 more), dx_add is under way
// from the start. The tile leaves through LDS (the W tile's, done with by
// then), so dx_add and dx move in 128-byte pieces of a row. Small tiles, so that
// several workgroups share a CU and one's loads run under another's MFMAs:
// three with dx_add (132 registers), four without. At T = 16384, d = 2048, 64
// experts 128 x 128 tiles at two per CU took 56 us, these 31 us (134 MB).
constexpr int kDxStrideW = 128 * 2 + 64;

template <bool ADD>
__global__ __launch_bounds__(256) void router_dx_mfma_kernel(const uint16_t* parts,
                                                             const uint16_t* w,
                                                             const uint16_t* dx_add, int T_, int d,
                                                             int N, uint16_t* dx) {
  __shared__ __attribute__((aligned(16))) float lds[4 * 32 * 68];
  static_assert(sizeof(lds) >= 64 * kDxStrideW, "the W tile shares it");
  char* const ws = reinterpret_cast<char*>(lds);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  float* const tile = lds + wave * (32 * 68);
  const unsigned item = xcd_item(), tiles = (d + 127) / 128;
  const int c0 = item % tiles * 128, np = router_parts_experts(N);
  const int t0 = (int)(item / tiles) * 64 + wm * 32;
  // (tokens past the end: whatever is there, in rows that are not stored)
  const uint16_t* ablock = parts + (size_t)(min(t0, T_ - 1) / 32) * (96 * (size_t)np) + lane * 8;
  // This lane's piece u of the tile: row (u * 64 + lane) / 8, 8 columns.
  const int cc = lane % 8 * 8, c = c0 + wn * 64 + cc;
  u32x4 add[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    add[u] = u32x4{0u, 0u, 0u, 0u};
    if constexpr (ADD)
      add[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(
          dx_add + (size_t)min(t0 + u * 8 + lane / 8, T_ - 1) * d + (c < d ? c : 0)));
  }
  uint32_t off[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) off[j] = tr_offset<kDxStrideW>(wn * 64 + 32 * j, lane);
  f32x16 acc[2] = {f32x16{}, f32x16{}};

  for (int e0 = 0; e0 < np; e0 += 64) {
    u32x4 a[4][3];
#pragma unroll
    for (int sl = 0; sl < 4; ++sl)
#pragma unroll
      for (int p = 0; p < 3; ++p)
        a[sl][p] =
            *reinterpret_cast<const u32x4*>(ablock + ((size_t)(e0 / 16 + sl) * 3 + p) * 512);
    u32x4 b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = e0 + (tid + u * 256) / 16, cb = c0 + (tid + u * 256) % 16 * 8;
      // (past the end: any row and column; the parts there are 0, and nothing
      // past d is stored)
      b[u] = *reinterpret_cast<const u32x4*>(w + (size_t)min(e, N - 1) * d + (cb < d ? cb : 0));
    }
    if (e0 > 0) __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *reinterpret_cast<u32x4*>(ws + (tid + u * 256) / 16 * kDxStrideW + (tid + u * 256) % 16 * 16) =
          b[u];
    __syncthreads();
#pragma unroll
    for (int sl = 0; sl < 4; ++sl) {
      bf16x8 bf[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) bf[j] = tr_read<kDxStrideW>(ws + off[j] + sl * 16 * kDxStrideW);
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a[sl][p]),
                                                           bf[j], acc[j], 0, 0, 0);
    }
  }
  __syncthreads();  // W is done with
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      tile[(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * 68 + 32 * j + (lane & 31)] = acc[j][r];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int row = u * 8 + lane / 8, t = t0 + row;
    if (t >= T_ || c >= d) continue;
    const float4 v0 = *reinterpret_cast<const float4*>(tile + row * 68 + cc);
    const float4 v1 = *reinterpret_cast<const float4*>(tile + row * 68 + cc + 4);
    u32x4 o;
    o[0] = pack_bf16x2(v0.x + bf16_lo(add[u][0]), v0.y + bf16_hi(add[u][0]));
    o[1] = pack_bf16x2(v0.z + bf16_lo(add[u][1]), v0.w + bf16_hi(add[u][1]));
    o[2] = pack_bf16x2(v1.x + bf16_lo(add[u][2]), v1.y + bf16_hi(add[u][2]));
    o[3] = pack_bf16x2(v1.z + bf16_lo(add[u][3]), v1.w + bf16_hi(add[u][3]));
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(dx + (size_t)t * d + c));
  }
}

// dW: 64 experts x 256 columns per workgroup and range of tokens, 8 waves of
// 32 x 64, 64 tokens per step; two LDS buffers filled through registers, one
// barrier per step.
constexpr int kDwStrideA = 192 * 2 + 64, kDwStrideB = 256 * 2 + 64;

__global__ __launch_bounds__(512) void router_dw_mfma_kernel(const uint16_t* parts,
                                                             const uint16_t* x, int T_, int d,
                                                             int N, int tokens_per_split,
                                                             float* out) {
  __shared__ __attribute__((aligned(16))) char as[2][64 * kDwStrideA];
  __shared__ __attribute__((aligned(16))) char bs[2][64 * kDwStrideB];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 2, wn = wave & 3;
  const int np = router_parts_experts(N);
  const unsigned item = xcd_item(), tiles_c = (d + 255) / 256, tiles = tiles_c * (np / 64);
  const unsigned split = item / tiles, tile = item % tiles;
  const int c0 = tile % tiles_c * 256, e0 = tile / tiles_c * 64;
  const size_t t0 = (size_t)split * tokens_per_split;
  const int rows = t0 < (size_t)T_ ? (int)min((size_t)tokens_per_split, (size_t)T_ - t0) : 0;
  const uint16_t* ap = parts + t0 / 32 * (96 * (size_t)np) + (size_t)(e0 / 16) * 1536;
  const uint16_t* bp = x + t0 * d + c0;
  const uint32_t offa = tr_offset<kDwStrideA>(wm * 96, lane);
  uint32_t offb[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) offb[j] = tr_offset<kDwStrideB>(wn * 64 + 32 * j, lane);
  f32x16 acc[2] = {f32x16{}, f32x16{}};
  u32x4 ra[2][3] = {}, rb[2][4] = {};
  // This thread's pieces of a step: offsets in the step's rows of the parts and
  // of x, and in LDS.
  int row_a[3], row_b[4];
  uint32_t at_a[3], at_b[4], lds_a[3], lds_b[4];
#pragma unroll
  for (int u = 0; u < 3; ++u) {
    // 16 bytes of the step's two token blocks, four slices of sixteen experts,
    // three parts and 64 lanes: a token's eight experts of one part
    const int piece = tid + u * 512, l = piece % 64, part = piece / 64 % 3;
    const int sl = piece / 192 % 4, e = sl * 16 + l / 32 * 8;
    row_a[u] = piece / 768 * 32 + l % 32;
    at_a[u] = (uint32_t)((sl * 3 + part) * 512 + l * 8);
    lds_a[u] = row_a[u] * kDwStrideA + (e / 32 * 96 + part * 32 + e % 32) * 2;
  }
  const int ch_b = tid % 32;
  const bool in_d = c0 + ch_b * 8 < d;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    row_b[u] = (tid + u * 512) / 32;
    at_b[u] = (uint32_t)(row_b[u] * d + (in_d ? ch_b * 8 : 0));
    lds_b[u] = row_b[u] * kDwStrideB + ch_b * 16;
  }
  // Rows past the end load the last row and become zeros on their way to LDS,
  // as do columns past d. Every step issues the same loads, without a branch:
  // only then do the compiler's waits for one step's leave the next in flight.
  auto load = [&](int r0, u32x4 (&a)[3], u32x4 (&b)[4]) {
    r0 = min(r0, rows - 1);
    const uint16_t* pb = bp + (size_t)r0 * d;
    const int most = rows - 1 - r0;
#pragma unroll
    for (int u = 0; u < 3; ++u) {  // (a block holds 32 tokens: those past the end are there)
      const int block = min(r0 / 32 + row_a[u] / 32, (rows - 1) / 32);
      a[u] = *reinterpret_cast<const u32x4*>(ap + (size_t)block * (96 * (size_t)np) + at_a[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      b[u] = *reinterpret_cast<const u32x4*>(pb +
                                             (at_b[u] - (uint32_t)(max(0, row_b[u] - most) * d)));
  };
  auto store = [&](int r0, int buf, const u32x4 (&a)[3], const u32x4 (&b)[4]) {
    const int left = rows - r0;
    const bool all = left >= 64 && c0 + 256 <= d;
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      u32x4 v = a[u];
      if (!all && row_a[u] >= left) v = u32x4{0u, 0u, 0u, 0u};
      *reinterpret_cast<u32x4*>(as[buf] + lds_a[u]) = v;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      u32x4 v = b[u];
      if (!all && (row_b[u] >= left || !in_d)) v = u32x4{0u, 0u, 0u, 0u};
      *reinterpret_cast<u32x4*>(bs[buf] + lds_b[u]) = v;
    }
  };
  auto multiply = [&](int buf) {
#pragma unroll
    for (int sl = 0; sl < 4; ++sl) {
      bf16x8 a[3], b[2];
#pragma unroll
      for (int p = 0; p < 3; ++p)
        a[p] = tr_read<kDwStrideA>(as[buf] + offa + p * 64 + sl * 16 * kDwStrideA);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        b[j] = tr_read<kDwStrideB>(bs[buf] + offb[j] + sl * 16 * kDwStrideB);
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[p], b[j], acc[j], 0, 0, 0);
    }
  };
  // Step r0 is in LDS buffer (r0 / 64) % 2 while the next two are under way to
  // registers. Steps past the end add zeros.
  if (rows > 0) {
    load(0, ra[0], rb[0]);
    load(64, ra[1], rb[1]);
    store(0, 0, ra[0], rb[0]);
    for (int r0 = 0; r0 < rows; r0 += 128) {
      load(r0 + 128, ra[0], rb[0]);
      lds_barrier();
      multiply(0);
      store(r0 + 64, 1, ra[1], rb[1]);
      load(r0 + 192, ra[1], rb[1]);
      lds_barrier();
      multiply(1);
      store(r0 + 128, 0, ra[0], rb[0]);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = c0 + wn * 64 + 32 * j + (lane & 31);
    if (c >= d) continue;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int e = e0 + wm * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
      if (e < N) out[((size_t)split * N + e) * d + c] = acc[j][r];
    }
  }
}

// ---- dense dl, fp32: fp32 MFMA ------------------------------------------------------
// v_mfma_f32_32x32x2_f32: lane l gives element (l % 32, l / 32) of A and (l / 32,
// l % 32) of B, straight from memory. Exact fp32 products at 1/16 of the bf16
// rate: 226 to 231 us at T = 16384, d = 2048, 64 experts, three times what its
// bytes take. The split of both operands into bf16 parts (six products) would
// be faster and is left out, fp32 layers being small here.
//
// dx: 64 tokens x 128 columns per workgroup, 4 waves of 32 x 64. Eight experts
// per step: half h of the wave takes experts 4 h .. 4 h + 3 of them (any order
// of a sum's terms will do, as long as A and B agree), so its dl come as one
// 16-byte load (VEC: N is a multiple of 4).
template <bool VEC>
__global__ __launch_bounds__(256) void router_dx_f32_kernel(const float* dl, const float* w,
                                                            const float* dx_add, int T_, int d,
                                                            int N, float* dx) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int half = lane >> 5, col = lane & 31;
  const size_t t0 = (size_t)grid_block_z() * 64 + wave / 2 * 32;
  if (t0 >= (size_t)T_) return;  // (no barrier below)
  const int c0 = blockIdx.y * 128 + wave % 2 * 64;
  const float* row = dl + min(t0 + col, (size_t)T_ - 1) * N;
  const int ca = min(c0 + col, d - 1), cb = min(c0 + 32 + col, d - 1);
  f32x16 acc[2] = {f32x16{}, f32x16{}};
  for (int e0 = 0; e0 < N; e0 += 8) {
    float a[4], b0[4], b1[4];
    const int eh = e0 + 4 * half;
    if constexpr (VEC) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(row + min(eh, N - 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = row[min(eh + i, N - 1)];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* we = w + (size_t)min(eh + i, N - 1) * d;
      b0[i] = we[ca];
      b1[i] = we[cb];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = eh + i < N;
      const float x = in ? a[i] : 0.f;
      acc[0] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, in ? b0[i] : 0.f, acc[0], 0, 0, 0);
      acc[1] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, in ? b1[i] : 0.f, acc[1], 0, 0, 0);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const size_t t = t0 + 8 * (r >> 2) + 4 * half + (r & 3);
      const int c = c0 + 32 * j + col;
      if (t < (size_t)T_ && c < d) dx[t * d + c] = acc[j][r] + (dx_add ? dx_add[t * d + c] : 0.f);
    }
}

// dW: 64 experts x 64 columns per wave and range of tokens, two tokens per MFMA
// step, eight steps loaded ahead.
constexpr int kF32Rows = 16;

__global__ __launch_bounds__(64) void router_dw_f32_kernel(const float* dl, const float* x, int T_,
                                                           int d, int N, int tokens_per_split,
                                                           float* out) {
  const int lane = threadIdx.x, half = lane >> 5, col = lane & 31;
  const int c0 = blockIdx.x * 64, e0 = blockIdx.y * 64;
  const size_t t0 = (size_t)blockIdx.z * tokens_per_split;
  const size_t t1 = min(t0 + tokens_per_split, (size_t)T_);
  int e[2], c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    e[i] = min(e0 + 32 * i + col, N - 1);
    c[i] = min(c0 + 32 * i + col, d - 1);
  }
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
  for (size_t t = t0; t < t1; t += kF32Rows) {
    float a[8][2], b[8][2];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const size_t tr = min(t + 2 * u + half, t1 - 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[u][i] = dl[tr * N + e[i]];
        b[u][i] = x[tr * d + c[i]];
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool in = t + 2 * u + half < t1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[u][i] = in ? a[u][i] : 0.f;
        b[u][i] = in ? b[u][i] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[u][i], b[u][j], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int ee = e0 + 32 * i + 8 * (r >> 2) + 4 * half + (r & 3), cc = c0 + 32 * j + col;
        if (ee < N && cc < d) out[((size_t)blockIdx.z * N + ee) * d + cc] = acc[i][j][r];
      }
}

}  // namespace

// Tokens per range: 1024 at most (four ranges per dW workgroup), and shorter
// (down to 32) until the dW role has 4096 workgroups (T = 16384, d = 2048, 64
// experts: 55 us, with 2048 67 us, with 512 81 us).
int router_range_tokens(int T, int d, int N) {
  const int chunks = (d + 511) / 512;
  int r = 1024;
  while (r > 32 && ((long long)T + 4 * r - 1) / (4 * r) * N * chunks < 4096) r /= 2;
  return r;
}

hipError_t launch_router_bwd_sparse(bmoe_dtype dt, int T, int d, int N, int k, const void* x,
                                    const void* w, const RouterPairs& rp, const void* dx_add,
                                    void* dx, float* dw, float* part, hipStream_t s) {
  if (dt == BMOE_BF16)
    return sparse_t(T, d, N, k, static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w),
                    rp, static_cast<const uint16_t*>(dx_add), static_cast<uint16_t*>(dx), dw, part,
                    s);
  return sparse_t(T, d, N, k, static_cast<const float*>(x), static_cast<const float*>(w), rp,
                  static_cast<const float*>(dx_add), static_cast<float*>(dx), dw, part, s);
}

// Token ranges of the dense dW: one workgroup per CU (its LDS), at least four
// steps each.
int router_dense_splits(int T, int d, int N) {
  const int tiles = (d + 255) / 256 * (router_parts_experts(N) / 64);
  int S = (256 + tiles - 1) / tiles;
  const int most = (int)(((long long)T + 255) / 256);
  if (S > most) S = most;
  return S < 1 ? 1 : S;
}

hipError_t launch_router_bwd_parts(int T, int d, int N, const uint16_t* x, const uint16_t* w,
                                   const uint16_t* parts, const uint16_t* dx_add, uint16_t* dx,
                                   float* dw, float* part, hipStream_t s) {
  const dim3 gx(((unsigned)T + 63) / 64 * ((d + 127) / 128));
  hipError_t e = dx_add ? launch_kernel(router_dx_mfma_kernel<true>, gx, dim3(256), 0, s,
                                        KernelTiming{}, parts, w, dx_add, T, d, N, dx)
                        : launch_kernel(router_dx_mfma_kernel<false>, gx, dim3(256), 0, s,
                                        KernelTiming{}, parts, w, dx_add, T, d, N, dx);
  if (e != hipSuccess) return e;
  const int S = router_dense_splits(T, d, N);
  const int per = (int)((((long long)T + S - 1) / S + 63) / 64 * 64);
  e = launch_kernel(router_dw_mfma_kernel,
                    dim3((d + 255) / 256 * (router_parts_experts(N) / 64) * S), dim3(512), 0, s,
                    KernelTiming{}, parts, x, T, d, N, per, S == 1 ? dw : part);
  if (e != hipSuccess || S == 1) return e;
  const size_t n4 = (size_t)N * d / 4;
  return launch_kernel(router_dw_join_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, s,
                       KernelTiming{}, reinterpret_cast<const float4*>(part), S, n4,
                       reinterpret_cast<float4*>(dw));
}

// Token ranges of the fp32 dW: 2048 waves, at least 128 tokens each.
int router_f32_splits(int T, int d, int N) {
  const int tiles = (d + 63) / 64 * ((N + 63) / 64);
  int S = (2048 + tiles - 1) / tiles;
  const int most = (int)(((long long)T + 127) / 128);
  if (S > most) S = most;
  return S < 1 ? 1 : S;
}

hipError_t launch_router_bwd_f32(int T, int d, int N, const float* x, const float* w,
                                 const float* dl, const float* dx_add, float* dx, float* dw,
                                 float* part, hipStream_t s) {
  hipError_t e = hipSuccess;
  const dim3 gx = grid_rows_z(((unsigned)T + 63) / 64, (d + 127) / 128);
  if (T > 0)
    e = N % 4 == 0 ? launch_kernel(router_dx_f32_kernel<true>, gx, dim3(256), 0, s, KernelTiming{},
                                   dl, w, dx_add, T, d, N, dx)
                   : launch_kernel(router_dx_f32_kernel<false>, gx, dim3(256), 0, s,
                                   KernelTiming{}, dl, w, dx_add, T, d, N, dx);
  if (e != hipSuccess) return e;
  const int S = router_f32_splits(T, d, N);
  const int per = (int)((((long long)T + S - 1) / S + kF32Rows - 1) / kF32Rows * kF32Rows);
  e = launch_kernel(router_dw_f32_kernel, dim3((d + 63) / 64, (N + 63) / 64, S), dim3(64), 0, s,
                    KernelTiming{}, dl, x, T, d, N, per, S == 1 ? dw : part);
  if (e != hipSuccess || S == 1) return e;
  const size_t n4 = (size_t)N * d / 4;
  return launch_kernel(router_dw_join_kernel, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, s,
                       KernelTiming{}, reinterpret_cast<const float4*>(part), S, n4,
                       reinterpret_cast<float4*>(dw));
}

}  // namespace bmoe
