// Tiles of matrix products C = A B through LDS rings, shared by the grouped
// products and the Newton-Schulz products.
//
// An operand's memory rows run either along the output (kOutRows: [m][k], the
// reduction contiguous) or along the reduction (kRedRows: [k][m]). A K-step is
// 64 bytes of reduction per output row: 32 values of 16 bits, 16 of fp32. Its
// 16-byte chunks go to LDS by DMA, XOR-swizzled so that fragment reads spread
// over the banks; kRedRows fragments of 16-bit types are gathered by gfx950's
// transposing LDS read. Steps past the reduction's end, and chunks past it,
// read zeros, so every step issues the same number of DMA instructions and the
// counted waits are exact.
//
// ALIGNED = false serves rows that are no multiple of 16 bytes: chunks are put
// together from single elements in registers and written to the same places.
//
// PARTS = 2: operands are pairs (hi, lo) whose sum is the value; the product
// is hi hi + hi lo + lo hi (three MFMAs per pair of fragments read, so LDS and
// L2 traffic per MFMA are two thirds of a plain product's).
#pragma once

#include "common.h"

namespace bmoe {
namespace tile {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint64_t u64x2v __attribute__((ext_vector_type(2)));

enum Elem { kBf16, kF16, kF32 };
enum Mode { kOutRows, kRedRows };

// Sixteen zero bytes: the DMA source of what lies past the reduction's end.
__device__ const uint4 kZeros = {0u, 0u, 0u, 0u};

template <int E_, int PARTS_, int BM_, int BN_, int WM_, int WN_, int NSTAGE_, int AMODE_,
          int BMODE_, bool ALIGNED_>
struct Cfg {
  static constexpr int E = E_, PARTS = PARTS_, BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int NSTAGE = NSTAGE_, AHEAD = NSTAGE - 1, AMODE = AMODE_, BMODE = BMODE_;
  static constexpr bool ALIGNED = ALIGNED_;
  static constexpr int ES = E == kF32 ? 4 : 2;  // bytes per element
  static constexpr int EPC = 16 / ES;           // elements per chunk
  static constexpr int BK = 64 / ES;            // reduction per K-step
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  static constexpr int A_PART = BM * 64, B_PART = BN * 64;
  static constexpr int A_BYTES = PARTS * A_PART, B_BYTES = PARTS * B_PART;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int A_LOADS = A_PART / 1024 / WAVES, B_LOADS = B_PART / 1024 / WAVES;
  static constexpr int V = PARTS * (A_LOADS + B_LOADS);  // DMA instructions per wave and step
  static_assert(A_LOADS >= 1 && B_LOADS >= 1 && AHEAD * V <= 63, "DMA counts");
  static_assert(FM >= 1 && FN >= 1 && FM * FN * 16 <= 256, "accumulators");
  static_assert(NSTAGE * STAGE <= 160 * 1024, "LDS budget");
};

template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | (((N >> 4) & 3) << 14));
}

__device__ __forceinline__ void dma16(const void* g, char* lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                   (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

// `n` elements at p (n <= 0: none) as one chunk, the rest zeros.
template <int ES>
__device__ __forceinline__ u32x4 partial_chunk(const char* p, int n) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if constexpr (ES == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n)
        v[i / 2] |= (uint32_t) * reinterpret_cast<const uint16_t*>(p + 2 * i) << (16 * (i & 1));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) v[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
  }
  return v;
}

// ---- kOutRows: LDS rows of 64 bytes -------------------------------------------
// Four rows fill the 256 bytes of the banks once; sixteen lanes reading one
// chunk of sixteen rows meet every bank group once with this swizzle.
__device__ __forceinline__ int out_swz(int row, int ch) { return ch ^ ((row >> 2) & 3); }

template <class C, int R, int LOADS>
struct OutRowsSource {
  const char* p[LOADS];  // this lane's chunk of step 0
  int k0[LOADS];         // its first reduction index
  int K;
  size_t part;           // bytes between the parts
  // row_of(r): address of the row of output row r (0 <= r < R; any valid row
  // for those past the end, whose outputs are not stored).
  template <typename F>
  __device__ __forceinline__ void init(F row_of, int K_, size_t part_, int lane, int wave) {
    K = K_;
    part = part_;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int e = (wave * LOADS + j) * 64 + lane;
      const int row = e >> 2, ch = out_swz(row, e & 3);
      p[j] = row_of(row) + ch * 16;
      k0[j] = ch * C::EPC;
    }
  }
  __device__ __forceinline__ void load(char* region, int step, int lane, int wave) const {
#pragma unroll
    for (int q = 0; q < C::PARTS; ++q)
#pragma unroll
      for (int j = 0; j < LOADS; ++j) {
        const int left = K - k0[j] - step * C::BK;
        const char* g = p[j] + q * part + (size_t)step * 64;
        char* dst = region + q * (R * 64) + (wave * LOADS + j) * 1024;
        if constexpr (C::ALIGNED) {
          dma16(left > 0 ? (const void*)g : (const void*)&kZeros, dst);
        } else {
          *reinterpret_cast<u32x4*>(dst + lane * 16) = partial_chunk<C::ES>(g, left);
        }
      }
  }
};

// ---- kRedRows: LDS rows of R elements -------------------------------------------
// The four rows of a transposing read (fp32: the rows of the two lane halves)
// land on different bank ranges.
template <int ES, int R>
__device__ __forceinline__ int red_swz(int r, int ch) {
  if constexpr (ES == 4) return ch ^ (((r >> 2) & 1) << 3);
  else if constexpr (R >= 128) return ch ^ ((r & 3) << 2);
  else return ch ^ (((r >> 1) & 1) << 2);
}

// The memory row of reduction index k: k itself, or a row number that the
// workgroup put in LDS.
struct SameRow {
  __device__ __forceinline__ size_t operator()(int k) const { return (size_t)k; }
};
struct ListedRow {
  const int32_t* list;
  __device__ __forceinline__ size_t operator()(int k) const { return (size_t)list[k]; }
};

template <class C, int R, int LOADS, class MAP>
struct RedRowsSource {
  const char* base;
  size_t ld, part;      // bytes per row, between the parts
  int r[LOADS];         // row within a step
  uint32_t col[LOADS];  // byte offset of the chunk's column
  int cols_left[LOADS]; // columns from it on (ALIGNED = false)
  int K;
  MAP map;
  // Columns c0 .. of `cols`; ALIGNED needs cols to be whole chunks (chunks past
  // the last repeat it: their outputs are not stored).
  __device__ __forceinline__ void init(const char* base_, size_t ld_, int c0, int cols, int K_,
                                       size_t part_, MAP map_, int lane, int wave) {
    static_assert(R * C::ES / 16 >= 8, "swizzle range");
    base = base_;
    ld = ld_;
    part = part_;
    K = K_;
    map = map_;
    constexpr int CH = R / C::EPC;  // chunks per row
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int e = (wave * LOADS + j) * 64 + lane;
      r[j] = e / CH;
      const int c = c0 + red_swz<C::ES, R>(r[j], e % CH) * C::EPC;
      cols_left[j] = cols - c;
      col[j] = (uint32_t)((C::ALIGNED ? min(c, cols - C::EPC) : min(c, cols - 1)) * C::ES);
    }
  }
  __device__ __forceinline__ void load(char* region, int step, int lane, int wave) const {
#pragma unroll
    for (int q = 0; q < C::PARTS; ++q)
#pragma unroll
      for (int j = 0; j < LOADS; ++j) {
        const int k = step * C::BK + r[j];
        const bool in = k < K;
        const char* g = base + q * part + map(in ? k : 0) * ld + col[j];
        char* dst = region + q * (R * 64) + (wave * LOADS + j) * 1024;
        if constexpr (C::ALIGNED) {
          dma16(in ? (const void*)g : (const void*)&kZeros, dst);
        } else {
          *reinterpret_cast<u32x4*>(dst + lane * 16) =
              partial_chunk<C::ES>(g, in ? cols_left[j] : 0);
        }
      }
  }
};

// ---- fragments --------------------------------------------------------------------
// 16-bit types: lane l holds output row l % 32 of its block, reduction 8 (l /
// 32) + 0..7 of a slice of 16 (one MFMA). fp32: reduction 4 (l / 32) + 0..3 of
// a slice of 8 (four MFMAs of two each). A K-step is two slices.
template <class C, int MODE, int R, int F>
struct Reader {
  uint32_t off[MODE == kOutRows ? 2 : F];
  __device__ __forceinline__ void init(int row0, int lane) {
    if constexpr (MODE == kOutRows) {
      const int row = row0 + (lane & 31);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) off[kk] = row * 64 + 16 * out_swz(row, 2 * kk + (lane >> 5));
    } else if constexpr (C::ES == 2) {
      // In each 16-lane group, lane 4j + q points at row kb + j, columns 4q ..
      // 4q + 3 of the group's 16; the read hands lane i column i of these rows.
      const int gr = lane >> 4, L = lane & 15;
      const int r0 = 8 * (gr >> 1) + (L >> 2);
#pragma unroll
      for (int i = 0; i < F; ++i) {
        const int c = row0 + 32 * i + 16 * (gr & 1) + 4 * (L & 3);
        off[i] = r0 * (R * 2) + red_swz<2, R>(r0, c >> 3) * 16 + (c & 7) * 2;
      }
    } else {
      const int r0 = 4 * (lane >> 5);
#pragma unroll
      for (int i = 0; i < F; ++i) {
        const int c = row0 + 32 * i + (lane & 31);
        off[i] = r0 * (R * 4) + red_swz<4, R>(r0, c >> 2) * 16 + (c & 3) * 4;
      }
    }
  }
  // The F fragments of slice KK, part q.
  template <int KK>
  __device__ __forceinline__ void read(u32x4 (&f)[F], const char* region, int q) const {
    const char* s = region + q * (R * 64);
#pragma unroll
    for (int i = 0; i < F; ++i) {
      if constexpr (MODE == kOutRows) {
        f[i] = *reinterpret_cast<const u32x4*>(s + off[KK] + i * 32 * 64);
      } else if constexpr (C::ES == 2) {
        typedef __attribute__((address_space(3))) v4s lds_v4s;
        const char* p = s + off[i] + KK * 16 * R * 2;
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p);
        const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * R * 2));
        const u64x2v x = {__builtin_bit_cast(uint64_t, lo), __builtin_bit_cast(uint64_t, hi)};
        f[i] = __builtin_bit_cast(u32x4, x);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f[i][j] = *reinterpret_cast<const uint32_t*>(s + off[i] + (8 * KK + j) * R * 4);
      }
    }
  }
};

template <int E>
__device__ __forceinline__ void mma(f32x16& acc, const u32x4& a, const u32x4& b) {
  if constexpr (E == kBf16) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  } else if constexpr (E == kF16) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                 __builtin_bit_cast(f16x8, b), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[j]), __uint_as_float(b[j]), acc,
                                                 0, 0, 0);
  }
}

template <class C>
using Acc = f32x16[C::FM][C::FN];

template <class C>
__device__ __forceinline__ void clear(Acc<C>& acc) {
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
}

template <class C, int KK, class RA, class RB>
__device__ __forceinline__ void read_slice(u32x4 (&fa)[C::PARTS][C::FM],
                                           u32x4 (&fb)[C::PARTS][C::FN], const char* stg,
                                           const RA& ra, const RB& rb) {
#pragma unroll
  for (int q = 0; q < C::PARTS; ++q) {
    ra.template read<KK>(fa[q], stg, q);
    rb.template read<KK>(fb[q], stg + C::A_BYTES, q);
  }
}

template <class C>
__device__ __forceinline__ void mma_slice(Acc<C>& acc, const u32x4 (&fa)[C::PARTS][C::FM],
                                          const u32x4 (&fb)[C::PARTS][C::FN]) {
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      if constexpr (C::PARTS == 2) {
        mma<C::E>(acc[i][j], fa[0][i], fb[1][j]);
        mma<C::E>(acc[i][j], fa[1][i], fb[0][j]);
      }
      mma<C::E>(acc[i][j], fa[0][i], fb[0][j]);
    }
}

template <class C, class SA, class SB>
__device__ __forceinline__ void issue(char* stg, const SA& a, const SB& b, int step, int lane,
                                      int wave) {
  a.load(stg, step, lane, wave);
  b.load(stg + C::A_BYTES, step, lane, wave);
  __asm__ volatile("" ::: "memory");
}

// One K-step out of ring stage S (the stages are separate arrays and S is a
// constant, so the compiler can tell the stage read from the stages being
// filled and waits only for these reads).
template <class C, int S, class SA, class SB, class RA, class RB>
__device__ __forceinline__ void step(Acc<C>& acc, char* const (&ring)[C::NSTAGE], const SA& a,
                                     const SB& b, const RA& ra, const RB& rb, int kt, int lane,
                                     int wave) {
  __asm__ volatile("" ::: "memory");
  // this wave's part of step kt has landed once only the later steps' are out
  wait_vm<(C::AHEAD - 1) * C::V>();
  // every wave's has, and every wave is done with step kt - 1, whose stage the
  // next DMA overwrites
  lds_barrier();
  issue<C>(ring[(S + C::AHEAD) % C::NSTAGE], a, b, kt + C::AHEAD, lane, wave);
  u32x4 fa[C::PARTS][C::FM], fb[C::PARTS][C::FN], ga[C::PARTS][C::FM], gb[C::PARTS][C::FN];
  read_slice<C, 0>(fa, fb, ring[S], ra, rb);
  read_slice<C, 1>(ga, gb, ring[S], ra, rb);
  mma_slice<C>(acc, fa, fb);
  mma_slice<C>(acc, ga, gb);
}

// acc += the product over steps [0, nsteps), taken in whole rounds of the ring
// (the steps past nsteps add zeros; leaving a round early would cost a copy of
// the accumulators per exit). All of the workgroup's waves call it with the
// same nsteps; on return no DMA is in flight, but other waves may still be
// reading the ring.
template <class C, class SA, class SB, class RA, class RB>
__device__ __forceinline__ void run(Acc<C>& acc, char* const (&ring)[C::NSTAGE], const SA& a,
                                    const SB& b, const RA& ra, const RB& rb, int nsteps, int lane,
                                    int wave) {
#pragma unroll
  for (int s = 0; s < C::AHEAD; ++s) issue<C>(ring[s], a, b, s, lane, wave);
  for (int kt = 0; kt < nsteps; kt += C::NSTAGE) {
    step<C, 0>(acc, ring, a, b, ra, rb, kt, lane, wave);
    step<C, 1>(acc, ring, a, b, ra, rb, kt + 1, lane, wave);
    if constexpr (C::NSTAGE > 2) step<C, 2>(acc, ring, a, b, ra, rb, kt + 2, lane, wave);
    if constexpr (C::NSTAGE > 3) step<C, 3>(acc, ring, a, b, ra, rb, kt + 3, lane, wave);
  }
  wait_vm<0>();
}

// Row and column, within its 32 x 32 block, of accumulator register r of a lane.
__device__ __forceinline__ int acc_row(int r, int lane) {
  return 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
}
__device__ __forceinline__ int acc_col(int lane) { return lane & 31; }

// Workgroups are dealt to the eight XCDs in turn: the work item of workgroup b,
// so that runs of `run` consecutive items share an XCD's L2.
__device__ __forceinline__ int xcd_item(int b, int run) {
  const int super = 8 * run;
  return b / super * super + (b % 8) * run + (b % super) / 8;
}

}  // namespace tile
}  // namespace bmoe
