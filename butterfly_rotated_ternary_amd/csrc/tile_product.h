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
// ALIGNED = false serves rows that are no multiple of 16 bytes: chunks go through
// registers, loaded before a step's MFMAs and written to the same places behind
// them. 8192 rows, 64 experts of 1000 x 500 bf16, c, da and dW: 23, 34 and 44 us
// (38, 82 and 69 with the loads waited for at once), of 1000 x 504 by DMA 22, 24
// and 40.
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

// KB: bytes of reduction per output row and K-step, 64 or 128.
template <int E_, int PARTS_, int BM_, int BN_, int WM_, int WN_, int NSTAGE_, int AMODE_,
          int BMODE_, bool ALIGNED_, int KB_ = 64>
struct Cfg {
  static constexpr int E = E_, PARTS = PARTS_, BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int NSTAGE = NSTAGE_, AHEAD = NSTAGE - 1, AMODE = AMODE_, BMODE = BMODE_;
  static constexpr bool ALIGNED = ALIGNED_;
  static constexpr int ES = E == kF32 ? 4 : 2;  // bytes per element
  static constexpr int EPC = 16 / ES;           // elements per chunk
  static constexpr int KB = KB_, BK = KB / ES;  // reduction per K-step
  static constexpr int SLICES = KB / 32;        // of two chunks each
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  // a stage's A rows, rounded up so that every wave issues as many loads (the
  // rows past BM repeat others)
  static constexpr int GRAN = 1024 / KB * WAVES, AR = (BM + GRAN - 1) / GRAN * GRAN;
  static constexpr int A_PART = AR * KB, B_PART = BN * KB;
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

// !ALIGNED: chunks are single accesses, whatever their alignment; the chunk at a
// row's end takes the row's last 16 bytes, and end_chunk() moves its n elements
// down once they are needed. Rows shorter than a chunk are read element by
// element: n of them at p (n <= 0: none).
template <int ES>
__device__ __forceinline__ u32x4 short_chunk(const char* p, int n) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if constexpr (ES == 2) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n)
        v[i / 2] |= (uint32_t) * reinterpret_cast<const uint16_t*>(p + 2 * i) << (16 * (i & 1));
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < n) v[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
  }
  return v;
}
template <int ES>
__device__ __forceinline__ void end_chunk(u32x4& v, int n, int len) {
  constexpr int EPC = 16 / ES;
  if (n <= 0 || n >= EPC || len < EPC) return;
  const int bytes = (EPC - n) * ES;
  if (bytes & 8) v = u32x4{v[2], v[3], 0u, 0u};
  if (bytes & 4) v = u32x4{v[1], v[2], v[3], 0u};
  if (ES == 2 && (bytes & 2))
    v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
}

// ---- kOutRows: LDS rows of KB bytes -------------------------------------------
// Four (two) rows fill the 256 bytes of the banks once; sixteen lanes reading
// one chunk of sixteen rows meet every bank group once with this swizzle.
template <int KB>
__device__ __forceinline__ int out_swz(int row, int ch) {
  return KB == 64 ? ch ^ ((row >> 2) & 3) : ch ^ ((row >> 1) & 7);
}

// Rows: SPREAD = false: row r lies r ld bytes (below 2^32 in all) behind a base
// that is the same for the workgroup; true: anywhere.
template <class C, int R, int LOADS, bool SPREAD = false>
struct OutRowsSource {
  const char* base;
  uint32_t off[LOADS];                // this lane's chunk of step 0: base + off
  const char* p[SPREAD ? LOADS : 1];  // or, for rows anywhere, its address
  static constexpr int CH = C::KB / 16;
  int K;
  size_t part;                        // bytes between the parts
  u32x4 held[C::ALIGNED ? 1 : LOADS];  // !ALIGNED: the chunks of the step loaded last
  // row_of(r): offset (SPREAD: address) of the row of output row r (0 <= r < R;
  // any valid row for those past the end, whose outputs are not stored).
  template <typename F>
  __device__ __forceinline__ void init(const char* base_, F row_of, int K_, size_t part_, int lane,
                                       int wave) {
    base = base_;
    K = K_;
    part = part_;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int e = (wave * LOADS + j) * 64 + lane;
      const int row = e / CH, ch = out_swz<C::KB>(row, e % CH);
      if constexpr (SPREAD) p[j] = row_of(row) + ch * 16;
      else off[j] = row_of(row) + ch * 16;
    }
  }
  // Number of steps that lie wholly before K.
  __device__ __forceinline__ int whole_steps() const { return K / C::BK; }
  // WHOLE: the step lies before K.
  template <bool WHOLE>
  __device__ __forceinline__ void load(char* region, int step, int lane, int wave) {
#pragma unroll
    for (int q = 0; q < C::PARTS; ++q) {
      const char* b = base + (q * part + (size_t)step * C::KB);
#pragma unroll
      for (int j = 0; j < LOADS; ++j) {
        const char* g;
        if constexpr (SPREAD) g = p[j] + (q * part + (size_t)step * C::KB);
        else g = b + off[j];
        char* dst = region + q * (R * C::KB) + (wave * LOADS + j) * 1024;
        const int e = (wave * LOADS + j) * 64 + lane;
        const int left = K - step * C::BK - out_swz<C::KB>(e / CH, e % CH) * C::EPC;
        if constexpr (!C::ALIGNED) {
          if (K < C::EPC) {
            held[j] = short_chunk<C::ES>(g, left);
          } else {
            if (!WHOLE && left < C::EPC)
              g = left > 0 ? g - (C::EPC - left) * C::ES : reinterpret_cast<const char*>(&kZeros);
            __builtin_memcpy(&held[j], g, 16);
          }
        } else if constexpr (WHOLE) {
          dma16(g, dst);
        } else {
          dma16(left > 0 ? (const void*)g : (const void*)&kZeros, dst);
        }
      }
    }
  }
  // !ALIGNED: the step's chunks to their places.
  template <bool WHOLE>
  __device__ __forceinline__ void put(char* region, int step, int lane, int wave) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int e = (wave * LOADS + j) * 64 + lane;
      if constexpr (!WHOLE)
        end_chunk<C::ES>(held[j], K - step * C::BK - out_swz<C::KB>(e / CH, e % CH) * C::EPC, K);
      *reinterpret_cast<u32x4*>(region + (wave * LOADS + j) * 1024 + lane * 16) = held[j];
    }
  }
};

// ---- kRedRows: LDS rows of R elements -------------------------------------------
// The four rows of a transposing read land on different 64-byte bank ranges
// (rows of whole 256 bytes all start on one bank, others alternate between two);
// of fp32, the rows of the two lane halves on different 128-byte ranges.
template <int ES, int R>
__device__ __forceinline__ int red_swz(int r, int ch) {
  if constexpr (ES == 4) return ch ^ (((r >> 2) & 1) << 3);
  else if constexpr (R % 128 == 0) return ch ^ ((r & 3) << 2);
  else return ch ^ (((r >> 1) & 1) << 2);
}

// The memory row of reduction index k: k itself, or a row number that the
// workgroup put in LDS.
struct SameRow {
  static constexpr bool SAME = true;
};
struct ListedRow {
  static constexpr bool SAME = false;
  const int32_t* list;
};

template <class C, int R, int LOADS, class MAP>
struct RedRowsSource {
  const char* base;
  size_t ld, part;      // bytes per row, between the parts
  uint32_t off[LOADS];  // byte offset of this lane's chunk's column (SameRow: in its row)
  int c0, cols, K;
  MAP map;
  static constexpr bool SAME = MAP::SAME;
  // ListedRow: the rows of the step that is loaded next (steps are loaded in
  // order), read a step ahead so that no load waits for LDS.
  int32_t row[SAME ? 1 : LOADS];
  u32x4 held[C::ALIGNED ? 1 : LOADS];  // (as above)
  static constexpr int CH = R / C::EPC;  // chunks per row
  // Columns c0 .. of `cols`; ALIGNED needs cols to be whole chunks (chunks past
  // the last read the row's last 16 bytes: their outputs are not stored). A step's
  // rows (SameRow) span less than 2^32 bytes.
  __device__ __forceinline__ void init(const char* base_, size_t ld_, int c0_, int cols_, int K_,
                                       size_t part_, MAP map_, int lane, int wave) {
    static_assert(R % 64 == 0, "swizzle range");
    base = base_;
    ld = ld_;
    part = part_;
    c0 = c0_;
    cols = cols_;
    K = K_;
    map = map_;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int e = (wave * LOADS + j) * 64 + lane, r = e / CH;
      const int c = c0 + red_swz<C::ES, R>(r, e % CH) * C::EPC;
      off[j] = (uint32_t)((C::ALIGNED || cols >= C::EPC ? min(c, cols - C::EPC) : c) * C::ES);
      if constexpr (SAME) off[j] += (uint32_t)(r * ld);
      else row[j] = map.list[min(r, K - 1)];
    }
  }
  __device__ __forceinline__ int whole_steps() const { return K / C::BK; }
  template <bool WHOLE>
  __device__ __forceinline__ void load(char* region, int step, int lane, int wave) {
#pragma unroll
    for (int q = 0; q < C::PARTS; ++q) {
      const char* b = base + q * part;
      if constexpr (SAME) b += (size_t)step * C::BK * ld;
#pragma unroll
      for (int j = 0; j < LOADS; ++j) {
        const int e = (wave * LOADS + j) * 64 + lane, r = e / CH;
        const int k = step * C::BK + r;
        const bool in = WHOLE || k < K;
        const char* g = b + off[j];
        if constexpr (!SAME) {
          g += (size_t)row[j] * ld;
          row[j] = map.list[min(k + C::BK, K - 1)];
        }
        char* dst = region + q * (R * C::KB) + (wave * LOADS + j) * 1024;
        if constexpr (!C::ALIGNED) {
          if (cols < C::EPC) {
            held[j] = short_chunk<C::ES>(
                g, in ? cols - c0 - red_swz<C::ES, R>(r, e % CH) * C::EPC : 0);
          } else {
            __builtin_memcpy(&held[j], in ? g : reinterpret_cast<const char*>(&kZeros), 16);
          }
        } else if constexpr (WHOLE) {
          dma16(g, dst);
        } else {
          dma16(in ? (const void*)g : (const void*)&kZeros, dst);
        }
      }
    }
  }
  template <bool WHOLE>
  __device__ __forceinline__ void put(char* region, int step, int lane, int wave) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int e = (wave * LOADS + j) * 64 + lane, r = e / CH;
      if (c0 + R > cols)  // the last columns' tile
        end_chunk<C::ES>(held[j], cols - c0 - red_swz<C::ES, R>(r, e % CH) * C::EPC, cols);
      *reinterpret_cast<u32x4*>(region + (wave * LOADS + j) * 1024 + lane * 16) = held[j];
    }
  }
};

// ---- fragments --------------------------------------------------------------------
// 16-bit types: lane l holds output row l % 32 of its block, reduction 8 (l /
// 32) + 0..7 of a slice of 16 (one MFMA). fp32: reduction 4 (l / 32) + 0..3 of
// a slice of 8 (four MFMAs of two each).
template <class C, int MODE, int R, int F>
struct Reader {
  uint32_t off[MODE == kOutRows ? C::SLICES : F];
  __device__ __forceinline__ void init(int row0, int lane) {
    if constexpr (MODE == kOutRows) {
      const int row = row0 + (lane & 31);
#pragma unroll
      for (int kk = 0; kk < C::SLICES; ++kk)
        off[kk] = row * C::KB + 16 * out_swz<C::KB>(row, 2 * kk + (lane >> 5));
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
    const char* s = region + q * (R * C::KB);
#pragma unroll
    for (int i = 0; i < F; ++i) {
      if constexpr (MODE == kOutRows) {
        f[i] = *reinterpret_cast<const u32x4*>(s + off[KK] + i * 32 * C::KB);
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

// The fragments of slice KK. Of pairs, the hi parts first, then the lo parts of
// b and of a: in the order in which the products below leave registers free.
template <class C, int KK, class RA, class RB>
__device__ __forceinline__ void read_slice(u32x4 (&fa)[C::PARTS][C::FM],
                                           u32x4 (&fb)[C::PARTS][C::FN], const char* stg,
                                           const RA& ra, const RB& rb) {
  ra.template read<KK>(fa[0], stg, 0);
  rb.template read<KK>(fb[0], stg + C::A_BYTES, 0);
  if constexpr (C::PARTS == 2) {
    rb.template read<KK>(fb[1], stg + C::A_BYTES, 1);
    ra.template read<KK>(fa[1], stg, 1);
  }
}

template <class C>
__device__ __forceinline__ void mma_blocks(Acc<C>& acc, const u32x4 (&a)[C::FM],
                                           const u32x4 (&b)[C::FN]) {
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) mma<C::E>(acc[i][j], a[i], b[j]);
}
// Of pairs, the lo products first: b's lo part is done with after a third of
// them, a's after two thirds, and the next slice's are read into their registers.
template <class C>
__device__ __forceinline__ void mma_slice(Acc<C>& acc, const u32x4 (&fa)[C::PARTS][C::FM],
                                          const u32x4 (&fb)[C::PARTS][C::FN]) {
  if constexpr (C::PARTS == 2) {
    mma_blocks<C>(acc, fa[0], fb[1]);
    mma_blocks<C>(acc, fa[1], fb[0]);
  }
  mma_blocks<C>(acc, fa[0], fb[0]);
}

template <class C, bool WHOLE, class SA, class SB>
__device__ __forceinline__ void issue(char* stg, SA& a, SB& b, int step, int lane,
                                      int wave) {
  a.template load<WHOLE>(stg, step, lane, wave);
  b.template load<WHOLE>(stg + C::A_BYTES, step, lane, wave);
}
// What issue() loaded to its place, where no DMA puts it there.
template <class C, bool WHOLE, class SA, class SB>
__device__ __forceinline__ void settle(char* stg, SA& a, SB& b, int step, int lane, int wave) {
  if constexpr (!C::ALIGNED) {
    static_assert(C::PARTS == 1, "chunks held of one part");
    a.template put<WHOLE>(stg, step, lane, wave);
    b.template put<WHOLE>(stg + C::A_BYTES, step, lane, wave);
  }
}

// How many LDS reads a slice of one part of an operand takes.
template <class C, int MODE, int F>
constexpr int reads_of() {
  return F * (MODE == kOutRows ? 1 : C::ES == 2 ? 2 : 4);
}

// Order of one run of MFMAs: NDS LDS reads and NVM DMA issues spread between
// them from the start.
template <class C, int NDS, int NVM>
__device__ __forceinline__ void interleave_blocks() {
  constexpr int NMF = C::FM * C::FN * (C::E == kF32 ? 4 : 1);
  constexpr int PER = (NDS + NMF - 1) / NMF, PERV = (NVM + NMF - 1) / NMF;
#pragma unroll
  for (int i = 0; i < NMF; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                           // MFMA
    if (i * PER < NDS) __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);      // LDS read
    if (i * PERV < NVM) __builtin_amdgcn_sched_group_barrier(0x020, PERV, 0);    // DMA
    __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);                           // VALU
  }
}
// Order of one slice's section: its MFMAs under which the next slice is read
// and (DMA) a step's loads are issued.
template <class C, bool DMA>
__device__ __forceinline__ void interleave() {
  constexpr int A = reads_of<C, C::AMODE, C::FM>(), B = reads_of<C, C::BMODE, C::FN>();
  constexpr int NVM = DMA && C::ALIGNED ? C::V : 0;
  interleave_blocks<C, A + B, NVM>();
  if constexpr (C::PARTS == 2) {
    interleave_blocks<C, B, 0>();
    interleave_blocks<C, A, 0>();
  }
  __builtin_amdgcn_sched_barrier(0);
}

template <class C>
struct Frags {
  u32x4 a[C::PARTS][C::FM], b[C::PARTS][C::FN];
};

// One K-step out of ring stage S (the stages are separate arrays and S is a
// constant, so the compiler can tell the stage read from the stages being
// filled and waits only for these reads). On entry f holds slice 0 of step kt,
// on return slice 0 of step kt + 1: each slice's reads run under the MFMAs of
// the slice before.
template <class C, int S, bool WHOLE, class SA, class SB, class RA, class RB>
__device__ __forceinline__ void step(Acc<C>& acc, Frags<C>& f, char* const (&ring)[C::NSTAGE],
                                     SA& a, SB& b, const RA& ra, const RB& rb, int kt,
                                     int lane, int wave) {
  // Every wave is done with step kt - 1 (the barrier in it), whose stage this
  // DMA overwrites.
  issue<C, WHOLE>(ring[(S + C::AHEAD) % C::NSTAGE], a, b, kt + C::AHEAD, lane, wave);
  Frags<C> g;
  read_slice<C, 1>(g.a, g.b, ring[S], ra, rb);
  mma_slice<C>(acc, f.a, f.b);
  interleave<C, true>();
  if constexpr (C::SLICES == 4) {
    read_slice<C, 2>(f.a, f.b, ring[S], ra, rb);
    mma_slice<C>(acc, g.a, g.b);
    interleave<C, false>();
    read_slice<C, 3>(g.a, g.b, ring[S], ra, rb);
    mma_slice<C>(acc, f.a, f.b);
    interleave<C, false>();
  }
  settle<C, WHOLE>(ring[(S + C::AHEAD) % C::NSTAGE], a, b, kt + C::AHEAD, lane, wave);
  __asm__ volatile("" ::: "memory");
  // this wave's part of step kt + 1 has landed once only the later steps' are out
  wait_vm<(C::AHEAD - 1) * C::V>();
  lds_barrier();
  read_slice<C, 0>(f.a, f.b, ring[(S + 1) % C::NSTAGE], ra, rb);
  mma_slice<C>(acc, g.a, g.b);
  interleave<C, false>();
}

template <class C, bool WHOLE, class SA, class SB, class RA, class RB>
__device__ __forceinline__ void round(Acc<C>& acc, Frags<C>& f, char* const (&ring)[C::NSTAGE],
                                      SA& a, SB& b, const RA& ra, const RB& rb, int kt,
                                      int lane, int wave) {
  step<C, 0, WHOLE>(acc, f, ring, a, b, ra, rb, kt, lane, wave);
  step<C, 1, WHOLE>(acc, f, ring, a, b, ra, rb, kt + 1, lane, wave);
  if constexpr (C::NSTAGE > 2) step<C, 2, WHOLE>(acc, f, ring, a, b, ra, rb, kt + 2, lane, wave);
  if constexpr (C::NSTAGE > 3) step<C, 3, WHOLE>(acc, f, ring, a, b, ra, rb, kt + 3, lane, wave);
}

// acc += the product over steps [0, nsteps), taken in whole rounds of the ring
// (the steps past nsteps add zeros; leaving a round early would cost a copy of
// the accumulators per exit). All of the workgroup's waves call it with the
// same nsteps; on return no DMA is in flight, but other waves may still be
// reading the ring.
template <class C, class SA, class SB, class RA, class RB>
__device__ __forceinline__ void run(Acc<C>& acc, char* const (&ring)[C::NSTAGE], SA& a, SB& b,
                                    const RA& ra, const RB& rb, int nsteps, int lane,
                                    int wave) {
#pragma unroll
  for (int s = 0; s < C::AHEAD; ++s) {
    issue<C, false>(ring[s], a, b, s, lane, wave);
    settle<C, false>(ring[s], a, b, s, lane, wave);
    __asm__ volatile("" ::: "memory");
  }
  wait_vm<(C::AHEAD - 1) * C::V>();
  lds_barrier();
  Frags<C> f;
  read_slice<C, 0>(f.a, f.b, ring[0], ra, rb);
  int kt = 0;
  // rounds whose loads all lie before the reduction's end need no checks
  for (const int whole = a.whole_steps() - C::AHEAD; kt + C::NSTAGE <= whole; kt += C::NSTAGE)
    round<C, true>(acc, f, ring, a, b, ra, rb, kt, lane, wave);
  for (; kt < nsteps; kt += C::NSTAGE)
    round<C, false>(acc, f, ring, a, b, ra, rb, kt, lane, wave);
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
