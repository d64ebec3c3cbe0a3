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
// second time, out of L2, because dy needs sums over the row). 32768 tokens of
// 4 rows of 4096 bf16, 1.88 GB: 349 us (5.4 TB/s); the gradient of 16384 tokens of 2
// rows of 2048, 0.54 GB: 118 + 5 us (4.5 TB/s); one token of 8 rows 5.5 us. A row
// belongs to TPR threads (sixteen, a wave, or a whole workgroup), a thread to EPC * NV
// of its values, held in registers between the sums - but in the gradient of rows above
// 4096, whose sixteen values a thread of each array leave 42 to 63 registers in scratch
// memory in fp32 (8192 tokens of 2 rows of 8192: 491 us, 4.4 TB/s) and two in bf16 with
// several picks (234 us, 4.6 TB/s). With eps = 0 a row of zeros, a token without picks
// too, has 0 / 0 for its norm: NaN; squares have to be within fp32.
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
  static constexpr bool AHEAD = VALS <= 8;       // the gradient loads a token ahead
  static constexpr int THREADS = TPR > kThreads ? TPR : kThreads;
  static constexpr int ROWS = THREADS / TPR;     // per workgroup
};

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16_bits(v); }

// The chunk of a row at column c: values c .. c + EPC - 1 of d, zeros past it.
// Rows that are not aligned take 16-byte accesses all the same (the memory
// system splits them); a row's last chunk takes the row's last 16 bytes and moves
// them down. Rows shorter than that are read value by value.
template <class C>
__device__ __forceinline__ uint4 load_chunk(const typename C::T* p, int c, int d) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (C::ALIGNED) {
    if (c < d) v = *reinterpret_cast<const uint4*>(p + c);
  } else if (d >= C::EPC) {
    const int at = min(c, d - C::EPC), past = c - at;  // values to drop
    __builtin_memcpy(&v, p + at, 16);
    if (past & (C::EPC / 2)) v = make_uint4(v.z, v.w, 0u, 0u);
    if (past & (C::EPC / 4)) v = make_uint4(v.y, v.z, v.w, 0u);
    if (C::EPC == 8 && (past & 1))
      v = make_uint4(v.x >> 16 | v.y << 16, v.y >> 16 | v.z << 16, v.z >> 16 | v.w << 16, v.w >> 16);
    if (past >= C::EPC) v = make_uint4(0u, 0u, 0u, 0u);
  } else {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < C::EPC - 1; ++e)
      if (c + e < d) {
        if constexpr (C::EPC == 8)
          w[e / 2] |= (uint32_t)p[c + e] << (16 * (e & 1));
        else
          w[e] = __float_as_uint(p[c + e]);
      }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}
template <class C>
__device__ __forceinline__ void widen(uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < C::EPC; ++e)
    f[e] = C::EPC == 4 ? __uint_as_float(w[e]) : (e & 1) == 0 ? bf16_lo(w[e / 2]) : bf16_hi(w[e / 2]);
}

// This thread's values of a row of d: chunks lane, lane + TPR, ... (zeros past d).
template <class C>
__device__ __forceinline__ void load_row(const typename C::T* row, int d, int lane,
                                         float (&v)[C::VALS]) {
#pragma unroll
  for (int i = 0; i < C::NV; ++i)
    widen<C>(load_chunk<C>(row, (i * C::TPR + lane) * C::EPC, d), v + i * C::EPC);
}
template <class C>
__device__ __forceinline__ void store_row(typename C::T* row, int d, int lane,
                                          const float (&v)[C::VALS], float scale) {
#pragma unroll
  for (int i = 0; i < C::NV; ++i) {
    const int c = (i * C::TPR + lane) * C::EPC;
    if constexpr (C::ALIGNED) {
      if (c < d) store16(v + i * C::EPC, row + c, scale);
    } else if (c + C::EPC <= d) {
      typename C::T w[C::EPC];
#pragma unroll
      for (int e = 0; e < C::EPC; ++e) put(w + e, v[i * C::EPC + e] * scale);
      __builtin_memcpy(row + c, w, 16);
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

// The sum over a wave's lanes, in a fixed order: DPP shifts by 1, 2, 4 and 8
// within rows of 16 lanes, then across the rows; the last lane has it all.
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(
                 __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, ROWS == 0xF));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = add_dpp<0x111, 0xF>(v);
  v = add_dpp<0x112, 0xF>(v);
  v = add_dpp<0x114, 0xF>(v);
  v = add_dpp<0x118, 0xF>(v);
  v = add_dpp<0x142, 0xA>(v);  // lane 15 (47) of the row before, into rows 1 and 3
  v = add_dpp<0x143, 0xC>(v);  // lane 31, into rows 2 and 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), kWave - 1));
}

// The sum over each sixteen lanes, the same bits in all of them: DPP swaps of
// neighbours, of pairs, of fours and of eights.
__device__ __forceinline__ float narrow_sum(float v) {
  v = add_dpp<0xB1, 0xF>(v);   // lanes 1 0 3 2
  v = add_dpp<0x4E, 0xF>(v);   // lanes 2 3 0 1
  v = add_dpp<0x141, 0xF>(v);  // eight lanes mirrored
  return add_dpp<0x140, 0xF>(v);  // sixteen lanes mirrored
}

// Sums of N values over the TPR threads of a row, the same in all of them.
// lds: N floats per wave.
template <class C, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* lds) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = C::TPR < kWave ? narrow_sum(v[i]) : wave_sum(v[i]);
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

// A thread's values of a row as they are in memory: chunk i * TPR + lane.
template <class C>
struct RawRow {
  uint4 v[C::NV];
  __device__ __forceinline__ void load(const void* base, size_t row, int d, int lane) {
    const typename C::T* p = static_cast<const typename C::T*>(base) + row * d;
#pragma unroll
    for (int i = 0; i < C::NV; ++i) v[i] = load_chunk<C>(p, (i * C::TPR + lane) * C::EPC, d);
  }
  __device__ __forceinline__ void get(float (&f)[C::VALS]) const {
#pragma unroll
    for (int i = 0; i < C::NV; ++i) widen<C>(v[i], f + i * C::EPC);
  }
};

// A token's picks (k <= 64): the row of u, -1 for one outside it, and the gate, all
// loaded at once. Pick j is in lane j of each wave; of rows of sixteen lanes, in
// lane j % 16, register j / 16.
template <class C>
struct Picks {
  static constexpr int LANES = C::TPR < kWave ? C::TPR : kWave, REGS = kWave / LANES;
  int32_t row[REGS], g[REGS];  // (the gate's bits)
  __device__ __forceinline__ void load(const NormCall& p, long long t) {
#pragma unroll
    for (int i = 0; i < REGS; ++i) {
      const int j = i * LANES + threadIdx.x % LANES;
      row[i] = -1;
      g[i] = __float_as_int(1.f);
      if (!p.u || j >= p.k || t >= p.T) continue;
      const int32_t at = (int32_t)(t * p.k + j);
      row[i] = p.inv ? p.inv[at] : at;
      if (row[i] >= p.M) row[i] = -1;
      if (p.gates) g[i] = __float_as_int(p.gates[at]);
    }
  }
  __device__ __forceinline__ int pick(const int (&v)[REGS], int j) const {
    if constexpr (REGS == 1) {
      return __builtin_amdgcn_readlane(v[0], j);
    } else {
      static_assert(REGS == 4, "rows of sixteen lanes");
      const int x = j < 16 ? v[0] : j < 32 ? v[1] : j < 48 ? v[2] : v[3];
      return __shfl(x, j % LANES, LANES);
    }
  }
  __device__ __forceinline__ int32_t row_of(int j) const { return pick(row, j); }
  __device__ __forceinline__ float gate_of(int j) const { return __int_as_float(pick(g, j)); }
};

// y += the picks j0 .. k - 1, ascending, eight rows of u in flight where a thread has
// one chunk of a row, else four.
template <class C>
__device__ __forceinline__ void add_picks(const NormCall& p, const Picks<C>& picks, int j0, int lane,
                                          float (&y)[C::VALS]) {
  constexpr int U = C::NV == 1 ? 8 : 4;
  for (int j = j0; j < p.k; j += U) {
    RawRow<C> u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (j + i >= p.k) continue;
      const int32_t row = picks.row_of(j + i);
      if (row >= 0) u[i].load(p.u, (size_t)row, p.d, lane);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (j + i >= p.k || picks.row_of(j + i) < 0) continue;  // the same in the whole row
      const float g = picks.gate_of(j + i);
      float v[C::VALS];
      u[i].get(v);
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) y[e] = fmaf(g, v[e], y[e]);
    }
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
  const long long t64 = (long long)grid_block() * C::ROWS + threadIdx.x / C::TPR;
  // all TPR threads of a row: its sums and picks use no lane outside of them (sixteen
  // lanes within a wave, whole waves, or the workgroup whose barriers they share)
  if (t64 >= p.T) return;
  const int t = (int)t64;
  const size_t at = (size_t)t * p.d;
  Picks<C> picks;
  picks.load(p, t);
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
#pragma unroll
    for (int e = 0; e < C::VALS; ++e) y[e] = 0.f;
    add_picks<C>(p, picks, 0, lane, y);
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

// What the gradient reads of a token, loaded a token ahead: its rows, and the
// first K picks' rows of u (the picks two tokens ahead).
template <class C, int K>
struct TokenLoads {
  RawRow<C> x, dn, dr, u[K];
  Picks<C> picks;
  __device__ __forceinline__ void load(const NormCall& p, long long t, int lane) {
    if (t >= p.T) return;
    if (p.w_pre) {
      x.load(p.x, (size_t)t, p.d, lane);
      dn.load(p.dn, (size_t)t, p.d, lane);
    }
    if (p.dr_out) dr.load(p.dr_out, (size_t)t, p.d, lane);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int32_t row = picks.row_of(j);
      if (row >= 0) u[j].load(p.u, (size_t)row, p.d, lane);
    }
  }
};

// fp32 weights of this thread's columns: kept, or read again for each token
// where a thread has many.
template <class C>
struct Weights {
  static constexpr bool KEPT = C::VALS <= 8;
  const float* p;
  float v[KEPT ? C::VALS : 1];
  __device__ __forceinline__ void init(const float* w, int d, int lane) {
    p = w;
    if constexpr (KEPT)
      if (w) load_weight<C>(w, d, lane, v);
  }
  __device__ __forceinline__ void get(int d, int lane, float (&w)[C::VALS]) const {
    if constexpr (KEPT) {
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) w[e] = v[e];
    } else {
      load_weight<C>(p, d, lane, w);
    }
  }
};

// One workgroup takes ROWS tokens at a time, `gridDim.x` apart, and keeps the
// weights' gradients of its columns in registers; they end as partial sums
// part[side][workgroup][d], added in order by a second launch. A token is a
// chain of loads, sums over its row and barriers, so the next token's loads are
// issued before it. Its first K picks stay in registers for their dgates;
// further ones are read again.
template <class C, int K>
__global__ __launch_bounds__(C::THREADS) void norm_bwd_kernel(NormCall p, float* part) {
  __shared__ float lds[(K > 3 ? K : 3) * (C::THREADS / kWave)];
  __shared__ float fold[C::ROWS > 1 ? C::ROWS * C::TPR * C::VALS : 1];
  using T = typename C::T;
  const int lane = threadIdx.x % C::TPR, sub = threadIdx.x / C::TPR;
  const long long stride = (long long)gridDim.x * C::ROWS;
  float dpre[C::VALS], dpost[C::VALS];
#pragma unroll
  for (int e = 0; e < C::VALS; ++e) dpre[e] = dpost[e] = 0.f;
  const long long first = (long long)blockIdx.x * C::ROWS + sub;
  TokenLoads<C, K> next;
  next.picks.load(p, first);
  if constexpr (C::AHEAD) next.load(p, first, lane);
  Picks<C> after;
  after.load(p, first + stride);
  Weights<C> w_pre, w_post;
  w_pre.init(p.w_pre, p.d, lane);
  w_post.init(p.w_post, p.d, lane);
  // (the threads of a row leave it together, as in norm_kernel)
  for (long long t64 = first; t64 < p.T; t64 += stride) {
    const size_t at = (size_t)t64 * p.d;
    if constexpr (!C::AHEAD) next.load(p, t64, lane);
    const TokenLoads<C, K> now = next;
    next.picks = after;
    after.load(p, t64 + 2 * stride);
    if constexpr (C::AHEAD) next.load(p, t64 + stride, lane);
    float dr[C::VALS], y[C::VALS];
#pragma unroll
    for (int e = 0; e < C::VALS; ++e) y[e] = 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (now.picks.row_of(j) < 0) continue;
      const float g = now.picks.gate_of(j);
      float v[C::VALS];
      now.u[j].get(v);
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) y[e] = fmaf(g, v[e], y[e]);
    }
    if (p.u) add_picks<C>(p, now.picks, K, lane, y);
    if (p.dr_out) {
      now.dr.get(dr);
    } else {
#pragma unroll
      for (int e = 0; e < C::VALS; ++e) dr[e] = 0.f;
    }
    float s[3] = {0.f, 0.f, 0.f};  // r'^2, w_pre dn r', y^2
#pragma unroll
    for (int e = 0; e < C::VALS; ++e) s[2] = fmaf(y[e], y[e], s[2]);
    if (p.w_pre) {
      float x[C::VALS], dn[C::VALS], w[C::VALS];
      now.x.get(x);
      now.dn.get(dn);
      w_pre.get(p.d, lane, w);
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
      w_post.get(p.d, lane, w);
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
    float dg[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      dg[j] = 0.f;
      const int32_t row = now.picks.row_of(j);
      if (row < 0) continue;
      if (p.du)
        store_row<C>(static_cast<T*>(p.du) + (size_t)row * p.d, p.d, lane, dr, now.picks.gate_of(j));
      if (p.dgates) {
        float v[C::VALS];
        now.u[j].get(v);
#pragma unroll
        for (int e = 0; e < C::VALS; ++e) dg[j] = fmaf(dr[e], v[e], dg[j]);
      }
    }
    if (p.dgates) {
      row_sum<C, K>(dg, lds);
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (lane == 0 && j < p.k) p.dgates[t64 * p.k + j] = dg[j];
    }
    for (int j0 = K; j0 < p.k; j0 += 2) {
      float d2[2] = {0.f, 0.f};
      RawRow<C> u[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t row = j0 + i < p.k ? now.picks.row_of(j0 + i) : -1;
        if (row >= 0 && p.dgates) u[i].load(p.u, (size_t)row, p.d, lane);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t row = j0 + i < p.k ? now.picks.row_of(j0 + i) : -1;
        if (row < 0) continue;
        if (p.du)
          store_row<C>(static_cast<T*>(p.du) + (size_t)row * p.d, p.d, lane, dr,
                       now.picks.gate_of(j0 + i));
        if (p.dgates) {
          float v[C::VALS];
          u[i].get(v);
#pragma unroll
          for (int e = 0; e < C::VALS; ++e) d2[i] = fmaf(dr[e], v[e], d2[i]);
        }
      }
      if (p.dgates) {
        row_sum<C, 2>(d2, lds);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (lane == 0 && j0 + i < p.k) p.dgates[t64 * p.k + j0 + i] = d2[i];
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
  // for fill_rows: a row's pick (here, where no token's values are live: in the loop
  // it took registers, and of some widths a wave per SIMD)
  if (p.marks && p.inv) {
    const long long picks = (long long)p.T * p.k, all = (long long)gridDim.x * C::THREADS;
    for (long long i = (long long)blockIdx.x * C::THREADS + threadIdx.x; i < picks; i += all) {
      const int32_t row = p.inv[i];
      if (row >= 0 && row < p.M) p.marks[row] = (int32_t)i;
    }
  }
}

// The rows of du that no pick names become 0, 64 rows a wave at a time. A row that a
// pick names holds a pick that names it in marks; of the others, where marks holds
// whatever the workspace did, no pick can name them.
constexpr int kSumWaves = 16;
struct FillArgs {
  const int32_t *inv, *marks;
  long long rows, picks;
  size_t row_bytes;
  char* du;
};
__device__ __forceinline__ void fill_rows(const FillArgs& f, int lane, int wave) {
  const long long step = (long long)gridDim.x * kSumWaves * kWave;
  for (long long r0 = ((long long)blockIdx.x * kSumWaves + wave) * kWave; r0 < f.rows; r0 += step) {
    const long long r = r0 + lane;
    bool named = r >= f.rows || (!f.inv && r < f.picks);
    if (!named && f.inv) {
      const int32_t m = f.marks[r];
      named = m >= 0 && m < f.picks && f.inv[m] == r;
    }
    for (uint64_t left = __ballot(!named); left; left &= left - 1) {
      char* row = f.du + (size_t)(r0 + __ffsll((unsigned long long)left) - 1) * f.row_bytes;
      if (f.row_bytes % 16 == 0) {
        for (size_t i = 16 * lane; i < f.row_bytes; i += 16 * kWave)
          *reinterpret_cast<uint4*>(row + i) = make_uint4(0u, 0u, 0u, 0u);
      } else {
        for (size_t i = 2 * lane; i < f.row_bytes; i += 2 * kWave)
          *reinterpret_cast<uint16_t*>(row + i) = 0;
      }
    }
  }
}

// dw[c] = the partial sums of column c, in order and in 64 bits: 64 columns a
// workgroup, sixteen waves taking a sixteenth of the parts each. blockIdx.y = 2:
// fill_rows.
__global__ __launch_bounds__(64 * kSumWaves) void norm_weights_kernel(const float* part, int parts,
                                                                      int d, float* dw_pre,
                                                                      float* dw_post, FillArgs fill) {
  __shared__ double lds[kSumWaves][64];
  if (blockIdx.y == 2) return fill_rows(fill, threadIdx.x % 64, threadIdx.x / 64);
  float* dst = blockIdx.y ? dw_post : dw_pre;
  if (!dst || blockIdx.x * 64 >= (unsigned)d) return;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, col = blockIdx.x * 64 + lane;
  const int n = (parts + kSumWaves - 1) / kSumWaves, lo = min(parts, wave * n),
            hi = min(parts, lo + n);
  double s = 0.0;
  if (col < d) {
    const float* src = part + (size_t)blockIdx.y * parts * d + col;
#pragma unroll 8
    for (int i = lo; i < hi; ++i) s += (double)src[(size_t)i * d];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < d) {
    for (int w = 1; w < kSumWaves; ++w) s += lds[w][lane];
    dst[col] = (float)s;
  }
}

// Workgroups of the gradient: enough rows each that their partial sums stay few.
constexpr int kBwdGroups = 768;
constexpr unsigned kFillGroups = 256;  // of fill_rows, at most

template <class C>
hipError_t launch_norm_cfg(const NormCall& c, hipStream_t s) {
  const size_t groups = ((size_t)c.T + C::ROWS - 1) / C::ROWS;
  return launch_kernel(norm_kernel<C>, grid_rows(groups), dim3(C::THREADS), 0, s, KernelTiming{},
                       c);
}
template <class C>
hipError_t launch_norm_bwd_cfg(const NormCall& c, float* part, hipStream_t s) {
  const size_t want = ((size_t)c.T + C::ROWS - 1) / C::ROWS;
  // T = 0: no sums, dw = 0. Two rounds at most: as many rows in each (1000 x 4096 fp32
  // 36.5 -> 32 us; more rounds gain nothing by it)
  const int groups = want > kBwdGroups && want <= 2 * kBwdGroups ? (int)((want + 1) / 2)
                     : want < kBwdGroups                         ? (int)want
                                                                 : kBwdGroups;
  const auto launch = [&](auto kernel) {
    return launch_kernel(kernel, dim3(groups), dim3(C::THREADS), 0, s, KernelTiming{}, c, part);
  };
  hipError_t e = hipSuccess;
  if (groups) e = !c.u || c.k == 1 ? launch(norm_bwd_kernel<C, 1>) : launch(norm_bwd_kernel<C, 2>);
  if (e != hipSuccess || (!c.dw_pre && !c.dw_post && !c.fill)) return e;
  FillArgs fill = {};
  unsigned wide = (c.d + 63) / 64;
  if (c.fill) {
    fill.inv = c.inv;
    fill.marks = c.marks;
    fill.rows = c.M;
    fill.picks = (long long)c.T * c.k;
    fill.row_bytes = (size_t)c.d * sizeof(typename C::T);
    fill.du = static_cast<char*>(c.du);
    const long long most = (c.M + kSumWaves * kWave - 1) / (kSumWaves * kWave);
    if (most > wide) wide = most < kFillGroups ? (unsigned)most : kFillGroups;
  }
  return launch_kernel(norm_weights_kernel, dim3(wide, c.fill ? 3 : 2), dim3(64 * kSumWaves), 0, s,
                       KernelTiming{}, (const float*)part, groups, c.d, c.dw_pre, c.dw_post, fill);
}

// f(config) for rows of d values (EPC per 16 bytes): sixteen lanes per row up to 16
// chunks (32768 rows of 128 bf16 18 -> 12.5 us, their gradient 39 -> 25), a wave up to
// 128, then a workgroup. The gradient holds about ten values per column and
// thread, so its long rows go to 512 threads (1024 would leave each 128
// registers; fp32 above 4096, four chunks a thread, does not fit 256 either).
template <bool BACK, typename T, bool ALIGNED, typename F>
hipError_t with_width(int d, F f) {
  constexpr int EPC = 16 / sizeof(T);
  if (d <= 16 * EPC) return f(NormCfg<T, 16, 1, ALIGNED>{});
  if (d <= 64 * EPC) return f(NormCfg<T, 64, 1, ALIGNED>{});
  if (d <= 128 * EPC) return f(NormCfg<T, 64, 2, ALIGNED>{});
  if (d <= 256 * EPC) return f(NormCfg<T, 256, 1, ALIGNED>{});
  if constexpr (BACK) {
    if (d <= 512 * EPC) return f(NormCfg<T, 512, 1, ALIGNED>{});
    if (d <= 1024 * EPC) return f(NormCfg<T, 512, 2, ALIGNED>{});
    if constexpr (EPC == 4) return f(NormCfg<T, 512, 4, ALIGNED>{});
  } else {
    if (d <= 512 * EPC) return f(NormCfg<T, 256, 2, ALIGNED>{});
    if (d <= 1024 * EPC) return f(NormCfg<T, 1024, 1, ALIGNED>{});
    if constexpr (EPC == 4) return f(NormCfg<T, 1024, 2, ALIGNED>{});
  }
  return hipErrorInvalidValue;
}
template <bool BACK, typename F>
hipError_t with_cfg(bmoe_dtype dt, int d, F f) {
  if (dt == BMOE_BF16)
    return d % 8 == 0 ? with_width<BACK, uint16_t, true>(d, f)
                      : with_width<BACK, uint16_t, false>(d, f);
  return d % 4 == 0 ? with_width<BACK, float, true>(d, f) : with_width<BACK, float, false>(d, f);
}

}  // namespace

size_t norm_part_bytes(int T, int d) {
  const size_t groups = T < kBwdGroups ? T : kBwdGroups;
  return 2 * groups * d * sizeof(float);
}

hipError_t launch_norm(bmoe_dtype dt, const NormCall& c, hipStream_t s) {
  return with_cfg<false>(dt, c.d, [&](auto cfg) { return launch_norm_cfg<decltype(cfg)>(c, s); });
}

hipError_t launch_norm_bwd(bmoe_dtype dt, const NormCall& c, float* part, hipStream_t s) {
  return with_cfg<true>(
      dt, c.d, [&](auto cfg) { return launch_norm_bwd_cfg<decltype(cfg)>(c, part, s); });
}

}  // namespace bmoe
