// Global norm of a list of gradients, and the gradients scaled to a largest
// norm:
//   norm = sqrt(sum over all tensors and entries of g^2)
//   out  = g * (max_norm / norm  if max_norm < norm < infinity, else 1)
// Squares are summed in 64 bits (no overflow, and a sum over 10^9 entries
// keeps its bits; the fp64 FMA runs at the fp32 rate here, far above what
// memory delivers) in an order that the sizes and alignments alone fix:
// thread, wave, workgroup, then the workgroups' partial sums in their order.
//
// Bound by HBM: the norm reads every byte once, the scaling reads and writes
// it once. The tensors are cut into chunks of 256 16-byte vectors, numbered
// through the list; a workgroup takes a run of consecutive chunks, so it looks
// its tensor up once, and streams 8 chunks (32 KB) per step. The scaling walks
// its run backwards and neither keeps what it loads nor what it stores; the
// norm's loads stay cached for it up to 256 MB (the last-level cache) of the
// whole list, above that they stream too (300 tensors of 2 MB in three tables:
// 340 us, 378 us when each table's own size decided). Measured, norm and
// scaling apart, plain against streaming accesses: 128 MB 84 -> 65 us (73 if
// the norm streams), 0.96 GB 569 -> 517 us (557 if it does not), against 533 us
// for its three passes at the rate of a large copy (5.4 TB/s). An out tensor
// that is not aligned as its gradient is (modulo 16) is written entry by entry:
// 128 MB of fp32 87 us, of bf16 133 us.
#include "common.h"
#include "kernels.h"

namespace bmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;  // vectors in flight per thread

__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += lds[w];
  return s;
}

// The norm from the partial sums, the same in every workgroup that asks.
__device__ __forceinline__ float norm_of(const double* part, int n, double* lds) {
  double acc = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) acc += part[i];
  return (float)sqrt(block_sum(acc, lds));
}

// ---- the entries of one tensor, by 16-byte vectors of its address ----------------
// Vector v of a tensor holds its entries W v - head ... W v - head + W - 1, W
// per 16 bytes, head the entries between the aligned address and the first.
struct Span {
  const char* src;  // rounded down to 16 bytes
  char* dst;        // src's offset from it, not rounded
  long long count;
  int head, bf16;
};
__device__ __forceinline__ Span span_of(const GradEntry& t) {
  Span s;
  const uintptr_t a = reinterpret_cast<uintptr_t>(t.src);
  s.src = reinterpret_cast<const char*>(a & ~(uintptr_t)15);
  s.dst = static_cast<char*>(t.dst) - (a & 15);
  s.count = (long long)t.count;
  s.bf16 = t.bf16;
  s.head = (int)(a & 15) / (t.bf16 ? 2 : 4);
  return s;
}

// Whether all entries of vectors [v0, v1) exist.
__device__ __forceinline__ bool whole(const Span& s, long long v0, long long v1) {
  const int w = s.bf16 ? 8 : 4;
  return v0 * w >= s.head && v1 * w - s.head <= s.count;
}

// f(value, byte offset) for the entries that vector v has.
template <typename F>
__device__ __forceinline__ void each_entry(const Span& s, long long v, F f) {
  const int w = s.bf16 ? 8 : 4;
  for (int i = 0; i < w; ++i) {
    const long long e = v * w + i - s.head;
    if (e < 0 || e >= s.count) continue;
    const long long at = v * 16 + i * (16 / w);
    f(s.bf16 ? bf16_lo(*reinterpret_cast<const uint16_t*>(s.src + at))
             : *reinterpret_cast<const float*>(s.src + at),
      at);
  }
}

__device__ __forceinline__ double add_sq(double acc, float g) {
  return fma((double)g, (double)g, acc);
}
template <bool BF16>
__device__ __forceinline__ void add_sq(double& a, double& b, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      a = add_sq(a, bf16_lo(w[i]));
      b = add_sq(b, bf16_hi(w[i]));
    } else {
      double& x = i & 1 ? b : a;
      x = add_sq(x, __uint_as_float(w[i]));
    }
  }
}

// Index of the entry that chunk c belongs to.
template <typename Table>
__device__ __forceinline__ int find(const Table& tab, uint32_t c) {
  int lo = 0, hi = tab.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (tab.t[mid].first <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// This workgroup's run of chunks.
template <typename Table>
__device__ __forceinline__ uint32_t run_start(const Table& tab, uint32_t b) {
  return (uint32_t)((uint64_t)tab.chunks * b / gridDim.x);
}

// Streaming accesses, for data that no cache will hold until its next use.
__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)));
}
__device__ __forceinline__ void st_once(uint4* p, uint4 v) {
  __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(p));
}

template <bool BF16, bool ONCE>
__device__ __forceinline__ void sq_chunks(const Span& s, long long c0, long long c1, double& a,
                                          double& b) {
  const uint4* p = reinterpret_cast<const uint4*>(s.src) + threadIdx.x;
  for (long long c = c0; c < c1;) {
    if (c + kAhead <= c1 && whole(s, c * 256, (c + kAhead) * 256)) {
      uint4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) v[u] = ONCE ? ld_once(p + (c + u) * 256) : p[(c + u) * 256];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) add_sq<BF16>(a, b, v[u]);
      c += kAhead;
    } else {
      const long long v = c * 256 + threadIdx.x;
      if (whole(s, v, v + 1)) add_sq<BF16>(a, b, p[c * 256]);
      else each_entry(s, v, [&](float g, long long) { a = add_sq(a, g); });
      ++c;
    }
  }
}

template <bool ONCE, typename Table>
__global__ __launch_bounds__(kThreads) void grad_sq_kernel(Table tab, double* part) {
  __shared__ double lds[kThreads / 64];
  double a = 0.0, b = 0.0;
  uint32_t c = run_start(tab, blockIdx.x);
  const uint32_t end = run_start(tab, blockIdx.x + 1);
  for (int n = find(tab, c); c < end; ++n) {
    const Span s = span_of(tab.t[n]);
    const uint32_t first = tab.t[n].first, next = n + 1 < tab.n ? tab.t[n + 1].first : tab.chunks;
    const uint32_t stop = next < end ? next : end;
    if (s.bf16) sq_chunks<true, ONCE>(s, c - first, stop - first, a, b);
    else sq_chunks<false, ONCE>(s, c - first, stop - first, a, b);
    c = stop;
  }
  const double sum = block_sum(a + b, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const double* part, int n,
                                                             float* norm) {
  __shared__ double lds[kThreads / 64];
  const float v = norm_of(part, n, lds);
  if (threadIdx.x == 0) *norm = v;
}

__device__ __forceinline__ uint4 scaled(uint4 v, float f, int bf16) {
  uint4 r;
  if (bf16) {
    r.x = pack_bf16x2(bf16_lo(v.x) * f, bf16_hi(v.x) * f);
    r.y = pack_bf16x2(bf16_lo(v.y) * f, bf16_hi(v.y) * f);
    r.z = pack_bf16x2(bf16_lo(v.z) * f, bf16_hi(v.z) * f);
    r.w = pack_bf16x2(bf16_lo(v.w) * f, bf16_hi(v.w) * f);
  } else {
    r.x = __float_as_uint(__uint_as_float(v.x) * f);
    r.y = __float_as_uint(__uint_as_float(v.y) * f);
    r.z = __float_as_uint(__uint_as_float(v.z) * f);
    r.w = __float_as_uint(__uint_as_float(v.w) * f);
  }
  return r;
}

// Chunks [c0, c1) of a tensor, the last first: what the norm read last is the
// likeliest to be in the caches still.
__device__ __forceinline__ void scale_chunks(const Span& s, long long c0, long long c1, float f) {
  const uint4* p = reinterpret_cast<const uint4*>(s.src) + threadIdx.x;
  uint4* o = reinterpret_cast<uint4*>(s.dst) + threadIdx.x;
  const bool same = (reinterpret_cast<uintptr_t>(s.dst) & 15) == 0;  // as aligned as src
  for (long long c = c1; c > c0;) {
    if (same && c - kAhead >= c0 && whole(s, (c - kAhead) * 256, c * 256)) {
      c -= kAhead;
      uint4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) v[u] = ld_once(p + (c + u) * 256);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) st_once(o + (c + u) * 256, scaled(v[u], f, s.bf16));
    } else {
      --c;
      const long long v = c * 256 + threadIdx.x;
      if (same && whole(s, v, v + 1)) {
        o[c * 256] = scaled(p[c * 256], f, s.bf16);
      } else {
        each_entry(s, v, [&](float g, long long at) {
          if (s.bf16) *reinterpret_cast<uint16_t*>(s.dst + at) = (uint16_t)f32_to_bf16_bits(g * f);
          else *reinterpret_cast<float*>(s.dst + at) = g * f;
        });
      }
    }
  }
}

// norm: read, or (part not NULL) taken from the n_part partial sums and
// written by the first workgroup.
template <typename Table>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(Table tab, const double* part,
                                                              int n_part, float* norm,
                                                              float max_norm, int in_place) {
  __shared__ double lds[kThreads / 64];
  float nv;
  if (part) {
    nv = norm_of(part, n_part, lds);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = nv;
  } else {
    nv = *norm;
  }
  const float coef = nv > max_norm && nv < INFINITY ? max_norm / nv : 1.f;
  if (in_place && coef == 1.f) return;
  uint32_t end = run_start(tab, blockIdx.x + 1);
  const uint32_t c = run_start(tab, blockIdx.x);
  for (int n = find(tab, end - 1); end > c; --n) {
    const uint32_t first = tab.t[n].first;
    const uint32_t start = first > c ? first : c;
    scale_chunks(span_of(tab.t[n]), start - first, end - first, coef);
    end = start;
  }
}

// A table of few tensors: kernel arguments of 3.6 KB cost each launch about
// 0.5 us of host time, which short lists wait for (one layer's four tensors:
// 17.5 us a call, 18.6 with the large table).
constexpr int kFew = 8;
struct FewTable {
  int n;
  uint32_t chunks;
  GradEntry t[kFew];
};
FewTable few(const GradTable& tab) {
  FewTable r{tab.n, tab.chunks, {}};
  for (int i = 0; i < tab.n; ++i) r.t[i] = tab.t[i];
  return r;
}

// A workgroup per chunk up to what is resident at once.
int grid_of(const GradTable& tab) {
  return tab.chunks < (uint32_t)kGradParts ? (int)tab.chunks : kGradParts;
}

}  // namespace

uint32_t grad_chunks(const void* src, size_t count, int bf16) {
  const size_t w = bf16 ? 8 : 4;
  const size_t head = (reinterpret_cast<uintptr_t>(src) & 15) / (16 / w);
  return (uint32_t)(((head + count + w - 1) / w + 255) / 256);
}

hipError_t launch_grad_sq(const GradTable& tab, size_t list_chunks, double* part, int* n_part,
                          hipStream_t s) {
  *n_part = grid_of(tab);
  const dim3 grid(*n_part), block(kThreads);
  if (list_chunks > (256u << 20) / 4096)
    return launch_kernel(grad_sq_kernel<true, GradTable>, grid, block, 0, s, KernelTiming{}, tab,
                         part);
  if (tab.n <= kFew)
    return launch_kernel(grad_sq_kernel<false, FewTable>, grid, block, 0, s, KernelTiming{},
                         few(tab), part);
  return launch_kernel(grad_sq_kernel<false, GradTable>, grid, block, 0, s, KernelTiming{}, tab,
                       part);
}

hipError_t launch_grad_norm(const double* part, int n_part, float* norm, hipStream_t s) {
  return launch_kernel(grad_norm_kernel, dim3(1), dim3(kThreads), 0, s, KernelTiming{}, part,
                       n_part, norm);
}

hipError_t launch_grad_scale(const GradTable& tab, const double* part, int n_part, float* norm,
                             float max_norm, int in_place, hipStream_t s) {
  const dim3 grid(grid_of(tab)), block(kThreads);
  if (tab.n <= kFew)
    return launch_kernel(grad_scale_kernel<FewTable>, grid, block, 0, s, KernelTiming{}, few(tab),
                         part, n_part, norm, max_norm, in_place);
  return launch_kernel(grad_scale_kernel<GradTable>, grid, block, 0, s, KernelTiming{}, tab, part,
                       n_part, norm, max_norm, in_place);
}

}  // namespace bmoe
