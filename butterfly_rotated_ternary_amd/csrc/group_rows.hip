// Routed rows grouped by expert: a stable counting sort of the M = T k ids.
//   offsets[e] .. offsets[e + 1]  the sorted slots of expert e
//   perm[slot] = r                experts ascending, r ascending within one
//   inv[r] = slot                 (-1 for an id outside [0, N): a padded pick)
// Padded picks take the slots behind the last expert's, in order of r.
//
// Bound by latency: the ids are 4 M bytes. They are cut into at most 256
// chunks. One launch counts each chunk's experts, a second gives every chunk
// the counts before it (at most 256 x N words from L2) and ranks its own rows
// (64 at a time, one ballot per bit of the expert). One chunk needs no counts
// from elsewhere: a single launch. In the trace 8 ids of 256 experts take 3.3 to 3.8 us,
// 3009 of 60 5.2, 8192 of 64 8.9 to 9.4, 131072 of 256 3.3 + 8.9 call after call and
// 6.2 + 10.6 where other work has been in between.
#include "common.h"
#include "kernels.h"

namespace bmoe {
namespace {

constexpr int kThreads = 256;  // of the count
constexpr int kMostChunks = 256;
constexpr int kLeastChunk = 2048;

// Waves of the scatter, each with a cursor per expert in LDS: sixteen (131072 ids of
// 256 experts 8.6 us, four 17), or four where sixteen would pass 64 KB.
int waves_of(int N) { return 17 * (N + 1) * (int)sizeof(int) + 64 <= 65536 ? 16 : 4; }

struct GroupArgs {
  const int32_t* ids;
  int32_t *offsets, *perm, *inv;
  int* count;  // [chunks][N + 1]
  int M, N, chunk, chunks, nbits;
};

// Expert N is the padded picks'.
__device__ __forceinline__ int key_of(const GroupArgs& p, int r) {
  const int e = p.ids[r];
  return (unsigned)e < (unsigned)p.N ? e : p.N;
}

__global__ __launch_bounds__(kThreads) void group_count_kernel(GroupArgs p) {
  extern __shared__ int cnt[];
  const int n = p.N + 1;
  for (int e = threadIdx.x; e < n; e += kThreads) cnt[e] = 0;
  __syncthreads();
  const long long r0 = (long long)blockIdx.x * p.chunk;
  const int len = (int)min((long long)p.chunk, p.M - r0);
  for (int i = threadIdx.x; i < len; i += kThreads) atomicAdd(&cnt[key_of(p, (int)(r0 + i))], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += kThreads) p.count[(size_t)blockIdx.x * n + e] = cnt[e];
}

template <int WAVES>
__global__ __launch_bounds__(64 * WAVES) void group_scatter_kernel(GroupArgs p) {
  constexpr int THREADS = 64 * WAVES;
  extern __shared__ int sh[];  // [WAVES][n] cursors, [n] bases
  __shared__ int scratch[WAVES];
  const int n = p.N + 1, tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  int* base = sh + WAVES * n;
  const long long r0 = (long long)blockIdx.x * p.chunk;
  const int len = (int)min((long long)p.chunk, p.M - r0);
  for (int i = tid; i < WAVES * n; i += THREADS) sh[i] = 0;
  __syncthreads();
  // each wave owns a contiguous share of the chunk and counts it
  const int share = (len + WAVES - 1) / WAVES;
  const int wb = min(len, wave * share), we = min(len, wb + share);
  int* cur = sh + wave * n;
  for (int i = wb + lane; i < we; i += kWave) atomicAdd(&cur[key_of(p, (int)(r0 + i))], 1);
  __syncthreads();
  // per expert: the rows of all chunks, and of those before this one
  for (int e = tid; e < n; e += THREADS) {
    int total = 0, before = 0;
    if (p.chunks == 1) {
#pragma unroll
      for (int w = 0; w < WAVES; ++w) total += sh[w * n + e];
    } else {
      // 16 loads in flight (131072 ids in 64 chunks: 33 us one by one)
      for (int c0 = 0; c0 < p.chunks; c0 += 16) {
        int v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          v[i] = c0 + i < p.chunks ? p.count[(size_t)(c0 + i) * n + e] : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          total += v[i];
          before += c0 + i < (int)blockIdx.x ? v[i] : 0;
        }
      }
    }
    base[e] = total;
    // the wave's own counts become cursors relative to the expert's base
    int at = before;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const int v = sh[w * n + e];
      sh[w * n + e] = at;
      at += v;
    }
  }
  __syncthreads();
  // exclusive prefix sum of the totals: each thread owns a run of experts
  const int per = (n + THREADS - 1) / THREADS;
  const int lo = min(n, tid * per), hi = min(n, lo + per);
  int seg = 0;
  for (int e = lo; e < hi; ++e) seg += base[e];
  const int incl = wave_incl_scan(seg);
  if (lane == kWave - 1) scratch[wave] = incl;
  __syncthreads();
  int at = incl - seg;
  for (int w = 0; w < wave; ++w) at += scratch[w];
  for (int e = lo; e < hi; ++e) {
    const int v = base[e];
    base[e] = at;
    if (blockIdx.x == 0) p.offsets[e] = at;  // e = N: where the padded picks begin
    at += v;
  }
  __syncthreads();
  // stable ranks: lanes with the same expert found by one ballot per bit
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (kWave - lane);
  for (int i0 = wb; i0 < we; i0 += kWave) {
    const bool valid = i0 + lane < we;
    const int r = (int)(r0 + i0 + lane);
    const int e = valid ? key_of(p, r) : 0;
    uint64_t same = __ballot(valid);
    for (int b = 0; b < p.nbits; ++b) {
      const bool bit = (e >> b) & 1;
      const uint64_t has = __ballot(bit);
      same &= bit ? has : ~has;
    }
    const int rank = __popcll(same & below), group = __popcll(same);
    const int c = valid ? cur[e] : 0;
    __builtin_amdgcn_wave_barrier();
    if (valid) {
      const int slot = base[e] + c + rank;
      p.perm[slot] = r;
      p.inv[r] = e < p.N ? slot : -1;
      if (rank == group - 1) cur[e] = c + group;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// One chunk as long as a wave has at most eight times 64 rows. On the device one launch
// is the shorter way up to about 5000 ids (64 experts, in a captured graph: 4096 6.2
// against 7.2 us, 6144 7.9 against 7.6, 8192 9.5 against 7.7), but the host pays 2.5 us
// for the second one (any of these, call after call: 11.8 against 14.3 us; alone, with
// the GPU waited for, 8192 28.1 against 26.1).
int chunk_of(int M, int N) {
  if (M <= 512 * waves_of(N)) return 512 * waves_of(N);
  const int c = (int)(((long long)M + kMostChunks - 1) / kMostChunks);
  return c < kLeastChunk ? kLeastChunk : c;
}

}  // namespace

size_t group_count_bytes(int M, int N) {
  const size_t chunk = chunk_of(M, N), chunks = (M + chunk - 1) / chunk;
  return chunks > 1 ? chunks * (N + 1) * sizeof(int) : 0;
}

hipError_t launch_group_rows(const int32_t* ids, int M, int N, int32_t* offsets, int32_t* perm,
                             int32_t* inv, int* count, hipStream_t s) {
  GroupArgs p;
  p.ids = ids;
  p.offsets = offsets;
  p.perm = perm;
  p.inv = inv;
  p.count = count;
  p.M = M;
  p.N = N;
  p.chunk = chunk_of(M, N);
  p.chunks = M > 0 ? (int)(((long long)M + p.chunk - 1) / p.chunk) : 1;
  p.nbits = 0;
  while ((1 << p.nbits) < N + 1) ++p.nbits;
  if (p.chunks > 1) {
    const hipError_t e = launch_kernel(group_count_kernel, dim3(p.chunks), dim3(kThreads),
                                       (uint32_t)(sizeof(int) * (N + 1)), s, KernelTiming{}, p);
    if (e != hipSuccess) return e;
  }
  if (waves_of(N) == 16)
    return launch_kernel(group_scatter_kernel<16>, dim3(p.chunks), dim3(64 * 16),
                         (uint32_t)(sizeof(int) * 17 * (N + 1)), s, KernelTiming{}, p);
  const size_t lds = sizeof(int) * (size_t)5 * (N + 1);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(group_scatter_kernel<4>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  return launch_kernel(group_scatter_kernel<4>, dim3(p.chunks), dim3(64 * 4), (uint32_t)lds, s,
                       KernelTiming{}, p);
}

}  // namespace bmoe
