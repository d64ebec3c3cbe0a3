// Routing from logits: scores, the choice of experts and the gates; the
// gradient of the gates with respect to the logits; the loads of the experts
// and the update of the balance bias. The layer is a top-k mixture of experts
// (ButterflyMoE abstract; gist.science summary, §2.3) whose pages give no
// router formula; the readings are stated in the C header.
//
//   s = softmax(l) or sigmoid(l),  c = s + b   (c = -inf where l = -inf)
//   groups kept by the largest, or the sum of the two largest, c of a group
//   ids = the k largest c of the kept groups, ties to the lower id
//   g   = scale * s,  or scale * s / (sum of the chosen s)
#include "common.h"
#include "kernels.h"

namespace bmoe {
namespace {

// ---- order-preserving keys -----------------------------------------------------
// Unsigned integers in the order of the reals: 0 = not a candidate (taken, or
// of a group that is not kept), 1 = NaN (after -inf), -0 = +0.
__device__ __forceinline__ uint64_t key_of(double c) {
  if (c != c) return 1u;
  const int64_t b = __double_as_longlong(c + 0.0);
  return (uint64_t)b ^ ((uint64_t)(b >> 63) | 0x8000000000000000ull);
}

template <int LPT>
__device__ __forceinline__ double sub_max(double v) {
#pragma unroll
  for (int o = LPT / 2; o >= 1; o >>= 1) v = fmax(v, __shfl_xor(v, o, 64));
  return v;
}
template <int LPT>
__device__ __forceinline__ double sub_sum(double v) {
#pragma unroll
  for (int o = LPT / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

template <typename T>
__device__ __forceinline__ float ld_logit(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_lo(*reinterpret_cast<const uint16_t*>(p));
  else return *p;
}

// Gate of one chosen logit before the renormalisation, times e^(-shift) for
// the sigmoid (so the ratios keep their bits where every chosen score is tiny).
__device__ __forceinline__ double sigmoid_shifted(double l, double shift) {
  return l >= 0.0 ? 1.0 / (1.0 + exp(-l)) * exp(-shift) : exp(l - shift) / (1.0 + exp(l));
}

// LPT lanes per token, PER experts per lane (lane q of a token holds experts
// q * PER ... q * PER + PER - 1, so the lowest lane holds the lowest ids).
template <int LPT, int PER, typename T>
__global__ __launch_bounds__(256) void route_kernel(const T* logits, const float* bias, int T_,
                                                    int N, int k, RouteSpec sp, int32_t* ids,
                                                    float* gates) {
  const int q = threadIdx.x % LPT;
  const long long tok = (long long)blockIdx.x * (256 / LPT) + threadIdx.x / LPT;
  const bool live = tok < T_;
  const T* row = logits + (size_t)(live ? tok : 0) * N;
  const int base = q * PER;
  const bool softmax = sp.score == BMOE_SCORE_SOFTMAX;

  double l[PER];
  bool bad = false;
  double m = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = base + i;
    l[i] = e < N ? (double)ld_logit(row + e) : -INFINITY;
    bad |= l[i] != l[i] || (softmax && l[i] == INFINITY);
    m = fmax(m, l[i]);
  }
  const uint64_t own = LPT == 64 ? ~0ull : ((1ull << (LPT & 63)) - 1) << ((threadIdx.x & 63) / LPT * LPT);
  bad = (__ballot(bad) & own) != 0;
  m = sub_max<LPT>(m);

  // scores; the softmax's only up to its common factor where no bias is added
  double total = 0.0;
  if (softmax) {
#pragma unroll
    for (int i = 0; i < PER; ++i) total += l[i] == -INFINITY ? 0.0 : exp(l[i] - m);
    total = sub_sum<LPT>(total);
  }
  double c[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = base + i;
    if (bias == nullptr && !(sp.groups > 1 && sp.group_score == BMOE_GROUP_TOP2)) {
      c[i] = l[i];  // the scores rise with the logits
    } else {
      const double s = softmax ? exp(l[i] - m) / total : 1.0 / (1.0 + exp(-l[i]));
      c[i] = l[i] == -INFINITY ? -INFINITY : s + (bias && e < N ? (double)bias[e] : 0.0);
    }
  }

  // groups
  uint64_t keep = ~0ull;
  const int size = N / sp.groups;
  if (sp.groups > 1) {
    double mine = -INFINITY;  // lane g: the score of group g
    for (int g = 0; g < sp.groups; ++g) {
      double a = -INFINITY, b = -INFINITY;  // the two largest
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = base + i;
        if (e >= g * size && e < (g + 1) * size) {
          if (c[i] > a) { b = a; a = c[i]; }
          else if (c[i] > b) b = c[i];
        }
      }
#pragma unroll
      for (int o = LPT / 2; o >= 1; o >>= 1) {
        const double oa = __shfl_xor(a, o, 64), ob = __shfl_xor(b, o, 64);
        b = fmax(fmin(a, oa), a > oa ? b : ob);
        a = fmax(a, oa);
      }
      const double v = sp.group_score == BMOE_GROUP_MAX || b == -INFINITY ? a : a + b;
      if (q == g) mine = v;
    }
    int rank = 0;
    for (int h = 0; h < sp.groups; ++h) {
      const double v = __shfl(mine, (threadIdx.x & 63) / LPT * LPT + h, 64);
      rank += v > mine || (v == mine && h < q);
    }
    keep = __ballot(q < sp.groups && rank < sp.keep) >> ((threadIdx.x & 63) / LPT * LPT);
  }
  uint64_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = base + i;
    // without a bias the experts' order is that of their logits
    const double v = bias ? c[i] : l[i];
    key[i] = e < N && (sp.groups == 1 || (keep >> (e / size) & 1u)) ? key_of(v) : 0u;
  }

  // k rounds: the largest key, the lower id on ties; pick j stays in lane j
  int mine_id = 0;
  for (int j = 0; j < k; ++j) {
    uint64_t bk = 0;
    int bi = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] > bk) {
        bk = key[i];
        bi = base + i;
      }
#pragma unroll
    for (int o = LPT / 2; o >= 1; o >>= 1) {
      const uint64_t ok = __shfl_xor((unsigned long long)bk, o, 64);
      const int oi = __shfl_xor(bi, o, 64);
      if (ok > bk || (ok == bk && oi < bi)) {
        bk = ok;
        bi = oi;
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (base + i == bi) key[i] = 0;
    if (q == j) mine_id = bi;
  }

  // gates
  const bool pick = q < k;
  const double lj = pick ? (double)ld_logit(row + mine_id) : -INFINITY;
  double g;
  if (sp.renorm) {
    const double mc = sub_max<LPT>(lj);
    const double shift = softmax ? mc : fmin(mc, 0.0);
    const double u = !pick || lj == -INFINITY ? 0.0
                     : softmax ? exp(lj - shift) : sigmoid_shifted(lj, shift);
    const double sum = sub_sum<LPT>(u);
    g = sum > 0.0 ? u / sum : 0.0;
  } else {
    g = lj == -INFINITY ? 0.0 : softmax ? exp(lj - m) / total : 1.0 / (1.0 + exp(-lj));
  }
  if (live && pick) {
    ids[(size_t)tok * k + q] = mine_id;
    gates[(size_t)tok * k + q] = bad ? NAN : (float)((double)sp.scale * g);
  }
}

// ---- gradient of the gates --------------------------------------------------------
// What pick (id, u) of its LPT lanes' token adds to dl[id], for the specs
// under which only the picks move. l: the pick's logit, -inf for no pick.
template <int LPT>
__device__ __forceinline__ double pick_grad(double l, double u, const RouteSpec& sp) {
  const bool softmax = sp.score == BMOE_SCORE_SOFTMAX;
  double v;
  if (sp.renorm) {
    const double mc = sub_max<LPT>(l);
    const double shift = softmax ? mc : fmin(mc, 0.0);
    const double w = l == -INFINITY ? 0.0 : softmax ? exp(l - shift) : sigmoid_shifted(l, shift);
    const double sum = sub_sum<LPT>(w);
    const double p = sum > 0.0 ? w / sum : 0.0;
    v = p * (u - sub_sum<LPT>(u * p));
    if (!softmax) v *= 1.0 / (1.0 + exp(l));
  } else {
    v = u * (1.0 / (1.0 + exp(-l))) * (1.0 / (1.0 + exp(l)));
  }
  return l == -INFINITY ? 0.0 : v;
}

// One wave per token; lane j < k holds pick j. With u_j the gates' gradient
// times scale:
//   renormalised:  dl_j = p_j (u_j - sum_i u_i p_i) [ (1 - s_j) ],  p = s / sum
//   sigmoid:       dl_j = u_j s_j (1 - s_j)
//   softmax:       dl_e = s_e (sum over j with id_j = e of u_j  -  sum_i u_i s_i)
// An id outside [0, N) contributes nothing; equal ids add up in their order.
template <typename T>
__global__ __launch_bounds__(256) void route_bwd_kernel(const T* logits, const int32_t* ids,
                                                        const float* dgates, int T_, int N, int k,
                                                        RouteSpec sp, float* dlogits) {
  const int lane = threadIdx.x & 63;
  const size_t tok = (size_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (tok >= (size_t)T_) return;  // whole wave
  const T* row = logits + tok * N;
  float* out = dlogits + tok * N;
  const bool softmax = sp.score == BMOE_SCORE_SOFTMAX;
  const int id = lane < k ? ids[tok * k + lane] : -1;
  const bool pick = id >= 0 && id < N;
  const float l = pick ? ld_logit(row + id) : -INFINITY;
  const float u = pick ? sp.scale * dgates[tok * k + lane] : 0.f;
  double m = -INFINITY, total = 0.0, v = u;  // v: this pick's dl, or (dense) its u
  const bool dense = softmax && !sp.renorm;
  if (!dense) {
    v = pick_grad<64>((double)l, (double)u, sp);
  } else {
    for (int e = lane; e < N; e += 64) m = fmax(m, (double)ld_logit(row + e));
    m = sub_max<64>(m);
    for (int e = lane; e < N; e += 64) {
      const double x = ld_logit(row + e);
      total += x == -INFINITY ? 0.0 : exp(x - m);
    }
    total = sub_sum<64>(total);
  }
  if (!pick || l == -INFINITY) v = 0.0;
  double d = 0.0;
  if (dense) d = sub_sum<64>(l == -INFINITY ? 0.0 : u * (exp((double)l - m) / total));
  for (int e = lane; e - lane < N; e += 64) {
    double a = 0.0;
    for (int j = 0; j < k; ++j) {
      const int ij = __shfl(id, j, 64);
      const double vj = __shfl(v, j, 64);
      if (ij == e) a += vj;
    }
    if (e >= N) continue;
    if (dense) {
      const double x = ld_logit(row + e);
      a = x == -INFINITY ? 0.0 : exp(x - m) / total * (a - d);
    }
    out[e] = (float)a;
  }
}

// The picks' (id, coefficient) pairs of one range of tokens, and the same
// listed by expert (stable): one workgroup per range. Each wave owns a
// contiguous share of the range's picks; equal experts within 64 picks are
// ranked by ballots over the id's bits.
template <int LPT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void route_pairs_kernel(
    const float* logits, const int32_t* ids, const float* dgates, int T_, int N, int k, int nbits,
    RouteSpec sp, RouterPairs rp) {
  extern __shared__ int cur[];  // [WAVES][N]: counts, then cursors
  __shared__ int wsum[WAVES];
  constexpr int kThreads = WAVES * 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const size_t t0 = (size_t)blockIdx.x * rp.tokens;
  const int nt = (int)min((size_t)rp.tokens, (size_t)T_ - t0);
  for (int i = tid; i < WAVES * N; i += kThreads) cur[i] = 0;
  const int q = tid % LPT;
  for (int i = tid / LPT; i - tid / LPT < nt; i += kThreads / LPT) {
    const size_t tok = t0 + i;
    const bool mine = i < nt && q < k;
    const int id = mine ? ids[tok * k + q] : -1;
    const bool pick = id >= 0 && id < N;
    const float l = pick ? logits[tok * N + id] : -INFINITY;
    const float u = pick ? sp.scale * dgates[tok * k + q] : 0.f;
    const float v = (float)pick_grad<LPT>((double)l, (double)u, sp);
    if (mine) rp.pairs[tok * k + q] = make_int2(pick ? id : 0, __float_as_int(pick ? v : 0.f));
  }
  __syncthreads();

  const int M = nt * k;
  const int2* pairs = rp.pairs + t0 * k;
  const int share = ((M + WAVES - 1) / WAVES + 63) / 64 * 64;
  const int wb = min(M, wave * share), we = min(M, wb + share);
  int* mycur = cur + wave * N;
  for (int r = wb + lane; r < we; r += 64) {
    const int2 p = pairs[r];
    if (__int_as_float(p.y) != 0.f) atomicAdd(&mycur[p.x], 1);
  }
  __syncthreads();
  // exclusive scan over (expert, wave); a thread owns consecutive experts
  const int per = (N + kThreads - 1) / kThreads;
  const int lo = min(N, tid * per), hi = min(N, lo + per);
  int seg = 0;
  for (int e = lo; e < hi; ++e)
    for (int w = 0; w < WAVES; ++w) seg += cur[w * N + e];
  const int incl = wave_incl_scan(seg);
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int run = (int)(t0 * k) + incl - seg;
  for (int w = 0; w < wave; ++w) run += wsum[w];
  int32_t* off = rp.off + (size_t)blockIdx.x * (N + 1);
  for (int e = lo; e < hi; ++e) {
    off[e] = run;
    for (int w = 0; w < WAVES; ++w) {
      const int c = cur[w * N + e];
      cur[w * N + e] = run;
      run += c;
    }
  }
  if (tid == kThreads - 1) off[N] = run;
  __syncthreads();
  const uint64_t lt = (1ull << lane) - 1;
  for (int base = wb; base < we; base += 64) {
    const int r = base + lane;
    const int2 p = r < we ? pairs[r] : make_int2(0, 0);
    const bool valid = r < we && __int_as_float(p.y) != 0.f;
    uint64_t mask = __ballot(valid);
    for (int b = 0; b < nbits; ++b) {
      const bool bit = (p.x >> b) & 1;
      const uint64_t bal = __ballot(bit);
      mask &= bit ? bal : ~bal;
    }
    const int rank = __popcll(mask & lt), grp = __popcll(mask);
    const int at = valid ? mycur[p.x] : 0;
    __builtin_amdgcn_wave_barrier();
    if (valid) {
      rp.list[at + rank] = make_int2((int)(t0 + r / k), p.y);
      if (rank == grp - 1) mycur[p.x] = at + grp;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- loads and the balance bias -----------------------------------------------------
// One workgroup: a histogram in LDS (integers, so the order does not matter),
// then bias[e] += rate * sign(mean - load[e]) with the comparison in integers
// (sum of the loads against N * load).
__global__ __launch_bounds__(1024) void balance_kernel(const int32_t* ids, long long M, int N,
                                                       int accumulate, float rate, int32_t* load,
                                                       float* bias) {
  __shared__ int hist[kMaxExperts];
  __shared__ long long sum;
  if (threadIdx.x == 0) sum = 0;
  for (int e = threadIdx.x; e < N; e += 1024) hist[e] = accumulate ? load[e] : 0;
  __syncthreads();
  for (long long r = threadIdx.x; r < M; r += 1024) {
    const int e = ids[r];
    if (e >= 0 && e < N) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  long long part = 0;
  for (int e = threadIdx.x; e < N; e += 1024) part += hist[e];
  if (part) atomicAdd((unsigned long long*)&sum, (unsigned long long)part);
  __syncthreads();
  for (int e = threadIdx.x; e < N; e += 1024) {
    load[e] = hist[e];
    if (bias) {
      const long long diff = sum - (long long)N * hist[e];
      bias[e] += diff > 0 ? rate : diff < 0 ? -rate : 0.f;
    }
  }
}

template <typename T>
hipError_t route_t(const T* logits, const float* bias, int Tn, int N, int k, const RouteSpec& sp,
                   int32_t* ids, float* gates, hipStream_t s) {
  const int need = k > sp.groups ? k : sp.groups;  // picks and group scores sit one per lane
#define BMOE_ROUTE(LPT, PER)                                                                  \
  return launch_kernel(route_kernel<LPT, PER, T>, dim3(((unsigned)Tn + 256 / LPT - 1) / (256 / LPT)),   \
                       dim3(256), 0, s, KernelTiming{}, logits, bias, Tn, N, k, sp, ids, gates)
  if (need <= 16 && N <= 64) BMOE_ROUTE(16, 4);
  if (need <= 16 && N <= 256) BMOE_ROUTE(16, 16);
  if (N <= 256) BMOE_ROUTE(64, 4);
  if (N <= 1024) BMOE_ROUTE(64, 16);
  BMOE_ROUTE(64, 64);
#undef BMOE_ROUTE
}

}  // namespace

hipError_t launch_route(bmoe_dtype dt, int T, int N, int k, const RouteSpec& sp,
                        const void* logits, const float* bias, int32_t* ids, float* gates,
                        hipStream_t s) {
  if (dt == BMOE_BF16)
    return route_t(static_cast<const uint16_t*>(logits), bias, T, N, k, sp, ids, gates, s);
  return route_t(static_cast<const float*>(logits), bias, T, N, k, sp, ids, gates, s);
}

hipError_t launch_route_bwd(bmoe_dtype dt, int T, int N, int k, const RouteSpec& sp,
                            const void* logits, const int32_t* ids, const float* dgates,
                            float* dlogits, hipStream_t s) {
  const dim3 grid(((unsigned)T + 3) / 4), block(256);
  if (dt == BMOE_BF16)
    return launch_kernel(route_bwd_kernel<uint16_t>, grid, block, 0, s, KernelTiming{},
                         static_cast<const uint16_t*>(logits), ids, dgates, T, N, k, sp, dlogits);
  return launch_kernel(route_bwd_kernel<float>, grid, block, 0, s, KernelTiming{},
                       static_cast<const float*>(logits), ids, dgates, T, N, k, sp, dlogits);
}

hipError_t launch_route_pairs(int T, int N, int k, const RouteSpec& sp, const float* logits,
                              const int32_t* ids, const float* dgates, const RouterPairs& rp,
                              hipStream_t s) {
  int nbits = 0;
  while ((1 << nbits) < N) ++nbits;
  // 16 waves while their cursors take 32 KB at most, else 4 (64 KB at 4096)
#define BMOE_PAIRS(LPT)                                                                        \
  return N <= 512 ? launch_kernel(route_pairs_kernel<LPT, 16>, dim3(rp.ranges), dim3(1024),    \
                                  16 * N * 4, s, KernelTiming{}, logits, ids, dgates, T, N, k, \
                                  nbits, sp, rp)                                               \
                  : launch_kernel(route_pairs_kernel<LPT, 4>, dim3(rp.ranges), dim3(256),      \
                                  4 * N * 4, s, KernelTiming{}, logits, ids, dgates, T, N, k,  \
                                  nbits, sp, rp)
  if (k <= 2) BMOE_PAIRS(2);
  if (k <= 4) BMOE_PAIRS(4);
  if (k <= 8) BMOE_PAIRS(8);
  if (k <= 16) BMOE_PAIRS(16);
  BMOE_PAIRS(64);
#undef BMOE_PAIRS
}

hipError_t launch_balance(long long M, int N, const int32_t* ids, int accumulate, float rate,
                          int32_t* load, float* bias, hipStream_t s) {
  return launch_kernel(balance_kernel, dim3(1), dim3(1024), 0, s, KernelTiming{}, ids, M, N,
                       accumulate, rate, load, bias);
}

}  // namespace bmoe
