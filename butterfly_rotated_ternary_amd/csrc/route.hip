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

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kU = 5.9604644775390625e-8f;  // 2^-24: half a step of fp32, relative

// ---- exchanges among the LPT lanes of one token ------------------------------------
// All-reduce by DPP inside 16 lanes (each step pairs lanes whose groups hold
// one value: lane ^ 1, lane ^ 2, the mirrored half row, the mirrored row) and
// by gfx950's row and half swaps above. No LDS round trips.
template <int O>
__device__ __forceinline__ uint32_t partner(uint32_t v) {
  if constexpr (O == 1) return __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);
  else if constexpr (O == 2) return __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);
  else if constexpr (O == 4) return __builtin_amdgcn_mov_dpp(v, 0x141, 0xF, 0xF, true);
  else return __builtin_amdgcn_mov_dpp(v, 0x140, 0xF, 0xF, true);
}
template <int LPT, typename F>
__device__ __forceinline__ uint32_t sub_reduce(uint32_t v, F f) {
  if constexpr (LPT >= 2) v = f(v, partner<1>(v));
  if constexpr (LPT >= 4) v = f(v, partner<2>(v));
  if constexpr (LPT >= 8) v = f(v, partner<4>(v));
  if constexpr (LPT >= 16) v = f(v, partner<8>(v));
  if constexpr (LPT >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = f(r[0], r[1]);
  }
  if constexpr (LPT >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = f(r[0], r[1]);
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t sub_max(uint32_t v) {
  return sub_reduce<LPT>(v, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
}
template <int LPT>
__device__ __forceinline__ uint32_t sub_min(uint32_t v) {
  return sub_reduce<LPT>(v, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
}
template <int LPT>
__device__ __forceinline__ float sub_max(float v) {
  return __uint_as_float(sub_reduce<LPT>(__float_as_uint(v), [](uint32_t x, uint32_t y) {
    return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y)));
  }));
}
template <int LPT>
__device__ __forceinline__ float sub_sum(float v) {
  return __uint_as_float(sub_reduce<LPT>(__float_as_uint(v), [](uint32_t x, uint32_t y) {
    return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
  }));
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
template <int LPT>
__device__ __forceinline__ uint64_t sub_max(uint64_t v) {
#pragma unroll
  for (int o = LPT / 2; o >= 1; o >>= 1) {
    const uint64_t w = __shfl_xor((unsigned long long)v, o, 64);
    v = w > v ? w : v;
  }
  return v;
}

// Lanes of this lane's token in a ballot, moved to bit 0.
template <int LPT>
__device__ __forceinline__ uint64_t own_bits(uint64_t ballot) {
  if constexpr (LPT == 64) return ballot;
  else return ballot >> ((threadIdx.x & 63) / LPT * LPT) & ((1ull << LPT) - 1);
}

// ---- order-preserving keys -----------------------------------------------------
// Unsigned integers in the order of the reals: 0 = not a candidate (taken, or
// of a group that is not kept), 1 = NaN (after -inf), -0 = +0.
__device__ __forceinline__ uint32_t key_of(float c) {
  const int32_t b = __float_as_int(c + 0.f);
  return c != c ? 1u : (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(double c) {
  const int64_t b = __double_as_longlong(c + 0.0);
  return c != c ? 1ull : (uint64_t)b ^ ((uint64_t)(b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// ---- scores ----------------------------------------------------------------------
// e^v on the exponential unit: off by (1.3 |v| + 2) 2^-24, relative (the
// product with log2 e, that constant, the unit's last place); a difference v
// brings |v| 2^-24 more.
__device__ __forceinline__ float exp_of(float v) { return __builtin_amdgcn_exp2f(v * kLog2e); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }
__device__ __forceinline__ float inv_of(float v) { return __builtin_amdgcn_rcpf(v); }
__device__ __forceinline__ double inv_of(double v) { return 1.0 / v; }

// Sigmoid of l times e^(-shift), shift <= 0 and 0 unless every l of interest
// is negative: ratios of such scores keep their bits where all are tiny.
template <typename R>
__device__ __forceinline__ R sigmoid_shifted(R l, R shift) {
  return l >= R(0) ? inv_of(R(1) + exp_of(-l)) : exp_of(l - shift) * inv_of(R(1) + exp_of(l));
}

template <typename T>
__device__ __forceinline__ float ld_logit(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_lo(*reinterpret_cast<const uint16_t*>(p));
  else return *p;
}

// This lane's PER consecutive values of a row of n from `base` on, `fill`
// past its end. VEC: n is a multiple of the vector's length.
template <int PER, bool VEC, typename T>
__device__ __forceinline__ void ld_row(const T* row, int base, int n, float fill,
                                       float (&v)[PER]) {
  constexpr int W = 16 / sizeof(T) < PER ? 16 / sizeof(T) : PER;  // values per load
  if constexpr (VEC && W > 1) {
#pragma unroll
    for (int i = 0; i < PER; i += W) {
      const bool in = base + i < n;
      const T* p = row + (in ? base + i : 0);
      float f[W];
      if constexpr (sizeof(T) == 4) {
        if constexpr (W == 4) {
          const float4 x = *reinterpret_cast<const float4*>(p);
          f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(p);
          f[0] = x.x; f[1] = x.y;
        }
      } else {
        uint32_t d[W / 2];
        if constexpr (W == 8) {
          const uint4 x = *reinterpret_cast<const uint4*>(p);
          d[0] = x.x; d[1] = x.y; d[2] = x.z; d[3] = x.w;
        } else if constexpr (W == 4) {
          const uint2 x = *reinterpret_cast<const uint2*>(p);
          d[0] = x.x; d[1] = x.y;
        } else {
          d[0] = *reinterpret_cast<const uint32_t*>(p);
        }
#pragma unroll
        for (int u = 0; u < W / 2; ++u) {
          f[2 * u] = bf16_lo(d[u]);
          f[2 * u + 1] = bf16_hi(d[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < W; ++u) v[i + u] = in ? f[u] : fill;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool in = base + i < n;
      const float f = ld_logit(row + (in ? base + i : 0));
      v[i] = in ? f : fill;
    }
  }
}

// ---- the choice ------------------------------------------------------------------
// k picks of one token by its LPT lanes, PER experts per lane (lane q holds
// experts q PER ... q PER + PER - 1, so the lowest lane has the lowest ids).
// Returns pick j's id in lane j. In fp32 (R = float) scores are a few units
// off, so *unsure is set for a token whose picks, or kept groups, are not
// further apart than the errors allow (bounded below); the caller then decides
// that token with R = double. Without a bias the keys are the logits
// themselves and nothing is unsure but sums of two scores.
template <int LPT, int PER, typename R, typename T>
__device__ __forceinline__ int choose(const T* row, const float* bias, const float (&l)[PER],
                                      const float (&b)[PER], int base, int N, int k,
                                      const RouteSpec& sp, float lmax, bool* unsure) {
  constexpr bool kFast = sizeof(R) == 4;
  using K = decltype(key_of(R(0)));
  const bool biased = bias != nullptr;
  const int q = threadIdx.x % LPT;
  const bool softmax = sp.score == BMOE_SCORE_SOFTMAX;
  const bool scored = biased || (sp.groups > 1 && sp.group_score == BMOE_GROUP_TOP2);
  const R m = softmax ? (R)lmax : R(0);
  // A score s of a logit at distance x from m is off by s u (3 |x| + A) at
  // most: the difference, its product with log2 e and that constant, then the
  // exponential's, sum's (PER + 6 additions) and quotient's last places.
  constexpr float kA = PER + 24;
  R c[PER], smax = R(1);
  if (scored) {
    R inv = R(1);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      c[i] = softmax ? (l[i] == -INFINITY ? R(0) : exp_of((R)l[i] - m))
                     : inv_of(R(1) + exp_of(-(R)l[i]));
    if (softmax) {
      R total = R(0);
#pragma unroll
      for (int i = 0; i < PER; ++i) total += c[i];
      inv = R(1) / sub_sum<LPT>(total);
      smax = inv;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      c[i] = l[i] == -INFINITY ? R(-INFINITY) : c[i] * inv + (R)b[i];
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = (R)l[i];
  }

  uint64_t keep = 1;  // bit g: group g is kept
  const int size = N / sp.groups;
  if (sp.groups > 1) {
    R mine = R(-INFINITY), slack = R(0);  // lane g: the score of group g, its error
    for (int g = 0; g < sp.groups; ++g) {
      R a = R(-INFINITY), a2 = R(-INFINITY);  // the two largest
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const R v = base + i >= g * size && base + i < (g + 1) * size ? c[i] : R(-INFINITY);
        if (v > a) { a2 = a; a = v; }
        else if (v > a2) a2 = v;
      }
#pragma unroll
      for (int o = LPT / 2; o >= 1; o >>= 1) {
        const R oa = __shfl_xor(a, o, 64), ob = __shfl_xor(a2, o, 64);
        a2 = fmax(fmin(a, oa), a > oa ? a2 : ob);
        a = fmax(a, oa);
      }
      const bool one = sp.group_score == BMOE_GROUP_MAX || a2 == R(-INFINITY);
      if (q == g) {
        mine = one ? a : a + a2;
        if (kFast && scored)
          slack = R(kU) * (R(2) * smax * R(kA + 1.f) + R(3) * (fabs(a) + (one ? R(0) : fabs(a2))));
      }
    }
    int rank = 0;
    for (int h = 0; h < sp.groups; ++h) {
      const R v = __shfl(mine, (threadIdx.x & 63) / LPT * LPT + h, 64);
      rank += v > mine || (v == mine && h < q);
    }
    const bool kept = q < sp.groups && rank < sp.keep;
    keep = own_bits<LPT>(__ballot(kept));
    if constexpr (kFast) {
      if (scored) {
        // the lowest that a kept group, and the highest that another can be
        const float lowest = -sub_max<LPT>(kept ? -(mine - slack) : -INFINITY);
        const float highest =
            sub_max<LPT>(q < sp.groups && !kept ? mine + slack : -INFINITY);
        *unsure |= !(lowest > highest);
      }
    }
  }

  K key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = base + i;
    const bool in = e < N && (sp.groups == 1 || (keep >> (e / size) & 1u));
    key[i] = in ? key_of(biased ? c[i] : (R)l[i]) : K(0);
  }

  // k rounds: the largest key, the lower id on ties
  int id = 0;
  K top = 0;
  for (int j = 0; j < k; ++j) {
    K best = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) best = key[i] > best ? key[i] : best;
    best = sub_max<LPT>(best);
    uint32_t at = 0x7fffffff;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) at = key[i] == best ? (uint32_t)(base + i) : at;
    at = sub_min<LPT>(at);
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = at == (uint32_t)(base + i) ? K(0) : key[i];
    if (q == j) {
      id = (int)at;
      top = best;
    }
  }
  if constexpr (kFast) {
    if (biased) {
      // Each pick's choice minus its error has to be above the next pick's
      // plus that one's, and the last's above every expert left. Experts of
      // the same logit and bias tie exactly, and so do equal infinities: the
      // ids have ordered those.
      auto err = [&](float cv, float lv, float bv) {
        const float s = fabsf(cv - bv), x = softmax ? lmax - lv : fabsf(lv);
        return kU * (s * (3.f * x + kA) + 3.f * fabsf(cv));
      };
      auto ties = [](float c0, float l0, float b0, float c1, float l1, float b1) {
        return (l0 == l1 && b0 == b1) || (c0 == c1 && fabsf(c0) == INFINITY);
      };
      const bool pick = q < k;
      const float lj = pick ? ld_logit(row + id) : 0.f, bj = pick ? bias[id] : 0.f;
      const float cj = value_of(top);
      const float ej = fabsf(cj) == INFINITY ? 0.f : err(cj, lj, bj);
      const int here = threadIdx.x & 63, last = here / LPT * LPT + k - 1;
      const float cn = __shfl(cj, here + 1, 64), en = __shfl(ej, here + 1, 64);
      const float ln = __shfl(lj, here + 1, 64), bn = __shfl(bj, here + 1, 64);
      bool ok = q >= k - 1 || ties(cj, lj, bj, cn, ln, bn) || cj - ej > cn + en;
      const float ck = __shfl(cj, last, 64), ek = __shfl(ej, last, 64);
      const float lk = __shfl(lj, last, 64), bk = __shfl(bj, last, 64);
      float left = -INFINITY;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float cv = value_of(key[i]);
        if (key[i] != 0 && !ties(ck, lk, bk, cv, l[i], b[i]))
          left = fmaxf(left, fabsf(cv) == INFINITY ? cv : cv + err(cv, l[i], b[i]));
      }
      ok &= left == -INFINITY ? ck == ck : ck - ek > left;
      *unsure |= !ok;
    }
  }
  return id;
}

// ---- routing ----------------------------------------------------------------------
template <int LPT, int PER, bool VEC, typename T>
__global__ __launch_bounds__(256) void route_kernel(const T* logits, const float* bias, int T_,
                                                    int N, int k, RouteSpec sp, int32_t* ids,
                                                    float* gates) {
  constexpr int kTok = 256 / LPT;  // tokens per workgroup
  const int q = threadIdx.x % LPT, base = q * PER;
  const bool softmax = sp.score == BMOE_SCORE_SOFTMAX;
  float b[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) b[i] = 0.f;
  if (bias) ld_row<PER, VEC>(bias, base, N, 0.f, b);
  for (size_t t0 = (size_t)blockIdx.x * kTok; t0 < (size_t)T_; t0 += (size_t)gridDim.x * kTok) {
    const size_t tok = t0 + threadIdx.x / LPT;
    const bool live = tok < (size_t)T_;
    const T* row = logits + (live ? tok : 0) * N;
    float l[PER];
    ld_row<PER, VEC>(row, base, N, -INFINITY, l);
    bool bad = false;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      bad |= l[i] != l[i];
      m = fmaxf(m, l[i]);
    }
    m = sub_max<LPT>(m);
    bad = own_bits<LPT>(__ballot(bad)) != 0 || (softmax && m == INFINITY);

    bool unsure = false;
    int id = choose<LPT, PER, float>(row, bias, l, b, base, N, k, sp, m, &unsure);
    if (__any(unsure)) id = choose<LPT, PER, double>(row, bias, l, b, base, N, k, sp, m, &unsure);

    const bool pick = q < k;
    const float lj = pick ? ld_logit(row + id) : -INFINITY;
    float g;
    if (sp.renorm) {
      const float mc = sub_max<LPT>(lj);
      const float shift = softmax ? mc : fminf(mc, 0.f);
      const float u = lj == -INFINITY ? 0.f
                      : softmax ? exp_of(lj - shift) : sigmoid_shifted(lj, shift);
      const float sum = sub_sum<LPT>(u);
      g = sum > 0.f ? u / sum : 0.f;
    } else if (softmax) {
      float total = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) total += l[i] == -INFINITY ? 0.f : exp_of(l[i] - m);
      total = sub_sum<LPT>(total);
      g = lj == -INFINITY ? 0.f : exp_of(lj - m) / total;
    } else {
      g = lj == -INFINITY ? 0.f : inv_of(1.f + exp_of(-lj));
    }
    if (live && pick) {
      ids[tok * k + q] = id;
      gates[tok * k + q] = bad ? NAN : sp.scale * g;
    }
  }
}

// ---- gradient of the gates --------------------------------------------------------
// With u_j the gates' gradient times scale:
//   renormalised:  dl_j = p_j (u_j - sum_i u_i p_i) [ (1 - s_j) ],  p = s / sum
//   sigmoid:       dl_j = u_j s_j (1 - s_j)
//   softmax:       dl_e = s_e (sum over j with id_j = e of u_j  -  sum_i u_i s_i)
// An id outside [0, N) contributes nothing; equal ids add up in their order.

// What pick (l, u) of its LPT lanes' token adds to its logit's gradient, for
// the specs under which only the picks move. l = -inf: no pick, or masked.
template <int LPT>
__device__ __forceinline__ float pick_grad(float l, float u, const RouteSpec& sp) {
  const bool softmax = sp.score == BMOE_SCORE_SOFTMAX;
  float v;
  if (sp.renorm) {
    const float mc = sub_max<LPT>(l);
    const float shift = softmax ? mc : fminf(mc, 0.f);
    const float w = l == -INFINITY ? 0.f : softmax ? exp_of(l - shift) : sigmoid_shifted(l, shift);
    const float sum = sub_sum<LPT>(w);
    const float p = sum > 0.f ? w / sum : 0.f;
    v = p * (u - sub_sum<LPT>(u * p));
    if (!softmax) v *= inv_of(1.f + exp_of(l));
  } else {
    v = u * inv_of(1.f + exp_of(-l)) * inv_of(1.f + exp_of(l));
  }
  return l == -INFINITY ? 0.f : v;
}

template <int LPT, int PER, bool VEC, typename T>
__global__ __launch_bounds__(256) void route_bwd_kernel(const T* logits, const int32_t* ids,
                                                        const float* dgates, int T_, int N, int k,
                                                        RouteSpec sp, float* dlogits) {
  const int q = threadIdx.x % LPT, base = q * PER;
  const size_t tok = (size_t)blockIdx.x * (256 / LPT) + threadIdx.x / LPT;
  const bool live = tok < (size_t)T_;
  const T* row = logits + (live ? tok : 0) * N;
  const bool dense = sp.score == BMOE_SCORE_SOFTMAX && !sp.renorm;
  const int id = live && q < k ? ids[tok * k + q] : -1;
  const bool pick = id >= 0 && id < N;
  const float lj = pick ? ld_logit(row + id) : -INFINITY;
  const float u = pick ? sp.scale * dgates[tok * k + q] : 0.f;
  float a[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) a[i] = 0.f;
  const float v = dense ? (lj == -INFINITY ? 0.f : u) : pick_grad<LPT>(lj, u, sp);
  const int sub = (threadIdx.x & 63) / LPT * LPT;
  for (int j = 0; j < k; ++j) {
    const int at = __shfl(id, sub + j, 64) - base;
    const float vj = __shfl(v, sub + j, 64);
#pragma unroll
    for (int i = 0; i < PER; ++i) a[i] += at == i ? vj : 0.f;
  }
  if (dense) {
    float l[PER], m = -INFINITY, total = 0.f;
    ld_row<PER, VEC>(row, base, N, -INFINITY, l);
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, l[i]);
    m = sub_max<LPT>(m);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      l[i] = l[i] == -INFINITY ? 0.f : exp_of(l[i] - m);
      total += l[i];
    }
    const float inv = 1.f / sub_sum<LPT>(total);
    const float d = sub_sum<LPT>(lj == -INFINITY ? 0.f : u * (exp_of(lj - m) * inv));
#pragma unroll
    for (int i = 0; i < PER; ++i) a[i] = l[i] == 0.f ? 0.f : l[i] * inv * (a[i] - d);
  }
  if (!live) return;
  float* out = dlogits + tok * N;
  if constexpr (VEC && PER % 4 == 0) {
#pragma unroll
    for (int i = 0; i < PER; i += 4)
      if (base + i < N)
        *reinterpret_cast<float4*>(out + base + i) = make_float4(a[i], a[i + 1], a[i + 2], a[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (base + i < N) out[base + i] = a[i];
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
    const float v = pick_grad<LPT>(l, u, sp);
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

// Lanes per token and experts per lane: 16 lanes (4 tokens per wave) up to 256
// experts and 16 picks or groups (they sit one per lane), else a whole wave
// per token.
#define BMOE_BY_SHAPE(CALL)                          \
  if (need <= 16 && N <= 64) { CALL(16, 4); }        \
  if (need <= 16 && N <= 256) { CALL(16, 16); }      \
  if (N <= 256) { CALL(64, 4); }                     \
  if (N <= 1024) { CALL(64, 16); }                   \
  CALL(64, 64)

template <bool VEC, typename T>
hipError_t route_t(const T* logits, const float* bias, int Tn, int N, int k, const RouteSpec& sp,
                   int32_t* ids, float* gates, hipStream_t s) {
  const int need = k > sp.groups ? k : sp.groups;
#define BMOE_CALL(LPT, PER)                                                                     \
  const unsigned blocks = ((unsigned)Tn + 256 / LPT - 1) / (256 / LPT);                         \
  return launch_kernel(route_kernel<LPT, PER, VEC, T>, dim3(blocks < 2048 ? blocks : 2048),     \
                       dim3(256), 0, s, KernelTiming{}, logits, bias, Tn, N, k, sp, ids, gates)
  BMOE_BY_SHAPE(BMOE_CALL);
#undef BMOE_CALL
}

template <bool VEC, typename T>
hipError_t route_bwd_t(const T* logits, const int32_t* ids, const float* dgates, int Tn, int N,
                       int k, const RouteSpec& sp, float* dlogits, hipStream_t s) {
  const int need = k;
#define BMOE_CALL(LPT, PER)                                                                      \
  return launch_kernel(route_bwd_kernel<LPT, PER, VEC, T>,                                       \
                       dim3(((unsigned)Tn + 256 / LPT - 1) / (256 / LPT)), dim3(256), 0, s,      \
                       KernelTiming{}, logits, ids, dgates, Tn, N, k, sp, dlogits)
  BMOE_BY_SHAPE(BMOE_CALL);
#undef BMOE_CALL
}

}  // namespace

hipError_t launch_route(bmoe_dtype dt, int T, int N, int k, const RouteSpec& sp,
                        const void* logits, const float* bias, int32_t* ids, float* gates,
                        hipStream_t s) {
  // whole vectors of a row: 16 bytes of logits (and 4 fp32 of the bias)
  if (dt == BMOE_BF16) {
    const uint16_t* l = static_cast<const uint16_t*>(logits);
    return N % 8 == 0 ? route_t<true>(l, bias, T, N, k, sp, ids, gates, s)
                      : route_t<false>(l, bias, T, N, k, sp, ids, gates, s);
  }
  const float* l = static_cast<const float*>(logits);
  return N % 4 == 0 ? route_t<true>(l, bias, T, N, k, sp, ids, gates, s)
                    : route_t<false>(l, bias, T, N, k, sp, ids, gates, s);
}

hipError_t launch_route_bwd(bmoe_dtype dt, int T, int N, int k, const RouteSpec& sp,
                            const void* logits, const int32_t* ids, const float* dgates,
                            float* dlogits, hipStream_t s) {
  if (dt == BMOE_BF16) {
    const uint16_t* l = static_cast<const uint16_t*>(logits);
    return N % 8 == 0 ? route_bwd_t<true>(l, ids, dgates, T, N, k, sp, dlogits, s)
                      : route_bwd_t<false>(l, ids, dgates, T, N, k, sp, dlogits, s);
  }
  const float* l = static_cast<const float*>(logits);
  return N % 4 == 0 ? route_bwd_t<true>(l, ids, dgates, T, N, k, sp, dlogits, s)
                    : route_bwd_t<false>(l, ids, dgates, T, N, k, sp, dlogits, s);
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
