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
// The same for 64-bit values, as two halves.
template <int LPT, typename F>
__device__ __forceinline__ uint64_t sub_reduce64(uint64_t v, F f) {
  auto both = [](uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; };
#define BMOE_STEP(O) \
  if constexpr (LPT > O) v = f(v, both(partner<O>((uint32_t)v), partner<O>((uint32_t)(v >> 32))));
  BMOE_STEP(1)
  BMOE_STEP(2)
  BMOE_STEP(4)
  BMOE_STEP(8)
#undef BMOE_STEP
  if constexpr (LPT >= 32) {
    const auto l = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
    const auto h = __builtin_amdgcn_permlane16_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
    v = f(both(l[0], h[0]), both(l[1], h[1]));
  }
  if constexpr (LPT >= 64) {
    const auto l = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
    const auto h = __builtin_amdgcn_permlane32_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
    v = f(both(l[0], h[0]), both(l[1], h[1]));
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ uint64_t sub_max(uint64_t v) {
  return sub_reduce64<LPT>(v, [](uint64_t x, uint64_t y) { return x > y ? x : y; });
}
template <int LPT>
__device__ __forceinline__ double sub_sum(double v) {
  return __longlong_as_double(sub_reduce64<LPT>(__double_as_longlong(v), [](uint64_t x, uint64_t y) {
    return (uint64_t)__double_as_longlong(__longlong_as_double(x) + __longlong_as_double(y));
  }));
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
__device__ __forceinline__ uint64_t key_of(double c) {
  const int64_t b = __double_as_longlong(c + 0.0);
  return c != c ? 1ull : (uint64_t)b ^ ((uint64_t)(b >> 63) | 0x8000000000000000ull);
}

// ---- scores ----------------------------------------------------------------------
// e^v on the exponential unit: off by (1.3 |v| + 2) 2^-24, relative (the
// product with log2 e, that constant, the unit's last place); a difference v
// brings |v| 2^-24 more.
__device__ __forceinline__ float exp_of(float v) { return __builtin_amdgcn_exp2f(v * kLog2e); }
__device__ __forceinline__ float inv_of(float v) { return __builtin_amdgcn_rcpf(v); }

// Sigmoid of l times e^(-shift), shift <= 0 and 0 unless every l of interest
// is negative: ratios of such scores keep their bits where all are tiny.
__device__ __forceinline__ float sigmoid_shifted(float l, float shift) {
  return l >= 0.f ? inv_of(1.f + exp_of(-l)) : exp_of(l - shift) * inv_of(1.f + exp_of(l));
}

template <typename T>
__device__ __forceinline__ float ld_logit(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_lo(*reinterpret_cast<const uint16_t*>(p));
  else return *p;
}

// This lane's values p[0 .. cnt), cnt <= PER, `fill` past them. VEC: p is
// aligned to, and cnt a multiple of, the vector's length.
template <int PER, bool VEC, typename T>
__device__ __forceinline__ void ld_row(const T* src, int cnt, float fill, float (&v)[PER]) {
  constexpr int W = 16 / sizeof(T) < PER ? 16 / sizeof(T) : PER;  // values per load
  if constexpr (VEC && W > 1) {
#pragma unroll
    for (int i = 0; i < PER; i += W) {
      float f[W];
      const T* p = src + i;
      const bool in = i < cnt;
      if (!in) {
#pragma unroll
        for (int u = 0; u < W; ++u) v[i + u] = fill;
        continue;
      }
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
      for (int u = 0; u < W; ++u) v[i + u] = f[u];
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      v[i] = fill;
      if (i < cnt) v[i] = ld_logit(src + i);
    }
  }
}

// ---- the choice ------------------------------------------------------------------
// A token's lanes and its experts: LPT lanes, PER consecutive experts per lane.
// With groups, a group takes lpg lanes (a power of two), so its lanes hold no
// other group's experts; the lowest lanes still hold the lowest ids.
struct LaneMap {
  int lpg;    // lanes per group; 0: the map does not fit
  int lpg64;  // the same where a wave takes one token of LPT PER experts
  int shift;  // log2 lpg
  int size;   // experts per group
  bool fits() const { return lpg && lpg64; }
};
inline int lanes_per_group(int lanes, int per, int N, int groups) {
  const int size = N / groups;
  int lpg = 1;
  while (lpg * per < size && lpg < lanes) lpg *= 2;
  if (groups == 1) lpg = lanes;
  return lpg * per < size || groups * lpg > lanes ? 0 : lpg;
}
template <int LPT, int PER>
LaneMap lane_map(int N, int groups) {
  const int lpg = lanes_per_group(LPT, PER, N, groups);
  int shift = 0;
  while (1 << shift < lpg) ++shift;
  return {lpg, lanes_per_group(64, LPT * PER / 64, N, groups), shift, N / groups};
}

// Group scores from the lanes' two largest choices: (a, a2) over `lpg` lanes.
template <int LPT>
__device__ __forceinline__ void top2_lanes(float& a, float& a2, int lpg) {
  auto merge = [&](uint32_t ob, uint32_t ob2) {
    const float o = __uint_as_float(ob), o2 = __uint_as_float(ob2);
    a2 = fmaxf(fminf(a, o), fmaxf(a2, o2));
    a = fmaxf(a, o);
  };
  if (lpg > 1) merge(partner<1>(__float_as_uint(a)), partner<1>(__float_as_uint(a2)));
  if (lpg > 2) merge(partner<2>(__float_as_uint(a)), partner<2>(__float_as_uint(a2)));
  if (lpg > 4) merge(partner<4>(__float_as_uint(a)), partner<4>(__float_as_uint(a2)));
  if (lpg > 8) merge(partner<8>(__float_as_uint(a)), partner<8>(__float_as_uint(a2)));
  if constexpr (LPT >= 32) {
    if (lpg > 16) merge(__shfl_xor(__float_as_uint(a), 16, 64), __shfl_xor(__float_as_uint(a2), 16, 64));
    if (lpg > 32) merge(__shfl_xor(__float_as_uint(a), 32, 64), __shfl_xor(__float_as_uint(a2), 32, 64));
  }
}

// The picks of one token in 64 bits, by a whole wave, from row; m: the row's
// largest logit. LANES: `lpg` lanes hold a group each, else a lane's experts
// may be of several. Returns pick j's id in lane j. Rare, so its code is seldom
// in the instruction cache and fetching that is what one costs: it is kept
// short (the exponential and the quotient once each, in loops that turn the
// lane's values around) and on DPP and scalar reads of lanes.
template <int PER, bool LANES, typename T>
__device__ int choose_exact(const T* row, const float* bias, int N, int k, const RouteSpec& sp,
                            int lpg, float m) {
  const int q = threadIdx.x & 63;
  const bool softmax = sp.score == BMOE_SCORE_SOFTMAX;
  const int size = N / sp.groups;
  const int mine_g = LANES ? q / lpg : 0, in_group = LANES ? q % lpg * PER : q * PER;
  const int base = LANES ? mine_g * size + in_group : in_group;
  const int cnt =
      LANES ? (mine_g < sp.groups ? min(PER, size - in_group) : 0) : min(PER, N - in_group);
  float l[PER];
  double c[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float v = ld_logit(row + min(base + i, N - 1));
    l[i] = i < cnt ? v : -INFINITY;
    c[i] = l[i];
  }
  if (bias || (sp.groups > 1 && sp.group_score == BMOE_GROUP_TOP2)) {
    // f(l, c, slot) for each slot in turn, its result the slot's new c
    auto each = [&](auto f) {
#pragma unroll 1
      for (int i = 0; i < PER; ++i) {
        const float l0 = l[0];
        const double c0 = f(l0, c[0], i);
#pragma unroll
        for (int u = 0; u + 1 < PER; ++u) {
          l[u] = l[u + 1];
          c[u] = c[u + 1];
        }
        l[PER - 1] = l0;
        c[PER - 1] = c0;
      }
    };
    double total = 0.0;
    each([&](float v, double, int) {
      const double e = exp(softmax ? (double)v - m : -(double)v);
      total += v == -INFINITY ? 0.0 : e;
      return e;
    });
    total = softmax ? sub_sum<64>(total) : 1.0;
    each([&](float v, double e, int i) {
      const double s = (softmax ? e : 1.0) / (softmax ? total : 1.0 + e);
      return v == -INFINITY ? -INFINITY : s + (bias ? (double)bias[min(base + i, N - 1)] : 0.0);
    });
  }
  uint64_t keep = ~0ull;  // bit g: group g is kept
  if (sp.groups > 1) {
    double mine = -INFINITY;  // lane g * lpg (LANES) or g: the score of group g
    // (no branches: those were compiled to a pair of values in scratch memory)
    auto top2 = [&](double& a, double& a2, double v) {
      v = v == v ? v : -INFINITY;
      a2 = fmax(a2, fmin(a, v));
      a = fmax(a, v);
    };
    auto merge = [&](double& a, double& a2, int o) {
      const double oa = __shfl_xor(a, o, 64), ob = __shfl_xor(a2, o, 64);
      a2 = fmax(fmin(a, oa), fmax(a2, ob));
      a = fmax(a, oa);
    };
    const bool by_max = sp.group_score == BMOE_GROUP_MAX;
    if constexpr (LANES) {
      double a = -INFINITY, a2 = -INFINITY;
#pragma unroll
      for (int i = 0; i < PER; ++i) top2(a, a2, c[i]);
      for (int o = 1; o < lpg; o *= 2) merge(a, a2, o);
      mine = by_max || a2 == -INFINITY ? a : a + a2;
    } else {
      for (int g = 0; g < sp.groups; ++g) {
        double a = -INFINITY, a2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          top2(a, a2, base + i >= g * size && base + i < (g + 1) * size ? c[i] : -INFINITY);
        for (int o = 32; o >= 1; o /= 2) merge(a, a2, o);
        if (q == g) mine = by_max || a2 == -INFINITY ? a : a + a2;
      }
    }
    const int step = LANES ? lpg : 1, g = q / step;
    int rank = 0;
    for (int h = 0; h < sp.groups; ++h) {
      const uint64_t bits = __double_as_longlong(mine);
      const double v = __longlong_as_double(
          (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(bits >> 32), h * step) << 32 |
          (uint32_t)__builtin_amdgcn_readlane((int)bits, h * step));
      rank += v > mine || (v == mine && h < g);
    }
    const bool kept = g < sp.groups && rank < sp.keep;
    keep = __ballot(kept);
    if (LANES) keep = kept ? ~0ull : 0;
  }
  uint64_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const bool in = i < cnt && (sp.groups == 1 || LANES ? keep != 0 : keep >> ((base + i) / size) & 1u);
    // without a bias the experts' order is that of their logits
    const uint64_t x = key_of(bias ? c[i] : (double)l[i]);
    key[i] = in ? x : 0;
  }
  int id = 0;
  for (int j = 0; j < k; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = key[i] > best ? key[i] : best;
    best = sub_max<64>(best);
    uint32_t at = 0x7fffffff;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) at = key[i] == best ? (uint32_t)(base + i) : at;
    at = sub_min<64>(at);
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = at == (uint32_t)(base + i) ? 0 : key[i];
    if (q == j) id = (int)at;
  }
  return id;
}

// The picks: pick j's id in lane j. fp32 finds them and the one after them,
// 64 bits put those in order. `open` is set for a token that this does not
// decide: kept groups, or the last pick and the experts not looked at again,
// closer than the errors bounded below, no k finite choices, a seventh pick from
// one lane; choose_exact then decides it. Without a bias the
// choices are the logits themselves, and only sums of two scores have errors.
// l, b: this lane's logits and biases from expert `base` on (-inf and 0 past
// its last).
template <int LPT, int PER, typename T>
__device__ __forceinline__ int choose(const T* row, const float* bias, const float (&l)[PER],
                                      const float (&b)[PER], float bmax, int base, int k,
                                      const RouteSpec& sp, const LaneMap& map, float m, bool& open) {
  const int q = threadIdx.x % LPT, here = threadIdx.x & 63, sub = here / LPT * LPT;
  const bool softmax = sp.score == BMOE_SCORE_SOFTMAX;
  // A score s of a logit at distance x from m is off by s u (3 |x| + A) at
  // most: the difference, its product with log2 e and that constant, then the
  // exponential's, sum's (PER + 6 additions) and quotient's last places. The
  // sigmoid has x = |l| and none of the sum.
  const float kA = softmax ? PER + 26 : 8;
  float c[PER], smax = 1.f;
  const bool scored = bias || (sp.groups > 1 && sp.group_score == BMOE_GROUP_TOP2);
  if (!scored) {
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = l[i];
  } else if (softmax) {
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = exp_of(l[i] - m);  // (a row of -inf: NaN, left open below)
      total += c[i];
    }
    smax = 1.f / sub_sum<LPT>(total);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      c[i] = l[i] == -INFINITY ? -INFINITY : fmaf(c[i], smax, b[i]);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      c[i] = l[i] == -INFINITY ? -INFINITY : inv_of(1.f + exp_of(-l[i])) + b[i];
  }

  if (sp.groups > 1) {
    float a = -INFINITY, a2 = -INFINITY;  // the two largest
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      a2 = fmaxf(a2, fminf(a, c[i]));
      a = fmaxf(a, c[i]);
    }
    top2_lanes<LPT>(a, a2, map.lpg);
    const bool one = sp.group_score == BMOE_GROUP_MAX || a2 == -INFINITY;
    const float score = one ? a : a + a2;
    const int g = q >> map.shift;
    int rank = 0;
    for (int h = 0; h < sp.groups; ++h) {
      const float v = __shfl(score, sub + (h << map.shift), 64);
      rank += v > score || (v == score && h < g);
    }
    const bool real = g < sp.groups, kept = real && rank < sp.keep;
    if (scored) {
      const float slack = kU * (2.f * smax * (kA + 2.f) + 3.f * (fabsf(a) + (one ? 0.f : fabsf(a2))));
      // the lowest that a kept group, and the highest that another can be
      const float lowest = -sub_max<LPT>(kept ? slack - score : -INFINITY);
      const float highest = sub_max<LPT>(real && !kept ? score + slack : -INFINITY);
      open |= !(lowest > highest);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = !kept ? -INFINITY : bias ? c[i] : l[i];
    }
  }

  // Each lane sorts integer keys (the choice's bits in order, the last ones
  // replaced by the place in the lane, so that a comparison is a min and a max)
  // into its kDepth largest; a round looks at the lanes' heads only. Keys equal
  // above the replaced bits go by id.
  constexpr uint32_t kLow = PER - 1;
  constexpr int kDepth = PER < 6 ? PER : 6;
  uint32_t h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  auto order = [](uint32_t& x, uint32_t& y) {  // x >= y
    const uint32_t hi = x > y ? x : y;
    y = x > y ? y : x;
    x = hi;
  };
  auto four = [&](uint32_t* f, int i0) {  // the lane's choices i0 .. i0 + 3, sorted
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int32_t bits = __float_as_int(c[i0 + u]);
      f[u] = (((uint32_t)bits ^ ((uint32_t)(bits >> 31) | 0x80000000u)) & ~kLow) | (kLow - (i0 + u));
    }
    order(f[0], f[1]);
    order(f[2], f[3]);
    order(f[0], f[2]);
    order(f[1], f[3]);
    order(f[1], f[2]);
  };
  auto merge8 = [&](uint32_t (&f)[8]) {  // sorts a bitonic eight
#pragma unroll
    for (int u = 0; u < 4; ++u) order(f[u], f[u + 4]);
#pragma unroll
    for (int u = 0; u < 8; u += 4) {
      order(f[u], f[u + 2]);
      order(f[u + 1], f[u + 3]);
    }
#pragma unroll
    for (int u = 0; u < 8; u += 2) order(f[u], f[u + 1]);
  };
  if constexpr (PER == 4) {
    four(h, 0);
  } else {
#pragma unroll
    for (int i0 = 0; i0 < PER; i0 += 8) {
      uint32_t f[8], g[4];
      four(f, i0);
      four(g, i0 + 4);
#pragma unroll
      for (int u = 0; u < 4; ++u) f[4 + u] = g[3 - u];
      merge8(f);
      if (i0 == 0) {
#pragma unroll
        for (int u = 0; u < 8; ++u) h[u] = f[u];
      } else {  // the eight largest of two sorted eights, sorted
#pragma unroll
        for (int u = 0; u < 8; ++u) h[u] = h[u] > f[7 - u] ? h[u] : f[7 - u];
        merge8(h);
      }
    }
  }
  auto value_of = [](uint32_t k0) {
    return __uint_as_float(k0 & 0x80000000u ? k0 ^ 0x80000000u : ~k0);
  };
  // the largest that a lane's list does not hold
  const uint32_t spare = PER > kDepth ? h[kDepth] & ~kLow : 0;
  int id = 0;  // pick q's; in lane k (if there is one) the expert's after the picks
  uint32_t key = 0, beyond = 0;
  for (int j = 0; j <= k; ++j) {
    const uint32_t v = h[0] & ~kLow;
    const uint32_t best = sub_max<LPT>(v);
    const uint32_t mine = v == best ? (uint32_t)base + kLow - (h[0] & kLow) : 0x7fffffffu;
    const uint32_t first = sub_min<LPT>(mine);
    const bool out = mine == first;
    // (a bit select: written as a choice between two entries it is compiled
    // as an indexed read of h, eleven instructions each)
    const uint32_t gone = out ? ~0u : 0u;
#pragma unroll
    for (int u = 0; u + 1 < kDepth; ++u) h[u] = (h[u] & ~gone) | (h[u + 1] & gone);
    h[kDepth - 1] &= ~gone;
    if (q == j) {
      id = (int)first;
      key = best;
    }
    if (j == LPT) beyond = best;
  }
  // the largest of the experts that no lane has
  const uint32_t left = max(sub_max<LPT>(h[0] ? h[0] & ~kLow : spare), beyond);

  // The candidates in 64 bits, a lane each, and put in order: keys equal above
  // the replaced bits, or off by the errors of c, may have them wrong. The sum
  // behind a softmax's scores is off by kA u still.
  const bool pick = q < k, last = q == k - 1;
  const float v32 = value_of(key);
  const bool fine = q <= k && fabsf(v32) < INFINITY;
  open |= pick && !fine;
  const float lq = fine ? ld_logit(row + id) : 0.f;
  double s = 0.0, v = fine ? (double)lq : -INFINITY;
  if (bias) {
    const float bq = fine ? bias[id] : 0.f;
    const double e = exp(softmax ? (double)lq - m : -(double)lq);
    s = softmax ? e * (double)smax : 1.0 / (1.0 + e);
    v = fine ? s + (double)bq : -INFINITY;
  }
  const bool follows = pick && q + 1 < LPT;  // the next lane has a candidate
  auto wrong = [&] {
    const double vn = __shfl(v, (here + 1) & 63, 64);
    const int in = __shfl(id, (here + 1) & 63, 64);
    return follows && !(v > vn || (v == vn && id < in));
  };
  for (int pass = 0; pass <= k && __any(wrong()); ++pass) {  // odd-even transposition
    const int other = (q + pass) & 1 ? q - 1 : q + 1;
    const bool two = other >= 0 && max(q, other) <= k && other < LPT;
    const int from = two ? sub + other : here;
    const double vo = __shfl(v, from, 64), so = __shfl(s, from, 64);
    const int io = __shfl(id, from, 64);
    const bool before = v > vo || (v == vo && id < io);
    if (two && before != (other > q)) {
      v = vo;
      s = so;
      id = io;
    }
  }
  if (bias && softmax) {
    const double dv = v - __shfl(v, (here + 1) & 63, 64), ds = s - __shfl(s, (here + 1) & 63, 64);
    open |= follows && !(dv > fabs(ds) * (double)(kA * kU) + 1e-15) && !(dv == 0.0 && ds == 0.0);
  }
  // None left has a choice above `up`, so none a score above S, and none an
  // error above E (s x <= S (1 + ln(smax / S)) for a score s <= S).
  const float up = value_of(left | kLow);
  double bound = up, low = v;
  if (bias) {
    const float S = fminf(smax, fmaxf(up + bmax, 1e-30f));
    bound += kU * (S * (3.f + 2.1f * __builtin_amdgcn_logf(smax / S) + kA) + 3.f * fabsf(up));
    if (softmax) low -= s * (double)(kA * kU);
  }
  open |= last && up > -INFINITY && !(low > bound);
  return id;
}

// Gate of pick q < k of a token (lj: its logit, -inf where there is none).
// total: the row's sum of e^(l - m), for softmax gates without renorm.
template <int LPT>
__device__ __forceinline__ float gate_of(float lj, const RouteSpec& sp, float m, float total) {
  const bool softmax = sp.score == BMOE_SCORE_SOFTMAX;
  float g;
  if (sp.renorm) {
    const float mc = sub_max<LPT>(lj);
    const float shift = softmax ? mc : fminf(mc, 0.f);
    const float u = lj == -INFINITY ? 0.f
                    : softmax ? exp_of(lj - shift) : sigmoid_shifted(lj, shift);
    const float sum = sub_sum<LPT>(u);
    g = sum > 0.f ? u / sum : 0.f;
  } else if (softmax) {
    g = lj == -INFINITY ? 0.f : exp_of(lj - m) / total;
  } else {
    g = lj == -INFINITY ? 0.f : inv_of(1.f + exp_of(-lj));
  }
  return sp.scale * g;
}

// ---- routing ----------------------------------------------------------------------
// Tokens left open are decided one at a time by the whole wave. In a launch of
// their own after this one they cost more (at 32768 tokens of 256 experts 24 us
// for that launch). Of ordinary fp32 logits 1 token in 10^4 is open. Without a
// bias every token is whose last pick has a value equal to another expert's
// past the candidates: of unit-variance bf16 logits 0.6% at 256 experts and top
// 8, 4% at 1024 and 16, 31% at 4096 and 64, and every constant row.
// Bound by the VALU: 32768 tokens, 256 experts in 8 groups, top 8, with a bias
// 20.7 us, about 3 us of it the wait for the last open token; without groups
// 14.7 us, without bias too 11.5 us (bf16 13.9 us; constant rows 49 us). 512
// experts in 8 groups with a bias 39 us. 8192 tokens of 4096 experts, top 64:
// 243 us, bf16 1.02 ms; 64 experts in a lane take 256 VGPRs (one wave per SIMD)
// and spill scalar registers.
template <int LPT, int PER, bool VEC, typename T>
__global__ __launch_bounds__(256) void route_kernel(const T* logits, const float* bias, int T_,
                                                    int N, int k, RouteSpec sp, LaneMap map,
                                                    int32_t* ids, float* gates) {
  constexpr int kTok = 256 / LPT;  // tokens per workgroup
  const int q = threadIdx.x % LPT;
  const bool softmax = sp.score == BMOE_SCORE_SOFTMAX;
  const int in_group = (q & (map.lpg - 1)) * PER;  // this lane's first expert within its group
  const int base = (q >> map.shift) * map.size + in_group;
  const int cnt = q >> map.shift < sp.groups ? max(0, min(PER, map.size - in_group)) : 0;
  float b[PER], bmax = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) b[i] = 0.f;
  if (bias) {
    ld_row<PER, VEC>(bias + base, cnt, 0.f, b);
#pragma unroll
    for (int i = 0; i < PER; ++i) bmax = fmaxf(bmax, fabsf(b[i]));
    bmax = sub_max<LPT>(bmax);
  }
  // (No loop over tokens: in one the compiler keeps the conditions on spec and
  // shape as masks, more than there are scalar registers; their spills made
  // the 32768 x 256 case 26.0 us instead of 23.4.)
  const size_t t0 = (size_t)grid_block() * kTok;
  if (t0 >= (size_t)T_) return;
  const size_t tok = t0 + threadIdx.x / LPT;
  const bool live = tok < (size_t)T_;
  const T* row = logits + (live ? tok : 0) * N;
  float l[PER];
  ld_row<PER, VEC>(row + base, cnt, -INFINITY, l);
  bool bad = false;
  float m = -INFINITY, total = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    bad |= l[i] != l[i];
    m = fmaxf(m, l[i]);
  }
  m = sub_max<LPT>(m);
  if (softmax && !sp.renorm) {
#pragma unroll
    for (int i = 0; i < PER; ++i) total += l[i] == -INFINITY ? 0.f : exp_of(l[i] - m);
    total = sub_sum<LPT>(total);
  }
  const bool has_nan = own_bits<LPT>(__ballot(bad)) != 0;

  bool open = has_nan || m == INFINITY || !(bmax < INFINITY);
  int id = choose<LPT, PER>(row, bias, l, b, bmax, base, k, sp, map, m, open);
  uint64_t todo = __ballot(open && live);
  const bool pick = live && q < k;  // (a lane without a token may hold no id)
  while (todo) {
    const int sub = (int)__builtin_ctzll(todo) / LPT * LPT;
    todo &= ~(LPT == 64 ? ~0ull : ((1ull << (LPT & 63)) - 1) << sub);
    const size_t t = t0 + ((threadIdx.x & ~63) + sub) / LPT;
    const int x = choose_exact<LPT * PER / 64, true>(logits + t * N, bias, N, k, sp, map.lpg64,
                                               __shfl(m, sub, 64));
    const int y = __shfl(x, q, 64);
    if ((threadIdx.x & 63) / LPT * LPT == sub) id = y;
  }
  const bool nan = has_nan || (softmax && m == INFINITY);
  const float g = gate_of<LPT>(pick ? ld_logit(row + id) : -INFINITY, sp, m, total);
  if (pick) {
    ids[tok * k + q] = id;
    gates[tok * k + q] = nan ? NAN : g;
  }
}

// Every token in 64 bits, a wave each: groups whose lanes route_kernel does not
// have (more than 32 groups of more than 64 experts).
template <typename T>
__global__ __launch_bounds__(256) void route_exact_kernel(const T* logits, const float* bias,
                                                          int T_, int N, int k, RouteSpec sp,
                                                          int32_t* ids, float* gates) {
  constexpr int PER = 64;
  const int q = threadIdx.x & 63;
  const bool softmax = sp.score == BMOE_SCORE_SOFTMAX;
  const size_t t = (size_t)grid_block() * 4 + (threadIdx.x >> 6);
  if (t >= (size_t)T_) return;  // whole wave
  const T* row = logits + t * N;
  float m = -INFINITY, total = 0.f;
  bool nan = false;
  for (int e = q; e < N; e += 64) {
    const float l = ld_logit(row + e);
    nan |= l != l;
    m = fmaxf(m, l);
  }
  m = sub_max<64>(m);
  nan = __any(nan) || (softmax && m == INFINITY);
  if (softmax && !sp.renorm) {
    for (int e = q; e < N; e += 64) {
      const float l = ld_logit(row + e);
      total += l == -INFINITY ? 0.f : exp_of(l - m);
    }
    total = sub_sum<64>(total);
  }
  const int id = choose_exact<PER, false>(row, bias, N, k, sp, 0, m);
  const float g = gate_of<64>(q < k ? ld_logit(row + id) : -INFINITY, sp, m, total);
  if (q < k) {
    ids[t * k + q] = id;
    gates[t * k + q] = nan ? NAN : g;
  }
}

// ---- gradient of the gates --------------------------------------------------------
// With u_j the gates' gradient times scale:
//   renormalised:  dl_j = p_j (u_j - sum_i u_i p_i) [ (1 - s_j) ],  p = s / sum
//   sigmoid:       dl_j = u_j s_j (1 - s_j)
//   softmax:       dl_e = s_e (sum over j with id_j = e of u_j  -  sum_i u_i s_i)
// An id outside [0, N) contributes nothing; equal ids add up in their order. Nor
// does a masked pick, whose gate is constant: what arrives as its gradient may
// be NaN or infinite, so it becomes 0 before any product.

// What pick (l, u) of its LPT lanes' token adds to its logit's gradient, for
// the specs under which only the picks move. l = -inf: no pick, or masked (u 0).
template <int LPT>
__device__ __forceinline__ float pick_grad(float l, float u, const RouteSpec& sp) {
  const bool softmax = sp.score == BMOE_SCORE_SOFTMAX;
  float v;
  if (sp.renorm) {
    const float mc = sub_max<LPT>(l);
    const float shift = softmax ? mc : fminf(mc, 0.f);
    const float w = l == -INFINITY ? 0.f : softmax ? exp_of(l - shift) : sigmoid_shifted(l, shift);
    const float sum = sub_sum<LPT>(w);
    const float p = sum == 0.f ? 0.f : w / sum;  // (a NaN stays one)
    v = p * (u - sub_sum<LPT>(u * p));
    if (!softmax) v *= inv_of(1.f + exp_of(l));
  } else {
    v = u * inv_of(1.f + exp_of(-l)) * inv_of(1.f + exp_of(l));
  }
  return l == -INFINITY ? 0.f : v;
}

// dl is written as fp32 [T][N], or (PARTS) as three bf16 parts whose sum is
// dl to fp32's last bits, in the order of MFMA operands (router_parts_*).
template <int LPT, int PER, bool VEC, bool PARTS, typename T>
__global__ __launch_bounds__(256) void route_bwd_kernel(const T* logits, const int32_t* ids,
                                                        const float* dgates, int T_, int N, int k,
                                                        RouteSpec sp, float* dlogits,
                                                        uint16_t* parts) {
  // Lanes of a token side by side in memory: slot i of lane q is expert
  // q QUAD + off(i). (No order among lanes matters here, as it does for the
  // choice. PER consecutive experts per lane, 16-byte pieces 64 bytes apart,
  // took 18.0 us instead of 11.4 at T = 32768, N = 256, dense: 67 MB.)
  constexpr int QUAD = VEC || PARTS ? 4 : 1;
  static_assert(PER % 4 == 0, "whole quads");
  auto off = [](int i) { return i / QUAD * (QUAD * LPT) + i % QUAD; };
  const int q = threadIdx.x % LPT, base = q * QUAD;
  const size_t tok = (size_t)grid_block() * (256 / LPT) + threadIdx.x / LPT;
  const bool live = tok < (size_t)T_;
  const T* row = logits + (live ? tok : 0) * N;
  const bool dense = sp.score == BMOE_SCORE_SOFTMAX && !sp.renorm;
  const int id = live && q < k ? ids[tok * k + q] : -1;
  const bool pick = id >= 0 && id < N;
  const float lj = pick ? ld_logit(row + id) : -INFINITY;
  const float dg = pick ? dgates[tok * k + q] : 0.f;
  const float u = lj == -INFINITY ? 0.f : sp.scale * dg;
  float a[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) a[i] = 0.f;
  const float v = dense ? u : pick_grad<LPT>(lj, u, sp);
  const int sub = (threadIdx.x & 63) / LPT * LPT;
  for (int j = 0; j < k; ++j) {
    const int at = __shfl(id, sub + j, 64) - base;
    const float vj = __shfl(v, sub + j, 64);
#pragma unroll
    for (int i = 0; i < PER; ++i) a[i] += at == off(i) ? vj : 0.f;
  }
  if (dense) {
    float l[PER], m = -INFINITY, total = 0.f;
#pragma unroll
    for (int i = 0; i < PER; i += QUAD) {
      const int e = base + off(i);
      float f[QUAD];
      ld_row<QUAD, VEC>(row + min(e, N), max(0, min(QUAD, N - e)), -INFINITY, f);
#pragma unroll
      for (int u = 0; u < QUAD; ++u) l[i + u] = f[u];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, l[i]);
    m = sub_max<LPT>(m);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      l[i] = l[i] == -INFINITY ? 0.f : exp_of(l[i] - m);
      total += l[i];
    }
    total = sub_sum<LPT>(total);
    const float inv = 1.f / total;
    const float none = total != total ? total : 0.f;  // a NaN or +inf logit: NaN, not 0
    const float d = sub_sum<LPT>(lj == -INFINITY ? 0.f : u * (exp_of(lj - m) * inv));
#pragma unroll
    for (int i = 0; i < PER; ++i) a[i] = l[i] == 0.f ? none : l[i] * inv * (a[i] - d);
    // a row without a pick is 0 whatever it holds (a branch, rarely taken: in the
    // line above the condition cost 0.5 of 11.5 us)
    if (own_bits<LPT>(__ballot(lj != -INFINITY)) == 0) {
#pragma unroll
      for (int i = 0; i < PER; ++i) a[i] = 0.f;
    }
  }
  if (!live) return;
  if constexpr (PARTS) {
    const int np = router_parts_experts(N);
    uint16_t* out = parts + tok / 32 * (96 * (size_t)np) + tok % 32 * 8;
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      const int e = base + off(i);
      if (e >= np) continue;
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = e + u < N ? a[i + u] : 0.f;
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        uint2 w;
        w.x = pack_bf16x2(v[0], v[1]);
        w.y = pack_bf16x2(v[2], v[3]);
        *reinterpret_cast<uint2*>(out + (e / 16 * 3 + p) * 512 + e % 16 / 8 * 256 + e % 8) = w;
        v[0] -= bf16_lo(w.x);
        v[1] -= bf16_hi(w.x);
        v[2] -= bf16_lo(w.y);
        v[3] -= bf16_hi(w.y);
      }
    }
    return;
  }
  float* out = dlogits + tok * N;
#pragma unroll
  for (int i = 0; i < PER; i += QUAD) {
    const int e = base + off(i);
    if (e >= N) continue;
    if constexpr (QUAD == 4)
      *reinterpret_cast<float4*>(out + e) = make_float4(a[i], a[i + 1], a[i + 2], a[i + 3]);
    else
      out[e] = a[i];
  }
}

// Token i of `nt` from t0 on: its picks' (id, coefficient) pairs, by THREADS
// threads.
template <int LPT, int THREADS>
__device__ __forceinline__ void make_pairs(const float* logits, const int32_t* ids,
                                           const float* dgates, size_t t0, int nt, int N, int k,
                                           const RouteSpec& sp, int2* pairs) {
  const int q = threadIdx.x % LPT;
  for (int i = threadIdx.x / LPT; i - (int)threadIdx.x / LPT < nt; i += THREADS / LPT) {
    const size_t tok = t0 + i;
    const bool mine = i < nt && q < k;
    const int id = mine ? ids[tok * k + q] : -1;
    const bool pick = id >= 0 && id < N;
    const float l = pick ? logits[tok * N + id] : -INFINITY;
    const float dg = pick ? dgates[tok * k + q] : 0.f;
    const float u = l == -INFINITY ? 0.f : sp.scale * dg;
    const float v = pick_grad<LPT>(l, u, sp);
    if (mine) pairs[tok * k + q] = make_int2(pick ? id : 0, __float_as_int(pick ? v : 0.f));
  }
}

template <int LPT>
__global__ __launch_bounds__(256) void route_pairs_kernel(const float* logits, const int32_t* ids,
                                                          const float* dgates, int T_, int N,
                                                          int k, RouteSpec sp, int2* pairs) {
  const size_t t0 = (size_t)grid_block() * (256 / LPT);
  if (t0 >= (size_t)T_) return;
  const int nt = (int)min((size_t)(256 / LPT), (size_t)T_ - t0);
  make_pairs<LPT, 256>(logits, ids, dgates, t0, nt, N, k, sp, pairs);
}

// The pairs of one range of tokens listed by expert (stable): one workgroup
// per range. Each wave owns a contiguous share of the range's picks; equal
// experts within 64 picks are ranked by ballots over the id's bits. MAKE: the
// workgroup makes its range's pairs first (short ranges, one launch less).
template <int LPT, int WAVES, bool MAKE>
__global__ __launch_bounds__(WAVES * 64) void route_lists_kernel(
    const float* logits, const int32_t* ids, const float* dgates, int T_, int N, int k, int nbits,
    RouteSpec sp, RouterPairs rp) {
  extern __shared__ int cur[];  // [WAVES][N]: counts, then cursors
  __shared__ int wsum[WAVES];
  constexpr int kThreads = WAVES * 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const size_t t0 = (size_t)blockIdx.x * rp.tokens;
  const int nt = (int)min((size_t)rp.tokens, (size_t)T_ - t0);
  for (int i = tid; i < WAVES * N; i += kThreads) cur[i] = 0;
  if constexpr (MAKE)
    make_pairs<LPT, kThreads>(logits, ids, dgates, t0, nt, N, k, sp, rp.pairs);
  __syncthreads();

  const int M = nt * k;
  const int2* pairs = rp.pairs + t0 * k;
  const int share = ((M + WAVES - 1) / WAVES + 63) / 64 * 64;
  const int wb = min(M, wave * share), we = min(M, wb + share);
  int* mycur = cur + wave * N;
#pragma unroll 8
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
// Histograms in LDS (integers, so no order matters), then bias[e] += rate *
// sign(mean - load[e]) with the comparison in integers (sum of the loads
// against N * load). Few ids: one workgroup does it all. More: 64 workgroups
// count a share each and write their histograms; a second launch
// adds them (no counters to clear, nothing left between calls). Bound by
// latency: 2^18 ids are 1 MB. Measured at 262144 ids, 256 experts: one
// workgroup 42 us, shares 12 us (two launches).
constexpr int kBalanceShares = 64, kBalanceOne = 16384;  // ids that one workgroup takes

__device__ __forceinline__ void count_ids(const int32_t* ids, long long r0, long long r1, int N,
                                          int* hist) {
  // r0 is a multiple of 4: 16-byte loads, eight in flight per thread
  const int4* p = reinterpret_cast<const int4*>(ids);
  const long long v1 = r1 / 4;
  auto add = [&](int e) {
    if (e >= 0 && e < N) atomicAdd(&hist[e], 1);
  };
  for (long long v0 = r0 / 4; v0 < v1; v0 += 8 * 1024) {
    int4 x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const long long v = v0 + u * 1024 + threadIdx.x;
      x[u] = v < v1 ? p[v] : make_int4(-1, -1, -1, -1);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      add(x[u].x);
      add(x[u].y);
      add(x[u].z);
      add(x[u].w);
    }
  }
  for (long long r = v1 * 4 + threadIdx.x; r < r1; r += 1024) add(ids[r]);
}

// hist: the experts' loads. Writes load and moves the bias.
__device__ __forceinline__ void finish_loads(const int* hist, int N, float rate, int32_t* load,
                                             float* bias, long long* sum) {
  long long part = 0;
  for (int e = threadIdx.x; e < N; e += 1024) part += hist[e];
  if (part) atomicAdd((unsigned long long*)sum, (unsigned long long)part);
  __syncthreads();
  for (int e = threadIdx.x; e < N; e += 1024) {
    load[e] = hist[e];
    if (bias) {
      const long long diff = *sum - (long long)N * hist[e];
      bias[e] += diff > 0 ? rate : diff < 0 ? -rate : 0.f;
    }
  }
}

__global__ __launch_bounds__(1024) void balance_kernel(const int32_t* ids, long long M, int N,
                                                       int accumulate, float rate, int32_t* load,
                                                       float* bias) {
  __shared__ int hist[kMaxExperts];
  __shared__ long long sum;
  if (threadIdx.x == 0) sum = 0;
  for (int e = threadIdx.x; e < N; e += 1024) hist[e] = accumulate ? load[e] : 0;
  __syncthreads();
  count_ids(ids, 0, M, N, hist);
  __syncthreads();
  finish_loads(hist, N, rate, load, bias, &sum);
}

// part [kBalanceShares][N]: each workgroup's counts of its share.
__global__ __launch_bounds__(1024) void balance_count_kernel(const int32_t* ids, long long M,
                                                             int N, long long share, int* part) {
  __shared__ int hist[kMaxExperts];
  for (int e = threadIdx.x; e < N; e += 1024) hist[e] = 0;
  __syncthreads();
  const long long r0 = blockIdx.x * share;
  if (r0 < M) count_ids(ids, r0, r0 + share < M ? r0 + share : M, N, hist);
  __syncthreads();
  for (int e = threadIdx.x; e < N; e += 1024) part[(size_t)blockIdx.x * N + e] = hist[e];
}

__global__ __launch_bounds__(1024) void balance_join_kernel(const int* part, int N, int accumulate,
                                                            float rate, int32_t* load,
                                                            float* bias) {
  __shared__ int hist[kMaxExperts];
  __shared__ long long sum;
  if (threadIdx.x == 0) sum = 0;
  for (int e = threadIdx.x; e < N; e += 1024) hist[e] = accumulate ? load[e] : 0;
  __syncthreads();
  // a thread adds several shares of one expert; N threads side by side
  const int lanes = N < 1024 ? N : 1024, rows = 1024 / lanes;
  const int row = threadIdx.x / lanes;
  if (row < rows)
    for (int e = threadIdx.x % lanes; e < N; e += lanes) {
      int c = 0;
#pragma unroll 8
      for (int w = row; w < kBalanceShares; w += rows) c += part[(size_t)w * N + e];
      if (c) atomicAdd(&hist[e], c);
    }
  __syncthreads();
  finish_loads(hist, N, rate, load, bias, &sum);
}

// Workgroups of 256 threads for T tokens of `lanes` lanes each.
inline dim3 token_grid(int T, int lanes) {
  const unsigned per = 256 / lanes;
  return grid_rows(((unsigned)T + per - 1) / per);
}

// Lanes per token and experts per lane: 16 lanes (4 tokens per wave) up to 256
// experts and 16 picks, 32 up to 512 and 32, else a whole wave per token.
template <bool VEC, typename T>
hipError_t route_t(const T* logits, const float* bias, int Tn, int N, int k, const RouteSpec& sp,
                   int32_t* ids, float* gates, hipStream_t s) {
  const bool few = Tn <= 1024;  // a wave per token still leaves SIMDs without one
  LaneMap map;
#define BMOE_CALL(LPT, PER, WHEN)                                                               \
  if ((WHEN) && N <= LPT * PER && k <= LPT && (map = lane_map<LPT, PER>(N, sp.groups)).fits()) { \
    return launch_kernel(route_kernel<LPT, PER, VEC, T>, token_grid(Tn, LPT), dim3(256), 0, s,  \
                         KernelTiming{}, logits, bias, Tn, N, k, sp, map, ids, gates);          \
  }
  BMOE_CALL(16, 4, true)
  BMOE_CALL(16, 16, !few)
  BMOE_CALL(64, 4, true)
  BMOE_CALL(16, 16, true)
  BMOE_CALL(32, 16, true)
  BMOE_CALL(64, 16, true)
  BMOE_CALL(64, 64, true)
#undef BMOE_CALL
  return launch_kernel(route_exact_kernel<T>, token_grid(Tn, 64), dim3(256), 0, s,
                       KernelTiming{}, logits, bias, Tn, N, k, sp, ids, gates);
}

#define BMOE_BY_SHAPE(CALL)                    \
  if (k <= 16 && N <= 64) { CALL(16, 4); }     \
  if (k <= 16 && N <= 256) { CALL(16, 16); }   \
  if (N <= 256) { CALL(64, 4); }               \
  if (N <= 1024) { CALL(64, 16); }             \
  CALL(64, 64)

template <bool VEC, bool PARTS, typename T>
hipError_t route_bwd_t(const T* logits, const int32_t* ids, const float* dgates, int Tn, int N,
                       int k, const RouteSpec& sp, float* dlogits, uint16_t* parts,
                       hipStream_t s) {
#define BMOE_CALL(LPT, PER)                                                                      \
  return launch_kernel(route_bwd_kernel<LPT, PER, VEC, PARTS, T>,                                \
                       token_grid(Tn, LPT), dim3(256), 0, s, KernelTiming{}, logits, ids,        \
                       dgates, Tn, N, k, sp, dlogits, parts)
  BMOE_BY_SHAPE(BMOE_CALL);
#undef BMOE_CALL
}

}  // namespace

hipError_t launch_route(bmoe_dtype dt, int T, int N, int k, const RouteSpec& sp,
                        const void* logits, const float* bias, int32_t* ids, float* gates,
                        hipStream_t s) {
  // whole vectors (16 bytes) of a row and of each group in it
  const int size = N / sp.groups;
  if (dt == BMOE_BF16) {
    const uint16_t* l = static_cast<const uint16_t*>(logits);
    return size % 8 == 0 ? route_t<true>(l, bias, T, N, k, sp, ids, gates, s)
                         : route_t<false>(l, bias, T, N, k, sp, ids, gates, s);
  }
  const float* l = static_cast<const float*>(logits);
  return size % 4 == 0 ? route_t<true>(l, bias, T, N, k, sp, ids, gates, s)
                       : route_t<false>(l, bias, T, N, k, sp, ids, gates, s);
}

hipError_t launch_route_bwd(bmoe_dtype dt, int T, int N, int k, const RouteSpec& sp,
                            const void* logits, const int32_t* ids, const float* dgates,
                            float* dlogits, hipStream_t s) {
  if (dt == BMOE_BF16) {
    const uint16_t* l = static_cast<const uint16_t*>(logits);
    return N % 8 == 0 ? route_bwd_t<true, false>(l, ids, dgates, T, N, k, sp, dlogits, nullptr, s)
                      : route_bwd_t<false, false>(l, ids, dgates, T, N, k, sp, dlogits, nullptr, s);
  }
  const float* l = static_cast<const float*>(logits);
  return N % 4 == 0 ? route_bwd_t<true, false>(l, ids, dgates, T, N, k, sp, dlogits, nullptr, s)
                    : route_bwd_t<false, false>(l, ids, dgates, T, N, k, sp, dlogits, nullptr, s);
}

hipError_t launch_route_bwd_parts(int T, int N, int k, const RouteSpec& sp, const float* logits,
                                  const int32_t* ids, const float* dgates, uint16_t* parts,
                                  hipStream_t s) {
  return N % 4 == 0 ? route_bwd_t<true, true>(logits, ids, dgates, T, N, k, sp, nullptr, parts, s)
                    : route_bwd_t<false, true>(logits, ids, dgates, T, N, k, sp, nullptr, parts, s);
}

hipError_t launch_route_pairs(int T, int N, int k, const RouteSpec& sp, const float* logits,
                              const int32_t* ids, const float* dgates, const RouterPairs& rp,
                              hipStream_t s) {
  int nbits = 0;
  while ((1 << nbits) < N) ++nbits;
  // Ranges of up to 2048 lanes' worth of picks make their pairs themselves;
  // longer ones wait too long for their gathers, so a launch over all CUs makes
  // them. 16 waves for those while their cursors take 32 KB at most, else 4
  // (64 KB at 4096 experts).
  const int lpt = k <= 2 ? 2 : k <= 4 ? 4 : k <= 8 ? 8 : k <= 16 ? 16 : 64;
  const bool make = (long long)rp.tokens * lpt <= 2048;
#define BMOE_LISTS(LPT, WAVES, MAKE)                                                            \
  launch_kernel(route_lists_kernel<LPT, WAVES, MAKE>, dim3(rp.ranges), dim3(WAVES * 64),        \
                WAVES * N * 4, s, KernelTiming{}, logits, ids, dgates, T, N, k, nbits, sp, rp)
#define BMOE_PAIRS(LPT)                                                                         \
  do {                                                                                          \
    if (make) return BMOE_LISTS(LPT, 4, true);                                                  \
    const hipError_t e =                                                                        \
        launch_kernel(route_pairs_kernel<LPT>, token_grid(T, LPT), dim3(256), 0, s,             \
                      KernelTiming{}, logits, ids, dgates, T, N, k, sp, rp.pairs);              \
    if (e != hipSuccess) return e;                                                              \
    return N <= 512 ? BMOE_LISTS(2, 16, false) : BMOE_LISTS(2, 4, false);                       \
  } while (0)
  if (k <= 2) BMOE_PAIRS(2);
  if (k <= 4) BMOE_PAIRS(4);
  if (k <= 8) BMOE_PAIRS(8);
  if (k <= 16) BMOE_PAIRS(16);
  BMOE_PAIRS(64);
#undef BMOE_LISTS
#undef BMOE_PAIRS
}

size_t balance_part_bytes(long long M, int N) {
  return M > kBalanceOne ? (size_t)kBalanceShares * N * sizeof(int) : 0;
}

hipError_t launch_balance(long long M, int N, const int32_t* ids, int accumulate, float rate,
                          int32_t* load, float* bias, int* part, hipStream_t s) {
  if (M <= kBalanceOne)
    return launch_kernel(balance_kernel, dim3(1), dim3(1024), 0, s, KernelTiming{}, ids, M, N,
                         accumulate, rate, load, bias);
  const long long share = ((M + kBalanceShares - 1) / kBalanceShares + 3) / 4 * 4;
  const hipError_t e = launch_kernel(balance_count_kernel, dim3(kBalanceShares), dim3(1024), 0, s,
                                     KernelTiming{}, ids, M, N, share, part);
  if (e != hipSuccess) return e;
  return launch_kernel(balance_join_kernel, dim3(1), dim3(1024), 0, s, KernelTiming{},
                       static_cast<const int*>(part), N, accumulate, rate, load, bias);
}

}  // namespace bmoe
