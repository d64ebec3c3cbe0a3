// Global norm of a list of gradients, and the gradients scaled to a largest
// norm:
//   norm = sqrt(sum over all tensors and entries of g^2)
//   out  = g * (max_norm / norm  if max_norm < norm < infinity, else 1)
// Squares are summed in 64 bits (no overflow, and a sum over 10^9 entries
// keeps its bits) in an order that the sizes alone fix: thread, wave,
// workgroup, then the workgroups' partial sums in their order.
#include <cmath>

#include "common.h"
#include "kernels.h"

namespace bmoe {
namespace {

constexpr int kThreads = 256;

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

__device__ __forceinline__ float ld_grad(const GradEntry& t, size_t i) {
  return t.bf16 ? bf16_lo(static_cast<const uint16_t*>(t.src)[i])
                : static_cast<const float*>(t.src)[i];
}

__global__ __launch_bounds__(kThreads) void grad_sq_kernel(GradTable tab, double* part) {
  __shared__ double lds[kThreads / 64];
  double acc = 0.0;
  for (int n = 0; n < tab.n; ++n) {
    const GradEntry t = tab.t[n];
    for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < t.count;
         i += (size_t)gridDim.x * kThreads) {
      const double g = ld_grad(t, i);
      acc = fma(g, g, acc);
    }
  }
  const double s = block_sum(acc, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void grad_norm_kernel(const double* part, int n,
                                                             float* norm) {
  __shared__ double lds[kThreads / 64];
  double acc = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) acc += part[i];
  const double s = block_sum(acc, lds);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

__global__ __launch_bounds__(kThreads) void grad_scale_kernel(GradTable tab, const float* norm,
                                                              float max_norm, int in_place) {
  const float nv = *norm;
  const float coef = nv > max_norm && nv < INFINITY ? max_norm / nv : 1.f;
  if (in_place && coef == 1.f) return;
  for (int n = 0; n < tab.n; ++n) {
    const GradEntry t = tab.t[n];
    for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < t.count;
         i += (size_t)gridDim.x * kThreads) {
      const float v = ld_grad(t, i) * coef;
      if (t.bf16) static_cast<uint16_t*>(t.dst)[i] = (uint16_t)f32_to_bf16_bits(v);
      else static_cast<float*>(t.dst)[i] = v;
    }
  }
}

int grid_of(const GradTable& tab) {
  size_t most = 0;
  for (int n = 0; n < tab.n; ++n) most = tab.t[n].count > most ? tab.t[n].count : most;
  const size_t g = (most + kThreads - 1) / kThreads;
  return g < 1 ? 1 : g > kGradParts ? kGradParts : (int)g;
}

}  // namespace

hipError_t launch_grad_sq(const GradTable& tab, double* part, int* n_part, hipStream_t s) {
  *n_part = grid_of(tab);
  return launch_kernel(grad_sq_kernel, dim3(*n_part), dim3(kThreads), 0, s, KernelTiming{}, tab,
                       part);
}

hipError_t launch_grad_norm(const double* part, int n_part, float* norm, hipStream_t s) {
  return launch_kernel(grad_norm_kernel, dim3(1), dim3(kThreads), 0, s, KernelTiming{}, part,
                       n_part, norm);
}

hipError_t launch_grad_scale(const GradTable& tab, const float* norm, float max_norm, int in_place,
                             hipStream_t s) {
  return launch_kernel(grad_scale_kernel, dim3(grid_of(tab)), dim3(kThreads), 0, s, KernelTiming{},
                       tab, norm, max_norm, in_place);
}

}  // namespace bmoe
