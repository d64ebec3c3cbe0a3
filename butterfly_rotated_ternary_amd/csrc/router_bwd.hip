// Gradient of the router's product l = x W_r^T, from the gradient of its
// logits dl [T][N] (fp32):
//   dx[t][c] = dx_add[t][c] + sum_e dl[t][e] W_r[e][c]
//   dW[e][c] = sum_t dl[t][e] x[t][c]
// fp32 FMA, 64 x 64 outputs per workgroup, 4 x 4 per thread, the reduction in
// chunks of 16 through LDS, in ascending order.
#include "common.h"
#include "kernels.h"

namespace bmoe {
namespace {

constexpr int kRb = 16;

template <typename T>
__device__ __forceinline__ float ld_act(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_lo(*reinterpret_cast<const uint16_t*>(p));
  else return *p;
}
template <typename T>
__device__ __forceinline__ void st_act(T* p, float v) {
  if constexpr (sizeof(T) == 2) *p = (uint16_t)f32_to_bf16_bits(v);
  else *p = v;
}

template <typename T>
__global__ __launch_bounds__(256) void router_dx_kernel(const float* dl, const T* w,
                                                        const T* dx_add, int T_, int d, int N,
                                                        T* dx) {
  __shared__ float as[kRb][65], bs[kRb][65];
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const int t0 = blockIdx.x * 64, c0 = blockIdx.y * 64;
  float acc[4][4] = {};
  for (int e0 = 0; e0 < N; e0 += kRb) {
    for (int u = tid; u < 64 * kRb; u += 256) {
      const int r = u / kRb, ke = u % kRb;
      as[ke][r] = t0 + r < T_ && e0 + ke < N ? dl[(size_t)(t0 + r) * N + e0 + ke] : 0.f;
      const int kb = u / 64, cb = u % 64;
      bs[kb][cb] = e0 + kb < N && c0 + cb < d ? ld_act(w + (size_t)(e0 + kb) * d + c0 + cb) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kRb; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[u][ty + 16 * i], bs[u][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + ty + 16 * i, c = c0 + tx + 16 * j;
      if (t >= T_ || c >= d) continue;
      const size_t o = (size_t)t * d + c;
      st_act(dx + o, acc[i][j] + (dx_add ? ld_act(dx_add + o) : 0.f));
    }
}

template <typename T>
__global__ __launch_bounds__(256) void router_dw_kernel(const float* dl, const T* x, int T_, int d,
                                                        int N, float* dw) {
  __shared__ float as[kRb][65], bs[kRb][65];
  const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16;
  const int e0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  float acc[4][4] = {};
  for (int t0 = 0; t0 < T_; t0 += kRb) {
    for (int u = tid; u < 64 * kRb; u += 256) {
      const int r = u / 64, c = u % 64;
      const bool ok = t0 + r < T_;
      as[r][c] = ok && e0 + c < N ? dl[(size_t)(t0 + r) * N + e0 + c] : 0.f;
      bs[r][c] = ok && c0 + c < d ? ld_act(x + (size_t)(t0 + r) * d + c0 + c) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kRb; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[u][ty + 16 * i], bs[u][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = e0 + ty + 16 * i, c = c0 + tx + 16 * j;
      if (e < N && c < d) dw[(size_t)e * d + c] = acc[i][j];
    }
}

template <typename T>
hipError_t bwd_t(int Tn, int d, int N, const T* x, const T* w, const float* dl, const T* dx_add,
                 T* dx, float* dw, hipStream_t s) {
  const hipError_t e =
      Tn == 0 ? hipSuccess :
      launch_kernel(router_dx_kernel<T>, dim3(((unsigned)Tn + 63) / 64, (d + 63) / 64), dim3(256), 0, s,
                    KernelTiming{}, dl, w, dx_add, Tn, d, N, dx);
  if (e != hipSuccess) return e;
  return launch_kernel(router_dw_kernel<T>, dim3((d + 63) / 64, (N + 63) / 64), dim3(256), 0, s,
                       KernelTiming{}, dl, x, Tn, d, N, dw);
}

}  // namespace

hipError_t launch_router_bwd(bmoe_dtype dt, int T, int d, int N, const void* x, const void* w,
                             const float* dl, const void* dx_add, void* dx, float* dw,
                             hipStream_t s) {
  if (dt == BMOE_BF16)
    return bwd_t(T, d, N, static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w), dl,
                 static_cast<const uint16_t*>(dx_add), static_cast<uint16_t*>(dx), dw, s);
  return bwd_t(T, d, N, static_cast<const float*>(x), static_cast<const float*>(w), dl,
               static_cast<const float*>(dx_add), static_cast<float*>(dx), dw, s);
}

}  // namespace bmoe
