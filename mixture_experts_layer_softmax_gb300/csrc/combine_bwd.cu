// Gradient of the combine y[t] = sum_k w[t,k] y_perm[dst_row[t,k]]:
//   dy_perm[dst_row[t,k]] = w[t,k] dy[t],   dw[t,k] = <dy[t], y_perm[dst_row[t,k]]>
// A block of threads a token: dy[t] is read once, each y_perm row once, each
// dy_perm row written once; the dot products are fp32 in a fixed order.
#include "common.cuh"

namespace moe {

namespace {

template <typename T, int KMAX>
__global__ void __launch_bounds__(128)
    combine_bwd_kernel(const T* __restrict__ dy, const T* __restrict__ y_perm,
                       const int32_t* __restrict__ dst_row, const float* __restrict__ w, int ntok,
                       int K, int h, T* __restrict__ dy_perm, float* __restrict__ dw, int* status) {
  constexpr int V = Vec<T>::N;
  __shared__ int64_t s_off[KMAX];
  __shared__ float s_w[KMAX], s_dot[4][KMAX];
  const int64_t t = blockIdx.x, P = (int64_t)ntok * K;
  if (threadIdx.x < KMAX) {
    const int k = threadIdx.x;
    int64_t off = -1;
    if (k < K) {
      const int r = __ldg(dst_row + t * K + k);
      if (r >= 0 && r < P)
        off = (int64_t)r * h;
      else if (r != -1)
        report(status, MOE_ERR_DEVICE_BOUNDS);
    }
    s_off[k] = off;
    s_w[k] = off >= 0 && w ? __ldg(w + t * K + k) : 1.f;
  }
  __syncthreads();
  float dot[KMAX] = {};
  const int nvec = h / V;
  for (int v = threadIdx.x; v < nvec; v += 128) {
    Vec<T> u[KMAX];
    const Vec<T> g = ld16_stream(dy + t * h + (int64_t)v * V);
    if (y_perm) {
#pragma unroll
      for (int k = 0; k < KMAX; ++k)
        if (s_off[k] >= 0) u[k] = ld16_stream(y_perm + s_off[k] + (int64_t)v * V);
    }
#pragma unroll
    for (int k = 0; k < KMAX; ++k)
      if (s_off[k] >= 0) {
        Vec<T> o;
#pragma unroll
        for (int q = 0; q < V; ++q) o.v[q] = from_f32<T>(s_w[k] * to_f32(g.v[q]));
        st16(dy_perm + s_off[k] + (int64_t)v * V, o);
        if (y_perm) {
#pragma unroll
          for (int q = 0; q < V; ++q) dot[k] = fmaf(to_f32(g.v[q]), to_f32(u[k].v[q]), dot[k]);
        }
      }
  }
  if (!dw) return;
#pragma unroll
  for (int k = 0; k < KMAX; ++k) {
#pragma unroll
    for (int o = 16; o; o >>= 1) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], o);
    if ((threadIdx.x & 31) == 0) s_dot[threadIdx.x >> 5][k] = dot[k];
  }
  __syncthreads();
  if (threadIdx.x < K) {
    const int k = threadIdx.x;
    dw[t * K + k] = (s_dot[0][k] + s_dot[1][k]) + (s_dot[2][k] + s_dot[3][k]);
  }
}

template <typename T>
cudaError_t combine_bwd_t(const moe_config_t& c, const void* dy, const void* y_perm,
                          const int32_t* dst_row, const float* w, void* dy_perm, float* dw,
                          int* status, cudaStream_t s) {
#define MOE_CB(KM)                                                                             \
  combine_bwd_kernel<T, KM><<<(unsigned)c.T, 128, 0, s>>>(                                     \
      static_cast<const T*>(dy), static_cast<const T*>(y_perm), dst_row, w, c.T, c.K, c.h,     \
      static_cast<T*>(dy_perm), dw, status)
  if (c.K <= 2) MOE_CB(2);
  else if (c.K <= 4) MOE_CB(4);
  else if (c.K <= 8) MOE_CB(8);
  else MOE_CB(16);
#undef MOE_CB
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_combine_bwd(const moe_config_t& c, const void* dy, const void* y_perm,
                               const int32_t* dst_row, const float* w, void* dy_perm, float* dw,
                               int* status, cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  if (c.dtype == MOE_BF16)
    return combine_bwd_t<__nv_bfloat16>(c, dy, y_perm, dst_row, w, dy_perm, dw, status, s);
  return combine_bwd_t<float>(c, dy, y_perm, dst_row, w, dy_perm, dw, status, s);
}

}  // namespace moe
