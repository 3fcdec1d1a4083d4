// Gradient of the combine y[t] = sum_k w[t,k] y_perm[dst_row[t,k]]:
//   dy_perm[dst_row[t,k]] = w[t,k] dy[t],   dw[t,k] = <dy[t], y_perm[dst_row[t,k]]>
// (slots of a token that share a row, as a token that names an expert twice has them, add
// their weights: the combine adds the row once for each).
// dy[t] is read once, each y_perm row once, each dy_perm row written once: bound by HBM.
// The dot products are fp32 in a fixed order.
#include "common.cuh"
#include "pdl.cuh"

namespace moe {

namespace {

// W warps a token; below four, several tokens a block of 128 threads.
template <typename T, int KMAX, int W>
__global__ void __launch_bounds__(W > 4 ? 32 * W : 128, W > 4 ? 1 : KMAX <= 8 ? 5 : 4)
    combine_bwd_kernel(const T* __restrict__ dy, const T* __restrict__ y_perm,
                       const int32_t* __restrict__ dst_row, const float* __restrict__ w, int ntok,
                       int K, int h, T* __restrict__ dy_perm, float* __restrict__ dw, int* status) {
  constexpr int V = Vec<T>::N, B = W > 4 ? 1 : 4 / W;
  __shared__ int64_t s_off[B][KMAX];
  __shared__ float s_w[B][KMAX], s_dot[B * W][KMAX];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, b = warp / W, tx = threadIdx.x - b * (32 * W);
  const int64_t t = (int64_t)blockIdx.x * B + b, P = (int64_t)ntok * K;
  if (tx < 32) {  // the token's first warp, a lane a slot
    const int k = tx;
    int row = -2 - k;  // of no other slot
    if (k < K && t < ntok) {
      const int r = __ldg(dst_row + t * K + k);
      if (r >= 0 && r < P)
        row = r;
      else if (r != -1)
        report(status, MOE_ERR_DEVICE_BOUNDS);
    }
    float wk = row >= 0 && w ? __ldg(w + t * K + k) : 1.f;
    // every slot of a shared row gets the sum, and so writes the same values
    const unsigned same = __match_any_sync(0xffffffffu, row);
    if (__any_sync(0xffffffffu, (same & (same - 1)) != 0)) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        const float wj = __shfl_sync(0xffffffffu, wk, j);
        if ((same >> j) & 1u) sum += wj;
      }
      wk = sum;
    }
    if (k < KMAX) {
      s_off[b][k] = row >= 0 ? (int64_t)row * h : -1;
      s_w[b][k] = wk;
    }
  }
  __syncthreads();
  float dot[KMAX] = {};
  const int nvec = t < ntok ? h / V : 0;
  for (int v = tx; v < nvec; v += 32 * W) {
    Vec<T> u[KMAX];
    const Vec<T> g = ld16_stream(dy + t * h + (int64_t)v * V);
    if (y_perm) {
#pragma unroll
      for (int k = 0; k < KMAX; ++k)
        if (s_off[b][k] >= 0) u[k] = ld16_stream(y_perm + s_off[b][k] + (int64_t)v * V);
    }
#pragma unroll
    for (int k = 0; k < KMAX; ++k)
      if (s_off[b][k] >= 0) {
        Vec<T> o;
#pragma unroll
        for (int q = 0; q < V; ++q) o.v[q] = from_f32<T>(s_w[b][k] * to_f32(g.v[q]));
        st16(dy_perm + s_off[b][k] + (int64_t)v * V, o);
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
    if ((threadIdx.x & 31) == 0) s_dot[warp][k] = dot[k];
  }
  __syncthreads();
  if (tx < K && t < ntok) {
    float s = s_dot[b * W][tx];
#pragma unroll
    for (int i = 1; i < W; ++i) s += s_dot[b * W + i][tx];
    dw[t * K + tx] = s;
  }
}

template <typename T>
cudaError_t combine_bwd_t(const moe_config_t& c, const void* dy, const void* y_perm,
                          const int32_t* dst_row, const float* w, void* dy_perm, float* dw,
                          int sms, int* status, cudaStream_t s) {
  // two vectors a thread or more, if the row has them; 16 warps a token where there is
  // not a token for every SM twice over (100 tokens of 7168, top-8: 20.5 -> 12.3 us)
  const int nvec = c.h / Vec<T>::N;
#define MOE_CB(KM, W)                                                                          \
  return pdl_launch(combine_bwd_kernel<T, KM, W>,                                              \
                    dim3((unsigned)ceil_div(c.T, W > 4 ? 1 : 4 / W)),                          \
                    dim3(W > 4 ? 32 * W : 128), 0, s, static_cast<const T*>(dy),               \
                    static_cast<const T*>(y_perm), dst_row, w, c.T, c.K, c.h,                  \
                    static_cast<T*>(dy_perm), dw, status)
#define MOE_CBW(KM)                                                                            \
  if (nvec < 128) MOE_CB(KM, 1);                                                               \
  else if (nvec < 256) MOE_CB(KM, 2);                                                          \
  else if (c.T > 2 * sms) MOE_CB(KM, 4);                                                       \
  else MOE_CB(KM, 16)
  if (c.K <= 2) { MOE_CBW(2); }
  if (c.K <= 4) { MOE_CBW(4); }
  if (c.K <= 8) { MOE_CBW(8); }
  MOE_CBW(16);
#undef MOE_CBW
#undef MOE_CB
}

}  // namespace

cudaError_t launch_combine_bwd(const moe_config_t& c, const void* dy, const void* y_perm,
                               const int32_t* dst_row, const float* w, void* dy_perm, float* dw,
                               int sms, int* status, cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  if (c.dtype == MOE_BF16)
    return combine_bwd_t<__nv_bfloat16>(c, dy, y_perm, dst_row, w, dy_perm, dw, sms, status, s);
  return combine_bwd_t<float>(c, dy, y_perm, dst_row, w, dy_perm, dw, sms, status, s);
}

}  // namespace moe
