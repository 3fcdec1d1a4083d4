// FP8 tensors with a scale for each block of 128 (fp8.cuh): the quantisers of
// activations (1 x 128 blocks) and of expert weights (128 x 128 blocks, with the
// transposed tensor for data gradients on request), and the dispatch of rows
// that are in 8 bits already.
//
// "Scalable Training of Mixture-of-Experts Models with Megatron Core" (review),
// §5.3, the blockwise FP8 recipe: E4M3, activations in 1 x 128 tiles, weights in
// 128 x 128 blocks.
#include "fp8.cuh"

namespace moe {

namespace {

using fp8::BLOCK;

// 16 threads a 1 x 128 block, 8 values each; two blocks a warp.
__global__ void __launch_bounds__(256)
    fp8_quantize_kernel(const __nv_bfloat16* __restrict__ x, int64_t blocks,
                        uint8_t* __restrict__ q, float* __restrict__ sf) {
  const int lane = threadIdx.x & 31, sub = lane & 15;
  const int64_t nwarps = (int64_t)gridDim.x * 8;
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); 2 * w < blocks; w += nwarps) {
    const int64_t b = 2 * w + (lane >> 4);
    const bool valid = b < blocks;
    Vec<__nv_bfloat16> u = {};
    if (valid) u = ld16_stream(x + b * BLOCK + sub * 8);
    float v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = to_f32(u.v[i]);
      m = max(m, fp8::mag_bits(v[i]));
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float a = fp8::block_top(m);
    if (!valid) continue;
    *reinterpret_cast<uint2*>(q + b * BLOCK + sub * 8) = fp8::codes8(v, a);
    if (sub == 0) sf[b] = fp8::block_scale(a);
  }
}

// One block of threads a 128 x 128 block of w; group g's N rows of K columns.
__global__ void __launch_bounds__(256)
    fp8_quantize_weights_kernel(const __nv_bfloat16* __restrict__ w, int N, int K,
                                uint8_t* __restrict__ q, float* __restrict__ sf,
                                uint8_t* __restrict__ q_t, float* __restrict__ sf_t) {
  __shared__ uint32_t s_max[8];
  __shared__ uint8_t s_q[BLOCK][BLOCK + 4];
  const int NB = N / BLOCK, KB = K / BLOCK;
  const int kb = blockIdx.x % KB, gn = blockIdx.x / KB;
  const int nb = gn % NB;
  const int64_t g = gn / NB;
  const int r0 = threadIdx.x >> 4, c = (threadIdx.x & 15) * 8;
  const __nv_bfloat16* src = w + (g * N + (int64_t)nb * BLOCK) * K + (int64_t)kb * BLOCK + c;
  Vec<__nv_bfloat16> u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = ld16_stream(src + (int64_t)(r0 + 16 * i) * K);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, fp8::mag_bits(to_f32(u[i].v[j])));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
  const float a = fp8::block_top(m);
  uint8_t* dst = q + (g * N + (int64_t)nb * BLOCK) * K + (int64_t)kb * BLOCK + c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = to_f32(u[i].v[j]);
    const uint2 cd = fp8::codes8(v, a);
    *reinterpret_cast<uint2*>(dst + (int64_t)(r0 + 16 * i) * K) = cd;
    if (q_t) {
      uint32_t* row = reinterpret_cast<uint32_t*>(&s_q[r0 + 16 * i][c]);
      row[0] = cd.x;
      row[1] = cd.y;
    }
  }
  if (threadIdx.x == 0) {
    sf[(g * NB + nb) * KB + kb] = fp8::block_scale(a);
    if (sf_t) sf_t[(g * KB + kb) * NB + nb] = fp8::block_scale(a);
  }
  if (!q_t) return;
  __syncthreads();
  uint8_t* dt = q_t + (g * K + (int64_t)kb * BLOCK) * N + (int64_t)nb * BLOCK + c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = r0 + 16 * i;
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j >> 2] |= (uint32_t)s_q[c + j][k] << (8 * (j & 3));
    *reinterpret_cast<uint2*>(dt + (int64_t)k * N) = make_uint2(o[0], o[1]);
  }
}

// One warp a token: its h codes and h / 128 scales to its K rows.
template <int KMAX>
__global__ void __launch_bounds__(256)
    fp8_scatter_kernel(const uint8_t* __restrict__ x_q, const float* __restrict__ x_sf,
                       const int32_t* __restrict__ dst_row, int T, int K, int h,
                       uint8_t* __restrict__ q, float* __restrict__ sf, int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= T) return;
  const int64_t P = (int64_t)T * K;
  int64_t row[KMAX];
#pragma unroll
  for (int k = 0; k < KMAX; ++k) {
    row[k] = -1;
    if (k < K) {
      const int r = __ldg(dst_row + t * K + k);
      if (r >= 0 && r < P)
        row[k] = r;
      else if (r != -1)
        report(status, MOE_ERR_DEVICE_BOUNDS);
    }
  }
  const int nvec = h / 16, KB = h / BLOCK;
  const uint4* src = reinterpret_cast<const uint4*>(x_q + t * h);
  for (int v = lane; v < nvec; v += 32) {
    const uint4 u = __ldg(src + v);
#pragma unroll
    for (int k = 0; k < KMAX; ++k)
      if (row[k] >= 0) reinterpret_cast<uint4*>(q + row[k] * h)[v] = u;
  }
  for (int b = lane; b < KB; b += 32) {
    const float s = __ldg(x_sf + t * KB + b);
#pragma unroll
    for (int k = 0; k < KMAX; ++k)
      if (row[k] >= 0) sf[row[k] * KB + b] = s;
  }
}

}  // namespace

cudaError_t launch_fp8_quantize(int64_t rows, int K, const void* x, uint8_t* q, float* sf, int sms,
                                cudaStream_t s) {
  const int64_t blocks = rows * (K / BLOCK), need = ceil_div(blocks, 16);
  const int grid = (int)(need < 8LL * sms ? need : 8LL * sms);
  fp8_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(x), blocks, q, sf);
  return cudaGetLastError();
}

cudaError_t launch_fp8_quantize_weights(int groups, int N, int K, const void* w, uint8_t* q,
                                        float* sf, uint8_t* q_t, float* sf_t, cudaStream_t s) {
  const unsigned grid = (unsigned)((int64_t)groups * (N / BLOCK) * (K / BLOCK));
  fp8_quantize_weights_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(w), N, K, q,
                                                   sf, q_t, sf_t);
  return cudaGetLastError();
}

cudaError_t launch_fp8_scatter(const moe_config_t& c, const uint8_t* x_q, const float* x_sf,
                               const int32_t* dst_row, uint8_t* q, float* sf, int* status,
                               cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  const unsigned grid = (unsigned)ceil_div(c.T, 8);
#define MOE_FS(KM) \
  fp8_scatter_kernel<KM><<<grid, 256, 0, s>>>(x_q, x_sf, dst_row, c.T, c.K, c.h, q, sf, status)
  if (c.K <= 2) MOE_FS(2);
  else if (c.K <= 4) MOE_FS(4);
  else if (c.K <= 8) MOE_FS(8);
  else MOE_FS(16);
#undef MOE_FS
  return cudaGetLastError();
}

}  // namespace moe
