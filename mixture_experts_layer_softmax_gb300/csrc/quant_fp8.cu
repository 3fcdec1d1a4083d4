// FP8 tensors with a scale for each block of 128 (fp8.cuh): the quantisers of
// activations (1 x 128 blocks) and of expert weights (128 x 128 blocks, with the
// transposed tensor for data gradients on request), and the dispatch of rows
// that are in 8 bits already.
//
// "Scalable Training of Mixture-of-Experts Models with Megatron Core" (review),
// §5.3, the blockwise FP8 recipe: E4M3, activations in 1 x 128 tiles, weights in
// 128 x 128 blocks.
//
// All are bound by HBM: weights of 8 x 28672 x 4096 with their transposes 549 us (3.76 GB,
// 6.85 TB/s), rows of 16384 x 4096 to 8 experts each 92 us without the maps (626 MB).
#include "fp8.cuh"
#include "pdl.cuh"

namespace moe {

namespace {

using fp8::BLOCK;

// Eight threads a 1 x 128 block, 16 values each: a warp's 16-byte stores fill lines.
// Each thread has the loads of U blocks in flight.
template <int U>
__global__ void __launch_bounds__(256)
    fp8_quantize_kernel(const __nv_bfloat16* __restrict__ x, int64_t blocks,
                        uint8_t* __restrict__ q, float* __restrict__ sf) {
  pdl_wait();
  pdl_trigger();
  const int sub = threadIdx.x & 7;
  const int64_t b0 = (int64_t)blockIdx.x * (32 * U) + (threadIdx.x >> 3);
  uint4 u[U][2];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int64_t b = b0 + 32 * k;
    u[k][0] = u[k][1] = make_uint4(0, 0, 0, 0);
    if (b < blocks) {
      const uint4* src = reinterpret_cast<const uint4*>(x + b * BLOCK) + 2 * sub;
      u[k][0] = __ldcs(src);
      u[k][1] = __ldcs(src + 1);
    }
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int64_t b = b0 + 32 * k;
    uint32_t m = __vmaxu2(fp8::mag_max2(u[k][0]), fp8::mag_max2(u[k][1]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (b >= blocks) continue;
    const float a = fp8::block_top(fp8::mag_bits2(m)), inv = fp8::block_inverse(a);
    const uint2 lo = fp8::codes8(u[k][0], inv), hi = fp8::codes8(u[k][1], inv);
    reinterpret_cast<uint4*>(q + b * BLOCK)[sub] = make_uint4(lo.x, lo.y, hi.x, hi.y);
    if (sub == 0) sf[b] = fp8::block_scale(a);
  }
}

// A block of threads a 128 x 128 block of w (group g's N rows of K columns): thread
// (r, c) has columns 16 c .. 16 c + 15 of rows r, r + 32, r + 64, r + 96.  For the
// transposed codes the block passes through shared memory as words of four columns,
// word w of row n at place w ^ 4 (n / 16) of its row: then the stores and the loads
// of a warp each fall into different banks.  On the way out a thread has four
// columns k of 16 rows n: 16 words, transposed four by four with byte permutes.
__global__ void __launch_bounds__(256)
    fp8_quantize_weights_kernel(const __nv_bfloat16* __restrict__ w, int N, int K,
                                uint8_t* __restrict__ q, float* __restrict__ sf,
                                uint8_t* __restrict__ q_t, float* __restrict__ sf_t) {
  __shared__ uint32_t s_max[8];
  __shared__ __align__(16) uint32_t s_q[BLOCK][32];
  pdl_wait();
  pdl_trigger();
  const int NB = N / BLOCK, KB = K / BLOCK;
  const int kb = blockIdx.x % KB, gn = blockIdx.x / KB;
  const int nb = gn % NB;
  const int64_t g = gn / NB;
  const int r = threadIdx.x >> 3, c = threadIdx.x & 7;
  const int64_t row0 = g * N + (int64_t)nb * BLOCK, col0 = (int64_t)kb * BLOCK + c * 16;
  uint4 u[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4* src = reinterpret_cast<const uint4*>(w + (row0 + r + 32 * i) * K + col0);
    u[i][0] = __ldcs(src);
    u[i][1] = __ldcs(src + 1);
  }
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m2 = __vmaxu2(m2, __vmaxu2(fp8::mag_max2(u[i][0]), fp8::mag_max2(u[i][1])));
  uint32_t m = __reduce_max_sync(0xffffffffu, fp8::mag_bits2(m2));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
  const float a = fp8::block_top(m), inv = fp8::block_inverse(a);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint2 lo = fp8::codes8(u[i][0], inv), hi = fp8::codes8(u[i][1], inv);
    const uint4 v = make_uint4(lo.x, lo.y, hi.x, hi.y);
    const int n = r + 32 * i;
    *reinterpret_cast<uint4*>(q + (row0 + n) * K + col0) = v;
    if (q_t) *reinterpret_cast<uint4*>(&s_q[n][(4 * c) ^ (4 * (n >> 4))]) = v;
  }
  if (threadIdx.x == 0) {
    sf[(g * NB + nb) * KB + kb] = fp8::block_scale(a);
    if (sf_t) sf_t[(g * KB + kb) * NB + nb] = fp8::block_scale(a);
  }
  if (!q_t) return;
  __syncthreads();
  const int k4 = r, n16 = c;  // columns 4 k4 .. + 3 of rows 16 n16 .. + 15
  uint32_t o[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = s_q[16 * n16 + 4 * i + j][k4 ^ (4 * n16)];
    const uint32_t a0 = __byte_perm(v[0], v[1], 0x5140), a1 = __byte_perm(v[2], v[3], 0x5140);
    const uint32_t b0 = __byte_perm(v[0], v[1], 0x7362), b1 = __byte_perm(v[2], v[3], 0x7362);
    o[0][i] = __byte_perm(a0, a1, 0x5410);
    o[1][i] = __byte_perm(a0, a1, 0x7632);
    o[2][i] = __byte_perm(b0, b1, 0x5410);
    o[3][i] = __byte_perm(b0, b1, 0x7632);
  }
  uint8_t* dt = q_t + (g * K + (int64_t)kb * BLOCK + 4 * k4) * N + (int64_t)nb * BLOCK + 16 * n16;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(dt + (int64_t)j * N) = make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]);
}

// One warp V x 512 bytes of a token's codes (grid.y of them a row), to its K rows, and
// the row's h / 128 scales with the first.  What it reads is in registers before the
// maps' last step has ended (programmatic dependent launch); the destinations are read
// after it.
template <int KMAX, int V>
__global__ void __launch_bounds__(256)
    fp8_scatter_kernel(const uint8_t* __restrict__ x_q, const float* __restrict__ x_sf,
                       const int32_t* __restrict__ dst_row, int T, int K, int h,
                       uint8_t* __restrict__ q, float* __restrict__ sf, int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= T) {
    pdl_wait();
    return;
  }
  const int64_t P = (int64_t)T * K;
  const int nvec = h / 16, KB = h / BLOCK, v0 = blockIdx.y * (32 * V) + lane;
  const uint4* src = reinterpret_cast<const uint4*>(x_q + t * h);
  uint4 u[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (v0 + i * 32 < nvec) u[i] = __ldcs(src + v0 + i * 32);
  float s0 = blockIdx.y == 0 && lane < KB ? __ldg(x_sf + t * KB + lane) : 0.f;
  pdl_wait();
  pdl_trigger();
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
#pragma unroll
  for (int k = 0; k < KMAX; ++k) {
    if (row[k] < 0) continue;
    uint4* dst = reinterpret_cast<uint4*>(q + row[k] * h);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (v0 + i * 32 < nvec) dst[v0 + i * 32] = u[i];
  }
  if (blockIdx.y) return;
  for (int b = lane; b < KB; b += 32) {
    if (b >= 32) s0 = __ldg(x_sf + t * KB + b);
#pragma unroll
    for (int k = 0; k < KMAX; ++k)
      if (row[k] >= 0) sf[row[k] * KB + b] = s0;
  }
}

}  // namespace

cudaError_t launch_fp8_quantize(int64_t rows, int K, const void* x, uint8_t* q, float* sf, int sms,
                                cudaStream_t s) {
  const int64_t blocks = rows * (K / BLOCK);
  const __nv_bfloat16* xs = static_cast<const __nv_bfloat16*>(x);
  // four blocks a thread while that leaves every SM four blocks of threads
  if (blocks >= 32LL * 4 * 4 * sms)
    return pdl_launch(fp8_quantize_kernel<4>, dim3((unsigned)ceil_div(blocks, 128)), dim3(256), 0, s, xs,
                      blocks, q, sf);
  return pdl_launch(fp8_quantize_kernel<1>, dim3((unsigned)ceil_div(blocks, 32)), dim3(256), 0, s, xs,
                    blocks, q, sf);
}

cudaError_t launch_fp8_quantize_weights(int groups, int N, int K, const void* w, uint8_t* q,
                                        float* sf, uint8_t* q_t, float* sf_t, cudaStream_t s) {
  const unsigned grid = (unsigned)((int64_t)groups * (N / BLOCK) * (K / BLOCK));
  return pdl_launch(fp8_quantize_weights_kernel, dim3(grid), dim3(256), 0, s,
                    static_cast<const __nv_bfloat16*>(w), N, K, q, sf, q_t, sf_t);
}

cudaError_t launch_fp8_scatter(const moe_config_t& c, const uint8_t* x_q, const float* x_sf,
                               const int32_t* dst_row, uint8_t* q, float* sf, int sms, int* status,
                               cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  // 8 vectors a thread; 2 while that leaves an SM less than 16 warps
  const bool small = c.T * ceil_div(c.h, 4096) < 16LL * sms;
  const int per = small ? 1024 : 4096;
  const dim3 grid((unsigned)ceil_div(c.T, 8), (unsigned)ceil_div(c.h, per));
  // (directly behind the maps' steps on the stream: see the kernel)
#define MOE_FS(KM)                                                                                  \
  (small ? pdl_launch(fp8_scatter_kernel<KM, 2>, grid, dim3(256), 0, s, x_q, x_sf, dst_row, c.T,    \
                      c.K, c.h, q, sf, status)                                                      \
         : pdl_launch(fp8_scatter_kernel<KM, 8>, grid, dim3(256), 0, s, x_q, x_sf, dst_row, c.T,    \
                      c.K, c.h, q, sf, status))
  return c.K <= 2 ? MOE_FS(2) : c.K <= 4 ? MOE_FS(4) : c.K <= 8 ? MOE_FS(8) : MOE_FS(16);
#undef MOE_FS
}

}  // namespace moe
