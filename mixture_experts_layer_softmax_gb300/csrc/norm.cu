// RMS norm with the residual's addition, in front of the layer, and its gradient:
//   v = x + res,  r = (mean(v^2) + eps)^(-1/2),  y = v r w
// y goes out in the activations' type (the router's rows) and / or in FP8 with a
// scale for each 128 columns (the experts' rows, fp8.cuh), both from the fp32 y.
// With n = v r and g = dy w the gradient is
//   dv = r (g - n mean(g n)) + dsum,   dw = sum over the rows of dy n
// (dsum: what arrives at v itself by the residual stream; x and res both get dv).
// Sums are fp32 in a fixed order.
#include "fp8.cuh"

namespace moe {

namespace {

constexpr int kCols = 8;  // columns a thread holds per vector

// Columns [c, c + 8) of a row: one 16-byte load of bf16, two of fp32 (the second
// only where the row goes on: fp32 rows are multiples of 4).  Plain loads: the
// outputs may be the inputs' own buffers.
MOE_D void load8(const __nv_bfloat16* p, int left, float* v) {
  (void)left;
  Vec<__nv_bfloat16> u;
  *reinterpret_cast<uint4*>(&u) = *reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = to_f32(u.v[i]);
}
MOE_D void load8(const float* p, int left, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
  if (left > 4) b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
MOE_D void store8(__nv_bfloat16* p, int left, const float* v) {
  (void)left;
  Vec<__nv_bfloat16> u;
#pragma unroll
  for (int i = 0; i < 8; ++i) u.v[i] = from_f32<__nv_bfloat16>(v[i]);
  st16(p, u);
}
MOE_D void store8(float* p, int left, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  if (left > 4) *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Sum over the block's threads, in the same order for every thread; `slot` holds
// a float a warp.
MOE_D float block_sum(float v, float* slot) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int nw = blockDim.x >> 5;
  if (nw == 1) return v;
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < nw; ++i) t += slot[i];
  __syncthreads();
  return t;
}

// A block of threads a row, which stays in its registers (NV vectors a thread).
template <typename T, int NV>
__global__ void __launch_bounds__(1024)
    rmsnorm_fwd_kernel(const T* x, const T* res, const float* __restrict__ w, float eps, int h,
                       T* sum, T* y, uint8_t* __restrict__ q, float* __restrict__ sf,
                       float* __restrict__ rstd) {
  __shared__ float slot[32];
  const int64_t row = blockIdx.x;
  const int nt = blockDim.x;
  float v[NV][kCols];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + threadIdx.x) * kCols;
#pragma unroll
    for (int j = 0; j < kCols; ++j) v[i][j] = 0.f;
    if (c < h) {
      load8(x + row * h + c, h - c, v[i]);
      if (res) {
        float u[kCols];
        load8(res + row * h + c, h - c, u);
#pragma unroll
        for (int j = 0; j < kCols; ++j) v[i][j] += u[j];
      }
    }
#pragma unroll
    for (int j = 0; j < kCols; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  }
  ss = block_sum(ss, slot);
  const float r = 1.f / sqrtf(ss / (float)h + eps);
  if (rstd && threadIdx.x == 0) rstd[row] = r;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + threadIdx.x) * kCols;
    const bool in = c < h;
    float o[kCols] = {};
    if (in) {
      if (sum) store8(sum + row * h + c, h - c, v[i]);
      float g[kCols];
      load8(w + c, h - c, g);
#pragma unroll
      for (int j = 0; j < kCols; ++j) o[j] = v[i][j] * r * g[j];
      if (y) store8(y + row * h + c, h - c, o);
    }
    if (q) {  // h is a multiple of 128: a block's 16 threads are all in or all out
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < kCols; ++j) m = max(m, fp8::mag_bits(o[j]));
#pragma unroll
      for (int s = 1; s < 16; s <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
      const float a = fp8::block_top(m);
      if (in) {
        *reinterpret_cast<uint2*>(q + row * h + c) = fp8::codes8(o, a);
        if ((threadIdx.x & 15) == 0)
          sf[row * (h / fp8::BLOCK) + c / fp8::BLOCK] = fp8::block_scale(a);
      }
    }
  }
}

// A block of threads takes rows blockIdx.x, + gridDim.x, ...; each thread keeps
// its columns' part of dw in registers and writes it once, to part[blockIdx.x].
template <typename T, int NV>
__global__ void __launch_bounds__(1024)
    rmsnorm_bwd_kernel(const T* dy, const T* sum, const float* __restrict__ rstd,
                       const float* __restrict__ w, const T* dsum, int64_t rows, int h, T* dx,
                       float* __restrict__ part) {
  __shared__ float slot[32];
  const int nt = blockDim.x;
  float acc[NV][kCols] = {};
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float r = __ldg(rstd + row);
    float n[NV][kCols], g[NV][kCols];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * nt + threadIdx.x) * kCols;
#pragma unroll
      for (int j = 0; j < kCols; ++j) n[i][j] = g[i][j] = 0.f;
      if (c < h) {
        float ww[kCols];
        load8(sum + row * h + c, h - c, n[i]);
        load8(dy + row * h + c, h - c, g[i]);
        load8(w + c, h - c, ww);
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          n[i][j] *= r;
          acc[i][j] = fmaf(g[i][j], n[i][j], acc[i][j]);
          g[i][j] *= ww[j];
          dot = fmaf(g[i][j], n[i][j], dot);
        }
      }
    }
    const float mean = block_sum(dot, slot) / (float)h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * nt + threadIdx.x) * kCols;
      if (c < h) {
        float o[kCols], d[kCols] = {};
        if (dsum) load8(dsum + row * h + c, h - c, d);
#pragma unroll
        for (int j = 0; j < kCols; ++j) o[j] = fmaf(r, fmaf(-n[i][j], mean, g[i][j]), d[j]);
        store8(dx + row * h + c, h - c, o);
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + threadIdx.x) * kCols;
    if (c < h) store8(part + (int64_t)blockIdx.x * h + c, h - c, acc[i]);
  }
}

// dw = the parts added in order, a thread a column.
__global__ void __launch_bounds__(128)
    rmsnorm_dw_kernel(const float* __restrict__ part, int parts, int h, float* __restrict__ dw) {
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (c >= h) return;
  float s = 0.f;
  for (int i = 0; i < parts; ++i) s += __ldg(part + (int64_t)i * h + c);
  dw[c] = s;
}

constexpr int kMaxParts = 512;

// Vectors a thread and threads a block for rows of h columns.
struct Shape {
  int nv, threads;
};
Shape row_shape(int h) {
  const int nvec = (int)ceil_div(h, kCols);
  int nv = 1;
  while (nv < 8 && ceil_div(nvec, nv) > (nv < 4 ? 256 : 1024)) nv *= 2;
  return {nv, (int)align_up((size_t)ceil_div(nvec, nv), 32)};
}

template <typename T>
cudaError_t fwd_t(int64_t rows, int h, const void* x, const void* res, const float* w, float eps,
                  void* sum, void* y, uint8_t* q, float* sf, float* rstd, cudaStream_t s) {
  const Shape sh = row_shape(h);
#define MOE_NF(NV)                                                                                \
  rmsnorm_fwd_kernel<T, NV><<<(unsigned)rows, sh.threads, 0, s>>>(                                \
      static_cast<const T*>(x), static_cast<const T*>(res), w, eps, h, static_cast<T*>(sum),      \
      static_cast<T*>(y), q, sf, rstd)
  if (sh.nv == 1) MOE_NF(1);
  else if (sh.nv == 2) MOE_NF(2);
  else if (sh.nv == 4) MOE_NF(4);
  else MOE_NF(8);
#undef MOE_NF
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_t(int64_t rows, int h, const void* dy, const void* sum, const float* rstd,
                  const float* w, const void* dsum, void* dx, float* dw, float* part, int sms,
                  cudaStream_t s) {
  const Shape sh = row_shape(h);
  const int64_t want = rows < 2LL * sms ? rows : 2LL * sms;
  const unsigned grid = (unsigned)(want < kMaxParts ? want : kMaxParts);
#define MOE_NB(NV)                                                                                \
  rmsnorm_bwd_kernel<T, NV><<<grid, sh.threads, 0, s>>>(                                          \
      static_cast<const T*>(dy), static_cast<const T*>(sum), rstd, w,                             \
      static_cast<const T*>(dsum), rows, h, static_cast<T*>(dx), dw ? part : nullptr)
  if (sh.nv == 1) MOE_NB(1);
  else if (sh.nv == 2) MOE_NB(2);
  else if (sh.nv == 4) MOE_NB(4);
  else MOE_NB(8);
#undef MOE_NB
  if (dw) rmsnorm_dw_kernel<<<(unsigned)ceil_div(h, 128), 128, 0, s>>>(part, (int)grid, h, dw);
  return cudaGetLastError();
}

}  // namespace

size_t rmsnorm_bwd_workspace(int64_t rows, int h) {
  const int64_t parts = rows < kMaxParts ? rows : kMaxParts;
  return align_up((size_t)parts * h * 4, 256);
}

cudaError_t launch_rmsnorm_fwd(int64_t rows, int h, int dtype, const void* x, const void* res,
                               const float* w, float eps, void* sum, void* y, uint8_t* q,
                               float* sf, float* rstd, cudaStream_t s) {
  if (dtype == MOE_BF16)
    return fwd_t<__nv_bfloat16>(rows, h, x, res, w, eps, sum, y, q, sf, rstd, s);
  return fwd_t<float>(rows, h, x, res, w, eps, sum, y, q, sf, rstd, s);
}

cudaError_t launch_rmsnorm_bwd(int64_t rows, int h, int dtype, const void* dy, const void* sum,
                               const float* rstd, const float* w, const void* dsum, void* dx,
                               float* dw, float* part, int sms, cudaStream_t s) {
  if (dtype == MOE_BF16)
    return bwd_t<__nv_bfloat16>(rows, h, dy, sum, rstd, w, dsum, dx, dw, part, sms, s);
  return bwd_t<float>(rows, h, dy, sum, rstd, w, dsum, dx, dw, part, sms, s);
}

}  // namespace moe
