// FP8 expert products with a scale for each block of 128 (fp8.cuh):
//   z[r, n] = sum_b sa[r, b] sw[n / 128, b] sum_{k in block b} a[r, k] w[n, k]
// for the rows r of each expert, and FC1's epilogue a = p silu(gate) up.
#include "fp8.cuh"

namespace moe {

namespace {

using fp8::BLOCK;

struct Fp8Params {
  const int32_t* offsets;  // [E+1]
  const float* prob;       // FC1: [P] or null
  const uint8_t* a;        // [P, Kd]
  const float* a_sf;       // [P, Kd/128]
  const uint8_t* w;        // [E * Nw, Kd]
  const float* w_sf;       // [E * Nw/128, Kd/128]
  __nv_bfloat16* save;     // FC1: [P, 2N] pre-activation or null
  __nv_bfloat16* out;      // [P, N] or null
  uint8_t* out_q;          // FC1: [P, N] or null
  float* out_sf;           // FC1: [P, N/128]
  int P, E, Kd, N, Nw;     // Nw: weight rows an expert (2N or N)
};

constexpr int BM = 16;

// 16 rows x two blocks of 128 columns (FC1: gate and up) a block of threads;
// thread c + 128 i takes rows 8 i .. 8 i + 7 of column c of both.
template <bool SWIGLU>
__global__ void __launch_bounds__(256) fp8_product_simple_kernel(const Fp8Params p) {
  __shared__ float sA[BM][33], sW[256][33], sO[BM][BLOCK + 1], sTop[BM];
  __shared__ int s_e, s_row, s_end, s_nb;
  const int nblk = SWIGLU ? p.N / BLOCK : (p.N + 255) / 256;
  if (threadIdx.x == 0) {
    int64_t left = blockIdx.x;
    s_e = -1;
    for (int e = 0; e < p.E; ++e) {
      const int lo = min(max(p.offsets[e], 0), p.P), hi = min(max(p.offsets[e + 1], 0), p.P);
      const int64_t tiles = hi > lo ? (int64_t)((hi - lo + BM - 1) / BM) * nblk : 0;
      if (left < tiles) {
        s_e = e;
        s_nb = (int)(left % nblk);
        s_row = lo + (int)(left / nblk) * BM;
        s_end = hi;
        break;
      }
      left -= tiles;
    }
  }
  __syncthreads();
  if (s_e < 0) return;
  const int e = s_e, row0 = s_row, end = s_end, nb = s_nb;
  const int KB = p.Kd / BLOCK;
  const int col0 = SWIGLU ? nb * BLOCK : nb * 256, col1 = SWIGLU ? p.N + nb * BLOCK : col0 + 128;
  const bool two = col1 < p.Nw;
  const int c = threadIdx.x & 127, rh = (threadIdx.x >> 7) * 8;
  float acc[2][8] = {};
  for (int kb = 0; kb < KB; ++kb) {
    float part[2][8] = {};
    for (int k0 = 0; k0 < BLOCK; k0 += 32) {
      __syncthreads();
      for (int i = threadIdx.x; i < BM * 32; i += 256) {
        const int r = row0 + i / 32;
        sA[i / 32][i % 32] =
            r < end ? fp8::decode(p.a[(int64_t)r * p.Kd + kb * BLOCK + k0 + i % 32]) : 0.f;
      }
      for (int i = threadIdx.x; i < 256 * 32; i += 256) {
        const int n = i / 32 < 128 ? col0 + i / 32 : col1 + i / 32 - 128;
        sW[i / 32][i % 32] =
            n < p.Nw ? fp8::decode(p.w[((int64_t)e * p.Nw + n) * p.Kd + kb * BLOCK + k0 + i % 32])
                     : 0.f;
      }
      __syncthreads();
      for (int k = 0; k < 32; ++k) {
        const float w0 = sW[c][k], w1 = sW[128 + c][k];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          part[0][i] = fmaf(sA[rh + i][k], w0, part[0][i]);
          part[1][i] = fmaf(sA[rh + i][k], w1, part[1][i]);
        }
      }
    }
    const int64_t wb = (int64_t)e * (p.Nw / BLOCK);
    const float s0 = p.w_sf[(wb + col0 / BLOCK) * KB + kb];
    const float s1 = two ? p.w_sf[(wb + col1 / BLOCK) * KB + kb] : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sa = row0 + rh + i < end ? p.a_sf[(int64_t)(row0 + rh + i) * KB + kb] : 0.f;
      acc[0][i] = fmaf(part[0][i], sa * s0, acc[0][i]);
      acc[1][i] = fmaf(part[1][i], sa * s1, acc[1][i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = row0 + rh + i;
    if (r >= end) continue;
    if (SWIGLU) {
      const float pr = p.prob ? p.prob[r] : 1.f;
      const float v = pr * (silu_f(acc[0][i]) * acc[1][i]);
      if (p.save) {
        p.save[r * p.Nw + col0 + c] = from_f32<__nv_bfloat16>(acc[0][i]);
        p.save[r * p.Nw + col1 + c] = from_f32<__nv_bfloat16>(acc[1][i]);
      }
      if (p.out) p.out[r * p.N + col0 + c] = from_f32<__nv_bfloat16>(v);
      sO[rh + i][c] = v;
    } else {
      p.out[r * p.N + col0 + c] = from_f32<__nv_bfloat16>(acc[0][i]);
      if (two) p.out[r * p.N + col1 + c] = from_f32<__nv_bfloat16>(acc[1][i]);
    }
  }
  if (!SWIGLU || !p.out_q) return;
  __syncthreads();
  for (int i = threadIdx.x >> 5; i < BM; i += 8) {
    uint32_t m = 0;
    for (int j = threadIdx.x & 31; j < BLOCK; j += 32) m = max(m, fp8::mag_bits(sO[i][j]));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) sTop[i] = fp8::block_top(m);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < BM * 64; i += 256) {
    const int64_t r = row0 + i / 64;
    const int j = 2 * (i % 64);
    if (r >= end) continue;
    const float a = sTop[i / 64], d = a * 0x1p-9f;
    *reinterpret_cast<uint16_t*>(p.out_q + r * p.N + col0 + j) = (uint16_t)fp8::codes2(
        fp8::ratio(sO[i / 64][j], d), fp8::ratio(sO[i / 64][j + 1], d));
    if (j == 0) p.out_sf[r * (p.N / BLOCK) + nb] = fp8::block_scale(a);
  }
}

}  // namespace

// swiglu (FC1): w = W1 codes [E * 2N, Kd] (gate rows, then up rows, per expert);
// plain (FC2): w = W2 codes [E * N, Kd].
cudaError_t launch_fp8_product(bool swiglu, int P, const uint8_t* a, const float* a_sf, int Kd,
                               const uint8_t* w, const float* w_sf, int E, int N,
                               const int32_t* offsets, const float* prob, void* save, void* out,
                               uint8_t* out_q, float* out_sf, int sms, int* status,
                               cudaStream_t s) {
  (void)sms;
  (void)status;
  if (P == 0) return cudaSuccess;
  Fp8Params p{};
  p.offsets = offsets; p.prob = prob; p.a = a; p.a_sf = a_sf; p.w = w; p.w_sf = w_sf;
  p.save = static_cast<__nv_bfloat16*>(save); p.out = static_cast<__nv_bfloat16*>(out);
  p.out_q = out_q; p.out_sf = out_sf;
  p.P = P; p.E = E; p.Kd = Kd; p.N = N; p.Nw = swiglu ? 2 * N : N;
  const int nblk = swiglu ? N / BLOCK : (N + 255) / 256;
  const int64_t tiles = (ceil_div(P, BM) + (E < P ? E : P)) * (int64_t)nblk;
  if (swiglu)
    fp8_product_simple_kernel<true><<<(unsigned)tiles, 256, 0, s>>>(p);
  else
    fp8_product_simple_kernel<false><<<(unsigned)tiles, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
