// RMS norm with the residual's addition, in front of the layer, and its gradient:
//   v = x + res,  r = (mean(v^2) + eps)^(-1/2),  y = v r w
// y goes out in the activations' type (the router's rows) and / or in FP8 with a
// scale for each 128 columns (the experts' rows, fp8.cuh), both from the fp32 y.
// With n = v r and g = dy w the gradient is
//   dv = r (g - n mean(g n)) + dsum,   dw = sum over the rows of dy n
// (dsum: what arrives at v itself by the residual stream; x and res both get dv).
// Sums are fp32 in a fixed order.
//
// Both directions are bound by HBM.  Forward of 8192 x 4096, bf16, all outputs: 44.4 us on
// the device (303 MB, 6.8 TB/s).  Gradient of 4096 x 7168: 43 us and 5 for dw's sum
// (235 MB); as blocks that load, add up and store row by row it took 152 us, with one
// group of eight warps behind a ring of bulk copies 49 + 5.
#include "fp8.cuh"
#include "pdl.cuh"
#include "tc_ptx.cuh"

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

// Eight columns as loaded: asked for together before any is used.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
  uint4 a;
  MOE_D void load(const __nv_bfloat16* p, int) { a = *reinterpret_cast<const uint4*>(p); }
  MOE_D void zero() { a = make_uint4(0, 0, 0, 0); }
  MOE_D void values(float* v) const {
    v[0] = fp8::bf16_lo(a.x); v[1] = fp8::bf16_hi(a.x); v[2] = fp8::bf16_lo(a.y);
    v[3] = fp8::bf16_hi(a.y); v[4] = fp8::bf16_lo(a.z); v[5] = fp8::bf16_hi(a.z);
    v[6] = fp8::bf16_lo(a.w); v[7] = fp8::bf16_hi(a.w);
  }
};
template <> struct Raw<float> {
  float4 a, b;
  MOE_D void load(const float* p, int left) {
    a = *reinterpret_cast<const float4*>(p);
    b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (left > 4) b = *reinterpret_cast<const float4*>(p + 4);
  }
  MOE_D void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  MOE_D void values(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

MOE_D float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// blockDim.x threads a row (whole warps, NV vectors a thread), blockDim.y rows a
// block: a row stays in its threads' registers (8192 x 4096, bf16, 47 us), but for the
// widest: four vectors a thread of 1024 spill a little in fp32, eight (above 32768 columns)
// much, and go through the L1 (2048 x 16384 50 us, 1024 x 65536 145, in fp32 512 x 65536
// 245, for 45, 89 and 84 us of bytes).  Bound by HBM: every byte moves once.
template <typename T, int NV, int NT>
__global__ void __launch_bounds__(NT)
    rmsnorm_fwd_kernel(const T* x, const T* res, const float* __restrict__ w, float eps,
                       int64_t rows, int h, T* sum, T* y, uint8_t* __restrict__ q,
                       float* __restrict__ sf, float* __restrict__ rstd) {
  __shared__ float slot[NT / 32];
  pdl_wait();
  pdl_trigger();
  const int nt = blockDim.x;
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool here = row < rows;
  Raw<T> a[NV], b[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + threadIdx.x) * kCols;
    a[i].zero();
    b[i].zero();
    if (here && c < h) {
      a[i].load(x + row * h + c, h - c);
      if (res) b[i].load(res + row * h + c, h - c);
    }
  }
  // one vector a thread is a call of few rows, where w's latency would show
  float w1[kCols] = {};
  if (NV == 1 && (int)threadIdx.x * kCols < h) load8(w + threadIdx.x * kCols, h - (int)threadIdx.x * kCols, w1);
  float v[NV][kCols];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    a[i].values(v[i]);
    if (res) {
      float u[kCols];
      b[i].values(u);
#pragma unroll
      for (int j = 0; j < kCols; ++j) v[i][j] += u[j];
    }
#pragma unroll
    for (int j = 0; j < kCols; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  }
  ss = warp_sum(ss);
  const int nw = nt >> 5;
  if (nw > 1) {
    const int first = threadIdx.y * nw;
    if ((threadIdx.x & 31) == 0) slot[first + (threadIdx.x >> 5)] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < nw; ++i) ss += slot[first + i];
  }
  if (!here) return;  // (whole warps: the shuffles below are within a warp)
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
      if (NV > 1) load8(w + c, h - c, g);
#pragma unroll
      for (int j = 0; j < kCols; ++j) o[j] = v[i][j] * r * (NV > 1 ? g[j] : w1[j]);
      if (y) store8(y + row * h + c, h - c, o);
    }
    if (q) {  // h is a multiple of 128: a block's 16 threads are all in or all out
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < kCols; ++j) m = max(m, fp8::mag_bits(o[j]));
#pragma unroll
      for (int s = 1; s < 16; s <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
      const float top = fp8::block_top(m), inv = fp8::block_inverse(top);
      if (in) {
        *reinterpret_cast<uint2*>(q + row * h + c) = fp8::codes8(o, inv);
        if ((threadIdx.x & 15) == 0)
          sf[row * (h / fp8::BLOCK) + c / fp8::BLOCK] = fp8::block_scale(top);
      }
    }
  }
}

// ---- gradient ------------------------------------------------------------------
// Rows of up to 8192 columns.  A persistent block: G groups of W warps, each a row at a
// time with a ring of shared-memory stages of its own (R rows each, more than one where
// they are short), and one warp that fills the rings with bulk copies (dy, sum and dsum
// of a stage's rows), as many stages ahead as fit: no load of a row to come waits for a
// sum over the present one, and while one group adds up its dot product the others
// compute.  A thread reads its columns from the stage twice, before and after the sum,
// and keeps its part of dw in registers; the groups' are added at the end, a block
// writes one part, and a second kernel adds the blocks' in order.
constexpr int kBwdWarps = 16;
constexpr int kRing = 8;                 // stages a group at most
constexpr int kRingBytes = 216 * 1024;   // shared memory of w and the stages

enum BwdStage { kManyRows, kOneRow, kOneRowAlone };  // (the last: w stays where it is)

template <typename T, int NV, BwdStage MODE>
__global__ void __launch_bounds__(32 * kBwdWarps + 32, 1)
    rmsnorm_bwd_kernel(const T* dy, const T* sum, const float* __restrict__ rstd,
                       const float* __restrict__ w, const T* dsum, int64_t rows, int h, int W,
                       int G, int r_stage, int stages, T* dx, float* __restrict__ part, int* status) {
  constexpr bool ONE = MODE != kManyRows, w_shared = MODE != kOneRowAlone;
  const int R = ONE ? 1 : r_stage;
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ uint64_t full[kBwdWarps][kRing], empty[kBwdWarps][kRing];
  __shared__ float slot[2][kBwdWarps];
  __shared__ int abort[kBwdWarps][2], quit;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int arrays = dsum ? 3 : 2;
  const float* s_w = w_shared ? reinterpret_cast<float*>(dyn) : w;
  const uint32_t array_bytes = (uint32_t)(R * h * sizeof(T)), stage_bytes = arrays * array_bytes;
  const int64_t chunks = (rows + R - 1) / R;
  uint8_t* ring = dyn + (w_shared ? align_up((size_t)h * 4, 128) : 0);  // [group][stage][array]
  if (threadIdx.x == 0) {
    for (int g = 0; g < G; ++g) {
      for (int s = 0; s < stages; ++s) {
        tc::mbar_init(tc::smem_u32(&full[g][s]), 1);
        tc::mbar_init(tc::smem_u32(&empty[g][s]), W);
      }
      abort[g][0] = abort[g][1] = 0;
    }
    quit = 0;
    tc::fence_barrier_init();
  }
  if (w_shared)
    for (int c = threadIdx.x * 4; c < h; c += blockDim.x * 4)
      *reinterpret_cast<float4*>(dyn + 4 * c) = __ldg(reinterpret_cast<const float4*>(w + c));
  __syncthreads();
  if (warp == kBwdWarps) {
    if (lane == 0) {
      const tc::WaitCtl wc{status, &quit, 2000000000ull, 0};
      const tc::WaitCtl wd{status, nullptr, 1000000000ull, 0};
      int stage = 0, g = 0;
      uint32_t phase = 0, laps = 0;  // laps: stages filled by all groups so far
      int64_t issued = 0;
      for (int64_t c = (int64_t)blockIdx.x * G; c < chunks;) {
        if (!tc::mbar_wait(tc::smem_u32(&empty[g][stage]), phase ^ 1, wc)) break;
        const uint32_t fb = tc::smem_u32(&full[g][stage]);
        const uint32_t dst = tc::smem_u32(ring) + (uint32_t)(g * stages + stage) * stage_bytes;
        const int64_t at = c * R * h, left = rows - c * R;
        const uint32_t bytes = left < R ? (uint32_t)(left * h * sizeof(T)) : array_bytes;
        tc::mbar_arrive_expect_tx(fb, arrays * bytes);
        tc::bulk_load(dst, dy + at, bytes, fb);
        tc::bulk_load(dst + array_bytes, sum + at, bytes, fb);
        if (dsum) tc::bulk_load(dst + 2 * array_bytes, dsum + at, bytes, fb);
        ++issued;
        if (++g == G) {
          g = 0;
          ++laps;
          c += (int64_t)(gridDim.x - 1) * G + 1;
          if (++stage == stages) { stage = 0; phase ^= 1; }
        } else {
          ++c;
        }
      }
      // no copy is under way when the block ends: the last one of every stage has come
      const int64_t n = (int64_t)G * stages;
      for (int64_t k = issued > n ? issued - n : 0; k < issued; ++k) {
        const int64_t lap = k / G;
        tc::mbar_wait(tc::smem_u32(&full[k % G][lap % stages]), (uint32_t)(lap / stages) & 1u, wd);
      }
    }
    return;
  }
  const int g = warp / W, tx = (warp % W) * 32 + lane, nt = W * 32;
  if (g >= G) return;
  float acc[NV][kCols] = {};
  int stage = 0, parity = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int64_t c = (int64_t)blockIdx.x * G + g; c < chunks && ok; c += (int64_t)gridDim.x * G) {
    // a wait that gave up is known to every warp of the group behind the next barrier, by
    // a flag of that row's parity (the other may be raised before all have read it)
    const tc::WaitCtl wc{status, &abort[g][parity], 2000000000ull, 0};
    const int64_t row0 = c * R;
    const int n_rows = ONE ? 1 : rows - row0 < R ? (int)(rows - row0) : R;
    float r = __ldg(rstd + row0);
    tc::mbar_wait(tc::smem_u32(&full[g][stage]), phase, wc);
    const T* s_dy = reinterpret_cast<const T*>(ring + (size_t)(g * stages + stage) * stage_bytes);
    for (int k = 0; k < n_rows; ++k, parity ^= 1, s_dy += h) {
      const T *s_sum = s_dy + R * h, *s_ds = s_dy + 2 * R * h;
      const int64_t row = row0 + k;
      const float r_next = k + 1 < n_rows ? __ldg(rstd + row + 1) : 0.f;
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * nt + tx) * kCols;
        if (col < h) {
          float n[kCols], d[kCols], ww[kCols];
          load8(s_sum + col, h - col, n);
          load8(s_dy + col, h - col, d);
          load8(s_w + col, h - col, ww);
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            n[j] *= r;
            acc[i][j] = fmaf(d[j], n[j], acc[i][j]);
            dot = fmaf(d[j] * ww[j], n[j], dot);
          }
        }
      }
      dot = warp_sum(dot);
      if (lane == 0) slot[parity][warp] = dot;
      asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "r"(nt) : "memory");
      if (abort[g][parity]) {
        quit = 1;
        ok = false;
        break;
      }
      dot = 0.f;
      for (int i = 0; i < W; ++i) dot += slot[parity][g * W + i];
      const float mr = dot / (float)h * r;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * nt + tx) * kCols;
        if (col < h) {
          float n[kCols], d[kCols], ww[kCols], o[kCols] = {};
          load8(s_sum + col, h - col, n);
          load8(s_dy + col, h - col, d);
          load8(s_w + col, h - col, ww);
          if (dsum) load8(s_ds + col, h - col, o);
#pragma unroll
          for (int j = 0; j < kCols; ++j) o[j] = fmaf(r, fmaf(-n[j], mr, d[j] * ww[j]), o[j]);
          store8(dx + row * h + col, h - col, o);
        }
      }
      r = r_next;
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(tc::smem_u32(&empty[g][stage]));
    if (++stage == stages) { stage = 0; phase ^= 1; }
  }
  if (!part) return;
  // the groups' parts, added in order by the first one: the others leave theirs in the
  // stages, which no copy is under way to once every group has had all its rows
  const int threads = G * nt;
  float* left = reinterpret_cast<float*>(ring);
  asm volatile("bar.sync 9, %0;" ::"r"(threads) : "memory");
  if (g > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * nt + tx) * kCols;
      if (c < h) store8(left + (size_t)(g - 1) * h + c, h - c, acc[i]);
    }
  }
  asm volatile("bar.sync 9, %0;" ::"r"(threads) : "memory");
  if (g > 0) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * nt + tx) * kCols;
    if (c >= h) continue;
    for (int k = 1; k < G; ++k) {
      float v[kCols];
      load8(left + (size_t)(k - 1) * h + c, h - c, v);
#pragma unroll
      for (int j = 0; j < kCols; ++j) acc[i][j] += v[j];
    }
    store8(part + (int64_t)blockIdx.x * h + c, h - c, acc[i]);
  }
}

// Few rows: one launch, whose first `rows` blocks have a row of dx each and whose others
// 32 columns of dw, summed by 8 threads each over every 8th row and then in order (the
// inputs come a second time, from the L2).
template <typename T>
__global__ void __launch_bounds__(256)
    rmsnorm_bwd_few_kernel(const T* dy, const T* sum, const float* __restrict__ rstd,
                           const float* __restrict__ w, const T* dsum, int rows, int h, T* dx,
                           float* __restrict__ dw) {
  __shared__ float slot[8][33];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x >= (unsigned)rows) {
    const int c = (blockIdx.x - rows) * 32 + lane;
    float v = 0.f;
    if (c < h) {
#pragma unroll 4
      for (int i = warp; i < rows; i += 8)
        v = fmaf(to_f32(dy[(int64_t)i * h + c]), to_f32(sum[(int64_t)i * h + c]) * __ldg(rstd + i), v);
    }
    slot[warp][lane] = v;
    __syncthreads();
    if (warp || c >= h) return;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += slot[i][lane];
    dw[c] = v;
    return;
  }
  const int64_t at = (int64_t)blockIdx.x * h;
  const float r = __ldg(rstd + blockIdx.x);
  float dot = 0.f;
  for (int c = threadIdx.x * kCols; c < h; c += 256 * kCols) {
    float n[kCols], d[kCols], ww[kCols];
    load8(sum + at + c, h - c, n);
    load8(dy + at + c, h - c, d);
    load8(w + c, h - c, ww);
#pragma unroll
    for (int j = 0; j < kCols; ++j) dot = fmaf(d[j] * ww[j], n[j] * r, dot);
  }
  dot = warp_sum(dot);
  if (lane == 0) slot[warp][0] = dot;
  __syncthreads();
  dot = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) dot += slot[i][0];
  const float mr = dot / (float)h * r;
  for (int c = threadIdx.x * kCols; c < h; c += 256 * kCols) {
    float n[kCols], d[kCols], ww[kCols], o[kCols] = {};
    load8(sum + at + c, h - c, n);
    load8(dy + at + c, h - c, d);
    load8(w + c, h - c, ww);
    if (dsum) load8(dsum + at + c, h - c, o);
#pragma unroll
    for (int j = 0; j < kCols; ++j) o[j] = fmaf(r, fmaf(-n[j], mr, d[j] * ww[j]), o[j]);
    store8(dx + at + c, h - c, o);
  }
}

// Longer rows: a block of threads takes rows blockIdx.x, + gridDim.x, ... and reads each
// twice, loads, sum and stores one after the other (2048 x 16384, bf16, with dsum: 100 us
// for 40 of bytes; eight vectors a thread spill as well, 1024 x 65536 225 for 79).
template <typename T, int NV>
__global__ void __launch_bounds__(1024)
    rmsnorm_bwd_long_kernel(const T* dy, const T* sum, const float* __restrict__ rstd,
                            const float* __restrict__ w, const T* dsum, int64_t rows, int h, T* dx,
                            float* __restrict__ part) {
  __shared__ float slot[2][32];
  const int nt = blockDim.x, nw = nt >> 5;
  float acc[NV][kCols] = {};
  int parity = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, parity ^= 1) {
    const float r = __ldg(rstd + row);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * nt + threadIdx.x) * kCols;
      if (c < h) {
        float n[kCols], g[kCols], ww[kCols];
        load8(sum + row * h + c, h - c, n);
        load8(dy + row * h + c, h - c, g);
        load8(w + c, h - c, ww);
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          n[j] *= r;
          acc[i][j] = fmaf(g[j], n[j], acc[i][j]);
          dot = fmaf(g[j] * ww[j], n[j], dot);
        }
      }
    }
    dot = warp_sum(dot);
    if ((threadIdx.x & 31) == 0) slot[parity][threadIdx.x >> 5] = dot;
    __syncthreads();
    dot = 0.f;
    for (int i = 0; i < nw; ++i) dot += slot[parity][i];
    const float mean = dot / (float)h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * nt + threadIdx.x) * kCols;
      if (c < h) {
        float n[kCols], g[kCols], ww[kCols], d[kCols] = {};
        load8(sum + row * h + c, h - c, n);
        load8(dy + row * h + c, h - c, g);
        load8(w + c, h - c, ww);
        if (dsum) load8(dsum + row * h + c, h - c, d);
#pragma unroll
        for (int j = 0; j < kCols; ++j) g[j] = fmaf(r, fmaf(-(n[j] * r), mean, g[j] * ww[j]), d[j]);
        store8(dx + row * h + c, h - c, g);
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

// dw: 32 columns a block, each summed by 16 threads over every 16th part and then
// over the threads, in order.
__global__ void __launch_bounds__(512)
    rmsnorm_dw_kernel(const float* __restrict__ part, int parts, int h, float* __restrict__ dw) {
  __shared__ float s[16][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  pdl_wait();
  pdl_trigger();
  float v = 0.f;
  if (c < h) {
#pragma unroll 4
    for (int i = threadIdx.y; i < parts; i += 16) v += __ldg(part + (int64_t)i * h + c);
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y || c >= h) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) v += s[i][threadIdx.x];
  dw[c] = v;
}

constexpr int kMaxBlocks = 256;  // of the gradient's first kernel
// Rows up to which the gradient is one launch (bf16, with 5 us of the event pair's own: 512 x
// 2048 12.3 us against 14.3, 512 x 7168 14.3 against 20.5; 1024 x 2048 22.5 against 16.4).
constexpr int kFewRows = 512;

// Warps a row in the gradient (the fewest that hold it in 4 vectors a thread) and groups
// a block: at most 8, which have a barrier each, and so many that each has two stages.
int bwd_warps(int h) {
  int w = 1;
  while (w < 8 && h > w * 32 * 4 * kCols) w *= 2;
  return w;
}
int bwd_groups(int h, int W, size_t stage) {
  int g = kBwdWarps / W < 8 ? kBwdWarps / W : 8;
  while (g > 1 && 2 * g * stage > kRingBytes - align_up((size_t)h * 4, 128)) g /= 2;
  return g;
}
constexpr int kBwdMaxCols = 8 * 32 * 4 * kCols;

template <typename T, int NV, int NT>
cudaError_t fwd_launch(int64_t rows, int h, int threads, const void* x, const void* res,
                       const float* w, float eps, void* sum, void* y, uint8_t* q, float* sf,
                       float* rstd, cudaStream_t s) {
  // short rows: several a block, up to 128 threads
  const int per = threads >= 128 ? 1 : 128 / threads;
  return pdl_launch(rmsnorm_fwd_kernel<T, NV, NT>, dim3((unsigned)ceil_div(rows, per)),
                    dim3(threads, per), 0, s, static_cast<const T*>(x), static_cast<const T*>(res), w,
                    eps, rows, h, static_cast<T*>(sum), static_cast<T*>(y), q, sf, rstd);
}

template <typename T>
cudaError_t fwd_t(int64_t rows, int h, const void* x, const void* res, const float* w, float eps,
                  void* sum, void* y, uint8_t* q, float* sf, float* rstd, int sms, cudaStream_t s) {
  const int nvec = (int)ceil_div(h, kCols);
  auto threads = [&](int nv) { return (int)align_up((size_t)ceil_div(nvec, nv), 32); };
#define MOE_NF(NV, NT) \
  return fwd_launch<T, NV, NT>(rows, h, threads(NV), x, res, w, eps, sum, y, q, sf, rstd, s)
  if (nvec <= 128) MOE_NF(1, 128);
  // few rows: as many threads a row as it has vectors (7 rows of 7168 take 4.6 us on the
  // device, 6.0 with four a thread)
  if (nvec <= 1024 && rows <= sms) MOE_NF(1, 1024);
  if (nvec <= 256) MOE_NF(2, 128);
  if (nvec <= 1024) MOE_NF(4, 256);
  if (nvec <= 4096) MOE_NF(4, 1024);
  MOE_NF(8, 1024);
#undef MOE_NF
}

template <typename T>
cudaError_t bwd_t(int64_t rows, int h, const void* dy, const void* sum, const float* rstd,
                  const float* w, const void* dsum, void* dx, float* dw, float* part, int sms,
                  int* status, cudaStream_t s) {
  const T* a = static_cast<const T*>(dy);
  const T* b = static_cast<const T*>(sum);
  const T* d = static_cast<const T*>(dsum);
  T* o = static_cast<T*>(dx);
  float* pt = dw ? part : nullptr;
  const int most = sms < kMaxBlocks ? sms : kMaxBlocks;
  if (rows <= kFewRows && (!dw || (a != o && b != o))) {
    // (in place, dx would go where the blocks for dw still read)
    return pdl_launch(rmsnorm_bwd_few_kernel<T>, dim3((unsigned)(rows + (dw ? ceil_div(h, 32) : 0))),
                      dim3(256), 0, s, a, b, rstd, w, d, (int)rows, h, o, dw);
  }
  int parts;
  if (h <= kBwdMaxCols) {
    const size_t row = (size_t)h * sizeof(T);
    size_t head = align_up((size_t)h * 4, 128);
    int W = bwd_warps(h);
    const int G = bwd_groups(h, W, row * (d ? 3 : 2));
    while (G * W < kBwdWarps && h > W * 256) W *= 2;  // warps that would be idle: fewer vectors a thread
    // short rows come in copies of up to 4 KB (one thread issues them all), while every
    // group has some
    const int64_t share = rows / ((int64_t)most * G), want = 4096 / (int64_t)row;
    const int R = (int)(share < 2 || want < 2 ? 1 : share < want ? share : want);
    const size_t stage = R * row * (d ? 3 : 2);
    if (2 * G * stage > kRingBytes - head) head = 0;  // w in shared memory would cost the second stage
    const int64_t blocks = ceil_div(ceil_div(rows, R), G);
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    const int fit = (int)((kRingBytes - head) / (G * stage)), stages = fit < kRing ? fit : kRing;
#define MOE_BWD(MODE)                                             \
  (h <= W * 256   ? rmsnorm_bwd_kernel<T, 1, MODE>                \
   : h <= W * 512 ? rmsnorm_bwd_kernel<T, 2, MODE>                \
                  : rmsnorm_bwd_kernel<T, 4, MODE>)
    auto kern = R > 1 ? MOE_BWD(kManyRows) : head ? MOE_BWD(kOneRow) : MOE_BWD(kOneRowAlone);
#undef MOE_BWD
    const size_t smem = head + G * stages * stage;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = pdl_launch(kern, dim3(grid), dim3(32 * kBwdWarps + 32), smem, s, a, b, rstd, w, d, rows, h, W, G,
                   R, stages, o, pt, status);
    if (e != cudaSuccess) return e;
    parts = (int)grid;
  } else {
    const unsigned grid = (unsigned)(rows < most ? rows : most);
    const int nvec = (int)ceil_div(h, kCols);
    if (nvec <= 4096)
      rmsnorm_bwd_long_kernel<T, 4><<<grid, (unsigned)align_up(ceil_div(nvec, 4), 32), 0, s>>>(
          a, b, rstd, w, d, rows, h, o, pt);
    else
      rmsnorm_bwd_long_kernel<T, 8><<<grid, (unsigned)align_up(ceil_div(nvec, 8), 32), 0, s>>>(
          a, b, rstd, w, d, rows, h, o, pt);
    parts = (int)grid;
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dw) return e;
  return pdl_launch(rmsnorm_dw_kernel, dim3((unsigned)ceil_div(h, 32)), dim3(32, 16), 0, s,
                    (const float*)part, parts, h, dw);
}

}  // namespace

size_t rmsnorm_bwd_workspace(int64_t rows, int h) {
  const int64_t blocks = rows < kMaxBlocks ? rows : kMaxBlocks;
  return align_up((size_t)blocks * h * 4, 256);
}

cudaError_t launch_rmsnorm_fwd(int64_t rows, int h, int dtype, const void* x, const void* res,
                               const float* w, float eps, void* sum, void* y, uint8_t* q,
                               float* sf, float* rstd, int sms, cudaStream_t s) {
  if (dtype == MOE_BF16)
    return fwd_t<__nv_bfloat16>(rows, h, x, res, w, eps, sum, y, q, sf, rstd, sms, s);
  return fwd_t<float>(rows, h, x, res, w, eps, sum, y, q, sf, rstd, sms, s);
}

cudaError_t launch_rmsnorm_bwd(int64_t rows, int h, int dtype, const void* dy, const void* sum,
                               const float* rstd, const float* w, const void* dsum, void* dx,
                               float* dw, float* part, int sms, int* status, cudaStream_t s) {
  if (dtype == MOE_BF16)
    return bwd_t<__nv_bfloat16>(rows, h, dy, sum, rstd, w, dsum, dx, dw, part, sms, status, s);
  return bwd_t<float>(rows, h, dy, sum, rstd, w, dsum, dx, dw, part, sms, status, s);
}

}  // namespace moe
