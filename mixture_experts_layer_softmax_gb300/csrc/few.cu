// The whole MoE layer for a few tokens (T <= 64): the call of a decoding step.
//
//   l = W_r x (+ b_r), top-K and p as in the layer pass;
//   y_t = sum_k p_tk E_{e_tk}(x_t)  (+ S(x_t)).
//
// The expert weights are the traffic: each busy expert's matrices are read
// from HBM for a handful of rows.  bf16 weights, or MXFP4 weights (E2M1 codes
// with one E8M0 scale per 32 columns) whose values are exact in fp32.
//
// "Scalable Training of Mixture-of-Experts Models with Megatron Core" (review),
// §2.1 (the four steps), §2.2 (router); the same formulas and options as
// moe_layer_fwd.
#include "few.cuh"
#include "router_select.cuh"

namespace moe {

namespace {

// ---- route ----------------------------------------------------------------------
// Partial logits: one warp per (expert, slice of h), eight tokens at a time.
// x is exact in fp32 and the products and sums are fp32, each lane over its
// own columns, the lanes added as a tree.
constexpr int kRouteTok = 8;
__global__ void __launch_bounds__(256)
    few_router_kernel(const __nv_bfloat16* __restrict__ x, const float* __restrict__ w_r, int T,
                      int E, int h, int kparts, float* __restrict__ parts) {
  const int unit = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (unit >= E * kparts) return;
  const int e = unit % E, part = unit / E;
  const int vecs = h / 8;  // 16-byte vectors of x
  const int v0 = (int)((int64_t)vecs * part / kparts), v1 = (int)((int64_t)vecs * (part + 1) / kparts);
  const float* w = w_r + (int64_t)e * h;
  for (int t0 = 0; t0 < T; t0 += kRouteTok) {
    float acc[kRouteTok];
#pragma unroll
    for (int j = 0; j < kRouteTok; ++j) acc[j] = 0.f;
    for (int v = v0 + lane; v < v1; v += 32) {
      const Vec<float> wa = ldg16(w + v * 8), wb = ldg16(w + v * 8 + 4);
#pragma unroll
      for (int j = 0; j < kRouteTok; ++j) {
        if (t0 + j >= T) break;
        const Vec<__nv_bfloat16> xv = ldg16(x + (int64_t)(t0 + j) * h + v * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[j] = fmaf(to_f32(xv.v[i]), wa.v[i], acc[j]);
          acc[j] = fmaf(to_f32(xv.v[i + 4]), wb.v[i], acc[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kRouteTok; ++j) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
      if (lane == 0 && t0 + j < T) parts[((int64_t)part * T + t0 + j) * E + e] = acc[j];
    }
  }
}

template <int J>
MOE_D void few_select_token(const float* parts, int kparts, const float* gate_bias, int t,
                            const RouterArgs& r, int lane) {
  float l[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = lane + 32 * j;
    float s = 0.f;
    if (e < r.E) {
      for (int p = 0; p < kparts; ++p) s += parts[((int64_t)p * r.T + t) * r.E + e];
      if (gate_bias) s += __ldg(gate_bias + e);
    }
    l[j] = s;
  }
  select_and_write<J>(l, t, r, lane);
}

__global__ void __launch_bounds__(32)
    few_select_kernel(const float* __restrict__ parts, int kparts, const float* gate_bias,
                      RouterArgs r, int32_t* idx_out, float* prob_out) {
  const int t = blockIdx.x, lane = threadIdx.x;
  if (r.E <= 32) few_select_token<1>(parts, kparts, gate_bias, t, r, lane);
  else if (r.E <= 64) few_select_token<2>(parts, kparts, gate_bias, t, r, lane);
  else if (r.E <= 128) few_select_token<4>(parts, kparts, gate_bias, t, r, lane);
  else few_select_token<8>(parts, kparts, gate_bias, t, r, lane);
  __syncwarp();
  if (lane < r.K) {
    if (idx_out) idx_out[t * r.K + lane] = r.topk_idx[t * r.K + lane];
    if (prob_out) prob_out[t * r.K + lane] = r.topk_prob[t * r.K + lane];
  }
}

// ---- experts --------------------------------------------------------------------
// Eight consecutive weights of a row in fp32.
template <bool W4>
MOE_D void load_w8(const void* w, const uint8_t* sf, int e, int rows, int cols, int row, int k,
                   float (&v)[8]) {
  if constexpr (W4) {
    const int64_t r = (int64_t)e * rows + row;
    const uint32_t q = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(w) +
                                                               (r * cols + k) / 2));
    const int64_t tile = (int64_t)e * ((rows + 127) / 128) + row / 128;
    const int i = row & 127;
    const uint32_t c = __ldg(sf + (tile * (cols / 128) + k / 128) * 512 + 16 * (i & 31) +
                             4 * (i >> 5) + (k >> 5 & 3));
    const float s = c == 255u ? __uint_as_float(0x7fc00000u)
                              : (c ? __uint_as_float(c << 23) : __uint_as_float(0x00400000u));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t n = q >> (4 * j);
      const int ex = n >> 1 & 3, m = n & 1;
      const float mag = ex ? (float)((2 + m) << ex) * 0.25f : 0.5f * m;
      v[j] = ((n & 8) ? -mag : mag) * s;
    }
  } else {
    const Vec<__nv_bfloat16> u =
        ldg16(static_cast<const __nv_bfloat16*>(w) + ((int64_t)e * rows + row) * cols + k);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = to_f32(u.v[j]);
  }
}

// Whether slot p (token p / K) is beyond its expert's capacity: the number of
// earlier tokens' slots of the same expert.  All lanes return the answer.
MOE_D bool few_dropped(const int32_t* idx, int p, int e, int capacity, int lane) {
  if (capacity <= 0) return false;
  int n = 0;
  for (int q = lane; q < p; q += 32) n += idx[q] == e ? 1 : 0;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n >= capacity;
}

MOE_D float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// a[s, f]: one warp per value; slots P .. P + T - 1 are the shared expert's.
template <bool W4>
__global__ void __launch_bounds__(256) few_fc1_kernel(FewArgs A, const int32_t* idx, float* a) {
  const moe_config_t& c = A.c;
  const int P = c.T * c.K, S = P + (c.n_shared ? c.T : 0), lane = threadIdx.x & 31;
  const int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (u >= (int64_t)S * c.F) return;
  const int s = (int)(u / c.F), f = (int)(u % c.F);
  const bool shared = s >= P;
  const int t = shared ? s - P : s / c.K, e = shared ? 0 : idx[s];
  if (e < 0 || e >= c.E) { report(A.status, MOE_ERR_DEVICE_BOUNDS); return; }
  const bool glu = c.act == MOE_ACT_SWIGLU;
  const int rows = glu ? 2 * c.F : c.F;
  const void* w = shared ? A.w1.ws : A.w1.w;
  const uint8_t* sf = shared ? A.w1.ws_sf : A.w1.sf;
  float g = 0.f, v = 0.f;
  for (int k = lane * 8; k < c.h; k += 256) {
    const Vec<__nv_bfloat16> xv = ldg16(A.x + (int64_t)t * c.h + k);
    float w8[8];
    load_w8<W4>(w, sf, e, rows, c.h, f, k, w8);
#pragma unroll
    for (int j = 0; j < 8; ++j) g = fmaf(to_f32(xv.v[j]), w8[j], g);
    if (glu) {
      load_w8<W4>(w, sf, e, rows, c.h, c.F + f, k, w8);
#pragma unroll
      for (int j = 0; j < 8; ++j) v = fmaf(to_f32(xv.v[j]), w8[j], v);
    }
  }
  g = warp_sum(g);
  v = warp_sum(v);
  if (lane == 0) {
    if (c.has_bias && !shared) g += to_f32(A.b1[(int64_t)e * c.F + f]);
    a[(int64_t)s * c.F + f] = glu ? silu_f(g) * v : gelu_f(g);
  }
}

// y[t, j]: one warp per value, the slots in order.
template <bool W4>
__global__ void __launch_bounds__(256)
    few_fc2_kernel(FewArgs A, const int32_t* idx, const float* prob, const float* a) {
  const moe_config_t& c = A.c;
  const int P = c.T * c.K, lane = threadIdx.x & 31;
  const int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (u >= (int64_t)c.T * c.h) return;
  const int t = (int)(u / c.h), j = (int)(u % c.h);
  float y = 0.f;
  for (int k = 0; k < c.K + (c.n_shared ? 1 : 0); ++k) {
    const bool shared = k == c.K;
    const int s = shared ? P + t : t * c.K + k, e = shared ? 0 : idx[s];
    if (e < 0 || e >= c.E) { report(A.status, MOE_ERR_DEVICE_BOUNDS); continue; }
    if (!shared && few_dropped(idx, s, e, c.capacity, lane)) continue;
    float d = 0.f;
    for (int f = lane * 8; f < c.F; f += 256) {
      float w8[8];
      load_w8<W4>(shared ? A.w2.ws : A.w2.w, shared ? A.w2.ws_sf : A.w2.sf, e, c.h, c.F, j, f, w8);
      const Vec<float> a0 = ldg16(a + (int64_t)s * c.F + f), a1 = ldg16(a + (int64_t)s * c.F + f + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d = fmaf(a0.v[i], w8[i], d);
        d = fmaf(a1.v[i], w8[i + 4], d);
      }
    }
    d = warp_sum(d);
    if (c.has_bias && !shared) d += to_f32(A.b2[(int64_t)e * c.h + j]);
    y += shared ? d : prob[s] * d;
  }
  if (lane == 0) A.y[(int64_t)t * c.h + j] = __float2bfloat16_rn(y);
}

}  // namespace

cudaError_t launch_few(const FewArgs& a, bool mxfp4, cudaStream_t s) {
  const moe_config_t& c = a.c;
  const FewLayout L = few_layout(c);
  float* parts = reinterpret_cast<float*>(a.ws + L.parts);
  int32_t* idx = reinterpret_cast<int32_t*>(a.ws + L.idx);
  float* prob = reinterpret_cast<float*>(a.ws + L.prob);
  float* act = reinterpret_cast<float*>(a.ws + L.a);
  const int kparts = few_kparts(c);
  few_router_kernel<<<(unsigned)ceil_div((int64_t)c.E * kparts, 8), 256, 0, s>>>(
      a.x, a.w_r, c.T, c.E, c.h, kparts, parts);
  RouterArgs r{};
  r.T = c.T; r.E = c.E; r.K = c.K; r.h = c.h; r.score = c.score;
  r.renorm = (c.flags & MOE_FLAG_RENORM) != 0;
  r.force_balance = (c.flags & MOE_FLAG_FORCE_BALANCE) != 0;
  r.sel_bias = a.sel_bias; r.topk_idx = idx; r.topk_prob = prob;
  few_select_kernel<<<c.T, 32, 0, s>>>(parts, kparts, a.gate_bias, r, a.idx_out, a.prob_out);
  const int64_t S = (int64_t)c.T * c.K + (c.n_shared ? c.T : 0);
  const unsigned g1 = (unsigned)ceil_div(S * c.F, 8), g2 = (unsigned)ceil_div((int64_t)c.T * c.h, 8);
  if (mxfp4) {
    few_fc1_kernel<true><<<g1, 256, 0, s>>>(a, idx, act);
    few_fc2_kernel<true><<<g2, 256, 0, s>>>(a, idx, prob, act);
  } else {
    few_fc1_kernel<false><<<g1, 256, 0, s>>>(a, idx, act);
    few_fc2_kernel<false><<<g2, 256, 0, s>>>(a, idx, prob, act);
  }
  return cudaGetLastError();
}

}  // namespace moe
