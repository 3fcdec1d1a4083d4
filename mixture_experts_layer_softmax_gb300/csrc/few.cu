// The whole MoE layer for a few tokens (T <= 64): the call of a decoding step.
//
//   l = W_r x (+ b_r), top-K and p as in the layer pass;
//   y_t = sum_k p_tk E_{e_tk}(x_t)  (+ S(x_t)).
//
// The expert weights are the traffic: each busy expert's matrices are read
// from HBM for a handful of rows.  bf16 weights, or MXFP4 weights (E2M1 codes
// with one E8M0 scale per 32 columns).
//
// Two launches.  few_router_kernel writes partial logits (and, for MXFP4
// weights, the tokens in fp16).  few_kernel does the rest, one block per SM:
//   every block selects the experts of all tokens and sorts the (token, slot)
//   pairs by expert (the same list everywhere), then takes units of work from
//   one counter: first all of FC1's units (an expert, a block of its rows),
//   then FC2's (an expert, a block of rows of h, a slice of F).  An FC2 unit
//   waits until its expert's FC1 units are done.  Units are taken in order, so
//   every FC1 unit that an FC2 unit waits for belongs to a block that already
//   runs and waits for nothing: no block needs any other to become resident.
//   When all FC2 units are done every block adds its share of the slots'
//   results, in slot order, and writes y.
// Within a block: two producer warps stream the unit's weight rows and the
// expert's token rows through a ring of shared-memory stages (512 columns a
// stage, TMA boxes of many rows: a copy per row costs its issuing warp about
// 95 cycles whatever its size, which held an earlier form of this kernel at 10 bytes a
// cycle and SM).  The weight producer runs ahead of the arithmetic, into the
// next unit and from FC1 into FC2, so that HBM stays busy across unit and
// phase borders; only the token producer waits for FC1's results.  NW consumer
// warps split a stage's columns and multiply with m16n8k16 tensor-core
// instructions, weight rows as M, tokens as N: the weights are read once from
// HBM however many tokens share them, and a product with up to 32 tokens costs
// less than the loads.  (tcgen05 wants 128 weight rows a tile; that would
// leave too few units to balance the SMs, and the mma rate is not what bounds
// this kernel.)
// At a unit's end the warps' sums meet in shared memory, in warp order.
//
// "Scalable Training of Mixture-of-Experts Models with Megatron Core" (review),
// §2.1 (the four steps), §2.2 (router); the same formulas and options as
// moe_layer_fwd.
#include <cuda_fp16.h>

#include "few.cuh"
#include "mx.cuh"
#include "router_select.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

MOE_D void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
MOE_D void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The power of two that brings a largest magnitude (fp32 bits m) into
// [2^14, 2^15) when the values are divided by it; 1 for a row with an infinity or
// a NaN (they stay what they are), the smallest useful one below 2^-86.
MOE_D float f16_block_scale(uint32_t m) {
  const int e = (int)(m >> 23);
  if (e == 255) return 1.f;
  return __uint_as_float((uint32_t)(max(e, 41) - 14) << 23);
}
// Tokens in fp16: x = xh * xs with xs a power of two that puts the token's
// largest magnitude into [2^14, 2^15).  Exact for values down to 2^-29 of the
// largest; below, the error is at most 2^-40 of it, far under the fp32 sums'.
__device__ void few_convert_token(const __nv_bfloat16* __restrict__ x, int h,
                                  __half* __restrict__ xh, float* __restrict__ xs) {
  __shared__ uint32_t s_max[8];
  uint32_t m = 0;
  for (int v = threadIdx.x; v < h / 8; v += blockDim.x) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(x) + v);
    for (uint32_t w : {u.x, u.y, u.z, u.w}) m = max(m, max((w << 16) & 0x7fff0000u, w & 0x7fff0000u));
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int w = 0; w < 8; ++w) m = max(m, s_max[w]);
  const float scale = f16_block_scale(m), inv = 1.f / scale;
  if (threadIdx.x == 0) *xs = scale;
  for (int v = threadIdx.x; v < h / 8; v += blockDim.x) {
    const Vec<__nv_bfloat16> u = ldg16(x + v * 8);
    __half o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __float2half_rn(to_f32(u.v[i]) * inv);
    *reinterpret_cast<uint4*>(xh + v * 8) = *reinterpret_cast<const uint4*>(o);
  }
}

// ---- route ----------------------------------------------------------------------
// Partial logits: one warp per (expert, slice of h), eight tokens at a time.
// x is exact in fp32 and the products and sums are fp32, each lane over its
// own columns, the lanes added as a tree.  The blocks past the router's convert
// one token each; block 0 clears the counters of few_kernel.
constexpr int kRouteTok = 8;
__global__ void __launch_bounds__(256)
    few_router_kernel(const __nv_bfloat16* __restrict__ x, const float* __restrict__ w_r, int T,
                      int E, int h, int kparts, float* __restrict__ parts, int route_blocks,
                      __half* xh, float* xs, int32_t* sync, int sync_words) {
  pdl_trigger();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < sync_words; i += blockDim.x) sync[i] = 0;
  if ((int)blockIdx.x >= route_blocks) {
    const int t = blockIdx.x - route_blocks;
    few_convert_token(x + (int64_t)t * h, h, xh + (int64_t)t * h, xs + t);
    return;
  }
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

// One token's logits (the slices added in order) and its selection: a warp.
// All experts' loads of four slices go out together: their latency, not their
// number, is what a decoding step waits for here.
template <int J>
MOE_D void few_select_token(const float* parts, int kparts, const float* gate_bias, int t,
                            const RouterArgs& r, int lane) {
  float l[J];
#pragma unroll
  for (int j = 0; j < J; ++j) l[j] = 0.f;
  for (int p0 = 0; p0 < kparts; p0 += 4) {
    float v[J][4];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = lane + 32 * j;
        v[j][i] = e < r.E && p0 + i < kparts
                      ? __ldcg(parts + ((int64_t)(p0 + i) * r.T + t) * r.E + e) : 0.f;
      }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) l[j] += v[j][i];
  }
  if (gate_bias)
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (lane + 32 * j < r.E) l[j] += __ldg(gate_bias + lane + 32 * j);
  select_and_write<J>(l, t, r, lane);
}

// ---- units ------------------------------------------------------------------------
enum { kEnd = 0, kFC1 = 1, kFC2 = 2 };

// What a stage holds: part of a unit's columns.
struct alignas(16) FewStage {
  int kind;   // kEnd, kFC1, kFC2
  int last;   // the unit's last stage
  int entry;  // busy expert (index into the list)
  int pos0;   // first row of the unit in the sorted pair list
  int n;      // its rows (tokens)
  int r0;     // first weight row (FC1: first hidden unit)
  int k0, kc; // its columns in this stage
  int ks;     // slice of F (FC2)
  int pad[3];
};

constexpr int kMaxEntries = 257, kMaxPairs = kFewMaxT * 16, kMaxStages = 12;

struct FewCtl {
  uint64_t full_w[kMaxStages];  // weights (and the stage's description) are there
  uint64_t full_t[kMaxStages];  // token rows are there
  uint64_t told[kMaxStages];    // the stage's description is there
  uint64_t empty[kMaxStages], meet;
  alignas(16) FewStage st[kMaxStages];
  int abort;
  int pairs, units1, units2, fc2_writers;
  int ent_e[kMaxEntries];        // expert (E: the shared one)
  int ent_start[kMaxEntries];    // first sorted pair
  int ent_n[kMaxEntries];        // pairs
  int cum1[kMaxEntries + 1], cum2[kMaxEntries + 1];  // units before entry j
  int start[kMaxEntries];                // first sorted pair of an expert
  unsigned long long mask[kMaxEntries];  // tokens of an expert
  int4 part[9];                          // a 32-expert chunk's entries, pairs, sub-units, writers
  int idx[kMaxPairs];
  float prob[kMaxPairs];
  int16_t pos_of[kMaxPairs];     // sorted position of pair p, -1: dropped
  uint8_t tok_of[kMaxPairs + kFewMaxT];  // token of a sorted position
};

struct FewParams {
  // weights as (columns, rows of one half, halves of the experts); tokens, the
  // hidden values and their scales as (columns, rows)
  CUtensorMap w1, w2, w1s, w2s, x, act, act_s;
  FewArgs a;
  RouterArgs r;
  const float* parts;
  int kparts;
  int32_t* sync;
  const float* xs;
  void* hidden;      // bf16, or fp16 with hidden_s (MXFP4 weights)
  float* hidden_s;
  float* ypart;
  int S;            // rows of act and ypart: T K (+ T)
  int ksplit, stages;
  uint64_t wait_limit_ns;
};

// RT = 16 MT weight rows of a unit, NB = 8 NT tokens, NW consumer warps: MT of
// them share a slice of a stage's KC columns, one m-tile each.
template <bool W4_, int MT_, int NT_, int NW_, int KC_>
struct FewTile {
  static constexpr bool W4 = W4_;
  static constexpr int MT = MT_, NT = NT_, NW = NW_, KC = KC_;
  static constexpr int RT = 16 * MT;  // weight rows of a unit
  static constexpr int NB = 8 * NT;   // tokens of a unit
  static constexpr int KG = NW / MT, KW = KC / KG;  // slices and their columns
  // A stage holds KC / 256 boxes of 256 columns, rows one after the other.
  // bf16 rows are 512 bytes, unswizzled: two of a quarter-warp's eight 16-byte
  // loads meet in a bank, which the shared-memory bandwidth has room for.
  // MXFP4 rows are 128 bytes with the 128-byte swizzle, without conflicts.
  static constexpr int KB = 256, NKB = KC / KB;
  static constexpr int A_ROW = W4 ? 128 : 512, B_ROW = 512;
  static constexpr int A_BYTES = NKB * RT * A_ROW, B_BYTES = NKB * NB * B_ROW;
  static constexpr int SF = W4 ? 2 * (KC / 128) * mx::ATOM : 0;
  static constexpr int BS_ROW = W4 ? KC / 32 * 4 : 0;
  static constexpr int STAGE = (A_BYTES + B_BYTES + SF + NB * BS_ROW + 1023) / 1024 * 1024;
  static constexpr int RED_TOK = RT + 4;  // padded token stride of the meeting buffer
  static constexpr int RED = 2 * KG * NB * RED_TOK * 4;  // two units in turn
  static constexpr int THREADS = 32 * (NW + 2);
  static_assert(NW % MT == 0 && NW >= 8 && KW % (W4 ? 128 : 32) == 0, "whole scale words per warp");
};

// Warps that write the results of a unit of n tokens by `width` values, and of
// an expert's n tokens in units of nb.
MOE_HD int few_writers(int n, int width, int warps) {
  const int w = (n * width + 31) / 32;
  return w < warps ? w : warps;
}
MOE_HD int few_writers_of(int n, int nb, int width, int warps) {
  return n / nb * few_writers(nb, width, warps) + few_writers(n % nb, width, warps);
}

// Sorts the pairs by expert (tokens ascending) and lays out the units; every
// thread of the block calls it.  A token picks an expert at most once, so the
// tokens of an expert are a 64-bit mask: a pair's place is the number of set
// bits below its token, whatever the order the bits were set in.
template <class L>
__device__ void few_build_list(FewCtl& c, const moe_config_t& cf, int nrb1, int nrb2, int ksplit,
                               int* status) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, P = cf.T * cf.K;
  for (int p = threadIdx.x; p < P; p += L::THREADS) {
    const int e = c.idx[p];
    if (e < 0 || e >= cf.E) report(status, MOE_ERR_DEVICE_BOUNDS);
    else atomicOr(&c.mask[e], 1ull << (p / cf.K));
  }
  if (threadIdx.x == 0 && cf.n_shared) c.mask[cf.E] = ~0ull >> (64 - cf.T);
  __syncthreads();
  // a 32-expert chunk a warp; the shared expert is one more expert
  const int last = cf.E + (cf.n_shared ? 1 : 0), chunks = (last + 31) / 32;
  for (int ch = warp; ch < chunks; ch += L::NW + 2) {
    const int e = ch * 32 + lane;
    int n = e < last ? __popcll(c.mask[e]) : 0;
    if (e < cf.E && cf.capacity > 0) n = min(n, cf.capacity);
    int ie = n > 0 ? 1 : 0, ip = n, is = (n + L::NB - 1) / L::NB;
    int iw = few_writers_of(n, L::NB, L::RT, L::NW);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, ie, o), b = __shfl_up_sync(0xffffffffu, ip, o),
                d = __shfl_up_sync(0xffffffffu, is, o), f = __shfl_up_sync(0xffffffffu, iw, o);
      if (lane >= o) { ie += a; ip += b; is += d; iw += f; }
    }
    if (lane == 31) c.part[ch] = make_int4(ie, ip, is, iw);
    if (e < last) {  // within the chunk, for now
      c.start[e] = ip - n;
      c.cum1[e] = is - (n + L::NB - 1) / L::NB;
      c.cum2[e] = n > 0 ? ie - 1 : -1;
    }
  }
  __syncthreads();
  int4 all = make_int4(0, 0, 0, 0);
  for (int ch = 0; ch < chunks; ++ch) {
    const int4 v = c.part[ch];
    all.x += v.x; all.y += v.y; all.z += v.z; all.w += v.w;
  }
  // experts and their entries: read everything, then write
  constexpr int kPer = (kMaxEntries + L::THREADS - 1) / L::THREADS;
  int4 mine[kPer];  // entry, first pair, sub-units before, pairs
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x + i * L::THREADS;
    mine[i].x = -1;
    if (e >= last) continue;
    int4 b = make_int4(0, 0, 0, 0);
    for (int ch = 0; ch < e / 32; ++ch) {
      const int4 v = c.part[ch];
      b.x += v.x; b.y += v.y; b.z += v.z;
    }
    int n = __popcll(c.mask[e]);
    if (e < cf.E && cf.capacity > 0) n = min(n, cf.capacity);
    mine[i] = make_int4(c.cum2[e] < 0 ? -1 : b.x + c.cum2[e], b.y + c.start[e], b.z + c.cum1[e], n);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = threadIdx.x + i * L::THREADS, j = mine[i].x;
    if (e >= last) continue;
    c.start[e] = mine[i].y;
    if (j < 0) continue;
    c.ent_e[j] = e;
    c.ent_start[j] = mine[i].y;
    c.ent_n[j] = mine[i].w;
    c.cum1[j] = mine[i].z * nrb1;
    c.cum2[j] = mine[i].z * nrb2 * ksplit;
  }
  if (threadIdx.x == 0) {
    c.pairs = all.y;
    c.cum1[all.x] = c.units1 = all.z * nrb1;
    c.cum2[all.x] = c.units2 = all.z * nrb2 * ksplit;
    c.fc2_writers = all.w * nrb2 * ksplit;
  }
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += L::THREADS) {
    const int e = c.idx[p], t = p / cf.K;
    int pos = -1;
    if (e >= 0 && e < cf.E) {
      const int rank = __popcll(c.mask[e] & ((1ull << t) - 1));
      if (cf.capacity == 0 || rank < cf.capacity) {
        pos = c.start[e] + rank;
        c.tok_of[pos] = (uint8_t)t;
      }
    }
    c.pos_of[p] = (int16_t)pos;
  }
  if (cf.n_shared)
    for (int t = threadIdx.x; t < cf.T; t += L::THREADS) c.tok_of[c.start[cf.E] + t] = (uint8_t)t;
  __syncthreads();
}

MOE_D int ld_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
MOE_D void red_release(int32_t* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Orders this thread's global accesses through the generic proxy with those of
// bulk copies (the hidden values are written by stores and read by copies).
MOE_D void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// Waits until *p reaches v; bounded as mbar_wait is.
MOE_D bool wait_count(const int32_t* p, int v, const tc::WaitCtl& w) {
  if (ld_acquire(p) >= v) return true;
  const uint64_t t0 = tc::globaltimer_ns();
  for (int64_t i = 1;; ++i) {
    if (ld_acquire(p) >= v) return true;
    if ((i & 15) == 0) {
      if (w.abort && *w.abort) return false;
      if (tc::globaltimer_ns() - t0 > w.limit_ns) {
        report(w.status, MOE_ERR_TIMEOUT);
        if (w.abort) *w.abort = 1;
        return false;
      }
    }
  }
}

template <bool F16>
MOE_D void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                    uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight E2M1 codes -> eight fp16 values (exact), in order.
MOE_D void e2m1x8_to_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// A box of a 3-D tensor map (as tc::tma_load_2d).
MOE_D void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                       uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

MOE_D uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
MOE_D uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}

// Rows of FC1's output of a unit: hidden units (a SwiGLU unit holds the gate
// and up rows of RT / 2 of them, in groups of eight: each m-tile has eight
// gate rows above the matching eight up rows).
template <class L> MOE_HD int few_rows1(bool glu) { return glu ? L::RT / 2 : L::RT; }

template <class L>
__global__ void __launch_bounds__(L::THREADS, 1) few_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const moe_config_t& cf = p.a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool glu = cf.act == MOE_ACT_SWIGLU;
  uint8_t* ring = smem;
  float* red = reinterpret_cast<float*>(smem + (size_t)p.stages * L::STAGE);
  FewCtl& ctl = *reinterpret_cast<FewCtl*>(reinterpret_cast<uint8_t*>(red) + L::RED);
  const uint32_t ring0 = tc::smem_u32(ring);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      tc::mbar_init(tc::smem_u32(&ctl.full_w[s]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.full_t[s]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.told[s]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.empty[s]), L::NW);
    }
    tc::mbar_init(tc::smem_u32(&ctl.meet), L::NW);
    ctl.abort = 0;
    tc::fence_barrier_init();
    tc::fence_proxy_async_smem();
    for (const CUtensorMap* m : {&p.w1, &p.w2, &p.x, &p.act}) tc::prefetch_tensormap(m);
  }
  for (int e = threadIdx.x; e < kMaxEntries; e += L::THREADS) ctl.mask[e] = 0ull;
  pdl_wait();  // the partial logits, the cleared counters, the fp16 tokens
  int32_t* claim = p.sync;
  // the first unit's number comes while the experts are selected
  const int first_claim = threadIdx.x == 32 * L::NW ? atomicAdd(claim, 1) : 0;
  {
    RouterArgs r = p.r;
    r.topk_idx = ctl.idx;
    r.topk_prob = ctl.prob;
    for (int t = warp; t < cf.T; t += L::NW + 2) {
      if (cf.E <= 32) few_select_token<1>(p.parts, p.kparts, p.a.gate_bias, t, r, lane);
      else if (cf.E <= 64) few_select_token<2>(p.parts, p.kparts, p.a.gate_bias, t, r, lane);
      else if (cf.E <= 128) few_select_token<4>(p.parts, p.kparts, p.a.gate_bias, t, r, lane);
      else few_select_token<8>(p.parts, p.kparts, p.a.gate_bias, t, r, lane);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < cf.T * cf.K; i += L::THREADS) {
      if (p.a.idx_out) p.a.idx_out[i] = ctl.idx[i];
      if (p.a.prob_out) p.a.prob_out[i] = ctl.prob[i];
    }
  }
  const int nrb1 = ((glu ? 2 * cf.F : cf.F) + L::RT - 1) / L::RT;
  few_build_list<L>(ctl, cf, nrb1, (cf.h + L::RT - 1) / L::RT, p.ksplit, p.a.status);

  int32_t* done = p.sync + 2;   // warps that wrote FC1 results, per busy expert
  int32_t* done2 = p.sync + 1;  // warps that wrote FC2 results
  const int width1 = few_rows1<L>(glu);
  const int total = ctl.units1 + ctl.units2;
  tc::WaitCtl wc{p.a.status, &ctl.abort, p.wait_limit_ns, 0};
  tc::WaitCtl wdrain{p.a.status, nullptr, 1000000000ull, 0};

  if (warp == L::NW) {
    // ================= weights =================
    if (lane == 0) {
      int stage = 0, j1 = 0, j2 = 0;
      uint32_t phase = 0, issued = 0, issued_par = 0;
      int next = first_claim;
      bool ok = true;
      while (ok) {
        const int u = next;
        if (u < total) next = atomicAdd(claim, 1);  // the next unit, while this one streams
        FewStage st{};
        int kbeg = 0, kend = 1, cols = 0, nrows = 0;
        const CUtensorMap* map = nullptr;
        const uint8_t* sf = nullptr;
        int half0 = 0;  // the map's third coordinate
        bool pairs_of_rows = false;
        if (u < total) {
          int j;
          if (u < ctl.units1) {
            while (ctl.cum1[j1 + 1] <= u) ++j1;
            j = j1;
            const int sub = (ctl.ent_n[j] + L::NB - 1) / L::NB, loc = u - ctl.cum1[j];
            st.kind = kFC1;
            st.r0 = loc / sub * few_rows1<L>(glu);
            st.pos0 = loc % sub * L::NB;
            nrows = glu ? 2 * cf.F : cf.F;
            kend = cols = cf.h;
            pairs_of_rows = glu;
          } else {
            const int u2 = u - ctl.units1;
            while (ctl.cum2[j2 + 1] <= u2) ++j2;
            j = j2;
            const int sub = (ctl.ent_n[j] + L::NB - 1) / L::NB, loc = u2 - ctl.cum2[j];
            const int rest = loc / sub;
            st.kind = kFC2;
            st.ks = rest % p.ksplit;
            st.r0 = rest / p.ksplit * L::RT;
            st.pos0 = loc % sub * L::NB;
            nrows = cf.h;
            cols = cf.F;
            const int nst = (cf.F + L::KC - 1) / L::KC;
            kbeg = nst * st.ks / p.ksplit * L::KC;
            kend = min(cf.F, nst * (st.ks + 1) / p.ksplit * L::KC);
          }
          st.entry = j;
          st.n = min(L::NB, ctl.ent_n[j] - st.pos0);
          st.pos0 += ctl.ent_start[j];
          const int e = ctl.ent_e[j];
          const bool shared = e == cf.E;
          map = st.kind == kFC1 ? (shared ? &p.w1s : &p.w1) : (shared ? &p.w2s : &p.w2);
          half0 = shared ? 0 : e * (pairs_of_rows ? 2 : 1);
          if (L::W4) {
            const FewWeights& W = st.kind == kFC1 ? p.a.w1 : p.a.w2;
            sf = shared ? W.ws_sf
                        : W.sf + (int64_t)e * (nrows / 128) * (cols / 128) * mx::ATOM;
          }
        }
        for (int k0 = kbeg; k0 < kend; k0 += L::KC) {
          if (!tc::mbar_wait(tc::smem_u32(&ctl.empty[stage]), phase ^ 1, wc)) { ok = false; break; }
          const uint32_t fb = tc::smem_u32(&ctl.full_w[stage]);
          st.kc = min(L::KC, kend - k0);
          st.k0 = k0;
          st.last = k0 + L::KC >= kend;
          ctl.st[stage] = st;
          const int nkb = (st.kc + L::KB - 1) / L::KB;
          const uint32_t sf_bytes = L::W4 ? st.kc / 128 * mx::ATOM : 0;
          const uint32_t tx = nkb * L::RT * L::A_ROW + sf_bytes * (pairs_of_rows ? 2 : 1);
          tc::mbar_arrive_expect_tx(fb, st.kind == kEnd ? 0 : tx);
          tc::mbar_arrive(tc::smem_u32(&ctl.told[stage]));
          if (st.kind == kEnd) {
            issued &= ~(1u << stage);  // its copies are consumed, its barrier a phase further
            ok = false;
            break;
          }
          const uint32_t a_dst = ring0 + stage * L::STAGE;
          for (int b = 0; b < nkb; ++b)
            tma_load_3d(a_dst + b * L::RT * L::A_ROW, map, (k0 + b * L::KB) / (L::W4 ? 2 : 1),
                        st.r0, half0, fb);
          if (L::W4) {  // the scales of the unit's rows: atoms of their 128-row tile
            const uint32_t sf_dst = a_dst + L::A_BYTES + L::B_BYTES;
            for (int i = 0; i < (pairs_of_rows ? 2 : 1); ++i) {
              const int row = st.r0 + i * cf.F;
              tc::bulk_load(sf_dst + i * (L::SF / 2),
                            sf + ((int64_t)(row / 128) * (cols / 128) + k0 / 128) * mx::ATOM,
                            sf_bytes, fb);
            }
          }
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == p.stages) { stage = 0; phase ^= 1; }
        }
      }
      for (int s = 0; s < p.stages; ++s)
        if ((issued >> s) & 1u)
          tc::mbar_wait(tc::smem_u32(&ctl.full_w[s]), (issued_par >> s) & 1u, wdrain);
    }
    __syncwarp();
  } else if (warp == L::NW + 1) {
    // ================= tokens =================
    if (lane == 0) {
      int stage = 0, ready = -1;
      uint32_t phase = 0, issued = 0, issued_par = 0;
      for (;;) {
        if (!tc::mbar_wait(tc::smem_u32(&ctl.told[stage]), phase, wc)) break;
        const FewStage st = ctl.st[stage];
        if (st.kind == kEnd) break;
        if (st.kind == kFC2 && ready != st.entry) {  // the expert's hidden values
          const int writers = few_writers_of(ctl.ent_n[st.entry], L::NB, width1, L::NW);
          if (!wait_count(done + st.entry, nrb1 * writers, wc)) break;
          fence_proxy_async_global();
          ready = st.entry;
        }
        const uint32_t fb = tc::smem_u32(&ctl.full_t[stage]);
        const uint32_t b_dst = ring0 + stage * L::STAGE + L::A_BYTES;
        const int nkb = (st.kc + L::KB - 1) / L::KB;
        if (st.kind == kFC1) {  // tokens anywhere: four rows a load, the last one repeated
          const int n4 = (st.n + 3) / 4;
          tc::mbar_arrive_expect_tx(fb, nkb * n4 * 4 * L::B_ROW);
          for (int i = 0; i < n4; ++i) {
            int row[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) row[r] = ctl.tok_of[st.pos0 + min(4 * i + r, st.n - 1)];
            for (int b = 0; b < nkb; ++b)
              tc::tma_gather4(b_dst + (b * L::NB + 4 * i) * L::B_ROW, &p.x, st.k0 + b * L::KB,
                              row[0], row[1], row[2], row[3], fb);
          }
        } else {  // rows of the sorted list: boxes of eight
          const int n8 = (st.n + 7) / 8;
          tc::mbar_arrive_expect_tx(fb, n8 * (nkb * 8 * L::B_ROW + 8 * L::BS_ROW));
          for (int i = 0; i < n8; ++i) {
            for (int b = 0; b < nkb; ++b)
              tc::tma_load_2d(b_dst + (b * L::NB + 8 * i) * L::B_ROW, &p.act, st.k0 + b * L::KB,
                              st.pos0 + 8 * i, fb);
            if (L::W4)
              tc::tma_load_2d(b_dst + L::B_BYTES + L::SF + 8 * i * L::BS_ROW, &p.act_s, st.k0 / 32,
                              st.pos0 + 8 * i, fb);
          }
        }
        issued |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        if (++stage == p.stages) { stage = 0; phase ^= 1; }
      }
      for (int s = 0; s < p.stages; ++s)
        if ((issued >> s) & 1u)
          tc::mbar_wait(tc::smem_u32(&ctl.full_t[s]), (issued_par >> s) & 1u, wdrain);
    }
    __syncwarp();
  } else {
    // ================= consumers =================
    const int g = lane >> 2, q = lane & 3;
    int stage = 0;
    uint32_t phase = 0;
    const int mi = warp % L::MT, ki = warp / L::MT;  // its m-tile and slice of the columns
    float acc[L::NT][4];
#pragma unroll
    for (int n = 0; n < L::NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    // A barrier of the consumer warps that gives up like every other wait (a
    // hardware barrier would hang if one warp had left after a timeout).
    uint32_t meet_par = 0;
    auto meet = [&]() -> bool {
      const uint32_t b = tc::smem_u32(&ctl.meet);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(b);
      const bool go = tc::mbar_wait(b, meet_par, wc);
      meet_par ^= 1;
      return go;
    };
    int unit = 0;  // units this block has finished
    bool finish = false;
    for (;;) {
      if (!tc::mbar_wait(tc::smem_u32(&ctl.full_w[stage]), phase, wc)) break;
      const FewStage st = ctl.st[stage];
      if (st.kind == kEnd) { finish = true; break; }
      if (!tc::mbar_wait(tc::smem_u32(&ctl.full_t[stage]), phase, wc)) break;
      const uint32_t a_s = ring0 + stage * L::STAGE, b_s = a_s + L::A_BYTES;
      const uint32_t sf_s = b_s + L::B_BYTES, bs_s = sf_s + L::SF;
      const int ntiles = (st.n + 7) >> 3;
      // rows of an m-tile's two halves: gate and up rows lie in two blocks
      const bool two = glu && st.kind == kFC1;
      const int m_row = (two ? 8 : 16) * mi + g, hi_row = two ? 8 * L::MT : 8;
      uint32_t sw0 = 0, sw1 = 0;  // the scales of 128 columns of the lane's two rows
#pragma unroll
      for (int c = 0; c < L::KW / 32; ++c) {
        const int kb = ki * L::KW + c * 32;  // 32 columns (zeros past the matrix)
        if (kb >= st.kc) break;
        uint32_t b[L::NT][4];
#pragma unroll
        for (int n = 0; n < L::NT; ++n) {
          if (n < ntiles) {
            const int row = min(8 * n + g, st.n - 1);
            const uint4 v = lds128(b_s + (kb / L::KB * L::NB + row) * L::B_ROW + (kb % L::KB + 8 * q) * 2);
            b[n][0] = v.x; b[n][1] = v.y; b[n][2] = v.z; b[n][3] = v.w;
          }
        }
        if constexpr (!L::W4) {
          const uint32_t at = a_s + (kb / L::KB * L::RT + m_row) * L::A_ROW + (kb % L::KB + 8 * q) * 2;
          const uint4 lo = lds128(at), hi = lds128(at + hi_row * L::A_ROW);
#pragma unroll
          for (int n = 0; n < L::NT; ++n)
            if (n < ntiles) {
              mma16816<false>(acc[n], lo.x, hi.x, lo.y, hi.y, b[n][0], b[n][1]);
              mma16816<false>(acc[n], lo.z, hi.z, lo.w, hi.w, b[n][2], b[n][3]);
            }
        } else {
          // the fp16 products of one 32-column block, then its scales in fp32
          if (c % 4 == 0) {
            const int i0 = (st.r0 + m_row) & 127, i1 = two ? i0 : i0 + 8;
            const uint32_t at = sf_s + kb / 128 * mx::ATOM;
            sw0 = lds32(at + 16 * (i0 & 31) + 4 * (i0 >> 5));
            sw1 = lds32(at + (two ? L::SF / 2 : 0) + 16 * (i1 & 31) + 4 * (i1 >> 5));
          }
          uint32_t lo[4], hi[4];
          // 16 bytes hold the block's codes of a row; the swizzle moves them by
          // the row's place in its group of eight, which is g
          const uint32_t at = a_s + (kb / L::KB * L::RT + m_row) * L::A_ROW +
                              (((kb % L::KB) / 32) ^ g) * 16 + 4 * q;
          e2m1x8_to_f16(lds32(at), lo);
          e2m1x8_to_f16(lds32(at + hi_row * L::A_ROW), hi);
          const float s0 = mx::e8m0_value(sw0 >> (8 * (c & 3)) & 255u);
          const float s1 = mx::e8m0_value(sw1 >> (8 * (c & 3)) & 255u);
#pragma unroll
          for (int n = 0; n < L::NT; ++n)
            if (n < ntiles) {
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma16816<true>(d, lo[0], hi[0], lo[1], hi[1], b[n][0], b[n][1]);
              mma16816<true>(d, lo[2], hi[2], lo[3], hi[3], b[n][2], b[n][3]);
              if (st.kind == kFC2) {  // the tokens' own scales of these columns
                const float b0 = __uint_as_float(lds32(bs_s + min(8 * n + 2 * q, st.n - 1) * L::BS_ROW + kb / 32 * 4));
                const float b1 = __uint_as_float(lds32(bs_s + min(8 * n + 2 * q + 1, st.n - 1) * L::BS_ROW + kb / 32 * 4));
                d[0] *= b0; d[1] *= b1; d[2] *= b0; d[3] *= b1;
              }
              acc[n][0] = fmaf(d[0], s0, acc[n][0]);
              acc[n][1] = fmaf(d[1], s0, acc[n][1]);
              acc[n][2] = fmaf(d[2], s1, acc[n][2]);
              acc[n][3] = fmaf(d[3], s1, acc[n][3]);
            }
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.empty[stage]));
      if (++stage == p.stages) { stage = 0; phase ^= 1; }
      if (!st.last) continue;

      // ---- the unit's end: the warps' sums meet ----
      // One meeting a unit: the buffers alternate, so the next unit's sums go
      // elsewhere while this unit's are read, and the unit after that comes
      // past the next meeting.  The results are written by the first warps,
      // counted from a warp that moves on with every unit, so that the wait for
      // the stores' way to the L2 falls on another warp each time.
      float* mine = red + (unit & 1) * (L::RED / 8);
#pragma unroll
      for (int n = 0; n < L::NT; ++n) {
        if (n < ntiles) {
          float* d = mine + (ki * L::NB + 8 * n + 2 * q) * L::RED_TOK + 16 * mi + g;
          d[0] = acc[n][0];
          d[L::RED_TOK] = acc[n][1];
          d[8] = acc[n][2];
          d[L::RED_TOK + 8] = acc[n][3];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
      }
      if (!meet()) break;
      auto sum = [&](int tok, int row) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < L::KG; ++w) v += mine[(w * L::NB + tok) * L::RED_TOK + row];
        return v;
      };
      const int rw = (warp + L::NW - unit % L::NW) % L::NW;  // place among the writers
      ++unit;
      const int width = st.kind == kFC1 ? width1 : L::RT;
      if (rw >= few_writers(st.n, width, L::NW)) continue;
      const int items = st.n * width;
      if (st.kind == kFC1) {
        const int e = ctl.ent_e[st.entry];
        for (int i0 = rw * 32; i0 < items; i0 += 32 * L::NW) {  // whole warps (shuffles below)
          const int i = i0 + lane;
          const int tok = min(i / width, st.n - 1), f = i % width;
          const bool valid = i < items && st.r0 + f < cf.F;
          const int pos = st.pos0 + tok;
          float v;
          const float s = L::W4 ? __ldg(p.xs + ctl.tok_of[pos]) : 1.f;
          if (glu) {
            const int row = f / 8 * 16 + (f & 7);
            v = silu_f(sum(tok, row) * s) * (sum(tok, row + 8) * s);
          } else {
            float z = sum(tok, f);
            if (cf.has_bias && e < cf.E && valid) z += to_f32(p.a.b1[(int64_t)e * cf.F + st.r0 + f]);
            v = gelu_f(z);
          }
          const int64_t at = (int64_t)pos * cf.F + st.r0 + f;
          if constexpr (L::W4) {
            // one token's 32 hidden units are a warp's: fp16 with a power-of-two
            // scale of their own (11 significant bits, half a step 2^-11 of
            // values down to 2^-29 of the largest)
            uint32_t m = __float_as_uint(v) & 0x7fffffffu;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float bsc = f16_block_scale(m);
            if (valid) {
              static_cast<__half*>(p.hidden)[at] = __float2half_rn(v * (1.f / bsc));
              if (f == 0) p.hidden_s[(int64_t)pos * (cf.F / 32) + st.r0 / 32] = bsc;
            }
          } else {
            // bf16, as moe_layer_fwd keeps them: FC2's operand type
            if (valid) static_cast<__nv_bfloat16*>(p.hidden)[at] = __float2bfloat16_rn(v);
          }
        }
        fence_proxy_async_global();
        __syncwarp();
        if (lane == 0) red_release(done + st.entry, 1);
      } else {
        for (int i = rw * 32 + lane; i < items; i += 32 * L::NW) {
          const int tok = i / L::RT, row = i % L::RT;
          if (st.r0 + row < cf.h)
            __stcg(p.ypart + ((int64_t)st.ks * p.S + st.pos0 + tok) * cf.h + st.r0 + row, sum(tok, row));
        }
        __syncwarp();
        if (lane == 0) red_release(done2, 1);
      }
    }
    // ---- combine: every block's share, two columns a thread ----
    int all = 0;
    if (finish && lane == 0) all = wait_count(done2, ctl.fc2_writers, wc);
    if (__shfl_sync(0xffffffffu, all, 0)) {
      ld_acquire(done2);  // every lane's own
      const int64_t pairs2 = (int64_t)cf.T * cf.h / 2;
      const int slots = cf.K + (cf.n_shared ? 1 : 0);
      for (int64_t i = ((int64_t)warp * gridDim.x + blockIdx.x) * 32 + lane; i < pairs2;
           i += (int64_t)gridDim.x * L::NW * 32) {
        const int t = (int)(2 * i / cf.h), r = (int)(2 * i - (int64_t)t * cf.h);
        float2 y = make_float2(0.f, 0.f);
        constexpr int kBatch = 4;  // slots whose loads go out together
        for (int k0 = 0; k0 < slots; k0 += kBatch) {
          float2 o[kBatch];
          float w[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int k = k0 + j;
            const bool shared = k == cf.K;
            const int pr = t * cf.K + min(k, cf.K - 1);
            const int pos = shared ? ctl.pairs - cf.T + t : ctl.pos_of[pr];
            const bool there = k < slots && pos >= 0;  // else past the end, or dropped
            w[j] = shared ? 1.f : ctl.prob[pr];
            o[j] = make_float2(0.f, 0.f);
            if (!there) w[j] = 0.f;
            if (there && cf.has_bias && !shared) {
              const __nv_bfloat16* b = p.a.b2 + (int64_t)ctl.idx[pr] * cf.h + r;
              o[j] = make_float2(to_f32(b[0]), to_f32(b[1]));
            }
            if (there) {
              const float* src = p.ypart + (int64_t)pos * cf.h + r;
              const int64_t step = (int64_t)p.S * cf.h;
              for (int s = 0; s < p.ksplit; ++s) {
                const float2 v = __ldcg(reinterpret_cast<const float2*>(src + s * step));
                o[j].x += v.x;
                o[j].y += v.y;
              }
            }
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            y.x = fmaf(w[j], o[j].x, y.x);
            y.y = fmaf(w[j], o[j].y, y.y);
          }
        }
        *reinterpret_cast<__nv_bfloat162*>(p.a.y + (int64_t)t * cf.h + r) = __floats2bfloat162_rn(y.x, y.y);
      }
    }
  }
  __syncthreads();
}

// A map of up to three dimensions, zero fill outside.
bool few_encode(CUtensorMap* m, CUtensorMapDataType type, int elem, const void* base, int rank,
                uint64_t cols, uint64_t rows, uint64_t halves, int box_cols, int box_rows,
                int box_halves, bool swizzle) {
  tc::EncodeTiledFn fn = tc::encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cols, rows, halves};
  const cuuint64_t strides[2] = {cols * elem, cols * rows * elem};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, (cuuint32_t)box_halves};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, type, rank, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class L>
cudaError_t few_launch(FewParams& p, const __half* xh, cudaStream_t s) {
  const moe_config_t& c = p.a.c;
  const bool glu = c.act == MOE_ACT_SWIGLU;
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const auto u16 = CU_TENSOR_MAP_DATA_TYPE_UINT16;
  // weights: rows of F or h, the gate and up halves of an expert one after the other
  auto weights = [&](CUtensorMap* m, const void* w, uint64_t cols, uint64_t rows, uint64_t halves,
                     int pair) {
    return L::W4 ? few_encode(m, u8, 1, w, 3, cols / 2, rows, halves, L::A_ROW, L::RT / pair, pair, true)
                 : few_encode(m, u16, 2, w, 3, cols, rows, halves, L::KB, L::RT / pair, pair, false);
  };
  const int pair = glu ? 2 : 1;
  bool ok = weights(&p.w1, p.a.w1.w, c.h, c.F, (uint64_t)c.E * pair, pair) &&
            weights(&p.w2, p.a.w2.w, c.F, c.h, c.E, 1);
  if (c.n_shared)
    ok = ok && weights(&p.w1s, p.a.w1.ws, c.h, c.F, pair, pair) &&
         weights(&p.w2s, p.a.w2.ws, c.F, c.h, 1, 1);
  const void* x = L::W4 ? static_cast<const void*>(xh) : p.a.x;
  ok = ok && few_encode(&p.x, u16, 2, x, 2, c.h, c.T, 1, L::KB, 1, 1, false) &&
       few_encode(&p.act, u16, 2, p.hidden, 2, c.F, p.S, 1, L::KB, 8, 1, false);
  if (L::W4)
    ok = ok && few_encode(&p.act_s, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, p.hidden_s, 2, c.F / 32, p.S,
                          1, L::KC / 32, 8, 1, false);
  if (!ok) return cudaErrorInvalidValue;
  constexpr int kMost = 227 * 1024;
  const int fixed = 1024 + L::RED + (int)sizeof(FewCtl);  // 1024: the ring's alignment
  int stages = (kMost - fixed) / L::STAGE;
  if (stages > kMaxStages) stages = kMaxStages;
  p.stages = stages;
  const int smem = stages * L::STAGE + fixed;
  cudaError_t e = cudaFuncSetAttribute(few_kernel<L>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.a.sms);
  cfg.blockDim = dim3(L::THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<L>, p);
}

}  // namespace

cudaError_t launch_few(const FewArgs& a, bool mxfp4, cudaStream_t s) {
  const moe_config_t& c = a.c;
  const FewLayout L = few_layout(c);
  FewParams p{};
  p.a = a;
  p.parts = reinterpret_cast<float*>(a.ws + L.parts);
  p.kparts = few_kparts(c);
  p.sync = reinterpret_cast<int32_t*>(a.ws + L.sync);
  __half* xh = reinterpret_cast<__half*>(a.ws + L.xh);
  p.xs = reinterpret_cast<float*>(a.ws + L.xs);
  p.hidden = a.ws + L.a;
  p.hidden_s = reinterpret_cast<float*>(a.ws + L.as);
  p.ypart = reinterpret_cast<float*>(a.ws + L.ypart);
  p.S = c.T * c.K + (c.n_shared ? c.T : 0);
  p.ksplit = few_ksplit(c);
  p.wait_limit_ns = 2000000000ull;
  p.r.T = c.T; p.r.E = c.E; p.r.K = c.K; p.r.h = c.h; p.r.score = c.score;
  p.r.renorm = (c.flags & MOE_FLAG_RENORM) != 0;
  p.r.force_balance = (c.flags & MOE_FLAG_FORCE_BALANCE) != 0;
  p.r.sel_bias = a.sel_bias;
  const int route_blocks = (int)ceil_div((int64_t)c.E * p.kparts, 8);
  few_router_kernel<<<route_blocks + (mxfp4 ? c.T : 0), 256, 0, s>>>(
      a.x, a.w_r, c.T, c.E, c.h, p.kparts, const_cast<float*>(p.parts), route_blocks,
      xh, const_cast<float*>(p.xs), p.sync, (int)few_sync_words(c));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (mxfp4)
    return c.T <= 8 ? few_launch<FewTile<true, 4, 1, 16, 512>>(p, xh, s)
                    : few_launch<FewTile<true, 4, 2, 16, 512>>(p, xh, s);
  if (c.T <= 8) return few_launch<FewTile<false, 2, 1, 8, 512>>(p, xh, s);
  if (c.T <= 16) return few_launch<FewTile<false, 2, 2, 8, 512>>(p, xh, s);
  return few_launch<FewTile<false, 2, 4, 8, 256>>(p, xh, s);
}

}  // namespace moe
