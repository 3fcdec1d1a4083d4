// The whole MoE layer for a few tokens (T <= 64): the call of a decoding step.
//
//   l = W_r x (+ b_r), top-K and p as in the layer pass;
//   y_t = sum_k p_tk E_{e_tk}(x_t)  (+ S(x_t)).
//
// The expert weights are the traffic: each busy expert's matrices are read
// from HBM for a handful of rows.  bf16 weights, or MXFP4 weights (E2M1 codes
// with one E8M0 scale per 32 columns).
//
// Three launches, each started while the one before drains (programmatic
// dependent launch).  few_router_kernel writes partial logits (and, for MXFP4
// weights, the tokens as E2M1 parts); few_select_kernel adds them and selects, a block
// a token.  few_kernel does the rest, one block per SM:
//   every block sorts the (token, slot) pairs by expert (the same list
//   everywhere), then takes units of work from one counter: first all of FC1's
//   units (an expert, a block of its rows), then FC2's (an expert, a block of
//   rows of h, a slice of F).  An FC2 unit waits until its expert's FC1 units
//   are done.  Units are taken in order, so every FC1 unit that an FC2 unit
//   waits for belongs to a block that already runs and waits for nothing: no
//   block needs any other to become resident.
//   When all FC2 units are done every block adds its share of the slots'
//   results, in a fixed order, and writes y.
// Within a block: two producer warps stream the unit's weight rows and the
// expert's token rows through a ring of shared-memory stages (256 columns a
// stage, TMA boxes of many rows: a copy per row costs its issuing warp about
// 95 cycles whatever its size, which held an earlier form of this kernel at 10 bytes a
// cycle and SM).  The weight producer runs ahead of the arithmetic, into the
// next unit and from FC1 into FC2, so that HBM stays busy across unit and
// phase borders; only the token producer waits for FC1's results.  NW consumer
// warps split a stage's columns and multiply with m16n8k16 tensor-core
// instructions, weight rows as M, tokens as N: the weights are read once from
// HBM however many tokens share them, and a product with up to 16 tokens costs
// less than the loads.  (Beside bf16 weights the mma rate is not what bounds
// this kernel, and 64-row units balance the SMs better than tcgen05's 128.
// MXFP4 weights have a kernel of their own, few_mx_kernel, below.)
// At a unit's end the warps' sums meet in shared memory, in warp order.
//
// "Scalable Training of Mixture-of-Experts Models with Megatron Core" (review),
// §2.1 (the four steps), §2.2 (router); the same formulas and options as
// moe_layer_fwd.
#include <cuda_fp4.h>

#include <type_traits>

#include "few.cuh"
#include "mx.cuh"
#include "router_select.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

MOE_D void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
MOE_D void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---- E2M1 parts --------------------------------------------------------------------
// A block of 32 values, four a lane of eight lanes, as a sum of kParts E2M1 blocks,
// each with a scale of its own: part 0 rounds v / s, s the power of two that puts
// the largest magnitude into [2, 4), and each further part what the ones before
// left.  There E2M1's steps are at most 1, so part 0 leaves at most s / 2; at s / 4
// that is at most 2, steps of 1/2, and from then on every part takes three bits: six
// leave at most s / 65536, 2^-17 of the block's largest value (a bf16 number's own half
// step is 2^-8 of it), or 2^-129 where the scales end at 2^-127.  What a part leaves is
// kept in units of that part's scale, where every difference is exact and none overflows
// (4 s is infinite for a block above 3.5 2^126).  A block with an infinity or a NaN gets
// the NaN scale.  code[i]: the lane's four codes of part i, the first lowest.
MOE_D void e2m1_parts(float (&v)[4], uint32_t (&code)[kParts], uint32_t (&scale)[kParts]) {
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int e = (int)(m >> 23);
  int x = max(e - 1, 0);
  const float inv = __uint_as_float((uint32_t)(254 - x) << 23);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] *= inv;
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    scale[i] = e == 255 ? (i == 0 ? 255u : 0u) : (uint32_t)x;
    uint32_t c = 0u;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      c |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(v[2 * j], v[2 * j + 1]), __NV_E2M1,
                                              cudaRoundNearest) << (8 * j);
    code[i] = e == 255 ? 0u : c;
    const int next = max(e - 1 - (3 * i + 2), 0);
    const float up = __uint_as_float((uint32_t)(127 + x - next) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t b = c >> (4 * j);
      v[j] = (v[j] - __uint_as_float((b & 8u) << 28 | (b & 7u) << 22) * 0x1p126f) * up;
    }
    x = next;
  }
}

// A token's columns b0 .. b1 - 1 (blocks of 32) as parts: four blocks a warp.
__device__ void few_split_token(const __nv_bfloat16* __restrict__ x, int h, int b0, int b1,
                                uint8_t* __restrict__ q, uint8_t* __restrict__ sf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 3, l = lane & 7;
  for (int b = b0 + 4 * warp; b < b1; b += blockDim.x / 8) {  // (b1 - b0 is a multiple of four)
    const __nv_bfloat162* src = reinterpret_cast<const __nv_bfloat162*>(x + (b + g) * 32 + 4 * l);
    const float2 lo = __bfloat1622float2(src[0]), hi = __bfloat1622float2(src[1]);
    float v[4] = {lo.x, lo.y, hi.x, hi.y};
    uint32_t code[kParts], scale[kParts];
    e2m1_parts(v, code, scale);
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      *reinterpret_cast<uint16_t*>(q + (int64_t)i * (h / 2) + (b + g) * 16 + 2 * l) = (uint16_t)code[i];
      if (l == 0) sf[(int64_t)i * (h / 32) + b + g] = (uint8_t)scale[i];
    }
  }
}

// ---- route ----------------------------------------------------------------------
// Partial logits: one warp per (expert, slice of h, TOK tokens).  x is exact in
// fp32 and the products and sums are fp32, each lane over its own columns, the
// lanes added as a tree.  The blocks past the router's split kSplitCols columns of
// a token each; block 0 clears the counters of few_kernel.
constexpr int kSplitCols = 1024;
template <int TOK>
__global__ void __launch_bounds__(256)
    few_router_kernel(const __nv_bfloat16* __restrict__ x, const float* __restrict__ w_r, int T,
                      int E, int h, int kparts, float* __restrict__ parts, int route_blocks,
                      uint8_t* xq, uint8_t* xs, int32_t* sync, int sync_words) {
  pdl_trigger();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < sync_words; i += blockDim.x) sync[i] = 0;
  if ((int)blockIdx.x >= route_blocks) {
    const int per = (h + kSplitCols - 1) / kSplitCols, i = blockIdx.x - route_blocks;
    const int t = i / per, b0 = i % per * (kSplitCols / 32);
    few_split_token(x + (int64_t)t * h, h, b0, min(b0 + kSplitCols / 32, h / 32),
                    xq + (int64_t)t * kParts * (h / 2), xs + (int64_t)t * kParts * (h / 32));
    return;
  }
  const int unit = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (unit >= E * kparts * (int)ceil_div(T, TOK)) return;
  const int e = unit % E, part = unit / E % kparts, t0 = unit / (E * kparts) * TOK;
  const int vecs = h / 8;  // 16-byte vectors of x
  const int v0 = (int)((int64_t)vecs * part / kparts), v1 = (int)((int64_t)vecs * (part + 1) / kparts);
  const float* w = w_r + (int64_t)e * h;
  {
    float acc[TOK];
#pragma unroll
    for (int j = 0; j < TOK; ++j) acc[j] = 0.f;
    for (int v = v0 + lane; v < v1; v += 32) {
      const Vec<float> wa = ldg16(w + v * 8), wb = ldg16(w + v * 8 + 4);
#pragma unroll
      for (int j = 0; j < TOK; ++j) {
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
    for (int j = 0; j < TOK; ++j) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
      if (lane == 0 && t0 + j < T) parts[((int64_t)part * T + t0 + j) * E + e] = acc[j];
    }
  }
}

// The full selection on one token's logits (router_select.cuh), by a warp; out of
// line, for the rare token whose fp32 sigmoid keys are too close to rank.
__device__ __noinline__ void few_select_exact(const float* logit, int t, RouterArgs r, int lane) {
  float l[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) l[j] = lane + 32 * j < r.E ? logit[lane + 32 * j] : 0.f;
  select_and_write<8>(l, t, r, lane);
}

// Adds the partial logits and selects: a block a token, a thread an expert, with
// select_and_write's choices.  (A warp a token with the logits in registers, as the
// large router has it, took 9.5 us for one token of 64 experts and 16 us of 256.)
// The biases are read before the partial logits are there: the router, a plain
// launch, runs, so what came before it on the stream is done.  The results are
// written kFewCopies times: each block of few_kernel reads one of the copies.
__global__ void __launch_bounds__(256)
    few_select_kernel(const float* __restrict__ parts, int kparts, const float* gate_bias,
                      RouterArgs r, int pairs_pad, int32_t* idx_out, float* prob_out) {
  __shared__ float s_logit[256];
  __shared__ __align__(16) uint32_t s_key[256];
  __shared__ int s_sel[32];
  __shared__ float s_prob[16];
  const unsigned FULL = 0xffffffffu;
  const int e = threadIdx.x, t = blockIdx.x, lane = threadIdx.x & 31;
  constexpr int kBatch = 8;
  const bool sig = r.score == MOE_SCORE_SIGMOID;
  pdl_trigger();
  const float gb = gate_bias && e < r.E ? __ldg(gate_bias + e) : 0.f;
  const float sb = r.sel_bias && e < r.E ? __ldg(r.sel_bias + e) : 0.f;
  pdl_wait();
  float l = 0.f;
  uint32_t key = 0u;  // order-preserving; 0 past E and for what was picked
  if (e < r.E) {
    for (int p0 = 0; p0 < kparts; p0 += kBatch) {  // all of a batch under way, added in order
      float v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        v[i] = p0 + i < kparts ? __ldcg(parts + ((int64_t)(p0 + i) * r.T + t) * r.E + e) : 0.f;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) l += v[i];
    }
    l += gb;
    const float fast = sig ? sigmoid_f(l) : l;  // selection_key_fast
    key = max(sortable_key(r.sel_bias ? __fadd_rn(fast, sb) : fast), 1u);
  }
  s_logit[e] = l;
  s_key[e] = key;
  __syncthreads();
  if (e >= 32) return;
  // One warp picks: the largest key of its 256, the lowest expert among equals, and
  // again without it.  (Each thread counting the keys above its own, bound by the
  // shared-memory reads: 4.8 us for the kernel with 256 experts and one token; this
  // 2.7.)  The (K+1)-th too: its gap is looked at below.
  int my = 0;
  if (r.force_balance) {
    my = lane < r.K ? (int)(((int64_t)t * r.K + lane) % r.E) : 0;
  } else {
    uint32_t k[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) k[j] = s_key[lane + 32 * j];
#pragma unroll 1
    for (int i = 0; i < min(r.K + 1, r.E); ++i) {
      const uint32_t best = __reduce_max_sync(FULL, max(max(max(k[0], k[1]), max(k[2], k[3])),
                                                        max(max(k[4], k[5]), max(k[6], k[7]))));
      unsigned at = 256u;
#pragma unroll
      for (int j = 7; j >= 0; --j)
        if (k[j] == best) at = lane + 32 * j;
      at = __reduce_min_sync(FULL, at);
      if (lane == i) my = (int)at;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at == lane + 32 * j) k[j] = 0u;
    }
  }
  if (lane < r.K) s_sel[lane] = my;
  __syncwarp();
  const int before = __shfl_up_sync(FULL, my, 1);
  bool close = false;  // sigmoid: two of the best K + 1 keys within their error bound
  if (sig && !r.force_balance && lane >= 1 && lane < min(r.K + 1, r.E)) {
    const float prev = from_sortable_key(s_key[before]), cur = from_sortable_key(s_key[my]);
    close = !(prev - cur > 4e-6f * (1.f + fabsf(prev) + fabsf(cur)));
  }
  if (__any_sync(FULL, close)) {
    RouterArgs w = r;  // the results in shared memory, as below
    w.topk_idx = s_sel - (int64_t)t * r.K;
    w.topk_prob = s_prob - (int64_t)t * r.K;
    few_select_exact(s_logit, t, w, lane);
  } else {
    const bool active = lane < r.K;
    const float ml = s_logit[my];
    float m = 0.f, num, den = 0.f;
    if (!sig) {
      m = active ? ml : -INFINITY;
      if (!r.renorm)
        for (int j = lane; j < r.E; j += 32) m = fmaxf(m, s_logit[j]);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
    }
    num = active ? (sig ? sigmoid_f(ml) : expf(ml - m)) : 0.f;
    if (r.renorm) den = num;
    else
      for (int j = lane; j < r.E; j += 32) den += sig ? sigmoid_f(s_logit[j]) : expf(s_logit[j] - m);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) den += __shfl_xor_sync(FULL, den, o);
    if (active) s_prob[lane] = num / den;
  }
  __syncwarp();
  for (int i = lane; i < kFewCopies * r.K; i += 32) {
    const int k = i % r.K, at = i / r.K * pairs_pad + t * r.K + k;
    r.topk_idx[at] = s_sel[k];
    r.topk_prob[at] = s_prob[k];
  }
  if (lane < r.K) {
    if (idx_out) idx_out[t * r.K + lane] = s_sel[lane];
    if (prob_out) prob_out[t * r.K + lane] = s_prob[lane];
  }
}

// ---- units ------------------------------------------------------------------------
enum { kEnd = 0, kFC1 = 1, kFC2 = 2 };

// What a stage holds: part of a unit's columns.
struct alignas(16) FewStage {
  int kind;   // kEnd, kFC1, kFC2
  int last;   // the unit's last stage
  int kc;     // columns in this stage
  int entry;  // busy expert (index into the list)
  int pos0;   // first row of the unit in the sorted pair list
  int n;      // its rows (tokens)
  int r0;     // first weight row (FC1: first hidden unit)
  int ks;     // slice of F (FC2)
  int k0;     // first column
  int pad[3];
};

constexpr uint16_t kNoExpert = 0xffff;
constexpr int kMaxChunks = 9;  // of 32 experts, the shared one included
constexpr int kMaxEntries = 257, kMaxPairs = kFewMaxT * 16, kMaxStages = 12;

struct FewCtl {
  uint64_t full_w[kMaxStages];  // weights (and the stage's description) are there
  uint64_t full_t[kMaxStages];  // token rows are there
  uint64_t told[kMaxStages];    // the stage's description is there
  uint64_t empty[kMaxStages], meet;
  alignas(16) FewStage st[kMaxStages];
  int abort;
  int entries, pairs, units1, units2, fc2_writers;
  int ent_e[kMaxEntries];        // expert (E: the shared one)
  int ent_start[kMaxEntries];    // first sorted pair
  int ent_n[kMaxEntries];        // pairs
  int cum1[kMaxEntries + 1], cum2[kMaxEntries + 1];  // units before entry j
  int start[kMaxEntries];                // first sorted pair of an expert
  alignas(16) int4 part[kMaxChunks];     // busy experts, pairs, units and writers of 32 experts
  uint32_t mask[2][kMaxEntries];         // tokens of an expert: 0 .. 31, 32 .. 63
  uint16_t idx[kMaxPairs];       // expert of a pair (kNoExpert: out of range)
  int16_t pos_of[kMaxPairs];     // sorted position of pair p, -1: dropped
  uint8_t tok_of[kMaxPairs + kFewMaxT];  // token of a sorted position
};

struct FewParams {
  // weights as (columns, rows of one half, halves of the experts); tokens, the
  // hidden values and their scales as (columns, rows)
  CUtensorMap w1, w2, w1s, w2s, x, act;
  FewArgs a;
  const int32_t* idx;  // kFewCopies copies of the selection, pairs_pad apart
  const float* prob;
  int pairs_pad;
  int32_t* sync;
  void* hidden;         // bf16, two rows a pair, or E2M1 parts (MXFP4 weights) with
  uint8_t* hidden_s;    // their block scales
  const uint32_t* xs;   // block scales of the tokens' parts
  float* ypart;
  int S;            // rows of act and ypart: T K (+ T)
  int ksplit, stages;
  int more1, more2;  // added to the awaited counts of FC1's and FC2's results: 0 but for a test
  uint64_t wait_limit_ns;
};

// RT = 16 MT weight rows of a unit, NB = 8 NT tokens, NW consumer warps of MPW
// m-tiles each: MT / MPW of them share a slice of a stage's KC columns.
template <int MT_, int MPW_, int NT_, int NW_, int KC_>
struct FewTile {
  static constexpr int MT = MT_, MPW = MPW_, NT = NT_, NW = NW_, KC = KC_;
  static constexpr int RT = 16 * MT;  // weight rows of a unit
  static constexpr int NB = 8 * NT;   // tokens of a unit
  static constexpr int MG = MT / MPW, KG = NW / MG, KW = KC / KG;  // slices and their columns
  // A stage holds KC / 256 boxes of 256 columns, rows one after the other.
  // Rows are 512 bytes, unswizzled: two of a quarter-warp's eight 16-byte
  // loads meet in a bank, which the shared-memory bandwidth has room for.
  static constexpr int KB = 256, NKB = KC / KB;
  static constexpr int A_ROW = 512, B_ROW = 512;
  // Rows of FC2's hidden values a token: two bf16 numbers a value, the second what the
  // first left, within 2^-16 of it (with one the result's error is 1.4 times the output
  // rounding's).  They cost 1 to 2 percent with 8 tokens a unit and 4 with 16 (32 tokens,
  // 2 of 8: 425 us with one number, 444 with two).
  static constexpr int HR = 2;
  static constexpr int NBR = HR * NB;
  static constexpr int A_BYTES = NKB * RT * A_ROW, B_BYTES = NKB * NBR * B_ROW;
  static constexpr int STAGE = (A_BYTES + B_BYTES + 1023) / 1024 * 1024;
  static constexpr int RED_TOK = RT + 4;  // padded token stride of the meeting buffer
  // Meeting buffers: with 16 tokens the second one's place holds a fourth stage
  // (456 us with two buffers and three stages, 444 so).
  static constexpr int REDS = NT > 1 ? 1 : 2;
  static constexpr int RED1 = KG * NB * RED_TOK * 4, RED = REDS * RED1;
  static constexpr int THREADS = 32 * (NW + 2);
  // warps that write the results of a unit of n tokens by `width` values
  static MOE_HD int writers(int n, int width) {
    const int w = (n * width + 31) / 32;
    return w < NW ? w : NW;
  }
  static_assert(MT % MPW == 0 && NW % MG == 0 && NW >= 8 && KB % KW == 0 && KW % 32 == 0, "whole blocks per warp");
};

// Warps that write the results of an expert's n tokens, in units of L::NB, by
// `width` values.
template <class L> MOE_HD int few_writers_of(int n, int width) {
  return n / L::NB * L::writers(L::NB, width) + L::writers(n % L::NB, width);
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
    if (e == kNoExpert) {
      report(status, MOE_ERR_DEVICE_BOUNDS);
    } else {
      const int t = p / cf.K;
      atomicOr(&c.mask[t >> 5][e], 1u << (t & 31));
    }
  }
  if (threadIdx.x < 2 && cf.n_shared) {
    const int n = cf.T - 32 * (int)threadIdx.x;  // tokens in this word
    c.mask[threadIdx.x][cf.E] = n >= 32 ? ~0u : n > 0 ? (1u << n) - 1 : 0u;
  }
  __syncthreads();
  // busy experts in order (the shared expert is one more): a warp takes 32 experts,
  // counts, and continues after the warps before it
  const int last = cf.E + (cf.n_shared ? 1 : 0), chunks = (last + 31) / 32;
  static_assert(L::THREADS / 32 >= kMaxChunks, "a warp for every 32 experts");
  {
    const int e = warp * 32 + lane;
    int n = warp < chunks && e < last ? __popc(c.mask[0][e]) + __popc(c.mask[1][e]) : 0;
    if (e < cf.E && cf.capacity > 0) n = min(n, cf.capacity);
    const uint32_t busy = __ballot_sync(0xffffffffu, n > 0);
    const int sub = (n + L::NB - 1) / L::NB;
    int ip = n, is = sub;
    if (!__any_sync(0xffffffffu, n > 1)) {  // at most one token an expert: count the busy ones
      ip = is = __popc(busy & (0xffffffffu >> (31 - lane)));
    } else {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, ip, o), b = __shfl_up_sync(0xffffffffu, is, o);
        if (lane >= o) { ip += a; is += b; }
      }
    }
    const int writers = __reduce_add_sync(0xffffffffu, few_writers_of<L>(n, L::RT));
    if (lane == 31 && warp < chunks) c.part[warp] = make_int4(__popc(busy), ip, is, writers);
    __syncthreads();
    int4 before = make_int4(0, 0, 0, 0);
    for (int ch = 0; ch < min(warp, chunks); ++ch) {
      const int4 v = c.part[ch];
      before.x += v.x; before.y += v.y; before.z += v.z; before.w += v.w;
    }
    if (n > 0) {
      const int j = before.x + __popc(busy & ((1u << lane) - 1)), u = before.z + is - sub;
      c.start[e] = c.ent_start[j] = before.y + ip - n;
      c.ent_e[j] = e;
      c.ent_n[j] = n;
      c.cum1[j] = u * nrb1;
      c.cum2[j] = u * nrb2 * ksplit;
    }
    if (warp == L::THREADS / 32 - 1 && lane == 0) {  // past every chunk but perhaps its own
      if (warp < chunks) {
        const int4 v = c.part[warp];
        before.x += v.x; before.y += v.y; before.z += v.z; before.w += v.w;
      }
      c.entries = before.x;
      c.pairs = before.y;
      c.cum1[before.x] = c.units1 = before.z * nrb1;
      c.cum2[before.x] = c.units2 = before.z * nrb2 * ksplit;
      c.fc2_writers = before.w * nrb2 * ksplit;
    }
  }
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += L::THREADS) {
    const int e = c.idx[p], t = p / cf.K;
    int pos = -1;
    if (e != kNoExpert) {
      const uint32_t below = (1u << (t & 31)) - 1;
      const int rank = t < 32 ? __popc(c.mask[0][e] & below)
                              : __popc(c.mask[0][e]) + __popc(c.mask[1][e] & below);
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

// Unit u of the list (FC1's, then FC2's): all of its first stage but the columns,
// which are kbeg .. kend - 1.  The whole warp calls it: the lanes look for the entry
// together (one going on from the last unit's entry step by step, with divisions
// that most lists do without: 64 tokens of 64 experts 54.7 us, so 54.3; one of 256
// 50.7 and 50.2).  rows1: hidden units of an FC1 unit.
template <class L>
MOE_D FewStage few_unit(const FewCtl& c, const moe_config_t& cf, int u, int ksplit, int rows1, int lane,
                        int& kbeg, int& kend) {
  FewStage st{};
  const bool fc1 = u < c.units1;
  const int v = fc1 ? u : u - c.units1;
  const int* cum = fc1 ? c.cum1 : c.cum2;
  int j = -1;
  for (int i = 0; i < c.entries; i += 32)
    j += __popc(__ballot_sync(0xffffffffu, i + lane < c.entries && cum[i + lane] <= v));
  const int n = c.ent_n[j], loc = v - cum[j];
  int rest = loc, part = 0;  // the unit's rows, its tokens
  if (n > L::NB) {
    const int sub = (n + L::NB - 1) / L::NB;
    rest = loc / sub;
    part = loc - rest * sub;
  }
  st.kind = fc1 ? kFC1 : kFC2;
  kbeg = 0;
  kend = fc1 ? cf.h : cf.F;
  if (fc1) {
    st.r0 = rest * rows1;
  } else if (ksplit == 1) {
    st.r0 = rest * L::RT;
  } else {
    st.ks = rest % ksplit;
    st.r0 = rest / ksplit * L::RT;
    const int nst = (cf.F + L::KC - 1) / L::KC;
    kbeg = nst * st.ks / ksplit * L::KC;
    kend = min(cf.F, nst * (st.ks + 1) / ksplit * L::KC);
  }
  st.entry = j;
  st.n = min(L::NB, n - part * L::NB);
  st.pos0 = c.ent_start[j] + part * L::NB;
  return st;
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

MOE_D void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A box of a 3-D tensor map (as tc::tma_load_2d), first to leave the L2: weights
// are read once, and what they would push out is the code, the router's weight
// and the hidden values.
MOE_D uint64_t evict_first_policy() {
  uint64_t v;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(v));
  return v;
}
MOE_D void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                       uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}

// Loads from the ring: ordinary loads, which the compiler may move among the
// products but not across a barrier's wait.
MOE_D uint4 lds128(const uint8_t* a) { return *reinterpret_cast<const uint4*>(a); }

// Rows of FC1's output of a unit: hidden units (a SwiGLU unit holds the gate
// and up rows of RT / 2 of them, in groups of eight: each m-tile has eight
// gate rows above the matching eight up rows).
template <class L> MOE_HD int few_rows1(bool glu) { return glu ? L::RT / 2 : L::RT; }

// The combine: a warp takes 64 columns of a token, eight slots at once: lanes
// 4 s + c hold columns 16 i + 4 c .. + 3 of slot s, and a tree adds the slots (a
// fixed order).  `at`: the block's copy of the selection.
constexpr int kCols = 64;
MOE_D int64_t few_combine_items(const moe_config_t& cf) {
  return (int64_t)cf.T * ((cf.h + kCols - 1) / kCols);
}
__device__ __forceinline__ void few_combine(const FewParams& p, const FewCtl& ctl, int64_t at, int warp,
                                            int warps, int lane) {
  const moe_config_t& cf = p.a.c;
  const int g = lane >> 2, q = lane & 3;
  const int col_blocks = (cf.h + kCols - 1) / kCols;
  const int64_t items = few_combine_items(cf);
  const int slots = cf.K + (cf.n_shared ? 1 : 0);
  for (int64_t i = (int64_t)warp * gridDim.x + blockIdx.x; i < items; i += (int64_t)gridDim.x * warps) {
    const int t = (int)(i / col_blocks), r = (int)(i - (int64_t)t * col_blocks) * kCols + 4 * q;
    float4 y[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k = g; k < slots; k += 8) {
      const bool shared = k == cf.K;
      const int pr = t * cf.K + k;
      const int pos = shared ? ctl.pairs - cf.T + t : ctl.pos_of[pr];
      if (pos < 0) continue;  // dropped
      const float w = shared ? 1.f : __ldcg(p.prob + at + pr);
      const float* src = p.ypart + (int64_t)pos * cf.h + r;
      float4 o[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (cf.has_bias && !shared) {
        const __nv_bfloat16* b = p.a.b2 + (int64_t)ctl.idx[pr] * cf.h + r;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (r + 16 * c < cf.h)
            o[c] = make_float4(to_f32(b[16 * c]), to_f32(b[16 * c + 1]), to_f32(b[16 * c + 2]), to_f32(b[16 * c + 3]));
      }
#pragma unroll 2
      for (int s = 0; s < p.ksplit; ++s) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (r + 16 * c < cf.h) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src + (int64_t)s * p.S * cf.h + 16 * c));
            o[c].x += v.x; o[c].y += v.y; o[c].z += v.z; o[c].w += v.w;
          }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        y[c].x = fmaf(w, o[c].x, y[c].x); y[c].y = fmaf(w, o[c].y, y[c].y);
        y[c].z = fmaf(w, o[c].z, y[c].z); y[c].w = fmaf(w, o[c].w, y[c].w);
      }
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) {
        y[c].x += __shfl_xor_sync(0xffffffffu, y[c].x, o);
        y[c].y += __shfl_xor_sync(0xffffffffu, y[c].y, o);
        y[c].z += __shfl_xor_sync(0xffffffffu, y[c].z, o);
        y[c].w += __shfl_xor_sync(0xffffffffu, y[c].w, o);
      }
      if (g == c && r + 16 * c < cf.h) {
        __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(p.a.y + (int64_t)t * cf.h + r + 16 * c);
        dst[0] = __floats2bfloat162_rn(y[c].x, y[c].y);
        dst[1] = __floats2bfloat162_rn(y[c].z, y[c].w);
      }
    }
  }
}

// Weights that are needed whatever the selection, or nearly so, are asked for before
// it, by the blocks together (16 KB a request, one thread), up to about what HBM
// delivers until the list is there: the first experts' when there are twice as many
// pairs as experts or more, then the shared one's (five tokens of 256, bf16, 407.5 us
// without and 405.3).  Where tokens choose alike and independently an expert then stays
// idle once in e^2 at most (13 tokens, 2 of 8, MXFP4, 122.0 us without, 119.2 so, 118.7
// with 40 MB; 32 tokens, bf16, 422.3, 417.0 and 419.2); where they all choose experts
// past the first ones, the requests are 3 us of HBM for nothing.
constexpr int64_t kPrefetchBytes = 20 << 20;
constexpr int kPrefetchChunk = 16384, kPrefetchPairs = 2;
MOE_D void few_prefetch(const void* base, int64_t bytes, int64_t& room) {
  bytes = min(bytes, room);
  room -= bytes;
  for (int64_t at = (int64_t)blockIdx.x * kPrefetchChunk; at + kPrefetchChunk <= bytes;
       at += (int64_t)gridDim.x * kPrefetchChunk)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const uint8_t*>(base) + at),
                 "r"(kPrefetchChunk)
                 : "memory");
}

template <class L>
__global__ void __launch_bounds__(L::THREADS, 1) few_kernel(const __grid_constant__ FewParams p) {
  // (the ring's offset, not a rounded pointer: the compiler must see that its loads
  // are from shared memory)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
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
  for (int e = threadIdx.x; e < kMaxEntries; e += L::THREADS) ctl.mask[0][e] = ctl.mask[1][e] = 0u;
  if (threadIdx.x == 32 * (L::NW + 1)) {
    int64_t room = kPrefetchBytes;
    if (cf.T * cf.K >= kPrefetchPairs * cf.E)
      few_prefetch(p.a.w1.w, (int64_t)cf.E * (glu ? 2 : 1) * cf.F * cf.h * 2, room);
    if (!cf.n_shared) room = 0;
    few_prefetch(p.a.w1.ws, (int64_t)(glu ? 2 : 1) * cf.F * cf.h * 2, room);
    few_prefetch(p.a.w2.ws, (int64_t)cf.F * cf.h * 2, room);
  }
  pdl_wait();  // the selection, and with it the cleared counters
  int32_t* claim = p.sync;
  // the first unit's number comes while the list is made
  const int first_claim = threadIdx.x == 32 * L::NW ? atomicAdd(claim, 1) : 0;
  const int64_t at = (int64_t)(blockIdx.x % kFewCopies) * p.pairs_pad;  // this block's copy
  {
    for (int i = threadIdx.x; i < cf.T * cf.K; i += L::THREADS) {
      const int e = __ldcg(p.idx + at + i);
      ctl.idx[i] = e >= 0 && e < cf.E ? (uint16_t)e : kNoExpert;
    }
  }
  __syncthreads();
  const int nrb1 = ((glu ? 2 * cf.F : cf.F) + L::RT - 1) / L::RT;
  few_build_list<L>(ctl, cf, nrb1, (cf.h + L::RT - 1) / L::RT, p.ksplit, p.a.status);

  int32_t* done = p.sync + 2;   // warps that wrote FC1 results, per busy expert
  int32_t* done2 = p.sync + 1;  // warps that wrote FC2 results
  const int width1 = few_rows1<L>(glu);
  const int total = ctl.units1 + ctl.units2, all2 = ctl.fc2_writers + p.more2;
  tc::WaitCtl wc{p.a.status, &ctl.abort, p.wait_limit_ns, 0};
  tc::WaitCtl wdrain{p.a.status, nullptr, 1000000000ull, 0};

  if (warp == L::NW) {
    // ================= weights =================
    // (as for the tokens, one elected lane of the whole warp issues)
    {
      const bool elected = tc::elect_one();
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_par = 0;
      const uint64_t policy = evict_first_policy();
      int next = first_claim;
      bool ok = true;
      while (ok) {
        const int u = __shfl_sync(0xffffffffu, next, 0);
        if (u < total && lane == 0) next = atomicAdd(claim, 1);  // the next unit, while this one streams
        FewStage st{};
        int kbeg = 0, kend = 1;
        const CUtensorMap* map = nullptr;
        int half0 = 0;  // the map's third coordinate
        bool pairs_of_rows = false;
        if (u < total) {
          st = few_unit<L>(ctl, cf, u, p.ksplit, few_rows1<L>(glu), lane, kbeg, kend);
          pairs_of_rows = glu && st.kind == kFC1;
          const int e = ctl.ent_e[st.entry];
          const bool shared = e == cf.E;
          map = st.kind == kFC1 ? (shared ? &p.w1s : &p.w1) : (shared ? &p.w2s : &p.w2);
          half0 = shared ? 0 : e * (pairs_of_rows ? 2 : 1);
        }
        for (int k0 = kbeg; k0 < kend; k0 += L::KC) {
          if (!tc::mbar_wait(tc::smem_u32(&ctl.empty[stage]), phase ^ 1, wc)) { ok = false; break; }
          const uint32_t fb = tc::smem_u32(&ctl.full_w[stage]);
          st.kc = min(L::KC, kend - k0);
          st.k0 = k0;
          st.last = k0 + L::KC >= kend;
          const int nkb = (st.kc + L::KB - 1) / L::KB;
          const uint32_t tx = nkb * L::RT * L::A_ROW;
          const uint32_t a_dst = ring0 + stage * L::STAGE;
          if (elected) {
            ctl.st[stage] = st;
            tc::mbar_arrive_expect_tx(fb, st.kind == kEnd ? 0 : tx);
            tc::mbar_arrive(tc::smem_u32(&ctl.told[stage]));
            if (st.kind != kEnd) {
#pragma unroll
              for (int b = 0; b < L::NKB; ++b)
                if (b < nkb)
                  tma_load_3d(a_dst + b * L::RT * L::A_ROW, map, k0 + b * L::KB, st.r0, half0, fb, policy);
            }
          }
          __syncwarp();
          if (st.kind == kEnd) {
            issued &= ~(1u << stage);  // its copies are consumed, its barrier a phase further
            ok = false;
            break;
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
    // (the whole warp runs the loop, one elected lane issues: the addresses stay
    // in uniform registers)
    const bool elected = tc::elect_one();
    int stage = 0, ready = -1;
    uint32_t phase = 0, issued = 0, issued_par = 0;
    int row[2 * L::NT][4];  // FC1: the unit's tokens, four rows a load
    for (;;) {
      if (!tc::mbar_wait(tc::smem_u32(&ctl.told[stage]), phase, wc)) break;
      const FewStage st = ctl.st[stage];
      if (st.kind == kEnd) break;
      if (st.kind == kFC2 && ready != st.entry) {  // the expert's hidden values
        const int writers = few_writers_of<L>(ctl.ent_n[st.entry], width1);
        int up = 0;
        if (lane == 0) up = wait_count(done + st.entry, nrb1 * writers + p.more1, wc);
        if (!__shfl_sync(0xffffffffu, up, 0)) break;
        ld_acquire(done + st.entry);  // every lane's own
        fence_proxy_async_global();
        ready = st.entry;
      }
      const uint32_t fb = tc::smem_u32(&ctl.full_t[stage]);
      const uint32_t b_dst = ring0 + stage * L::STAGE + L::A_BYTES;
      const int nkb = (st.kc + L::KB - 1) / L::KB;
      if (st.kind == kFC1) {  // tokens anywhere: the last one repeated
        if (st.k0 == 0) {  // a unit's first stage
          const int mine = ctl.tok_of[st.pos0 + min(lane, st.n - 1)];
#pragma unroll
          for (int i = 0; i < 2 * L::NT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) row[i][r] = __shfl_sync(0xffffffffu, mine, 4 * i + r);
        }
        const int n4 = (st.n + 3) / 4;
        if (elected) {
          tc::mbar_arrive_expect_tx(fb, nkb * n4 * 4 * L::B_ROW);
#pragma unroll
          for (int i = 0; i < 2 * L::NT; ++i)
            if (i < n4)
              for (int b = 0; b < nkb; ++b)
                tc::tma_gather4(b_dst + (b * L::NBR + 4 * i) * L::B_ROW, &p.x, st.k0 + b * L::KB,
                                row[i][0], row[i][1], row[i][2], row[i][3], fb);
        }
      } else if (elected) {  // rows of the sorted list: boxes of eight
        const int n8 = (L::HR * st.n + 7) / 8;
        tc::mbar_arrive_expect_tx(fb, n8 * nkb * 8 * L::B_ROW);
        for (int i = 0; i < n8; ++i)
          for (int b = 0; b < nkb; ++b)
            tc::tma_load_2d(b_dst + (b * L::NBR + 8 * i) * L::B_ROW, &p.act, st.k0 + b * L::KB,
                            L::HR * st.pos0 + 8 * i, fb);
      }
      __syncwarp();
      issued |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == p.stages) { stage = 0; phase ^= 1; }
    }
    for (int s = 0; s < p.stages; ++s)
      if ((issued >> s) & 1u)
        tc::mbar_wait(tc::smem_u32(&ctl.full_t[s]), (issued_par >> s) & 1u, wdrain);
    __syncwarp();
  } else {
    // ================= consumers =================
    const int g = lane >> 2, q = lane & 3;
    int stage = 0;
    uint32_t phase = 0;
    const int mi = warp % L::MG * L::MPW, ki = warp / L::MG;  // its first m-tile, its columns
    const int k_w = ki * L::KW;
    float acc[L::MPW][L::NT][4];
#pragma unroll
    for (int m = 0; m < L::MPW; ++m)
#pragma unroll
      for (int n = 0; n < L::NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
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
    // The stages of one unit, the first of which is there (its weights).  TWO: a
    // SwiGLU FC1 unit, whose m-tiles' upper halves (up rows) lie in a block of
    // their own.  ROWS: rows a token, which add up in the same sums.
    // What does not change from stage to stage is worked out once.
    auto stages = [&](auto two_c, auto rows_c, const FewStage& st) -> bool {
      constexpr bool TWO = decltype(two_c)::value;
      constexpr int ROWS = decltype(rows_c)::value;
      constexpr int M_STEP = TWO ? 8 : 16, HI = (TWO ? 8 * L::MT : 8) * L::A_ROW;
      const int ntiles = (st.n + 7) >> 3;
      const int m_row = M_STEP * mi + g;
      // offsets within a stage: the lane's weight rows and token rows (past the
      // last token, the last)
      const uint32_t a_off = (k_w / L::KB * L::RT + m_row) * L::A_ROW +
                             (k_w % L::KB + 8 * q) * 2;
      uint32_t b_off[L::NT];
#pragma unroll
      for (int n = 0; n < L::NT; ++n)
        b_off[n] = L::A_BYTES + (k_w / L::KB * L::NBR + ROWS * min(8 * n + g, st.n - 1)) * L::B_ROW +
                   (k_w % L::KB + 8 * q) * 2;
      int kc = st.kc, last = st.last;
      for (;;) {
        if (!tc::mbar_wait(tc::smem_u32(&ctl.full_t[stage]), phase, wc)) return false;
        const uint8_t* base = ring + stage * L::STAGE;
        const uint8_t* a_at = base + a_off;
#pragma unroll
        for (int c = 0; c < L::KW / 32; ++c) {
          if (k_w + c * 32 >= kc) break;  // (the boxes are zero past the matrix)
          uint4 b[ROWS][L::NT];
#pragma unroll
          for (int n = 0; n < L::NT; ++n)
            if (L::NT == 1 || n < ntiles) {
#pragma unroll
              for (int r = 0; r < ROWS; ++r) b[r][n] = lds128(base + b_off[n] + r * L::B_ROW + c * 64);
            }
#pragma unroll
          for (int m = 0; m < L::MPW; ++m) {
            const uint4 lo = lds128(a_at + m * M_STEP * L::A_ROW + c * 64);
            const uint4 hi = lds128(a_at + m * M_STEP * L::A_ROW + HI + c * 64);
#pragma unroll
            for (int n = 0; n < L::NT; ++n)
              if (L::NT == 1 || n < ntiles) {
#pragma unroll
                for (int r = ROWS - 1; r >= 0; --r) {
                  mma16816(acc[m][n], lo.x, hi.x, lo.y, hi.y, b[r][n].x, b[r][n].y);
                  mma16816(acc[m][n], lo.z, hi.z, lo.w, hi.w, b[r][n].z, b[r][n].w);
                }
              }
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.empty[stage]));
        if (++stage == p.stages) { stage = 0; phase ^= 1; }
        if (last) return true;
        if (!tc::mbar_wait(tc::smem_u32(&ctl.full_w[stage]), phase, wc)) return false;
        const int4 h = *reinterpret_cast<const int4*>(&ctl.st[stage]);
        last = h.y;
        kc = h.z;
      }
    };
    for (;;) {
      if (!tc::mbar_wait(tc::smem_u32(&ctl.full_w[stage]), phase, wc)) break;
      const FewStage st = ctl.st[stage];
      if (st.kind == kEnd) { finish = true; break; }
      bool done_all;
      using One = std::integral_constant<int, 1>;
      if (st.kind == kFC2) done_all = stages(std::false_type{}, std::integral_constant<int, L::HR>{}, st);
      else if (glu) done_all = stages(std::true_type{}, One{}, st);
      else done_all = stages(std::false_type{}, One{}, st);
      if (!done_all) break;
      const int ntiles = (st.n + 7) >> 3;

      // ---- the unit's end: the warps' sums meet ----
      // One meeting a unit where there are two buffers: they alternate, so the next unit's sums go
      // elsewhere while this unit's are read, and the unit after that comes
      // past the next meeting.  The results are written by the first warps,
      // counted from a warp that moves on with every unit, so that the wait for
      // the stores' way to the L2 falls on another warp each time.
      float* mine = red + (L::REDS == 2 ? (unit & 1) * (L::RED1 / 4) : 0);
      if (L::REDS == 1 && unit > 0 && !meet()) break;  // one buffer: the last unit's sums are read
#pragma unroll
      for (int m = 0; m < L::MPW; ++m)
#pragma unroll
        for (int n = 0; n < L::NT; ++n) {
          if (n < ntiles) {
            float* d = mine + (ki * L::NB + 8 * n + 2 * q) * L::RED_TOK + 16 * (mi + m) + g;
            d[0] = acc[m][n][0];
            d[L::RED_TOK] = acc[m][n][1];
            d[8] = acc[m][n][2];
            d[L::RED_TOK + 8] = acc[m][n][3];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
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
      const int writers = L::writers(st.n, width);
      if (rw >= writers) continue;
      const int items = st.n * width;
      if (st.kind == kFC1) {
        const int e = ctl.ent_e[st.entry];
        for (int i0 = rw * 32; i0 < items; i0 += 32 * writers) {  // whole warps (shuffles below)
          const int i = i0 + lane;
          const int tok = min(i / width, st.n - 1), f = i % width;
          const bool valid = i < items && st.r0 + f < cf.F;
          const int pos = st.pos0 + tok;
          float v;
          if (glu) {
            const int row = f / 8 * 16 + (f & 7);
            v = silu_f(sum(tok, row)) * sum(tok, row + 8);
          } else {
            float z = sum(tok, f);
            if (cf.has_bias && e < cf.E && valid) z += to_f32(p.a.b1[(int64_t)e * cf.F + st.r0 + f]);
            v = gelu_f(z);
          }
          if (valid) {
            __nv_bfloat16* at = static_cast<__nv_bfloat16*>(p.hidden) + (int64_t)pos * L::HR * cf.F + st.r0 + f;
            const __nv_bfloat16 first = __float2bfloat16_rn(v);
            at[0] = first;
            const float left = v - to_f32(first);
            at[cf.F] = __float2bfloat16_rn(isfinite(left) ? left : 0.f);
          }
        }
        fence_proxy_async_global();
        __syncwarp();
        if (lane == 0) red_release(done + st.entry, 1);
      } else {
        for (int i = rw * 32 + lane; i < items; i += 32 * writers) {
          const int tok = i / L::RT, row = i % L::RT;
          if (st.r0 + row < cf.h)
            __stcg(p.ypart + ((int64_t)st.ks * p.S + st.pos0 + tok) * cf.h + st.r0 + row, sum(tok, row));
        }
        __syncwarp();
        if (lane == 0) red_release(done2, 1);
      }
    }
    // ---- combine: every block's share ----
    finish = finish && blockIdx.x < few_combine_items(cf);
    if (finish && warp == 0) {  // one warp of a block that has a share watches the count
      int all = 0;
      if (lane == 0) all = wait_count(done2, all2, wc);
      __shfl_sync(0xffffffffu, all, 0);
    }
    if (finish && meet() && ld_acquire(done2) >= all2) {
      few_combine(p, ctl, at, warp, L::NW, lane);
    }
  }
  __syncthreads();
}

// ---- MXFP4 weights -----------------------------------------------------------------
// The same units, list, counter and order as few_kernel, the products on the
// 5th-generation tensor cores: tcgen05.mma kind::mxf4, 128 weight rows as M
// (FC1: 64 gate rows and the matching 64 up rows), the tokens' E2M1 parts as N
// (six rows a token), the block scales of both operands applied by the MMA, fp32
// accumulators in TMEM (two, for two units in turn).  Decoding the codes on the
// ALUs for m16n8k16 products (tokens in fp16) took 34 warp instructions for 16 x
// 32 weights: T = 13, 2 of 8 experts / T = 64, 8 of 64 / T = 5, 8 of 256 ran in
// 156 / 92 / 165 us; this takes 121 / 58 / 124.
//   warp 0  weights: 128-row boxes of 256 codes and the rows' scale atoms; 512
//           columns a stage (256 a stage, seven or eight stages: the scale warp's
//           work a stage bounds it, 161 / 68 / 171 us);
//   warp 1  TMEM owner and MMA issuer (one elected lane);
//   warps 2, 8, 9  tokens: their parts (FC1: token by token; FC2: one box);
//   warp 3  scales: an FC1 unit's atoms put together from the halves of two
//           tiles, the tokens' scale words gathered into atoms;
//   warps 4-7  epilogue, a TMEM lane quarter each: adds the parts, FC1: SwiGLU
//           (gate and up meet in shared memory) and the hidden values' parts;
//           FC2: partial results.
template <int NT_>
struct FewMxTile {
  static constexpr int NT = NT_, NB = 8 * NT, N = NB * kParts, RT = 128, KC = 512, KB = 256;
  static constexpr int NKB = KC / KB, NKA = KC / 128;  // boxes and scale atoms along K (uint4 loads below)
  static constexpr int A_BOX = RT * 128, B_BOX = N * 128;  // bytes of 256 columns
  static constexpr int A_BYTES = NKB * A_BOX, B_BYTES = NKB * B_BOX;
  static constexpr int SF = NKA * mx::ATOM;                // atoms of 128 rows
  static constexpr int B_OFF = A_BYTES, RAW = B_OFF + B_BYTES, SFA = RAW + 2 * SF, SFB = SFA + SF;
  static constexpr int STAGE = SFB + SF;
  static constexpr int EX = NB * 64, EX_BYTES = 2 * 2 * EX * 4;  // gate and up, two units in turn
  static constexpr int TOKEN_WARPS = 3;  // warps 2, 8 and 9
  static constexpr int THREADS = 320;
  static constexpr uint32_t ACC = 128, SF_COL0 = 256, SF_COLS = 8 * NKA, TMEM = 512;  // TMEM columns
  static constexpr int MAX_STAGES = (TMEM - SF_COL0) / SF_COLS;
  static MOE_HD int writers(int n, int) { return n > 0 ? 4 : 0; }
  static_assert(N <= (int)ACC && STAGE % 1024 == 0 && SFA % 128 == 0, "TMEM columns, swizzle alignment");
};

struct FewMxCtl {
  FewCtl c;
  uint64_t full_s[kMaxStages];                      // the stage's scales are there
  uint64_t unit_told[2], tmem_full[2], tmem_empty[2], drain;
  alignas(16) FewStage unit[2];
  uint32_t tmem_base;
};

// A box of a 3-D tensor map without a cache hint.
MOE_D void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                       uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// 32 lanes x NG groups of 16 columns, one wait.
template <int NG>
MOE_D void tmem_ld_x16(uint32_t taddr, float (&v)[16 * NG]) {
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    float* d = v + 16 * i;
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]), "=f"(d[4]), "=f"(d[5]), "=f"(d[6]),
          "=f"(d[7]), "=f"(d[8]), "=f"(d[9]), "=f"(d[10]), "=f"(d[11]), "=f"(d[12]), "=f"(d[13]),
          "=f"(d[14]), "=f"(d[15])
        : "r"(taddr + 16 * i)
        : "memory");
  }
}

template <class L>
__global__ void __launch_bounds__(L::THREADS, 1) few_mx_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  const moe_config_t& cf = p.a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* ex = reinterpret_cast<float*>(ring + (size_t)p.stages * L::STAGE);
  FewMxCtl& mc = *reinterpret_cast<FewMxCtl*>(reinterpret_cast<uint8_t*>(ex) + L::EX_BYTES);
  FewCtl& ctl = mc.c;
  const uint32_t ring0 = tc::smem_u32(ring);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      for (uint64_t* b : {&ctl.full_w[s], &ctl.told[s], &ctl.empty[s], &mc.full_s[s]})
        tc::mbar_init(tc::smem_u32(b), 1);
      tc::mbar_init(tc::smem_u32(&ctl.full_t[s]), L::TOKEN_WARPS);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(tc::smem_u32(&mc.unit_told[b]), 1);
      tc::mbar_init(tc::smem_u32(&mc.tmem_full[b]), 1);
      tc::mbar_init(tc::smem_u32(&mc.tmem_empty[b]), 4);
    }
    tc::mbar_init(tc::smem_u32(&mc.drain), 1);
    tc::mbar_init(tc::smem_u32(&ctl.meet), 4);
    ctl.abort = 0;
    tc::fence_barrier_init();
    tc::fence_proxy_async_smem();
    for (const CUtensorMap* m : {&p.w1, &p.w2, &p.x, &p.act}) tc::prefetch_tensormap(m);
  }
  if (warp == 1) {
    tc::tmem_alloc(tc::smem_u32(&mc.tmem_base), L::TMEM);
    tc::tmem_relinquish();
  }
  for (int e = threadIdx.x; e < kMaxEntries; e += L::THREADS) ctl.mask[0][e] = ctl.mask[1][e] = 0u;
  if (threadIdx.x == 32 * 3) {
    int64_t room = kPrefetchBytes;
    if (cf.T * cf.K >= kPrefetchPairs * cf.E) {
      few_prefetch(p.a.w1.sf, (int64_t)cf.E * cf.F * cf.h / 16, room);
      few_prefetch(p.a.w1.w, (int64_t)cf.E * cf.F * cf.h, room);
    }
    if (!cf.n_shared) room = 0;
    few_prefetch(p.a.w1.ws, (int64_t)cf.F * cf.h, room);
    few_prefetch(p.a.w2.ws, (int64_t)cf.F * cf.h / 2, room);
    few_prefetch(p.a.w1.ws_sf, (int64_t)cf.F * cf.h / 16, room);
    few_prefetch(p.a.w2.ws_sf, (int64_t)cf.F * cf.h / 32, room);
  }
  pdl_wait();  // the selection, and with it the cleared counters and the tokens' parts
  int32_t* claim = p.sync;
  const int first_claim = threadIdx.x == 0 ? atomicAdd(claim, 1) : 0;
  const int64_t at = (int64_t)(blockIdx.x % kFewCopies) * p.pairs_pad;  // this block's copy
  for (int i = threadIdx.x; i < cf.T * cf.K; i += L::THREADS) {
    const int e = __ldcg(p.idx + at + i);
    ctl.idx[i] = e >= 0 && e < cf.E ? (uint16_t)e : kNoExpert;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const int nrb1 = 2 * cf.F / L::RT;
  few_build_list<L>(ctl, cf, nrb1, cf.h / L::RT, p.ksplit, p.a.status);

  int32_t* done = p.sync + 2;   // warps that wrote FC1 results, per busy expert
  int32_t* done2 = p.sync + 1;  // warps that wrote FC2 results
  const int total = ctl.units1 + ctl.units2;
  const uint32_t tmem = mc.tmem_base;
  tc::WaitCtl wc{p.a.status, &ctl.abort, p.wait_limit_ns, 0};
  tc::WaitCtl wdrain{p.a.status, nullptr, 1000000000ull, 0};
  const bool elected = tc::elect_one();
  int stage = 0;
  uint32_t phase = 0, issued = 0, issued_par = 0;
  // (each role's own copies of these)
  auto next_stage = [&] { if (++stage == p.stages) { stage = 0; phase ^= 1; } };
  auto note_issued = [&] {
    issued |= 1u << stage;
    issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
  };
  // Waits until an FC2 unit's expert has all its hidden values.
  auto hidden_ready = [&](int entry) -> bool {
    int up = 0;
    if (lane == 0) up = wait_count(done + entry, nrb1 * few_writers_of<L>(ctl.ent_n[entry], 0) + p.more1, wc);
    if (!__shfl_sync(0xffffffffu, up, 0)) return false;
    ld_acquire(done + entry);  // every lane's own
    return true;
  };

  if (warp == 0) {
    // ================= weights =================
    int next = first_claim;
    const uint64_t policy = evict_first_policy();
    bool ok = true;
    while (ok) {
      const int u = __shfl_sync(0xffffffffu, next, 0);
      if (u < total && lane == 0) next = atomicAdd(claim, 1);  // the next unit, while this one streams
      FewStage st{};
      int kbeg = 0, kend = 1, half0 = 0;
      const CUtensorMap* map = nullptr;
      const uint8_t *sf0 = nullptr, *sf1 = nullptr;  // scales of the rows, of the up rows
      if (u < total) {
        st = few_unit<L>(ctl, cf, u, p.ksplit, L::RT / 2, lane, kbeg, kend);
        const int e = ctl.ent_e[st.entry];
        const bool shared = e == cf.E, fc1 = st.kind == kFC1;
        map = fc1 ? (shared ? &p.w1s : &p.w1) : (shared ? &p.w2s : &p.w2);
        half0 = shared ? 0 : e * (fc1 ? 2 : 1);
        const FewWeights& W = fc1 ? p.a.w1 : p.a.w2;
        const int64_t row_atoms = (fc1 ? cf.h : cf.F) / 128;
        const uint8_t* sf = shared ? W.ws_sf
                                   : W.sf + (int64_t)e * ((fc1 ? 2 * cf.F : cf.h) / 128) * row_atoms * mx::ATOM;
        sf0 = sf + st.r0 / 128 * row_atoms * mx::ATOM;
        sf1 = sf + (st.r0 + cf.F) / 128 * row_atoms * mx::ATOM;
      }
      for (int k0 = kbeg; k0 < kend; k0 += L::KC) {
        if (!tc::mbar_wait(tc::smem_u32(&ctl.empty[stage]), phase ^ 1, wc)) { ok = false; break; }
        const uint32_t fb = tc::smem_u32(&ctl.full_w[stage]);
        st.kc = min(L::KC, kend - k0);
        st.k0 = k0;
        st.last = k0 + L::KC >= kend;
        const int nkb = (st.kc + L::KB - 1) / L::KB;
        const uint32_t sf_bytes = st.kc / 128 * mx::ATOM;
        const bool fc1 = st.kind == kFC1;
        const uint32_t dst = ring0 + stage * L::STAGE;
        if (elected) {
          ctl.st[stage] = st;
          tc::mbar_arrive_expect_tx(fb, st.kind == kEnd ? 0 : nkb * L::A_BOX + sf_bytes * (fc1 ? 2 : 1));
          tc::mbar_arrive(tc::smem_u32(&ctl.told[stage]));
          if (st.kind != kEnd) {
#pragma unroll
            for (int b = 0; b < L::NKB; ++b)
              if (b < nkb) tma_load_3d(dst + b * L::A_BOX, map, (k0 + b * L::KB) / 2, st.r0, half0, fb, policy);
            const int64_t off = (int64_t)(k0 / 128) * mx::ATOM;
            tc::bulk_load(dst + (fc1 ? L::RAW : L::SFA), sf0 + off, sf_bytes, fb);
            if (fc1) tc::bulk_load(dst + L::RAW + L::SF, sf1 + off, sf_bytes, fb);
          }
        }
        __syncwarp();
        if (st.kind == kEnd) {
          issued &= ~(1u << stage);  // its copies are consumed, its barrier a phase further
          ok = false;
          break;
        }
        note_issued();
        next_stage();
      }
    }
    for (int s = 0; s < p.stages; ++s)
      if ((issued >> s) & 1u)
        tc::mbar_wait(tc::smem_u32(&ctl.full_w[s]), (issued_par >> s) & 1u, wdrain);
  } else if (warp == 1) {
    // ================= MMA issuer =================
    const uint64_t a_desc = tc::desc_kmajor_sw128(ring0), b_desc = tc::desc_kmajor_sw128(ring0 + L::B_OFF);
    const uint64_t sfa_desc = tc::desc_sf_atom(ring0 + L::SFA), sfb_desc = tc::desc_sf_atom(ring0 + L::SFB);
    int unit = 0;
    bool first = true, ok = true;
    while (ok) {
      if (!tc::mbar_wait(tc::smem_u32(&ctl.full_w[stage]), phase, wc)) break;
      const FewStage st = ctl.st[stage];
      const int buf = unit & 1;
      if (first &&  // the epilogue is done with this buffer's last unit
          !tc::mbar_wait(tc::smem_u32(&mc.tmem_empty[buf]), ((unit >> 1) & 1) ^ 1, wc)) break;
      if (st.kind != kEnd) {
        if (!tc::mbar_wait(tc::smem_u32(&ctl.full_t[stage]), phase, wc)) break;
        if (!tc::mbar_wait(tc::smem_u32(&mc.full_s[stage]), phase, wc)) break;
        tc::fence_after_sync();
        const uint32_t so = stage * (L::STAGE >> 4);  // descriptors count 16 bytes
        const uint32_t d = tmem + buf * L::ACC;
        const uint32_t sfa = tmem + L::SF_COL0 + stage * L::SF_COLS, sfb = sfa + 4 * L::NKA;
        const int nk = st.kc / 128;
        if (elected) {
#pragma unroll
          for (int k = 0; k < L::NKA; ++k) {
            if (k >= nk) break;
            tc::tmem_cp_32x128b_warpx4(sfa + 4 * k, sfa_desc + so + k * (mx::ATOM >> 4));
            tc::tmem_cp_32x128b_warpx4(sfb + 4 * k, sfb_desc + so + k * (mx::ATOM >> 4));
            const uint64_t ad = a_desc + so + (k >> 1) * (L::A_BOX >> 4) + (k & 1) * 4;
            const uint64_t bd = b_desc + so + (k >> 1) * (L::B_BOX >> 4) + (k & 1) * 4;
            tc::mma_mxf4(d, ad, bd, tc::idesc_mxf4_e2m1(128, L::N, 0, 0), sfa + 4 * k, sfb + 4 * k,
                         !first || k > 0);
            tc::mma_mxf4(d, ad + 2, bd + 2, tc::idesc_mxf4_e2m1(128, L::N, 2, 2), sfa + 4 * k, sfb + 4 * k, 1);
          }
          tc::mma_commit(tc::smem_u32(&ctl.empty[stage]));
        }
        __syncwarp();
        first = false;
      }
      if (st.kind == kEnd || st.last) {
        if (elected) {
          mc.unit[buf] = st;
          tc::mbar_arrive(tc::smem_u32(&mc.unit_told[buf]));
          if (st.kind != kEnd) tc::mma_commit(tc::smem_u32(&mc.tmem_full[buf]));
        }
        __syncwarp();
        ++unit;
        first = true;
      }
      ok = st.kind != kEnd;
      if (ok) next_stage();
    }
    if (ctl.abort) {  // let every issued MMA finish before TMEM is freed
      if (elected) tc::mma_commit(tc::smem_u32(&mc.drain));
      tc::mbar_wait(tc::smem_u32(&mc.drain), 0, wdrain);
    }
  } else if (warp == 2 || warp >= 8) {
    // ================= tokens =================
    // A token's parts are a box of their own (FC1): three warps share the issue (one
    // token of 256 experts 55.8 us with one warp, 54.8 so; 13 tokens of 8 127.9, 127.3).
    const int tw = warp == 2 ? 0 : warp - 7;
    int ready = -1, mine = 0;
    for (;;) {
      if (!tc::mbar_wait(tc::smem_u32(&ctl.told[stage]), phase, wc)) break;
      const FewStage st = ctl.st[stage];
      if (st.kind == kEnd) break;
      if (tw == 0 && st.kind == kFC2 && ready != st.entry) {
        if (!hidden_ready(st.entry)) break;
        fence_proxy_async_global();
        ready = st.entry;
      }
      const uint32_t fb = tc::smem_u32(&ctl.full_t[stage]);
      const uint32_t dst = ring0 + stage * L::STAGE + L::B_OFF;
      const int nkb = (st.kc + L::KB - 1) / L::KB;
      if (st.kind == kFC1) {  // tokens anywhere: a token's parts a box
        if (st.k0 == 0) mine = ctl.tok_of[st.pos0 + min(lane, st.n - 1)];
        const int mine_n = (st.n - tw + L::TOKEN_WARPS - 1) / L::TOKEN_WARPS;  // tokens tw, tw + 3, ..
        if (elected) tc::mbar_arrive_expect_tx(fb, nkb * mine_n * kParts * 128);
        for (int i = tw; i < st.n; i += L::TOKEN_WARPS) {
          const int t = __shfl_sync(0xffffffffu, mine, i);
          if (elected)
            for (int b = 0; b < nkb; ++b)
              tma_load_3d(dst + b * L::B_BOX + i * kParts * 128, &p.x, (st.k0 + b * L::KB) / 2, 0, t, fb);
        }
      } else if (elected) {  // rows of the sorted list: one box
        tc::mbar_arrive_expect_tx(fb, tw == 0 ? nkb * L::B_BOX : 0);
        if (tw == 0)
          for (int b = 0; b < nkb; ++b)
            tma_load_3d(dst + b * L::B_BOX, &p.act, (st.k0 + b * L::KB) / 2, 0, st.pos0, fb);
      }
      __syncwarp();
      if (st.kind == kFC1 || tw == 0) note_issued();
      else issued &= ~(1u << stage);  // no copies of its own; the stage's last ones are consumed
      next_stage();
    }
    for (int s = 0; s < p.stages; ++s)
      if ((issued >> s) & 1u)
        tc::mbar_wait(tc::smem_u32(&ctl.full_t[s]), (issued_par >> s) & 1u, wdrain);
  } else if (warp == 3) {
    // ================= scales =================
    // The tokens' scale words come from the L2, asked for while the stage's weights
    // are under way.  (Asked for a stage earlier, they are waited for by the stage's
    // proxy fence all the same: 13 tokens of 8 experts 123.6 us, so 122.2; a word a
    // load, not a stage's words in one: 127.5.)
    int ready = -1;
    constexpr int NR = (L::N + 31) / 32;  // rows (token, part) a lane
    for (;;) {
      if (!tc::mbar_wait(tc::smem_u32(&ctl.told[stage]), phase, wc)) break;
      const FewStage st = ctl.st[stage];
      if (st.kind == kEnd) break;
      if (st.kind == kFC2 && ready != st.entry) {
        if (!hidden_ready(st.entry)) break;
        ready = st.entry;
      }
      const bool fc1 = st.kind == kFC1;
      const int nk = st.kc / 128, words = (fc1 ? cf.h : cf.F) / 128;
      alignas(16) uint32_t w[NR][L::NKA];
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int r = lane + 32 * i, tok = r / kParts;
        const int src = tok < st.n ? (fc1 ? ctl.tok_of[st.pos0 + tok] : st.pos0 + tok) : -1;
        const uint32_t* base = fc1 ? p.xs : reinterpret_cast<const uint32_t*>(p.hidden_s);
        base += ((int64_t)src * kParts + r % kParts) * words + st.k0 / 128;
#pragma unroll
        for (int k = 0; k < L::NKA; ++k) w[i][k] = 0u;
        if (src < 0) continue;
        if (nk == L::NKA && words % L::NKA == 0) {  // a stage's words, aligned
          *reinterpret_cast<uint4*>(w[i]) = __ldcg(reinterpret_cast<const uint4*>(base));
        } else {
#pragma unroll
          for (int k = 0; k < L::NKA; ++k)
            if (k < nk) w[i][k] = __ldcg(base + k);
        }
      }
      uint8_t* sp = ring + stage * L::STAGE;
      if (!tc::mbar_wait(tc::smem_u32(&ctl.full_w[stage]), phase, wc)) break;
      if (fc1) {  // rows r0 .. r0 + 63 of the gate tile, then the same of the up tile
        const int hb = (st.r0 & 127) >> 6;
#pragma unroll
        for (int k = 0; k < L::NKA; ++k)
          if (k < nk) {
            const uint8_t* raw = sp + L::RAW + k * mx::ATOM + 16 * lane + 8 * hb;
            const uint2 g = *reinterpret_cast<const uint2*>(raw);
            const uint2 u = *reinterpret_cast<const uint2*>(raw + L::SF);
            *reinterpret_cast<uint4*>(sp + L::SFA + k * mx::ATOM + 16 * lane) = make_uint4(g.x, g.y, u.x, u.y);
          }
      }
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int k = 0; k < L::NKA; ++k)
          if (k < nk)
            *reinterpret_cast<uint32_t*>(sp + L::SFB + k * mx::ATOM + 16 * lane + 4 * i) = w[i][k];
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&mc.full_s[stage]));
      next_stage();
    }
  } else if (warp < 8) {
    // ================= epilogue =================
    const int q = warp & 3;  // TMEM lane quarter
    uint32_t meet_par = 0;
    for (int unit = 0;; ++unit) {
      const int buf = unit & 1;
      const uint32_t par = (unit >> 1) & 1;
      if (!tc::mbar_wait(tc::smem_u32(&mc.unit_told[buf]), par, wc)) break;
      const FewStage st = mc.unit[buf];
      if (st.kind == kEnd) break;
      if (!tc::mbar_wait(tc::smem_u32(&mc.tmem_full[buf]), par, wc)) break;
      tc::fence_after_sync();
      float v[L::N];
      tmem_ld_x16<L::N / 16>(tmem + ((uint32_t)(q * 32) << 16) + buf * L::ACC, v);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&mc.tmem_empty[buf]));
      float y[L::NB];
#pragma unroll
      for (int t = 0; t < L::NB; ++t) {
        y[t] = v[kParts * t + kParts - 1];  // the smallest part first
#pragma unroll
        for (int i = kParts - 2; i >= 0; --i) y[t] += v[kParts * t + i];
      }
      if (st.kind == kFC1) {
        float* eb = ex + buf * 2 * L::EX;
#pragma unroll
        for (int t = 0; t < L::NB; ++t) eb[(q >> 1) * L::EX + t * 64 + (q & 1) * 32 + lane] = y[t];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.meet));
        if (!tc::mbar_wait(tc::smem_u32(&ctl.meet), meet_par, wc)) break;
        meet_par ^= 1;
        // blocks of 32 hidden units of a token, eight lanes a block, four blocks a warp
        // (a block a warp, a value a lane: 64 tokens of 64 experts 69.1 us, so 54.1)
        const int l = lane & 7;
        for (int i0 = 4 * q; i0 < 2 * st.n; i0 += 16) {  // whole warps (shuffles)
          const int i = i0 + (lane >> 3), t = i >> 1, f = (i & 1) * 32;
          const bool valid = t < st.n;
          const int at4 = (valid ? t * 64 + f : 0) + 4 * l;
          const float4 z = *reinterpret_cast<const float4*>(eb + at4), u = *reinterpret_cast<const float4*>(eb + L::EX + at4);
          float v4[4] = {silu_f(z.x) * u.x, silu_f(z.y) * u.y, silu_f(z.z) * u.z, silu_f(z.w) * u.w};
          uint32_t code[kParts], scale[kParts];
          e2m1_parts(v4, code, scale);
          if (!valid) continue;
          const int64_t row = (int64_t)(st.pos0 + t) * kParts;
#pragma unroll
          for (int k = 0; k < kParts; ++k) {
            *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(p.hidden) + (row + k) * (cf.F / 2) +
                                         (st.r0 + f) / 2 + 2 * l) = (uint16_t)code[k];
            if (l == 0) p.hidden_s[(row + k) * (cf.F / 32) + (st.r0 + f) / 32] = (uint8_t)scale[k];
          }
        }
        fence_proxy_async_global();
        __syncwarp();
        if (lane == 0) red_release(done + st.entry, 1);
      } else {
        float* dst = p.ypart + ((int64_t)st.ks * p.S + st.pos0) * cf.h + st.r0 + q * 32 + lane;
#pragma unroll
        for (int t = 0; t < L::NB; ++t)
          if (t < st.n) __stcg(dst + (int64_t)t * cf.h, y[t]);
        __syncwarp();
        if (lane == 0) red_release(done2, 1);
      }
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, L::TMEM);
  }
  // ---- combine: every block's share ----
  const bool share = !ctl.abort && blockIdx.x < few_combine_items(cf);
  if (share && threadIdx.x == 0) mc.tmem_base = wait_count(done2, ctl.fc2_writers + p.more2, wc);  // (its address is read)
  __syncthreads();
  if (share && mc.tmem_base != 0) {
    ld_acquire(done2);  // every thread's own
    few_combine(p, ctl, at, warp, L::THREADS / 32, lane);
  }
}

// Launches a kernel that may start while the one before it drains; it waits
// (pdl_wait) before it reads what that one writes.
template <typename... KArgs, typename... Args>
cudaError_t few_pdl_launch(void (*kern)(KArgs...), int grid, int block, size_t smem, cudaStream_t s,
                           const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
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

// Launches a kernel with a ring of as many stages as fit beside `fixed` bytes, at
// most `most`.
cudaError_t few_launch_ring(void (*kern)(const FewParams), int threads, int stage, int most, int fixed,
                            FewParams& p, cudaStream_t s) {
  fixed += 1024;  // the ring's alignment
  p.stages = (227 * 1024 - fixed) / stage;
  if (p.stages > most) p.stages = most;
  const int smem = p.stages * stage + fixed;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return few_pdl_launch(kern, p.a.sms, threads, smem, s, p);
}

// The launch with MXFP4 weights.
template <class L>
cudaError_t few_mx_launch(FewParams& p, const uint8_t* xq, cudaStream_t s) {
  const moe_config_t& c = p.a.c;
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  auto weights = [&](CUtensorMap* m, const void* w, uint64_t cols, uint64_t rows, uint64_t halves,
                     int pair) {
    return few_encode(m, u8, 1, w, 3, cols / 2, rows, halves, 128, L::RT / pair, pair, true);
  };
  bool ok = weights(&p.w1, p.a.w1.w, c.h, c.F, (uint64_t)c.E * 2, 2) &&
            weights(&p.w2, p.a.w2.w, c.F, c.h, c.E, 1);
  if (c.n_shared)
    ok = ok && weights(&p.w1s, p.a.w1.ws, c.h, c.F, 2, 2) && weights(&p.w2s, p.a.w2.ws, c.F, c.h, 1, 1);
  ok = ok && few_encode(&p.x, u8, 1, xq, 3, c.h / 2, kParts, c.T, 128, kParts, 1, true) &&
       few_encode(&p.act, u8, 1, p.hidden, 3, c.F / 2, kParts, p.S, 128, kParts, L::NB, true);
  if (!ok) return cudaErrorInvalidValue;
  return few_launch_ring(few_mx_kernel<L>, L::THREADS, L::STAGE, L::MAX_STAGES, L::EX_BYTES + (int)sizeof(FewMxCtl), p, s);
}

template <class L>
cudaError_t few_launch(FewParams& p, cudaStream_t s) {
  const moe_config_t& c = p.a.c;
  const bool glu = c.act == MOE_ACT_SWIGLU;
  const auto u16 = CU_TENSOR_MAP_DATA_TYPE_UINT16;
  // weights: rows of F or h, the gate and up halves of an expert one after the other
  auto weights = [&](CUtensorMap* m, const void* w, uint64_t cols, uint64_t rows, uint64_t halves,
                     int pair) {
    return few_encode(m, u16, 2, w, 3, cols, rows, halves, L::KB, L::RT / pair, pair, false);
  };
  const int pair = glu ? 2 : 1;
  bool ok = weights(&p.w1, p.a.w1.w, c.h, c.F, (uint64_t)c.E * pair, pair) &&
            weights(&p.w2, p.a.w2.w, c.F, c.h, c.E, 1);
  if (c.n_shared)
    ok = ok && weights(&p.w1s, p.a.w1.ws, c.h, c.F, pair, pair) &&
         weights(&p.w2s, p.a.w2.ws, c.F, c.h, 1, 1);
  ok = ok && few_encode(&p.x, u16, 2, p.a.x, 2, c.h, c.T, 1, L::KB, 1, 1, false) &&
       few_encode(&p.act, u16, 2, p.hidden, 2, c.F, (uint64_t)L::HR * p.S, 1, L::KB, 8, 1, false);
  if (!ok) return cudaErrorInvalidValue;
  return few_launch_ring(few_kernel<L>, L::THREADS, L::STAGE, kMaxStages, L::RED + (int)sizeof(FewCtl), p, s);
}

}  // namespace

cudaError_t launch_few(const FewArgs& a, bool mxfp4, cudaStream_t s) {
  const moe_config_t& c = a.c;
  const FewLayout L = few_layout(c);
  FewParams p{};
  p.a = a;
  float* parts = reinterpret_cast<float*>(a.ws + L.parts);
  const int kparts = few_kparts(c);
  p.idx = reinterpret_cast<int32_t*>(a.ws + L.idx);
  p.prob = reinterpret_cast<float*>(a.ws + L.prob);
  p.pairs_pad = few_pairs_pad(c);
  p.sync = reinterpret_cast<int32_t*>(a.ws + L.sync);
  uint8_t* xq = reinterpret_cast<uint8_t*>(a.ws + L.xq);
  uint8_t* xs = reinterpret_cast<uint8_t*>(a.ws + L.xs);
  p.xs = reinterpret_cast<uint32_t*>(xs);
  p.hidden = a.ws + L.a;
  p.hidden_s = reinterpret_cast<uint8_t*>(a.ws + L.as);
  p.ypart = reinterpret_cast<float*>(a.ws + L.ypart);
  p.S = c.T * c.K + (c.n_shared ? c.T : 0);
  p.ksplit = few_ksplit(c);
  p.more1 = a.starve == 1;
  p.more2 = a.starve == 2;
  p.wait_limit_ns = a.starve ? 20000000ull : 2000000000ull;
  RouterArgs r{};
  r.T = c.T; r.E = c.E; r.K = c.K; r.h = c.h; r.score = c.score;
  r.renorm = (c.flags & MOE_FLAG_RENORM) != 0;
  r.force_balance = (c.flags & MOE_FLAG_FORCE_BALANCE) != 0;
  r.sel_bias = a.sel_bias;
  r.topk_idx = const_cast<int32_t*>(p.idx);
  r.topk_prob = const_cast<float*>(p.prob);
  // Tokens a warp of the router takes: as many as leave 26 warps an SM.  us with 8 / 4 /
  // 2 / 1 (MXFP4): 64 tokens of 64 experts 54.8 / 55.8 / 56.5 / 59.4, 24 tokens 48.1 /
  // 46.7 / 46.5 / 47.9, 5 tokens of 256 129.3 / 126.3 / 124.9 / 123.0.
  auto warps = [&](int tok) { return (int64_t)c.E * kparts * ceil_div(c.T, tok); };
  int tok = 8;
  while (tok > 1 && warps(tok) < 26 * a.sms) tok /= 2;
  const int route_blocks = (int)ceil_div(warps(tok), 8);
  auto* route = tok == 1 ? few_router_kernel<1> : tok == 2 ? few_router_kernel<2>
                : tok == 4 ? few_router_kernel<4> : few_router_kernel<8>;
  route<<<route_blocks + (mxfp4 ? c.T * (int)ceil_div(c.h, kSplitCols) : 0), 256, 0, s>>>(
      a.x, a.w_r, c.T, c.E, c.h, kparts, parts, route_blocks,
      xq, xs, p.sync, (int)few_sync_words(c));
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = few_pdl_launch(few_select_kernel, c.T, 256, 0, s,
                       const_cast<const float*>(parts), kparts, a.gate_bias, r, p.pairs_pad,
                       a.idx_out, a.prob_out);
  if (e != cudaSuccess) return e;
  // Tokens a unit holds: 8 while experts have at most that many on average or
  // half of it (what is more becomes a second unit, whose weights come from the
  // L2), 16 beyond.  us with 8 / 16: T = 32, 2 of 8, bf16, 485 / 439; T = 64, 8 of 64,
  // MXFP4, 63.5 / 58.1; T = 13, 2 of 8, MXFP4 (3.25 tokens an expert), 118 to 125 / 129.
  const bool many = c.T > 8 && (int64_t)c.T * c.K > 4LL * c.E;
  if (mxfp4)
    return many ? few_mx_launch<FewMxTile<2>>(p, xq, s) : few_mx_launch<FewMxTile<1>>(p, xq, s);
  return many ? few_launch<FewTile<4, 2, 2, 8, 256>>(p, s) : few_launch<FewTile<4, 2, 1, 16, 256>>(p, s);
}

}  // namespace moe
