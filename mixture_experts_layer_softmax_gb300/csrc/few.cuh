// Workspace of the layer for a few tokens (few.cu), laid over the bytes of the
// whole-layer workspace: a call of one never needs what the other left.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kFewMaxT = 64;  // tokens of one moe_layer_fwd_few call
// E2M1 blocks that a block of tokens or hidden values beside MXFP4 weights is the sum of:
// within 2^(1 - 3 kParts) of its largest value.  Four (2^-11) left an error 1.15 times the
// output rounding's, and in a block with an outlier lost what is 2^-11 of it; six (2^-17)
// leave the output rounding, as two bf16 numbers do beside bf16 weights.  us with 4 / 6 / 8:
// one token of 256 experts 52.1 / 51.4 / 54.6, 13 of 8 120.6 / 121.2 / 122.3, 64 of 64
// 56.5 / 57.6 / 61.2.
constexpr int kParts = 6;

// Slices of the router's h reduction: enough (expert, slice) pairs to give
// every SM 16 warps, slices of at least 256 columns, at most 32 of them.  (us for 5
// tokens of 256 experts, MXFP4, with 4 / 8 / 16 / 32 warps: 129.4 / 125.0 / 122.1 /
// 126.0; slices of 128 columns: 64 tokens of 64 59.9 against 54.4.)  152 is the GB300's
// SM count, not the device's own: the workspace's size, which this sets, and the sums'
// order are the config's alone.
inline int few_kparts(const moe_config_t& c) {
  const int64_t most = ceil_div(c.h, 256);
  int64_t p = ceil_div(16 * 152, c.E);
  if (p > most) p = most;
  if (p > 32) p = 32;
  return p < 1 ? 1 : (int)p;
}

// FC2's reduction (F) is cut into slices of at most 4096 columns whose partial
// results are added in order: units stay small enough to spread evenly.
inline int few_ksplit(const moe_config_t& c) {
  return (int)ceil_div(c.F, 4096);
}

// The selection (expert and weight of every pair) is kept in several copies,
// whole 128-byte lines apart, so that the SMs do not all read the same lines.
constexpr int kFewCopies = 16;
inline int few_pairs_pad(const moe_config_t& c) { return (c.T * c.K + 31) / 32 * 32; }

// Whether every count of units and of finished warps fits 31 bits, with the
// smallest units (8 tokens, 64 rows) and the most writers (16 a unit).
inline bool few_counts_fit(const moe_config_t& c) {
  const int64_t subs = (int64_t)c.T * c.K + (c.n_shared ? ceil_div(c.T, 8) : 0);
  const int64_t r1 = c.act == MOE_ACT_SWIGLU ? 2LL * c.F : c.F, most = (1LL << 31) / 16;
  return subs * ceil_div(r1, 64) < most && subs * ceil_div(c.h, 64) * few_ksplit(c) < most;
}

// Whether the few-token calls take the config, but for the number of its tokens.
inline bool few_takes(const moe_config_t& c) {
  return c.dtype == MOE_BF16 && !(c.flags & MOE_FLAG_SAVE_FOR_BWD) && c.aux_loss_coeff == 0.f &&
         c.z_loss_coeff == 0.f && few_counts_fit(c);
}

struct FewLayout {
  size_t sync, parts, idx, prob, xq, xs, a, as, ypart, total;
};
// int32 words at `sync`: the unit counter, the warps that finished FC2 results,
// and those that finished FC1 results per busy expert (E + 1).
inline size_t few_sync_words(const moe_config_t& c) { return 2 + c.E + 1; }

inline FewLayout few_layout(const moe_config_t& c) {
  FewLayout w{};
  if (c.T < 1 || c.T > kFewMaxT || !few_takes(c)) return w;
  const size_t T = (size_t)c.T, S = T * c.K + (c.n_shared ? T : 0);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  w.sync = take(few_sync_words(c) * 4);
  w.parts = take((size_t)few_kparts(c) * T * c.E * 4);
  w.idx = take((size_t)kFewCopies * few_pairs_pad(c) * 4);
  w.prob = take((size_t)kFewCopies * few_pairs_pad(c) * 4);
  w.xq = take(T * c.h * kParts / 2);    // tokens in E2M1 parts (MXFP4 weights)
  w.xs = take(T * ceil_div(c.h, 32) * kParts);  // and their block scales
  w.a = take(S * c.F * 4);              // hidden values: two bf16 numbers each, or parts
  w.as = take(S * ceil_div(c.F, 32) * kParts);  // and their block scales
  w.ypart = take((size_t)few_ksplit(c) * S * c.h * 4);
  w.total = off;
  return w;
}

// The expert matrices of one projection: bf16 [E][rows][cols], or MXFP4 codes
// with their scale atoms (uniform groups of `rows` rows, 128-row tiles).
struct FewWeights {
  const void* w;        // routed experts
  const uint8_t* sf;    // their scales (MXFP4)
  const void* ws;       // shared expert or null
  const uint8_t* ws_sf;
};

struct FewArgs {
  moe_config_t c;
  const __nv_bfloat16* x;
  const float* w_r;
  const float* gate_bias;
  const float* sel_bias;
  FewWeights w1, w2;
  const __nv_bfloat16* b1;
  const __nv_bfloat16* b2;
  __nv_bfloat16* y;
  int32_t* idx_out;   // or null
  float* prob_out;    // or null
  char* ws;           // few_layout
  int* status;
  int sms;
  int starve;         // 0, or the wait on counts that is to run out: 1 FC1's results, 2 FC2's
};

cudaError_t launch_few(const FewArgs& a, bool mxfp4, cudaStream_t s);

}  // namespace moe
