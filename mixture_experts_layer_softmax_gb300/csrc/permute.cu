// Dispatch: expert-contiguous permutation of the T*K (token, slot) pairs.
//
// "Scalable Training of Mixture-of-Experts Models with Megatron Core" (review),
// §2.1 "Dispatch" (tokens are permuted so each expert's rows are contiguous,
// with per-expert counts and offsets) and §4.3.1 (permutation fusion);
// §4.3.3 asks for sync-free kernels: counts and offsets never leave the device.
//
// Positions are decided without atomics, so the permutation is unique and
// bit-reproducible: inside an expert's segment rows are in ascending token
// order.  Tokens are cut into chunks of 32 (one warp each):
//   1. chunk_hist:   hist[c][e] = pairs of chunk c routed to e
//   2. chunk_scan:   base[c][e] = sum_{c' < c} hist[c'][e]; counts[e];
//                    for small batches (ceil(T/32) * E <= 8192) every block of
//                    step 3 redoes this scan in shared memory instead (one
//                    launch fewer)
//   3. chunk_ranks:  offsets = exclusive scan of counts; for every pair
//                    dst_row = offsets[e] + base[c][e] + rank inside the chunk
//                    (a bit per token in a word per expert);
//                    src_token, perm_prob are the inverse maps.
//   With an expert capacity C (skill page "emerging-techniques-moe-training",
//   "Capacity Factor Tuning"), counts[e] = min(slots, C) and a pair whose
//   position base + rank inside its expert is >= C is dropped (dst_row = -1):
//   every expert keeps its first C slots in ascending token order.
//   4. scatter_rows: each token's row is read once and written to its K
//                    destinations with 16-byte vectors.
#include "common.cuh"
#include "pdl.cuh"

namespace moe {

constexpr int kChunk = 32;

// ---- per-warp steps ----------------------------------------------------------

// hist[c][e] for chunk c; `my` is this warp's [E] shared-memory counter row.
MOE_D void hist_chunk(int c, int lane, int32_t* my, const int32_t* __restrict__ idx, int T, int K,
                      int E, int32_t* __restrict__ hist, int* status) {
  for (int e = lane; e < E; e += 32) my[e] = 0;
  __syncwarp();
  const int64_t t = (int64_t)c * kChunk + lane;
  if (t < T)
    for (int k = 0; k < K; ++k) {
      const int e = __ldg(idx + t * K + k);
      if (e >= 0 && e < E)
        atomicAdd(&my[e], 1);
      else
        report(status, MOE_ERR_DEVICE_BOUNDS);
    }
  __syncwarp();
  for (int e = lane; e < E; e += 32) hist[(int64_t)c * E + e] = my[e];
  __syncwarp();
}

// Exclusive scan of hist[:, e] over the chunks into base[:, e]; counts[e] =
// the slots expert e keeps (all of them, or at most `cap` when cap > 0).
MOE_D void scan_expert(int e, int lane, const int32_t* hist, int NC, int E, int cap,
                       int32_t* base, int32_t* counts) {
  int running = 0;
  for (int c0 = 0; c0 < NC; c0 += 32) {
    const int c = c0 + lane;
    const int v = c < NC ? hist[(int64_t)c * E + e] : 0;  // global or shared memory
    int incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    if (c < NC) base[(int64_t)c * E + e] = running + incl - v;
    running += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) counts[e] = (cap > 0 && running > cap) ? cap : running;
}

// Whole block (256 threads): s_off[0..E] = exclusive scan of counts[0..E)
// (zero past E, s_off[256] the total); block 0 also writes offsets_out.
MOE_D void block_offsets(const int32_t* __restrict__ counts, int E, int32_t* s_off,
                         int32_t* s_warp, int32_t* offsets_out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = threadIdx.x;
  const int v = e < E ? __ldg(counts + e) : 0;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int wbase = 0;
  for (int w = 0; w < warp; ++w) wbase += s_warp[w];
  s_off[e] = wbase + incl - v;
  if (e == 255) s_off[256] = wbase + incl;
  __syncthreads();
  if (blockIdx.x == 0 && offsets_out && e <= E) offsets_out[e] = s_off[e];
  if (blockIdx.x == 0 && offsets_out && E == 256 && e == 0) offsets_out[256] = s_off[256];
}

// A pair's destination row: offsets[e] + its position among expert e's slots, or -1
// when cap > 0 and position >= cap (dropped: beyond the expert's capacity).
// src_token and perm_prob are the inverse maps of the kept pairs.
MOE_D void place_pair(int64_t t, int k, int e, int pos, int T, int K, int cap,
                      const float* __restrict__ prob, const int32_t* s_off,
                      int32_t* __restrict__ dst_row, int32_t* __restrict__ src_token,
                      float* __restrict__ perm_prob, int* status) {
  const int64_t i = t * K + k;
  if (e < 0 || (cap > 0 && pos >= cap)) {
    dst_row[i] = -1;
    return;
  }
  const int r = s_off[e] + pos;
  if (r < 0 || (int64_t)r >= (int64_t)T * K) {  // histograms that do not match idx
    report(status, MOE_ERR_DEVICE_BOUNDS);
    dst_row[i] = -1;
    return;
  }
  dst_row[i] = r;
  src_token[r] = (int32_t)t;
  if (perm_prob) perm_prob[r] = prob ? __ldg(prob + i) : 1.f;
}

// Destination rows of chunk c's pairs: the pair's position among expert e's
// slots is base[c][e] + its rank among the chunk's earlier tokens routed to e.
// Every expert has a word of `my` ([E], this warp's) with a bit for each token
// routed to it, so a rank is the number of lower bits.  (A token that names an
// expert twice, which no router of this library does, has one bit for both: such
// a chunk counts in order of the tokens.)  Expert ids outside [0, E) get dst_row = -1
// (reported by the histogram step).
MOE_D void ranks_chunk(int c, int lane, uint32_t* my, const int32_t* __restrict__ idx,
                       const float* __restrict__ prob, int T, int K, int E, int cap,
                       const int32_t* base, const int32_t* s_off, int32_t* __restrict__ dst_row,
                       int32_t* __restrict__ src_token, float* __restrict__ perm_prob,
                       int* status) {
  const int64_t t = (int64_t)c * kChunk + lane;
  const bool valid = t < T;
  const unsigned lt_mask = (1u << lane) - 1u;
  for (int e = lane; e < E; e += 32) my[e] = 0;
  __syncwarp();
  bool twice = false;
  if (valid) {
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
      const int e = __ldg(idx + t * K + k);
      if (e >= 0 && e < E) twice |= (atomicOr(&my[e], 1u << lane) >> lane) & 1u;
    }
  }
  __syncwarp();
  if (!__any_sync(0xffffffffu, twice)) {
    if (!valid) return;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
      int e = __ldg(idx + t * K + k);
      if (e < 0 || e >= E) e = -1;
      const int pos = e < 0 ? 0 : base[(int64_t)c * E + e] + __popc(my[e] & lt_mask);
      place_pair(t, k, e, pos, T, K, cap, prob, s_off, dst_row, src_token, perm_prob, status);
    }
    return;
  }
  // such a chunk: as many tokens at a time as the warp has lanes for their slots, with a
  // count of an expert's pairs so far in its word (9 ballots for each pair of slots, as it
  // was: 210 us for the maps of 200000 tokens, top-16 of 256, and 91 without such tokens)
  __syncwarp();
  for (int e = lane; e < E; e += 32) my[e] = 0;
  __syncwarp();
  const int tokens = min(kChunk, T - c * kChunk), per = 32 / K, g = lane / K, k = lane - g * K;
  const unsigned earlier = (1u << (g * K)) - 1u;  // lanes of the tokens before this lane's
  for (int i = g; i - g < tokens; i += per) {
    const bool in = g < per && i < tokens;
    const int64_t ti = (int64_t)c * kChunk + i;
    int e = in ? __ldg(idx + ti * K + k) : -1;
    if (e < 0 || e >= E) e = -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int pos = e < 0 ? 0 : base[(int64_t)c * E + e] + (int)my[e] + __popc(same & earlier);
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) my[e] += __popc(same);
    __syncwarp();
    // (of a token's slots that share the row, the last one's probability stays)
    const unsigned token = ((1u << K) - 1u) << (g * K);
    const bool last = ((same & token) >> lane) == 1u;
    if (in)
      place_pair(ti, k, e, pos, T, K, cap, prob, s_off, dst_row, src_token, last ? perm_prob : nullptr,
                 status);
  }
}

// Token t's row, read once (16-byte vectors, up to 8 per lane in flight) and
// written to its K destination rows.  The first batch of the row's vectors is
// loaded before pdl_wait: x is never written by the map steps this kernel
// follows (and was final before they started), so under programmatic
// dependent launch that read overlaps the previous kernel's tail; the
// destination rows are read only after the wait.
template <typename T, int KMAX>
MOE_D void scatter_token(int64_t t, int lane, const T* __restrict__ x,
                         const int32_t* __restrict__ dst_row,
                         int ntok, int K, int h, T* __restrict__ x_perm, int* status) {
  constexpr int V = Vec<T>::N;
  constexpr int kMaxVec = 8;
  const int nvec = h / V;
  const int64_t P = (int64_t)ntok * K;
  const T* src = x + t * h;
  Vec<T> buf[kMaxVec];
#pragma unroll
  for (int i = 0; i < kMaxVec; ++i) {
    const int v = i * 32 + lane;
    if (v < nvec) buf[i] = ld16_stream(src + (int64_t)v * V);
  }
  pdl_wait();
  T* dst[KMAX];
#pragma unroll
  for (int k = 0; k < KMAX; ++k) {
    dst[k] = nullptr;
    if (k < K) {
      const int r = __ldg(dst_row + t * K + k);
      if (r >= 0 && r < P)
        dst[k] = x_perm + (int64_t)r * h;
      else if (r >= P)
        report(status, MOE_ERR_DEVICE_BOUNDS);
    }
  }
  for (int v0 = 0; v0 < nvec; v0 += 32 * kMaxVec) {
    if (v0 > 0) {
#pragma unroll
      for (int i = 0; i < kMaxVec; ++i) {
        const int v = v0 + i * 32 + lane;
        if (v < nvec) buf[i] = ld16_stream(src + (int64_t)v * V);
      }
    }
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
      if (!dst[k]) continue;
#pragma unroll
      for (int i = 0; i < kMaxVec; ++i) {
        const int v = v0 + i * 32 + lane;
        if (v < nvec) st16(dst[k] + (int64_t)v * V, buf[i]);
      }
    }
  }
}

// ---- separate kernels -------------------------------------------------------

// One warp per chunk of 32 tokens; 8 warps per block.
__global__ void __launch_bounds__(256) chunk_hist_kernel(const int32_t* __restrict__ idx, int T,
                                                         int K, int E, int NC,
                                                         int32_t* __restrict__ hist, int* status) {
  extern __shared__ int32_t sh[];  // [8][E]
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 8 + warp;
  if (c < NC) hist_chunk(c, lane, sh + warp * E, idx, T, K, E, hist, status);
}

// 32 experts a block (a lane each, so that a warp's loads are whole lines), the chunks
// shared among 32 warps: each adds up its chunks, the sums are scanned, and each writes
// the exclusive scan of its own.
__global__ void __launch_bounds__(1024) chunk_scan_kernel(const int32_t* __restrict__ hist, int NC,
                                                          int E, int cap,
                                                          int32_t* __restrict__ base,
                                                          int32_t* __restrict__ counts) {
  __shared__ int32_t s_sum[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  const int per = (NC + 31) / 32, c0 = min(warp * per, NC), c1 = min(c0 + per, NC);
  pdl_wait();
  pdl_trigger();
  int sum = 0;
  if (e < E) {
#pragma unroll 8
    for (int c = c0; c < c1; ++c) sum += __ldg(hist + (int64_t)c * E + e);
  }
  s_sum[lane][warp] = sum;
  __syncthreads();
  {  // warp w scans expert w's 32 sums
    const int v = s_sum[warp][lane];
    int incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    s_sum[warp][lane] = incl - v;
    const int ew = blockIdx.x * 32 + warp;
    if (lane == 31 && ew < E) counts[ew] = (cap > 0 && incl > cap) ? cap : incl;
  }
  __syncthreads();
  if (e >= E) return;
  int run = s_sum[lane][warp];
#pragma unroll 8
  for (int c = c0; c < c1; ++c) {
    const int v = __ldg(hist + (int64_t)c * E + e);
    base[(int64_t)c * E + e] = run;
    run += v;
  }
}

// Block: exclusive scan of counts into shared offsets, then one warp per chunk
// computes every pair's destination row.
__global__ void __launch_bounds__(256) chunk_ranks_kernel(
    const int32_t* __restrict__ idx, const float* __restrict__ prob, int T, int K, int E, int cap,
    int NC, const int32_t* __restrict__ base, const int32_t* __restrict__ counts,
    int32_t* __restrict__ offsets_out, int32_t* __restrict__ dst_row,
    int32_t* __restrict__ src_token, float* __restrict__ perm_prob, int* status) {
  __shared__ int32_t s_off[257];
  __shared__ int32_t s_warp[8];
  extern __shared__ uint32_t s_bits[];  // [8][E]
  pdl_wait();
  pdl_trigger();
  block_offsets(counts, E, s_off, s_warp, offsets_out);
  const int c = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (c < NC)
    ranks_chunk(c, threadIdx.x & 31, s_bits + (threadIdx.x >> 5) * E, idx, prob, T, K, E, cap, base,
                s_off, dst_row, src_token, perm_prob, status);
}

// Steps 2 and 3 in one kernel for small batches (NC * E <= kScanInBlock):
// every block copies the chunk histograms into shared memory and scans them
// per expert itself (a few thousand integers, L2-resident), so the separate
// scan launch goes away; block 0 writes counts and offsets.  Same per-warp
// steps, same maps.
constexpr int64_t kScanInBlock = 8192;

__global__ void __launch_bounds__(256) chunk_scan_ranks_kernel(
    const int32_t* __restrict__ idx, const float* __restrict__ prob, int T, int K, int E, int cap,
    int NC, const int32_t* __restrict__ hist, int32_t* __restrict__ counts_out,
    int32_t* __restrict__ offsets_out, int32_t* __restrict__ dst_row,
    int32_t* __restrict__ src_token, float* __restrict__ perm_prob, int* status) {
  extern __shared__ int32_t sh[];
  pdl_wait();
  pdl_trigger();
  int32_t* s_base = sh;                        // [NC][E]: hist, then base in place
  int32_t* s_cnt = s_base + (int64_t)NC * E;   // [E]
  int32_t* s_off = s_cnt + E;                  // [E + 1]
  uint32_t* s_bits = reinterpret_cast<uint32_t*>(s_off + E + 1);  // [8][E]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 8
  for (int i = threadIdx.x; i < NC * E; i += 256) s_base[i] = __ldg(hist + i);
  __syncthreads();
  if (NC <= 64) {  // a thread an expert (at most 256), else a warp
    const int e = threadIdx.x;
    int run = 0;
    if (e < E) {
      for (int c = 0; c < NC; ++c) {
        const int v = s_base[c * E + e];
        s_base[c * E + e] = run;
        run += v;
      }
      s_cnt[e] = (cap > 0 && run > cap) ? cap : run;
    }
  } else {
    for (int e = warp; e < E; e += 8) scan_expert(e, lane, s_base, NC, E, cap, s_base, s_cnt);
  }
  __syncthreads();
  if (warp == 0) {  // s_off = exclusive scan of the counts
    int running = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int v = e < E ? s_cnt[e] : 0;
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      if (e < E) {
        s_off[e] = running + incl - v;
        if (blockIdx.x == 0) {
          offsets_out[e] = running + incl - v;
          counts_out[e] = v;
        }
      }
      running += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      s_off[E] = running;
      if (blockIdx.x == 0) offsets_out[E] = running;
    }
  }
  __syncthreads();
  const int c = blockIdx.x * 8 + warp;
  if (c < NC)
    ranks_chunk(c, lane, s_bits + warp * E, idx, prob, T, K, E, cap, s_base, s_off, dst_row,
                src_token, perm_prob, status);
}

// One warp per token (the grid covers every token, so the block scheduler
// balances the load).
template <typename T, int KMAX>
__global__ void __launch_bounds__(256) scatter_rows_kernel(const T* __restrict__ x,
                                                           const int32_t* __restrict__ dst_row,
                                                           int ntok, int K, int h,
                                                           T* __restrict__ x_perm, int* status) {
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t < ntok)
    scatter_token<T, KMAX>(t, threadIdx.x & 31, x, dst_row, ntok, K, h, x_perm, status);
  else
    pdl_wait();
}

int num_chunks(int T) { return (int)ceil_div(T, kChunk); }

// Step 1 alone: the per-chunk histograms of idx (the router's hand-off to
// the dispatch when its own epilogue does not produce them).
cudaError_t launch_chunk_hist(const moe_config_t& c, const int32_t* idx, int32_t* hist,
                              int* status, cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  const int NC = num_chunks(c.T);
  chunk_hist_kernel<<<(unsigned)ceil_div(NC, 8), 256, 8 * c.E * sizeof(int32_t), s>>>(
      idx, c.T, c.K, c.E, NC, hist, status);
  return cudaGetLastError();
}

// hist_ready: hist already holds idx's chunk histograms (written by the
// router), so step 1 is skipped.
cudaError_t launch_permute_maps(const moe_config_t& c, const int32_t* idx, const float* prob,
                                int32_t* hist, int32_t* base, int32_t* counts, int32_t* offsets,
                                int32_t* dst_row, int32_t* src_token, float* perm_prob,
                                int* status, cudaStream_t s, bool hist_ready) {
  const int NC = num_chunks(c.T);
  if (c.T == 0) {
    // no rows: counts and offsets are all zero
    cudaError_t e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * c.E, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(offsets, 0, sizeof(int32_t) * (c.E + 1), s);
    return e;
  }
  const int blocks = (int)ceil_div(NC, 8);
  if (!hist_ready) {
    const cudaError_t e = launch_chunk_hist(c, idx, hist, status, s);
    if (e != cudaSuccess) return e;
  }
  if ((int64_t)NC * c.E <= kScanInBlock) {
    const size_t bytes = sizeof(int32_t) * ((size_t)NC * c.E + 2 * c.E + 1 + 8 * c.E);
    return pdl_launch(chunk_scan_ranks_kernel, dim3(blocks), dim3(256), bytes, s, idx, prob, c.T,
                      c.K, c.E, c.capacity, NC, (const int32_t*)hist, counts, offsets, dst_row,
                      src_token, perm_prob, status);
  }
  // each step may be scheduled while the one before it ends (it waits for it first)
  cudaError_t e = pdl_launch(chunk_scan_kernel, dim3((unsigned)ceil_div(c.E, 32)), dim3(1024), 0, s,
                             (const int32_t*)hist, NC, c.E, c.capacity, base, counts);
  if (e != cudaSuccess) return e;
  return pdl_launch(chunk_ranks_kernel, dim3(blocks), dim3(256), 8 * c.E * sizeof(uint32_t), s, idx,
                    prob, c.T, c.K, c.E, c.capacity, NC, (const int32_t*)base,
                    (const int32_t*)counts, offsets, dst_row, src_token, perm_prob, status);
}

int scatter_grid(int ntok, int sms) {
  const int64_t need = ceil_div(ntok, 8);
  const int64_t cap = (int64_t)sms * 8;
  return (int)(need < cap ? (need > 0 ? need : 1) : cap);
}

template <typename T>
static cudaError_t scatter_t(const moe_config_t& c, const void* x, const int32_t* dst_row,
                             void* x_perm, int* status, cudaStream_t s, bool pdl) {
  const unsigned grid = (unsigned)ceil_div(c.T, 8);
  const T* xs = static_cast<const T*>(x);
  T* xp = static_cast<T*>(x_perm);
  if (c.K <= 2)
    return launch_maybe_pdl(pdl, scatter_rows_kernel<T, 2>, dim3(grid), dim3(256), 0, s, xs, dst_row,
                            c.T, c.K, c.h, xp, status);
  else if (c.K <= 4)
    return launch_maybe_pdl(pdl, scatter_rows_kernel<T, 4>, dim3(grid), dim3(256), 0, s, xs, dst_row,
                            c.T, c.K, c.h, xp, status);
  else if (c.K <= 8)
    return launch_maybe_pdl(pdl, scatter_rows_kernel<T, 8>, dim3(grid), dim3(256), 0, s, xs, dst_row,
                            c.T, c.K, c.h, xp, status);
  else
    return launch_maybe_pdl(pdl, scatter_rows_kernel<T, 16>, dim3(grid), dim3(256), 0, s, xs, dst_row,
                            c.T, c.K, c.h, xp, status);
  return cudaGetLastError();
}

// after_maps: the launch directly follows this library's map steps on the
// stream, so it may overlap their tail (programmatic dependent launch); any
// other caller gets a plain launch.
cudaError_t launch_scatter_rows(const moe_config_t& c, const void* x, const int32_t* dst_row,
                                void* x_perm, int sms, int* status, cudaStream_t s,
                                bool after_maps) {
  (void)sms;
  if (c.T == 0) return cudaSuccess;
  if (c.dtype == MOE_BF16)
    return scatter_t<__nv_bfloat16>(c, x, dst_row, x_perm, status, s, after_maps);
  return scatter_t<float>(c, x, dst_row, x_perm, status, s, after_maps);
}

}  // namespace moe
