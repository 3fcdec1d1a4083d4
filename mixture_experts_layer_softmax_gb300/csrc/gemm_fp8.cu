// FP8 expert products with a scale for each block of 128 (fp8.cuh):
//   z[r, n] = sum_b sa[r, b] sw[n / 128, b] sum_{k in block b} a[r, k] w[n, k]
// for the rows r of each expert, and FC1's epilogue a = p silu(gate) up.
//
// The scales are fp32 numbers, which the tensor cores do not apply: the products
// of one block of 128 columns (4 MMAs of K = 32, kind::f8f6f4) are summed in TMEM
// and joined in registers, acc += (sa sw) t, an FMA a value and block.
//
// Persistent kernel, one CTA an SM, tiles of 128 rows x 256 weight rows (FC1: 128
// gate and the matching 128 up rows):
//   warp 0     TMA producer: 4 stages of {A 128 x 128 B, W 256 x 128 B}.
//   warps 1-2  MMA issuers (warp 1 owns TMEM): a stage's products go to one of two
//              256-column accumulators, each given back once a block.
//   warp 3     scales: each row's sa sw of eight blocks at a time, to shared memory
//              (a joining thread that reads its own row's scales touches a line of its
//              own with each, and keeps registers for them).
//   warps 4-11 two warps a TMEM lane quarter (32 rows), each one half of the
//              columns: a thread keeps 128 fp32 sums of one row.
// While they evaluate and store a tile the MMAs run at most two blocks ahead.
// Every wait is bounded; one that gives up records MOE_ERR_TIMEOUT and every role
// leaves its loop.
//
// FC1 of 16384 rows, 8 experts, 4096 -> 2 x 14336: 1515 us in a burst, 2.54 PFLOP/s (1005
// us at twice the measured bf16 rate), 1.69 to 1.73 ms in a long run (1400 W); 8-bit a
// instead of bf16 the same, with the pre-activation 1.63 and 1.84 ms.  Evaluating and
// storing a tile takes a time of its own whatever K is: FC2 of 16384 rows to 4096 columns
// 70, 93, 138 and 236 us at K = 512, 1024, 2048 and 4096.  What bounds the FC1, by leaving
// parts of the work out when a burst took 1552: the stages' copies alone 1100 us (48 KB a
// 512-cycle step, 75 bytes a clock and SM), the MMAs and the hand-over 944, the joining
// alone 1190 (a packed FMA takes an SM quarter 2.3 to 3 cycles, a TMEM load of 16 columns
// its latency), all but SiLU and stores 1444.
// Steps: 4.0 ms with the joining's registers capped at 168 a thread (spills), 2.2 ms with
// a register split, 1.78 with 16-column loads and intrinsics for the packed FMA (half the
// moves), 1.65 with the scales in a warp of their own, 1.57 with 32-byte stores, 1.55 with
// two MMA issuers, 1.515 with the joining loop unrolled twice.
// Slower were a tile of 128 x 128 (four accumulators, 2.1 ms: the MMAs read A twice), 16
// joining warps (2.1 ms), and rows exchanged between four lanes so that a store covers 8
// rows x 128 bytes instead of 32 x 32 (1.62 ms: the exchange costs more than the lines).
#include "fp8.cuh"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

using fp8::BLOCK;

constexpr int TM = 128, TN = 256;
constexpr int A_BYTES = TM * BLOCK, W_BYTES = TN * BLOCK;
constexpr int STAGES = 4;
constexpr int kThreads = 384;
// Registers a thread: 384 x 168 at launch; the first warpgroup gives some back and
// the joining ones take them.
constexpr int kRegsIssue = 88, kRegsJoin = 208;
static_assert(kRegsIssue + 2 * kRegsJoin <= 3 * 168, "more registers than the launch brings");

constexpr int SB = 8;  // blocks of scales at a time

struct Ctl {
  float2 scale[2][SB][TM + 4];  // [block][row]: sa times the scales of the tile's two weight blocks
  uint64_t full[STAGES], empty[STAGES], tfull[2], tempty[2], sfull[2], sempty[2], meet[4], drain[2];
  uint32_t tmem_base;
  int abort;
  int off[257], tile_start[257], part[8];
  uint32_t top[2][2][TM];  // tile parity, half of the columns, row
};
constexpr size_t kSmem = 1024 + (size_t)STAGES * (A_BYTES + W_BYTES) + sizeof(Ctl);
static_assert(kSmem <= 227 * 1024, "shared memory");

struct TcParams {
  const int32_t* offsets;  // [E+1]
  const float* prob;       // FC1: [P] or null
  const float* a_sf;       // [P, KB]
  const float* w_sf;       // [E * Nw/128, KB]
  __nv_bfloat16* save;     // FC1: [P, 2N] pre-activation or null
  __nv_bfloat16* out;      // [P, N] or null
  uint8_t* out_q;          // FC1: [P, N] or null
  float* out_sf;           // FC1: [P, N/128]
  int P, E, KB, N, Nw;     // KB: blocks of K; Nw: weight rows an expert (2N or N)
  bool wide;               // every output is 32-byte aligned (their rows are multiples of 64 bytes)
  bool once;               // weights are read about once: they leave the L2 first
  int* status;
  uint64_t wait_limit_ns;
};

// acc += s t for N values, two in one packed FMA.
template <int N> MOE_D void join(float2* acc, const uint32_t (&t)[N], float s) {
#pragma unroll
  for (int j = 0; j < N / 2; ++j)
    acc[j] = __ffma2_rn(make_float2(__uint_as_float(t[2 * j]), __uint_as_float(t[2 * j + 1])),
                        make_float2(s, s), acc[j]);
}
// 16 columns of the warp's 32 lanes, arrived.
MOE_D void tmem_ld(uint32_t addr, uint32_t (&r)[16]) {
  tc::tmem_ld_32x32b_x16_nowait(addr, r);
  tc::tmem_ld_wait_x16(r);
}
MOE_D uint32_t pack_bf16x2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// SiLU with CUDA's expf and the approximate quotient, bounded by 2 ulp; a quotient
// below 2^-126 (z < -87) is 0.
MOE_D float silu_f32(float z) { return z * __fdividef(1.f, 1.f + expf(-z)); }
// 32 bytes of a row: one store where the row is 32-byte aligned (a warp's rows are
// lines apart, so its stores cost by their number: 16-byte ones took 4096 cycles a tile).
MOE_D void store32(void* dst, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// 64 values of a row to 64 bf16.
MOE_D void store64(__nv_bfloat16* dst, const float2* v, bool wide) {
#pragma unroll
  for (int j = 0; j < 32; j += 8) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(v[j + k].x, v[j + k].y);
    store32(dst + 2 * j, w, wide);
  }
}

struct Tile {
  int e, row, rows, nb;  // expert, first row, rows of the expert from there, column tile
};
template <int ROWS, class C> MOE_D Tile tile_at(const C& c, int E, int tile) {
  int lo = 0, hi = E - 1;  // largest e with tile_start[e] <= tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c.tile_start[mid] <= tile) lo = mid; else hi = mid - 1;
  }
  const int local = tile - c.tile_start[lo], n = c.off[lo + 1] - c.off[lo];
  const int mblk = (n + ROWS - 1) / ROWS;
  const int nb = local / mblk, mb = local - nb * mblk;
  return {lo, c.off[lo] + mb * ROWS, n - mb * ROWS, nb};
}

// Expert boundaries kept within the rows and ascending (c.off), and the tiles before
// each expert (c.tile_start; nblk column tiles for every ROWS of its rows).  Every
// thread of the block calls it, at least 256; thread e has expert e.
template <int ROWS, class C>
MOE_D void load_tiles(C& c, const int32_t* __restrict__ offsets, int E, int P, int nblk) {
  const int e = threadIdx.x, lane = e & 31, w = e >> 5;
  const int first = min(max(__ldg(offsets), 0), P);
  int end = e < E ? max(min(max(__ldg(offsets + e + 1), 0), P), first) : first;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {  // an expert's end: the largest offset so far
    const int t = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end = max(end, t);
  }
  if (lane == 31 && w < 8) c.part[w] = end;
  __syncthreads();
  for (int i = 0; i < min(w, 8); ++i) end = max(end, c.part[i]);
  if (e < E) c.off[e + 1] = end;
  if (e == 0) c.off[0] = first;
  __syncthreads();
  const int tiles = e < E ? (end - c.off[e] + ROWS - 1) / ROWS * nblk : 0;
  int sum = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += t;
  }
  if (lane == 31 && w < 8) c.part[w] = sum;
  __syncthreads();
  for (int i = 0; i < min(w, 8); ++i) sum += c.part[i];
  if (e < E) c.tile_start[e] = sum - tiles;
  if (e == E - 1) c.tile_start[E] = sum;
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_product_kernel(const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmW, const TcParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sW = sA + STAGES * A_BYTES;
  Ctl& ctl = *reinterpret_cast<Ctl*>(sW + STAGES * W_BYTES);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E, KB = p.KB;
  const int nblk = SWIGLU ? p.N / BLOCK : (p.N + TN - 1) / TN;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(tc::smem_u32(&ctl.full[s]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(tc::smem_u32(&ctl.tfull[b]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.tempty[b]), 8);
      tc::mbar_init(tc::smem_u32(&ctl.sfull[b]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.sempty[b]), 8);
      tc::mbar_init(tc::smem_u32(&ctl.drain[b]), 1);
    }
    for (int q = 0; q < 4; ++q) tc::mbar_init(tc::smem_u32(&ctl.meet[q]), 2);
    ctl.abort = 0;
    tc::fence_barrier_init();
    tc::fence_proxy_async_smem();
    tc::prefetch_tensormap(&tmA);
    tc::prefetch_tensormap(&tmW);
  }
  if (warp == 1) {
    tc::tmem_alloc(tc::smem_u32(&ctl.tmem_base), 512);
    tc::tmem_relinquish();
  }
  pdl_wait();  // before here only the block's own state
  pdl_trigger();
  load_tiles<TM>(ctl, p.offsets, E, p.P, nblk);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem_base = ctl.tmem_base;
  const int total = ctl.tile_start[E];
  tc::WaitCtl wc{p.status, &ctl.abort, p.wait_limit_ns, 0};
  tc::WaitCtl wdrain{p.status, nullptr, 1000000000ull, 0};

  if (warp < 4) {
    tc::regs_dec<kRegsIssue>();
    if (warp == 0) {
      // ================= TMA producer: the warp runs the loop, one lane issues =================
      const bool elected = tc::elect_one();
      const uint64_t policy = p.once ? tc::evict_first_policy() : tc::evict_normal_policy();
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_par = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const Tile t = tile_at<TM>(ctl, E, tile);
        const int w0 = t.e * p.Nw + (SWIGLU ? t.nb * BLOCK : t.nb * TN);
        // the second half: FC1's up rows; FC2's next 128 rows, where an odd last tile
        // takes rows of the next expert (or, past the tensor, zeros) that go nowhere
        const int w1 = SWIGLU ? w0 + p.N : w0 + BLOCK;
        for (int kb = 0; kb < KB; ++kb) {
          if (!tc::mbar_wait(tc::smem_u32(&ctl.empty[stage]), phase ^ 1, wc)) { ok = false; break; }
          if (elected) {
            const uint32_t fb = tc::smem_u32(&ctl.full[stage]);
            const uint32_t wd = tc::smem_u32(sW + stage * W_BYTES);
            tc::mbar_arrive_expect_tx(fb, A_BYTES + W_BYTES);
            tc::tma_load_2d(tc::smem_u32(sA + stage * A_BYTES), &tmA, kb * BLOCK, t.row, fb);
            tc::tma_load_2d_hint(wd, &tmW, kb * BLOCK, w0, fb, policy);
            tc::tma_load_2d_hint(wd + W_BYTES / 2, &tmW, kb * BLOCK, w1, fb, policy);
          }
          __syncwarp();
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
      }
      for (int s = 0; s < STAGES; ++s)
        if ((issued >> s) & 1u)
          tc::mbar_wait(tc::smem_u32(&ctl.full[s]), (issued_par >> s) & 1u, wdrain);
      __syncwarp();
    } else if (warp <= 2) {
      // ================= MMA issuers: likewise, one for each accumulator =================
      // (a step's two waits, four MMAs and two commits in one warp for both: 1567 us for
      // FC1 of 16384 rows, against 1552)
      const bool elected = tc::elect_one();
      const uint32_t buf = warp - 1;
      const uint64_t a_base = tc::desc_kmajor_sw128(tc::smem_u32(sA));
      const uint64_t w_base = tc::desc_kmajor_sw128(tc::smem_u32(sW));
      const int tiles = (total - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
      const int64_t steps = tiles > 0 ? (int64_t)tiles * KB : 0;
      for (int64_t step = buf; step < steps; step += 2) {
        const uint32_t stage = (uint32_t)step % STAGES;
        if (!tc::mbar_wait(tc::smem_u32(&ctl.tempty[buf]), ((uint32_t)(step >> 1) & 1) ^ 1, wc) ||
            !tc::mbar_wait(tc::smem_u32(&ctl.full[stage]), (uint32_t)(step / STAGES) & 1, wc))
          break;
        tc::fence_after_sync();
        const uint64_t ad = a_base + stage * (A_BYTES >> 4), wd = w_base + stage * (W_BYTES >> 4);
        if (elected) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_f8(tmem_base + buf * TN, ad + 2 * k, wd + 2 * k, tc::idesc_e4m3_f32(TM, TN), k != 0);
          tc::mma_commit(tc::smem_u32(&ctl.empty[stage]));
          tc::mma_commit(tc::smem_u32(&ctl.tfull[buf]));
        }
        __syncwarp();
      }
      __syncwarp();
      if (ctl.abort) {  // let every issued MMA finish before TMEM is freed
        if (elected) tc::mma_commit(tc::smem_u32(&ctl.drain[buf]));
        tc::mbar_wait(tc::smem_u32(&ctl.drain[buf]), 0, wdrain);
      }
      __syncwarp();
    } else {
      // ================= scales: a lane has one block of every fourth row =================
      const int j = lane & 7, r0 = lane >> 3;
      const int wblk = p.Nw / BLOCK;
      uint32_t n = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const Tile t = tile_at<TM>(ctl, E, tile);
        // FC1: gate and up; FC2: neighbours (the last block twice where there is one)
        const float* sw0 = p.w_sf + ((int64_t)t.e * wblk + (SWIGLU ? t.nb : 2 * t.nb)) * KB;
        const float* sw1 = p.w_sf + ((int64_t)t.e * wblk + (SWIGLU ? wblk / 2 + t.nb : min(2 * t.nb + 1, wblk - 1))) * KB;
        const float* sa = p.a_sf + (int64_t)t.row * KB;
        for (int kb = 0; kb < KB; kb += SB, ++n) {
          const uint32_t buf = n & 1;
          const int k = min(kb + j, KB - 1);
          const float w0 = __ldg(sw0 + k), w1 = __ldg(sw1 + k);
#pragma unroll 1
          for (int r = r0; r < TM; r += 64) {
            float a[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)  // (a row behind the expert's takes its last row's, which go nowhere)
              a[i] = __ldg(sa + (int64_t)min(r + 4 * i, t.rows - 1) * KB + k);
            if (r == r0 && !tc::mbar_wait(tc::smem_u32(&ctl.sempty[buf]), ((n >> 1) & 1) ^ 1, wc)) { ok = false; break; }
#pragma unroll
            for (int i = 0; i < 16; ++i) ctl.scale[buf][j][r + 4 * i] = make_float2(a[i] * w0, a[i] * w1);
          }
          if (!ok) break;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.sfull[buf]));
        }
      }
    }
  } else {
    tc::regs_inc<kRegsJoin>();
    // ================= joining and epilogue (warps 4..11) =================
    const int q = warp & 3;          // TMEM lane quarter this warp may access
    const int hf = (warp - 4) >> 2;  // which half of the columns (FC1: 64 gate and the matching up ones)
    // a warp's TMEM columns: FC1's gate and up, FC2's one half
    const uint32_t c0 = SWIGLU ? hf * 64 : hf * 128, c1 = SWIGLU ? 128 + hf * 64 : hf * 128 + 64;
    const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16);
    const int i = q * 32 + lane;  // row within the tile
    uint32_t step = 0, n = 0, parity = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const Tile t = tile_at<TM>(ctl, E, tile);
      const int n0 = SWIGLU ? t.nb * BLOCK + hf * 64 : t.nb * TN + hf * 128;  // first column
      float2 acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.f, 0.f);
#pragma unroll 2  // (one at a time 1552 us, four 2841: spills)
      for (int kb = 0; kb < KB; ++kb, ++step) {
        const int j = kb & (SB - 1);
        const uint32_t sb = n & 1, buf = step & 1;
        if ((j == 0 && !tc::mbar_wait(tc::smem_u32(&ctl.sfull[sb]), (n >> 1) & 1, wc)) ||
            !tc::mbar_wait(tc::smem_u32(&ctl.tfull[buf]), (step >> 1) & 1, wc)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const float2 s = ctl.scale[sb][j][i];
        const float g = SWIGLU || hf == 0 ? s.x : s.y, u = SWIGLU ? s.y : g;
        const uint32_t b0 = tbase + buf * TN + c0, b1 = tbase + buf * TN + c1;
        constexpr int LD = 16;
        uint32_t v[LD];
#pragma unroll
        for (int c = 0; c < 128 / LD; ++c) {
          const int col = c * LD;
          tmem_ld(col < 64 ? b0 + col : b1 + col - 64, v);
          if (c < 128 / LD - 1) join(acc + col / 2, v, col < 64 ? g : u);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.tempty[buf]));
        join(acc + 64 - LD / 2, v, u);
        if (j == SB - 1 || kb == KB - 1) {
          if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.sempty[sb]));
          ++n;
        }
      }
      if (!ok) break;
      const bool valid = i < t.rows;
      const int64_t row = (int64_t)t.row + i;
      if (SWIGLU) {
        if (p.save && valid) {
          store64(p.save + row * p.Nw + n0, acc, p.wide);
          store64(p.save + row * p.Nw + p.N + n0, acc + 32, p.wide);
        }
        const float pr = p.prob && valid ? __ldg(p.prob + row) : 1.f;
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          acc[j].x = pr * (silu_f32(acc[j].x) * acc[32 + j].x);
          acc[j].y = pr * (silu_f32(acc[j].y) * acc[32 + j].y);
          m = max(m, max(fp8::mag_bits(acc[j].x), fp8::mag_bits(acc[j].y)));
        }
        if (p.out && valid) store64(p.out + row * p.N + n0, acc, p.wide);
        if (p.out_q) {
          // the block's other 64 columns are the other warp's of this lane quarter; a
          // buffer is written again two tiles on, behind the next tile's meeting
          ctl.top[parity][hf][i] = m;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.meet[q]));
          if (!tc::mbar_wait(tc::smem_u32(&ctl.meet[q]), parity, wc)) break;
          const float a = fp8::block_top(max(m, ctl.top[parity][hf ^ 1][i])), inv = fp8::block_inverse(a);
          if (valid) {
#pragma unroll
            for (int j = 0; j < 32; j += 16) {
              uint32_t w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float2 x = acc[j + 2 * k], y = acc[j + 2 * k + 1];
                w[k] = fp8::codes4(x.x * inv, x.y * inv, y.x * inv, y.y * inv);
              }
              store32(p.out_q + row * p.N + n0 + 2 * j, w, p.wide);
            }
            if (hf == 0) p.out_sf[row * (p.N / BLOCK) + t.nb] = fp8::block_scale(a);
          }
          parity ^= 1;
        }
      } else if (valid && n0 < p.N) {
        store64(p.out + row * p.N + n0, acc, p.wide);
        store64(p.out + row * p.N + n0 + 64, acc + 32, p.wide);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem_base, 512);
  }
}

// ---- a few rows an expert --------------------------------------------------------
// The time is the weights' bytes, so the weights are the MMAs' 128 rows and up to 16
// of an expert's tokens their columns: a unit is 128 output columns (FC1: of the gate
// and of the up rows) of at most 16 tokens, a stage 128 weight rows x 256 columns of K
// (256 consecutive bytes a row for the DRAM; FC1's stages take gate and up in turn).
// A block's products are then 128 x 16, which four warps join in a few cycles, and
// eight accumulators stand ready, so that no MMA waits for one.  T = 13 of 64 experts,
// 2048 -> 2 x 1024: 32 us among other calls, T = 1 of 256, 2048 -> 7168: 21.6.  By itself,
// with 5 us of the event pair's own and without dependent launches, 39 (the kernel above
// 49; without evict-first weights 45) and 28.7 (36.9; 32.8).  At 16 rows an expert on
// average it takes 0.78 to 1.08 times the other's time (8, 64 and 32 experts), at 32 rows
// 1.06 to 1.31 times.  The choice knows the average alone: rows that all go to a few of
// many experts read those experts' weights again (from the L2) for every 16 of them, 4096
// rows on 64 of 256 experts 508 us against the other kernel's 311, on one 506 against 107.
//   warp 0     TMA producer, 6 stages
//   warp 1     TMEM owner and MMA issuer
//   warp 2     scales: the products sa sw of each token and block, to shared memory
//   warps 4-7  a TMEM lane quarter each; a thread is one output column
constexpr int FT = 16, FSTAGES = 6, FBUFS = 8, FS = 16;
constexpr int F_W_BYTES = 2 * BLOCK * BLOCK, F_A_BYTES = 2 * FT * BLOCK;
constexpr int kFewThreads = 256;
constexpr int kFewRows = 16;  // rows an expert, on average, up to which this kernel is taken

struct FewCtl {
  float scale[FS][2][FT];  // ring of stages: sa sw of the stage's two blocks
  uint64_t full[FSTAGES], empty[FSTAGES], tfull[FBUFS], tempty[FBUFS], sfull[FS], sempty[FS], meet, drain;
  uint32_t tmem_base;
  int abort;
  int off[257], tile_start[257], part[8];
  uint32_t top[2][4][FT];  // unit parity, warp, token
};
constexpr size_t kFewSmem = 1024 + (size_t)FSTAGES * (F_W_BYTES + F_A_BYTES) + sizeof(FewCtl);
static_assert(kFewSmem <= 227 * 1024, "shared memory");

// acc[j] += t[j] s[j] for the 16 tokens.
MOE_D void join_few(float (&acc)[FT], const uint32_t (&t)[FT], const float* s) {
#pragma unroll
  for (int j = 0; j < FT; j += 4) {
    const float4 v = *reinterpret_cast<const float4*>(s + j);
    acc[j] = fmaf(__uint_as_float(t[j]), v.x, acc[j]);
    acc[j + 1] = fmaf(__uint_as_float(t[j + 1]), v.y, acc[j + 1]);
    acc[j + 2] = fmaf(__uint_as_float(t[j + 2]), v.z, acc[j + 2]);
    acc[j + 3] = fmaf(__uint_as_float(t[j + 3]), v.w, acc[j + 3]);
  }
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kFewThreads, 1)
    fp8_product_few_kernel(const __grid_constant__ CUtensorMap tmA,
                           const __grid_constant__ CUtensorMap tmW, const TcParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sW = smem;
  uint8_t* sA = sW + FSTAGES * F_W_BYTES;
  FewCtl& ctl = *reinterpret_cast<FewCtl*>(sA + FSTAGES * F_A_BYTES);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E, KB = p.KB;
  const int nblk = p.N / BLOCK;
  const int KS = (SWIGLU ? 2 : 1) * ((KB + 1) / 2);  // stages of a unit
  // stage ks: FC1 gate (even) or up (odd); its blocks 2 pair and, where there is one, 2 pair + 1
  const auto pair_of = [](int ks) { return SWIGLU ? ks >> 1 : ks; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < FSTAGES; ++s) {
      tc::mbar_init(tc::smem_u32(&ctl.full[s]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.empty[s]), 1);
    }
    for (int b = 0; b < FBUFS; ++b) {
      tc::mbar_init(tc::smem_u32(&ctl.tfull[b]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.tempty[b]), 4);
    }
    for (int s = 0; s < FS; ++s) {
      tc::mbar_init(tc::smem_u32(&ctl.sfull[s]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.sempty[s]), 4);
    }
    tc::mbar_init(tc::smem_u32(&ctl.meet), 4);
    tc::mbar_init(tc::smem_u32(&ctl.drain), 1);
    ctl.abort = 0;
    tc::fence_barrier_init();
    tc::fence_proxy_async_smem();
    tc::prefetch_tensormap(&tmA);
    tc::prefetch_tensormap(&tmW);
  }
  if (warp == 1) {
    tc::tmem_alloc(tc::smem_u32(&ctl.tmem_base), FBUFS * 2 * FT);
    tc::tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  load_tiles<FT>(ctl, p.offsets, E, p.P, nblk);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem_base = ctl.tmem_base;
  const int total = ctl.tile_start[E];
  tc::WaitCtl wc{p.status, &ctl.abort, p.wait_limit_ns, 0};
  tc::WaitCtl wdrain{p.status, nullptr, 1000000000ull, 0};

  if (warp == 0) {
    const bool elected = tc::elect_one();
    const uint64_t policy = tc::evict_first_policy();
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_par = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const Tile t = tile_at<FT>(ctl, E, tile);
      const int w0 = t.e * p.Nw + t.nb * BLOCK;
      for (int ks = 0; ks < KS; ++ks) {
        if (!tc::mbar_wait(tc::smem_u32(&ctl.empty[stage]), phase ^ 1, wc)) { ok = false; break; }
        if (elected) {
          const uint32_t fb = tc::smem_u32(&ctl.full[stage]);
          const uint32_t wd = tc::smem_u32(sW + stage * F_W_BYTES), ad = tc::smem_u32(sA + stage * F_A_BYTES);
          const int kb = 2 * pair_of(ks), blocks = kb + 1 < KB ? 2 : 1;
          const int wr = SWIGLU && (ks & 1) ? w0 + p.N : w0;
          tc::mbar_arrive_expect_tx(fb, blocks * (BLOCK + FT) * BLOCK);
          for (int b = 0; b < blocks; ++b)
            tc::tma_load_2d_hint(wd + b * (BLOCK * BLOCK), &tmW, (kb + b) * BLOCK, wr, fb, policy);
          for (int b = 0; b < blocks; ++b)
            tc::tma_load_2d(ad + b * (FT * BLOCK), &tmA, (kb + b) * BLOCK, t.row, fb);
        }
        __syncwarp();
        issued |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        if (++stage == FSTAGES) { stage = 0; phase ^= 1; }
      }
    }
    for (int s = 0; s < FSTAGES; ++s)
      if ((issued >> s) & 1u)
        tc::mbar_wait(tc::smem_u32(&ctl.full[s]), (issued_par >> s) & 1u, wdrain);
    __syncwarp();
  } else if (warp == 1) {
    const bool elected = tc::elect_one();
    int stage = 0;
    uint32_t phase = 0, step = 0;
    bool ok = true;
    const uint64_t a_base = tc::desc_kmajor_sw128(tc::smem_u32(sA));
    const uint64_t w_base = tc::desc_kmajor_sw128(tc::smem_u32(sW));
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      for (int ks = 0; ks < KS; ++ks, ++step) {
        const uint32_t buf = step % FBUFS;
        if (!tc::mbar_wait(tc::smem_u32(&ctl.tempty[buf]), ((step / FBUFS) & 1) ^ 1, wc) ||
            !tc::mbar_wait(tc::smem_u32(&ctl.full[stage]), phase, wc)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint64_t ad = a_base + (uint32_t)(stage * (F_A_BYTES >> 4));
        const uint64_t wd = w_base + (uint32_t)(stage * (F_W_BYTES >> 4));
        const uint32_t d = tmem_base + buf * (2 * FT);
        const bool two = 2 * pair_of(ks) + 1 < KB;
        if (elected) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_f8(d, wd + 2 * k, ad + 2 * k, tc::idesc_e4m3_f32(BLOCK, FT), k != 0);
          if (two) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_f8(d + FT, wd + (BLOCK * BLOCK >> 4) + 2 * k, ad + (FT * BLOCK >> 4) + 2 * k,
                         tc::idesc_e4m3_f32(BLOCK, FT), k != 0);
          }
          tc::mma_commit(tc::smem_u32(&ctl.empty[stage]));
          tc::mma_commit(tc::smem_u32(&ctl.tfull[buf]));
        }
        __syncwarp();
        if (++stage == FSTAGES) { stage = 0; phase ^= 1; }
      }
    }
    __syncwarp();
    if (ctl.abort) {  // let every issued MMA finish before TMEM is freed
      if (elected) tc::mma_commit(tc::smem_u32(&ctl.drain));
      tc::mbar_wait(tc::smem_u32(&ctl.drain), 0, wdrain);
    }
    __syncwarp();
  } else if (warp == 2) {
    // lane = token + 16 (first or second block of the stage); four stages asked for at a time
    const int tok = lane & 15, half = lane >> 4;
    uint32_t step = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const Tile t = tile_at<FT>(ctl, E, tile);
      const int wblk = p.Nw / BLOCK;
      // (a token behind the expert's takes its last one's scales, which go nowhere)
      const float* sa = p.a_sf + (int64_t)(t.row + min(tok, t.rows - 1)) * KB;
      const float* sw = p.w_sf + ((int64_t)t.e * wblk + t.nb) * KB;
      for (int k0 = 0; k0 < KS && ok; k0 += 4) {
        float s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = min(2 * pair_of(k0 + j) + half, KB - 1);
          s[j] = __ldg(sa + k) * __ldg(sw + (SWIGLU && (j & 1) ? (int64_t)(wblk / 2) * KB : 0) + k);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (k0 + j >= KS) break;
          const uint32_t r = step % FS;
          if (!tc::mbar_wait(tc::smem_u32(&ctl.sempty[r]), ((step / FS) & 1) ^ 1, wc)) { ok = false; break; }
          ctl.scale[r][half][tok] = s[j];
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.sfull[r]));
          ++step;
        }
      }
    }
  } else if (warp >= 4) {
    const int q = warp & 3;
    const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16);
    uint32_t step = 0, parity = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const Tile t = tile_at<FT>(ctl, E, tile);
      float acc[FT], up[FT];
#pragma unroll
      for (int j = 0; j < FT; ++j) acc[j] = up[j] = 0.f;
      for (int ks = 0; ks < KS; ++ks, ++step) {
        const uint32_t buf = step % FBUFS, s = step % FS;
        if (!tc::mbar_wait(tc::smem_u32(&ctl.sfull[s]), (step / FS) & 1, wc) ||
            !tc::mbar_wait(tc::smem_u32(&ctl.tfull[buf]), (step / FBUFS) & 1, wc)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint32_t d = tbase + buf * (2 * FT);
        uint32_t v[FT], w[FT];
        tmem_ld(d, v);
        tmem_ld(d + FT, w);  // (without a second block, what an earlier stage left)
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.tempty[buf]));
        const bool two = 2 * pair_of(ks) + 1 < KB;
        if (SWIGLU && (ks & 1)) {
          join_few(up, v, ctl.scale[s][0]);
          if (two) join_few(up, w, ctl.scale[s][1]);
        } else {
          join_few(acc, v, ctl.scale[s][0]);
          if (two) join_few(acc, w, ctl.scale[s][1]);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.sempty[s]));
      }
      if (!ok) break;
      const int n = t.nb * BLOCK + q * 32 + lane;  // this thread's column
      uint32_t m = 0;                              // lane's token's largest magnitude in the warp's columns
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        if (j >= t.rows) break;
        const int64_t row = t.row + j;
        if (SWIGLU) {
          if (p.save) {
            p.save[row * p.Nw + n] = from_f32<__nv_bfloat16>(acc[j]);
            p.save[row * p.Nw + p.N + n] = from_f32<__nv_bfloat16>(up[j]);
          }
          acc[j] = (p.prob ? __ldg(p.prob + row) : 1.f) * (silu_f32(acc[j]) * up[j]);
          if (p.out_q) {
            const uint32_t r = __reduce_max_sync(0xffffffffu, fp8::mag_bits(acc[j]));
            if (lane == j) m = r;
          }
        }
        if (p.out) p.out[row * p.N + n] = from_f32<__nv_bfloat16>(acc[j]);
      }
      if (SWIGLU && p.out_q) {
        // a unit's 128 columns are one block of each token: its four warps meet, and
        // each lane has a token's scale; a buffer is written again two units on, behind
        // the next unit's meeting
        if (lane < FT) ctl.top[parity][q][lane] = m;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.meet));
        if (!tc::mbar_wait(tc::smem_u32(&ctl.meet), parity, wc)) break;
        const uint32_t(&tp)[4][FT] = ctl.top[parity];
        const int k = lane & (FT - 1);
        const float a = fp8::block_top(max(max(tp[0][k], tp[1][k]), max(tp[2][k], tp[3][k])));
        const float inv = fp8::block_inverse(a);
        if (q == 0 && lane < min(t.rows, FT)) p.out_sf[(int64_t)(t.row + lane) * nblk + t.nb] = fp8::block_scale(a);
#pragma unroll
        for (int j = 0; j < FT; ++j) {
          if (j >= t.rows) break;
          p.out_q[(int64_t)(t.row + j) * p.N + n] =
              (uint8_t)fp8::codes2(acc[j] * __shfl_sync(0xffffffffu, inv, j), 0.f);
        }
        parity ^= 1;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem_base, FBUFS * 2 * FT);
  }
}

// 2-D uint8 [rows, cols] map with a {128, box_rows} box, 128-byte swizzle, zero fill.
bool encode_u8(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  tc::EncodeTiledFn fn = tc::encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols};
  const cuuint32_t box[2] = {(cuuint32_t)BLOCK, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// swiglu (FC1): w = W1 codes [E * 2N, Kd] (gate rows, then up rows, per expert);
// plain (FC2): w = W2 codes [E * N, Kd].
cudaError_t launch_fp8_product(bool swiglu, int P, const uint8_t* a, const float* a_sf, int Kd,
                               const uint8_t* w, const float* w_sf, int E, int N,
                               const int32_t* offsets, const float* prob, void* save, void* out,
                               uint8_t* out_q, float* out_sf, int sms, int* status,
                               cudaStream_t s) {
  if (P == 0) return cudaSuccess;
  const int Nw = swiglu ? 2 * N : N;
  const bool few = P <= (int64_t)kFewRows * E;
  CUtensorMap ma, mw;
  if (!encode_u8(&ma, a, (uint64_t)P, (uint64_t)Kd, few ? 16 : TM)) return cudaErrorInvalidValue;
  if (!encode_u8(&mw, w, (uint64_t)E * Nw, (uint64_t)Kd, BLOCK)) return cudaErrorInvalidValue;
  TcParams p{};
  p.offsets = offsets; p.prob = prob; p.a_sf = a_sf; p.w_sf = w_sf;
  p.save = static_cast<__nv_bfloat16*>(save); p.out = static_cast<__nv_bfloat16*>(out);
  p.out_q = out_q; p.out_sf = out_sf;
  p.P = P; p.E = E; p.KB = Kd / BLOCK; p.N = N; p.Nw = Nw;
  p.wide = ((reinterpret_cast<uintptr_t>(save) | reinterpret_cast<uintptr_t>(out) |
             reinterpret_cast<uintptr_t>(out_q)) & 31u) == 0;
  // up to 64 rows an expert on average most have one row tile: evict-first is 5 to 12%
  // faster at 32 and 64, and 2 to 5% slower at 128 and 256, where tiles share weights
  p.once = P <= 64LL * E;
  p.status = status;
  p.wait_limit_ns = 2000000000ull;
  const int nblk = swiglu || few ? N / BLOCK : (N + TN - 1) / TN;
  const int64_t tiles_max = (ceil_div(P, few ? FT : TM) + (E < P ? E : P)) * (int64_t)nblk;
  const int grid = (int)(tiles_max < sms ? tiles_max : sms);
  auto kern = few ? (swiglu ? fp8_product_few_kernel<true> : fp8_product_few_kernel<false>)
                  : (swiglu ? fp8_product_kernel<true> : fp8_product_kernel<false>);
  const int threads = few ? kFewThreads : kThreads;
  const size_t smem = few ? kFewSmem : kSmem;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return pdl_launch(kern, dim3(grid), dim3(threads), smem, s, ma, mw, p);
}

}  // namespace moe
