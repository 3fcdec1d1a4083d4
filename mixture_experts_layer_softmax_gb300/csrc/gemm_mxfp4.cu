// MXFP4: quantisation, its inverse, and the expert GEMMs on 4-bit operands:
// E2M1 codes with one E8M0 scale per 1 x 32 block along K, block-scaled MMAs on
// the 5th-generation tensor cores (tcgen05.mma kind::mxf4, scales in TMEM),
// fp32 accumulate.
//
// "Scalable Training of Mixture-of-Experts Models with Megatron Core" (review),
// §5.3 low-precision recipes: the microscaled formats native to Blackwell.
// Element and scale rules are the OCP Microscaling v1.0 ones of MXFP4: shared
// exponent X = floor(log2 max|x|) - 2 (E2M1's largest binade is 2^2), element =
// x / 2^X rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the
// even code), saturated to +-6.
//
// Operand format (written by mxfp4_quantize_kernel or by the FC1 epilogue):
//   codes  [rows, K / 2] uint8, two columns a byte (the even column in bits
//          0-3), code = sign << 3 | exponent << 1 | mantissa;
//   scales in the atoms of mx.cuh, the same as MXFP8's.
//
// GEMM kernel (persistent, 1 CTA per SM, 576 threads), the roles of the MXFP8
// kernel with twice the columns per stage:
//   warp 0     TMA producer: 4 stages of {A 128 x 128 B, B 256 x 128 B} = 256
//              columns (128-byte swizzle) plus two scale atoms per 128 rows.
//   warp 1     TMEM owner and MMA issuer: per stage, tcgen05.cp of six atoms
//              into the stage's 24 TMEM columns, then 4 MMAs M128 N256 K64
//              (atom k / 2, scale bytes 2 (k % 2) and the next).
//   warps 2-17 epilogue; FC1 can re-quantise a.
// K is a multiple of 128; an odd last 128 columns are half a stage (the box's
// other half is zero fill and gets no MMA).
// Every wait is bounded; a wait that gives up records MOE_ERR_TIMEOUT and
// every role leaves its loop.
#include <cuda_fp4.h>

#include "mx.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

using mx::ATOM;
constexpr int BM = 128, BN = 256;
constexpr int BK = 256, BKB = 128;  // K elements and bytes per row and stage
constexpr int A_BYTES = BM * BKB;   // 16 KB
constexpr int B_BYTES = BN * BKB;   // 32 KB
constexpr int SF_BYTES = 6 * ATOM;  // two atoms per 128 rows of A and B
constexpr int STAGES = 4;
constexpr int kEpiWarps = 16;  // four per TMEM lane quarter, each a quarter of the columns
constexpr int kThreads = 64 + 32 * kEpiWarps;  // producer, MMA, epilogue
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t SF_COL0 = 256, SF_STRIDE = 32;  // per stage: A scales +0..7, B +8..23

enum Mx4Mode { kSwiGLU = 0, kPlain = 1 };

struct Mx4Params {
  const int32_t* offsets;  // [E+1]
  const float* prob;       // FC1: [P] or null
  const uint8_t* a_sf;     // A scale atoms
  const uint8_t* b_sf;     // B scale atoms (uniform groups of Nb rows)
  __nv_bfloat16* out;      // [P, N] bf16 or null
  uint8_t* out_q;          // FC1: codes of a [P, N / 2] or null
  uint8_t* out_sf;         // FC1: scale atoms of a
  int P, E, Kd, N, Nb;
  bool wide;               // out is 32-byte aligned (its rows are multiples of 256 bytes)
  int* status;
  uint64_t wait_limit_ns;
};

struct Mx4Ctl {
  uint64_t full[STAGES], empty[STAGES], tmem_full, tmem_empty, drain;
  uint32_t tmem_base;
  int abort;
  int tile_start[257];  // GEMM tiles before expert e
  int rtile[257];       // 128-row tiles before expert e (scale atom numbering)
  int off[257];
};

constexpr size_t kSmem = 1024 + (size_t)STAGES * (A_BYTES + B_BYTES + SF_BYTES) + sizeof(Mx4Ctl);

// ---- E8M0 / E2M1 helpers ------------------------------------------------------
// E8M0 code of a block whose largest magnitude has the fp32 bits `abits`: X + 127
// with X = floor(log2 amax) - 2 clamped at -127.  A block that holds an infinity
// or a NaN (exponent field 255) gets 255, the format's NaN.
MOE_D uint32_t e8m0_code(uint32_t abits) {
  const uint32_t e = abits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^-X for scale code c; 0 for the NaN block (its codes are 0).
MOE_D float e8m0_inverse(uint32_t c) { return c == 255u ? 0.f : __uint_as_float((254u - c) << 23); }

// 8 values (already divided by the scale) -> 8 E2M1 codes, the first in the
// low bits, round to nearest even with saturation.
MOE_D uint32_t e2m1x8(const float* v) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_E2M1,
                                            cudaRoundNearest)
         << (8 * i);
  return w;
}

MOE_D uint32_t pack_bf16x2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// SiLU with the approximate exponential and reciprocal: the exact ones kept the
// epilogue warps busy for longer than the tile's MMAs.  CUDA bounds __expf(-z) by
// 2 + |1.173 z| units in the last place and __fdividef by 2, so the value is off by
// 2^-23 (5 + 1.2 |z|) of itself: below 2^-16 for every z whose SiLU is a normal number
// (z > -92), beside half steps of 2^-8 (bf16) and 2^-2 (E2M1).  A reciprocal below
// 2^-126 is 0, and exp(-z) overflowing gives -0, SiLU's limit; NaN stays.
MOE_D float silu_fast(float z) { return z * __fdividef(1.f, 1.f + __expf(-z)); }

// 32 lanes x two groups of 32 columns: both loads in flight, then one wait, in one
// asm statement (no register is read before the data has arrived).
MOE_D void tmem_ld_x32x2(uint32_t ta, uint32_t tb, float (&a)[32], float (&b)[32]) {
#define MOE_F8(v, i) "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3]), "=f"(v[i + 4]), \
                     "=f"(v[i + 5]), "=f"(v[i + 6]), "=f"(v[i + 7])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : MOE_F8(a, 0), MOE_F8(a, 8), MOE_F8(a, 16), MOE_F8(a, 24), MOE_F8(b, 0), MOE_F8(b, 8),
        MOE_F8(b, 16), MOE_F8(b, 24)
      : "r"(ta), "r"(tb)
      : "memory");
#undef MOE_F8
}

// 32 values of a row as bf16: 32-byte stores (whole sectors) where the output
// allows them, 16-byte ones elsewhere.
MOE_D void store_row32(__nv_bfloat16* dst, const float (&a)[32], bool wide) {
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = pack_bf16x2(a[2 * j], a[2 * j + 1]);
  if (wide) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + 16 * j),
                   "r"(w[8 * j]), "r"(w[8 * j + 1]), "r"(w[8 * j + 2]), "r"(w[8 * j + 3]),
                   "r"(w[8 * j + 4]), "r"(w[8 * j + 5]), "r"(w[8 * j + 6]), "r"(w[8 * j + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<uint4*>(dst + 8 * j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  }
}

// ---- quantiser and its inverse ----------------------------------------------------
// A block takes units of 128 rows (a scale tile) by 128 columns: eight threads a
// row, 16 columns each, rows 32 apart in turn, so that a thread's four rows have
// their scale words side by side and a unit's 512-byte atom is stored whole.
// (Whole rows at a time, with a 4-byte scale store a chunk, measured 4.6 TB/s.)
// All of a thread's loads go out before the first is used.
// Groups: offsets [G+1] on the device, or uniform groups of `urows` rows; rows of
// no group (before the first, after the last) form tiles without scales.
struct Tiles {
  int off[257], rt[257];
};
struct Tile {
  int row0, rows;    // first row, rows (at most 128)
  int64_t scale;     // scale tile, -1: none
};

// Scale tiles a buffer has room for (descending offsets could ask for more).
MOE_D int64_t tiles_room(int rows, int G) { return ((int64_t)rows + 127) / 128 + G; }

MOE_D int64_t tiles_total(const Tiles& t, bool ragged, int rows, int G, int urows) {
  if (!ragged) return (int64_t)G * ((urows + 127) / 128);
  return (int64_t)t.rt[G] + (t.off[0] + 127) / 128 + (rows - t.off[G] + 127) / 128;
}

MOE_D Tile tile_at(const Tiles& t, bool ragged, int rows, int G, int urows, int64_t i) {
  Tile o;
  o.scale = i;
  if (!ragged) {
    const int per = (urows + 127) / 128;
    const int g = (int)(i / per), lr = (int)(i - (int64_t)g * per) * 128;
    o.row0 = g * urows + lr;
    o.rows = min(128, urows - lr);
  } else if (i < t.rt[G]) {
    int lo = 0, hi = G - 1;  // the last group with rt[g] <= i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.rt[mid] <= i) lo = mid; else hi = mid - 1;
    }
    o.row0 = t.off[lo] + (int)(i - t.rt[lo]) * 128;
    o.rows = min(128, t.off[lo + 1] - o.row0);
    if (i >= tiles_room(rows, G)) o.scale = -1;
  } else {
    int k = (int)(i - t.rt[G]);
    const int before = (t.off[0] + 127) / 128;
    o.scale = -1;
    o.row0 = k < before ? k * 128 : t.off[G] + (k - before) * 128;
    o.rows = min(128, (k < before ? t.off[0] : rows) - o.row0);
  }
  return o;
}

__global__ void __launch_bounds__(256)
    mxfp4_quantize_kernel(const __nv_bfloat16* __restrict__ x, int rows, int K, int G,
                          const int32_t* __restrict__ offsets, int urows,
                          uint8_t* __restrict__ q, uint8_t* __restrict__ sf) {
  __shared__ Tiles s_t;
  const bool ragged = offsets != nullptr;
  if (ragged) mx::load_groups(offsets, G, rows, s_t.off, s_t.rt);
  const int KB = K / 128;
  const int sub = threadIdx.x & 7, row = threadIdx.x >> 3;
  const int64_t units = tiles_total(s_t, ragged, rows, G, urows) * KB;
  for (int64_t un = blockIdx.x; un < units; un += gridDim.x) {
    const int64_t ti = un / KB;
    const int kb = (int)(un - ti * KB);
    const Tile tile = tile_at(s_t, ragged, rows, G, urows, ti);
    uint4 raw[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int lr = 32 * u + row;
      raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
      if (lr < tile.rows) {
        const uint4* src = reinterpret_cast<const uint4*>(x + (int64_t)(tile.row0 + lr) * K + kb * 128 + sub * 16);
        raw[u][0] = __ldcs(src);
        raw[u][1] = __ldcs(src + 1);
      }
    }
    uint32_t words[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int lr = 32 * u + row;
      const uint32_t w[8] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w,
                             raw[u][1].x, raw[u][1].y, raw[u][1].z, raw[u][1].w};
      uint32_t hi = 0, lo = 0;  // largest magnitudes of the odd and even columns, as bits
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        hi = max(hi, w[i] & 0x7fff0000u);
        lo = max(lo, w[i] & 0x00007fffu);
      }
      uint32_t abits = max(hi, lo << 16);
      abits = max(abits, __shfl_xor_sync(0xffffffffu, abits, 1));  // two threads a block
      const uint32_t code = e8m0_code(abits);
      const float inv = e8m0_inverse(code);
      float v[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // exact: a power of two
        v[2 * i] = __uint_as_float(w[i] << 16) * inv;
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * inv;
      }
      uint2 codes = make_uint2(e2m1x8(v), e2m1x8(v + 8));
      if (code == 255u) codes = make_uint2(0u, 0u);
      const uint32_t c1 = __shfl_down_sync(0xffffffffu, code, 2);
      const uint32_t c2 = __shfl_down_sync(0xffffffffu, code, 4);
      const uint32_t c3 = __shfl_down_sync(0xffffffffu, code, 6);
      words[u] = code | (c1 << 8) | (c2 << 16) | (c3 << 24);
      if (lr < tile.rows)
        *reinterpret_cast<uint2*>(q + (int64_t)(tile.row0 + lr) * (K / 2) + kb * 64 + sub * 8) = codes;
    }
    if (sub == 0 && tile.scale >= 0)  // past the group's end: scale 2^-127 of zeros
      *reinterpret_cast<uint4*>(sf + mx::atom_word(tile.scale, KB, kb, row)) =
          make_uint4(words[0], words[1], words[2], words[3]);
  }
}

// Eight E2M1 codes times a block's scale -> eight bf16 values, exact: the code's
// exponent and mantissa bits placed in a bf16's give value / 2^126 (the zero
// exponent's 0.5 too, as a subnormal), which 2^126 and the scale bring back.
MOE_D uint4 e2m1x8_to_bf16(uint32_t w, float scale) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t c = w >> (8 * j + 4 * b);
      v[b] = __uint_as_float((c & 8u) << 28 | (c & 7u) << 22) * 0x1p126f * scale;
    }
    o[j] = pack_bf16x2(v[0], v[1]);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Codes and scales -> bf16 values, in the quantiser's units; 16 threads a row,
// eight columns each, so that a warp's 16-byte stores fill whole sectors (16
// columns a thread in two stores: 4.5 TB/s over 940M values, this 6.2).  Rows of no group
// are left as they are.
__global__ void __launch_bounds__(256)
    mxfp4_dequantize_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sf, int rows,
                            int K, int G, const int32_t* __restrict__ offsets, int urows,
                            __nv_bfloat16* __restrict__ x) {
  __shared__ Tiles s_t;
  const bool ragged = offsets != nullptr;
  if (ragged) mx::load_groups(offsets, G, rows, s_t.off, s_t.rt);
  const int KB = K / 128;
  const int sub = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int64_t units = (ragged ? (int64_t)s_t.rt[G] : tiles_total(s_t, false, rows, G, urows)) * KB;
  for (int64_t un = blockIdx.x; un < units; un += gridDim.x) {
    const int64_t ti = un / KB;
    const int kb = (int)(un - ti * KB);
    const Tile tile = tile_at(s_t, ragged, rows, G, urows, ti);
    if (tile.scale < 0) continue;
    uint32_t codes[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int lr = 16 * u + row;
      codes[u] = 0u;
      if (lr < tile.rows)
        codes[u] = __ldcs(reinterpret_cast<const uint32_t*>(q + (int64_t)(tile.row0 + lr) * (K / 2) + kb * 64 + sub * 4));
    }
    // rows i and i + 16, each with the words of rows 32, 64 and 96 further on
    const uint8_t* atom = sf + mx::atom_word(tile.scale, KB, kb, row);
    const uint4 w0 = __ldg(reinterpret_cast<const uint4*>(atom));
    const uint4 w1 = __ldg(reinterpret_cast<const uint4*>(atom + 256));
    const uint32_t words[8] = {w0.x, w1.x, w0.y, w1.y, w0.z, w1.z, w0.w, w1.w};
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int lr = 16 * u + row;
      if (lr >= tile.rows) continue;
      const float s = mx::e8m0_value(words[u] >> (8 * (sub >> 2)) & 255u);
      __stcs(reinterpret_cast<uint4*>(x + (int64_t)(tile.row0 + lr) * K + kb * 128 + sub * 8),
             e2m1x8_to_bf16(codes[u], s));
    }
  }
}

// ---- GEMM -------------------------------------------------------------------------
MOE_D void decode_tile(const Mx4Ctl& c, int E, int tile, int& e, int& mb, int& nb) {
  int lo = 0, hi = E - 1;  // largest e with tile_start[e] <= tile
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c.tile_start[mid] <= tile) lo = mid; else hi = mid - 1;
  }
  e = lo;
  const int local = tile - c.tile_start[e];
  const int mblk = (c.off[e + 1] - c.off[e] + BM - 1) / BM;
  nb = local / mblk;
  mb = local - nb * mblk;
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_mxfp4_kernel(const __grid_constant__ CUtensorMap tmA,
                              const __grid_constant__ CUtensorMap tmB, const Mx4Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * A_BYTES;
  uint8_t* sSF = sB + STAGES * B_BYTES;
  Mx4Ctl& ctl = *reinterpret_cast<Mx4Ctl*>(sSF + STAGES * SF_BYTES);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E;
  const int nblk = MODE == kSwiGLU ? (p.N + 127) / 128 : (p.N + BN - 1) / BN;
  const int KB = p.Kd / 128;     // scale atoms along K
  const int KS = (p.Kd + BK - 1) / BK;  // stages along K; the last may hold one atom
  const int nbt = p.Nb / 128;  // B row tiles per expert

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      tc::mbar_init(tc::smem_u32(&ctl.full[s]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.empty[s]), 1);
    }
    tc::mbar_init(tc::smem_u32(&ctl.tmem_full), 1);
    tc::mbar_init(tc::smem_u32(&ctl.tmem_empty), kEpiWarps);
    tc::mbar_init(tc::smem_u32(&ctl.drain), 1);
    ctl.abort = 0;
    tc::fence_barrier_init();
    tc::fence_proxy_async_smem();
    tc::prefetch_tensormap(&tmA);
    tc::prefetch_tensormap(&tmB);
  }
  if (warp == 1) {
    tc::tmem_alloc(tc::smem_u32(&ctl.tmem_base), TMEM_COLS);
    tc::tmem_relinquish();
  }
  // (kept within the rows here, and ascending below: no offsets reach past a tensor)
  for (int e = threadIdx.x; e <= E; e += kThreads) ctl.off[e] = min(max(__ldg(p.offsets + e), 0), p.P);
  __syncthreads();
  if (warp == 2) {  // tile_start and rtile: exclusive scans over the experts
    int run_t = 0, run_r = 0, run_o = ctl.off[0];
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      int end = max(run_o, e < E ? ctl.off[e + 1] : 0);  // expert e's end: the largest offset so far
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end = max(end, t);
      }
      const int prev = __shfl_up_sync(0xffffffffu, end, 1), beg = lane ? prev : run_o;
      if (e < E) ctl.off[e + 1] = end;
      run_o = __shfl_sync(0xffffffffu, end, 31);
      const int mblk = (end - beg + BM - 1) / BM;
      int it = mblk * nblk, ir = mblk;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, it, o);
        const int r = __shfl_up_sync(0xffffffffu, ir, o);
        if (lane >= o) { it += t; ir += r; }
      }
      if (e < E) {
        ctl.tile_start[e] = run_t + it - mblk * nblk;
        ctl.rtile[e] = run_r + ir - mblk;
      }
      run_t += __shfl_sync(0xffffffffu, it, 31);
      run_r += __shfl_sync(0xffffffffu, ir, 31);
    }
    if (lane == 0) ctl.tile_start[E] = run_t;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem_base = ctl.tmem_base;
  const int total = ctl.tile_start[E];
  tc::WaitCtl wc{p.status, &ctl.abort, p.wait_limit_ns, 0};
  tc::WaitCtl wdrain{p.status, nullptr, 1000000000ull, 0};

  if (warp == 0) {
    // ================= TMA producer =================
    {  // the whole warp, one elected lane issuing: see the MMA issuer
      const bool elected = tc::elect_one();
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_par = 0;
      for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
        int e, mb, nb;
        decode_tile(ctl, E, tile, e, mb, nb);
        const int a_row = ctl.off[e] + mb * BM;
        const int64_t a_atom = (int64_t)(ctl.rtile[e] + mb) * KB;
        int b_row0, b_row1;
        int64_t b_atom0, b_atom1;
        bool two_b = true;
        if (MODE == kSwiGLU) {  // gate rows nb*128.., up rows N + nb*128..
          b_row0 = e * p.Nb + nb * 128;
          b_row1 = e * p.Nb + p.N + nb * 128;
          b_atom0 = ((int64_t)e * nbt + nb) * KB;
          b_atom1 = ((int64_t)e * nbt + p.N / 128 + nb) * KB;
        } else {
          b_row0 = e * p.Nb + nb * BN;
          b_row1 = b_row0 + 128;
          b_atom0 = ((int64_t)e * nbt + 2 * nb) * KB;
          b_atom1 = b_atom0 + KB;
          two_b = nb * BN + 128 < p.N;  // a half past N has no scale atom to read
        }
        bool ok = true;
        for (int ks = 0; ks < KS; ++ks) {
          if (!tc::mbar_wait(tc::smem_u32(&ctl.empty[stage]), phase ^ 1, wc)) { ok = false; break; }
          const int kb = 2 * ks;
          const uint32_t sfb = (kb + 1 < KB ? 2 : 1) * ATOM;  // scale bytes per 128 rows
          const uint32_t fb = tc::smem_u32(&ctl.full[stage]);
          if (elected) {
            tc::mbar_arrive_expect_tx(fb, A_BYTES + B_BYTES + (two_b ? 3 : 2) * sfb);
            const uint32_t a_dst = tc::smem_u32(sA + stage * A_BYTES);
            const uint32_t b_dst = tc::smem_u32(sB + stage * B_BYTES);
            const uint32_t sf_dst = tc::smem_u32(sSF + stage * SF_BYTES);
            tc::tma_load_2d(a_dst, &tmA, ks * BKB, a_row, fb);
            tc::tma_load_2d(b_dst, &tmB, ks * BKB, b_row0, fb);
            tc::tma_load_2d(b_dst + B_BYTES / 2, &tmB, ks * BKB, b_row1, fb);
            tc::bulk_load(sf_dst, p.a_sf + (a_atom + kb) * ATOM, sfb, fb);
            tc::bulk_load(sf_dst + 2 * ATOM, p.b_sf + (b_atom0 + kb) * ATOM, sfb, fb);
            if (two_b) tc::bulk_load(sf_dst + 4 * ATOM, p.b_sf + (b_atom1 + kb) * ATOM, sfb, fb);
          }
          __syncwarp();
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
      }
      for (int s = 0; s < STAGES; ++s)
        if ((issued >> s) & 1u)
          tc::mbar_wait(tc::smem_u32(&ctl.full[s]), (issued_par >> s) & 1u, wdrain);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ================= MMA issuer =================
    // The whole warp runs the loop, so that the descriptors are warp-uniform and
    // stay in uniform registers; one elected lane issues.  (One lane running the
    // loop alone moves every operand of every instruction there first: 1130
    // cycles a stage against the MMAs' 512.)
    {
      const bool elected = tc::elect_one();
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      const uint64_t a_base = tc::desc_kmajor_sw128(tc::smem_u32(sA));
      const uint64_t b_base = tc::desc_kmajor_sw128(tc::smem_u32(sB));
      const uint64_t sf_base = tc::desc_sf_atom(tc::smem_u32(sSF));
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        if (!tc::mbar_wait(tc::smem_u32(&ctl.tmem_empty), acc_phase ^ 1, wc)) break;
        tc::fence_after_sync();
        for (int ks = 0; ks < KS; ++ks) {
          if (!tc::mbar_wait(tc::smem_u32(&ctl.full[stage]), phase, wc)) { ok = false; break; }
          tc::fence_after_sync();
          // addresses in 16-byte units, added to the descriptors
          const uint64_t ad = a_base + (uint32_t)(stage * (A_BYTES >> 4));
          const uint64_t bd = b_base + (uint32_t)(stage * (B_BYTES >> 4));
          const uint64_t sd = sf_base + (uint32_t)(stage * (SF_BYTES >> 4));
          const uint32_t sfa = tmem_base + SF_COL0 + stage * SF_STRIDE;
          const bool two = 2 * ks + 1 < KB;  // both atoms
          if (elected) {
            // atom j: A scales in columns 4j .. 4j+3, B scales in 8 + 8j .. 8 + 8j + 7
            tc::tmem_cp_32x128b_warpx4(sfa, sd);
            tc::tmem_cp_32x128b_warpx4(sfa + 8, sd + 2 * (ATOM >> 4));
            tc::tmem_cp_32x128b_warpx4(sfa + 12, sd + 4 * (ATOM >> 4));
            // 64 columns (32 bytes, two blocks) an MMA
            tc::mma_mxf4(tmem_base, ad, bd, tc::idesc_mxf4_e2m1(BM, BN, 0, 0), sfa, sfa + 8, ks != 0);
            tc::mma_mxf4(tmem_base, ad + 2, bd + 2, tc::idesc_mxf4_e2m1(BM, BN, 2, 2), sfa, sfa + 8, 1);
            if (two) {
              tc::tmem_cp_32x128b_warpx4(sfa + 4, sd + (ATOM >> 4));
              tc::tmem_cp_32x128b_warpx4(sfa + 16, sd + 3 * (ATOM >> 4));
              tc::tmem_cp_32x128b_warpx4(sfa + 20, sd + 5 * (ATOM >> 4));
              tc::mma_mxf4(tmem_base, ad + 4, bd + 4, tc::idesc_mxf4_e2m1(BM, BN, 0, 0), sfa + 4, sfa + 16, 1);
              tc::mma_mxf4(tmem_base, ad + 6, bd + 6, tc::idesc_mxf4_e2m1(BM, BN, 2, 2), sfa + 4, sfa + 16, 1);
            }
            tc::mma_commit(tc::smem_u32(&ctl.empty[stage]));
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        if (elected) tc::mma_commit(tc::smem_u32(&ctl.tmem_full));
        acc_phase ^= 1;
      }
      __syncwarp();
      if (ctl.abort) {  // let every issued MMA finish before TMEM is freed
        if (elected) tc::mma_commit(tc::smem_u32(&ctl.drain));
        tc::mbar_wait(tc::smem_u32(&ctl.drain), 0, wdrain);
      }
    }
    __syncwarp();
  } else {
    // ================= epilogue (warps 2..17) =================
    // four warps per TMEM lane quarter, each taking a quarter of the tile's
    // columns; each releases the accumulator as soon as its TMEM reads are done
    // (eight warps with twice the columns spilled, and left too few instructions
    // in flight: FC1 at 16384 rows 698 us)
    const int q = warp & 3;          // TMEM lane quarter this warp may access
    const int qt = (warp - 2) >> 2;  // which quarter of the columns
    uint32_t acc_phase = 0;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
      int e, mb, nb;
      decode_tile(ctl, E, tile, e, mb, nb);
      if (!tc::mbar_wait(tc::smem_u32(&ctl.tmem_full), acc_phase, wc)) break;
      tc::fence_after_sync();
      const int m_e = ctl.off[e + 1] - ctl.off[e];
      const int i = q * 32 + lane;  // row within the tile
      const bool valid = mb * BM + i < m_e;
      const int64_t row = (int64_t)ctl.off[e] + mb * BM + i;
      const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16);
      // all of the warp's TMEM reads in flight together, then the release, then
      // the math; a warp whose rows are all past the expert's end only releases
      const bool any = mb * BM + q * 32 < m_e;
      float v[2][32];
      if (any) {
        const uint32_t c0 = MODE == kSwiGLU ? qt * 32 : qt * 64;
        const uint32_t c1 = MODE == kSwiGLU ? 128 + qt * 32 : qt * 64 + 32;
        tmem_ld_x32x2(tbase + c0, tbase + c1, v[0], v[1]);
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.tmem_empty));
      acc_phase ^= 1;
      if (!any) continue;
      if (MODE == kSwiGLU) {
        // columns: gate qt*32 .. +31 and the matching up columns
        const float pr = (p.prob && valid) ? __ldg(p.prob + row) : 1.f;
        const int n = nb * 128 + qt * 32;
        float (&a)[32] = v[0];
#pragma unroll
        for (int j = 0; j < 32; ++j) a[j] = pr * (silu_fast(v[0][j]) * v[1][j]);
        if (valid && p.out) store_row32(p.out + row * p.N + n, a, p.wide);
        if (p.out_q) {  // one block of FC2's A operand
          uint32_t abits = 0;
#pragma unroll
          for (int j = 0; j < 32; ++j) abits = max(abits, __float_as_uint(a[j]) & 0x7fffffffu);
          const uint32_t code = e8m0_code(abits);
          const float inv = e8m0_inverse(code);
#pragma unroll
          for (int j = 0; j < 32; ++j) a[j] *= inv;
          if (valid) {
            const uint32_t keep = code == 255u ? 0u : ~0u;  // codes of a NaN block: 0, as the quantiser's
            *reinterpret_cast<uint4*>(p.out_q + (row * p.N + n) / 2) =
                make_uint4(e2m1x8(a) & keep, e2m1x8(a + 8) & keep, e2m1x8(a + 16) & keep, e2m1x8(a + 24) & keep);
            // its scale: atom (rtile[e] + mb, kb = nb), row i, block qt
            p.out_sf[mx::atom_word(ctl.rtile[e] + mb, p.N / 128, nb, i) + qt] = (uint8_t)code;
          }
        }
      } else if (valid) {
        // columns qt*64 .. +63
        const int n = nb * BN + qt * 64;
        if (n < p.N) {
          store_row32(p.out + row * p.N + n, v[0], p.wide);
          store_row32(p.out + row * p.N + n + 32, v[1], p.wide);
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ---- host side ----------------------------------------------------------------------
// 2-D uint8 [rows, bytes] map with a {128, 128} box, 128-byte swizzle, zero fill.
bool encode_codes(CUtensorMap* m, const void* base, uint64_t rows, uint64_t bytes) {
  tc::EncodeTiledFn fn = tc::encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {bytes, rows};
  const cuuint64_t strides[1] = {bytes};
  const cuuint32_t box[2] = {(cuuint32_t)BKB, 128};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks for the quantiser and its inverse: as many as run at once, fewer where
// there are fewer units (counted from above for ragged groups).
int unit_grid(int rows, int groups, bool ragged, int KB, int sms) {
  const int64_t tiles = ragged ? ceil_div(rows, 128) + (groups < rows ? groups : rows) + 2
                               : (int64_t)groups * ceil_div(rows / groups, 128);
  const int64_t most = 4LL * sms;
  return (int)(tiles * KB < most ? tiles * KB : most);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(int rows, int K, int groups, const int32_t* offsets,
                                  const void* x, uint8_t* q, uint8_t* sf, int sms,
                                  cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const int grid = unit_grid(rows, groups, offsets != nullptr, K / 128, sms);
  mxfp4_quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(x), rows, K, groups,
                                             offsets, offsets ? 0 : rows / groups, q, sf);
  return cudaGetLastError();
}

cudaError_t launch_mxfp4_dequantize(int rows, int K, int groups, const int32_t* offsets,
                                    const uint8_t* q, const uint8_t* sf, void* x, int sms,
                                    cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const int grid = unit_grid(rows, groups, offsets != nullptr, K / 128, sms);
  mxfp4_dequantize_kernel<<<grid, 256, 0, s>>>(q, sf, rows, K, groups, offsets,
                                               offsets ? 0 : rows / groups,
                                               static_cast<__nv_bfloat16*>(x));
  return cudaGetLastError();
}

// One MXFP4 grouped GEMM.  swiglu (FC1): A = x_perm [P, Kd], B = W1 [E * 2N, Kd]
// (gate rows then up rows per expert), out = a [P, N] bf16 (or null) and/or
// out_q / out_sf = a re-quantised for FC2; prob scales a.  Plain (FC2): B = W2
// [E * N, Kd], out [P, N] bf16.
cudaError_t launch_grouped_gemm_mxfp4(bool swiglu, int P, const uint8_t* A, const uint8_t* A_sf,
                                      int Kd, const uint8_t* B, const uint8_t* B_sf, int Nb,
                                      int E, int N, const int32_t* offsets, const float* prob,
                                      void* out, uint8_t* out_q, uint8_t* out_sf, int sms,
                                      int* status, cudaStream_t s) {
  if (P == 0) return cudaSuccess;
  CUtensorMap ma, mb;
  if (!encode_codes(&ma, A, (uint64_t)P, (uint64_t)Kd / 2)) return cudaErrorInvalidValue;
  if (!encode_codes(&mb, B, (uint64_t)E * Nb, (uint64_t)Kd / 2)) return cudaErrorInvalidValue;
  Mx4Params p{};
  p.offsets = offsets; p.prob = prob; p.a_sf = A_sf; p.b_sf = B_sf;
  p.out = static_cast<__nv_bfloat16*>(out); p.out_q = out_q; p.out_sf = out_sf;
  p.P = P; p.E = E; p.Kd = Kd; p.N = N; p.Nb = Nb;
  p.wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  p.status = status;
  p.wait_limit_ns = 2000000000ull;
  const int nblk = swiglu ? (N + 127) / 128 : (N + BN - 1) / BN;
  const int64_t tiles_max = (ceil_div(P, BM) + E) * (int64_t)nblk;
  const int grid = (int)(tiles_max < sms ? tiles_max : sms);
  auto kern = swiglu ? grouped_gemm_mxfp4_kernel<kSwiGLU> : grouped_gemm_mxfp4_kernel<kPlain>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, kSmem, s>>>(ma, mb, p);
  return cudaGetLastError();
}

}  // namespace moe
