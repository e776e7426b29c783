// The E4M3 product with one scale per token and 128 deep group and one per 128 x 128
// block of the weight:
//
//   y[t,n] = sum_g xs[t,g] ws[n/128,g] sum_{k in g} xq[t,k] wq[n,k]
//
// Both operands are stored with the contraction contiguous.  A block is 128 x 128 both
// ways, so the codes of W [H,N] transposed serve the forward and, as they are, the
// gradient dx = dy W^T with the same scales.  Each group's sums start from zero, are
// scaled once by xs ws in float32 and added in group order (by each of the waves or parts that
// share a column tile's groups, whose sums are then added in their order).
//
// In every kernel the weight is the matrix instruction's first operand (its rows are
// the output's columns) and the tokens the second, so that a lane of the accumulator
// holds ONE token and several output columns: a token's scale is then one register of
// the lane, and a block's a scalar.
//
// Measured: 5 tokens at H = 7168, N = 4096 10.4 us (29 MB: 2.8 TB/s, latency counts);
// 8192 tokens there 33 us for the codes and 205 us for the product, 2.3 PFLOP/s, as the
// fastest of a run, 245 us at the clock that a sustained run leaves (the scaling's vector
// operations share the issue slots and the power with the matrix instructions, which are
// busy 60% of the time; a library product without scales takes 177 us).
#include "gemm_common.h"
#include "kernels.h"
#include "quant_core.h"

namespace hmm {
namespace {

constexpr int G = 128;  // group and block size

// ------------------------------------------------------------ weight quantiser
// One workgroup per block: every thread keeps 8 rows of an 8-column chunk, the maximum
// crosses the workgroup once, and the codes go out as they are and, through LDS, transposed.
// Bound by HBM and, at a few megabytes, by its one round of workgroups: 4096 x 2048 9.1 us (34 MB).
constexpr int QB_THREADS = 256;
constexpr int QB_PITCH = G + 8;

__global__ void __launch_bounds__(QB_THREADS) quant_block(const uint16_t* __restrict__ w, int64_t H, int64_t N, int hbs,
                                                          int nbs, uint8_t* __restrict__ qt, uint8_t* __restrict__ q,
                                                          float* __restrict__ ds) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[G * QB_PITCH];
  __shared__ float wmax[QB_THREADS / 64];
  const int64_t b = blockIdx.x;
  const int nb = (int)(b % nbs), hb = (int)(b / nbs % hbs);
  const int64_t e = b / nbs / hbs;
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4;  // column chunk, group of 8 rows
  const int64_t n = (int64_t)nb * G + c * 8, h = (int64_t)hb * G + r * 8;
  const bool in = n < N;
  u32x4 raw[8];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    raw[i] = in ? *reinterpret_cast<const u32x4*>(w + (e * H + h + i) * N + n) : u32x4{0, 0, 0, 0};
    float v[8];
    unpack8(raw[i], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < QB_THREADS / 64; ++k) m = fmaxf(m, wmax[k]);
  const float sc = block_scale_of(m);
  if (threadIdx.x == 0) ds[(e * nbs + nb) * hbs + hb] = 1.f / sc;
  float s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = sc;
  uint2 code[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v[8];
    unpack8(raw[i], v);
    code[i] = to_e4m3x8(v, s);
    if (q && in) *reinterpret_cast<uint2*>(q + (e * H + h + i) * N + n) = code[i];
  }
  if (!qt) return;  // the same for every thread
  // 8 x 8 bytes transposed in registers: column j's 8 rows become 8 bytes
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint2 col;
    const int sh = 8 * (j & 3);
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = ((j < 4 ? code[i].x : code[i].y) >> sh) & 0xffu;
    col.x = x[0] | x[1] << 8 | x[2] << 16 | x[3] << 24;
    col.y = x[4] | x[5] << 8 | x[6] << 16 | x[7] << 24;
    *reinterpret_cast<uint2*>(tile + (c * 8 + j) * QB_PITCH + r * 8) = col;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < G * G / 8 / QB_THREADS; ++k) {
    const int i = threadIdx.x + k * QB_THREADS;
    const int row = i / (G / 8), ch = i % (G / 8);
    const int64_t on = (int64_t)nb * G + row;
    if (on < N)
      *reinterpret_cast<uint2*>(qt + (e * N + on) * H + (int64_t)hb * G + ch * 8) =
          *reinterpret_cast<const uint2*>(tile + row * QB_PITCH + ch * 8);
  }
}

// ------------------------------------------------------------- token quantiser
// 16 consecutive lanes hold a group (8 elements each); H / 8 is a multiple of 16, so a
// group's lanes are active together.  Bound by HBM: 8192 x 7168 tokens 33 us (178 MB: 5.4 TB/s)
// with the descales side by side per group, 29.5 us in memory order.
constexpr int QR_THREADS = 256;
constexpr int QR_TOKENS = QR_THREADS / 16;
constexpr int64_t QR_MAX_BLOCKS = 1 << 20;

// One chunk of a group: its codes at chunk c, and the group's descale.
__device__ __forceinline__ void quant_chunk(const uint16_t* __restrict__ x, int64_t c, uint8_t* __restrict__ xq,
                                            float* __restrict__ descale) {
  float v[8], s[8];
  unpack8(*reinterpret_cast<const u32x4*>(x + c * 8), v);
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float sc = block_scale_of(m);
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = sc;
  *reinterpret_cast<uint2*>(xq + c * 8) = to_e4m3x8(v, s);
  if ((threadIdx.x & 15) == 0) *descale = 1.f / sc;
}

// Descales [T][H / 128]: chunks in memory order.
__global__ void __launch_bounds__(QR_THREADS) quant_rows_block(const uint16_t* __restrict__ x, int64_t chunks,
                                                               uint8_t* __restrict__ xq, float* __restrict__ xs) {
  for (int64_t c = (int64_t)blockIdx.x * QR_THREADS + threadIdx.x; c < chunks; c += (int64_t)gridDim.x * QR_THREADS)
    quant_chunk(x, c, xq, xs + (c >> 4));
}

// Descales [H / 128][T], so that the product reads those of a group side by side.  A workgroup
// takes one group of 16 tokens: their descales are one 64-byte line of one L2.
__global__ void __launch_bounds__(QR_THREADS) quant_cols_block(const uint16_t* __restrict__ x, int64_t T, int groups, int64_t tiles,
                                                               uint8_t* __restrict__ xq, float* __restrict__ xs) {
  for (int64_t b = blockIdx.x; b < tiles; b += gridDim.x) {
    const int64_t g = b % groups, t = b / groups * QR_TOKENS + (threadIdx.x >> 4);
    if (t < T) quant_chunk(x, (t * groups + g) * 16 + (threadIdx.x & 15), xq, xs + g * T + t);
  }
}

// ------------------------------------------------------------------- few rows
// Bound by the weight's bytes, and below a few tens of megabytes by the latency of its one round
// of loads.  A workgroup owns 16 columns; its RW waves take the groups in
// turn, streaming codes from global memory into two register sets (six: 12.7 us where two take
// 10.4), and add their sums up in LDS
// at the end.  Lane l holds 32 codes of a group, k = 32 (l / 16) + 0.., of weight row and of
// token l % 16.
struct BlockArgs {
  const uint8_t *xq, *wq;
  const float *xs, *ws;
  int64_t T, H, N;
  int ws_n, ws_g;      // steps of ws from one column block and from one group to the next
  int64_t xs_t, xs_g;  // and of xs from one token and from one group to the next
  uint16_t* y;
  int mt, nt;          // tiles of the many-row kernel
};

// y of 16 columns and the tokens 16 n + 0..15 from the waves' sums
template <int RW>
__device__ __forceinline__ void put_rows(float (&part)[RW][16][20], f32x4 acc, int n, int64_t T, int64_t N, int64_t n0,
                                         uint16_t* y) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  *reinterpret_cast<f32x4*>(&part[wave][lane & 15][4 * (lane >> 4)]) = acc;
  __syncthreads();
  const int t = threadIdx.x >> 4, col = threadIdx.x & 15;
  if (threadIdx.x < 256 && n * 16 + t < T && n0 + col < N) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < RW; ++q) s += part[q][t][col];
    y[(int64_t)(n * 16 + t) * N + n0 + col] = f2bf(s);
  }
  __syncthreads();
}

// Up to 16 bf16 tokens, quantised in registers (a group of a token is held by the four lanes that
// share it), which gives exactly the codes of the token quantiser in one launch.  (Every workgroup
// quantises the same tokens: 5 at 7168 x 4096 take 10.4 us so, 2.4 + 10.7 us as two launches;
// 24 took 18.8 us against 2.4 + 13.)  Codes of both
// operands become bf16 (exact) for the 16x16x32 instruction: products are exact, sums float32.
template <int RW>
__global__ void __launch_bounds__(RW * 64) block_rows(const uint16_t* __restrict__ x, const uint8_t* __restrict__ wq,
                                                      const float* __restrict__ ws, int T, int64_t H, int64_t N,
                                                      uint16_t* __restrict__ y) {
  __shared__ float part[RW][16][20];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int row = lane & 15, quad = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int groups = (int)(H / G);
  const uint8_t* wp = wq + min(n0 + row, N - 1) * H + 32 * quad;
  const uint16_t* xp = x + (int64_t)min(row, T - 1) * H + 32 * quad;
  const float* wsp = ws + (n0 / G) * groups;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  u32x4 w[2][2], b[2][4];
  auto load = [&](int g, u32x4 (&wr)[2], u32x4 (&br)[4]) {
    if (g >= groups) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) wr[i] = *reinterpret_cast<const u32x4*>(wp + (int64_t)g * G + 16 * i);
#pragma unroll
    for (int q = 0; q < 4; ++q) br[q] = *reinterpret_cast<const u32x4*>(xp + (int64_t)g * G + 8 * q);
    __builtin_amdgcn_sched_barrier(0);  // the loads go out here, not where their data is needed
  };
  auto bf16_of = [](uint32_t v, bool high) {
    return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
  };
  auto group = [&](int g, const u32x4 (&w)[2], const u32x4 (&b)[4]) {
    if (g >= groups) return;
    float v[4][8], m = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      unpack8(b[q], v[q]);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[q][j]));
    }
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    const float sc = block_scale_of(m);
    const float s[8] = {sc, sc, sc, sc, sc, sc, sc, sc};
    f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint2 code = to_e4m3x8(v[q], s);
      const uint32_t w0 = w[q >> 1][2 * (q & 1)], w1 = w[q >> 1][2 * (q & 1) + 1];
      const u32x4 a = {bf16_of(w0, false), bf16_of(w0, true), bf16_of(w1, false), bf16_of(w1, true)};
      const u32x4 c = {bf16_of(code.x, false), bf16_of(code.x, true), bf16_of(code.y, false), bf16_of(code.y, true)};
      t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, c), t, 0, 0, 0);
    }
    const float sx = wsp[g] * (1.f / sc);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(sx, t[i], acc[i]);
  };
  load(wave, w[0], b[0]);
  load(wave + RW, w[1], b[1]);
  for (int g = wave; g < groups; g += 2 * RW) {
    group(g, w[0], b[0]);
    load(g + 2 * RW, w[0], b[0]);
    group(g + RW, w[1], b[1]);
    load(g + 3 * RW, w[1], b[1]);
  }
  put_rows<RW>(part, acc, 0, T, N, n0, y);
}

// Up to 16 NT tokens' codes: one 16x16x128 instruction a group and row tile.
template <int NT, int RW>
__global__ void __launch_bounds__(RW * 64) block_codes(const BlockArgs A) {
  __shared__ float part[RW][16][20];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int row = lane & 15, quad = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int groups = (int)(A.H / G);
  const uint8_t* wp = A.wq + min(n0 + row, A.N - 1) * A.H + 32 * quad;
  const uint8_t* xp[NT];
  const float* sp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int64_t t = min((int64_t)(n * 16 + row), A.T - 1);
    xp[n] = A.xq + t * A.H + 32 * quad;
    sp[n] = A.xs + t * A.xs_t;
  }
  const float* wsp = A.ws + (n0 / G) * A.ws_n;
  f32x4 acc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Set {
    u32x4 w[2], b[NT][2];
    float s[NT];
  } set[2];
  auto load = [&](int g, Set& S) {
    if (g >= groups) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) S.w[i] = *reinterpret_cast<const u32x4*>(wp + (int64_t)g * G + 16 * i);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) S.b[n][i] = *reinterpret_cast<const u32x4*>(xp[n] + (int64_t)g * G + 16 * i);
      S.s[n] = sp[n][g * A.xs_g];
    }
    __builtin_amdgcn_sched_barrier(0);  // the loads go out here, not where their data is needed
  };
  auto join = [](const u32x4 (&v)[2]) {
    return i32x8{(int)v[0][0], (int)v[0][1], (int)v[0][2], (int)v[0][3], (int)v[1][0], (int)v[1][1], (int)v[1][2], (int)v[1][3]};
  };
  auto group = [&](int g, const Set& S) {
    if (g >= groups) return;
    const float sw = wsp[(int64_t)g * A.ws_g];
    const i32x8 a = join(S.w);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
      const f32x4 t = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, join(S.b[n]), zero, 0, 0, 0, 127, 0, 127);
      const float s = S.s[n] * sw;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = __builtin_fmaf(s, t[i], acc[n][i]);
    }
  };
  load(wave, set[0]);
  load(wave + RW, set[1]);
  for (int g = wave; g < groups; g += 2 * RW) {
    group(g, set[0]);
    load(g + 2 * RW, set[0]);
    group(g + RW, set[1]);
    load(g + 3 * RW, set[1]);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) put_rows<RW>(part, acc[n], n, A.T, A.N, n0, A.y);
}

// ------------------------------------------------------------------- many rows
// Bound by the matrix instructions and the scaling between them (one float32 operation per
// accumulator element and group, which takes about as many issue cycles as a group's two
// 32x32x64 instructions of a tile, hence the interleaving).  The 16x16x128 instruction, with the
// scaling of its shorter sums, was slower: 238 us against 202 at 8192 x 7168 x 4096.
// BM tokens by BN columns a workgroup, one group of 128 a step, NS stages of LDS filled
// by loads that bypass the registers (the tokens' scales among them).  A row of a stage is 128
// bytes, half of the banks; its 16-byte chunk c sits at position c ^ (row / 2 % 8), so the 16-byte reads of 16 consecutive
// rows cover every bank once.  (The loads write LDS in lane order, so the permutation is applied to the
// global address, inside one 128-byte line.)
// KS parts of the workgroup take the steps in turn, each with stages of its own, and their sums are
// added at the end (part 0 first).
template <int BM_, int BN_, int WM_, int WN_, int NS_, int KS_>
struct BlockTile {
  static constexpr int SPREAD = 5;  // tiles of a step that its stage loads are spread over
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_, KS = KS_;
  static constexpr int HT = WM * WN * 64, NTHR = KS * HT;  // threads of a part, of the workgroup
  static constexpr int TM = BM / WM, TN = BN / WN, MB = TM / 32, NB = TN / 32;
  static constexpr int STAGE = (BM + BN) * G + BM * 4;  // weight rows, token rows, token scales
  static constexpr int LDO = BN + 8;  // output tile pitch, elements
  static constexpr int LDS = KS * NS * STAGE > BM * LDO * 2 ? KS * NS * STAGE : BM * LDO * 2;
  static_assert(TN <= G && G % TN == 0, "a wave's columns lie in one weight block");
  static_assert(BM * 8 % HT == 0 && BN * 8 % HT == 0 && BM < HT && BM % (HT / 64) == 0, "whole loads a stage");
  static_assert(KS == 1 || BM * BN * 4 <= LDS, "the second part's sums fit");
};

// the words of make_rsrc's buffer resource, for assembly
__device__ __forceinline__ u32x4 rsrc_words(const void* base, int64_t bytes) {
  const uint64_t p = (uint64_t)base;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)p), (uint32_t)__builtin_amdgcn_readfirstlane((int)(p >> 32)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}

// 16 bytes per lane from global memory to LDS at lds + 16 lane (lds: uniform).  Written in
// assembly because the compiler, which cannot tell the two stages apart, would wait for a
// load of the next stage before every read of this one; it has no register to return, and
// the kernel waits for it itself (vmcnt) before the barrier that publishes the stage.
__device__ __forceinline__ void load_lds16(u32x4 r, uint32_t lds, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(r), "s"(soff)
               : "memory");
}
// The same of 4 bytes per lane, of the lanes in ``mask`` only; the wave's 64 lanes are active
// before and after.
__device__ __forceinline__ void load_lds4(u32x4 r, uint32_t lds, uint32_t voff, uint32_t soff, uint64_t mask) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_mov_b64 exec, %4\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds\n\ts_mov_b64 exec, -1"
      :
      : "s"(lds), "v"(voff), "s"(r), "s"(soff), "s"(mask)
      : "memory");
}

__device__ __forceinline__ i32x8 frag(const uint8_t* base, int row, int kk, int half) {
  const int c = 4 * kk + half;
  const u32x4 lo = *reinterpret_cast<const u32x4*>(base + row * G + ((c ^ ((row >> 1) & 7)) * 16));
  const u32x4 hi = *reinterpret_cast<const u32x4*>(base + row * G + (((c + 2) ^ ((row >> 1) & 7)) * 16));
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

template <class C>
__global__ void __launch_bounds__(C::NTHR) block_gemm(const BlockArgs A) {
  __shared__ __attribute__((aligned(128))) uint8_t smem[C::LDS];
  const int nblocks = gridDim.x;
  int mt, nt;
  const int logical = xcd_remap(blockIdx.x, nblocks);
  if (logical >= A.mt * A.nt) return;
  raster(logical, A.mt, A.nt, mt, nt);
  const int64_t m0 = (int64_t)mt * C::BM, n0 = (int64_t)nt * C::BN;
  const int lane = threadIdx.x & 63;
  const int waves = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int part = waves / (C::HT / 64), wave = waves % (C::HT / 64), tid = threadIdx.x % C::HT;
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int half = lane >> 5, l32 = lane & 31;
  const uint32_t pitch = (uint32_t)A.H;
  const u32x4 rx = rsrc_words(A.xq + m0 * A.H, min((int64_t)C::BM, A.T - m0) * A.H);
  const u32x4 rw = rsrc_words(A.wq + n0 * A.H, min((int64_t)C::BN, A.N - n0) * A.H);
  const int groups = (int)(A.H / G);
  const u32x4 rs = rsrc_words(A.xs + m0 * A.xs_t, (A.T * groups - m0 * A.xs_t) * 4);
  const float* wsp = A.ws + ((n0 + wn * C::TN) / G < (A.N + G - 1) / G ? (n0 + wn * C::TN) / G : 0) * A.ws_n;

  f32x16 acc[C::NB][C::MB];
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
    for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[nb][mb][r] = 0.f;

  const uint8_t* mine = smem + part * C::NS * C::STAGE;  // the part's stages
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem + part * C::NS * C::STAGE;
  // A load takes 8 lanes a row, so the workgroup's i-th one starts RPL rows (a multiple of 16,
  // the permutation's period) further: one offset register serves all of them, and both operands.
  constexpr int RPL = C::HT / 8, LW = C::BN / RPL, LOADS = LW + C::BM / RPL;
  static_assert(RPL % 16 == 0, "permutation period");
  const uint32_t voff = (tid >> 3) * pitch + (((tid & 7) ^ ((tid >> 4) & 7)) * 16);
  constexpr int TPW = C::BM * 64 / C::HT;  // tokens whose scales a wave loads
  const uint32_t soff = (uint32_t)min((int64_t)(wave * TPW + lane), A.T - 1 - m0) * (uint32_t)A.xs_t * 4;
  // Loads [from, to) of stage g into its buffer (past the last stage: of the last one again,
  // unused); the last of them is the scales', BM / waves tokens a wave.  Rows past the tensors' ends are
  // beyond the resources and come back as zeros; the scalar offset stays inside.
  auto stage = [&](int g, int buf, int from, int to) {
    const uint32_t at = lds0 + (uint32_t)buf * C::STAGE;
    const int gc = min(g, groups - 1);
#pragma unroll
    for (int i = from; i < to; ++i)
      if (i < LOADS)
        load_lds16(i < LW ? rw : rx, at + (uint32_t)(i * C::HT + wave * 64) * 16,
                   voff + (uint32_t)(i < LW ? i : i - LW) * RPL * pitch, (uint32_t)gc * G);
      else
        load_lds4(rs, at + (C::BM + C::BN) * G + (uint32_t)wave * TPW * 4, soff, (uint32_t)(gc * A.xs_g) * 4, (1ull << TPW) - 1);
  };
  constexpr int TILES = C::NB * C::MB, ALL = LOADS + 1, OVER = C::SPREAD < TILES ? C::SPREAD : TILES;
  constexpr int PER = (ALL + OVER - 1) / OVER;
#pragma unroll
  for (int q = 0; q < C::NS - 1; ++q) stage(q * C::KS + part, q, 0, ALL);
  // the block's scales: lane l holds that of the part's step i0 + l, reloaded every 64 steps
  float wl = 0.f;
  int buf = 0, fill = C::NS - 1;
  for (int step = 0; step * C::KS < groups; ++step) {
    const bool live = C::KS == 1 || step * C::KS + part < groups;  // false in an odd last step of part 1
    if ((step & 63) == 0) {
      wl = wsp[(int64_t)min((step + lane) * C::KS + part, groups - 1) * A.ws_g];
      asm volatile("" : "+v"(wl));  // waits for it here, once in 64 steps
    }
    // this step's stage has landed (NS - 2 later ones may be on their way), and the last one is done with
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"i"((C::NS - 2) * ALL) : "memory");
    const float sw = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wl), step & 63));
    const uint8_t* sw_ = mine + buf * C::STAGE;
    const uint8_t* sx_ = sw_ + C::BN * G;
    const float* ss_ = reinterpret_cast<const float*>(sx_ + C::BM * G);
    i32x8 fb[C::MB][2], fa[2][2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      fa[0][kk] = frag(sw_, wn * C::TN + l32, kk, half);
#pragma unroll
      for (int mb = 0; mb < C::MB; ++mb) fb[mb][kk] = frag(sx_, wm * C::TM + mb * 32 + l32, kk, half);
    }
    float s[C::MB];
#pragma unroll
    for (int mb = 0; mb < C::MB; ++mb) s[mb] = ss_[wm * C::TM + mb * 32 + l32] * sw;
    // The matrix instructions of tile i run while the sums of tile i - 1 are scaled and added;
    // the next stage's loads go out one by one between them (all at once they would fill the
    // address unit's queue, and each wave's later instructions wait behind its own).
    f32x16 t[2];
#pragma unroll
    for (int i = 0; i <= TILES; ++i) {
      const int nb = i / C::MB, mb = i % C::MB;
      if (i < TILES) {
        if (mb == 0 && nb + 1 < C::NB)
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) fa[(nb + 1) & 1][kk] = frag(sw_, wn * C::TN + (nb + 1) * 32 + l32, kk, half);
        const f32x16 zero = {};
        t[i & 1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[nb & 1][0], fb[mb][0], zero, 0, 0, 0, 127, 0, 127);
        t[i & 1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[nb & 1][1], fb[mb][1], t[i & 1], 0, 0, 0, 127, 0, 127);
        __builtin_amdgcn_sched_barrier(0);
        stage((step + C::NS - 1) * C::KS + part, fill, min(i * PER, ALL), min((i + 1) * PER, ALL));
      }
      if (i > 0 && live) {
        const int pn = (i - 1) / C::MB, pm = (i - 1) % C::MB;
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[pn][pm][r] = __builtin_fmaf(s[pm], t[(i - 1) & 1][r], acc[pn][pm][r]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    buf = buf + 1 == C::NS ? 0 : buf + 1;
    fill = fill + 1 == C::NS ? 0 : fill + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the loads past the last stage write into LDS
  __syncthreads();
  if constexpr (C::KS == 2) {  // part 1's sums through LDS, added by part 0
    float* sums = reinterpret_cast<float*>(smem) + wave * (C::NB * C::MB * 16 * 64) + lane;
    if (part == 1)
#pragma unroll
      for (int i = 0; i < C::NB * C::MB * 16; ++i) sums[i * 64] = acc[i / 16 / C::MB][i / 16 % C::MB][i % 16];
    __syncthreads();
    if (part == 0)
#pragma unroll
      for (int i = 0; i < C::NB * C::MB * 16; ++i) acc[i / 16 / C::MB][i / 16 % C::MB][i % 16] += sums[i * 64];
    __syncthreads();
  }
  // the tile in bf16 through LDS, so that stores are rows of 16-byte chunks
  uint16_t* out = reinterpret_cast<uint16_t*>(smem);
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
    for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
      for (int q = 0; q < 4 && part == 0; ++q) {
        uint2 v;
        v.x = (uint32_t)f2bf(acc[nb][mb][4 * q]) | ((uint32_t)f2bf(acc[nb][mb][4 * q + 1]) << 16);
        v.y = (uint32_t)f2bf(acc[nb][mb][4 * q + 2]) | ((uint32_t)f2bf(acc[nb][mb][4 * q + 3]) << 16);
        *reinterpret_cast<uint2*>(out + (wm * C::TM + mb * 32 + l32) * C::LDO + wn * C::TN + nb * 32 + 8 * q + 4 * half) = v;
      }
  __syncthreads();
  constexpr int CPR = C::BN / 8;
#pragma unroll 4
  for (int i = threadIdx.x; i < C::BM * CPR; i += C::NTHR) {
    const int r = i / CPR, c = i % CPR * 8;
    if (m0 + r < A.T && n0 + c < A.N)
      store16_stream(A.y + (m0 + r) * A.N + n0 + c, *reinterpret_cast<const u32x4*>(out + r * C::LDO + c));
  }
}

template <class C>
hipError_t launch_gemm(BlockArgs a, hipStream_t stream) {
  a.mt = (int)((a.T + C::BM - 1) / C::BM);
  a.nt = (int)((a.N + C::BN - 1) / C::BN);
  const int64_t blocks = ((int64_t)a.mt * a.nt + 7) / 8 * 8;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  block_gemm<C><<<(unsigned)blocks, C::NTHR, 0, stream>>>(a);
  return hipGetLastError();
}

template <int NT, int RW>
hipError_t launch_codes(const BlockArgs& a, hipStream_t stream) {
  block_codes<NT, RW><<<(unsigned)((a.N + 15) / 16), RW * 64, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_block(const uint16_t* w, int64_t E, int64_t H, int64_t N, uint8_t* qt, uint8_t* q, float* ds,
                              hipStream_t stream) {
  const int64_t hbs = H / G, nbs = (N + G - 1) / G;
  if (E * hbs * nbs > 0x7fffffff) return hipErrorInvalidValue;
  quant_block<<<(unsigned)(E * hbs * nbs), QB_THREADS, 0, stream>>>(w, H, N, (int)hbs, (int)nbs, qt, q, ds);
  return hipGetLastError();
}

hipError_t launch_quant_rows_block(const uint16_t* x, int64_t T, int64_t H, uint8_t* xq, float* xs, bool cols,
                                   hipStream_t stream) {
  if (T <= 0) return hipSuccess;
  const int64_t groups = H / G, chunks = T * (H / 8);
  const int64_t blocks = cols ? (T + QR_TOKENS - 1) / QR_TOKENS * groups : (chunks + QR_THREADS - 1) / QR_THREADS;
  const unsigned grid = (unsigned)(blocks < QR_MAX_BLOCKS ? blocks : QR_MAX_BLOCKS);
  if (cols)
    quant_cols_block<<<grid, QR_THREADS, 0, stream>>>(x, T, (int)groups, blocks, xq, xs);
  else
    quant_rows_block<<<grid, QR_THREADS, 0, stream>>>(x, chunks, xq, xs);
  return hipGetLastError();
}

hipError_t launch_block_rows(const uint16_t* x, const uint8_t* wq, const float* ws, int T, int64_t H, int64_t N, uint16_t* y,
                             hipStream_t stream) {
  block_rows<8><<<(unsigned)((N + 15) / 16), 8 * 64, 0, stream>>>(x, wq, ws, T, H, N, y);
  return hipGetLastError();
}

hipError_t launch_block_gemm(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, int64_t T, int64_t H,
                             int64_t N, bool xs_cols, bool ws_transposed, uint16_t* y, hipStream_t stream) {
  const int groups = (int)(H / G), nbs = (int)((N + G - 1) / G);
  const BlockArgs a{xq, wq, xs, ws, T, H, N, ws_transposed ? 1 : groups, ws_transposed ? nbs : 1, xs_cols ? 1 : groups,
                    xs_cols ? T : 1, y, 0, 0};
  // Few rows and columns leave CUs without a 64 x 64 tile, and 16-column workgroups win; with
  // many columns the tiles cover the chip and read the tokens' codes less often.  16 rows: 12.3
  // against 13.8 us at N = 8192 (H = 4096), 22 against 19.6 at N = 14336; 32 rows: 14.6 against
  // 21 at N = 4096 (H = 7168), 9.8 against 8.5 at N = 6144 (H = 2048).
  if (T <= 16 && N <= 8192) return launch_codes<1, 8>(a, stream);
  if (T <= 32 && N <= 4096) return launch_codes<2, 8>(a, stream);
  const auto tiles = [&](int64_t bm, int64_t bn) { return ((T + bm - 1) / bm) * ((N + bn - 1) / bn); };
  // The fewest rounds of the 256 CUs, then the largest tile.  160 tiles of 256 x 256 in one round
  // take 53.9 us against 68.6 of 320 of 256 x 128 in two (5000 x 4096 x 2048); 128 against 256 leave
  // half of the chip idle, 52 to 40 us (4096 x 4096 x 2048).  Below 128 of those, smaller tiles:
  // 24.7 against 32.6 us (1536 x 4096 x 2048), at 128 34.5 against 33.2 (1024 x 4096 x 4096).
  // Between these sizes the product is at 2.5 to 3 times its operations' time.  128 tiles of 256 x 128
  // take nearly as long as 256 of them (33 and 39 us, 32 steps each): a CU with a tile is at three
  // quarters of its rate, and half have none.  The small tiles stage four times the bytes a matrix
  // instruction that 256 x 256 tiles do: 1536 x 4096 x 2048 moves 409 MB into LDS, 16.5 TB/s, matrix
  // instructions busy a fifth of the time.
  if (tiles(256, 256) > 128) return launch_gemm<BlockTile<256, 256, 4, 2, 2, 1>>(a, stream);
  if (tiles(256, 128) >= 128) return launch_gemm<BlockTile<256, 128, 4, 2, 3, 1>>(a, stream);
  // Small tiles: up to one a CU, two parts of a workgroup share a tile's groups (64 x 7168 x 4096
  // 17.9 us against 21.7, 130 x 2048 x 2048 7.6 against 9.1); with more, two workgroups a CU overlap
  // as well and the parts only cost LDS (1003 x 2048 x 1552, 400 tiles: 14.8 against 11.3).
  if (tiles(64, 64) <= 256) return launch_gemm<BlockTile<64, 64, 2, 2, 3, 2>>(a, stream);
  return launch_gemm<BlockTile<64, 64, 2, 2, 3, 1>>(a, stream);
}

}  // namespace hmm
