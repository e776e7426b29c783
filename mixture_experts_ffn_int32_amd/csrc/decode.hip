// A whole mixture-of-experts layer for a few tokens (T <= 64), where every byte
// of the chosen experts' weights is read once and used for a handful of rows:
//
//   l[t,e] = x[t] . Wr[e];  ids[t], w[t] = the K largest logits and their softmax
//   [g|u]  = x[t] . W1[e];  a = silu(g) u;  y[t] = sum_k w[t,k] a . W2[ids[t,k]]
//
// Bound by HBM: an expert's 3 H I weights for 6 H I flop a row.  So nothing of
// the large products' tiling is of use here.  A workgroup owns a column tile of
// one chosen expert; its waves split the contraction, each streaming weights
// from global memory straight into the matrix instruction's operand registers
// (no LDS, no barrier in the loop, the next step's loads in flight), with up to
// 16 rows a 16x16x32 instruction.  The waves' sums meet in LDS once, at the end.
//
// The choice of experts is decided by the order of the logits, so they are
// summed in 64 bits: products of two bf16 are exact in it, and their sum is
// exact or off by far less than any gap, in whatever order it is taken.  All
// other sums are float32; a stays a bf16 pair (hi + lo, 16 significant bits),
// for the instruction has time to spare; y is rounded once.
//
// Three or four launches on one stream, no state kept between calls:
//   logits, top-k        (with a router weight)
//   up-projection        one workgroup per (chosen expert, 64 or 32 columns of I)
//   down-projection      one workgroup per (chosen expert, 128 or 64 columns of H);
//                        the last one of a column tile to finish adds the rows up
// The last step needs no wait: a workgroup stores its rows at the device-wide
// coherence point, counts itself, and only the one that counts last reads them,
// in a fixed order, so the sum has the same bits on every run.
#include "gemm_common.h"
#include "kernels.h"

namespace hmm {
namespace {

constexpr int DT = DECODE_MAX_TOKENS;
constexpr int MAX_SLOTS = DT * 16;
static_assert(DT == 64, "the rows of an expert are one 64-bit lane mask");

// ------------------------------------------------------------------------ router

// logits[t][e] in float64: a workgroup takes EE experts and TT tokens, its
// threads split H in 16-byte chunks.
constexpr int GE = 2, GT = 4, GTHR = 512;

template <class W>
__device__ __forceinline__ void router8(const W* p, double (&v)[8]);
template <>
__device__ __forceinline__ void router8<uint16_t>(const uint16_t* p, double (&v)[8]) {
  float f[8];
  unpack8(*reinterpret_cast<const u32x4*>(p), f);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = f[j];
}
template <>
__device__ __forceinline__ void router8<float>(const float* p, double (&v)[8]) {
  const f32x4* q = reinterpret_cast<const f32x4*>(p);
  const f32x4 a = q[0], b = q[1];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[4 + j] = b[j];
  }
}

template <class W>
__global__ void __launch_bounds__(GTHR) router_logits(const uint16_t* __restrict__ x, const W* __restrict__ wr, int T,
                                                      int64_t H, int E, double* __restrict__ logits) {
  __shared__ double part[GTHR / 64][GE * GT];
  const int e0 = blockIdx.x * GE, t0 = blockIdx.y * GT;
  double acc[GE][GT] = {};
  for (int64_t c = (int64_t)threadIdx.x * 8; c < H; c += GTHR * 8) {
    double xv[GT][8], wv[8];
#pragma unroll
    for (int t = 0; t < GT; ++t) router8<uint16_t>(x + (int64_t)min(t0 + t, T - 1) * H + c, xv[t]);
#pragma unroll
    for (int e = 0; e < GE; ++e) {
      router8<W>(wr + (int64_t)min(e0 + e, E - 1) * H + c, wv);
#pragma unroll
      for (int t = 0; t < GT; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[e][t] = __builtin_fma(xv[t][j], wv[j], acc[e][t]);
    }
  }
#pragma unroll
  for (int e = 0; e < GE; ++e)
#pragma unroll
    for (int t = 0; t < GT; ++t) {
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) acc[e][t] += __shfl_xor(acc[e][t], d);
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][e * GT + t] = acc[e][t];
    }
  __syncthreads();
  if (threadIdx.x < GE * GT) {
    const int e = e0 + threadIdx.x / GT, t = t0 + threadIdx.x % GT;
    double s = 0.;
#pragma unroll
    for (int q = 0; q < GTHR / 64; ++q) s += part[q][threadIdx.x];
    if (e < E && t < T) logits[(int64_t)t * E + e] = s;
  }
}

// One wave per token: K times the largest remaining logit (ties to the lower
// index, a NaN ranks last), then the weights: exp(l - max) over its sum over the
// chosen (renorm) or over all experts.
constexpr int TK_PER = MAX_EXPERTS / 64;
__global__ void __launch_bounds__(64) router_topk(const double* __restrict__ logits, int E, int K, int renorm,
                                                  int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int t = blockIdx.x, lane = threadIdx.x;
  double v[TK_PER];
  uint32_t open = 0;  // bit j: expert lane + 64 j is still to be chosen
#pragma unroll
  for (int j = 0; j < TK_PER; ++j) {
    v[j] = -__builtin_inf();
    if (64 * j < E && lane + 64 * j < E) {
      const double l = logits[(int64_t)t * E + lane + 64 * j];
      if (l == l) v[j] = l;
      open |= 1u << j;
    }
  }
  double top = 0.;
  float mine = 0.f, sum = 0.f;
  int my_id = 0;
  for (int k = 0; k < K; ++k) {
    double b = -__builtin_inf();
    int bi = 0x7fffffff;
#pragma unroll
    for (int j = 0; j < TK_PER; ++j)
      if (64 * j < E && ((open >> j) & 1) && (bi == 0x7fffffff || v[j] > b)) {
        b = v[j];
        bi = lane + 64 * j;
      }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      const double ob = __shfl_xor(b, d);
      const int oi = __shfl_xor(bi, d);
      if (oi != 0x7fffffff && (bi == 0x7fffffff || ob > b || (ob == b && oi < bi))) {
        b = ob;
        bi = oi;
      }
    }
    if (k == 0) top = b;
    const float e = expf((float)(b - top));
    sum += e;
    if (lane == k) {
      mine = e;
      my_id = bi;
    }
    if ((bi & 63) == lane) open &= ~(1u << (bi >> 6));
  }
  if (!renorm) {
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < TK_PER; ++j)
      if (64 * j < E && lane + 64 * j < E) sum += expf((float)(v[j] - top));
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
  }
  if (lane < K) {
    ids[t * K + lane] = my_id;
    weights[t * K + lane] = mine / sum;
  }
}

// ------------------------------------------------------------------- expert tiles

// What a workgroup finds out first: the i-th expert that some token chose, and
// the rows (tokens) it has.  A token that names an expert twice is one row.
struct Rows {
  int32_t ids[MAX_SLOTS];
  uint32_t chosen[MAX_EXPERTS / 32];
  int32_t tok[DT];
  int32_t slot[DT];  // t * K + the first k that names the expert
  int flag;
};

// false if fewer than i + 1 experts are chosen; nact: how many are
template <int DW>
__device__ __forceinline__ bool find_rows(Rows& L, const DecodeArgs& A, int i, int& e, int& rows, int& nact) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int S = A.T * A.K;
  if (tid < MAX_EXPERTS / 32) L.chosen[tid] = 0;
  __syncthreads();
  for (int s = tid; s < S; s += DW * 64) {
    const int id = A.ids[s];
    L.ids[s] = id;
    if (id >= 0 && id < A.E) atomicOr(&L.chosen[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
  const uint32_t w = lane < MAX_EXPERTS / 32 ? L.chosen[lane] : 0u;
  int inc = __popc(w);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  nact = __shfl(inc, 31);
  if (i >= nact) return false;
  const int word = __ffsll((unsigned long long)__ballot(lane < 32 && inc > i)) - 1;
  uint32_t bits = (uint32_t)__shfl((int)w, word);
  int skip = i - (__shfl(inc, word) - __popc(bits));
  while (skip--) bits &= bits - 1;
  e = word * 32 + __ffs(bits) - 1;
  int first = -1;
  if (lane < A.T)
    for (int k = A.K - 1; k >= 0; --k)
      if (L.ids[lane * A.K + k] == e) first = k;
  const uint64_t mask = __ballot(first >= 0);
  rows = __popcll(mask);
  if (first >= 0 && tid < 64) {
    const int r = __popcll(mask & ((1ull << lane) - 1));
    L.tok[r] = lane;
    L.slot[r] = lane * A.K + first;
  }
  __syncthreads();
  return true;
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// A wave's share of a tile: acc[c][nt] += the 16 columns of sub-tile c times 16 rows.
// In the accumulator, lane l holds row l % 16 and the columns 4 (l / 16) + 0..3 of the sub-tile.
//
// bf16 weights [K][N] (columns contiguous), 128 columns a wave and 32 deep a step:
// lane l loads the 16-byte column chunk l % 16 of the 8 rows k = 8 (l / 16) + 0..7, which
// after a transposition in registers (one v_perm_b32 per pair) is its operand for each of
// the 8 columns of the chunk.  Sub-tile c holds the columns 8 m + c of chunk m.
struct Bf16Weights {
  static constexpr int SUB = 8, COLS = 128, DEPTH = 32, LOADS = 8;
  static constexpr int ROW_LOADS = 1;  // 16-byte loads of a row (token) per step
  static __device__ __forceinline__ int column(int c, int m) { return 8 * m + c; }

  const char* p;    // this lane's chunk at step 0
  int64_t pitch;    // bytes between rows k
  // chunks below half come from base0, the others from base1 (gate and up columns)
  __device__ __forceinline__ void init(const void* w, int64_t, int64_t N, int64_t c0, int64_t c1, const float*, int64_t,
                                       int lane) {
    const int m = lane & 15;
    const int64_t col = m < 8 ? c0 + 8 * m : c1 + 8 * (m - 8);
    pitch = N * 2;
    p = static_cast<const char*>(w) + (int64_t)(8 * (lane >> 4)) * pitch + col * 2;
  }
  __device__ __forceinline__ void load(int step, u32x4 (&r)[LOADS]) const {
    const char* q = p + (int64_t)step * DEPTH * pitch;
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = *reinterpret_cast<const u32x4*>(q + j * pitch);
  }
  static __device__ __forceinline__ int row_offset(int lane) { return 8 * (lane >> 4); }
  template <int NT, int PARTS>
  __device__ __forceinline__ void mul(int, const u32x4 (&r)[LOADS], const u32x4 (&b)[NT][PARTS][ROW_LOADS], int nt,
                                      f32x4 (&acc)[SUB][NT]) const {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      u32x4 a;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        a[q] = __builtin_amdgcn_perm(r[2 * q + 1][c >> 1], r[2 * q][c >> 1], (c & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n < nt)
#pragma unroll
          for (int h = 0; h < PARTS; ++h)
            acc[c][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                                __builtin_bit_cast(bf16x8, b[n][h][0]), acc[c][n], 0, 0, 0);
    }
  }
};

// E4M3 weights [N][K] (the contraction contiguous), 64 columns a wave and D deep a
// step (128, one scale block, or 64 where registers are short): lane l loads the D / 4
// codes k = (D / 4) (l / 16) + 0.. of column l % 16 of each sub-tile, turns them into
// bf16 (exact), and the step's sums, started from zero, are scaled by the block's
// descale in float32.
template <int D>
struct Fp8Weights {
  static constexpr int SUB = 4, COLS = 64, DEPTH = D, CL = D / 64, LOADS = 4 * CL;  // CL: loads per column
  static constexpr int ROW_LOADS = 2 * CL;
  static __device__ __forceinline__ int column(int c, int m) { return 16 * c + m; }

  const char *p0, *p1;   // this lane's codes at step 0, sub-tiles 0,1 and 2,3
  int64_t pitch;         // bytes between columns
  const float *d0, *d1;  // descales of step 0
  __device__ __forceinline__ void init(const void* w, int64_t K, int64_t, int64_t c0, int64_t c1, const float* ds,
                                       int64_t groups, int lane) {
    pitch = K;
    const char* b = static_cast<const char*>(w) + (int64_t)(lane & 15) * pitch + row_offset(lane);
    p0 = b + c0 * pitch;
    p1 = b + c1 * pitch;
    d0 = ds + (c0 >> 7) * groups;
    d1 = ds + (c1 >> 7) * groups;
  }
  __device__ __forceinline__ void load(int step, u32x4 (&r)[LOADS]) const {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const char* q = (c < 2 ? p0 : p1) + (int64_t)step * DEPTH + (c & 1) * 16 * pitch;
#pragma unroll
      for (int i = 0; i < CL; ++i) r[CL * c + i] = *reinterpret_cast<const u32x4*>(q + 16 * i);
    }
  }
  static __device__ __forceinline__ int row_offset(int lane) { return D / 4 * (lane >> 4); }
  template <int NT, int PARTS>
  __device__ __forceinline__ void mul(int step, const u32x4 (&r)[LOADS], const u32x4 (&b)[NT][PARTS][ROW_LOADS], int nt,
                                      f32x4 (&acc)[SUB][NT]) const {
    const float s0 = d0[step * D / 128], s1 = d1[step * D / 128];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      u32x4 a[2 * CL];
#pragma unroll
      for (int q = 0; q < 2 * CL; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t v = r[CL * c + (q >> 1)][2 * (q & 1) + i];
          a[q][2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, false));
          a[q][2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, true));
        }
      const float s = c < 2 ? s0 : s1;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n < nt) {
          f32x4 g = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 2 * CL; ++q)
#pragma unroll
            for (int h = 0; h < PARTS; ++h)
              g = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[q]),
                                                          __builtin_bit_cast(bf16x8, b[n][h][q]), g, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[c][n][i] = __builtin_fmaf(s, g[i], acc[c][n][i]);
        }
    }
  }
};

// The wave's sums over its steps (wave, wave + DW, ...) of the tile.  src[n]: this
// lane's row of row tile n (rows past the last one repeat row 0's data: their
// columns of the accumulator are never read); part: elements between a row's parts.
template <class WT, int NT, int PARTS, int DW>
__device__ __forceinline__ void stream_tile(const WT& W, const uint16_t* const (&src)[NT], int64_t part, int steps,
                                            int wave, int lane, int nt, f32x4 (&acc)[WT::SUB][NT]) {
#pragma unroll
  for (int c = 0; c < WT::SUB; ++c)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[c][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (wave >= steps) return;
  // The loads return in order: with one row tile its data is fetched a step ahead
  // with the weights; with more (registers) right before the next step's weights, so
  // that waiting for it leaves those in flight.
  constexpr bool AHEAD = NT == 1;
  u32x4 w[WT::LOADS], b[NT][PARTS][WT::ROW_LOADS];
  auto load_rows = [&](int s, u32x4 (&br)[NT][PARTS][WT::ROW_LOADS]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (n < nt)
#pragma unroll
        for (int h = 0; h < PARTS; ++h)
#pragma unroll
          for (int q = 0; q < WT::ROW_LOADS; ++q)
            br[n][h][q] = *reinterpret_cast<const u32x4*>(src[n] + h * part + (int64_t)s * WT::DEPTH + 8 * q);
  };
  W.load(wave, w);
  if constexpr (AHEAD) load_rows(wave, b);
  for (int s = wave; s < steps; s += DW) {
    u32x4 wn[WT::LOADS], bn[NT][PARTS][WT::ROW_LOADS];
    if constexpr (!AHEAD) load_rows(s, b);
    if (s + DW < steps) {
      W.load(s + DW, wn);
      if constexpr (AHEAD) load_rows(s + DW, bn);
    }
    W.template mul<NT, PARTS>(s, w, b, nt, acc);
#pragma unroll
    for (int j = 0; j < WT::LOADS; ++j) w[j] = wn[j];
    if constexpr (AHEAD)
#pragma unroll
      for (int h = 0; h < PARTS; ++h)
#pragma unroll
        for (int q = 0; q < WT::ROW_LOADS; ++q) b[0][h][q] = bn[0][h][q];
  }
}

// LDS of the waves' sums of one row tile: [DW][16 rows][COLS + 4] floats (a pitch of
// 4 banks more than a multiple of 64: the 16 rows of a store fall into distinct banks)
template <class WT, int DW>
struct Sums {
  static constexpr int LD = WT::COLS + 4;
  float v[DW][16][LD];
};
template <class WT, int NT, int DW>
__device__ __forceinline__ void put_sums(Sums<WT, DW>& L, const f32x4 (&acc)[WT::SUB][NT], int n, int wave, int lane) {
#pragma unroll
  for (int c = 0; c < WT::SUB; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) L.v[wave][lane & 15][WT::column(c, 4 * (lane >> 4) + i)] = acc[c][n][i];
}
template <class WT, int DW>
__device__ __forceinline__ float get_sum(const Sums<WT, DW>& L, int row, int col) {
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < DW; ++q) s += L.v[q][row][col];
  return s;
}

// up-projection: COLS / 2 gate columns and the matching up columns of one expert
template <class WT, int NT, int DW>
__global__ void __launch_bounds__(DW * 64) decode_up(const DecodeArgs A) {
  constexpr int HC = WT::COLS / 2;
  __shared__ Rows L;
  __shared__ Sums<WT, DW> P;
  const int tiles = (int)(A.I / HC);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  // the down-projection's counters, cleared one launch ahead of their use
  for (int64_t g = (int64_t)blockIdx.x * DW * 64 + threadIdx.x; g < A.col_tiles; g += (int64_t)gridDim.x * DW * 64)
    A.count[g] = 0;
  int e, rows, nact;
  const int n0 = (blockIdx.x % tiles) * HC;
  if (!find_rows<DW>(L, A, blockIdx.x / tiles, e, rows, nact)) return;
  e = __builtin_amdgcn_readfirstlane(e);
  const int nt = __builtin_amdgcn_readfirstlane((rows + 15) >> 4);
  WT W;
  W.init(static_cast<const char*>(A.up) + (int64_t)e * A.H * 2 * A.I * A.wbytes, A.H, 2 * A.I, n0, A.I + n0,
         A.up_descale + (int64_t)e * (2 * A.I / 128) * (A.H / 128), A.H / 128, lane);
  const uint16_t* src[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = n * 16 + (lane & 15);
    src[n] = A.x + (int64_t)L.tok[r < rows ? r : 0] * A.H + WT::row_offset(lane);
  }
  f32x4 acc[WT::SUB][NT];
  stream_tile<WT, NT, 1, DW>(W, src, 0, (int)(A.H / WT::DEPTH), wave, lane, nt, acc);
  for (int n = 0; n < nt; ++n) {
#pragma unroll
    for (int q = 0; q < NT; ++q)
      if (q == n) put_sums<WT, NT, DW>(P, acc, q, wave, lane);
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * HC; i += DW * 64) {
      const int row = n * 16 + i / HC, col = i % HC;
      if (row < rows) {
        const float gv = get_sum(P, i / HC, col), u = get_sum(P, i / HC, HC + col);
        const float a = gv * sigmoidf_(gv) * u;
        uint16_t* out = A.a + (int64_t)L.slot[row] * 2 * A.I + n0 + col;
        const uint16_t hi = f2bf(a);
        const float rest = a - bf2f(hi);
        out[0] = hi;
        out[A.I] = __builtin_isfinite(rest) ? f2bf(rest) : 0;  // an infinite a has no rest
      }
    }
    __syncthreads();
  }
}

// down-projection: COLS columns of one expert's rows, then, by the workgroup that
// finishes the column tile, the weighted sum of each token's rows
template <class WT, int NT, int DW>
__global__ void __launch_bounds__(DW * 64) decode_down(const DecodeArgs A) {
  constexpr int C = WT::COLS;
  __shared__ Rows L;
  __shared__ Sums<WT, DW> P;
  const int tiles = A.col_tiles;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int ct = blockIdx.x % tiles;
  const int n0 = ct * C;
  const int width = min(C, (int)A.H - n0);  // H is a multiple of 64: a last tile may be half as wide
  int e, rows, nact;
  const int i = blockIdx.x / tiles;
  const bool have = find_rows<DW>(L, A, i, e, rows, nact);
  if (!have && !(i == 0 && nact == 0)) return;
  const rsrc_t o = make_rsrc(A.o, (int64_t)A.T * A.K * A.H * 4);
  bool last = true;
  if (have) {
    e = __builtin_amdgcn_readfirstlane(e);
    const int nt = __builtin_amdgcn_readfirstlane((rows + 15) >> 4);
    // a half tile's missing columns read its first half again (and are not stored)
    const int64_t c1 = width > C / 2 ? n0 + C / 2 : n0;
    WT W;
    W.init(static_cast<const char*>(A.down) + (int64_t)e * A.H * A.I * A.wbytes, A.I, A.H, n0, c1,
           A.down_descale + (int64_t)e * (A.H / 128) * (A.I / 128), A.I / 128, lane);
    const uint16_t* src[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = n * 16 + (lane & 15);
      src[n] = A.a + (int64_t)L.slot[r < rows ? r : 0] * 2 * A.I + WT::row_offset(lane);
    }
    f32x4 acc[WT::SUB][NT];
    stream_tile<WT, NT, 2, DW>(W, src, A.I, (int)(A.I / WT::DEPTH), wave, lane, nt, acc);
    for (int n = 0; n < nt; ++n) {
#pragma unroll
      for (int q = 0; q < NT; ++q)
        if (q == n) put_sums<WT, NT, DW>(P, acc, q, wave, lane);
      __syncthreads();
      for (int c = threadIdx.x; c < 16 * C / 4; c += DW * 64) {
        const int row = n * 16 + c / (C / 4), col = c % (C / 4) * 4;
        if (row < rows && col < width) {
          f32x4 v;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = get_sum(P, c / (C / 4), col + j);
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), o,
                                                 (int)(uint32_t)(((int64_t)L.slot[row] * A.H + n0 + col) * 4), 0, 16);
        }
      }
      __syncthreads();
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the rows have reached the coherence point
    __syncthreads();
    if (threadIdx.x == 0)
      L.flag = __hip_atomic_fetch_add(A.count + ct, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)nact - 1;
    __syncthreads();
    last = L.flag != 0;
  }
  if (!last) return;
  const int cpr = width / 4;
  for (int c = threadIdx.x; c < A.T * cpr; c += DW * 64) {
    const int t = c / cpr, col = n0 + c % cpr * 4;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < A.K; ++k) {
      const int id = L.ids[t * A.K + k];
      if (id < 0 || id >= A.E) continue;
      int first = k;
      for (int q = 0; q < k; ++q)
        if (L.ids[t * A.K + q] == id) {
          first = q;
          break;
        }
      const float w = A.weights[t * A.K + k];
      const f32x4 v = __builtin_bit_cast(f32x4, bload_coh(o, (uint32_t)(((int64_t)(t * A.K + first) * A.H + col) * 4), 0));
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = __builtin_fmaf(w, v[j], y[j]);
    }
    uint2 out;
    out.x = (uint32_t)f2bf(y[0]) | ((uint32_t)f2bf(y[1]) << 16);
    out.y = (uint32_t)f2bf(y[2]) | ((uint32_t)f2bf(y[3]) << 16);
    *reinterpret_cast<uint2*>(A.y + (int64_t)t * A.H + col) = out;
  }
}

template <class WT, int NT, int DW>
hipError_t launch_experts(const DecodeArgs& A, hipStream_t stream) {
  const int64_t act = A.E < A.T * A.K ? A.E : A.T * A.K;
  decode_up<WT, NT, DW><<<(unsigned)(act * (A.I / (WT::COLS / 2))), DW * 64, 0, stream>>>(A);
  decode_down<WT, NT, DW><<<(unsigned)(act * A.col_tiles), DW * 64, 0, stream>>>(A);
  return hipGetLastError();
}

}  // namespace

int decode_col_tiles(int64_t H, bool fp8) {
  const int c = fp8 ? Fp8Weights<128>::COLS : Bf16Weights::COLS;
  return (int)((H + c - 1) / c);
}

hipError_t launch_router(const uint16_t* x, const void* wr, bool wr_f32, int T, int64_t H, int E, int K, bool renorm,
                         double* logits, int32_t* ids, float* weights, hipStream_t stream) {
  const dim3 grid((E + GE - 1) / GE, (T + GT - 1) / GT);
  if (wr_f32)
    router_logits<float><<<grid, GTHR, 0, stream>>>(x, (const float*)wr, T, H, E, logits);
  else
    router_logits<uint16_t><<<grid, GTHR, 0, stream>>>(x, (const uint16_t*)wr, T, H, E, logits);
  router_topk<<<T, 64, 0, stream>>>(logits, E, K, renorm, ids, weights);
  return hipGetLastError();
}

hipError_t launch_moe_decode(const DecodeArgs& A, bool fp8, hipStream_t stream) {
  // an expert has at most T rows: T / 16 row tiles.  Four of them on bf16 weights
  // hold 128 accumulator registers: four waves a workgroup, one a SIMD.
  if (A.T <= 16)
    return fp8 ? launch_experts<Fp8Weights<128>, 1, 8>(A, stream) : launch_experts<Bf16Weights, 1, 8>(A, stream);
  if (A.T <= 32)
    return fp8 ? launch_experts<Fp8Weights<128>, 2, 8>(A, stream) : launch_experts<Bf16Weights, 2, 8>(A, stream);
  return fp8 ? launch_experts<Fp8Weights<64>, 4, 8>(A, stream) : launch_experts<Bf16Weights, 4, 4>(A, stream);
}

}  // namespace hmm
