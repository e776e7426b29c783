// A whole mixture-of-experts layer for a few tokens (T <= 64), where a chosen
// expert's weights are streamed for a handful of rows:
//
//   l[t,e] = x[t] . Wr[e];  ids[t], w[t] = the K largest logits and their softmax
//   [g|u]  = x[t] . W1[e];  a = silu(g) u;  y[t] = sum_k w[t,k] a . W2[ids[t,k]]
//
// Bound by HBM: an expert's 3 H I weights for 6 H I flop a row, read once for up to 16 or
// 32 rows (one or two row tiles, launch_experts) and again for the next ones.  So nothing of
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
// Two to five launches on one stream, no state kept between calls:
//   logits, top-k        (with a router weight)
//   up-projection        a unit: one chosen expert, 32 to 128 columns of I
//   down-projection      a unit: one chosen expert, 64 to 256 columns of H
//   sum of the rows      above SUM_TOKENS tokens; for fewer of them the workgroup that
//                        finishes a column tile last adds its rows up
// That last step needs no wait: a workgroup stores its rows at the device-wide
// coherence point, counts itself, and only the one that counts last reads them.  Either
// way a token's rows are added in the order of its slots: the same bits on every run.
//
// Measured, bf16, E = 32, H = 7168, I = 2048, K = 8: 1 token: logits 4.7, top-k 4.9, up 88 us
// (470 MB: 5.3 TB/s), down 47 us (235 MB: 5.0 TB/s); 64 tokens: 6, 5, 334 us (1880 MB: 5.6
// TB/s), 199 us (940 MB: 4.7 TB/s), sum 6 us.  E = 128, H = 2048, I = 768, 17 tokens: up 89, down
// 47 us (5.7 and 5.4 TB/s).  E4M3 weights, 8 tokens: up 141 us (5.6 TB/s), down 95 us (4.2
// TB/s).  Reads alone reach 6.2 TB/s here, a copy 5.2.  Experts with more rows than their tiles
// hold: 64 tokens, 8 experts, K = 4 (24 to 41 rows, 11 passes over 8 experts' weights): up 146 us
// (655 MB fetched for 470), down 80 (344 for 235); 4 experts, K = 4 (64 rows, every weight twice):
// 126 and 52 us.
#include "gemm_common.h"
#include "kernels.h"

namespace hmm {
namespace {

constexpr int DT = DECODE_MAX_TOKENS;
constexpr int MAX_SLOTS = DT * 16;
// Workgroups of an expert launch: two a CU (their registers allow no more), each taking units in
// turn and loading across their borders.
constexpr int MAX_GROUPS = 512;
static_assert(DT == 64, "the rows of an expert are one 64-bit lane mask");

// ------------------------------------------------------------------------ router

// logits[t][e] in float64: a workgroup takes one expert and GT tokens, its threads split H in
// 16-byte chunks.  Latency counts: 64 tokens, 32 experts, H = 7168 5.6 us with GT = 4, 5.3 with 2,
// 6.2 with two experts a workgroup; 256 experts 24, 26 and 23 us.
constexpr int GTHR = 512;

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

template <class W, int GT>
__global__ void __launch_bounds__(GTHR) router_logits(const uint16_t* __restrict__ x, const W* __restrict__ wr, int T,
                                                      int64_t H, int E, double* __restrict__ logits) {
  __shared__ double part[GTHR / 64][GT];
  const int e = blockIdx.x, t0 = blockIdx.y * GT;
  double acc[GT] = {};
  for (int64_t c = (int64_t)threadIdx.x * 8; c < H; c += GTHR * 8) {
    double xv[GT][8], wv[8];
#pragma unroll
    for (int t = 0; t < GT; ++t) router8<uint16_t>(x + (int64_t)min(t0 + t, T - 1) * H + c, xv[t]);
    router8<W>(wr + (int64_t)e * H + c, wv);
#pragma unroll
    for (int t = 0; t < GT; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[t] = __builtin_fma(xv[t][j], wv[j], acc[t]);
  }
#pragma unroll
  for (int t = 0; t < GT; ++t) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) acc[t] += __shfl_xor(acc[t], d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][t] = acc[t];
  }
  __syncthreads();
  if (threadIdx.x < GT && t0 + threadIdx.x < T) {
    double s = 0.;
#pragma unroll
    for (int q = 0; q < GTHR / 64; ++q) s += part[q][threadIdx.x];
    logits[(int64_t)(t0 + threadIdx.x) * E + e] = s;
  }
}

// One workgroup per token, one thread per expert: an expert's rank is the number of
// experts before it (a larger logit, or the same and a lower index; a NaN counts as
// -infinity), and ranks below K are the choice.  Then the weights: exp(l - max) over its
// sum over the chosen (renorm) or over all experts, added in a fixed order.
template <int NT>
__global__ void __launch_bounds__(NT) router_topk(const double* __restrict__ logits, int E, int K, int renorm,
                                                  int32_t* __restrict__ ids, float* __restrict__ weights) {
  __shared__ __attribute__((aligned(16))) double l[NT + 2];
  __shared__ float chosen[16];
  __shared__ float part[NT / 64];
  __shared__ double top;
  const int t = blockIdx.x, e = threadIdx.x;
  double v = -__builtin_inf();
  if (e < E) {
    const double x = logits[(int64_t)t * E + e];
    if (x == x) v = x;
  }
  l[e] = v;
  __syncthreads();
  int rank = 0;
  if (e < E) {
    const double2* p = reinterpret_cast<const double2*>(l);
    // threads past E hold -infinity at a higher index: they are before nobody
#pragma unroll 4
    for (int j = 0; j < E; j += 2) {
      const double2 o = p[j >> 1];
      rank += (o.x > v) | ((o.x == v) & (j < e));
      rank += (o.y > v) | ((o.y == v) & (j + 1 < e));
    }
    if (rank == 0) top = v;
  }
  __syncthreads();
  const float x = e < E ? expf((float)(v - top)) : 0.f;
  if (e < E && rank < K) {
    ids[t * K + rank] = e;
    chosen[rank] = x;
  }
  if (!renorm) {
    float s = x;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d);
    if ((e & 63) == 0) part[e >> 6] = s;
  }
  __syncthreads();
  if (e < K) {
    float sum = 0.f;
    if (renorm)
      for (int k = 0; k < K; ++k) sum += chosen[k];
    else
      for (int k = 0; k < NT / 64; ++k) sum += part[k];
    weights[t * K + e] = chosen[e] / sum;
  }
}

// ------------------------------------------------------------------- expert tiles

// What a workgroup finds out first: the experts that some token chose, in ascending order.
struct Chosen {
  int32_t ids[MAX_SLOTS];
  uint32_t bits[MAX_EXPERTS / 32];
  uint16_t expert[MAX_EXPERTS];
  int flag;
};

// LDS written before is readable after, by every wave; loads from global memory stay in flight
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// returns how many experts are chosen
template <int DW>
__device__ __forceinline__ int find_chosen(Chosen& L, const DecodeArgs& A) {
  const int tid = threadIdx.x;
  const int S = A.T * A.K;
  if (tid < MAX_EXPERTS / 32) L.bits[tid] = 0;
  __syncthreads();
  for (int s = tid; s < S; s += DW * 64) {
    const int id = A.ids[s];
    L.ids[s] = id;
    if (id >= 0 && id < A.E) atomicOr(&L.bits[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
  const int lane = tid & 63;
  uint32_t w = lane < MAX_EXPERTS / 32 ? L.bits[lane] : 0u;
  int inc = __popc(w);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  if (tid < MAX_EXPERTS / 32)
    for (int at = inc - __popc(w); w; w &= w - 1) L.expert[at++] = (uint16_t)(tid * 32 + __ffs(w) - 1);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(__shfl(inc, 31));
}

// The rows (tokens) of an expert, found by a wave on its own: their number, and in
// lane r the slot t K + k of row r (k: the first that names the expert; a token that
// names it twice is one row).
__device__ __forceinline__ int find_rows(const Chosen& L, const DecodeArgs& A, int e, int lane, int& slot) {
  int first = -1;
  if (lane < A.T)
    for (int k = A.K - 1; k >= 0; --k)
      if (L.ids[lane * A.K + k] == e) first = k;
  const uint64_t mask = __ballot(first >= 0);
  const int rows = __popcll(mask);
  const uint64_t below = mask & ((1ull << lane) - 1);
  // rows go to the lowest lanes in order, the other lanes behind them: a permutation
  const int to = first >= 0 ? __popcll(below) : rows + lane - __popcll(below);
  slot = __builtin_amdgcn_ds_permute(4 * to, lane * A.K + first);
  return rows;
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
  static constexpr bool WIDE = true;
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
        if (NT == 1 || n < nt)
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
  static constexpr bool WIDE = false;
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
        if (NT == 1 || n < nt) {
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

// A unit of work: a column tile of one expert, for up to 16 NT of its rows (an expert with
// more takes the tile again for the next ones).
template <class WT, int NT>
struct Unit {
  int index, chunk;           // unit number, chunk of 16 NT rows
  int e, tile, rows, nt;      // rows of the expert; row tiles of this chunk
  int slot;                   // lane r: slot of the expert's row r
  WT W;
  const uint16_t* src[NT];    // this lane's row of each row tile
};

// The waves of a tile take the steps of a unit in turn: first, first + DS, ... and load one
// step ahead, across the end of a unit into the next one.  ``next()`` fills a unit with the
// following one and is false at the end.  The rows of a step are fetched with its weights
// (NT == 1), or right before the next step's weights, so that waiting for them leaves those
// in flight (loads return in order).  Rows past the last one repeat row 0: their columns of
// the accumulator are never read.
template <class WT, int NT, int PARTS, int DS>
struct Stream {
  static constexpr bool AHEAD = NT == 1;
  u32x4 w[2][WT::LOADS], b[AHEAD ? 2 : 1][NT][PARTS][WT::ROW_LOADS];
  f32x4 acc[WT::SUB][NT];

  template <int P>
  __device__ __forceinline__ void load_rows(const Unit<WT, NT>& U, int s, int64_t part) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      if (NT == 1 || n < U.nt)
#pragma unroll
        for (int h = 0; h < PARTS; ++h)
#pragma unroll
          for (int q = 0; q < WT::ROW_LOADS; ++q)
            b[AHEAD ? P : 0][n][h][q] = *reinterpret_cast<const u32x4*>(U.src[n] + h * part + (int64_t)s * WT::DEPTH + 8 * q);
  }
  // step s into register set P
  template <int P>
  __device__ __forceinline__ void load(const Unit<WT, NT>& U, int s, int64_t part) {
    U.W.load(s, w[P]);
    if constexpr (AHEAD) load_rows<P>(U, s, part);
    __builtin_amdgcn_sched_barrier(0);  // the loads go out here, not where their data is needed
  }
  // step s from register set P; the rows now, where they are not fetched ahead
  template <int P>
  __device__ __forceinline__ void rows_now(const Unit<WT, NT>& U, int s, int64_t part) {
    if constexpr (!AHEAD) load_rows<0>(U, s, part);
    __builtin_amdgcn_sched_barrier(0);
  }
  template <int P>
  __device__ __forceinline__ void mul(const Unit<WT, NT>& U, int s) {
    U.W.template mul<NT, PARTS>(s, w[P], b[AHEAD ? P : 0], U.nt, acc);
  }
  __device__ __forceinline__ void begin(const Unit<WT, NT>& U, int64_t part, int steps, int first) {
    if (first < steps) load<0>(U, first, part);
  }
  // The sums of U's steps; then U is the next unit with its first step on the way in set 0,
  // or the result is false.
  template <class Next>
  __device__ __forceinline__ bool run(Unit<WT, NT>& U, int64_t part, int steps, int first, Next&& next) {
#pragma unroll
    for (int c = 0; c < WT::SUB; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[c][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    int s = first;
    for (; s + 2 * DS < steps; s += 2 * DS) {
      rows_now<0>(U, s, part);
      load<1>(U, s + DS, part);
      mul<0>(U, s);
      rows_now<1>(U, s + DS, part);
      load<0>(U, s + 2 * DS, part);
      mul<1>(U, s + DS);
    }
    if (s + DS < steps) {
      rows_now<0>(U, s, part);
      load<1>(U, s + DS, part);
      mul<0>(U, s);
      s += DS;
      rows_now<1>(U, s, part);
      Unit<WT, NT> V = U;
      const bool more = next(V);
      if (more) load<0>(V, first, part);
      mul<1>(U, s);
      U = V;
      return more;
    }
    if (s < steps) {
      rows_now<0>(U, s, part);
      mul<0>(U, s);
    }
    const bool more = next(U);
    if (more && first < steps) load<0>(U, first, part);
    return more;
  }
};

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
// the sum of the waves [first, first + N)
template <int N, class WT, int DW>
__device__ __forceinline__ float get_sum(const Sums<WT, DW>& L, int first, int row, int col) {
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < N; ++q) s += L.v[first + q][row][col];
  return s;
}

// up-projection: HC gate columns and the matching up columns of one expert a unit.  Narrow:
// every wave has COLS / 2 of each.  Wide: half of the waves have COLS gate columns, the
// others the up columns, so that a row's bytes lie together (bf16: 256 instead of twice 128).
template <class WT, int NT, int DW, bool WIDE>
__global__ void __launch_bounds__(DW * 64, 2) decode_up(const DecodeArgs A) {
  constexpr int HC = WIDE ? WT::COLS : WT::COLS / 2, DS = WIDE ? DW / 2 : DW;
  __shared__ Chosen L;
  __shared__ Sums<WT, DW> P;
  const int tiles = (int)(A.I / HC), steps = (int)(A.H / WT::DEPTH);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  // the down-projection's counters, cleared one launch ahead of their use
  for (int64_t g = (int64_t)blockIdx.x * DW * 64 + threadIdx.x; g < A.col_tiles; g += (int64_t)gridDim.x * DW * 64)
    A.count[g] = 0;
  const int units = find_chosen<DW>(L, A) * tiles;
  typedef Unit<WT, NT> U;
  auto rows_of = [&](U& u) {
    u.nt = min(NT, (u.rows - u.chunk * 16 * NT + 15) >> 4);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = (u.chunk * NT + n) * 16 + (lane & 15);
      const int slot = __shfl(u.slot, r < u.rows ? r : 0);
      u.src[n] = A.x + (int64_t)(slot / A.K) * A.H + WT::row_offset(lane);
    }
  };
  auto set = [&](U& u, int index) {
    u.index = index;
    u.chunk = 0;
    u.tile = index % tiles;
    u.e = __builtin_amdgcn_readfirstlane((int)L.expert[index / tiles]);
    u.rows = __builtin_amdgcn_readfirstlane(find_rows(L, A, u.e, lane, u.slot));
    const int64_t n0 = (int64_t)u.tile * HC;
    u.W.init(static_cast<const char*>(A.up) + (int64_t)u.e * A.H * 2 * A.I * A.wbytes, A.H, 2 * A.I,
             WIDE && wave >= DS ? A.I + n0 : n0, WIDE ? (wave >= DS ? A.I : 0) + n0 + HC / 2 : A.I + n0,
             A.up_descale + (int64_t)u.e * (2 * A.I / 128) * (A.H / 128), A.H / 128, lane);
    rows_of(u);
  };
  auto next = [&](U& u) {
    if ((u.chunk + 1) * 16 * NT < u.rows) {
      ++u.chunk;
      rows_of(u);
      return true;
    }
    const int index = u.index + (int)gridDim.x;
    if (index >= units) return false;
    set(u, index);
    return true;
  };
  if ((int)blockIdx.x >= units) return;
  U u;
  set(u, blockIdx.x);
  Stream<WT, NT, 1, DS> S;
  const int first = WIDE && wave >= DS ? wave - DS : wave;
  S.begin(u, 0, steps, first);
  for (bool more = true; more;) {
    const int nt = u.nt, row0 = u.chunk * 16 * NT, rows = u.rows, n0 = u.tile * HC, slot_of = u.slot;
    more = S.run(u, 0, steps, first, next);
    for (int n = 0; n < nt; ++n) {
#pragma unroll
      for (int q = 0; q < NT; ++q)
        if (q == n) put_sums<WT, NT, DW>(P, S.acc, q, wave, lane);
      lds_barrier();
      for (int i = threadIdx.x; i < 16 * HC; i += DW * 64) {
        const int row = row0 + n * 16 + i / HC, col = i % HC;
        const int slot = __shfl(slot_of, row & 63);
        if (row < rows) {
          const float gv = get_sum<DS>(P, 0, i / HC, col);
          const float uv = get_sum<DS>(P, DW - DS, i / HC, WIDE ? col : HC + col);
          const float a = gv * sigmoidf_(gv) * uv;
          uint16_t* out = A.a + (int64_t)slot * 2 * A.I + n0 + col;
          const uint16_t hi = f2bf(a);
          const float rest = a - bf2f(hi);
          out[0] = hi;
          out[A.I] = __builtin_isfinite(rest) ? f2bf(rest) : 0;  // an infinite a has no rest
        }
      }
      lds_barrier();
    }
  }
}

// The weighted sum of a token's rows at 4 columns, in the order of its slots, four rows'
// loads at a time.  COH: the rows were written in this launch.
template <bool COH, class Ids>
__device__ __forceinline__ void combine4(const Ids& ids, const DecodeArgs& A, rsrc_t o, int t, int col) {
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < A.K; k0 += 4) {
    f32x4 v[4];
    float w[4];
    bool has[4];  // a dropped slot adds nothing, whatever its weight
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = k0 + j;
      w[j] = 0.f;
      has[j] = false;
      v[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (k >= A.K) continue;
      const int id = ids[t * A.K + k];
      if (id < 0 || id >= A.E) continue;
      int first = 0;  // a repeated expert's row is that of its first slot
      while (ids[t * A.K + first] != id) ++first;
      has[j] = true;
      w[j] = A.weights[t * A.K + k];
      const uint32_t at = (uint32_t)(((int64_t)(t * A.K + first) * A.H + col) * 4);
      v[j] = __builtin_bit_cast(f32x4, COH ? bload_coh(o, at, 0) : bload(o, at, 0));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (has[j])
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = __builtin_fmaf(w[j], v[j][q], y[q]);
  }
  uint2 out;
  out.x = (uint32_t)f2bf(y[0]) | ((uint32_t)f2bf(y[1]) << 16);
  out.y = (uint32_t)f2bf(y[2]) | ((uint32_t)f2bf(y[3]) << 16);
  *reinterpret_cast<uint2*>(A.y + (int64_t)t * A.H + col) = out;
}

template <int THREADS>
__device__ __forceinline__ void combine_tile(const Chosen& L, const DecodeArgs& A, rsrc_t o, int n0, int width) {
  const int cpr = width / 4;
  for (int c = threadIdx.x; c < A.T * cpr; c += THREADS) combine4<true>(L.ids, A, o, c / cpr, n0 + c % cpr * 4);
}

constexpr int CT = 256;
__global__ void __launch_bounds__(CT) decode_combine(const DecodeArgs A) {
  const rsrc_t o = make_rsrc(A.o, (int64_t)A.T * A.K * A.H * 4);
  const int col = (blockIdx.x * CT + threadIdx.x) * 4;
  if (col < A.H) combine4<false>(A.ids, A, o, blockIdx.y, col);
}

// down-projection: CS COLS columns of one expert's rows a unit (a CS-th of the waves for each
// COLS of them), then (SUM) by the workgroup that finishes the column tile the weighted sum of
// each token's rows
template <class WT, int NT, int DW, int CS, bool SUM>
__global__ void __launch_bounds__(DW * 64, 2) decode_down(const DecodeArgs A) {
  constexpr int C = WT::COLS * CS, DS = DW / CS;
  __shared__ Chosen L;
  __shared__ Sums<WT, DW> P;
  const int tiles = (int)((A.H + C - 1) / C), steps = (int)(A.I / WT::DEPTH);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int nact = find_chosen<DW>(L, A), units = nact * tiles;
  const rsrc_t o = make_rsrc(A.o, (int64_t)A.T * A.K * A.H * 4);
  // H is a multiple of 64: a last tile may be narrower
  auto width_of = [&](int tile) { return min(C, (int)A.H - tile * C); };
  if (SUM && units == 0)  // no valid id at all: y is zero
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) combine_tile<DW * 64>(L, A, o, t * C, width_of(t));
  typedef Unit<WT, NT> U;
  auto rows_of = [&](U& u) {
    u.nt = min(NT, (u.rows - u.chunk * 16 * NT + 15) >> 4);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = (u.chunk * NT + n) * 16 + (lane & 15);
      u.src[n] = A.a + (int64_t)__shfl(u.slot, r < u.rows ? r : 0) * 2 * A.I + WT::row_offset(lane);
    }
  };
  auto set = [&](U& u, int index) {
    u.index = index;
    u.chunk = 0;
    u.tile = index % tiles;
    u.e = __builtin_amdgcn_readfirstlane((int)L.expert[index / tiles]);
    u.rows = __builtin_amdgcn_readfirstlane(find_rows(L, A, u.e, lane, u.slot));
    // columns past the last one: the wave reads its first half, or the tile, again (and does not store it)
    int64_t n0 = (int64_t)u.tile * C + wave / DS * WT::COLS;
    if (n0 >= A.H) n0 = (int64_t)u.tile * C;
    u.W.init(static_cast<const char*>(A.down) + (int64_t)u.e * A.H * A.I * A.wbytes, A.I, A.H, n0,
             n0 + WT::COLS / 2 < A.H ? n0 + WT::COLS / 2 : n0, A.down_descale + (int64_t)u.e * (A.H / 128) * (A.I / 128), A.I / 128,
             lane);
    rows_of(u);
  };
  auto next = [&](U& u) {
    if ((u.chunk + 1) * 16 * NT < u.rows) {
      ++u.chunk;
      rows_of(u);
      return true;
    }
    const int index = u.index + (int)gridDim.x;
    if (index >= units) return false;
    set(u, index);
    return true;
  };
  if ((int)blockIdx.x >= units) return;
  U u;
  set(u, blockIdx.x);
  Stream<WT, NT, 2, DS> S;
  const int first = wave % DS;
  S.begin(u, A.I, steps, first);
  for (bool more = true; more;) {
    const int nt = u.nt, row0 = u.chunk * 16 * NT, rows = u.rows, tile = u.tile, slot_of = u.slot;
    const int n0 = tile * C, width = width_of(tile);
    const bool done = row0 + 16 * NT >= rows;  // the expert's last chunk
    more = S.run(u, A.I, steps, first, next);
    for (int n = 0; n < nt; ++n) {
#pragma unroll
      for (int q = 0; q < NT; ++q)
        if (q == n) put_sums<WT, NT, DW>(P, S.acc, q, wave, lane);
      lds_barrier();
      for (int c = threadIdx.x; c < 16 * C / 4; c += DW * 64) {
        const int row = row0 + n * 16 + c / (C / 4), col = c % (C / 4) * 4;
        const int slot = __shfl(slot_of, row & 63);
        if (row < rows && col < width) {
          f32x4 v;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = get_sum<DS>(P, col / WT::COLS * DS, c / (C / 4), col % WT::COLS + j);
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), o,
                                                 (int)(uint32_t)(((int64_t)slot * A.H + n0 + col) * 4), 0, SUM ? 16 : 0);
        }
      }
      lds_barrier();
    }
    if (!SUM || !done) continue;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the rows have reached the coherence point
    lds_barrier();
    if (threadIdx.x == 0)
      L.flag = __hip_atomic_fetch_add(A.count + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)nact - 1;
    __syncthreads();
    if (L.flag) combine_tile<DW * 64>(L, A, o, n0, width);
    lds_barrier();  // the flag has been read
  }
}

template <class W>
void launch_logits(const uint16_t* x, const W* wr, int T, int64_t H, int E, double* logits, hipStream_t stream) {
  if (T == 1)  // four tokens would only repeat it
    router_logits<W, 1><<<E, GTHR, 0, stream>>>(x, wr, T, H, E, logits);
  else
    router_logits<W, 4><<<dim3(E, (T + 3) / 4), GTHR, 0, stream>>>(x, wr, T, H, E, logits);
}

template <class WT, int NT, int DW, bool WIDE>
void launch_up(const DecodeArgs& A, int64_t act, hipStream_t stream) {
  const int64_t units = act * (A.I / (WIDE ? WT::COLS : WT::COLS / 2));
  decode_up<WT, NT, DW, WIDE><<<(unsigned)(units < MAX_GROUPS ? units : MAX_GROUPS), DW * 64, 0, stream>>>(A);
}
template <class WT, int NT, int DW, int CS, bool SUM>
void launch_down(const DecodeArgs& A, int64_t act, hipStream_t stream) {
  const int64_t units = act * ((A.H + WT::COLS * CS - 1) / (WT::COLS * CS));
  decode_down<WT, NT, DW, CS, SUM><<<(unsigned)(units < MAX_GROUPS ? units : MAX_GROUPS), DW * 64, 0, stream>>>(A);
}

constexpr int SUM_TOKENS = 4;  // up to which the down-projection adds the rows up (both sides: launch_experts)

// WA: one row tile at a time, for experts with up to 16 rows (with more, the tile is read again for
// the next 16); WB: two.  One where an expert has 8 rows or fewer on average: up + down of 17 tokens,
// 128 experts, K = 8 (1 row) 89 + 47 us against 93 + 57; 64 tokens, 64 E4M3 experts, K = 8 (8 rows)
// 73 + 49 against 88 + 53; but 64 tokens, 32 experts, K = 6 (12 rows) 409 + 200 against 329 + 190.
// Wide tiles (a wave's 128 columns side by side) where they still give every workgroup a unit:
// up-projection of 32 experts, H = 7168, I = 2048, 64 tokens 332 us wide, 371 narrow; 86 chosen
// experts, H = 2048, I = 768, 17 tokens 91 / 95; down-projection of the latter 56 / 61, of the
// former 200 / 198.  With E4M3 weights wide tiles gained nothing (93 / 89).
template <class WA, class WB, int DW>
hipError_t launch_experts(const DecodeArgs& A, hipStream_t stream) {
  const int64_t act = A.E < A.T * A.K ? A.E : A.T * A.K;  // experts that may be chosen
  const bool few = A.T <= 16 || A.T * A.K <= 8 * A.E;
  bool up = false, down = false;
  if constexpr (WA::WIDE) {
    if (A.I % WA::COLS == 0 && act * (A.I / WA::COLS) >= MAX_GROUPS) {
      few ? launch_up<WA, 1, DW, true>(A, act, stream) : launch_up<WB, 2, DW, true>(A, act, stream);
      up = true;
    }
  }
  if (!up) few ? launch_up<WA, 1, DW, false>(A, act, stream) : launch_up<WB, 2, DW, false>(A, act, stream);
  // Up to 4 tokens the down-projection adds the rows up itself (1 token, 32 experts: 47.5 us, 42.9
  // and 4.8 with the sum as a launch of its own; 64 tokens 244 us, 197 and 6).
  if (A.T <= SUM_TOKENS) {
    launch_down<WA, 1, DW, 1, true>(A, act, stream);
    return hipGetLastError();
  }
  if constexpr (WA::WIDE) {
    if (act * (A.H / (2 * WA::COLS)) >= MAX_GROUPS) {
      few ? launch_down<WA, 1, DW, 2, false>(A, act, stream) : launch_down<WB, 2, DW, 2, false>(A, act, stream);
      down = true;
    }
  }
  if (!down) few ? launch_down<WA, 1, DW, 1, false>(A, act, stream) : launch_down<WB, 2, DW, 1, false>(A, act, stream);
  decode_combine<<<dim3((unsigned)((A.H / 4 + CT - 1) / CT), A.T), CT, 0, stream>>>(A);
  return hipGetLastError();
}

}  // namespace

int decode_col_tiles(int64_t H, bool fp8) {
  const int c = fp8 ? Fp8Weights<128>::COLS : Bf16Weights::COLS;
  return (int)((H + c - 1) / c);
}

hipError_t launch_router(const uint16_t* x, const void* wr, bool wr_f32, int T, int64_t H, int E, int K, bool renorm,
                         double* logits, int32_t* ids, float* weights, hipStream_t stream) {
  if (wr_f32)
    launch_logits(x, (const float*)wr, T, H, E, logits, stream);
  else
    launch_logits(x, (const uint16_t*)wr, T, H, E, logits, stream);
  if (E <= 128)
    router_topk<128><<<T, 128, 0, stream>>>(logits, E, K, renorm, ids, weights);
  else
    router_topk<MAX_EXPERTS><<<T, MAX_EXPERTS, 0, stream>>>(logits, E, K, renorm, ids, weights);
  return hipGetLastError();
}

hipError_t launch_moe_decode(const DecodeArgs& A, bool fp8, hipStream_t stream) {
  return fp8 ? launch_experts<Fp8Weights<128>, Fp8Weights<64>, 4>(A, stream)
             : launch_experts<Bf16Weights, Bf16Weights, 4>(A, stream);
}

}  // namespace hmm
