// The norms before and after a block, fused with the block's gate and the
// residual sum, and their gradients.
//
//   u  = y rho_y,  rho_y = (mean_H y^2 + eps)^-1/2      (post-norm; u = y without a post weight)
//   r' = round(r + s g wp u)                            (the residual stream as it is stored)
//   n  = r' rho w, rho   = (mean_H r'^2 + eps)^-1/2     (the next block's pre-norm)
//
// and, with t the whole gradient of r' (tr that of its output, dn that of n):
//   x  = r' rho;   a = dn w;   t = tr + rho (a - x mean(a x));   dr = t
//   b  = s t g wp;  dy = rho_y (b - u mean(b u))  (dy = b without a post weight)
//   dw = sum_t dn x;  dwp = sum_t s t g u;  dg = s t wp u, summed over what g is broadcast over
//
// The gradients are taken of the normalised rows x and u, at most sqrt(H) in size: rho^3 as a
// factor of its own leaves float32 for rows of 1e14 and for an eps below 2e-26.
//
// n is taken of the stored (rounded) r', so that the backward, which reads the
// stored r', is the gradient of exactly what the forward computed.
//
// All of it is bound by HBM: a row is read once, kept in registers between the
// reductions (two in the forward, two in the backward), and written once; every
// sum is float32.  A row belongs to one wave (H <= 1024) or one workgroup, V
// 16-byte chunks per thread; the next row's loads are in flight while this one is
// reduced and written.  The backward's column sums stay in registers
// while a workgroup walks its rows (one fixed set of workgroups, whatever the
// device), then go to the workspace as one partial row per workgroup, and a
// second launch adds those in order: no atomics, the same bits on every run.
//
// Measured: 8192 rows of 7168, bf16: forward 85-96 us for 470 MB (4.9-5.5 TB/s),
// backward 132-142 us for 705 MB (5.0-5.3 TB/s) and 4 us for the sums; 4001 rows of
// 2048 with a float32 stream: 21 us (98 MB, in part from the L2 caches and the
// infinity cache), 28 us and 4 us; 16384 rows of 512: 14, 22 and 4 us.  A large copy reaches 5.2 TB/s.  One row: 3.9 us.
#include "device.h"
#include "kernels.h"

namespace hmm {
namespace {

constexpr int MAX_THREADS_PER_ROW = 1024;

// 8 consecutive elements at index i of a bf16 or float32 array
__device__ __forceinline__ void load8(const void* p, bool f32, int64_t i, float (&v)[8]) {
  if (f32) {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  } else {
    unpack8(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i), v);
  }
}
__device__ __forceinline__ void store8(void* p, bool f32, int64_t i, const float (&v)[8], bool stream = false) {
  if (f32) {
    f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + i);
    q[0] = f32x4{v[0], v[1], v[2], v[3]};
    q[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else if (stream) {
    store16_stream(static_cast<uint16_t*>(p) + i, pack8(v));
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = pack8(v);
  }
}

// 1 / sqrt(m): the hardware's v_rsq_f32 (one ulp) and one Newton step
__device__ __forceinline__ float rsqrt_(float m) {
  const float r = __builtin_amdgcn_rsqf(m);
  const float c = __builtin_fmaf(0.5f * r, __builtin_fmaf(-m * r, r, 1.0f), r);
  return __builtin_isfinite(c) ? c : r;  // m infinite: 0, of which the step would make a NaN
}

// sums of N values over the NT threads of a row, in a fixed order, to every thread
template <int NT, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* lds) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor(v[k], d);
  if constexpr (NT > 64) {
    constexpr int NW = NT / 64;
    __syncthreads();  // the previous reduction's values have been read
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) lds[(threadIdx.x >> 6) * N + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < NW; ++q) s += lds[q * N + k];
      v[k] = s;
    }
  }
}

// gate of 8 columns of row t
__device__ __forceinline__ void gate8(const NormArgs& A, int64_t t, int64_t i, float (&g)[8]) {
  if (A.gate_kind == NORM_GATE_TOKEN) {
    const float v = bf2f(A.gate[t]);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = v;
  } else if (A.gate_kind == NORM_GATE_CHANNEL) {
    load8(A.gate, false, i, g);
  } else if (A.gate_kind == NORM_GATE_FULL) {
    load8(A.gate, false, t * A.H + i, g);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 1.f;
  }
}

template <int NT>
constexpr int rows_per_block() { return NT == 64 ? 4 : 1; }

// 8 elements as they were loaded: bf16, or float32 where F32
template <bool F32>
struct Raw8 {
  u32x4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const char*>(p) + i * (F32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < (F32 ? 2 : 1); ++k) v[k] = q[k];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < (F32 ? 2 : 1); ++k) v[k] = u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(v[j >> 2][j & 3]);
    } else {
      unpack8(v[0], f);
    }
  }
};

// RF, WF: the residual stream and the weights are float32.
template <int NT, int V, bool RF, bool WF>
__global__ void __launch_bounds__(NT == 64 ? 256 : NT) residual_norm_fwd(const NormArgs A) {
  constexpr int RPB = rows_per_block<NT>();
  __shared__ float lds[MAX_THREADS_PER_ROW / 64];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int slot = NT == 64 ? threadIdx.x >> 6 : 0;
  const float invH = 1.f / (float)A.H;
  Raw8<WF> w[V], wp[V];
  // a row's data is loaded while the row before it is reduced and written
  struct Row {
    Raw8<RF> r[V];
    Raw8<false> y[V];
  };
  auto load = [&](Row& R, int64_t t) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int64_t i = (int64_t)(tid + k * NT) * 8;
      R.r[k].zero();
      R.y[k].zero();
      if (i >= A.H) continue;
      R.r[k].load(A.residual, t * A.H + i);
      if (A.y) R.y[k].load(A.y, t * A.H + i);
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t t = (int64_t)blockIdx.x * RPB + slot;
  Row R;
  if (t < A.T) load(R, t);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int64_t i = (int64_t)(tid + k * NT) * 8;
    w[k].zero();
    wp[k].zero();
    if (i >= A.H) continue;
    w[k].load(A.norm_weight, i);
    if (A.post_weight) wp[k].load(A.post_weight, i);
  }
  for (; t < A.T; t += step) {
    Row N;
    load(N, t + step < A.T ? t + step : t);
    __builtin_amdgcn_sched_barrier(0);
    float r[V][8];
    float sum[1] = {0.f};
#pragma unroll
    for (int k = 0; k < V; ++k) R.r[k].get(r[k]);
    if (A.y) {
      float rho_y = 1.f;
      if (A.post_weight) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          float y[8];
          R.y[k].get(y);
#pragma unroll
          for (int j = 0; j < 8; ++j) sum[0] = __builtin_fmaf(y[j], y[j], sum[0]);
        }
        row_sum<NT>(sum, lds);
        rho_y = rsqrt_(__builtin_fmaf(sum[0], invH, A.eps));
      }
      if (tid == 0 && A.rstd) A.rstd[t] = rho_y;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int64_t i = (int64_t)(tid + k * NT) * 8;
        if (i >= A.H) continue;
        float g[8], y[8], wpv[8];
        gate8(A, t, i, g);
        R.y[k].get(y);
        if (A.post_weight) {
          wp[k].get(wpv);
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] *= rho_y * wpv[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          r[k][j] = __builtin_fmaf(A.scale * g[j], y[j], r[k][j]);
          if (!RF) r[k][j] = round_bf(r[k][j]);
        }
        store8(A.residual_out, RF, t * A.H + i, r[k], A.stream);
      }
    }
    sum[0] = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[0] = __builtin_fmaf(r[k][j], r[k][j], sum[0]);
    row_sum<NT>(sum, lds);
    const float rho = rsqrt_(__builtin_fmaf(sum[0], invH, A.eps));
    if (tid == 0 && A.rstd) A.rstd[A.T + t] = rho;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int64_t i = (int64_t)(tid + k * NT) * 8;
      if (i >= A.H) continue;
      float wv[8], n[8];
      w[k].get(wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) n[j] = r[k][j] * rho * wv[j];
      store8(A.normed, false, t * A.H + i, n, A.stream);
    }
    R = N;
  }
}

// RF, WF: the residual stream and the weights are float32; CHAN: the gate is per channel.
template <int NT, int V, bool RF, bool WF, bool CHAN>
__global__ void __launch_bounds__(NT == 64 ? 256 : NT) residual_norm_bwd(const NormArgs A, const NormGradArgs G) {
  constexpr int RPB = rows_per_block<NT>();
  __shared__ float lds[2 * MAX_THREADS_PER_ROW / 64];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int slot = NT == 64 ? threadIdx.x >> 6 : 0;
  const float invH = 1.f / (float)A.H;
  constexpr bool AHEAD = NT * V <= 1024;  // wider rows have no registers for two of them
  float cw[V][8], cp[V][8], cg[CHAN ? V : 1][8];  // column sums of dw, dwp, dg
  Raw8<WF> w[V], wp[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int64_t i = (int64_t)(tid + k * NT) * 8;
    w[k].zero();
    wp[k].zero();
    if (i < A.H) {
      w[k].load(A.norm_weight, i);
      if (A.post_weight) wp[k].load(A.post_weight, i);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) cw[k][j] = cp[k][j] = cg[CHAN ? k : 0][j] = 0.f;
  }
  // a row's data is loaded while the row before it is reduced and written
  struct Row {
    Raw8<RF> r[V], tr[V];
    Raw8<false> d[V], y[V];
    float rho, rho_y;
  };
  auto load = [&](Row& R, int64_t t) {
    R.rho = A.rstd[A.T + t];
    R.rho_y = A.y ? A.rstd[t] : 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int64_t i = (int64_t)(tid + k * NT) * 8;
      R.r[k].zero();
      R.tr[k].zero();
      R.d[k].zero();
      R.y[k].zero();
      if (i >= A.H) continue;
      R.r[k].load(A.residual, t * A.H + i);
      if (G.d_normed) R.d[k].load(G.d_normed, t * A.H + i);
      if (G.d_residual_out) R.tr[k].load(G.d_residual_out, t * A.H + i);
      if (A.y) R.y[k].load(A.y, t * A.H + i);
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t t = (int64_t)blockIdx.x * RPB + slot;
  Row R;
  if (AHEAD && t < A.T) load(R, t);
  for (; t < A.T; t += step) {
    Row N;
    if constexpr (AHEAD) {
      load(N, t + step < A.T ? t + step : t);
      __builtin_amdgcn_sched_barrier(0);
    } else {
      load(R, t);
    }
    const float rho = R.rho;
    float d[V][8], tr[V][8];
    float s1[1] = {0.f};
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float r[8], wv[8];
      R.r[k].get(r);
      R.d[k].get(d[k]);
      w[k].get(wv);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = r[j] * rho;
        cw[k][j] = __builtin_fmaf(d[k][j], x, cw[k][j]);
        d[k][j] *= wv[j];
        s1[0] = __builtin_fmaf(d[k][j], x, s1[0]);
      }
    }
    row_sum<NT>(s1, lds);
    const float m1 = s1[0] * invH;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int64_t i = (int64_t)(tid + k * NT) * 8;
      float r[8];
      R.r[k].get(r);
      R.tr[k].get(tr[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        tr[k][j] = __builtin_fmaf(rho, __builtin_fmaf(-m1, r[j] * rho, d[k][j]), tr[k][j]);
      if (i < A.H) store8(G.d_residual, RF, t * A.H + i, tr[k], A.stream);
    }
    if (A.y) {  // the same for every thread
      const float rho_y = R.rho_y;
      float s2[2] = {0.f, 0.f};  // sum b u, sum s t wp u
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int64_t i = (int64_t)(tid + k * NT) * 8;
        if (i >= A.H) continue;
        float g[8], wpv[8], dg[8], y[8];
        gate8(A, t, i, g);
        R.y[k].get(y);
        if (A.post_weight)
          wp[k].get(wpv);
        else
#pragma unroll
          for (int j = 0; j < 8; ++j) wpv[j] = 1.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float st = A.scale * tr[k][j], u = y[j] * rho_y;
          dg[j] = st * wpv[j] * u;
          if constexpr (CHAN) cg[k][j] += dg[j];
          s2[1] += dg[j];
          cp[k][j] = __builtin_fmaf(st * g[j], u, cp[k][j]);
          tr[k][j] = st * g[j] * wpv[j];  // b
          s2[0] = __builtin_fmaf(tr[k][j], u, s2[0]);
        }
        if (A.gate_kind == NORM_GATE_FULL) store8(G.d_gate, false, t * A.H + i, dg);
      }
      row_sum<NT>(s2, lds);
      if (A.gate_kind == NORM_GATE_TOKEN && tid == 0) static_cast<uint16_t*>(G.d_gate)[t] = f2bf(s2[1]);
      const float m2 = A.post_weight ? s2[0] * invH : 0.f;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int64_t i = (int64_t)(tid + k * NT) * 8;
        if (i >= A.H) continue;
        float dy[8], y[8];
        R.y[k].get(y);
#pragma unroll
        for (int j = 0; j < 8; ++j) dy[j] = rho_y * __builtin_fmaf(-m2, y[j] * rho_y, tr[k][j]);
        store8(G.d_y, false, t * A.H + i, dy, A.stream);
      }
    }
    if constexpr (AHEAD) R = N;
  }

  // one partial row per workgroup: dw, then dwp, then dg (those that are asked for)
  float* p = G.partial + (int64_t)blockIdx.x * A.H;
  const int64_t next = (int64_t)gridDim.x * A.H;
  auto put = [&](const float (&c)[V][8]) {
    if constexpr (RPB > 1) {  // the waves' sums in LDS first, added in the waves' order
      __shared__ __attribute__((aligned(16))) float waves[RPB][NT * V * 8];
      __syncthreads();  // the previous array has been read
#pragma unroll
      for (int k = 0; k < V; ++k) store8(waves[slot], true, (tid + k * NT) * 8, c[k]);
      __syncthreads();
      const int i = threadIdx.x * 8;
      if (threadIdx.x < NT * V && i < A.H) {
        float s[8], v[8];
        load8(waves[0], true, i, s);
#pragma unroll
        for (int q = 1; q < RPB; ++q) {
          load8(waves[q], true, i, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[j] += v[j];
        }
        store8(p, true, i, s);
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int64_t i = (int64_t)(tid + k * NT) * 8;
        if (i < A.H) store8(p, true, i, c[k]);
      }
    }
    p += next;
  };
  static_assert(RPB == 1 || NT * V <= NT * RPB, "a thread for each chunk");
  put(cw);
  if (A.post_weight) put(cp);
  if constexpr (CHAN) put(cg);
}

// out[c] = sum of the np partial rows of column c, in order: 16 row groups of 64
// columns each, then the groups.  blockIdx.y names the array.
constexpr int PS_GROUPS = 16;
__global__ void __launch_bounds__(64 * PS_GROUPS) norm_partial_sum(const float* __restrict__ partial, int np, int64_t H,
                                                                   const NormSums S) {
  __shared__ float part[PS_GROUPS][64];
  const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const int q = threadIdx.x >> 6;
  const int per = (np + PS_GROUPS - 1) / PS_GROUPS;
  const float* p = partial + (int64_t)blockIdx.y * np * H;
  float s = 0.f;
  if (c < H)
#pragma unroll 8
    for (int r = q * per; r < min(np, (q + 1) * per); ++r) s += p[(int64_t)r * H + c];
  part[q][threadIdx.x & 63] = s;
  __syncthreads();
  if (q || c >= H) return;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < PS_GROUPS; ++k) s += part[k][threadIdx.x];
  void* out = S.out[blockIdx.y];
  if (S.f32[blockIdx.y])
    static_cast<float*>(out)[c] = s;
  else
    static_cast<uint16_t*>(out)[c] = f2bf(s);
}

// Calls f<threads per row, chunks per thread> for rows of H elements.  Few waves a row, so that
// several rows overlap on a CU, as far as registers hold a row and the next one.  Forward /
// backward of 8192 rows of 7168: 512 threads 85 / 132 us, 1024 106 / 140, 256 100 / 162; of 4096:
// 256 threads 48 / 74, 512 52 / 72, 128 59 / 92; of 2048: 256 threads 25 / 40, 128 26 / 50;
// 32000 of 1408: 192 threads 76 / 118, 256 84 / 137 us; 2000
// rows of 16384: 1024 threads 52 / 160, 512 54 / 144.
template <class F>
hipError_t for_width(int64_t H, F&& f) {
  if (H <= 512) return f.template operator()<64, 1>();
  if (H <= 1024) return f.template operator()<64, 2>();
  if (H <= 1536) return f.template operator()<192, 1>();
  if (H <= 2048) return f.template operator()<256, 1>();
  if (H <= 4096) return f.template operator()<256, 2>();
  if (H <= 8192) return f.template operator()<512, 2>();
  return f.template operator()<F::LONGEST, 2048 / F::LONGEST>();
}

// Threads of a forward launch: as many as the 256 CUs hold.  Each row walker takes rows in turn.
constexpr int FWD_THREADS = 1 << 19;
struct FwdLaunch {
  static constexpr int LONGEST = 1024;  // threads of rows above 8192
  const NormArgs& A;
  hipStream_t stream;
  template <int NT, int V, bool RF, bool WF>
  void launch() {
    constexpr int R = rows_per_block<NT>(), B = NT == 64 ? 256 : NT;
    const int64_t rows = (A.T + R - 1) / R, most = FWD_THREADS / B;
    residual_norm_fwd<NT, V, RF, WF><<<(unsigned)(rows < most ? rows : most), B, 0, stream>>>(A);
  }
  template <int NT, int V>
  hipError_t operator()() {
    if (A.res_f32)
      A.w_f32 ? launch<NT, V, true, true>() : launch<NT, V, true, false>();
    else
      A.w_f32 ? launch<NT, V, false, true>() : launch<NT, V, false, false>();
    return hipGetLastError();
  }
};
struct BwdLaunch {
  static constexpr int LONGEST = 512;
  const NormArgs& A;
  const NormGradArgs& G;
  int blocks;
  hipStream_t stream;
  template <int NT, int V>
  hipError_t operator()() {
    if (A.res_f32)
      A.w_f32 ? launch<NT, V, true, true>() : launch<NT, V, true, false>();
    else
      A.w_f32 ? launch<NT, V, false, true>() : launch<NT, V, false, false>();
    return hipGetLastError();
  }
  template <int NT, int V, bool RF, bool WF>
  void launch() {
    constexpr int B = NT == 64 ? 256 : NT;
    if (A.gate_kind == NORM_GATE_CHANNEL)
      residual_norm_bwd<NT, V, RF, WF, true><<<blocks, B, 0, stream>>>(A, G);
    else
      residual_norm_bwd<NT, V, RF, WF, false><<<blocks, B, 0, stream>>>(A, G);
  }
};

// Workgroups of the backward, each with one partial row: 512 (of 256 threads with two chunks
// each: two waves a SIMD, as the registers allow), 768 of one chunk (three), 256 of 512 threads.
// 8192 rows of 7168: 256 of them 132 us and 4 us for their sums, 512 136 + 6; 16000 rows of 2048: 768 74 + 4, 512 84 + 4; 16384 rows of 512: 256 28 + 4,
// 512 22 + 4, 1024 24 + 5.
inline int bwd_blocks(int64_t T, int64_t H) {
  const int64_t rpb = H <= 1024 ? 4 : 1;
  const int64_t b = (T + rpb - 1) / rpb, most = H > 4096 ? 256 : H > 1024 && H <= 2048 ? 768 : 512;
  return (int)(b < most ? b : most);
}

}  // namespace

int64_t norm_partial_rows(int64_t T, int64_t H) { return bwd_blocks(T, H); }

// Outputs past the L2 caches' 32 MB are stored with the streaming hint (8192 rows of 7168,
// backward: 144 us with it, 154 without).
inline bool streams(const NormArgs& A) { return A.T * A.H * 2 > (32 << 20); }

hipError_t launch_residual_norm(const NormArgs& args, hipStream_t stream) {
  NormArgs A = args;
  A.stream = streams(A);
  if (A.T == 0) return hipSuccess;
  return for_width(A.H, FwdLaunch{A, stream});
}

hipError_t launch_residual_norm_bwd(const NormArgs& args, const NormGradArgs& G, hipStream_t stream) {
  NormArgs A = args;
  A.stream = streams(A);
  if (A.T > 0) {
    const hipError_t e = for_width(A.H, BwdLaunch{A, G, bwd_blocks(A.T, A.H), stream});
    if (e != hipSuccess) return e;
  }
  NormSums S{};
  int n = 0;
  S.out[n] = G.d_norm_weight;
  S.f32[n++] = A.w_f32;
  if (A.post_weight) {
    S.out[n] = G.d_post_weight;
    S.f32[n++] = A.w_f32;
  }
  if (A.gate_kind == NORM_GATE_CHANNEL) {
    S.out[n] = G.d_gate;
    S.f32[n++] = false;
  }
  norm_partial_sum<<<dim3((unsigned)((A.H + 63) / 64), n), 64 * PS_GROUPS, 0, stream>>>(
      G.partial, (int)norm_partial_rows(A.T, A.H), A.H, S);
  return hipGetLastError();
}

}  // namespace hmm
