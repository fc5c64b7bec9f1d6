// CUDA-core kernels of the gated recurrence (every shape and type that the
// tensor-core kernels of la2_gated_sm100.cuh do not take), and the small fp32
// kernels both paths share: the scan of chunk states, the pool update after a
// prefill, and the gradient of the gates.
//
// Per (b, h) sequence, with one log gate l_t a token (-inf: the state restarts):
//
//   KV_t = e^(l_t) KV_(t-1) + k_t^T v_t,      o_t = q_t KV_t
//
// so o = ((q k^T) ⊙ D) v with D[t][s] = e^(l_(s+1) + ... + l_t) for s <= t.
// Blocks of 64 rows: with c_t the running sum of the gates inside a block, the
// state KV before it and c_R its last sum,
//
//   O_t  = sum_{j<=t} e^(c_t - c_j) (q_t . k_j) v_j + e^(c_t) q_t KV
//   KV  <- e^(c_R) KV + sum_j e^(c_R - c_j) k_j^T v_j
//
// and walking back, with U = sum over later rows t of D[t][R] q_t^T dO_t,
//
//   dK_j = sum_{t>=j} e^(c_t - c_j) (dO_t . v_j) q_t + e^(c_R - c_j) v_j U^T   (dV alike)
//   U   <- e^(c_R) U + sum_t e^(c_t) q_t^T dO_t
//
// No exponent is ever positive unless a gate is: nothing is divided by a decay.
// The sums c are fp64 here (their differences are what is exponentiated; in fp32
// a sum of 64 gates of -1 would leave the weights 4e-6 off, a fifth of what an
// fp32 result may be); a gate of -inf counts as kLogZero, whose exponential is 0.
//
// The gate's gradient is the flow of pairs across its token,
//   dl_t = sum_{i >= t > j} D[i][j] (q_i . k_j)(dO_i . v_j),
// and satisfies dl_t = dl_(t+1) + q_t . dq_t - k_t . dk_t. The row dots leave the
// dQ and dK passes in fp32; the flow at a chunk's end is <KV, U> of the two chunk
// states there, so the running difference only spans one chunk.
//
// What bounds it: shared-memory reads (8 words for 16 multiply-adds per thread),
// about half of the fp32 rate; the workload is short sequences in fp32.
#pragma once

#include <algorithm>

#include "la2_common.cuh"

namespace la2 {
namespace gated {

constexpr int kThreads = 256;
constexpr int kRows = 64;
constexpr double kLogZero = -1.0e4;

// A log gate as the sums take it. A comparison, not fmax: NaN stays NaN.
__device__ __forceinline__ double gate_log(float x) {
  return x < static_cast<float>(kLogZero) ? kLogZero : static_cast<double>(x);
}
__host__ __device__ __forceinline__ int odd(int w) { return w | 1; }  // row stride of a tile in smem

// out(r, c) = sum_k a(r, k) b(k, c), optionally scaled per row and continued with
// a second sum: r < R, c < Cn. Threads are 16 x 16; a thread owns rows tr + 16 i
// and columns tc + 16 j, so neighbouring lanes read neighbouring (or odd-strided)
// words. ep(r, c, value) returns what the row's dot adds; rowend(r, dot) is called
// by one lane a row, always the same one, after each tile of 64 columns.
template <class A1, class B1, class SC, class A2, class B2, class EP, class RE>
__device__ __forceinline__ void tile_product(int R, int Cn, int K1, A1 a1, B1 b1, SC scale, int K2, A2 a2,
                                             B2 b2, EP ep, RE rowend) {
  const int tc = threadIdx.x & 15, tr = threadIdx.x >> 4;
  for (int c0 = 0; c0 < Cn; c0 += 64) {
    for (int r0 = 0; r0 < R; r0 += 64) {
      float acc[4][4];
      int rr[4], cc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rr[i] = min(r0 + tr + 16 * i, R - 1);
        cc[i] = min(c0 + tc + 16 * i, Cn - 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
      }
#pragma unroll 4
      for (int k = 0; k < K1; ++k) {
        float x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) { x[i] = a1(rr[i], k); y[i] = b1(k, cc[i]); }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = scale(rr[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] *= f;
      }
#pragma unroll 4
      for (int k = 0; k < K2; ++k) {
        float x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) { x[i] = a2(rr[i], k); y[i] = b2(k, cc[i]); }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + tr + 16 * i;
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = c0 + tc + 16 * j;
          if (r < R && c < Cn) dot += ep(r, c, acc[i][j]);
        }
        rowend(r, dot, tc);
      }
    }
  }
}

// Sum of `x` over the 16 lanes of a half warp.
__device__ __forceinline__ float half_warp_sum(float x) {
#pragma unroll
  for (int m = 8; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

struct Zero2 { __device__ float operator()(int, int) const { return 0.f; } };
struct One1 { __device__ float operator()(int) const { return 1.f; } };
struct NoRow { __device__ void operator()(int, float, int) const {} };

// Rows [0, rows) of a [*, w] tensor into an fp32 tile of stride odd(w); the rest zero.
__device__ __forceinline__ void load_rows(float* dst, const float* __restrict__ src, int rows, int w) {
  const int ld = odd(w);
  for (int i = threadIdx.x; i < kRows * w; i += kThreads) {
    const int r = i / w, c = i - r * w;
    dst[r * ld + c] = r < rows ? src[i] : 0.f;
  }
}

// The block's gate sums: c[t] for t < kRows (rows behind the last one repeat it)
// and the weights e^(c_t) and e^(c_R - c_t). `start`: the block opens its sequence,
// where nothing comes before the first token for its gate to pass on (0, unless NaN).
// Ends with a barrier.
__device__ __forceinline__ void gate_tables(const float* __restrict__ gate, int rows, bool start, double* c,
                                            float* head, float* tail) {
  if (threadIdx.x < 32) {
    const int i = 2 * threadIdx.x;
    double x = i < rows ? gate_log(gate[i]) : 0.0;
    if (start && i == 0 && x == x) x = 0.0;
    const double y = i + 1 < rows ? gate_log(gate[i + 1]) : 0.0;
    double s = x + y;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, s, m);
      if (threadIdx.x >= m) s += up;
    }
    c[i] = s - y;
    c[i + 1] = s;
  }
  __syncthreads();
  if (threadIdx.x < kRows) {
    head[threadIdx.x] = expf(static_cast<float>(c[threadIdx.x]));
    tail[threadIdx.x] = expf(static_cast<float>(c[kRows - 1] - c[threadIdx.x]));
  }
  __syncthreads();
}

__device__ __forceinline__ float pair_weight(const double* c, int t, int s) {
  return s <= t ? expf(static_cast<float>(c[t] - c[s])) : 0.f;
}

// state (d x dv, stride odd(dv)) <- e^(c_R) state + sum_t w_t a_t^T b_t
template <class W>
__device__ __forceinline__ void update_state(float* S, const float* a, const float* b, W w, int d, int dv,
                                             int rows, float whole) {
  const int la = odd(d), lb = odd(dv);
  tile_product(
      d, dv, rows, [&](int r, int k) { return w(k) * a[k * la + r]; },
      [&](int k, int c) { return b[k * lb + c]; }, One1{}, 0, Zero2{}, Zero2{},
      [&](int r, int c, float x) {
        S[r * lb + c] = fmaf(whole, S[r * lb + c], x);
        return 0.f;
      },
      NoRow{});
}

__device__ __forceinline__ void load_state_tile(float* S, const float* __restrict__ src, int d, int dv) {
  const int ld = odd(dv);
  for (int i = threadIdx.x; i < d * dv; i += kThreads) {
    const int r = i / dv, c = i - r * dv;
    S[r * ld + c] = src ? src[i] : 0.f;
  }
}

struct Shape {
  int64_t N, L, C;
  int d, dv;
};

// Floats of shared memory: a state, `a` tiles of d and `b` of dv columns, `s` score tiles, the tables.
__host__ __device__ __forceinline__ size_t smem_bytes(int d, int dv, int a, int b, int s) {
  return kRows * sizeof(double) +
         sizeof(float) * ((size_t)d * odd(dv) + (size_t)kRows * (a * odd(d) + b * odd(dv)) +
                          (size_t)s * kRows * odd(kRows) + 3 * kRows);
}

// Own state of every chunk: SUFFIX false, sum_s e^(rest of the chunk's gates) a_s^T b_s
// (the state after the chunk); SUFFIX true, sum_t e^(the chunk's gates up to t)
// a_t^T b_t (decayed back to the row before the chunk). tot: the chunk's sum of gates.
template <bool SUFFIX>
__global__ void __launch_bounds__(kThreads)
chunk_state_kernel(const float* __restrict__ a, const float* __restrict__ b, const float* __restrict__ gate,
                   float* __restrict__ out, double* __restrict__ tot, const Shape sh) {
  extern __shared__ double smem_d[];
  double* c = smem_d;
  float* S = reinterpret_cast<float*>(c + kRows);
  float* As = S + sh.d * odd(sh.dv);
  float* Bs = As + kRows * odd(sh.d);
  float *head = Bs + kRows * odd(sh.dv), *tail = head + kRows;
  const int64_t bh = blockIdx.x / sh.C, ch = blockIdx.x % sh.C;
  const int64_t t0 = ch * sh.L, t1 = imin64(sh.N, t0 + sh.L);
  const int nblk = static_cast<int>((t1 - t0 + kRows - 1) / kRows);
  load_state_tile(S, nullptr, sh.d, sh.dv);
  double sum = 0.0;
  for (int n = 0; n < nblk; ++n) {
    const int64_t i0 = t0 + static_cast<int64_t>(SUFFIX ? nblk - 1 - n : n) * kRows;
    const int rows = static_cast<int>(imin64(kRows, t1 - i0));
    __syncthreads();
    load_rows(As, a + (bh * sh.N + i0) * sh.d, rows, sh.d);
    load_rows(Bs, b + (bh * sh.N + i0) * sh.dv, rows, sh.dv);
    gate_tables(gate + bh * sh.N + i0, rows, false, c, head, tail);
    sum += c[kRows - 1];
    const float whole = head[kRows - 1];
    const float* w = SUFFIX ? head : tail;
    update_state(S, As, Bs, [&](int k) { return w[k]; }, sh.d, sh.dv, rows, whole);
  }
  __syncthreads();
  float* o = out + static_cast<int64_t>(blockIdx.x) * sh.d * sh.dv;
  for (int i = threadIdx.x; i < sh.d * sh.dv; i += kThreads) o[i] = S[(i / sh.dv) * odd(sh.dv) + i % sh.dv];
  if (threadIdx.x == 0) tot[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads)
fwd_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
           const float* __restrict__ gate, float* __restrict__ o, const float* __restrict__ states, const Shape sh) {
  extern __shared__ double smem_d[];
  const int d = sh.d, dv = sh.dv, ld = odd(d), lv = odd(dv), ls = odd(kRows);
  double* c = smem_d;
  float* S = reinterpret_cast<float*>(c + kRows);
  float* Qs = S + d * lv;
  float* Ks = Qs + kRows * ld;
  float* Vs = Ks + kRows * ld;
  float* P = Vs + kRows * lv;
  float *head = P + kRows * ls, *tail = head + kRows;
  const int64_t bh = blockIdx.x / sh.C, ch = blockIdx.x % sh.C;
  const int64_t t0 = ch * sh.L, t1 = imin64(sh.N, t0 + sh.L);
  load_state_tile(S, states ? states + static_cast<int64_t>(blockIdx.x) * d * dv : nullptr, d, dv);
  for (int64_t i0 = t0; i0 < t1; i0 += kRows) {
    const int rows = static_cast<int>(imin64(kRows, t1 - i0));
    const int64_t row = bh * sh.N + i0;
    __syncthreads();
    load_rows(Qs, q + row * d, rows, d);
    load_rows(Ks, k + row * d, rows, d);
    load_rows(Vs, v + row * dv, rows, dv);
    gate_tables(gate + row, rows, i0 == 0, c, head, tail);
    tile_product(
        rows, rows, d, [&](int r, int x) { return Qs[r * ld + x]; }, [&](int x, int j) { return Ks[j * ld + x]; },
        One1{}, 0, Zero2{}, Zero2{},
        [&](int t, int j, float x) {
          P[t * ls + j] = j <= t ? x * pair_weight(c, t, j) : 0.f;
          return 0.f;
        },
        NoRow{});
    __syncthreads();
    float* ob = o + row * dv;
    tile_product(
        rows, dv, d, [&](int r, int x) { return Qs[r * ld + x]; }, [&](int x, int e) { return S[x * lv + e]; },
        [&](int r) { return head[r]; }, rows, [&](int r, int j) { return P[r * ls + j]; },
        [&](int j, int e) { return Vs[j * lv + e]; },
        [&](int t, int e, float x) {
          ob[t * dv + e] = x;
          return 0.f;
        },
        NoRow{});
    __syncthreads();
    update_state(S, Ks, Vs, [&](int j) { return tail[j]; }, d, dv, rows, head[kRows - 1]);
  }
}

// dQ_t = sum_{j<=t} e^(c_t - c_j) (dO_t . v_j) k_j + e^(c_t) dO_t KV^T, and q_t . dq_t.
__global__ void __launch_bounds__(kThreads)
bwd_dq_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
              const float* __restrict__ gate, const float* __restrict__ dout, float* __restrict__ dq,
              float* __restrict__ qdq, const float* __restrict__ states, const Shape sh) {
  extern __shared__ double smem_d[];
  const int d = sh.d, dv = sh.dv, ld = odd(d), lv = odd(dv), ls = odd(kRows);
  double* c = smem_d;
  float* S = reinterpret_cast<float*>(c + kRows);
  float* Ks = S + d * lv;
  float* Vs = Ks + kRows * ld;
  float* Gs = Vs + kRows * lv;
  float* A = Gs + kRows * lv;
  float *head = A + kRows * ls, *tail = head + kRows, *dots = tail + kRows;
  const int64_t bh = blockIdx.x / sh.C, ch = blockIdx.x % sh.C;
  const int64_t t0 = ch * sh.L, t1 = imin64(sh.N, t0 + sh.L);
  load_state_tile(S, states ? states + static_cast<int64_t>(blockIdx.x) * d * dv : nullptr, d, dv);
  for (int64_t i0 = t0; i0 < t1; i0 += kRows) {
    const int rows = static_cast<int>(imin64(kRows, t1 - i0));
    const int64_t row = bh * sh.N + i0;
    __syncthreads();
    load_rows(Ks, k + row * d, rows, d);
    load_rows(Vs, v + row * dv, rows, dv);
    load_rows(Gs, dout + row * dv, rows, dv);
    if (threadIdx.x < kRows) dots[threadIdx.x] = 0.f;
    gate_tables(gate + row, rows, i0 == 0, c, head, tail);
    tile_product(
        rows, rows, dv, [&](int r, int x) { return Gs[r * lv + x]; }, [&](int x, int j) { return Vs[j * lv + x]; },
        One1{}, 0, Zero2{}, Zero2{},
        [&](int t, int j, float x) {
          A[t * ls + j] = j <= t ? x * pair_weight(c, t, j) : 0.f;
          return 0.f;
        },
        NoRow{});
    __syncthreads();
    const float* qb = q + row * d;
    float* ob = dq + row * d;
    tile_product(
        rows, d, dv, [&](int r, int e) { return Gs[r * lv + e]; }, [&](int e, int x) { return S[x * lv + e]; },
        [&](int r) { return head[r]; }, rows, [&](int r, int j) { return A[r * ls + j]; },
        [&](int j, int x) { return Ks[j * ld + x]; },
        [&](int t, int x, float y) {
          ob[t * d + x] = y;
          return qb[t * d + x] * y;
        },
        [&](int r, float dot, int tc) {
          dot = half_warp_sum(dot);
          if (tc == 0 && r < rows) dots[r] += dot;
        });
    __syncthreads();
    if (threadIdx.x < rows) qdq[row + threadIdx.x] = dots[threadIdx.x];
    update_state(S, Ks, Vs, [&](int j) { return tail[j]; }, d, dv, rows, head[kRows - 1]);
  }
}

// dK, dV and k_j . dk_j, blocks of a chunk last to first.
__global__ void __launch_bounds__(kThreads)
bwd_dkdv_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                const float* __restrict__ gate, const float* __restrict__ dout, float* __restrict__ dk,
                float* __restrict__ dvv, float* __restrict__ kdk, const float* __restrict__ states,
                const Shape sh) {
  extern __shared__ double smem_d[];
  const int d = sh.d, dv = sh.dv, ld = odd(d), lv = odd(dv), ls = odd(kRows);
  double* c = smem_d;
  float* U = reinterpret_cast<float*>(c + kRows);
  float* Qs = U + d * lv;
  float* Ks = Qs + kRows * ld;
  float* Vs = Ks + kRows * ld;
  float* Gs = Vs + kRows * lv;
  float* P = Gs + kRows * lv;
  float *head = P + kRows * ls, *tail = head + kRows, *dots = tail + kRows;
  const int64_t bh = blockIdx.x / sh.C, ch = blockIdx.x % sh.C;
  const int64_t t0 = ch * sh.L, t1 = imin64(sh.N, t0 + sh.L);
  const int nblk = static_cast<int>((t1 - t0 + kRows - 1) / kRows);
  load_state_tile(U, states ? states + static_cast<int64_t>(blockIdx.x) * d * dv : nullptr, d, dv);
  for (int n = nblk - 1; n >= 0; --n) {
    const int64_t i0 = t0 + static_cast<int64_t>(n) * kRows;
    const int rows = static_cast<int>(imin64(kRows, t1 - i0));
    const int64_t row = bh * sh.N + i0;
    __syncthreads();
    load_rows(Qs, q + row * d, rows, d);
    load_rows(Ks, k + row * d, rows, d);
    load_rows(Vs, v + row * dv, rows, dv);
    load_rows(Gs, dout + row * dv, rows, dv);
    if (threadIdx.x < kRows) dots[threadIdx.x] = 0.f;
    gate_tables(gate + row, rows, i0 == 0, c, head, tail);
    // P[t][j] = D (q_t . k_j), then dV; the same tile then holds D (dO_t . v_j) for dK
    tile_product(
        rows, rows, d, [&](int r, int x) { return Qs[r * ld + x]; }, [&](int x, int j) { return Ks[j * ld + x]; },
        One1{}, 0, Zero2{}, Zero2{},
        [&](int t, int j, float x) {
          P[t * ls + j] = j <= t ? x * pair_weight(c, t, j) : 0.f;
          return 0.f;
        },
        NoRow{});
    __syncthreads();
    float* vb = dvv + row * dv;
    tile_product(
        rows, dv, d, [&](int j, int x) { return Ks[j * ld + x]; }, [&](int x, int e) { return U[x * lv + e]; },
        [&](int j) { return tail[j]; }, rows, [&](int j, int t) { return P[t * ls + j]; },
        [&](int t, int e) { return Gs[t * lv + e]; },
        [&](int j, int e, float y) {
          vb[j * dv + e] = y;
          return 0.f;
        },
        NoRow{});
    __syncthreads();
    tile_product(
        rows, rows, dv, [&](int r, int x) { return Gs[r * lv + x]; }, [&](int x, int j) { return Vs[j * lv + x]; },
        One1{}, 0, Zero2{}, Zero2{},
        [&](int t, int j, float x) {
          P[t * ls + j] = j <= t ? x * pair_weight(c, t, j) : 0.f;
          return 0.f;
        },
        NoRow{});
    __syncthreads();
    float* kb = dk + row * d;
    tile_product(
        rows, d, dv, [&](int j, int e) { return Vs[j * lv + e]; }, [&](int e, int x) { return U[x * lv + e]; },
        [&](int j) { return tail[j]; }, rows, [&](int j, int t) { return P[t * ls + j]; },
        [&](int t, int x) { return Qs[t * ld + x]; },
        [&](int j, int x, float y) {
          kb[j * d + x] = y;
          return Ks[j * ld + x] * y;
        },
        [&](int j, float dot, int tc) {
          dot = half_warp_sum(dot);
          if (tc == 0 && j < rows) dots[j] += dot;
        });
    __syncthreads();
    if (threadIdx.x < rows) kdk[row + threadIdx.x] = dots[threadIdx.x];
    update_state(U, Qs, Gs, [&](int t) { return head[t]; }, d, dv, rows, head[kRows - 1]);
  }
}

// ------------------------------------------------ shared with the tensor cores

// In place, per (sequence, element): the chunks' own states become the state
// before each chunk (mode 0) or the decayed sum of the later chunks (mode 1).
// Grid: ceil(nel / 256) blocks a sequence.
__global__ void __launch_bounds__(kThreads)
scan_kernel(float* __restrict__ s, const double* __restrict__ tot, int64_t C, int nel, int mode) {
  pdl_launch_dependents();
  pdl_wait();
  const int nb = (nel + kThreads - 1) / kThreads;
  const int64_t bh = blockIdx.x / nb;
  const int e = static_cast<int>(blockIdx.x % nb) * kThreads + threadIdx.x;
  if (e >= nel) return;
  float* p = s + bh * C * nel + e;
  const double* g = tot + bh * C;
  constexpr int U = 8;  // independent loads in flight
  float run = 0.f;
  for (int64_t i0 = 0; i0 < C; i0 += U) {
    float x[U], f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t ch = mode == 0 ? i0 + u : C - 1 - (i0 + u);
      const bool on = i0 + u < C;
      x[u] = on ? p[ch * nel] : 0.f;
      f[u] = on ? expf(static_cast<float>(g[ch])) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t ch = mode == 0 ? i0 + u : C - 1 - (i0 + u);
      if (i0 + u < C) p[ch * nel] = run;
      run = fmaf(f[u], run, x[u]);
    }
  }
}

// Slot of batch row b, or -1 where nothing is to be done: a negative index (a
// padded row), or an index out of the pool or named by an earlier row already,
// which are errors that la2_check reports (two rows must not update one state).
// Called by every thread of a block; contains a barrier.
__device__ __forceinline__ int64_t checked_slot(const int32_t* __restrict__ slots, int64_t b, int64_t n_slots) {
  if (!slots) return b;
  const int32_t s = slots[b];
  int bad = 0;
  if (s >= 0) {
    for (int64_t i = threadIdx.x; i < b; i += blockDim.x) bad |= slots[i] == s;
    bad |= s >= n_slots;
  }
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) record_error(DEV_ERR_INDEX, 60);
  return bad || s < 0 ? -1 : s;
}

// pool[slot of b][h] <- e^(all gates) pool[slot][h] + the chunks' states decayed to
// the last token, added in chunk order. A chunk's state is `nel_c` floats; ld > 0: in
// the tensor cores' layout of ld rows (float4 j of row r at j*ld + r). Grid: ceil(d*dv / 256) blocks a sequence.
__global__ void __launch_bounds__(kThreads)
pool_update_kernel(const float* __restrict__ chunks, const double* __restrict__ tot, float* __restrict__ pool,
                   const int32_t* __restrict__ slots, int64_t n_slots, int64_t C, int H, int d, int dv,
                   int nel_c, int ld) {
  pdl_launch_dependents();
  pdl_wait();
  const int nel = d * dv, nb = (nel + kThreads - 1) / kThreads;
  const int64_t bh = blockIdx.x / nb, b = bh / H;
  const int64_t slot = checked_slot(slots, b, n_slots);
  const int e = static_cast<int>(blockIdx.x % nb) * kThreads + threadIdx.x;
  if (slot < 0 || e >= nel) return;
  const int r = e / dv, c = e % dv;
  const float* p = chunks + bh * C * nel_c + (ld ? ((c >> 2) * ld + r) * 4 + (c & 3) : e);
  float* out = pool + (slot * H + (bh - b * H)) * nel + e;
  float run = *out;
  for (int64_t ch = 0; ch < C; ++ch)
    run = fmaf(expf(static_cast<float>(tot[bh * C + ch])), run, p[ch * nel_c]);
  *out = run;
}

// dl_t = flow at the chunk's end + sum over the chunk's rows from t on of
// (q . dq - k . dk). The flow at the end of chunk c is <state before chunk c + 1, U
// behind chunk c> (0 for the last chunk); elements in any common order. One CTA a
// (sequence, chunk). `per` = 0: prefix and suffix hold those states, scanned;
// otherwise they hold K pieces' own states, `per` a chunk, and are summed here,
// nearest first, each decayed over the nearer ones (at most kMaxPieces).
constexpr int kGradThreads = 1024;
constexpr int kMaxPieces = 16;
template <typename T>
__global__ void __launch_bounds__(kGradThreads)
gate_grad_kernel(const T* __restrict__ gate, const float* __restrict__ qdq, const float* __restrict__ kdk,
                 const float* __restrict__ prefix, const float* __restrict__ suffix,
                 const double* __restrict__ tot, T* __restrict__ dgate, int64_t N, int64_t L, int64_t C, int nel,
                 int64_t K, int64_t per) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kWarps = kGradThreads / 32;
  __shared__ double part[kWarps];
  __shared__ float weight[2][kMaxPieces];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t bh = blockIdx.x / C, ch = blockIdx.x % C;
  const int64_t t0 = ch * L, t1 = imin64(N, t0 + L);
  double carry = 0.0;
  if (ch + 1 < C) {
    const int64_t edge = (ch + 1) * per;  // first piece behind the chunk
    const int n_pre = per ? static_cast<int>(edge) : 1, n_suf = per ? static_cast<int>(K - edge) : 1;
    const float* a = prefix + (bh * K + (per ? edge - 1 : ch + 1)) * nel;
    const float* b = suffix + (bh * K + (per ? edge : ch)) * nel;
    if (threadIdx.x < 2) {
      float f = 1.f;
      const int n = threadIdx.x ? n_suf : n_pre;
      for (int j = 0; j < n; ++j) {
        weight[threadIdx.x][j] = f;
        if (j + 1 < n) f *= expf(static_cast<float>(tot[bh * K + (threadIdx.x ? edge + j : edge - 1 - j)]));
      }
    }
    __syncthreads();
    double x = 0.0;
    auto term = [&](int i) {
      float u = 0.f, v = 0.f;
      for (int j = 0; j < n_pre; ++j) u = fmaf(weight[0][j], a[i - static_cast<int64_t>(j) * nel], u);
      for (int j = 0; j < n_suf; ++j) v = fmaf(weight[1][j], b[i + static_cast<int64_t>(j) * nel], v);
      x += static_cast<double>(u) * v;
    };
    auto term4 = [&](int i) {
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
#pragma unroll 4
      for (int j = 0; j < n_pre; ++j) {
        const float4 y = *reinterpret_cast<const float4*>(a + i - static_cast<int64_t>(j) * nel);
        const float f = weight[0][j];
        u = make_float4(fmaf(f, y.x, u.x), fmaf(f, y.y, u.y), fmaf(f, y.z, u.z), fmaf(f, y.w, u.w));
      }
#pragma unroll 4
      for (int j = 0; j < n_suf; ++j) {
        const float4 y = *reinterpret_cast<const float4*>(b + i + static_cast<int64_t>(j) * nel);
        const float f = weight[1][j];
        v = make_float4(fmaf(f, y.x, v.x), fmaf(f, y.y, v.y), fmaf(f, y.z, v.z), fmaf(f, y.w, v.w));
      }
      x += (static_cast<double>(u.x) * v.x + static_cast<double>(u.y) * v.y) +
           (static_cast<double>(u.z) * v.z + static_cast<double>(u.w) * v.w);
    };
    if (nel % 4 == 0)
      for (int i = 4 * threadIdx.x; i < nel; i += 4 * kGradThreads) term4(i);
    else
      for (int i = threadIdx.x; i < nel; i += kGradThreads) term(i);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    if (lane == 0) part[w] = x;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) carry += part[i];
    __syncthreads();
  }
  // rows of the chunk from its last; thread x holds row hi - x
  for (int64_t hi = t1 - 1; hi >= t0; hi -= kGradThreads) {
    const int64_t t = hi - threadIdx.x, at = bh * N + t;
    double x = t >= t0 ? static_cast<double>(qdq[at]) - static_cast<double>(kdk[at]) : 0.0;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, x, m);
      if (lane >= m) x += up;
    }
    if (lane == 31) part[w] = x;
    __syncthreads();
    double before = carry;
    for (int i = 0; i < kWarps; ++i) {
      if (i < w) before += part[i];
      carry += part[i];
    }
    if (t >= t0) {
      const float l = to_f32(gate[at]);
      // a gate of 0 passes nothing on, and its own factor is 0; there is nothing
      // before the first token for its gate to pass on
      const bool none = t == 0 || l < static_cast<float>(kLogZero);
      dgate[at] = from_f32<T>(none ? 0.f : static_cast<float>(before + x));
    }
    __syncthreads();
  }
}

}  // namespace gated
}  // namespace la2
