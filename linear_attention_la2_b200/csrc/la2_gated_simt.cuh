// CUDA-core kernels of the gated recurrence in fp32 (bf16 is on the tensor cores, see
// la2_gated_sm100.cuh), and the small fp32
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
// fp32 result may be); a restart counts as kLogZero, whose exponential is 0.
//
// The gate's gradient is the flow of pairs across its token,
//   dl_t = sum_{i >= t > j} D[i][j] (q_i . k_j)(dO_i . v_j),
// and satisfies dl_t = dl_(t+1) + q_t . dq_t - k_t . dk_t. The row dots leave the
// dQ and dK passes in fp32; the flow at a chunk's end is <KV, U> of the two chunk
// states there, so the running difference only spans one chunk. The pairs i = j are in
// both dots and cancel; of a head that forgets within a token the dots hold little else,
// and what is left would be their rounding (12 % of dl at log gates of -12 over 500
// rows). These kernels leave the pairs i = j out of both dots; the tensor cores' do not, and
// where all gates around a token are that low its few pairs are summed instead (see
// sum_near_pairs).
//
// The workload is short sequences in fp32: what counts is how many blocks run at once
// and how long one takes. A chunk may be a single block; a call's independent parts
// (both states, both gradients) share a launch.
#pragma once

#include <algorithm>

#include "la2_common.cuh"

namespace la2 {
namespace gated {

constexpr int kThreads = 256;
constexpr int kRows = 64;
// A log gate below this is 0 (a restart), as its exponential in fp32 is. In the fp64 sums
// such a gate counts as kLogZero, which no gates above 0 outweigh in fp32 ones.
constexpr float kRestart = -104.f;
constexpr double kLogZero = -1.0e4;

// A log gate as the sums take it. A comparison, not fmax: NaN stays NaN.
__device__ __forceinline__ double gate_log(float x) {
  return x < kRestart ? kLogZero : static_cast<double>(x);
}
__host__ __device__ __forceinline__ int round4(int w) { return (w + 3) & ~3; }
// Row stride of a tile of w columns: whole float4s, an odd number of them, so that a
// float4 of eight neighbouring rows comes from eight different groups of banks.
__host__ __device__ __forceinline__ int stride_of(int w) { return ((w + 3) / 4 | 1) * 4; }

// Products of 64 x 64 outputs: threads are 16 x 16 and own rows 4 tr + i and columns
// 4 tc + j (WIDE) or tc + 16 j. An operand's values lie along k within a row of its
// tile (AK, BK: read as float4 of four k) or across rows (read as float4 of four
// rows, columns; of columns tc + 16 j one by one). Four steps of k take 8 (or 20)
// reads for 64 multiply-adds a thread; with one word a read (8 for 16) the forward
// kernel took 222 us instead of 130 (B2 H8 N2K, 128 wide).
__device__ __forceinline__ int tile_col() { return threadIdx.x & 15; }
__device__ __forceinline__ int tile_row() { return 4 * (threadIdx.x >> 4); }

// acc += sum over k < K (a multiple of 4) of [w_k] a(r0 + i, k) b(k, cc[j]) (WIDE: cc[0] + j)
template <bool AK, bool BK, bool WIDE, bool WEIGHT>
__device__ __forceinline__ void accumulate(float (&acc)[4][4], const float* a, int la, int r0, const float* b, int lb,
                                           const int (&cc)[4], int K, const float* w) {
#pragma unroll 2
  for (int k = 0; k < K; k += 4) {
    float x[4][4], y[4][4];  // [k][row], [k][column]
    if constexpr (AK) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(a + (r0 + i) * la + k);
        x[0][i] = v.x; x[1][i] = v.y; x[2][i] = v.z; x[3][i] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 v = *reinterpret_cast<const float4*>(a + (k + e) * la + r0);
        x[e][0] = v.x; x[e][1] = v.y; x[e][2] = v.z; x[e][3] = v.w;
      }
    }
    if constexpr (BK) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(b + cc[j] * lb + k);
        y[0][j] = v.x; y[1][j] = v.y; y[2][j] = v.z; y[3][j] = v.w;
      }
    } else if constexpr (WIDE) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 v = *reinterpret_cast<const float4*>(b + (k + e) * lb + cc[0]);
        y[e][0] = v.x; y[e][1] = v.y; y[e][2] = v.z; y[e][3] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int j = 0; j < 4; ++j) y[e][j] = b[(k + e) * lb + cc[j]];
    }
    if constexpr (WEIGHT) {
      const float4 v = *reinterpret_cast<const float4*>(w + k);
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[e][i] *= f[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[e][i], y[e][j], acc[i][j]);
  }
}
__device__ __forceinline__ void clear(float (&acc)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
}
__device__ __forceinline__ void scale_rows(float (&acc)[4][4], const float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = f[tile_row() + i];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] *= x;
  }
}
// Columns c0 + tc + 16 j, the last one standing in for those behind it.
__device__ __forceinline__ void spread_columns(int (&cc)[4], int c0, int n) {
#pragma unroll
  for (int j = 0; j < 4; ++j) cc[j] = min(c0 + tile_col() + 16 * j, n - 1);
}

// Sum of `x` over the 16 lanes of a half warp.
__device__ __forceinline__ float half_warp_sum(float x) {
#pragma unroll
  for (int m = 8; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// Starts the copies of rows [0, rows) of a [*, w] tensor into a tile; the rest of its
// 64 rows and round4(w) columns become zeros. copies_done() and a barrier end them.
template <int BYTES>
__device__ __forceinline__ void copy_or_zero(float* dst, const float* src, bool on) {
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(on ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void load_rows(float* dst, const float* __restrict__ src, int rows, int w) {
  const int ld = stride_of(w);
  if (w % 4 == 0) {
#pragma unroll
    for (int u = 0; u < kRows / 16; ++u) {
      const int r = (threadIdx.x >> 4) + 16 * u;
      for (int c = 4 * (threadIdx.x & 15); c < w; c += 64)
        copy_or_zero<16>(dst + r * ld + c, r < rows ? src + r * w + c : src, r < rows);
    }
  } else {
#pragma unroll
    for (int u = 0; u < kRows / 16; ++u) {
      const int r = (threadIdx.x >> 4) + 16 * u;
      for (int c = threadIdx.x & 15; c < round4(w); c += 16) {
        const bool on = r < rows && c < w;
        copy_or_zero<4>(dst + r * ld + c, on ? src + r * w + c : src, on);
      }
    }
  }
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The block's gate sums: c[t] for t < kRows (rows behind the last one repeat it)
// and the weights e^(c_t) and e^(c_R - c_t). `start`: the block opens its sequence,
// where nothing comes before the first token for its gate to pass on (0, unless NaN).
// Waits for the thread's copies; ends with a barrier.
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
  copies_done();
  __syncthreads();
}

// P[t][j] = e^(c_t - c_j) (a_t . b_j) for j <= t, else 0, over all 64 rows. With `diag`
// the products a_t . b_t go there and P has zeros in their place.
__device__ __forceinline__ void scores(float* P, const float* a, const float* b, int ld, int K, const double* c,
                                       float* diag) {
  float acc[4][4];
  int cc[4];
  clear(acc);
  spread_columns(cc, 0, kRows);
  accumulate<true, true, false, false>(acc, a, ld, tile_row(), b, ld, cc, K, nullptr);
  const int lp = stride_of(kRows);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = tile_row() + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool own = diag && cc[j] == t;
      P[t * lp + cc[j]] = cc[j] <= t && !own ? acc[i][j] * expf(static_cast<float>(c[t] - c[cc[j]])) : 0.f;
      if (own) diag[t] = acc[i][j];
    }
  }
}

// Four values of a row from column c on, w columns wide.
__device__ __forceinline__ void store4(float* row, int c, int w, const float (&x)[4]) {
  if (w % 4 == 0) {
    *reinterpret_cast<float4*>(row + c) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < w) row[c + j] = x[j];
  }
}

// S (d rows) <- e^(c_R) S + sum over K rows of w_t a_t^T b_t (`fresh`: S was 0), into
// S or, as dense rows of dv, into `out`.
__device__ __forceinline__ void update_state(float* S, const float* a, const float* b, const float* w, int d, int dv,
                                             int K, float whole, bool fresh, float* out) {
  const int la = stride_of(d), lb = stride_of(dv);
  for (int c0 = 0; c0 < dv; c0 += 64)
    for (int r0 = 0; r0 < d; r0 += 64) {
      const int c = c0 + 4 * tile_col(), r = r0 + tile_row();
      const int cc[4] = {min(c, round4(dv) - 4), 0, 0, 0};
      float acc[4][4];
      clear(acc);
      accumulate<false, false, true, true>(acc, a, la, min(r, round4(d) - 4), b, lb, cc, K, w);
      if (c < dv)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (r + i >= d) break;
          float4* s = reinterpret_cast<float4*>(S + (r + i) * lb + c);
          if (!fresh) {
            float4 x = *s;
            if (whole == 0.f) x = make_float4(0.f, 0.f, 0.f, 0.f);  // (a restart drops it, be it no number)
            acc[i][0] = fmaf(whole, x.x, acc[i][0]);
            acc[i][1] = fmaf(whole, x.y, acc[i][1]);
            acc[i][2] = fmaf(whole, x.z, acc[i][2]);
            acc[i][3] = fmaf(whole, x.w, acc[i][3]);
          }
          if (out)
            store4(out + (r + i) * dv, c, dv, acc[i]);
          else
            *s = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        }
    }
}

struct Shape {
  int64_t N, L, C;
  int d, dv;
  int pieces;  // 1: the chunks add up the others' own states; 0: a scan has done it
};

// The state that chunk ch of a sequence starts from, in rows of stride_of(dv), zeros
// around it: the scanned one, or the own states of the chunks before it (BACK: behind
// it), nearest first, each decayed over the nearer ones. With `sum`, it also goes there
// ([BH][C][d*dv], for the gates' gradient).
template <bool BACK>
__device__ __forceinline__ void load_state(float* S, const float* __restrict__ states, const double* __restrict__ tot,
                                           int64_t bh, int64_t ch, const Shape& sh, float* sum) {
  const int ld = stride_of(sh.dv), w = ld / 4, nel = sh.d * sh.dv;
  const int n = !states ? 0 : sh.pieces ? static_cast<int>(BACK ? sh.C - 1 - ch : ch) : 1;
  const int64_t first = bh * sh.C + (sh.pieces ? (BACK ? ch + 1 : ch - 1) : ch);
  const int step = BACK ? 1 : -1;
  for (int i = threadIdx.x; i < round4(sh.d) * w; i += kThreads) {
    const int r = i / w, c = 4 * (i - r * w);
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (r < sh.d && c < sh.dv) {
      float f = 1.f;
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const float* src = states + (first + j * step) * nel + r * sh.dv + c;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (sh.dv % 4 == 0) {
          const float4 u = *reinterpret_cast<const float4*>(src);
          v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < sh.dv) v[e] = src[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = f == 0.f ? x[e] : fmaf(f, v[e], x[e]);  // (dropped, be it no number)
        if (j + 1 < n) f *= expf(static_cast<float>(tot[first + j * step]));
      }
    }
    if (sum && r < sh.d && c < sh.dv) store4(sum + (bh * sh.C + ch) * nel + r * sh.dv, c, sh.dv, x);
    *reinterpret_cast<float4*>(S + r * ld + c) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

// Bytes of shared memory: a state, `a` tiles of d and `b` of dv columns, `s` score tiles with
// their diagonals, the tables.
__host__ __device__ __forceinline__ size_t smem_bytes(int d, int dv, int a, int b, int s) {
  return kRows * sizeof(double) +
         sizeof(float) * ((size_t)round4(d) * stride_of(dv) + (size_t)kRows * (a * stride_of(d) + b * stride_of(dv)) +
                          (size_t)s * kRows * (stride_of(kRows) + 1) + 2 * kRows);
}

// Own state of every chunk: prefix (blockIdx.y 0, of k and v), sum_s e^(rest of the
// chunk's gates) a_s^T b_s, the state after the chunk; suffix (blockIdx.y 1, of q and
// dO), sum_t e^(the chunk's gates up to t) a_t^T b_t, decayed back to the row before
// the chunk. tot: the chunk's sum of gates. `all` false: not the last chunk's prefix
// nor the first one's suffix, which nothing starts from.
struct StateArgs {
  const float *a[2], *b[2], *gate;
  float* out[2];
  double* tot;
  int all;
};
__global__ void __launch_bounds__(kThreads, 2)
chunk_state_kernel(const StateArgs p, const Shape sh) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ double smem_d[];
  const int d = sh.d, dv = sh.dv;
  double* c = smem_d;
  float *head = reinterpret_cast<float*>(c + kRows), *tail = head + kRows;
  float* S = tail + kRows;
  float* As = S + round4(d) * stride_of(dv);
  float* Bs = As + kRows * stride_of(d);
  const bool suffix = blockIdx.y;
  const int64_t bh = blockIdx.x / sh.C, ch = blockIdx.x % sh.C;
  const int64_t t0 = ch * sh.L, t1 = imin64(sh.N, t0 + sh.L);
  const int nblk = static_cast<int>((t1 - t0 + kRows - 1) / kRows);
  if (!p.all && (suffix ? ch == 0 : ch + 1 == sh.C)) return;
  double sum = 0.0;
  for (int n = 0; n < nblk; ++n) {
    const int64_t i0 = t0 + static_cast<int64_t>(suffix ? nblk - 1 - n : n) * kRows;
    const int rows = static_cast<int>(imin64(kRows, t1 - i0));
    __syncthreads();
    load_rows(As, p.a[suffix] + (bh * sh.N + i0) * d, rows, d);
    load_rows(Bs, p.b[suffix] + (bh * sh.N + i0) * dv, rows, dv);
    gate_tables(p.gate + bh * sh.N + i0, rows, false, c, head, tail);
    sum += c[kRows - 1];
    update_state(S, As, Bs, suffix ? head : tail, d, dv, round4(rows), head[kRows - 1], n == 0,
                 n + 1 < nblk ? nullptr : p.out[suffix] + static_cast<int64_t>(blockIdx.x) * d * dv);
  }
  // (of both launches' chunks each sum is written once: its blocks add up in another order)
  if (threadIdx.x == 0 && (!suffix || ch + 1 == sh.C)) p.tot[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads, 2)
fwd_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
           const float* __restrict__ gate, float* __restrict__ o, const float* __restrict__ states,
           const double* __restrict__ tot, const Shape sh) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ double smem_d[];
  const int d = sh.d, dv = sh.dv, ld = stride_of(d), lv = stride_of(dv), lp = stride_of(kRows);
  double* c = smem_d;
  float *head = reinterpret_cast<float*>(c + kRows), *tail = head + kRows;
  float* S = tail + kRows;
  float* Qs = S + round4(d) * lv;
  float* Ks = Qs + kRows * ld;
  float* Vs = Ks + kRows * ld;
  float* P = Vs + kRows * lv;
  const int64_t bh = blockIdx.x / sh.C, ch = blockIdx.x % sh.C;
  const int64_t t0 = ch * sh.L, t1 = imin64(sh.N, t0 + sh.L);
  for (int64_t i0 = t0; i0 < t1; i0 += kRows) {
    const int rows = static_cast<int>(imin64(kRows, t1 - i0));
    const int64_t row = bh * sh.N + i0;
    __syncthreads();
    load_rows(Qs, q + row * d, rows, d);
    load_rows(Ks, k + row * d, rows, d);
    load_rows(Vs, v + row * dv, rows, dv);
    if (i0 == t0) load_state<false>(S, states, tot, bh, ch, sh, nullptr);
    gate_tables(gate + row, rows, i0 == 0, c, head, tail);
    scores(P, Qs, Ks, ld, round4(d), c, nullptr);
    __syncthreads();
    for (int c0 = 0; c0 < dv; c0 += 64) {
      const int col = c0 + 4 * tile_col(), cc[4] = {min(col, round4(dv) - 4), 0, 0, 0};
      float acc[4][4];
      clear(acc);
      accumulate<true, false, true, false>(acc, Qs, ld, tile_row(), S, lv, cc, round4(d), nullptr);
      scale_rows(acc, head);
      accumulate<true, false, true, false>(acc, P, lp, tile_row(), Vs, lv, cc, round4(rows), nullptr);
      if (col < dv)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (tile_row() + i < rows) store4(o + (row + tile_row() + i) * dv, col, dv, acc[i]);
    }
    if (i0 + kRows < t1) {  // (the state past the chunk's last block is not needed)
      __syncthreads();
      update_state(S, Ks, Vs, tail, d, dv, round4(rows), head[kRows - 1], false, nullptr);
    }
  }
}

struct BwdArgs {
  const float *q, *k, *v, *gate, *dout;
  float *dq, *dk, *dv;
  float *qdq, *kdk;                // the rows' dots
  const float *prefix, *suffix;    // chunk states, or null
  float *prefix_sum, *suffix_sum;  // where the chunks' starts go, or null
  const double* tot;
};
// Rows' values 4 tr + i of columns cc[j] out, and their dots with `x` (row stride lx)
// added to dot. The pairs of a token with itself, diag_t z_t, are in the values and not
// in the dots: they cancel between the two passes, and beside the pairs that a head
// which forgets within a token keeps, their rounding would be all that was left.
__device__ __forceinline__ void store_spread(float* out, int w, const float* x, int lx, const float (&acc)[4][4], int c0,
                                             int rows, const float* diag, const float* z, float (&dot)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = tile_row() + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + tile_col() + 16 * j;
      if (t < rows && c < w) {
        out[t * w + c] = fmaf(diag[t], z[t * lx + c], acc[i][j]);
        dot[i] = fmaf(x[t * lx + c], acc[i][j], dot[i]);
      }
    }
  }
}
__device__ __forceinline__ void store_dots(float* out, float (&dot)[4], int rows) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = half_warp_sum(dot[i]);
    if (tile_col() == 0 && tile_row() + i < rows) out[tile_row() + i] = x;
  }
}

// dQ_t = sum_{j<=t} e^(c_t - c_j) (dO_t . v_j) k_j + e^(c_t) dO_t KV^T, and q_t . dq_t of j < t.
__device__ __forceinline__ void bwd_dq(const BwdArgs& p, const Shape& sh, double* smem_d) {
  const int d = sh.d, dv = sh.dv, ld = stride_of(d), lv = stride_of(dv), lp = stride_of(kRows);
  double* c = smem_d;
  float *head = reinterpret_cast<float*>(c + kRows), *tail = head + kRows;
  float* S = tail + kRows;
  float* Ks = S + round4(d) * lv;
  float* Vs = Ks + kRows * ld;
  float* Gs = Vs + kRows * lv;
  float* Qs = Gs + kRows * lv;
  float* A = Qs + kRows * ld;
  float* diag = A + kRows * lp;
  const int64_t bh = blockIdx.x / sh.C, ch = blockIdx.x % sh.C;
  const int64_t t0 = ch * sh.L, t1 = imin64(sh.N, t0 + sh.L);
  for (int64_t i0 = t0; i0 < t1; i0 += kRows) {
    const int rows = static_cast<int>(imin64(kRows, t1 - i0));
    const int64_t row = bh * sh.N + i0;
    __syncthreads();
    load_rows(Gs, p.dout + row * dv, rows, dv);
    load_rows(Vs, p.v + row * dv, rows, dv);
    load_rows(Ks, p.k + row * d, rows, d);
    load_rows(Qs, p.q + row * d, rows, d);
    if (i0 == t0) load_state<false>(S, p.prefix, p.tot, bh, ch, sh, p.prefix_sum);
    gate_tables(p.gate + row, rows, i0 == 0, c, head, tail);
    scores(A, Gs, Vs, lv, round4(dv), c, diag);
    __syncthreads();
    float dot[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < d; c0 += 64) {
      float acc[4][4];
      int cc[4];
      clear(acc);
      spread_columns(cc, c0, d);
      accumulate<true, true, false, false>(acc, Gs, lv, tile_row(), S, lv, cc, round4(dv), nullptr);
      scale_rows(acc, head);
      accumulate<true, false, false, false>(acc, A, lp, tile_row(), Ks, ld, cc, round4(rows), nullptr);
      store_spread(p.dq + row * d, d, Qs, ld, acc, c0, rows, diag, Ks, dot);
    }
    store_dots(p.qdq + row, dot, rows);
    if (i0 + kRows < t1) {
      __syncthreads();
      update_state(S, Ks, Vs, tail, d, dv, round4(rows), head[kRows - 1], false, nullptr);
    }
  }
}

// dK, dV and k_j . dk_j of t > j, blocks of a chunk last to first.
__device__ __forceinline__ void bwd_dkdv(const BwdArgs& p, const Shape& sh, double* smem_d) {
  const int d = sh.d, dv = sh.dv, ld = stride_of(d), lv = stride_of(dv), lp = stride_of(kRows);
  double* c = smem_d;
  float *head = reinterpret_cast<float*>(c + kRows), *tail = head + kRows;
  float* U = tail + kRows;
  float* Qs = U + round4(d) * lv;
  float* Ks = Qs + kRows * ld;
  float* Vs = Ks + kRows * ld;
  float* Gs = Vs + kRows * lv;
  float* P = Gs + kRows * lv;
  float* diag = P + kRows * lp;
  const int64_t bh = blockIdx.x / sh.C, ch = blockIdx.x % sh.C;
  const int64_t t0 = ch * sh.L, t1 = imin64(sh.N, t0 + sh.L);
  const int nblk = static_cast<int>((t1 - t0 + kRows - 1) / kRows);
  for (int n = nblk - 1; n >= 0; --n) {
    const int64_t i0 = t0 + static_cast<int64_t>(n) * kRows;
    const int rows = static_cast<int>(imin64(kRows, t1 - i0));
    const int64_t row = bh * sh.N + i0;
    __syncthreads();
    load_rows(Qs, p.q + row * d, rows, d);
    load_rows(Ks, p.k + row * d, rows, d);
    load_rows(Gs, p.dout + row * dv, rows, dv);
    load_rows(Vs, p.v + row * dv, rows, dv);
    if (n == nblk - 1) load_state<true>(U, p.suffix, p.tot, bh, ch, sh, p.suffix_sum);
    gate_tables(p.gate + row, rows, i0 == 0, c, head, tail);
    // P[t][j] = D (q_t . k_j), then dV; the same tile then holds D (dO_t . v_j) for dK
    scores(P, Qs, Ks, ld, round4(d), c, nullptr);
    __syncthreads();
    for (int c0 = 0; c0 < dv; c0 += 64) {
      const int col = c0 + 4 * tile_col(), cc[4] = {min(col, round4(dv) - 4), 0, 0, 0};
      float acc[4][4];
      clear(acc);
      accumulate<true, false, true, false>(acc, Ks, ld, tile_row(), U, lv, cc, round4(d), nullptr);
      scale_rows(acc, tail);
      accumulate<false, false, true, false>(acc, P, lp, tile_row(), Gs, lv, cc, round4(rows), nullptr);
      if (col < dv)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (tile_row() + i < rows) store4(p.dv + (row + tile_row() + i) * dv, col, dv, acc[i]);
    }
    __syncthreads();
    scores(P, Gs, Vs, lv, round4(dv), c, diag);
    __syncthreads();
    float dot[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < d; c0 += 64) {
      float acc[4][4];
      int cc[4];
      clear(acc);
      spread_columns(cc, c0, d);
      accumulate<true, true, false, false>(acc, Vs, lv, tile_row(), U, lv, cc, round4(dv), nullptr);
      scale_rows(acc, tail);
      accumulate<false, false, false, false>(acc, P, lp, tile_row(), Qs, ld, cc, round4(rows), nullptr);
      store_spread(p.dk + row * d, d, Ks, ld, acc, c0, rows, diag, Qs, dot);
    }
    store_dots(p.kdk + row, dot, rows);
    if (n > 0) {
      __syncthreads();
      update_state(U, Qs, Gs, head, d, dv, round4(rows), head[kRows - 1], false, nullptr);
    }
  }
}

// Both gradients in one launch, the longer one's CTAs first: neither reads the other's.
__global__ void __launch_bounds__(kThreads, 2)
bwd_kernel(const BwdArgs p, const Shape sh) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ double smem_d[];
  if (blockIdx.y == 0)
    bwd_dkdv(p, sh, smem_d);
  else
    bwd_dq(p, sh, smem_d);
}

// ------------------------------------------------ shared with the tensor cores

// In place, per (sequence, element): the chunks' own states become the state
// before each chunk (mode 0) or the decayed sum of the later chunks (mode 1).
// Grid: ceil(nel / 256) blocks a sequence; blockIdx.y 1 scans s1 in mode 1.
__global__ void __launch_bounds__(kThreads)
scan_kernel(float* __restrict__ s0, float* __restrict__ s1, const double* __restrict__ tot, int64_t C, int nel,
            int mode0) {
  float* s = blockIdx.y ? s1 : s0;
  const int mode = blockIdx.y ? 1 : mode0;
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
      run = f[u] == 0.f ? x[u] : fmaf(f[u], run, x[u]);  // (a restart drops what may be no number)
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
// the tensor cores' layout of ld rows (float4 j of row r at j*ld + r). V values a
// thread, dv a multiple of V; in that layout a warp takes 4 rows x 8 float4s, so that
// both sides move in whole sectors. Grid: ceil(d*dv / (256 V)) blocks a sequence.
template <int V>
__global__ void __launch_bounds__(kThreads)
pool_update_kernel(const float* __restrict__ chunks, const double* __restrict__ tot, float* __restrict__ pool,
                   const int32_t* __restrict__ slots, int64_t n_slots, int64_t C, int H, int d, int dv,
                   int nel_c, int ld) {
  pdl_launch_dependents();
  pdl_wait();
  const int nel = d * dv, nb = (nel + kThreads * V - 1) / (kThreads * V);
  const int64_t bh = blockIdx.x / nb, b = bh / H;
  const int64_t slot = checked_slot(slots, b, n_slots);
  const int i = static_cast<int>(blockIdx.x % nb) * kThreads + threadIdx.x;
  if (slot < 0 || i * V >= nel) return;
  int to = i * V, from = to;
  if (V == 4 && ld) {
    const int tiles = dv / 32, t = i >> 5, r = t / tiles * 4 + (i & 3), j = t % tiles * 8 + ((i & 31) >> 2);
    to = r * dv + 4 * j;
    from = (j * ld + r) * 4;
  }
  const float* p = chunks + bh * C * nel_c + from;
  float* out = pool + (slot * H + (bh - b * H)) * nel + to;
  float run[V];
  auto get = [](const float* src, float (&x)[V]) {
    if constexpr (V == 4) {
      const float4 y = *reinterpret_cast<const float4*>(src);
      x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
    } else {
      x[0] = *src;
    }
  };
  get(out, run);
#pragma unroll 4
  for (int64_t ch = 0; ch < C; ++ch) {
    float x[V];
    get(p + ch * nel_c, x);
    const float f = expf(static_cast<float>(tot[bh * C + ch]));
#pragma unroll
    for (int e = 0; e < V; ++e)  // (a restart drops what was there, be it no number)
      run[e] = f == 0.f ? x[e] : fmaf(f, run[e], x[e]);
  }
  if constexpr (V == 4)
    *reinterpret_cast<float4*>(out) = make_float4(run[0], run[1], run[2], run[3]);
  else
    *out = run[0];
}

// Sum of x over the lanes up to this one, from the last that is cut on; cut: whether one is.
__device__ __forceinline__ void sum_up_to_cut(double& x, bool& cut, int lane) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const double up = __shfl_up_sync(0xffffffffu, x, m);
    const bool up_cut = __shfl_up_sync(0xffffffffu, cut, m);
    if (lane >= m && !cut) {
      x += up;
      cut = up_cut;
    }
  }
}

// Where the gates of a bf16 sequence are below this for kNear tokens on both sides of a
// token, the gate's gradient is summed over pairs at most kNear tokens apart: the
// others carry e^-20 of its factor. Above it the running difference loses less
// than e^5 2^-24 = 9e-6 of the pairs a row, at random signs.
constexpr float kForgets = -5.f;
constexpr int kNear = 4;

// dl_t of the lanes that want it, lane l the row top - l of its sequence: the sum over
// i >= t > j, i - j <= kNear of e^(l_(j+1) + ... + l_i) (q_i . k_j)(dO_i . v_j). A warp walks
// the rows i with the last kNear rows of k and v in registers, each lane two or four
// columns; the eight dots of a row meet in nine shuffles, and each lane takes the
// distances that reach across its t. With d and dv from 64 to 128 in steps of 64. Out
// of line: it is rarely run and would cost the scan registers. (Gradients of B2 H32 N8K:
// 490 us with no such token, 759 us with all gates at -8; with the rows read anew for every
// distance 1163 us.)
struct NearRow {
  uint32_t x[2];  // columns 2 lane, + 1 and 64 + 2 lane, + 1
  __device__ __forceinline__ void load(const __nv_bfloat16* base, int64_t row, int w, int lane) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(base + row * w) + lane;
    x[0] = row >= 0 ? p[0] : 0u;
    x[1] = row >= 0 && w == 128 ? p[32] : 0u;
  }
  __device__ __forceinline__ float dot(const NearRow& o) const {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(o.x[e] << 16), s);
      s = fmaf(__uint_as_float(x[e] & 0xffff0000u), __uint_as_float(o.x[e] & 0xffff0000u), s);
    }
    return s;
  }
};
__device__ __noinline__ float sum_near_pairs(const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                                             const __nv_bfloat16* dout, const __nv_bfloat16* gate, int64_t N, int d,
                                             int dv, int64_t top, unsigned wanted, int lane) {
  const int64_t t = top - lane, first = top - (31 - __clz(wanted));
  const int64_t last = imin64(N - 1, top - (__ffs(wanted) - 1) + kNear - 1);
  const int apart = (lane >> 2 & 3) + 1;  // the distance whose pair this lane ends up with
  NearRow kr[kNear], vr[kNear];           // rows i - 1, i - 2, ...
  float gr[kNear];                        // gates i, i - 1, ...
#pragma unroll
  for (int a = 0; a < kNear; ++a) {
    kr[a].load(k, first - 1 - a, d, lane);
    vr[a].load(v, first - 1 - a, dv, lane);
    gr[a] = first - 1 - a >= 0 ? to_f32(gate[first - 1 - a]) : 0.f;  // (gate i is put in front)
  }
  float sum = 0.f;
  q += first * d;
  k += first * d;
  v += first * dv;
  dout += first * dv;
  NearRow qi, oi, ki, vi;
  float gi;
  auto fetch = [&](int64_t i) {
    qi.load(q, 0, d, lane);
    oi.load(dout, 0, dv, lane);
    ki.load(k, 0, d, lane);
    vi.load(v, 0, dv, lane);
    gi = to_f32(gate[i]);
    q += d;
    k += d;
    v += dv;
    dout += dv;
  };
  fetch(first);
#pragma unroll 4
  for (int64_t i = first; i <= last; ++i) {
    float s[8];
#pragma unroll
    for (int a = 0; a < kNear; ++a) {
      s[a] = qi.dot(kr[a]);
      s[4 + a] = oi.dot(vr[a]);
    }
#pragma unroll
    for (int a = kNear - 1; a > 0; --a) {
      kr[a] = kr[a - 1];
      vr[a] = vr[a - 1];
      gr[a] = gr[a - 1];
    }
    kr[0] = ki;
    vr[0] = vi;
    gr[0] = gi;
    if (i < last) fetch(i + 1);
#pragma unroll
    for (int step = 0; step < 3; ++step) {  // each lane keeps half: lanes from 16 on the dots of dO and v
      const int keep = 4 >> step, bit = 16 >> step;
      const bool up = lane & bit;
#pragma unroll
      for (int e = 0; e < keep; ++e) {
        const float mine = up ? s[e + keep] : s[e], other = up ? s[e] : s[e + keep];
        s[e] = mine + __shfl_xor_sync(0xffffffffu, other, bit);
      }
    }
    float x = s[0];
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x *= __shfl_xor_sync(0xffffffffu, x, 16);
    const float l = gr[0] + (apart > 1 ? gr[1] : 0.f) + (apart > 2 ? gr[2] : 0.f) + (apart > 3 ? gr[3] : 0.f);
    x = i >= apart ? x * expf(l) : 0.f;
    const int64_t behind = i - t;
#pragma unroll
    for (int a = 0; a < kNear; ++a) {
      const float pair = __shfl_sync(0xffffffffu, x, 4 * a);
      if (behind >= 0 && behind <= a) sum += pair;
    }
  }
  return sum;
}

// dl_t = flow at the chunk's end + sum over the chunk's rows from t on of
// (q . dq - k . dk), and 0 at a restart, from which the sum starts anew. The flow at
// the end of chunk c is <state before chunk c + 1, U behind chunk c> (0 for the last
// chunk): the starts of the dQ and dK passes' chunks,
// which those passes (or a scan) left there; elements in any common order. One CTA a
// (sequence, chunk). (Adding those states up from the chunks' pieces here, up to 12 of
// 64 KB a CTA, took 31 us at B2 H32 N8K.)
constexpr int kGradThreads = 1024;
template <typename T>
__global__ void __launch_bounds__(kGradThreads)
gate_grad_kernel(const T* __restrict__ gate, const float* __restrict__ qdq, const float* __restrict__ kdk,
                 const float* __restrict__ prefix, const float* __restrict__ suffix, T* __restrict__ dgate, int64_t N,
                 int64_t L, int64_t C, int nel, const T* __restrict__ q, const T* __restrict__ k,
                 const T* __restrict__ v, const T* __restrict__ dout, int d, int dv) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kWarps = kGradThreads / 32;
  __shared__ double part[kWarps];
  __shared__ int part_cut[kWarps];
  static_assert(kWarps == 32, "a flag a lane");
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t bh = blockIdx.x / C, ch = blockIdx.x % C;
  const int64_t t0 = ch * L, t1 = imin64(N, t0 + L);
  double carry = 0.0;
  if (ch + 1 < C) {
    const float* a = prefix + (bh * C + ch + 1) * nel;
    const float* b = suffix + (bh * C + ch) * nel;
    double x = 0.0;
    if (nel % 4 == 0) {
#pragma unroll 4
      for (int i = 4 * threadIdx.x; i < nel; i += 4 * kGradThreads) {
        const float4 u = *reinterpret_cast<const float4*>(a + i), v = *reinterpret_cast<const float4*>(b + i);
        x += (static_cast<double>(u.x) * v.x + static_cast<double>(u.y) * v.y) +
             (static_cast<double>(u.z) * v.z + static_cast<double>(u.w) * v.w);
      }
    } else {
      for (int i = threadIdx.x; i < nel; i += kGradThreads) x += static_cast<double>(a[i]) * b[i];
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    if (lane == 0) part[w] = x;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) carry += part[i];
    __syncthreads();
  }
  // rows of the chunk from its last; thread x holds row hi - x. A gate of 0 passes
  // nothing on and its own factor is 0: what has been summed behind it ends there, so
  // the sums of one document do not reach the gates of another. There is nothing
  // before the first token for its gate to pass on.
  for (int64_t hi = t1 - 1; hi >= t0; hi -= kGradThreads) {
    const int64_t t = hi - threadIdx.x, at = bh * N + t;
    const float l = t >= t0 ? to_f32(gate[at]) : 0.f;
    bool cut = t >= t0 && (t == 0 || l < kRestart);
    double x = t >= t0 && !cut ? static_cast<double>(qdq[at]) - static_cast<double>(kdk[at]) : 0.0;
    float near = 0.f;
    bool forgets = false;
    if constexpr (sizeof(T) == 2) {
      forgets = l < kForgets && !cut;
      for (int u = 1; u <= kNear && forgets; ++u)  // (the first token's gate decides nothing)
        forgets = (t - u < 1 || to_f32(gate[at - u]) < kForgets) && (t + u >= N || to_f32(gate[at + u]) < kForgets);
      const unsigned wanted = __ballot_sync(0xffffffffu, forgets);
      if (wanted)
        near = sum_near_pairs(q + bh * N * d, k + bh * N * d, v + bh * N * dv, dout + bh * N * dv, gate + bh * N, N, d,
                              dv, t + lane, wanted, lane);
    }
    sum_up_to_cut(x, cut, lane);
    if (lane == 31) {
      part[w] = x;
      part_cut[w] = cut;
    }
    __syncthreads();
    double sum = part[lane];  // (every warp sums the warps' own up)
    bool any = part_cut[lane];
    sum_up_to_cut(sum, any, lane);
    if (!any) sum += carry;
    const double before = w ? __shfl_sync(0xffffffffu, sum, w - 1) : carry;
    carry = __shfl_sync(0xffffffffu, sum, 31);
    if (t >= t0) dgate[at] = from_f32<T>(forgets ? near : static_cast<float>(cut ? x : before + x));
    __syncthreads();
  }
}

}  // namespace gated
}  // namespace la2
