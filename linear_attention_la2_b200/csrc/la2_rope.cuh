// RMS norm of every query and key head with the position rotation in the same
// pass, and its gradients. Included at the end of la2.cu.
//
// A row x of d values (one token, one head), weight w, position angles a_i:
//
//   r = 1 / sqrt(mean(x^2) + eps),  y = w (r x),
//   (z_i, z_(i+h)) = (y_i cos a_i - y_(i+h) sin a_i, y_i sin a_i + y_(i+h) cos a_i),  i < h = rot / 2,
//   z_i = y_i for i >= rot;  out = scale z.
//
// Pair i turns by a_i = pos[axis(i)][token] base^(-2i/rot): with several axes
// (time, height, width) each takes a run of pairs. Backwards, with g the
// gradient turned back by -a and scaled (the rotation is orthogonal):
//
//   dw = sum over rows of g (r x),   u = w g,   dx = r (u - (r x) mean(u (r x))).
//
// The input rows are slices of the [B, N, heads, d] projections (any batch,
// token and head strides), the output the dense [B, H, N, d] tensors that the
// attention entry points read, so the transposition costs no pass of its own.
//
// Bound by HBM: each row is read once and written once (backwards: two reads).
// A CTA takes a tile of consecutive tokens and their heads. The angles are computed
// once a token: the turns in fp64 (at position 2^20 an fp32 product is 0.06 rad off),
// and only their fraction goes on to fp32. A group of lanes, each with two 16-byte
// pieces of a row that are one another's pairs, keeps one token's cosines and sines in
// registers and walks the heads; its neighbours hold the next tokens, so that the
// tile's rows of a head leave as one piece of the output. Rows arrive by
// asynchronous copies into places of the loading thread's own, several ahead: in
// registers as many would halve the warps.
#pragma once

namespace la2 {
namespace rope {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxD = 256;
constexpr int kMaxAxes = 4;
constexpr int kRowTile = kWarps;  // tokens of a CTA, a warp a row

struct Params {
  const void* x[2];        // queries, keys (backward: the forward's inputs)
  const void* w[2];        // weights, or null for ones
  void* out[2];            // forward: [B,H,N,d]; backward: dx [B,N,H,d]
  const void* dy[2];       // backward: [B,H,N,d]
  float* dw_part;          // backward: [grid][2][d]
  const int32_t* pos;      // [axes][B*N], or null: 0..N-1
  int64_t sb[2], sn[2], sh[2];  // input strides in elements
  int64_t N, tokens;       // tokens = B * N
  int32_t heads[2];
  int32_t d, half, tile, splits, axes;
  float eps, scale[2];
  double turn[kMaxD / 2];  // base^(-2i/rot) / (2 pi)
  uint8_t axis[kMaxD / 2];
};

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int m = G / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// A lane's 16 bytes of a row as packed pairs of fp32 (8 bf16 or 4 fp32 values): the
// rows' arithmetic is two values an instruction, and the shuffles and reads below move
// the row's raw words. One value an instruction made both passes issue-bound (46 and
// 67 us at B4 N2K, 32 heads, against 21 and 31 us of traffic).
using gated::f2;
using gated::fma2;
using gated::mul2;
using gated::unpack;
template <int VEC>
__device__ __forceinline__ void widen(const uint4& u, uint64_t (&x)[VEC / 2]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    if constexpr (VEC == 8)
      x[i] = f2(w[i] << 16, w[i] & 0xffff0000u);
    else
      x[i] = f2(w[2 * i], w[2 * i + 1]);
  }
}
template <int VEC>
__device__ __forceinline__ uint4 narrow(const uint64_t (&x)[VEC / 2]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) {
    if constexpr (VEC == 8)
      w[i] = gated::pack2(x[i]);
    else
      unpack(x[i], w[2 * i], w[2 * i + 1]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int N>
__device__ __forceinline__ float sum_products(const uint64_t (&x)[2][N], const uint64_t (&y)[2][N]) {
  uint64_t s = mul2(x[0][0], y[0][0]);
#pragma unroll
  for (int i = 1; i < 2 * N; ++i) s = fma2(x[i / N][i % N], y[i / N][i % N], s);
  float a, b;
  unpack(s, a, b);
  return a + b;
}
// A lane's pieces of a weight as stored (loaded ahead), and widened times f (f where
// there is no weight).
template <typename T>
__device__ __forceinline__ void fetch_weight(const void* w, const int (&at)[2], uint4 (&raw)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (w && at[i] >= 0) raw[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(w) + at[i]);
  }
}
template <int VEC>
__device__ __forceinline__ void widen_weight(const void* w, const uint4 (&raw)[2], float f, uint64_t (&x)[2][VEC / 2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    widen<VEC>(raw[i], x[i]);
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) x[i][e] = w ? mul2(x[i][e], f2(f, f)) : f2(f, f);
  }
}

// The two pieces (of VEC values) of lane l of a row's group. With half a multiple of VEC
// (STAGE false) the first half / VEC lanes hold the pairs, and the pieces behind the
// rotated ones are halved over the lanes after them; otherwise all pieces are halved
// over the lanes, and the pairs meet in shared memory. A lane may have one or none (-1).
template <int VEC, bool STAGE>
__device__ __forceinline__ void pieces_of(int l, int half, int d, int (&at)[2]) {
  const int n = d / VEC, hl = STAGE ? 0 : half / VEC;
  if (l < hl) {
    at[0] = l * VEC;
    at[1] = (l + hl) * VEC;
  } else {
    const int rest = n - 2 * hl, k = l - hl, first = (rest + 1) / 2;
    at[0] = k < first ? (2 * hl + k) * VEC : -1;
    at[1] = k < first && first + k < rest ? (2 * hl + first + k) * VEC : -1;
  }
}
// Lanes that a row takes.
template <int VEC>
__host__ __device__ __forceinline__ int lanes_of(int half, int d) {
  const int n = d / VEC, hl = half % VEC ? 0 : half / VEC;
  return hl + (n - 2 * hl + 1) / 2;
}

// Frequencies and axes of the pairs, out of the parameters (whose bank serves one
// address at a time) into shared memory. A barrier must follow.
struct Pairs {
  double turn[kMaxD / 2];
  uint8_t axis[kMaxD / 2];
};
__device__ __forceinline__ void load_pairs(const Params& p, Pairs& s) {
  for (int i = threadIdx.x; i < p.half; i += kThreads) {
    s.turn[i] = p.turn[i];
    s.axis[i] = p.axis[i];
  }
}
// A token's positions on every axis.
struct Positions {
  int32_t at[kMaxAxes];
};
__device__ __forceinline__ Positions positions_of(const Params& p, int64_t tok, int64_t n) {
  Positions x;
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a)
    x.at[a] = !p.pos ? static_cast<int32_t>(n) : a < p.axes ? p.pos[a * p.tokens + tok] : 0;
  return x;
}
// (cos, sin) of pair j.
__device__ __forceinline__ float2 angle_of(const Pairs& s, const Positions& at, int j) {
  const int ax = s.axis[j];
  const int32_t n = ax == 0 ? at.at[0] : ax == 1 ? at.at[1] : ax == 2 ? at.at[2] : at.at[3];
  const double a = static_cast<double>(n) * s.turn[j];
  float2 r;
  sincospif(2.f * static_cast<float>(a - rint(a)), &r.y, &r.x);
  return r;
}

// One token's turn of a lane's two pieces: value <- own value + other (its pair's other
// value). STAGE false: the pieces are each other's, own = cos and other = -+ sin.
template <int VEC, bool STAGE>
struct Turn {
  uint64_t own[STAGE ? 2 : 1][VEC / 2], other[STAGE ? 2 : 1][VEC / 2];
};
// sign -1 turns back.
template <int VEC, bool STAGE>
__device__ __forceinline__ void load_turn(Turn<VEC, STAGE>& c, const Pairs& s, const Positions& pos, const int (&at)[2],
                                          int half, float sign) {
#pragma unroll
  for (int i = 0; i < (STAGE ? 2 : 1); ++i)
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      float o[2], t[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int v = at[i] + 2 * e + u;
        o[u] = 1.f;
        t[u] = 0.f;
        if (at[i] >= 0 && v < 2 * half && (STAGE || v < half)) {
          const float2 a = angle_of(s, pos, v < half ? v : v - half);
          o[u] = a.x;
          t[u] = STAGE && v < half ? -sign * a.y : sign * a.y;
        }
      }
      c.own[i][e] = f2(o[0], o[1]);
      c.other[i][e] = f2(t[0], t[1]);
    }
}
// The staging row of a group: 9 words for every 8, so that lanes meet few conflicts.
template <int VEC, bool STAGE>
__device__ __forceinline__ void turn_row(uint64_t (&x)[2][VEC / 2], const Turn<VEC, STAGE>& c, const int (&at)[2],
                                         int half, float* stage) {
  if constexpr (!STAGE) {
    const uint64_t minus = f2(-1.f, -1.f);
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) {
      const uint64_t a = fma2(mul2(x[1][e], minus), c.other[0][e], mul2(x[0][e], c.own[0][e]));
      x[1][e] = fma2(x[0][e], c.other[0][e], mul2(x[1][e], c.own[0][e]));
      x[0][e] = a;
    }
  } else {
    auto word = [](int i) { return i + (i >> 3); };
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (at[i] >= 0)
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e)
          unpack(x[i][e], stage[word(at[i] + 2 * e)], stage[word(at[i] + 2 * e + 1)]);
    __syncwarp();
    auto other = [&](int v) { return stage[word(v < half ? v + half : (v < 2 * half ? v - half : v))]; };
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (at[i] >= 0)
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e)
          x[i][e] = fma2(f2(other(at[i] + 2 * e), other(at[i] + 2 * e + 1)), c.other[i][e], mul2(x[i][e], c.own[i][e]));
  }
}
// Floats of a group's staging row.
__host__ __device__ constexpr int stage_floats(int vec, int g) { return 2 * vec * g + 2 * vec * g / 8; }

// The token and first head of a thread's group: groups run over the tile's tokens,
// then over its share of the heads (`slots` heads at a time).
struct Place {
  int t, slot, slots;
  bool on;          // the token exists
  int64_t b, n, tok;
};
template <int G>
__device__ __forceinline__ Place place_of(const Params& p, int64_t tok0) {
  Place x;
  const int g = threadIdx.x / G;
  x.t = g % p.tile;
  const int own = kThreads / G / p.tile;
  x.slots = own * p.splits;
  x.slot = g / p.tile + own * blockIdx.y;
  x.tok = tok0 + x.t;
  x.on = x.tok < p.tokens;
  if (!x.on) x.tok = tok0;
  x.b = static_cast<uint32_t>(x.tok) / static_cast<uint32_t>(p.N);
  x.n = x.tok - x.b * p.N;
  return x;
}

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
constexpr int kDepth = 4;   // rows a thread has in flight, of two pieces (backwards: 3, of two times two)
constexpr int kDepthBwd = 3;

template <typename T, int VEC, int G, bool STAGE>
__global__ void __launch_bounds__(kThreads, 5)
rope_fwd_vec_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint4 ring_all[];  // [kDepth][2][kThreads]
  __shared__ Pairs pairs;
  __shared__ float stage_all[STAGE ? kThreads / G * stage_floats(VEC, G) : 1];
  load_pairs(p, pairs);
  pdl_launch_dependents();
  pdl_wait();
  const Place at = place_of<G>(p, static_cast<int64_t>(blockIdx.x) * p.tile);
  const int half = p.half;
  int pc[2];
  pieces_of<VEC, STAGE>(threadIdx.x % G, half, p.d, pc);
  const float inv_d = 1.f / static_cast<float>(p.d), eps = p.eps;
  float* stage = stage_all + (STAGE ? threadIdx.x / G * stage_floats(VEC, G) : 0);
  // rows k of the thread: its share of the queries' heads, then of the keys'
  const int nq = (p.heads[0] + at.slots - 1) / at.slots, total = nq + (p.heads[1] + at.slots - 1) / at.slots;
  uint4* ring = ring_all + threadIdx.x;
  // what is fetched next: the row's place, its head, and the step to the next
  const T* src = nullptr;
  int64_t src_step = 0;
  int fetch_k = 0, fetch_h = 0, fetch_heads = 0, fetch_at = 0;
  auto fetch = [&]() {
    if (fetch_k == 0 || fetch_k == nq) {
      const int which = fetch_k >= nq;
      src = static_cast<const T*>(p.x[which]) + at.b * p.sb[which] + at.n * p.sn[which] + at.slot * p.sh[which];
      src_step = at.slots * p.sh[which];
      fetch_h = at.slot;
      fetch_heads = at.on ? p.heads[which] : 0;
    }
    if (fetch_h < fetch_heads) {
      const uint32_t to = sm100::smem_u32(ring + fetch_at * 2 * kThreads);
      if (pc[0] >= 0) copy_async16(to, src + pc[0]);
      if (pc[1] >= 0) copy_async16(to + kThreads * 16, src + pc[1]);
    }
    copy_commit();
    src += src_step;
    fetch_h += at.slots;
    ++fetch_k;
    fetch_at = fetch_at + 1 == kDepth ? 0 : fetch_at + 1;
  };
#pragma unroll 1
  for (int k = 0; k < kDepth - 1; ++k) fetch();
  const Positions pos = positions_of(p, at.tok, at.n);
  uint4 w_raw[2][2];
  fetch_weight<T>(p.w[0], pc, w_raw[0]);
  fetch_weight<T>(p.w[1], pc, w_raw[1]);
  __syncthreads();
  Turn<VEC, STAGE> c;
  load_turn<VEC, STAGE>(c, pairs, pos, pc, half, 1.f);
  uint64_t w[2][VEC / 2];
  T* dst = nullptr;
  int64_t dst_step = 0;
  int h = 0, heads = 0, from = 0;
#pragma unroll 1
  for (int k = 0; k < total; ++k) {  // (the same for all lanes of a warp)
    if (k == 0 || k == nq) {
      const int which = k >= nq;
      widen_weight<VEC>(p.w[which], which ? w_raw[1] : w_raw[0], p.scale[which], w);
      dst = static_cast<T*>(p.out[which]) + ((at.b * p.heads[which] + at.slot) * p.N + at.n) * p.d;
      dst_step = at.slots * p.N * p.d;
      h = at.slot;
      heads = at.on ? p.heads[which] : 0;
    }
    fetch();
    copy_wait<kDepth - 1>();
    const bool on = h < heads;
    uint64_t x[2][VEC / 2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      widen<VEC>(on && pc[i] >= 0 ? ring[(2 * from + i) * kThreads] : make_uint4(0u, 0u, 0u, 0u), x[i]);
    from = from + 1 == kDepth ? 0 : from + 1;
    const float r = rsqrtf(fmaf(group_sum<G>(sum_products(x, x)), inv_d, eps));
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) x[i][e] = mul2(x[i][e], w[i][e]);
    turn_row<VEC, STAGE>(x, c, pc, half, stage);
    const uint64_t rr = f2(r, r);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) x[i][e] = mul2(x[i][e], rr);
      if (on && pc[i] >= 0) *reinterpret_cast<uint4*>(dst + pc[i]) = narrow<VEC>(x[i]);
    }
    dst += dst_step;
    h += at.slots;
  }
}

// Adds a CTA's per-thread sums of dw up in a fixed order: dw[2][d] of the CTA.
__device__ __forceinline__ void store_dw(const Params& p, const float* smem_dw) {
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.d; i += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += smem_dw[w * 2 * p.d + i];
    p.dw_part[static_cast<int64_t>(blockIdx.x) * 2 * p.d + i] = s;
  }
}

template <typename T, int VEC, int G, bool STAGE>
__global__ void __launch_bounds__(kThreads, 4)
rope_bwd_vec_kernel(const __grid_constant__ Params p) {
  constexpr int D = kDepthBwd;
  extern __shared__ uint4 ring_all[];  // [D][4][kThreads]: two pieces of x, two of dy
  float* sdw = reinterpret_cast<float*>(ring_all + 4 * D * kThreads);  // [kWarps][2][d]
  __shared__ Pairs pairs;
  __shared__ float stage_all[STAGE ? kThreads / G * stage_floats(VEC, G) : 1];
  load_pairs(p, pairs);
  pdl_launch_dependents();
  pdl_wait();
  const int d = p.d, half = p.half;
  int pc[2];
  pieces_of<VEC, STAGE>(threadIdx.x % G, half, d, pc);
  const float inv_d = 1.f / static_cast<float>(d), eps = p.eps;
  float* stage = stage_all + (STAGE ? threadIdx.x / G * stage_floats(VEC, G) : 0);
  float* my_dw = sdw + (threadIdx.x >> 5) * 2 * d;
  uint4* ring = ring_all + threadIdx.x;
  for (int i = threadIdx.x & 31; i < 2 * d; i += 32) my_dw[i] = 0.f;
  uint4 w_raw[2][2];
  fetch_weight<T>(p.w[0], pc, w_raw[0]);
  fetch_weight<T>(p.w[1], pc, w_raw[1]);
  __syncthreads();
  for (int64_t tok0 = static_cast<int64_t>(blockIdx.x) * p.tile; tok0 < p.tokens;
       tok0 += static_cast<int64_t>(gridDim.x) * p.tile) {
    const Place at = place_of<G>(p, tok0);
    const int nq = (p.heads[0] + at.slots - 1) / at.slots, total = nq + (p.heads[1] + at.slots - 1) / at.slots;
    const T *xs = nullptr, *gs = nullptr;  // fetched next
    int64_t x_step = 0, g_step = 0;
    int fetch_k = 0, fetch_h = 0, fetch_heads = 0, fetch_at = 0;
    auto fetch = [&]() {
      if (fetch_k == 0 || fetch_k == nq) {
        const int which = fetch_k >= nq;
        xs = static_cast<const T*>(p.x[which]) + at.b * p.sb[which] + at.n * p.sn[which] + at.slot * p.sh[which];
        gs = static_cast<const T*>(p.dy[which]) + ((at.b * p.heads[which] + at.slot) * p.N + at.n) * d;
        x_step = at.slots * p.sh[which];
        g_step = at.slots * p.N * d;
        fetch_h = at.slot;
        fetch_heads = at.on ? p.heads[which] : 0;
      }
      if (fetch_h < fetch_heads) {
        const uint32_t to = sm100::smem_u32(ring + fetch_at * 4 * kThreads);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (pc[i] >= 0) {
            copy_async16(to + i * kThreads * 16, xs + pc[i]);
            copy_async16(to + (2 + i) * kThreads * 16, gs + pc[i]);
          }
      }
      copy_commit();
      xs += x_step;
      gs += g_step;
      fetch_h += at.slots;
      ++fetch_k;
      fetch_at = fetch_at + 1 == D ? 0 : fetch_at + 1;
    };
#pragma unroll 1
    for (int k = 0; k < D - 1; ++k) fetch();
    Turn<VEC, STAGE> c;
    load_turn<VEC, STAGE>(c, pairs, positions_of(p, at.tok, at.n), pc, half, -1.f);
    uint64_t w[2][VEC / 2], dw[2][VEC / 2];
    T* dst = nullptr;
    int64_t dst_step = 0;
    int h = 0, heads = 0, from = 0;
    auto add_dw = [&](int which) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          float a, b;
          unpack(dw[i][e], a, b);
#pragma unroll
          for (int m = G; m < 32; m <<= 1) {  // the groups of a warp
            a += __shfl_xor_sync(0xffffffffu, a, m);
            b += __shfl_xor_sync(0xffffffffu, b, m);
          }
          if ((threadIdx.x & 31) < G && pc[i] >= 0) {
            my_dw[which * d + pc[i] + 2 * e] += a;
            my_dw[which * d + pc[i] + 2 * e + 1] += b;
          }
        }
    };
#pragma unroll 1
    for (int k = 0; k < total; ++k) {  // (the same for all lanes of a warp)
      if (k == 0 || k == nq) {
        if (k > 0) add_dw(0);
        const int which = k >= nq;
        widen_weight<VEC>(p.w[which], which ? w_raw[1] : w_raw[0], 1.f, w);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < VEC / 2; ++e) dw[i][e] = 0;
        dst = static_cast<T*>(p.out[which]) + (at.tok * p.heads[which] + at.slot) * d;
        dst_step = at.slots * d;
        h = at.slot;
        heads = at.on ? p.heads[which] : 0;
      }
      fetch();
      copy_wait<D - 1>();
      const bool on = h < heads;
      uint64_t x[2][VEC / 2], g[2][VEC / 2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool have = on && pc[i] >= 0;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        widen<VEC>(have ? ring[(4 * from + i) * kThreads] : zero, x[i]);
        widen<VEC>(have ? ring[(4 * from + 2 + i) * kThreads] : zero, g[i]);
      }
      from = from + 1 == D ? 0 : from + 1;
      // (a group without a row adds zeros to dw: with eps = 0 the root would make them NaN)
      const float square = fmaf(group_sum<G>(sum_products(x, x)), inv_d, eps), r = on ? rsqrtf(square) : 0.f;
      const uint64_t rr = f2(r, r), ff = f2(k >= nq ? p.scale[1] : p.scale[0], k >= nq ? p.scale[1] : p.scale[0]);
      turn_row<VEC, STAGE>(g, c, pc, half, stage);  // back
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          x[i][e] = mul2(x[i][e], rr);
          g[i][e] = mul2(g[i][e], ff);
          dw[i][e] = fma2(g[i][e], x[i][e], dw[i][e]);
          g[i][e] = mul2(g[i][e], w[i][e]);
        }
      const float dot = -group_sum<G>(sum_products(g, x)) * inv_d;
      const uint64_t dd = f2(dot, dot);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) g[i][e] = mul2(fma2(x[i][e], dd, g[i][e]), rr);
        if (on && pc[i] >= 0) *reinterpret_cast<uint4*>(dst + pc[i]) = narrow<VEC>(g[i]);
      }
      dst += dst_step;
      h += at.slots;
    }
    if (total > 0) add_dw(total > nq ? 1 : 0);
  }
  store_dw(p, sdw);
}

// A warp a row. Value slots of a lane: M pairs (a, b), then (REST: rot < d) 2M single
// values. A warp keeps one token: its angles and both weights stay in the lanes'
// registers while it walks the heads (with rows found one by one, and the slots behind
// the rotated values always there, 88 and 147 us at B4 N2K, 32 heads of 90).
template <typename T, int M, bool REST>
struct WarpRow {
  static constexpr int R = REST ? 2 * M : 0, SLOTS = 2 * M + R;
  float x[SLOTS];  // a, b, rest
  __device__ __forceinline__ void load(const T* p, int lane, int half, int d) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int j = lane + 32 * m;
      x[m] = j < half ? to_f32(p[j]) : 0.f;
      x[M + m] = j < half ? to_f32(p[half + j]) : 0.f;
    }
#pragma unroll
    for (int m = 0; m < R; ++m) {
      const int j = 2 * half + lane + 32 * m;
      x[2 * M + m] = j < d ? to_f32(p[j]) : 0.f;
    }
  }
  __device__ __forceinline__ void store(T* p, int lane, int half, int d) const {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int j = lane + 32 * m;
      if (j < half) {
        p[j] = from_f32<T>(x[m]);
        p[half + j] = from_f32<T>(x[M + m]);
      }
    }
#pragma unroll
    for (int m = 0; m < R; ++m) {
      const int j = 2 * half + lane + 32 * m;
      if (j < d) p[j] = from_f32<T>(x[2 * M + m]);
    }
  }
  __device__ __forceinline__ void turn(const float2 (&cs)[M], float sign) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const float u = x[m], v = x[M + m], sn = sign * cs[m].y;
      x[m] = fmaf(u, cs[m].x, -sn * v);
      x[M + m] = fmaf(v, cs[m].x, sn * u);
    }
  }
};
// Both weights' values of a lane, times f (f where there is no weight).
template <typename T, int M, bool REST>
__device__ __forceinline__ void load_weights(const Params& p, WarpRow<T, M, REST> (&w)[2], int lane, float f0, float f1) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (p.w[i]) w[i].load(static_cast<const T*>(p.w[i]), lane, p.half, p.d);
#pragma unroll
    for (int e = 0; e < w[i].SLOTS; ++e) w[i].x[e] = (p.w[i] ? w[i].x[e] : 1.f) * (i ? f1 : f0);
  }
}
// cos and sin of a lane's pairs.
template <int M>
__device__ __forceinline__ void load_angles(const Params& p, const Place& at, int lane, float2 (&cs)[M]) {
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int j = lane + 32 * m;
    cs[m] = make_float2(1.f, 0.f);
    if (j < p.half) {
      const int64_t n = p.pos ? p.pos[p.axis[j] * p.tokens + at.tok] : at.n;
      const double a = static_cast<double>(n) * p.turn[j];
      sincospif(2.f * static_cast<float>(a - rint(a)), &cs[m].y, &cs[m].x);
    }
  }
}

template <typename T, int M, bool REST>
__global__ void __launch_bounds__(kThreads)
rope_fwd_row_kernel(const __grid_constant__ Params p) {
  using Row = WarpRow<T, M, REST>;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, d = p.d, half = p.half;
  const float inv_d = 1.f / static_cast<float>(d);
  const Place at = place_of<32>(p, static_cast<int64_t>(blockIdx.x) * p.tile);
  if (!at.on) return;
  float2 cs[M];
  load_angles(p, at, lane, cs);
  Row w[2];
  load_weights(p, w, lane, p.scale[0], p.scale[1]);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const T* src = static_cast<const T*>(p.x[which]) + at.b * p.sb[which] + at.n * p.sn[which] + at.slot * p.sh[which];
    T* dst = static_cast<T*>(p.out[which]) + ((at.b * p.heads[which] + at.slot) * p.N + at.n) * d;
    const int64_t src_step = at.slots * p.sh[which], dst_step = at.slots * p.N * d;
#pragma unroll 1
    for (int h = at.slot; h < p.heads[which]; h += 2 * at.slots) {
      const bool two = h + at.slots < p.heads[which];
      Row x[2];
      x[0].load(src, lane, half, d);
      x[1].load(two ? src + src_step : src, lane, half, d);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (u && !two) break;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < Row::SLOTS; ++e) s = fmaf(x[u].x[e], x[u].x[e], s);
        const float r = rsqrtf(fmaf(group_sum<32>(s), inv_d, p.eps));
#pragma unroll
        for (int e = 0; e < Row::SLOTS; ++e) x[u].x[e] *= r * w[which].x[e];
        x[u].turn(cs, 1.f);
        x[u].store(dst + u * dst_step, lane, half, d);
      }
      src += 2 * src_step;
      dst += 2 * dst_step;
    }
  }
}

template <typename T, int M, bool REST>
__global__ void __launch_bounds__(kThreads)
rope_bwd_row_kernel(const __grid_constant__ Params p) {
  using Row = WarpRow<T, M, REST>;
  extern __shared__ float row_dw[];  // [kWarps][2][d]
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, d = p.d, half = p.half;
  const float inv_d = 1.f / static_cast<float>(d);
  Row w[2];
  load_weights(p, w, lane, 1.f, 1.f);
  WarpRow<float, M, REST> dw[2];
#pragma unroll
  for (int e = 0; e < Row::SLOTS; ++e) dw[0].x[e] = dw[1].x[e] = 0.f;
  for (int64_t tok0 = static_cast<int64_t>(blockIdx.x) * p.tile; tok0 < p.tokens;
       tok0 += static_cast<int64_t>(gridDim.x) * p.tile) {
    const Place at = place_of<32>(p, tok0);
    if (!at.on) continue;
    float2 cs[M];
    load_angles(p, at, lane, cs);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const T* xs = static_cast<const T*>(p.x[which]) + at.b * p.sb[which] + at.n * p.sn[which] + at.slot * p.sh[which];
      const T* gs = static_cast<const T*>(p.dy[which]) + ((at.b * p.heads[which] + at.slot) * p.N + at.n) * d;
      T* dst = static_cast<T*>(p.out[which]) + (at.tok * p.heads[which] + at.slot) * d;
      const int64_t x_step = at.slots * p.sh[which], g_step = at.slots * p.N * d, dst_step = at.slots * d;
#pragma unroll 1
      for (int h = at.slot; h < p.heads[which]; h += 2 * at.slots) {
        const bool two = h + at.slots < p.heads[which];
        Row x[2], g[2];
        x[0].load(xs, lane, half, d);
        g[0].load(gs, lane, half, d);
        x[1].load(two ? xs + x_step : xs, lane, half, d);
        g[1].load(two ? gs + g_step : gs, lane, half, d);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (u && !two) break;
          float s = 0.f;
#pragma unroll
          for (int e = 0; e < Row::SLOTS; ++e) s = fmaf(x[u].x[e], x[u].x[e], s);
          const float r = rsqrtf(fmaf(group_sum<32>(s), inv_d, p.eps));
          g[u].turn(cs, -1.f);
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < Row::SLOTS; ++e) {
            x[u].x[e] *= r;
            g[u].x[e] *= p.scale[which];
            dw[which].x[e] = fmaf(g[u].x[e], x[u].x[e], dw[which].x[e]);
            g[u].x[e] *= w[which].x[e];
            dot = fmaf(g[u].x[e], x[u].x[e], dot);
          }
          dot = group_sum<32>(dot) * inv_d;
#pragma unroll
          for (int e = 0; e < Row::SLOTS; ++e) g[u].x[e] = r * fmaf(-x[u].x[e], dot, g[u].x[e]);
          g[u].store(dst + u * dst_step, lane, half, d);
        }
        xs += 2 * x_step;
        gs += 2 * g_step;
        dst += 2 * dst_step;
      }
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which)
    dw[which].store(row_dw + ((threadIdx.x >> 5) * 2 + which) * d, lane, half, d);
  store_dw(p, row_dw);
}

// dw of the queries' and keys' weights from the CTAs' sums, in fp64 and a fixed order.
constexpr int kDwWarps = 32;
template <typename T>
__global__ void __launch_bounds__(32 * kDwWarps)
dw_kernel(const float* __restrict__ part, int n, int d, T* __restrict__ dwq, T* __restrict__ dwk) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ double sum[kDwWarps][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
  double s = 0.0;
  if (i < 2 * d) {
#pragma unroll 8
    for (int c = w; c < n; c += kDwWarps) s += part[static_cast<int64_t>(c) * 2 * d + i];
  }
  sum[w][lane] = s;
  __syncthreads();
  if (w == 0 && i < 2 * d) {
    for (int x = 1; x < kDwWarps; ++x) s += sum[x][lane];
    T* o = i < d ? dwq : dwk;
    if (o) o[i < d ? i : i - d] = from_f32<T>(static_cast<float>(s));
  }
}

// ---------------------------------------------------------------------- host

struct Args {
  const void *q, *k, *wq, *wk;
  int64_t qs[3], ks[3];
  const int32_t* pos;
  int64_t B, N, H, Hkv, d, rot, axes;
  const int64_t* sections;
  double base, eps, q_scale, k_scale;
  la2_dtype dt;
};

static la2_status check(const Args& a) {
  if (a.B < 0 || a.N < 0 || a.H < 0 || a.Hkv < 0 || a.d < 1 || a.rot < 0 || a.rot > a.d || a.rot % 2)
    return LA2_ERR_INVALID_ARG;
  if (a.dt != LA2_F32 && a.dt != LA2_BF16) return LA2_ERR_INVALID_ARG;
  if (a.axes < 1 || !(a.base > 0.0) || !(a.eps >= 0.0) || !std::isfinite(a.base) || !std::isfinite(a.eps) ||
      !std::isfinite(a.q_scale) || !std::isfinite(a.k_scale))
    return LA2_ERR_INVALID_ARG;
  if (a.d > kMaxD || a.axes > kMaxAxes) return LA2_ERR_UNSUPPORTED;
  if (!a.sections && a.axes != 1) return LA2_ERR_INVALID_ARG;
  if (a.sections) {
    int64_t sum = 0;
    for (int i = 0; i < a.axes; ++i) {
      if (a.sections[i] < 0 || a.sections[i] > a.rot) return LA2_ERR_INVALID_ARG;
      sum += a.sections[i];
    }
    if (sum != a.rot / 2) return LA2_ERR_INVALID_ARG;
  }
  for (int i = 0; i < 3; ++i)
    if (a.qs[i] < 0 || a.ks[i] < 0 || a.qs[i] > (int64_t(1) << 48) || a.ks[i] > (int64_t(1) << 48))
      return LA2_ERR_INVALID_ARG;
  if (double(a.B) * double(a.N) * (double(a.H) + double(a.Hkv)) * double(a.d) > 9.0e17) return LA2_ERR_INVALID_ARG;
  if (a.B > 0x7fffffff || a.N > 0x7fffffff || a.H + a.Hkv > (1 << 20)) return LA2_ERR_UNSUPPORTED;
  if (double(a.B) * double(a.N) > 2147483647.0) return LA2_ERR_UNSUPPORTED;
  return LA2_OK;
}

// Bytes from the first to behind the last element of a strided [B, N, heads, d] slice.
static size_t extent(const Args& a, const int64_t* s, int64_t heads, size_t es) {
  if (a.B == 0 || a.N == 0 || heads == 0) return 0;
  return ((size_t)((a.B - 1) * s[0] + (a.N - 1) * s[1] + (heads - 1) * s[2] + a.d)) * es;
}

// Lanes of a row's group, a power of two (the kernels are instantiated for 4 to 32).
static int group_of(const Args& a) {
  const int half = (int)a.rot / 2, d = (int)a.d;
  const int lanes = a.dt == LA2_BF16 ? lanes_of<8>(half, d) : lanes_of<4>(half, d);
  return lanes <= 4 ? 4 : lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32;
}
// Tokens of a tile, a power of two: one for each group of a CTA, whose set-up (angles,
// coefficients) is then done once a token and whose rows of a head leave as one piece
// (B4 N2K, 32 heads of 128, bf16: 16 tokens 27.9 and 43.3 us forward and back, 8 tokens
// 31.1 and 48.1); fewer where that would leave an SM less than three tiles. A warp a row
// hides its loads behind other warps: few tokens, many CTAs.
static int tile_of(const Args& a, bool vec, int sms) {
  int64_t t = vec ? kThreads / group_of(a) : kRowTile;
  while (t > 1 && a.B * a.N < t * 3 * sms) t /= 2;
  return static_cast<int>(t);
}

// CTAs of the backward: each leaves its sums of dw, so a bounded number (8 an SM, of which
// 4 run at once: 128 registers a thread), which take further tiles in turn.
static int bwd_grid(const Args& a, int tile, int sms) {
  const int64_t tiles = (a.B * a.N + tile - 1) / tile;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(tiles, 8 * (int64_t)sms)));
}

static Params params(const Args& a, int tile) {
  Params p{};
  p.x[0] = a.q;
  p.x[1] = a.k;
  p.w[0] = a.wq;
  p.w[1] = a.wk;
  p.pos = a.pos;
  p.sb[0] = a.qs[0]; p.sn[0] = a.qs[1]; p.sh[0] = a.qs[2];
  p.sb[1] = a.ks[0]; p.sn[1] = a.ks[1]; p.sh[1] = a.ks[2];
  p.N = a.N;
  p.tokens = a.B * a.N;
  p.heads[0] = (int)a.H;
  p.heads[1] = (int)a.Hkv;
  p.d = (int)a.d;
  p.half = (int)a.rot / 2;
  p.tile = tile;
  p.splits = 1;
  p.axes = (int)a.axes;
  p.eps = (float)a.eps;
  p.scale[0] = (float)a.q_scale;
  p.scale[1] = (float)a.k_scale;
  int i = 0;
  for (int ax = 0; ax < a.axes; ++ax)
    for (int64_t n = a.sections ? a.sections[ax] : a.rot / 2; n > 0; --n, ++i) p.axis[i] = (uint8_t)ax;
  // base^(-2i/rot) / (2 pi) as products of two powers, i mod 16 and the rest (a call of
  // pow for each took 3 us of the call, as long as the launch): three roundings of fp64
  double lo[16], hi[kMaxD / 32];
  const double step = p.half ? -2.0 / static_cast<double>(a.rot) : 0.0;
  for (i = 0; i < std::min(16, p.half); ++i) lo[i] = std::pow(a.base, i * step);
  for (i = 0; 16 * i < p.half; ++i) hi[i] = std::pow(a.base, 16 * i * step) / 6.283185307179586476925286766559;
  for (i = 0; i < p.half; ++i) p.turn[i] = lo[i % 16] * hi[i / 16];
  return p;
}

// Whether rows can be taken in 16-byte pieces.
static bool vec_ok(const Args& a, const void* const* more, int n) {
  const int64_t es = a.dt == LA2_BF16 ? 2 : 4, vec = 16 / es;
  if (a.d % vec) return false;
  for (int i = 0; i < 3; ++i)
    if (a.qs[i] % vec || a.ks[i] % vec) return false;
  if (!is_aligned(a.q, 16) || !is_aligned(a.k, 16) || !is_aligned(a.wq, 16) || !is_aligned(a.wk, 16)) return false;
  for (int i = 0; i < n; ++i)
    if (!is_aligned(more[i], 16)) return false;
  return true;
}

using Kernel = void (*)(const Params);
template <typename T, bool BWD, int G, bool STAGE>
static Kernel vec_kernel() {
  if constexpr (BWD)
    return rope_bwd_vec_kernel<T, 16 / sizeof(T), G, STAGE>;
  else
    return rope_fwd_vec_kernel<T, 16 / sizeof(T), G, STAGE>;
}
template <typename T, bool BWD, bool STAGE>
static Kernel vec_kernel(int g) {
  return g == 4   ? vec_kernel<T, BWD, 4, STAGE>()
         : g == 8  ? vec_kernel<T, BWD, 8, STAGE>()
         : g == 16 ? vec_kernel<T, BWD, 16, STAGE>()
                   : vec_kernel<T, BWD, 32, STAGE>();
}
template <typename T, bool BWD>
static Kernel vec_kernel(const Args& a) {
  // (pairs a whole number of 16-byte pieces apart stay within a lane)
  return (a.rot / 2) % (16 / (int)sizeof(T)) ? vec_kernel<T, BWD, true>(group_of(a))
                                             : vec_kernel<T, BWD, false>(group_of(a));
}

template <typename T, bool BWD, int M>
static Kernel row_kernel_of(bool rest) {
  if constexpr (BWD)
    return rest ? rope_bwd_row_kernel<T, M, true> : rope_bwd_row_kernel<T, M, false>;
  else
    return rest ? rope_fwd_row_kernel<T, M, true> : rope_fwd_row_kernel<T, M, false>;
}
template <typename T, bool BWD>
static Kernel row_kernel(const Args& a) {
  const bool rest = a.rot < a.d;
  return a.d <= 64 ? row_kernel_of<T, BWD, 1>(rest) : a.d <= 128 ? row_kernel_of<T, BWD, 2>(rest)
                                                                : row_kernel_of<T, BWD, 4>(rest);
}

// Dynamic shared memory beyond the default limit (wide rows, with their static part).
static bool allow_smem(Kernel kern, size_t bytes) {
  return bytes <= 32 * 1024 ||
         cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

template <typename T>
static la2_status launch_fwd(const Args& a, Params p, bool vec, int sms, cudaStream_t st) {
  const int64_t tiles = (p.tokens + p.tile - 1) / p.tile;
  // few tokens (a decode batch): their heads over several CTAs
  const int64_t rows = (int64_t)p.tile * (a.H + a.Hkv);
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(3 * sms / tiles, (rows + 15) / 16));
  const size_t smem = vec ? (size_t)2 * kDepth * kThreads * 16 : 0;
  const dim3 grid((unsigned)tiles, (unsigned)p.splits), block(kThreads);
  const Kernel kern = vec ? vec_kernel<T, false>(a) : row_kernel<T, false>(a);
  if (!allow_smem(kern, smem)) return LA2_ERR_CUDA;
  LaunchTimer t(K_QK_ROPE, st);
  if (launch_pdl(kern, grid, block, smem, st, p) != cudaSuccess) return LA2_ERR_CUDA;
  return launch_status();
}

template <typename T>
static la2_status launch_bwd(const Args& a, const Params& p, bool vec, int grid, void* dwq, void* dwk,
                             cudaStream_t st) {
  const size_t smem = (size_t)kWarps * 2 * p.d * sizeof(float) +
                      (vec ? (size_t)4 * kDepthBwd * kThreads * 16 : 0);
  const Kernel kern = vec ? vec_kernel<T, true>(a) : row_kernel<T, true>(a);
  if (!allow_smem(kern, smem)) return LA2_ERR_CUDA;
  {
    LaunchTimer t(K_QK_ROPE_BWD, st);
    if (launch_pdl(kern, dim3(grid), dim3(kThreads), smem, st, p) != cudaSuccess) return LA2_ERR_CUDA;
    if (dwq || dwk)
      if (launch_pdl(dw_kernel<T>, dim3((2 * p.d + 31) / 32), dim3(32 * kDwWarps), 0, st,
                     static_cast<const float*>(p.dw_part), grid, p.d, static_cast<T*>(dwq),
                     static_cast<T*>(dwk)) != cudaSuccess)
        return LA2_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace rope
}  // namespace la2

extern "C" {

la2_status la2_qk_norm_rope(const void* q, const void* k, const int64_t* q_strides, const int64_t* k_strides,
                            const void* wq, const void* wk, const int32_t* positions, void* q_out,
                            void* k_out, int64_t B, int64_t N, int64_t H, int64_t Hkv, int64_t d,
                            int64_t rot, int64_t n_axes, const int64_t* sections, double base, double eps,
                            double q_scale, double k_scale, la2_dtype dt, la2_stream_t stream) {
  if (!q_strides || !k_strides) return LA2_ERR_INVALID_ARG;
  rope::Args a{q, k, wq, wk, {q_strides[0], q_strides[1], q_strides[2]},
               {k_strides[0], k_strides[1], k_strides[2]}, positions, B, N, H, Hkv, d, rot, n_axes, sections,
               base, eps, q_scale, k_scale, dt};
  la2_status s = rope::check(a);
  if (s != LA2_OK) return s;
  if (B == 0 || N == 0 || H + Hkv == 0) return LA2_OK;
  const size_t es = dt == LA2_BF16 ? 2 : 4;
  if ((H > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !k_out))) return LA2_ERR_INVALID_ARG;
  const void* ptr[6] = {q, k, wq, wk, q_out, k_out};
  for (const void* x : ptr)
    if (!is_aligned(x, es)) return LA2_ERR_INVALID_ARG;
  if (!is_aligned(positions, 4)) return LA2_ERR_INVALID_ARG;
  const size_t nq = (size_t)B * N * H * d * es, nk = (size_t)B * N * Hkv * d * es;
  const gated::Span in[5] = {{q, rope::extent(a, a.qs, H, es)}, {k, rope::extent(a, a.ks, Hkv, es)},
                             {wq, wq ? (size_t)d * es : 0}, {wk, wk ? (size_t)d * es : 0},
                             {positions, positions ? (size_t)n_axes * B * N * 4 : 0}};
  for (const gated::Span& x : in)
    if (x.n && (overlaps(q_out, nq, x.p, x.n) || overlaps(k_out, nk, x.p, x.n))) return LA2_ERR_INVALID_ARG;
  if (nq && nk && overlaps(q_out, nq, k_out, nk)) return LA2_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LA2_ERR_CUDA;
  const void* outs[2] = {q_out, k_out};
  const bool vec = rope::vec_ok(a, outs, 2);
  rope::Params p = rope::params(a, rope::tile_of(a, vec, sms));
  p.out[0] = q_out;
  p.out[1] = k_out;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dt == LA2_BF16 ? rope::launch_fwd<__nv_bfloat16>(a, p, vec, sms, st)
                        : rope::launch_fwd<float>(a, p, vec, sms, st);
}

size_t la2_qk_norm_rope_backward_workspace_size(int64_t B, int64_t N, int64_t H, int64_t Hkv, int64_t d) {
  if (B < 0 || N < 0 || H < 0 || Hkv < 0 || d < 1 || d > rope::kMaxD) return (size_t)-1;
  if (double(B) * double(N) > 2147483647.0) return (size_t)-1;
  if (B == 0 || N == 0 || H + Hkv == 0) return 0;
  const int sms = device_sm_count();
  if (sms <= 0) return (size_t)-1;
  rope::Args a{};
  a.B = B;
  a.N = N;
  return (size_t)rope::bwd_grid(a, 1, sms) * 2 * d * sizeof(float);  // (the type and its tile are not known here)
}

la2_status la2_qk_norm_rope_backward(const void* dq_out, const void* dk_out, const void* q, const void* k,
                                     const int64_t* q_strides, const int64_t* k_strides, const void* wq,
                                     const void* wk, const int32_t* positions, void* dq, void* dk, void* dwq,
                                     void* dwk, int64_t B, int64_t N, int64_t H, int64_t Hkv, int64_t d,
                                     int64_t rot, int64_t n_axes, const int64_t* sections, double base,
                                     double eps, double q_scale, double k_scale, la2_dtype dt,
                                     void* workspace, size_t workspace_bytes, la2_stream_t stream) {
  if (!q_strides || !k_strides) return LA2_ERR_INVALID_ARG;
  rope::Args a{q, k, wq, wk, {q_strides[0], q_strides[1], q_strides[2]},
               {k_strides[0], k_strides[1], k_strides[2]}, positions, B, N, H, Hkv, d, rot, n_axes, sections,
               base, eps, q_scale, k_scale, dt};
  la2_status s = rope::check(a);
  if (s != LA2_OK) return s;
  // a weight and its gradient come together
  if ((wq == nullptr) != (dwq == nullptr) || (wk == nullptr) != (dwk == nullptr)) return LA2_ERR_INVALID_ARG;
  const size_t es = dt == LA2_BF16 ? 2 : 4;
  const void* ptr[10] = {dq_out, dk_out, q, k, wq, wk, dq, dk, dwq, dwk};
  for (const void* x : ptr)
    if (!is_aligned(x, es)) return LA2_ERR_INVALID_ARG;
  if (!is_aligned(positions, 4)) return LA2_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0 || N == 0 || H + Hkv == 0) {  // sums over no rows
    if (dwq && cudaMemsetAsync(dwq, 0, d * es, st) != cudaSuccess) return LA2_ERR_CUDA;
    if (dwk && cudaMemsetAsync(dwk, 0, d * es, st) != cudaSuccess) return LA2_ERR_CUDA;
    return LA2_OK;
  }
  if ((H > 0 && (!q || !dq || !dq_out)) || (Hkv > 0 && (!k || !dk || !dk_out))) return LA2_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LA2_ERR_CUDA;
  const void* more[4] = {dq, dk, dq_out, dk_out};
  const bool vec = rope::vec_ok(a, more, 4);
  const int tile = rope::tile_of(a, vec, sms), grid = rope::bwd_grid(a, tile, sms);
  const size_t need = (size_t)grid * 2 * d * sizeof(float);
  if (!workspace || workspace_bytes < need) return LA2_ERR_WORKSPACE;
  if (!is_aligned(workspace, 256)) return LA2_ERR_INVALID_ARG;
  const size_t nq = (size_t)B * N * H * d * es, nk = (size_t)B * N * Hkv * d * es;
  const gated::Span in[7] = {{q, rope::extent(a, a.qs, H, es)}, {k, rope::extent(a, a.ks, Hkv, es)},
                             {wq, wq ? (size_t)d * es : 0}, {wk, wk ? (size_t)d * es : 0},
                             {positions, positions ? (size_t)n_axes * B * N * 4 : 0}, {dq_out, nq}, {dk_out, nk}};
  const gated::Span out[5] = {{dq, nq}, {dk, nk}, {dwq, dwq ? (size_t)d * es : 0},
                              {dwk, dwk ? (size_t)d * es : 0}, {workspace, need}};
  for (int i = 0; i < 5; ++i) {
    if (!out[i].n) continue;
    for (const gated::Span& x : in)
      if (x.n && overlaps(out[i].p, out[i].n, x.p, x.n)) return LA2_ERR_INVALID_ARG;
    for (int j = i + 1; j < 5; ++j)
      if (out[j].n && overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return LA2_ERR_INVALID_ARG;
  }
  rope::Params p = rope::params(a, tile);
  p.out[0] = dq;
  p.out[1] = dk;
  p.dy[0] = dq_out;
  p.dy[1] = dk_out;
  p.dw_part = static_cast<float*>(workspace);
  return dt == LA2_BF16 ? rope::launch_bwd<__nv_bfloat16>(a, p, vec, grid, dwq, dwk, st)
                        : rope::launch_bwd<float>(a, p, vec, grid, dwq, dwk, st);
}

}  // extern "C"
