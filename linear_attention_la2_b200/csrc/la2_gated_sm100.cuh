// Tensor-core kernels of the gated recurrence (bf16, d and dv 64 or 128, sm_100a); the
// formulas are at the top of la2_gated_simt.cuh. The PTX wrappers, operand
// descriptors, bounded waits and TMEM layouts are those of la2_sm100.cuh.
//
// One kernel does all four products of a layer, as out_t = sum over the kept s of
// w(t, s) (x_t . y_s) z_s with (x, y, z) in the query, key and value places:
//
//             x   y   z    walk      kept     w                  state (z x y)
//   O         q   k   v    forward   s <= t   e^(c_t - c_s)      KV^T = v^T k
//   dQ        dO  v   k    forward   s <= t   e^(c_t - c_s)      KV = k^T v
//   dV        k   q   dO   back      s >= t   e^(c_s - c_t)      U^T = dO^T q
//   dK        v   dO  q    back      s >= t   e^(c_s - c_t)      U = q^T dO
//
// Per block of 64 rows, walking a chunk of one (b, h) sequence in one CTA:
//   S     = X Y^T                      tcgen05 -> TMEM
//   P     = bf16(S w)                  mask warps, TMEM -> shared memory
//   near  = Z^T P^T                    tcgen05 -> TMEM, transposed: M = 128 lanes, 64
//   far   = state X^T                  columns each; the state's bf16 copy is the A
//                                      operand, read from TMEM
//   out   = head far + near            epilogue warps: the row's e^(c_t) (walking
//                                      back e^(c_R - c_t)) is applied in fp32
//   state <- e^(c_R) state + Z^T Y~    tcgen05, Y~ = rows scaled by e^(c_R - c_s)
//                                      (walking back e^(c_s))
// far and near are separate accumulators, so X needs no scaling. Y~ is made in place
// once S has read Y, as a bf16 value there and its bf16 remainder beside it (two
// MMAs): one rounding fewer in the outputs, and states good to 2^-17. The state stays
// in TMEM: the state warps read it once a block, write its bf16 copy for far, and put
// e^(c_R) times it back, which the block's update adds onto. The loop-carried path is
// update -> copy -> update; S of the next block is issued before it, and the second
// buffers of far and P let the epilogue and the mask trail.
//
// What bounds it: no unit alone. A 64-row block takes about 3600 cycles (B1 H32 N16K: 120 us
// for 64 blocks a CTA), its share of HBM 2850 at 148 SMs, shared memory about 2200 of 128
// bytes by count (tile loads, operand reads, the scaling, P and the output tile; GRAD 2900;
// the state's copy as an operand there took 500, GRAD 1000, more), the tensor pipe a third, the
// issue slots half. What is left are the waits of the chain update -> copy -> update and
// between the roles.
//
// Gate sums: c in base 2, fp32, at most 64 terms; a restart counts as 0 there and cuts the
// weights made of them.
//
// NaN and infinities: a restart drops the state and what chunks start from; inside the 64
// rows of a block the products mix all rows (0 times NaN).
//
// GRAD (dQ, dK) also returns the rows' dots q . dq and k . dk (fp32, from the
// unrounded rows) for the gates' gradient, a running difference of them: their
// errors have to cancel over a chunk. P is rounded alike in both passes (the same
// products, the same weights), so the near parts agree; for the far parts the state's
// copy is kept as value and remainder too (2^-17 instead of 2^-9). The dots' rows are
// loaded into the output's staging tile, read there and overwritten by the output.
//
// Widths of 64 run as 128: the tensor maps end at the tensor's width, so that the tiles'
// second 64 columns arrive as zeros and are not stored, and the chunk states' other rows
// and columns are zeros. The blocks' time is that of 128, a third of the CUDA cores' at
// 64 (B4 H4 N2K: forward 97 -> 31 us, gradients 245 -> 83 us).
//
// Roundings: P and, in O and dV, the state's copy are one bf16 value each, as in the plain
// and decayed forms' kernels: with Y~ and the sums finer, an output is 2.35e-3 off
// (relative Frobenius) where its own rounding alone is 1.66e-3. A second value of P
// would be another product of 64 x 128 x 64 a block and 16 KB that are not there.
//
// The roles' inner loops stay rolled: five roles share each scheduler, and unrolled
// over a block their instructions came from beyond its instruction cache.
#pragma once

#include "la2_gated_simt.cuh"
#include "la2_sm100.cuh"

namespace la2 {
namespace gated {

namespace s = sm100;

constexpr int kTile = 64 * 128 * 2;       // one 64 x 128 bf16 tile
constexpr int kMainThreads = 768;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kTabs = 8, kTab = 452;      // gate tables in flight, their floats (see the table warp)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Running sums of 64 gates over a warp: lane l gets those of rows 2l and 2l + 1.
__device__ __forceinline__ void warp_sums(float x, float y, int lane, float& a, float& b) {
  float t = x + y;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const float up = __shfl_up_sync(0xffffffffu, t, m);
    if (lane >= m) t += up;
  }
  b = t;
  // (a as t - y would be NaN - NaN or lose y's digits next to a restart)
  const float before = __shfl_up_sync(0xffffffffu, t, 1);
  a = (lane ? before : 0.f) + x;
}

// Sums of the gates behind each row instead, of all 64 in `all`.
__device__ __forceinline__ void warp_sums_behind(float x, float y, int lane, float& a, float& b, float& all) {
  float t = x + y;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const float down = __shfl_down_sync(0xffffffffu, t, m);
    if (lane + m < 32) t += down;
  }
  all = __shfl_sync(0xffffffffu, t, 0);
  const float next = __shfl_down_sync(0xffffffffu, t, 1);
  b = lane < 31 ? next : 0.f;
  a = y + b;
}
// (NaN is none.)
__device__ __forceinline__ bool is_restart(__nv_bfloat16 x) { return to_f32(x) < kRestart; }
// Restarts of a block as ballots of its even and odd rows: whether one lies at or before
// row 2 lane + odd, or behind it.
__device__ __forceinline__ bool restart_upto(uint32_t even, uint32_t odd_rows, int lane, int odd) {
  const uint32_t to = 0xffffffffu >> (31 - lane);
  return (even & to) | (odd_rows & (odd ? to : to >> 1));
}
__device__ __forceinline__ bool restart_behind(uint32_t even, uint32_t odd_rows, int lane, int odd) {
  const uint32_t from = 0xffffffffu << lane;
  return (even & (from << 1)) | (odd_rows & (odd ? from << 1 : from));
}
// Bits 0..7 to the even places.
__device__ __forceinline__ uint32_t spread_bits(uint32_t x) {
  x = (x | x << 4) & 0x0f0fu;
  x = (x | x << 2) & 0x3333u;
  return (x | x << 1) & 0x5555u;
}
// The columns that are kept of row l of a square on the diagonal, as bits: those up to l
// from the last restart at or before it on (BACK: those from l to the restart behind it).
template <bool BACK>
__device__ __forceinline__ uint32_t kept_bits(uint32_t restarts, int l) {
  const uint32_t upto = (2u << l) - 1;
  if (BACK) {
    const uint32_t behind = restarts & ~upto;
    return ((behind & -behind) - 1) & 0xffffu & ~(upto >> 1);
  }
  const uint32_t before = restarts & upto;
  return before ? upto & ~((1u << (31 - __clz(before))) - 1) : upto;
}

// One lane of the warp, the same for every MMA and commit of the issuing loop.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}
// N MMAs of 16 k each by the elected lane; the operands' descriptors step by da and db
// (bytes / 16) from MMA to MMA, and from every fourth to the next by ja, jb more.
template <int N>
__device__ __forceinline__ void mma_run(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t da, uint32_t db,
                                        uint32_t ja, uint32_t jb, uint32_t idesc, uint32_t accumulate) {
  if (lead) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      s::mma_bf16_ss(d, a + k * da + (k >> 2) * ja, b + k * db + (k >> 2) * jb, idesc, k > 0 ? 1u : accumulate);
  }
  __syncwarp();
}
// D[tmem] (+)= A[tmem] B[smem] by the calling thread (A: M lanes, two bf16 a column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint64_t* bar) {
  if (lead) s::mma_commit(bar);
  __syncwarp();
}

// Calls f(i, x, y) for the blocks i < n in turn, x and y the gates of rows 2 lane and
// 2 lane + 1 of block i (get(i, r) reads one). Loads run four blocks ahead: under load
// one takes about as long as a block. f's code is there once, not once a load in flight: as four
// copies it cost the gradients 20 us of 500 (B2 H32 N8K) in instruction fetches.
template <class G, class F>
__device__ __forceinline__ void for_gates(int n, int lane, G get, F f) {
  __nv_bfloat162 now[4], next[4];
  auto load = [&](int i) {
#pragma unroll
    for (int u = 0; u < 4; ++u) next[u] = __nv_bfloat162(get(i + u, 2 * lane), get(i + u, 2 * lane + 1));
  };
  load(0);
#pragma unroll 1
  for (int i = 0; i < n; i += 4) {
#pragma unroll
    for (int u = 0; u < 4; ++u) now[u] = next[u];
    load(i + 4);
#pragma unroll 1
    for (int u = 0; u < min(4, n - i); ++u) {
      const __nv_bfloat162 g = u < 2 ? (u ? now[1] : now[0]) : (u == 2 ? now[2] : now[3]);
      if (!f(i + u, g.x, g.y)) return;
    }
  }
}

// Launches of one call that do not read one another's results (the two state passes;
// dQ, dV and dK) run side by side: all but the first are `beside` the one before. Such a
// grid does not wait for it at its start: that one let this grid start only once all
// its CTAs had passed their own wait (or were beside theirs), so everything older is
// complete. It waits at its end instead, so that whoever waits for it finds the whole
// group done. (Gradients of B2 H32 N8K 510 -> 487 us, of
// B4 H16 N2K 203 -> 188 us: the launches' tails overlap.)
__device__ __forceinline__ void begin_grid(int beside) {
  if (!beside) pdl_wait();
  pdl_launch_dependents();
}
__device__ __forceinline__ void end_grid(int beside) {
  if (beside) pdl_wait();
}

struct TcParams {
  const __nv_bfloat16* gate;   // [BH][N]
  const float* init;           // [BH][K][128*128] (state_f4): states of the sequence's pieces, or null
  const double* tot;           // [BH][K]: sums of their gates
  float* dots;                 // GRAD: [BH][N]
  float* sum;                  // GRAD, per > 0: [BH][C][128*128], where each chunk leaves the state it starts from
  int64_t N, L, C, spin_limit;
  // Pieces: `per` a chunk; a chunk starts from all pieces before it (walking back:
  // behind it), each decayed over those between. per = 0: init holds one state a
  // chunk, scanned already.
  int32_t K, per;
  int32_t halves;  // 64-column halves of an output row
  int32_t beside;  // the launch before is independent: see begin_grid
};

template <bool GRAD>
struct TcCfg {
  static constexpr int KS = 3;                     // stages of X, Y, Z
  static constexpr int PARTS = GRAD ? 2 : 1;       // bf16 parts of the state's copy (64 columns each)
  static constexpr int OFF_LO = KS * 3 * kTile;    // remainder of Y~
  static constexpr int OFF_P = OFF_LO + kTile;
  static constexpr int OFF_OUT = OFF_P + 2 * 64 * 64 * 2;
  static constexpr int OFF_TAB = OFF_OUT + 2 * kTile;
  static constexpr int OFF_DOT = OFF_TAB + kTabs * kTab * 4;
  static constexpr int OFF_BAR = OFF_DOT + (GRAD ? 2 * 4 * 64 * 4 : 0);
  static constexpr int NBAR = 4 * KS + 3 + 4 + 2 + 3 + 2 + 4 + kTabs + 1;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};
// TMEM columns: the state, its copy (value, remainder), S, two buffers of far, near
constexpr uint32_t kColState = 0, kColCopy = 128, kColS = 256, kColFar = 320, kColNear = 448;

// Packed fp32 pairs (two multiply-adds an instruction: the roles share the issue slots).
__device__ __forceinline__ uint64_t f2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ uint64_t f2(uint32_t x, uint32_t y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ void unpack(uint64_t a, uint32_t& x, uint32_t& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(a));
}
__device__ __forceinline__ void unpack(uint64_t a, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack2(uint64_t a) {  // to bf16
  float x, y;
  unpack(a, x, y);
  return s::pack_bf16x2(x, y);
}
__device__ __forceinline__ uint32_t bfma2(uint32_t a, uint32_t b, uint32_t c) {  // bf16 pairs
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// A factor as two bf16 values, each twice: f = h + l to 2^-17.
struct Factor {
  uint32_t h, l;
};
__device__ __forceinline__ Factor factor(float f) {
  Factor r;
  r.h = s::pack_bf16x2(f, f);
  const float l = f - __uint_as_float(r.h & 0xffff0000u);
  r.l = s::pack_bf16x2(l, l);
  return r;
}
// Two bf16 values times f: the rounded products, and what they are off to 2^-17. The
// remainder of x h against its rounding has at most 8 bits: the second product is exact.
__device__ __forceinline__ void split_scaled(uint32_t x, const Factor& f, uint32_t& hi, uint32_t& lo) {
  hi = bfma2(x, f.h, 0x80008000u);  // (-0: keeps the sign of a zero product)
  lo = bfma2(x, f.l, bfma2(x, f.h, hi ^ 0x80008000u));
}

// Two 8-column fragments of 16 TMEM lanes: thread 4 g + j of the warp gets, of each,
// columns 2 j and 2 j + 1 of lane g and then of lane g + 8.
__device__ __forceinline__ void tmem_ld_frag2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// Four 8 x 8 bf16 matrices, transposed, from and to rows of 16 bytes (lane l: row l % 8 of matrix l / 8).
__device__ __forceinline__ void ldmatrix_t4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stmatrix_t4(uint32_t addr, const uint32_t* r) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

// Thread t of the warp writes 8 consecutive columns of TMEM lane (lane field) + t.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Thread t of the warp reads 16 consecutive columns of TMEM lane (lane field) + t.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

template <bool BACK, bool GRAD>
__global__ void __launch_bounds__(kMainThreads, 1)
gated_sm100_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y,
                   const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_o,
                   const __grid_constant__ CUtensorMap tm_dot, const TcParams prm) {
  using CF = TcCfg<GRAD>;
  constexpr int KS = CF::KS, PARTS = CF::PARTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  // (from lane 0, so that the compiler takes what depends on it as warp-uniform)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int wg = warp >> 2, w4 = warp & 3;

  uint64_t* in_full = reinterpret_cast<uint64_t*>(smem + CF::OFF_BAR);
  uint64_t* in_empty = in_full + KS;
  uint64_t* z_full = in_empty + KS;  // (in: X and Y)
  uint64_t* z_empty = z_full + KS;
  uint64_t* s_full = z_empty + KS;
  uint64_t* s_empty = s_full + 2;
  uint64_t *p_full = s_empty + 1, *p_empty = p_full + 2;
  uint64_t *y_full = p_empty + 2, *y_empty = y_full + 1;
  uint64_t *copy_full = y_empty + 1, *copy_empty = copy_full + 1, *updated = copy_empty + 1;
  uint64_t *o_full = updated + 1, *o_empty = o_full + 1;
  uint64_t *staged = o_empty + 1, *tile_free = staged + 2;
  uint64_t* tab_full = tile_free + 2;
  uint64_t* drain = tab_full + kTabs;
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base + 1);
  float* tab = reinterpret_cast<float*>(smem + CF::OFF_TAB);

  const int64_t bh = blockIdx.x / prm.C, ch = blockIdx.x % prm.C;
  const int64_t t0 = ch * prm.L, t1 = min(prm.N, t0 + prm.L);
  const int n = static_cast<int>((t1 - t0 + 63) / 64);
  const bool has_init = prm.init && (BACK ? ch + 1 < prm.C : ch > 0);
  const int first_copy = has_init ? 0 : 1;  // the first block that has a far part
  auto row_of = [&](int i) { return t0 + static_cast<int64_t>(BACK ? n - 1 - i : i) * 64; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) {
      s::mbar_init(&in_full[i], 1);
      s::mbar_init(&in_empty[i], 1);
      s::mbar_init(&z_full[i], 1);
      s::mbar_init(&z_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      s::mbar_init(&s_full[i], 1);
      s::mbar_init(&p_full[i], 128);
      s::mbar_init(&p_empty[i], 1);
      s::mbar_init(&tile_free[i], 1);
      s::mbar_init(&staged[i], 128);
    }
    s::mbar_init(s_empty, 128);
    s::mbar_init(o_full, 1);
    s::mbar_init(o_empty, 128);
    s::mbar_init(y_full, 128);
    s::mbar_init(y_empty, 1);
    s::mbar_init(copy_full, 256);
    s::mbar_init(copy_empty, 1);
    s::mbar_init(updated, 1);
    for (int i = 0; i < kTabs; ++i) s::mbar_init(&tab_full[i], 32);
    s::mbar_init(drain, 1);
    *abort_flag = 0;
    s::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    s::tma_prefetch(&tm_x);
    s::tma_prefetch(&tm_y);
    s::tma_prefetch(&tm_z);
    s::tma_prefetch(&tm_o);
    if (GRAD) s::tma_prefetch(&tm_dot);
  }
  if (warp == 1) {
    s::tmem_alloc(tmem_base, 512);
    s::tmem_relinquish();
  }
  s::tc_fence_before();
  __syncthreads();
  s::tc_fence_after();
  const uint32_t tmem = *tmem_base;
  const int64_t lim = prm.spin_limit;
  begin_grid(prm.beside);  // global memory is touched only after this point

  auto wait = [&](uint64_t* bar, uint32_t parity, int where) -> bool {
    return __all_sync(0xffffffffu, s::wait_bar(bar, parity, lim, abort_flag, where));
  };
  auto tab_of = [&](int i, int where) -> const float* {  // the block's gate sums, or null after an abort
    return wait(&tab_full[i % kTabs], (i / kTabs) & 1, where) ? tab + (i % kTabs) * kTab : nullptr;
  };
  const uint32_t lane_off = static_cast<uint32_t>(32 * w4) << 16;

  if (warp == 0) {
    // ================================================================ loads
    if (lane == 0) {
      int issued = 0, issued_z = 0;
      for (int i = 0; i < n; ++i) {
        const int st = i % KS, row = static_cast<int>(row_of(i)), z = static_cast<int>(bh);
        uint8_t* dst = smem + st * 3 * kTile;
        if (!s::wait_bar(&in_empty[st], ((i / KS) & 1) ^ 1, lim, abort_flag, 70)) break;
        s::mbar_expect_tx(&in_full[st], 2 * kTile);
        for (int p = 0; p < 2; ++p) s::tma_load_3d(dst + p * 8192, &tm_x, &in_full[st], 64 * p, row, z);
        for (int p = 0; p < 2; ++p) s::tma_load_3d(dst + kTile + p * 8192, &tm_y, &in_full[st], 64 * p, row, z);
        ++issued;
        if (!s::wait_bar(&z_empty[st], ((i / KS) & 1) ^ 1, lim, abort_flag, 87)) break;
        s::mbar_expect_tx(&z_full[st], kTile);
        for (int p = 0; p < 2; ++p) s::tma_load_3d(dst + 2 * kTile + p * 8192, &tm_z, &z_full[st], 64 * p, row, z);
        ++issued_z;
      }
      // Every load lands before the CTA exits, also where another role has given up and
      // nobody else waits for the last ones.
      for (int j = max(0, issued - KS); j < issued; ++j) s::drain_wait(&in_full[j % KS], (j / KS) & 1);
      for (int j = max(0, issued_z - KS); j < issued_z; ++j) s::drain_wait(&z_full[j % KS], (j / KS) & 1);
    }
  } else if (warp == 1) {
    // ================================================================== MMA
    constexpr uint32_t ID_S = s::make_idesc(64, 64, false, false);
    constexpr uint32_t ID_FAR = s::make_idesc(128, 64, false, false);
    constexpr uint32_t ID_UPD = s::make_idesc(128, 128, true, true);
    constexpr uint32_t ID_NEAR = s::make_idesc(128, 64, true, false);
    const uint32_t lead = elect_one();
    const uint32_t base = s::smem_u32(smem);
    // Operand descriptors at their first 16 k: X and Y by rows (S, far), Y~ and Z by
    // columns (update, near) of stage 0; a stage further on is 3 kTile.
    constexpr uint32_t kStage = 3 * kTile / 16, kY = kTile / 16, kZ = 2 * kTile / 16;
    const uint64_t row_d = s::make_desc(base, 16, 1024), col_d = s::make_desc(base, 8192, 1024);
    const uint64_t lo_d = s::make_desc(base + CF::OFF_LO, 8192, 1024), p_d = s::make_desc(base + CF::OFF_P, 16, 1024);
    auto scores = [&](int i) -> bool {  // S of block i
      if (!wait(&in_full[i % KS], (i / KS) & 1, 71)) return false;
      if (!wait(s_empty, (i & 1) ^ 1, 72)) return false;
      s::tc_fence_after();
      const uint32_t st = (i % KS) * kStage;
      mma_run<8>(lead, tmem + kColS, row_d + st, row_d + st + kY, 2, 2, 504, 504, ID_S, 0);
      commit(lead, &s_full[i & 1]);
      return true;
    };
    bool ok = scores(0);
    for (int i = 0; i < n && ok; ++i) {
      const uint32_t st = (i % KS) * kStage;
      const bool far = i >= first_copy;
      ok = false;
      if (i + 1 < n && !scores(i + 1)) break;
      if (!wait(&z_full[i % KS], (i / KS) & 1, 87)) break;
      if (far && !wait(copy_full, (i - first_copy) & 1, 74)) break;
      if (i + 1 < n) {  // the state past the chunk's last block is not needed
        if (!wait(y_full, i & 1, 75)) break;
        s::tc_fence_after();
        mma_run<4>(lead, tmem + kColState, col_d + st + kZ, col_d + st + kY, 128, 128, 0, 0, ID_UPD, far);
        mma_run<4>(lead, tmem + kColState, col_d + st + kZ, lo_d, 128, 128, 0, 0, ID_UPD, 1);
        commit(lead, updated);
        commit(lead, y_empty);
      }
      if (far) {  // (its buffer: the epilogue has read block i - 2, see near of i - 1)
        s::tc_fence_after();
        if (lead) {
#pragma unroll
          for (int k = 0; k < 8 * PARTS; ++k)
            mma_ts(tmem + kColFar + 64 * (i & 1), tmem + kColCopy + 8 * k,
                   row_d + st + ((k & 7) >> 2) * 512 + (k & 3) * 2, ID_FAR, k > 0);
        }
        __syncwarp();
        commit(lead, copy_empty);
      }
      commit(lead, &in_empty[i % KS]);  // X and Y are done with, Z is not
      if (!wait(&p_full[i & 1], (i >> 1) & 1, 76)) break;
      if (!wait(o_empty, (i & 1) ^ 1, 73)) break;  // the epilogue has read near of block i - 1
      s::tc_fence_after();
      mma_run<4>(lead, tmem + kColNear, col_d + st + kZ, p_d + (i & 1) * 512, 128, 2, 0, 0, ID_NEAR, 0);
      commit(lead, o_full);
      commit(lead, &p_empty[i & 1]);
      commit(lead, &z_empty[i % KS]);
      ok = true;
    }
    commit(lead, drain);  // every MMA issued must finish before TMEM is released
    s::drain_wait(drain, 0);
  } else if (warp == 2) {
    // =========================================================== gate tables
    // Per block: the running sums c [64]; the epilogue's factors of far [64]; for
    // the mask, whose rows and columns meet in 16 x 16 squares, e^(c_E(s) - c_s) [64]
    // with E(s) the last row of s' sixteen, and e^(c_t - c_E) for the first three E
    // [3][64] (read for later t only): off the diagonal e^(c_t - c_s) is one of each,
    // neither above 1 unless gates are; the factors of Y~ [64]; and the restarts of each
    // sixteen as bits [4]. Restarts count as 0 in the sums, which keep their digits, and
    // cut the factors: one that spans a restart is 0, however the gates behind it
    // grow; squares on the diagonal go by the bits. Table i goes into slot i % 8 when block i - KS
    // has released its stage (z_empty): everything of it is done but its epilogue,
    // and before its near was issued the epilogue had read block i - KS - 1 (o_empty),
    // so readers of block i - 8 are long done.
    const __nv_bfloat16* g = prm.gate + bh * prm.N;
    for_gates(
        n, lane,
        [&](int i, int r) {
          const int64_t t = row_of(i) + r;
          return i < n && t < t1 ? g[t] : __float2bfloat16(0.f);
        },
        [&](int i, __nv_bfloat16 gx, __nv_bfloat16 gy) {
          // nothing comes before the first token for its gate to pass on: 0, unless NaN (not where it
          // is loaded: four blocks ahead, the warp would wait for it there)
          if (lane == 0 && row_of(i) == 0 && !__hisnan(gx)) gx = __float2bfloat16(0.f);
          const bool cx = is_restart(gx), cy = is_restart(gy);
          const uint32_t ex = __ballot_sync(0xffffffffu, cx), ey = __ballot_sync(0xffffffffu, cy);
          float a, b;
          warp_sums(cx ? 0.f : to_f32(gx) * kLog2e, cy ? 0.f : to_f32(gy) * kLog2e, lane, a, b);
          const float all = __shfl_sync(0xffffffffu, b, 31);
          const float end = __shfl_sync(0xffffffffu, b, lane | 7);
          float2 head = make_float2(ex2(a), ex2(b)), tail = make_float2(ex2(all - a), ex2(all - b));
          float2 to_end = make_float2(ex2(end - a), ex2(end - b)), from_end[3];
#pragma unroll
          for (int h = 0; h < 3; ++h) {
            const float e = __shfl_sync(0xffffffffu, b, 8 * h + 7);
            from_end[h] = make_float2(ex2(a - e), ex2(b - e));
          }
          uint32_t bits = 0;
          if (ex | ey) {
            auto cut = [](float2& f, bool x, bool y) { f = make_float2(x ? 0.f : f.x, y ? 0.f : f.y); };
            const uint32_t own = 0xffu << (lane & 24);  // the row's sixteen
            cut(head, restart_upto(ex, ey, lane, 0), restart_upto(ex, ey, lane, 1));
            cut(tail, restart_behind(ex, ey, lane, 0), restart_behind(ex, ey, lane, 1));
            cut(to_end, restart_behind(ex & own, ey & own, lane, 0), restart_behind(ex & own, ey & own, lane, 1));
#pragma unroll
            for (int h = 0; h < 3; ++h) {
              const uint32_t later = 0xffffff00u << (8 * h);
              cut(from_end[h], restart_upto(ex & later, ey & later, lane, 0), restart_upto(ex & later, ey & later, lane, 1));
            }
            const int byte = 8 * (lane & 3);
            bits = spread_bits(ex >> byte & 0xffu) | spread_bits(ey >> byte & 0xffu) << 1;
          }
          // (the wait last: what it waits for is what the block's mask waits for next)
          if (i >= KS && !wait(&z_empty[i % KS], (i / KS - 1) & 1, 77)) return false;
          float* slot = tab + (i % kTabs) * kTab;
          float2* t = reinterpret_cast<float2*>(slot);
          t[lane] = make_float2(a, b);
          t[32 + lane] = BACK ? tail : head;
          t[64 + lane] = to_end;
#pragma unroll
          for (int h = 0; h < 3; ++h) t[96 + 32 * h + lane] = from_end[h];
          t[192 + lane] = BACK ? head : tail;
          if (lane < 4) reinterpret_cast<uint32_t*>(slot)[448 + lane] = bits;
          s::mbar_arrive(&tab_full[i % kTabs]);
          return true;
        });
  } else if (wg == 4) {
    // ===================================================================== Y~
    // Two threads a row: the value over Y once S has read it, the remainder into its
    // tile once the update of the block before has read that.
    const int r = threadIdx.x & 63, half = (threadIdx.x >> 6) & 1;
    const uint32_t lo_t = s::smem_u32(smem + CF::OFF_LO) + half * 8192 + r * 128;
    for (int i = 0; i + 1 < n; ++i) {
      const float* c = tab_of(i, 78);
      if (!c) break;
      const Factor f = factor(c[384 + r]);
      if (!wait(&s_full[i & 1], (i >> 1) & 1, 79)) break;
      if (!wait(y_empty, (i & 1) ^ 1, 90)) break;
      const uint32_t ya = s::smem_u32(smem + (i % KS) * 3 * kTile + kTile) + half * 8192 + r * 128;
#pragma unroll 2
      for (int ch = 0; ch < 8; ++ch) {
        const uint32_t off = (ch ^ (r & 7)) << 4;
        uint32_t x[4], hi[4], lo[4];
        s::ld_shared_v4(ya + off, x[0], x[1], x[2], x[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) split_scaled(x[e], f, hi[e], lo[e]);
        s::st_shared_v4(ya + off, hi[0], hi[1], hi[2], hi[3]);
        s::st_shared_v4(lo_t + off, lo[0], lo[1], lo[2], lo[3]);
      }
      s::fence_proxy_async();
      s::mbar_arrive(y_full);
    }
  } else if (wg == 1) {
    // ======================================================== S -> P, weighted
    // A warp's 16 rows (lanes 0-15) against the columns in sixteens: h = w4 lies on
    // the diagonal; those beyond it are not kept, and zero in both buffers from the
    // start. The products of weights are taken in one order, (S e^(c_E - c_s))
    // e^(c_t - c_E), whichever of t and s is the row: dQ and dK round alike.
    const int r = s::acc_row<64>(w4, lane);
    const uint32_t prow = s::smem_u32(smem + CF::OFF_P) + (r < 0 ? 0 : r) * 128;
    auto p_at = [&](int buf, int q) { return prow + buf * 8192 + ((q ^ (r & 7)) << 4); };
    if (r >= 0)
      for (int q = 0; q < 16; ++q) s::st_shared_v4(p_at(q >> 3, q & 7), 0u, 0u, 0u, 0u);
    const int h0 = BACK ? w4 : 0, h1 = BACK ? 3 : w4;
    for (int i = 0; i < n; ++i) {
      const float* c = tab_of(i, 80);
      if (!c) break;
      if (!wait(&s_full[i & 1], (i >> 1) & 1, 81)) break;
      s::tc_fence_after();
      if (!wait(&p_empty[i & 1], ((i >> 1) & 1) ^ 1, 82)) break;  // near of block i - 2 has read its P
#pragma unroll 1
      for (int h = h0; h <= h1; ++h) {
        uint32_t v[16], w[8];
        tmem_ld16(tmem + kColS + 16 * h + lane_off, v);
        s::tmem_ld_wait();
        if (r >= 0) {
          if (h == w4) {
            const float cr = c[r];
            const uint32_t kept = kept_bits<BACK>(reinterpret_cast<const uint32_t*>(c)[448 + w4], lane);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int col = 16 * h + 2 * e;
              const float2 cc = *reinterpret_cast<const float2*>(c + col);
              const float wa = ex2(BACK ? cc.x - cr : cr - cc.x), wb = ex2(BACK ? cc.y - cr : cr - cc.y);
              const float a = kept & (1u << (2 * e)) ? __uint_as_float(v[2 * e]) * wa : 0.f;
              const float b = kept & (2u << (2 * e)) ? __uint_as_float(v[2 * e + 1]) * wb : 0.f;
              w[e] = s::pack_bf16x2(a, b);
            }
          } else {
            const float* cols = c + (BACK ? 192 + 64 * w4 : 128) + 16 * h;
            const float f = c[BACK ? 128 + r : 192 + 64 * h + r];
            const uint64_t ff = f2(f, f);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(cols + 2 * e);
              const uint64_t a = f2(v[2 * e], v[2 * e + 1]), b = f2(v[2 * e + 2], v[2 * e + 3]);
              w[e] = pack2(BACK ? mul2(mul2(a, ff), x.x) : mul2(mul2(a, x.x), ff));
              w[e + 1] = pack2(BACK ? mul2(mul2(b, ff), x.y) : mul2(mul2(b, x.y), ff));
            }
          }
          s::st_shared_v4(p_at(i & 1, 2 * h), w[0], w[1], w[2], w[3]);
          s::st_shared_v4(p_at(i & 1, 2 * h + 1), w[4], w[5], w[6], w[7]);
        }
      }
      s::tc_fence_before();
      s::mbar_arrive(s_empty);
      s::fence_proxy_async();
      s::mbar_arrive(&p_full[i & 1]);
    }
  } else if (wg == 2 || wg == 5) {
    // ==================================== the state's bf16 copy, and its decay
    // One warpgroup the first 64 columns, the other the rest.
    const int col0 = wg == 2 ? 0 : 64;
    const int r = 32 * w4 + lane;  // state row
    const uint32_t ts = tmem + kColState + col0 + lane_off, tc = tmem + kColCopy + col0 / 2 + lane_off;
    // 16 columns of row r into the copy, and times f into the state
    auto put = [&](uint32_t (&v)[16], int h, float f, bool keep) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = __uint_as_float(v[2 * e]), b = __uint_as_float(v[2 * e + 1]);
        hi[e] = s::pack_bf16x2(a, b);
        if (PARTS == 2)
          lo[e] = s::pack_bf16x2(a - __uint_as_float(hi[e] << 16), b - __uint_as_float(hi[e] & 0xffff0000u));
      }
      tmem_st8(tc + 8 * h, hi);
      if (PARTS == 2) tmem_st8(tc + 64 + 8 * h, lo);
      if (keep) {
        if (f == 0.f) {  // (a restart drops the state, be it no number)
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = 0u;
        } else {
          const uint64_t ff = f2(f, f);
#pragma unroll
          for (int e = 0; e < 16; e += 2) unpack(mul2(f2(v[e], v[e + 1]), ff), v[e], v[e + 1]);
        }
        s::tmem_st16(ts + h * 16, v);
      }
    };
    auto done = [&]() {
      s::tmem_st_wait();
      s::tc_fence_before();
      s::mbar_arrive(copy_full);
    };
    bool ok = true;
    if (has_init) {
      const float* c = tab_of(0, 83);
      ok = c != nullptr;
      if (ok) {
        // the pieces between this chunk and the sequence's start (walking back: its
        // end), nearest first, each decayed over the nearer ones
        const int pieces = prm.per == 0 ? 1 : static_cast<int>(BACK ? prm.K - (ch + 1) * prm.per : ch * prm.per);
        const float whole = c[BACK ? 447 : 127];  // e^(c_R)
#pragma unroll 1
        for (int h = 0; h < 4; ++h) {
          float x[16];
          uint32_t v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0.f;
          float f = 1.f;
#pragma unroll 1
          for (int j = 0; j < pieces; ++j) {
            const int64_t at = bh * prm.K + (prm.per == 0 ? ch : BACK ? (ch + 1) * prm.per + j : ch * prm.per - 1 - j);
            const float4* src = reinterpret_cast<const float4*>(prm.init + at * 128 * 128);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 y = src[s::state_f4<128>(r, col0 / 4 + h * 4 + q)];
              x[4 * q] = fmaf(f, y.x, x[4 * q]);
              x[4 * q + 1] = fmaf(f, y.y, x[4 * q + 1]);
              x[4 * q + 2] = fmaf(f, y.z, x[4 * q + 2]);
              x[4 * q + 3] = fmaf(f, y.w, x[4 * q + 3]);
            }
            if (j + 1 < pieces) f *= expf(static_cast<float>(prm.tot[at]));
            if (f == 0.f) break;  // (what a restart has dropped may be no number)
          }
          if (GRAD && prm.sum) {
            float4* dst = reinterpret_cast<float4*>(prm.sum + (bh * prm.C + ch) * 128 * 128);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              dst[s::state_f4<128>(r, col0 / 4 + h * 4 + q)] =
                  make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(x[e]);
          put(v, h, whole, n > 1);
        }
        done();
      }
    }
    for (int i = 1; i < n && ok; ++i) {
      const float* c = tab_of(i, 83);
      if (!c) break;
      const float whole = c[BACK ? 447 : 127];
      if (!wait(updated, (i - 1) & 1, 84)) break;
      // far of the block before has read the copy
      if (i > first_copy && !wait(copy_empty, (i - 1 - first_copy) & 1, 88)) break;
      s::tc_fence_after();
#pragma unroll 1
      for (int h = 0; h < 4; ++h) {
        uint32_t v[16];
        tmem_ld16(ts + 16 * h, v);
        s::tmem_ld_wait();
        put(v, h, whole, i + 1 < n);
      }
      done();
    }
  } else if (wg == 3) {
    // =========================================== out = head far + near -> HBM
    // TMEM holds out transposed: lane e (column of the output), 64 columns t. Read in
    // 16 x 8 fragments, thread 4 g + j of the warp has lanes g and g + 8, columns 2 j
    // and 2 j + 1 of each, which is what stmatrix writes, transposed, into the staging
    // tile's rows t (and ldmatrix reads the dots' rows from there in).
    const uint32_t tile = s::smem_u32(smem + CF::OFF_OUT);
    float* dotbuf = reinterpret_cast<float*>(smem + CF::OFF_DOT);
    const int m = lane >> 3, i8 = lane & 7;  // matrix of four, its row, that this lane addresses
    for (int i = 0; i < n; ++i) {
      const bool far = i >= first_copy;
      const float* head = tab_of(i, 85);
      if (!head) break;
      head += 64 + 2 * (lane & 3);
      // the tile: the dots' rows have landed (GRAD), or the store of block i - 2 has read it
      if (!wait(&tile_free[i & 1], ((i >> 1) & 1) ^ (GRAD ? 0 : 1), 89)) break;
      if (!wait(o_full, i & 1, 86)) break;
      s::tc_fence_after();
      uint64_t dot[8];  // columns 8 g + 2 j, + 1 of this thread, summed over its lanes
#pragma unroll
      for (int e = 0; e < 8; ++e) dot[e] = 0;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const uint32_t t_lane = lane_off + (static_cast<uint32_t>(16 * half) << 16);
        const int e8 = 4 * w4 + 2 * half + (m & 1);  // eight columns of the output
        const uint32_t row0 = tile + (i & 1) * kTile + (e8 >> 3) * 8192 + (8 * (m >> 1) + i8) * 128 + (((e8 & 7) ^ i8) << 4);
#pragma unroll
        for (int part = 0; part < 4; ++part) {  // 16 rows of the output
          uint32_t near[8], v[8], x[4], pk[4];
          tmem_ld_frag2(tmem + kColNear + 16 * part + t_lane, near);
          if (far) tmem_ld_frag2(tmem + kColFar + 64 * (i & 1) + 16 * part + t_lane, v);
          if (GRAD) ldmatrix_t4(row0 + part * 2048, x);
          s::tmem_ld_wait();
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const uint64_t hd = *reinterpret_cast<const uint64_t*>(head + 16 * part + 8 * g);
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // lane g, lane g + 8
              uint64_t o = f2(near[4 * g + 2 * e], near[4 * g + 2 * e + 1]);
              if (far) o = fma2(hd, f2(v[4 * g + 2 * e], v[4 * g + 2 * e + 1]), o);
              pk[2 * g + e] = pack2(o);
              if (GRAD) {
                const uint32_t xx = x[2 * g + e];
                dot[2 * part + g] = fma2(o, f2(xx << 16, xx & 0xffff0000u), dot[2 * part + g]);
              }
            }
          }
          stmatrix_t4(row0 + part * 2048, pk);
        }
      }
      s::tc_fence_before();
      s::mbar_arrive(o_empty);
      if (GRAD) {
        // over the eight threads with the same columns: each keeps half at every step
        float d[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) unpack(dot[e], d[2 * e], d[2 * e + 1]);
#pragma unroll
        for (int step = 0; step < 3; ++step) {
          const int keep = 8 >> step, bit = 16 >> step;
          const bool up = lane & bit;
#pragma unroll
          for (int e = 0; e < keep; ++e) {
            const float a = up ? d[e + keep] : d[e], z = up ? d[e] : d[e + keep];
            d[e] = a + __shfl_xor_sync(0xffffffffu, z, bit);
          }
        }
        const int g = (lane >> 4) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
        *reinterpret_cast<float2*>(dotbuf + (i & 1) * 256 + w4 * 64 + 8 * g + 2 * (lane & 3)) = make_float2(d[0], d[1]);
      }
      s::fence_proxy_async();
      s::mbar_arrive(&staged[i & 1]);
    }
  } else if (warp == 3) {
    // ==================================== stores, and the rows of the dots (GRAD)
    // A staging tile: [dots' rows loaded ->] output written (staged) -> store has
    // read it -> free (tile_free: then, or when the dots' rows two blocks on have landed). Each
    // tile has its own staged: with one for both, a pair of blocks that are staged before
    // this warp comes back to wait would look like none. The
    // dots of a block meet here, before its tile and their buffer are free again.
    const float* dotbuf = reinterpret_cast<const float*>(smem + CF::OFF_DOT);
    auto load_dot_rows = [&](int i) {
      uint8_t* dst = smem + CF::OFF_OUT + (i & 1) * kTile;
      s::mbar_expect_tx(&tile_free[i & 1], kTile);
      for (int p = 0; p < 2; ++p)
        s::tma_load_3d(dst + p * 8192, &tm_dot, &tile_free[i & 1], 64 * p, static_cast<int>(row_of(i)), static_cast<int>(bh));
    };
    int issued = 0;
    if (GRAD)
      for (; issued < min(n, 2); ++issued)
        if (lane == 0) load_dot_rows(issued);
    for (int i = 0; i < n; ++i) {
      if (!wait(&staged[i & 1], (i >> 1) & 1, 91)) break;
      if (lane == 0) {
        // A chunk ends on a block boundary or at N, where the tensor map clips.
        for (int p = 0; p < prm.halves; ++p)
          s::tma_store_3d(&tm_o, smem + CF::OFF_OUT + (i & 1) * kTile + p * 8192, 64 * p,
                          static_cast<int>(row_of(i)), static_cast<int>(bh));
        s::bulk_commit_group();
      }
      if (GRAD) {
        const float* db = dotbuf + (i & 1) * 256 + 2 * lane;
        const int64_t row = row_of(i) + 2 * lane;
        float2 a[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) a[w] = *reinterpret_cast<const float2*>(db + 64 * w);
        float* d = prm.dots + bh * prm.N + row;
        if (row < t1) d[0] = (a[0].x + a[1].x) + (a[2].x + a[3].x);
        if (row + 1 < t1) d[1] = (a[0].y + a[1].y) + (a[2].y + a[3].y);
        __syncwarp();
      }
      if (lane == 0) {
        s::bulk_wait_group_read<0>();  // the store has read the tile
        if (!GRAD) s::mbar_arrive(&tile_free[i & 1]);
        else if (i + 2 < n) load_dot_rows(i + 2);
      }
      if (GRAD && i + 2 < n) ++issued;
      __syncwarp();
    }
    if (lane == 0) {
      // loads still in flight after an abort, and the stores, are done before exit
      if (GRAD)
        for (int j = max(0, issued - 2); j < issued; ++j) s::drain_wait(&tile_free[j & 1], (j >> 1) & 1);
      s::bulk_wait_group<0>();
    }
  }

  end_grid(prm.beside);
  s::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    s::tc_fence_after();
    s::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- chunk states
//
// Own state of every piece of L rows (see chunk_state_kernel), SUFFIX false from (k, v), true
// from (q, dO): sum of w_t y_t^T z_t with the weight taken to the piece's end (its
// start), so the accumulator is never decayed: the blocks are walked from that edge,
// and the sum of the gates walked so far goes into the scale of the rows. Y~ is value
// and remainder: a state that only starts chunks is good to 2^-17, well under the
// rounding of the outputs made from it. FULL: a state that the caller receives in fp32 (a
// pool's, after a prefill). Its Y~ is fp32's 24 bits as three bf16 values, the first over Y,
// and the other two have a sum of their own, so that the first's loses no digits to as
// many small addends again (B3 H16 N3001: 7e-7 off, as la2_kv_state's exact products are, in 33 us;
// with value and remainder 4.5e-6 in 28 us). Bound by HBM, where K and V are read once, and, FULL,
// by shared memory (192 KB a block: 1500 cycles against 1350 of HBM). Warps: 0 loads,
// 1 MMA, 2 the rows' factors, 4-11 scale rows (four threads a row) and write the
// state out. Two CTAs an SM: one's scaling (about 1000 cycles a block) runs beside the
// other's waits, loads and MMAs; one CTA with twice the buffers was 1.4 times slower.
constexpr int kStateTab = 68;  // the rows' factors, and whether the block lies beyond a restart
struct StateCfg {
  static constexpr int KS = 2;
  static constexpr int OFF_Y2 = KS * 2 * kTile;            // value and remainder (FULL: two remainders)
  static constexpr int OFF_TAB = OFF_Y2 + 2 * kTile;       // kTabs blocks' tables
  static constexpr int OFF_BAR = OFF_TAB + kTabs * kStateTab * 4;
  static constexpr int NBAR = 2 * KS + 2 + 2 + kTabs;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  static_assert(SMEM <= 113 * 1024, "two CTAs an SM");
};

struct TcStateParams {
  const __nv_bfloat16* gate;
  float* out;      // [BH][K][128*128] (state_f4)
  float* out_t;    // its transpose, or null
  double* tot;     // [BH][K]
  int64_t N, L, K, first, count, spin_limit;  // pieces [first, first + count) of the K of every sequence
  // First piece whose sum this launch writes: the prefixes' and the suffixes' passes walk a
  // piece in opposite orders, which may end on other bits, and run side by side.
  int64_t tot_from;
  int32_t beside;  // the launch before is independent: see begin_grid
};

// A pair as three bf16 values each.
__device__ __forceinline__ void split3(uint64_t x, uint32_t& a, uint32_t& b, uint32_t& c) {
  const uint64_t minus = f2(-1.f, -1.f);
  a = pack2(x);
  x = fma2(f2(a << 16, a & 0xffff0000u), minus, x);
  b = pack2(x);
  c = pack2(fma2(f2(b << 16, b & 0xffff0000u), minus, x));
}

// ROWS_Z: the state's rows are z's columns (what O and dV start from), else y's.
template <bool SUFFIX, bool ROWS_Z, bool FULL>
__global__ void __launch_bounds__(384, 2)
gated_state_sm100_kernel(const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_z,
                         const TcStateParams prm) {
  using CF = StateCfg;
  constexpr int KS = CF::KS;
  constexpr uint32_t kCols = FULL ? 256 : 128;  // (two CTAs an SM share 512)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  // (from lane 0, so that the compiler takes what depends on it as warp-uniform)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  uint64_t* in_full = reinterpret_cast<uint64_t*>(smem + CF::OFF_BAR);
  uint64_t* in_empty = in_full + KS;
  uint64_t* y2_full = in_empty + KS;
  uint64_t* y2_empty = y2_full + 1;
  uint64_t *done = y2_empty + 1, *drain = done + 1;
  uint64_t* tab_full = drain + 1;
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(tab_full + kTabs);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base + 1);
  float* tab = reinterpret_cast<float*>(smem + CF::OFF_TAB);

  const int64_t bh = blockIdx.x / prm.count, ch = prm.first + blockIdx.x % prm.count;
  const int64_t t0 = ch * prm.L, t1 = min(prm.N, t0 + prm.L);
  const int n = static_cast<int>((t1 - t0 + 63) / 64);
  auto row_of = [&](int i) { return t0 + static_cast<int64_t>(SUFFIX ? i : n - 1 - i) * 64; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) { s::mbar_init(&in_full[i], 1); s::mbar_init(&in_empty[i], 1); }
    s::mbar_init(y2_full, 256);
    s::mbar_init(y2_empty, 1);
    for (int i = 0; i < kTabs; ++i) s::mbar_init(&tab_full[i], 32);
    s::mbar_init(done, 1);
    s::mbar_init(drain, 1);
    *abort_flag = 0;
    s::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    s::tma_prefetch(&tm_y);
    s::tma_prefetch(&tm_z);
  }
  if (warp == 1) {
    s::tmem_alloc(tmem_base, kCols);
    s::tmem_relinquish();
  }
  s::tc_fence_before();
  __syncthreads();
  s::tc_fence_after();
  const uint32_t tmem = *tmem_base;
  const int64_t lim = prm.spin_limit;
  begin_grid(prm.beside);
  auto wait = [&](uint64_t* bar, uint32_t parity, int where) -> bool {
    return __all_sync(0xffffffffu, s::wait_bar(bar, parity, lim, abort_flag, where));
  };

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (int i = 0; i < n; ++i) {
        const int st = i % KS;
        if (!s::wait_bar(&in_empty[st], ((i / KS) & 1) ^ 1, lim, abort_flag, 90)) break;
        const int row = static_cast<int>(row_of(i)), z = static_cast<int>(bh);
        uint8_t* dst = smem + st * 2 * kTile;
        s::mbar_expect_tx(&in_full[st], 2 * kTile);
        for (int p = 0; p < 2; ++p) s::tma_load_3d(dst + p * 8192, &tm_y, &in_full[st], 64 * p, row, z);
        for (int p = 0; p < 2; ++p) s::tma_load_3d(dst + kTile + p * 8192, &tm_z, &in_full[st], 64 * p, row, z);
        ++issued;
      }
      // (every load lands before the CTA exits, whoever has given up)
      for (int j = max(0, issued - KS); j < issued; ++j) s::drain_wait(&in_full[j % KS], (j / KS) & 1);
    }
  } else if (warp == 1) {
    constexpr uint32_t ID_UPD = s::make_idesc(128, 128, true, true);
    const uint32_t lead = elect_one();
    const uint64_t in_d = s::make_desc(s::smem_u32(smem), 8192, 1024);
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      ok = wait(&in_full[i % KS], (i / KS) & 1, 91) && wait(y2_full, i & 1, 92);
      if (!ok) break;
      s::tc_fence_after();
      if (tab[(i % kTabs) * kStateTab + 64] != 0.f) {  // beyond a restart: nothing to add, be it no number
        commit(lead, y2_empty);
        commit(lead, &in_empty[i % KS]);
        continue;
      }
      const uint64_t y2 = in_d + CF::OFF_Y2 / 16, y = in_d + (i % KS) * 2 * kTile / 16, z = y + kTile / 16;
      const uint64_t lo = y2 + kTile / 16;
      if constexpr (FULL) {
        mma_run<4>(lead, tmem, y, z, 128, 128, 0, 0, ID_UPD, i > 0);
        mma_run<4>(lead, tmem + 128, y2, z, 128, 128, 0, 0, ID_UPD, i > 0);
        mma_run<4>(lead, tmem + 128, lo, z, 128, 128, 0, 0, ID_UPD, 1);
      } else {
        mma_run<4>(lead, tmem, ROWS_Z ? z : y2, ROWS_Z ? y2 : z, 128, 128, 0, 0, ID_UPD, i > 0);
        mma_run<4>(lead, tmem, ROWS_Z ? z : lo, ROWS_Z ? lo : z, 128, 128, 0, 0, ID_UPD, 1);
      }
      commit(lead, y2_empty);
      commit(lead, &in_empty[i % KS]);
    }
    if (ok) commit(lead, done);
    commit(lead, drain);
    s::drain_wait(drain, 0);
  } else if (warp == 2) {
    // the rows' factors, a block's when block i - KS has released its stage. Each is the
    // exponential of a sum over the gates between the row and the piece's edge alone
    // (walking from the end: those behind the row), so no large sums are subtracted, and 0 beyond
    // a restart: as a large negative gate in those sums it would cost them their digits.
    const __nv_bfloat16* g = prm.gate + bh * prm.N;
    double run = 0.0;   // sum of the gates of the blocks walked
    bool dead = false;  // a restart among them: nothing further reaches the edge
    for_gates(
        n, lane,
        [&](int i, int r) {
          const int64_t t = row_of(i) + r;
          return i < n && t < t1 ? g[t] : __float2bfloat16(0.f);
        },
        [&](int i, __nv_bfloat16 gx, __nv_bfloat16 gy) {
          if (i >= KS && !wait(&in_empty[i % KS], (i / KS - 1) & 1, 96)) return false;
          const bool cx = is_restart(gx), cy = is_restart(gy);
          const uint32_t ex = __ballot_sync(0xffffffffu, cx), ey = __ballot_sync(0xffffffffu, cy);
          const float x = cx ? 0.f : to_f32(gx) * kLog2e, y = cy ? 0.f : to_f32(gy) * kLog2e;
          float a, b, all;
          bool za, zb;
          if constexpr (SUFFIX) {
            warp_sums(x, y, lane, a, b);
            all = __shfl_sync(0xffffffffu, b, 31);
            za = restart_upto(ex, ey, lane, 0);
            zb = restart_upto(ex, ey, lane, 1);
          } else {
            warp_sums_behind(x, y, lane, a, b, all);
            // (NaN among the gates reaches every row, as it does in the sum of all)
            a += 0.f * all;
            b += 0.f * all;
            za = restart_behind(ex, ey, lane, 0);
            zb = restart_behind(ex, ey, lane, 1);
          }
          float* slot = tab + (i % kTabs) * kStateTab;
          if (lane == 0) slot[64] = dead;
          reinterpret_cast<float2*>(slot)[lane] =
              make_float2(dead || za ? 0.f : ex2(static_cast<float>(run + static_cast<double>(a))),
                          dead || zb ? 0.f : ex2(static_cast<float>(run + static_cast<double>(b))));
          run += static_cast<double>(all);
          dead |= (ex | ey) != 0;
          s::mbar_arrive(&tab_full[i % kTabs]);
          return true;
        });
    // (natural log; -infinity: its exponential is 0 whatever gates above 0 the piece has)
    if (lane == 0 && ch >= prm.tot_from) prm.tot[bh * prm.K + ch] = dead ? -INFINITY : run * 0.693147180559945309417;
  } else if (warp >= 4) {
    const int r = (warp - 4) * 8 + (lane >> 2), ch0 = (lane & 3) * 4;
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      ok = wait(&tab_full[i % kTabs], (i / kTabs) & 1, 97) && wait(&in_full[i % KS], (i / KS) & 1, 93) &&
           wait(y2_empty, (i & 1) ^ 1, 94);
      if (!ok) break;
      const float factor_r = tab[(i % kTabs) * kStateTab + r];
      const Factor f = factor(factor_r);
      const uint32_t y2 = s::smem_u32(smem + CF::OFF_Y2);
      const uint32_t ya = s::smem_u32(smem + (i % KS) * 2 * kTile);
#pragma unroll
      for (int ch = ch0; ch < ch0 + 4; ++ch) {
        const uint32_t off = (ch >> 3) * 8192 + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
        uint32_t x[4], hi[4], lo[4];
        s::ld_shared_v4(ya + off, x[0], x[1], x[2], x[3]);
        if constexpr (FULL) {
          uint32_t mid[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            split3(mul2(f2(x[e] << 16, x[e] & 0xffff0000u), f2(factor_r, factor_r)), hi[e], mid[e], lo[e]);
          s::st_shared_v4(ya + off, hi[0], hi[1], hi[2], hi[3]);
          s::st_shared_v4(y2 + off, mid[0], mid[1], mid[2], mid[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) split_scaled(x[e], f, hi[e], lo[e]);
          s::st_shared_v4(y2 + off, hi[0], hi[1], hi[2], hi[3]);
        }
        s::st_shared_v4(y2 + kTile + off, lo[0], lo[1], lo[2], lo[3]);
      }
      s::fence_proxy_async();
      s::mbar_arrive(y2_full);
    }
    if (ok && wait(done, 0, 95)) {  // warps 4-7 the first 64 columns, 8-11 the others
      s::tc_fence_after();
      const int row = 32 * (warp & 3) + lane;
      float4* dst = reinterpret_cast<float4*>(prm.out + (bh * prm.K + ch) * 128 * 128);
      float* dst_t = prm.out_t ? prm.out_t + (bh * prm.K + ch) * 128 * 128 + (row >> 2) * 512 + (row & 3) : nullptr;
#pragma unroll 1
      for (int c32 = warp < 8 ? 0 : 2; c32 < (warp < 8 ? 2 : 4); ++c32) {
        uint32_t v[32];
        const uint32_t at = tmem + c32 * 32 + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        s::tmem_ld32(at, v);
        s::tmem_ld_wait();
        if constexpr (FULL) {
          uint32_t u[32];
          s::tmem_ld32(at + 128, u);
          s::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(u[e]));
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          dst[s::state_f4<128>(row, c32 * 8 + q)] =
              make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                          __uint_as_float(v[4 * q + 3]));
        if (dst_t)
#pragma unroll
          for (int e = 0; e < 32; ++e) dst_t[(c32 * 32 + e) * 4] = __uint_as_float(v[e]);
      }
    }
  }

  end_grid(prm.beside);
  s::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    s::tc_fence_after();
    s::tmem_dealloc(tmem, kCols);
  }
}

// -------------------------------------------------------------------- launches

// A [BH, N, w] tensor and its map (64 rows x 64 columns a copy), made once a call.
struct Tile {
  CUtensorMap map;
  int w;
  bool ok;
  Tile(const void* base, int64_t BH, int64_t N, int w_) : w(w_), ok(make_tmap_3d(&map, base, BH, N, w_, 64)) {}
};

template <bool SUFFIX, bool ROWS_Z, bool FULL>
inline cudaError_t launch_state_sm100(const Tile& y, const Tile& z, const TcStateParams& p, int64_t BH, cudaStream_t st) {
  if (!y.ok || !z.ok) return cudaErrorInvalidValue;
  auto kern = gated_state_sm100_kernel<SUFFIX, ROWS_Z, FULL>;
  static bool done[128];
  if (!smem_attribute_set(kern, StateCfg::SMEM, done)) return cudaErrorInvalidValue;
  return launch_pdl(kern, dim3((unsigned)(BH * p.count)), dim3(384), StateCfg::SMEM, st, y.map, z.map, p);
}

// dot_rows: GRAD (else any).
template <bool BACK, bool GRAD>
inline cudaError_t launch_sm100(const Tile& x, const Tile& y, const Tile& z, const Tile& o, const Tile& dot_rows,
                                TcParams p, int64_t BH, cudaStream_t st) {
  if (!x.ok || !y.ok || !z.ok || !o.ok || !dot_rows.ok) return cudaErrorInvalidValue;
  p.halves = o.w / 64;
  auto kern = gated_sm100_kernel<BACK, GRAD>;
  static bool done[128];
  if (!smem_attribute_set(kern, TcCfg<GRAD>::SMEM, done)) return cudaErrorInvalidValue;
  return launch_pdl(kern, dim3((unsigned)(BH * p.C)), dim3(kMainThreads), TcCfg<GRAD>::SMEM, st, x.map, y.map, z.map,
                    o.map, dot_rows.map, p);
}

}  // namespace gated
}  // namespace la2
