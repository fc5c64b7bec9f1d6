// Tensor-core kernels of the gated recurrence (bf16, d = dv = 128, sm_100a); the
// formulas are at the top of la2_gated_simt.cuh. The PTX wrappers, operand
// descriptors, bounded waits and TMEM layouts are those of la2_sm100.cuh.
//
// One kernel does all four products of a layer, as out_t = sum over the kept s of
// w(t, s) (x_t . y_s) z_s with (x, y, z) in the query, key and value places:
//
//             x   y   z    walk      kept     w                  state (c x e)
//   O         q   k   v    forward   s <= t   e^(c_t - c_s)      KV = k^T v
//   dQ        dO  v   k    forward   s <= t   e^(c_t - c_s)      KV, read transposed
//   dV        k   q   dO   back      s >= t   e^(c_s - c_t)      U = q^T dO
//   dK        v   dO  q    back      s >= t   e^(c_s - c_t)      U, read transposed
//
// Per block of 64 rows, walking a chunk of one (b, h) sequence in one CTA:
//   S     = X Y^T                      tcgen05 -> TMEM
//   P     = bf16(S w)                  mask warps, TMEM -> shared memory
//   near  = P Z                        tcgen05 -> TMEM
//   far   = X state                    tcgen05 -> TMEM, from a bf16 copy of the state
//   out   = head far + near            epilogue warps: the row's e^(c_t) (walking
//                                      back e^(c_R - c_t)) is applied in fp32
//   state <- e^(c_R) state + Y~^T Z    tcgen05, Y~ = bf16 rows scaled by e^(c_R - c_s)
//                                      (walking back e^(c_s))
// X and Y stay unscaled in shared memory: Y~ is a copy that two warps make as soon
// as the tile has landed, off the path S -> P -> near, and X needs no scaling since
// far and near are separate accumulators. The state stays in TMEM: the state warps
// read it once a block, write its bf16 copy and put e^(c_R) times it back, which the
// block's update adds onto. S of the next block is issued before P of this one is
// waited for.
//
// Gate sums: c in base 2, fp32, at most 64 terms; a log gate under kLog2Zero (in
// base 2) counts as that, its exponential is 0, so a restart cuts exactly and costs
// the differences of later sums at most 2^-17 * (number of restarts in the block).
//
// GRAD (dQ, dK) also returns the rows' dots q . dq and k . dk (fp32, from the
// unrounded rows) for the gates' gradient, a running difference of them: their
// errors have to cancel over a chunk. P is rounded alike in both passes (the same
// products, the same weights), so the near parts agree; for the far parts the state's
// copy and Y~ are kept as two bf16 tiles, value and remainder (2^-17 instead of 2^-9;
// a second MMA each, into the same accumulator).
#pragma once

#include "la2_gated_simt.cuh"
#include "la2_sm100.cuh"

namespace la2 {
namespace gated {

namespace s = sm100;

constexpr int kTile = 64 * 128 * 2;       // one 64 x 128 bf16 tile
constexpr int kCopy = 128 * 128 * 2;      // the state's bf16 copy
constexpr float kLog2Zero = -160.f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kTabs = 4;                  // gate tables in flight (see the table warp)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A log gate in base 2. A comparison, not fmaxf: NaN stays NaN.
__device__ __forceinline__ float gate_log2(__nv_bfloat16 x) {
  const float y = to_f32(x) * kLog2e;
  return y < kLog2Zero ? kLog2Zero : y;
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
  a = t - y;
  // (a from b would be NaN - NaN or lose y's digits next to a restart)
  const float before = __shfl_up_sync(0xffffffffu, t, 1);
  a = (lane ? before : 0.f) + x;
}

struct TcParams {
  const __nv_bfloat16* gate;   // [BH][N]
  const float* init;           // [BH][C][128*128] (state_f4): state next to each chunk, or null
  const __nv_bfloat16* dot_x;  // GRAD: [BH][N][128], the rows of the dots
  float* dots;                 // GRAD: [BH][N]
  int64_t N, L, C, spin_limit;
};

template <bool GRAD>
struct TcCfg {
  static constexpr int KS = GRAD ? 2 : 3;          // stages of X, Y, Z
  static constexpr int PARTS = GRAD ? 2 : 1;       // bf16 tiles of Y~ and of the state's copy
  static constexpr int OFF_Y2 = KS * 3 * kTile;
  static constexpr int OFF_P = OFF_Y2 + PARTS * kTile;
  static constexpr int OFF_COPY = OFF_P + 64 * 64 * 2;
  static constexpr int OFF_OUT = OFF_COPY + PARTS * kCopy;
  static constexpr int OFF_TAB = OFF_OUT + kTile;
  static constexpr int OFF_BAR = OFF_TAB + kTabs * 64 * 4;
  static constexpr int NBAR = 2 * KS + 2 + 2 + 2 + 2 + 2 + 2 + kTabs + 1;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};
// TMEM columns
constexpr uint32_t kColState = 0, kColFar = 128, kColNear = 256, kColS = 384;  // S: two buffers of 64

// Row r of a [64 x 128] swizzled tile times f: the value, and with two parts its remainder.
template <int PARTS>
__device__ __forceinline__ void scaled_copy(uint32_t src, uint32_t dst, int r, float f, int ch0, int n) {
#pragma unroll 4
  for (int ch = ch0; ch < ch0 + n; ++ch) {
    const uint32_t off = (ch >> 3) * 64 * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
    uint32_t x[4], hi[4], lo[4];
    s::ld_shared_v4(src + off, x[0], x[1], x[2], x[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = __uint_as_float(x[e] << 16) * f, b = __uint_as_float(x[e] & 0xffff0000u) * f;
      hi[e] = s::pack_bf16x2(a, b);
      if (PARTS == 2)
        lo[e] = s::pack_bf16x2(a - __uint_as_float(hi[e] << 16), b - __uint_as_float(hi[e] & 0xffff0000u));
    }
    s::st_shared_v4(dst + off, hi[0], hi[1], hi[2], hi[3]);
    if (PARTS == 2) s::st_shared_v4(dst + kTile + off, lo[0], lo[1], lo[2], lo[3]);
  }
}

template <bool BACK, bool GRAD>
__global__ void __launch_bounds__(512, 1)
gated_sm100_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_y,
                   const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_o,
                   const TcParams prm) {
  using CF = TcCfg<GRAD>;
  constexpr int KS = CF::KS, PARTS = CF::PARTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wg = warp >> 2, w4 = warp & 3;

  uint64_t* in_full = reinterpret_cast<uint64_t*>(smem + CF::OFF_BAR);
  uint64_t* in_empty = in_full + KS;
  uint64_t* s_full = in_empty + KS;
  uint64_t* s_empty = s_full + 2;
  uint64_t *p_full = s_empty + 2, *p_empty = p_full + 1;
  uint64_t *y2_full = p_empty + 1, *y2_empty = y2_full + 1;
  uint64_t *copy_full = y2_empty + 1, *updated = copy_full + 1;
  uint64_t *o_full = updated + 1, *o_empty = o_full + 1;
  uint64_t* tab_full = o_empty + 1;
  uint64_t* drain = tab_full + kTabs;
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base + 1);
  float* tab = reinterpret_cast<float*>(smem + CF::OFF_TAB);

  const int64_t bh = blockIdx.x / prm.C, ch = blockIdx.x % prm.C;
  const int64_t t0 = ch * prm.L, t1 = min(prm.N, t0 + prm.L);
  const int n = static_cast<int>((t1 - t0 + 63) / 64);
  const bool has_init = prm.init && (BACK ? ch + 1 < prm.C : ch > 0);
  auto row_of = [&](int i) { return t0 + static_cast<int64_t>(BACK ? n - 1 - i : i) * 64; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) { s::mbar_init(&in_full[i], 1); s::mbar_init(&in_empty[i], 1); }
    for (int i = 0; i < 2; ++i) { s::mbar_init(&s_full[i], 1); s::mbar_init(&s_empty[i], 128); }
    s::mbar_init(p_full, 128);
    s::mbar_init(p_empty, 1);
    s::mbar_init(y2_full, 64);
    s::mbar_init(y2_empty, 1);
    s::mbar_init(copy_full, 128);
    s::mbar_init(updated, 1);
    s::mbar_init(o_full, 1);
    s::mbar_init(o_empty, 128);
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
  pdl_launch_dependents();  // global memory is touched only after this point
  pdl_wait();

  auto wait = [&](uint64_t* bar, uint32_t parity, int where) -> bool {
    return __all_sync(0xffffffffu, s::wait_bar(bar, parity, lim, abort_flag, where));
  };
  auto tab_of = [&](int i, int where) -> const float* {  // the block's gate sums, or null after an abort
    return wait(&tab_full[i % kTabs], (i / kTabs) & 1, where) ? tab + (i % kTabs) * 64 : nullptr;
  };
  const uint32_t lane_off = static_cast<uint32_t>(32 * w4) << 16;

  if (warp == 0) {
    // ================================================================ loads
    if (lane == 0) {
      int issued = 0;
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int st = i % KS;
        if (!s::wait_bar(&in_empty[st], ((i / KS) & 1) ^ 1, lim, abort_flag, 70)) { ok = false; break; }
        const int row = static_cast<int>(row_of(i)), z = static_cast<int>(bh);
        uint8_t* dst = smem + st * 3 * kTile;
        s::mbar_expect_tx(&in_full[st], 3 * kTile);
        for (int p = 0; p < 2; ++p) s::tma_load_3d(dst + p * 8192, &tm_x, &in_full[st], 64 * p, row, z);
        for (int p = 0; p < 2; ++p) s::tma_load_3d(dst + kTile + p * 8192, &tm_y, &in_full[st], 64 * p, row, z);
        for (int p = 0; p < 2; ++p) s::tma_load_3d(dst + 2 * kTile + p * 8192, &tm_z, &in_full[st], 64 * p, row, z);
        ++issued;
      }
      if (!ok)  // let every load this thread issued land before the CTA exits
        for (int j = max(0, issued - KS); j < issued; ++j) s::drain_wait(&in_full[j % KS], (j / KS) & 1);
    }
  } else if (warp == 1) {
    // ================================================================== MMA
    constexpr uint32_t ID_S = s::make_idesc(64, 64, false, false);
    constexpr uint32_t ID_FAR = s::make_idesc(64, 128, false, !GRAD);  // GRAD: the state read transposed
    constexpr uint32_t ID_UPD = s::make_idesc(128, 128, true, true);
    constexpr uint32_t ID_NEAR = s::make_idesc(64, 128, false, true);
    const uint32_t base = s::smem_u32(smem);
    const uint32_t y2 = base + CF::OFF_Y2, pa = base + CF::OFF_P, cp = base + CF::OFF_COPY;
    auto scores = [&](int i) -> bool {  // S of block i
      if (!wait(&in_full[i % KS], (i / KS) & 1, 71)) return false;
      if (!wait(&s_empty[i & 1], ((i >> 1) & 1) ^ 1, 72)) return false;
      s::tc_fence_after();
      const uint32_t xa = base + (i % KS) * 3 * kTile, ya = xa + kTile;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t off = (k >> 2) * 8192 + (k & 3) * 32;
        s::mma_bf16_ss_warp(tmem + kColS + 64 * (i & 1), s::make_desc(xa + off, 16, 1024),
                            s::make_desc(ya + off, 16, 1024), ID_S, k > 0);
      }
      s::mma_commit_warp(&s_full[i & 1]);
      return true;
    };
    int copies = 0;
    bool ok = scores(0);
    for (int i = 0; i < n && ok; ++i) {
      const uint32_t xa = base + (i % KS) * 3 * kTile, za = xa + 2 * kTile;
      const bool far = i > 0 || has_init;
      ok = false;
      if (!wait(o_empty, (i & 1) ^ 1, 73)) break;
      if (far) {
        if (!wait(copy_full, copies & 1, 74)) break;
        ++copies;
        s::tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8 * PARTS; ++k) {
          const uint32_t a = xa + ((k & 7) >> 2) * 8192 + (k & 3) * 32;
          const uint32_t b = cp + (k >> 3) * kCopy;
          const uint64_t bd = GRAD ? s::make_desc(b + ((k & 7) >> 2) * 16384 + (k & 3) * 32, 16, 1024)
                                   : s::make_desc(b + (k & 7) * 2048, 16384, 1024);
          s::mma_bf16_ss_warp(tmem + kColFar, s::make_desc(a, 16, 1024), bd, ID_FAR, k > 0);
        }
      }
      if (i + 1 < n) {  // the state past the chunk's last block is not needed
        if (!wait(y2_full, i & 1, 75)) break;
        s::tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4 * PARTS; ++k) {
          const uint64_t yd = s::make_desc(y2 + (k >> 2) * kTile + (k & 3) * 2048, 8192, 1024);
          const uint64_t zd = s::make_desc(za + (k & 3) * 2048, 8192, 1024);
          s::mma_bf16_ss_warp(tmem + kColState, GRAD ? zd : yd, GRAD ? yd : zd, ID_UPD, far || k > 0);
        }
        s::mma_commit_warp(updated);
        s::mma_commit_warp(y2_empty);
        if (!scores(i + 1)) break;
      }
      if (!wait(p_full, i & 1, 76)) break;
      s::tc_fence_after();
#pragma unroll
      for (int k = 0; k < 4; ++k)
        s::mma_bf16_ss_warp(tmem + kColNear, s::make_desc(pa + k * 32, 16, 1024),
                            s::make_desc(za + k * 2048, 8192, 1024), ID_NEAR, k > 0);
      s::mma_commit_warp(o_full);
      s::mma_commit_warp(p_empty);
      s::mma_commit_warp(&in_empty[i % KS]);
      ok = true;
    }
    s::mma_commit_warp(drain);  // every MMA issued must finish before TMEM is released
    s::drain_wait(drain, 0);
  } else if (warp < 4) {
    // ============================================ gate tables (warp 2) and Y~
    // Table i goes into slot i % 4. Warp 2 writes it after its Y~ of block i - 1,
    // which waited for the update of block i - 2, which is issued after everything
    // of block i - 3 but its epilogue's reads, and after those (o_empty): the slot's
    // last readers, of block i - 4, are done.
    const int r = threadIdx.x - 64;
    const __nv_bfloat16* g = prm.gate + bh * prm.N;
    auto gate_at = [&](int64_t t) { return t < t1 ? g[t] : __float2bfloat16(0.f); };
    __nv_bfloat16 gx = gate_at(row_of(0) + 2 * lane), gy = gate_at(row_of(0) + 2 * lane + 1);
    for (int i = 0; i < n; ++i) {
      if (warp == 2) {
        float a, b;
        warp_sums(gate_log2(gx), gate_log2(gy), lane, a, b);
        reinterpret_cast<float2*>(tab + (i % kTabs) * 64)[lane] = make_float2(a, b);
        s::mbar_arrive(&tab_full[i % kTabs]);
        if (i + 1 < n) {
          gx = gate_at(row_of(i + 1) + 2 * lane);
          gy = gate_at(row_of(i + 1) + 2 * lane + 1);
        }
      }
      if (i + 1 == n) break;
      const float* c = tab_of(i, 77);
      if (!c) break;
      if (!wait(&in_full[i % KS], (i / KS) & 1, 78)) break;
      if (!wait(y2_empty, (i & 1) ^ 1, 79)) break;
      const float f = ex2(BACK ? c[r] : c[63] - c[r]);
      scaled_copy<PARTS>(s::smem_u32(smem + (i % KS) * 3 * kTile + kTile), s::smem_u32(smem + CF::OFF_Y2), r, f, 0, 16);
      s::fence_proxy_async();
      s::mbar_arrive(y2_full);
    }
  } else if (wg == 1) {
    // ======================================================== S -> P, weighted
    const int r = s::acc_row<64>(w4, lane);
    const uint32_t pbase = s::smem_u32(smem + CF::OFF_P);
    for (int i = 0; i < n; ++i) {
      const float* c = tab_of(i, 80);
      if (!c) break;
      const float cr = r >= 0 ? c[r] : 0.f;
      if (!wait(&s_full[i & 1], (i >> 1) & 1, 81)) break;
      s::tc_fence_after();
      uint32_t w[32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
        s::tmem_ld32(tmem + kColS + 64 * (i & 1) + 32 * h + lane_off, v);
        s::tmem_ld_wait();
        if (r >= 0) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int col = 32 * h + 2 * e;
            const float2 cc = *reinterpret_cast<const float2*>(c + col);
            const float wa = ex2(BACK ? cc.x - cr : cr - cc.x), wb = ex2(BACK ? cc.y - cr : cr - cc.y);
            const float a = (BACK ? col >= r : col <= r) ? __uint_as_float(v[2 * e]) * wa : 0.f;
            const float b = (BACK ? col + 1 >= r : col + 1 <= r) ? __uint_as_float(v[2 * e + 1]) * wb : 0.f;
            w[16 * h + e] = s::pack_bf16x2(a, b);
          }
        }
      }
      s::tc_fence_before();
      s::mbar_arrive(&s_empty[i & 1]);
      if (!wait(p_empty, (i & 1) ^ 1, 82)) break;  // near of the block before has read P
      if (r >= 0)
#pragma unroll
        for (int q = 0; q < 8; ++q)
          s::st_shared_v4(pbase + r * 128 + ((q ^ (r & 7)) << 4), w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
      s::fence_proxy_async();
      s::mbar_arrive(p_full);
    }
  } else if (wg == 2) {
    // ==================================== the state's bf16 copy, and its decay
    const int r = 32 * w4 + lane;  // state row
    const uint32_t ts = tmem + kColState + lane_off;
    const uint32_t cbase = s::smem_u32(smem + CF::OFF_COPY);
    const float4* init =
        has_init ? reinterpret_cast<const float4*>(prm.init + static_cast<int64_t>(blockIdx.x) * 128 * 128) : nullptr;
    for (int i = has_init ? 0 : 1; i < n; ++i) {
      const float* c = tab_of(i, 83);
      if (!c) break;
      const float whole = ex2(c[63]);
      if (i > 0) {
        if (!wait(updated, (i - 1) & 1, 84)) break;
        s::tc_fence_after();
      }
#pragma unroll
      for (int c32 = 0; c32 < 4; ++c32) {
        uint32_t v[32];
        if (i == 0) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 x = init[s::state_f4<128>(r, c32 * 8 + q)];
            v[4 * q] = __float_as_uint(x.x);
            v[4 * q + 1] = __float_as_uint(x.y);
            v[4 * q + 2] = __float_as_uint(x.z);
            v[4 * q + 3] = __float_as_uint(x.w);
          }
        } else {
          s::tmem_ld32(ts + c32 * 32, v);
          s::tmem_ld_wait();
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t off = (c32 >> 1) * 16384 + r * 128 + ((((c32 & 1) * 4 + q) ^ (r & 7)) << 4);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = __uint_as_float(v[8 * q + 2 * e]), b = __uint_as_float(v[8 * q + 2 * e + 1]);
            hi[e] = s::pack_bf16x2(a, b);
            if (PARTS == 2)
              lo[e] = s::pack_bf16x2(a - __uint_as_float(hi[e] << 16), b - __uint_as_float(hi[e] & 0xffff0000u));
          }
          s::st_shared_v4(cbase + off, hi[0], hi[1], hi[2], hi[3]);
          if (PARTS == 2) s::st_shared_v4(cbase + kCopy + off, lo[0], lo[1], lo[2], lo[3]);
        }
        if (i + 1 < n) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(whole * __uint_as_float(v[e]));
          s::tmem_st32(ts + c32 * 32, v);
        }
      }
      s::tmem_st_wait();
      s::fence_proxy_async();
      s::tc_fence_before();
      s::mbar_arrive(copy_full);
    }
  } else {
    // =========================================== out = head far + near -> HBM
    const int r = s::acc_row<64>(w4, lane);
    const int rl = lane & 15;
    uint8_t* stage = smem + CF::OFF_OUT + w4 * 16 * 128;
    for (int i = 0; i < n; ++i) {
      const bool far = i > 0 || has_init;
      const int64_t row = row_of(i) + r;
      const bool valid = r >= 0 && row < t1;
      const uint4* xr = GRAD ? reinterpret_cast<const uint4*>(prm.dot_x + (bh * prm.N + (valid ? row : t0)) * 128) : nullptr;
      uint4 x[4];
      if (GRAD && valid)
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = xr[q];
      const float* c = tab_of(i, 85);
      if (!c) break;
      const float head = r >= 0 && far ? ex2(BACK ? c[63] - c[r] : c[r]) : 0.f;
      if (!wait(o_full, i & 1, 86)) break;
      s::tc_fence_after();
      if (lane == 0) s::bulk_wait_group_read<0>();  // the store of the block before has read the stage
      __syncwarp();
      float dot = 0.f;
#pragma unroll
      for (int c32 = 0; c32 < 4; ++c32) {
        uint32_t near[32], v[32];
        s::tmem_ld32(tmem + kColNear + c32 * 32 + lane_off, near);
        if (far) s::tmem_ld32(tmem + kColFar + c32 * 32 + lane_off, v);
        s::tmem_ld_wait();
        if (r >= 0) {
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = far ? fmaf(head, __uint_as_float(v[e]), __uint_as_float(near[e])) : __uint_as_float(near[e]);
          if (GRAD) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t u[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                dot = fmaf(o[8 * q + 2 * e], __uint_as_float(u[e] << 16), dot);
                dot = fmaf(o[8 * q + 2 * e + 1], __uint_as_float(u[e] & 0xffff0000u), dot);
              }
              if (valid && c32 < 3) x[q] = xr[4 * (c32 + 1) + q];
            }
          }
          const uint32_t base = s::smem_u32(stage + (c32 >> 1) * 8192) + rl * 128;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            s::st_shared_v4(base + ((((c32 & 1) * 4 + q) ^ (rl & 7)) << 4), s::pack_bf16x2(o[8 * q], o[8 * q + 1]),
                            s::pack_bf16x2(o[8 * q + 2], o[8 * q + 3]), s::pack_bf16x2(o[8 * q + 4], o[8 * q + 5]),
                            s::pack_bf16x2(o[8 * q + 6], o[8 * q + 7]));
        }
      }
      s::tc_fence_before();
      s::mbar_arrive(o_empty);
      if (GRAD && valid) prm.dots[bh * prm.N + row] = dot;
      s::fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        // A chunk ends on a block boundary or at N, where the tensor map clips.
        const int64_t y = row_of(i) + 16 * w4;
        if (y < t1)
          for (int p = 0; p < 2; ++p)
            s::tma_store_3d(&tm_o, stage + p * 8192, 64 * p, static_cast<int>(y), static_cast<int>(bh));
        s::bulk_commit_group();
      }
    }
    if (lane == 0) s::bulk_wait_group<0>();  // stores done before exit
  }

  s::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    s::tc_fence_after();
    s::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- chunk states
//
// Own state of every chunk (see chunk_state_kernel), SUFFIX false from (k, v), true
// from (q, dO): sum of w_t y_t^T z_t with the weight taken to the chunk's end (its
// start), so the accumulator is never decayed: the blocks are walked from that edge,
// and the sum of the gates walked so far goes into the scale of the rows. Y~ is value
// and remainder, so the fp32 state is good to 2^-17: it is what the caller's pool
// receives after a prefill. Bound by HBM: K and V are read once. Warps: 0 loads,
// 1 MMA, 4-11 scale rows (four threads a row), 4-7 write the state out.
struct StateCfg {
  static constexpr int KS = 3;
  static constexpr int OFF_Y2 = KS * 2 * kTile;            // two buffers of value and remainder
  static constexpr int OFF_BAR = OFF_Y2 + 4 * kTile;
  static constexpr int NBAR = 2 * KS + 4 + 2;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

struct TcStateParams {
  const __nv_bfloat16* gate;
  float* out;      // [BH][C][128*128] (state_f4)
  double* tot;     // [BH][C]
  int64_t N, L, C, first, count, spin_limit;  // chunks [first, first + count) of every sequence
};

template <bool SUFFIX>
__global__ void __launch_bounds__(384, 1)
gated_state_sm100_kernel(const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_z,
                         const TcStateParams prm) {
  using CF = StateCfg;
  constexpr int KS = CF::KS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* in_full = reinterpret_cast<uint64_t*>(smem + CF::OFF_BAR);
  uint64_t* in_empty = in_full + KS;
  uint64_t* y2_full = in_empty + KS;
  uint64_t* y2_empty = y2_full + 2;
  uint64_t *done = y2_empty + 2, *drain = done + 1;
  uint32_t* tmem_base = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base + 1);

  const int64_t bh = blockIdx.x / prm.count, ch = prm.first + blockIdx.x % prm.count;
  const int64_t t0 = ch * prm.L, t1 = min(prm.N, t0 + prm.L);
  const int n = static_cast<int>((t1 - t0 + 63) / 64);
  auto row_of = [&](int i) { return t0 + static_cast<int64_t>(SUFFIX ? i : n - 1 - i) * 64; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < KS; ++i) { s::mbar_init(&in_full[i], 1); s::mbar_init(&in_empty[i], 1); }
    for (int i = 0; i < 2; ++i) { s::mbar_init(&y2_full[i], 256); s::mbar_init(&y2_empty[i], 1); }
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
    s::tmem_alloc(tmem_base, 128);
    s::tmem_relinquish();
  }
  s::tc_fence_before();
  __syncthreads();
  s::tc_fence_after();
  const uint32_t tmem = *tmem_base;
  const int64_t lim = prm.spin_limit;
  pdl_launch_dependents();
  pdl_wait();
  auto wait = [&](uint64_t* bar, uint32_t parity, int where) -> bool {
    return __all_sync(0xffffffffu, s::wait_bar(bar, parity, lim, abort_flag, where));
  };

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int st = i % KS;
        if (!s::wait_bar(&in_empty[st], ((i / KS) & 1) ^ 1, lim, abort_flag, 90)) { ok = false; break; }
        const int row = static_cast<int>(row_of(i)), z = static_cast<int>(bh);
        uint8_t* dst = smem + st * 2 * kTile;
        s::mbar_expect_tx(&in_full[st], 2 * kTile);
        for (int p = 0; p < 2; ++p) s::tma_load_3d(dst + p * 8192, &tm_y, &in_full[st], 64 * p, row, z);
        for (int p = 0; p < 2; ++p) s::tma_load_3d(dst + kTile + p * 8192, &tm_z, &in_full[st], 64 * p, row, z);
        ++issued;
      }
      if (!ok)
        for (int j = max(0, issued - KS); j < issued; ++j) s::drain_wait(&in_full[j % KS], (j / KS) & 1);
    }
  } else if (warp == 1) {
    constexpr uint32_t ID_UPD = s::make_idesc(128, 128, true, true);
    const uint32_t base = s::smem_u32(smem);
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      ok = wait(&in_full[i % KS], (i / KS) & 1, 91) && wait(&y2_full[i & 1], (i >> 1) & 1, 92);
      if (!ok) break;
      s::tc_fence_after();
      const uint32_t y2 = base + CF::OFF_Y2 + (i & 1) * 2 * kTile, za = base + (i % KS) * 2 * kTile + kTile;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        s::mma_bf16_ss_warp(tmem, s::make_desc(y2 + (k >> 2) * kTile + (k & 3) * 2048, 8192, 1024),
                            s::make_desc(za + (k & 3) * 2048, 8192, 1024), ID_UPD, i > 0 || k > 0);
      s::mma_commit_warp(&y2_empty[i & 1]);
      s::mma_commit_warp(&in_empty[i % KS]);
    }
    if (ok) s::mma_commit_warp(done);
    s::mma_commit_warp(drain);
    s::drain_wait(drain, 0);
  } else if (warp >= 4) {
    const int r = (warp - 4) * 8 + (lane >> 2), ch0 = (lane & 3) * 4;
    const __nv_bfloat16* g = prm.gate + bh * prm.N;
    auto gate_at = [&](int64_t t) { return t < t1 ? g[t] : __float2bfloat16(0.f); };
    __nv_bfloat16 gx = gate_at(row_of(0) + 2 * lane), gy = gate_at(row_of(0) + 2 * lane + 1);
    double run = 0.0;  // sum of the gates of the blocks walked
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      float a, b;
      warp_sums(gate_log2(gx), gate_log2(gy), lane, a, b);
      const float ca = __shfl_sync(0xffffffffu, a, r >> 1), cb = __shfl_sync(0xffffffffu, b, r >> 1);
      const float c = (r & 1) ? cb : ca, all = __shfl_sync(0xffffffffu, b, 31);
      const float f = ex2(static_cast<float>(run + static_cast<double>(SUFFIX ? c : all - c)));
      run += static_cast<double>(all);
      if (i + 1 < n) {
        gx = gate_at(row_of(i + 1) + 2 * lane);
        gy = gate_at(row_of(i + 1) + 2 * lane + 1);
      }
      ok = wait(&in_full[i % KS], (i / KS) & 1, 93) && wait(&y2_empty[i & 1], ((i >> 1) & 1) ^ 1, 94);
      if (!ok) break;
      scaled_copy<2>(s::smem_u32(smem + (i % KS) * 2 * kTile), s::smem_u32(smem + CF::OFF_Y2 + (i & 1) * 2 * kTile), r,
                     f, ch0, 4);
      s::fence_proxy_async();
      s::mbar_arrive(&y2_full[i & 1]);
    }
    if (warp == 4 && lane == 0) prm.tot[bh * prm.C + ch] = run * 0.693147180559945309417;  // natural log
    if (ok && warp < 8 && wait(done, 0, 95)) {
      s::tc_fence_after();
      const int row = 32 * (warp & 3) + lane;
      float4* dst = reinterpret_cast<float4*>(prm.out + (bh * prm.C + ch) * 128 * 128);
#pragma unroll
      for (int c32 = 0; c32 < 4; ++c32) {
        uint32_t v[32];
        s::tmem_ld32(tmem + c32 * 32 + (static_cast<uint32_t>(32 * (warp & 3)) << 16), v);
        s::tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 8; ++q)
          dst[s::state_f4<128>(row, c32 * 8 + q)] =
              make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                          __uint_as_float(v[4 * q + 3]));
      }
    }
  }

  s::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    s::tc_fence_after();
    s::tmem_dealloc(tmem, 128);
  }
}

// -------------------------------------------------------------------- launches

template <bool SUFFIX>
inline cudaError_t launch_state_sm100(const void* y, const void* z, const TcStateParams& p, int64_t BH, cudaStream_t st) {
  CUtensorMap ty, tz;
  if (!make_tmap_3d(&ty, y, BH, p.N, 128, 64) || !make_tmap_3d(&tz, z, BH, p.N, 128, 64)) return cudaErrorInvalidValue;
  auto kern = gated_state_sm100_kernel<SUFFIX>;
  static bool done[128];
  if (!smem_attribute_set(kern, StateCfg::SMEM, done)) return cudaErrorInvalidValue;
  return launch_pdl(kern, dim3((unsigned)(BH * p.count)), dim3(384), StateCfg::SMEM, st, ty, tz, p);
}

template <bool BACK, bool GRAD>
inline cudaError_t launch_sm100(const void* x, const void* y, const void* z, void* o, const TcParams& p, int64_t BH,
                                cudaStream_t st) {
  CUtensorMap tx, ty, tz, to;
  if (!make_tmap_3d(&tx, x, BH, p.N, 128, 64) || !make_tmap_3d(&ty, y, BH, p.N, 128, 64) ||
      !make_tmap_3d(&tz, z, BH, p.N, 128, 64) || !make_tmap_3d(&to, o, BH, p.N, 128, 16))
    return cudaErrorInvalidValue;
  auto kern = gated_sm100_kernel<BACK, GRAD>;
  static bool done[128];
  if (!smem_attribute_set(kern, TcCfg<GRAD>::SMEM, done)) return cudaErrorInvalidValue;
  return launch_pdl(kern, dim3((unsigned)(BH * p.C)), dim3(512), TcCfg<GRAD>::SMEM, st, tx, ty, tz, to, p);
}

}  // namespace gated
}  // namespace la2
