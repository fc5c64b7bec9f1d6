// A pool of state slots, [n_slots, H, d, dv] fp32: copies between slots (fork,
// fresh slots) and compaction. Included at the end of la2.cu.
//
// Both move whole slots once, read and write, and nothing else: bound by HBM.
// The index lists live on the device (a serving loop captured in a graph changes
// them between replays), so the kernels check them; what they refuse is skipped
// and reported by la2_check.
#pragma once

namespace la2 {
namespace slots {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;  // 16-byte pieces a thread has in flight
constexpr int kPiece = kThreads * kUnroll;
constexpr int kMaxCompact = 32768;  // slots whose plan fits in shared memory

// Copies (src >= 0) or zeroes (src < 0) piece `part` of a slot of `n` elements.
template <typename V>
__device__ __forceinline__ void move_piece(V* __restrict__ dst, const V* __restrict__ src, bool zero,
                                           int64_t part, int64_t n) {
  V x[kUnroll];
  const int64_t at = part * kPiece + threadIdx.x;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    x[u] = V{};
    if (!zero && at + u * kThreads < n) x[u] = src[at + u * kThreads];
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (at + u * kThreads < n) dst[at + u * kThreads] = x[u];
}

// Entry i: pool[dst[i]] <- pool[src[i]], or 0 for src[i] = -1; nothing for
// dst[i] = -1 or dst[i] = src[i]. All sources hold their values from before the
// call: an entry whose destination another entry reads, or an earlier one writes,
// is not carried out (and is an error), so no order between CTAs matters.
template <typename V>
__global__ void __launch_bounds__(kThreads)
copy_kernel(V* __restrict__ pool, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int64_t n,
            int64_t n_slots, int64_t slot, int64_t parts) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t i = blockIdx.x / parts, part = blockIdx.x % parts;
  const int32_t s = src[i], d = dst[i];
  int bad = d < -1 || d >= n_slots || s < -1 || s >= n_slots;
  if (!bad) {
    if (d == -1 || d == s) return;
    for (int64_t j = threadIdx.x; j < n; j += kThreads) {
      const int32_t sj = src[j], dj = dst[j];
      bad |= j != i && dj != -1 && ((sj == d && dj != d) || (dj == d && j < i));
    }
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    if (threadIdx.x == 0) record_error(DEV_ERR_INDEX, 61);
    return;
  }
  move_piece(pool + d * slot, pool + (s < 0 ? 0 : s) * slot, s < 0, part, slot);
}

// New place of every slot: live slots below n_live stay, the k-th live slot from
// n_live on goes into the k-th hole below it, -1 for the others. One CTA; the
// holes are listed in shared memory.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads)
compact_plan_kernel(const int32_t* __restrict__ live, int32_t* __restrict__ moved, int n) {
  extern __shared__ int32_t hole[];
  __shared__ int warp_sum[kPlanThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int count = 0;
  for (int i = threadIdx.x; i < n; i += kPlanThreads) count += live[i] != 0;
  count = __reduce_add_sync(0xffffffffu, count);
  if (lane == 0) warp_sum[w] = count;
  __syncthreads();
  int n_live = 0;
  for (int x = 0; x < kPlanThreads / 32; ++x) n_live += warp_sum[x];
  __syncthreads();
  // pass 0 ranks the holes below n_live, pass 1 the live slots from n_live on
  for (int pass = 0; pass < 2; ++pass) {
    int base = 0;
    for (int i0 = pass ? n_live : 0; i0 < (pass ? n : n_live); i0 += kPlanThreads) {
      const int i = i0 + threadIdx.x;
      const bool in = i < (pass ? n : n_live);
      const bool on = in && live[i] != 0;
      const bool mark = in && on == (pass == 1);
      const unsigned ballot = __ballot_sync(0xffffffffu, mark);
      if (lane == 0) warp_sum[w] = __popc(ballot);
      __syncthreads();
      int rank = base + __popc(ballot & ((1u << lane) - 1u));
      for (int x = 0; x < kPlanThreads / 32; ++x) {
        if (x < w) rank += warp_sum[x];
        base += warp_sum[x];
      }
      if (pass == 0) {
        if (mark) hole[rank] = i;
        if (in) moved[i] = on ? i : -1;
      } else if (in) {
        moved[i] = mark ? hole[rank] : -1;
      }
      __syncthreads();
    }
  }
}

// Up to kSmall slots: plan and moves in one launch. CTA (k, part) finds the k-th live
// slot from n_live on and the k-th hole below it (there are at most n / 2) and moves its
// piece; k = 0, part 0 also writes `moved` of the slots that stay or are dead. Every CTA
// reads all flags, four a thread (48 slots of 2 MB, 32 live: 10.2 us, with a launch for
// the plan 14.2).
constexpr int kSmall = 4 * kThreads;
template <typename V>
__global__ void __launch_bounds__(kThreads)
compact_small_kernel(V* __restrict__ pool, const int32_t* __restrict__ live, int32_t* __restrict__ moved, int n,
                     int64_t slot, int64_t parts) {
  __shared__ int sums[kThreads / 32], from_to[2];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t k = blockIdx.x / parts, part = blockIdx.x % parts;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  bool on[4];
  int count = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = 4 * threadIdx.x + u;
    on[u] = i < n && live[i] != 0;
    count += on[u];
  }
  count = __reduce_add_sync(0xffffffffu, count);
  if (lane == 0) sums[w] = count;
  if (threadIdx.x < 2) from_to[threadIdx.x] = -1;
  __syncthreads();
  int n_live = 0;
#pragma unroll
  for (int x = 0; x < kThreads / 32; ++x) n_live += sums[x];
  __syncthreads();
  // running counts of the slots to move (low half) and of the holes (high half)
  auto mark = [&](int u) {
    const int i = 4 * threadIdx.x + u;
    return i >= n ? 0 : i < n_live ? (on[u] ? 0 : 1 << 16) : (on[u] ? 1 : 0);
  };
  const int own = mark(0) + mark(1) + mark(2) + mark(3);
  int run = own;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, run, m);
    if (lane >= m) run += up;
  }
  if (lane == 31) sums[w] = run;
  __syncthreads();
  run -= own;
  for (int x = 0; x < w; ++x) run += sums[x];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = 4 * threadIdx.x + u, x = mark(u);
    if (x & 0xffff && (run & 0xffff) == k) from_to[0] = i;
    if (x >> 16 && run >> 16 == k) from_to[1] = i;
    if (blockIdx.x == 0 && i < n && !(x & 0xffff)) moved[i] = on[u] ? i : -1;
    run += x;
  }
  __syncthreads();
  if (from_to[0] < 0) return;  // as many holes as slots to move
  if (part == 0 && threadIdx.x == 0) moved[from_to[0]] = from_to[1];
  move_piece(pool + from_to[1] * slot, pool + from_to[0] * slot, false, part, slot);
}

// Slot i to moved[i]. Sources lie at or behind n_live, destinations below it.
template <typename V>
__global__ void __launch_bounds__(kThreads)
compact_move_kernel(V* __restrict__ pool, const int32_t* __restrict__ moved, int64_t slot, int64_t parts) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t i = blockIdx.x / parts, part = blockIdx.x % parts;
  const int32_t d = moved[i];
  if (d < 0 || d == i) return;
  move_piece(pool + d * slot, pool + i * slot, false, part, slot);
}

static la2_status check(int64_t n_slots, int64_t H, int64_t d, int64_t dv) {
  if (n_slots < 0 || H < 0 || d < 1 || dv < 1) return LA2_ERR_INVALID_ARG;
  if (n_slots > 0x7fffffff || double(n_slots) * double(H) * double(d) * double(dv) > 2.0e18)
    return LA2_ERR_INVALID_ARG;
  return LA2_OK;
}

}  // namespace slots
}  // namespace la2

extern "C" {

la2_status la2_state_copy(float* state, const int32_t* src, const int32_t* dst, int64_t n, int64_t n_slots,
                          int64_t H, int64_t d, int64_t dv, la2_stream_t stream) {
  la2_status s = slots::check(n_slots, H, d, dv);
  if (s != LA2_OK || n < 0) return s != LA2_OK ? s : LA2_ERR_INVALID_ARG;
  if (n == 0 || n_slots == 0 || H == 0) return LA2_OK;
  if (!state || !src || !dst || !is_aligned(state, 4) || !is_aligned(src, 4) || !is_aligned(dst, 4))
    return LA2_ERR_INVALID_ARG;
  const int64_t slot = H * d * dv;
  const size_t ns = (size_t)n_slots * slot * sizeof(float), ni = (size_t)n * sizeof(int32_t);
  if (overlaps(state, ns, src, ni) || overlaps(state, ns, dst, ni)) return LA2_ERR_INVALID_ARG;
  const bool vec = slot % 4 == 0 && is_aligned(state, 16);
  const int64_t elems = vec ? slot / 4 : slot, parts = (elems + slots::kPiece - 1) / slots::kPiece;
  if (double(n) * double(parts) > 2147483647.0) return LA2_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)(n * parts)), block(slots::kThreads);
  LaunchTimer t(K_STATE_COPY, st);
  const cudaError_t e =
      vec ? launch_pdl(slots::copy_kernel<float4>, grid, block, 0, st, reinterpret_cast<float4*>(state), src, dst,
                       n, n_slots, elems, parts)
          : launch_pdl(slots::copy_kernel<float>, grid, block, 0, st, state, src, dst, n, n_slots, elems, parts);
  if (e != cudaSuccess) return LA2_ERR_CUDA;
  return launch_status();
}

la2_status la2_state_compact(float* state, const int32_t* live, int32_t* moved, int64_t n_slots, int64_t H,
                             int64_t d, int64_t dv, la2_stream_t stream) {
  la2_status s = slots::check(n_slots, H, d, dv);
  if (s != LA2_OK) return s;
  if (n_slots == 0 || H == 0) return LA2_OK;
  if (n_slots > slots::kMaxCompact) return LA2_ERR_UNSUPPORTED;
  if (!state || !live || !moved || !is_aligned(state, 4) || !is_aligned(live, 4) || !is_aligned(moved, 4))
    return LA2_ERR_INVALID_ARG;
  const int64_t slot = H * d * dv;
  const size_t ns = (size_t)n_slots * slot * sizeof(float), ni = (size_t)n_slots * sizeof(int32_t);
  if (overlaps(state, ns, live, ni) || overlaps(state, ns, moved, ni) || overlaps(live, ni, moved, ni))
    return LA2_ERR_INVALID_ARG;
  const bool vec = slot % 4 == 0 && is_aligned(state, 16);
  const int64_t elems = vec ? slot / 4 : slot, parts = (elems + slots::kPiece - 1) / slots::kPiece;
  if (double(n_slots) * double(parts) > 2147483647.0) return LA2_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (n_slots <= slots::kSmall) {
    const dim3 grid((unsigned)(std::max<int64_t>(1, n_slots / 2) * parts)), block(slots::kThreads);
    LaunchTimer t(K_STATE_COMPACT, st);
    const cudaError_t e =
        vec ? launch_pdl(slots::compact_small_kernel<float4>, grid, block, 0, st, reinterpret_cast<float4*>(state),
                         live, moved, (int)n_slots, elems, parts)
            : launch_pdl(slots::compact_small_kernel<float>, grid, block, 0, st, state, live, moved, (int)n_slots,
                         elems, parts);
    return e == cudaSuccess ? launch_status() : LA2_ERR_CUDA;
  }
  const size_t smem = ni;
  static bool attr_done[128];
  if (smem > 48 * 1024 &&
      !smem_attribute_set(slots::compact_plan_kernel, slots::kMaxCompact * (int)sizeof(int32_t), attr_done))
    return LA2_ERR_CUDA;
  LaunchTimer t(K_STATE_COMPACT, st);
  if (launch_pdl(slots::compact_plan_kernel, dim3(1), dim3(slots::kPlanThreads), smem, st, live, moved,
                 (int)n_slots) != cudaSuccess)
    return LA2_ERR_CUDA;
  const dim3 grid((unsigned)(n_slots * parts)), block(slots::kThreads);
  const int32_t* to = moved;
  const cudaError_t e = vec ? launch_pdl(slots::compact_move_kernel<float4>, grid, block, 0, st,
                                         reinterpret_cast<float4*>(state), to, elems, parts)
                            : launch_pdl(slots::compact_move_kernel<float>, grid, block, 0, st, state, to, elems, parts);
  if (e != cudaSuccess) return LA2_ERR_CUDA;
  return launch_status();
}

}  // extern "C"
