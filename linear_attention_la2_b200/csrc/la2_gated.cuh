// Host side of the gated recurrence: shapes, plan, launches and the C entry
// points la2_forward_gated, la2_backward_gated, la2_kv_state_gated and
// la2_decode_step_gated. Included at the end of la2.cu.
#pragma once

namespace la2 {
namespace gated {

struct Plan {
  int64_t L = 0, C = 1;
  bool tc = false;
  int nel = 0;  // floats of a chunk's state in the workspace
  // Tensor cores: the pieces whose own states are computed (Ls rows, K a sequence,
  // `per` a chunk); per = 0 (and K = C): a scan turns them into the chunks' states.
  int64_t Ls = 0, K = 1, per = 0;
  size_t off_suffix = 0, off_suffix_t = 0, off_sum = 0, off_tot = 0, off_qdq = 0, off_kdk = 0;  // prefix states at 0
  size_t bytes = 0;
};

constexpr int64_t kSumPieces = 12;  // pieces a chunk adds up itself; more are scanned

enum Need { NEED_FWD, NEED_BWD, NEED_STATE };

static size_t round256(size_t n) { return (n + 255) / 256 * 256; }

static la2_status check(int64_t B, int64_t H, int64_t N, int64_t d, int64_t dv, la2_dtype dt) {
  if (B < 0 || H < 0 || N < 0 || d < 1 || dv < 1) return LA2_ERR_INVALID_ARG;
  if (dt != LA2_F32 && dt != LA2_BF16) return LA2_ERR_INVALID_ARG;
  if (double(B) * double(H) * double(N) * double(std::max(d, dv)) > 9.0e18) return LA2_ERR_INVALID_ARG;
  if (d > 128 || dv > 128) return LA2_ERR_UNSUPPORTED;
  if (dt == LA2_BF16 && ((d != 64 && d != 128) || (dv != 64 && dv != 128))) return LA2_ERR_UNSUPPORTED;
  if (N > 0x7fffffff - kRows) return LA2_ERR_UNSUPPORTED;  // rows are TMA coordinates
  // one CTA a (sequence, chunk of at least a block), 256 elements of a state a CTA
  const double nel = dt == LA2_BF16 ? 128.0 * 128.0 : double(d) * double(dv), nb = std::ceil(nel / kThreads);
  if (double(B) * double(H) * std::max(std::ceil(double(N) / kRows), nb) > 2147483647.0)
    return LA2_ERR_UNSUPPORTED;
  return LA2_OK;
}

// Chunks of a sequence run in parallel: the count is the one whose waves of CTAs, times
// blocks a chunk and a fixed cost, are shortest; more than one chunk adds the pass over
// the chunks' own states. CUDA cores: in the backward at most 512 rows a chunk, over
// which the gates' gradient is a running difference of row dots (see la2_gated_simt.cuh).
static Plan make_plan_uncached(int64_t B, int64_t H, int64_t N, int64_t d, int64_t dv, la2_dtype dt, Need need,
                               int sms) {
  Plan p;
  const int64_t BH = B * H, T = (N + kRows - 1) / kRows;
  p.tc = dt == LA2_BF16;
  p.nel = p.tc ? 128 * 128 : static_cast<int>(d * dv);
  int64_t per = 1;
  if (g_chunk_len > 0) {
    p.L = (g_chunk_len + kRows - 1) / kRows * kRows;
  } else if (p.tc) {
    // in blocks of the main pass: what a launch of it and of the state pass costs
    // beside its blocks, a block of the state pass (two CTAs an SM), a piece's state that
    // a chunk adds up, and the scan, for itself and for a state. (Gradients in 2 chunks a sequence of 1, 2, 3, 4, 5, 6
    // pieces: B2 H32 N8K 561, 506, 483, 473, 507, 521 us, where a pass of 4 is the last
    // that fits in one wave; B4 H16 N2K 173, 164, 177, 173, -, 200 us.)
    constexpr double kFixed = 6.0, kStateFixed = 5.0, kStateBlock = 0.7, kPiece = 1.0, kScan = 4.0, kScanState = 0.0125;
    const double passes = need == NEED_BWD ? 2 : 1, launches = need == NEED_BWD ? 3 : 1;  // state, main
    const int64_t G = std::max(sms, 1), most = std::max<int64_t>(1, T / 2);
    auto waves = [](int64_t units, int64_t slots) { return static_cast<double>((units + slots - 1) / slots); };
    auto blocks = [&](int64_t parts) { return static_cast<double>((T + parts - 1) / parts); };
    int64_t best_c = 1;
    double best = -1.0;
    for (int64_t c = 1; c <= most && (c == 1 || BH * (c - 1) < 8 * G); ++c) {
      const int64_t mmax = need == NEED_STATE || c == 1 ? 1 : std::max<int64_t>(1, std::min(kSumPieces, T) / c);
      for (int64_t m = 1; m <= mmax; ++m) {
        double cost = need == NEED_STATE ? 0.0 : launches * waves(BH * c, G) * (blocks(c * m) * m + kFixed);
        if (need == NEED_STATE || c > 1)
          cost += passes * waves(BH * (need == NEED_STATE ? c : (c - 1) * m), 2 * G) *
                  (blocks(c * m) * kStateBlock + kStateFixed);
        if (need != NEED_STATE)
          cost += c > kSumPieces ? passes * (kScan + kScanState * static_cast<double>(BH * c))
                                 : launches * kPiece * static_cast<double>((c - 1) * m);
        if (best < 0.0 || cost < best) {
          best = cost;
          best_c = c;
          per = m;
        }
      }
    }
    p.Ls = (T + best_c * per - 1) / (best_c * per) * kRows;
    p.L = p.Ls * per;
  } else {
    // in blocks of the main pass (both gradients count as two of its CTAs): its waves,
    // a block of the state pass, and the launches that more than one chunk adds
    const double block = need == NEED_BWD ? 0.25 : 0.4;
    const size_t smem = need == NEED_BWD   ? smem_bytes((int)d, (int)dv, 2, 2, 1)
                        : need == NEED_FWD ? smem_bytes((int)d, (int)dv, 2, 1, 1)
                                           : smem_bytes((int)d, (int)dv, 1, 1, 0);
    const int64_t slots = std::max(sms, 1) * (smem <= 113 * 1024 ? 2 : 1), ctas = need == NEED_BWD ? 2 : 1;
    auto waves = [&](int64_t units) { return static_cast<double>((units + slots - 1) / slots); };
    double best = -1.0;
    for (int64_t c = 1; c <= T && (c == 1 || BH * (c - 1) < 4 * slots); ++c) {
      const int64_t rows = (T + c - 1) / c;
      double cost = need == NEED_STATE ? 0.0 : waves(ctas * BH * c) * (static_cast<double>(rows) + 0.3);
      if (need == NEED_STATE || c > 1) cost += waves(ctas * BH * c) * (block * static_cast<double>(rows) + 0.3);
      if (c > kSumPieces) cost += 0.4;
      if (best < 0.0 || cost < best) {
        best = cost;
        p.L = rows * kRows;
      }
    }
    if (need == NEED_BWD) p.L = std::min<int64_t>(p.L, 512);
  }
  p.L = std::max<int64_t>(p.L, kRows);
  p.C = std::max<int64_t>(1, (N + p.L - 1) / p.L);
  p.K = p.C;
  if (p.tc && p.Ls == 0) p.Ls = p.L;
  if (!p.tc) {
    p.per = p.C <= kSumPieces ? 1 : 0;
  } else if (need != NEED_STATE) {
    p.K = std::max<int64_t>(1, (N + p.Ls - 1) / p.Ls);
    p.per = p.K <= kSumPieces ? p.L / p.Ls : 0;
  }
  const bool states = p.C > 1 || need == NEED_STATE;
  const size_t one = states ? round256((size_t)BH * p.K * p.nel * sizeof(float)) : 0;
  size_t at = one;
  p.off_suffix = at;
  if (need == NEED_BWD) at += one;
  p.off_suffix_t = at;  // tensor cores: the suffix states transposed, for dV
  if (need == NEED_BWD && p.tc) at += one;
  // the starts of the dQ and then of the dK pass's chunks, where the chunks add them up
  p.off_sum = at;
  if (need == NEED_BWD && states && p.per > 0) at += 2 * round256((size_t)BH * p.C * p.nel * sizeof(float));
  p.off_tot = at;
  if (states) at += round256((size_t)BH * p.K * sizeof(double));
  p.off_qdq = at;
  if (need == NEED_BWD) at += round256((size_t)BH * N * sizeof(float));
  p.off_kdk = at;
  if (need == NEED_BWD) at += round256((size_t)BH * N * sizeof(float));
  p.bytes = at;
  return p;
}

// Plans are pure functions of the arguments, the split override and the SM count; a
// workspace query and its call ask for the same one, so recent plans are kept.
static Plan make_plan(int64_t B, int64_t H, int64_t N, int64_t d, int64_t dv, la2_dtype dt, Need need, int sms) {
  struct Key {
    int64_t v[9];
    bool operator==(const Key& o) const { return std::memcmp(v, o.v, sizeof(v)) == 0; }
  };
  constexpr int kSlots = 16;
  static Key keys[kSlots];
  static Plan plans[kSlots];
  static int used = 0, next_slot = 0;
  static std::mutex mu;
  const Key k{{B, H, N, d, dv, dt, need, sms, g_chunk_len}};
  {
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
      if (keys[i] == k) return plans[i];
  }
  const Plan p = make_plan_uncached(B, H, N, d, dv, dt, need, sms);
  std::lock_guard<std::mutex> lock(mu);
  keys[next_slot] = k;
  plans[next_slot] = p;
  next_slot = (next_slot + 1) % kSlots;
  used = used < kSlots ? used + 1 : kSlots;
  return p;
}

// Lets a CUDA-core kernel take what a CTA may have (once a device).
template <auto KERNEL>
static bool raise_smem() {
  static bool done[128];
  return smem_attribute_set(KERNEL, 227 * 1024, done);
}

// CUDA cores: the chunks' own states of (a0, b0) as prefixes and, with out1, of
// (a1, b1) as suffixes; `all`: every chunk's.
static la2_status chunk_states(const void* a0, const void* b0, const void* a1, const void* b1, const void* gate,
                               float* out0, float* out1, double* tot, bool all, int64_t BH, const Shape& sh,
                               cudaStream_t st) {
  const size_t smem = smem_bytes(sh.d, sh.dv, 1, 1, 0);
  if (!raise_smem<chunk_state_kernel>()) return LA2_ERR_CUDA;
  StateArgs p{};
  p.a[0] = static_cast<const float*>(a0);
  p.b[0] = static_cast<const float*>(b0);
  p.a[1] = static_cast<const float*>(a1);
  p.b[1] = static_cast<const float*>(b1);
  p.gate = static_cast<const float*>(gate);
  p.out[0] = out0;
  p.out[1] = out1;
  p.tot = tot;
  p.all = all;
  LaunchTimer t(K_GATED_STATE, st);
  if (launch_pdl(chunk_state_kernel, dim3((unsigned)(BH * sh.C), out1 ? 2 : 1), dim3(kThreads), smem, st, p, sh) !=
      cudaSuccess)
    return LA2_ERR_CUDA;
  return launch_status();
}

// Scans s0 in mode0 and, where given, s1 in mode 1 (see scan_kernel).
static la2_status scan(float* s0, float* s1, const double* tot, int64_t BH, const Shape& sh, int nel, int mode0,
                       cudaStream_t st) {
  const int nb = (nel + kThreads - 1) / kThreads;
  LaunchTimer t(K_GATED_SCAN, st);
  if (launch_pdl(scan_kernel, dim3((unsigned)(BH * nb), s1 ? 2 : 1), dim3(kThreads), 0, st, s0, s1, tot, sh.C, nel,
                 mode0) != cudaSuccess)
    return LA2_ERR_CUDA;
  return launch_status();
}

static la2_status forward(const void* q, const void* k, const void* v, const void* gate, void* o, char* ws,
                          const Plan& p, int64_t BH, const Shape& sh, cudaStream_t st) {
  float* states = p.C > 1 ? reinterpret_cast<float*>(ws) : nullptr;
  double* tot = reinterpret_cast<double*>(ws + p.off_tot);
  la2_status s = LA2_OK;
  if (states) {
    // (all: the scan reads every chunk's)
    if ((s = chunk_states(k, v, nullptr, nullptr, gate, states, nullptr, tot, !p.per, BH, sh, st)) != LA2_OK) return s;
    if (!p.per && (s = scan(states, nullptr, tot, BH, sh, p.nel, 0, st)) != LA2_OK) return s;
  }
  const size_t smem = smem_bytes(sh.d, sh.dv, 2, 1, 1);
  if (!raise_smem<fwd_kernel>()) return LA2_ERR_CUDA;
  LaunchTimer t(K_GATED_FWD, st);
  if (launch_pdl(fwd_kernel, dim3((unsigned)(BH * sh.C)), dim3(kThreads), smem, st, static_cast<const float*>(q),
                 static_cast<const float*>(k), static_cast<const float*>(v), static_cast<const float*>(gate),
                 static_cast<float*>(o), static_cast<const float*>(states), static_cast<const double*>(tot),
                 sh) != cudaSuccess)
    return LA2_ERR_CUDA;
  return launch_status();
}

// Tensor cores: states of the pieces that a chunk starts from, and their scan where
// the chunks do not add them up themselves. kind: what they are for.
enum States { FOR_O, FOR_DQ, FOR_DK_DV, FOR_POOL };
static la2_status states_tc(const Tile& y, const Tile& z, const void* gate, float* out, float* out_t, double* tot,
                            int64_t BH, const Shape& sh, const Plan& pl, States kind, cudaStream_t st) {
  const int64_t per = std::max<int64_t>(1, pl.per);
  TcStateParams p{};
  p.gate = static_cast<const __nv_bfloat16*>(gate);
  p.out = out;
  p.out_t = out_t;
  p.tot = tot;
  p.N = sh.N;
  p.L = pl.Ls;
  p.K = pl.K;
  p.first = kind == FOR_DK_DV ? per : 0;
  p.count = kind == FOR_POOL ? pl.K : kind == FOR_DK_DV ? pl.K - per : (pl.C - 1) * per;
  p.tot_from = kind == FOR_DK_DV ? (pl.C - 1) * per : 0;  // (the others are the prefixes' pass')
  p.beside = kind == FOR_DK_DV && pl.per > 0;  // (the prefixes' pass came before, without a scan)
  p.spin_limit = spin_limit();
  {
    LaunchTimer t(K_GATED_STATE, st);
    const cudaError_t e = kind == FOR_DK_DV ? launch_state_sm100<true, false, false>(y, z, p, BH, st)
                          : kind == FOR_O   ? launch_state_sm100<false, true, false>(y, z, p, BH, st)
                          : kind == FOR_DQ  ? launch_state_sm100<false, false, false>(y, z, p, BH, st)
                                            : launch_state_sm100<false, false, true>(y, z, p, BH, st);
    if (e != cudaSuccess) return LA2_ERR_CUDA;
  }
  la2_status s = launch_status();
  if (s != LA2_OK || kind == FOR_POOL || pl.per > 0) return s;
  return scan(out, out_t, tot, BH, sh, pl.nel, kind == FOR_DK_DV ? 1 : 0, st);  // (out_t: suffixes only)
}

static TcParams tc_params(const void* gate, const float* init, const double* tot, const Shape& sh, const Plan& pl) {
  TcParams p{};
  p.gate = static_cast<const __nv_bfloat16*>(gate);
  p.init = init;
  p.tot = tot;
  p.N = sh.N;
  p.L = sh.L;
  p.C = sh.C;
  p.spin_limit = spin_limit();
  p.K = static_cast<int32_t>(pl.K);
  p.per = static_cast<int32_t>(pl.per);
  return p;
}

static la2_status forward_tc(const void* q, const void* k, const void* v, const void* gate, void* o, char* ws,
                             const Plan& p, int64_t BH, const Shape& sh, cudaStream_t st) {
  float* states = p.C > 1 ? reinterpret_cast<float*>(ws) : nullptr;
  double* tot = reinterpret_cast<double*>(ws + p.off_tot);
  const Tile tq(q, BH, sh.N, sh.d), tk(k, BH, sh.N, sh.d), tv(v, BH, sh.N, sh.dv), to(o, BH, sh.N, sh.dv);
  if (states) {
    const la2_status s = states_tc(tk, tv, gate, states, nullptr, tot, BH, sh, p, FOR_O, st);
    if (s != LA2_OK) return s;
  }
  LaunchTimer t(K_GATED_FWD, st);
  if (launch_sm100<false, false>(tq, tk, tv, to, to, tc_params(gate, states, tot, sh, p), BH, st) != cudaSuccess)
    return LA2_ERR_CUDA;
  return launch_status();
}

// The gates' gradient, from the chunks' starts: the sums left by the gradient passes,
// or the scanned states.
template <typename T>
static la2_status gate_grad(const void* q, const void* k, const void* v, const void* gate, const void* dout,
                            const float* qdq, const float* kdk, const float* prefix, const float* suffix, void* dgate,
                            int64_t BH, const Shape& sh, const Plan& p, cudaStream_t st) {
  LaunchTimer t(K_GATED_GATE, st);
  if (launch_pdl(gate_grad_kernel<T>, dim3((unsigned)(BH * sh.C)), dim3(kGradThreads), 0, st,
                 static_cast<const T*>(gate), qdq, kdk, prefix, suffix, static_cast<T*>(dgate), sh.N, sh.L, sh.C,
                 p.nel, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v),
                 static_cast<const T*>(dout), sh.d, sh.dv) != cudaSuccess)
    return LA2_ERR_CUDA;
  return launch_status();
}

// Where the dQ (0) and dK (1) passes leave the chunks' starts, or null: no chunks, or scanned.
static float* start_sums(char* ws, const Plan& p, int64_t BH, int which) {
  if (p.C == 1 || p.per == 0) return nullptr;
  return reinterpret_cast<float*>(ws + p.off_sum + which * round256((size_t)BH * p.C * p.nel * sizeof(float)));
}

static la2_status backward_tc(const void* q, const void* k, const void* v, const void* gate, const void* dout,
                              void* dq, void* dk, void* dvv, void* dgate, char* ws, const Plan& p, int64_t BH,
                              const Shape& sh, cudaStream_t st) {
  float* prefix = p.C > 1 ? reinterpret_cast<float*>(ws) : nullptr;
  float* suffix = p.C > 1 ? reinterpret_cast<float*>(ws + p.off_suffix) : nullptr;
  float* suffix_t = p.C > 1 ? reinterpret_cast<float*>(ws + p.off_suffix_t) : nullptr;
  float* qdq = reinterpret_cast<float*>(ws + p.off_qdq);
  float* kdk = reinterpret_cast<float*>(ws + p.off_kdk);
  float *prefix_sum = start_sums(ws, p, BH, 0), *suffix_sum = start_sums(ws, p, BH, 1);
  double* tot = reinterpret_cast<double*>(ws + p.off_tot);
  const Tile tq(q, BH, sh.N, sh.d), tk(k, BH, sh.N, sh.d), tv(v, BH, sh.N, sh.dv), tdo(dout, BH, sh.N, sh.dv);
  const Tile tdq(dq, BH, sh.N, sh.d), tdk(dk, BH, sh.N, sh.d), tdv(dvv, BH, sh.N, sh.dv);
  la2_status s = LA2_OK;
  if (prefix) {
    if ((s = states_tc(tk, tv, gate, prefix, nullptr, tot, BH, sh, p, FOR_DQ, st)) != LA2_OK) return s;
    if ((s = states_tc(tq, tdo, gate, suffix, suffix_t, tot, BH, sh, p, FOR_DK_DV, st)) != LA2_OK) return s;
  }
  {
    TcParams t = tc_params(gate, prefix, tot, sh, p);
    t.dots = qdq;
    t.sum = prefix_sum;
    LaunchTimer lt(K_GATED_DQ, st);
    if (launch_sm100<false, true>(tdo, tv, tk, tdq, tq, t, BH, st) != cudaSuccess) return LA2_ERR_CUDA;
  }
  {
    TcParams t = tc_params(gate, suffix_t, tot, sh, p);
    t.beside = 1;
    LaunchTimer lt(K_GATED_DKDV, st);
    if (launch_sm100<true, false>(tk, tq, tdo, tdv, tdv, t, BH, st) != cudaSuccess) return LA2_ERR_CUDA;
    t.init = suffix;
    t.dots = kdk;
    t.sum = suffix_sum;
    if (launch_sm100<true, true>(tv, tdo, tq, tdk, tk, t, BH, st) != cudaSuccess) return LA2_ERR_CUDA;
  }
  if ((s = launch_status()) != LA2_OK) return s;
  return gate_grad<__nv_bfloat16>(q, k, v, gate, dout, qdq, kdk, prefix_sum ? prefix_sum : prefix,
                                  suffix_sum ? suffix_sum : suffix, dgate, BH, sh, p, st);
}

static la2_status backward(const void* q, const void* k, const void* v, const void* gate, const void* dout,
                           void* dq, void* dk, void* dvv, void* dgate, char* ws, const Plan& p, int64_t BH,
                           const Shape& sh, cudaStream_t st) {
  float* prefix = p.C > 1 ? reinterpret_cast<float*>(ws) : nullptr;
  float* suffix = p.C > 1 ? reinterpret_cast<float*>(ws + p.off_suffix) : nullptr;
  double* tot = reinterpret_cast<double*>(ws + p.off_tot);
  la2_status s = LA2_OK;
  if (prefix) {
    if ((s = chunk_states(k, v, q, dout, gate, prefix, suffix, tot, !p.per, BH, sh, st)) != LA2_OK) return s;
    if (!p.per && (s = scan(prefix, suffix, tot, BH, sh, p.nel, 0, st)) != LA2_OK) return s;
  }
  BwdArgs a{};
  a.q = static_cast<const float*>(q);
  a.k = static_cast<const float*>(k);
  a.v = static_cast<const float*>(v);
  a.gate = static_cast<const float*>(gate);
  a.dout = static_cast<const float*>(dout);
  a.dq = static_cast<float*>(dq);
  a.dk = static_cast<float*>(dk);
  a.dv = static_cast<float*>(dvv);
  a.qdq = reinterpret_cast<float*>(ws + p.off_qdq);
  a.kdk = reinterpret_cast<float*>(ws + p.off_kdk);
  a.prefix = prefix;
  a.suffix = suffix;
  a.prefix_sum = start_sums(ws, p, BH, 0);
  a.suffix_sum = start_sums(ws, p, BH, 1);
  a.tot = tot;
  {
    const size_t smem = smem_bytes(sh.d, sh.dv, 2, 2, 1);
    if (!raise_smem<bwd_kernel>()) return LA2_ERR_CUDA;
    LaunchTimer t(K_GATED_DKDV, st);  // (dQ too)
    if (launch_pdl(bwd_kernel, dim3((unsigned)(BH * sh.C), 2), dim3(kThreads), smem, st, a, sh) != cudaSuccess)
      return LA2_ERR_CUDA;
  }
  if ((s = launch_status()) != LA2_OK) return s;
  return gate_grad<float>(q, k, v, gate, dout, a.qdq, a.kdk, a.prefix_sum ? a.prefix_sum : prefix,
                          a.suffix_sum ? a.suffix_sum : suffix, dgate, BH, sh, p, st);
}

// Pointers of a call: every one non-null and aligned, no output over an input,
// another output or the workspace.
struct Span {
  const void* p;
  size_t n;
};
static bool spans_ok(const Span* in, int n_in, const Span* out, int n_out) {
  for (int i = 0; i < n_in; ++i)
    if (!in[i].p || !is_aligned(in[i].p, 16)) return false;
  for (int i = 0; i < n_out; ++i) {
    if (!out[i].p || !is_aligned(out[i].p, 16)) return false;
    for (int j = 0; j < n_in; ++j)
      if (overlaps(out[i].p, out[i].n, in[j].p, in[j].n)) return false;
    for (int j = i + 1; j < n_out; ++j)
      if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return false;
  }
  return true;
}
static la2_status workspace_ok(const void* ws, size_t have, size_t need, const Span* in, int n_in,
                               const Span* out, int n_out) {
  if (need == 0) return LA2_OK;
  if (!ws || have < need) return LA2_ERR_WORKSPACE;
  if (!is_aligned(ws, 256)) return LA2_ERR_INVALID_ARG;
  for (int i = 0; i < n_in; ++i)
    if (overlaps(ws, need, in[i].p, in[i].n)) return LA2_ERR_INVALID_ARG;
  for (int i = 0; i < n_out; ++i)
    if (overlaps(ws, need, out[i].p, out[i].n)) return LA2_ERR_INVALID_ARG;
  return LA2_OK;
}

static size_t workspace_size(int64_t B, int64_t H, int64_t N, int64_t d, int64_t dv, la2_dtype dt, Need need) {
  if (check(B, H, N, d, dv, dt) != LA2_OK) return (size_t)-1;
  if (B == 0 || H == 0 || N == 0) return 0;
  const int sms = device_sm_count();
  if (sms <= 0) return (size_t)-1;
  return make_plan(B, H, N, d, dv, dt, need, sms).bytes;
}

}  // namespace gated
}  // namespace la2

extern "C" {

size_t la2_workspace_size_gated(int64_t B, int64_t H, int64_t N, int64_t d, int64_t dv, la2_dtype dt,
                                int is_backward) {
  return gated::workspace_size(B, H, N, d, dv, dt, is_backward ? gated::NEED_BWD : gated::NEED_FWD);
}

la2_status la2_forward_gated(const void* q, const void* k, const void* v, const void* gate, void* o,
                             int64_t B, int64_t H, int64_t N, int64_t d, int64_t dv, la2_dtype dt,
                             void* workspace, size_t workspace_bytes, la2_stream_t stream) {
  la2_status s = gated::check(B, H, N, d, dv, dt);
  if (s != LA2_OK) return s;
  if (B == 0 || H == 0 || N == 0) return LA2_OK;
  const size_t es = dt == LA2_BF16 ? 2 : 4, rows = (size_t)B * H * N;
  const gated::Span in[4] = {{q, rows * d * es}, {k, rows * d * es}, {v, rows * dv * es}, {gate, rows * es}};
  const gated::Span out[1] = {{o, rows * dv * es}};
  if (!gated::spans_ok(in, 4, out, 1)) return LA2_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LA2_ERR_CUDA;
  const gated::Plan p = gated::make_plan(B, H, N, d, dv, dt, gated::NEED_FWD, sms);
  s = gated::workspace_ok(workspace, workspace_bytes, p.bytes, in, 4, out, 1);
  if (s != LA2_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const gated::Shape sh{N, p.L, p.C, (int)d, (int)dv, p.per > 0};
  char* ws = static_cast<char*>(workspace);
  if (p.tc) return gated::forward_tc(q, k, v, gate, o, ws, p, B * H, sh, st);
  return gated::forward(q, k, v, gate, o, ws, p, B * H, sh, st);
}

la2_status la2_backward_gated(const void* q, const void* k, const void* v, const void* gate,
                              const void* dout, void* dq, void* dk, void* dvv, void* dgate, int64_t B,
                              int64_t H, int64_t N, int64_t d, int64_t dv, la2_dtype dt, void* workspace,
                              size_t workspace_bytes, la2_stream_t stream) {
  la2_status s = gated::check(B, H, N, d, dv, dt);
  if (s != LA2_OK) return s;
  if (B == 0 || H == 0 || N == 0) return LA2_OK;
  const size_t es = dt == LA2_BF16 ? 2 : 4, rows = (size_t)B * H * N;
  const gated::Span in[5] = {{q, rows * d * es}, {k, rows * d * es}, {v, rows * dv * es},
                             {gate, rows * es},  {dout, rows * dv * es}};
  const gated::Span out[4] = {{dq, rows * d * es}, {dk, rows * d * es}, {dvv, rows * dv * es}, {dgate, rows * es}};
  if (!gated::spans_ok(in, 5, out, 4)) return LA2_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LA2_ERR_CUDA;
  const gated::Plan p = gated::make_plan(B, H, N, d, dv, dt, gated::NEED_BWD, sms);
  s = gated::workspace_ok(workspace, workspace_bytes, p.bytes, in, 5, out, 4);
  if (s != LA2_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const gated::Shape sh{N, p.L, p.C, (int)d, (int)dv, p.per > 0};
  char* ws = static_cast<char*>(workspace);
  if (p.tc) return gated::backward_tc(q, k, v, gate, dout, dq, dk, dvv, dgate, ws, p, B * H, sh, st);
  return gated::backward(q, k, v, gate, dout, dq, dk, dvv, dgate, ws, p, B * H, sh, st);
}

size_t la2_kv_state_gated_workspace_size(int64_t B, int64_t H, int64_t N, int64_t d, int64_t dv, la2_dtype dt) {
  return gated::workspace_size(B, H, N, d, dv, dt, gated::NEED_STATE);
}

la2_status la2_kv_state_gated(const void* k, const void* v, const void* gate, float* state,
                              const int32_t* slots, int64_t n_slots, int64_t B, int64_t H, int64_t N,
                              int64_t d, int64_t dv, la2_dtype dt, void* workspace, size_t workspace_bytes,
                              la2_stream_t stream) {
  la2_status s = gated::check(B, H, N, d, dv, dt);
  if (s != LA2_OK) return s;
  if (n_slots < 0 || n_slots > 0x7fffffff || (!slots && n_slots < B)) return LA2_ERR_INVALID_ARG;
  if (B == 0 || H == 0 || N == 0) return LA2_OK;
  const size_t es = dt == LA2_BF16 ? 2 : 4, rows = (size_t)B * H * N;
  const gated::Span in[4] = {{k, rows * d * es}, {v, rows * dv * es}, {gate, rows * es},
                             {slots, (size_t)B * sizeof(int32_t)}};
  const gated::Span out[1] = {{state, (size_t)n_slots * H * d * dv * sizeof(float)}};
  const int n_in = slots ? 4 : 3;
  if (slots && !is_aligned(slots, 4)) return LA2_ERR_INVALID_ARG;
  if (!gated::spans_ok(in, 3, out, 1)) return LA2_ERR_INVALID_ARG;
  if (slots && overlaps(in[3].p, in[3].n, out[0].p, out[0].n)) return LA2_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (sms <= 0) return LA2_ERR_CUDA;
  const gated::Plan p = gated::make_plan(B, H, N, d, dv, dt, gated::NEED_STATE, sms);
  s = gated::workspace_ok(workspace, workspace_bytes, p.bytes, in, n_in, out, 1);
  if (s != LA2_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const gated::Shape sh{N, p.L, p.C, (int)d, (int)dv, p.per > 0};
  float* chunks = static_cast<float*>(workspace);
  double* tot = reinterpret_cast<double*>(static_cast<char*>(workspace) + p.off_tot);
  if (p.tc)
    s = gated::states_tc(gated::Tile(k, B * H, N, (int)d), gated::Tile(v, B * H, N, (int)dv), gate, chunks, nullptr, tot,
                         B * H, sh, p, gated::FOR_POOL, st);
  else
    s = gated::chunk_states(k, v, nullptr, nullptr, gate, chunks, nullptr, tot, true, B * H, sh, st);
  if (s != LA2_OK) return s;
  const int V = dv % 4 == 0 ? 4 : 1;  // (state: 16-byte aligned, see spans_ok)
  const int64_t nb = (d * dv + gated::kThreads * V - 1) / (gated::kThreads * V);
  LaunchTimer t(K_GATED_POOL, st);
  if (launch_pdl(V == 4 ? gated::pool_update_kernel<4> : gated::pool_update_kernel<1>, dim3((unsigned)(B * H * nb)),
                 dim3(gated::kThreads), 0, st,
                 static_cast<const float*>(chunks), static_cast<const double*>(tot), state, slots, n_slots,
                 p.C, (int)H, (int)d, (int)dv, p.nel, p.tc ? 128 : 0) != cudaSuccess)
    return LA2_ERR_CUDA;
  return launch_status();
}

la2_status la2_decode_step_gated(const void* q, const void* k, const void* v, const void* gate, void* o,
                                 float* state, const int32_t* slots, int64_t n_slots, int64_t B, int64_t H,
                                 int64_t d, int64_t dv, la2_dtype dt, la2_stream_t stream) {
  if (B < 0 || H < 0 || d < 1 || dv < 1) return LA2_ERR_INVALID_ARG;
  if (dt != LA2_F32 && dt != LA2_BF16) return LA2_ERR_INVALID_ARG;
  if (n_slots < 0 || n_slots > 0x7fffffff || (!slots && n_slots < B)) return LA2_ERR_INVALID_ARG;
  if (double(std::max(B, n_slots)) * double(H) * double(d) * double(dv) > 2.0e18) return LA2_ERR_INVALID_ARG;
  if (B == 0 || H == 0) return LA2_OK;
  const size_t es = dt == LA2_BF16 ? 2 : 4, BH = (size_t)B * H;
  if (!q || !k || !v || !gate || !o || !state) return LA2_ERR_INVALID_ARG;
  if (!is_aligned(q, es) || !is_aligned(k, es) || !is_aligned(v, es) || !is_aligned(gate, es) ||
      !is_aligned(o, es) || !is_aligned(state, 4) || !is_aligned(slots, 4))
    return LA2_ERR_INVALID_ARG;
  if (BH > 0x7fffffff || (dv + 31) / 32 > 65535) return LA2_ERR_UNSUPPORTED;
  const gated::Span in[5] = {{q, BH * d * es}, {k, BH * d * es}, {v, BH * dv * es}, {gate, BH * es},
                             {slots, slots ? (size_t)B * sizeof(int32_t) : 0}};
  const size_t no = BH * dv * es, ns = (size_t)n_slots * H * d * dv * sizeof(float);
  for (const gated::Span& x : in)
    if (x.p && (overlaps(o, no, x.p, x.n) || overlaps(state, ns, x.p, x.n))) return LA2_ERR_INVALID_ARG;
  if (overlaps(o, no, state, ns)) return LA2_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  LaunchTimer t(K_GATED_DECODE, st);
  // Four columns per lane under the conditions of la2_decode_step's.
  const bool v4 = dv % 4 == 0 && d <= kDecodeWarps * kRows && is_aligned(state, 16) && is_aligned(v, 4 * es);
  const dim3 grid((unsigned)BH, (unsigned)(v4 ? (dv + 127) / 128 : (dv + 31) / 32)), block(32 * kDecodeWarps);
  auto launch = [&](auto tag) {
    using T = decltype(tag);
    auto kern = v4 ? decode_gated_v4_kernel<T> : decode_gated_kernel<T>;
    return launch_pdl(kern, grid, block, 0, st, static_cast<const T*>(q), static_cast<const T*>(k),
                      static_cast<const T*>(v), static_cast<const T*>(gate), static_cast<T*>(o), state, slots,
                      n_slots, (int)H, (int)d, (int)dv);
  };
  if ((dt == LA2_BF16 ? launch(__nv_bfloat16()) : launch(0.f)) != cudaSuccess) return LA2_ERR_CUDA;
  return launch_status();
}

}  // extern "C"
