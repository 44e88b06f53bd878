// kl_logp.cu -- C ABI of the operators on token log-probabilities through the
// LM output head: kl_logp_*, kl_policy_* and kl_preference_fwd (the mathematics
// and the row kernels are in kl_logp.cuh).
//
// Per chunk of C compact rows (the rows that take part; counted on the device):
//   logp_gather    hidden states, token and the token's logit r of the chunk's rows
//   gemm LOGP      logits tiles -> sums of e = 2^(x - r), and for a backward e in bf16
//   logp_rows      lse, logp, ent; the policy loss's row loss and gradient; the rows'
//                  gradient factors (e is dS up to one factor per row)
//   logp_dlogits   only with an entropy term: e -> dS in place
//                  (chunks that are recomputed: logp_coef, gemm DLOGP gives dS of the
//                  other tokens and logp_own that of the rows' own)
//   gemm ACCUM     dH parts = dS W, split over the vocabulary
//   logp_dh        parts summed, scattered to their rows; the others zeroed
//   gemm           dW (+)= dS^T H_c
// No host synchronisation anywhere: the grids are sized for N rows and the
// kernels read how many there are.
#include "kl_host.cuh"
#include "kl_logp.cuh"

using namespace ckl;

namespace {

// Rows per chunk by default.  In one pass 4096 are as fast (policy loss, 8192 to 32768
// rows, bf16 dW: d 4096, V 128256 20.3, 40.9 and 81.4 ms with 8192, 20.0, 39.9 and 79.1
// with 4096; d 2048, V 50257 3.9, 8.2 and 16.2 against 4.0, 8.1 and 16.0) in half the
// workspace; but where the backward follows a forward over all rows only the first
// chunk's logits are kept, and a row behind it costs a third more.
constexpr int64_t kLogpChunk = 8192;
constexpr int kMaxSeqs = 1 << 20;

struct LPlan {
  int64_t C = 0, C64 = 0, Vp = 0, dp = 0, nch = 0, part_rows = 0;
  int tiles_v = 0, parts_v = 0;
  size_t plan = 0, perm = 0, cid = 0, rowin = 0, factor = 0, clogp = 0, rowc = 0, rl = 0, Hc = 0,
         part = 0, E = 0, dHp = 0, dWf = 0, score = 0, count = 0, slope = 0, total = 0;
};

int check_shape(const kl_logp_problem* p) {
  if (p == nullptr) return KL_ERR_NULL;
  if (p->dtype != KL_DTYPE_BF16) return KL_ERR_DTYPE;
  if (p->dW_dtype != KL_DTYPE_BF16 && p->dW_dtype != KL_DTYPE_F32) return KL_ERR_DTYPE;
  if (p->ids_64 != 0 && p->ids_64 != 1) return KL_ERR_DTYPE;
  if (p->N < 0 || p->d < 1 || p->V < 1 || p->N > (int64_t(1) << 31) - 8192 ||
      p->V > (int64_t(1) << 31) - 512 || p->d > (int64_t(1) << 20))
    return KL_ERR_SHAPE;
  if (p->n_seqs < 0 || p->n_seqs > kMaxSeqs) return KL_ERR_SHAPE;
  if (!(p->T > 0.f) || !(p->T < INFINITY) || p->chunk_tokens < 0) return KL_ERR_ARG;
  if ((p->entropy != 0 && p->entropy != 1) || (p->keep_chunk != 0 && p->keep_chunk != 1))
    return KL_ERR_ARG;
  if (p->ldH != 0 && (p->ldH < p->d || p->ldH > (int64_t(1) << 32))) return KL_ERR_SHAPE;
  if (p->d % 8 != 0 || p->ldH % 8 != 0) return KL_ERR_ALIGN;
  return KL_OK;
}

int check(const kl_logp_problem* p) {
  KL_TRY(check_shape(p));
  if (p->N > 0) {
    if (p->H == nullptr || p->W == nullptr || p->ids == nullptr) return KL_ERR_NULL;
    if (p->n_seqs > 0 && p->cu_seqlens == nullptr) return KL_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(p->H) | reinterpret_cast<uintptr_t>(p->W)) & 15)
      return KL_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(p->ids) & (p->ids_64 ? 7 : 3)) return KL_ERR_ALIGN;
  }
  return KL_OK;
}

LPlan plan_of(const kl_logp_problem* p, int entry) {
  if (p->keep_chunk) entry = KL_ENTRY_FWD_BWD;  // one layout for the call pair
  LPlan l;
  const int64_t chunk = p->chunk_tokens > 0 ? p->chunk_tokens : kLogpChunk;
  l.C = p->N < chunk ? p->N : chunk;
  if (l.C < 1) l.C = 1;
  l.C64 = cdiv(l.C, 64) * 64;
  l.nch = p->N > 0 ? cdiv(p->N, l.C) : 0;
  // Row pitches of the library's own buffers are whole 128-byte lines: a TMA box
  // row that starts inside a 32-byte sector touches a fifth one.  Cycles per K block
  // of the logits GEMM, 1148 rows, V 50256: 868 at d = 1000 (2000-byte rows), 659 at
  // d = 1008, 595 at d = 1024; V = 50257 instead (rows of e): 667 at d = 1024.
  l.Vp = cdiv(p->V, 64) * 64;
  l.dp = cdiv(p->d, 64) * 64;
  l.tiles_v = static_cast<int>(cdiv(p->V, kBN));
  l.parts_v = l.tiles_v * kHalves;
  size_t off = 256;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += up256(bytes);
    return o;
  };
  const size_t C64 = static_cast<size_t>(l.C64), N = static_cast<size_t>(p->N > 0 ? p->N : 1);
  l.plan = take(static_cast<size_t>(l.nch > 0 ? l.nch : 1) * sizeof(ChunkPlan));
  l.perm = take(N * 4);
  l.cid = take(C64 * 4);
  l.rowin = take(C64 * sizeof(RowIn));
  l.factor = take(C64 * 4);
  l.clogp = take(C64 * 4);
  l.rowc = take(C64 * sizeof(float4));
  l.rl = take(N * 4);
  if (p->n_seqs > 0) {
    const size_t S = static_cast<size_t>(p->n_seqs);
    l.score = take(S * 8);
    l.count = take(S * 4);
    l.slope = take(S * 4);
  }
  l.Hc = take(C64 * l.dp * 2);
  l.part = take(C64 * l.parts_v * sizeof(float4));
  if (entry != KL_ENTRY_FWD) {
    l.E = take(C64 * l.Vp * 2);
    // dH parts, rows of 256: four K parts of a full chunk, up to 32 of a short one
    const int64_t full = 4 * cdiv(l.C, 256) * 256;
    l.part_rows = full > 32 * 256 ? full : 32 * 256;
    l.dHp = take(static_cast<size_t>(l.part_rows) * p->d * 4);
    if (p->dW_dtype == KL_DTYPE_BF16 && l.nch > 1)
      l.dWf = take(static_cast<size_t>(p->V) * p->d * 4);
  }
  l.total = off;
  return l;
}

struct LCtx {
  const kl_logp_problem* p;
  LPlan l;
  uint8_t* ws;
  Scalars* sc;
  cudaStream_t st;
  int sms;
  RowSelect sel;
  float normalizer = 0.f;
  template <typename T>
  T* at(size_t off) const {
    return reinterpret_cast<T*>(ws + off);
  }
  const ChunkPlan* plan(int64_t k) const { return at<const ChunkPlan>(l.plan) + k; }
  int64_t ldH() const { return p->ldH != 0 ? p->ldH : p->d; }
  int64_t in_chunk(int64_t k) const {
    const int64_t left = p->N - k * l.C;
    return left < l.C ? left : l.C;
  }
};

int begin(const kl_logp_problem* p, int entry, void* ws, size_t ws_bytes, void* stream, LCtx& c) {
  KL_TRY(check(p));
  DevInfo di;
  KL_TRY(current_device_info(&di));
  c.p = p;
  c.l = plan_of(p, entry);
  if (ws == nullptr) return KL_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(ws) & 255) return KL_ERR_ALIGN;
  if (ws_bytes < c.l.total) return KL_ERR_WORKSPACE;
  c.ws = static_cast<uint8_t*>(ws);
  c.sc = reinterpret_cast<Scalars*>(ws);
  c.st = static_cast<cudaStream_t>(stream);
  c.sms = di.sms;
  c.sel = RowSelect{p->ids, p->ids_64, p->mask, p->n_seqs > 0 ? p->cu_seqlens : nullptr,
                    static_cast<int>(p->n_seqs), p->N, static_cast<int>(p->V)};
  return KL_OK;
}

// dH on 256 x 512 tiles, whose halves share the rows of dS, unless parts of 16 K blocks
// cannot fill the CTA pairs: then 256 x 256 tiles need half as many parts to be
// written and summed (250 rows, d 1024, vocabulary 32000: GEMM and sum 38 to 33 us, timed
// launch by launch).
bool wide_dH(const LCtx& c) {
  const int64_t tiles = cdiv(c.in_chunk(0), 2 * kBM) * cdiv(c.p->d, 2 * kBN);
  return tiles * cdiv(c.p->V, 64 * 16) >= c.sms / 2;
}

Numbering numbering(const LCtx& c, float normalizer) {
  return Numbering{c.at<int>(c.l.perm), c.sc, c.at<ChunkPlan>(c.l.plan),
                   static_cast<int>(c.l.nch), static_cast<int>(c.l.C),
                   static_cast<int>(c.p->d), wide_dH(c) ? 2 : 1, c.sms / 2,
                   c.l.part_rows, normalizer};
}

// Few rows: the gather numbers them as well.
bool number_in_gather(const LCtx& c) {
  return c.l.nch == 1 && c.p->N <= kNumberRows && c.p->n_seqs <= kNumberRows;
}

// Start of a pass: numbers the rows (or leaves it to the gather).
int launch_compact(LCtx& c, float normalizer) {
  c.normalizer = normalizer;
  if (number_in_gather(c)) return KL_OK;
  LaunchScope ls("logp_compact", c.st, 0, static_cast<double>(c.p->N) * 9);
  return launch_dependent(logp_compact_kernel, 1, 1024, c.st, c.sel, c.p->T_row,
                          numbering(c, normalizer));
}

int launch_gather(LCtx& c, int64_t k) {
  const kl_logp_problem* p = c.p;
  LaunchScope ls("logp_gather", c.st, 0, 6.0 * c.in_chunk(k) * p->d);
  return launch_dependent(
      number_in_gather(c) ? logp_gather_kernel<true> : logp_gather_kernel<false>,
      static_cast<unsigned>(cdiv(c.in_chunk(k), 64) * 64), kGatherThreads, c.st,
      static_cast<const __nv_bfloat16*>(p->H), static_cast<const __nv_bfloat16*>(p->W),
      static_cast<int>(p->d), c.ldH(), c.sel, p->T_row, 1.f / p->T, numbering(c, c.normalizer),
      k * c.l.C, c.plan(k), c.at<__nv_bfloat16>(c.l.Hc), c.l.dp, c.at<int>(c.l.cid),
      c.at<RowIn>(c.l.rowin), c.l.E ? c.at<__nv_bfloat16>(c.l.E) : nullptr, c.l.Vp);
}

// Logits of chunk k: statistics, with e stored when `store` (EPI_LOGP), or dS from
// the rows' coefficients (EPI_DLOGP).
template <int EPI>
int gemm_rows(LCtx& c, int64_t k, bool store) {
  const kl_logp_problem* p = c.p;
  constexpr int kBKe = kRowBytes / 2;
  const int64_t d = p->d, rows = c.in_chunk(k);
  CUtensorMap ma, mb, mc;
  if (!make_map(&ma, c.at<void>(c.l.Hc), KL_DTYPE_BF16, d, c.l.C64, c.l.dp * 2, kBKe, kBM) ||
      !make_map(&mb, p->W, KL_DTYPE_BF16, d, p->V, d * 2, kBKe, kBN / 2))
    return KL_ERR_CUDA;
  mc = mb;
  if (store && !make_out_map(&mc, c.at<void>(c.l.E), KL_DTYPE_BF16, p->V, c.l.C64, c.l.Vp * 2))
    return KL_ERR_CUDA;
  GemmParams gp{};
  gp.tiles_m = static_cast<int>(cdiv(rows, 2 * kBM));
  gp.tiles_n = c.l.tiles_v;
  gp.num_kb = static_cast<int>(cdiv(d, kBKe));
  gp.m_fastest = 1;
  gp.store = store ? STORE_EXP : STORE_NONE;
  gp.rows_valid = static_cast<int>(rows);
  gp.cols_valid = static_cast<int>(p->V);
  gp.partials = c.at<float4>(c.l.part);
  gp.status = &c.sc->status;
  gp.spin_limit = spin_limit();
  gp.dyn = c.plan(k);
  gp.ids = c.at<int>(c.l.cid);
  gp.rowin = c.at<float4>(c.l.rowin);
  gp.entropy = p->entropy;
  gp.rowc = c.at<float4>(c.l.rowc);
  return launch_gemm<__nv_bfloat16, 0, 0, EPI, 1, 0, 0, kHalves, 1>(
      EPI == EPI_LOGP ? "gemm_logp" : "gemm_dlogp", c.st, c.sms, ma, mb, mc, gp,
      2.0 * rows * p->V * d);
}

int launch_rows(LCtx& c, int64_t k, const PolicyRows* pol, const RowOut& o, const RowBack& back) {
  const unsigned grid = static_cast<unsigned>(cdiv(c.in_chunk(k), 8));
  LaunchScope ls("logp_rows", c.st, 0,
                 c.in_chunk(k) * (c.l.parts_v * 16.0 + (back.E && !back.dense ? 4.0 * c.p->d : 0)));
  auto go = [&](auto kern, const PolicyRows& q) {
    return launch_dependent(kern, grid, 256, c.st, c.at<float4>(c.l.part), c.l.parts_v, c.plan(k),
                            k * c.l.C, static_cast<int>(c.in_chunk(k)), c.p->N, c.at<int>(c.l.perm),
                            c.at<int>(c.l.cid), c.at<RowIn>(c.l.rowin), c.p->entropy, q, c.sc, o,
                            back);
  };
  return pol != nullptr ? go(logp_rows_kernel<1>, *pol) : go(logp_rows_kernel<0>, PolicyRows{});
}

// The gradient's part of launch_rows.  dense: it has an entropy term.
RowBack row_back(LCtx& c, bool dense) {
  RowBack b{};
  b.E = c.at<__nv_bfloat16>(c.l.E);
  b.ld = c.l.Vp;
  b.dense = dense ? 1 : 0;
  b.H = static_cast<const __nv_bfloat16*>(c.p->H);
  b.ldH = c.ldH();
  b.Hc = c.at<__nv_bfloat16>(c.l.Hc);
  b.ldh = c.l.dp;
  b.d = static_cast<int>(c.p->d);
  b.V = static_cast<int>(c.p->V);
  b.factor = c.at<float>(c.l.factor);
  b.rowc = c.at<float4>(c.l.rowc);
  b.clogp = c.at<float>(c.l.clogp);
  b.g_host = 1.f;
  return b;
}

int launch_dlogits(LCtx& c, int64_t k) {
  LaunchScope ls("logp_dlogits", c.st, 0, 4.0 * c.in_chunk(k) * c.p->V);
  return launch_dependent(logp_dlogits_kernel, static_cast<unsigned>(c.in_chunk(k)), 512, c.st,
                          c.at<__nv_bfloat16>(c.l.E), c.l.Vp, static_cast<int>(c.p->V),
                          c.at<float4>(c.l.part), c.l.parts_v, c.plan(k), c.at<int>(c.l.cid),
                          c.at<float>(c.l.clogp), c.at<float4>(c.l.rowc));
}

// The own tokens' entries after gemm_rows<EPI_DLOGP>.
int launch_own(LCtx& c, int64_t k) {
  LaunchScope ls("logp_own", c.st, 0, c.in_chunk(k) * (4.0 * c.l.parts_v + 38));
  return launch_dependent(logp_own_kernel, static_cast<unsigned>(cdiv(c.in_chunk(k), 8)), 256, c.st,
                          c.at<__nv_bfloat16>(c.l.E), c.l.Vp, static_cast<int>(c.p->V),
                          c.at<float>(c.l.part), c.l.parts_v, c.plan(k),
                          static_cast<int>(c.in_chunk(k)), c.at<int>(c.l.cid),
                          c.at<RowIn>(c.l.rowin), c.at<float4>(c.l.rowc));
}

int launch_mean(LCtx& c, const float* x, int64_t n, bool norm, float given, float* loss) {
  LaunchScope ls("logp_mean", c.st, 0, 4.0 * n);
  return launch_dependent(logp_mean_kernel, 1, 1024, c.st, x, n, norm ? &c.sc->norm : nullptr,
                          given, loss);
}

// A bf16 dW from the fp32 sums over all chunks.
int launch_round_dW(LCtx& c, void* dW) {
  const int64_t n = c.p->V * c.p->d;
  LaunchScope ls("logp_round", c.st, 0, 6.0 * n);
  return launch_dependent(logp_round_kernel, static_cast<unsigned>(c.sms * 8), 256, c.st,
                          c.at<float>(c.l.dWf), static_cast<__nv_bfloat16*>(dW), n / 8);
}

// dH rows of chunk k and its share of dW (beta: added to what dW holds) from dS, either
// of them where wanted.  loss, where not nullptr: the mean of the row losses, with the
// last chunk.
int grads(LCtx& c, int64_t k, void* dH, void* dW, int beta, const float* row_loss = nullptr,
          float* loss = nullptr) {
  const kl_logp_problem* p = c.p;
  constexpr int kBKe = kRowBytes / 2, kMNe = kRowBytes / 2;
  const int64_t d = p->d, rows = c.in_chunk(k);
  void* E = c.at<void>(c.l.E);
  const bool mean = loss != nullptr && k == c.l.nch - 1;
  if (dH != nullptr) {
    CUtensorMap ma, mb, mc;
    if (!make_map(&ma, E, KL_DTYPE_BF16, p->V, c.l.C64, c.l.Vp * 2, kBKe, kBM) ||
        !make_map(&mb, p->W, KL_DTYPE_BF16, d, p->V, d * 2, kMNe, kBKe) ||
        !make_out_map(&mc, c.at<void>(c.l.dHp), KL_DTYPE_F32, d, c.l.part_rows, d * 4))
      return KL_ERR_CUDA;
    GemmParams gp{};
    gp.tiles_m = static_cast<int>(cdiv(rows, 2 * kBM));
    const bool wide = wide_dH(c);
    gp.tiles_n = static_cast<int>(cdiv(d, wide ? 2 * kBN : kBN));
    gp.num_kb = static_cast<int>(cdiv(p->V, kBKe));
    gp.m_fastest = 1;
    gp.ksplit = 32;  // the most; the kernel takes the plan's
    gp.rows_valid = static_cast<int>(rows);
    gp.cols_valid = static_cast<int>(d);
    gp.status = &c.sc->status;
    gp.spin_limit = spin_limit();
    gp.dyn = c.plan(k);
    const double flops = 2.0 * rows * p->V * d;
    if (wide)
      KL_TRY((launch_gemm<__nv_bfloat16, 0, 1, EPI_ACCUM, 1, 1, 0, 1, 1>("gemm_dH", c.st, c.sms, ma,
                                                                         mb, mc, gp, flops)));
    else
      KL_TRY((launch_gemm<__nv_bfloat16, 0, 1, EPI_ACCUM, 1, 0, 0, 1, 1>("gemm_dH", c.st, c.sms, ma,
                                                                         mb, mc, gp, flops)));
    LaunchScope ls("logp_dh", c.st, 0, 6.0 * rows * d);
    KL_TRY(launch_dependent(logp_dh_kernel, static_cast<unsigned>(rows + (mean ? 1 : 0)), 256, c.st,
                            c.at<float>(c.l.dHp), c.plan(k), k * c.l.C, c.at<int>(c.l.perm),
                            c.at<float>(c.l.factor), static_cast<int>(d),
                            static_cast<__nv_bfloat16*>(dH), static_cast<int>(rows),
                            c.l.part_rows, row_loss, p->N, c.sc, loss));
  } else if (mean) {
    KL_TRY(launch_mean(c, row_loss, p->N, true, 0.f, loss));
  }
  if (dW == nullptr) return KL_OK;
  const bool direct = p->dW_dtype == KL_DTYPE_BF16 && c.l.nch == 1;
  void* out = p->dW_dtype == KL_DTYPE_F32 || direct ? dW : c.at<void>(c.l.dWf);
  CUtensorMap ma, mb, mc;
  if (!make_map(&ma, E, KL_DTYPE_BF16, p->V, c.l.C64, c.l.Vp * 2, kMNe, kBKe) ||
      !make_map(&mb, c.at<void>(c.l.Hc), KL_DTYPE_BF16, d, c.l.C64, c.l.dp * 2, kMNe, kBKe) ||
      !make_out_map(&mc, out, direct ? KL_DTYPE_BF16 : KL_DTYPE_F32, d, p->V,
                    d * (direct ? 2 : 4)))
    return KL_ERR_CUDA;
  GemmParams gp{};
  gp.tiles_m = static_cast<int>(cdiv(p->V, 2 * kBM));
  gp.tiles_n = static_cast<int>(cdiv(d, kBN));
  gp.num_kb = static_cast<int>(cdiv(rows, kBKe));
  gp.m_fastest = 0;
  gp.rows_valid = static_cast<int>(p->V);
  gp.cols_valid = static_cast<int>(d);
  gp.beta = beta;
  gp.status = &c.sc->status;
  gp.spin_limit = spin_limit();
  gp.dyn = c.plan(k);
  gp.dyn_k = 1;
  const double flops = 2.0 * rows * p->V * d;
  if (direct)
    return launch_gemm<__nv_bfloat16, 1, 1, EPI_STORE, 1, 0, 0, 2, 1>("gemm_dW", c.st, c.sms, ma,
                                                                      mb, mc, gp, flops);
  KL_TRY((launch_gemm<__nv_bfloat16, 1, 1, EPI_ACCUM, 1, 0, 0, 1, 1>("gemm_dW", c.st, c.sms, ma,
                                                                     mb, mc, gp, flops)));
  if (p->dW_dtype == KL_DTYPE_BF16 && k == c.l.nch - 1)
    return launch_round_dW(c, dW);
  return KL_OK;
}

// No rows at all: dW gets zeros unless it accumulates.
int empty_dW(LCtx& c, void* dW, int accumulate) {
  if (accumulate || dW == nullptr) return KL_OK;
  const size_t bytes =
      static_cast<size_t>(c.p->V) * c.p->d * (c.p->dW_dtype == KL_DTYPE_F32 ? 4 : 2);
  return cudaMemsetAsync(dW, 0, bytes, c.st) == cudaSuccess ? KL_OK : KL_ERR_CUDA;
}

// Forward over the chunks, the first chunk last: it is the one that always holds
// rows, and keep_chunk leaves its exponentials for the backward.
int run_fwd(LCtx& c, const PolicyRows* pol, float normalizer, const RowOut& o) {
  KL_TRY(launch_compact(c, normalizer));
  for (int64_t k = c.l.nch - 1; k >= 0; --k) {
    KL_TRY(launch_gather(c, k));
    KL_TRY(gemm_rows<EPI_LOGP>(c, k, c.p->keep_chunk && k == 0));
    KL_TRY(launch_rows(c, k, pol, o, RowBack{}));
  }
  return KL_OK;
}

int check_grads(const kl_logp_problem* p, const void* dH, const void* dW, int accumulate) {
  if (p->N > 0 && dW == nullptr && dH == nullptr) return KL_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(dH) | reinterpret_cast<uintptr_t>(dW)) & 15)
    return KL_ERR_ALIGN;
  if (accumulate && p->dW_dtype != KL_DTYPE_F32) return KL_ERR_DTYPE;
  return KL_OK;
}

int check_policy(const kl_logp_problem* p, const kl_policy* q) {
  if (q == nullptr) return KL_ERR_NULL;
  if (!(q->clip_low >= 0.f && q->clip_low <= 1.f) || !(q->clip_high >= 0.f) ||
      !(q->dual_clip == 0.f || q->dual_clip > 1.f) || !(q->kl_coef >= 0.f) ||
      !(q->kl_coef < INFINITY) || !(fabsf(q->entropy_coef) < INFINITY) ||
      !(q->normalizer >= 0.f) || !(q->normalizer < INFINITY))
    return KL_ERR_ARG;
  if (q->entropy_coef != 0.f && !p->entropy) return KL_ERR_ARG;
  if (p->N > 0 && (q->advantage == nullptr || (q->kl_coef != 0.f && q->ref_logp == nullptr)))
    return KL_ERR_NULL;
  return KL_OK;
}

PolicyRows policy_rows(const kl_policy* q) {
  return PolicyRows{q->advantage, q->old_logp,  q->ref_logp, q->row_weight,  q->clip_low,
                    q->clip_high, q->dual_clip, q->kl_coef,  q->entropy_coef};
}

}  // namespace

extern "C" {

size_t kl_logp_workspace_bytes(const kl_logp_problem* p, int entry) {
  if (check_shape(p) != KL_OK || entry < KL_ENTRY_FWD || entry > KL_ENTRY_FWD_BWD) return 0;
  return plan_of(p, entry).total;
}

int kl_logp_fwd(const kl_logp_problem* p, void* ws, size_t ws_bytes, float* logp, float* entropy,
                float* lse, void* stream) {
  LCtx c;
  KL_TRY(check(p));
  if (p->N > 0 && (logp == nullptr || (p->entropy && entropy == nullptr))) return KL_ERR_NULL;
  KL_TRY(begin(p, KL_ENTRY_FWD, ws, ws_bytes, stream, c));
  RowOut o{};
  o.logp = logp;
  o.ent = p->entropy ? entropy : nullptr;
  o.lse = lse;
  return run_fwd(c, nullptr, 0.f, o);
}

int kl_logp_bwd(const kl_logp_problem* p, void* ws, size_t ws_bytes, const float* lse,
                const float* entropy, const float* g_logp, const float* g_entropy,
                const float* grad_loss, void* dH, void* dW, int accumulate_dW, void* stream) {
  LCtx c;
  KL_TRY(check(p));
  if (p->N > 0 && (lse == nullptr || g_logp == nullptr ||
                   (g_entropy != nullptr && entropy == nullptr)))
    return KL_ERR_NULL;
  KL_TRY(check_grads(p, dH, dW, accumulate_dW));
  KL_TRY(begin(p, KL_ENTRY_BWD, ws, ws_bytes, stream, c));
  // keep_chunk: the forward left the rows' numbering and the first chunk's rows too
  if (!p->keep_chunk) KL_TRY(launch_compact(c, 0.f));
  if (p->N == 0) return empty_dW(c, dW, accumulate_dW);
  for (int64_t k = 0; k < c.l.nch; ++k) {
    if (!p->keep_chunk || k > 0) KL_TRY(launch_gather(c, k));
    if (p->keep_chunk && k == 0) {
      RowBack b = row_back(c, g_entropy != nullptr);
      b.g_logp = g_logp;
      b.g_ent = g_entropy;
      b.ent = entropy;
      b.g_dev = grad_loss;
      KL_TRY(launch_rows(c, k, nullptr, RowOut{}, b));
      if (b.dense) KL_TRY(launch_dlogits(c, k));
    } else {
      {
        LaunchScope ls("logp_coef", c.st, 0, 36.0 * c.in_chunk(k));
        KL_TRY(launch_dependent(logp_coef_kernel,
                                static_cast<unsigned>(cdiv(c.in_chunk(k), 128)), 128, c.st,
                                c.plan(k), k * c.l.C, static_cast<int>(c.in_chunk(k)), p->N,
                                c.at<int>(c.l.perm), c.at<RowIn>(c.l.rowin), lse, entropy, g_logp,
                                g_entropy, grad_loss, c.at<float4>(c.l.rowc),
                                c.at<float>(c.l.factor)));
      }
      KL_TRY(gemm_rows<EPI_DLOGP>(c, k, true));
      KL_TRY(launch_own(c, k));
    }
    KL_TRY(grads(c, k, dH, dW, accumulate_dW || k > 0));
  }
  return KL_OK;
}

int kl_policy_fwd(const kl_logp_problem* p, const kl_policy* q, void* ws, size_t ws_bytes,
                  float* loss, float* row_loss, float* logp, float* entropy, float* lse,
                  float* g_logp, float* g_entropy, void* stream) {
  LCtx c;
  KL_TRY(check(p));
  KL_TRY(check_policy(p, q));
  if (loss == nullptr ||
      (p->N > 0 && g_logp != nullptr && q->entropy_coef != 0.f && g_entropy == nullptr))
    return KL_ERR_NULL;
  KL_TRY(begin(p, KL_ENTRY_FWD, ws, ws_bytes, stream, c));
  RowOut o{};
  o.logp = logp;
  o.ent = p->entropy ? entropy : nullptr;
  o.lse = lse;
  o.row_loss = row_loss != nullptr ? row_loss : c.at<float>(c.l.rl);
  o.g_logp = g_logp;
  o.g_ent = g_entropy;
  const PolicyRows pol = policy_rows(q);
  KL_TRY(run_fwd(c, &pol, q->normalizer, o));
  return launch_mean(c, o.row_loss, p->N, true, 0.f, loss);
}

int kl_policy_fwd_bwd(const kl_logp_problem* p, const kl_policy* q, void* ws, size_t ws_bytes,
                      float grad_loss, float* loss, float* row_loss, float* logp, float* entropy,
                      void* dH, void* dW, int accumulate_dW, void* stream) {
  LCtx c;
  KL_TRY(check(p));
  KL_TRY(check_policy(p, q));
  if (p->keep_chunk) return KL_ERR_ARG;
  if (loss == nullptr) return KL_ERR_NULL;
  KL_TRY(check_grads(p, dH, dW, accumulate_dW));
  KL_TRY(begin(p, KL_ENTRY_FWD_BWD, ws, ws_bytes, stream, c));
  RowOut o{};
  o.logp = logp;
  o.ent = p->entropy ? entropy : nullptr;
  o.row_loss = row_loss != nullptr ? row_loss : c.at<float>(c.l.rl);
  RowBack back = row_back(c, q->entropy_coef != 0.f);
  back.g_host = grad_loss;
  const PolicyRows pol = policy_rows(q);
  KL_TRY(launch_compact(c, q->normalizer));
  if (p->N == 0) KL_TRY(empty_dW(c, dW, accumulate_dW));
  for (int64_t k = 0; k < c.l.nch; ++k) {
    KL_TRY(launch_gather(c, k));
    KL_TRY(gemm_rows<EPI_LOGP>(c, k, true));
    KL_TRY(launch_rows(c, k, &pol, o, back));
    if (back.dense) KL_TRY(launch_dlogits(c, k));
    KL_TRY(grads(c, k, dH, dW, accumulate_dW || k > 0, o.row_loss, loss));
  }
  return p->N > 0 ? KL_OK : launch_mean(c, o.row_loss, 0, true, 0.f, loss);
}

int kl_preference_fwd(const kl_logp_problem* p, const kl_preference* q, void* ws, size_t ws_bytes,
                      float* loss, float* pair_loss, float* seq_logp, float* logp, float* lse,
                      float* g_logp, void* stream) {
  LCtx c;
  KL_TRY(check(p));
  if (q == nullptr) return KL_ERR_NULL;
  if (q->n_pairs < 0 || q->n_pairs > kMaxSeqs) return KL_ERR_SHAPE;
  if (q->pairs == nullptr && 2 * q->n_pairs != p->n_seqs) return KL_ERR_SHAPE;
  if (q->n_pairs > 0 && p->n_seqs == 0) return KL_ERR_SHAPE;
  if (q->loss < KL_PREFERENCE_SIGMOID || q->loss > KL_PREFERENCE_HINGE ||
      !(q->beta > 0.f && q->beta < INFINITY) || !(q->label_smoothing >= 0.f) ||
      !(q->label_smoothing < 0.5f) || !(fabsf(q->margin) < INFINITY) ||
      (q->average != 0 && q->average != 1) || !(q->normalizer >= 0.f) ||
      !(q->normalizer < INFINITY) ||
      (q->label_smoothing != 0.f && q->loss != KL_PREFERENCE_SIGMOID) ||
      (q->margin != 0.f && q->loss == KL_PREFERENCE_SQUARED))
    return KL_ERR_ARG;
  if (loss == nullptr || (q->n_pairs > 0 && pair_loss == nullptr) ||
      (p->N > 0 && (logp == nullptr || g_logp == nullptr)))
    return KL_ERR_NULL;
  KL_TRY(begin(p, KL_ENTRY_FWD, ws, ws_bytes, stream, c));
  RowOut o{};
  o.logp = logp;
  o.lse = lse;
  KL_TRY(run_fwd(c, nullptr, 0.f, o));
  const int S = static_cast<int>(p->n_seqs), P = static_cast<int>(q->n_pairs);
  const float divisor = q->normalizer > 0.f ? q->normalizer : static_cast<float>(P);
  const PrefPairs pp{q->pairs, P, S, q->ref_logp, q->loss, q->beta, q->label_smoothing, q->margin};
  const PrefScores ps{c.at<double>(c.l.score), c.at<int>(c.l.count), c.at<float>(c.l.slope),
                      seq_logp, q->average, divisor};
  if (p->N > 0 && p->N <= kPrefSmall && S <= kPrefSmall && P <= kPrefSmall && S > 0) {
    LaunchScope ls("pref_small", c.st, 0, 22.0 * p->N);
    return launch_dependent(pref_small_kernel, 1, 1024, c.st, c.sel, logp, c.sc, pp, ps, pair_loss,
                            g_logp, &c.sc->status, loss);
  }
  if (S > 0) {
    {
      LaunchScope ls("pref_sum", c.st, 0, 9.0 * p->N);
      KL_TRY(launch_dependent(pref_sum_kernel, static_cast<unsigned>(S), 256, c.st, c.sel, logp,
                              c.sc, ps));
    }
    LaunchScope ls("pref_pair", c.st, 0, 0);
    KL_TRY(launch_dependent(pref_pair_kernel, static_cast<unsigned>(cdiv(S > P ? S : P, 8)), 256,
                            c.st, pp, ps, pair_loss, &c.sc->status));
  }
  LaunchScope ls("pref_rows", c.st, 0, 13.0 * p->N);
  return launch_dependent(pref_rows_kernel, static_cast<unsigned>(cdiv(p->N, 256) + 1), 256, c.st,
                          c.sel, c.sc, c.at<float>(c.l.slope), g_logp, pair_loss, S > 0 ? P : 0,
                          divisor, loss);
}

}  // extern "C"
