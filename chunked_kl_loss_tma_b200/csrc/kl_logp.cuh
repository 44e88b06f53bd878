// kl_logp.cuh -- row kernels of the token log-probability operators: the log-
// probability and entropy of each row's token under softmax(H W^T / T), the
// clipped policy loss and the preference loss built on them, and their
// gradients with respect to the logits.
//
//   z = s / T,  lse = log sum_j exp z_j,  p = exp(z - lse)
//   logp = z_id - lse,   ent = lse - sum_j p_j z_j
//   d logp / d z_j = [j = id] - p_j,   d ent / d z_j = -p_j (ln p_j + ent)
//
// so with g = dL/dlogp and h = dL/dent every loss here has
//   dS_j = a [j = id] - p_j (a + b (ln p_j + ent)),   a = g / T,  b = h / T.
//
// Rows that take no part (masked, a negative token id, behind the last packed
// sequence) are left out before the contractions: the rows that do are numbered
// consecutively (compact rows), their hidden states are gathered, and the
// contractions run over them alone, with the counts read on the device.  In a
// policy step with 35% of the rows masked that is a third of the work; the
// gather costs 6 d bytes a row (17 us for 2663 of 4096 rows at d 4096, of 6.7 ms).
#pragma once
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "kl_gemm.cuh"
#include "kl_rowutil.cuh"

namespace ckl {

// Epilogue groups of the logits GEMMs, each with half the columns of a tile: half the
// tail of the last tile, and shorter epilogues where they bind (2048 rows, d 256: the
// MMA thread still waits for them half of its time; at d 1000 it does not, and one
// group or two take 127 us).
constexpr int kHalves = 2;
constexpr int kPartVecs = kBN / kHalves / 8;  // vectors of 8 columns that share a partial

// What selects the rows that take part.
struct RowSelect {
  const void* ids;       // [N] int32 or int64
  int ids_64;
  const uint8_t* mask;   // [N] or nullptr
  const int* cu;         // [S + 1] packed sequence offsets, or nullptr
  int S;
  int64_t N;
  int V;
};

// The row's token, or -1 when the row takes no part; *bad: an id >= V.
__device__ __forceinline__ int row_token(const RowSelect& s, int64_t row, bool* bad) {
  if (s.mask != nullptr && s.mask[row] == 0) return -1;
  const int64_t id = s.ids_64 ? static_cast<const int64_t*>(s.ids)[row]
                              : static_cast<const int32_t*>(s.ids)[row];
  if (id >= s.V) {
    *bad = true;
    return -1;
  }
  return id < 0 ? -1 : static_cast<int>(id);
}

// K parts of the dH contraction of one chunk: `tiles` output tiles of 256 x 256 wide,
// num_kb K blocks, `units` CTA pairs, at most cap <= 32 parts; lane s - 1 weighs s
// parts.  In units of one K block of a 256 x 256 tile (0.4 us): waves x (K blocks of
// a part + 5 for the tile's epilogue) x wide + the parts' write and read, 8 bytes per
// value and part at about 5 TB/s from L2.
__device__ __forceinline__ int plan_ksplit(int rows, int d, int tiles, int wide, int num_kb,
                                           int units, int cap) {
  const int s = (threadIdx.x & 31) + 1;
  const int kbs = (num_kb + s - 1) / s;
  const int waves = (tiles * s + units - 1) / units;
  float cost = static_cast<float>(waves * wide) * (kbs + 5) +
               static_cast<float>(s) * rows * d * (1.f / 250000.f);
  // no part shorter than 8 blocks, none empty
  if (s > 1 && (s > cap || kbs < 8 || (s - 1) * kbs >= num_kb)) cost = 3.4e38f;
  float best = cost;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, o));
  return __ffs(__ballot_sync(0xffffffffu, cost == best));
}

// Rows of a chunk and the row behind a compact one, kept within their buffers: a kept
// workspace that is not the forward's holds anything.
__device__ __forceinline__ int rows_of(const ChunkPlan* plan, int most) {
  return max(0, min(plan->rows, most));
}
__device__ __forceinline__ int row_of(const int* perm, int64_t at, int64_t N) {
  const int row = perm[at];
  return row >= 0 && row < N ? row : 0;
}

// What the numbering of the rows leaves for the other kernels.
struct Numbering {
  int* perm;        // [N]: the rows that take part in order, then the others from the end back
  Scalars* sc;      // status word reset, count, the loss's divisor
  ChunkPlan* plan;  // [nch]
  int nch, C, d, wide, units;
  int64_t part_rows;
  float normalizer;
};

// Numbers the rows that take part, by one CTA of THREADS threads, 4 rows a thread and
// step.  WRITE: leaves the Numbering; else only finds the row numbered `want`.  Returns
// the number of rows; *found (shared) the wanted row.
template <int THREADS>
__device__ __forceinline__ int number_rows(const RowSelect& sel, const float* T_row,
                                           const Numbering& o, bool write, int want, int* found) {
  constexpr int kWarps = THREADS / 32;
  __shared__ int wsum[kWarps];
  __shared__ int status, total;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    status = 0;
    total = 0;
  }
  __syncthreads();
  int64_t lo = 0, hi = sel.N;
  if (sel.cu != nullptr) {
    bool ok = true;
    for (int s = threadIdx.x; s < sel.S; s += THREADS)
      ok &= sel.cu[s] >= 0 && sel.cu[s + 1] >= sel.cu[s] && sel.cu[s + 1] <= sel.N;
    if (!__syncthreads_and(ok)) {
      if (threadIdx.x == 0) atomicCAS(&status, 0, kStatusIndex);
      hi = 0;  // bad offsets: no row takes part
    } else {
      lo = sel.cu[0];
      hi = sel.cu[sel.S];
    }
  }
  for (int64_t base = 0; base < sel.N; base += 4 * THREADS) {
    const int64_t r0 = base + 4 * threadIdx.x;
    int keep = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = r0 + i;
      if (row < lo || row >= hi || row >= sel.N) continue;
      bool bad = false;
      const int id = row_token(sel, row, &bad);
      if (bad) atomicCAS(&status, 0, kStatusIndex);
      if (id >= 0) {
        keep |= 1 << i;
        if (T_row != nullptr && !(T_row[row] > 0.f)) atomicCAS(&status, 0, kStatusArg);
      }
    }
    const int n = __popc(keep);
    int incl = n;
#pragma unroll
    for (int o2 = 1; o2 < 32; o2 <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o2);
      if (lane >= o2) incl += t;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      int v = lane < kWarps ? wsum[lane] : 0;
#pragma unroll
      for (int o2 = 1; o2 < kWarps; o2 <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, v, o2);
        if (lane >= o2) v += t;
      }
      if (lane < kWarps) wsum[lane] = v;
    }
    __syncthreads();
    int pos = total + (warp > 0 ? wsum[warp - 1] : 0) + incl - n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = r0 + i;
      if (row >= sel.N) break;
      if (keep >> i & 1) {
        if (write) o.perm[pos] = static_cast<int>(row);
        if (pos == want) *found = static_cast<int>(row);
        ++pos;
      } else if (write) {
        o.perm[sel.N - 1 - (row - pos)] = static_cast<int>(row);  // row - pos: left out before it
      }
    }
    __syncthreads();
    if (threadIdx.x == 0) total += wsum[kWarps - 1];
    __syncthreads();
  }
  if (write) {
    if (threadIdx.x == 0) {
      o.sc->status = status;
      o.sc->n_valid = total;
      o.sc->norm = o.normalizer > 0.f ? o.normalizer : static_cast<float>(total);
    }
    for (int k = warp; k < o.nch; k += kWarps) {
      const int64_t left = total - static_cast<int64_t>(k) * o.C;
      const int rows = left <= 0 ? 0 : left < o.C ? static_cast<int>(left) : o.C;
      const int tm = (rows + 2 * kBM - 1) / (2 * kBM);
      const int tn = (o.d + o.wide * kBN - 1) / (o.wide * kBN);
      int ks = 1;
      if (tm > 0 && o.part_rows > 0) {
        const int64_t fit = o.part_rows / (tm * 2 * kBM);
        ks = plan_ksplit(rows, o.d, tm * tn, o.wide, (sel.V + 63) / 64, o.units,
                         fit < 32 ? static_cast<int>(fit) : 32);
      }
      if (lane == 0) o.plan[k] = ChunkPlan{rows, ks};
    }
  }
  return total;
}

__global__ void __launch_bounds__(1024)
    logp_compact_kernel(RowSelect sel, const float* T_row, Numbering o) {
  grid_dep_wait();
  number_rows<1024>(sel, T_row, o, true, -1, nullptr);
}

// The tensor core adds each K = 16 step into the fp32 accumulator and truncates towards
// zero, which takes a share of what the accumulator holds at each step.  Over a logit
// whose products add up in one direction that is between nothing (all of it in one step,
// the others add 0) and twice c steps (all of it in the first step, small products in the
// others); c steps where it grows evenly, as with products that are alike along d.
// Measured slope of (logit - exact logit) on the exact logit there, d = 512 to 8192:
// -1.6e-8 per step (-4.1e-6 at d = 4096).  The logits' scale carries the inverse, the
// middle of the two.  The own token's logit is formed apart and needs none.  Rms errors
// of log-probabilities at d = 4096, without and with it: even growth 5.8e-7 and 3.4e-8
// (tokens at -0.12), 3.9e-6 and 4.0e-7 (at -9.5); cancelling halves 4.2e-7 and 5.2e-7;
// all of the logit in one step 2.7e-7 and 2.6e-5 (logits up to 32): within the bound
// that any input has, 2^-23 per step of the largest partial sum.
constexpr double kTruncPerStep = 1.62e-8;

// What the logits epilogue and the row kernels know of a compact row beforehand.
struct RowIn {
  float scale2;  // log2 e / T, with the truncation's inverse
  float ref;     // r: the logit of the row's own token in base 2, rounded,
  float ref_lo;  // and what the rounding left
  float invT;
};

// One CTA per compact row of the chunk: its hidden state, token and reference
// logit (fp32 products, exact in themselves, summed in fp32 within a thread and
// in fp64 across; 2 d bytes of W a row); zero hidden states up to a whole tile or
// the buffer's end, past which TMA fills zeros (and, in an empty chunk, zero dS rows E).
// NUMBER (up to kNumberRows rows, one step of the numbering): every CTA numbers the
// rows for itself and the first one leaves the numbering, so that short calls have
// one launch less (4 of 81 us at 250 rows).
constexpr int kGatherThreads = 128;
constexpr int kNumberRows = 4 * kGatherThreads;
template <bool NUMBER>
__global__ void __launch_bounds__(kGatherThreads)
    logp_gather_kernel(const __nv_bfloat16* H, const __nv_bfloat16* W,
                       int d, int64_t ldH, RowSelect sel, const float* T_row, float invT,
                       Numbering num, int64_t c0, const ChunkPlan* plan,
                       __nv_bfloat16* Hc, int64_t ldh, int* cid,
                       RowIn* rowin, __nv_bfloat16* E, int64_t ld) {
  grid_dep_wait();
  __shared__ int found;
  const int i = blockIdx.x;
  int rows, row = 0;
  if (NUMBER) {
    rows = number_rows<kGatherThreads>(sel, T_row, num, i == 0, i, &found);
    if (i < rows) row = found;  // written before number_rows' last barrier
  } else {
    rows = rows_of(plan, num.C);
    if (i < rows) row = row_of(num.perm, c0 + i, sel.N);
  }
  uint4* dst = reinterpret_cast<uint4*>(Hc + static_cast<int64_t>(i) * ldh);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (i >= rows) {
    if (i >= (rows + 255) / 256 * 256 && i >= 64) return;
    for (int v = threadIdx.x; v < d / 8; v += kGatherThreads) dst[v] = zero;
    if (rows == 0 && E != nullptr && i < 64) {
      uint4* e = reinterpret_cast<uint4*>(E + static_cast<int64_t>(i) * ld);
      for (int64_t v = threadIdx.x; v < ld / 8; v += kGatherThreads) e[v] = zero;
    }
    return;
  }
  __shared__ double red[kGatherThreads / 32];
  bool bad = false;
  const int id = max(row_token(sel, row, &bad), 0);
  const uint4* src = reinterpret_cast<const uint4*>(H + row * ldH);
  const uint4* w = reinterpret_cast<const uint4*>(W + static_cast<int64_t>(id) * d);
  float s = 0.f;
  for (int v0 = threadIdx.x; v0 < d / 8; v0 += 4 * kGatherThreads) {
    uint4 a[4], b[4];  // all loads before the first store
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = v0 + j * kGatherThreads;
      a[j] = v < d / 8 ? src[v] : zero;
      b[j] = v < d / 8 ? w[v] : zero;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = v0 + j * kGatherThreads;
      if (v < d / 8) dst[v] = a[j];
      const uint32_t x[4] = {a[j].x, a[j].y, a[j].z, a[j].w};
      const uint32_t y[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s = fmaf(__uint_as_float(x[k] << 16), __uint_as_float(y[k] << 16), s);
        s = fmaf(__uint_as_float(x[k] & 0xffff0000u), __uint_as_float(y[k] & 0xffff0000u), s);
      }
    }
  }
  const double t = warp_sum_d(s);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    double z = 0.0;
    for (int k = 0; k < kGatherThreads / 32; ++k) z += red[k];
    const float it = row_invT(T_row, row, invT);
    constexpr double kLog2eD = 1.4426950408889634;
    z *= kLog2eD * it;
    RowIn r;
    r.scale2 = static_cast<float>(kLog2eD * it * (1.0 + kTruncPerStep * ((d + 15) / 16)));
    r.ref = static_cast<float>(z);
    r.ref_lo = static_cast<float>(z - r.ref);
    r.invT = it;
    rowin[i] = r;
    cid[i] = id;
  }
}

// The clipped policy loss of a row (pointers over the original rows).
struct PolicyRows {
  const float* advantage;
  const float* old_logp;    // or nullptr: the current policy's own (ratio 1)
  const float* ref_logp;    // or nullptr when kl_coef is 0
  const float* row_weight;  // or nullptr
  float clip_low, clip_high, dual_clip, kl_coef, entropy_coef;
};

// l = max(-A r, -A clip(r, 1 - low, 1 + high)), r = exp(logp - old), bounded by
// -A dual_clip for A < 0 when dual_clip > 0; + kl_coef (e^t - t - 1) with
// t = ref - logp; - entropy_coef ent; times the row's weight.  g = dl/dlogp,
// h = dl/dent.  A zero advantage has no surrogate, whatever the ratio.  A NaN ratio stays
// NaN in l and g (the clip alone would make a number of it), and so does a NaN logp where
// the surrogate does not depend on it.
struct PolicyIn {
  float advantage, old_logp, ref_logp, weight;
};
__device__ __forceinline__ PolicyIn policy_in(const PolicyRows& q, int row) {
  return PolicyIn{q.advantage[row], q.old_logp != nullptr ? q.old_logp[row] : 0.f,
                  q.kl_coef != 0.f ? q.ref_logp[row] : 0.f,
                  q.row_weight != nullptr ? q.row_weight[row] : 1.f};
}
__device__ __forceinline__ float policy_row(const PolicyRows& q, const PolicyIn& in, float logp,
                                            float ent, float* g, float* h) {
  const float A = in.advantage;
  float l = 0.f, dl = 0.f;
  if (A != 0.f) {
    const float r = q.old_logp != nullptr ? expf(logp - in.old_logp) : 1.f;
    const float u = -A * r;
    const float c = -A * fminf(fmaxf(r, 1.f - q.clip_low), 1.f + q.clip_high);
    l = u < c ? c : u;
    dl = u < c ? 0.f : u;  // d(-A r)/dlogp = -A r
    if (A < 0.f && q.dual_clip > 0.f && l > -A * q.dual_clip) {
      l = -A * q.dual_clip;
      dl = 0.f;
    }
  }
  if (isnan(logp)) l = dl = logp;
  if (q.kl_coef != 0.f) {
    const float t = in.ref_logp - logp, em1 = expm1f(t);
    l += q.kl_coef * (em1 - t);
    dl -= q.kl_coef * em1;
  }
  const float w = in.weight;
  if (q.entropy_coef != 0.f) l -= q.entropy_coef * ent;
  *g = w * dl;
  *h = -w * q.entropy_coef;
  return w * l;
}

struct RowOut {
  float* logp;      // [N] each, original rows; 0 where a row takes no part; may be nullptr
  float* ent;
  float* lse;
  float* row_loss;  // policy
  float* g_logp;    // policy: dloss/dlogp and dloss/dent of the mean loss
  float* g_ent;
};

// What a row's gradient is formed from, and where it goes (fused passes).
//
// Without an entropy term dS_j = -(a / Z) (e_j - Z [j = id]), Z = sum_j e_j: the
// stored exponentials are dS up to one factor per row.  So no pass over the chunk
// turns them into dS.  The own token's entry becomes e_id - Z = -(sum of the
// others), accurate however near 1 its probability is; the factor goes onto the
// rows of dH as they are summed, and onto the rows of H that dW contracts.  So dW's
// products carry two roundings to bf16, of e and of the scaled row, where a stored dS
// has one: 2.3e-3 from the 64-bit dW, in fp32 or bf16, where one rounding of the result
// is 1.7e-3.  At 8192 rows and a vocabulary of 128256 the pass took 0.75 of 19.5 ms.
// With an entropy term (b != 0) the factor differs along the row and the pass runs
// (logp_dlogits_kernel).
struct RowBack {
  __nv_bfloat16* E;     // stored exponentials [.][ld], or nullptr: no gradient wanted
  int64_t ld;
  int dense;            // 1: the pass runs: write rowc, leave E and Hc
  const __nv_bfloat16* H;  // rows ldH apart
  int64_t ldH;
  __nv_bfloat16* Hc;    // gathered rows (ldh apart), scaled here
  int64_t ldh;
  int d, V;
  float* factor;        // per compact row, for dH
  float4* rowc;         // (a, b, ent, lse log2 e)
  float* clogp;
  const float* g_logp;  // given gradients (original rows), or nullptr: the policy's
  const float* g_ent;
  const float* ent;     // with g_ent: the forward's entropies (original rows)
  const float* g_dev;   // times *g_dev (nullptr: g_host)
  float g_host;
};

// Split-V merge (one warp per compact row; the rows left out follow and get
// zeros): partials of 128 columns (shift, sum e, sum e (x - shift), .) -> lse, logp, ent; with
// POLICY also the row's loss and gradient; with k.E the gradient's row factors.
//   logp = -log(1 + q), q = (sum of the others) / e_id: no large numbers are
// subtracted, so a log-probability near 0 keeps its relative accuracy.  Sums run
// in a fixed order.
template <int POLICY>
__global__ void __launch_bounds__(256)
    logp_rows_kernel(const float4* part, int parts_n,
                     const ChunkPlan* plan, int64_t c0, int in_chunk, int64_t N,
                     const int* perm, const int* cid,
                     const RowIn* rowin, int entropy, PolicyRows pol,
                     const Scalars* sc, RowOut o, RowBack k) {
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (i >= in_chunk) return;
  const int row = row_of(perm, c0 + i, N);
  if (i >= rows_of(plan, in_chunk)) {
    if (lane == 0) {
      if (o.logp != nullptr) o.logp[row] = 0.f;
      if (o.ent != nullptr) o.ent[row] = 0.f;
      if (o.lse != nullptr) o.lse[row] = 0.f;
      if (o.row_loss != nullptr) o.row_loss[row] = 0.f;
      if (o.g_logp != nullptr) o.g_logp[row] = 0.f;
      if (o.g_ent != nullptr) o.g_ent[row] = 0.f;
    }
    return;
  }
  const float4* pr = part + static_cast<int64_t>(i) * parts_n;
  const RowIn in = rowin[i];
  // everything that a row needs is asked for at once, before the sums
  PolicyIn pin{};
  float norm = 1.f, g = 0.f, h = 0.f, given_ent = 0.f;
  if (POLICY) {
    pin = policy_in(pol, row);
    norm = sc->norm > 0.f ? 1.f / sc->norm : 0.f;
  } else if (k.g_logp != nullptr) {
    g = k.g_logp[row];
    if (k.g_ent != nullptr) {
      h = k.g_ent[row];
      given_ent = k.ent[row];
    }
  }
  const bool scaled = k.E != nullptr && !k.dense;  // the row of H that dW contracts
  const int id = scaled ? min(max(cid[i], 0), k.V - 1) : 0;
  const float g_loss = k.g_dev != nullptr ? *k.g_dev : k.g_host;
  const uint4* hr = reinterpret_cast<const uint4*>(k.H + row * k.ldH);
  uint4 h4[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    h4[j] = scaled && lane + 32 * j < k.d / 8 ? hr[lane + 32 * j] : make_uint4(0, 0, 0, 0);
  // One pass over the partials as if none had moved from r, which hardly any has.
  float M = in.ref, Zo = 0.f, U = 0.f;
  bool moved = false;  // a part was done around its own maximum
#pragma unroll 8
  for (int t = lane; t < parts_n; t += 32) {
    const float4 v = pr[t];
    M = fmaxf(M, v.x);
    moved |= v.x != in.ref;
    Zo += v.y;
    U += v.z;
  }
  moved = __any_sync(0xffffffffu, moved);
  if (moved) {
    M = warp_max(M);
    Zo = U = 0.f;
    for (int t = lane; t < parts_n; t += 32) {
      const float4 v = pr[t];
      const float w = ex2_approx(v.x - M);
      Zo += w * v.y;
      if (w > 0.f) U += w * fmaf(v.x - M, v.y, v.z);  // sum e (x - M)
    }
  }
  Zo = warp_sum(Zo);
  U = warp_sum(U);
  const float zid = ex2_approx(in.ref - M + in.ref_lo);  // the token's own e
  const float Z = Zo + zid, q = Zo / zid;
  const float ref = in.ref + in.ref_lo;
  // past 2^90 the token's share is 0 in fp32 beside the others'
  const float logp = q < 0x1p90f ? -log1pf(q) : (in.ref - M + in.ref_lo - log2f(Z)) * kLn2;
  const float lse = fmaf(ref, kLn2, -logp);
  float ent = 0.f;
  if (entropy) {  // log Z - (sum e (x - M)) / Z around M
    const float lz = q < 0x1p90f ? (in.ref - M + in.ref_lo) * kLn2 + log1pf(q) : log2f(Z) * kLn2;
    if (zid > 0.f) U += zid * (in.ref - M + in.ref_lo);
    ent = lz - U / Z * kLn2;
  }
  if (POLICY) {
    const float l = policy_row(pol, pin, logp, ent, &g, &h);
    g *= norm;
    h *= norm;
    if (lane == 0) {
      if (o.row_loss != nullptr) o.row_loss[row] = l;
      if (o.g_logp != nullptr) o.g_logp[row] = g;
      if (o.g_ent != nullptr) o.g_ent[row] = h;
    }
  } else if (k.g_ent != nullptr) {
    ent = given_ent;
  }
  if (lane == 0) {
    if (o.logp != nullptr) o.logp[row] = logp;
    if (o.ent != nullptr) o.ent[row] = ent;
    if (o.lse != nullptr) o.lse[row] = lse;
  }
  if (k.E == nullptr) return;
  const float s = g_loss * in.invT;
  const float a = g * s;
  if (k.dense) {
    if (lane == 0) {
      k.rowc[i] = make_float4(a, h * s, ent, lse * kLog2e);
      k.clogp[i] = logp;
      k.factor[i] = 1.f;
    }
    return;
  }
  __nv_bfloat16* e = k.E + static_cast<int64_t>(i) * k.ld;
  if (moved) {  // bring every part to the shift M
    for (int t = 0; t < parts_n; ++t) {
      const float w = ex2_approx(pr[t].x - M);
      if (w == 1.f) continue;
      const int v1 = min((t + 1) * kPartVecs, (k.V + 7) >> 3);
      for (int v = t * kPartVecs + lane; v < v1; v += 32) {
        float f[8];
        load8<__nv_bfloat16>(e + v * 8, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = v * 8 + j < k.V ? f[j] * w : 0.f;
        store8<__nv_bfloat16>(e + v * 8, f);
      }
    }
    __syncwarp();
  }
  // The own token's entry is the largest part of most rows, and its rounding would
  // be the one with most effect; so the factor takes it back.
  const __nv_bfloat16 own = __float2bfloat16_rn(-Zo);
  const float back = -__bfloat162float(own);
  const float factor = -a / Z * (back > 0.f ? Zo / back : 1.f);
  if (lane == 0) {
    e[id] = own;
    k.factor[i] = factor;
  }
  __nv_bfloat16* hc = k.Hc + static_cast<int64_t>(i) * k.ldh;
  auto scale = [&](uint4 u, int v) {
    float f[8];
    load8<__nv_bfloat16>(reinterpret_cast<const __nv_bfloat16*>(&u), f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= factor;
    store8<__nv_bfloat16>(hc + v * 8, f);
  };
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (lane + 32 * j < k.d / 8) scale(h4[j], lane + 32 * j);
  for (int v0 = lane + 128; v0 < k.d / 8; v0 += 128) {  // four loads, then four stores
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h4[j] = v0 + 32 * j < k.d / 8 ? hr[v0 + 32 * j] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v0 + 32 * j < k.d / 8) scale(h4[j], v0 + 32 * j);
  }
}

// Backward of given row gradients where the logits are recomputed: compact (a, b,
// ent, lse log2 e), one thread a row.
__global__ void logp_coef_kernel(const ChunkPlan* plan, int64_t c0, int in_chunk, int64_t N,
                                 const int* perm, const RowIn* rowin,
                                 const float* lse, const float* ent,
                                 const float* g_logp, const float* g_ent,
                                 const float* g_loss, float4* rowc,
                                 float* factor) {
  grid_dep_wait();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= rows_of(plan, in_chunk)) return;
  const int row = row_of(perm, c0 + i, N);
  const float s = (g_loss != nullptr ? *g_loss : 1.f) * rowin[i].invT;
  rowc[i] = make_float4(s * g_logp[row], g_ent != nullptr ? s * g_ent[row] : 0.f,
                        ent != nullptr ? ent[row] : 0.f, lse[row] * kLog2e);
  factor[i] = 1.f;
}

// The own tokens' entries of a recomputed chunk, one warp per compact row, from the sums
// of the others' p (one per 128 columns, joined in a fixed order):
//   dS_id = a (1 - p) - p b (ln p + ent),  1 - p = sum_{j != id} p_j,
// where p near 1 comes from that sum too, and p elsewhere from the gathered logit.  For
// log-probabilities of -1e-5 and nearer to 0, a - a p was wrong by all of its value.
// 8192 rows, vocabulary 128256: 17 us beside the 6.8 ms of the chunk's logits (54 rows: 1.5
// of 39.5 us of the call).
__global__ void __launch_bounds__(256)
    logp_own_kernel(__nv_bfloat16* E, int64_t ld, int V, const float* part, int parts_n,
                    const ChunkPlan* plan, int in_chunk, const int* cid, const RowIn* rowin,
                    const float4* rowc) {
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (i >= rows_of(plan, in_chunk)) return;
  const float* pr = part + static_cast<int64_t>(i) * parts_n;
  float q = 0.f;
#pragma unroll 8
  for (int t = lane; t < parts_n; t += 32) q += pr[t];
  q = warp_sum(q);
  if (lane != 0) return;
  const float4 rc = rowc[i];
  const RowIn in = rowin[i];
  const float l2 = in.ref - rc.w + in.ref_lo;
  const float p = q < 0.5f ? 1.f - q : ex2_approx(l2);
  const float lnp = q < 0.5f ? log1pf(-q) : l2 * kLn2;
  const int id = min(max(cid[i], 0), V - 1);
  E[static_cast<int64_t>(i) * ld + id] =
      __float2bfloat16_rn(rc.x * q - p * rc.y * (lnp + rc.z));
}

// dS in place over the stored exponentials where the gradient has an entropy
// term, one CTA per compact row (zeros up to the padded end):
//   p_j = e_j 2^(shift - lse log2 e),  dS_j = -p_j (a + b (ln p_j + ent)),
// and at the token's own entry a (1 - p) = -a expm1(logp) takes the place of -p a.
__global__ void __launch_bounds__(512) logp_dlogits_kernel(
    __nv_bfloat16* E, int64_t ld, int V, const float4* part, int parts_n,
    const ChunkPlan* plan, const int* cid,
    const float* clogp, const float4* rowc) {
  grid_dep_wait();
  const int i = blockIdx.x;
  if (i >= rows_of(plan, static_cast<int>(gridDim.x))) return;  // those behind are 0 already
  __nv_bfloat16* e = E + static_cast<int64_t>(i) * ld;
  const int nvec = (V + 7) >> 3;
  const float4 rc = rowc[i];
  const float4* pr = part + static_cast<int64_t>(i) * parts_n;
  for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
    float f[8];
    load8<__nv_bfloat16>(e + v * 8, f);
    const float off = pr[v / kPartVecs].x - rc.w;
    const float scale = ex2_approx(off);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float p = scale * f[k];
      const float lnp = (__log2f(f[k]) + off) * kLn2;
      // p ln p = 0 where p is 0; a NaN p stays NaN
      f[k] = v * 8 + k < V && p != 0.f ? -p * fmaf(rc.y, lnp + rc.z, rc.x) : 0.f;
    }
    store8<__nv_bfloat16>(e + v * 8, f);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const float logp = clogp[i];
    const float ds = -rc.x * expm1f(logp) - expf(logp) * rc.y * (logp + rc.z);
    e[min(max(cid[i], 0), V - 1)] = __float2bfloat16_rn(ds);
  }
}

// dst = src rounded to bf16, n8 vectors of 8 values.
__global__ void __launch_bounds__(256)
    logp_round_kernel(const float* src, __nv_bfloat16* dst, int64_t n8) {
  grid_dep_wait();
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n8; i += gridDim.x * 256ll) {
    float f[8];
    load8<float>(src + i * 8, f);
    store8<__nv_bfloat16>(dst + i * 8, f);
  }
}

// loss = sum_n x[n] / divisor in fp64 in a fixed order (0 for divisor 0), by one CTA.
__device__ void mean_of(const float* x, int64_t n, float divisor, float* loss) {
  __shared__ double red[32];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) s += x[i];
  s = warp_sum_d(s);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = warp_sum_d(threadIdx.x < (blockDim.x >> 5) ? red[threadIdx.x] : 0.0);
    if (threadIdx.x == 0) *loss = divisor > 0.f ? static_cast<float>(s / divisor) : 0.f;
  }
}

// The mean alone; the divisor is *norm, or `given` where norm is nullptr.
__global__ void __launch_bounds__(1024) logp_mean_kernel(const float* x, int64_t n,
                                                         const float* norm, float given,
                                                         float* loss) {
  grid_dep_wait();
  mean_of(x, n, norm != nullptr ? *norm : given, loss);
}

// dH rows of the chunk: the K parts (fp32, split_rows apart) summed in order, times
// the row's factor, rounded once and written to the rows they came from; zeros to
// the rows left out.  One CTA per compact row, and one more for the mean of x [n]
// where loss is wanted (the last chunk: its rows' losses are there by now).
__global__ void logp_dh_kernel(const float* part, const ChunkPlan* plan,
                               int64_t c0, const int* perm,
                               const float* factor, int d,
                               __nv_bfloat16* dH, int in_chunk,
                               int64_t part_rows, const float* x, int64_t N, const Scalars* sc,
                               float* loss) {
  grid_dep_wait();
  const int i = blockIdx.x, rows = rows_of(plan, in_chunk);
  if (i == in_chunk) {
    mean_of(x, N, sc->norm, loss);
    return;
  }
  uint2* out = reinterpret_cast<uint2*>(dH + static_cast<int64_t>(row_of(perm, c0 + i, N)) * d);
  if (i >= rows) {
    for (int v = threadIdx.x; v < d / 4; v += blockDim.x) out[v] = make_uint2(0u, 0u);
    return;
  }
  const int64_t tile_rows = (rows + 2 * kBM - 1) / (2 * kBM) * (2 * kBM), slice = tile_rows * d;
  const int ks = min(plan->ksplit, static_cast<int>(part_rows / tile_rows));
  const float* src = part + static_cast<int64_t>(i) * d;
  const float k = factor[i];
  for (int v = threadIdx.x; v < d / 4; v += blockDim.x) {
    float4 a = reinterpret_cast<const float4*>(src)[v];
#pragma unroll 8
    for (int s = 1; s < ks; ++s) {
      const float4 b = reinterpret_cast<const float4*>(src + s * slice)[v];
      a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(k * a.x, k * a.y);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(k * a.z, k * a.w);
    out[v] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                        *reinterpret_cast<const uint32_t*>(&hi));
  }
}

// ------------------------------------------------------------------ preference loss

struct PrefPairs {
  const int* pairs;  // [P][2] (chosen, rejected) sequences, or nullptr: (i, P + i)
  int P, S;
  const float* ref;  // [S] reference scores, or nullptr (0)
  int loss;          // 0 sigmoid, 1 squared, 2 hinge
  float beta, smoothing, margin;
};

__device__ __forceinline__ bool pair_of(const PrefPairs& q, int i, int* a, int* b) {
  *a = q.pairs != nullptr ? q.pairs[2 * i] : i;
  *b = q.pairs != nullptr ? q.pairs[2 * i + 1] : q.P + i;
  return *a >= 0 && *a < q.S && *b >= 0 && *b < q.S;
}

// Loss of pair (a, b) and its slope with respect to x = (score - ref)[a] - (score - ref)[b].
__device__ __forceinline__ double pair_loss(const PrefPairs& q, const double* score, int a, int b,
                                            double* slope) {
  double x = score[a] - score[b];
  if (q.ref != nullptr) x -= static_cast<double>(q.ref[a]) - static_cast<double>(q.ref[b]);
  const double beta = q.beta;
  if (q.loss == 1) {
    const double y = x - 0.5 / beta;
    *slope = 2.0 * y;
    return y * y;
  }
  const double y = beta * x - q.margin;
  if (q.loss == 2) {
    *slope = y >= 1.0 ? 0.0 : y < 1.0 ? -beta : y;  // a NaN margin is no satisfied one
    return y >= 1.0 ? 0.0 : 1.0 - y;
  }
  // (1 - eps) softplus(-y) + eps softplus(y); d/dy = sigmoid(y) - (1 - eps)
  const double t = exp(-fabs(y)), soft = log1p(t), eps = q.smoothing;
  const double sig = y >= 0.0 ? 1.0 / (1.0 + t) : t / (1.0 + t);
  *slope = beta * (sig - (1.0 - eps));
  return (1.0 - eps) * (soft + fmax(-y, 0.0)) + eps * (soft + fmax(y, 0.0));
}

// The scores, kept in fp64: sums of thousands of log-probabilities are subtracted from
// each other and from the reference's.
struct PrefScores {
  double* score;    // [S]
  int* count;       // [S] rows that take part
  float* slope;     // [S] of the loss in each row's log-probability
  float* seq_logp;  // [S], or nullptr
  int average;
  float divisor;
};

// Share of one thread of a group of `size` in sequence s's sum and count.  Nothing is
// read through offsets that logp_compact found bad (n_valid is then 0).
__device__ __forceinline__ void score_share(const RowSelect& sel, const float* logp,
                                            const Scalars* sc, int s, int rank, int size,
                                            double* x, int* n) {
  *x = 0.0;
  *n = 0;
  if (sc->n_valid <= 0) return;
  for (int64_t r = sel.cu[s] + rank; r < sel.cu[s + 1]; r += size) {
    bool bad = false;
    if (row_token(sel, r, &bad) >= 0) {
      *x += logp[r];
      ++*n;
    }
  }
  *x = warp_sum_d(*x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) *n += __shfl_xor_sync(0xffffffffu, *n, o);
}

__device__ __forceinline__ void keep_score(const PrefScores& k, int s, double x, int n) {
  if (k.average && n > 0) x /= n;
  k.score[s] = x;
  k.count[s] = n;
  if (k.seq_logp != nullptr) k.seq_logp[s] = static_cast<float>(x);
}

// Pair i's loss (one thread).
__device__ __forceinline__ void one_pair(const PrefPairs& q, const PrefScores& k, int i,
                                         float* each, int* status) {
  int a, b;
  double d;
  const bool ok = pair_of(q, i, &a, &b);
  if (!ok) atomicCAS(status, 0, kStatusIndex);
  each[i] = ok ? static_cast<float>(pair_loss(q, k.score, a, b, &d)) : 0.f;
}

// Slope of the mean loss in each of sequence s's rows, summed over the pairs that hold
// it in a fixed order: lanes over the pairs, then the lanes (one warp).
__device__ __forceinline__ void one_slope(const PrefPairs& q, const PrefScores& k, int s) {
  const int lane = threadIdx.x & 31;
  int a, b;
  double d, sum = 0.0;
  if (q.pairs == nullptr) {  // sequence s is in pair s mod P alone (2 P = S)
    if (lane == 0) {
      pair_of(q, s < q.P ? s : s - q.P, &a, &b);
      pair_loss(q, k.score, a, b, &d);
      sum = s < q.P ? d : -d;
    }
  } else {
    for (int i = lane; i < q.P; i += 32) {
      if (!pair_of(q, i, &a, &b) || a == b || (a != s && b != s)) continue;
      pair_loss(q, k.score, a, b, &d);
      sum += a == s ? d : -d;
    }
    sum = warp_sum_d(sum);
  }
  if (lane == 0) {
    const double w = k.divisor > 0.f ? 1.0 / k.divisor : 0.0;
    const int n = k.count[s];
    k.slope[s] = static_cast<float>(sum * w / (k.average && n > 0 ? n : 1));
  }
}

// g_logp of row r: the slope of its sequence, 0 where the row takes no part.
__device__ __forceinline__ float row_slope(const RowSelect& sel, const Scalars* sc,
                                           const float* slope, int64_t r) {
  bool bad = false;
  if (sc->n_valid <= 0 || r < sel.cu[0] || r >= sel.cu[sel.S] || row_token(sel, r, &bad) < 0)
    return 0.f;
  int lo = 0, hi = sel.S;  // the sequence with cu[lo] <= r < cu[lo + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sel.cu[mid] <= r) lo = mid;
    else hi = mid;
  }
  return slope[lo];
}

// One CTA per packed sequence.
__global__ void __launch_bounds__(256) pref_sum_kernel(RowSelect sel, const float* logp,
                                                       const Scalars* sc, PrefScores k) {
  grid_dep_wait();
  __shared__ double red[8];
  __shared__ int redn[8];
  double x;
  int n;
  score_share(sel, logp, sc, blockIdx.x, threadIdx.x, 256, &x, &n);
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5] = x;
    redn[threadIdx.x >> 5] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) {
      x += red[w];
      n += redn[w];
    }
    keep_score(k, blockIdx.x, x, n);
  }
}

// Warps over max(S, P).
__global__ void __launch_bounds__(256)
    pref_pair_kernel(PrefPairs q, PrefScores k, float* each, int* status) {
  grid_dep_wait();
  const int w = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (w < q.P && (threadIdx.x & 31) == 0) one_pair(q, k, w, each, status);
  if (w < q.S) one_slope(q, k, w);
}

// Threads over the rows; the last CTA joins the pairs' losses.
__global__ void __launch_bounds__(256)
    pref_rows_kernel(RowSelect sel, const Scalars* sc, const float* slope,
                     float* g_logp, const float* each, int P,
                     float divisor, float* loss) {
  grid_dep_wait();
  if (blockIdx.x == gridDim.x - 1) {
    mean_of(each, P, divisor, loss);
    return;
  }
  const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (r < sel.N) g_logp[r] = row_slope(sel, sc, slope, r);
}

// The three above in one launch of one CTA, for few rows, sequences and pairs.
constexpr int kPrefSmall = 1024;
__global__ void __launch_bounds__(1024)
    pref_small_kernel(RowSelect sel, const float* logp, const Scalars* sc,
                      PrefPairs q, PrefScores k, float* each,
                      float* g_logp, int* status, float* loss) {
  grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int s = warp; s < q.S; s += 32) {
    double x;
    int n;
    score_share(sel, logp, sc, s, lane, 32, &x, &n);
    if (lane == 0) keep_score(k, s, x, n);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < q.P; i += 1024) one_pair(q, k, i, each, status);
  for (int s = warp; s < q.S; s += 32) one_slope(q, k, s);
  __syncthreads();
  if (threadIdx.x < sel.N) g_logp[threadIdx.x] = row_slope(sel, sc, k.slope, threadIdx.x);
  mean_of(each, q.P, k.divisor, loss);
}

}  // namespace ckl
