// kl_clip.cu -- the global gradient norm over many tensors, and clipping.
//
//   total = sum_i sum g_i^2 (or the largest |g|),  norm = sqrt(total),
//   dst_i = src_i * min(1, max_norm / (norm + 1e-6)), rounded once to dst's type.
//
// Bound by HBM: the norm reads every gradient once, and the scaling, which needs
// the norm first, reads and writes them again, so that (beyond the L2's 126 MB)
// 2 reads + 1 write is the least a clipped call moves; a call that stays under
// max_norm in place moves one read.  One launch covers up to 896 tensors of any
// sizes and types: their table travels in the kernel's arguments (no copy to the
// device, nothing to keep alive), and a persistent grid walks it in pieces of
// 8192 values.  Every piece goes to a fixed CTA and is summed in a fixed order:
// 64 values a thread in fp32, then fp64, so the norm is the same bits every time.
// The scaling pass walks backwards: what the norm read last is still in L2.  1.35e9
// values (1.05 GB fp32, 2.2 GB bf16) clipped into bf16: 1.40 ms, the norm at 7.2 TB/s
// and the scaling at 6.3 TB/s, where a plain copy reaches 6.55.
#include <algorithm>
#include <memory>
#include <new>

#include <cuda_fp16.h>

#include "kl_host.cuh"
#include "kl_rowutil.cuh"

using namespace ckl;

namespace {

constexpr int kPiece = 8192;      // values
constexpr int kClipThreads = 256;
// CTAs per SM.  5.9 GB of mixed gradients scaled into bf16: 0.95 ms with 8, 1.02 with
// 6, 1.16 with 4 (one vector a thread and step; with two 1.25, with four 1.48 ms:
// longer bursts of reads and writes in turn).  2.7 GB summed: 0.445 ms with 6, 0.485
// with 8 CTAs.
constexpr int kSumCtas = 6, kScaleCtas = 8;
constexpr int kMaxParts = 148 * kSumCtas;
constexpr int kSmallTable = 104, kBigTable = 896;  // 4 KB and 32 KB of kernel arguments

template <int CAP>
struct Table {
  kl_grad e[CAP];
  int first[CAP + 1];  // first piece of each tensor; first[count] = pieces
  int count;
};
static_assert(sizeof(Table<kBigTable>) <= 32764 - 64, "kernel arguments");

template <typename T>
__device__ __forceinline__ float value(T x);
template <>
__device__ __forceinline__ float value<float>(float x) { return x; }
template <>
__device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <>
__device__ __forceinline__ float value<__half>(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T rounded(float x);
template <>
__device__ __forceinline__ float rounded<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half rounded<__half>(float x) { return __float2half_rn(x); }

// Values of the 16-byte vector u.
template <typename T>
__device__ __forceinline__ void unpack(uint4 u, float* f) {
  const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
  for (int i = 0; i < 16 / static_cast<int>(sizeof(T)); ++i) f[i] = value<T>(t[i]);
}

// Values before the next 16-byte boundary (pointers are aligned to their type).
template <typename T>
__device__ __forceinline__ int head_of(const T* p) {
  return static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
}

// Sum of squares of n values, this thread's share; or (INF) the largest |x| as bits
// (a NaN's bits are larger than every number's, so it stays).  At most 64 values are
// summed in fp32.  Where their sum overflows (a value over 1.8e19), or is so small that
// squares below the subnormals' range count (under 2^-120, and not all values 0), they
// are summed again in fp64.
template <typename T, bool INF>
__device__ __forceinline__ double piece_sum(const T* p, int n, uint32_t& m) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(T));
  const int tid = threadIdx.x, head = min(head_of(p), n), nv = (n - head) / kVec;
  constexpr uint32_t kNotSign = sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu;
  float s = 0.f;
  uint32_t any = 0;  // the values' bits
  auto take = [&](float x) {
    if (INF) m = max(m, __float_as_uint(fabsf(x)));
    else s = fmaf(x, x, s);
  };
  auto take_one = [&](float x) {
    any |= __float_as_uint(x);
    take(x);
  };
  if (tid < head) take_one(value<T>(p[tid]));
  const uint4* v = reinterpret_cast<const uint4*>(p + head);
#pragma unroll 1
  for (int i = tid; i < nv; i += 4 * kClipThreads) {
    uint4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      u[k] = i + k * kClipThreads < nv ? v[i + k * kClipThreads] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f[kVec];
      unpack<T>(u[k], f);
      if (!INF) any |= (u[k].x | u[k].y) | (u[k].z | u[k].w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) take(f[j]);
    }
  }
  const int tail = head + nv * kVec + tid;
  if (tail < n) take_one(value<T>(p[tail]));
  if (INF || (s >= 0x1p-120f && s < INFINITY) || (any & kNotSign) == 0) return s;
  double wide = 0.0;
  auto again = [&](float x) { wide = fma(static_cast<double>(x), static_cast<double>(x), wide); };
  if (tid < head) again(value<T>(p[tid]));
#pragma unroll 1
  for (int i = tid; i < nv; i += kClipThreads) {
    float f[kVec];
    unpack<T>(v[i], f);
#pragma unroll
    for (int j = 0; j < kVec; ++j) again(f[j]);
  }
  if (tail < n) again(value<T>(p[tail]));
  return wide;
}

template <int CAP, bool INF>
__global__ void __launch_bounds__(kClipThreads)
    grad_sum_kernel(const __grid_constant__ Table<CAP> t, double* part) {
  grid_dep_wait();
  __shared__ double red[kClipThreads / 32];
  double acc = 0.0;
  uint32_t m = 0;
  int e = 0;
  const int pieces = t.first[t.count];
  for (int c = blockIdx.x; c < pieces; c += gridDim.x) {
    while (c >= t.first[e + 1]) ++e;
    const int64_t base = static_cast<int64_t>(c - t.first[e]) * kPiece;
    const int64_t left = t.e[e].n - base;
    const int n = left < kPiece ? static_cast<int>(left) : kPiece;
    const int ty = t.e[e].src_dtype;
    if (ty == KL_DTYPE_F32)
      acc += piece_sum<float, INF>(static_cast<const float*>(t.e[e].src) + base, n, m);
    else if (ty == KL_DTYPE_BF16)
      acc += piece_sum<__nv_bfloat16, INF>(static_cast<const __nv_bfloat16*>(t.e[e].src) + base, n,
                                           m);
    else
      acc += piece_sum<__half, INF>(static_cast<const __half*>(t.e[e].src) + base, n, m);
  }
  if (INF) {
    acc = static_cast<double>(__uint_as_float(__reduce_max_sync(0xffffffffu, m)));
  } else {
    acc = warp_sum_d(acc);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kClipThreads / 32; ++w) {
      if (!INF) acc += red[w];
      else if (!(acc >= red[w])) acc = isnan(acc) ? acc : red[w];
    }
    part[blockIdx.x] = acc;
  }
}

// The parts joined in a fixed order (whole CTA; the result in every thread).
template <bool INF>
__device__ double join_parts(const double* part, int parts) {
  __shared__ double red[kClipThreads / 32], all;
  double a = 0.0;
  for (int i = threadIdx.x; i < parts; i += kClipThreads) {
    const double b = part[i];
    if (!INF) a += b;
    else if (!(a >= b)) a = isnan(a) ? a : b;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double b = __shfl_xor_sync(0xffffffffu, a, o);
    if (!INF) a += b;
    else if (!(a >= b)) a = isnan(a) ? a : b;
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kClipThreads / 32; ++w) {
      if (!INF) a += red[w];
      else if (!(a >= red[w])) a = isnan(a) ? a : red[w];
    }
    all = a;
  }
  __syncthreads();
  return all;
}

template <bool INF>
__global__ void __launch_bounds__(kClipThreads)
    grad_total_kernel(const double* part, int parts, double* total, float* norm) {
  grid_dep_wait();
  const double t = join_parts<INF>(part, parts);
  if (threadIdx.x == 0) {
    if (total != nullptr) *total = t;
    if (norm != nullptr) *norm = static_cast<float>(INF ? t : sqrt(t));
  }
}

// dst = k * src for n values; 16-byte accesses where both reach a boundary together.
template <typename T, typename U>
__device__ __forceinline__ void piece_scale(const T* src, U* dst, int n, float k, bool stream) {
  constexpr int kIn = static_cast<int>(sizeof(T)) / 2, kOut = static_cast<int>(sizeof(U)) / 2;
  const int tid = threadIdx.x, head = min(head_of(dst), n);
  if (reinterpret_cast<uintptr_t>(src + head) & 15) {
    for (int i = tid; i < n; i += kClipThreads) dst[i] = rounded<U>(k * value<T>(src[i]));
    return;
  }
  if (tid < head) dst[tid] = rounded<U>(k * value<T>(src[tid]));
  const int nv = (n - head) / 8;
  const uint4* in = reinterpret_cast<const uint4*>(src + head);
  uint4* out = reinterpret_cast<uint4*>(dst + head);
  for (int i = tid; i < nv; i += kClipThreads) {
    uint4 u[kIn], w[kOut];
#pragma unroll
    for (int j = 0; j < kIn; ++j) u[j] = in[i * kIn + j];
    float f[8];
#pragma unroll
    for (int j = 0; j < kIn; ++j) unpack<T>(u[j], f + j * (8 / kIn));
    U* x = reinterpret_cast<U*>(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = rounded<U>(k * f[j]);
#pragma unroll
    for (int j = 0; j < kOut; ++j) {
      if (stream) __stcs(out + i * kOut + j, w[j]);
      else out[i * kOut + j] = w[j];
    }
  }
  const int tail = head + nv * 8 + tid;
  if (tail < n) dst[tail] = rounded<U>(k * value<T>(src[tail]));
}

template <typename T>
__device__ __forceinline__ void piece_scale_to(const kl_grad& g, int64_t base, int n, float k) {
  const T* src = static_cast<const T*>(g.src) + base;
  const bool stream = g.src != g.dst;  // written behind: leave L2 to what is still to be read
  if (g.dst_dtype == KL_DTYPE_F32)
    piece_scale(src, static_cast<float*>(g.dst) + base, n, k, stream);
  else if (g.dst_dtype == KL_DTYPE_BF16)
    piece_scale(src, static_cast<__nv_bfloat16*>(g.dst) + base, n, k, stream);
  else
    piece_scale(src, static_cast<__half*>(g.dst) + base, n, k, stream);
}

template <int CAP, bool INF>
__global__ void __launch_bounds__(kClipThreads)
    grad_scale_kernel(const __grid_constant__ Table<CAP> t, const double* part,
                      int parts, float max_norm, float* norm) {
  grid_dep_wait();
  const double total = join_parts<INF>(part, parts);
  const double nrm = INF ? total : sqrt(total);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(nrm);
  // a NaN norm gives NaN, an infinite one 0 (and NaN where a gradient is infinite)
  const double q = max_norm / (nrm + 1e-6);
  const float k = q > 1.0 ? 1.f : static_cast<float>(q);
  const int pieces = t.first[t.count];
  int e = t.count - 1;
  for (int c = pieces - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    while (c < t.first[e]) --e;
    const kl_grad& g = t.e[e];
    if (k == 1.f && g.src == g.dst) continue;  // nothing to change
    const int64_t base = static_cast<int64_t>(c - t.first[e]) * kPiece;
    const int64_t left = g.n - base;
    const int n = left < kPiece ? static_cast<int>(left) : kPiece;
    if (g.src_dtype == KL_DTYPE_F32) piece_scale_to<float>(g, base, n, k);
    else if (g.src_dtype == KL_DTYPE_BF16) piece_scale_to<__nv_bfloat16>(g, base, n, k);
    else piece_scale_to<__half>(g, base, n, k);
  }
}

// ------------------------------------------------------------------ host
int64_t dtype_bytes(int t) { return t == KL_DTYPE_F32 ? 4 : 2; }
bool known_dtype(int t) { return t == KL_DTYPE_F32 || t == KL_DTYPE_BF16 || t == KL_DTYPE_F16; }

constexpr int64_t kMaxValues = int64_t(1) << 40;

// At most 2^40 values in all (a list for the norm alone may name a tensor more than once),
// so that one table's pieces can be numbered in 32 bits and only its length splits a list.
int check_grads(const kl_grad* g, int64_t count, bool write) {
  if (count < 0 || count > (int64_t(1) << 20)) return KL_ERR_SHAPE;
  if (count > 0 && g == nullptr) return KL_ERR_NULL;
  int64_t left = kMaxValues;
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].n < 0 || g[i].n > left) return KL_ERR_SHAPE;
    left -= g[i].n;
    if (!known_dtype(g[i].src_dtype) || (write && !known_dtype(g[i].dst_dtype)))
      return KL_ERR_DTYPE;
    if (g[i].n == 0) continue;
    if (g[i].src == nullptr || (write && g[i].dst == nullptr)) return KL_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(g[i].src) % dtype_bytes(g[i].src_dtype) ||
        (write && reinterpret_cast<uintptr_t>(g[i].dst) % dtype_bytes(g[i].dst_dtype)))
      return KL_ERR_ALIGN;
  }
  return KL_OK;
}

// A destination may be its own source, and must share no byte with anything else.
// Returns KL_OK, KL_ERR_ARG, or KL_ERR_TOO_LARGE when there is no host memory for
// the list of a very long table.
int check_overlap(const kl_grad* g, int64_t count) {
  struct Span {
    uintptr_t a, b;
    bool write;
  };
  constexpr int64_t kOnStack = 2 * kSmallTable;
  Span few[kOnStack];
  std::unique_ptr<Span[]> many;
  Span* v = few;
  if (2 * count > kOnStack) {
    many.reset(new (std::nothrow) Span[static_cast<size_t>(count) * 2]);
    if (many == nullptr) return KL_ERR_TOO_LARGE;
    v = many.get();
  }
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].n == 0) continue;
    const uintptr_t s = reinterpret_cast<uintptr_t>(g[i].src);
    const uintptr_t d = reinterpret_cast<uintptr_t>(g[i].dst);
    v[n++] = {d, d + g[i].n * dtype_bytes(g[i].dst_dtype), true};
    if (s != d || g[i].src_dtype != g[i].dst_dtype)
      v[n++] = {s, s + g[i].n * dtype_bytes(g[i].src_dtype), false};
  }
  std::sort(v, v + n, [](const Span& x, const Span& y) { return x.a < y.a; });
  uintptr_t end_any = 0, end_write = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (v[i].a < end_write || (v[i].write && v[i].a < end_any)) return KL_ERR_ARG;
    end_any = std::max(end_any, v[i].b);
    if (v[i].write) end_write = std::max(end_write, v[i].b);
  }
  return KL_OK;
}

// Fills t with the tensors from `from` on that fit one table; returns the next one.
template <int CAP>
int64_t fill(Table<CAP>& t, const kl_grad* g, int64_t from, int64_t count) {
  int n = 0;
  int64_t pieces = 0, i = from;
  for (; i < count && n < CAP; ++i) {
    const int64_t k = cdiv(g[i].n, kPiece);
    if (k == 0) continue;
    t.e[n] = g[i];
    t.first[n++] = static_cast<int>(pieces);
    pieces += k;
  }
  t.first[n] = static_cast<int>(pieces);
  t.count = n;
  return i;
}

int64_t launches_of(int64_t count) { return cdiv(count > 0 ? count : 1, kSmallTable); }

template <int CAP, bool INF>
int launch_sum(const Table<CAP>& t, double* part, int grid, cudaStream_t st) {
  double bytes = 0;
  for (int i = 0; i < t.count; ++i)
    bytes += static_cast<double>(t.e[i].n) * dtype_bytes(t.e[i].src_dtype);
  LaunchScope ls("grad_sum", st, 0, bytes);
  return launch_dependent(grad_sum_kernel<CAP, INF>, grid, kClipThreads, st, t, part);
}

template <int CAP, bool INF>
int launch_scale(const Table<CAP>& t, const double* part, int parts, float max_norm, float* norm,
                 int grid, cudaStream_t st) {
  double bytes = 0;
  for (int i = 0; i < t.count; ++i)
    bytes += static_cast<double>(t.e[i].n) *
             (dtype_bytes(t.e[i].src_dtype) + dtype_bytes(t.e[i].dst_dtype));
  LaunchScope ls("grad_scale", st, 0, bytes);
  return launch_dependent(grad_scale_kernel<CAP, INF>, grid, kClipThreads, st, t, part, parts,
                          max_norm, norm);
}

template <int CAP, bool INF>
int sum_all(const kl_grad* g, int64_t count, double* part, int sms, cudaStream_t st, int* parts) {
  Table<CAP> t;
  *parts = 0;
  for (int64_t i = 0; i < count;) {
    i = fill(t, g, i, count);
    const int pieces = t.first[t.count];
    const int most = sms * kSumCtas < kMaxParts ? sms * kSumCtas : kMaxParts;
    if (pieces == 0) continue;
    const int grid = pieces < most ? pieces : most;
    KL_TRY((launch_sum<CAP, INF>(t, part + *parts, grid, st)));
    *parts += grid;
  }
  return KL_OK;
}

template <int CAP, bool INF>
int scale_all(const kl_grad* g, int64_t count, const double* part, int parts, float max_norm,
              float* norm, int sms, cudaStream_t st) {
  Table<CAP> t;
  bool any = false;
  for (int64_t i = 0; i < count;) {
    i = fill(t, g, i, count);
    const int pieces = t.first[t.count];
    if (pieces == 0) continue;
    const int grid = pieces < sms * kScaleCtas ? pieces : sms * kScaleCtas;
    KL_TRY((launch_scale<CAP, INF>(t, part, parts, max_norm, any ? nullptr : norm, grid, st)));
    any = true;
  }
  if (any || norm == nullptr) return KL_OK;
  LaunchScope ls("grad_total", st, 0, 0);  // no values at all
  return launch_dependent(grad_total_kernel<INF>, 1, kClipThreads, st, part, parts, nullptr, norm);
}

// The sums of all tensors into the workspace's parts.
int sums(const kl_grad* g, int64_t count, int inf, double* part, int sms, cudaStream_t st,
         int* parts) {
  if (count <= kSmallTable)
    return inf ? sum_all<kSmallTable, true>(g, count, part, sms, st, parts)
               : sum_all<kSmallTable, false>(g, count, part, sms, st, parts);
  return inf ? sum_all<kBigTable, true>(g, count, part, sms, st, parts)
             : sum_all<kBigTable, false>(g, count, part, sms, st, parts);
}

int scales(const kl_grad* g, int64_t count, int inf, const double* part, int parts, float max_norm,
           float* norm, int sms, cudaStream_t st) {
  if (count <= kSmallTable)
    return inf ? scale_all<kSmallTable, true>(g, count, part, parts, max_norm, norm, sms, st)
               : scale_all<kSmallTable, false>(g, count, part, parts, max_norm, norm, sms, st);
  return inf ? scale_all<kBigTable, true>(g, count, part, parts, max_norm, norm, sms, st)
             : scale_all<kBigTable, false>(g, count, part, parts, max_norm, norm, sms, st);
}

int begin(const kl_grad* g, int64_t count, int norm_type, bool write, void* ws, size_t ws_bytes,
          DevInfo* di) {
  KL_TRY(check_grads(g, count, write));
  if (norm_type != KL_NORM_2 && norm_type != KL_NORM_INF) return KL_ERR_ARG;
  if (write) KL_TRY(check_overlap(g, count));
  KL_TRY(current_device_info(di));
  if (ws == nullptr) return KL_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(ws) & 255) return KL_ERR_ALIGN;
  return ws_bytes < kl_grad_workspace_bytes(count) ? KL_ERR_WORKSPACE : KL_OK;
}

}  // namespace

extern "C" {

size_t kl_grad_workspace_bytes(int64_t count) {
  if (count < 0 || count > (int64_t(1) << 20)) return 0;
  return up256(static_cast<size_t>(launches_of(count)) * kMaxParts * sizeof(double));
}

int kl_grad_norm(const kl_grad* g, int64_t count, int norm_type, void* ws, size_t ws_bytes,
                 double* total, float* norm, void* stream) {
  DevInfo di;
  KL_TRY(begin(g, count, norm_type, false, ws, ws_bytes, &di));
  if (total == nullptr && norm == nullptr) return KL_ERR_NULL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(ws);
  const int inf = norm_type == KL_NORM_INF;
  int parts = 0;
  KL_TRY(sums(g, count, inf, part, di.sms, st, &parts));
  LaunchScope ls("grad_total", st, 0, 8.0 * parts);
  return launch_dependent(inf ? grad_total_kernel<true> : grad_total_kernel<false>, 1,
                          kClipThreads, st, part, parts, total, norm);
}

int kl_grad_clip(const kl_grad* g, int64_t count, int norm_type, float max_norm,
                 const double* total, void* ws, size_t ws_bytes, float* norm, void* stream) {
  DevInfo di;
  if (!(max_norm >= 0.f)) return KL_ERR_ARG;
  KL_TRY(begin(g, count, norm_type, true, ws, ws_bytes, &di));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(ws);
  const int inf = norm_type == KL_NORM_INF;
  int parts = 1;
  if (total == nullptr) KL_TRY(sums(g, count, inf, part, di.sms, st, &parts));
  return scales(g, count, inf, total != nullptr ? total : part, parts, max_norm, norm, di.sms, st);
}

}  // extern "C"
