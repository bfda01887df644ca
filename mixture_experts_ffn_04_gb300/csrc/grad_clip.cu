// grad_clip.cu -- global gradient norm over many tensors, and clipping
// (include/moe_train.h).
//
//   norm = sqrt(sum g^2),  coef = min(1, max_norm / (norm + 1e-6)),  dst = g coef
//
// Bound by HBM: every gradient is read for the norm before the first can be
// scaled, then read again and written.  The list is cut into chunks of
// kChunkMin to kChunkMax elements that never span two tensors (a table in the
// workspace, so one launch covers any list).  The norm pass goes through the chunks
// upwards and the scaling pass downwards: what the norm pass read last is still in L2
// when the scaling pass starts.  604 M bf16 values: norm 175 us (6.9 TB/s), scaling 350
// (6.9); 200 M values in 1500 tensors at odd offsets 91 (6.2) and 171 (6.6).
//
// Each chunk's squares are added in fp32 (at most 64 in a row in each of
// four sums of a thread) and its sum goes to the workspace; the last block to finish adds the
// chunks in fp64 in chunk order (no atomics on the sums, so the norm is the same
// in every run).  A chunk whose fp32 sum overflowed, or is small enough for
// squares to have underflowed, is added again with its values scaled by a power
// of two; a chunk of zeros is among them (200 M bf16 zeros: norm 73 us, else 65).
#include <algorithm>
#include <cmath>

#include "../../include/moe_train.h"
#include "common.cuh"
#include "internal.h"
#include "train.h"

namespace moe {
namespace {

// Elements of a chunk: the power of two that gives about eight chunks an SM, so
// that a small list covers the GPU and a large one spends little on table
// look-ups and block sums.
constexpr int kChunkMin = 2048, kChunkMax = 32768;
constexpr int kThreads = 256;

struct Entry {
  const void* src;
  void* dst;
  int64_t numel;
  int32_t src_dtype, dst_dtype;
  int64_t first;   // first chunk of the tensor
};

constexpr int kBatch = 64;   // entries a table launch carries in its arguments
struct Batch {
  Entry e[kBatch];
};

__global__ void table_kernel(const __grid_constant__ Batch b, int n, Entry* table, int64_t at) {
  if ((int)threadIdx.x < n) table[at + threadIdx.x] = b.e[threadIdx.x];
}
// chunk -> tensor
__global__ void __launch_bounds__(256) chunks_kernel(const Entry* table, int64_t tensors, int32_t* owner,
                                                      int64_t chunk) {
  for (int64_t t = blockIdx.x; t < tensors; t += gridDim.x) {
    const Entry e = table[t];
    const int64_t n = (e.numel + chunk - 1) / chunk;
    for (int64_t c = threadIdx.x; c < n; c += blockDim.x) owner[e.first + c] = (int32_t)t;
  }
}

struct Span {
  const char* src;
  char* dst;
  int64_t n;
  int sd, dd;
};
__device__ __forceinline__ Span span_of(const Entry* table, const int32_t* owner, int64_t c,
                                           int64_t chunk) {
  const Entry e = table[owner[c]];
  const int64_t at = (c - e.first) * chunk;
  Span s;
  s.sd = e.src_dtype;
  s.dd = e.dst_dtype;
  s.src = reinterpret_cast<const char*>(e.src) + at * (s.sd == MOE_F32 ? 4 : 2);
  s.dst = e.dst ? reinterpret_cast<char*>(e.dst) + at * (s.dd == MOE_F32 ? 4 : 2) : nullptr;
  s.n = e.numel - at < chunk ? e.numel - at : chunk;
  return s;
}

// Elements before the first 16-byte boundary of p, at most n.
template <typename T>
__device__ __forceinline__ int head_of(const char* p, int64_t n) {
  const int h = (int)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
  return h < n ? h : (int)n;
}

template <typename T>
__device__ __forceinline__ float chunk_squares(const Span& s, float scale) {
  constexpr int NV = Vec16<T>::N;
  const T* p = reinterpret_cast<const T*>(s.src);
  const int head = head_of<T>(s.src, s.n);
  const int nv = (int)((s.n - head) / NV);
  const uint4* v = reinterpret_cast<const uint4*>(p + head);
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  int i = threadIdx.x;
  for (; i + 3 * kThreads < nv; i += 4 * kThreads) {
    uint4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = v[i + k * kThreads];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f[NV];
      unpack16(u[k], f, (const T*)nullptr);
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        f[e] *= scale;
        a[k] = fmaf(f[e], f[e], a[k]);
      }
    }
  }
  for (; i < nv; i += kThreads) {
    float f[NV];
    unpack16(v[i], f, (const T*)nullptr);
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      f[e] *= scale;
      a[0] = fmaf(f[e], f[e], a[0]);
    }
  }
  // the elements before the first boundary and after the last whole vector
  const int tail = (int)(s.n - head) - nv * NV;
  if ((int)threadIdx.x < head) {
    const float f = to_f(p[threadIdx.x]) * scale;
    a[1] = fmaf(f, f, a[1]);
  } else if ((int)threadIdx.x < head + tail) {
    const float f = to_f(p[head + nv * NV + (threadIdx.x - head)]) * scale;
    a[1] = fmaf(f, f, a[1]);
  }
  return (a[0] + a[1]) + (a[2] + a[3]);
}

template <typename V>
__device__ __forceinline__ V block_sum(V v, V* sh) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  V t = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) t += sh[w];
  return t;
}

struct Head {   // the workspace's first bytes
  uint32_t flags;
  int32_t ticket;
  float coef;
  int32_t next;   // norm pass: chunks handed out beyond the blocks' first ones
};

constexpr int kNormPerSm = 6;   // resident blocks: one wave
__global__ void __launch_bounds__(kThreads, kNormPerSm) grad_norm_kernel(const Entry* table, const int32_t* owner,
                                                             int64_t chunks, double* sums, Head* head,
                                                             double max_norm, float* norm, int64_t chunk) {
  __shared__ float sh[kThreads / 32];
  __shared__ double shd[kThreads / 32];
  __shared__ int s_last;
  pdl_trigger();
  pdl_wait();
  // chunks of a ragged list differ in size: the next one is claimed while this
  // one is added up
  __shared__ int64_t s_next;
  for (int64_t c = blockIdx.x; c < chunks;) {
    if (threadIdx.x == 0) s_next = (int64_t)gridDim.x + atomicAdd(&head->next, 1);
    const Span s = span_of(table, owner, c, chunk);
    auto squares = [&](float scale) {
      return (double)block_sum(s.sd == MOE_F32 ? chunk_squares<float>(s, scale) : chunk_squares<bf16>(s, scale), sh);
    };
    double sum = squares(1.0f);
    // Below 1e-28 squares under the smallest normal number may be missing (the
    // values are then under 1e-14, and 2^80 times them safe); above 1e38 the sum
    // overflowed (2^-96 times any fp32 value squares safely).  Infinities and
    // NaN stay what they are.
    if (!(sum >= 1e-28)) sum = squares(0x1p80f) * 0x1p-160;
    else if (!(sum <= 1e38)) sum = squares(0x1p-96f) * 0x1p192;
    if (threadIdx.x == 0) sums[c] = sum;
    c = s_next;        // written before block_sum's barriers
    __syncthreads();
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(&head->ticket, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double a = 0.0;
  for (int64_t i = threadIdx.x; i < chunks; i += kThreads) a += __ldcg(sums + i);
  a = block_sum(a, shd);
  if (threadIdx.x == 0) {
    const double n = sqrt(a);
    float coef = 1.0f;
    if (isfinite(n)) {
      const double q = max_norm / (n + 1e-6);
      coef = q < 1.0 ? (float)q : 1.0f;
    }
    *norm = (float)n;
    head->coef = coef;
    head->ticket = 0;
    head->next = 0;
  }
}

template <typename S, typename D>
__device__ __forceinline__ void scale_chunk(const Span& s, float coef) {
  const S* p = reinterpret_cast<const S*>(s.src);
  D* o = reinterpret_cast<D*>(s.dst);
  constexpr int NS = Vec16<S>::N, ND = Vec16<D>::N;
  constexpr int N = NS > ND ? NS : ND;   // elements a step: whole vectors on both sides
  const int head = head_of<S>(s.src, s.n);
  const bool fits = (reinterpret_cast<uintptr_t>(o + head) & 15) == 0;
  const int steps = fits ? (int)((s.n - head) / N) : 0;
  constexpr int U = 4;
  int i = threadIdx.x;
  for (; i + (U - 1) * kThreads < steps; i += U * kThreads) {
    uint4 u[U][N / NS];
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int h = 0; h < N / NS; ++h)
        u[k][h] = reinterpret_cast<const uint4*>(p + head + (int64_t)(i + k * kThreads) * N)[h];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      float f[N];
#pragma unroll
      for (int h = 0; h < N / NS; ++h) unpack16(u[k][h], f + h * NS, (const S*)nullptr);
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] *= coef;
#pragma unroll
      for (int h = 0; h < N / ND; ++h)
        __stcs(reinterpret_cast<uint4*>(o + head + (int64_t)(i + k * kThreads) * N) + h,
               pack16(f + h * ND, (const D*)nullptr));
    }
  }
  for (; i < steps; i += kThreads) {
    float f[N];
#pragma unroll
    for (int h = 0; h < N / NS; ++h)
      unpack16(reinterpret_cast<const uint4*>(p + head + (int64_t)i * N)[h], f + h * NS, (const S*)nullptr);
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] *= coef;
#pragma unroll
    for (int h = 0; h < N / ND; ++h)
      __stcs(reinterpret_cast<uint4*>(o + head + (int64_t)i * N) + h, pack16(f + h * ND, (const D*)nullptr));
  }
  // before the first boundary, after the last whole step (all, where source
  // and destination never meet on one)
  for (int64_t j = threadIdx.x; j < head; j += kThreads) o[j] = from_f<D>(to_f(p[j]) * coef);
  for (int64_t j = head + (int64_t)steps * N + threadIdx.x; j < s.n; j += kThreads)
    o[j] = from_f<D>(to_f(p[j]) * coef);
}

__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const Entry* table, const int32_t* owner,
                                                              int64_t chunks, const Head* head,
                                                              int64_t chunk) {
  pdl_trigger();
  pdl_wait();
  const float coef = head->coef;
  for (int64_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const Span s = span_of(table, owner, chunks - 1 - i, chunk);
    if (s.dst == nullptr || (coef == 1.0f && s.dst == s.src)) continue;
    if (s.sd == MOE_F32) {
      if (s.dd == MOE_F32) scale_chunk<float, float>(s, coef);
      else scale_chunk<float, bf16>(s, coef);
    } else {
      if (s.dd == MOE_F32) scale_chunk<bf16, float>(s, coef);
      else scale_chunk<bf16, bf16>(s, coef);
    }
  }
}

struct ClipLayout {
  size_t head, table, owner, sums, total;
};
ClipLayout layout_clip(int64_t tensors, int64_t chunks) {
  ClipLayout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~(size_t)255;
    return at;
  };
  L.head = take(256);
  L.table = take((size_t)tensors * sizeof(Entry));
  L.owner = take((size_t)chunks * 4);
  L.sums = take((size_t)chunks * 8);
  L.total = off;
  return L;
}

moe_status check_list(const moe_grad_tensor* t, int64_t n, int64_t* chunks, int* chunk, const char** why) {
  if (n < 0 || n > 0x7fffffff || (n > 0 && !t)) {
    *why = "tensors must be an array of n >= 0 entries";
    return MOE_ERR_INVALID_ARG;
  }
  int64_t c = 0, all = 0;
  for (int64_t i = 0; i < n; ++i) {
    for (int32_t d : {t[i].src_dtype, t[i].dst_dtype})
      if (d != MOE_F32 && d != MOE_BF16) {
        *why = "dtypes must be MOE_F32 or MOE_BF16";
        return MOE_ERR_UNSUPPORTED;
      }
    if (t[i].numel < 0 || t[i].numel > (1ll << 40) || (t[i].numel > 0 && !t[i].src)) {
      *why = "every tensor needs a source and 0 <= numel <= 2^40";
      return MOE_ERR_INVALID_ARG;
    }
    const size_t se = t[i].src_dtype == MOE_F32 ? 4 : 2, de = t[i].dst_dtype == MOE_F32 ? 4 : 2;
    if ((uintptr_t)t[i].src % se || (uintptr_t)t[i].dst % de) {
      *why = "sources and destinations must be aligned to their elements";
      return MOE_ERR_INVALID_ARG;
    }
    if (t[i].dst == t[i].src && t[i].numel > 0 && t[i].dst_dtype != t[i].src_dtype) {
      *why = "in-place clipping keeps the type";
      return MOE_ERR_INVALID_ARG;
    }
    all += t[i].numel;
  }
  *chunk = kChunkMin;
  while (*chunk < kChunkMax && all / *chunk > 8 * 152) *chunk *= 2;
  for (int64_t i = 0; i < n; ++i) c += (t[i].numel + *chunk - 1) / *chunk;
  if (c > 0x7fffffff) {
    *why = "the list is too long";
    return MOE_ERR_UNSUPPORTED;
  }
  *chunks = c;
  return MOE_OK;
}

unsigned clip_grid(int64_t chunks, int per_sm) {
  const int64_t cap = (int64_t)tc_sm_count() * per_sm;
  return (unsigned)std::max<int64_t>(1, std::min(chunks, cap));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_grad_clip_workspace_bytes(const moe_grad_tensor* tensors, int64_t n) {
  int64_t chunks;
  int chunk;
  const char* why;
  if (check_list(tensors, n, &chunks, &chunk, &why) != MOE_OK) return 0;
  return layout_clip(n, chunks).total;
}

extern "C" moe_status moe_grad_clip_plan(const moe_grad_tensor* tensors, int64_t n, moe_grad_plan* plan,
                                         void* ws, size_t ws_bytes, void* stream) {
  reset_launch_count();
  int64_t chunks = 0;
  int chunk = 0;
  const char* why = "";
  moe_status e = check_list(tensors, n, &chunks, &chunk, &why);
  if (e != MOE_OK) return fail(e, why);
  if (!plan) return fail(MOE_ERR_INVALID_ARG, "plan must be non-NULL");
  const ClipLayout L = layout_clip(n, chunks);
  e = check_ws(ws, ws_bytes, L.total);
  if (e != MOE_OK) return e;
  char* b = static_cast<char*>(ws);
  cudaStream_t st = (cudaStream_t)stream;
  Entry* table = reinterpret_cast<Entry*>(b + L.table);
  CHECK_CUDA(cudaMemsetAsync(b + L.head, 0, sizeof(Head), st));
  int64_t first = 0;
  for (int64_t at = 0; at < n; at += kBatch) {
    Batch batch = {};
    const int m = (int)std::min<int64_t>(kBatch, n - at);
    for (int i = 0; i < m; ++i) {
      const moe_grad_tensor& t = tensors[at + i];
      batch.e[i] = {t.src, t.dst, t.numel, t.src_dtype, t.dst_dtype, first};
      first += (t.numel + chunk - 1) / chunk;
    }
    table_kernel<<<1, kBatch, 0, st>>>(batch, m, table, at);
    count_launch();
    CHECK_CUDA(cudaGetLastError());
  }
  if (chunks > 0) {
    chunks_kernel<<<clip_grid(n, 8), 256, 0, st>>>(table, n, reinterpret_cast<int32_t*>(b + L.owner),
                                                   chunk);
    count_launch();
    CHECK_CUDA(cudaGetLastError());
  }
  *plan = {n, chunks, chunk, 0};
  return MOE_OK;
}

extern "C" moe_status moe_grad_clip(const moe_grad_plan* plan, double max_norm, float* norm, void* ws,
                                    size_t ws_bytes, void* stream) {
  reset_launch_count();
  if (!plan || plan->chunk_elems < kChunkMin || plan->chunk_elems > kChunkMax || plan->tensors < 0 || plan->chunks < 0)
    return fail(MOE_ERR_INVALID_ARG, "plan was not made by moe_grad_clip_plan");
  if (!norm) return fail(MOE_ERR_INVALID_ARG, "norm must be non-NULL");
  if (!(max_norm > 0.0)) return fail(MOE_ERR_INVALID_ARG, "max_norm must be positive");
  const ClipLayout L = layout_clip(plan->tensors, plan->chunks);
  moe_status e = check_ws(ws, ws_bytes, L.total);
  if (e != MOE_OK) return e;
  char* b = static_cast<char*>(ws);
  cudaStream_t st = (cudaStream_t)stream;
  const Entry* table = reinterpret_cast<const Entry*>(b + L.table);
  const int32_t* owner = reinterpret_cast<const int32_t*>(b + L.owner);
  Head* head = reinterpret_cast<Head*>(b + L.head);
  CHECK_CUDA(launch_after(grad_norm_kernel, clip_grid(plan->chunks, kNormPerSm), kThreads, 0, st, 1, table, owner,
                          plan->chunks, reinterpret_cast<double*>(b + L.sums), head, max_norm, norm,
                          (int64_t)plan->chunk_elems));
  if (plan->chunks > 0 && std::isfinite(max_norm))
    CHECK_CUDA(launch_after(grad_scale_kernel, clip_grid(plan->chunks, 16), kThreads, 0, st, 1, table, owner,
                            plan->chunks, (const Head*)head, (int64_t)plan->chunk_elems));
  return MOE_OK;
}
