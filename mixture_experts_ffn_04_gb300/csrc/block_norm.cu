// block_norm.cu -- the norms before and after a block with its gate and residual,
// forward and backward (include/moe_model.h).
//
//   u = y r1 (w_post + o),  s = residual_scale x + g u,  h = s r2 (w_pre + o)
//
// Bound by HBM: the forward reads two rows a token and writes two, the backward
// reads four and writes two (s is not read back: from x and y it costs a few
// FMAs, and it has not been rounded).  A group of threads holds a whole row in
// registers, eight columns and their multiples a thread, so that both norms of the
// forward, and both row sums of the backward, come from one read.  Sums in fp32.
//
// The sums over tokens (dw_post, dgate of a channel gate, dw_pre) stay in the
// registers of the thread that owns the columns, over the rows its group meets (at
// most kFlush of them in one sum), go to the workspace, and a second kernel adds
// the groups' sums in a fixed order.
#include <algorithm>
#include <cmath>

#include "../../include/moe_model.h"
#include "common.cuh"
#include "internal.h"
#include "train.h"

namespace moe {
namespace bn {

constexpr int kFlush = 128;        // rows that one fp32 sum of a column takes
constexpr int kMaxWarps = 32;

struct NShape {
  int64_t T;
  int H, dtype, esize, gate;
  float off, res, eps;
};

// 8 columns of a row, as they stand in memory
template <typename T>
struct Eight {
  uint4 v[8 / Vec16<T>::N];
};
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p) {
  Eight<T> r;
#pragma unroll
  for (int i = 0; i < 8 / Vec16<T>::N; ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ Eight<T> zero8() {
  Eight<T> r;
#pragma unroll
  for (int i = 0; i < 8 / Vec16<T>::N; ++i) r.v[i] = make_uint4(0, 0, 0, 0);
  return r;
}
template <typename T>
__device__ __forceinline__ void open8(const Eight<T>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 8 / Vec16<T>::N; ++i) unpack16(r.v[i], f + i * Vec16<T>::N, (const T*)nullptr);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* f) {
#pragma unroll
  for (int i = 0; i < 8 / Vec16<T>::N; ++i)
    reinterpret_cast<uint4*>(p)[i] = pack16(f + i * Vec16<T>::N, (const T*)nullptr);
}

// Threads of a row: G, with a power of two up to 32 or whole warps beyond, so that
// the lanes of a sum are G apart from the next row's.  NG rows a block.
struct Geometry {
  int G, NG, vpt;
};
Geometry geometry(int H, int wide) {
  const int vecs = H / 8;
  Geometry g;
  if (vecs <= 32) {
    g.vpt = 1;
    g.G = 4;
    while (g.G < vecs) g.G *= 2;
  } else {
    g.vpt = vecs <= wide ? 1 : (vecs <= 1024 ? 2 : 4);
    g.G = ((vecs + g.vpt - 1) / g.vpt + 31) / 32 * 32;
  }
  g.NG = std::max(1, 256 / g.G);
  return g;
}

// Sum over a row's threads, the same in all of them.  G > 32: red holds a value a
// warp, `slot` alternates so that one barrier a sum is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int G, float (*red)[N][kMaxWarps], int& slot) {
  const int span = G < 32 ? G : 32;
  for (int o = span >> 1; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (G <= 32) return;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[slot][i][warp] = v[i];
  __syncthreads();
  const int first = (threadIdx.x / G) * (G >> 5);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = 0.0f;
    for (int w = 0; w < (G >> 5); ++w) t += red[slot][i][first + w];
    v[i] = t;
  }
  slot ^= 1;
}

template <typename T, int VPT>
__global__ void __launch_bounds__(1024) norm_forward_kernel(int64_t rows, int H, int G, int NG, int kind, float off,
                                                            float res, float eps, const T* x, const T* __restrict__ y,
                                                            const T* __restrict__ w_post, const void* __restrict__ gate,
                                                            const T* __restrict__ w_pre, T* s, T* __restrict__ h,
                                                            float2* __restrict__ rstd) {
  __shared__ float red[2][1][kMaxWarps];
  pdl_trigger();
  pdl_wait();
  const int g = threadIdx.x / G, lane = threadIdx.x - g * G;
  int slot = 0;
  const float inv_h = 1.0f / (float)H;
  // weights stay in registers over the rows
  Eight<T> wp[VPT], wg[VPT], wq[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (lane + v * G) * 8;
    const bool live = c < H;
    wp[v] = live && w_post ? load8<T>(w_post + c) : zero8<T>();
    wg[v] = live && kind == MOE_GATE_CHANNEL ? load8<T>(static_cast<const T*>(gate) + c) : zero8<T>();
    wq[v] = live && w_pre ? load8<T>(w_pre + c) : zero8<T>();
  }
  for (int64_t base = (int64_t)blockIdx.x * NG; base < rows; base += (int64_t)gridDim.x * NG) {
    const int64_t t = base + g;
    const bool on = t < rows;
    Eight<T> ux[VPT], uy[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (lane + v * G) * 8;
      ux[v] = on && c < H ? load8<T>(x + t * H + c) : zero8<T>();
      uy[v] = on && c < H && y ? load8<T>(y + t * H + c) : zero8<T>();
    }
    float gt = 1.0f;
    if (kind == MOE_GATE_TOKEN && on) gt = static_cast<const float*>(gate)[t];
    float r1 = 1.0f;
    if (w_post) {
      float sum[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        float f[8];
        open8<T>(uy[v], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = fmaf(f[e], f[e], sum[0]);
      }
      row_sum<1>(sum, G, red, slot);
      r1 = 1.0f / sqrtf(sum[0] * inv_h + eps);
    }
    float f[VPT][8];
    float sum[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float fy[8], w[8];
      open8<T>(ux[v], f[v]);
      open8<T>(uy[v], fy);
      if (w_post) {
        open8<T>(wp[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) fy[e] = fy[e] * r1 * (w[e] + off);
      }
      if (kind == MOE_GATE_CHANNEL) {
        open8<T>(wg[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) fy[e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[v][e] = y ? fmaf(res, f[v][e], gt * fy[e]) : res * f[v][e];
        sum[0] = fmaf(f[v][e], f[v][e], sum[0]);
      }
    }
    float r2 = 0.0f;
    if (w_pre) {
      row_sum<1>(sum, G, red, slot);
      r2 = 1.0f / sqrtf(sum[0] * inv_h + eps);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (lane + v * G) * 8;
      if (!on || c >= H) continue;
      if (s) store8<T>(s + t * H + c, f[v]);
      if (w_pre) {
        float w[8];
        open8<T>(wq[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[v][e] = f[v][e] * r2 * (w[e] + off);
        store8<T>(h + t * H + c, f[v]);
      }
    }
    if (rstd && on && lane == 0) rstd[t] = make_float2(w_post ? r1 : 0.0f, r2);
  }
}

struct BwdArgs {
  int64_t rows;
  int H, G, NG, kind, flushes;
  float off, res;
  const void *ds, *dh, *x, *y, *w_post, *gate, *w_pre;
  const float2* rstd;
  void *dx, *dy;
  float* dgate;      // of a token gate
  float* part;       // [flushes][blocks][NG][3][H], or NULL
};

template <typename T, int VPT>
__global__ void __launch_bounds__(VPT == 4 ? 1024 : 512) norm_backward_kernel(const BwdArgs a) {
  __shared__ float red[2][1][kMaxWarps];
  __shared__ float red2[2][2][kMaxWarps];
  pdl_trigger();
  pdl_wait();
  const int G = a.G, H = a.H;
  const int g = threadIdx.x / G, lane = threadIdx.x - g * G;
  int slot = 0, slot2 = 0;
  const float inv_h = 1.0f / (float)H;
  const T* w_post = static_cast<const T*>(a.w_post);
  const T* w_pre = static_cast<const T*>(a.w_pre);
  const T* ds = static_cast<const T*>(a.ds);
  const T* dh = static_cast<const T*>(a.dh);
  const T* x = static_cast<const T*>(a.x);
  const T* y = static_cast<const T*>(a.y);
  T* dx = static_cast<T*>(a.dx);
  T* dy = static_cast<T*>(a.dy);
  Eight<T> wp[VPT], wg[VPT], wq[VPT];
  float s_post[VPT][8], s_gate[VPT][8], s_pre[VPT][8];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (lane + v * G) * 8;
    const bool live = c < H;
    wp[v] = live && w_post ? load8<T>(w_post + c) : zero8<T>();
    wg[v] = live && a.kind == MOE_GATE_CHANNEL ? load8<T>(static_cast<const T*>(a.gate) + c) : zero8<T>();
    wq[v] = live && w_pre ? load8<T>(w_pre + c) : zero8<T>();
#pragma unroll
    for (int e = 0; e < 8; ++e) s_post[v][e] = s_gate[v][e] = s_pre[v][e] = 0.0f;
  }
  int count = 0, flush = 0;
  auto put_sums = [&]() {
    float* p = a.part + (((int64_t)flush * gridDim.x + blockIdx.x) * a.NG + g) * 3 * H;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (lane + v * G) * 8;
      if (c < H) {
        store8<float>(p + c, s_post[v]);
        store8<float>(p + H + c, s_gate[v]);
        store8<float>(p + 2 * H + c, s_pre[v]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s_post[v][e] = s_gate[v][e] = s_pre[v][e] = 0.0f;
    }
    ++flush;
    count = 0;
  };
  for (int64_t base = (int64_t)blockIdx.x * a.NG; base < a.rows; base += (int64_t)gridDim.x * a.NG) {
    const int64_t t = base + g;
    const bool on = t < a.rows;
    Eight<T> ux[VPT], uy[VPT], us[VPT], uh[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (lane + v * G) * 8;
      const bool live = on && c < H;
      ux[v] = live && w_pre ? load8<T>(x + t * H + c) : zero8<T>();
      uy[v] = live && y ? load8<T>(y + t * H + c) : zero8<T>();
      us[v] = live && ds ? load8<T>(ds + t * H + c) : zero8<T>();
      uh[v] = live && w_pre ? load8<T>(dh + t * H + c) : zero8<T>();
    }
    float2 r = make_float2(0.0f, 0.0f);
    if (on) r = a.rstd[t];
    if (!w_post) r.x = 1.0f;
    float gt = 1.0f;
    if (a.kind == MOE_GATE_TOKEN && on) gt = static_cast<const float*>(a.gate)[t];
    // D: first the row sum of dh w_pre sn
    float D[VPT][8];
    float c2[1] = {0.0f};
    if (w_pre) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        float fx[8], fy[8], fh[8], w[8];
        open8<T>(ux[v], fx);
        open8<T>(uy[v], fy);
        open8<T>(uh[v], fh);
        if (w_post) {
          open8<T>(wp[v], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) fy[e] = fy[e] * r.x * (w[e] + a.off);
        }
        if (a.kind == MOE_GATE_CHANNEL) {
          open8<T>(wg[v], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) fy[e] *= w[e];
        }
        open8<T>(wq[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float sn = (y ? fmaf(a.res, fx[e], gt * fy[e]) : a.res * fx[e]) * r.y;
          s_pre[v][e] = fmaf(fh[e], sn, s_pre[v][e]);
          const float b = fh[e] * (w[e] + a.off);
          c2[0] = fmaf(b, sn, c2[0]);
          D[v][e] = sn;   // until the sum is there
        }
      }
      row_sum<1>(c2, G, red, slot);
      c2[0] *= inv_h;
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float fs[8], fh[8], w[8];
      open8<T>(us[v], fs);
      if (w_pre) {
        open8<T>(uh[v], fh);
        open8<T>(wq[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          D[v][e] = fmaf(r.y, fmaf(-D[v][e], c2[0], fh[e] * (w[e] + a.off)), fs[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) D[v][e] = fs[e];
      }
      const int c = (lane + v * G) * 8;
      if (dx && on && c < H) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = a.res * D[v][e];
        store8<T>(dx + t * H + c, o);
      }
    }
    if (!y) { if (a.part && ++count == kFlush) put_sums(); continue; }
    // the block's side: row sums of b yn and of D u
    float c1[2] = {0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float fy[8], w[8], gg[8];
      open8<T>(uy[v], fy);
      open8<T>(wp[v], w);
      open8<T>(wg[v], gg);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float yn = fy[e] * r.x;
        const float wv = w_post ? w[e] + a.off : 1.0f;
        const float gv = a.kind == MOE_GATE_CHANNEL ? gg[e] : gt;
        const float du = D[v][e] * gv, dyn = D[v][e] * yn;
        s_post[v][e] = fmaf(du, yn, s_post[v][e]);
        s_gate[v][e] = fmaf(dyn, wv, s_gate[v][e]);
        c1[0] = fmaf(du * wv, yn, c1[0]);
        c1[1] = fmaf(dyn, wv, c1[1]);
        D[v][e] = du * wv;
      }
    }
    row_sum<2>(c1, G, red2, slot2);
    if (a.dgate && on && lane == 0) a.dgate[t] = c1[1];
    c1[0] *= inv_h;
    if (dy) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = (lane + v * G) * 8;
        if (!on || c >= H) continue;
        if (w_post) {
          float fy[8];
          open8<T>(uy[v], fy);
#pragma unroll
          for (int e = 0; e < 8; ++e) D[v][e] = r.x * fmaf(-(fy[e] * r.x), c1[0], D[v][e]);
        }
        store8<T>(dy + t * H + c, D[v]);
      }
    }
    if (a.part && ++count == kFlush) put_sums();
  }
  if (a.part)
    while (flush < a.flushes) put_sums();   // a group with fewer rows adds zeros
}

// The groups' column sums, added in order: eight warps take a part of them each.
constexpr int kJoinWarps = 8;
template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) norm_columns_kernel(const float* __restrict__ part, int64_t n, int H,
                                                                       T* dw_post, T* dgate, T* dw_pre) {
  __shared__ float4 sh[kJoinWarps][32];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = (blockIdx.x * 32 + lane) * 4;
  const int64_t each = (n + kJoinWarps - 1) / kJoinWarps, hi = min(n, (warp + 1) * each);
  float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (c < 3 * H) {
#pragma unroll 8
    for (int64_t i = warp * each; i < hi; ++i) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(part + i * 3 * H + c));
      f.x += u.x; f.y += u.y; f.z += u.z; f.w += u.w;
    }
  }
  sh[warp][lane] = f;
  __syncthreads();
  if (warp != 0 || c >= 3 * H) return;
  for (int w = 1; w < kJoinWarps; ++w) {
    const float4 u = sh[w][lane];
    f.x += u.x; f.y += u.y; f.z += u.z; f.w += u.w;
  }
  const int which = c / H, col = c - which * H;
  T* out = which == 0 ? dw_post : which == 1 ? dgate : dw_pre;
  if (out == nullptr) return;
  out[col] = from_f<T>(f.x);
  out[col + 1] = from_f<T>(f.y);
  out[col + 2] = from_f<T>(f.z);
  out[col + 3] = from_f<T>(f.w);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
moe_status decode(const moe_block_norm_shape* s, NShape* o, const char** why) {
  *why = "";
  if (!s) { *why = "shape is NULL"; return MOE_ERR_INVALID_ARG; }
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16) { *why = "dtype must be MOE_F32 or MOE_BF16"; return MOE_ERR_UNSUPPORTED; }
  if (s->tokens < 0 || s->tokens > (1ll << 28)) { *why = "tokens must be in [0, 2^28]"; return MOE_ERR_INVALID_ARG; }
  if (s->hidden <= 0 || s->hidden % 8) { *why = "hidden must be a positive multiple of 8"; return MOE_ERR_INVALID_ARG; }
  if (s->hidden > 32768) { *why = "hidden above 32768 is not supported"; return MOE_ERR_UNSUPPORTED; }
  if (s->gate < MOE_GATE_NONE || s->gate > MOE_GATE_TOKEN) { *why = "gate must be a moe_gate_kind"; return MOE_ERR_INVALID_ARG; }
  if (s->unit_offset != 0 && s->unit_offset != 1) { *why = "unit_offset must be 0 or 1"; return MOE_ERR_INVALID_ARG; }
  if (!std::isfinite((float)s->residual_scale)) { *why = "residual_scale must be finite in fp32"; return MOE_ERR_INVALID_ARG; }
  if (!((float)s->eps > 0.0f) || !std::isfinite((float)s->eps)) { *why = "eps must be positive and finite in fp32"; return MOE_ERR_INVALID_ARG; }
  o->T = s->tokens;
  o->H = s->hidden;
  o->dtype = s->dtype;
  o->esize = s->dtype == MOE_F32 ? 4 : 2;
  o->gate = s->gate;
  o->off = (float)s->unit_offset;
  o->res = (float)s->residual_scale;
  o->eps = (float)s->eps;
  return MOE_OK;
}

// The same on every device, so that a workspace's size and the sums do not depend on it.
struct Split {
  Geometry g;
  int64_t blocks;
  int flushes;
};
Split split_of(const NShape& s) {
  Split p;
  p.g = geometry(s.H, 256);
  const int threads = p.g.G * p.g.NG;
  const int per_sm = threads > 512 ? 1 : 512 / threads > 0 ? 1024 / threads / 2 + 1 : 1;
  p.blocks = std::min<int64_t>((s.T + p.g.NG - 1) / p.g.NG, 152ll * std::max(1, per_sm));
  if (p.blocks < 1) p.blocks = 1;
  const int64_t rows = (s.T + p.blocks * p.g.NG - 1) / (p.blocks * p.g.NG);   // of a group
  p.flushes = (int)std::max<int64_t>(1, (rows + kFlush - 1) / kFlush);
  return p;
}
size_t part_bytes(const NShape& s, const Split& p) {
  return (size_t)p.flushes * p.blocks * p.g.NG * 3 * s.H * 4;
}

template <typename T>
cudaError_t forward(const NShape& s, const void* x, const void* y, const void* w_post, const void* gate,
                    const void* w_pre, void* so, void* h, float* rstd, cudaStream_t st) {
  const Geometry g = geometry(s.H, 512);
  const unsigned threads = (unsigned)(g.G * g.NG);
  const int64_t need = (s.T + g.NG - 1) / g.NG, cap = (int64_t)tc_sm_count() * std::max(1u, 2048 / threads);
  const unsigned grid = (unsigned)std::min(need, cap);
  auto go = [&](auto kernel) {
    return launch_after(kernel, grid, threads, 0, st, 1, s.T, s.H, g.G, g.NG, s.gate, s.off, s.res, s.eps,
                        static_cast<const T*>(x), static_cast<const T*>(y), static_cast<const T*>(w_post), gate,
                        static_cast<const T*>(w_pre), static_cast<T*>(so), static_cast<T*>(h),
                        reinterpret_cast<float2*>(rstd));
  };
  if (g.vpt == 1) return go(norm_forward_kernel<T, 1>);
  if (g.vpt == 2) return go(norm_forward_kernel<T, 2>);
  return go(norm_forward_kernel<T, 4>);
}

template <typename T>
cudaError_t backward(const NShape& s, const Split& p, const BwdArgs& a, void* dw_post, void* dgate, void* dw_pre,
                     cudaStream_t st) {
  const unsigned threads = (unsigned)(p.g.G * p.g.NG);
  auto go = [&](auto kernel) { return launch_after(kernel, (unsigned)p.blocks, threads, 0, st, 1, a); };
  cudaError_t e = p.g.vpt == 1 ? go(norm_backward_kernel<T, 1>)
                  : p.g.vpt == 2 ? go(norm_backward_kernel<T, 2>) : go(norm_backward_kernel<T, 4>);
  if (e != cudaSuccess || !a.part) return e;
  return launch_after(norm_columns_kernel<T>, (unsigned)((3 * s.H + 127) / 128), 32 * kJoinWarps, 0, st, 1,
                      (const float*)a.part, (int64_t)p.flushes * p.blocks * p.g.NG, s.H, static_cast<T*>(dw_post),
                      static_cast<T*>(dgate), static_cast<T*>(dw_pre));
}

// What both directions ask of the inputs.
moe_status check_inputs(const NShape& s, const void* x, const void* y, const void* w_post, const void* gate,
                        const void* w_pre) {
  if (!x && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "x must be non-NULL");
  if (!y && (w_post || s.gate != MOE_GATE_NONE) && s.T > 0)
    return fail(MOE_ERR_INVALID_ARG, "w_post and a gate need y");
  if ((s.gate != MOE_GATE_NONE) != (gate != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "gate must be given iff the shape has one");
  if (!aligned16(x) || !aligned16(y) || !aligned16(w_post) || !aligned16(w_pre) ||
      (s.gate == MOE_GATE_CHANNEL && !aligned16(gate)))
    return fail(MOE_ERR_INVALID_ARG, "x, y, w_post, a channel gate and w_pre must be 16-byte aligned");
  if ((uintptr_t)gate & 3u) return fail(MOE_ERR_INVALID_ARG, "a token gate must be aligned to its elements");
  return MOE_OK;
}

}  // namespace bn
}  // namespace moe

using namespace moe;

#define DECODE_BN(shape, s)                                  \
  bn::NShape s;                                              \
  do {                                                       \
    const char* why_ = "";                                   \
    moe_status st_ = bn::decode(shape, &s, &why_);           \
    if (st_ != MOE_OK) return fail(st_, why_);               \
  } while (0)

extern "C" size_t moe_block_norm_workspace_bytes(const moe_block_norm_shape* shape) {
  bn::NShape s;
  const char* why;
  moe_status st = bn::decode(shape, &s, &why);
  if (st != MOE_OK) {
    fail(st, why);
    return 0;
  }
  return 256 + bn::part_bytes(s, bn::split_of(s));
}

extern "C" moe_status moe_block_norm_forward(const moe_block_norm_shape* shape, const void* x, const void* y,
                                             const void* w_post, const void* gate, const void* w_pre, void* so,
                                             void* h, float* rstd, void* stream) {
  reset_launch_count();
  DECODE_BN(shape, s);
  moe_status e = bn::check_inputs(s, x, y, w_post, gate, w_pre);
  if (e != MOE_OK) return e;
  if ((w_pre != nullptr) != (h != nullptr) && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "h must be given iff w_pre is");
  if (!so && !h && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "one of s and h must be non-NULL");
  if (!aligned16(so) || !aligned16(h)) return fail(MOE_ERR_INVALID_ARG, "s and h must be 16-byte aligned");
  if ((uintptr_t)rstd & 7u) return fail(MOE_ERR_INVALID_ARG, "rstd must be 8-byte aligned");
  if (s.T == 0) return MOE_OK;
  CHECK_CUDA(s.dtype == MOE_F32
                 ? bn::forward<float>(s, x, y, w_post, gate, w_pre, so, h, rstd, (cudaStream_t)stream)
                 : bn::forward<bf16>(s, x, y, w_post, gate, w_pre, so, h, rstd, (cudaStream_t)stream));
  return MOE_OK;
}

extern "C" moe_status moe_block_norm_backward(const moe_block_norm_shape* shape, const void* ds, const void* dh,
                                              const void* x, const void* y, const void* w_post, const void* gate,
                                              const void* w_pre, const float* rstd, void* dx, void* dy, void* dw_post,
                                              void* dgate, void* dw_pre, void* ws, size_t ws_bytes, void* stream) {
  reset_launch_count();
  DECODE_BN(shape, s);
  moe_status e = bn::check_inputs(s, x, y, w_post, gate, w_pre);
  if (e != MOE_OK) return e;
  if ((w_pre != nullptr) != (dh != nullptr) && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "dh must be given iff w_pre is");
  if (!ds && !dh && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "one of ds and dh must be non-NULL");
  if (!rstd && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "rstd must be non-NULL");
  if ((dy && !y && s.T > 0) || (dw_post && !w_post) || (dgate && !gate) || (dw_pre && !w_pre))
    return fail(MOE_ERR_INVALID_ARG, "a gradient's input must be non-NULL");
  if (!dx && !dy && !dw_post && !dgate && !dw_pre) return fail(MOE_ERR_INVALID_ARG, "no gradient is asked for");
  if (!aligned16(ds) || !aligned16(dh) || !aligned16(dx) || !aligned16(dy))
    return fail(MOE_ERR_INVALID_ARG, "ds, dh, dx and dy must be 16-byte aligned");
  if (((uintptr_t)dw_post | (uintptr_t)dw_pre | (uintptr_t)dgate) & (uintptr_t)(s.esize - 1) ||
      (s.gate == MOE_GATE_TOKEN && ((uintptr_t)dgate & 3u)))
    return fail(MOE_ERR_INVALID_ARG, "dw_post, dgate and dw_pre must be aligned to their elements");
  if ((uintptr_t)rstd & 7u) return fail(MOE_ERR_INVALID_ARG, "rstd must be 8-byte aligned");
  const bn::Split p = bn::split_of(s);
  e = check_ws(ws, ws_bytes, 256 + bn::part_bytes(s, p));
  if (e != MOE_OK) return e;
  const bool channel = s.gate == MOE_GATE_CHANNEL;
  bn::BwdArgs a = {};
  a.rows = s.T;
  a.H = s.H;
  a.G = p.g.G;
  a.NG = p.g.NG;
  a.kind = s.gate;
  a.flushes = p.flushes;
  a.off = s.off;
  a.res = s.res;
  a.ds = ds;
  a.dh = dh;
  a.x = x;
  a.y = y;
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.rstd = reinterpret_cast<const float2*>(rstd);
  a.dx = dx;
  a.dy = dy;
  a.dgate = channel ? nullptr : static_cast<float*>(dgate);
  // without tokens the columns' sums are zeros, written like any others
  if (dw_post || dw_pre || (channel && dgate)) a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
  if (s.T == 0 && !a.part) return MOE_OK;
  void* dcol = channel ? dgate : nullptr;
  CHECK_CUDA(s.dtype == MOE_F32 ? bn::backward<float>(s, p, a, dw_post, dcol, dw_pre, (cudaStream_t)stream)
                                : bn::backward<bf16>(s, p, a, dw_post, dcol, dw_pre, (cudaStream_t)stream));
  return MOE_OK;
}
