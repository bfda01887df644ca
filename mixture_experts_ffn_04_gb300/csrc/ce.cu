// ce.cu -- softmax cross entropy of a linear classifier over a vocabulary, and
// its gradient, without the [tokens, vocab] logits (include/moe_train.h).
//
//   z = x W^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,target
//   d = g (softmax(z) - onehot(target)),  dx = d W,  dW = d^T x
//
// The tokens that count are packed into a dense matrix first (one pass over x,
// small against W and the products), so ignored tokens cost nothing and what
// their rows hold reaches no sum.  Forward: one GEMM over all of W whose
// epilogue keeps, per row and 128 columns, a maximum and a sum of exponentials,
// and a kernel that merges them.  Backward: pieces of the vocabulary; per piece
// the logits again with d in the epilogue (kept for the piece only), then both
// gradient products in one launch.  8 T H V flops for loss and gradient, of
// which 2 T H V recompute the logits.
//
// Up to two rows (fp32: 32) the logits are not tiles' work but a pass over W, forward
// and backward; the gradient products are the same.
//
// Every exponential is of a difference from a maximum, and the backward's logits are
// added up exactly as the forward's: probabilities stay in [0, 1] whatever the logits'
// size.
//
// Measured (bf16): T = 4096, H = 2048, V = 131072 loss and gradient 5.66 to 5.84 ms
// from GPU to GPU, 1.5-1.55 PFLOP/s under the power cap (0.9 of the sustained
// matrix-product rate); of its launches packing, merging and adding up dx take 55 us.
#include <algorithm>

#include "../../include/moe_train.h"
#include "common.cuh"
#include "internal.h"
#include "train.h"

namespace moe {
namespace {

// Logit gradient of one piece.  T = 4096, V = 131072 (loss and gradient; one GPU, the
// gradient's logits then in chunks of 4096, 2 % faster than now): pieces of 64 MiB 5768
// us, 128 5613, 256 5525, 512 5478, all in one (1 GiB) 5446: each piece costs a launch
// pair's tail, and larger ones only memory.
constexpr int64_t kDlogitBytes = 512ll << 20;
// Tokens up to which a bf16 call keeps the logit gradient in two bf16 planes.  Its
// rounding to one adds the result's own error once more where it averages out (1.45
// times the error with weights per token, at 64 rows and at 1000), but up to 2.1 times
// at one row, 1.7 at 16, 1.6 at 32, where few large entries carry a result; the second
// plane costs a quarter of such a backward (H = 2048, V = 50257, 16 rows 165 us against
// 203), and as much as a third from 256 rows on (389 rows 250 against 363).
constexpr int kTwoPlaneRows = 32;
// Planes of one piece of an fp32 W.  T = 64, H = 2048, V = 50257: pieces of 512 MiB
// (two of them, four rounds of tiles) 494 us the loss and 1337 with the gradient, of 768
// (one, three rounds) 417 and 1158.
constexpr int64_t kPlaneBytes = 768ll << 20;

// packing: tokens of a tile, most blocks, tokens up to which each block counts for itself
constexpr int kPackTile = 256, kPackBlocks = 1024, kPackSelf = 4096;

// the few-row kernels: most rows of x, blocks an SM, shared memory of x
constexpr int kSkinnyRows = 32, kSkinnyPerSm = 4, kSkinnySmem = 220 * 1024;

struct CeShape {
  int64_t T, x_ld, w_ld;
  int H, V, dtype, reduction, ignore, esize, planes, d_planes;
};

moe_status decode_ce(const moe_ce_shape* s, CeShape* o, const char** why) {
  if (!s) { *why = "shape is NULL"; return MOE_ERR_INVALID_ARG; }
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16) {
    *why = "dtype must be MOE_F32 or MOE_BF16";
    return MOE_ERR_UNSUPPORTED;
  }
  if (s->tokens < 0 || s->tokens > (1ll << 28)) {
    *why = "tokens must be in [0, 2^28]";
    return MOE_ERR_INVALID_ARG;
  }
  if (s->hidden <= 0 || s->hidden % 8) {
    *why = "hidden must be a positive multiple of 8";
    return MOE_ERR_INVALID_ARG;
  }
  if (s->vocab < 1 || s->vocab > (1 << 30)) {
    *why = "vocab must be in [1, 2^30]";
    return MOE_ERR_INVALID_ARG;
  }
  if (s->reduction < MOE_CE_NONE || s->reduction > MOE_CE_MEAN) {
    *why = "reduction must be MOE_CE_NONE, MOE_CE_SUM or MOE_CE_MEAN";
    return MOE_ERR_INVALID_ARG;
  }
  if ((double)s->tokens * s->vocab >= (double)(1ll << 46)) {
    *why = "tokens * vocab must be below 2^46";
    return MOE_ERR_UNSUPPORTED;
  }
  o->x_ld = s->x_stride ? s->x_stride : s->hidden;
  o->w_ld = s->w_stride ? s->w_stride : s->hidden;
  if (o->x_ld < s->hidden || o->x_ld % 8 || o->w_ld < s->hidden || o->w_ld % 8 ||
      o->x_ld >= (1ll << 32) || o->w_ld >= (1ll << 32)) {
    *why = "x_stride and w_stride must be 0 or at least hidden, and multiples of 8";
    return MOE_ERR_INVALID_ARG;
  }
  o->T = s->tokens;
  o->H = s->hidden;
  o->V = s->vocab;
  o->dtype = s->dtype;
  o->reduction = s->reduction;
  o->ignore = s->ignore_index;
  o->esize = s->dtype == MOE_F32 ? 4 : 2;
  o->planes = s->dtype == MOE_F32 ? kPlanesF32 : 1;
  o->d_planes = s->dtype == MOE_F32 ? kPlanesF32 : s->tokens <= kTwoPlaneRows ? 2 : 1;
  return MOE_OK;
}

struct CeLayout {
  int64_t rows_pad, piece, npieces;   // vocabulary columns of a piece
  int64_t nctr;
  LinearSplit split;
  bool dx_direct, dw_direct;
  size_t flags, skinny, meta, ctr, count, rowmap, inv, tgt, g, rowstat, zt, loss, xc, wpl, stats, d, dx_part, dw_part, total;
};

CeLayout layout_ce(const CeShape& s) {
  CeLayout L;
  L.rows_pad = std::max<int64_t>(256, (s.T + 255) / 256 * 256);
  const int64_t vpad = ((int64_t)s.V + 255) / 256 * 256;
  int64_t piece = kDlogitBytes / (L.rows_pad * 2 * s.d_planes) / 256 * 256;
  if (s.planes > 1) piece = std::min(piece, kPlaneBytes / ((int64_t)s.H * 2 * s.planes) / 256 * 256);
  piece = std::max<int64_t>(piece, 256);
  L.npieces = (vpad + piece - 1) / piece;
  // pieces of equal size
  L.piece = ((vpad + L.npieces - 1) / L.npieces + 255) / 256 * 256;
  L.npieces = (vpad + L.piece - 1) / L.piece;
  L.split = linear_grad_split(s.T, L.piece, s.H);
  L.dx_direct = L.npieces == 1 && L.split.dx == 1;
  L.dw_direct = L.split.dw == 1;
  L.nctr = 2 * L.npieces;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~(size_t)255;
    return at;
  };
  const size_t T = (size_t)L.rows_pad;
  L.flags = take(256);   // status word; the few-row kernel's ticket at +32
  L.skinny = take(s.T <= kSkinnyRows ? (size_t)tc_sm_count() * kSkinnyPerSm * s.T * 8 : 0);
  L.meta = take(256);   // rows that count, the merge's ticket, the gradients' scale
  L.ctr = take((size_t)L.nctr * 4);
  L.count = take(kPackBlocks * 4);
  L.rowmap = take(T * 4);
  L.inv = take(T * 4);
  L.tgt = take(T * 4);
  L.g = take(T * 4);
  L.rowstat = take(T * 16);
  L.zt = take(T * 4);
  L.loss = take(T * 4);
  L.xc = take((size_t)s.planes * T * s.H * 2);
  L.wpl = take(s.planes > 1 ? (size_t)s.planes * L.piece * s.H * 2 : 0);
  const size_t base = off;
  L.stats = take((size_t)(vpad / 128) * T * 8);
  const size_t fwd_end = off;
  off = base;   // the backward's buffers take the forward statistics' place
  L.d = take((size_t)s.d_planes * T * L.piece * 2);
  L.dx_part = take(L.dx_direct ? 0 : (size_t)L.split.dx * T * s.H * 4);
  L.dw_part = take(L.dw_direct ? 0 : (size_t)L.split.dw * L.piece * s.H * 4);
  L.total = std::max(off, fwd_end);
  return L;
}

struct PrepArgs {
  const int32_t* target;
  const int32_t* count;   // of each block's tokens, or NULL
  int64_t T, rows_per_block;
  int V, ignore, H;
  const void* x;
  int64_t x_ld, plane;
  bf16* xc;
  int32_t *nrows, *ticket, *ctr, *rowmap, *inv, *tgt;
  float* scale;   // of the gradients, for the backward
  int64_t nctr;
  uint32_t* flags;
  // forward: zero the outputs of tokens that do not count
  float *loss, *lse_out;
  float4* stats_out;
  // backward
  const float4* rowstat;
  const float* dloss;
  float* g;
  float4* rowstat_c;
  int reduction;
  void* dx;   // zero the rows of tokens that do not count (direct dx), or NULL
};

__device__ __forceinline__ bool counts(int t, int V, int ignore) { return t != ignore && t >= 0 && t < V; }

// Tokens that count in each block's range, for more than kPackSelf tokens: with every
// block counting all of them, as below, the reads grow with the square of the tokens.
// Packing and a two-column loss at H = 8, counted here against each block for itself:
// T = 4096 25.2 / 25.1 us, 8192 27 / 33, 65536 92 / 140, 262144 287 / 486; H = 1024:
// 36 / 35, 35 / 37, 157 / 196, 560 / 734.
__global__ void __launch_bounds__(kPackTile) ce_count_kernel(const int32_t* __restrict__ target, int64_t T,
                                                             int64_t rows_per_block, int V, int ignore,
                                                             int32_t* count) {
  __shared__ int s_sum;
  pdl_trigger();
  pdl_wait();
  const int64_t beg = min(T, blockIdx.x * rows_per_block), end = min(T, beg + rows_per_block);
  if (threadIdx.x == 0) s_sum = 0;
  __syncthreads();
  int c = 0;
  for (int64_t i = beg + threadIdx.x; i < end; i += blockDim.x) c += counts(target[i], V, ignore) ? 1 : 0;
  c = __reduce_add_sync(0xffffffffu, c);
  if ((threadIdx.x & 31) == 0) atomicAdd(&s_sum, c);   // integers: the order does not matter
  __syncthreads();
  if (threadIdx.x == 0) count[blockIdx.x] = s_sum;
}

// Pack the tokens that count: block b takes rows_per_block tokens, counts those
// before its own (a pass over the targets, which every block reads from L2; over the
// blocks' counts where there are any) and copies its rows -- bf16 as they are, fp32 as
// planes.  Rows from the count up to a multiple of 64 are zeroed: the dW product's last
// k-block reads them.  Latency-bound at small T; at 8192 x 7168 bound by the copy.
template <typename T>
__global__ void __launch_bounds__(kPackTile) ce_prep_kernel(const PrepArgs a) {
  __shared__ int s_before, s_total, s_cnt[kPackTile], s_warp[kPackTile / 32];
  pdl_trigger();
  pdl_wait();
  const int64_t beg = min(a.T, blockIdx.x * a.rows_per_block), end = min(a.T, beg + a.rows_per_block);
  if (threadIdx.x == 0) s_before = s_total = 0;
  __syncthreads();
  int before = 0, total = 0;
  if (a.count) {
    for (int i = threadIdx.x; i < (int)gridDim.x; i += blockDim.x) {
      const int c = a.count[i];
      total += c;
      if (i < (int)blockIdx.x) before += c;
    }
  } else {
    for (int64_t i = threadIdx.x; i < a.T; i += blockDim.x) {
      const int c = counts(a.target[i], a.V, a.ignore) ? 1 : 0;
      total += c;
      if (i < beg) before += c;
    }
  }
  before = __reduce_add_sync(0xffffffffu, before);
  total = __reduce_add_sync(0xffffffffu, total);
  if ((threadIdx.x & 31) == 0) {
    atomicAdd(&s_before, before);   // integers: the order does not matter
    atomicAdd(&s_total, total);
  }
  __syncthreads();
  if (blockIdx.x == 0) {
    if (threadIdx.x == 0) {
      *a.nrows = s_total;
      *a.ticket = 0;
      // One factor of every token's gradient stays out of the logit gradient, where
      // its rounding to bf16 would be the same relative error in every entry.
      float g = 1.0f;
      if (a.g && a.reduction != MOE_CE_NONE) {
        if (a.dloss) g = a.dloss[0];
        if (a.reduction == MOE_CE_MEAN && s_total > 0) g /= (float)s_total;
      }
      *a.scale = g;
    }
    for (int64_t i = threadIdx.x; i < a.nctr; i += blockDim.x) a.ctr[i] = 0;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* x = reinterpret_cast<const T*>(a.x);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int nv = a.H / 8;
  int base = s_before;
  for (int64_t tile = beg; tile < end; tile += kPackTile) {
    // place of each of the tile's tokens among those that count
    const int64_t mine = tile + threadIdx.x;
    int t = a.ignore;
    if (mine < end) t = a.target[mine];
    const bool ok = mine < end && counts(t, a.V, a.ignore);
    if (mine < end && !ok && t != a.ignore) set_flag(a.flags, kFlagTarget);
    const uint32_t ball = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) s_warp[warp] = __popc(ball);
    __syncthreads();
    int pos = base;
    for (int w = 0; w < kPackTile / 32; ++w) {
      if (w < warp) pos += s_warp[w];
      base += s_warp[w];
    }
    pos += __popc(ball & ((1u << lane) - 1u));
    if (mine < end) {
      s_cnt[threadIdx.x] = ok ? pos : -1;
      a.inv[mine] = ok ? pos : -1;
      if (ok) {
        a.rowmap[pos] = (int32_t)mine;
        a.tgt[pos] = t;
        if (a.g) {
          a.g[pos] = a.reduction == MOE_CE_NONE ? a.dloss[mine] : 1.0f;
          a.rowstat_c[pos] = a.rowstat[mine];
        }
      } else {
        if (a.loss) a.loss[mine] = 0.0f;
        if (a.lse_out) a.lse_out[mine] = 0.0f;
        if (a.stats_out) a.stats_out[mine] = make_float4(0.0f, 1.0f, 0.0f, 0.0f);
      }
    }
    __syncthreads();
    // copy the rows: a warp a row
    for (int r = warp; r < kPackTile && tile + r < end; r += kPackTile / 32) {
      const int p = s_cnt[r];
      if (p < 0) {
        if (a.dx) {
          uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.dx) + (tile + r) * (int64_t)a.H);
          for (int v = lane; v < nv * (int)(sizeof(T) / 2); v += 32) o[v] = zero;
        }
        continue;
      }
      const T* src = x + (tile + r) * a.x_ld;
      bf16* dst = a.xc + (int64_t)p * a.H;
      if (sizeof(T) == 2) {
#pragma unroll 4
        for (int v = lane; v < nv; v += 32)
          reinterpret_cast<uint4*>(dst)[v] = reinterpret_cast<const uint4*>(src)[v];
      } else {
        for (int v = lane; v < nv; v += 32) {
          const float4 u = reinterpret_cast<const float4*>(src)[2 * v];
          const float4 w = reinterpret_cast<const float4*>(src)[2 * v + 1];
          float f[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
          for (int pl = 0; pl < kPlanesF32; ++pl) {
            float q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = take_plane(f[e]);
            reinterpret_cast<uint4*>(dst + pl * a.plane * a.H)[v] = pack16(q, (const bf16*)nullptr);
          }
        }
      }
    }
    __syncthreads();   // s_warp and s_cnt are the next tile's
  }
  const int total_rows = s_total, pad_end = (total_rows + 63) / 64 * 64;
  const int planes = sizeof(T) == 2 ? 1 : kPlanesF32;
  for (int r = total_rows + blockIdx.x; r < pad_end; r += gridDim.x)
    for (int pl = 0; pl < planes; ++pl)
      for (int v = threadIdx.x; v < nv; v += blockDim.x)
        reinterpret_cast<uint4*>(a.xc + (pl * a.plane + r) * a.H)[v] = zero;
}

// Maximum M and sum of exponentials S joined with another pair's.
__device__ __forceinline__ void merge_ms(float& M, float& S, float m, float s) {
  const float log2e = 1.4426950408889634f, n = fmaxf(M, m), mu = n == -INFINITY ? 0.0f : n;
  S = S * exp2f((M - mu) * log2e) + s * exp2f((m - mu) * log2e);
  M = n;
}

// A row from the maximum m and sum of exponentials of its other columns and its
// target's logit:  M = the larger of m and z_t, R = the others' sum under M, S = R +
// e^(z_t - M);  loss = ln(S / e_t) = log1p(R / e_t).  With the target apart neither
// the loss nor the gradient p_t - 1 = -R / S of a nearly certain target loses digits
// to 1 or to lse.
struct RowStat {
  float4 stat;   // M, S, R, 0
  float lse, loss;
};
__device__ __forceinline__ RowStat finish_row(float m, float s, float zt) {
  const float log2e = 1.4426950408889634f;
  const float M = fmaxf(m, zt), Mu = M == -INFINITY ? 0.0f : M;
  const float R = s * exp2f((m - Mu) * log2e), et = exp2f((zt - Mu) * log2e), S = R + et;
  RowStat r;
  r.stat = make_float4(Mu, S, R, 0.0f);
  r.lse = Mu + logf(S);
  r.loss = R <= et ? log1pf(R / et) : (Mu - zt) + logf(S);
  return r;
}

// Merge the row statistics of all half tiles (lanes: 32 rows, warps: slices of
// the half tiles): the other columns' maximum and sum, then the row (above).  The
// last block adds the rows' losses, in row order, in fp64.
// (T = 4096, V = 131072: 34 MB of statistics in 20 us, bound by their latency.)
constexpr int kMergeWarps = 32;
__global__ void __launch_bounds__(32 * kMergeWarps)
    ce_merge_kernel(const float2* __restrict__ stats, int64_t rows_pad, int parts,
                    const float* __restrict__ zt, const int32_t* __restrict__ rowmap,
                    const int32_t* nrows, int32_t* ticket, float* loss_c, float* loss, float* lse,
                    float4* rowstat, float* total, int mean) {
  pdl_trigger();
  pdl_wait();
  const int n = *nrows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float2 s_part[kMergeWarps][32];
  for (int64_t r0 = blockIdx.x * 32ll; r0 < n; r0 += gridDim.x * 32ll) {
    const int64_t row = r0 + lane;
    float M = -INFINITY, S = 0.0f;
    if (row < n) {
#pragma unroll 8
      for (int p = warp; p < parts; p += kMergeWarps) {
        const float2 v = __ldcs(stats + p * rows_pad + row);
        merge_ms(M, S, v.x, v.y);
      }
    }
    s_part[warp][lane] = make_float2(M, S);
    __syncthreads();
    if (warp == 0 && row < n) {
      for (int w = 1; w < kMergeWarps; ++w) {
        const float2 v = s_part[w][lane];
        merge_ms(M, S, v.x, v.y);
      }
      const RowStat r = finish_row(M, S, zt[row]);
      const float each = r.loss;
      const int t = rowmap[row];
      if (lse) lse[t] = r.lse;
      if (rowstat) rowstat[t] = r.stat;
      if (loss) loss[t] = each;
      loss_c[row] = each;
    }
    __syncthreads();
  }
  if (!total) return;
  __shared__ int s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(ticket, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double acc = 0.0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) acc += (double)__ldcg(loss_c + i);
  __shared__ double s_sum[kMergeWarps];
#pragma unroll
  for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) s_sum[warp] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int w = 0; w < kMergeWarps; ++w) v += s_sum[w];
    if (mean && n > 0) v /= (double)n;
    *total = (float)v;
  }
}

// The logits of R rows against vocabulary rows v .. vend: a warp takes NV rows of W at a
// time (all lanes across the row, 16 bytes a load) against the rows of x in shared
// memory (fp32); lane k R + r is handed the logit of row k and x row r.  Forward and
// backward both call it: the same sums in the same order, whatever R and NV are, so the
// backward's logits are those of the statistics.
template <typename T, int R, int NV, typename F>
__device__ __forceinline__ void skinny_logits(const T* w, int64_t w_ld, const float* s_x, int H, int64_t v,
                                              int64_t vend, F&& take) {
  static_assert(NV * R <= 32, "a lane a logit");
  constexpr int N = Vec16<T>::N;
  const int lane = threadIdx.x & 31;
  for (; v < vend; v += NV) {
    float acc[NV][R];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int r = 0; r < R; ++r) acc[k][r] = 0.0f;
    const T* wr[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) wr[k] = w + min(v + k, vend - 1) * w_ld;
#pragma unroll 4
    for (int i = lane * N; i < H; i += 32 * N) {
      uint4 u[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k) u[k] = __ldcs(reinterpret_cast<const uint4*>(wr[k] + i));
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float f[N];
        unpack16(u[k], f, (const T*)nullptr);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int e = 0; e < N; e += 4) {
            const float4 xv = *reinterpret_cast<const float4*>(s_x + r * H + i + e);
            acc[k][r] = fmaf(f[e], xv.x, acc[k][r]);
            acc[k][r] = fmaf(f[e + 1], xv.y, acc[k][r]);
            acc[k][r] = fmaf(f[e + 2], xv.z, acc[k][r]);
            acc[k][r] = fmaf(f[e + 3], xv.w, acc[k][r]);
          }
      }
    }
    float mine = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float z = acc[k][r];
#pragma unroll
        for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane == k * R + r) mine = z;
      }
    if (lane < NV * R && v + lane / R < vend) take(v + lane / R, mine);
  }
}

// Warps a block: more where a block's rows of x leave room for one or two blocks an SM.
template <int R>
constexpr int kFewWarps = R <= 8 ? 8 : 16;
template <int R>
constexpr int kFewBlocks = R <= 2 ? kSkinnyPerSm : R <= 8 ? 2 : 1;

// x of rows first .. first + R into shared memory (zeros where a row does not count,
// whatever x holds).
template <typename T, int R>
__device__ __forceinline__ void skinny_rows(const T* x, int64_t x_ld, const int32_t* target, int first, int rows,
                                            int H, int V, int ignore, float* s_x) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const bool ok = first + r < rows && counts(target[first + r], V, ignore);
    const T* xr = x + (first + r) * x_ld;
    for (int i = threadIdx.x; i < H; i += blockDim.x) s_x[r * H + i] = ok ? to_f(xr[i]) : 0.0f;
  }
  __syncthreads();
}

// Loss of few rows in one launch: W streams by, a running maximum and sum per row of x,
// and the last block merges the blocks.  More than R rows go in groups of R, whose
// blocks of the same part of W are neighbours, so that it comes from HBM once.  Bound by
// HBM up to R = 4: one token against 50257 x 2048 bf16 reads 206 MB in 38 us, 5.4 TB/s
// (0.80 of the copy); with two blocks an SM instead of four it took 63 (too few loads in
// flight).  From R = 8 on by the FMAs and the reads of x from shared memory.
struct SkinnyArgs {
  const void *x, *w;
  int64_t x_ld, w_ld;
  const int32_t* target;
  int T, H, V, ignore, reduction;
  float *loss, *lse, *total;
  float4* rowstat;   // [T] or NULL
  int groups;        // of R rows
  float2* part;      // [grid / groups][T]
  float* zt;         // [T]
  int32_t* ticket;   // 0 between calls
  uint32_t* flags;
};
template <typename T, int R, int NV>
__global__ void __launch_bounds__(32 * kFewWarps<R>, kFewBlocks<R>) ce_skinny_kernel(const SkinnyArgs a) {
  pdl_trigger();
  pdl_wait();
  constexpr int W = kFewWarps<R>;
  extern __shared__ __align__(16) float s_x[];   // [R][H]
  __shared__ float2 s_ms[W][R];
  __shared__ float s_loss[kSkinnyRows];
  __shared__ int s_last;
  const int first = blockIdx.x % a.groups * R, block = blockIdx.x / a.groups, blocks = gridDim.x / a.groups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  skinny_rows<T, R>(reinterpret_cast<const T*>(a.x), a.x_ld, a.target, first, a.T, a.H, a.V, a.ignore, s_x);
  if (blockIdx.x == 0 && (int)threadIdx.x < a.T) {
    const int t = a.target[threadIdx.x];
    if (t != a.ignore && !counts(t, a.V, a.ignore)) set_flag(a.flags, kFlagTarget);
  }
  const int row = first + lane % R, target = row < a.T ? a.target[row] : -1;
  float M = -INFINITY, S = 0.0f;
  // a contiguous range of rows a warp: every warp has the same number, but one
  const int64_t all = (int64_t)blocks * W, me = (int64_t)block * W + warp;
  skinny_logits<T, R, NV>(reinterpret_cast<const T*>(a.w), a.w_ld, s_x, a.H, a.V * me / all,
                          a.V * (me + 1) / all, [&](int64_t v, float z) {
                            if (target != (int)v) merge_ms(M, S, z, 1.0f);
                            else a.zt[row] = z;   // the target is merged by itself
                          });
#pragma unroll
  for (int o = R; o < NV * R; o <<= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, M, o), s2 = __shfl_xor_sync(0xffffffffu, S, o);
    merge_ms(M, S, m2, s2);
  }
  if (lane < R) s_ms[warp][lane] = make_float2(M, S);
  __syncthreads();
  if (threadIdx.x < R && first + (int)threadIdx.x < a.T) {
    float m = -INFINITY, s = 0.0f;
    for (int k = 0; k < W; ++k) merge_ms(m, s, s_ms[k][threadIdx.x].x, s_ms[k][threadIdx.x].y);
    a.part[block * a.T + first + threadIdx.x] = make_float2(m, s);
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  for (int r = warp; r < a.T; r += W) {
    float m = -INFINITY, s = 0.0f;
    for (int b = lane; b < blocks; b += 32) {
      const float2 p = __ldcg(a.part + b * a.T + r);
      merge_ms(m, s, p.x, p.y);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      merge_ms(m, s, m2, s2);
    }
    if (lane == 0) {
      const bool ok = counts(a.target[r], a.V, a.ignore);
      RowStat q = {make_float4(0.0f, 1.0f, 0.0f, 0.0f), 0.0f, 0.0f};
      if (ok) q = finish_row(m, s, __ldcg(a.zt + r));
      if (a.lse) a.lse[r] = q.lse;
      if (a.rowstat) a.rowstat[r] = q.stat;
      if (a.loss) a.loss[r] = q.loss;
      s_loss[r] = q.loss;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    if (a.total) {
      double t = 0.0;
      int n = 0;
      for (int r = 0; r < a.T; ++r)
        if (counts(a.target[r], a.V, a.ignore)) {
          t += (double)s_loss[r];
          ++n;
        }
      if (a.reduction == MOE_CE_MEAN && n > 0) t /= (double)n;
      *a.total = (float)t;
    }
    *a.ticket = 0;
  }
}

// The logit gradient of few rows, in the place of the tiles' (whose logits, added up in
// another order, differ from the statistics by their rounding: at logits of 1e5 that is
// a probability's whole size).  d [planes][plane][d_ld] of columns v0 .. v0 + vcols; row
// of d: the token's place among those that count.  The rows up to 64, which the dW
// product's k-block reads, and the columns past the vocabulary are zeroed.
struct SkinnyGradArgs {
  const void *x, *w;
  int64_t x_ld, w_ld;
  const int32_t* target;
  int T, H, V, ignore, planes, groups;
  const float4* rowstat;   // [T]
  const float* g;          // of the rows that count
  int64_t v0, vcols, plane, d_ld;
  bf16* d;
};
template <typename T, int R, int NV>
__global__ void __launch_bounds__(32 * kFewWarps<R>, kFewBlocks<R>)
    ce_skinny_grad_kernel(const SkinnyGradArgs a) {
  pdl_trigger();
  pdl_wait();
  constexpr int W = kFewWarps<R>;
  extern __shared__ __align__(16) float s_x[];   // [R][H]
  const int first = blockIdx.x % a.groups * R, block = blockIdx.x / a.groups, blocks = gridDim.x / a.groups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this lane's row: its place among those that count (-1: it does not)
  const int row = first + lane % R;
  int n = 0, pos = -1;
  for (int r = 0; r < a.T; ++r) {
    const bool ok = counts(a.target[r], a.V, a.ignore);
    if (ok && r == row) pos = n;
    n += ok ? 1 : 0;
  }
  float4 ms = make_float4(0.0f, 1.0f, 0.0f, 0.0f);
  float gs = 0.0f;
  int target = -1;
  if (pos >= 0) {
    ms = a.rowstat[row];
    gs = a.g[pos] / ms.y;
    target = a.target[row];
  }
  skinny_rows<T, R>(reinterpret_cast<const T*>(a.x), a.x_ld, a.target, first, a.T, a.H, a.V, a.ignore, s_x);
  auto put = [&](int row, int64_t c, float v) {
    for (int p = 0; p < a.planes; ++p) a.d[(p * a.plane + row) * a.d_ld + c] = __float2bfloat16_rn(take_plane(v));
  };
  const int64_t have = min(a.vcols, a.V - a.v0);
  const int64_t all = (int64_t)blocks * W, me = (int64_t)block * W + warp;
  skinny_logits<T, R, NV>(reinterpret_cast<const T*>(a.w) + a.v0 * a.w_ld, a.w_ld, s_x, a.H, have * me / all,
                          have * (me + 1) / all, [&](int64_t c, float z) {
                            if (pos < 0) return;
                            const float e = exp2f((z - ms.x) * 1.4426950408889634f) * gs;
                            put(pos, c, a.v0 + c == target ? -gs * ms.z : e);
                          });
  const int64_t tid = blockIdx.x * (int64_t)blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = tid; i < n * (a.vcols - have); i += step) put((int)(i % n), have + i / n, 0.0f);
  const int64_t per = a.vcols / 8;   // 16-byte pieces of a row (vcols: a multiple of 256)
  for (int64_t i = tid; i < a.planes * (64 - n) * per; i += step) {
    const int64_t row = i / per;
    const int64_t at = (row / (64 - n)) * a.plane + n + row % (64 - n);
    *reinterpret_cast<uint4*>(a.d + at * a.d_ld + (i % per) * 8) = make_uint4(0, 0, 0, 0);
  }
}

// Rows of x a block holds.
int skinny_group(const CeShape& s) {
  if (s.T <= 2) return (int)s.T;   // (all of bf16's)
  int r = s.T <= 4 ? 4 : s.T <= 8 ? 8 : 16;
  while (r > 4 && (size_t)r * s.H * 4 > (size_t)kSkinnySmem) r /= 2;
  return r;
}

// Both few-row kernels: R rows of x a block, `vocab` rows of W.
template <int R, int NV, typename Args>
cudaError_t launch_few(void (*kernel)(Args), int64_t vocab, Args a, cudaStream_t st) {
  constexpr int W = kFewWarps<R>;
  const size_t smem = (size_t)R * a.H * 4;
  if (smem > 40 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  a.groups = (a.T + R - 1) / R;
  const int64_t want = (vocab + W * NV - 1) / (W * NV);
  // as many blocks an SM as the kernel is compiled for, if x fits so often
  const int per = (int)std::max<size_t>(1, std::min<size_t>(kFewBlocks<R>, 220 * 1024 / (smem + 1024)));
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(want, (int64_t)tc_sm_count() * per / a.groups));
  return launch_after(kernel, (unsigned)(parts * a.groups), 32 * W, smem, st, 1, a);
}
cudaError_t launch_skinny(const CeShape& s, const SkinnyArgs& a, cudaStream_t st) {
  const bool f = s.dtype == MOE_F32;
  switch (skinny_group(s)) {
    case 1: return launch_few<1, 2>(f ? ce_skinny_kernel<float, 1, 2> : ce_skinny_kernel<bf16, 1, 2>, s.V, a, st);
    case 2: return launch_few<2, 2>(f ? ce_skinny_kernel<float, 2, 2> : ce_skinny_kernel<bf16, 2, 2>, s.V, a, st);
    case 4: return launch_few<4, 4>(ce_skinny_kernel<float, 4, 4>, s.V, a, st);
    case 8: return launch_few<8, 4>(ce_skinny_kernel<float, 8, 4>, s.V, a, st);
    default: return launch_few<16, 2>(ce_skinny_kernel<float, 16, 2>, s.V, a, st);
  }
}
cudaError_t launch_skinny_grad(const CeShape& s, const SkinnyGradArgs& a, cudaStream_t st) {
  const bool f = s.dtype == MOE_F32;
  const int64_t have = std::min<int64_t>(a.vcols, a.V - a.v0);
  switch (skinny_group(s)) {
    case 1:
      return launch_few<1, 2>(f ? ce_skinny_grad_kernel<float, 1, 2> : ce_skinny_grad_kernel<bf16, 1, 2>, have, a, st);
    case 2:
      return launch_few<2, 2>(f ? ce_skinny_grad_kernel<float, 2, 2> : ce_skinny_grad_kernel<bf16, 2, 2>, have, a, st);
    case 4: return launch_few<4, 4>(ce_skinny_grad_kernel<float, 4, 4>, have, a, st);
    case 8: return launch_few<8, 4>(ce_skinny_grad_kernel<float, 8, 4>, have, a, st);
    default: return launch_few<16, 2>(ce_skinny_grad_kernel<float, 16, 2>, have, a, st);
  }
}

// The few-row kernels against the tensor cores' tiles (which do the work of 256 rows
// whatever T is, fp32 after turning W into planes).  Loss, us, few-row / tiles:
//   H, V            bf16  T = 1    2         fp32  T = 1     4         8         16        32        48
//   2048, 50257     38 / 64   48 / 64        70 / 412  77 / 412  105 / 413 160 / 412 286 / 414 416 / 412
//   1024, 32001                              28 / 152  33 / 153   51 / 153  73 / 152 124 / 152 172 / 153
//   7168, 32768     79 / 120  99 / 120      148 / 915 204 / 915  330 / 917 586 / 916 (groups of 4)
// and with the gradient, fp32:
//   2048, 50257                             660       698       757 / 1154 863 / 1156 1128 / 1156 1397 / 1155
//   1024, 32001                             247       267       301 / 429  356 / 434   470 / 434   574 / 437
//   7168, 32768                            1601      1946      2330 / 2645 3151 / 2647
// bf16 takes four rows in 59 us against 64, at H = 7168 135 against 120.  So two rows in
// bf16, in fp32 two groups of as many rows as a block holds.
bool skinny_ok(const CeShape& s) {
  if (s.T < 1 || s.T > (s.dtype == MOE_F32 ? kSkinnyRows : 2)) return false;
  const int r = skinny_group(s);
  return s.T <= 2 * r && (size_t)r * s.H * 4 <= (size_t)kSkinnySmem;
}

cudaError_t run_prep(const CeShape& s, const CeLayout& L, char* ws, PrepArgs& p, cudaStream_t st) {
  p.T = s.T;
  // a warp a token up to 8192 tokens, then more; whole tiles above 2^18 tokens
  int64_t rpb = std::max<int64_t>(((s.T + kPackBlocks - 1) / kPackBlocks + 7) / 8 * 8, 8);
  if (rpb > kPackTile) rpb = (rpb + kPackTile - 1) / kPackTile * kPackTile;
  const int64_t blocks = std::max<int64_t>((s.T + rpb - 1) / rpb, 32);
  if (s.T > kPackSelf) {
    int32_t* count = reinterpret_cast<int32_t*>(ws + L.count);
    const cudaError_t e = launch_after(ce_count_kernel, (unsigned)blocks, kPackTile, 0, st, 1, p.target, s.T, rpb,
                                       s.V, s.ignore, count);
    if (e != cudaSuccess) return e;
    p.count = count;
  }
  p.rows_per_block = rpb;
  p.V = s.V;
  p.ignore = s.ignore;
  p.H = s.H;
  p.x_ld = s.x_ld;
  p.plane = L.rows_pad;
  p.xc = reinterpret_cast<bf16*>(ws + L.xc);
  p.nrows = reinterpret_cast<int32_t*>(ws + L.meta);
  p.ticket = p.nrows + 1;
  p.scale = reinterpret_cast<float*>(p.nrows + 2);
  p.ctr = reinterpret_cast<int32_t*>(ws + L.ctr);
  p.nctr = L.nctr;
  p.rowmap = reinterpret_cast<int32_t*>(ws + L.rowmap);
  p.inv = reinterpret_cast<int32_t*>(ws + L.inv);
  p.tgt = reinterpret_cast<int32_t*>(ws + L.tgt);
  p.flags = reinterpret_cast<uint32_t*>(ws);
  p.reduction = s.reduction;
  return launch_after(s.dtype == MOE_F32 ? ce_prep_kernel<float> : ce_prep_kernel<bf16>, (unsigned)blocks,
                      kPackTile, 0, st, 1, p);
}

// W's columns (vocabulary rows) v0 .. of this piece as a tensor-core operand:
// the caller's rows, or the piece's planes in the workspace.
struct Operand {
  const void* p;
  int64_t ld, plane, rows, v0;
};
cudaError_t piece_operand(const CeShape& s, const CeLayout& L, char* ws, const void* w, int64_t v0,
                          int64_t vcols, Operand* o, cudaStream_t st) {
  if (s.planes == 1) {
    *o = {w, s.w_ld, 0, s.V, v0};
    return cudaSuccess;
  }
  const int64_t have = std::min<int64_t>(vcols, s.V - v0);
  *o = {ws + L.wpl, s.H, L.piece, vcols, 0};
  return launch_planes(reinterpret_cast<const float*>(w) + v0 * s.w_ld, s.w_ld, have, vcols, s.H,
                       ws + L.wpl, L.piece, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

#define DECODE_CE(shape, s)                                  \
  CeShape s;                                                 \
  do {                                                       \
    const char* why_ = "";                                   \
    moe_status st_ = decode_ce(shape, &s, &why_);            \
    if (st_ != MOE_OK) return ::moe::fail(st_, why_);        \
  } while (0)

extern "C" size_t moe_linear_ce_workspace_bytes(const moe_ce_shape* shape) {
  CeShape s;
  const char* why;
  if (decode_ce(shape, &s, &why) != MOE_OK) return 0;
  return layout_ce(s).total;
}

extern "C" moe_status moe_linear_ce_forward(const moe_ce_shape* shape, const void* x, const void* w,
                                            const int32_t* target, float* loss, float* lse, float* stats,
                                            float* total, void* ws, size_t ws_bytes, void* stream) {
  reset_launch_count();
  DECODE_CE(shape, s);
  if (!w || (s.T > 0 && (!x || !target))) return fail(MOE_ERR_INVALID_ARG, "x, w and target must be non-NULL");
  if (!loss && !lse && !stats && !total)
    return fail(MOE_ERR_INVALID_ARG, "one of loss, lse, stats and total must be non-NULL");
  if (!aligned16(stats)) return fail(MOE_ERR_INVALID_ARG, "stats must be 16-byte aligned");
  if (s.reduction == MOE_CE_NONE && total)
    return fail(MOE_ERR_INVALID_ARG, "total must be NULL with MOE_CE_NONE");
  if (!aligned16(x) || !aligned16(w)) return fail(MOE_ERR_INVALID_ARG, "x and w must be 16-byte aligned");
  const CeLayout L = layout_ce(s);
  moe_status e = check_ws(ws, ws_bytes, L.total);
  if (e != MOE_OK) return e;
  char* b = static_cast<char*>(ws);
  cudaStream_t st = (cudaStream_t)stream;
  if (skinny_ok(s)) {
    SkinnyArgs k = {};
    k.x = x;
    k.w = w;
    k.x_ld = s.x_ld;
    k.w_ld = s.w_ld;
    k.target = target;
    k.T = (int)s.T;
    k.H = s.H;
    k.V = s.V;
    k.ignore = s.ignore;
    k.reduction = s.reduction;
    k.loss = loss;
    k.lse = lse;
    k.rowstat = reinterpret_cast<float4*>(stats);
    k.total = total;
    k.part = reinterpret_cast<float2*>(b + L.skinny);
    k.zt = reinterpret_cast<float*>(b + L.zt);
    k.flags = reinterpret_cast<uint32_t*>(b);
    k.ticket = reinterpret_cast<int32_t*>(b) + 8;
    CHECK_CUDA(launch_skinny(s, k, st));
    return MOE_OK;
  }
  PrepArgs p = {};
  p.target = target;
  p.x = x;
  p.loss = loss;
  p.lse_out = lse;
  p.stats_out = reinterpret_cast<float4*>(stats);
  CHECK_CUDA(run_prep(s, L, b, p, st));
  const int64_t vpad = ((int64_t)s.V + 255) / 256 * 256;
  // bf16 W is read where it is: one launch over the whole vocabulary
  const int64_t step = s.planes == 1 ? vpad : L.piece;
  int64_t c = 0;
  for (int64_t v0 = 0; v0 < vpad && s.T > 0; v0 += step, ++c) {
    const int64_t vcols = std::min(step, vpad - v0);
    Operand o;
    CHECK_CUDA(piece_operand(s, L, b, w, v0, vcols, &o, st));
    LogitsArgs a = {};
    a.planes = s.planes;
    a.x = b + L.xc;
    a.x_ld = s.H;
    a.x_plane = L.rows_pad;
    a.w = o.p;
    a.w_ld = o.ld;
    a.w_plane = o.plane;
    a.w_rows = o.rows;
    a.hidden = s.H;
    a.v0 = v0;
    a.w_v0 = o.v0;
    a.vcols = vcols;
    a.vocab = s.V;
    a.nrows = p.nrows;
    a.rows_bound = s.T;
    a.target = p.tgt;
    a.ctr = p.ctr + c;
    a.flags = p.flags;
    a.stats = reinterpret_cast<float2*>(b + L.stats);
    a.zt = reinterpret_cast<float*>(b + L.zt);
    a.rows_pad = L.rows_pad;
    CHECK_CUDA(launch_linear_logits(a, st));
  }
  int64_t blocks = std::min<int64_t>((s.T + 31) / 32, 4096);
  if (blocks < 1) blocks = 1;
  CHECK_CUDA(launch_after(ce_merge_kernel, (unsigned)blocks, 32 * kMergeWarps, 0, st, 1,
                          reinterpret_cast<const float2*>(b + L.stats), L.rows_pad, (int)(vpad / 128),
                          reinterpret_cast<const float*>(b + L.zt), p.rowmap, p.nrows, p.ticket,
                          reinterpret_cast<float*>(b + L.loss), loss, lse,
                          reinterpret_cast<float4*>(stats), total,
                          s.reduction == MOE_CE_MEAN ? 1 : 0));
  return MOE_OK;
}

extern "C" moe_status moe_linear_ce_backward(const moe_ce_shape* shape, const void* x, const void* w,
                                             const int32_t* target, const float* stats,
                                             const float* dloss, void* dx, void* dw, void* ws,
                                             size_t ws_bytes, void* stream) {
  reset_launch_count();
  DECODE_CE(shape, s);
  if (!w || (s.T > 0 && (!x || !target || !stats)))
    return fail(MOE_ERR_INVALID_ARG, "x, w, target and stats must be non-NULL");
  if (!aligned16(stats)) return fail(MOE_ERR_INVALID_ARG, "stats must be 16-byte aligned");
  if (s.reduction == MOE_CE_NONE && !dloss && s.T > 0)
    return fail(MOE_ERR_INVALID_ARG, "dloss must be non-NULL with MOE_CE_NONE");
  if (!dw && (!dx && s.T > 0)) return fail(MOE_ERR_INVALID_ARG, "one of dx and dw must be non-NULL");
  if (!aligned16(x) || !aligned16(w) || !aligned16(dx) || !aligned16(dw))
    return fail(MOE_ERR_INVALID_ARG, "x, w, dx and dw must be 16-byte aligned");
  const CeLayout L = layout_ce(s);
  moe_status e = check_ws(ws, ws_bytes, L.total);
  if (e != MOE_OK) return e;
  char* b = static_cast<char*>(ws);
  cudaStream_t st = (cudaStream_t)stream;
  PrepArgs p = {};
  p.target = target;
  p.x = x;
  p.rowstat = reinterpret_cast<const float4*>(stats);
  p.dloss = dloss;
  p.g = reinterpret_cast<float*>(b + L.g);
  p.rowstat_c = reinterpret_cast<float4*>(b + L.rowstat);
  p.dx = L.dx_direct ? dx : nullptr;
  CHECK_CUDA(run_prep(s, L, b, p, st));
  const int64_t vpad = ((int64_t)s.V + 255) / 256 * 256;
  int64_t c = 0;
  for (int64_t v0 = 0; v0 < vpad; v0 += L.piece, ++c) {
    const int64_t vcols = std::min(L.piece, vpad - v0);
    const int64_t have = std::min<int64_t>(vcols, s.V - v0);
    Operand o;
    CHECK_CUDA(piece_operand(s, L, b, w, v0, vcols, &o, st));
    if (skinny_ok(s)) {
      SkinnyGradArgs k = {};
      k.x = x;
      k.w = w;
      k.x_ld = s.x_ld;
      k.w_ld = s.w_ld;
      k.target = target;
      k.T = (int)s.T;
      k.H = s.H;
      k.V = s.V;
      k.ignore = s.ignore;
      k.planes = s.d_planes;
      k.rowstat = p.rowstat;
      k.g = p.g;
      k.v0 = v0;
      k.vcols = vcols;
      k.plane = L.rows_pad;
      k.d_ld = L.piece;
      k.d = reinterpret_cast<bf16*>(b + L.d);
      CHECK_CUDA(launch_skinny_grad(s, k, st));
    } else {
      LogitsArgs a = {};
      a.planes = s.planes;
      a.x = b + L.xc;
      a.x_ld = s.H;
      a.x_plane = L.rows_pad;
      a.w = o.p;
      a.w_ld = o.ld;
      a.w_plane = o.plane;
      a.w_rows = o.rows;
      a.hidden = s.H;
      a.v0 = v0;
      a.w_v0 = o.v0;
      a.vcols = vcols;
      a.vocab = s.V;
      a.nrows = p.nrows;
      a.rows_bound = s.T;
      a.target = p.tgt;
      a.ctr = p.ctr + 2 * c;
      a.flags = p.flags;
      a.rows_pad = L.rows_pad;
      a.gradient = true;
      a.d_planes = s.d_planes;
      a.rowstat = p.rowstat_c;
      a.g = p.g;
      a.d = b + L.d;
      a.d_ld = L.piece;
      CHECK_CUDA(launch_linear_logits(a, st));
    }
    LinearGradArgs q = {};
    q.planes = s.d_planes == 2 ? kPlanesD2 : s.planes;
    q.d = b + L.d;
    q.d_ld = L.piece;
    q.d_plane = L.rows_pad;
    q.x = b + L.xc;
    q.x_ld = s.H;
    q.x_plane = L.rows_pad;
    q.x_rows = L.rows_pad;
    q.w = o.p;
    q.w_ld = o.ld;
    q.w_plane = o.plane;
    q.w_rows = o.rows;
    q.scale = p.scale;
    q.hidden = s.H;
    q.v0 = v0;
    q.w_v0 = o.v0;
    q.vcols = vcols;
    q.vocab = s.V;
    q.nrows = p.nrows;
    q.rows_bound = s.T;
    q.ctr = p.ctr + 2 * c + 1;
    q.flags = p.flags;
    q.split = L.split;
    q.out_f32 = s.dtype == MOE_F32;
    q.rows_pad = L.rows_pad;
    q.accumulate = v0 > 0;
    if (dx && L.dx_direct) {
      q.dx = dx;
      q.rowmap = p.rowmap;
    } else if (dx) {
      q.dx_part = reinterpret_cast<float*>(b + L.dx_part);
    }
    q.dw_pad = L.piece;
    if (dw && L.dw_direct) q.dw = dw;
    else if (dw) q.dw_part = reinterpret_cast<float*>(b + L.dw_part);
    CHECK_CUDA(launch_linear_grad(q, st));
    if (q.dw_part)
      CHECK_CUDA(launch_reduce_parts(q.dw_part, L.split.dw, L.piece * s.H, have, s.H, nullptr, nullptr,
                                     static_cast<char*>(dw) + v0 * s.H * s.esize, q.out_f32, st));
  }
  if (dx && !L.dx_direct)
    CHECK_CUDA(launch_reduce_parts(reinterpret_cast<const float*>(b + L.dx_part), L.split.dx,
                                   L.rows_pad * s.H, s.T, s.H, p.inv, nullptr, dx, s.dtype == MOE_F32, st));
  return MOE_OK;
}
