// router_bwd.cu -- gradient of the top-k softmax router with its load-balance
// and z losses (include/moe_train.h).
//
// The logits are computed again (2 T H E flops, against the 4 T H E of the two
// gradient products): bf16 on the pairs of SMs, summed in chunks of K (the
// truncation of one long tensor-core sum shows in the z loss), fp32 by the
// forward's router GEMM.  One warp a token then turns them into the gradient of
// the logits:
//   dz_te = [norm]  sum_s [idx_s = e] w_s (D_s - dot)        w: softmax over the k
//           [full]  sum_s [idx_s = e] w_s D_s - p_te dot     w_s = p at idx_s
//           + p_te (cb (n_e - sum_j n_j p_tj) + 2 c_z / T lse_t)
// with dot = sum_s w_s D_s, D = d_topk_w, cb = balance_coef E / (T^2 k), and the
// gate column d_gate s (1 - s).  All of it in fp32.  dz goes into the gradient
// products dx = dz W_r (+ dx_add) and dW_r = dz^T x, one launch on the tensor
// cores, as two bf16 planes (fp32 layers: three): one plane would add its rounding
// to that of the results (dW_r 2.5e-3 off instead of 1.7e-3), and the MMAs are not
// what bounds them.
// What bounds it: HBM, x once for each product, dx_add and dx once; at few tokens
// the launches.  T = 8192, H = 7168, E = 256: 173 us, of which the gradient launch
// takes 103 (360 MB in and out, half of HBM's rate), the logits 31, dz 20, the
// histogram 8, the reduction of dW_r's parts 6.
#include <algorithm>
#include <cmath>

#include <cooperative_groups.h>

#include "../../include/moe_train.h"
#include "common.cuh"
#include "internal.h"
#include "train.h"

namespace moe {
namespace {

struct DzArgs {
  const float* logits;
  int64_t split_stride;
  int nsplit, ldl;
  int64_t T;
  int E, k, ncols, norm, gate;
  const int32_t* idx;
  const float* d_w;
  const float* d_gate;
  const int32_t* counts;
  int32_t *zctr, *gctr;  // tile counters of the logits and of the gradient launch
  uint32_t* flags;     // few slots (counts == NULL with `count`): each block counts
  int count;           // the slots itself, and flags the routes out of range
  float cb, cz2;       // balance_coef E / (T^2 k), 2 z_coef / T
  int planes;          // of dz
  bf16* dz;            // [planes][plane][ld]
  int64_t plane;
  int ld;
  int64_t rows;        // T rounded up to 64: the rest is zeroed
  double* part;        // [grid][2]
  int32_t* ticket;
  float* aux;
  double balance, zmean;   // scales of the sums of pn and lse^2
};

// Slots routed to each expert (integers: the order does not matter), by one
// cluster: each block counts its part in shared memory, then adds up its share of
// the experts over the blocks.  Nothing has to be zero before.  One block takes
// 18 us for 32768 slots (shared-memory atomics), eight 5.  meta: the ticket and
// the two tile counters, zeroed here too (after a call that ended early).
constexpr int kHistCluster = 8, kHistOneBlock = 4096, kFewSlots = 1024;
__global__ void __launch_bounds__(1024) route_hist_kernel(const int32_t* __restrict__ idx, int64_t n,
                                                          int E, int32_t* counts, int32_t* meta,
                                                          uint32_t* flags) {
  extern __shared__ int32_t s_h[];
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x < 3) meta[threadIdx.x] = 0;
  for (int e = threadIdx.x; e < E; e += blockDim.x) s_h[e] = 0;
  __syncthreads();
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int e = idx[i];
    if (e >= 0 && e < E) atomicAdd(&s_h[e], 1);
    else set_flag(flags, kFlagRoute);
  }
  if (gridDim.x == 1) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) counts[e] = s_h[e];
    return;
  }
  cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
  cl.sync();
  for (int e = blockIdx.x * blockDim.x + threadIdx.x; e < E; e += gridDim.x * blockDim.x) {
    int c = 0;
    for (int r = 0; r < kHistCluster; ++r) c += *cl.map_shared_rank(s_h + e, r);
    counts[e] = c;
  }
  cl.sync();   // the blocks' shared memory stays until all have read it
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// e^v by the hardware's 2^x: a few ulp for the arguments near 0 that carry the
// weight, |v| 2^-24 more for the others.
__device__ __forceinline__ float exp_of(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.4426950408889634f));
  return r;
}

// Every dz kernel zeroes the tile counters of the gradient launch that follows it and
// of the logits' launch, which is done: a call of few slots, of whatever shape, finds
// zeros in them without a launch of its own for that.
__device__ __forceinline__ void reset_counters(const DzArgs& a) {
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *a.gctr = 0;
    if (a.zctr) *a.zctr = 0;
  }
}

// The losses: block sums in fp64, the last block adds the blocks in order.
__device__ void finish_aux(const DzArgs& a, double sum_pn, double sum_l2) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  __shared__ double s_d[8][2];
  __shared__ int s_last;
  if (lane == 0) {
    s_d[warp][0] = sum_pn;
    s_d[warp][1] = sum_l2;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double x = 0.0, y = 0.0;
    for (int w = 0; w < warps; ++w) {
      x += s_d[w][0];
      y += s_d[w][1];
    }
    a.part[2 * blockIdx.x] = x;
    a.part[2 * blockIdx.x + 1] = y;
    __threadfence();
    s_last = atomicAdd(a.ticket, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last || warp != 0) return;
  __threadfence();
  double x = 0.0, y = 0.0;
  for (int i = lane; i < (int)gridDim.x; i += 32) {
    x += __ldcg(a.part + 2 * i);
    y += __ldcg(a.part + 2 * i + 1);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, o);
    y += __shfl_xor_sync(0xffffffffu, y, o);
  }
  if (lane == 0) {
    a.aux[0] = (float)(x * a.balance);
    a.aux[1] = (float)(y * a.zmean);
    *a.ticket = 0;
  }
}

// A warp a token, up to 64 * NP router columns and 32 slots: the token's logits
// in registers (columns 64 j + 2 lane, + 1), its slots one a lane, loaded with
// the logits; only the gather at the slots' experts and the scatter of their
// terms go through shared memory.  Bound by latency: 20 us at 8192 x 256, 9 at 64
// tokens; the kernel for any shape takes 15 and 5 us longer.
template <int NP>
__global__ void __launch_bounds__(256) router_dz_small_kernel(const DzArgs a) {
  extern __shared__ float s_f[];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  float* row = s_f + (size_t)warp * 64 * NP;
  reset_counters(a);
  float cnt[2 * NP];
#pragma unroll
  for (int j = 0; j < 2 * NP; ++j) cnt[j] = 0.0f;
  if (a.count) {
    int* h = reinterpret_cast<int*>(s_f);   // (before the rows need the space)
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) h[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < (int)a.T * a.k; i += blockDim.x) {
      const int e = a.idx[i];
      if (e >= 0 && e < a.E) atomicAdd(&h[e], 1);   // integers: the order does not matter
      else if (blockIdx.x == 0) set_flag(a.flags, kFlagRoute);
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 2 * NP; ++j) {
    const int e = 64 * (j / 2) + 2 * lane + (j & 1);
    if (e < a.E) cnt[j] = a.count ? (float)reinterpret_cast<const int*>(s_f)[e] : a.counts ? (float)a.counts[e] : 0.0f;
  }
  if (a.count) __syncthreads();
  // (fp64 arithmetic is slow on this GPU: a few tokens' terms first add up in fp32)
  double sum_pn = 0.0, sum_l2 = 0.0;
  float few_pn = 0.0f, few_l2 = 0.0f;
  int few = 0;
  for (int64_t t = blockIdx.x * (int64_t)warps + warp; t < a.rows; t += (int64_t)gridDim.x * warps) {
    if (t >= a.T) {   // rows the weight gradient's last k-block reads
      for (int p = 0; p < a.planes; ++p)
        for (int e = lane; e < a.ld; e += 32) a.dz[(p * a.plane + t) * a.ld + e] = __float2bfloat16_rn(0.0f);
      continue;
    }
    int slot = -1;
    float D = 0.0f;
    if (a.d_w && lane < a.k) {
      slot = a.idx[t * a.k + lane];
      D = a.d_w[t * a.k + lane];
    }
    if (slot < 0 || slot >= a.E) {   // dropped: whatever d_w holds there
      slot = -1;
      D = 0.0f;
    }
    const float dg = a.gate ? a.d_gate[t] : 0.0f;
    float z[2 * NP];
#pragma unroll
    for (int j = 0; j < 2 * NP; ++j) z[j] = 0.0f;
#pragma unroll 4
    for (int s = 0; s < a.nsplit; ++s) {
      const float* l = a.logits + s * a.split_stride + t * a.ldl + 2 * lane;
#pragma unroll
      for (int j = 0; j < NP; ++j)
        if (64 * j + 2 * lane < a.ncols) {
          const float2 v = *reinterpret_cast<const float2*>(l + 64 * j);   // ldl is a multiple of 4
          z[2 * j] += v.x;
          z[2 * j + 1] += v.y;
        }
    }
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < 2 * NP; ++j) {
      const int e = 64 * (j / 2) + 2 * lane + (j & 1);
      if (e < a.E) m = fmaxf(m, z[j]);
      row[e] = z[j];
    }
    __syncwarp();
    m = warp_max(m);
    float p[2 * NP], sum = 0.0f, pn = 0.0f;
#pragma unroll
    for (int j = 0; j < 2 * NP; ++j) {
      const int e = 64 * (j / 2) + 2 * lane + (j & 1);
      p[j] = e < a.E ? exp_of(z[j] - m) : 0.0f;
      sum += p[j];
      pn = fmaf(p[j], cnt[j], pn);
    }
    sum = warp_sum(sum);
    pn = warp_sum(pn) / sum;
    const float inv = 1.0f / sum, lse = m + logf(sum);
    few_pn += pn;
    few_l2 = fmaf(lse, lse, few_l2);
    if (++few == 8) {
      sum_pn += (double)few_pn;
      sum_l2 += (double)few_l2;
      few_pn = few_l2 = 0.0f;
      few = 0;
    }
    const float zs = slot >= 0 ? row[slot] : -INFINITY;
    __syncwarp();
    float w, dot = 0.0f, add = 0.0f;
    if (a.d_w) {
      float top = m, den = sum;
      if (a.norm) {
        top = warp_max(zs);
        den = warp_sum(slot >= 0 ? exp_of(zs - top) : 0.0f);
      }
      w = slot >= 0 ? exp_of(zs - top) / den : 0.0f;
      dot = warp_sum(w * D);
      add = a.norm ? w * (D - dot) : w * D;
      if (slot < 0) add = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) *reinterpret_cast<float2*>(row + 64 * j + 2 * lane) = make_float2(0.0f, 0.0f);
    __syncwarp();
    if (a.d_w) {
      // repeated routes add up in slot order
      const uint32_t same = __match_any_sync(0xffffffffu, slot);
      const bool dup = slot >= 0 && __popc(same) > 1;
      if (slot >= 0 && !dup) row[slot] = add;
      uint32_t left = __ballot_sync(0xffffffffu, dup);
      while (left) {
        const int s = __ffs(left) - 1;
        left &= left - 1;
        if (lane == s) row[slot] += add;
        __syncwarp();
      }
      __syncwarp();
    }
    const float base = (a.norm ? 0.0f : -dot) + a.cz2 * lse - a.cb * pn;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int e = 64 * j + 2 * lane;
      if (e >= a.ld) continue;
      const float2 c = *reinterpret_cast<const float2*>(row + e);
      float v[2] = {c.x, c.y};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (e + h < a.E) {
          v[h] += p[2 * j + h] * inv * (base + a.cb * cnt[2 * j + h]);
        } else if (e + h < a.ncols) {
          const float s = 1.0f / (1.0f + exp_of(-z[2 * j + h]));
          v[h] = dg * s * (1.0f - s);
        } else {
          v[h] = 0.0f;
        }
      }
      for (int pl = 0; pl < a.planes; ++pl) {
        *reinterpret_cast<uint32_t*>(a.dz + (pl * a.plane + t) * a.ld + e) = pack_bf16x2(v[0], v[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v[h] -= __bfloat162float(__float2bfloat16_rn(v[h]));
          if (!isfinite(v[h])) v[h] = 0.0f;
        }
      }
    }
    __syncwarp();
  }
  if (a.aux) finish_aux(a, sum_pn + (double)few_pn, sum_l2 + (double)few_l2);
}

// Any number of columns and slots: a warp a token; z and the slots'
// contributions of its token in shared memory (2 ncols floats a warp).
__global__ void __launch_bounds__(256) router_dz_kernel(const DzArgs a) {
  extern __shared__ float s_f[];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  reset_counters(a);
  float* z = s_f + (size_t)warp * 2 * a.ncols;
  float* acc = z + a.ncols;
  double sum_pn = 0.0, sum_l2 = 0.0;
  for (int64_t t = blockIdx.x * (int64_t)warps + warp; t < a.rows; t += (int64_t)gridDim.x * warps) {
    if (t >= a.T) {   // rows the weight gradient's last k-block reads
      for (int p = 0; p < a.planes; ++p)
        for (int e = lane; e < a.ld; e += 32) a.dz[(p * a.plane + t) * a.ld + e] = __float2bfloat16_rn(0.0f);
      continue;
    }
    float m = -INFINITY;
    for (int e = lane; e < a.ncols; e += 32) {
      float v = 0.0f;
      for (int s = 0; s < a.nsplit; ++s) v += a.logits[s * a.split_stride + t * a.ldl + e];
      z[e] = v;
      acc[e] = 0.0f;
      if (e < a.E) m = fmaxf(m, v);
    }
    __syncwarp();
    m = warp_max(m);
    float sum = 0.0f, pn = 0.0f;
    for (int e = lane; e < a.E; e += 32) {
      const float x = expf(z[e] - m);
      sum += x;
      if (a.counts) pn += x * (float)a.counts[e];
    }
    sum = warp_sum(sum);
    pn = warp_sum(pn) / sum;
    const float inv = 1.0f / sum, lse = m + logf(sum);
    sum_pn += (double)pn;
    sum_l2 += (double)lse * lse;
    // the slots: weights, then their contribution to the selected experts
    float dot = 0.0f;
    if (a.d_w) {
      float top = m, den = sum;
      if (a.norm) {
        top = -INFINITY;
        for (int s = lane; s < a.k; s += 32) {
          const int e = a.idx[t * a.k + s];
          if (e >= 0 && e < a.E) top = fmaxf(top, z[e]);
        }
        top = warp_max(top);
        den = 0.0f;
        for (int s = lane; s < a.k; s += 32) {
          const int e = a.idx[t * a.k + s];
          if (e >= 0 && e < a.E) den += expf(z[e] - top);
        }
        den = warp_sum(den);
      }
      const float di = den > 0.0f ? 1.0f / den : 0.0f;
      for (int s = lane; s < a.k; s += 32) {
        const int e = a.idx[t * a.k + s];
        if (e >= 0 && e < a.E) dot += expf(z[e] - top) * di * a.d_w[t * a.k + s];
      }
      dot = warp_sum(dot);
      // in slot order, so that a repeated route adds up the same every time
      for (int s = 0; s < a.k; ++s) {
        if (lane == (s & 31)) {
          const int e = a.idx[t * a.k + s];
          if (e >= 0 && e < a.E) {
            const float w = expf(z[e] - top) * di, d = a.d_w[t * a.k + s];
            acc[e] += a.norm ? w * (d - dot) : w * d;
          }
        }
        __syncwarp();
      }
    }
    const float base = (a.norm ? 0.0f : -dot) + a.cz2 * lse - a.cb * pn;
    for (int e = lane; e < a.ld; e += 32) {
      float v = 0.0f;
      if (e < a.E) {
        const float p = expf(z[e] - m) * inv;
        v = acc[e] + p * (base + (a.counts ? a.cb * (float)a.counts[e] : 0.0f));
      } else if (e < a.ncols) {
        const float s = 1.0f / (1.0f + expf(-z[e]));
        v = a.d_gate[t] * s * (1.0f - s);
      }
      for (int p = 0; p < a.planes; ++p) {
        const bf16 r = __float2bfloat16_rn(v);
        a.dz[(p * a.plane + t) * a.ld + e] = r;
        v -= __bfloat162float(r);
        if (!isfinite(v)) v = 0.0f;
      }
    }
    __syncwarp();
  }
  if (a.aux) finish_aux(a, sum_pn, sum_l2);
}

constexpr int kDzBlocks = 2048;

struct RbLayout {
  Layout L;
  int64_t rows_pad, cols_pad;
  int planes, dz_planes, zsplit;
  LinearSplit split;
  bool dx_direct, dw_direct;
  size_t counts, part, z, dz, xpl, wpl, dx_part, dw_part, total;
};
RbLayout layout_rb(const Shape& s) {
  RbLayout R;
  R.L = layout_for(s);
  R.rows_pad = std::max<int64_t>(256, (s.T + 255) / 256 * 256);
  R.cols_pad = ((int64_t)s.ncols + 63) / 64 * 64;
  R.planes = s.dtype == MOE_F32 ? kPlanesF32 : kPlanesD2;
  R.dz_planes = s.dtype == MOE_F32 ? kPlanesF32 : 2;
  R.zsplit = linear_product_split(s.T, R.cols_pad, s.H);
  R.split = linear_grad_split(s.T, R.cols_pad, s.H);
  R.dx_direct = R.split.dx == 1;
  R.dw_direct = R.split.dw == 1;
  size_t off = R.L.scratch_end;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~(size_t)255;
    return at;
  };
  R.counts = take((size_t)s.E * 4);
  R.part = take((size_t)kDzBlocks * 16);
  R.z = take(s.dtype == MOE_F32 ? 0 : (size_t)R.zsplit * R.rows_pad * R.cols_pad * 4);
  R.dz = take((size_t)R.dz_planes * R.rows_pad * R.cols_pad * 2);
  R.xpl = take(s.dtype == MOE_F32 ? (size_t)R.planes * R.rows_pad * s.H * 2 : 0);
  R.wpl = take(s.dtype == MOE_F32 ? (size_t)R.planes * R.cols_pad * s.H * 2 : 0);
  R.dx_part = take(R.dx_direct ? 0 : (size_t)R.split.dx * R.rows_pad * s.H * 4);
  const size_t dw_rows = ((size_t)s.ncols + 255) / 256 * 256;
  R.dw_part = take(R.dw_direct ? 0 : (size_t)R.split.dw * dw_rows * s.H * 4);
  R.total = off;
  return R;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_router_backward_workspace_bytes(const moe_shape* shape) {
  Shape s;
  const char* why;
  if (decode_shape(shape, &s, &why) != MOE_OK) return 0;
  return layout_rb(s).total;
}

extern "C" moe_status moe_router_backward(const moe_shape* shape, const void* x, const void* w_router,
                                          const int32_t* topk_idx, const float* d_topk_w,
                                          const float* d_gate, double balance_coef, double z_coef,
                                          const void* dx_add, void* dx, void* dw_router, float* aux,
                                          void* ws, size_t ws_bytes, void* stream) {
  reset_launch_count();
  DECODE(shape, s);
  if (!w_router || !dw_router || (s.T > 0 && (!x || !topk_idx || !dx)))
    return fail(MOE_ERR_INVALID_ARG, "x, w_router, topk_idx, dx and dw_router must be non-NULL");
  if (s.gate && !d_gate && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "shared_gate needs d_gate");
  if (!s.gate && d_gate) return fail(MOE_ERR_INVALID_ARG, "d_gate without shared_gate");
  if (!(balance_coef >= 0.0) || !(z_coef >= 0.0) || !std::isfinite(balance_coef) || !std::isfinite(z_coef))
    return fail(MOE_ERR_INVALID_ARG, "balance_coef and z_coef must be finite and >= 0");
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(dx_add) || !aligned16(dx) || !aligned16(dw_router))
    return fail(MOE_ERR_INVALID_ARG, "x, w_router, dx_add, dx and dw_router must be 16-byte aligned");
  const RbLayout R = layout_rb(s);
  moe_status e = check_ws(ws, ws_bytes, R.total);
  if (e != MOE_OK) return e;
  char* b = static_cast<char*>(ws);
  cudaStream_t st = (cudaStream_t)stream;
  if (s.T == 0) {
    CHECK_CUDA(cudaMemsetAsync(dw_router, 0, (size_t)s.ncols * s.H * s.esize, st));
    if (aux) CHECK_CUDA(cudaMemsetAsync(aux, 0, 8, st));
    return MOE_OK;
  }
  uint32_t* flags = reinterpret_cast<uint32_t*>(b);
  // ticket and tile counters, in the status word's block: zero from the workspace's
  // initialisation on; the ticket's last reader and each call's dz kernel (the
  // histogram too, for calls that have it) leave zeros for the next call, whose shape
  // may be another
  int32_t* meta = reinterpret_cast<int32_t*>(b) + 16;
  int32_t* counts = reinterpret_cast<int32_t*>(b + R.counts);
  const int64_t slots = s.T * s.k;
  // Few slots: every block of the small dz kernel counts them for itself, which
  // takes less than a launch does (T = 64, k = 4: 25 us a call, by the histogram
  // kernel 27 to 30).  The counters then have to be zero: dz zeroes them.
  const bool small = s.k <= 32 && s.ncols <= 512, few = small && slots <= kFewSlots;
  if (!few) {
    const unsigned hb = slots <= kHistOneBlock ? 1u : (unsigned)kHistCluster;
    // (the pass that finds routes out of range, so it runs in any case)
    if ((size_t)s.E * 4 > 48 * 1024)
      CHECK_CUDA(cudaFuncSetAttribute(route_hist_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, s.E * 4));
    CHECK_CUDA(launch_after(route_hist_kernel, hb, 1024, (size_t)s.E * 4, st, hb, topk_idx, slots, s.E, counts,
                            meta, flags));
  }
  DzArgs d = {};
  if (s.dtype == MOE_F32) {
    int nsplit = 1;
    e = router_gemm(s, R.L, b, x, w_router, &nsplit, st);
    if (e != MOE_OK) return e;
    d.logits = reinterpret_cast<const float*>(b + R.L.logits);
    d.split_stride = s.T * (int64_t)s.ldl;
    d.nsplit = nsplit;
    d.ldl = s.ldl;
  } else {
    ProductArgs z = {};
    z.x = x;
    z.x_ld = s.H;
    z.rows = s.T;
    z.w = w_router;
    z.w_ld = s.H;
    z.cols = s.ncols;
    z.hidden = s.H;
    z.split = R.zsplit;
    z.ctr = meta + 2;
    z.flags = flags;
    z.part = reinterpret_cast<float*>(b + R.z);
    z.rows_pad = R.rows_pad;
    z.ld = R.cols_pad;
    CHECK_CUDA(launch_linear_product(z, st));
    d.logits = z.part;
    d.split_stride = R.rows_pad * R.cols_pad;
    d.nsplit = R.zsplit;
    d.ldl = (int)R.cols_pad;
  }
  d.T = s.T;
  d.E = s.E;
  d.k = s.k;
  d.ncols = s.ncols;
  d.norm = s.norm;
  d.gate = s.gate;
  d.idx = topk_idx;
  d.d_w = d_topk_w;
  d.d_gate = d_gate;
  d.counts = balance_coef > 0.0 && !few ? counts : nullptr;
  d.count = few;
  d.flags = flags;
  d.gctr = meta + 1;
  d.zctr = s.dtype == MOE_F32 ? nullptr : meta + 2;
  const double cb = balance_coef * s.E / ((double)s.T * (double)s.T * s.k);
  d.cb = (float)cb;
  d.cz2 = (float)(2.0 * z_coef / (double)s.T);
  d.planes = R.dz_planes;
  d.dz = reinterpret_cast<bf16*>(b + R.dz);
  d.plane = R.rows_pad;
  d.ld = (int)R.cols_pad;
  d.rows = (s.T + 63) / 64 * 64;
  d.part = reinterpret_cast<double*>(b + R.part);
  d.ticket = meta;
  d.aux = aux;
  d.balance = cb;
  d.zmean = z_coef / (double)s.T;
  if (small) {
    const int np = s.ncols <= 64 ? 1 : s.ncols <= 128 ? 2 : s.ncols <= 256 ? 4 : 8;
    const int warps = 4;
    // one wave (64 to 80 registers: at least six blocks an SM)
    const unsigned blocks = (unsigned)std::min<int64_t>((d.rows + warps - 1) / warps, 6 * tc_sm_count());
    const size_t smem = (size_t)warps * 64 * np * 4;
    auto kernel = np == 1 ? router_dz_small_kernel<1> : np == 2 ? router_dz_small_kernel<2>
                : np == 4 ? router_dz_small_kernel<4> : router_dz_small_kernel<8>;
    CHECK_CUDA(launch_after(kernel, blocks, 32 * warps, smem, st, 1, d));
  } else {
    const size_t per_warp = 2 * (size_t)s.ncols * 4;
    const int warps = (int)std::max<size_t>(1, std::min<size_t>(8, 200 * 1024 / per_warp));
    if (per_warp * warps > 48 * 1024)
      CHECK_CUDA(cudaFuncSetAttribute(router_dz_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)(per_warp * warps)));
    const int64_t blocks = std::min<int64_t>((d.rows + warps - 1) / warps, kDzBlocks);
    CHECK_CUDA(launch_after(router_dz_kernel, (unsigned)blocks, 32 * warps, per_warp * warps, st, 1, d));
  }
  LinearGradArgs q = {};
  q.planes = R.planes;
  q.d = b + R.dz;
  q.d_ld = R.cols_pad;
  q.d_plane = R.rows_pad;
  q.x = x;
  q.x_ld = s.H;
  q.x_rows = s.T;
  q.w = w_router;
  q.w_ld = s.H;
  q.w_rows = s.ncols;
  if (s.dtype == MOE_F32) {
    CHECK_CUDA(launch_planes(static_cast<const float*>(x), s.H, s.T, d.rows, s.H, b + R.xpl, R.rows_pad, st));
    CHECK_CUDA(launch_planes(static_cast<const float*>(w_router), s.H, s.ncols, R.cols_pad, s.H, b + R.wpl,
                             R.cols_pad, st));
    q.x = b + R.xpl;
    q.x_plane = q.x_rows = R.rows_pad;
    q.w = b + R.wpl;
    q.w_plane = q.w_rows = R.cols_pad;
  }
  q.hidden = s.H;
  q.vcols = R.cols_pad;
  q.vocab = s.ncols;
  q.rows_bound = s.T;
  q.ctr = meta + 1;
  q.flags = flags;
  q.split = R.split;
  q.out_f32 = s.dtype == MOE_F32;
  q.rows_pad = R.rows_pad;
  if (R.dx_direct) {
    q.dx = dx;
    q.dx_add = dx_add;
  } else {
    q.dx_part = reinterpret_cast<float*>(b + R.dx_part);
  }
  q.dw_pad = ((int64_t)s.ncols + 255) / 256 * 256;
  if (R.dw_direct) q.dw = dw_router;
  else q.dw_part = reinterpret_cast<float*>(b + R.dw_part);
  CHECK_CUDA(launch_linear_grad(q, st));
  if (q.dx_part)
    CHECK_CUDA(launch_reduce_parts(q.dx_part, R.split.dx, R.rows_pad * s.H, s.T, s.H, nullptr, dx_add, dx,
                                   q.out_f32, st));
  if (q.dw_part)
    CHECK_CUDA(launch_reduce_parts(q.dw_part, R.split.dw, q.dw_pad * s.H, s.ncols, s.H, nullptr, nullptr,
                                   dw_router, q.out_f32, st));
  return MOE_OK;
}
