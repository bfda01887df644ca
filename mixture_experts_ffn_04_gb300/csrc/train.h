// train.h -- host-side plumbing of the training operators (vocabulary cross
// entropy, router gradient): the dense tensor-core GEMMs they share and the
// small kernels around them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#ifdef __CUDACC__
#include "common.cuh"
#endif
#include "internal.h"

namespace moe {

// Programmatic dependent launch: a kernel launched with launch_after may be
// scheduled while the one before it in the stream still runs; pdl_wait returns
// when that one has completed and its writes are visible, so nothing before it
// touches memory.  Every block waits, also those without work: a kernel then
// never completes before the one it was launched after.  pdl_trigger lets the
// next kernel be scheduled.
#ifdef __CUDACC__
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t st,
                         unsigned cluster, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}
#endif

// fp32 operands go through the bf16 tensor cores as three bf16 planes, x = x0 + x1 +
// x2 exactly (8 mantissa bits each, the range of fp32), stacked `plane` rows apart in
// one matrix; a product takes the six plane products above 2^-24.  Not two fp16 planes
// under a scale for the matrix, which need half the products: values 2^-50 below the
// matrix's largest vanish in them, which a masked row of 1e15, a rare column's
// gradient or a large feature that meets zeros does to all the rest, whatever the
// scale is taken over.
// bf16 gradients can keep D in two bf16 planes against one of x and w (two
// products): D's rounding, half of the gradients' error, then vanishes.
constexpr int kPlanesF32 = 3, kPlanesD2 = 4;

#ifdef __CUDACC__
// The next plane of v, which keeps the rest (none where the plane is not finite).  A
// finite value that would round to infinity takes the largest bf16 value instead:
// infinity times a zero on the other side would be NaN.
__device__ __forceinline__ float take_plane(float& v) {
  float p = __bfloat162float(__float2bfloat16_rn(v));
  if (fabsf(p) == INFINITY && fabsf(v) != INFINITY) p = copysignf(__uint_as_float(0x7F7F0000u), v);
  const float r = v - p;
  v = isfinite(r) ? r : 0.0f;
  return p;
}
#endif

// K or row tiles of the dense GEMMs: 256 x 256 output tiles, 64-wide k-blocks.
constexpr int kLinTile = 256, kLinK = 64;

// Work split of the gradient GEMM, the same on every device: rows is the
// caller's bound (the real count may be smaller).
struct LinearSplit {
  int dx, dw;   // K splits of a dX tile (K = vocabulary), a dW tile (K = rows)
};
LinearSplit linear_grad_split(int64_t rows, int64_t vocab, int hidden);

struct LogitsArgs {
  int planes;              // 1: bf16 operands, kPlanesF32: fp32 in planes
  int d_planes;            // of d: 1 or 2, or kPlanesF32
  const void* x;           // bf16 [planes * x_plane, x_ld], rows of `hidden`
  int64_t x_ld, x_plane;
  const void* w;           // bf16 [planes * w_plane, w_ld]
  int64_t w_ld, w_plane, w_rows;   // w_rows: rows of one plane that exist
  int hidden;
  int64_t v0;              // first vocabulary column of this call; row of w it
  int64_t w_v0;            // starts at
  int64_t vcols;           // columns computed (the last ones may pass `vocab`)
  int64_t vocab;
  const int32_t* nrows;    // device: rows that count
  int64_t rows_bound;
  const int32_t* target;   // [rows] compacted targets
  int32_t* ctr;            // zeroed tile counter
  uint32_t* flags;
  // statistics (gradient == false): (max, sum of e^(z - max)) of each row over each
  // 128-wide half tile without its target, at stats[(2 * tile + half) * rows_pad +
  // row], and the target's logit
  float2* stats;
  float* zt;
  int64_t rows_pad;
  // gradient (gradient == true): d = g e^(z - M) / S, at the target -g R / S, in bf16
  // planes [d_planes * rows_pad, d_ld], zeros past the rows (to the tile) and
  // past the vocabulary
  bool gradient;
  const float4* rowstat;   // (M, S, R, -) of the compacted rows
  const float* g;
  void* d;
  int64_t d_ld;
};
cudaError_t launch_linear_logits(const LogitsArgs& a, cudaStream_t st);

// z = x W^T of bf16 operands in fp32, K in `split` parts: part[s][rows_pad][ld] (ld a
// multiple of 64), to be added in order.
struct ProductArgs {
  const void* x;           // bf16 [rows, x_ld]
  int64_t x_ld, rows;
  const void* w;           // bf16 [cols, w_ld]
  int64_t w_ld, cols;
  int hidden, split;
  int32_t* ctr;            // zeroed tile counter
  uint32_t* flags;
  float* part;
  int64_t rows_pad, ld;
};
int linear_product_split(int64_t rows, int64_t cols, int hidden);
cudaError_t launch_linear_product(const ProductArgs& a, cudaStream_t st);

struct LinearGradArgs {
  int planes;              // 1, kPlanesD2 or kPlanesF32
  const void* d;           // bf16 [planes * d_plane, d_ld]: d [rows, vcols]
  int64_t d_ld, d_plane;
  const void* x;           // bf16 [planes * x_plane, x_ld]; rows past the count
  int64_t x_ld, x_plane;   // up to a multiple of 64 finite (or past x_rows)
  int64_t x_rows;
  const void* w;           // bf16 [planes * w_plane, w_ld]
  int64_t w_ld, w_plane, w_rows;
  const float* scale;      // device: factor of dx and dw, or NULL (not with dx_add)
  int hidden;
  int64_t v0, w_v0, vcols, vocab;
  const int32_t* nrows;    // device count, or NULL: rows_bound
  int64_t rows_bound;
  int32_t* ctr;
  uint32_t* flags;
  LinearSplit split;
  int out_f32;             // type of dx and dw
  // dx: fp32 partial sums [split.dx][rows_pad][hidden] (added to when
  // accumulate), or straight to dx rows (row r to rowmap[r]; dx_add added)
  float* dx_part;
  int64_t rows_pad;
  int accumulate;
  void* dx;
  const int32_t* rowmap;
  const void* dx_add;
  // dw rows v0 .. of [vocab, hidden], or fp32 partials
  // [split.dw][dw_pad][hidden] of this call's columns
  void* dw;
  float* dw_part;
  int64_t dw_pad;
};
cudaError_t launch_linear_grad(const LinearGradArgs& a, cudaStream_t st);

// out[r] = sum of the splits' partial rows (+ add[r]), rounded once; row r of
// the partials is inv[r] (inv == NULL: r), a negative inv gives a zero row.
cudaError_t launch_reduce_parts(const float* part, int splits, int64_t part_stride, int64_t rows,
                                int hidden, const int32_t* inv, const void* add, void* out,
                                int out_f32, cudaStream_t st);

// Rows of fp32 as three bf16 planes: dst [3][plane][hidden]; rows past `rows` up to
// `rows_zero` are zeros.
cudaError_t launch_planes(const float* src, int64_t ld, int64_t rows, int64_t rows_zero, int hidden,
                          void* dst, int64_t plane, cudaStream_t st);

}  // namespace moe
