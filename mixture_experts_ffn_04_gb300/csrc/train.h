// train.h -- host-side plumbing of the training operators (vocabulary cross
// entropy, router gradient): the dense tensor-core GEMMs they share and the
// small kernels around them.
#pragma once

#ifdef __CUDACC__
#include <cuda_fp16.h>
#endif
#include <cuda_runtime.h>
#include <stdint.h>

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

// fp32 operands go through the 16-bit tensor cores in planes, stacked `plane`
// rows apart in one matrix:
//  * three bf16 planes, x = x0 + x1 + x2 (8 mantissa bits each), any range, six
//    products;
//  * two fp16 planes, x s = h + l 2^-11 with one power of two s for the matrix
//    that brings its largest finite value to [2^14, 2^15): 22 mantissa bits down
//    to 2^-29 of the largest, three products.
// bf16 gradients can keep D in two bf16 planes against one of x and w (two
// products): D's rounding, half of the gradients' error, then vanishes.
constexpr int kPlanesF32 = 3, kPlanesHalf = 2, kPlanesD2 = 4;

#ifdef __CUDACC__
constexpr float kHalfLow = 2048.0f;   // scale of the low plane against the high one
// The power of two for a largest absolute value, given as its bits (a value that
// is not finite or zero: 1), and its reciprocal.
__device__ __forceinline__ float pow2_scale(uint32_t bits) {
  if (bits == 0u || bits >= 0x7F800000u) return 1.0f;
  int s = 14 - ilogbf(__uint_as_float(bits));
  s = s > 126 ? 126 : (s < -126 ? -126 : s);
  return __uint_as_float((uint32_t)(s + 127) << 23);
}
__device__ __forceinline__ float pow2_recip(float s) {
  return __uint_as_float((254u << 23) - __float_as_uint(s));
}
// What the high plane leaves for the low one (0 where it is not finite).
__device__ __forceinline__ float half_rest(float v) {
  const float r = (v - __half2float(__float2half_rn(v))) * kHalfLow;
  return isfinite(r) ? r : 0.0f;
}
__device__ __forceinline__ uint4 pack_half8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
#endif

// K or row tiles of the dense GEMMs: 256 x 256 output tiles, 64-wide k-blocks.
constexpr int kLinTile = 256, kLinK = 64;

// Work split of the gradient GEMM, the same on every device: rows is the
// caller's bound (the real count may be smaller).
struct LinearSplit {
  int dx, dw;   // K splits of a dX tile (K = vocabulary), a dW tile (K = rows)
};
LinearSplit linear_grad_split(int64_t rows, int64_t vocab, int hidden, int planes);

struct LogitsArgs {
  int planes;              // 1: bf16 operands, kPlanesHalf: fp32 in fp16 planes
  const float* scale;      // kPlanesHalf: device, the scales of x, w and d
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
  // planes [planes * rows_pad, d_ld], zeros past the rows (to the tile) and
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
  int planes;              // 1, kPlanesD2, kPlanesHalf or kPlanesF32
  const float* scale;      // kPlanesHalf: device, the scales of x, w and d
  const void* d;           // bf16 [planes * d_plane, d_ld]: d [rows, vcols]
  int64_t d_ld, d_plane;
  const void* x;           // bf16 [planes * x_plane, x_ld]; rows past the count
  int64_t x_ld, x_plane;   // up to a multiple of 64 finite (or past x_rows)
  int64_t x_rows;
  const void* w;           // bf16 [planes * w_plane, w_ld]
  int64_t w_ld, w_plane, w_rows;
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

// Rows of fp32 as bf16 planes (or bf16 rows copied): dst [planes][plane][hidden];
// rows past `rows` up to `rows_zero` are zeros.
cudaError_t launch_planes(const float* src, int64_t ld, int64_t rows, int64_t rows_zero, int hidden,
                          void* dst, int64_t plane, cudaStream_t st);

// The same as two fp16 planes; max: device, the bits of the matrix's largest
// finite absolute value.
cudaError_t launch_halves(const float* src, int64_t ld, int64_t rows, int64_t rows_zero, int hidden,
                          void* dst, int64_t plane, const uint32_t* max, cudaStream_t st);

int linear_clusters();   // clusters of two SMs the device runs at once

}  // namespace moe
