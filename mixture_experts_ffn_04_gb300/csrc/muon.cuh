// muon.cuh -- what the kernels of the orthogonalised update share: the tensors of a
// round, their elements, and the factor of a matrix.
#pragma once

#include "../../include/moe_model.h"
#include "common.cuh"
#include "orth.h"

namespace moe {
namespace muon {

constexpr int kSegs = 16;                       // tensors a launch carries in its arguments
constexpr int64_t kScratch = 3ll << 30;         // bytes of one round's matrices
constexpr int64_t kMaxRound = 16384;            // matrices of a round
constexpr int kPart = 8192;                     // elements of a partial sum of squares
constexpr int kTile = 64;

// Matrices of one tensor that take part in a round: `count` from its matrix
// `first`, the round's matrices `at` and on.
struct Seg {
  void* param;        // also the output of the matrices alone
  const void* grad;
  float* momentum;    // NULL: u is grad itself
  int64_t first;
  int32_t at, count;
  int32_t rows, cols, pdtype, gdtype;
  float size;         // lr * size of the update
};

struct Round {
  Seg seg[kSegs];
  int32_t segs, batch;
  int32_t m, n, ldx, parts;   // of a matrix: sides, row length in scratch, partial sums
  float beta, rest, keep;     // momentum, 1 - momentum; 1 - lr * weight_decay
  int32_t nesterov, update;   // update: param = keep param - size X, else out = X
  double eps;
  double* sums;               // [batch][parts]
  int32_t planes;             // of X: two of fp16, or one and 8-bit parts (orth.h)
  __half* x;                  // [planes][batch][m][ldx], the 8-bit parts behind
};

__device__ __forceinline__ const Seg& seg_of(const Round& r, int b) {
  int s = 0;
  while (s + 1 < r.segs && r.seg[s + 1].at <= b) ++s;
  return r.seg[s];
}

// 8 consecutive elements of a row or of the whole matrix, as floats; `n` of them
// exist.  vec: 16-byte aligned and all there.
__device__ __forceinline__ void read8(const void* p, int dtype, int64_t at, int n, bool vec, float* f) {
  if (dtype == MOE_F32) {
    const float* q = static_cast<const float*>(p) + at;
    if (vec) {
      unpack16(reinterpret_cast<const uint4*>(q)[0], f, (const float*)nullptr);
      unpack16(reinterpret_cast<const uint4*>(q)[1], f + 4, (const float*)nullptr);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = e < n ? q[e] : 0.0f;
    }
  } else {
    const bf16* q = static_cast<const bf16*>(p) + at;
    if (vec) {
      unpack16(reinterpret_cast<const uint4*>(q)[0], f, (const bf16*)nullptr);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = e < n ? __bfloat162float(q[e]) : 0.0f;
    }
  }
}
// 8 whole elements on a 16-byte boundary as memory has them, and as floats: several reads go
// out before the first value is looked at.
struct Raw8 {
  uint4 v[2];
};
__device__ __forceinline__ Raw8 load_raw(const void* p, int dtype, int64_t at, bool there) {
  Raw8 r;
  r.v[0] = r.v[1] = make_uint4(0, 0, 0, 0);
  if (there) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (dtype == MOE_F32 ? 4 : 2));
    r.v[0] = q[0];
    if (dtype == MOE_F32) r.v[1] = q[1];
  }
  return r;
}
__device__ __forceinline__ void open_raw(const Raw8& r, int dtype, float* f) {
  if (dtype == MOE_F32) {
    unpack16(r.v[0], f, (const float*)nullptr);
    unpack16(r.v[1], f + 4, (const float*)nullptr);
  } else {
    unpack16(r.v[0], f, (const bf16*)nullptr);
  }
}
__device__ __forceinline__ void write8(void* p, int dtype, int64_t at, int n, bool vec, const float* f) {
  if (dtype == MOE_F32) {
    float* q = static_cast<float*>(p) + at;
    if (vec) {
      reinterpret_cast<uint4*>(q)[0] = pack16(f, (const float*)nullptr);
      reinterpret_cast<uint4*>(q)[1] = pack16(f + 4, (const float*)nullptr);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) q[e] = f[e];
    }
  } else {
    bf16* q = static_cast<bf16*>(p) + at;
    if (vec) {
      *reinterpret_cast<uint4*>(q) = pack16(f, (const bf16*)nullptr);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) q[e] = __float2bfloat16_rn(f[e]);
    }
  }
}
__device__ __forceinline__ bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The direction's element from a gradient's and the new momentum's.
__device__ __forceinline__ float direction(const Round& r, float g, float v) {
  return r.nesterov ? fmaf(r.beta, v, r.rest * g) : v;
}

// Two factors whose product is 2^kOrthX / (norm + eps): one would leave fp32 for
// norms far from 1.  The square root and the quotient in fp32 (a common factor of the matrix,
// within 2^-23), the range in the exponents: fp64 roots and divisions take thousands of clocks
// here.
__device__ __forceinline__ float2 scale_of(double sum, double eps) {
  if (!isfinite(sum)) return make_float2(__int_as_float(0x7fc00000), 1.0f);
  if (sum == 0.0) return make_float2(0.0f, 0.0f);
  int e;
  double m = frexp(sum, &e);                   // sum = m 2^e, made even
  if (e & 1) {
    m *= 0.5;
    ++e;
  }
  int q;
  const double f = frexp(ldexp((double)sqrtf((float)m), e / 2) + eps, &q);      // norm + eps = f 2^q
  const int h = -q / 2;
  return make_float2(ldexpf(1.0f, h), ldexpf(1.0f / (float)f, kOrthX - q - h));
}

}  // namespace muon

// Matrices small enough for a cluster to hold (muon_small.cu): whether, and the update of a
// round's.
bool muon_small_fits(int m, int n, int planes);
cudaError_t launch_muon_small(const muon::Round& r, int planes, int steps, const double (*coef)[3], uint32_t* flags,
                              cudaStream_t st);

}  // namespace moe
