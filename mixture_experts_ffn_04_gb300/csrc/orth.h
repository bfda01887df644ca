// orth.h -- host-side plumbing of the orthogonalised update: the three products
// of one Newton-Schulz step over a batch of matrices (orth_tc.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// A matrix is held as one or two fp16 planes of its values times a power of two:
// the leading 11 bits, and the next 11.  X [m, n] with m <= n, its singular values at
// most 3.5; A = X X^T; B = b A + c A A, at most 100.
constexpr int kOrthX = 13, kOrthA = 11, kOrthB = 9;
constexpr double kOrthMaxX = 3.5, kOrthMaxB = 100.0;

// A batch in scratch.  x[0], x[1]: two planes each, [2][batch][m][ldx]; a, b: `planes`
// planes, [planes][batch][m][lda]; rows start on 16-byte boundaries.
struct OrthBatch {
  int64_t batch;
  int m, n, ldx, lda;
  int planes;        // of the products' operands: 1, or 2 for fp32 matrices
  void* x[2];
  void* a;
  void* b;
  uint32_t* flags;
};

// `steps` times X <- a X + (b A + c A A) X with (a, b, c) = coef[i], from x[0]; the
// last X is in x[steps & 1].
cudaError_t launch_orth_steps(const OrthBatch& t, int steps, const double (*coef)[3], cudaStream_t st);

}  // namespace moe
