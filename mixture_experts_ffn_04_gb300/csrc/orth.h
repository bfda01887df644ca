// orth.h -- host-side plumbing of the orthogonalised update: the three products
// of one Newton-Schulz step over a batch of matrices (orth_tc.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// A matrix is held as fp16 planes of its values times a power of two: the leading 11
// bits, and the next 11; X of bf16 matrices as one plane and an 8-bit part, the next 8 bits.
// X [m, n] with m <= n, its singular values at most 3.5; A = X X^T; B = b A + c A A, at most
// 100; R of two steps in one (below), at most 200.
constexpr int kOrthX = 13, kOrthA = 11, kOrthB = 9, kOrthR = 8;
constexpr double kOrthMaxX = 3.5, kOrthMaxB = 100.0, kOrthMaxR = 200.0;

// A batch in scratch.  x[0], x[1]: [planes][batch][m][ldx] each, with one plane the 8-bit
// parts [batch][m][ldx] behind it; a, b, c: [planes][batch][m][lda]; ldx a multiple of 128, lda of
// 64 (columns past m and n, up to there, are written, and read only into themselves).
// c: NULL, or (one plane) the first two steps go in one where steps follow them.  parts: of
// orth_parts_bytes.
struct OrthBatch {
  int64_t batch;
  int m, n, ldx, lda;
  int planes;        // of the products' operands: 1, or 2 for fp32 matrices
  void* x[2];
  void* a;
  void* b;
  void* c;
  float* parts;
  uint32_t* flags;
};

#ifdef __CUDACC__
// The 8-bit part of f whose leading fp16 plane is h (as fp32): how far f's bit pattern
// is from h's, in steps of 32 of at most 4096 either way (half of h's last bit), so h
// and the part hold 19 bits.  Integer steps at full rate: with a part in units of h's
// last bit, through float-integer conversions at a quarter of it, the epilogue took longer
// than the products.  Below fp16's normal range the part stops at its limit, closer to f
// than h alone.
__device__ __forceinline__ int orth_low_steps(float f, float h) {
  return (__float_as_int(f) - __float_as_int(h) + 16) >> 5;
}
// Four parts, each at its limit where it passes 8 bits, in one word, the first lowest.
__device__ __forceinline__ uint32_t orth_low_pack(int a, int b, int c, int d) {
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\t"
      "cvt.pack.sat.s8.s32.b32 t, %4, %3, 0;\n\t"
      "cvt.pack.sat.s8.s32.b32 %0, %2, %1, t;\n\t}\n"
      : "=r"(r)
      : "r"(a), "r"(b), "r"(c), "r"(d));
  return r;
}
// h and its part, byte `at` of `low`: one dot product of four bytes with 32 at that byte.
__device__ __forceinline__ float orth_with_low(float h, uint32_t low, int at) {
  return __int_as_float(__dp4a((int)low, 32 << (8 * at), __float_as_int(h)));
}
#endif

// Pieces that the sums of A = X X^T are cut into along n, where the tiles of `batch` matrices
// leave most of the GPU without one (1: whole); bytes of their partial sums for any batch of
// at most `most` (0: whole).
int orth_split(int64_t batch, int m, int n, int planes);
size_t orth_parts_bytes(int64_t most, int m, int n, int planes);

// `steps` times X <- a X + (b A + c A A) X with (a, b, c) = coef[i], from x[0]; the
// last X is in x[*last], of bf16 matrices without 8-bit parts.
cudaError_t launch_orth_steps(const OrthBatch& t, int steps, const double (*coef)[3], int* last, cudaStream_t st);

}  // namespace moe
