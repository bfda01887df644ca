// orth_tc.cu -- the products of a Newton-Schulz step over a batch of matrices, on
// pairs of SMs (tcgen05 cta_group::2, fp16 operands, fp32 sums):
//   kGram   A  = X X^T          X [m, n], m <= n, K = n
//   kPoly   B  = b A + c A A    K = m
//   kApply  X' = a X + B X      K = m, X read in its stored layout (MN-major)
// A and B are symmetric: only the tiles on and below the diagonal are computed,
// and each is written twice, the second time transposed.
//
// The first two steps of wide bf16 matrices are one: with B = b A + c A A of the first,
//   C = a A + B A,  A' = a C + B C (= X' X'^T),  B' = b' A' + c' A' A',
//   R = a B' + a' B + B' B,  X'' = a a' X + R X
// (polynomials in A commute), three products of K = m more in place of a kGram and a
// kApply, which is the slowest (2652 us against 2894 for 96 matrices 704 x 2816).
// a a' X stays apart, so that X keeps its 19 bits; simulated as below no less precise
// (normal entries 1.6e-3, rank 16 4.5e-4).  A later pair rounds R closer to the result
// (2.6e-3 with the third and fourth step in one too): not taken.
//
// Operands are the leading fp16 planes of X, A and B (11 bits); a X takes both planes
// of X, and X' is kept in both.  That matters more than the precision of the
// products: an error in X outside its row and column space grows by a in every
// step, 3.4445^5 = 484 in all, where one inside it meets the same polynomial as X
// itself.  Simulated at 512 x 1365 against 64 bits: X in one plane 3.6e-2 off for a
// matrix of rank 10 with a floor of 1e-2 (bf16 operands throughout: 0.29), in two planes
// 3.0e-4; normal entries 1.6e-3 (the polynomial in the rounded A, which b A takes from
// the same plane as A A: with b A exact instead 2.8e-3).  fp32 matrices take three
// products of two planes each, smallest first: 5.7e-7 (fp32 products: 7.2e-6), from stages with
// both planes of both operands.
//
// Few matrices with a long side (fewer tiles of A than half of the pairs of SMs) have kGram's
// sums cut into pieces along n, fp32 partial tiles that join_kernel adds in order (2 matrices 731
// x 8026 in fp32, 12 tiles: 1065 us for five steps whole, 725 in pieces).
//
// A pair of SMs computes 256 x 256 tiles (256 x 128 where there are few) over 64-wide k-blocks through six 32 KB
// stages (three of 64 KB).  Addend and result go between registers and memory as whole 128-byte rows, turned
// in a 4 KB slice of each epilogue warp between that layout and the one of TMEM (a lane a
// row), the addend asked for half a tile ahead.  By TMA boxes both stood in the TMA queue behind
// the operands of more than a tile: at m = 704, whose tiles have 11 k-blocks, 2800 of a
// tile's 14000 clocks went by waiting for the addend, 2000 issuing the result; by the
// lane that owns the row, 32 bytes at a time, each instruction took 32 lines (340 us for 96
// matrices 704 x 2816 against 312).
//
// At 704 x 2816 (96 matrices): kGram 126 us, kPoly 49 to 54 (with two addends 65), kApply 260
// with both 8-bit parts, 217 and 193 without; 2.46 ms for five steps, 0.47 of the tensor cores' measured
// rate by the formula's flops.  kGram is bound by the products (a k-block of a pair takes 650 clocks, what
// 256 x 256 x 64 takes at the peak), kApply and kPoly by their epilogues: with 11 k-blocks a tile's
// products take 7100 clocks, kApply's epilogue 9000 to 12000.
//
// Roles in each CTA: warp 0 TMA producer, warp 1 TMEM and (even CTA) the MMA
// issuer, warps 4-11 epilogue, two a 32-lane TMEM quarter.  Tiles are dealt out in a
// fixed order (all have the same K).  The sums of fp32 matrices leave TMEM in chunks of
// k-blocks, added in fp32 registers (the tensor cores cut the accumulator off at each K = 16
// step); with operands of 11 bits it would not show.  Every wait on an mbarrier is bounded,
// and a CTA that gives up waits, with a limit, for its copies and MMAs in flight.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "orth.h"
#include "tc_pair.cuh"
#include "tcgen05.cuh"
#include "train.h"

namespace moe {
namespace tc {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();   // gemm_tc.cu
}

namespace orth {

using namespace tc;

constexpr int BM = 256, BN = 256, BMC = BM / 2, BNC = BN / 2, BK = 64;
constexpr int A_BYTES = BMC * BK * 2, B_BYTES = BNC * BK * 2;   // of a plane
constexpr int BOX_BYTES = 64 * BK * 2;
constexpr int RING_BYTES = 6 * (A_BYTES + B_BYTES);              // six stages of a plane, three of two
constexpr int MAX_STAGES = 6;
constexpr int EPI_WARPS = 8;   // a warp: 32 rows, half of the columns
constexpr int THREADS = 32 * (4 + EPI_WARPS);
// 168 registers a thread at launch; 56 + 2 * 224 <= 3 * 168 (three groups of 4 warps)
constexpr int ROLE_REGS = 56, EPI_REGS = 224;
static_assert(ROLE_REGS + 2 * EPI_REGS <= 3 * 168, "register pool of the launch");
constexpr uint32_t TMEM_COLS = 512;
constexpr int BAR_BYTES = 256;
constexpr int STAGE_WARP = 4096;   // an epilogue warp's slice: 32 rows of 128 bytes
constexpr int SMEM_BYTES = 1024 + RING_BYTES + EPI_WARPS * STAGE_WARP + BAR_BYTES;
static_assert(SMEM_BYTES <= 232448, "shared memory budget of one CTA");
static_assert((2 * MAX_STAGES + 5) * 8 + 8 <= BAR_BYTES, "barrier area");
constexpr long long kDrainCycles = 1 << 21;
constexpr int kChunkExact = 3;   // k-blocks of 64, three products each

// kind::f16: D fp32, A and B fp16, M = 256 over the pair, N = n.
__host__ __device__ constexpr uint32_t idesc_of(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(BM >> 4) << 24); }
constexpr uint32_t IDESC_B_MN = 1u << 16;

enum Kind { kGram = 0, kPoly = 1, kApply = 2 };

struct Args {
  int m, n;               // of the output: m x m, or m x n
  int batch, planes;      // of matrices; of operands
  int kb;                 // k-blocks
  int mt, nt, per;        // row tiles, column tiles, tiles a matrix
  float add_scale, mul;   // result = add_scale * addend + mul * product
  const char* add;        // the addend's leading plane, rows add_ld bytes apart
  const char* add_low;    // its second plane, or its 8-bit parts
  int split;              // kGram: pieces of a tile's sum, neighbours in the tiles' order
  float* parts;           // [tiles][split][256][256] of them
  const char* add2;       // kOneTwice: the second addend
  float add2_scale;
  char* out;              // the result, the same
  char* out_low;
  int64_t add_ld, low_ld; // of the addend and the result, bytes
  uint32_t* flags;
};

struct Tile {
  int b, i, j, piece;
};
// A pair's tiles: every `step`th of all matrices' tiles, from its own.  Divisions by the
// number of tiles of a matrix are done once.
// NARROW: tiles of 128 columns, two to each whole one of kGram and kPoly.
template <int KIND, bool SPLIT = false, bool NARROW = false>
struct Walk {
  uint32_t t, l, b;             // tile; place in its matrix; matrix
  uint32_t step, step_l, step_b;
  float inv;                    // of the row tiles
  __device__ __forceinline__ Walk(const Args& a, uint32_t first, uint32_t step_) : t(first), step(step_) {
    b = first / (uint32_t)a.per;
    l = first - b * (uint32_t)a.per;
    step_b = step_ / (uint32_t)a.per;
    step_l = step_ - step_b * (uint32_t)a.per;
    inv = 1.0f / (float)a.mt;
  }
  __device__ __forceinline__ void next(const Args& a) {
    t += step;
    l += step_l;
    b += step_b;
    if (l >= (uint32_t)a.per) {
      l -= (uint32_t)a.per;
      ++b;
    }
  }
  __device__ __forceinline__ Tile tile(const Args& a) const {
    Tile r;
    r.b = (int)b;
    r.piece = 0;
    if (KIND == kApply) {
      int j = (int)((float)l * inv);      // within one of l / mt
      int i = (int)l - j * a.mt;
      if (i < 0) { --j; i += a.mt; }
      if (i >= a.mt) { ++j; i -= a.mt; }
      r.i = i;
      r.j = j;
    } else {
      uint32_t l = this->l;
      if (SPLIT) {
        const uint32_t whole = l / (uint32_t)a.split;
        r.piece = (int)(l - whole * (uint32_t)a.split);
        l = whole;
      }
      const uint32_t side = l & 1u;
      if (NARROW) l >>= 1;
      // row i of the lower triangle starts at i (i + 1) / 2
      int i = (int)((sqrtf(8.0f * (float)l + 1.0f) - 1.0f) * 0.5f);
      while ((uint32_t)i * (i + 1) / 2 > l) --i;
      while ((uint32_t)(i + 1) * (i + 2) / 2 <= l) ++i;
      r.i = i;
      r.j = (int)(l - (uint32_t)i * (i + 1) / 2);
      if (NARROW) r.j = 2 * r.j + (int)side;
    }
    return r;
  }
};

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// 32 rows of 128 bytes, ld bytes apart, as a warp moves them: lane l has 16 bytes l % 8
// of rows l / 8, + 4, .. + 28; rows from `rows` on are not there.
struct Block {
  uint4 v[8];
};
__device__ __forceinline__ void load_block(Block& b, const char* p, int64_t ld, int rows, int lane) {
  const char* at = p + (lane >> 3) * ld + (lane & 7) * 16;
  const int there = rows - (lane >> 3);
#pragma unroll
  for (int i = 0; i < 8; ++i, at += 4 * ld)
    b.v[i] = 4 * i < there ? *reinterpret_cast<const uint4*>(at) : make_uint4(0, 0, 0, 0);
}
// The block to and from a slice (put_piece's layout: piece j of row r at j ^ (r & 7)): where
// this lane's part of rows 0 .. 3 stands; of rows 4 i on it is 512 i behind, with bit 2 of the
// piece turned for odd i (a slice starts at a multiple of 128).
__device__ __forceinline__ uint32_t block_at(uint32_t stage, int lane, int i) {
  const int r = lane >> 3;
  const uint32_t at = stage + r * 128 + (((lane & 7) ^ r) << 4);
  return (i & 1 ? at ^ 64u : at) + 512 * i;
}
__device__ __forceinline__ void block_to_slice(const Block& b, uint32_t stage, int lane) {
  __syncwarp();   // what the slice held has been read
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(block_at(stage, lane, i)), "r"(b.v[i].x), "r"(b.v[i].y),
                 "r"(b.v[i].z), "r"(b.v[i].w)
                 : "memory");
  __syncwarp();
}
__device__ __forceinline__ uint4 load_piece(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ void slice_to_rows(uint32_t stage, char* p, int64_t ld, int rows, int lane) {
  __syncwarp();   // every lane's pieces are in the slice
  Block b;
#pragma unroll
  for (int i = 0; i < 8; ++i) b.v[i] = load_piece(block_at(stage, lane, i));
  char* at = p + (lane >> 3) * ld + (lane & 7) * 16;
  const int there = rows - (lane >> 3);
#pragma unroll
  for (int i = 0; i < 8; ++i, at += 4 * ld)
    if (4 * i < there) *reinterpret_cast<uint4*>(at) = b.v[i];
  __syncwarp();
}
// The same with rows of 64 bytes, half of a slice's (the 8-bit parts of 64 columns): lane l has
// 16 bytes l % 4 of rows l / 4, + 8, + 16, + 24.
__device__ __forceinline__ uint32_t half_at(uint32_t stage, int lane, int i) {
  const int r = 8 * i + (lane >> 2);
  return stage + r * 128 + (((lane & 3) ^ (r & 7)) << 4);
}
__device__ __forceinline__ void load_half(Block& b, const char* p, int64_t ld, int rows, int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    b.v[i] = r < rows ? *reinterpret_cast<const uint4*>(p + r * ld + (lane & 3) * 16) : make_uint4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ void half_to_slice(const Block& b, uint32_t stage, int lane) {
  __syncwarp();   // what the slice held has been read
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(half_at(stage, lane, i)), "r"(b.v[i].x), "r"(b.v[i].y),
                 "r"(b.v[i].z), "r"(b.v[i].w)
                 : "memory");
  __syncwarp();
}
__device__ __forceinline__ void half_to_rows(uint32_t stage, char* p, int64_t ld, int rows, int lane) {
  __syncwarp();   // every lane's pieces are in the slice
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = load_piece(half_at(stage, lane, i));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    if (r < rows) *reinterpret_cast<uint4*>(p + r * ld + (lane & 3) * 16) = v[i];
  }
  __syncwarp();
}
// The transposed image of 64 columns: value j of this lane's row goes to row j of 64 bytes
// (w: pairs of columns), then rows `cols` of them at p, whole (their ends may be padding).
__device__ __forceinline__ void mirror_rows(uint32_t stage, const uint32_t (&w)[32], char* p, int64_t ld, int cols,
                                            int lane) {
  __syncwarp();   // what the slice held has been read
#pragma unroll
  for (int j = 0; j < 64; ++j)
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(stage + j * 64 + lane * 2),
                 "h"((unsigned short)(w[j / 2] >> (j % 2 * 16)))
                 : "memory");
  __syncwarp();
  Block b;
#pragma unroll
  for (int i = 0; i < 8; ++i) b.v[i] = load_piece(stage + (8 * i + (lane >> 2)) * 64 + (lane & 3) * 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 8 * i + (lane >> 2);
    if (r < cols) *reinterpret_cast<uint4*>(p + r * ld + (lane & 3) * 16) = b.v[i];
  }
  __syncwarp();
}

// How addend and result are held: kOne: one fp16 plane; kTwo: two; kLow: one and the 8-bit
// part (X of bf16 matrices); kLowIn: the addend so, the result in one plane; kOneTwice: kOne
// with two addends.
enum Form { kOne = 0, kTwo = 1, kLow = 2, kLowIn = 3, kOneTwice = 4 };

// Operand maps are 3-D, {columns, rows, plane * batch + matrix}: boxes of 64 columns by
// 128 rows, kApply's B operand 64 by 64 in its stored layout.
struct Maps {
  CUtensorMap A, B;
};

// SPLIT: kGram's sums in pieces, which go to a.parts.  NB: columns of a tile.
template <int KIND, int FORM, bool SPLIT = false, int NB = 256>
__global__ void __launch_bounds__(THREADS, 1) orth_kernel(const __grid_constant__ Maps maps, const Args a) {
  constexpr int BN = NB, BNC = BN / 2, B_BYTES = BNC * BK * 2, EPI_COLS = BN / 2;
  constexpr bool NARROW = NB == 128;
  static_assert(!NARROW || !SPLIT, "pieces of a sum are whole tiles");
  // two planes: a stage has both of both operands, for the three products
  constexpr int PL = FORM == kTwo ? 2 : 1, S = MAX_STAGES / PL, STAGE_BYTES = PL * (A_BYTES + B_BYTES);
  constexpr bool LOW_IN = FORM == kLow || FORM == kLowIn, LOW_OUT = FORM == kLow;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* s_out = smem + RING_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_out + EPI_WARPS * STAGE_WARP);
  // bars: full[S] empty[S] tfull[2] tempty[2] final
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const uint32_t ring = smem_u32(smem);
  auto full = [&](int s) { return smem_u32(&bars[s]); };
  auto empty = [&](int s) { return smem_u32(&bars[S + s]); };
  auto tfull = [&](int b) { return smem_u32(&bars[2 * S + b]); };
  auto tempty = [&](int b) { return smem_u32(&bars[2 * S + 2 + b]); };
  const uint32_t final_bar = smem_u32(&bars[2 * S + 4]);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);      // the even CTA's producer (pair's bytes)
      mbar_init(empty(s), 1);     // the pair's MMA commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), 2 * EPI_WARPS);
    }
    mbar_init(final_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncwarp();
  __syncthreads();
  cluster_sync();   // barriers of both CTAs initialised before any remote arrive
  if (warp == 1) {
    tmem_alloc2(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish2();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  const uint32_t total = (uint32_t)a.per * (uint32_t)a.batch, first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const int steps = a.kb;   // k-blocks of a tile
  const int chunk = FORM == kTwo ? kChunkExact : steps;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ROLE_REGS));
    if (warp == 0 && lane == 0) {
      // ---------------- TMA producer ----------------
      int s = 0;
      uint32_t ph = 0, issued = 0;
      bool ok = true;
      const uint32_t full0 = map_to_rank(full(0), 0);   // the even CTA's "full" barriers
      for (Walk<KIND, SPLIT, NARROW> walk(a, first, step); ok && walk.t < total; walk.next(a)) {
        const Tile q = walk.tile(a);
        const int arow = q.i * BM + (int)rank * BMC, bcol = q.j * BN + (int)rank * BNC;
        // (a piece's last k-blocks may lie past n: zeros)
        const int k0 = SPLIT ? q.piece * a.kb * BK : 0;
        for (int k = k0; k < k0 + a.kb * BK; k += BK) {
          if (!wait_cl(empty(s), ph ^ 1u, abort_flag)) { ok = false; break; }
          const uint32_t sa = ring + s * STAGE_BYTES, sb = sa + PL * A_BYTES, fb = full0 + 8u * s;
          if (leader) mbar_expect_tx(full(s), 2 * STAGE_BYTES);
#pragma unroll
          for (int p = 0; p < PL; ++p) {
            const int z = p * a.batch + q.b;
            tma_load_3d_pair(sa + p * A_BYTES, &maps.A, k, arow, z, fb);
            if (KIND == kApply) {
              tma_load_3d_pair(sb + p * B_BYTES, &maps.B, bcol, k, z, fb);
              if (!NARROW) tma_load_3d_pair(sb + p * B_BYTES + BOX_BYTES, &maps.B, bcol + 64, k, z, fb);
            } else {
              tma_load_3d_pair(sb + p * B_BYTES, &maps.B, k, bcol, z, fb);
            }
          }
          ++issued;
          if (++s == S) { s = 0; ph ^= 1u; }
        }
      }
      if (*abort_flag) {
        // loads still in flight land before the pair goes away (the odd CTA's count on
        // the even CTA's barriers: it waits a thousand times a load's latency instead)
        if (leader) {
          for (uint32_t i = issued > (uint32_t)S ? issued - S : 0u; i < issued; ++i)
            wait2_quiet(full((int)(i % S)), (i / S) & 1u);
        } else {
          const long long t0 = clock64();
          while (clock64() - t0 < kDrainCycles) {}
        }
      }
    } else if (warp == 1 && lane == 0 && leader) {
      // ---------------- even CTA: MMA issuer for the pair ----------------
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      const uint32_t idesc = idesc_of(BN) | (KIND == kApply ? IDESC_B_MN : 0u);
      for (uint32_t t = first; ok && t < total; t += step) {
        for (int i0 = 0; i0 < steps && ok; i0 += chunk) {
          const int i1 = min(steps, i0 + chunk);
          if (!wait_cl(tempty(acc), aph ^ 1u, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)acc * BN;
          for (int i = i0; i < i1; ++i) {
            if (!wait_cl(full(s), ph, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sa = ring + s * STAGE_BYTES, sb = sa + PL * A_BYTES;
            // two planes: (1, 0), (0, 1), (0, 0)
#pragma unroll
            for (int p = 0; p < (PL == 2 ? 3 : 1); ++p) {
              const uint32_t oa = sa + (PL == 2 && p == 0 ? A_BYTES : 0), ob = sb + (PL == 2 && p == 1 ? B_BYTES : 0);
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk) {
                const uint64_t bd = KIND == kApply ? mn_desc(ob + kk * 2048) : sw128_desc(ob + kk * 32);
                mma2(d, sw128_desc(oa + kk * 32), bd, idesc, (i != i0 || p != 0 || kk != 0) ? 1u : 0u);
              }
            }
            commit2_both(empty(s));
            if (++s == S) { s = 0; ph ^= 1u; }
          }
          if (!ok) break;
          commit2_both(tfull(acc));
          acc ^= 1;
          if (acc == 0) aph ^= 1u;
        }
      }
      if (*abort_flag) {
        commit2_self(final_bar);
        wait2_quiet(final_bar, 0);
      }
    }
  } else {
    // ---------------- epilogue (warps 4..11, both CTAs) ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    const int q = warp & 3;                 // TMEM lanes 32q .. 32q+31
    const int c_lo = (warp - 4) / 4 * EPI_COLS;
    const uint32_t stage = smem_u32(s_out + (warp - 4) * STAGE_WARP);
    const int width = KIND == kApply ? a.n : a.m;
    int acc = 0;
    uint32_t aph = 0;
    bool ok = true;
    auto wait_acc = [&]() {
      int w = 1;
      if (lane == 0) w = wait_cl(tfull(acc), aph, abort_flag) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, w, 0);
      if (ok) tc_fence_after();
      return ok;
    };
    auto free_acc = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_relaxed(map_to_rank(tempty(acc), 0));
      acc ^= 1;
      if (acc == 0) aph ^= 1u;
    };
    auto tmem_at = [&]() { return tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)acc * BN + c_lo; };
    // a tile's part of this warp: its first row (of all matrices' rows) and column, and how
    // many rows there are; columns past the width go to the rows' padding
    struct Part {
      int64_t row;
      int n0, rows, r0;
    };
    auto part_of = [&](const Tile& d) {
      Part p;
      p.r0 = d.i * BM + (int)rank * BMC + q * 32;
      p.row = (int64_t)d.b * a.m + p.r0;
      p.n0 = d.j * BN + c_lo;
      p.rows = p.n0 < width ? min(32, a.m - p.r0) : 0;
      return p;
    };
    auto block_col = [&](const Tile& d) { return NARROW ? d.j >> 1 : d.j; };   // of 256 columns
    // the mirror image of 64 columns from `col`
    auto mirror = [&](char* out, const Tile& d, const Part& p, int col, const uint32_t (&w)[32]) {
      mirror_rows(stage, w, out + ((int64_t)d.b * a.m + col) * a.add_ld + 2 * p.r0, a.add_ld, a.m - col, lane);
    };
    // a lane's row of a partial tile
    auto part_row = [&](uint32_t t) {
      return a.parts + ((size_t)t * BM + (int)rank * BMC + q * 32 + lane) * BN + c_lo;
    };
    if constexpr (SPLIT && FORM == kOne) {
      for (uint32_t t = first; t < total; t += step) {
        if (!wait_acc()) break;
        float4* to = reinterpret_cast<float4*>(part_row(t));
#pragma unroll
        for (int c = 0; c < EPI_COLS / 32; ++c) {
          uint32_t r[32];
          tmem_ld32(tmem_at() + 32 * c, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            to[8 * c + j] = make_float4(__uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]),
                                        __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
        }
        free_acc();
      }
    } else if constexpr (FORM != kTwo) {
      // One sum a tile, 16 columns at a time from TMEM through the slice.  A block of the
      // addend is asked for as soon as the one before has gone into the slice: half a tile
      // ahead, the 8-bit parts a tile (more would not fit into the registers).
      Block hi, lo;
      auto ask_hi = [&](const Part& p, int h) {
        if (KIND != kGram)
          load_block(hi, a.add + p.row * a.add_ld + 2 * (p.n0 + 64 * h), a.add_ld, p.n0 + 64 * h < width ? p.rows : 0,
                     lane);
      };
      Block more;
      auto ask_more = [&](const Part& p, int h) {
        if (FORM == kOneTwice)
          load_block(more, a.add2 + p.row * a.add_ld + 2 * (p.n0 + 64 * h), a.add_ld,
                     p.n0 + 64 * h < width ? p.rows : 0, lane);
      };
      auto ask_lo = [&](const Part& p) {
        if (!LOW_IN) return;
        const char* at = a.add_low + p.row * a.low_ld + p.n0;
        if (NARROW) load_half(lo, at, a.low_ld, p.rows, lane);
        else load_block(lo, at, a.low_ld, p.rows, lane);
      };
      Walk<KIND, SPLIT, NARROW> walk(a, first, step);
      Tile d = walk.tile(a), dn = d;
      Part p = part_of(d), pn = p;
      ask_lo(p);
      ask_hi(p, 0);
      ask_more(p, 0);
      for (uint32_t t = first; t < total; t += step, d = dn, p = pn) {
        walk.next(a);
        if (walk.t < total) {
          dn = walk.tile(a);
          pn = part_of(dn);
        } else {
          pn.rows = 0;     // nothing more to ask for
        }
        uint32_t low[LOW_IN ? EPI_COLS / 4 : 1];     // this lane's 8-bit parts
        if (LOW_IN) {
          if (NARROW) half_to_slice(lo, stage, lane);
          else block_to_slice(lo, stage, lane);
          ask_lo(pn);
#pragma unroll
          for (int j = 0; j < EPI_COLS / 16; ++j) {
            const uint4 v = get_piece(stage, lane, j);
            low[4 * j] = v.x;
            low[4 * j + 1] = v.y;
            low[4 * j + 2] = v.z;
            low[4 * j + 3] = v.w;
          }
        }
        if (!wait_acc()) break;
        const uint32_t taddr = tmem_at();
        uint32_t r[2][16];
        tmem_ld16(taddr, r[0]);
#pragma unroll
        for (int h = 0; h < EPI_COLS / 64; ++h) {
          uint32_t second[FORM == kOneTwice ? 32 : 1];   // this lane's part of the second addend
          if (FORM == kOneTwice) {
            block_to_slice(more, stage, lane);
            if (NARROW) ask_more(pn, 0);
            else ask_more(h ? pn : p, h ^ 1);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint4 v = get_piece(stage, lane, j);
              second[4 * j] = v.x;
              second[4 * j + 1] = v.y;
              second[4 * j + 2] = v.z;
              second[4 * j + 3] = v.w;
            }
          }
          if (KIND != kGram) {
            block_to_slice(hi, stage, lane);
            if (NARROW) ask_hi(pn, 0);
            else ask_hi(h ? pn : p, h ^ 1);
          }
          uint32_t w[32];      // 64 columns, packed
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int k = 4 * h + c;
            tmem_wait_ld();
            if (k < EPI_COLS / 16 - 1) tmem_ld16(taddr + 16 * (k + 1), r[(k + 1) & 1]);
#pragma unroll
            for (int g = 0; g < 2; ++g) {       // 8 columns: a piece
              int steps8[8];
              uint4 add = make_uint4(0, 0, 0, 0);
              if (KIND != kGram) add = get_piece(stage, lane, 2 * c + g);
              const uint32_t h4[4] = {add.x, add.y, add.z, add.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float2 f = mul2(both(a.mul), make_float2(__uint_as_float(r[k & 1][8 * g + 2 * e]),
                                                         __uint_as_float(r[k & 1][8 * g + 2 * e + 1])));
                if (KIND != kGram) {
                  float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h4[e]));
                  if (LOW_IN) {
                    const uint32_t part = low[16 * h + 4 * c + 2 * g + e / 2];
                    x.x = orth_with_low(x.x, part, e % 2 * 2);
                    x.y = orth_with_low(x.y, part, e % 2 * 2 + 1);
                  }
                  f = fma2(both(a.add_scale), x, f);
                }
                if (FORM == kOneTwice) {
                  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&second[8 * c + 4 * g + e]));
                  f = fma2(both(a.add2_scale), x, f);
                }
                const uint32_t v = pack_half2(f.x, f.y);
                w[8 * c + 4 * g + e] = v;
                if (LOW_OUT) {
                  const float2 lead = __half22float2(*reinterpret_cast<const __half2*>(&v));
                  steps8[2 * e] = orth_low_steps(f.x, lead.x);
                  steps8[2 * e + 1] = orth_low_steps(f.y, lead.y);
                }
              }
              const uint32_t* v = w + 8 * c + 4 * g;
              put_piece(stage, lane, 2 * c + g, make_uint4(v[0], v[1], v[2], v[3]));
              if (LOW_OUT) {
                // the parts replace the addend's
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  low[16 * h + 4 * c + 2 * g + e] =
                      orth_low_pack(steps8[4 * e], steps8[4 * e + 1], steps8[4 * e + 2], steps8[4 * e + 3]);
              }
            }
          }
          if (h == EPI_COLS / 64 - 1) free_acc();
          const int col = p.n0 + 64 * h, rows = col < width ? p.rows : 0;
          slice_to_rows(stage, a.out + p.row * a.add_ld + 2 * col, a.add_ld, rows, lane);
          if (KIND != kApply && d.i != block_col(d) && rows > 0) mirror(a.out, d, p, col, w);
        }
        if (LOW_OUT) {
#pragma unroll
          for (int j = 0; j < EPI_COLS / 16; ++j)
            put_piece(stage, lane, j, make_uint4(low[4 * j], low[4 * j + 1], low[4 * j + 2], low[4 * j + 3]));
          char* to = a.out_low + p.row * a.low_ld + p.n0;
          if (NARROW) half_to_rows(stage, to, a.low_ld, p.rows, lane);
          else slice_to_rows(stage, to, a.low_ld, p.rows, lane);
        }
      }
    } else {
      for (Walk<KIND, SPLIT, NARROW> walk(a, first, step); ok && walk.t < total; walk.next(a)) {
        const Tile d = walk.tile(a);
        const Part p = part_of(d);
        float f[EPI_COLS];
#pragma unroll
        for (int j = 0; j < EPI_COLS; ++j) f[j] = 0.0f;
        if (KIND != kGram && p.rows > 0) {
          // start from the addend's two planes
#pragma unroll
          for (int h = 0; h < EPI_COLS / 64; ++h) {
            const int rows = p.n0 + 64 * h < width ? p.rows : 0;
            Block b[2];
            load_block(b[0], a.add + p.row * a.add_ld + 2 * (p.n0 + 64 * h), a.add_ld, rows, lane);
            load_block(b[1], a.add_low + p.row * a.add_ld + 2 * (p.n0 + 64 * h), a.add_ld, rows, lane);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              block_to_slice(b[k], stage, lane);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint4 v = get_piece(stage, lane, j);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
                  float* g = f + 64 * h + 8 * j + 2 * e;
                  g[0] = fmaf(a.add_scale, x.x, g[0]);
                  g[1] = fmaf(a.add_scale, x.y, g[1]);
                }
              }
            }
          }
        }
#pragma unroll 1
        for (int i0 = 0; i0 < steps; i0 += chunk) {
          const float mul = SPLIT ? 1.0f : a.mul;   // the parts are bare sums
          if (!wait_acc()) break;
          const uint32_t taddr = tmem_at();
#pragma unroll
          for (int c = 0; c < EPI_COLS; c += 32) {
            uint32_t r[32];
            tmem_ld32(taddr + c, r);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) f[c + j] = fmaf(mul, __uint_as_float(r[j]), f[c + j]);
          }
          free_acc();
        }
        if (!ok) break;
        if constexpr (SPLIT) {
          float4* to = reinterpret_cast<float4*>(part_row(walk.t));
#pragma unroll
          for (int j = 0; j < EPI_COLS / 4; ++j) to[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
          continue;
        }
        if (p.rows <= 0) continue;
#pragma unroll
        for (int h = 0; h < EPI_COLS / 64; ++h) {
          const int col = p.n0 + 64 * h;
          if (col >= width) continue;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            char* out = k == 0 ? a.out : a.out_low;
            uint32_t w[32];
            __syncwarp();   // what the slice held has been read
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float* g = f + 64 * h + 8 * j + 2 * e;
                w[4 * j + e] = pack_half2(g[0], g[1]);
                if (k == 0) {
                  // what the leading plane leaves
                  const float2 lead = __half22float2(*reinterpret_cast<const __half2*>(&w[4 * j + e]));
                  g[0] -= lead.x;
                  g[1] -= lead.y;
                }
              }
              put_piece(stage, lane, j, make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
            }
            slice_to_rows(stage, out + p.row * a.add_ld + 2 * col, a.add_ld, p.rows, lane);
            if (KIND != kApply && d.i != block_col(d)) mirror(out, d, p, col, w);
          }
        }
      }
    }
  }

  __syncwarp();     // the barriers below are for whole warps: roles end lane by lane
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync();   // no MMA, TMEM load or remote arrive of the pair in flight
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc2(tmem_base, TMEM_COLS);
  }
  if (threadIdx.x == 0 && *abort_flag) set_flag(a.flags, kFlagTimeout);
}

// A tile of A from its pieces, added in order, to the planes and below the diagonal to its
// mirror image: 32 x 32 elements a block, four a thread.
template <int PLANES>
__global__ void __launch_bounds__(256) join_kernel(const Args a, int lda) {
  __shared__ float sh[32][33];
  pdl_trigger();
  pdl_wait();
  Args whole = a;
  whole.split = 1;
  whole.per = a.per / a.split;
  const uint32_t t = blockIdx.x >> 6;
  const Tile d = Walk<kPoly>(whole, t, 1).tile(whole);
  const int r0 = (blockIdx.x >> 3 & 7) * 32, c0 = (blockIdx.x & 7) * 32;
  const int row0 = d.i * BM + r0, col0 = d.j * BN + c0;
  if (row0 >= a.m || col0 >= a.m) return;
  const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 4;
  const float* p = a.parts + (size_t)t * a.split * BM * BN + (size_t)(r0 + r) * BN + c0 + c;
  float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int s = 0; s < a.split; ++s) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(p + (size_t)s * BM * BN));
    f[0] += v.x;
    f[1] += v.y;
    f[2] += v.z;
    f[3] += v.w;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] *= a.mul;
  auto put = [&](int row, int col) {     // columns past m go to the rows' padding
    if (row >= a.m || col >= lda) return;
    const int64_t at = ((int64_t)d.b * a.m + row) * a.add_ld + 2 * col;
    const uint32_t h[2] = {pack_half2(f[0], f[1]), pack_half2(f[2], f[3])};
    *reinterpret_cast<uint2*>(a.out + at) = make_uint2(h[0], h[1]);
    if (PLANES == 2) {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h[0]));
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&h[1]));
      *reinterpret_cast<uint2*>(a.out_low + at) =
          make_uint2(pack_half2(f[0] - x.x, f[1] - x.y), pack_half2(f[2] - y.x, f[3] - y.y));
    }
  };
  put(row0 + r, col0 + c);
  if (d.i == d.j) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) sh[r][c + e] = f[e];
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = sh[c + e][r];
  put(col0 + r, row0 + c);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// `count` matrices [rows, cols] of fp16, rows ld elements apart; 128-byte swizzle.
static bool map3(CUtensorMap* m, const void* ptr, int64_t count, int rows, int cols, int ld, int box_cols, int box_rows) {
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
  cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * 2 * (cuuint64_t)rows};
  cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return encode_fn() != nullptr &&
         encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static std::atomic<int> g_clusters[64];

// Clusters of two CTAs that run at once, and the kernels' shared-memory limit
// (set once per device; several host threads may come here).
static cudaError_t prepare_device(int* clusters) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (g_clusters[dev] == 0) {
    const void* fn[] = {(const void*)orth_kernel<kPoly, kOneTwice>, (const void*)orth_kernel<kGram, kOne, true>,
                         (const void*)orth_kernel<kGram, kTwo, true>,
                         (const void*)orth_kernel<kGram, kOne, false, 128>, (const void*)orth_kernel<kGram, kTwo, false, 128>,
                         (const void*)orth_kernel<kPoly, kOne, false, 128>, (const void*)orth_kernel<kPoly, kTwo, false, 128>,
                         (const void*)orth_kernel<kPoly, kOneTwice, false, 128>,
                         (const void*)orth_kernel<kApply, kOne, false, 128>, (const void*)orth_kernel<kApply, kTwo, false, 128>,
                         (const void*)orth_kernel<kApply, kLow, false, 128>, (const void*)orth_kernel<kApply, kLowIn, false, 128>,
                         (const void*)orth_kernel<kGram, kOne>,  (const void*)orth_kernel<kGram, kTwo>,
                         (const void*)orth_kernel<kPoly, kOne>,  (const void*)orth_kernel<kPoly, kTwo>,
                         (const void*)orth_kernel<kApply, kLow>, (const void*)orth_kernel<kApply, kLowIn>,
                         (const void*)orth_kernel<kApply, kOne>, (const void*)orth_kernel<kApply, kTwo>};
    int least = 1 << 30;
    for (const void* f : fn) {
      e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
      if (e != cudaSuccess) return e;
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(2);
      cfg.blockDim = dim3(THREADS);
      cfg.dynamicSmemBytes = SMEM_BYTES;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, f, &cfg);
      if (e != cudaSuccess) return e;
      if (n < least) least = n;
    }
    g_clusters[dev] = least > 0 ? least : -1;
  }
  *clusters = g_clusters[dev].load();
  return *clusters > 0 ? cudaSuccess : cudaErrorNotSupported;
}

template <int KIND, int FORM, bool SPLIT = false, int NB = 256>
static cudaError_t launch(const Maps& maps, const Args& t, cudaStream_t st) {
  int mc = 0;
  cudaError_t e = prepare_device(&mc);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)t.per * t.batch;
  if (tiles <= 0) return cudaSuccess;
  if (tiles >= (1ll << 31)) return cudaErrorInvalidValue;
  const unsigned pairs = (unsigned)(tiles < mc ? tiles : mc);
  return launch_after(orth_kernel<KIND, FORM, SPLIT, NB>, 2 * pairs, THREADS, SMEM_BYTES, st, 2, maps, t);
}

static int gram_tiles(int m) {
  const int mt = (m + BM - 1) / BM;
  return mt * (mt + 1) / 2;
}
}  // namespace orth

// As many pieces as fill the pairs, of at least 8 k-blocks of 64, where the whole sum is long
// enough to pay for the partial tiles and their join: five steps with and without, 1 x 300 x 2200
// in fp32 264 us against 345, 4 x 55 x 3670 242 against 390, 2 x 731 x 8026 725 against 1065
// (bf16 395 against 465); bf16 1 x 704 x 2816 236 against 242, 1 x 300 x 1100 187 against 170,
// fp32 3 x 777 x 1001 388 against 390.
int orth_split(int64_t batch, int m, int n, int planes) {
  using namespace orth;
  constexpr int kPairs = 76, kLeast = 8, kLong = 48;   // fixed, so that the sums do not depend on the device
  const int64_t tiles = batch * gram_tiles(m), kb = (n + BK - 1) / BK;
  if (tiles <= 0 || 2 * tiles > kPairs || planes * kb < kLong) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(kPairs / tiles, kb / kLeast));
}
size_t orth_parts_bytes(int64_t most, int m, int n, int planes) {
  int64_t tiles = 0;
  for (int64_t b = 1; b <= most; ++b) {
    const int split = orth_split(b, m, n, planes);
    if (split > 1) tiles = std::max<int64_t>(tiles, b * orth::gram_tiles(m) * split);
    else break;   // nor does any larger batch
  }
  return (size_t)tiles * orth::BM * orth::BN * 4;
}

cudaError_t launch_orth_steps(const OrthBatch& t, int steps, const double (*coef)[3], int* last, cudaStream_t st) {
  using namespace orth;
  const int64_t B = t.batch, all = B * t.planes;
  const bool two = t.planes == 2;
  const int split = t.parts ? orth_split(B, t.m, t.n, t.planes) : 1;
  // the products' maps, those of X for either buffer as the source
  CUtensorMap of_a, of_b, of_c;
  // Tiles of 128 columns for kGram and kPoly where those of 256 leave half of the pairs idle: five
  // steps with and without, 3 x 777 x 1001 in fp32 307 us against 369, bf16 1 x 704 x 2816 189
  // against 222, 1 x 2048 x 7168 465 against 488, 37 x 200 x 300 (37 tiles) 132 against 142
  const bool narrow = 2 * B * gram_tiles(t.m) <= 76;
  const int b_rows = narrow ? 64 : 128;
  CUtensorMap as_b[3];   // a, b and c as the second operand
  Maps gram[2];
  CUtensorMap apply_x[2];
  if (!map3(&of_a, t.a, all, t.m, t.m, t.lda, 64, 128) || !map3(&of_b, t.b, all, t.m, t.m, t.lda, 64, 128) ||
      !map3(&of_c, t.c ? t.c : t.a, all, t.m, t.m, t.lda, 64, 128) ||
      !map3(&as_b[0], t.a, all, t.m, t.m, t.lda, 64, b_rows) || !map3(&as_b[1], t.b, all, t.m, t.m, t.lda, 64, b_rows) ||
      !map3(&as_b[2], t.c ? t.c : t.a, all, t.m, t.m, t.lda, 64, b_rows))
    return cudaErrorInvalidValue;
  for (int i = 0; i < 2; ++i) {
    // planes of X: two of fp16, or one with the 8-bit parts behind it
    const int64_t planes = (two ? 2 : 1) * B;
    if (!map3(&gram[i].A, t.x[i], planes, t.m, t.n, t.ldx, 64, 128) ||
        !map3(&apply_x[i], t.x[i], planes, t.m, t.n, t.ldx, 64, 64))
      return cudaErrorInvalidValue;
    gram[i].B = gram[i].A;
    if (narrow && split == 1 && !map3(&gram[i].B, t.x[i], planes, t.m, t.n, t.ldx, 64, b_rows)) return cudaErrorInvalidValue;
  }
  Args g = {};
  g.m = t.m;
  g.n = t.n;
  g.batch = (int)B;
  g.planes = t.planes;
  g.flags = t.flags;
  g.mt = (t.m + BM - 1) / BM;
  g.nt = (t.n + BN - 1) / BN;
  const int64_t rows = B * t.m, a_ld = (int64_t)t.lda * 2, x_ld = (int64_t)t.ldx * 2;
  char *pa = static_cast<char*>(t.a), *pb = static_cast<char*>(t.b), *pc = static_cast<char*>(t.c);
  // out = add_scale add (+ add2_scale add2) + mul P Q, symmetric, the scales with the powers of two
  auto poly = [&](const CUtensorMap& P, const CUtensorMap& Q, double mul, const char* add, double add_scale,
                  const char* add2, double add2_scale, char* out) {
    const Maps maps = {P, Q};
    g.kb = (t.m + BK - 1) / BK;
    g.per = gram_tiles(t.m) * (narrow ? 2 : 1);
    g.mul = (float)mul;
    g.add_scale = (float)add_scale;
    g.add = add;
    g.add_low = add + rows * a_ld;
    g.add2 = add2;
    g.add2_scale = (float)add2_scale;
    g.add_ld = g.low_ld = a_ld;
    g.out = out;
    g.out_low = out + rows * a_ld;
    if (narrow) {
      if (two) return launch<kPoly, kTwo, false, 128>(maps, g, st);
      return add2 ? launch<kPoly, kOneTwice, false, 128>(maps, g, st) : launch<kPoly, kOne, false, 128>(maps, g, st);
    }
    if (two) return launch<kPoly, kTwo>(maps, g, st);
    return add2 ? launch<kPoly, kOneTwice>(maps, g, st) : launch<kPoly, kOne>(maps, g, st);
  };
  g.parts = t.parts;
  // kApply's by the same rule: 1 x 704 x 2816 bf16 181 us against 190, 1 x 1024 x 1024 155 against
  // 168, fp32 265 against 300
  const bool narrow_x = 2 * B * g.mt * g.nt <= 76;
  auto two_to = [](int e) { return std::ldexp(1.0, e); };
  bool low = true;     // x[0] has its 8-bit parts
  int at = 0;          // the buffer that X is in
  for (int i = 0; i < steps; at ^= 1) {
    char *from = static_cast<char*>(t.x[at]), *to = static_cast<char*>(t.x[at ^ 1]);
    // A = X X^T
    g.split = split;
    g.kb = ((t.n + BK - 1) / BK + split - 1) / split;
    g.per = gram_tiles(t.m) * (split > 1 ? split : narrow ? 2 : 1);
    g.mul = ldexpf(1.0f, kOrthA - 2 * kOrthX);
    g.add_ld = g.low_ld = a_ld;
    g.out = pa;
    g.out_low = pa + rows * a_ld;
    cudaError_t e;
    if (split > 1) e = two ? launch<kGram, kTwo, true>(gram[at], g, st) : launch<kGram, kOne, true>(gram[at], g, st);
    else if (narrow)
      e = two ? launch<kGram, kTwo, false, 128>(gram[at], g, st) : launch<kGram, kOne, false, 128>(gram[at], g, st);
    else e = two ? launch<kGram, kTwo>(gram[at], g, st) : launch<kGram, kOne>(gram[at], g, st);
    if (e == cudaSuccess && split > 1) {
      const unsigned blocks = (unsigned)(B * gram_tiles(t.m) * 64);
      e = two ? launch_after(join_kernel<2>, blocks, 256, 0, st, 1, g, t.lda)
              : launch_after(join_kernel<1>, blocks, 256, 0, st, 1, g, t.lda);
    }
    if (e != cudaSuccess) return e;
    // B = b A + c A A, the polynomial in the planes that the product reads
    const double *c0 = coef[i], *c1 = coef[i + 1 < steps ? i + 1 : i];
    e = poly(of_a, as_b[0], c0[2] * two_to(kOrthB - 2 * kOrthA), pa, c0[1] * two_to(kOrthB - kOrthA), nullptr, 0.0, pb);
    const bool pair = t.c && i == 0 && steps > 2;
    if (pair) {
      // C, A', B', R to c, a, c, a
      if (e == cudaSuccess) e = poly(of_b, as_b[0], two_to(-kOrthB), pa, c0[0], nullptr, 0.0, pc);
      if (e == cudaSuccess) e = poly(of_b, as_b[2], two_to(-kOrthB), pc, c0[0], nullptr, 0.0, pa);
      if (e == cudaSuccess)
        e = poly(of_a, as_b[0], c1[2] * two_to(kOrthB - 2 * kOrthA), pa, c1[1] * two_to(kOrthB - kOrthA), nullptr, 0.0, pc);
      if (e == cudaSuccess)
        e = poly(of_c, as_b[1], two_to(kOrthR - 2 * kOrthB), pc, c0[0] * two_to(kOrthR - kOrthB), pb,
                 c1[0] * two_to(kOrthR - kOrthB), pa);
    }
    if (e != cudaSuccess) return e;
    i += pair ? 2 : 1;
    // X' = a X + B X, or a a' X + R X
    const Maps apply = {pair ? of_a : of_b, apply_x[at]};
    g.kb = (t.m + BK - 1) / BK;
    g.per = g.mt * (narrow_x ? (t.n + 127) / 128 : g.nt);
    g.add_scale = (float)(pair ? c0[0] * c1[0] : c0[0]);
    g.mul = ldexpf(1.0f, pair ? -kOrthR : -kOrthB);
    g.add_ld = x_ld;
    g.low_ld = t.ldx;
    g.add = from;
    g.add_low = from + rows * x_ld;
    g.out = to;
    g.out_low = to + rows * x_ld;
    // What the steps to come multiply an error outside X's rows and columns by: up to 4, 11
    // bits do (simulated as above, the last two X without their parts: 1.6e-3 again for
    // normal entries, rank 16 1.0e-3 instead of 4.3e-4; the last three: rank 16 2.5e-3).  A
    // later X that needs its parts takes them from this one's, so the most of any of them
    // counts (a = 3.44, 3.44, 0.005, then 3.44 five times: rank 4 1.0e-3, by this X's factor
    // alone 7.0e-2).
    double grows = 1.0, most = 1.0;
    for (int k = steps - 1; k >= i; --k) {
      grows *= fabs(coef[k][0]);
      most = std::max(most, grows);
    }
    const bool keep = most > 4.0;
    auto product = [&](auto columns) {
      constexpr int NB = decltype(columns)::value;
      if (two) return launch<kApply, kTwo, false, NB>(apply, g, st);
      if (keep) return launch<kApply, kLow, false, NB>(apply, g, st);   // (low: most only falls)
      if (low) return launch<kApply, kLowIn, false, NB>(apply, g, st);
      return launch<kApply, kOne, false, NB>(apply, g, st);
    };
    e = narrow_x ? product(std::integral_constant<int, 128>()) : product(std::integral_constant<int, 256>());
    if (e != cudaSuccess) return e;
    low = keep;
  }
  *last = at;
  return cudaSuccess;
}

}  // namespace moe
