// orth_tc.cu -- the products of a Newton-Schulz step over a batch of matrices, on
// pairs of SMs (tcgen05 cta_group::2, fp16 operands, fp32 sums):
//   kGram   A  = X X^T          X [m, n], m <= n, K = n
//   kPoly   B  = b A + c A A    K = m
//   kApply  X' = a X + B X      K = m, X read in its stored layout (MN-major)
// A and B are symmetric: only the tiles on and below the diagonal are computed,
// and each is written twice, the second time transposed.
//
// Operands are the leading fp16 planes of X, A and B (11 bits); a X takes both planes
// of X, and X' is kept in both.  That matters more than the precision of the
// products: an error in X outside its row and column space grows by a in every
// step, 3.4445^5 = 484 in all, where one inside it meets the same polynomial as X
// itself.  Simulated at 512 x 1365 against 64 bits: X in one plane 3.6e-2 off for a
// matrix of rank 10 with a floor of 1e-2 (bf16 operands throughout: 0.29), in two planes
// 3.0e-4; normal entries 1.6e-3 (the polynomial in the rounded A, which b A takes from
// the same plane as A A: with b A exact instead 2.8e-3).  fp32 matrices take three
// products of two planes each, smallest first: 5.7e-7 (fp32 products: 7.2e-6).
//
// A pair of SMs computes 256 x 256 tiles over 64-wide k-blocks through four 32 KB
// stages.  The sums of a tile leave TMEM in chunks of k-blocks (the tensor cores cut
// the accumulator off at each K = 16 step) into fp32 registers, which start from the
// addend a X or b A, read while the tile's products run.
//
// Roles in each CTA: warp 0 TMA producer, warp 1 TMEM and (even CTA) the MMA
// issuer, warps 4-19 epilogue, four a 32-lane TMEM quarter (with two, whose 128 columns a
// thread had two warps a scheduler to hide behind, a 256 x 256 tile of kApply took
// 8.3 us, three times its products).  Tiles are dealt out in a
// fixed order (all have the same K).  Every wait on an mbarrier is bounded, and a CTA
// that gives up waits, with a limit, for its copies and MMAs in flight.
#include <atomic>
#include <cuda.h>
#include <cudaTypedefs.h>

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
constexpr int S = 4;
constexpr int A_BYTES = BMC * BK * 2, B_BYTES = BNC * BK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int BOX_BYTES = 64 * BK * 2;
constexpr int RING_BYTES = S * STAGE_BYTES;
constexpr int EPI_WARPS = 16, EPI_COLS = 64;   // a warp: 32 rows, 64 columns
constexpr int THREADS = 32 * (4 + EPI_WARPS);
// 96 registers a thread at launch; 56 + 4 * 104 <= 5 * 96 (five groups of 4 warps)
constexpr int ROLE_REGS = 56, EPI_REGS = 104;
static_assert(ROLE_REGS + 4 * EPI_REGS <= 5 * 96, "register pool of the launch");
constexpr uint32_t TMEM_COLS = 512;
constexpr int BAR_BYTES = 512;
// staging of an epilogue warp: 32 rows of 64 fp16 values (128-byte swizzle), and of 64
// 8-bit parts (64-byte swizzle)
constexpr int HALF_BYTES = 4096, LOW_BYTES = 2048, STAGE_WARP = HALF_BYTES + LOW_BYTES;
constexpr int SMEM_BYTES = 1024 + RING_BYTES + EPI_WARPS * STAGE_WARP + BAR_BYTES;
static_assert(SMEM_BYTES <= 232448, "shared memory budget of one CTA");
static_assert((2 * S + 5 + 2 * EPI_WARPS) * 8 + 8 <= BAR_BYTES, "barrier area");
constexpr long long kDrainCycles = 1 << 21;
constexpr int kChunkExact = 8, kChunkHalf = 64;   // k-blocks: two planes, one plane

// kind::f16: D fp32, A and B fp16, M = 256 over the pair, N = 256.
constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
constexpr uint32_t IDESC_B_MN = 1u << 16;

enum Kind { kGram = 0, kPoly = 1, kApply = 2 };

struct Args {
  int m, n;               // of the output: m x m, or m x n
  int batch, planes;      // of matrices; of operands
  int kb;                 // k-blocks
  int mt, nt, per;        // row tiles, column tiles, tiles a matrix
  float add_scale, mul;   // result = add_scale * addend + mul * product
  const char* add;        // the addend's leading plane, rows ld bytes apart: for the L2
  const char* add_low;    // its second plane, or 8-bit parts
  int64_t add_ld, low_ld;
  uint32_t* flags;
};

struct Tile {
  int b, i, j;
};
template <int KIND>
__device__ __forceinline__ Tile decode(const Args& a, uint32_t t) {
  Tile r;
  r.b = (int)(t / (uint32_t)a.per);
  uint32_t l = t - (uint32_t)r.b * (uint32_t)a.per;
  if (KIND == kApply) {
    r.j = (int)(l / (uint32_t)a.mt);
    r.i = (int)(l - (uint32_t)r.j * (uint32_t)a.mt);
  } else {
    // row i of the lower triangle starts at i (i + 1) / 2
    int i = (int)((sqrtf(8.0f * (float)l + 1.0f) - 1.0f) * 0.5f);
    while ((uint32_t)i * (i + 1) / 2 > l) --i;
    while ((uint32_t)(i + 1) * (i + 2) / 2 <= l) ++i;
    r.i = i;
    r.j = (int)(l - (uint32_t)i * (i + 1) / 2);
  }
  return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void add_halves(float* f, uint4 v, float scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = fmaf(scale, h.x, f[2 * i]);
    f[2 * i + 1] = fmaf(scale, h.y, f[2 * i + 1]);
  }
}
__device__ __forceinline__ void box_out(const CUtensorMap* map, uint32_t stage, int lane, int col, int row, int z) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(col), "r"(row), "r"(z), "r"(stage)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// How X' and the addend are held: kOne: one fp16 plane (A, B); kTwo: two; kLow: one
// and the 8-bit part (X of bf16 matrices).
enum Form { kOne = 0, kTwo = 1, kLow = 2 };

// Maps are 3-D, {columns, rows, plane * batch + matrix}.  mA, mB: operand boxes
// (128 x 64; kApply's B operand 64 x 64 in its stored layout); mAdd, mOut: 32 rows of
// 64 columns; mAddLow, mOutLow: 32 rows of 64 8-bit parts; mT: 64 rows of 32 columns, for the
// transposed tile.
struct Maps {
  CUtensorMap A, B, Add, AddLow, Out, OutLow, T;
};

template <int KIND, int FORM>
__global__ void __launch_bounds__(THREADS, 1) orth_kernel(const __grid_constant__ Maps maps, const Args a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* s_out = smem + RING_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_out + EPI_WARPS * STAGE_WARP);
  // bars: full[S] empty[S] tfull[2] tempty[2] final addend[2 * EPI_WARPS]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5 + 2 * EPI_WARPS);
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
  auto addend = [&](int w) { return smem_u32(&bars[2 * S + 5 + w]); };

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
    for (int w = 0; w < 2 * EPI_WARPS; ++w) mbar_init(addend(w), 1);
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
  const int nprod = a.planes == 2 ? 3 : 1;
  const int chunk = a.planes == 2 ? kChunkExact : kChunkHalf;
  const int steps = a.kb * nprod;   // k-blocks of a tile

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ROLE_REGS));
    if (warp == 0 && lane == 0) {
      // ---------------- TMA producer ----------------
      int s = 0;
      uint32_t ph = 0, issued = 0;
      bool ok = true;
      const uint32_t full0 = map_to_rank(full(0), 0);   // the even CTA's "full" barriers
      for (uint32_t t = first; ok && t < total; t += step) {
        const Tile q = decode<KIND>(a, t);
        const int arow = q.i * BM + (int)rank * BMC, bcol = q.j * BN + (int)rank * BNC;
        for (int p = 0; p < nprod && ok; ++p) {
          // the products of planes (1, 0), (0, 1), (0, 0)
          const int pa = nprod == 3 && p == 0, pb = nprod == 3 && p == 1;
          const int za = pa * a.batch + q.b, zb = pb * a.batch + q.b;
          for (int k = 0; k < a.kb * BK; k += BK) {
            if (!wait_cl(empty(s), ph ^ 1u, abort_flag)) { ok = false; break; }
            const uint32_t sa = ring + s * STAGE_BYTES, sb = sa + A_BYTES, fb = full0 + 8u * s;
            if (leader) mbar_expect_tx(full(s), 2 * STAGE_BYTES);
            tma_load_3d_pair(sa, &maps.A, k, arow, za, fb);
            if (KIND == kApply) {
              tma_load_3d_pair(sb, &maps.B, bcol, k, zb, fb);
              tma_load_3d_pair(sb + BOX_BYTES, &maps.B, bcol + 64, k, zb, fb);
            } else {
              tma_load_3d_pair(sb, &maps.B, k, bcol, zb, fb);
            }
            ++issued;
            if (++s == S) { s = 0; ph ^= 1u; }
          }
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
      const uint32_t idesc = IDESC | (KIND == kApply ? IDESC_B_MN : 0u);
      for (uint32_t t = first; ok && t < total; t += step) {
        for (int i0 = 0; i0 < steps && ok; i0 += chunk) {
          const int i1 = min(steps, i0 + chunk);
          if (!wait_cl(tempty(acc), aph ^ 1u, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)acc * BN;
          for (int i = i0; i < i1; ++i) {
            if (!wait_cl(full(s), ph, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t sa = ring + s * STAGE_BYTES, sb = sa + A_BYTES;
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
              const uint64_t bd = KIND == kApply ? mn_desc(sb + kk * 2048) : sw128_desc(sb + kk * 32);
              mma2(d, sw128_desc(sa + kk * 32), bd, idesc, (i != i0 || kk != 0) ? 1u : 0u);
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
    // ---------------- epilogue (warps 4..19, both CTAs) ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    const int q = warp & 3;                 // TMEM lanes 32q .. 32q+31
    const int c_lo = (warp - 4) / 4 * EPI_COLS;
    const uint32_t half = smem_u32(s_out + (warp - 4) * STAGE_WARP), lows = half + HALF_BYTES;
    const uint32_t half_bar = addend(2 * (warp - 4)), low_bar = addend(2 * (warp - 4) + 1);
    const int width = KIND == kApply ? a.n : a.m;
    int acc = 0;
    uint32_t aph = 0, half_ph = 0, low_ph = 0;
    bool ok = true;
    // lane 0 waits for a box, the others' reads come after it
    auto landed = [&](uint32_t bar, uint32_t& ph) {
      int w = 1;
      if (lane == 0) {
        w = wait_cl(bar, ph, abort_flag) ? 1 : 0;
        // given up (perhaps for another warp's wait): the box still lands first
        if (!w) wait2_quiet(bar, ph);
      }
      ph ^= 1u;
      ok = __shfl_sync(0xffffffffu, w, 0) && ok;
      __syncwarp();   // (the exchange alone orders no memory)
    };
    auto ask = [&](uint32_t to, const CUtensorMap* map, int col, int row, int z, uint32_t bar, uint32_t bytes) {
      if (lane != 0) return;
      mbar_expect_tx(bar, bytes);
      tma_load_3d(to, map, col, row, z, bar);
    };
    // 16 bytes j of this lane's 64-byte row of 8-bit parts
    auto low_at = [&](int j) { return lows + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4); };
    for (uint32_t t = first; ok && t < total; t += step) {
      const Tile d = decode<KIND>(a, t);
      const int row0 = d.i * BM + (int)rank * BMC + q * 32, n0 = d.j * BN + c_lo;
      const bool live = row0 < a.m && n0 < width;
      float f[EPI_COLS];
#pragma unroll
      for (int j = 0; j < EPI_COLS; ++j) f[j] = 0.0f;
      if (KIND != kGram && live) {
        // start from the addend
        stage_free(lane);
        ask(half, &maps.Add, n0, row0, d.b, half_bar, HALF_BYTES);
        if (FORM == kLow) {
          ask(lows, &maps.AddLow, n0, row0, d.b, low_bar, LOW_BYTES);
          landed(half_bar, half_ph);
          landed(low_bar, low_ph);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 l;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(l.x), "=r"(l.y), "=r"(l.z), "=r"(l.w)
                         : "r"(low_at(j))
                         : "memory");
            const uint32_t low[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 v = get_piece(half, lane, 2 * j + h);
              const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w4[e]));
                const int at = 8 * h + 2 * e;    // of the 16 parts
                const uint32_t q2 = low[at / 4] >> (at % 4 * 8);
                f[16 * j + at] = a.add_scale * orth_with_low(x.x, (int)(int8_t)(q2 & 255u));
                f[16 * j + at + 1] = a.add_scale * orth_with_low(x.y, (int)(int8_t)((q2 >> 8) & 255u));
              }
            }
          }
        } else {
          landed(half_bar, half_ph);
#pragma unroll
          for (int j = 0; j < 8; ++j) add_halves(f + 8 * j, get_piece(half, lane, j), a.add_scale);
          if (FORM == kTwo) {
            __syncwarp();
            ask(half, &maps.Add, n0, row0, a.batch + d.b, half_bar, HALF_BYTES);
            landed(half_bar, half_ph);
#pragma unroll
            for (int j = 0; j < 8; ++j) add_halves(f + 8 * j, get_piece(half, lane, j), a.add_scale);
          }
        }
        __syncwarp();
        // the next tile's addend to the L2 while this one is worked on
        if (t + step < total) {
          const Tile e = decode<KIND>(a, t + step);
          const int row = e.i * BM + (int)rank * BMC + q * 32 + lane, col = e.j * BN + c_lo;
          if (row < a.m && col < width) {
            prefetch_l2(a.add + ((int64_t)e.b * a.m + row) * a.add_ld + 2 * col);
            if (FORM != kOne)
              prefetch_l2(a.add_low + ((int64_t)e.b * a.m + row) * a.low_ld + (FORM == kTwo ? 2 : 1) * col);
          }
        }
      }
      if (!ok) break;
#pragma unroll 1
      for (int i0 = 0; i0 < steps; i0 += chunk) {
        int w = 1;
        if (lane == 0) w = wait_cl(tfull(acc), aph, abort_flag) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, w, 0);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)acc * BN + c_lo;
#pragma unroll
        for (int c = 0; c < EPI_COLS; c += 16) {
          uint32_t r[16];
          tmem_ld16(taddr + c, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) f[c + j] = fmaf(a.mul, __uint_as_float(r[j]), f[c + j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_relaxed(map_to_rank(tempty(acc), 0));
        acc ^= 1;
        if (acc == 0) aph ^= 1u;
      }
      if (!ok) break;
      if (!live) continue;
      const bool mirror = KIND != kApply && d.i != d.j;
#pragma unroll
      for (int p = 0; p < (FORM == kTwo ? 2 : 1); ++p) {
        const int z = p * a.batch + d.b;
        stage_free(lane);
        if (FORM == kLow) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t l[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w4[4];
              int low[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float* v = f + 16 * j + 8 * h + 2 * e;
                w4[e] = pack_half2(v[0], v[1]);
                const float2 lead = __half22float2(*reinterpret_cast<const __half2*>(&w4[e]));
                low[2 * e] = orth_low_part(v[0], lead.x);
                low[2 * e + 1] = orth_low_part(v[1], lead.y);
              }
              put_piece(half, lane, 2 * j + h, make_uint4(w4[0], w4[1], w4[2], w4[3]));
              // the low bytes of four words
#pragma unroll
              for (int e = 0; e < 2; ++e)
                l[2 * h + e] = __byte_perm(__byte_perm(low[4 * e], low[4 * e + 1], 0x0040),
                                           __byte_perm(low[4 * e + 2], low[4 * e + 3], 0x0040), 0x5410);
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(low_at(j)), "r"(l[0]), "r"(l[1]), "r"(l[2]),
                         "r"(l[3])
                         : "memory");
          }
          box_out(&maps.OutLow, lows, lane, n0, row0, z);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float* v = f + 8 * j;
            put_piece(half, lane, j, make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]),
                                                pack_half2(v[6], v[7])));
          }
        }
        box_out(&maps.Out, half, lane, n0, row0, z);
        if (mirror) {
          // the transposed box: 64 rows (this warp's columns) of 32 values
          stage_free(lane);
#pragma unroll
          for (int j = 0; j < EPI_COLS; ++j) {
            const __half h = __float2half_rn(f[j]);
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(half + j * 64 + lane * 2),
                         "h"(*reinterpret_cast<const unsigned short*>(&h))
                         : "memory");
          }
          box_out(&maps.T, half, lane, row0, n0, z);
        }
        if (FORM == kTwo && p == 0) {
          // what the leading plane leaves
#pragma unroll
          for (int j = 0; j < EPI_COLS; ++j) f[j] -= __half2float(__float2half_rn(f[j]));
        }
      }
    }
    // the staging slices and what left them outlive the block's last tile
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
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

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// `count` matrices [rows, cols] of fp16 (or bytes), rows ld elements apart.
static bool map3(CUtensorMap* m, const void* ptr, int64_t count, int rows, int cols, int ld, int box_cols, int box_rows,
                 CUtensorMapSwizzle swizzle, int esize = 2) {
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
  cuuint64_t strides[2] = {(cuuint64_t)ld * esize, (cuuint64_t)ld * esize * (cuuint64_t)rows};
  cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return encode_fn() != nullptr &&
         encode_fn()(m, esize == 2 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
                     const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
    const void* fn[6] = {(const void*)orth_kernel<kGram, kOne>,  (const void*)orth_kernel<kGram, kTwo>,
                         (const void*)orth_kernel<kPoly, kOne>,  (const void*)orth_kernel<kPoly, kTwo>,
                         (const void*)orth_kernel<kApply, kLow>, (const void*)orth_kernel<kApply, kTwo>};
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

template <int KIND, int FORM>
static cudaError_t launch(const Maps& maps, const Args& t, cudaStream_t st) {
  int mc = 0;
  cudaError_t e = prepare_device(&mc);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)t.per * t.batch;
  if (tiles <= 0) return cudaSuccess;
  if (tiles >= (1ll << 31)) return cudaErrorInvalidValue;
  const unsigned pairs = (unsigned)(tiles < mc ? tiles : mc);
  return launch_after(orth_kernel<KIND, FORM>, 2 * pairs, THREADS, SMEM_BYTES, st, 2, maps, t);
}

}  // namespace orth

cudaError_t launch_orth_steps(const OrthBatch& t, int steps, const double (*coef)[3], cudaStream_t st) {
  using namespace orth;
  const int64_t B = t.batch, all = B * t.planes;
  const bool two = t.planes == 2;
  // the three products' maps, those of X for either buffer as the source
  Maps gram[2], poly, apply[2];
  CUtensorMap ak, aio;
  if (!map3(&ak, t.a, all, t.m, t.m, t.lda, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) || !map3(&aio, t.a, all, t.m, t.m, t.lda, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !map3(&gram[0].T, t.a, all, t.m, t.m, t.lda, 32, 64, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !map3(&apply[0].A, t.b, all, t.m, t.m, t.lda, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !map3(&poly.Out, t.b, all, t.m, t.m, t.lda, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !map3(&poly.T, t.b, all, t.m, t.m, t.lda, 32, 64, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  poly.A = poly.B = ak;
  poly.Add = poly.AddLow = aio;
  poly.OutLow = poly.Out;
  for (int i = 0; i < 2; ++i) {
    // planes of X: two of fp16, or one and the 8-bit parts behind it
    const int64_t planes = (two ? 2 : 1) * B;
    char* low = static_cast<char*>(t.x[i]) + B * t.m * (int64_t)t.ldx * 2;
    if (!map3(&gram[i].A, t.x[i], planes, t.m, t.n, t.ldx, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !map3(&apply[i].B, t.x[i], planes, t.m, t.n, t.ldx, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !map3(&apply[i].Add, t.x[i], planes, t.m, t.n, t.ldx, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !map3(&apply[i].AddLow, low, B, t.m, t.n, t.ldx, 64, 32, CU_TENSOR_MAP_SWIZZLE_64B, 1))
      return cudaErrorInvalidValue;
    gram[i].B = gram[i].Add = gram[i].AddLow = gram[i].A;
    gram[i].Out = gram[i].OutLow = aio;
    gram[i].T = gram[0].T;
    apply[i].A = apply[0].A;
    apply[i].T = poly.T;
  }
  for (int i = 0; i < 2; ++i) {
    apply[i].Out = apply[i ^ 1].Add;
    apply[i].OutLow = apply[i ^ 1].AddLow;
  }
  Args g = {};
  g.m = t.m;
  g.n = t.n;
  g.batch = (int)B;
  g.planes = t.planes;
  g.flags = t.flags;
  g.mt = (t.m + BM - 1) / BM;
  g.nt = (t.n + BN - 1) / BN;
  for (int i = 0; i < steps; ++i) {
    const int from = i & 1;
    // A = X X^T
    g.kb = (t.n + BK - 1) / BK;
    g.per = g.mt * (g.mt + 1) / 2;
    g.mul = ldexpf(1.0f, kOrthA - 2 * kOrthX);
    cudaError_t e = two ? launch<kGram, kTwo>(gram[from], g, st) : launch<kGram, kOne>(gram[from], g, st);
    if (e != cudaSuccess) return e;
    // B = b A + c A A, the polynomial in the planes that the product reads
    g.kb = (t.m + BK - 1) / BK;
    g.add_scale = ldexpf((float)coef[i][1], kOrthB - kOrthA);
    g.mul = ldexpf((float)coef[i][2], kOrthB - 2 * kOrthA);
    g.add_ld = g.low_ld = (int64_t)t.lda * 2;
    g.add = static_cast<const char*>(t.a);
    g.add_low = g.add + B * t.m * g.add_ld;
    e = two ? launch<kPoly, kTwo>(poly, g, st) : launch<kPoly, kOne>(poly, g, st);
    if (e != cudaSuccess) return e;
    // X' = a X + B X
    g.per = g.mt * g.nt;
    g.add_scale = (float)coef[i][0];
    g.mul = ldexpf(1.0f, -kOrthB);
    g.add_ld = (int64_t)t.ldx * 2;
    g.low_ld = two ? g.add_ld : t.ldx;
    g.add = static_cast<const char*>(t.x[from]);
    g.add_low = g.add + B * t.m * g.add_ld;
    e = two ? launch<kApply, kTwo>(apply[from], g, st) : launch<kApply, kLow>(apply[from], g, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
