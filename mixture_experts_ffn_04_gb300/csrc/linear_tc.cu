// linear_tc.cu -- the dense GEMMs of the training operators on pairs of SMs
// (tcgen05 cta_group::2): logits z = x W^T with the softmax statistics or the
// logit gradient in the epilogue, and the two gradient products
//   dX = D W   (D [rows, V], W [V, H])      K = vocabulary
//   dW = D^T x (D [rows, V], x [rows, H])   K = rows
// in one launch over one tile list; and the plain product x W^T in fp32 (a
// router's logits).
//
// A pair of SMs computes 256 x 256 output tiles over 64-wide k-blocks: CTA r
// keeps rows 128r .. of the A tile and columns 128r .. of the B tile, six
// 32 KB stages; per k-block an SM reads 32 KB of operands for 512 clocks of
// MMA.  Operands that are not K-major are read in their stored layout as
// 64-wide boxes with the 128-byte swizzle (MN-major descriptors), so neither D
// nor W nor x is ever transposed in memory.  The tile order is dynamic (one
// counter in global memory): the tiles in progress form one window, and within
// it groups of kGroupM row tiles pass over the column tiles, so the rows of a
// group stay in L2 while the other operand streams by once per group.
//
// The gradient launch puts the tiles with the longer K first (dX, K = vocabulary,
// unless the rows are more): the short ones run beside them and fill the SMs that
// the long ones leave idle at their end.  Where tiles are few and long, K is split and the fp32 partial
// sums are added in split order by a second kernel (no atomics: the result does
// not depend on the order of the tiles).
//
// The tensor cores cut the fp32 accumulator off at each K = 16 step (measured:
// the loss of one row over H = 2048 came out 4e-6 low in relative terms, as 128
// truncations predict), so a tile is summed in chunks of k-blocks: each chunk in
// one of the two TMEM accumulators, the chunks in fp32 registers with rounding to
// nearest, which frees the accumulator as soon as it is read.  Chunks of 512 for
// logits and all fp32 products, 4096 for gradients that are rounded to bf16 anyway.
//
// fp32 operands come in three bf16 planes (train.h): a tile's k-loop runs over the
// six plane products whose weight is above 2^-24, smallest first.
//
// Measured under a full clock (T = 4096, H = 2048, V = 131072): statistics 1.67
// PFLOP/s, the logit gradient 1.63, the gradient products 1.83, against 1.91 for the
// library's matrix product; back to back under the power cap 1.5-1.55 against 1.73.
// What bounds them is the MMA rate and the cap; tiles with few k-blocks (dW of few
// rows, dX of a router) are bound by their output.
//
// Roles in each CTA: warp 0 TMA producer, warp 1 TMEM and (even CTA) the MMA
// issuer, warp 2 the L2 prefetch of dX's addend, warps 4-11 epilogue: two per 32-lane TMEM quarter, one per half of
// the 256 columns.  Every wait on an mbarrier is bounded; a CTA that gives up raises
// its abort flag, its partner's waits run out in turn, copies and MMAs in flight are
// waited for, again with a limit, and both meet at the closing cluster barrier before
// TMEM is released.  Not bounded are the closing barriers themselves, which every warp
// reaches from whatever it was doing, and the waits for a warp's own output boxes.
#include <atomic>
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "internal.h"
#include "tc_pair.cuh"
#include "tcgen05.cuh"
#include "train.h"

namespace moe {
namespace tc {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();   // gemm_tc.cu
}

namespace lin {

using namespace tc;

constexpr int BM = kLinTile, BN = kLinTile, BMC = BM / 2, BNC = BN / 2, BK = kLinK;
constexpr int S = 6;
constexpr int A_BYTES = BMC * BK * 2, B_BYTES = BNC * BK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int BOX_BYTES = 64 * BK * 2;
constexpr int RING_BYTES = S * STAGE_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (4 + EPI_WARPS);
// Registers a thread: 168 at launch (384 threads), then 56 in the role warps'
// group and 224 in the two epilogue groups, which hold 128 sums each:
// 56 + 2 * 224 <= 3 * 168.
constexpr int ROLE_REGS = 56, EPI_REGS = 224;
static_assert(ROLE_REGS + 2 * EPI_REGS <= 3 * 168, "register pool of the launch");
constexpr uint32_t TMEM_COLS = 512;
constexpr int NSLOT = 4;
constexpr int READERS = 4 + 2 * EPI_WARPS;   // of a tile slot: odd producer, MMA, prefetch and epilogue warps
constexpr int BAR_BYTES = 512;
constexpr int STAGE_WARP = 4096;   // output staging of an epilogue warp: 32 rows of 128 bytes
constexpr int SMEM_BYTES = 1024 + RING_BYTES + EPI_WARPS * STAGE_WARP + BAR_BYTES;
static_assert(SMEM_BYTES <= 232448, "shared memory budget of one CTA");
static_assert((2 * S + 5 + 2 * NSLOT + EPI_WARPS) * 8 + 8 + NSLOT * 32 <= BAR_BYTES, "barrier area");
constexpr long long kDrainCycles = 1 << 21;   // about a millisecond
constexpr int kGroupM = 8;
constexpr int kChunkExact = 8, kChunkBf16 = 64;   // k-blocks of 64

// kind::f16: D fp32, A and B bf16, M = 256 over the pair, N = 256.
constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) |
                           ((uint32_t)(BM >> 4) << 24);
constexpr uint32_t IDESC_A_MN = 1u << 15, IDESC_B_MN = 1u << 16;

enum Kind { kStats = 0, kDlogit = 1, kGrad = 2, kProduct = 3 };

struct Args {
  int hidden, planes, d_planes;
  int64_t v0, w_v0, vcols, vocab;
  const int32_t* nrows;
  int64_t rows_bound;
  int32_t* ctr;
  uint32_t* flags;
  int64_t x_plane, w_plane, d_plane;
  const int32_t* target;
  float2* stats;
  float* zt;
  int64_t rows_pad;
  const float4* rowstat;
  const float* g;
  const float* scale;   // of dX and dW
  int ks_dx, ks_dw, out_f32;
  float* dx_part;
  int accumulate;
  void* dx;
  const int32_t* rowmap;
  const void* dx_add;
  float* dw_part;
  int64_t dw_pad;
  int want_dx, want_dw;
  int wide_in;   // x and w in maps of 64-wide column blocks (hidden a multiple of 64)
  int wide_dx;   // rows of dx on 32-byte boundaries
  int chunk;   // k-blocks the tensor cores add up before the fp32 registers do
};

// Plane products in ascending weight: (0,2) (2,0) (1,1) (0,1) (1,0) (0,0).
__device__ __forceinline__ void plane_pair(int planes, int i, int& pa, int& pb) {
  if (planes == 1) { pa = pb = 0; return; }
  if (planes == kPlanesD2) { pa = 1 - i; pb = 0; return; }
  const int t = i == 0 ? 0x02 : i == 1 ? 0x20 : i == 2 ? 0x11 : i == 3 ? 0x01 : i == 4 ? 0x10 : 0x00;
  pa = t >> 4;
  pb = t & 15;
}

// A tile as it stands in a slot: decoded once, by the taker (the divisions cost
// every reader about 1900 clocks a tile otherwise, a third of a short tile).
struct __align__(16) Tile {
  int type;        // 0: logits, 1: dX, 2: dW; -1: no tile left
  int mt, nt, sp;
  int kb0, kb1;    // k-blocks of one plane product
  int pad[2];
};

// m-tiles in groups of kGroupM, n-tiles outer within a group.
__device__ __forceinline__ void order_tile(uint32_t t, uint32_t MT, uint32_t NT, int& mt, int& nt) {
  const uint32_t per = kGroupM * NT, grp = t / per, first = grp * kGroupM;
  const uint32_t size = MT - first < (uint32_t)kGroupM ? MT - first : (uint32_t)kGroupM;
  const uint32_t r = t - grp * per;
  nt = (int)(r / size);
  mt = (int)(first + r % size);
}

template <int KIND>
struct Plan {
  int MTr, NTh, NTv, KBv, KBr;
  uint32_t n_dx, n_dw, total;   // tiles (the launcher bounds them by 2^31)
  bool dw_first;                // the longer parts come first
  int64_t rows;
  __device__ __forceinline__ void init(const Args& a) {
    rows = a.nrows ? (int64_t)*a.nrows : a.rows_bound;
    if (rows > a.rows_bound) rows = a.rows_bound;
    if (rows < 0) rows = 0;
    MTr = (int)((rows + BM - 1) / BM);
    NTh = (a.hidden + BN - 1) / BN;
    NTv = (int)((a.vcols + BN - 1) / BN);
    KBv = (int)((a.vcols + BK - 1) / BK);
    KBr = (int)((rows + BK - 1) / BK);
    n_dx = 0;
    if (KIND == kGrad) {
      n_dx = a.want_dx ? (uint32_t)MTr * NTh * a.ks_dx : 0u;
      n_dw = a.want_dw ? (uint32_t)NTv * NTh * a.ks_dw : 0u;
      total = n_dx + n_dw;
      dw_first = KBr / a.ks_dw > KBv / a.ks_dx;
    } else {
      total = (uint32_t)MTr * NTv * (KIND == kProduct ? a.ks_dx : 1);
    }
  }
  __device__ __forceinline__ Tile decode(const Args& a, uint32_t t) const {
    Tile r;
    r.sp = 0;
    if (KIND != kGrad) {
      r.type = 0;
      const uint32_t kb = (a.hidden + BK - 1) / BK, ks = KIND == kProduct ? a.ks_dx : 1;
      if (ks > 1) {
        r.sp = (int)(t % ks);
        t /= ks;
      }
      order_tile(t, MTr, NTv, r.mt, r.nt);
      part_range(kb, ks, r);
      return r;
    }
    const uint32_t lead = dw_first ? n_dw : n_dx;
    const bool dx = (t < lead) != dw_first;
    if (t >= lead) t -= lead;
    r.type = dx ? 1 : 2;
    const uint32_t ks = dx ? a.ks_dx : a.ks_dw, kb = dx ? KBv : KBr;
    if (ks > 1) {
      r.sp = (int)(t % ks);
      t /= ks;
    }
    order_tile(t, dx ? MTr : NTv, NTh, r.mt, r.nt);
    part_range(kb, ks, r);
    return r;
  }
  // the first kb % ks parts take one k-block more
  static __device__ __forceinline__ void part_range(uint32_t kb, uint32_t ks, Tile& r) {
    const uint32_t each = kb / ks, more = kb % ks;
    r.kb0 = (int)(r.sp * each + min((uint32_t)r.sp, more));
    r.kb1 = r.kb0 + (int)(each + ((uint32_t)r.sp < more ? 1u : 0u));
  }
};

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// b where i == j, else a: a select that stays one (the compiler would turn a
// chain of them over an array into an indexed copy in local memory).
__device__ __forceinline__ float pick(float a, float b, int i, int j) {
  float r;
  asm("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %3, %4;\n\tselp.f32 %0, %2, %1, p;\n\t}\n"
      : "=f"(r)
      : "f"(a), "f"(b), "r"(i), "r"(j));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// A warp's slice (tc_pair.cuh) out as one box; add: it is added to what is there (fp32).
__device__ __forceinline__ void stage_out(const CUtensorMap* map, uint32_t stage, int lane, int col, int row,
                                          bool add) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    if (add)
      asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                       reinterpret_cast<uint64_t>(map)),
                   "r"(col), "r"(row), "r"(stage)
                   : "memory");
    else
      asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                       reinterpret_cast<uint64_t>(map)),
                   "r"(col), "r"(row), "r"(stage)
                   : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

// Rows of dX that go to their tokens are stored by the lane that owns the row, in
// 32-byte sectors (rows that are only 16-byte aligned in halves).
struct Sector {
  uint32_t v[8];
};
__device__ __forceinline__ void store_sector(void* p, const Sector& s, bool wide, bool second) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(s.v[0]), "r"(s.v[1]),
                 "r"(s.v[2]), "r"(s.v[3]), "r"(s.v[4]), "r"(s.v[5]), "r"(s.v[6]), "r"(s.v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(s.v[0], s.v[1], s.v[2], s.v[3]);
    if (second) reinterpret_cast<uint4*>(p)[1] = make_uint4(s.v[4], s.v[5], s.v[6], s.v[7]);
  }
}
// 16 values as bf16, 8 as fp32.
__device__ __forceinline__ Sector pack_bf16(const float* f) {
  Sector s;
#pragma unroll
  for (int i = 0; i < 8; ++i) s.v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  return s;
}
__device__ __forceinline__ Sector pack_f32(const float* f) {
  Sector s;
#pragma unroll
  for (int i = 0; i < 8; ++i) s.v[i] = __float_as_uint(f[i]);
  return s;
}

template <int KIND>
__global__ void __launch_bounds__(THREADS, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                  const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmDt,
                  const __grid_constant__ CUtensorMap tmOx, const __grid_constant__ CUtensorMap tmOw,
                  const __grid_constant__ CUtensorMap tmAdd, const Args a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* s_out = smem + RING_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_out + EPI_WARPS * STAGE_WARP);
  // bars: full[S] empty[S] tfull[2] tempty[2] final tfill[NSLOT] tdrain[NSLOT]
  // addend[EPI_WARPS], then the scalars and the tile slots
  static_assert(sizeof(Tile) == 32, "a slot is two 16-byte pieces");
  unsigned char* s_slots = reinterpret_cast<unsigned char*>(bars) + BAR_BYTES - NSLOT * sizeof(Tile);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 5 + 2 * NSLOT + EPI_WARPS);
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
  auto tfill = [&](int i) { return smem_u32(&bars[2 * S + 5 + i]); };
  auto addend = [&](int w) { return smem_u32(&bars[2 * S + 5 + 2 * NSLOT + w]); };
  auto tdrain = [&](int i) { return smem_u32(&bars[2 * S + 5 + NSLOT + i]); };

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
    for (int i = 0; i < NSLOT; ++i) {
      mbar_init(tfill(i), 1);
      mbar_init(tdrain(i), READERS);
    }
    for (int w = 0; w < EPI_WARPS; ++w) mbar_init(addend(w), 1);
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
  pdl_wait();   // barriers, TMEM and descriptors are set up under the kernel before
  Plan<KIND> plan;
  plan.init(a);
  const int nprod = a.planes == 1 ? 1 : a.planes == kPlanesD2 ? 2 : 6;

  // Tile n of this pair (type -1 when there is none left, or a wait ran out).
  // The even CTA's producer takes it, one ahead, from the counter, decodes it and
  // writes it to slot n % NSLOT of both CTAs; the other readers read their CTA's
  // slot and tell the even CTA that they have.
  uint32_t reserve = threadIdx.x == 0 && leader ? (uint32_t)atomicAdd(a.ctr, 1) : 0u;
  auto take_tile = [&](int n) -> Tile {
    const int slot = n % NSLOT;
    const uint32_t use = (uint32_t)n / NSLOT;
    Tile t;
    t.type = -1;
    if (!wait_cl(tdrain(slot), (use & 1u) ^ 1u, abort_flag)) return t;
    const uint32_t id = reserve;
    if (id < plan.total) {
      reserve = (uint32_t)atomicAdd(a.ctr, 1);
      t = plan.decode(a, id);
    }
    const uint32_t mine = smem_u32(s_slots + slot * sizeof(Tile)), other = map_to_rank(mine, 1);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine), "r"(t.type), "r"(t.mt), "r"(t.nt),
                 "r"(t.sp)
                 : "memory");
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(mine + 16), "r"(t.kb0), "r"(t.kb1) : "memory");
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(other), "r"(t.type), "r"(t.mt),
                 "r"(t.nt), "r"(t.sp)
                 : "memory");
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(other + 16), "r"(t.kb0), "r"(t.kb1)
                 : "memory");
    mbar_arrive(tfill(slot));
    mbar_arrive_cluster(map_to_rank(tfill(slot), 1));
    return t;
  };
  auto load_slot = [&](int slot) -> Tile {
    Tile t;
    const uint32_t mine = smem_u32(s_slots + slot * sizeof(Tile));
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(t.type), "=r"(t.mt), "=r"(t.nt), "=r"(t.sp)
                 : "r"(mine)
                 : "memory");
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(t.kb0), "=r"(t.kb1) : "r"(mine + 16) : "memory");
    return t;
  };
  auto read_tile = [&](int n) -> Tile {
    const int slot = n % NSLOT;
    const uint32_t use = (uint32_t)n / NSLOT;
    Tile t;
    t.type = -1;
    if (!wait_cl(tfill(slot), use & 1u, abort_flag)) return t;
    t = load_slot(slot);
    // the slot has been read (the branch needs the values) when the arrival goes
    if ((t.type ^ t.mt ^ t.nt ^ t.sp ^ t.kb0 ^ t.kb1) != INT32_MIN) arrive_relaxed(map_to_rank(tdrain(slot), 0));
    return t;
  };

  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(ROLE_REGS));
  if (warp == 0 && lane == 0) {
    // ---------------- TMA producer ----------------
    // A k-block has 512 clocks of MMA: what does not change within a tile is
    // computed before it, and each kind of tile has a loop of its own.
    int s = 0;
    uint32_t ph = 0, issued = 0;
    bool ok = true;
    const uint32_t full0 = map_to_rank(full(0), 0);   // the even CTA's "full" barriers
    const bool paired = a.planes == kPlanesD2;
    const int outer = paired ? 1 : nprod;
    for (int n = 0; ok; ++n) {
      const Tile t = leader ? take_tile(n) : read_tile(n);
      if (t.type < 0) break;
      const int arow = t.mt * BM + (int)rank * BMC, bcol = t.nt * BN + (int)rank * BNC;
      // one stage: both CTAs' bytes count on the even CTA's barrier
      auto stage_load = [&](auto&& load) -> bool {
        if (!wait_cl(empty(s), ph ^ 1u, abort_flag)) return false;
        const uint32_t sa = ring + s * STAGE_BYTES;
        if (leader) mbar_expect_tx(full(s), 2 * STAGE_BYTES);
        load(sa, sa + A_BYTES, full0 + 8u * s);
        ++issued;
        if (++s == S) { s = 0; ph ^= 1u; }
        return true;
      };
      // Plane products one after the other; D's two planes side by side at each
      // k-block, so that the other operand's block comes from L2 the second time (a
      // router's dW otherwise reads x twice from memory).
      for (int po = 0; po < outer && ok; ++po) {
        int pa, pb;
        plane_pair(a.planes, po, pa, pb);
        const int d0 = (int)(pa * a.d_plane), d1 = paired ? 0 : d0;   // paired: plane 1, then 0
        const int w0 = (int)(pb * a.w_plane + a.w_v0), x0 = (int)((KIND == kGrad ? pb : pa) * a.x_plane);
        if (KIND != kGrad) {   // (kProduct: one plane)
          for (int k = t.kb0 * BK; k < t.kb1 * BK && ok; k += BK)
            ok = stage_load([&](uint32_t sa, uint32_t sb, uint32_t fb) {
              tma_load_2d_pair(sa, &tmX, k, x0 + arow, fb);
              tma_load_2d_pair(sb, &tmW, k, w0 + bcol, fb);
            });
        } else if (t.type == 1) {
          for (int k = t.kb0 * BK; k < t.kb1 * BK && ok; k += BK)
            for (int d = d0, h = 0; h <= (int)paired && ok; ++h, d = d1)
              ok = stage_load([&](uint32_t sa, uint32_t sb, uint32_t fb) {
                tma_load_2d_pair(sa, &tmD, k, d + arow, fb);
                if (a.wide_in) {
                  tma_load_3d_pair(sb, &tmW, 0, w0 + k, bcol / 64, fb);
                } else {
                  tma_load_2d_pair(sb, &tmW, bcol, w0 + k, fb);
                  tma_load_2d_pair(sb + BOX_BYTES, &tmW, bcol + 64, w0 + k, fb);
                }
              });
        } else {
          for (int k = t.kb0 * BK; k < t.kb1 * BK && ok; k += BK)
            for (int d = d0, h = 0; h <= (int)paired && ok; ++h, d = d1)
              ok = stage_load([&](uint32_t sa, uint32_t sb, uint32_t fb) {
                tma_load_3d_pair(sa, &tmDt, 0, d + k, arow / 64, fb);
                if (a.wide_in) {
                  tma_load_3d_pair(sb, &tmX, 0, x0 + k, bcol / 64, fb);
                } else {
                  tma_load_2d_pair(sb, &tmX, bcol, x0 + k, fb);
                  tma_load_2d_pair(sb + BOX_BYTES, &tmX, bcol + 64, x0 + k, fb);
                }
              });
        }
      }
    }
    if (*abort_flag) {
      // Loads still in flight land before the pair goes away.  The odd CTA's count on
      // the even CTA's barriers, which may have stopped expecting them: it waits a
      // thousand times a load's latency instead.
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
    for (int n = 0; ok; ++n) {
      const Tile t = read_tile(n);
      if (t.type < 0) break;
      const int steps = (t.kb1 - t.kb0) * nprod;   // 0 without rows: the epilogue writes zeros
      const uint32_t idesc = IDESC | (t.type == 2 ? IDESC_A_MN : 0u) | (t.type != 0 ? IDESC_B_MN : 0u);
      for (int i0 = 0; i0 < steps && ok; i0 += a.chunk) {
        const int i1 = min(steps, i0 + a.chunk);
        if (!wait_cl(tempty(acc), aph ^ 1u, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)acc * BN;
        for (int i = i0; i < i1; ++i) {
          if (!wait_cl(full(s), ph, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = ring + s * STAGE_BYTES, sb = sa + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = KIND == kGrad && t.type == 2 ? mn_desc(sa + kk * 2048) : sw128_desc(sa + kk * 32);
            const uint64_t bd = KIND == kGrad ? mn_desc(sb + kk * 2048) : sw128_desc(sb + kk * 32);
            mma2(d, ad, bd, idesc, (i != i0 || kk != 0) ? 1u : 0u);
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
  } else if (warp == 2) {
    // ---------------- L2 prefetch of dX's addend ----------------
    // a tile or two ahead of the epilogue, which otherwise waits a DRAM latency
    // for every tile
    const int esz = a.out_f32 ? 4 : 2;
    for (int n = 0;; ++n) {
      Tile t;
      {
        const int slot = n % NSLOT;
        int w = 0;
        if (lane == 0) w = wait_cl(tfill(slot), ((uint32_t)n / NSLOT) & 1u, abort_flag) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, w, 0)) break;
        t = load_slot(slot);
        __syncwarp();
        if (lane == 0) arrive_relaxed(map_to_rank(tdrain(slot), 0));
      }
      if (t.type < 0) break;
      if (KIND == kGrad && t.type == 1 && a.dx_add != nullptr) {
        const int n0 = t.nt * BN;
        // Line by line, not by cp.async.bulk.prefetch.L2: with that, one row an
        // instruction, this warp of one block once in some hundred launches did not
        // come back from it, and the launch never ended.  Its addresses and sizes were
        // multiples of 16 inside the matrix and the wait before it is bounded: the
        // code does not show why, so the instruction is not used.
        const int lines = (min(BN, a.hidden - n0) * esz + 127) / 128;
        for (int r = lane; r < BMC; r += 32) {
          const int64_t row = (int64_t)t.mt * BM + (int64_t)rank * BMC + r;
          if (row < plan.rows) {
            const char* p = reinterpret_cast<const char*>(a.dx_add) + (row * a.hidden + n0) * esz;
            for (int l = 0; l < lines; ++l)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(p + l * 128) : "memory");
          }
        }
      }
    }
  }
  } else {
    // ---------------- epilogue (warps 4..11, both CTAs) ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(EPI_REGS));
    const int q = warp & 3;                 // TMEM lanes 32q .. 32q+31
    const int half = (warp - 4) / 4;        // columns 128 half ..
    const int c_lo = half * (BN / 2);
    const uint32_t stage = smem_u32(s_out + (warp - 4) * STAGE_WARP);
    int acc = 0;
    uint32_t aph = 0, add_ph = 0;
    for (int n = 0;; ++n) {
      // each warp takes the tile for itself: no barrier among the warps
      Tile t;
      {
        const int slot = n % NSLOT;
        int w = 0;
        if (lane == 0) w = wait_cl(tfill(slot), ((uint32_t)n / NSLOT) & 1u, abort_flag) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, w, 0)) break;
        t = load_slot(slot);
        __syncwarp();
        if (lane == 0) arrive_relaxed(map_to_rank(tdrain(slot), 0));
      }
      if (t.type < 0) break;
      const int steps = (t.kb1 - t.kb0) * nprod;
      const int64_t row0 = (int64_t)t.mt * BM + (int64_t)rank * BMC + q * 32;
      const int64_t row = row0 + lane;
      // this lane's row of the tile, 128 columns, summed over the chunks;
      // gradients start from what they are added to, read while the tile's MMAs
      // run
      float f[BN / 2];
#pragma unroll
      for (int j = 0; j < BN / 2; ++j) f[j] = 0.0f;
      const bool is_dx = t.type == 1;
      const int n0 = t.nt * BN + c_lo;
      int nvalid = 0;
      bf16* hout = nullptr;    // rows of dX that go to their tokens: this lane's
      float* fout = nullptr;
      bool wide = true;        // its sectors are aligned
      bool fit = true;
      if (KIND == kGrad) {
        const int64_t nv = (is_dx ? plan.rows : min(a.vcols, a.vocab - a.v0)) - row0;
        nvalid = nv <= 0 ? 0 : (nv >= 32 ? 32 : (int)nv);
        if (is_dx && a.dx_part == nullptr) {
          wide = a.wide_dx;
          if (a.rowmap) {
            const int64_t orow = lane < nvalid ? a.rowmap[row] : 0;
            if (a.out_f32) fout = reinterpret_cast<float*>(a.dx) + orow * a.hidden + n0;
            else hout = reinterpret_cast<bf16*>(a.dx) + orow * a.hidden + n0;
          } else if (a.dx_add != nullptr && nvalid > 0) {
            // the addend by boxes through the slice, like the output (by the lanes'
            // own loads, 32 lines an instruction: 1 % slower at T = 8192)
            const int step = a.out_f32 ? 32 : 64;
#pragma unroll
            for (int c = 0; c < BN / 2; c += 32) {
              if (c % step != 0 || n0 + c >= a.hidden) continue;
              stage_free(lane);
              if (lane == 0) {
                mbar_expect_tx(addend(warp - 4), STAGE_WARP);
                tma_load_2d(stage, &tmAdd, n0 + c, (int)row0, addend(warp - 4));
              }
              int w = 1;
              if (lane == 0) {
                w = wait_cl(addend(warp - 4), add_ph, abort_flag) ? 1 : 0;
                // given up (perhaps for another warp's wait): the box still lands first
                if (!w) wait2_quiet(addend(warp - 4), add_ph);
              }
              add_ph ^= 1u;
              if (!__shfl_sync(0xffffffffu, w, 0)) { fit = false; break; }
              if (a.out_f32) {
#pragma unroll
                for (int j = 0; j < 8; ++j) unpack16(get_piece(stage, lane, j), f + c + 4 * j, (const float*)nullptr);
              } else if (c % 64 == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) unpack16(get_piece(stage, lane, j), f + c + 8 * j, (const bf16*)nullptr);
              }
              __syncwarp();
            }
          }
        }
      }
      if (!fit) break;
      bool ok = true;
#pragma unroll 1
      for (int i0 = 0; i0 < steps; i0 += a.chunk) {
        int w = 1;
        if (lane == 0) w = wait_cl(tfull(acc), aph, abort_flag) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, w, 0);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)acc * BN + c_lo;
#pragma unroll
        for (int c = 0; c < BN / 2; c += 64) {
          uint32_t r0[32], r1[32];
          tmem_ld32(taddr + c, r0);
          tmem_ld32(taddr + c + 32, r1);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            f[c + j] += __uint_as_float(r0[j]);
            f[c + 32 + j] += __uint_as_float(r1[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_relaxed(map_to_rank(tempty(acc), 0));
        acc ^= 1;
        if (acc == 0) aph ^= 1u;
      }
      if (!ok) break;
      if (KIND == kGrad && a.scale != nullptr) {
        const float scale = *a.scale;
#pragma unroll
        for (int j = 0; j < BN / 2; ++j) f[j] *= scale;
      }
      if (KIND == kStats) {
        // maximum of the row over this half of the tile and the sum of e^(z - maximum).
        // The difference is taken before the factor log2 e: a half tile of masked
        // columns has a maximum of -1e10 and more, whose product with log2 e is
        // rounded by more than exponents can be.
        const bool live = row < plan.rows;
        const int64_t col0 = a.v0 + (int64_t)t.nt * BN + c_lo;
        const int64_t left = a.vocab - col0;
        if (left < BN / 2) {
#pragma unroll
          for (int j = 0; j < BN / 2; ++j)
            if (j >= left) f[j] = -INFINITY;
        }
        const int64_t dt = live ? (int64_t)a.target[row] - col0 : -1;
        if (dt >= 0 && dt < BN / 2) {
          float zt = 0.0f;
#pragma unroll
          for (int j = 0; j < BN / 2; ++j) {
            zt = pick(zt, f[j], (int)dt, j);
            f[j] = pick(f[j], -INFINITY, (int)dt, j);   // the target is merged by itself
          }
          a.zt[row] = zt;
        }
        float m4[4] = {f[0], f[1], f[2], f[3]};
#pragma unroll
        for (int j = 4; j < BN / 2; ++j) m4[j & 3] = fmaxf(m4[j & 3], f[j]);
        const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        const float mu = m == -INFINITY ? 0.0f : m;
        float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < BN / 2; ++j) s4[j & 3] += ex2((f[j] - mu) * kLog2e);
        if (live)
          a.stats[(2 * (a.v0 / BN + t.nt) + half) * a.rows_pad + row] =
              make_float2(m, (s4[0] + s4[1]) + (s4[2] + s4[3]));
      } else if (KIND == kDlogit) {
        const bool live = row < plan.rows;
        const int64_t col0 = a.v0 + (int64_t)t.nt * BN + c_lo;
        const int64_t left = a.vocab - col0;
        const int64_t dt = live ? (int64_t)a.target[row] - col0 : -1;
        const float4 ms = live ? a.rowstat[row] : make_float4(0.0f, 1.0f, 0.0f, 0.0f);
        const float gs = live ? a.g[row] / ms.y : 0.0f;
#pragma unroll
        for (int j = 0; j < BN / 2; ++j) f[j] = ex2((f[j] - ms.x) * kLog2e) * gs;
        if (dt >= 0 && dt < BN / 2) {
#pragma unroll
          for (int j = 0; j < BN / 2; ++j) f[j] = pick(f[j], -gs * ms.z, (int)dt, j);
        }
        if (!live || left < BN / 2) {
#pragma unroll
          for (int j = 0; j < BN / 2; ++j) f[j] = live && j < left ? f[j] : 0.0f;
        }
#pragma unroll
        for (int c = 0; c < BN / 2; c += 64) {
          for (int pl = 0; pl < a.d_planes; ++pl) {
            stage_free(lane);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float q[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                q[e] = pl + 1 < a.d_planes ? take_plane(f[c + 8 * j + e]) : f[c + 8 * j + e];
              put_piece(stage, lane, j, pack16(q, (const bf16*)nullptr));
            }
            stage_out(&tmOx, stage, lane, t.nt * BN + c_lo + c, (int)(pl * a.d_plane + row0), false);
          }
        }
      } else if (KIND == kProduct) {
        const int orow = (int)((int64_t)t.sp * a.rows_pad + row0);
#pragma unroll
        for (int c = 0; c < BN / 2; c += 32)
          if (n0 + c < a.vcols && row0 < plan.rows) {
            stage_free(lane);
#pragma unroll
            for (int j = 0; j < 8; ++j) put_piece(stage, lane, j, pack16(f + c + 4 * j, (const float*)nullptr));
            stage_out(&tmOx, stage, lane, n0 + c, orow, false);
          }
      } else if (nvalid > 0) {
        const bool part = is_dx ? a.dx_part != nullptr : a.dw_part != nullptr;
        const CUtensorMap* map = is_dx ? &tmOx : &tmOw;
        if (fout != nullptr) {
#pragma unroll
          for (int c = 0; c < BN / 2; c += 8)
            if (n0 + c < a.hidden && lane < nvalid) store_sector(fout + c, pack_f32(f + c), wide, true);
        } else if (hout != nullptr) {
#pragma unroll
          for (int c = 0; c < BN / 2; c += 16)
            if (n0 + c < a.hidden && lane < nvalid)
              store_sector(hout + c, pack_bf16(f + c), wide && n0 + c + 16 <= a.hidden, n0 + c + 16 <= a.hidden);
        } else if (part || a.out_f32) {
          const int orow = (int)((part ? (int64_t)t.sp * (is_dx ? a.rows_pad : a.dw_pad) : is_dx ? 0 : a.v0) + row0);
#pragma unroll
          for (int c = 0; c < BN / 2; c += 32)
            if (n0 + c < a.hidden) {
              stage_free(lane);
#pragma unroll
              for (int j = 0; j < 8; ++j) put_piece(stage, lane, j, pack16(f + c + 4 * j, (const float*)nullptr));
              stage_out(map, stage, lane, n0 + c, orow, part && is_dx && a.accumulate);
            }
        } else {
          const int orow = (int)((is_dx ? 0 : a.v0) + row0);
#pragma unroll
          for (int c = 0; c < BN / 2; c += 64)
            if (n0 + c < a.hidden) {
              stage_free(lane);
#pragma unroll
              for (int j = 0; j < 8; ++j) put_piece(stage, lane, j, pack16(f + c + 8 * j, (const bf16*)nullptr));
              stage_out(map, stage, lane, n0 + c, orow, false);
            }
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

// out[r] = sum over the splits (in order) of part[s][row], + add[r].
template <typename T>
__global__ void __launch_bounds__(256) reduce_parts_kernel(const float* __restrict__ part, int splits,
                                                           int64_t stride, int64_t rows, int hidden,
                                                           const int32_t* __restrict__ inv,
                                                           const T* __restrict__ add,
                                                           T* __restrict__ out) {
  pdl_trigger();
  pdl_wait();
  const int per_row = hidden / 8;
  const int64_t items = rows * per_row;
  for (int64_t it = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; it < items;
       it += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = it / per_row;
    const int j0 = (int)(it - r * per_row) * 8;
    const int64_t src = inv ? (int64_t)inv[r] : r;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.0f;
    if (src >= 0) {
      for (int s = 0; s < splits; ++s) {
        const float4* p = reinterpret_cast<const float4*>(part + s * stride + src * hidden + j0);
        const float4 u = __ldcs(p), v = __ldcs(p + 1);
        f[0] += u.x; f[1] += u.y; f[2] += u.z; f[3] += u.w;
        f[4] += v.x; f[5] += v.y; f[6] += v.z; f[7] += v.w;
      }
    }
    constexpr int NV = Vec16<T>::N;
#pragma unroll
    for (int h = 0; h < 8 / NV; ++h) {
      if (add) {
        float b[8];
        unpack16(*reinterpret_cast<const uint4*>(add + r * hidden + j0 + h * NV), b, (const T*)nullptr);
#pragma unroll
        for (int e = 0; e < NV; ++e) f[h * NV + e] += b[e];
      }
      *reinterpret_cast<uint4*>(out + r * hidden + j0 + h * NV) = pack16(f + h * NV, (const T*)nullptr);
    }
  }
}

__global__ void __launch_bounds__(256) planes_kernel(const float* __restrict__ src, int64_t ld,
                                                     int64_t rows, int64_t rows_zero, int hidden,
                                                     bf16* __restrict__ dst, int64_t plane) {
  pdl_trigger();
  pdl_wait();
  const int per_row = hidden / 8;
  const int64_t items = rows_zero * per_row;
  for (int64_t it = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; it < items;
       it += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = it / per_row;
    const int j0 = (int)(it - r * per_row) * 8;
    float f[3][8];
    if (r < rows) {
      const float4 u = *reinterpret_cast<const float4*>(src + r * ld + j0);
      const float4 v = *reinterpret_cast<const float4*>(src + r * ld + j0 + 4);
      const float w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = w[e];
#pragma unroll
        for (int p = 0; p < 3; ++p) f[p][e] = take_plane(v);
      }
    } else {
#pragma unroll
      for (int p = 0; p < 3; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[p][e] = 0.0f;
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<uint4*>(dst + (p * plane + r) * hidden + j0) = pack16(f[p], (const bf16*)nullptr);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// bf16 rows of `width` elements, `ld` apart; box 64 x box_rows, 128-byte swizzle.
static bool map_rows(CUtensorMap* m, const void* ptr, int64_t rows, int64_t width, int64_t ld, int box_rows) {
  cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  return encode_fn() != nullptr &&
         encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same rows as {64, rows, width / 64}: one box of 64 rows brings two 64-wide
// column blocks, as the MN-major operand wants them (width a multiple of 64).
static bool map_blocks(CUtensorMap* m, const void* ptr, int64_t rows, int64_t width, int64_t ld) {
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(width / 64)};
  cuuint64_t strides[2] = {(cuuint64_t)ld * 2, 128};
  cuuint32_t box[3] = {64, BK, 2};
  cuuint32_t es[3] = {1, 1, 1};
  return encode_fn() != nullptr &&
         encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output boxes: 32 rows of 128 bytes (64 bf16 or 32 fp32 columns).
static bool map_out(CUtensorMap* m, void* ptr, int64_t rows, int64_t width, bool f32) {
  const int esz = f32 ? 4 : 2;
  cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)width * esz};
  cuuint32_t box[2] = {(cuuint32_t)(128 / esz), 32};
  cuuint32_t es[2] = {1, 1};
  return encode_fn() != nullptr &&
         encode_fn()(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, dims,
                     strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
    const void* fn[4] = {(const void*)linear_kernel<kStats>, (const void*)linear_kernel<kDlogit>,
                         (const void*)linear_kernel<kGrad>, (const void*)linear_kernel<kProduct>};
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

template <int KIND>
static cudaError_t launch(const CUtensorMap& mX, const CUtensorMap& mW, const CUtensorMap& mD,
                          const CUtensorMap& mDt, const CUtensorMap& mOx, const CUtensorMap& mOw,
                          const CUtensorMap& mAdd, const Args& t, int64_t tiles, cudaStream_t st) {
  int mc = 0;
  cudaError_t e = prepare_device(&mc);
  if (e != cudaSuccess) return e;
  if (tiles <= 0) return cudaSuccess;
  if (tiles >= (1ll << 31) - 4 * mc) return cudaErrorInvalidValue;
  const int64_t ncl = tiles < mc ? tiles : mc;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(2 * ncl));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, linear_kernel<KIND>, mX, mW, mD, mDt, mOx, mOw, mAdd, t);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

static unsigned elementwise_grid(int64_t items) {
  int64_t blocks = (items + 255) / 256;
  const int64_t cap = (int64_t)tc_sm_count() * 16;
  return (unsigned)(blocks > cap ? cap : blocks);
}

}  // namespace lin

LinearSplit linear_grad_split(int64_t rows, int64_t vocab, int hidden) {
  // A part longer than a pair's share of the work would leave the other SMs idle
  // at the end: split K until it is at most nine tenths of that share (at least 8
  // k-blocks a part, at most 16 parts, whose fp32 sums the reduction reads back).
  // Not shorter: the long parts start first and run beside the short tiles, so
  // that the reads of one kind overlap the writes of the other (HBM takes 4.1
  // TB/s of writes alone, 6.8 of both).
  const int64_t nth = (hidden + 255) / 256, mtr = (rows + 255) / 256, ntv = (vocab + 255) / 256;
  const int64_t kbv = (vocab + 63) / 64, kbr = (rows + 63) / 64;
  const int64_t total = mtr * nth * kbv + ntv * nth * kbr;
  int64_t part = total * 9 / (76 * 10);
  if (part < 8) part = 8;
  auto splits = [&](int64_t kb) {
    int64_t s = (kb + part - 1) / part;
    return (int)(s < 1 ? 1 : (s > 16 ? 16 : s));
  };
  return {splits(kbv), splits(kbr)};
}

cudaError_t launch_linear_logits(const LogitsArgs& a, cudaStream_t st) {
  using namespace lin;
  CUtensorMap mX, mW;
  if (!map_rows(&mX, a.x, a.planes * a.x_plane, a.hidden, a.x_ld, BMC) ||
      !map_rows(&mW, a.w, (a.planes - 1) * a.w_plane + a.w_rows, a.hidden, a.w_ld, BNC))
    return cudaErrorInvalidValue;
  Args t = {};
  t.hidden = a.hidden;
  t.planes = a.planes;
  t.v0 = a.v0;
  t.w_v0 = a.w_v0;
  t.vcols = a.vcols;
  t.vocab = a.vocab;
  t.nrows = a.nrows;
  t.rows_bound = a.rows_bound;
  t.ctr = a.ctr;
  t.flags = a.flags;
  t.x_plane = a.x_plane;
  t.w_plane = a.w_plane;
  t.d_plane = a.rows_pad;
  t.target = a.target;
  t.stats = a.stats;
  t.zt = a.zt;
  t.rows_pad = a.rows_pad;
  t.rowstat = a.rowstat;
  t.g = a.g;
  // the same chunks for the gradient's logits as for the statistics: with chunks of
  // their own (4096 of K) they differed from them by 1e-5 of their size, which at
  // logits of 1e4 is a third of a probability
  t.chunk = kChunkExact;
  const int64_t tiles = ((a.rows_bound + BM - 1) / BM) * ((a.vcols + BN - 1) / BN);
  if (!a.gradient) return launch<kStats>(mX, mW, mX, mX, mX, mX, mX, t, tiles, st);
  CUtensorMap mO;
  t.d_planes = a.d_planes;
  if (!map_out(&mO, a.d, a.d_planes * a.rows_pad, a.d_ld, false)) return cudaErrorInvalidValue;
  return launch<kDlogit>(mX, mW, mX, mX, mO, mO, mO, t, tiles, st);
}

int linear_product_split(int64_t rows, int64_t cols, int hidden) {
  // few tiles: as many parts of K as the 76 pairs of SMs take in one round, at
  // least 4 k-blocks each, at most 8 (the reader adds them up)
  const int64_t tiles = ((rows + 255) / 256) * ((cols + 255) / 256), kb = (hidden + 63) / 64;
  int64_t s = tiles > 0 ? 76 / tiles : 1;
  s = s < kb / 4 ? s : kb / 4;
  return (int)(s < 1 ? 1 : (s > 8 ? 8 : s));
}

cudaError_t launch_linear_product(const ProductArgs& a, cudaStream_t st) {
  using namespace lin;
  CUtensorMap mX, mW, mO;
  if (!map_rows(&mX, a.x, a.rows, a.hidden, a.x_ld, BMC) || !map_rows(&mW, a.w, a.cols, a.hidden, a.w_ld, BNC) ||
      !map_out(&mO, a.part, a.split * a.rows_pad, a.ld, true))
    return cudaErrorInvalidValue;
  Args t = {};
  t.hidden = a.hidden;
  t.planes = 1;
  t.vcols = a.ld;
  t.vocab = a.cols;
  t.rows_bound = a.rows;
  t.ctr = a.ctr;
  t.flags = a.flags;
  t.rows_pad = a.rows_pad;
  t.ks_dx = a.split;
  t.chunk = kChunkExact;
  const int64_t tiles = ((a.rows + BM - 1) / BM) * ((a.ld + BN - 1) / BN) * a.split;
  return launch<kProduct>(mX, mW, mX, mX, mO, mO, mO, t, tiles, st);
}

cudaError_t launch_linear_grad(const LinearGradArgs& a, cudaStream_t st) {
  using namespace lin;
  CUtensorMap mX, mW, mD, mDt;
  const int64_t drows = (a.planes == kPlanesD2 ? 2 : a.planes) * a.d_plane;
  const int64_t more = a.planes == kPlanesD2 ? 0 : a.planes - 1;   // planes of x and w after the first
  const int64_t xrows = more * a.x_plane + a.x_rows, wrows = more * a.w_plane + a.w_rows;
  const bool wide = a.hidden % 64 == 0;
  if (a.d_ld % 64 || !map_rows(&mD, a.d, drows, a.d_ld, a.d_ld, BMC) || !map_blocks(&mDt, a.d, drows, a.d_ld, a.d_ld))
    return cudaErrorInvalidValue;
  if (wide ? !map_blocks(&mX, a.x, xrows, a.hidden, a.x_ld) || !map_blocks(&mW, a.w, wrows, a.hidden, a.w_ld)
           : !map_rows(&mX, a.x, xrows, a.hidden, a.x_ld, BK) || !map_rows(&mW, a.w, wrows, a.hidden, a.w_ld, BK))
    return cudaErrorInvalidValue;
  Args t = {};
  t.hidden = a.hidden;
  t.planes = a.planes;
  t.v0 = a.v0;
  t.w_v0 = a.w_v0;
  t.vcols = a.vcols;
  t.vocab = a.vocab;
  t.nrows = a.nrows;
  t.rows_bound = a.rows_bound;
  t.ctr = a.ctr;
  t.flags = a.flags;
  t.x_plane = a.x_plane;
  t.w_plane = a.w_plane;
  t.d_plane = a.d_plane;
  t.rows_pad = a.rows_pad;
  t.ks_dx = a.split.dx;
  t.ks_dw = a.split.dw;
  t.wide_in = wide;
  t.out_f32 = a.out_f32;
  t.chunk = a.out_f32 ? kChunkExact : kChunkBf16;
  t.dx_part = a.dx_part;
  t.accumulate = a.accumulate;
  t.dx = a.dx;
  t.rowmap = a.rowmap;
  t.dx_add = a.dx_add;
  t.dw_part = a.dw_part;
  t.dw_pad = a.dw_pad;
  auto aligned32 = [](const void* p) { return ((uintptr_t)p & 31u) == 0; };
  t.wide_dx = a.hidden * (a.out_f32 ? 4 : 2) % 32 == 0 && aligned32(a.dx);
  t.want_dx = a.dx_part != nullptr || a.dx != nullptr;
  t.want_dw = a.dw_part != nullptr || a.dw != nullptr;
  t.scale = a.scale;
  if (a.dx_add && (a.rowmap || a.scale)) return cudaErrorInvalidValue;
  if ((t.want_dx && t.ks_dx > 1 && !a.dx_part) || (t.want_dw && t.ks_dw > 1 && !a.dw_part))
    return cudaErrorInvalidValue;
  const int64_t nth = (a.hidden + BN - 1) / BN;
  const int64_t tiles = (t.want_dx ? ((a.rows_bound + BM - 1) / BM) * nth * t.ks_dx : 0) +
                        (t.want_dw ? ((a.vcols + BN - 1) / BN) * nth * t.ks_dw : 0);
  CUtensorMap mOx = mX, mOw = mX, mAdd = mX;   // not used where nothing goes by box
  if (a.dx_add && !a.dx_part && !map_out(&mAdd, const_cast<void*>(a.dx_add), a.rows_bound > 0 ? a.rows_bound : 1, a.hidden, a.out_f32))
    return cudaErrorInvalidValue;
  if (t.want_dx && (a.dx_part ? !map_out(&mOx, a.dx_part, a.split.dx * a.rows_pad, a.hidden, true)
                              : !map_out(&mOx, a.dx, a.rows_bound > 0 ? a.rows_bound : 1, a.hidden, a.out_f32)))
    return cudaErrorInvalidValue;
  if (t.want_dw && (a.dw_part ? !map_out(&mOw, a.dw_part, a.split.dw * a.dw_pad, a.hidden, true)
                              : !map_out(&mOw, a.dw, a.vocab, a.hidden, a.out_f32)))
    return cudaErrorInvalidValue;
  return launch<kGrad>(mX, mW, mD, mDt, mOx, mOw, mAdd, t, tiles, st);
}

cudaError_t launch_reduce_parts(const float* part, int splits, int64_t part_stride, int64_t rows,
                                int hidden, const int32_t* inv, const void* add, void* out, int out_f32,
                                cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  const unsigned grid = lin::elementwise_grid(rows * (hidden / 8));
  if (out_f32)
    return launch_after(lin::reduce_parts_kernel<float>, grid, 256, 0, st, 1, part, splits, part_stride, rows,
                        hidden, inv, reinterpret_cast<const float*>(add), reinterpret_cast<float*>(out));
  return launch_after(lin::reduce_parts_kernel<bf16>, grid, 256, 0, st, 1, part, splits, part_stride, rows,
                      hidden, inv, reinterpret_cast<const bf16*>(add), reinterpret_cast<bf16*>(out));
}

cudaError_t launch_planes(const float* src, int64_t ld, int64_t rows, int64_t rows_zero, int hidden,
                          void* dst, int64_t plane, cudaStream_t st) {
  if (rows_zero <= 0) return cudaSuccess;
  return launch_after(lin::planes_kernel, lin::elementwise_grid(rows_zero * (hidden / 8)), 256, 0, st, 1, src, ld,
                      rows, rows_zero, hidden, reinterpret_cast<bf16*>(dst), plane);
}

}  // namespace moe
