// muon_small.cu -- the orthogonalised update of matrices whose smaller side is at most
// 128, in one launch: a cluster of up to 16 CTAs holds a matrix from gradient to
// parameter.
//
// X [m, n], m <= 128, is split by columns: a CTA has 256 of them (fp32 matrices: 128), in
// fp32 in the registers of its threads, laid out as TMEM is (a lane a row), and as
// fp16 planes in shared memory for the tensor cores (tcgen05, 128 x 128 and 128 x 256
// products).  A step is
//   P = X_slab X_slab^T in each CTA, summed over the cluster through distributed shared
//       memory (each CTA adds up its share of the rows, in rank order, and hands it to all):  A
//   B = b A + c A A in each CTA,   X_slab <- a X_slab + B X_slab
// with the operand precision of the general path (one fp16 plane, or three products of two
// planes), and X itself in fp32.
//
// Bound by latency: two cluster barriers and three short chains of products a step.  A
// 128 x 2048 matrix takes 55 us; through the general path's 18 launches it took 155.
#include <algorithm>
#include <atomic>

#include "../../include/moe_model.h"
#include "common.cuh"
#include "internal.h"
#include "muon.cuh"
#include "orth.h"
#include "tc_pair.cuh"
#include "tcgen05.cuh"
#include "train.h"

namespace moe {
namespace muon {

using namespace tc;

constexpr int kSide = 128;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kSquare = kSide * kSide * 2;              // an fp16 plane of A or B
constexpr int kPartial = kSide * kSide * 4;             // P, then the planes of B
__host__ __device__ constexpr int slab_of(int planes) { return planes == 2 ? 128 : 256; }
__host__ __device__ constexpr int x_bytes_of(int planes) { return planes * kSide * slab_of(planes) * 2; }
constexpr int smem_of(int planes) { return 1024 + x_bytes_of(planes) + kPartial + planes * kSquare + 256; }
static_assert(smem_of(1) <= 232448 && smem_of(2) <= 232448, "shared memory budget of one CTA");
static_assert(2 * kSquare <= kPartial, "B's planes take P's place");

struct Coefs {
  int32_t steps;
  float c[MOE_ORTH_MAX_STEPS][3];
};

// An operand of 64-column blocks [128 rows][128 bytes], 128-byte swizzle: 16 bytes j of
// row r of block b.
__device__ __forceinline__ uint32_t op_at(uint32_t base, int b, int r, int j) {
  return base + b * (kSide * 128) + r * 128 + ((j ^ (r & 7)) << 4);
}
// The same blocks as an MN-major operand: 64 columns a block, the next 16384 bytes on.
__device__ __forceinline__ uint64_t block_mn_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((kSide * 128) >> 4) << 16;   // next 64 columns
  d |= (uint64_t)(1024 >> 4) << 32;            // next 8 k-rows
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
__host__ __device__ constexpr uint32_t idesc_of(int n, bool b_mn) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kSide >> 4) << 24) | (b_mn ? 1u << 16 : 0u);
}

__device__ __forceinline__ void st4(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ void st2_cluster(uint32_t at, uint32_t x, uint32_t y) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ float4 ld4_cluster(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async;" ::: "memory"); }

// 8 values as planes of fp16.
template <int PLANES>
__device__ __forceinline__ void halves8(const float* f, uint4 (&out)[PLANES]) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 a = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    h[i] = *reinterpret_cast<const uint32_t*>(&a);
    if (PLANES == 2) {
      const float2 v = __half22float2(a);
      const __half2 b = __floats2half2_rn(f[2 * i] - v.x, f[2 * i + 1] - v.y);
      l[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  out[0] = make_uint4(h[0], h[1], h[2], h[3]);
  if (PLANES == 2) out[PLANES - 1] = make_uint4(l[0], l[1], l[2], l[3]);
}

// The staging square: [128][columns] floats, whose columns change places by the row and by
// themselves, so that neither a warp's 32 rows of one column meet in a bank, nor its columns 8
// apart of one row, nor its rows 8 apart of one column.
__device__ __forceinline__ int row_turn(int r) { return (r & 31) ^ ((r >> 5) & 3); }
__device__ __forceinline__ int col_turn(int c) { return c ^ ((c >> 5) & 7); }
template <int COLS>
__device__ __forceinline__ float* square_at(float* s, int r, int c) { return s + r * COLS + (col_turn(c) ^ row_turn(r)); }

// Eight elements that lie side by side in memory: of row `line` of X from column `place`,
// or, where X is the transposed matrix, of column `line` from row `place` (a multiple of 8).
// Their places in the square, e = 0 .. 7, without the turns worked out for each.
template <int COLS, bool TALL>
struct Places {
  float* p;
  int turn;
  __device__ __forceinline__ Places(float* s, int line, int place) {
    if (TALL) {
      p = s + place * COLS;
      turn = col_turn(line) ^ row_turn(place);       // row_turn(place + e) = row_turn(place) ^ e
    } else {
      turn = col_turn(place) ^ row_turn(line);       // col_turn(place + e) = col_turn(place) ^ e
      p = s + line * COLS;
    }
  }
  __device__ __forceinline__ float& operator[](int e) const { return TALL ? p[e * COLS + (turn ^ e)] : p[turn ^ e]; }
};

template <int PLANES>
__global__ void __launch_bounds__(kThreads, 1) small_kernel(const __grid_constant__ Round r,
                                                            const __grid_constant__ Coefs k, int cols_of, int ctas,
                                                            uint32_t* flags) {
  constexpr int SLAB = slab_of(PLANES), MINE = SLAB / 4, XP = kSide * SLAB * 2;   // XP: a plane of X
  static_assert(kSide * SLAB * 4 <= x_bytes_of(PLANES) + kPartial, "the staging square lies over X's planes and P");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* square = reinterpret_cast<float*>(smem);
  unsigned char* s_p = smem + x_bytes_of(PLANES);
  unsigned char* s_a = s_p + kPartial;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_a + PLANES * kSquare);
  double* sums = reinterpret_cast<double*>(bars + 2);          // of the warps, then the CTA's
  float2* factor = reinterpret_cast<float2*>(sums + kWarps + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(factor + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = ctas > 1 ? (int)cluster_rank() : 0;
  const uint32_t xs = smem_u32(smem), ps = smem_u32(s_p), as = smem_u32(s_a), bar = smem_u32(bars);
  if (tid == 0) {
    mbar_init(bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    proxy_fence();
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // A's rows and columns past m stay zero
  for (int i = tid; i < PLANES * kSquare / 16; i += kThreads) st4(as + 16 * i, make_uint4(0, 0, 0, 0));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t d_gram = tmem, d_poly = tmem + 128, d_apply = tmem + 256;
  pdl_wait();

  const int b = (int)blockIdx.x / ctas;
  const Seg& s = seg_of(r, b);
  const bool tall = s.rows > s.cols;
  const int64_t base = (s.first + (b - s.at)) * (int64_t)s.rows * s.cols;
  const int col0 = rank * cols_of, cols = max(0, min(cols_of, r.n - col0));   // of this CTA
  const bool ok8 = s.cols % 8 == 0 && aligned(s.grad) && aligned(s.momentum) && aligned(s.param);
  // 8 elements of this CTA's columns as memory has them: `line` (a row of X, or a column
  // where it is tall) and 8 places from `place`; n of them exist
  struct Piece {
    int64_t at;
    int line, place, n;
  };
  constexpr int PIECES = kSide * SLAB / 8 / kThreads, BATCH = 4;
  auto piece = [&](int it) {
    Piece p;
    const int i = it * kThreads + tid;
    if (tall) {
      p.line = i / 16;
      p.place = i % 16 * 8;
      p.n = p.line < cols ? min(8, r.m - p.place) : 0;
      p.at = base + (int64_t)(col0 + p.line) * s.cols + p.place;
    } else {
      p.line = i / (SLAB / 8);
      p.place = i % (SLAB / 8) * 8;
      p.n = p.line < r.m ? min(8, cols - p.place) : 0;
      p.at = base + (int64_t)p.line * s.cols + col0 + p.place;
    }
    return p;
  };
  auto to_square = [&](const Piece& p, const float* f) {
    if (tall) {
      const Places<SLAB, true> at(square, p.line, p.place);
#pragma unroll
      for (int e = 0; e < 8; ++e) at[e] = f[e];
    } else {
      const Places<SLAB, false> at(square, p.line, p.place);
#pragma unroll
      for (int e = 0; e < 8; ++e) at[e] = f[e];
    }
  };
  auto from_square = [&](const Piece& p, float* f) {
    if (tall) {
      const Places<SLAB, true> at(square, p.line, p.place);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = at[e];
    } else {
      const Places<SLAB, false> at(square, p.line, p.place);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = at[e];
    }
  };
  // All threads of the matrix (the cluster barrier is for whole warps).
  auto meet = [&]() {
    __syncwarp();
    if (ctas > 1) cluster_sync();
    else __syncthreads();
  };
  const int row = 32 * (warp & 3) + lane, part = warp >> 2;   // this thread's row, and MINE columns of it
  float x[MINE];
  float sum = 0.0f;
  // where pieces are whole (or not there) and on 16-byte boundaries, a batch's reads go out
  // together, before anything looks at their values
  const bool small_g = s.gdtype == MOE_BF16, moves = s.momentum != nullptr;
#pragma unroll 1
  for (int i0 = 0; i0 < PIECES; i0 += BATCH) {
    float g[BATCH][8], v[BATCH][8];
    if (ok8) {
      uint4 a[BATCH][2], c[BATCH][2];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const Piece p = piece(i0 + i);
        a[i][0] = a[i][1] = c[i][0] = c[i][1] = make_uint4(0, 0, 0, 0);
        if (p.n > 0) {
          const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(s.grad) + p.at * (small_g ? 2 : 4));
          a[i][0] = q[0];
          if (!small_g) a[i][1] = q[1];
          if (moves) {
            c[i][0] = reinterpret_cast<const uint4*>(s.momentum + p.at)[0];
            c[i][1] = reinterpret_cast<const uint4*>(s.momentum + p.at)[1];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        if (small_g) {
          unpack16(a[i][0], g[i], (const bf16*)nullptr);
        } else {
          unpack16(a[i][0], g[i], (const float*)nullptr);
          unpack16(a[i][1], g[i] + 4, (const float*)nullptr);
        }
        unpack16(c[i][0], v[i], (const float*)nullptr);
        unpack16(c[i][1], v[i] + 4, (const float*)nullptr);
      }
    } else {
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const Piece p = piece(i0 + i);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[i][e] = v[i][e] = 0.0f;
        if (p.n > 0) {
          read8(s.grad, s.gdtype, p.at, p.n, false, g[i]);
          if (moves) read8(s.momentum, MOE_F32, p.at, p.n, false, v[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const Piece p = piece(i0 + i);    // (what is not there was read as zeros)
      if (moves) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[i][e] = fmaf(r.beta, v[i][e], r.rest * g[i][e]);
          g[i][e] = direction(r, g[i][e], v[i][e]);
        }
        if (p.n > 0) write8(s.momentum, MOE_F32, p.at, p.n, ok8, v[i]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(g[i][e], g[i][e], sum);
      to_square(p, g[i]);
    }
  }
  // squares as in the general path: in fp32 over a warp's elements, once more and scaled
  // where they leave the range, in fp64 beyond
  {
    auto over = [](float v) {
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    };
    auto scaled = [&](float scale) {
      float t = 0.0f;
      for (int i = 0; i < PIECES; ++i) {
        float f[8];
        from_square(piece(i), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = f[e] * scale;
          t = fmaf(v, v, t);
        }
      }
      return over(t);
    };
    float total = over(sum);
    double unit = 1.0;
    if (!(total >= 1e-28f)) {
      total = scaled(0x1p80f);
      unit = 0x1p-160;
    } else if (!(total <= 1e38f)) {
      total = scaled(0x1p-96f);
      unit = 0x1p192;
    }
    if (lane == 0) sums[warp] = (double)total * unit;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < MINE; ++j) x[j] = *square_at<SLAB>(square, row, part * MINE + j);
  if (warp == 0) {
    double t = lane < kWarps ? sums[lane] : 0.0;
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) sums[kWarps] = t;
  }
  meet();
  if (warp == 0) {
    double t = 0.0;
    if (lane < ctas)
      asm volatile("ld.shared::cluster.f64 %0, [%1];"
                   : "=d"(t)
                   : "r"(map_to_rank(smem_u32(sums + kWarps), (uint32_t)lane))
                   : "memory");
#pragma unroll
    for (int o = kMaxCluster / 2; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) *factor = scale_of(t, r.eps);
  }
  __syncthreads();
  {
    const float2 f = *factor;
#pragma unroll
    for (int j = 0; j < MINE; ++j) x[j] = x[j] * f.x * f.y;
  }

  uint32_t phase = 0;
  // Products issued by one thread, waited for by all.
  auto multiply = [&](auto issue) {
    proxy_fence();          // this thread's writes of operands
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      issue();
      tc_commit(bar);
    }
    mbar_wait(bar, phase & 1u, abort_flag);
    phase ^= 1u;
    __syncwarp();           // each lane polls its own way out; what follows is for whole warps
    tc_fence_after();
  };
  auto put_x = [&]() {
#pragma unroll
    for (int j = 0; j < MINE / 8; ++j) {
      uint4 v[PLANES];
      halves8<PLANES>(x + 8 * j, v);
      const int c = part * MINE / 8 + j;
#pragma unroll
      for (int p = 0; p < PLANES; ++p) st4(op_at(xs + p * XP, c / 8, row, c % 8), v[p]);
    }
  };
  // the products of planes above 2^-22, smallest first
  constexpr int PRODUCTS = PLANES == 2 ? 3 : 1;
  auto plane_a = [](int i) { return PRODUCTS == 3 && i == 0 ? 1 : 0; };
  auto plane_b = [](int i) { return PRODUCTS == 3 && i == 1 ? 1 : 0; };
  const int blocks = (cols + 63) / 64;       // of X with columns
  put_x();
  for (int step = 0; step < k.steps; ++step) {
    const float ca = k.c[step][0], cb = k.c[step][1], cc = k.c[step][2];
    // P = X X^T over this CTA's columns
    multiply([&]() {
      uint32_t more = 0;
      for (int i = 0; i < PRODUCTS; ++i)
        for (int q = 0; q < blocks * 4; ++q, more = 1) {
          const uint32_t at = xs + (q / 4) * (kSide * 128) + (q % 4) * 32;
          tc_mma(d_gram, sw128_desc(at + plane_a(i) * XP), sw128_desc(at + plane_b(i) * XP), idesc_of(128, false), more);
        }
    });
    // row `row`, 32 columns, to the partial square in units of 16 bytes (turned by the row)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t v[16];
      tmem_ld16(d_gram + ((uint32_t)(32 * (warp & 3)) << 16) + part * 32 + 16 * c, v);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int unit = part * 8 + 4 * c + j;
        const uint4 w = blocks > 0 ? make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]) : make_uint4(0, 0, 0, 0);
        st4(ps + row * 512 + ((unit ^ (row & 31)) << 4), w);
      }
    }
    meet();
    // This CTA's rows of A: the partial squares in rank order, to every CTA.  What goes
    // between SMs takes the longest of a step (some 14 bytes a clock into an SM); with the units
    // that reach the diagonal alone, and the other side filled in by each CTA, it took as long.
    {
      const int share = (kSide + ctas - 1) / ctas, r0 = rank * share, r1 = min(r.m, r0 + share);
      for (int it = tid; it < (r1 - r0) * 32; it += kThreads) {
        const int rr = r0 + it / 32, unit = it % 32;       // 4 columns
        const uint32_t from = ps + rr * 512 + ((unit ^ (rr & 31)) << 4);
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (ctas == 1) {
          const uint4 u = ld4(from);
          f[0] = __uint_as_float(u.x);
          f[1] = __uint_as_float(u.y);
          f[2] = __uint_as_float(u.z);
          f[3] = __uint_as_float(u.w);
        } else {
          for (int q0 = 0; q0 < ctas; q0 += 8) {
            float4 u[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              u[q] = q0 + q < ctas ? ld4_cluster(map_to_rank(from, (uint32_t)(q0 + q))) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              f[0] += u[q].x; f[1] += u[q].y; f[2] += u[q].z; f[3] += u[q].w;
            }
          }
        }
        uint32_t h[2], l[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f0 = f[2 * e] * 0x1p-15f, f1 = f[2 * e + 1] * 0x1p-15f;    // 2^(kOrthA - 2 kOrthX)
          const __half2 a = __floats2half2_rn(f0, f1);
          const float2 lead = __half22float2(a);
          const __half2 c = __floats2half2_rn(f0 - lead.x, f1 - lead.y);
          h[e] = *reinterpret_cast<const uint32_t*>(&a);
          l[e] = *reinterpret_cast<const uint32_t*>(&c);
        }
        const uint32_t to = op_at(as, unit / 16, rr, unit % 16 / 2) + (unit & 1) * 8;
        for (int q = 0; q < ctas; ++q) {
          const uint32_t at = map_to_rank(to, (uint32_t)q);
          st2_cluster(at, h[0], h[1]);
          if (PLANES == 2) st2_cluster(at + kSquare, l[0], l[1]);
        }
      }
      proxy_fence();
    }
    meet();
    // B = b A + c A A
    multiply([&]() {
      uint32_t more = 0;
      for (int i = 0; i < PRODUCTS; ++i)
        for (int q = 0; q < 8; ++q, more = 1) {
          const uint32_t at = as + (q / 4) * (kSide * 128) + (q % 4) * 32;
          tc_mma(d_poly, sw128_desc(at + plane_a(i) * kSquare), sw128_desc(at + plane_b(i) * kSquare), idesc_of(128, false), more);
        }
    });
    const float kb = cb * 0.25f, kc = cc * 0x1p-13f;     // 2^(kOrthB - kOrthA), 2^(kOrthB - 2 kOrthA)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t v[16];
      tmem_ld16(d_poly + ((uint32_t)(32 * (warp & 3)) << 16) + part * 32 + 16 * c, v);
      tmem_wait_ld();
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int j = part * 4 + 2 * c + g;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.0f;
#pragma unroll
        for (int p = PLANES - 1; p >= 0; --p) {
          const uint4 h = ld4(op_at(as + p * kSquare, j / 8, row, j % 8));
          const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
            f[2 * e] += y.x;
            f[2 * e + 1] += y.y;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fmaf(kc, __uint_as_float(v[8 * g + e]), kb * f[e]);
        uint4 o[PLANES];
        halves8<PLANES>(f, o);
#pragma unroll
        for (int p = 0; p < PLANES; ++p) st4(op_at(ps + p * kSquare, j / 8, row, j % 8), o[p]);
      }
    }
    // X = a X + B X
    multiply([&]() {
      uint32_t more = 0;
      for (int i = 0; i < PRODUCTS; ++i)
        for (int q = 0; q < 8; ++q, more = 1)
          tc_mma(d_apply, sw128_desc(ps + plane_a(i) * kSquare + (q / 4) * (kSide * 128) + (q % 4) * 32),
                 block_mn_desc(xs + plane_b(i) * XP + q * 2048), idesc_of(SLAB, true), more);
    });
#pragma unroll
    for (int c = 0; c < MINE / 16; ++c) {
      uint32_t v[16];
      tmem_ld16(d_apply + ((uint32_t)(32 * (warp & 3)) << 16) + part * MINE + 16 * c, v);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) x[16 * c + e] = fmaf(0x1p-9f, __uint_as_float(v[e]), ca * x[16 * c + e]);
    }
    if (step + 1 < k.steps) put_x();
  }
  static_assert(kOrthX == 13 && kOrthA == 11 && kOrthB == 9, "the powers of two above");

  // the update, through the square again (the last product has read X's planes)
  __syncthreads();
#pragma unroll
  for (int j = 0; j < MINE; ++j) *square_at<SLAB>(square, row, part * MINE + j) = x[j] * 0x1p-13f;
  __syncthreads();
#pragma unroll 1
  for (int i0 = 0; i0 < PIECES; i0 += BATCH) {
    float w[BATCH][8];
    if (ok8) {
      const bool small_w = s.pdtype == MOE_BF16;
      uint4 a[BATCH][2];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const Piece p = piece(i0 + i);
        a[i][0] = a[i][1] = make_uint4(0, 0, 0, 0);
        if (p.n > 0 && r.update) {
          const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(s.param) + p.at * (small_w ? 2 : 4));
          a[i][0] = q[0];
          if (!small_w) a[i][1] = q[1];
        }
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        if (small_w) {
          unpack16(a[i][0], w[i], (const bf16*)nullptr);
        } else {
          unpack16(a[i][0], w[i], (const float*)nullptr);
          unpack16(a[i][1], w[i] + 4, (const float*)nullptr);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const Piece p = piece(i0 + i);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[i][e] = 0.0f;
        if (p.n > 0 && r.update) read8(s.param, s.pdtype, p.at, p.n, false, w[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const Piece p = piece(i0 + i);
      if (p.n <= 0) continue;
      float f[8];
      from_square(p, f);
      if (r.update)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fmaf(-s.size, f[e], r.keep * w[i][e]);
      write8(s.param, s.pdtype, p.at, p.n, ok8, f);
    }
  }
  if (*abort_flag) {
    // a product that never ended: long enough for it to be over before TMEM goes
    const long long t0 = clock64();
    while (clock64() - t0 < (1 << 21)) {}
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_flag(flags, kFlagTimeout);
  meet();   // no CTA leaves while its shared memory may be read
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// CTAs of a matrix: a power of two.
static int ctas_of(int n, int planes) {
  int c = 1;
  while (c * slab_of(planes) < n) c *= 2;
  return c;
}

static std::atomic<int> g_most[2][64];   // CTAs of the largest cluster that runs, + 1

// Shared memory and cluster sizes of this device, found out once.
static cudaError_t prepare(int planes, int* most) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::atomic<int>& slot = g_most[planes - 1][dev];
  if (slot == 0) {
    const void* f = planes == 2 ? (const void*)small_kernel<2> : (const void*)small_kernel<1>;
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(planes));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    int found = 1;
    for (int c = kMaxCluster; c > 1 && found == 1; c /= 2) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = c;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(c);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = smem_of(planes);
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, f, &cfg);
      if (e != cudaSuccess) return e;
      if (n > 0) found = c;
    }
    slot = found + 1;
  }
  *most = slot.load() - 1;
  return cudaSuccess;
}

}  // namespace muon

bool muon_small_fits(int m, int n, int planes) {
  return m <= muon::kSide && muon::ctas_of(n, planes) <= muon::kMaxCluster;
}

cudaError_t launch_muon_small(const muon::Round& r, int planes, int steps, const double (*coef)[3], uint32_t* flags,
                              cudaStream_t st) {
  using namespace muon;
  int most = 0;
  cudaError_t e = prepare(planes, &most);
  if (e != cudaSuccess) return e;
  const int ctas = ctas_of(r.n, planes);
  if (ctas > most) return cudaErrorNotSupported;
  const int cols = ((r.n + ctas - 1) / ctas + 7) / 8 * 8;   // of a CTA
  Coefs k = {};
  k.steps = steps;
  for (int i = 0; i < steps; ++i)
    for (int j = 0; j < 3; ++j) k.c[i][j] = (float)coef[i][j];
  const unsigned grid = (unsigned)(r.batch * ctas);
  if (planes == 2)
    return launch_after(small_kernel<2>, grid, kThreads, smem_of(2), st, (unsigned)ctas, r, k, cols, ctas, flags);
  return launch_after(small_kernel<1>, grid, kThreads, smem_of(1), st, (unsigned)ctas, r, k, cols, ctas, flags);
}

}  // namespace moe
