// block_norm.cu -- the norms before and after a block with its gate and residual,
// forward and backward (include/moe_model.h).
//
//   u = y r1 (w_post + o),  s = residual_scale x + g u,  h = s r2 (w_pre + o)
//
// The forward reads two rows a token and writes two, the backward reads four and
// writes two (s is not read back: from x and y it costs a few FMAs, and it has not been
// rounded).  At 8192 rows of 7168 columns in bf16 that takes 74 us (470 MB, 6.4 TB/s: 94 % of
// the rate of a copy) and 142 us (705 MB, 5.0 TB/s: 73 %), by the rings below; few rows are
// bound by latency (one row of 2048: 4.5 us on the device).  1 / sqrt by rsqrtf, within two
// units of fp32's last place: exactly rounded root and quotient, in every thread for its row,
// cost 4 % of the forward.  A group of threads holds a whole row in
// registers, eight columns and their multiples a thread, so that both norms of the
// forward, and both row sums of the backward, come from one read.  Sums in fp32.
//
// The sums over tokens (dw_post, dgate of a channel gate, dw_pre) stay in the
// registers of the thread that owns the columns, over the rows its group meets (at
// most kFlush of them in one sum), go to the workspace, and a second kernel adds
// the groups' sums in a fixed order.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>

#include "../../include/moe_model.h"
#include "../../include/moe_testing.h"
#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"
#include "train.h"

namespace moe {
namespace bn {

constexpr int kFlush = 128;        // rows that one fp32 sum of a column takes
constexpr int kMaxWarps = 32;

struct NShape {
  int64_t T;
  int H, dtype, esize, gate;
  float off, res, eps;
};

// 8 columns of a row, as they stand in memory
template <typename T>
struct Eight {
  uint4 v[8 / Vec16<T>::N];
};
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p) {
  Eight<T> r;
#pragma unroll
  for (int i = 0; i < 8 / Vec16<T>::N; ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ Eight<T> zero8() {
  Eight<T> r;
#pragma unroll
  for (int i = 0; i < 8 / Vec16<T>::N; ++i) r.v[i] = make_uint4(0, 0, 0, 0);
  return r;
}
template <typename T>
__device__ __forceinline__ void open8(const Eight<T>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 8 / Vec16<T>::N; ++i) unpack16(r.v[i], f + i * Vec16<T>::N, (const T*)nullptr);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* f) {
#pragma unroll
  for (int i = 0; i < 8 / Vec16<T>::N; ++i)
    reinterpret_cast<uint4*>(p)[i] = pack16(f + i * Vec16<T>::N, (const T*)nullptr);
}

// Threads of a row: G, with a power of two up to 32 or whole warps beyond, so that
// the lanes of a sum are G apart from the next row's.  NG rows a block.
struct Geometry {
  int G, NG, vpt;
};
Geometry geometry(int H) {
  const int vecs = H / 8;
  Geometry g;
  if (vecs <= 32) {
    g.vpt = 1;
    g.G = 4;
    while (g.G < vecs) g.G *= 2;
  } else {
    g.vpt = vecs <= 512 ? 1 : (vecs <= 1024 ? 2 : 4);
    g.G = ((vecs + g.vpt - 1) / g.vpt + 31) / 32 * 32;
  }
  g.NG = std::max(1, 256 / g.G);
  return g;
}

// Sum over a row's threads, the same in all of them.  G > 32: red holds a value a
// warp, `slot` alternates so that one barrier a sum is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int G, float (*red)[N][kMaxWarps], int& slot) {
  const int span = G < 32 ? G : 32;
  for (int o = span >> 1; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (G <= 32) return;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[slot][i][warp] = v[i];
  __syncthreads();
  const int first = (threadIdx.x / G) * (G >> 5);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = 0.0f;
    for (int w = 0; w < (G >> 5); ++w) t += red[slot][i][first + w];
    v[i] = t;
  }
  slot ^= 1;
}

template <typename T, int VPT>
__global__ void __launch_bounds__(1024) norm_forward_kernel(int64_t rows, int H, int G, int NG, int kind, float off,
                                                            float res, float eps, const T* x, const T* __restrict__ y,
                                                            const T* __restrict__ w_post, const void* __restrict__ gate,
                                                            const T* __restrict__ w_pre, T* s, T* __restrict__ h,
                                                            float2* __restrict__ rstd) {
  __shared__ float red[2][1][kMaxWarps];
  pdl_trigger();
  pdl_wait();
  const int g = threadIdx.x / G, lane = threadIdx.x - g * G;
  int slot = 0;
  const float inv_h = 1.0f / (float)H;
  // weights stay in registers over the rows
  Eight<T> wp[VPT], wg[VPT], wq[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (lane + v * G) * 8;
    const bool live = c < H;
    wp[v] = live && w_post ? load8<T>(w_post + c) : zero8<T>();
    wg[v] = live && kind == MOE_GATE_CHANNEL ? load8<T>(static_cast<const T*>(gate) + c) : zero8<T>();
    wq[v] = live && w_pre ? load8<T>(w_pre + c) : zero8<T>();
  }
  for (int64_t base = (int64_t)blockIdx.x * NG; base < rows; base += (int64_t)gridDim.x * NG) {
    const int64_t t = base + g;
    const bool on = t < rows;
    Eight<T> ux[VPT], uy[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (lane + v * G) * 8;
      ux[v] = on && c < H ? load8<T>(x + t * H + c) : zero8<T>();
      uy[v] = on && c < H && y ? load8<T>(y + t * H + c) : zero8<T>();
    }
    float gt = 1.0f;
    if (kind == MOE_GATE_TOKEN && on) gt = static_cast<const float*>(gate)[t];
    float r1 = 1.0f;
    if (w_post) {
      float sum[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        float f[8];
        open8<T>(uy[v], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = fmaf(f[e], f[e], sum[0]);
      }
      row_sum<1>(sum, G, red, slot);
      r1 = rsqrtf(sum[0] * inv_h + eps);
    }
    float f[VPT][8];
    float sum[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float fy[8], w[8];
      open8<T>(ux[v], f[v]);
      open8<T>(uy[v], fy);
      if (w_post) {
        open8<T>(wp[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) fy[e] = fy[e] * r1 * (w[e] + off);
      }
      if (kind == MOE_GATE_CHANNEL) {
        open8<T>(wg[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) fy[e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[v][e] = y ? fmaf(res, f[v][e], gt * fy[e]) : res * f[v][e];
        sum[0] = fmaf(f[v][e], f[v][e], sum[0]);
      }
    }
    float r2 = 0.0f;
    if (w_pre) {
      row_sum<1>(sum, G, red, slot);
      r2 = rsqrtf(sum[0] * inv_h + eps);
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (lane + v * G) * 8;
      if (!on || c >= H) continue;
      if (s) store8<T>(s + t * H + c, f[v]);
      if (w_pre) {
        float w[8];
        open8<T>(wq[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[v][e] = f[v][e] * r2 * (w[e] + off);
        store8<T>(h + t * H + c, f[v]);
      }
    }
    if (rstd && on && lane == 0) rstd[t] = make_float2(w_post ? r1 : 0.0f, r2);
  }
}


// ---------------------------------------------------------------------------
// Many rows: each team of threads (a row's threads, or a warp with several short
// rows) is fed by bulk copies into a ring of its own, two steps deep, so that the
// next rows are under way while this one's sums wait on each other; the weights
// stand in shared memory.  Held in registers without the ring, a row's loads, two
// row sums and stores followed one another: the forward at T = 4096, H = 2816 took 39 us
// (by the ring 25 then, 18 now), the backward at T = 8192, H = 7168 340 (160 then, 142 now).  x in
// registers a step ahead instead of by the ring: 104 us at 8192 x 7168 forward (84 then, 74 now).
// ---------------------------------------------------------------------------
struct RingShape {
  int G;        // threads of a team (whole warps)
  int Gs, R;    // threads of a row, rows a step: R > 1 within a warp
  int NG;       // teams of a block
  int vpt, depth;
  int smem;
  int per_sm;   // blocks
  long long limit;   // clocks of a wait
};

constexpr int kBarBytes = 512;   // barriers of all teams, 16-byte rows after them

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// Waits for a phase, `limit` clocks at most (0: gives up at once).  A copy that has not come by
// then may still do so: a thousand times its latency, so that it is not in flight when its
// slot is used for something else or the block ends.
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, long long limit) {
  long long t0;
  if (limit > 0) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    t0 = clock64();
    do {
      if (tc::mbar_try_wait(bar, parity)) return true;
    } while (clock64() - t0 <= limit);
  }
  t0 = clock64();
  while (clock64() - t0 < (1 << 21) && !tc::mbar_try_wait(bar, parity)) {}
  return false;
}

// What a team knows of its place.
struct Team {
  int g, tt, row, lane;      // team, thread in it, row of the step, thread in the row
  int G, Gs;
  __device__ __forceinline__ explicit Team(const RingShape& q) : G(q.G), Gs(q.Gs) {
    g = threadIdx.x / G;
    tt = threadIdx.x - g * G;
    row = tt / Gs;
    lane = tt - row * Gs;
  }
  // (Its warps have to be whole: lanes come from loops of their own, a wait or one lane's store.)
  __device__ __forceinline__ void sync() const {
    __syncwarp();
    if (G > 32) asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(G) : "memory");
  }
  // Sums over a row's threads; red: two values a warp of the block, 32 apart.
  __device__ __forceinline__ float sum(float v, float* red, int& slot) const {
    if (Gs < 32) {
      for (int o = Gs >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (Gs == 32) return v;
    const int lane32 = tt & 31, warps = G >> 5;
    float* r = red + slot * 32 + g * warps;
    if (lane32 == 0) r[tt >> 5] = v;
    sync();
    v = lane32 < warps ? r[lane32] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    slot ^= 1;
    return v;
  }
};

// What y and s are multiplied by, to shared memory in fp32: w1 = (w_post + o) g of a
// channel gate, w2 = w_pre + o (opened and combined once instead of in every row).  Of
// each eight columns the first four stand in the first half and the others in the second:
// a thread's eight side by side would put two of every eight lanes in the same banks.
template <typename T>
__device__ __forceinline__ void stage_weights(float* w1, float* w2, const T* w_post, const T* gate, const T* w_pre,
                                              float off, int H) {
  for (int c = threadIdx.x * 8; c < H; c += blockDim.x * 8) {
    float a[8], g[8], b[8];
    open8<T>(w_post ? load8<T>(w_post + c) : zero8<T>(), a);
    open8<T>(gate ? load8<T>(gate + c) : zero8<T>(), g);
    open8<T>(w_pre ? load8<T>(w_pre + c) : zero8<T>(), b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int to = (e >> 2) * (H >> 1) + (c >> 1) + (e & 3);
      w1[to] = (w_post ? a[e] + off : 1.0f) * (gate ? g[e] : 1.0f);
      w2[to] = w_pre ? b[e] + off : 0.0f;
    }
  }
}
// A team's rows: `steps` steps of R rows, NG * R rows apart, through its ring.
template <int STREAMS>
struct Feed {
  const char* src[STREAMS];   // NULL: not loaded
  int rows, first;            // rows in all; the team's first
  int step;                   // rows between a team's steps
  int R, row_bytes, depth;
  long long limit;
  uint32_t ring, bars;        // of the team
  const unsigned char* rows_at;   // the team's ring
  int at;                     // the slot that is read, its wait's parity; kept from step to
  uint32_t parity;            // step, since a division a step was a tenth of the instructions

  __device__ __forceinline__ void init(int64_t all, int bytes, const RingShape& q, int steps, const Team& m,
                                       unsigned char* smem, unsigned char* rings) {
    rows = (int)all;
    R = q.R;
    first = ((int)blockIdx.x * steps * q.NG + m.g) * R;
    step = q.NG * R;
    row_bytes = bytes;
    depth = q.depth;
    limit = q.limit;
    rows_at = rings + (size_t)m.g * depth * STREAMS * R * row_bytes;
    ring = tc::smem_u32(rows_at);
    at = 0;
    parity = 0;
    bars = tc::smem_u32(smem) + 8u * m.g * depth;
    if (m.tt == 0) {
      for (int i = 0; i < depth; ++i) tc::mbar_init(bars + 8u * i, 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
  }
  __device__ __forceinline__ bool wait() const { return ring_wait(bars + 8u * at, parity, limit); }
  __device__ __forceinline__ const unsigned char* here() const { return rows_at + at * STREAMS * R * row_bytes; }
  __device__ __forceinline__ void next() {
    if (++at == depth) {
      at = 0;
      parity ^= 1u;
    }
  }
  // Called by one thread of the team.
  __device__ __forceinline__ void load(int i, int steps, int to_slot) const {
    if (i >= steps) return;
    const int r = first + i * step;
    if (r >= rows) return;
    const int n = min(rows - r, R);
    const uint32_t bytes = (uint32_t)n * row_bytes, bar = bars + 8u * to_slot;
    const uint32_t to = ring + (uint32_t)to_slot * STREAMS * R * row_bytes;
    uint32_t all = 0;
#pragma unroll
    for (int k = 0; k < STREAMS; ++k) all += src[k] ? bytes : 0u;
    tc::mbar_expect_tx(bar, all);
#pragma unroll
    for (int k = 0; k < STREAMS; ++k)
      if (src[k]) bulk_load(to + k * R * row_bytes, src[k] + (int64_t)r * row_bytes, bytes, bar);
  }
  __device__ __forceinline__ void start(int steps) const {
    for (int i = 0; i < depth - 1; ++i) load(i, steps, i);
  }
  // Into the slot of the step before `i`, which every thread has left.
  __device__ __forceinline__ void refill(int i, int steps) const { load(i + depth - 1, steps, (at ? at : depth) - 1); }
};

// What bounds the kernels below, once the ring hides the memory, is the instructions they
// issue: fp32 arithmetic in pairs.
// Eight columns as four pairs.
struct Pairs {
  float2 p[4];
};
template <typename T>
__device__ __forceinline__ Pairs open_pairs(const Eight<T>& r) {
  float f[8];
  open8<T>(r, f);
  Pairs o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = make_float2(f[2 * i], f[2 * i + 1]);
  return o;
}
// Of the staged weights, w the address of the thread's first four, `half` floats between
// the halves.
__device__ __forceinline__ Pairs weight_pairs(const float* w, int half) {
  const float4 a = *reinterpret_cast<const float4*>(w), b = *reinterpret_cast<const float4*>(w + half);
  Pairs o;
  o.p[0] = make_float2(a.x, a.y);
  o.p[1] = make_float2(a.z, a.w);
  o.p[2] = make_float2(b.x, b.y);
  o.p[3] = make_float2(b.z, b.w);
  return o;
}
template <typename T>
__device__ __forceinline__ void store_pairs(T* to, const Pairs& v) {
  const float f[8] = {v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y, v.p[2].x, v.p[2].y, v.p[3].x, v.p[3].y};
  store8<T>(to, f);
}

template <typename T, int VPT>
__global__ void __launch_bounds__(1024, 1) norm_forward_ring_kernel(
    int64_t rows, int H, const RingShape q, int steps, int kind, float off, float res, float eps, const T* x,
    const T* __restrict__ y, const T* __restrict__ w_post, const void* __restrict__ gate, const T* __restrict__ w_pre,
    T* s, T* __restrict__ h, float2* __restrict__ rstd) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float red[2 * 32];
  __shared__ volatile int lost;   // a copy of the block never came
  if (threadIdx.x == 0) lost = 0;
  float* w1 = reinterpret_cast<float*>(smem + kBarBytes);
  float* w2 = w1 + H;
  unsigned char* ring = reinterpret_cast<unsigned char*>(w2 + H);
  const Team m(q);
  Feed<2> f;
  f.init(rows, H * (int)sizeof(T), q, steps, m, smem, ring);
  f.src[0] = reinterpret_cast<const char*>(x);
  f.src[1] = reinterpret_cast<const char*>(y);
  pdl_trigger();
  pdl_wait();
  if (m.tt == 0) f.start(steps);
  stage_weights<T>(w1, w2, w_post, kind == MOE_GATE_CHANNEL ? static_cast<const T*>(gate) : nullptr, w_pre, off, H);
  __syncthreads();
  const float inv_h = 1.0f / (float)H;
  const int half = H >> 1, span = q.Gs * 8, c0 = m.lane * 8;
  int slot = 0;
  bool fed = true, came = true;        // the copies: the block's, this thread's (the polling warp's)
  int t = f.first + m.row;             // the row
  int64_t to = (int64_t)t * H + c0;    // the thread's first column in it
  for (int i = 0; i < steps && t - m.row < rows; ++i, t += f.step, to += (int64_t)f.step * H, f.next()) {
    if (m.tt < 32) {
      came = came && f.wait();
      if (!came) lost = 1;                      // the barrier hands it on to the team
    }
    m.sync();                                   // the step before is behind every thread
    if (m.tt == 0 && came) f.refill(i, steps);  // into its slot
    fed = !lost;
    const bool on = t < rows;
    bool live[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) live[k] = on && c0 + k * span < H;
    const T* bx = reinterpret_cast<const T*>(f.here()) + (size_t)m.row * H + c0;
    const T* by = bx + (size_t)q.R * H;
    float gt = 1.0f;
    if (kind == MOE_GATE_TOKEN && on) gt = static_cast<const float*>(gate)[t];
    Pairs v[VPT];
    float r1 = 1.0f;
    if (w_post) {
      float2 sq = both(0.0f);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        if (!live[k]) continue;
        const Pairs fy = open_pairs<T>(load8<T>(by + k * span));
#pragma unroll
        for (int e = 0; e < 4; ++e) sq = fma2(fy.p[e], fy.p[e], sq);
      }
      r1 = rsqrtf(m.sum(sq.x + sq.y, red, slot) * inv_h + eps);
    }
    if (!fed) r1 = __int_as_float(0x7fc00000);
    const float2 rg = both(r1 * gt), rx = both(fed ? res : r1);
    float2 sq = both(0.0f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (!live[k]) continue;
      v[k] = open_pairs<T>(load8<T>(bx + k * span));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[k].p[e] = mul2(rx, v[k].p[e]);
      if (y) {
        const Pairs fy = open_pairs<T>(load8<T>(by + k * span));
        const Pairs w = weight_pairs(w1 + ((c0 + k * span) >> 1), half);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k].p[e] = fma2(rg, mul2(fy.p[e], w.p[e]), v[k].p[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sq = fma2(v[k].p[e], v[k].p[e], sq);
      if (s) store_pairs<T>(s + to + k * span, v[k]);
    }
    float r2 = 0.0f;
    if (w_pre) {
      r2 = rsqrtf(m.sum(sq.x + sq.y, red, slot) * inv_h + eps);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        if (!live[k]) continue;
        const Pairs w = weight_pairs(w2 + ((c0 + k * span) >> 1), half);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k].p[e] = mul2(v[k].p[e], mul2(both(r2), w.p[e]));
        store_pairs<T>(h + to + k * span, v[k]);
      }
    }
    if (rstd && on && m.lane == 0) rstd[t] = make_float2(w_post ? r1 : 0.0f, r2);
  }
}

struct BwdArgs {
  int64_t rows;
  int H, kind, flushes;
  float off, res;
  const void *ds, *dh, *x, *y, *w_post, *gate, *w_pre;
  const float2* rstd;
  void *dx, *dy;
  float* dgate;      // of a token gate
  float* part;       // [flushes][blocks][2][H] (rings: [blocks][2][H]), or NULL
  uint32_t* flags;
};

// Rows too wide for a ring of two steps beside the weights (fp32 from H = 5792, bf16 from 8200): a
// block a row, held in registers, of which there are too few (four vectors a thread: 32, the rest
// in local memory).  4096 rows: fp32 of 5784 columns by the ring 101 us, of 5792 185, of 7168 213; bf16
// of 8192 by the ring 78 us, of 8200 947, of 16384 1214.
template <typename T, int VPT>
__global__ void __launch_bounds__(VPT == 4 ? 1024 : 512) norm_backward_kernel(const BwdArgs a) {
  __shared__ float red[2][1][kMaxWarps];
  __shared__ float red2[2][2][kMaxWarps];
  pdl_trigger();
  pdl_wait();
  const int G = blockDim.x, H = a.H, lane = threadIdx.x;
  int slot = 0, slot2 = 0;
  const float inv_h = 1.0f / (float)H;
  const T* w_post = static_cast<const T*>(a.w_post);
  const T* w_pre = static_cast<const T*>(a.w_pre);
  const T* ds = static_cast<const T*>(a.ds);
  const T* dh = static_cast<const T*>(a.dh);
  const T* x = static_cast<const T*>(a.x);
  const T* y = static_cast<const T*>(a.y);
  T* dx = static_cast<T*>(a.dx);
  T* dy = static_cast<T*>(a.dy);
  Eight<T> wp[VPT], wg[VPT], wq[VPT];
  float s_e[VPT][8], s_pre[VPT][8];   // of g D yn (g of the token) and dh sn
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = (lane + v * G) * 8;
    const bool live = c < H;
    wp[v] = live && w_post ? load8<T>(w_post + c) : zero8<T>();
    wg[v] = live && a.kind == MOE_GATE_CHANNEL ? load8<T>(static_cast<const T*>(a.gate) + c) : zero8<T>();
    wq[v] = live && w_pre ? load8<T>(w_pre + c) : zero8<T>();
#pragma unroll
    for (int e = 0; e < 8; ++e) s_e[v][e] = s_pre[v][e] = 0.0f;
  }
  int count = 0, flush = 0;
  auto put_sums = [&]() {
    float* p = a.part + ((int64_t)flush * gridDim.x + blockIdx.x) * 2 * H;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (lane + v * G) * 8;
      if (c < H) {
        store8<float>(p + c, s_e[v]);
        store8<float>(p + H + c, s_pre[v]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s_e[v][e] = s_pre[v][e] = 0.0f;
    }
    ++flush;
    count = 0;
  };
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    Eight<T> ux[VPT], uy[VPT], us[VPT], uh[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = (lane + v * G) * 8;
      const bool live = c < H;
      ux[v] = live && w_pre ? load8<T>(x + t * H + c) : zero8<T>();
      uy[v] = live && y ? load8<T>(y + t * H + c) : zero8<T>();
      us[v] = live && ds ? load8<T>(ds + t * H + c) : zero8<T>();
      uh[v] = live && w_pre ? load8<T>(dh + t * H + c) : zero8<T>();
    }
    float2 r = a.rstd[t];
    if (!w_post) r.x = 1.0f;
    float gt = 1.0f;
    if (a.kind == MOE_GATE_TOKEN) gt = static_cast<const float*>(a.gate)[t];
    // D: first the row sum of dh w_pre sn
    float D[VPT][8];
    float c2[1] = {0.0f};
    if (w_pre) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        float fx[8], fy[8], fh[8], w[8];
        open8<T>(ux[v], fx);
        open8<T>(uy[v], fy);
        open8<T>(uh[v], fh);
        if (w_post) {
          open8<T>(wp[v], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) fy[e] = fy[e] * r.x * (w[e] + a.off);
        }
        if (a.kind == MOE_GATE_CHANNEL) {
          open8<T>(wg[v], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) fy[e] *= w[e];
        }
        open8<T>(wq[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float sn = (y ? fmaf(a.res, fx[e], gt * fy[e]) : a.res * fx[e]) * r.y;
          s_pre[v][e] = fmaf(fh[e], sn, s_pre[v][e]);
          const float b = fh[e] * (w[e] + a.off);
          c2[0] = fmaf(b, sn, c2[0]);
          D[v][e] = sn;   // until the sum is there
        }
      }
      row_sum<1>(c2, G, red, slot);
      c2[0] *= inv_h;
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float fs[8], fh[8], w[8];
      open8<T>(us[v], fs);
      if (w_pre) {
        open8<T>(uh[v], fh);
        open8<T>(wq[v], w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          D[v][e] = fmaf(r.y, fmaf(-D[v][e], c2[0], fh[e] * (w[e] + a.off)), fs[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) D[v][e] = fs[e];
      }
      const int c = (lane + v * G) * 8;
      if (dx && c < H) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = a.res * D[v][e];
        store8<T>(dx + t * H + c, o);
      }
    }
    if (!y) { if (a.part && ++count == kFlush) put_sums(); continue; }
    // the block's side: row sums of b yn and of D u
    float c1[2] = {0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float fy[8], w[8], gg[8];
      open8<T>(uy[v], fy);
      open8<T>(wp[v], w);
      open8<T>(wg[v], gg);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float yn = fy[e] * r.x;
        const float wv = w_post ? w[e] + a.off : 1.0f;
        const float gv = a.kind == MOE_GATE_CHANNEL ? gg[e] : gt;
        const float du = D[v][e] * gv, dyn = D[v][e] * yn;
        s_e[v][e] = fmaf(gt, dyn, s_e[v][e]);
        c1[0] = fmaf(du * wv, yn, c1[0]);
        c1[1] = fmaf(dyn, wv, c1[1]);
        D[v][e] = du * wv;
      }
    }
    row_sum<2>(c1, G, red2, slot2);
    if (a.dgate && lane == 0) a.dgate[t] = c1[1];
    c1[0] *= inv_h;
    if (dy) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = (lane + v * G) * 8;
        if (c >= H) continue;
        if (w_post) {
          float fy[8];
          open8<T>(uy[v], fy);
#pragma unroll
          for (int e = 0; e < 8; ++e) D[v][e] = r.x * fmaf(-(fy[e] * r.x), c1[0], D[v][e]);
        }
        store8<T>(dy + t * H + c, D[v]);
      }
    }
    if (a.part && ++count == kFlush) put_sums();
  }
  if (a.part)
    while (flush < a.flushes) put_sums();   // a block with fewer rows adds zeros
}


// Two vectors a thread in 14 warps halve the instructions of the row sums, waits and
// addresses for each element: at 8192 x 7168 160 us when it was measured (142 now) against 172 with
// one vector in 28 warps.  Nothing may spill: beside rings that leave the L1 no room a spilled
// register is an access of L2 (72 registers with a few spills: 195 to 270 us).  One barrier a row
// instead of three, by finishing dy a step later, took as long.
template <typename T, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 896 : 512, 1) norm_backward_ring_kernel(const BwdArgs a, const RingShape q,
                                                                                     int steps) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float red[2 * 32];
  __shared__ volatile int lost;   // a copy of the block never came
  if (threadIdx.x == 0) lost = 0;
  const int H = a.H;
  float* w1 = reinterpret_cast<float*>(smem + kBarBytes);
  float* w2 = w1 + H;
  unsigned char* ring = reinterpret_cast<unsigned char*>(w2 + H);
  const Team m(q);
  const bool with_y = a.y != nullptr, pre = a.w_pre != nullptr, post = a.w_post != nullptr;
  Feed<4> f;
  f.init(a.rows, H * (int)sizeof(T), q, steps, m, smem, ring);
  f.src[0] = static_cast<const char*>(pre ? a.x : nullptr);
  f.src[1] = static_cast<const char*>(a.y);
  f.src[2] = static_cast<const char*>(a.dh);
  f.src[3] = static_cast<const char*>(a.ds);
  T* dx = static_cast<T*>(a.dx);
  T* dy = static_cast<T*>(a.dy);
  pdl_trigger();
  pdl_wait();
  // (false without tokens alone, which need no ds or dh; with the conditions on it the compiler's
  // order of the loop is the better one: 8192 x 7168 142 us, without them 144)
  const bool feeds = pre || with_y || a.ds;
  if (m.tt == 0 && feeds) f.start(steps);
  stage_weights<T>(w1, w2, static_cast<const T*>(a.w_post),
                   a.kind == MOE_GATE_CHANNEL ? static_cast<const T*>(a.gate) : nullptr, static_cast<const T*>(a.w_pre),
                   a.off, H);
  __syncthreads();
  const float inv_h = 1.0f / (float)H;
  int slot = 0;
  bool fed = true, came = true;   // the copies: the block's, this thread's (the polling warp's)
  Pairs c_e[VPT], c_pre[VPT];   // the columns' sums over this team's rows
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) c_e[k].p[e] = c_pre[k].p[e] = both(0.0f);
  const int half = H >> 1, span = q.Gs * 8, c0 = m.lane * 8;
  int t = f.first + m.row;             // the row
  int64_t to = (int64_t)t * H + c0;    // the thread's first column in it
  float2 r_next = make_float2(0.0f, 0.0f);        // a step ahead
  float gate_next = 1.0f;
  auto ask = [&](int row) {
    if (row >= a.rows) return;
    r_next = a.rstd[row];
    if (a.kind == MOE_GATE_TOKEN) gate_next = static_cast<const float*>(a.gate)[row];
  };
  ask(t);
  for (int i = 0; i < steps && t - m.row < a.rows; ++i, t += f.step, to += (int64_t)f.step * H, f.next()) {
    const bool on = t < a.rows;
    bool live[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) live[k] = on && c0 + k * span < H;
    float2 r = r_next;
    const float gt = gate_next;
    ask(t + f.step);
    if (!post) r.x = 1.0f;
    if (m.tt < 32 && feeds) {
      came = came && f.wait();
      if (!came) lost = 1;                               // the barrier hands it on to the team
    }
    m.sync();                                            // the step before is behind every thread
    if (m.tt == 0 && feeds && came) f.refill(i, steps);  // into its slot
    fed = !lost;
    if (!fed) r.x = r.y = __int_as_float(0x7fc00000);
    const T* bx = reinterpret_cast<const T*>(f.here()) + (size_t)m.row * H + c0;
    const T *by = bx + (size_t)q.R * H, *bh = by + (size_t)q.R * H, *bs = bh + (size_t)q.R * H;
    Pairs D[VPT];
    if (pre) {
      float2 sum = both(0.0f);
      // under an eps near fp32's smallest the product of both norms of a row of zeros leaves
      // the range, and infinity times its zeros would be NaN
      float r12 = gt * r.x * r.y;
      r12 = r12 > FLT_MAX ? FLT_MAX : r12 < -FLT_MAX ? -FLT_MAX : r12;
      const float2 rx = both(a.res * r.y), ry = both(r12);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        if (!live[k]) continue;
        D[k] = open_pairs<T>(load8<T>(bx + k * span));
#pragma unroll
        for (int e = 0; e < 4; ++e) D[k].p[e] = mul2(rx, D[k].p[e]);
        if (with_y) {
          const Pairs fy = open_pairs<T>(load8<T>(by + k * span));
          const Pairs w = weight_pairs(w1 + ((c0 + k * span) >> 1), half);
#pragma unroll
          for (int e = 0; e < 4; ++e) D[k].p[e] = fma2(ry, mul2(fy.p[e], w.p[e]), D[k].p[e]);
        }
        const Pairs fh = open_pairs<T>(load8<T>(bh + k * span));
        const Pairs w = weight_pairs(w2 + ((c0 + k * span) >> 1), half);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c_pre[k].p[e] = fma2(fh.p[e], D[k].p[e], c_pre[k].p[e]);
          const float2 b = mul2(fh.p[e], w.p[e]);
          sum = fma2(b, D[k].p[e], sum);   // D is sn until the sum is there
        }
      }
      const float2 mean = both(-m.sum(sum.x + sum.y, red, slot) * inv_h), ry2 = both(r.y);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        if (!live[k]) continue;
        const Pairs fs = open_pairs<T>(a.ds ? load8<T>(bs + k * span) : zero8<T>()), fh = open_pairs<T>(load8<T>(bh + k * span));
        const Pairs w = weight_pairs(w2 + ((c0 + k * span) >> 1), half);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          D[k].p[e] = fma2(ry2, fma2(D[k].p[e], mean, mul2(fh.p[e], w.p[e])), fs.p[e]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
        D[k] = open_pairs<T>(on && c0 + k * span < H && a.ds ? load8<T>(bs + k * span) : zero8<T>());
    }
    // D, and the block's side: the row sum of D yn w1, which is the token gate's
    // gradient too
    float2 sum = both(0.0f);
    const float2 ge = both(gt * r.x);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (!live[k]) continue;
      if (dx) {
        Pairs o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o.p[e] = mul2(both(fed ? a.res : r.x), D[k].p[e]);
        store_pairs<T>(dx + to + k * span, o);
      }
      if (!with_y) continue;
      const Pairs fy = open_pairs<T>(load8<T>(by + k * span));
      const Pairs w = weight_pairs(w1 + ((c0 + k * span) >> 1), half);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c_e[k].p[e] = fma2(mul2(D[k].p[e], ge), fy.p[e], c_e[k].p[e]);
        D[k].p[e] = mul2(D[k].p[e], w.p[e]);
        sum = fma2(D[k].p[e], fy.p[e], sum);
      }
    }
    if (!with_y) continue;
    float c1 = (sum.x + sum.y) * r.x;
    if (post || a.dgate) c1 = m.sum(c1, red, slot);
    if (a.dgate && on && m.lane == 0) a.dgate[t] = c1;
    if (!dy) continue;
    const float2 mine = both(gt * r.x), back = both(post ? -(c1 * (inv_h * r.x)) * (gt * r.x) : 0.0f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (!live[k]) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) D[k].p[e] = mul2(mine, D[k].p[e]);
      if (post) {
        const Pairs fy = open_pairs<T>(load8<T>(by + k * span));
#pragma unroll
        for (int e = 0; e < 4; ++e) D[k].p[e] = fma2(fy.p[e], back, D[k].p[e]);
      }
      store_pairs<T>(dy + to + k * span, D[k]);
    }
  }
  if (!fed && m.tt == 0) set_flag(a.flags, kFlagTimeout);
  if (!a.part) return;
  // The rows' sums of the block in the ring, which no copy fills any more: a thread's
  // columns lie at its own row of its team, then added in that order.
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring);     // [NG][R][2][H]
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int c = (m.lane + k * q.Gs) * 8;
    if (c >= H) continue;
    float* p = sums + (size_t)(m.g * q.R + m.row) * 2 * H + c;
    store_pairs<float>(p, c_e[k]);
    store_pairs<float>(p + H, c_pre[k]);
  }
  __syncthreads();
  float* out = a.part + (int64_t)blockIdx.x * 2 * H;
  for (int c = threadIdx.x * 4; c < 2 * H; c += blockDim.x * 4) {
    float4 v = *reinterpret_cast<const float4*>(sums + c);
    for (int n = 1; n < q.NG * q.R; ++n) {
      const float4 u = *reinterpret_cast<const float4*>(sums + (size_t)n * 2 * H + c);
      v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
    }
    *reinterpret_cast<float4*>(out + c) = v;
  }
}

// The blocks' column sums, added in order: sixteen warps take a part of them each.
// With E = sum_t D yn (times the token's gate): dw_post = gate E, dgate = (w_post + o) E.
constexpr int kJoinWarps = 16;
template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) norm_columns_kernel(const float* __restrict__ part, int64_t n, int H,
                                                                       const T* __restrict__ w_post,
                                                                       const T* __restrict__ gate, float off,
                                                                       T* dw_post, T* dgate, T* dw_pre) {
  __shared__ float sh[kJoinWarps][32];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane, col = c < H ? c : c - H;
  const bool live = c < 2 * H && (c < H ? dw_post != nullptr || dgate != nullptr : dw_pre != nullptr);
  const int64_t each = (n + kJoinWarps - 1) / kJoinWarps, hi = min(n, (warp + 1) * each);
  float f = 0.0f;
  if (live) {
#pragma unroll 8
    for (int64_t i = warp * each; i < hi; ++i) f += __ldcg(part + i * 2 * H + c);
  }
  sh[warp][lane] = f;
  __syncthreads();
  if (warp != 0 || !live) return;
  for (int w = 1; w < kJoinWarps; ++w) f += sh[w][lane];
  if (c >= H) {
    dw_pre[col] = from_f<T>(f);
    return;
  }
  if (dw_post) dw_post[col] = from_f<T>(gate ? f * to_f(gate[col]) : f);
  if (dgate) dgate[col] = from_f<T>(w_post ? f * (to_f(w_post[col]) + off) : f);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
moe_status decode(const moe_block_norm_shape* s, NShape* o, const char** why) {
  *why = "";
  if (!s) { *why = "shape is NULL"; return MOE_ERR_INVALID_ARG; }
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16) { *why = "dtype must be MOE_F32 or MOE_BF16"; return MOE_ERR_UNSUPPORTED; }
  if (s->tokens < 0 || s->tokens > (1ll << 28)) { *why = "tokens must be in [0, 2^28]"; return MOE_ERR_INVALID_ARG; }
  if (s->hidden <= 0 || s->hidden % 8) { *why = "hidden must be a positive multiple of 8"; return MOE_ERR_INVALID_ARG; }
  if (s->hidden > 32768) { *why = "hidden above 32768 is not supported"; return MOE_ERR_UNSUPPORTED; }
  if (s->gate < MOE_GATE_NONE || s->gate > MOE_GATE_TOKEN) { *why = "gate must be a moe_gate_kind"; return MOE_ERR_INVALID_ARG; }
  if (s->unit_offset != 0 && s->unit_offset != 1) { *why = "unit_offset must be 0 or 1"; return MOE_ERR_INVALID_ARG; }
  if (!std::isfinite((float)s->residual_scale)) { *why = "residual_scale must be finite in fp32"; return MOE_ERR_INVALID_ARG; }
  if (!((float)s->eps > 0.0f) || !std::isfinite((float)s->eps)) { *why = "eps must be positive and finite in fp32"; return MOE_ERR_INVALID_ARG; }
  o->T = s->tokens;
  o->H = s->hidden;
  o->dtype = s->dtype;
  o->esize = s->dtype == MOE_F32 ? 4 : 2;
  o->gate = s->gate;
  o->off = (float)s->unit_offset;
  o->res = (float)s->residual_scale;
  o->eps = (float)s->eps;
  return MOE_OK;
}

// Rings for rows of H columns, `streams` of them in and two fp32 weight vectors beside
// them, one vector of 8 columns a thread up to `wide` vectors, at most `threads`
// threads of an SM (two vectors: threads2): as many teams as fit with two steps in their
// rings (three or four steps took as long or longer to start: the forward at 4096 x 2816 with
// three 27 us, with two 25 then and 18 now).  depth 0: none fits.
constexpr int kSmemBlock = 227 * 1024, kSmemSm = 228 * 1024;   // 1 KB of the latter goes with each block
constexpr int kStatic = 512;                                    // what the kernels declare besides
RingShape ring_shape(int H, int esize, int streams, int wide, int threads, int threads2) {
  RingShape q = {};
  const int vecs = H / 8;
  if (vecs <= 32) {
    q.vpt = 1;
    q.Gs = 4;
    while (q.Gs < vecs) q.Gs *= 2;
    q.G = 32;
    q.R = 32 / q.Gs;
  } else {
    q.vpt = vecs <= wide ? 1 : 2;
    q.Gs = q.G = ((vecs + q.vpt - 1) / q.vpt + 31) / 32 * 32;
    q.R = 1;
  }
  const int most_threads = q.vpt == 1 ? threads : threads2;
  const int row = H * esize, weights = kBarBytes + 2 * H * 4;
  const int step = streams * q.R * row;
  int best = 0;
  for (int b = 1; b <= 8; ++b)
    for (int ng = 1; ng <= 15 && b * ng * q.G <= most_threads; ++ng) {
      const int most = std::min(kSmemSm / b - 1024, kSmemBlock) - kStatic;
      const int depth = std::min(2, std::max(0, most - weights) / (ng * step));
      const int smem = std::max(weights + ng * depth * step, weights + ng * q.R * 2 * H * 4);
      if (depth < 2 || smem > most) continue;
      const int score = ng * b * 8 + depth;
      if (score <= best) continue;
      best = score;
      q.NG = ng;
      q.depth = depth;
      q.smem = smem;
      q.per_sm = b;
    }
  return q;
}

// The backward's work split, the same on every device, so that a workspace's size
// and the sums do not depend on it.  Rows in rings, at most kFlush a team; those too wide for
// one, a block each, as they come.
struct Split {
  RingShape q;
  int steps;       // of a team
  int G, vpt;      // without rings: threads, vectors of each
  int64_t blocks;
  int flushes;
};
Split split_of(const NShape& s) {
  Split p = {};
  p.q = ring_shape(s.H, s.esize, 4, 64, 896, 512);
  if (p.q.depth > 0) {
    const int64_t per = (int64_t)p.q.NG * p.q.R;   // rows of a block's step
    const int64_t resident = 152ll * p.q.per_sm;
    const int64_t rows = (s.T + per - 1) / per;
    const int64_t waves = std::max<int64_t>(1, (rows + resident * kFlush - 1) / (resident * kFlush));
    p.steps = (int)std::max<int64_t>(1, (rows + resident * waves - 1) / (resident * waves));
    p.blocks = std::max<int64_t>(1, (rows + p.steps - 1) / p.steps);
    return p;
  }
  const int vecs = s.H / 8;
  p.vpt = s.dtype == MOE_F32 && vecs <= 1024 ? 2 : 4;
  p.G = ((vecs + p.vpt - 1) / p.vpt + 31) / 32 * 32;
  p.blocks = std::max<int64_t>(1, std::min<int64_t>(s.T, p.G > 512 ? 152 : 2 * 152));
  p.flushes = (int)std::max<int64_t>(1, ((s.T + p.blocks - 1) / p.blocks + kFlush - 1) / kFlush);
  return p;
}
int64_t parts_of(const Split& p) { return p.q.depth > 0 ? p.blocks : (int64_t)p.flushes * p.blocks; }
size_t part_bytes(const NShape& s, const Split& p) { return (size_t)parts_of(p) * 2 * s.H * 4; }

std::atomic<int64_t> g_wait{-1};   // moe_testing_set_norm_wait
long long wait_limit() {
  const int64_t v = g_wait.load(std::memory_order_relaxed);
  return v < 0 || v > tc::kWaitCycles ? tc::kWaitCycles : v;
}

template <typename T>
cudaError_t forward(const NShape& s, const void* x, const void* y, const void* w_post, const void* gate,
                    const void* w_pre, void* so, void* h, float* rstd, cudaStream_t st) {
  RingShape q = ring_shape(s.H, s.esize, 2, 64, 1024, 1024);
  q.limit = wait_limit();
  const int64_t per = (int64_t)q.NG * q.R, rows = (s.T + std::max<int64_t>(per, 1) - 1) / std::max<int64_t>(per, 1);
  const int64_t resident = (int64_t)tc_sm_count() * q.per_sm;
  if (q.depth > 0 && rows > 2 * resident) {
    const int steps = (int)((rows + resident - 1) / resident);
    const unsigned grid = (unsigned)((rows + steps - 1) / steps);
    static std::atomic<uint64_t> done[2];
    auto go = [&](auto kernel) {
      const cudaError_t e = allow_smem(kernel, kSmemBlock - kStatic, done[q.vpt - 1]);
      if (e != cudaSuccess) return e;
      return launch_after(kernel, grid, (unsigned)(q.G * q.NG), q.smem, st, 1, s.T, s.H, q, steps, s.gate, s.off, s.res,
                          s.eps, static_cast<const T*>(x), static_cast<const T*>(y), static_cast<const T*>(w_post), gate,
                          static_cast<const T*>(w_pre), static_cast<T*>(so), static_cast<T*>(h),
                          reinterpret_cast<float2*>(rstd));
    };
    return q.vpt == 1 ? go(norm_forward_ring_kernel<T, 1>) : go(norm_forward_ring_kernel<T, 2>);
  }
  const Geometry g = geometry(s.H);
  const unsigned threads = (unsigned)(g.G * g.NG);
  const int64_t need = (s.T + g.NG - 1) / g.NG, cap = (int64_t)tc_sm_count() * std::max(1u, 2048 / threads);
  const unsigned grid = (unsigned)std::min(need, cap);
  auto go = [&](auto kernel) {
    return launch_after(kernel, grid, threads, 0, st, 1, s.T, s.H, g.G, g.NG, s.gate, s.off, s.res, s.eps,
                        static_cast<const T*>(x), static_cast<const T*>(y), static_cast<const T*>(w_post), gate,
                        static_cast<const T*>(w_pre), static_cast<T*>(so), static_cast<T*>(h),
                        reinterpret_cast<float2*>(rstd));
  };
  if (g.vpt == 1) return go(norm_forward_kernel<T, 1>);
  if (g.vpt == 2) return go(norm_forward_kernel<T, 2>);
  return go(norm_forward_kernel<T, 4>);
}

template <typename T>
cudaError_t backward(const NShape& s, const Split& p, BwdArgs a, void* dw_post, void* dgate, void* dw_pre,
                     cudaStream_t st) {
  cudaError_t e;
  if (p.q.depth > 0) {
    static std::atomic<uint64_t> done[2];
    RingShape q = p.q;
    q.limit = wait_limit();
    auto go = [&](auto kernel) {
      const cudaError_t f = allow_smem(kernel, kSmemBlock - kStatic, done[p.q.vpt - 1]);
      if (f != cudaSuccess) return f;
      return launch_after(kernel, (unsigned)p.blocks, (unsigned)(p.q.G * p.q.NG), p.q.smem, st, 1, a, q, p.steps);
    };
    e = p.q.vpt == 1 ? go(norm_backward_ring_kernel<T, 1>) : go(norm_backward_ring_kernel<T, 2>);
  } else {
    a.flushes = p.flushes;
    auto go = [&](auto kernel) { return launch_after(kernel, (unsigned)p.blocks, (unsigned)p.G, 0, st, 1, a); };
    if constexpr (sizeof(T) == 4) e = p.vpt == 2 ? go(norm_backward_kernel<T, 2>) : go(norm_backward_kernel<T, 4>);
    else e = go(norm_backward_kernel<T, 4>);
  }
  if (e != cudaSuccess || !a.part) return e;
  return launch_after(norm_columns_kernel<T>, (unsigned)((2 * s.H + 31) / 32), 32 * kJoinWarps, 0, st, 1,
                      (const float*)a.part, parts_of(p), s.H, static_cast<const T*>(a.w_post),
                      a.kind == MOE_GATE_CHANNEL ? static_cast<const T*>(a.gate) : nullptr, a.off,
                      static_cast<T*>(dw_post), static_cast<T*>(dgate), static_cast<T*>(dw_pre));
}

// What both directions ask of the inputs.
moe_status check_inputs(const NShape& s, const void* x, const void* y, const void* w_post, const void* gate,
                        const void* w_pre) {
  if (!x && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "x must be non-NULL");
  if (!y && (w_post || s.gate != MOE_GATE_NONE) && s.T > 0)
    return fail(MOE_ERR_INVALID_ARG, "w_post and a gate need y");
  const bool empty_gate = s.gate == MOE_GATE_TOKEN && s.T == 0;   // an array of none has no address
  if ((s.gate != MOE_GATE_NONE) != (gate != nullptr || empty_gate))
    return fail(MOE_ERR_INVALID_ARG, "gate must be given iff the shape has one");
  if (!aligned16(x) || !aligned16(y) || !aligned16(w_post) || !aligned16(w_pre) ||
      (s.gate == MOE_GATE_CHANNEL && !aligned16(gate)))
    return fail(MOE_ERR_INVALID_ARG, "x, y, w_post, a channel gate and w_pre must be 16-byte aligned");
  if ((uintptr_t)gate & 3u) return fail(MOE_ERR_INVALID_ARG, "a token gate must be aligned to its elements");
  return MOE_OK;
}

}  // namespace bn
}  // namespace moe

using namespace moe;

#define DECODE_BN(shape, s)                                  \
  bn::NShape s;                                              \
  do {                                                       \
    const char* why_ = "";                                   \
    moe_status st_ = bn::decode(shape, &s, &why_);           \
    if (st_ != MOE_OK) return fail(st_, why_);               \
  } while (0)

extern "C" size_t moe_block_norm_workspace_bytes(const moe_block_norm_shape* shape) {
  bn::NShape s;
  const char* why;
  moe_status st = bn::decode(shape, &s, &why);
  if (st != MOE_OK) {
    fail(st, why);
    return 0;
  }
  return 256 + bn::part_bytes(s, bn::split_of(s));
}

extern "C" moe_status moe_block_norm_forward(const moe_block_norm_shape* shape, const void* x, const void* y,
                                             const void* w_post, const void* gate, const void* w_pre, void* so,
                                             void* h, float* rstd, void* stream) {
  reset_launch_count();
  DECODE_BN(shape, s);
  moe_status e = bn::check_inputs(s, x, y, w_post, gate, w_pre);
  if (e != MOE_OK) return e;
  if ((w_pre != nullptr) != (h != nullptr) && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "h must be given iff w_pre is");
  if (!so && !h && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "one of s and h must be non-NULL");
  if (!aligned16(so) || !aligned16(h)) return fail(MOE_ERR_INVALID_ARG, "s and h must be 16-byte aligned");
  if ((uintptr_t)rstd & 7u) return fail(MOE_ERR_INVALID_ARG, "rstd must be 8-byte aligned");
  if (s.T == 0) return MOE_OK;
  CHECK_CUDA(s.dtype == MOE_F32
                 ? bn::forward<float>(s, x, y, w_post, gate, w_pre, so, h, rstd, (cudaStream_t)stream)
                 : bn::forward<bf16>(s, x, y, w_post, gate, w_pre, so, h, rstd, (cudaStream_t)stream));
  return MOE_OK;
}

extern "C" moe_status moe_block_norm_backward(const moe_block_norm_shape* shape, const void* ds, const void* dh,
                                              const void* x, const void* y, const void* w_post, const void* gate,
                                              const void* w_pre, const float* rstd, void* dx, void* dy, void* dw_post,
                                              void* dgate, void* dw_pre, void* ws, size_t ws_bytes, void* stream) {
  reset_launch_count();
  DECODE_BN(shape, s);
  moe_status e = bn::check_inputs(s, x, y, w_post, gate, w_pre);
  if (e != MOE_OK) return e;
  if ((w_pre != nullptr) != (dh != nullptr) && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "dh must be given iff w_pre is");
  if (!ds && !dh && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "one of ds and dh must be non-NULL");
  if (!rstd && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "rstd must be non-NULL");
  if ((dy && !y && s.T > 0) || (dw_post && !w_post) || (dgate && !gate) || (dw_pre && !w_pre))
    return fail(MOE_ERR_INVALID_ARG, "a gradient's input must be non-NULL");
  if (!dx && !dy && !dw_post && !dgate && !dw_pre && s.T > 0) return fail(MOE_ERR_INVALID_ARG, "no gradient is asked for");
  if (!aligned16(ds) || !aligned16(dh) || !aligned16(dx) || !aligned16(dy))
    return fail(MOE_ERR_INVALID_ARG, "ds, dh, dx and dy must be 16-byte aligned");
  if (((uintptr_t)dw_post | (uintptr_t)dw_pre | (uintptr_t)dgate) & (uintptr_t)(s.esize - 1) ||
      (s.gate == MOE_GATE_TOKEN && ((uintptr_t)dgate & 3u)))
    return fail(MOE_ERR_INVALID_ARG, "dw_post, dgate and dw_pre must be aligned to their elements");
  if ((uintptr_t)rstd & 7u) return fail(MOE_ERR_INVALID_ARG, "rstd must be 8-byte aligned");
  const bn::Split p = bn::split_of(s);
  e = check_ws(ws, ws_bytes, 256 + bn::part_bytes(s, p));
  if (e != MOE_OK) return e;
  const bool channel = s.gate == MOE_GATE_CHANNEL;
  bn::BwdArgs a = {};
  a.rows = s.T;
  a.H = s.H;
  a.kind = s.gate;
  a.off = s.off;
  a.res = s.res;
  a.ds = ds;
  a.dh = dh;
  a.x = x;
  a.y = y;
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.rstd = reinterpret_cast<const float2*>(rstd);
  a.dx = dx;
  a.dy = dy;
  a.dgate = channel ? nullptr : static_cast<float*>(dgate);
  a.flags = static_cast<uint32_t*>(ws);
  // without tokens the columns' sums are zeros, written like any others
  if (dw_post || dw_pre || (channel && dgate)) a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
  if (s.T == 0 && !a.part) return MOE_OK;
  void* dcol = channel ? dgate : nullptr;
  CHECK_CUDA(s.dtype == MOE_F32 ? bn::backward<float>(s, p, a, dw_post, dcol, dw_pre, (cudaStream_t)stream)
                                : bn::backward<bf16>(s, p, a, dw_post, dcol, dw_pre, (cudaStream_t)stream));
  return MOE_OK;
}

extern "C" int64_t moe_testing_set_norm_wait(int64_t max_cycles) {
  return bn::g_wait.exchange(max_cycles < 0 ? -1 : max_cycles);
}
