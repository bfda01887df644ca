// embed.cu -- token embedding and its gradient (include/moe_model.h).
//
//   y_t = scale w[id_t],   dw_v = dw_add_v + scale sum_{t : id_t = v} dy_t
//
// Both are bound by HBM: a lookup reads and writes a row a token (8192 tokens of 7168
// columns in bf16 29 us; frequent rows come from L2), the gradient reads a row a token and writes
// (and, with dw_add elsewhere, reads) one a vocabulary entry: 4096 tokens, 131072 x 2048 in bf16 with
// dw_add 191 us, of them 167 for the sums and the rows without tokens (1.09 GB, 6.5 TB/s);
// 60001 tokens, 32001 x 1000 in fp32 113 us, of them 63 for the sums (368 MB, 5.8 TB/s) and
// 39 for the sort's three launches.
//
// Gradient: the tokens are sorted by id (stable, so a row's tokens stay in
// order; up to kSmallT by counting, more by radix passes), the sorted list is cut into chunks of equal length, and one warp walks a
// chunk over 256 columns with its sum in fp32 registers: a row whose tokens lie
// inside the chunk is written at once, a row that crosses a chunk's border leaves
// a partial sum.  A second launch adds those up in chunk order.  So a frequent
// token (a tenth of a batch is not rare) is spread over as many warps as it has
// chunks, and nothing depends on the order in which blocks run.  Rows without tokens
// are written by further warps of the first launch.
//
// Tokens without a gradient (padding, ids out of range) get the key `vocab`, which
// sorts behind every row.  Up to kFewT tokens take one launch and no list.
#include <algorithm>
#include <cmath>

#include "../../include/moe_model.h"
#include "common.cuh"
#include "internal.h"
#include "train.h"

namespace moe {
namespace emb {

constexpr int kSmallT = 16384;      // tokens whose places are counted, not sorted
constexpr int kMaxBits = 9;         // of a radix digit
constexpr int kMaxBins = 1 << kMaxBits;
constexpr int kTileWarps = 16, kTileMin = 1024;
static_assert(32 * kTileWarps == kMaxBins, "a thread a digit");
constexpr int kMaxTiles = 256;      // blocks of a radix pass

struct EShape {
  int64_t T, w_ld;
  int H, V, pad, dtype, esize;
  float scale;
};

struct Digits {
  int passes, bits;
};
inline Digits digits_for(int V) {
  int b = 1;
  while (((int64_t)1 << b) <= V) ++b;   // keys 0 .. V
  Digits d;
  d.passes = (b + kMaxBits - 1) / kMaxBits;
  d.bits = (b + d.passes - 1) / d.passes;
  return d;
}

__device__ __forceinline__ uint32_t key_of(int id, int V, int pad) {
  return (uint32_t)id >= (uint32_t)V || id == pad ? (uint32_t)V : (uint32_t)id;
}

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
constexpr int kLookThreads = 256, kLookVecs = 4;

template <typename T>
__global__ void __launch_bounds__(kLookThreads) embed_kernel(const T* __restrict__ w, int64_t w_ld,
                                                             const int32_t* __restrict__ ids, int64_t vecs,
                                                             int per_row, int V, float scale,
                                                             T* __restrict__ y, uint32_t* flags) {
  pdl_trigger();
  pdl_wait();
  constexpr int NV = Vec16<T>::N;
  const int64_t step = (int64_t)kLookThreads * kLookVecs;
  for (int64_t at = blockIdx.x * step + threadIdx.x; at < vecs; at += gridDim.x * step) {
    uint4 u[kLookVecs];
#pragma unroll
    for (int k = 0; k < kLookVecs; ++k) {
      const int64_t i = at + k * kLookThreads;
      u[k] = make_uint4(0, 0, 0, 0);
      if (i < vecs) {
        const int64_t t = vecs <= 0xffffffffll ? (int64_t)((uint32_t)i / (uint32_t)per_row) : i / per_row;
        const int j = (int)(i - t * per_row);
        const int id = __ldg(ids + t);
        if ((uint32_t)id < (uint32_t)V) u[k] = __ldg(reinterpret_cast<const uint4*>(w + id * w_ld) + j);
        else if (j == 0) set_flag(flags, kFlagToken);
      }
    }
#pragma unroll
    for (int k = 0; k < kLookVecs; ++k) {
      const int64_t i = at + k * kLookThreads;
      if (i < vecs) {
        float f[NV];
        unpack16(u[k], f, (const T*)nullptr);
#pragma unroll
        for (int e = 0; e < NV; ++e) f[e] *= scale;
        __stcs(reinterpret_cast<uint4*>(y) + i, pack16(f, (const T*)nullptr));
      }
    }
  }
}

// ---------------------------------------------------------------------------
// sorting the tokens by id, stable
// ---------------------------------------------------------------------------

// Radix passes: one warp counts (or places) 32 items at a time in order: the lanes with
// the same digit find each other, the lowest of them keeps the warp's counter.
__device__ __forceinline__ void count_digit(uint32_t* cnt, uint32_t digit, bool live) {
  const uint32_t all = __ballot_sync(0xffffffffu, live);
  if (live) {
    const uint32_t same = __match_any_sync(all, digit);
    if ((__ffs(same) - 1) == (int)(threadIdx.x & 31)) cnt[digit] += __popc(same);
  }
  __syncwarp();
}
__device__ __forceinline__ uint32_t place_digit(uint32_t* cnt, uint32_t digit, bool live) {
  const uint32_t all = __ballot_sync(0xffffffffu, live);
  uint32_t at = 0, same = 0;
  const int lane = threadIdx.x & 31;
  if (live) {
    same = __match_any_sync(all, digit);
    at = cnt[digit] + __popc(same & ((1u << lane) - 1u));
  }
  __syncwarp();
  if (live && (__ffs(same) - 1) == lane) cnt[digit] += __popc(same);
  __syncwarp();
  return at;
}

// Marks a row as having tokens.  Frequent rows are marked thousands of times: the
// word is read first.
__device__ __forceinline__ void mark(uint32_t* present, uint32_t row) {
  const uint32_t bit = 1u << (row & 31);
  if (!(__ldcg(present + (row >> 5)) & bit)) atomicOr(present + (row >> 5), bit);
}

// Up to kSmallT tokens: a token's place is the number of tokens before it in the
// sorted order, T comparisons each (T = 4096: 17 M over all SMs, 1.5 us of a launch;
// one block with a radix sort in shared memory took 26).  A block finds the places of
// 32 tokens, a lane each; its warps take a part of every kRankKeys keys.
constexpr int kRankWarps = 8, kRankKeys = 4096;
__global__ void __launch_bounds__(32 * kRankWarps) rank_kernel(const int32_t* __restrict__ ids, int T, int V, int pad,
                                                               uint32_t* __restrict__ keys,
                                                               int32_t* __restrict__ toks, uint32_t* present,
                                                               uint32_t* flags) {
  __shared__ __align__(16) uint32_t key[kRankKeys];
  __shared__ uint32_t part[kRankWarps][32];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = blockIdx.x * 32, t = first + lane;
  const int id = t < T ? ids[t] : 0;
  const uint32_t mine = t < T ? key_of(id, V, pad) : 0u;
  uint32_t n = 0;
  for (int base = 0; base < T; base += kRankKeys) {
    __syncthreads();
    for (int i = threadIdx.x; i < kRankKeys; i += 32 * kRankWarps)
      key[i] = base + i < T ? key_of(ids[base + i], V, pad) : ~0u;    // ~0: before no token
    __syncthreads();
    constexpr int each = kRankKeys / kRankWarps;
    const int lo = warp * each, hi = min(lo + each, T - base);
    // four keys a step; those before the block's tokens count when equal, those behind
    // them do not (first is a multiple of 32, so a step lies on one side of it or in it)
    for (int i = lo; i < hi; i += 4) {
      const uint4 k = *reinterpret_cast<const uint4*>(key + i);
      const int at = base + i;
      if (at + 4 <= first || at >= first + 32) {
        const uint32_t lim = mine + (at < first ? 1u : 0u);
        n += (k.x < lim) + (k.y < lim) + (k.z < lim) + (k.w < lim);
      } else {
        n += (k.x < mine + (at < t)) + (k.y < mine + (at + 1 < t)) + (k.z < mine + (at + 2 < t)) +
             (k.w < mine + (at + 3 < t));
      }
    }
  }
  part[warp][lane] = n;
  __syncthreads();
  if (warp != 0 || t >= T) return;
  for (int w = 1; w < kRankWarps; ++w) n += part[w][lane];
  keys[n] = mine;
  toks[n] = t;
  if ((uint32_t)id >= (uint32_t)V) set_flag(flags, kFlagToken);
  if (present != nullptr && mine < (uint32_t)V) mark(present, mine);
}

// More tokens: each pass cuts the list into at most kMaxTiles tiles of `tile`
// items; hist[tile][bins] counts the digits of this pass's input.
__global__ void __launch_bounds__(512) hist_kernel(const int32_t* __restrict__ ids, int64_t T, int64_t tile,
                                                   int V, int pad, int bins, uint32_t* __restrict__ hist,
                                                   uint32_t* present, uint32_t* flags) {
  constexpr int kSeen = 1024;
  __shared__ uint32_t cnt[kMaxBins], seen[kSeen];
  pdl_trigger();
  pdl_wait();
  for (int d = threadIdx.x; d < bins; d += 512) cnt[d] = 0;
  for (int d = threadIdx.x; d < kSeen; d += 512) seen[d] = ~0u;
  __syncthreads();
  const int64_t lo = blockIdx.x * tile, hi = min(T, lo + tile);
  // A frequent row is marked by few threads of a block (a warp's equal keys once, and not
  // again while its key stands in `seen`): thousands of atomics on one word are a queue.
  // Whole warps go round (those past the end with the key ~0, which no token has).
  for (int64_t i = lo + threadIdx.x; i - (threadIdx.x & 31) < hi; i += 512) {
    const int id = i < hi ? ids[i] : 0;
    if ((uint32_t)id >= (uint32_t)V) set_flag(flags, kFlagToken);
    const uint32_t k = i < hi ? key_of(id, V, pad) : ~0u, same = __match_any_sync(0xffffffffu, k);
    if (k != ~0u && (__ffs(same) - 1) == (int)(threadIdx.x & 31)) {
      atomicAdd(cnt + (k & (bins - 1)), (uint32_t)__popc(same));
      if (present != nullptr && k < (uint32_t)V && atomicExch(seen + (k & (kSeen - 1)), k) != k) mark(present, k);
    }
    __syncwarp();
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += 512) hist[(int64_t)blockIdx.x * bins + d] = cnt[d];
}

// One pass: items to their places, and the next pass's counts (integers, so
// their atomics leave no trace of the order).  ids: the first pass.
__global__ void __launch_bounds__(32 * kTileWarps) scatter_kernel(
    const int32_t* __restrict__ ids, const uint32_t* __restrict__ kin, const int32_t* __restrict__ tin, int64_t T,
    int64_t tile, int V, int pad, int pass, int bits, const uint32_t* __restrict__ hist, uint32_t* next,
    uint32_t* __restrict__ kout, int32_t* __restrict__ tout) {
  __shared__ uint32_t cnt[kTileWarps * kMaxBins];
  __shared__ uint32_t sums[kTileWarps];
  pdl_trigger();
  pdl_wait();
  const int bins = 1 << bits, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // where this tile's items of a digit (a thread's each) start: all items of smaller
  // digits, then the earlier tiles' items of this one
  uint32_t before = 0, all = 0;
  const int digit = threadIdx.x;
  if (digit < bins) {
#pragma unroll 16
    for (unsigned b = 0; b < gridDim.x; ++b) {
      const uint32_t v = __ldcg(hist + (int64_t)b * bins + digit);
      before += b < blockIdx.x ? v : 0u;
      all += v;
    }
  }
  uint32_t incl = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  uint32_t start = before + incl - all;
  for (int w = 0; w < warp; ++w) start += sums[w];
  const int64_t t0 = blockIdx.x * tile, t1 = min(T, t0 + tile), per = tile / kTileWarps;
  const int64_t lo = min(t1, t0 + warp * per), hi = min(t1, lo + per);
  uint32_t* mine = cnt + warp * bins;
  for (int d = lane; d < bins; d += 32) mine[d] = 0;
  __syncwarp();
  const int shift = pass * bits;
  auto key_at = [&](int64_t i) { return ids != nullptr ? key_of(ids[i], V, pad) : kin[i]; };
  for (int64_t i = lo; i < hi; i += 32) {
    const bool live = i + lane < hi;
    count_digit(mine, live ? (key_at(i + lane) >> shift) & (bins - 1) : 0u, live);
  }
  __syncthreads();
  if (digit < bins) {
#pragma unroll
    for (int w = 0; w < kTileWarps; ++w) {
      const uint32_t v = cnt[w * bins + digit];
      cnt[w * bins + digit] = start;
      start += v;
    }
  }
  __syncthreads();
  for (int64_t i = lo; i < hi; i += 32) {
    const bool live = i + lane < hi;
    const uint32_t k = live ? key_at(i + lane) : 0u;
    const uint32_t at = place_digit(mine, (k >> shift) & (bins - 1), live);
    if (live) {
      kout[at] = k;
      tout[at] = ids != nullptr ? (int32_t)(i + lane) : tin[i + lane];
      if (next != nullptr)
        atomicAdd(next + (int64_t)(at / (uint32_t)tile) * bins + ((k >> (shift + bits)) & (bins - 1)), 1u);
    }
  }
}

// ---------------------------------------------------------------------------
// sums over the sorted tokens
// ---------------------------------------------------------------------------
struct SumArgs {
  const uint32_t* keys;
  const int32_t* toks;
  int64_t T;
  int H, V, chunk, slabs;     // slabs of 32 x 8 columns
  int64_t chunks;
  float scale;
  float* left;                // [chunks][H]: sums of a row that starts in an earlier chunk
  float* right;               // [chunks][H]: of a row that starts here and goes on
  int64_t acc_blocks;         // blocks of sum_kernel that walk chunks; the others fill
  const uint32_t* present;    // rows with tokens, or NULL: no row is filled
};

constexpr int kSumWarps = 8;
constexpr int kAhead = 8;     // rows of dy in flight for a warp

// 8 columns of one row
template <typename T>
struct Eight {
  uint4 v[8 / Vec16<T>::N];
};
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p) {
  Eight<T> r;
#pragma unroll
  for (int i = 0; i < 8 / Vec16<T>::N; ++i) r.v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
template <typename T>
__device__ __forceinline__ void add8(const Eight<T>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 8 / Vec16<T>::N; ++i) {
    float g[Vec16<T>::N];
    unpack16(r.v[i], g, (const T*)nullptr);
#pragma unroll
    for (int e = 0; e < Vec16<T>::N; ++e) f[i * Vec16<T>::N + e] += g[e];
  }
}
// dw row = dw_add row + scale * sum
template <typename T>
__device__ __forceinline__ void write8(const float* sum, float scale, const T* add, T* dw, int64_t at) {
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = 0.0f;
  if (add != nullptr) {
    // not through the read-only path: dw_add may be dw
    Eight<T> r;
#pragma unroll
    for (int i = 0; i < 8 / Vec16<T>::N; ++i) r.v[i] = reinterpret_cast<const uint4*>(add + at)[i];
    add8<T>(r, f);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = fmaf(sum[e], scale, f[e]);
#pragma unroll
  for (int i = 0; i < 8 / Vec16<T>::N; ++i)
    reinterpret_cast<uint4*>(dw + at)[i] = pack16(f + i * Vec16<T>::N, (const T*)nullptr);
}
__device__ __forceinline__ void write_part(float* p, const float* f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// A row without tokens: dw_add's, or zeros.
template <typename T>
__device__ __forceinline__ void fill_row(const T* add, T* dw, int64_t v, int H, int lane) {
  const int vecs = H / Vec16<T>::N;
  uint4* out = reinterpret_cast<uint4*>(dw + v * H);
  if (add == nullptr) {
    for (int j = lane; j < vecs; j += 32) __stcs(out + j, make_uint4(0, 0, 0, 0));
    return;
  }
  const uint4* in = reinterpret_cast<const uint4*>(add + v * H);
  int j = lane;
  for (; j + 96 < vecs; j += 128) {
    uint4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) u[k] = __ldcs(in + j + 32 * k);
#pragma unroll
    for (int k = 0; k < 4; ++k) __stcs(out + j + 32 * k, u[k]);
  }
  for (; j < vecs; j += 32) __stcs(out + j, __ldcs(in + j));
}

// Up to kFewT tokens in one launch, without a sorted list: a warp a token and 256 columns
// compares the token's id with all, and the first of an id adds up its tokens in order; the
// other warps fill the rows whose id no token has.  64 tokens of different ids (of one id), with
// and without: 131072 x 264 16 (23) us against 32 (34), 50257 x 2048 with dw_add 68 against 77, 80
// x 7168 8 (18) against 20; more tokens of one id would be too many for a warp.
constexpr int kFewT = 64;
template <typename T>
__global__ void __launch_bounds__(32 * kSumWarps) few_kernel(const int32_t* __restrict__ ids, int count, int V, int pad,
                                                             int H, int slabs, float scale, int sum_blocks,
                                                             const T* __restrict__ dy, const T* add, T* dw,
                                                             uint32_t* flags) {
  __shared__ uint32_t key[kFewT];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < kFewT) {
    const int id = threadIdx.x < count ? ids[threadIdx.x] : -1;
    key[threadIdx.x] = threadIdx.x < count ? key_of(id, V, pad) : (uint32_t)V;
    if (blockIdx.x == 0 && (int)threadIdx.x < count && (uint32_t)id >= (uint32_t)V) set_flag(flags, kFlagToken);
  }
  __syncthreads();
  const uint32_t k0 = key[lane], k1 = key[lane + 32];
  auto tokens_of = [&](uint32_t row) {
    return (uint64_t)__ballot_sync(0xffffffffu, k0 == row) | (uint64_t)__ballot_sync(0xffffffffu, k1 == row) << 32;
  };
  if ((int)blockIdx.x >= sum_blocks) {
    const int64_t step = (int64_t)(gridDim.x - sum_blocks) * kSumWarps;
    for (int64_t v = (int64_t)(blockIdx.x - sum_blocks) * kSumWarps + warp; v < V; v += step)
      if (!tokens_of((uint32_t)v)) fill_row<T>(add, dw, v, H, lane);
    return;
  }
  const int task = blockIdx.x * kSumWarps + warp, t = task / slabs, col = (task - t * slabs) * 256 + lane * 8;
  if (t >= count) return;
  const uint32_t row = key[t];
  uint64_t left = tokens_of(row);
  if (row >= (uint32_t)V || __ffsll((long long)left) - 1 != t || col >= H) return;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  while (left) {
    Eight<T> r[kAhead];
    int n = 0;
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (left) {
        r[j] = load8<T>(dy + (int64_t)(__ffsll((long long)left) - 1) * H + col);
        left &= left - 1;
        ++n;
      }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (j < n) add8<T>(r[j], acc);
  }
  write8<T>(acc, scale, add, dw, (int64_t)row * H + col);
}

template <typename T>
__global__ void __launch_bounds__(32 * kSumWarps) sum_kernel(const SumArgs a, const T* __restrict__ dy, const T* add,
                                                             T* dw) {
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x >= a.acc_blocks) {
    // rows without tokens
    const int64_t nw = (int64_t)(gridDim.x - a.acc_blocks) * kSumWarps;
    for (int64_t v = (blockIdx.x - a.acc_blocks) * kSumWarps + warp; v < a.V; v += nw) {
      if ((a.present[v >> 5] >> (v & 31)) & 1u) continue;
      fill_row<T>(add, dw, v, a.H, lane);
    }
    return;
  }
  const int64_t task = (int64_t)blockIdx.x * kSumWarps + warp;
  const int64_t c = task / a.slabs;
  if (c >= a.chunks) return;
  const int col = (int)(task - c * a.slabs) * 256 + lane * 8;
  const bool live = col < a.H;
  const int64_t p0 = c * a.chunk, p1 = min(a.T, p0 + a.chunk);
  const uint32_t V = (uint32_t)a.V;
  const uint32_t before = p0 > 0 ? a.keys[p0 - 1] : ~0u, after = p1 < a.T ? a.keys[p1] : ~0u;
  float acc[8];
  uint32_t cur = ~0u;      // row of the sum; ~0: none yet
  bool from_left = false;  // it started in an earlier chunk
  auto close = [&](bool goes_on) {
    if (cur == ~0u || !live) return;
    if (from_left) write_part(a.left + c * a.H + col, acc);
    else if (goes_on) write_part(a.right + c * a.H + col, acc);
    else write8<T>(acc, a.scale, add, dw, (int64_t)cur * a.H + col);
  };
  bool done = false;
  for (int64_t b = p0; b < p1 && !done; b += 32) {
    const uint32_t k32 = b + lane < p1 ? a.keys[b + lane] : V;
    const int32_t t32 = b + lane < p1 ? a.toks[b + lane] : 0;
    for (int j0 = 0; j0 < 32 && !done; j0 += kAhead) {
      Eight<T> r[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const uint32_t k = __shfl_sync(0xffffffffu, k32, j0 + j);
        const int64_t t = __shfl_sync(0xffffffffu, t32, j0 + j);
        if (k < V && live) r[j] = load8<T>(dy + t * a.H + col);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const uint32_t k = __shfl_sync(0xffffffffu, k32, j0 + j);
        if (k >= V) { done = true; break; }   // the tokens without a gradient, or the chunk's end
        if (k != cur) {
          close(false);
          from_left = cur == ~0u && k == before;
          cur = k;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
        }
        if (live) add8<T>(r[j], acc);
      }
    }
  }
  close(cur == after);
}

// The rows that cross borders: the block of the chunk where such a row starts
// adds its partial sums, eight warps a part each, the parts in order.
template <typename T>
__global__ void __launch_bounds__(32 * kSumWarps) join_kernel(const SumArgs a, const T* add, T* dw) {
  __shared__ float part[kSumWarps][256];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = blockIdx.x;
  const int64_t p0 = c * a.chunk, p1 = p0 + a.chunk;
  if (p1 >= a.T) return;
  const uint32_t row = a.keys[p1];
  if (row >= (uint32_t)a.V || a.keys[p1 - 1] != row) return;       // none goes on from here
  if (p0 > 0 && a.keys[p0 - 1] == row) return;                     // it started earlier
  // chunks after c whose first token is of the row
  int64_t n = 0;
  for (;;) {
    const int64_t q = (c + 1 + n + lane) * a.chunk;
    const uint32_t in = __ballot_sync(0xffffffffu, q < a.T && a.keys[q < a.T ? q : 0] == row);
    const int m = __ffs(~in) - 1;
    n += m < 0 ? 32 : m;
    if (m >= 0) break;
  }
  const int64_t each = (n + kSumWarps - 1) / kSumWarps, hi = min(n, (warp + 1) * each);
  for (int slab = blockIdx.y; slab < a.slabs; slab += gridDim.y) {
    const int col = slab * 256 + lane * 8;
    const bool live = col < a.H;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.0f;
    if (live) {
      auto take = [&](const float* p) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(p)), v = __ldcg(reinterpret_cast<const float4*>(p) + 1);
        f[0] += u.x; f[1] += u.y; f[2] += u.z; f[3] += u.w;
        f[4] += v.x; f[5] += v.y; f[6] += v.z; f[7] += v.w;
      };
      if (warp == 0) take(a.right + c * a.H + col);
#pragma unroll 4
      for (int64_t i = warp * each; i < hi; ++i) take(a.left + (c + 1 + i) * a.H + col);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) part[warp][lane * 8 + e] = f[e];
    __syncthreads();
    if (warp == 0 && live) {
      for (int w = 1; w < kSumWarps; ++w)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] += part[w][lane * 8 + e];
      write8<T>(f, a.scale, add, dw, (int64_t)row * a.H + col);
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Chunks for some 16 warps an SM, which are all there at once (a border costs a row of fp32
// written and read), of 8 to 256 tokens.  60001 tokens, 32001 x 1000 in fp32: 113 us with the
// sort, in powers of two 123, for 24 warps an SM 131; 30000, 50257 x 2048 in bf16 150, 166, 147
int64_t chunk_of(int64_t T, int slabs) {
  return std::min<int64_t>(256, std::max<int64_t>(8, (T * slabs / (16 * 152) + 7) / 8 * 8));
}
int slabs_of(int H) { return (H + 255) / 256; }

moe_status decode(const moe_embed_shape* s, EShape* o, const char** why) {
  *why = "";
  if (!s) { *why = "shape is NULL"; return MOE_ERR_INVALID_ARG; }
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16) { *why = "dtype must be MOE_F32 or MOE_BF16"; return MOE_ERR_UNSUPPORTED; }
  if (s->tokens < 0 || s->tokens > (1ll << 28)) { *why = "tokens must be in [0, 2^28]"; return MOE_ERR_INVALID_ARG; }
  if (s->hidden <= 0 || s->hidden % 8) { *why = "hidden must be a positive multiple of 8"; return MOE_ERR_INVALID_ARG; }
  if (s->hidden > (1 << 28)) { *why = "hidden must be at most 2^28"; return MOE_ERR_INVALID_ARG; }
  if (s->vocab < 1 || s->vocab > (1 << 30)) { *why = "vocab must be in [1, 2^30]"; return MOE_ERR_INVALID_ARG; }
  if (s->padding_idx < -1 || s->padding_idx >= s->vocab) { *why = "padding_idx must be -1 or in [0, vocab)"; return MOE_ERR_INVALID_ARG; }
  if (!std::isfinite(s->scale) || !std::isfinite((float)s->scale)) { *why = "scale must be finite in fp32"; return MOE_ERR_INVALID_ARG; }
  if (s->w_stride != 0 && (s->w_stride < s->hidden || s->w_stride % 8)) {
    *why = "w_stride must be 0, or at least hidden and a multiple of 8";
    return MOE_ERR_INVALID_ARG;
  }
  const int slabs = slabs_of(s->hidden);
  const int64_t chunk = chunk_of(s->tokens, slabs);
  if ((s->tokens + chunk - 1) / chunk * slabs > 0x7fffffff) {    // warps of the gradient's sums
    *why = "tokens times hidden is too large";
    return MOE_ERR_UNSUPPORTED;
  }
  o->T = s->tokens;
  o->H = s->hidden;
  o->V = s->vocab;
  o->pad = s->padding_idx;
  o->dtype = s->dtype;
  o->esize = s->dtype == MOE_F32 ? 4 : 2;
  o->scale = (float)s->scale;
  o->w_ld = s->w_stride ? s->w_stride : s->hidden;
  return MOE_OK;
}

struct Layout {
  size_t flags, keys[2], toks[2], present, hist, left, right, total;
  size_t zero_end;       // present and the counts of the later passes are zeroed together
  int64_t chunks, tiles, tile;
  int chunk, slabs;
  Digits dig;
};

Layout layout_of(const EShape& s) {
  Layout L = {};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~(size_t)255;
    return at;
  };
  L.dig = digits_for(s.V);
  L.slabs = slabs_of(s.H);
  const int64_t chunk = chunk_of(s.T, L.slabs);
  L.chunk = (int)chunk;
  L.chunks = (s.T + chunk - 1) / chunk;
  L.tile = ((s.T + kMaxTiles - 1) / kMaxTiles + kTileMin - 1) / kTileMin * kTileMin;
  if (L.tile < kTileMin) L.tile = kTileMin;
  L.tiles = (s.T + L.tile - 1) / L.tile;
  const bool small = s.T <= kSmallT;
  L.flags = take(256);
  for (int i = 0; i < (small ? 1 : 2); ++i) {
    L.keys[i] = take((size_t)s.T * 4);
    L.toks[i] = take((size_t)s.T * 4);
  }
  L.present = take(((size_t)s.V + 31) / 32 * 4);
  const size_t per = (size_t)L.tiles << L.dig.bits;
  L.hist = take(small ? 0 : per * 4 * L.dig.passes);
  L.zero_end = off;
  L.left = take((size_t)L.chunks * s.H * 4);
  L.right = take((size_t)L.chunks * s.H * 4);
  L.total = off;
  return L;
}

template <typename T>
cudaError_t launch_join(const SumArgs& a, const T* add, T* dw, cudaStream_t st) {
  // most chunks have no row to join: one check for a chunk's slabs, up to four at once
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)a.chunks, (unsigned)std::min(a.slabs, 4));
  cfg.blockDim = dim3(32 * kSumWarps);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, join_kernel<T>, a, add, dw);
  if (e != cudaSuccess) return e;
  count_launch();
  return cudaGetLastError();
}

template <typename T>
moe_status backward(const EShape& s, const Layout& L, char* b, const int32_t* ids, const void* dy, const void* add,
                    void* dw, cudaStream_t st) {
  uint32_t* flags = reinterpret_cast<uint32_t*>(b + L.flags);
  const bool fill = add != dw;
  uint32_t* present = fill ? reinterpret_cast<uint32_t*>(b + L.present) : nullptr;
  uint32_t* hist = reinterpret_cast<uint32_t*>(b + L.hist);
  const size_t per = (size_t)L.tiles << L.dig.bits;
  int at = 0;    // where the sorted list is
  int64_t fill_blocks = 0;
  if (fill) fill_blocks = std::min<int64_t>(((int64_t)s.V + kSumWarps - 1) / kSumWarps, 8 * (int64_t)tc_sm_count());
  if (s.T > 0 && s.T <= kFewT) {
    const int sum_blocks = ((int)s.T * L.slabs + kSumWarps - 1) / kSumWarps;
    CHECK_CUDA(launch_after(few_kernel<T>, (unsigned)(sum_blocks + fill_blocks), 32 * kSumWarps, 0, st, 1, ids, (int)s.T,
                            s.V, s.pad, s.H, L.slabs, s.scale, sum_blocks, static_cast<const T*>(dy),
                            static_cast<const T*>(add), static_cast<T*>(dw), flags));
    return MOE_OK;
  }
  if (s.T > kSmallT || fill) CHECK_CUDA(cudaMemsetAsync(b + L.present, 0, L.zero_end - L.present, st));
  if (s.T > 0 && s.T <= kSmallT) {
    CHECK_CUDA(launch_after(rank_kernel, (unsigned)((s.T + 31) / 32), 32 * kRankWarps, 0, st, 1, ids, (int)s.T, s.V, s.pad,
                            reinterpret_cast<uint32_t*>(b + L.keys[0]), reinterpret_cast<int32_t*>(b + L.toks[0]),
                            present, flags));
  } else if (s.T > 0) {
    CHECK_CUDA(launch_after(hist_kernel, (unsigned)L.tiles, 512, 0, st, 1, ids, s.T, L.tile, s.V, s.pad, 1 << L.dig.bits,
                            hist, present, flags));
    for (int p = 0; p < L.dig.passes; ++p) {
      const int to = p & 1;
      CHECK_CUDA(launch_after(scatter_kernel, (unsigned)L.tiles, 32 * kTileWarps, 0, st, 1, p == 0 ? ids : nullptr,
                              reinterpret_cast<const uint32_t*>(b + L.keys[to ^ 1]),
                              reinterpret_cast<const int32_t*>(b + L.toks[to ^ 1]), s.T, L.tile, s.V, s.pad, p, L.dig.bits,
                              hist + p * per, p + 1 < L.dig.passes ? hist + (p + 1) * per : nullptr,
                              reinterpret_cast<uint32_t*>(b + L.keys[to]), reinterpret_cast<int32_t*>(b + L.toks[to])));
      at = to;
    }
  }
  SumArgs a = {};
  a.keys = reinterpret_cast<const uint32_t*>(b + L.keys[at]);
  a.toks = reinterpret_cast<const int32_t*>(b + L.toks[at]);
  a.T = s.T;
  a.H = s.H;
  a.V = s.V;
  a.chunk = L.chunk;
  a.slabs = L.slabs;
  a.chunks = L.chunks;
  a.scale = s.scale;
  a.left = reinterpret_cast<float*>(b + L.left);
  a.right = reinterpret_cast<float*>(b + L.right);
  a.acc_blocks = (L.chunks * L.slabs + kSumWarps - 1) / kSumWarps;
  a.present = present;
  if (a.acc_blocks + fill_blocks > 0)
    CHECK_CUDA(launch_after(sum_kernel<T>, (unsigned)(a.acc_blocks + fill_blocks), 32 * kSumWarps, 0, st, 1, a,
                            static_cast<const T*>(dy), static_cast<const T*>(add), static_cast<T*>(dw)));
  if (L.chunks > 1)
    CHECK_CUDA(launch_join<T>(a, static_cast<const T*>(add), static_cast<T*>(dw), st));
  return MOE_OK;
}

}  // namespace emb
}  // namespace moe

using namespace moe;

#define DECODE_EMB(shape, s)                                  \
  emb::EShape s;                                              \
  do {                                                        \
    const char* why_ = "";                                    \
    moe_status st_ = emb::decode(shape, &s, &why_);           \
    if (st_ != MOE_OK) return fail(st_, why_);                \
  } while (0)

extern "C" size_t moe_embed_workspace_bytes(const moe_embed_shape* shape) {
  emb::EShape s;
  const char* why;
  moe_status st = emb::decode(shape, &s, &why);
  if (st != MOE_OK) {
    fail(st, why);
    return 0;
  }
  return emb::layout_of(s).total;
}

extern "C" moe_status moe_embed_forward(const moe_embed_shape* shape, const void* w, const int32_t* ids, void* y,
                                        void* ws, size_t ws_bytes, void* stream) {
  reset_launch_count();
  DECODE_EMB(shape, s);
  if (!w || (s.T > 0 && (!ids || !y))) return fail(MOE_ERR_INVALID_ARG, "w, ids and y must be non-NULL");
  if (!aligned16(w) || !aligned16(y)) return fail(MOE_ERR_INVALID_ARG, "w and y must be 16-byte aligned");
  if ((uintptr_t)ids & 3u) return fail(MOE_ERR_INVALID_ARG, "ids must be aligned to its elements");
  moe_status e = check_ws(ws, ws_bytes, emb::layout_of(s).total);
  if (e != MOE_OK) return e;
  if (s.T == 0) return MOE_OK;
  uint32_t* flags = static_cast<uint32_t*>(ws);
  const int per_row = s.H * s.esize / 16;
  const int64_t vecs = s.T * per_row, each = emb::kLookThreads * emb::kLookVecs;
  const unsigned grid = (unsigned)std::min<int64_t>((vecs + each - 1) / each, 16 * (int64_t)tc_sm_count());
  if (s.dtype == MOE_F32)
    CHECK_CUDA(launch_after(emb::embed_kernel<float>, grid, emb::kLookThreads, 0, (cudaStream_t)stream, 1,
                            static_cast<const float*>(w), s.w_ld, ids, vecs, per_row, s.V, s.scale,
                            static_cast<float*>(y), flags));
  else
    CHECK_CUDA(launch_after(emb::embed_kernel<bf16>, grid, emb::kLookThreads, 0, (cudaStream_t)stream, 1,
                            static_cast<const bf16*>(w), s.w_ld, ids, vecs, per_row, s.V, s.scale,
                            static_cast<bf16*>(y), flags));
  return MOE_OK;
}

extern "C" moe_status moe_embed_backward(const moe_embed_shape* shape, const int32_t* ids, const void* dy,
                                         const void* dw_add, void* dw, void* ws, size_t ws_bytes, void* stream) {
  reset_launch_count();
  DECODE_EMB(shape, s);
  if (!dw || (s.T > 0 && (!ids || !dy))) return fail(MOE_ERR_INVALID_ARG, "ids, dy and dw must be non-NULL");
  if (!aligned16(dy) || !aligned16(dw) || !aligned16(dw_add))
    return fail(MOE_ERR_INVALID_ARG, "dy, dw_add and dw must be 16-byte aligned");
  if ((uintptr_t)ids & 3u) return fail(MOE_ERR_INVALID_ARG, "ids must be aligned to its elements");
  const emb::Layout L = emb::layout_of(s);
  moe_status e = check_ws(ws, ws_bytes, L.total);
  if (e != MOE_OK) return e;
  char* b = static_cast<char*>(ws);
  if (s.dtype == MOE_F32) return emb::backward<float>(s, L, b, ids, dy, dw_add, dw, (cudaStream_t)stream);
  return emb::backward<bf16>(s, L, b, ids, dy, dw_add, dw, (cudaStream_t)stream);
}
