// muon.cu -- orthogonalised update of weight matrices (include/moe_model.h): the
// momentum, the matrices' norms, the fp16 planes that the products of orth_tc.cu
// read, and the update of the parameters.
//
// Tensors with the same smaller and larger side and the same precision form a
// bucket, whose matrices go through the products together, at most so many at a time
// as kScratch bytes of scratch hold.  A matrix is laid out with its smaller side as
// rows (one with more rows than columns is transposed on the way in and out), so the
// products see one shape.
//
// Bound by HBM: a bf16 parameter reads gradient and momentum twice (for the norm, then
// for the scaled planes), writes the momentum, and passes once more for the update.  Of 96
// matrices 704 x 2816, a third of them transposed, the momentum takes 285 us (6.7 TB/s), the
// planes 282 (6.1; with three blocks an SM instead of four 320), the update 199 (5.7;
// with the second piece of X read after the first was opened 239).  Tiles of 64 x 128 instead
// of 64 x 64: planes 317, update 359 (two blocks an SM).
#include <algorithm>
#include <cmath>

#include "../../include/moe_model.h"
#include "common.cuh"
#include "internal.h"
#include "muon.cuh"
#include "orth.h"
#include "train.h"

namespace moe {
namespace muon {

// Momentum, and the sum of u^2 over kPart elements of a matrix: in fp32 over a warp's
// elements, in fp64 beyond.  A warp whose sum overflowed, or is small enough for
// squares to have underflowed, adds again with its values scaled by a power of two.
__global__ void __launch_bounds__(256) momentum_kernel(const __grid_constant__ Round r) {
  __shared__ double sh[8];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tasks = (int64_t)r.batch * r.parts;
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int b = (int)(task / r.parts), part = (int)(task - (int64_t)b * r.parts);
    const Seg& s = seg_of(r, b);
    const int64_t each = (int64_t)s.rows * s.cols;
    const int64_t base = (s.first + (b - s.at)) * each;      // the matrix in its tensor
    const bool ok = each % 8 == 0 && aligned(s.grad) && aligned(s.momentum);
    constexpr int PIECES = kPart / 256 / 8;
    float u[PIECES][8];
    float sum = 0.0f;
    auto at_of = [&](int k) { return (int64_t)part * kPart + (k * 256 + threadIdx.x) * 8; };
    if (ok) {
      Raw8 g[PIECES], v[PIECES];
#pragma unroll
      for (int k = 0; k < PIECES; ++k) {
        const int64_t at = at_of(k);
        g[k] = load_raw(s.grad, s.gdtype, base + at, at < each);
        v[k] = load_raw(s.momentum, MOE_F32, base + at, at < each && s.momentum != nullptr);
      }
#pragma unroll
      for (int k = 0; k < PIECES; ++k) {
        const int64_t at = at_of(k);
        open_raw(g[k], s.gdtype, u[k]);
        if (s.momentum != nullptr) {
          float m[8];
          open_raw(v[k], MOE_F32, m);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            m[e] = fmaf(r.beta, m[e], r.rest * u[k][e]);
            u[k][e] = direction(r, u[k][e], m[e]);
          }
          if (at < each) write8(s.momentum, MOE_F32, base + at, 8, true, m);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < PIECES; ++k) {
        const int64_t at = at_of(k);
        const int n = at >= each ? 0 : (each - at < 8 ? (int)(each - at) : 8);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[k][e] = 0.0f;
        if (n <= 0) continue;
        read8(s.grad, s.gdtype, base + at, n, false, u[k]);
        if (s.momentum != nullptr) {
          float m[8];
          read8(s.momentum, MOE_F32, base + at, n, false, m);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            m[e] = fmaf(r.beta, m[e], r.rest * u[k][e]);
            u[k][e] = e < n ? direction(r, u[k][e], m[e]) : 0.0f;
          }
          write8(s.momentum, MOE_F32, base + at, n, false, m);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < PIECES; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(u[k][e], u[k][e], sum);
    auto all = [](float v) {
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    };
    auto squares = [&](float scale) {
      float t = 0.0f;
#pragma unroll
      for (int k = 0; k < kPart / 256 / 8; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = u[k][e] * scale;
          t = fmaf(v, v, t);
        }
      return (double)all(t);
    };
    double total = (double)all(sum);
    if (!(total >= 1e-28)) total = squares(0x1p80f) * 0x1p-160;
    else if (!(total <= 1e38)) total = squares(0x1p-96f) * 0x1p192;
    __syncthreads();
    if (lane == 0) sh[warp] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
      double t = 0.0;
      for (int w = 0; w < 8; ++w) t += sh[w];
      r.sums[task] = t;
    }
  }
}

// ALL16: gradients and parameters are bf16 in every segment, which leaves registers for more
// blocks an SM.
template <bool ALL16>
__device__ __forceinline__ int type_of(int dtype) { return ALL16 ? (int)MOE_BF16 : dtype; }

// 8 values to X, from `at` elements of the round's first plane.
template <bool ALL16>
__device__ __forceinline__ void put8(const Round& r, int64_t at, const float* f) {
  uint32_t h[4];
  float lead[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 a = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    const float2 v = __half22float2(a);
    lead[2 * i] = v.x;
    lead[2 * i + 1] = v.y;
    h[i] = *reinterpret_cast<const uint32_t*>(&a);
  }
  *reinterpret_cast<uint4*>(r.x + at) = make_uint4(h[0], h[1], h[2], h[3]);
  const int64_t plane = (int64_t)r.batch * r.m * r.ldx;
  if (!ALL16 && r.planes == 2) {
    uint32_t l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 c = __floats2half2_rn(f[2 * i] - lead[2 * i], f[2 * i + 1] - lead[2 * i + 1]);
      l[i] = *reinterpret_cast<const uint32_t*>(&c);
    }
    *reinterpret_cast<uint4*>(r.x + plane + at) = make_uint4(l[0], l[1], l[2], l[3]);
  } else {
    uint32_t l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      l[i] = orth_low_pack(orth_low_steps(f[4 * i], lead[4 * i]), orth_low_steps(f[4 * i + 1], lead[4 * i + 1]),
                           orth_low_steps(f[4 * i + 2], lead[4 * i + 2]), orth_low_steps(f[4 * i + 3], lead[4 * i + 3]));
    *reinterpret_cast<uint2*>(reinterpret_cast<char*>(r.x + plane) + at) = make_uint2(l[0], l[1]);
  }
}
// 8 values of the last X (which has no 8-bit parts: no step is left to need them), as they
// stand, and as floats.
struct RawX {
  uint4 hi, lo;
};
template <bool ALL16>
__device__ __forceinline__ RawX load_x(const Round& r, int64_t at, bool there) {
  RawX x;
  x.hi = x.lo = make_uint4(0, 0, 0, 0);
  if (there) {
    x.hi = *reinterpret_cast<const uint4*>(r.x + at);
    if (!ALL16 && r.planes == 2) x.lo = *reinterpret_cast<const uint4*>(r.x + (int64_t)r.batch * r.m * r.ldx + at);
  }
  return x;
}
template <bool ALL16>
__device__ __forceinline__ void open_x(const RawX& x, float* f) {
  const uint32_t h[4] = {x.hi.x, x.hi.y, x.hi.z, x.hi.w}, l[4] = {x.lo.x, x.lo.y, x.lo.z, x.lo.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    if (!ALL16) {
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&l[i]));
      a.x += b.x;
      a.y += b.y;
    }
    f[2 * i] = a.x * 0x1p-13f;
    f[2 * i + 1] = a.y * 0x1p-13f;
  }
}
static_assert(kOrthX == 13, "open_x's factor");

struct TileAt {
  int b, r0, c0;   // matrix of the round; first row and column of the tile in its tensor
};
__device__ __forceinline__ TileAt tile_at(const Round& r, int64_t task, const Seg*& s) {
  // tiles of kTile x kTile over the larger and smaller side, whichever way round
  const int tm = (r.m + kTile - 1) / kTile, tn = (r.n + kTile - 1) / kTile;
  TileAt t;
  t.b = (int)(task / ((int64_t)tm * tn));
  const int l = (int)(task - (int64_t)t.b * tm * tn);
  s = &seg_of(r, t.b);
  const int tc = s->rows <= s->cols ? tn : tm;   // tiles along a row of the tensor
  t.r0 = l / tc * kTile;
  t.c0 = l % tc * kTile;
  return t;
}

// u / (norm + eps) as X is held, its smaller side as rows.
template <bool ALL16>
__global__ void __launch_bounds__(256, ALL16 ? 4 : 3) planes_kernel(const __grid_constant__ Round r) {
  __shared__ float sh[kTile][kTile + 1];
  __shared__ double part[8];
  __shared__ float2 factor;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int64_t tiles = (int64_t)((r.m + kTile - 1) / kTile) * ((r.n + kTile - 1) / kTile);
  int last = -1;
  // a block takes neighbouring tiles, so that a matrix's norm is added up once
  const int64_t all = tiles * r.batch, each = (all + gridDim.x - 1) / gridDim.x;
  const int64_t end = min(all, (blockIdx.x + 1) * each);
  for (int64_t task = blockIdx.x * each; task < end; ++task) {
    const Seg* s;
    const TileAt t = tile_at(r, task, s);
    if (t.b != last) {
      last = t.b;
      double v = 0.0;
      for (int i = tid; i < r.parts; i += 256) v += __ldcg(r.sums + (int64_t)t.b * r.parts + i);
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      __syncthreads();
      if ((tid & 31) == 0) part[tid >> 5] = v;
      __syncthreads();
      if (tid == 0) {
        double w = 0.0;
        for (int i = 0; i < 8; ++i) w += part[i];
        factor = scale_of(w, r.eps);
      }
      __syncthreads();
    }
    const float2 q = factor;
    const bool tall = s->rows > s->cols;
    const int64_t base = (s->first + (t.b - s->at)) * (int64_t)s->rows * s->cols;
    const bool ok = s->cols % 8 == 0 && aligned(s->grad) && aligned(s->momentum);
    const int64_t x = (int64_t)t.b * r.m * r.ldx;   // of the matrix in the planes
    if (tall) __syncthreads();   // the last tile's readers are done
    Raw8 g[2], v[2];
    if (ok)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = t.r0 + k * 32 + tid / 8, col = t.c0 + tid % 8 * 8;
        const bool there = row < s->rows && col < s->cols;
        const int64_t at = base + (int64_t)row * s->cols + col;
        g[k] = load_raw(s->grad, type_of<ALL16>(s->gdtype), at, there);
        v[k] = load_raw(s->momentum, MOE_F32, at, there && s->momentum != nullptr);
      }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int lr = k * 32 + tid / 8, lc = tid % 8 * 8;
      const int row = t.r0 + lr, col = t.c0 + lc;
      const int n = row >= s->rows || col >= s->cols ? 0 : min(8, s->cols - col);
      float f[8], m[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = m[e] = 0.0f;
      if (ok) {
        open_raw(g[k], type_of<ALL16>(s->gdtype), f);
        open_raw(v[k], MOE_F32, m);
      } else if (n > 0) {
        const int64_t at = base + (int64_t)row * s->cols + col;
        read8(s->grad, type_of<ALL16>(s->gdtype), at, n, false, f);
        if (s->momentum != nullptr) read8(s->momentum, MOE_F32, at, n, false, m);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (s->momentum != nullptr) f[e] = direction(r, f[e], m[e]);
        f[e] = f[e] * q.x * q.y;
      }
      if (!tall) {
        if (n > 0) put8<ALL16>(r, x + (int64_t)row * r.ldx + col, f);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) sh[lr][lc + e] = e < n ? f[e] : 0.0f;
      }
    }
    if (!tall) continue;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int lr = k * 32 + tid / 8, lc = tid % 8 * 8;   // of the transposed tile
      const int row = t.c0 + lr, col = t.r0 + lc;
      if (row >= r.m || col >= r.n) continue;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = sh[lc + e][lr];
      put8<ALL16>(r, x + (int64_t)row * r.ldx + col, f);
    }
  }
}

// param = keep param - size X, or out = X.
template <bool ALL16>
__global__ void __launch_bounds__(256) update_kernel(const __grid_constant__ Round r) {
  __shared__ float sh[kTile][kTile + 1];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x;
  const int64_t all = (int64_t)((r.m + kTile - 1) / kTile) * ((r.n + kTile - 1) / kTile) * r.batch;
  const int64_t each = (all + gridDim.x - 1) / gridDim.x, end = min(all, (blockIdx.x + 1) * each);
  for (int64_t task = blockIdx.x * each; task < end; ++task) {
    const Seg* s;
    const TileAt t = tile_at(r, task, s);
    const bool tall = s->rows > s->cols;
    const int64_t base = (s->first + (t.b - s->at)) * (int64_t)s->rows * s->cols;
    const bool ok = s->cols % 8 == 0 && aligned(s->param);   // pieces are whole and on 16-byte boundaries
    const int64_t x = (int64_t)t.b * r.m * r.ldx;
    // everything that is read first
    Raw8 w[2];
    float f[2][8];
    if (r.update && ok)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = t.r0 + k * 32 + tid / 8, col = t.c0 + tid % 8 * 8;
        w[k] = load_raw(s->param, type_of<ALL16>(s->pdtype), base + (int64_t)row * s->cols + col, row < s->rows && col < s->cols);
      }
    RawX raw[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int row = (tall ? t.c0 : t.r0) + k * 32 + tid / 8, col = (tall ? t.r0 : t.c0) + tid % 8 * 8;
      raw[k] = load_x<ALL16>(r, x + (int64_t)row * r.ldx + col, row < r.m && col < r.n);
    }
    if (tall) __syncthreads();   // the last tile's readers are done
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int lr = k * 32 + tid / 8, lc = tid % 8 * 8;
      open_x<ALL16>(raw[k], f[k]);
      if (tall)
#pragma unroll
        for (int e = 0; e < 8; ++e) sh[lc + e][lr] = f[k][e];
    }
    if (tall) __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int lr = k * 32 + tid / 8, lc = tid % 8 * 8;
      const int row = t.r0 + lr, col = t.c0 + lc;
      const int n = row >= s->rows || col >= s->cols ? 0 : min(8, s->cols - col);
      if (n <= 0) continue;
      const int64_t at = base + (int64_t)row * s->cols + col;
      if (tall) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[k][e] = e < n ? sh[lr][lc + e] : 0.0f;
      }
      if (r.update) {
        float p[8];
        if (ok) open_raw(w[k], type_of<ALL16>(s->pdtype), p);
        else read8(s->param, type_of<ALL16>(s->pdtype), at, n, false, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[k][e] = fmaf(-s->size, f[k][e], r.keep * p[e]);
      }
      write8(s->param, type_of<ALL16>(s->pdtype), at, n, ok, f[k]);
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct Bucket {
  int m, n, planes;
  int64_t batch;
  int ldx, lda, parts;
  bool pair;       // the first two steps in one
  int64_t each;    // scratch bytes of a matrix
  int64_t round;   // matrices at a time
};

// Bytes of one X: two fp16 planes, or one and the 8-bit parts.
int64_t x_bytes(const Bucket& b) { return (int64_t)b.m * b.ldx * (b.planes == 2 ? 4 : 3); }

Bucket bucket_of(int m, int n, int planes, int64_t batch) {
  Bucket b = {};
  b.m = m;
  b.n = n;
  b.planes = planes;
  b.batch = batch;
  b.ldx = (n + 127) / 128 * 128;
  b.lda = (m + 63) / 64 * 64;
  b.parts = (int)(((int64_t)m * n + kPart - 1) / kPart);
  const bool small = muon_small_fits(m, n, planes);   // needs none
  // Three products of m in place of one of n and the slowest of the step: 2652 us against 2894
  // for 96 matrices 704 x 2816, 1376 against 1534 for 4 of 2048 x 7168; at n = 1.5 m (1024 x
  // 1536) 711 to 725 against 726 to 773, 64 of 512 x 768 650 against 630, at n = m as long.
  b.pair = planes == 1 && n >= 2ll * m;
  b.each = small ? 1 : 2 * x_bytes(b) + (b.pair ? 3ll : 2ll) * planes * m * b.lda * 2 + 8ll * b.parts;
  b.round = std::max<int64_t>(1, std::min<int64_t>(batch, std::min<int64_t>(kMaxRound, kScratch / b.each)));
  return b;
}

struct RoundLayout {
  size_t sums, x[2], a, b, c, parts, total;
};
RoundLayout layout_of(const Bucket& q) {
  RoundLayout L = {};
  size_t off = 256;
  L.total = off;
  if (muon_small_fits(q.m, q.n, q.planes)) return L;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~(size_t)255;
    return at;
  };
  L.sums = take((size_t)q.round * q.parts * 8);
  for (int i = 0; i < 2; ++i) L.x[i] = take((size_t)q.round * x_bytes(q));
  L.a = take((size_t)q.round * q.planes * q.m * q.lda * 2);
  L.b = take((size_t)q.round * q.planes * q.m * q.lda * 2);
  L.c = take(q.pair ? (size_t)q.round * q.planes * q.m * q.lda * 2 : 0);
  L.parts = take(orth_parts_bytes(q.round, q.m, q.n, q.planes));
  L.total = off;
  return L;
}

// Largest |a s + b s^3 + d s^5| and |b s^2 + d s^4| for s in [0, top].
void extremes(const double (&coef)[3], double top, double* x, double* y) {
  const double a = coef[0], b = coef[1], d = coef[2];
  *x = *y = 0.0;
  auto look = [&](double s2) {
    if (!(s2 > 0.0) || s2 > top * top) return;
    const double s = std::sqrt(s2);
    *x = std::max(*x, std::fabs(s * (a + s2 * (b + s2 * d))));
    *y = std::max(*y, std::fabs(s2 * (b + s2 * d)));
  };
  look(top * top);
  if (d != 0.0) {
    look(-b / (2.0 * d));
    const double disc = 9.0 * b * b - 20.0 * a * d;
    if (disc >= 0.0) {
      look((-3.0 * b + std::sqrt(disc)) / (10.0 * d));
      look((-3.0 * b - std::sqrt(disc)) / (10.0 * d));
    }
  } else if (b != 0.0) {
    look(-a / (3.0 * b));
  }
}

const char* check_coefs(const moe_orth_coefs& c) {
  if (c.steps < 1 || c.steps > MOE_ORTH_MAX_STEPS) return "steps must be in [1, MOE_ORTH_MAX_STEPS]";
  if (!(c.eps >= 0.0) || !std::isfinite(c.eps)) return "eps must be finite and >= 0";
  if (c.reserved != 0) return "reserved must be 0";
  double top = 1.0;   // of the singular values before the step
  for (int i = 0; i < c.steps; ++i) {
    for (double v : c.coef[i])
      if (!std::isfinite(v)) return "coefficients must be finite";
    double x, y;
    extremes(c.coef[i], top, &x, &y);
    if (!(x <= kOrthMaxX)) return "a step's coefficients take singular values past 3.5";
    if (!(y <= kOrthMaxB)) return "a step's b s^2 + c s^4 passes 100";
    top = x;
  }
  return nullptr;
}

// Whether R = a B' + a' B + B' B of the first two steps stays below its limit.
bool pair_fits(const moe_orth_coefs& c) {
  if (c.steps < 2) return false;
  double x0, y0, x1, y1;
  extremes(c.coef[0], 1.0, &x0, &y0);
  extremes(c.coef[1], x0, &x1, &y1);
  return std::fabs(c.coef[0][0]) * y1 + std::fabs(c.coef[1][0]) * y0 + y0 * y1 <= kOrthMaxR;
}

const char* check_sides(int64_t batch, int32_t rows, int32_t cols) {
  if (batch < 0 || batch > (1 << 24)) return "batch must be in [0, 2^24]";
  if (rows < 1 || cols < 1 || rows > 65536 || cols > 65536) return "rows and cols must be in [1, 65536]";
  return nullptr;
}

// One round: the update of the matrices in r's segments.
cudaError_t run_round(Round& r, const Bucket& q, const RoundLayout& L, char* ws, const moe_orth_coefs& c,
                      cudaStream_t st) {
  r.m = q.m;
  r.n = q.n;
  r.ldx = q.ldx;
  r.parts = q.parts;
  r.planes = q.planes;
  r.eps = c.eps;
  if (muon_small_fits(q.m, q.n, q.planes))
    return launch_muon_small(r, q.planes, c.steps, c.coef, reinterpret_cast<uint32_t*>(ws), st);
  r.sums = reinterpret_cast<double*>(ws + L.sums);
  r.x = reinterpret_cast<__half*>(ws + L.x[0]);
  const int64_t sms = tc_sm_count(), tiles = (int64_t)((q.m + kTile - 1) / kTile) * ((q.n + kTile - 1) / kTile) * r.batch;
  cudaError_t e = launch_after(momentum_kernel, (unsigned)std::min<int64_t>((int64_t)r.batch * q.parts, 16 * sms), 256, 0,
                               st, 1, r);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)std::min<int64_t>(tiles, 16 * sms);
  bool all16 = true;
  for (int i = 0; i < r.segs; ++i) all16 = all16 && r.seg[i].pdtype == MOE_BF16 && r.seg[i].gdtype == MOE_BF16;
  e = all16 ? launch_after(planes_kernel<true>, grid, 256, 0, st, 1, r) : launch_after(planes_kernel<false>, grid, 256, 0, st, 1, r);
  if (e != cudaSuccess) return e;
  OrthBatch t = {};
  t.batch = r.batch;
  t.m = q.m;
  t.n = q.n;
  t.ldx = q.ldx;
  t.lda = q.lda;
  t.planes = q.planes;
  t.x[0] = ws + L.x[0];
  t.x[1] = ws + L.x[1];
  t.a = ws + L.a;
  t.b = ws + L.b;
  t.c = q.pair && pair_fits(c) ? ws + L.c : nullptr;
  t.parts = reinterpret_cast<float*>(ws + L.parts);
  t.flags = reinterpret_cast<uint32_t*>(ws);
  int last = 0;
  e = launch_orth_steps(t, c.steps, c.coef, &last, st);
  if (e != cudaSuccess) return e;
  r.x = reinterpret_cast<__half*>(ws + L.x[last]);
  return all16 ? launch_after(update_kernel<true>, grid, 256, 0, st, 1, r)
               : launch_after(update_kernel<false>, grid, 256, 0, st, 1, r);
}

moe_status check_list(const moe_muon_tensor* t, int64_t n, const moe_muon_config* c, const char** why) {
  *why = nullptr;
  if (n < 0 || n > 65536 || (n > 0 && !t)) *why = "tensors must be an array of 0 to 65536 entries";
  else if (!c) *why = "config is NULL";
  else *why = check_coefs(c->coefs);
  if (*why) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(c->lr) || !std::isfinite(c->weight_decay) || !(c->momentum >= 0.0 && c->momentum < 1.0))
    *why = "lr and weight_decay must be finite, momentum in [0, 1)";
  else if (c->nesterov != 0 && c->nesterov != 1) *why = "nesterov must be 0 or 1";
  else if (c->scale < MOE_MUON_SCALE_NONE || c->scale > MOE_MUON_SCALE_RMS) *why = "scale must be a moe_muon_scale";
  if (*why) return MOE_ERR_INVALID_ARG;
  for (int64_t i = 0; i < n; ++i) {
    for (int32_t d : {t[i].param_dtype, t[i].grad_dtype})
      if (d != MOE_F32 && d != MOE_BF16) {
        *why = "dtypes must be MOE_F32 or MOE_BF16";
        return MOE_ERR_UNSUPPORTED;
      }
    *why = check_sides(t[i].batch, t[i].rows, t[i].cols);
    if (*why) return MOE_ERR_INVALID_ARG;
    if (t[i].batch == 0) continue;
    if (!t[i].param || !t[i].grad || !t[i].momentum) *why = "param, grad and momentum must be non-NULL";
    else if ((uintptr_t)t[i].param % (t[i].param_dtype == MOE_F32 ? 4 : 2) ||
             (uintptr_t)t[i].grad % (t[i].grad_dtype == MOE_F32 ? 4 : 2) || (uintptr_t)t[i].momentum % 4)
      *why = "param, grad and momentum must be aligned to their elements";
    if (*why) return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

struct Key {
  int m, n, planes;
};
Key key_of(const moe_muon_tensor& t) {
  return {std::min(t.rows, t.cols), std::max(t.rows, t.cols), t.param_dtype == MOE_F32 ? 2 : 1};
}
bool same(const Key& a, const Key& b) { return a.m == b.m && a.n == b.n && a.planes == b.planes; }

// Calls f(bucket, its first tensor) for every bucket, in the order of first tensors.
template <class F>
moe_status each_bucket(const moe_muon_tensor* t, int64_t n, F f) {
  for (int64_t i = 0; i < n; ++i) {
    const Key k = key_of(t[i]);
    bool seen = false;
    for (int64_t j = 0; j < i && !seen; ++j) seen = same(key_of(t[j]), k);
    if (seen) continue;
    int64_t batch = 0;
    for (int64_t j = i; j < n; ++j)
      if (same(key_of(t[j]), k)) batch += t[j].batch;
    if (batch == 0) continue;
    const moe_status st = f(bucket_of(k.m, k.n, k.planes, batch), i);
    if (st != MOE_OK) return st;
  }
  return MOE_OK;
}

float size_of(const moe_muon_config& c, const moe_muon_tensor& t) {
  double s = 1.0;
  if (c.scale == MOE_MUON_SCALE_SPECTRAL) s = std::sqrt(std::max(1.0, (double)t.rows / t.cols));
  if (c.scale == MOE_MUON_SCALE_RMS) s = 0.2 * std::sqrt((double)std::max(t.rows, t.cols));
  return (float)(c.lr * s);
}

moe_status check_shape(const moe_orth_shape* s, const moe_orth_coefs* c, const char** why) {
  *why = nullptr;
  if (!s || !c) *why = "shape and coefs must be non-NULL";
  else if (s->dtype != MOE_F32 && s->dtype != MOE_BF16) {
    *why = "dtype must be MOE_F32 or MOE_BF16";
    return MOE_ERR_UNSUPPORTED;
  } else if (s->reserved != 0) *why = "reserved must be 0";
  else *why = check_sides(s->batch, s->rows, s->cols);
  if (!*why) *why = check_coefs(*c);
  return *why ? MOE_ERR_INVALID_ARG : MOE_OK;
}
Bucket bucket_of(const moe_orth_shape& s) {
  return bucket_of(std::min(s.rows, s.cols), std::max(s.rows, s.cols), s.dtype == MOE_F32 ? 2 : 1, s.batch);
}

}  // namespace muon
}  // namespace moe

using namespace moe;

extern "C" size_t moe_orthogonalize_workspace_bytes(const moe_orth_shape* shape, const moe_orth_coefs* coefs) {
  const char* why;
  const moe_status st = muon::check_shape(shape, coefs, &why);
  if (st != MOE_OK) {
    fail(st, why);
    return 0;
  }
  return muon::layout_of(muon::bucket_of(*shape)).total;
}

extern "C" moe_status moe_orthogonalize(const moe_orth_shape* shape, const moe_orth_coefs* coefs, const void* x,
                                        void* out, void* ws, size_t ws_bytes, void* stream) {
  reset_launch_count();
  const char* why;
  moe_status st = muon::check_shape(shape, coefs, &why);
  if (st != MOE_OK) return fail(st, why);
  if (shape->batch > 0 && (!x || !out)) return fail(MOE_ERR_INVALID_ARG, "x and out must be non-NULL");
  const size_t esz = shape->dtype == MOE_F32 ? 4 : 2;
  if ((uintptr_t)x % esz || (uintptr_t)out % esz) return fail(MOE_ERR_INVALID_ARG, "x and out must be aligned to their elements");
  const muon::Bucket q = muon::bucket_of(*shape);
  const muon::RoundLayout L = muon::layout_of(q);
  st = check_ws(ws, ws_bytes, L.total);
  if (st != MOE_OK) return st;
  for (int64_t at = 0; at < shape->batch; at += q.round) {
    muon::Round r = {};
    r.batch = (int32_t)std::min<int64_t>(q.round, shape->batch - at);
    r.segs = 1;
    r.seg[0] = {out, x, nullptr, at, 0, r.batch, shape->rows, shape->cols, shape->dtype, shape->dtype, 0.0f};
    CHECK_CUDA(muon::run_round(r, q, L, static_cast<char*>(ws), *coefs, (cudaStream_t)stream));
  }
  return MOE_OK;
}

extern "C" size_t moe_muon_workspace_bytes(const moe_muon_tensor* tensors, int64_t n, const moe_muon_config* config) {
  const char* why;
  const moe_status st = muon::check_list(tensors, n, config, &why);
  if (st != MOE_OK) {
    fail(st, why);
    return 0;
  }
  size_t need = 256;
  muon::each_bucket(tensors, n, [&](const muon::Bucket& q, int64_t) {
    need = std::max(need, muon::layout_of(q).total);
    return MOE_OK;
  });
  return need;
}

extern "C" moe_status moe_muon_step(const moe_muon_tensor* tensors, int64_t n, const moe_muon_config* config, void* ws,
                                    size_t ws_bytes, void* stream) {
  reset_launch_count();
  const char* why;
  moe_status st = muon::check_list(tensors, n, config, &why);
  if (st != MOE_OK) return fail(st, why);
  st = check_ws(ws, ws_bytes, moe_muon_workspace_bytes(tensors, n, config));
  if (st != MOE_OK) return st;
  return muon::each_bucket(tensors, n, [&](const muon::Bucket& q, int64_t i) -> moe_status {
    const muon::RoundLayout L = muon::layout_of(q);
    const muon::Key k = muon::key_of(tensors[i]);
    muon::Round r = {};
    auto flush = [&]() -> moe_status {
      if (r.batch == 0) return MOE_OK;
      CHECK_CUDA(muon::run_round(r, q, L, static_cast<char*>(ws), config->coefs, (cudaStream_t)stream));
      r = {};
      return MOE_OK;
    };
    for (int64_t j = i; j < n; ++j) {
      const moe_muon_tensor& t = tensors[j];
      if (!muon::same(muon::key_of(t), k)) continue;
      for (int64_t at = 0; at < t.batch;) {
        if (r.segs == muon::kSegs || r.batch == q.round) {
          const moe_status e = flush();
          if (e != MOE_OK) return e;
        }
        const int32_t m = (int32_t)std::min<int64_t>(t.batch - at, q.round - r.batch);
        r.seg[r.segs++] = {t.param, t.grad, t.momentum, at, r.batch, m, t.rows, t.cols, t.param_dtype, t.grad_dtype,
                           muon::size_of(*config, t)};
        r.batch += m;
        r.update = 1;
        r.nesterov = config->nesterov;
        r.beta = (float)config->momentum;
        r.rest = (float)(1.0 - config->momentum);
        r.keep = (float)(1.0 - config->lr * config->weight_decay);
        at += m;
      }
    }
    return flush();
  });
}
