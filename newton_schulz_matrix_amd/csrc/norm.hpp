// norm.hpp - layer norm over the rows of a matrix, forward and backward.
//
//   mean_i = sum_j x_ij / n,  rstd_i = 1 / sqrt(sum_j (x_ij - mean_i)^2 / n + eps)
//   xhat = (x - mean) rstd,   y = w xhat + b
//   a = w dy,  dx = rstd (a - mean_j(a) - xhat mean_j(a xhat))
//   dw_j = sum_i dy_ij xhat_ij,   db_j = sum_i dy_ij
//
// Both passes are bound by memory: forward reads and writes each element
// once, backward reads x and dy and writes dx once.  A row therefore lives in
// registers from its one read to its one write: TPR threads hold E elements
// each, in 16-byte vectors where the row allows it (V elements), one by one
// otherwise (V = 1).  The variance is the sum of squared deviations from the
// finished mean, taken over the registers, so it does not lose its digits
// when the mean is large against the spread.  All statistics and sums are
// fp32; y, dx, dw and db are rounded once when stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "products.hpp"

namespace nsk {

// V consecutive elements of a row as floats; V = 1 is the unaligned form.
template <typename IO, int V>
__device__ __forceinline__ void load_vec(const IO* p, float (&f)[V]) {
  if constexpr (V * sizeof(IO) == 16) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const IO* e = reinterpret_cast<const IO*>(&q);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = to_f32<IO>(e[k]);
  } else if constexpr (V * sizeof(IO) == 32) {
    const uint4 q0 = reinterpret_cast<const uint4*>(p)[0], q1 = reinterpret_cast<const uint4*>(p)[1];
    const IO *e0 = reinterpret_cast<const IO*>(&q0), *e1 = reinterpret_cast<const IO*>(&q1);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      f[k] = to_f32<IO>(e0[k]);
      f[V / 2 + k] = to_f32<IO>(e1[k]);
    }
  } else {
    static_assert(V == 1, "a vector is 16 or 32 bytes");
    f[0] = to_f32<IO>(*p);
  }
}

template <typename IO, int V>
__device__ __forceinline__ void store_vec(IO* p, const float (&f)[V]) {
  if constexpr (V * sizeof(IO) == 16) {
    uint4 q;
    IO* e = reinterpret_cast<IO*>(&q);
#pragma unroll
    for (int k = 0; k < V; ++k) e[k] = from_f32<IO>(f[k]);
    *reinterpret_cast<uint4*>(p) = q;
  } else {
    static_assert(V == 1, "a vector is 16 bytes");
    p[0] = from_f32<IO>(f[0]);
  }
}

template <typename IO, int V>
__device__ __forceinline__ bool rounds_to_nonfinite(const float (&f)[V]) {
  bool bad = false;
#pragma unroll
  for (int k = 0; k < V; ++k) bad |= !(fabsf(f[k]) < kRoundsToInf<IO>);
  return bad;
}

// Sum of one float per thread over the TPR threads of a row; every thread of
// the row gets it, the same value in a fixed order.  `sh` holds one float
// per wave and is not touched when a row is one wave.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* sh) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  if constexpr (TPR > 64) {
    constexpr int kWaves = TPR / 64;
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) v += sh[i];
    __syncthreads();
  }
  return v;
}

// Rows handled by one block: four one-wave rows, or one.
template <int TPR> inline constexpr int kNormThreads = TPR == 64 ? 256 : TPR;
template <int TPR> inline constexpr int kNormRows = kNormThreads<TPR> / TPR;

struct NormFwdArgs {
  const void* X;
  void* Y;
  const void *W, *B;  // either may be null (1 and 0)
  float *mean, *rstd;  // either may be null
  int64_t rows, ldx, ldy;
  int cols;
  float eps;
  int32_t* d_status;
  int32_t status_bits;
};

template <typename IO, typename PT, int V, int E, int TPR>
__global__ void __launch_bounds__(kNormThreads<TPR>) k_norm_fwd(NormFwdArgs p) {
  constexpr int NV = E / V;
  __shared__ float sh[kNormThreads<TPR> / 64];
  const int t = threadIdx.x % TPR;
  bool bad = false;
  // The trip count differs between the waves of a block only when a row is
  // one wave, and then no barrier is inside.
  for (int64_t row = (int64_t)blockIdx.x * kNormRows<TPR> + threadIdx.x / TPR; row < p.rows;
       row += (int64_t)gridDim.x * kNormRows<TPR>) {
    const IO* x = reinterpret_cast<const IO*>(p.X) + row * p.ldx;
    float f[NV][V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      if (c < p.cols) {
        load_vec<IO, V>(x + c, f[i]);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) f[i][k] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) s += f[i][k];
    const float n = (float)p.cols;
    const float mean = row_sum<TPR>(s, sh) / n;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = (i * TPR + t) * V < p.cols;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        f[i][k] -= mean;
        q = in ? fmaf(f[i][k], f[i][k], q) : q;
      }
    }
    const float rstd = 1.f / sqrtf(row_sum<TPR>(q, sh) / n + p.eps);
    IO* y = reinterpret_cast<IO*>(p.Y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      if (c >= p.cols) continue;
      float w[V], b[V];
      if (p.W) load_vec<PT, V>(reinterpret_cast<const PT*>(p.W) + c, w);
      if (p.B) load_vec<PT, V>(reinterpret_cast<const PT*>(p.B) + c, b);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        f[i][k] *= rstd;
        if (p.W) f[i][k] *= w[k];
        if (p.B) f[i][k] += b[k];
      }
      bad |= rounds_to_nonfinite<IO, V>(f[i]);
      store_vec<IO, V>(y + c, f[i]);
    }
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
}

// Rows too long for registers: three passes over the row, the later two
// served by the cache.
template <typename IO, typename PT>
__global__ void __launch_bounds__(1024) k_norm_fwd_long(NormFwdArgs p) {
  __shared__ float sh[16];
  bool bad = false;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const IO* x = reinterpret_cast<const IO*>(p.X) + row * p.ldx;
    IO* y = reinterpret_cast<IO*>(p.Y) + row * p.ldy;
    const PT *W = reinterpret_cast<const PT*>(p.W), *B = reinterpret_cast<const PT*>(p.B);
    const float n = (float)p.cols;
    float s = 0.f, q = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) s += to_f32<IO>(x[c]);
    const float mean = row_sum<1024>(s, sh) / n;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float d = to_f32<IO>(x[c]) - mean;
      q = fmaf(d, d, q);
    }
    const float rstd = 1.f / sqrtf(row_sum<1024>(q, sh) / n + p.eps);
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      float v = (to_f32<IO>(x[c]) - mean) * rstd;
      if (W) v *= to_f32<PT>(W[c]);
      if (B) v += to_f32<PT>(B[c]);
      bad |= !(fabsf(v) < kRoundsToInf<IO>);
      y[c] = from_f32<IO>(v);
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
}

// ---------------------------------------------------------------------------
// Backward.
// ---------------------------------------------------------------------------
struct NormBwdArgs {
  const void *dY, *X, *W;  // W may be null (1)
  void* dX;
  const float *mean, *rstd;
  float* partial;  // [blocks][2][cols]: this block's share of dw and db; null when neither is wanted
  int64_t rows, lddy, ldx, lddx;
  int cols;
  int32_t* d_status;
  int32_t status_bits;
};

// Each block walks rows blockIdx.x, blockIdx.x + gridDim.x, ... (groups of
// kNormRows) and keeps its columns' dw and db in registers; they leave once,
// as one partial row per block, so the sums' order is fixed by the sizes.
template <typename IO, typename PT, int V, int E, int TPR>
__global__ void __launch_bounds__(kNormThreads<TPR>) k_norm_bwd(NormBwdArgs p) {
  constexpr int NV = E / V, R = kNormRows<TPR>;
  __shared__ float sh[kNormThreads<TPR> / 64];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  float dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) dw[i][k] = db[i][k] = 0.f;
  const float inv_n = 1.f / (float)p.cols;
  bool bad = false;
  for (int64_t row = (int64_t)blockIdx.x * R + sub; row < p.rows; row += (int64_t)gridDim.x * R) {
    const IO* x = reinterpret_cast<const IO*>(p.X) + row * p.ldx;
    const IO* dy = reinterpret_cast<const IO*>(p.dY) + row * p.lddy;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float xh[NV][V], a[NV][V];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      if (c < p.cols) {
        load_vec<IO, V>(x + c, xh[i]);
        load_vec<IO, V>(dy + c, a[i]);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) xh[i][k] = a[i][k] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      if (c >= p.cols) continue;
      float w[V];
      if (p.W) load_vec<PT, V>(reinterpret_cast<const PT*>(p.W) + c, w);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        xh[i][k] = (xh[i][k] - mean) * rstd;
        dw[i][k] = fmaf(a[i][k], xh[i][k], dw[i][k]);
        db[i][k] += a[i][k];
        if (p.W) a[i][k] *= w[k];
        s1 += a[i][k];
        s2 = fmaf(a[i][k], xh[i][k], s2);
      }
    }
    const float c1 = row_sum<TPR>(s1, sh) * inv_n, c2 = row_sum<TPR>(s2, sh) * inv_n;
    IO* dx = reinterpret_cast<IO*>(p.dX) + row * p.lddx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      if (c >= p.cols) continue;
#pragma unroll
      for (int k = 0; k < V; ++k) a[i][k] = rstd * (a[i][k] - c1 - xh[i][k] * c2);
      bad |= rounds_to_nonfinite<IO, V>(a[i]);
      store_vec<IO, V>(dx + c, a[i]);
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
  if (!p.partial) return;
  float* out = p.partial + (int64_t)blockIdx.x * 2 * p.cols;
  if constexpr (R > 1) {
    // The four one-wave rows of the block join in wave order.
    __shared__ float join[2 * E * 64];
    for (int r = 0; r < R; ++r) {
      if (sub == r) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) {
            float* j = join + ((i * V + k) * 2) * 64 + t;
            if (r > 0) {
              dw[i][k] += j[0];
              db[i][k] += j[64];
            }
            j[0] = dw[i][k];
            j[64] = db[i][k];
          }
      }
      __syncthreads();
    }
    if (sub != R - 1) return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * V;
    if (c >= p.cols) continue;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      out[c + k] = dw[i][k];
      out[p.cols + c + k] = db[i][k];
    }
  }
}

// Rows too long for registers: dx here, the parameters' gradients in
// k_norm_cols.
template <typename IO, typename PT>
__global__ void __launch_bounds__(1024) k_norm_bwd_long(NormBwdArgs p) {
  __shared__ float sh[16];
  bool bad = false;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const IO* x = reinterpret_cast<const IO*>(p.X) + row * p.ldx;
    const IO* dy = reinterpret_cast<const IO*>(p.dY) + row * p.lddy;
    IO* dx = reinterpret_cast<IO*>(p.dX) + row * p.lddx;
    const PT* W = reinterpret_cast<const PT*>(p.W);
    const float mean = p.mean[row], rstd = p.rstd[row], inv_n = 1.f / (float)p.cols;
    float s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float a = to_f32<IO>(dy[c]) * (W ? to_f32<PT>(W[c]) : 1.f);
      s1 += a;
      s2 = fmaf(a, (to_f32<IO>(x[c]) - mean) * rstd, s2);
    }
    const float c1 = row_sum<1024>(s1, sh) * inv_n, c2 = row_sum<1024>(s2, sh) * inv_n;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float a = to_f32<IO>(dy[c]) * (W ? to_f32<PT>(W[c]) : 1.f);
      const float v = rstd * (a - c1 - (to_f32<IO>(x[c]) - mean) * rstd * c2);
      bad |= !(fabsf(v) < kRoundsToInf<IO>);
      dx[c] = from_f32<IO>(v);
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
}

// partial[blockIdx.y][{dw, db}][c] over the rows blockIdx.y, + gridDim.y, ...
template <typename IO>
__global__ void __launch_bounds__(256) k_norm_cols(NormBwdArgs p) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float dw = 0.f, db = 0.f;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float g = to_f32<IO>(reinterpret_cast<const IO*>(p.dY)[row * p.lddy + c]);
    const float x = to_f32<IO>(reinterpret_cast<const IO*>(p.X)[row * p.ldx + c]);
    dw = fmaf(g, (x - p.mean[row]) * p.rstd[row], dw);
    db += g;
  }
  float* out = p.partial + (int64_t)blockIdx.y * 2 * p.cols;
  out[c] = dw;
  out[p.cols + c] = db;
}

// dw and db from `parts` partial rows: 16 groups of threads take every 16th
// partial of 64 columns each, and join in a fixed order.
template <typename PT>
__global__ void __launch_bounds__(1024) k_norm_join(const float* partial, int parts, int cols, PT* dw, PT* db) {
  __shared__ float sh[16][64];
  const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane, width = 2 * (int64_t)cols;
  float s = 0.f;
  if (c < width) {
#pragma unroll 8
    for (int i = g; i < parts; i += 16) s += partial[i * width + c];
  }
  sh[g][lane] = s;
  __syncthreads();
  if (g == 0 && c < width) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sh[i][lane];
    if (c < cols) {
      if (dw) dw[c] = from_f32<PT>(s);
    } else {
      if (db) db[c - cols] = from_f32<PT>(s);
    }
  }
}

}  // namespace nsk
