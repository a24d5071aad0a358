// norm.hpp - layer norm over the rows of a matrix, forward and backward.
//
//   mean_i = sum_j x_ij / n,  rstd_i = 1 / sqrt(sum_j (x_ij - mean_i)^2 / n + eps)
//   xhat = (x - mean) rstd,   y = w xhat + b
//   a = w dy,  dx = rstd (a - mean_j(a) - xhat mean_j(a xhat))
//   dw_j = sum_i dy_ij xhat_ij,   db_j = sum_i dy_ij
//
// Both passes are bound by memory: forward reads and writes each element
// once, backward reads x and dy and writes dx once.  A row therefore lives in
// registers from its one read to its one write: TPR threads hold NV vectors
// of 16 bytes each.  (The backward builds of 1024 threads, for rows past 8192
// columns, have more than their 128 registers to hold and spill.)  The
// variance is the sum of squared deviations from the finished mean, taken
// over the registers, so it does not lose its digits when the mean is large
// against the spread.  All statistics and sums are fp32; y, dx, dw and db are
// rounded once when stored.
//
// Measured (MI355X, bf16): forward 16384 x 768 13 us (3.9 TB/s, a launch's
// ramp included), 8192 x 4096 24 us (5.6 TB/s), one row of 4096 2.6 us;
// backward 8192 x 4096 42 us (4.7 TB/s) and 4 us for the parameters' join,
// 4096 x 12288 523 us (0.57 TB/s: the spills).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "products.hpp"

namespace nsk {

// ---------------------------------------------------------------------------
// Rows in 16-byte vectors at any element boundary.  The hardware takes
// unaligned vector loads and stores, so rows of an odd width (all but the
// first off every boundary) go in vectors too; only a row's last, partial
// vector is taken element by element.
// ---------------------------------------------------------------------------
template <typename IO> inline constexpr int kVec = 16 / (int)sizeof(IO);
template <int ALIGN> struct Vec16;
template <> struct Vec16<4> {
  typedef u32x4_t type __attribute__((aligned(4)));
};
template <> struct Vec16<2> {
  typedef u32x4_t type __attribute__((aligned(2)));
};

// How a row's width meets the vectors; a template argument, so that each
// build holds only its own case.
enum RowForm {
  kEven = 0,    // whole vectors
  kRagged = 1,  // a partial vector at the end
  kTiny = 2     // less than one vector
};

// Loading goes in two steps, so that the loads of a whole batch are in flight
// before the first is looked at.  issue16 loads without a branch: a lane whose
// vector would pass the row's end takes the row's last kVec columns instead.
// settle16 then moves those to their place and zeroes what lies past the row.
template <int FORM, typename IO>
__device__ __forceinline__ u32x4_t issue16(const IO* row, int c, int cols) {
  constexpr int V = kVec<IO>;
  if constexpr (FORM == kTiny) return u32x4_t{0u, 0u, 0u, 0u};
  return *reinterpret_cast<const typename Vec16<sizeof(IO)>::type*>(row + (c + V <= cols ? c : cols - V));
}
template <int FORM, typename IO>
__device__ __forceinline__ u32x4_t settle16(u32x4_t q, const IO* row, int c, int cols) {
  constexpr int V = kVec<IO>;
  if constexpr (FORM == kTiny) {
    IO* e = reinterpret_cast<IO*>(&q);
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (c + k < cols) e[k] = row[c + k];
    return q;
  }
  const int s = c + V - cols;  // elements past the end
  if constexpr (FORM == kRagged) {
    // Down by s elements where 0 < s < V, in steps of 8, 4 and 2 bytes.
    const int bytes = s > 0 ? s * (int)sizeof(IO) : 0;
    q = bytes & 8 ? u32x4_t{q[2], q[3], 0u, 0u} : q;
    q = bytes & 4 ? u32x4_t{q[1], q[2], q[3], 0u} : q;
    if constexpr (sizeof(IO) == 2)
      q = bytes & 2 ? u32x4_t{(q[0] >> 16) | (q[1] << 16), (q[1] >> 16) | (q[2] << 16), (q[2] >> 16) | (q[3] << 16),
                              q[3] >> 16}
                    : q;
  }
  return s >= V ? u32x4_t{0u, 0u, 0u, 0u} : q;
}

template <typename IO>
__device__ __forceinline__ void unpack(const u32x4_t& q, float (&f)[kVec<IO>]) {
  const IO* e = reinterpret_cast<const IO*>(&q);
#pragma unroll
  for (int k = 0; k < kVec<IO>; ++k) f[k] = to_f32<IO>(e[k]);
}

// Rounds and stores columns c .. c + kVec - 1, up to `cols`.
template <int FORM, typename IO>
__device__ __forceinline__ void store16v(IO* row, int c, int cols, const float (&f)[kVec<IO>]) {
  constexpr int V = kVec<IO>;
  u32x4_t q;
  IO* e = reinterpret_cast<IO*>(&q);
#pragma unroll
  for (int k = 0; k < V; ++k) e[k] = from_f32<IO>(f[k]);
  if (c + V <= cols) {
    *reinterpret_cast<typename Vec16<sizeof(IO)>::type*>(row + c) = q;
  } else if constexpr (FORM != kEven) {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (c + k < cols) row[c + k] = e[k];
  }
}

// V consecutive parameters as raw vectors (one, or two fp32 ones beside
// 16-bit data), and as floats.
template <int FORM, typename PT, int V>
struct Params {
  static constexpr int PV = kVec<PT>, N = V / PV;
  static_assert(V % PV == 0, "a data vector holds whole parameter vectors");
  u32x4_t q[N];
  __device__ __forceinline__ void issue(const PT* p, int c, int cols) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = issue16<FORM, PT>(p, c + i * PV, cols);
  }
  __device__ __forceinline__ void settle(const PT* p, int c, int cols) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = settle16<FORM, PT>(q[i], p, c + i * PV, cols);
  }
  __device__ __forceinline__ float get(int k) const {
    return to_f32<PT>(reinterpret_cast<const PT*>(&q[k / PV])[k % PV]);
  }
};

template <typename IO, int V>
__device__ __forceinline__ bool rounds_to_nonfinite(const float (&f)[V]) {
  bool bad = false;
#pragma unroll
  for (int k = 0; k < V; ++k) bad |= !(fabsf(f[k]) < kRoundsToInf<IO>);
  return bad;
}

// ---------------------------------------------------------------------------
// Sum over the TPR threads of a row; every thread gets it, in a fixed order.
// Within a wave the lanes exchange registers directly (data-parallel moves in
// a row of 16 lanes, the row and half swaps across them), which saves the
// round trips through the LDS crossbar that a shuffle takes.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false);
  return v + __builtin_bit_cast(float, o);
}
template <int TPR>
__device__ __forceinline__ float wave_row_sum(float v) {
  v = add_dpp<0xB1>(v);   // lane ^ 1
  v = add_dpp<0x4E>(v);   // lane ^ 2
  v = add_dpp<0x141>(v);  // mirrored in 8: the other quad
  v = add_dpp<0x140>(v);  // mirrored in 16: the other 8
  uint32_t u = __float_as_uint(v);
  auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  if constexpr (TPR >= 64) {
    u = __float_as_uint(v);
    p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return v;
}

// N sums at once; `sh` holds N floats per wave and is used when a row is
// more than a wave.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* sh) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = wave_row_sum<TPR>(v[j]);
  if constexpr (TPR > 64) {
    constexpr int kWaves = TPR / 64;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int j = 0; j < N; ++j) sh[(threadIdx.x >> 6) * N + j] = v[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      v[j] = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) v[j] += sh[i * N + j];
    }
    __syncthreads();
  }
}
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* sh) {
  float s[1] = {v};
  row_sums<TPR, 1>(s, sh);
  return s[0];
}

// Rows handled by one block at a time: rows of up to a wave share a block of
// 256 threads, wider ones have a block of their own.
template <int TPR> inline constexpr int kNormThreads = TPR <= 64 ? 256 : TPR;
template <int TPR> inline constexpr int kNormRows = kNormThreads<TPR> / TPR;

struct NormFwdArgs {
  const void* X;
  void* Y;
  const void *W, *B;   // either may be null (1 and 0)
  float *mean, *rstd;  // either may be null
  int64_t rows, ldx, ldy;
  int cols;
  float eps;
  int32_t* d_status;
  int32_t status_bits;
};

// A block walks rows blockIdx.x, + gridDim.x, ... (groups of kNormRows).
// A block of one wide row keeps the parameters in registers and loads its next
// row while it works on one; narrow rows, several to a block, take the
// parameters from the cache for each row: their registers are worth more as
// waves in flight.
template <typename IO, typename PT, int NV, int TPR, int FORM>
__global__ void __launch_bounds__(kNormThreads<TPR>) k_norm_fwd(NormFwdArgs p) {
  constexpr int V = kVec<IO>;
  __shared__ float sh[kNormThreads<TPR> / 64];
  const int t = threadIdx.x % TPR;
  const float n = (float)p.cols;
  auto in = [&](int c, int k) { return (FORM == kEven ? c : c + k) < p.cols; };  // column c + k is in the row
  const PT *W = reinterpret_cast<const PT*>(p.W), *B = reinterpret_cast<const PT*>(p.B);
  const int64_t stride = (int64_t)gridDim.x * kNormRows<TPR>;
  int64_t row = (int64_t)blockIdx.x * kNormRows<TPR> + threadIdx.x / TPR;
  u32x4_t raw[NV];
  auto fetch = [&](int64_t r) {
    const IO* x = reinterpret_cast<const IO*>(p.X) + r * p.ldx;
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i] = issue16<FORM, IO>(x, (i * TPR + t) * V, p.cols);
  };
  Params<FORM, PT, V> w[NV], b[NV];
  auto fetch_params = [&] {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (W) w[i].issue(W, (i * TPR + t) * V, p.cols);
      if (B) b[i].issue(B, (i * TPR + t) * V, p.cols);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (W) w[i].settle(W, (i * TPR + t) * V, p.cols);
      if (B) b[i].settle(B, (i * TPR + t) * V, p.cols);
    }
  };
  constexpr bool kHold = TPR > 64;
  if (kHold && row < p.rows) {
    fetch(row);
    fetch_params();
  }
  bool bad = false;
  // The trip count differs between the threads of a block only when a row is
  // at most a wave, and then no barrier is inside.
  for (; row < p.rows; row += stride) {
    const IO* x = reinterpret_cast<const IO*>(p.X) + row * p.ldx;
    if (!kHold) fetch(row);
    float f[NV][V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack<IO>(settle16<FORM, IO>(raw[i], x, (i * TPR + t) * V, p.cols), f[i]);
#pragma unroll
      for (int k = 0; k < V; ++k) s += f[i][k];
    }
    if (kHold && row + stride < p.rows) fetch(row + stride);
    const float mean = row_sum<TPR>(s, sh) / n;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        f[i][k] -= mean;
        q = in(c, k) ? fmaf(f[i][k], f[i][k], q) : q;
      }
    }
    // Squares past fp32 make rstd 0, and y finite but not the formula's: reported.
    const float var = row_sum<TPR>(q, sh) / n, rstd = 1.f / sqrtf(var + p.eps);
    bad |= !(var < __builtin_inff());
    if constexpr (!kHold) fetch_params();
    IO* y = reinterpret_cast<IO*>(p.Y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      if (c >= p.cols) continue;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        f[i][k] *= rstd;
        if (W) f[i][k] *= w[i].get(k);
        if (B) f[i][k] += b[i].get(k);
        bad |= in(c, k) && !(fabsf(f[i][k]) < kRoundsToInf<IO>);
      }
      store16v<FORM, IO>(y, c, p.cols, f[i]);
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
  const PT *W = reinterpret_cast<const PT*>(p.W), *B = reinterpret_cast<const PT*>(p.B);
  const float n = (float)p.cols;
  bool bad = false;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const IO* x = reinterpret_cast<const IO*>(p.X) + row * p.ldx;
    IO* y = reinterpret_cast<IO*>(p.Y) + row * p.ldy;
    float s = 0.f, q = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += 1024) s += to_f32<IO>(x[c]);
    const float mean = row_sum<1024>(s, sh) / n;
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float d = to_f32<IO>(x[c]) - mean;
      q = fmaf(d, d, q);
    }
    const float var = row_sum<1024>(q, sh) / n, rstd = 1.f / sqrtf(var + p.eps);
    bad |= !(var < __builtin_inff());
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
// The blocks are few (their partials are written and read again), so a block
// loads its next row while it works on one.
template <typename IO, typename PT, int NV, int TPR, int FORM>
__global__ void __launch_bounds__(kNormThreads<TPR>) k_norm_bwd(NormBwdArgs p) {
  constexpr int V = kVec<IO>, R = kNormRows<TPR>;
  __shared__ float sh[kNormThreads<TPR> / 64 * 2];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  float dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) dw[i][k] = db[i][k] = 0.f;
  const float inv_n = 1.f / (float)p.cols;
  auto in = [&](int c, int k) { return (FORM == kEven ? c : c + k) < p.cols; };  // column c + k is in the row
  const int64_t stride = (int64_t)gridDim.x * R;
  int64_t row = (int64_t)blockIdx.x * R + sub;
  u32x4_t rx[NV], rg[NV];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](int64_t r) {
    const IO* x = reinterpret_cast<const IO*>(p.X) + r * p.ldx;
    const IO* dy = reinterpret_cast<const IO*>(p.dY) + r * p.lddy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      rx[i] = issue16<FORM, IO>(x, c, p.cols);
      rg[i] = issue16<FORM, IO>(dy, c, p.cols);
    }
    mean = p.mean[r];
    rstd = p.rstd[r];
  };
  const PT* W = reinterpret_cast<const PT*>(p.W);
  Params<FORM, PT, V> w[NV];
  if (row < p.rows) {
    fetch(row);
    if (W) {
#pragma unroll
      for (int i = 0; i < NV; ++i) w[i].issue(W, (i * TPR + t) * V, p.cols);
#pragma unroll
      for (int i = 0; i < NV; ++i) w[i].settle(W, (i * TPR + t) * V, p.cols);
    }
  }
  bool bad = false;
  for (; row < p.rows; row += stride) {
    float xh[NV][V], a[NV][V];
    float s[2] = {0.f, 0.f};
    const float r = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      unpack<IO>(settle16<FORM, IO>(rx[i], reinterpret_cast<const IO*>(p.X) + row * p.ldx, c, p.cols), xh[i]);
      unpack<IO>(settle16<FORM, IO>(rg[i], reinterpret_cast<const IO*>(p.dY) + row * p.lddy, c, p.cols), a[i]);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        // Past the row dy is zero and xhat some number that meets it only.
        xh[i][k] = (xh[i][k] - mean) * r;
        dw[i][k] = fmaf(a[i][k], xh[i][k], dw[i][k]);
        db[i][k] += a[i][k];
        if (W) a[i][k] *= w[i].get(k);
        s[0] += a[i][k];
        s[1] = fmaf(a[i][k], xh[i][k], s[1]);
      }
    }
    if (row + stride < p.rows) fetch(row + stride);
    row_sums<TPR, 2>(s, sh);
    const float c1 = s[0] * inv_n, c2 = s[1] * inv_n;
    IO* dx = reinterpret_cast<IO*>(p.dX) + row * p.lddx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      if (c >= p.cols) continue;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        a[i][k] = r * (a[i][k] - c1 - xh[i][k] * c2);
        bad |= in(c, k) && !(fabsf(a[i][k]) < kRoundsToInf<IO>);
      }
      store16v<FORM, IO>(dx, c, p.cols, a[i]);
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
  if (!p.partial) return;
  float* out = p.partial + (int64_t)blockIdx.x * 2 * p.cols;
  if constexpr (R > 1) {
    // The block's rows join in their order.
    __shared__ float join[2 * NV * V * TPR];
    for (int j = 0; j < R; ++j) {
      if (sub == j) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) {
            float* q = join + (i * V + k) * 2 * TPR + t;
            if (j > 0) {
              dw[i][k] += q[0];
              db[i][k] += q[TPR];
            }
            q[0] = dw[i][k];
            q[TPR] = db[i][k];
          }
      }
      __syncthreads();
    }
    if (sub != R - 1) return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + t) * V;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (in(c, k)) {
        out[c + k] = dw[i][k];
        out[p.cols + c + k] = db[i][k];
      }
    }
  }
}

// Rows too long for registers: dx here, the parameters' gradients in
// k_norm_cols.
template <typename IO, typename PT>
__global__ void __launch_bounds__(1024) k_norm_bwd_long(NormBwdArgs p) {
  __shared__ float sh[32];
  const PT* W = reinterpret_cast<const PT*>(p.W);
  const float inv_n = 1.f / (float)p.cols;
  bool bad = false;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const IO* x = reinterpret_cast<const IO*>(p.X) + row * p.ldx;
    const IO* dy = reinterpret_cast<const IO*>(p.dY) + row * p.lddy;
    IO* dx = reinterpret_cast<IO*>(p.dX) + row * p.lddx;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float a = to_f32<IO>(dy[c]) * (W ? to_f32<PT>(W[c]) : 1.f);
      s[0] += a;
      s[1] = fmaf(a, (to_f32<IO>(x[c]) - mean) * rstd, s[1]);
    }
    row_sums<1024, 2>(s, sh);
    const float c1 = s[0] * inv_n, c2 = s[1] * inv_n;
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
__global__ void __launch_bounds__(1024) k_norm_join(const float* partial, int parts, int cols, PT* dw, PT* db,
                                                    int32_t* d_status, int32_t status_bits) {
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
    PT* out = c < cols ? dw : db;
    if (out) out[c < cols ? c : c - cols] = from_f32<PT>(s);
    if (d_status) report_status(d_status, status_bits, out && !(fabsf(s) < kRoundsToInf<PT>));
  }
}

}  // namespace nsk
