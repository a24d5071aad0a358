// resnorm.hpp - the root-mean-square norms before and after a block, fused
// with the block's gate and the scaled residual, forward and backward.
//
//   rb_i = 1 / sqrt(sum_j z_ij^2 / n + eps),  bhat = z rb,  nb = bhat wb
//   s = scale x + gate nb                                 (the new stream)
//   rs_i = 1 / sqrt(sum_j s_ij^2 / n + eps),  shat = s rs,  y = shat w
//
//   u = w dy,    G = ds + rs (u - shat mean_j(u shat)),   dx = scale G
//   q = gate G,  a = wb q,  dz = rb (a - bhat mean_j(a bhat))
//   dgate = sum over the gate's rows of G nb
//   dwb_j = sum_i q bhat,   dw_j = sum_i dy shat
//
// Both passes are bound by memory: forward reads x and z and writes s and y,
// backward reads ds, dy, s and z and writes dx and dz, each once, where the
// steps one by one would take two and a half times that.  As in norm.hpp a
// row lives in registers from its one read to its one write, TPR threads with
// NV vectors of 16 bytes of each operand.  Statistics and sums are fp32; s, y
// and the gradients are rounded once, when stored: y comes from the stream
// before its rounding, so it carries one rounding and not two.
//
// Measured (MI355X): forward 8192 x 4096 in bf16 46 us (5.8 TB/s with its inputs
// in the cache, 55 us and 4.9 without); backward 16384 x 768 with fp32
// parameters 38 us (4.0 TB/s) and 5 for the join, 5003 x 1001 in fp32 30 and 4,
// 8192 x 4096 in bf16 102 both (3.9 TB/s).  The norm alone, 8192 x 4096: 27 us
// forward (5.0 TB/s), 45 backward (4.4).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "xent.hpp"

namespace nsk {

struct ResNormFwdArgs {
  const void *X, *Z;            // Z null: no block output, s is x
  const void *gate, *wb, *w;    // each may be null (1)
  void *S, *Y;                  // S null without Z; Y null: no second norm
  float *rb, *rs;               // each may be null
  int64_t rows, ldx, ldz, lds, ldy;
  uint32_t gate_rows;           // consecutive rows that share a row of the gate
  int cols;
  float scale, eps;
  int norm_branch;
  int32_t* d_status;
  int32_t status_bits;
};

// Gate and weights wait in LDS: read from the cache where a row needs them,
// behind the sums that come before, their latency was a third of a row's time
// (16384 x 768 27 us forward, 19.5 without parameters).  ones where there are
// none, so that the rows' loop has no branch for them.
//
// A thread's V parameters of vector i are V / PV chunks of 16 bytes, chunk j
// of all threads side by side: with a thread's own chunks side by side (fp32
// parameters of 16-bit data) neighbours would meet in the banks.
template <typename PT, int NV, int TPR, int V>
struct alignas(16) ParamRow {
  static constexpr int PV = kVec<PT>, C = V / PV;
  u32x4_t v[NV * C * TPR];
  // Threads `first`, + `count`, ... of the block fill it.
  __device__ __forceinline__ void fill(const PT* src, int cols, int first, int count) {
    for (int q = first; q < NV * C * TPR; q += count) {
      const int t = q % TPR, j = q / TPR % C, i = q / (TPR * C);
      const int c = (i * TPR + t) * V + j * PV;
      u32x4_t x;
      PT* e = reinterpret_cast<PT*>(&x);
      if (src && c + PV <= cols) {
        x = *reinterpret_cast<const typename Vec16<sizeof(PT)>::type*>(src + c);
      } else {
#pragma unroll
        for (int k = 0; k < PV; ++k) e[k] = src ? (c + k < cols ? src[c + k] : from_f32<PT>(0.f)) : from_f32<PT>(1.f);
      }
      v[q] = x;
    }
  }
  // The parameters of thread t's vector i.
  __device__ __forceinline__ void get(int i, int t, float (&f)[V]) const {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const u32x4_t q = v[(i * C + j) * TPR + t];
#pragma unroll
      for (int k = 0; k < PV; ++k) f[j * PV + k] = to_f32<PT>(reinterpret_cast<const PT*>(&q)[k]);
    }
  }
};

// Rounds and stores a vector like store16v; adds nonfinite_bits of it to
// `found` (a float test per value costs four times that).
template <int FORM, typename IO>
__device__ __forceinline__ void put16v(IO* row, int c, int cols, const float (&f)[kVec<IO>], uint32_t& found) {
  constexpr int V = kVec<IO>;
  u32x4_t q;
  IO* e = reinterpret_cast<IO*>(&q);
#pragma unroll
  for (int k = 0; k < V; ++k) e[k] = from_f32<IO>(f[k]);
#pragma unroll
  for (int k = 0; k < 4; ++k) found |= nonfinite_bits<IO>(q[k]);
  if (c + V <= cols) {
    *reinterpret_cast<typename Vec16<sizeof(IO)>::type*>(row + c) = q;
  } else if constexpr (FORM != kEven) {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (c + k < cols) row[c + k] = e[k];
  }
}

// A row's sum as norm.hpp's row_sum, with one barrier where a row is more than
// a wave: successive sums of a block alternate between two buffers.
template <int TPR>
struct RowSums {
  static constexpr int kWaves = kNormThreads<TPR> / 64;
  float (*sh)[kWaves];  // [2]
  int turn = 0;
  __device__ __forceinline__ float operator()(float v) {
    v = wave_row_sum<TPR>(v);
    if constexpr (TPR > 64) {
      float* b = sh[turn];
      turn ^= 1;
      if ((threadIdx.x & 63) == 0) b[threadIdx.x >> 6] = v;
      __syncthreads();
      v = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) v += b[i];
    }
    return v;
  }
};

template <typename IO, typename PT, int NV, int TPR, int FORM>
__global__ void __launch_bounds__(kNormThreads<TPR>) k_resnorm_fwd(ResNormFwdArgs p) {
  constexpr int V = kVec<IO>, R = kNormRows<TPR>, T = kNormThreads<TPR>;
  __shared__ float sums[2][T / 64];
  __shared__ ParamRow<PT, NV, TPR, V> w_row, wb_row, gate_row;
  const int t = threadIdx.x % TPR;
  const float inv_n = 1.f / (float)p.cols;
  auto col = [&](int i) { return (i * TPR + t) * V; };
  const int64_t stride = (int64_t)gridDim.x * R;
  RowSums<TPR> row_total{sums};
  const bool shared_gate = !p.gate || (int64_t)p.gate_rows == p.rows;
  u32x4_t rx[NV], rz[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      rx[i] = issue16<FORM, IO>(reinterpret_cast<const IO*>(p.X) + row * p.ldx, col(i), p.cols);
      if (p.Z) rz[i] = issue16<FORM, IO>(reinterpret_cast<const IO*>(p.Z) + row * p.ldz, col(i), p.cols);
    }
  };
  int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / TPR;
  if (row < p.rows) fetch(row);
  w_row.fill(reinterpret_cast<const PT*>(p.w), p.cols, threadIdx.x, T);
  if (p.Z) {
    wb_row.fill(reinterpret_cast<const PT*>(p.wb), p.cols, threadIdx.x, T);
    if (shared_gate) gate_row.fill(reinterpret_cast<const PT*>(p.gate), p.cols, threadIdx.x, T);
  }
  __syncthreads();
  bool bad = false;
  uint32_t found = 0;
  // The trip count differs between the threads of a block only when a row is
  // at most a wave, and then no barrier is inside.
  for (; row < p.rows; row += stride) {
    const IO* x = reinterpret_cast<const IO*>(p.X) + row * p.ldx;
    float f[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) unpack<IO>(settle16<FORM, IO>(rx[i], x, col(i), p.cols), f[i]);
    if (p.Z) {
      const IO* z = reinterpret_cast<const IO*>(p.Z) + row * p.ldz;
      float b[NV][V], gv[NV][V], q = 0.f, rb = 1.f;
      if (!shared_gate) {
        const PT* gate = reinterpret_cast<const PT*>(p.gate) + (int64_t)((uint32_t)row / p.gate_rows) * p.cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          Params<FORM, PT, V> g;
          g.issue(gate, col(i), p.cols);
          g.settle(gate, col(i), p.cols);
#pragma unroll
          for (int k = 0; k < V; ++k) gv[i][k] = g.get(k);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        unpack<IO>(settle16<FORM, IO>(rz[i], z, col(i), p.cols), b[i]);
#pragma unroll
        for (int k = 0; k < V; ++k) q = fmaf(b[i][k], b[i][k], q);
      }
      if (row + stride < p.rows) fetch(row + stride);
      if (p.norm_branch) {
        const float mean = row_total(q) * inv_n;
        rb = 1.f / sqrtf(mean + p.eps);
        // Squares past fp32 make rb 0, and s finite but not the formula's: reported.
        bad |= !(mean < __builtin_inff());
        if (t == 0 && p.rb) p.rb[row] = rb;
      }
      IO* s = reinterpret_cast<IO*>(p.S) + row * p.lds;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = col(i);
        float wv[V];
        wb_row.get(i, t, wv);
        if (shared_gate) gate_row.get(i, t, gv[i]);
#pragma unroll
        for (int k = 0; k < V; ++k) f[i][k] = p.scale * f[i][k] + gv[i][k] * (b[i][k] * rb * wv[k]);
        if (c < p.cols) put16v<FORM, IO>(s, c, p.cols, f[i], found);
      }
    } else if (row + stride < p.rows) {
      fetch(row + stride);
    }
    if (!p.Y) continue;
    // Past the row x, z and so f are zeros.
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) q = fmaf(f[i][k], f[i][k], q);
    const float mean = row_total(q) * inv_n, rs = 1.f / sqrtf(mean + p.eps);
    bad |= !(mean < __builtin_inff());
    if (t == 0 && p.rs) p.rs[row] = rs;
    IO* y = reinterpret_cast<IO*>(p.Y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col(i);
      float wv[V];
      w_row.get(i, t, wv);
#pragma unroll
      for (int k = 0; k < V; ++k) f[i][k] = f[i][k] * rs * wv[k];
      if (c < p.cols) put16v<FORM, IO>(y, c, p.cols, f[i], found);
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad || (found & kNonfiniteMask<IO>));
}

// Rows of less than a vector or too long for registers: three passes over the
// row, the later two served by the cache (4096 x 16384 in bf16 508 us, 1.1 TB/s).
// S may be X and Y may be Z: the last pass reads an element and then writes it.
template <typename IO, typename PT>
__global__ void __launch_bounds__(1024) k_resnorm_fwd_long(ResNormFwdArgs p) {
  __shared__ float sh[16];
  const float inv_n = 1.f / (float)p.cols;
  const PT *W = reinterpret_cast<const PT*>(p.w), *WB = reinterpret_cast<const PT*>(p.wb);
  bool bad = false;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const IO* x = reinterpret_cast<const IO*>(p.X) + row * p.ldx;
    const IO* z = p.Z ? reinterpret_cast<const IO*>(p.Z) + row * p.ldz : nullptr;
    const PT* gate = p.gate ? reinterpret_cast<const PT*>(p.gate) + (int64_t)((uint32_t)row / p.gate_rows) * p.cols : nullptr;
    IO* s = z ? reinterpret_cast<IO*>(p.S) + row * p.lds : nullptr;
    IO* y = p.Y ? reinterpret_cast<IO*>(p.Y) + row * p.ldy : nullptr;
    float rb = 1.f, rs = 0.f, q = 0.f;
    if (z && p.norm_branch) {
      for (int c = threadIdx.x; c < p.cols; c += 1024) q = fmaf(to_f32<IO>(z[c]), to_f32<IO>(z[c]), q);
      const float mean = row_sum<1024>(q, sh) * inv_n;
      rb = 1.f / sqrtf(mean + p.eps);
      bad |= !(mean < __builtin_inff());
      if (threadIdx.x == 0 && p.rb) p.rb[row] = rb;
    }
    auto value = [&](int c) {
      float v = to_f32<IO>(x[c]);
      if (z) {
        const float wv = WB ? to_f32<PT>(WB[c]) : 1.f, gv = gate ? to_f32<PT>(gate[c]) : 1.f;
        v = p.scale * v + gv * (to_f32<IO>(z[c]) * rb * wv);
      }
      return v;
    };
    if (y) {
      q = 0.f;
      for (int c = threadIdx.x; c < p.cols; c += 1024) {
        const float v = value(c);
        q = fmaf(v, v, q);
      }
      const float mean = row_sum<1024>(q, sh) * inv_n;
      rs = 1.f / sqrtf(mean + p.eps);
      bad |= !(mean < __builtin_inff());
      if (threadIdx.x == 0 && p.rs) p.rs[row] = rs;
    }
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float v = value(c);
      if (s) {
        bad |= !(fabsf(v) < kRoundsToInf<IO>);
        s[c] = from_f32<IO>(v);
      }
      if (y) {
        const float o = v * rs * (W ? to_f32<PT>(W[c]) : 1.f);
        bad |= !(fabsf(o) < kRoundsToInf<IO>);
        y[c] = from_f32<IO>(o);
      }
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
}

// ---------------------------------------------------------------------------
// Backward.
// ---------------------------------------------------------------------------
struct ResNormBwdArgs {
  const void *dS, *dY;          // either may be null (0)
  const void *S, *Z;            // S may be null without dY; Z null: no block output
  const float *rb, *rs;         // rb null: the block's output is not normed
  const void *gate, *wb, *w;    // each may be null (1)
  void *dX, *dZ;                // dX may be null; dZ null without Z
  void* dgate_rows;             // the gate's gradient where each row has a gate of its own, or null
  int64_t rows, ldds, lddy, lds, ldz, lddx, lddz;
  uint32_t gate_rows;
  int cols;
  float scale;
  // The rows are cut into segments that share a row of the gate: `groups`
  // groups of group_rows rows, each dealt to `split` segments.  A block takes
  // segments blockIdx.x, + gridDim.x, ...; with split > 1 there is a block
  // for each.
  int64_t groups, group_rows;
  int split;
  float* partial;               // [blocks][3][partial_stride]: dw, dwb, and with split > 1 the segment's dgate
  void* dgate;                  // with split == 1: written when a segment ends
  int want_w, want_wb;          // whether dw and dwb are wanted
  int want_gate;                // whether the segments' dgate is
  int e_gated;                  // segments hold rows of several gates: want_gate is 0
  float* c_row;                 // [rows] (k_resnorm_*_long): mean_j(u shat)
  int32_t* d_status;
  int32_t status_bits;
};

// One array of column sums of a block's R rows, joined in their order (the two
// halves of a wave first): the threads of the first row hold the result.  `sh`
// holds three rows; all threads of the block call it.
template <int NV, int V, int TPR, int R>
__device__ __forceinline__ void join_rows(float (&v)[NV][V], float (*sh)[NV * V * TPR]) {
  if constexpr (TPR == 32) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const uint32_t u = __float_as_uint(v[i][k]);
        const auto q = __builtin_amdgcn_permlane32_swap(u, u, false, false);
        v[i][k] = __uint_as_float(q[0]) + __uint_as_float(q[1]);
      }
  }
  if constexpr (R > 1) {
    static_assert(TPR <= 64, "several rows share a block of four waves");
    const int wave = threadIdx.x >> 6, t = threadIdx.x % TPR;
    __syncthreads();  // readers of an earlier call are done
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) sh[wave - 1][(i * V + k) * TPR + t] = v[i][k];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int w = 0; w < 3; ++w)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) v[i][k] += sh[w][(i * V + k) * TPR + t];
    }
  }
}

// A packed vector that the compiler may not look through: unpacked again in
// each phase, it costs a few shifts; kept unpacked it would hold V registers
// from one phase to the next.
__device__ __forceinline__ void repack(u32x4_t& q) { asm volatile("" : "+v"(q)); }

// Partial rows in the workspace are whole vectors.
__host__ __device__ inline int64_t partial_stride(int64_t cols) { return (cols + 63) / 64 * 64; }

template <int V>
__device__ __forceinline__ void put_partial(float* row, int c, const float (&f)[V]) {
#pragma unroll
  for (int k = 0; k < V; k += 4) *reinterpret_cast<f32x4*>(row + c + k) = f32x4{f[k], f[k + 1], f[k + 2], f[k + 3]};
}

// A row goes through three phases over its packed registers: the mean of
// u shat; G, dx and the mean of a bhat; dz.  Two column sums live in registers
// beside them, dw and e = sum G bhat.  While the gate is the same for all rows
// of a segment, dgate is wb e and dwb gate e, added up in LDS when a segment
// ends; where rows of one segment have gates of their own, e holds dwb itself.
template <typename IO, typename PT, int NV, int TPR, int FORM>
__global__ void __launch_bounds__(kNormThreads<TPR>, 2) k_resnorm_bwd(ResNormBwdArgs p) {
  constexpr int V = kVec<IO>, R = kNormRows<TPR>, T = kNormThreads<TPR>, N = NV * TPR * V;
  __shared__ float sums[2][T / 64];
  __shared__ float join[R > 1 ? 3 : 1][R > 1 ? N : 1];
  __shared__ alignas(16) float wb_sum[N];  // dwb of the segments done
  __shared__ ParamRow<PT, NV, TPR, V> w_row, wb_row, gate_row;
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv_n = 1.f / (float)p.cols;
  auto col = [&](int i) { return (i * TPR + t) * V; };
  auto row_of = [&](const void* base, int64_t row, int64_t ld) { return reinterpret_cast<const IO*>(base) + row * ld; };
  RowSums<TPR> row_total{sums};
  w_row.fill(reinterpret_cast<const PT*>(p.w), p.cols, threadIdx.x, T);
  wb_row.fill(reinterpret_cast<const PT*>(p.wb), p.cols, threadIdx.x, T);
  for (int c = threadIdx.x; c < N; c += T) wb_sum[c] = 0.f;
  float dw[NV][V], e[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) dw[i][k] = e[i][k] = 0.f;
  uint32_t found = 0;
  bool bad = false;
  const int64_t segments = p.groups * p.split, step = (int64_t)p.split * R;
  float* partial = p.partial + (int64_t)blockIdx.x * 3 * partial_stride(p.cols);
  for (int64_t seg = blockIdx.x; seg < segments; seg += gridDim.x) {
    const int64_t group = seg / p.split, end = (group + 1) * p.group_rows;
    if (!p.e_gated) {
      // The segment's gate, for all its rows.
      const int64_t g = p.gate ? (int64_t)((uint32_t)(end - 1) / p.gate_rows) : 0;
      __syncthreads();
      gate_row.fill(p.gate ? reinterpret_cast<const PT*>(p.gate) + g * p.cols : nullptr, p.cols, threadIdx.x, T);
    }
    __syncthreads();
    for (int64_t row = group * p.group_rows + (seg - group * p.split) * R + sub; row < end; row += step) {
      u32x4_t rd[NV], ry[NV], rS[NV], rz[NV];
      Params<FORM, PT, V> rg[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (p.dY) {
          ry[i] = issue16<FORM, IO>(row_of(p.dY, row, p.lddy), col(i), p.cols);
          rS[i] = issue16<FORM, IO>(row_of(p.S, row, p.lds), col(i), p.cols);
        }
        if (p.dS) rd[i] = issue16<FORM, IO>(row_of(p.dS, row, p.ldds), col(i), p.cols);
        if (p.Z) rz[i] = issue16<FORM, IO>(row_of(p.Z, row, p.ldz), col(i), p.cols);
      }
      const PT* gate = p.e_gated ? reinterpret_cast<const PT*>(p.gate) + (int64_t)((uint32_t)row / p.gate_rows) * p.cols : nullptr;
      if (p.e_gated) {
#pragma unroll
        for (int i = 0; i < NV; ++i) rg[i].issue(gate, col(i), p.cols);
      }
      const float rs = p.dY ? p.rs[row] : 0.f, rb = p.rb ? p.rb[row] : 1.f;
      float m = 0.f;
      if (p.dY) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float u[V], s[V], wv[V];
          ry[i] = settle16<FORM, IO>(ry[i], row_of(p.dY, row, p.lddy), col(i), p.cols);
          rS[i] = settle16<FORM, IO>(rS[i], row_of(p.S, row, p.lds), col(i), p.cols);
          unpack<IO>(ry[i], u);
          unpack<IO>(rS[i], s);
          w_row.get(i, t, wv);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const float shat = s[k] * rs;
            dw[i][k] = fmaf(u[k], shat, dw[i][k]);
            m = fmaf(u[k] * wv[k], shat, m);
          }
          repack(ry[i]);
          repack(rS[i]);
        }
        m = row_total(m) * inv_n;
      }
      float a[NV][V], m2 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = col(i);
        float G[V];
        if (p.dS) {
          unpack<IO>(settle16<FORM, IO>(rd[i], row_of(p.dS, row, p.ldds), c, p.cols), G);
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k) G[k] = 0.f;
        }
        if (p.dY) {
          float u[V], s[V], wv[V];
          unpack<IO>(ry[i], u);
          unpack<IO>(rS[i], s);
          w_row.get(i, t, wv);
#pragma unroll
          for (int k = 0; k < V; ++k) G[k] += rs * (u[k] * wv[k] - s[k] * rs * m);
        }
        if (p.dX && c < p.cols) {
          float o[V];
#pragma unroll
          for (int k = 0; k < V; ++k) o[k] = p.scale * G[k];
          put16v<FORM, IO>(reinterpret_cast<IO*>(p.dX) + row * p.lddx, c, p.cols, o, found);
        }
        if (!p.Z) continue;
        float b[V], wv[V], gv[V];
        rz[i] = settle16<FORM, IO>(rz[i], row_of(p.Z, row, p.ldz), c, p.cols);
        unpack<IO>(rz[i], b);
        wb_row.get(i, t, wv);
        if (p.e_gated) {
          rg[i].settle(gate, c, p.cols);
#pragma unroll
          for (int k = 0; k < V; ++k) gv[k] = rg[i].get(k);
        } else {
          gate_row.get(i, t, gv);
        }
        if (p.dgate_rows && c < p.cols) {
          float o[V];
          uint32_t off = 0;
#pragma unroll
          for (int k = 0; k < V; ++k) o[k] = G[k] * (b[k] * rb) * wv[k];
          PT* out = reinterpret_cast<PT*>(p.dgate_rows) + row * p.cols;
          if constexpr (sizeof(PT) == sizeof(IO)) {
            put16v<FORM, PT>(out, c, p.cols, o, off);
          } else {
            // fp32 gates beside 16-bit data: two vectors.
            float half[2][4];
#pragma unroll
            for (int k = 0; k < V; ++k) half[k / 4][k % 4] = o[k];
            put16v<kRagged, PT>(out, c, p.cols, half[0], off);
            if (c + 4 < p.cols) put16v<kRagged, PT>(out, c + 4, p.cols, half[1], off);
          }
          bad |= (off & kNonfiniteMask<PT>) != 0;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
          // Past the row z is zero, and G some number that meets it only.
          const float bhat = b[k] * rb, q = gv[k] * G[k];
          e[i][k] = fmaf(p.e_gated ? q : G[k], bhat, e[i][k]);
          a[i][k] = wv[k] * q;
          m2 = fmaf(a[i][k], bhat, m2);
        }
        repack(rz[i]);
      }
      if (!p.Z) continue;
      m2 = p.rb ? row_total(m2) * inv_n : 0.f;
      IO* dz = reinterpret_cast<IO*>(p.dZ) + row * p.lddz;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = col(i);
        float b[V];
        unpack<IO>(rz[i], b);
#pragma unroll
        for (int k = 0; k < V; ++k) a[i][k] = rb * (a[i][k] - b[k] * rb * m2);
        if (c < p.cols) put16v<FORM, IO>(dz, c, p.cols, a[i], found);
      }
    }
    // The segment's end (once, after all rows, where e holds dwb itself).
    if (!(p.want_gate || p.want_wb)) continue;
    if (p.e_gated && seg + gridDim.x < segments) continue;
    if constexpr (R > 1) join_rows<NV, V, TPR, R>(e, join);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = col(i);
      if (sub == 0 && c < p.cols) {
        float gv[V], wv[V], dg[V];
        gate_row.get(i, t, gv);
        wb_row.get(i, t, wv);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          wb_sum[c + k] += p.e_gated ? e[i][k] : gv[k] * e[i][k];
          dg[k] = wv[k] * e[i][k];
        }
        if (p.want_gate && p.split > 1) {
          put_partial(partial + 2 * partial_stride(p.cols), c, dg);
        } else if (p.want_gate) {
#pragma unroll
          for (int k = 0; k < V; ++k) {
            if (c + k >= p.cols) continue;
            reinterpret_cast<PT*>(p.dgate)[group * p.cols + c + k] = from_f32<PT>(dg[k]);
            bad |= !(fabsf(dg[k]) < kRoundsToInf<PT>);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < V; ++k) e[i][k] = 0.f;
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad || (found & kNonfiniteMask<IO>));
  if constexpr (R > 1) {
    if (p.want_w) join_rows<NV, V, TPR, R>(dw, join);
  }
  if (sub != 0) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = col(i);
    if (c >= p.cols) continue;
    if (p.want_w) put_partial(partial, c, dw[i]);
    if (p.want_wb) {
      float o[V];
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] = wb_sum[c + k];
      put_partial(partial + partial_stride(p.cols), c, o);
    }
  }
}

// Rows of less than a vector or too long for registers: first each row's
// mean_j(u shat), then the column sums from it, then dx and dz (which may be
// written over ds and dy).  4096 x 16384 in bf16 1240 us, 0.65 TB/s.
template <typename IO, typename PT>
struct ResNormElement {
  const ResNormBwdArgs& p;
  __device__ __forceinline__ static float at(const void* base, int64_t i) {
    return to_f32<IO>(reinterpret_cast<const IO*>(base)[i]);
  }
  __device__ __forceinline__ static float param(const void* base, int64_t i) {
    return base ? to_f32<PT>(reinterpret_cast<const PT*>(base)[i]) : 1.f;
  }
  __device__ __forceinline__ float shat(int64_t row, int c) const { return at(p.S, row * p.lds + c) * p.rs[row]; }
  __device__ __forceinline__ float grad(int64_t row, int c, float m) const {
    float g = p.dS ? at(p.dS, row * p.ldds + c) : 0.f;
    if (p.dY) g += p.rs[row] * (param(p.w, c) * at(p.dY, row * p.lddy + c) - shat(row, c) * m);
    return g;
  }
  __device__ __forceinline__ float gate(int64_t row, int c) const {
    return param(p.gate, (int64_t)((uint32_t)row / p.gate_rows) * p.cols + c);
  }
  __device__ __forceinline__ float bhat(int64_t row, int c) const {
    return at(p.Z, row * p.ldz + c) * (p.rb ? p.rb[row] : 1.f);
  }
};

template <typename IO, typename PT>
__global__ void __launch_bounds__(1024) k_resnorm_rows_long(ResNormBwdArgs p) {
  __shared__ float sh[16];
  const ResNormElement<IO, PT> e{p};
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    float m = 0.f;
    for (int c = threadIdx.x; c < p.cols; c += 1024)
      m = fmaf(e.param(p.w, c) * e.at(p.dY, row * p.lddy + c), e.shat(row, c), m);
    m = row_sum<1024>(m, sh) / (float)p.cols;
    if (threadIdx.x == 0) p.c_row[row] = m;
  }
}

// A sum of up to millions of terms by one thread: runs of kSumRun terms, whose
// totals are added up apart, so that its error grows with the runs and their
// number and not with the number of terms (one running sum of terms of one
// sign is off by a step of itself for each, and ends to grow at 2^24 of them).
constexpr int kSumRun = 256;
struct LongSum {
  float total = 0.f, run = 0.f;
  __device__ __forceinline__ void add(float a, float b) { run = fmaf(a, b, run); }
  __device__ __forceinline__ void fold() {
    total += run;
    run = 0.f;
  }
  __device__ __forceinline__ float value() const { return total + run; }
};

// R rows of a segment at a time, 256 / R columns a block: rows of less than a
// vector share a block, and their sums are joined in LDS in their order.
template <typename IO, typename PT, int R>
__global__ void __launch_bounds__(256) k_resnorm_cols_long(ResNormBwdArgs p) {
  constexpr int C = 256 / R;
  __shared__ float sh[R > 1 ? R : 1][C];
  const int sub = threadIdx.x / C, c = blockIdx.x * C + threadIdx.x % C;
  const bool in = c < p.cols;
  // The sum of all rows' values, in the first one's threads.
  auto joined = [&](float v) {
    if constexpr (R > 1) {
      __syncthreads();
      sh[sub][threadIdx.x % C] = v;
      __syncthreads();
      v = 0.f;
      if (sub == 0)
        for (int i = 0; i < R; ++i) v += sh[i][threadIdx.x % C];
    }
    return v;
  };
  const ResNormElement<IO, PT> e{p};
  LongSum dw, dwb;
  int terms = 0;
  bool bad = false;
  const int64_t segments = p.groups * p.split, step = (int64_t)p.split * R;
  for (int64_t seg = blockIdx.y; seg < segments; seg += gridDim.y) {
    const int64_t group = seg / p.split, end = (group + 1) * p.group_rows;
    LongSum dg;
    for (int64_t row = group * p.group_rows + (seg - group * p.split) * R + sub; in && row < end; row += step) {
      if (++terms == kSumRun) {
        terms = 0;
        dw.fold();
        dwb.fold();
        dg.fold();
      }
      if (p.dY) dw.add(e.at(p.dY, row * p.lddy + c), e.shat(row, c));
      if (!p.Z) continue;
      const float g = e.grad(row, c, p.dY ? p.c_row[row] : 0.f), b = e.bhat(row, c);
      dg.add(g, b * e.param(p.wb, c));
      dwb.add(e.gate(row, c) * g, b);
    }
    if (!p.want_gate) continue;
    const float sum = joined(dg.value());
    if (!in || sub > 0) continue;
    if (p.split > 1) {
      p.partial[((int64_t)blockIdx.y * 3 + 2) * partial_stride(p.cols) + c] = sum;
    } else {
      reinterpret_cast<PT*>(p.dgate)[group * p.cols + c] = from_f32<PT>(sum);
      bad |= !(fabsf(sum) < kRoundsToInf<PT>);
    }
  }
  const float w = joined(dw.value()), wb = joined(dwb.value());
  float* out = p.partial + (int64_t)blockIdx.y * 3 * partial_stride(p.cols);
  if (in && sub == 0 && p.want_w) out[c] = w;
  if (in && sub == 0 && p.want_wb) out[partial_stride(p.cols) + c] = wb;
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
}

template <typename IO, typename PT>
__global__ void __launch_bounds__(1024) k_resnorm_bwd_long(ResNormBwdArgs p) {
  __shared__ float sh[16];
  const ResNormElement<IO, PT> e{p};
  bool bad = false;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const float m = p.dY ? p.c_row[row] : 0.f;
    float m2 = 0.f;
    if (p.Z && p.rb) {
      for (int c = threadIdx.x; c < p.cols; c += 1024)
        m2 = fmaf(e.param(p.wb, c) * (e.gate(row, c) * e.grad(row, c, m)), e.bhat(row, c), m2);
      m2 = row_sum<1024>(m2, sh) / (float)p.cols;
    }
    for (int c = threadIdx.x; c < p.cols; c += 1024) {
      const float g = e.grad(row, c, m);
      float o = 0.f, d = 0.f;
      if (p.Z) {
        const float b = e.bhat(row, c), wv = e.param(p.wb, c);
        d = g * b * wv;
        o = (p.rb ? p.rb[row] : 1.f) * (wv * (e.gate(row, c) * g) - b * m2);
      }
      if (p.dX) {
        bad |= !(fabsf(p.scale * g) < kRoundsToInf<IO>);
        reinterpret_cast<IO*>(p.dX)[row * p.lddx + c] = from_f32<IO>(p.scale * g);
      }
      if (!p.Z) continue;
      bad |= !(fabsf(o) < kRoundsToInf<IO>);
      reinterpret_cast<IO*>(p.dZ)[row * p.lddz + c] = from_f32<IO>(o);
      if (p.dgate_rows) {
        bad |= !(fabsf(d) < kRoundsToInf<PT>);
        reinterpret_cast<PT*>(p.dgate_rows)[row * p.cols + c] = from_f32<PT>(d);
      }
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
}

// The parameters' gradients from the blocks' partial rows, a block for 32
// columns of one of them: dw and dwb, from all partial rows, then the gate's
// rows, each from the `split` rows of its own.  32 half-waves take every 32nd
// partial row, all their loads in flight at once, and join in a fixed order.
struct ResNormJoinArgs {
  const float* partial;
  int blocks, split, cols;
  int64_t first;           // the launch's first row of dw, dwb and those of dgate
  void *dw, *dwb, *dgate;  // null: not wanted
  int32_t* d_status;
  int32_t status_bits;
};
template <typename PT>
__global__ void __launch_bounds__(1024) k_resnorm_join(ResNormJoinArgs p) {
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int64_t output = p.first + blockIdx.y;
  const int which = output < 2 ? (int)output : 2;
  void* out = which == 0 ? p.dw : which == 1 ? p.dwb : p.dgate;
  if (!out) return;
  const int64_t group = which == 2 ? output - 2 : 0, first = group * p.split;
  const int count = which == 2 ? p.split : p.blocks;
  float s = 0.f;
  if (c < p.cols) {
    const int64_t stride = partial_stride(p.cols);
    const float* src = p.partial + (first * 3 + which) * stride + c;
#pragma unroll 16
    for (int i = g; i < count; i += 32) s += src[(int64_t)i * 3 * stride];
  }
  sh[g][lane] = s;
  __syncthreads();
  if (g == 0 && c < p.cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += sh[i][lane];
    reinterpret_cast<PT*>(out)[group * p.cols + c] = from_f32<PT>(s);
    if (p.d_status) report_status(p.d_status, p.status_bits, !(fabsf(s) < kRoundsToInf<PT>));
  }
}

}  // namespace nsk
