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
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "norm.hpp"

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

// V parameters (1 where there are none) as floats.
template <int FORM, typename PT, int V>
__device__ __forceinline__ void param_values(const PT* p, int c, int cols, float (&f)[V]) {
  if (p) {
    Params<FORM, PT, V> q;
    q.issue(p, c, cols);
    q.settle(p, c, cols);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = q.get(k);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = 1.f;
  }
}

template <typename IO, typename PT, int NV, int TPR, int FORM>
__global__ void __launch_bounds__(kNormThreads<TPR>) k_resnorm_fwd(ResNormFwdArgs p) {
  constexpr int V = kVec<IO>;
  __shared__ float sh[kNormThreads<TPR> / 64];
  const int t = threadIdx.x % TPR;
  const float inv_n = 1.f / (float)p.cols;
  auto in = [&](int c, int k) { return (FORM == kEven ? c : c + k) < p.cols; };  // column c + k is in the row
  const PT *W = reinterpret_cast<const PT*>(p.w), *WB = reinterpret_cast<const PT*>(p.wb);
  const int64_t stride = (int64_t)gridDim.x * kNormRows<TPR>;
  bool bad = false;
  // The trip count differs between the threads of a block only when a row is
  // at most a wave, and then no barrier is inside.
  for (int64_t row = (int64_t)blockIdx.x * kNormRows<TPR> + threadIdx.x / TPR; row < p.rows; row += stride) {
    const IO* x = reinterpret_cast<const IO*>(p.X) + row * p.ldx;
    const IO* z = p.Z ? reinterpret_cast<const IO*>(p.Z) + row * p.ldz : nullptr;
    const PT* gate = p.gate ? reinterpret_cast<const PT*>(p.gate) + (int64_t)((uint32_t)row / p.gate_rows) * p.cols : nullptr;
    u32x4_t rx[NV], rz[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      rx[i] = issue16<FORM, IO>(x, c, p.cols);
      if (z) rz[i] = issue16<FORM, IO>(z, c, p.cols);
    }
    float f[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      unpack<IO>(settle16<FORM, IO>(rx[i], x, c, p.cols), f[i]);
    }
    if (z) {
      float b[NV][V], q = 0.f, rb = 1.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        unpack<IO>(settle16<FORM, IO>(rz[i], z, (i * TPR + t) * V, p.cols), b[i]);
#pragma unroll
        for (int k = 0; k < V; ++k) q = fmaf(b[i][k], b[i][k], q);
      }
      if (p.norm_branch) {
        const float mean = row_sum<TPR>(q, sh) * inv_n;
        rb = 1.f / sqrtf(mean + p.eps);
        // Squares past fp32 make rb 0, and s finite but not the formula's: reported.
        bad |= !(mean < __builtin_inff());
        if (t == 0 && p.rb) p.rb[row] = rb;
      }
      IO* s = reinterpret_cast<IO*>(p.S) + row * p.lds;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        float wv[V], gv[V];
        param_values<FORM, PT, V>(WB, c, p.cols, wv);
        param_values<FORM, PT, V>(gate, c, p.cols, gv);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          f[i][k] = p.scale * f[i][k] + gv[k] * (b[i][k] * rb * wv[k]);
          bad |= in(c, k) && !(fabsf(f[i][k]) < kRoundsToInf<IO>);
        }
        if (c < p.cols) store16v<FORM, IO>(s, c, p.cols, f[i]);
      }
    }
    if (!p.Y) continue;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) q = in((i * TPR + t) * V, k) ? fmaf(f[i][k], f[i][k], q) : q;
    const float mean = row_sum<TPR>(q, sh) * inv_n, rs = 1.f / sqrtf(mean + p.eps);
    bad |= !(mean < __builtin_inff());
    if (t == 0 && p.rs) p.rs[row] = rs;
    IO* y = reinterpret_cast<IO*>(p.Y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      if (c >= p.cols) continue;
      float wv[V];
      param_values<FORM, PT, V>(W, c, p.cols, wv);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        f[i][k] = f[i][k] * rs * wv[k];
        bad |= in(c, k) && !(fabsf(f[i][k]) < kRoundsToInf<IO>);
      }
      store16v<FORM, IO>(y, c, p.cols, f[i]);
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
}

// Rows of less than a vector or too long for registers: three passes over the
// row, the later two served by the cache.  S may be X and Y may be Z: the
// last pass reads an element and then writes it.
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
  float* partial;               // [blocks][3][cols]: dw, dwb, and with split > 1 the segment's dgate
  void* dgate;                  // with split == 1: written when a segment ends
  int want_w, want_wb;          // whether dw and dwb are wanted
  int want_gate;                // whether the segments' dgate is
  float* c_row;                 // [rows] (k_resnorm_*_long): mean_j(u shat)
  int32_t* d_status;
  int32_t status_bits;
};

// One array of column sums of a block's R rows, joined in their order; the
// last row's threads hold the result.
template <int NV, int V, int TPR, int R>
__device__ __forceinline__ void join_rows(float (&v)[NV][V], float* sh) {
  if constexpr (R > 1) {
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    for (int j = 0; j < R; ++j) {
      if (sub == j) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) {
            float* q = sh + (i * V + k) * TPR + t;
            if (j > 0) v[i][k] += *q;
            *q = v[i][k];
          }
      }
      __syncthreads();
    }
  }
}

template <typename IO, typename PT, int NV, int TPR, int FORM>
__global__ void __launch_bounds__(kNormThreads<TPR>) k_resnorm_bwd(ResNormBwdArgs p) {
  constexpr int V = kVec<IO>, R = kNormRows<TPR>;
  __shared__ float sh[kNormThreads<TPR> / 64];
  __shared__ float join[R > 1 ? NV * V * TPR : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv_n = 1.f / (float)p.cols;
  auto in = [&](int c, int k) { return (FORM == kEven ? c : c + k) < p.cols; };
  const PT *W = reinterpret_cast<const PT*>(p.w), *WB = reinterpret_cast<const PT*>(p.wb);
  float dw[NV][V], dwb[NV][V], dg[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) dw[i][k] = dwb[i][k] = dg[i][k] = 0.f;
  bool bad = false;
  u32x4_t rd[NV], ry[NV], rS[NV], rz[NV];
  auto row_of = [&](const void* base, int64_t row, int64_t ld) { return reinterpret_cast<const IO*>(base) + row * ld; };
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + t) * V;
      if (p.dS) rd[i] = issue16<FORM, IO>(row_of(p.dS, row, p.ldds), c, p.cols);
      if (p.dY) {
        ry[i] = issue16<FORM, IO>(row_of(p.dY, row, p.lddy), c, p.cols);
        rS[i] = issue16<FORM, IO>(row_of(p.S, row, p.lds), c, p.cols);
      }
      if (p.Z) rz[i] = issue16<FORM, IO>(row_of(p.Z, row, p.ldz), c, p.cols);
    }
  };
  const int64_t segments = p.groups * p.split, step = (int64_t)p.split * R;
  for (int64_t seg = blockIdx.x; seg < segments; seg += gridDim.x) {
    const int64_t group = seg / p.split, end = (group + 1) * p.group_rows;
    int64_t row = group * p.group_rows + (seg - group * p.split) * R + sub;
    if (row < end) fetch(row);
    for (; row < end; row += step) {
      const PT* gate = p.gate ? reinterpret_cast<const PT*>(p.gate) + (int64_t)((uint32_t)row / p.gate_rows) * p.cols : nullptr;
      float G[NV][V], b[NV][V];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (p.dS) {
          unpack<IO>(settle16<FORM, IO>(rd[i], row_of(p.dS, row, p.ldds), c, p.cols), G[i]);
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k) G[i][k] = 0.f;
        }
        if (p.Z) unpack<IO>(settle16<FORM, IO>(rz[i], row_of(p.Z, row, p.ldz), c, p.cols), b[i]);
      }
      if (p.dY) {
        const float rs = p.rs[row];
        float u[NV][V], s[NV][V], m = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * TPR + t) * V;
          float wv[V];
          unpack<IO>(settle16<FORM, IO>(ry[i], row_of(p.dY, row, p.lddy), c, p.cols), u[i]);
          unpack<IO>(settle16<FORM, IO>(rS[i], row_of(p.S, row, p.lds), c, p.cols), s[i]);
          param_values<FORM, PT, V>(W, c, p.cols, wv);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            s[i][k] *= rs;
            dw[i][k] = fmaf(u[i][k], s[i][k], dw[i][k]);
            u[i][k] *= wv[k];
            m = fmaf(u[i][k], s[i][k], m);
          }
        }
        if (row + step < end) fetch(row + step);
        m = row_sum<TPR>(m, sh) * inv_n;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) G[i][k] += rs * (u[i][k] - s[i][k] * m);
      } else if (row + step < end) {
        fetch(row + step);
      }
      if (p.dX) {
        IO* dx = reinterpret_cast<IO*>(p.dX) + row * p.lddx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (i * TPR + t) * V;
          if (c >= p.cols) continue;
          float o[V];
#pragma unroll
          for (int k = 0; k < V; ++k) {
            o[k] = p.scale * G[i][k];
            bad |= in(c, k) && !(fabsf(o[k]) < kRoundsToInf<IO>);
          }
          store16v<FORM, IO>(dx, c, p.cols, o);
        }
      }
      if (!p.Z) continue;
      const float rb = p.rb ? p.rb[row] : 1.f;
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        float wv[V], gv[V], o[V];
        param_values<FORM, PT, V>(WB, c, p.cols, wv);
        param_values<FORM, PT, V>(gate, c, p.cols, gv);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          // Past the row z is zero, and G some number that meets it only.
          b[i][k] *= rb;
          o[k] = G[i][k] * b[i][k] * wv[k];
          dg[i][k] += o[k];
          const float q = gv[k] * G[i][k];
          dwb[i][k] = fmaf(q, b[i][k], dwb[i][k]);
          G[i][k] = wv[k] * q;
          m = fmaf(G[i][k], b[i][k], m);
        }
        if (p.dgate_rows && c < p.cols) {
#pragma unroll
          for (int k = 0; k < V; ++k) bad |= in(c, k) && !(fabsf(o[k]) < kRoundsToInf<PT>);
          PT* out = reinterpret_cast<PT*>(p.dgate_rows) + row * p.cols;
          if constexpr (sizeof(PT) == sizeof(IO)) {
            store16v<FORM, PT>(out, c, p.cols, o);
          } else {
            // fp32 gates beside 16-bit data: two vectors.
            float half[2][4];
#pragma unroll
            for (int k = 0; k < V; ++k) half[k / 4][k % 4] = o[k];
            store16v<kRagged, PT>(out, c, p.cols, half[0]);
            if (c + 4 < p.cols) store16v<kRagged, PT>(out, c + 4, p.cols, half[1]);
          }
        }
      }
      m = p.rb ? row_sum<TPR>(m, sh) * inv_n : 0.f;
      IO* dz = reinterpret_cast<IO*>(p.dZ) + row * p.lddz;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + t) * V;
        if (c >= p.cols) continue;
#pragma unroll
        for (int k = 0; k < V; ++k) {
          G[i][k] = rb * (G[i][k] - b[i][k] * m);
          bad |= in(c, k) && !(fabsf(G[i][k]) < kRoundsToInf<IO>);
        }
        store16v<FORM, IO>(dz, c, p.cols, G[i]);
      }
    }
    if (p.want_gate) {
      // The segment's share of its gate row, or all of it.
      join_rows<NV, V, TPR, R>(dg, join);
      if (sub == R - 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const int c = (i * TPR + t) * V + k;
            if (c >= p.cols) continue;
            if (p.split > 1) {
              p.partial[((int64_t)blockIdx.x * 3 + 2) * p.cols + c] = dg[i][k];
            } else {
              reinterpret_cast<PT*>(p.dgate)[group * p.cols + c] = from_f32<PT>(dg[i][k]);
              bad |= !(fabsf(dg[i][k]) < kRoundsToInf<PT>);
            }
          }
      }
      if constexpr (R > 1) __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) dg[i][k] = 0.f;
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
  auto leave = [&](float (&v)[NV][V], int which) {
    join_rows<NV, V, TPR, R>(v, join);
    if (sub == R - 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int c = (i * TPR + t) * V + k;
          if (c < p.cols) p.partial[((int64_t)blockIdx.x * 3 + which) * p.cols + c] = v[i][k];
        }
    }
    if constexpr (R > 1) __syncthreads();
  };
  if (p.want_w) leave(dw, 0);
  if (p.want_wb) leave(dwb, 1);
}

// Rows of less than a vector or too long for registers: first each row's
// mean_j(u shat), then the column sums from it, then dx and dz (which may be
// written over ds and dy).
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

template <typename IO, typename PT>
__global__ void __launch_bounds__(256) k_resnorm_cols_long(ResNormBwdArgs p) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  const ResNormElement<IO, PT> e{p};
  float dw = 0.f, dwb = 0.f;
  bool bad = false;
  const int64_t segments = p.groups * p.split;
  for (int64_t seg = blockIdx.y; seg < segments; seg += gridDim.y) {
    const int64_t group = seg / p.split, end = (group + 1) * p.group_rows;
    float dg = 0.f;
    for (int64_t row = group * p.group_rows + (seg - group * p.split); row < end; row += p.split) {
      if (p.dY) dw = fmaf(e.at(p.dY, row * p.lddy + c), e.shat(row, c), dw);
      if (!p.Z) continue;
      const float g = e.grad(row, c, p.dY ? p.c_row[row] : 0.f), b = e.bhat(row, c);
      dg = fmaf(g, b * e.param(p.wb, c), dg);
      dwb = fmaf(e.gate(row, c) * g, b, dwb);
    }
    if (!p.want_gate) continue;
    if (p.split > 1) {
      p.partial[((int64_t)blockIdx.y * 3 + 2) * p.cols + c] = dg;
    } else {
      reinterpret_cast<PT*>(p.dgate)[group * p.cols + c] = from_f32<PT>(dg);
      bad |= !(fabsf(dg) < kRoundsToInf<PT>);
    }
  }
  float* out = p.partial + (int64_t)blockIdx.y * 3 * p.cols;
  if (p.want_w) out[c] = dw;
  if (p.want_wb) out[p.cols + c] = dwb;
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

// The parameters' gradients from the blocks' partial rows, a block for 64
// columns of one of them: dw and dwb, from all partial rows, then the gate's
// rows, each from the `split` rows of its own.
struct ResNormJoinArgs {
  const float* partial;
  int blocks, split, cols;
  void *dw, *dwb, *dgate;  // null: not wanted
  int32_t* d_status;
  int32_t status_bits;
};
template <typename PT>
__global__ void __launch_bounds__(1024) k_resnorm_join(ResNormJoinArgs p) {
  __shared__ float sh[16][64];
  const int slices = (p.cols + 63) / 64, output = blockIdx.x / slices, which = output < 2 ? output : 2;
  const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int c = (blockIdx.x % slices) * 64 + lane;
  void* out = which == 0 ? p.dw : which == 1 ? p.dwb : p.dgate;
  if (!out) return;
  const int64_t group = which == 2 ? output - 2 : 0;
  const int first = which == 2 ? (int)group * p.split : 0, count = which == 2 ? p.split : p.blocks;
  float s = 0.f;
  if (c < p.cols) {
    const float* src = p.partial + ((int64_t)first * 3 + which) * p.cols + c;
#pragma unroll 8
    for (int i = g; i < count; i += 16) s += src[(int64_t)i * 3 * p.cols];
  }
  sh[g][lane] = s;
  __syncthreads();
  if (g == 0 && c < p.cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sh[i][lane];
    reinterpret_cast<PT*>(out)[group * p.cols + c] = from_f32<PT>(s);
    if (p.d_status) report_status(p.d_status, p.status_bits, !(fabsf(s) < kRoundsToInf<PT>));
  }
}

}  // namespace nsk
