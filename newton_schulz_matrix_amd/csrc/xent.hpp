// xent.hpp - softmax cross entropy of an output projection over a large
// vocabulary, without ever holding the logits, and its gradients.
//
//   z = H W^T (H: n x d hidden states, W: v x d weights)
//   lse_i = log sum_j exp z_ij,   loss_i = lse_i - z_{i, t_i}
//   dz_ij = g_i (exp(z_ij - lse_i) - [j = t_i])   (g: the losses' gradients)
//   dH = dz W,   dW = dz^T H
//
// Forward is one product whose epilogue reduces each tile of logits to a
// maximum and a sum of exponentials per row; the tiles' pairs are joined by
// a second, small kernel, and only the target's logit is kept beside them.
// Backward goes over the vocabulary in pieces: a piece's logits are made
// again, turned into dz in the product's epilogue, and used at once for
// dW's rows of that piece and for dH, which adds up over the pieces in fp32.
// One piece of dz (in both orientations) is all that is stored.
//
// Both are bound by the matrix cores (2 n v d forward, 4 n v d and the
// logits again backward) unless n is small, where reading W bounds them.
// The products run on the caller's type with fp32 accumulation; logits,
// maxima, sums and dH's running sum are fp32.  dz is rounded to the operands'
// type, because it is an operand itself: one rounding of half a step per
// term, of the size of the result's own (see xent_scale).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "norm.hpp"

namespace nsk {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// ---------------------------------------------------------------------------
// Rows: targets and coefficients.
// ---------------------------------------------------------------------------
constexpr int kTargetNone = -1;  // ignored (or a padding row)
constexpr int kTargetBad = -2;   // outside the vocabulary

struct XentRowArgs {
  const void* targets;
  int targets64;
  int64_t ignore_index;
  int64_t n, n_pad, vocab;
  int32_t* tgt;        // n_pad
  const float* dloss;  // n, or null (forward)
  const float* lse;    // n (backward)
  float *coef, *lse_pad;  // n_pad (backward): dloss or 0, lse or 0
  float* gmax;         // backward: max |coef| over the rows, cleared beforehand
  int32_t* d_status;
  int32_t index_bit;
};

static __global__ void k_xent_clear(float* gmax) { *gmax = 0.f; }

// rows x cols zeros (dW when there is no row).
template <typename T>
__global__ void __launch_bounds__(256) k_xent_zero(T* dst, int64_t ld, int cols) {
  for (int c = threadIdx.x; c < cols; c += 256) dst[(int64_t)blockIdx.x * ld + c] = from_f32<T>(0.f);
}

static __global__ void __launch_bounds__(256) k_xent_rows(XentRowArgs p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  int t = kTargetNone;
  if (i < p.n) {
    const int64_t id = p.targets64 ? reinterpret_cast<const int64_t*>(p.targets)[i]
                                   : (int64_t) reinterpret_cast<const int32_t*>(p.targets)[i];
    t = id == p.ignore_index ? kTargetNone : id >= 0 && id < p.vocab ? (int)id : kTargetBad;
  }
  if (i < p.n_pad) p.tgt[i] = t;
  if (p.coef) {
    const float g = t >= 0 ? p.dloss[i] : 0.f;
    if (i < p.n_pad) {
      p.coef[i] = g;
      p.lse_pad[i] = i < p.n ? p.lse[i] : 0.f;
    }
    // The maximum of non-negative floats is that of their bit patterns; a
    // NaN's is above all of them and stays.
    uint32_t m = __float_as_uint(fabsf(g));
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      const uint32_t o = __shfl_xor(m, off, 64);
      m = o > m ? o : m;
    }
    if ((threadIdx.x & 63) == 0 && m) atomicMax(reinterpret_cast<uint32_t*>(p.gmax), m);
  }
  if (p.d_status) report_status(p.d_status, p.index_bit, t == kTargetBad);
}

// dst (rows_pad x cols_pad) = src's rows x cols corner, zeros elsewhere: the
// staging copy of an operand whose rows are not whole k-tiles or not aligned.
template <typename T>
__global__ void __launch_bounds__(256) k_xent_pad(const T* src, int64_t ld, int64_t rows, int cols, T* dst,
                                                  int cols_pad) {
  const int64_t r = blockIdx.x;
  for (int c = threadIdx.x; c < cols_pad; c += 256)
    dst[r * cols_pad + c] = r < rows && c < cols ? src[r * ld + c] : from_f32<T>(0.f);
}

// dst (cols_pad x ldd) = the transpose of src's rows x cols, zeros elsewhere,
// through 64 x 64 tiles in LDS.
template <typename T>
__global__ void __launch_bounds__(256) k_xent_transpose(const T* src, int64_t ld, int64_t rows, int cols, T* dst,
                                                        int64_t ldd) {
  __shared__ T tile[64][64 + 4 / sizeof(T)];
  const int64_t r0 = (int64_t)blockIdx.x * 64;
  const int c0 = blockIdx.y * 64, x = threadIdx.x & 63, y = threadIdx.x >> 6;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int64_t r = r0 + y + 4 * k;
    tile[y + 4 * k][x] = r < rows && c0 + x < cols ? src[r * ld + c0 + x] : from_f32<T>(0.f);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 16; ++k) dst[(int64_t)(c0 + y + 4 * k) * ldd + r0 + x] = tile[x][y + 4 * k];
}

// ---------------------------------------------------------------------------
// The products.
// ---------------------------------------------------------------------------
struct XentArgs {
  const void *H, *W;      // n x k and v x k, rows of whole k-tiles
  int64_t ldh, ldw;       // row strides in bytes
  uint32_t row_bytes;     // bytes of a row that may be read (k elements)
  int k;                  // a multiple of the k-tile
  int64_t n, v;           // valid rows of H and of W
  int tiles_m, tiles_n;
  const int32_t* tgt;     // n_pad
  int64_t n_pad;
  // forward
  float2* parts;          // [2 tiles_n][n_pad]: maximum and sum of exponentials
  float* zt;              // [n_pad]: the target's logit
  // backward: W, tgt and v are those of one piece of the vocabulary
  int v0;                 // its first id
  const float *coef, *lse, *gmax;
  void *dz, *dzt;         // n_pad x ldz and ldz x n_pad
  int64_t ldz;
};

// One tile of logits into acc.
template <typename T, int TM, int TN, int G>
__device__ __forceinline__ void xent_logits(const XentArgs& p, int tm, int tn, Acc<T, TM, TN>& acc) {
  constexpr int BK = kRowBytes / sizeof(T);
  const int64_t row0 = (int64_t)tm * TM, col0 = (int64_t)tn * TN;
  const RowBound bl{(int)(p.n - row0 < TM ? p.n - row0 : TM), p.row_bytes};
  const RowBound br{(int)(p.v - col0 < TN ? p.v - col0 : TN), p.row_bytes};
  acc_zero(acc);
  mainloop<T, TM, TN, 0, G>(reinterpret_cast<const char*>(p.H) + row0 * p.ldh, p.ldh,
                            reinterpret_cast<const char*>(p.W) + col0 * p.ldw, p.ldw, 0, p.k / BK, acc, false, [] {},
                            [](int, const char*, const FragAddr&) {}, &bl, &br);
}

// Forward: each wave owns TN / 2 columns of its rows, half of them in each
// half wave; a row's maximum and sum over them leave as one pair.
template <typename T, int TM, int TN, int G>
__global__ void __launch_bounds__(kThreads, G) k_xent_fwd(XentArgs p) {
  using A = Acc<T, TM, TN>;
  int tm, tn;
  grouped_tile(xcd_order(blockIdx.x, p.tiles_m * p.tiles_n), p.tiles_m, p.tiles_n, tm, tn);
  A acc;
  xent_logits<T, TM, TN, G>(p, tm, tn, acc);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int lr = lane & 31, h = lane >> 5;
  const int wr = (w >> 1) * (TM / 2), wc = (w & 1) * (TN / 2);
  const int64_t row0 = (int64_t)tm * TM, col0 = (int64_t)tn * TN;
  const float inf = __builtin_inff();
  if (col0 + TN > p.v) {
#pragma unroll
    for (int fm = 0; fm < A::FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (col0 + wc + 32 * fn + 8 * (e >> 2) + 4 * h + (e & 3) >= p.v) acc.v[fm][fn][e] = -inf;
  }
#pragma unroll
  for (int fm = 0; fm < A::FM; ++fm) {
    const int64_t row = row0 + wr + fm * 32 + lr;
    const int64_t at = (int64_t)p.tgt[row] - col0 - wc - 4 * h;  // the target's column in this lane's part
    if (__any(at >= 0 && at < TN / 2)) {
#pragma unroll
      for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (at == 32 * fn + 8 * (e >> 2) + (e & 3)) p.zt[row] = acc.v[fm][fn][e];
    }
    float m = -inf;
#pragma unroll
    for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
      for (int e = 0; e < 16; ++e) m = fmaxf(m, acc.v[fm][fn][e]);
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    // A part without a finite logit (all columns past the vocabulary, or all
    // -inf) keeps m = -inf and a sum of zeros.
    const float ref = m == -inf ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
      for (int e = 0; e < 16; ++e) s += __builtin_amdgcn_exp2f((acc.v[fm][fn][e] - ref) * kLog2e);
    s += __shfl_xor(s, 32, 64);
    if (h == 0) p.parts[(int64_t)(2 * tn + (w & 1)) * p.n_pad + row] = float2{m, s};
  }
}

// Joins the parts of each row: 16 rows per block, 64 threads each.
struct XentJoinArgs {
  const float2* parts;
  int count;
  int64_t n, n_pad;
  const float* zt;
  const int32_t* tgt;
  float *loss, *lse;
  int32_t* d_status;
  int32_t status_bits;
};

static __global__ void __launch_bounds__(1024) k_xent_join(XentJoinArgs p) {
  __shared__ float2 sh[64][17];
  const int r = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int64_t row = (int64_t)blockIdx.x * 16 + r;  // below n_pad, which is a multiple of 16
  const float inf = __builtin_inff();
  float m = -inf, s = 0.f;
  auto join = [&](float2 o) {
    const float t = fmaxf(m, o.x);
    if (t == -inf) {  // both empty: zeros, or a NaN to keep
      s += o.y;
      return;
    }
    s = s * __builtin_amdgcn_exp2f((m - t) * kLog2e) + o.y * __builtin_amdgcn_exp2f((o.x - t) * kLog2e);
    m = t;
  };
#pragma unroll 4
  for (int i = g; i < p.count; i += 64) join(p.parts[(int64_t)i * p.n_pad + row]);
  sh[g][r] = float2{m, s};
  __syncthreads();
  if (g == 0 && row < p.n) {
    for (int i = 1; i < 64; ++i) join(sh[i][r]);
    const float lse = m + kLn2 * __builtin_amdgcn_logf(s);
    const int t = p.tgt[row];
    p.lse[row] = lse;
    p.loss[row] = t >= 0 ? lse - p.zt[row] : t == kTargetBad ? __builtin_nanf("") : 0.f;
    if (p.d_status && !(fabsf(lse) < inf)) atomicOr(p.d_status, p.status_bits);
  }
}

// 16-bit types hold dz in units of max|g|: bf16 as dz / max|g|, whose entries
// at the targets then lie just below 1, where the type's relative step is
// finest; fp16 as dz * 2^15 / max|g|, its largest entry just inside the type
// and probabilities down to 2^-39 of it still held.  The products' results
// are taken back in fp32.  (Coefficients so small that the quotient
// overflows give gradients below 2^-100: the limit keeps them finite on the
// way.)
template <typename T> inline constexpr float kDzUnit = __is_same(T, _Float16) ? 0x1p15f : 1.f;
template <typename T>
__device__ __forceinline__ float xent_scale(const float* gmax) {
  if constexpr (sizeof(T) == 2) {
    const float g = *gmax;
    return g > 0.f ? fminf(kDzUnit<T> / g, 1e34f) : g;  // 0 stays 0, NaN stays NaN
  }
  return 1.f;
}
template <typename T>
__device__ __forceinline__ float xent_unscale(const float* gmax) {
  if constexpr (sizeof(T) == 2) return *gmax / kDzUnit<T>;
  return 1.f;
}

// Backward, first product: dz of one tile, stored in both orientations.
template <typename T, int TM, int TN, int G>
__global__ void __launch_bounds__(kThreads, G) k_xent_dz(XentArgs p) {
  using A = Acc<T, TM, TN>;
  using TL = TileLds<T, TM, TN, G>;
  int tm, tn;
  grouped_tile(xcd_order(blockIdx.x, p.tiles_m * p.tiles_n), p.tiles_m, p.tiles_n, tm, tn);
  A acc;
  xent_logits<T, TM, TN, G>(p, tm, tn, acc);
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int lr = lane & 31, h = lane >> 5;
  const int wr = (w >> 1) * (TM / 2), wc = (w & 1) * (TN / 2);
  const int64_t row0 = (int64_t)tm * TM, col0 = (int64_t)tn * TN;
  const float unit = xent_scale<T>(p.gmax);
#pragma unroll
  for (int fm = 0; fm < A::FM; ++fm) {
    const int il = wr + fm * 32 + lr;
    const float c = p.coef[row0 + il] * unit, l = p.lse[row0 + il];
    const int64_t at = (int64_t)p.tgt[row0 + il] - p.v0 - col0;
#pragma unroll
    for (int fn = 0; fn < A::FN; ++fn) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int jl = wc + fn * 32 + 8 * g + 4 * h;
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float q = __builtin_amdgcn_exp2f((acc.v[fm][fn][4 * g + e] - l) * kLog2e);
          if (at == jl + e) q -= 1.f;
          // A row without a gradient, and the columns past the vocabulary,
          // are exact zeros whatever their logits.
          v[e] = c == 0.f || col0 + jl + e >= p.v ? 0.f : c * q;
        }
        Quad<T>::store(reinterpret_cast<T*>(TL::at(il, jl)), v);
      }
    }
  }
  __syncthreads();
  constexpr int kEC = TL::kEC, kChunks = TM * TL::kCPR;
  static_assert(kChunks % kThreads == 0, "whole chunks per thread");
  T* dz = reinterpret_cast<T*>(p.dz);
  T* dzt = reinterpret_cast<T*>(p.dzt);
#pragma unroll 6
  for (int it = 0; it < kChunks / kThreads; ++it) {
    const int q = it * kThreads + threadIdx.x;
    const int r = q / TL::kCPR, c = q % TL::kCPR;
    store16<false>(dz + (row0 + r) * p.ldz + col0 + c * kEC, *reinterpret_cast<const uint4*>(TL::chunk(r, c)));
  }
  constexpr int kRB = TM / kEC, kBlocks = kRB * TL::kCPR;
#pragma unroll 1
  for (int q = threadIdx.x; q < kBlocks; q += kThreads) {
    const int rb = q % kRB, cb = q / kRB;
    uint4 cols[kEC];
    TL::block_t(rb, cb, cols);
#pragma unroll
    for (int e = 0; e < kEC; ++e)
      store16<false>(dzt + (col0 + cb * kEC + e) * p.n_pad + row0 + rb * kEC, cols[e]);
  }
}

// dW rows of one piece: dzt (pieces rows x n_pad) times H^T (d_pad x n_pad).
struct XentDwArgs {
  const void *L, *R;
  int64_t ldl, ldr;  // bytes
  int k;
  int tiles_m, tiles_n;
  void* out;
  int64_t ldo, rows, cols;  // valid rows and columns of out
  const float* gmax;
};

template <typename T, int TM, int TN, int G>
__global__ void __launch_bounds__(kThreads, G) k_xent_dw(XentDwArgs p) {
  using A = Acc<T, TM, TN>;
  using TL = TileLds<T, TM, TN, G>;
  int tm, tn;
  grouped_tile(xcd_order(blockIdx.x, p.tiles_m * p.tiles_n), p.tiles_m, p.tiles_n, tm, tn);
  const int64_t row0 = (int64_t)tm * TM, col0 = (int64_t)tn * TN;
  constexpr int BK = kRowBytes / sizeof(T);
  A acc;
  acc_zero(acc);
  mainloop<T, TM, TN, 0, G>(reinterpret_cast<const char*>(p.L) + row0 * p.ldl, p.ldl,
                            reinterpret_cast<const char*>(p.R) + col0 * p.ldr, p.ldr, 0, p.k / BK, acc, false, [] {},
                            [](int, const char*, const FragAddr&) {});
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int lr = lane & 31, h = lane >> 5;
  const int wr = (w >> 1) * (TM / 2), wc = (w & 1) * (TN / 2);
  const float s = xent_unscale<T>(p.gmax);
#pragma unroll
  for (int fm = 0; fm < A::FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = s * acc.v[fm][fn][4 * g + e];
        Quad<T>::store(reinterpret_cast<T*>(TL::at(wr + fm * 32 + lr, wc + fn * 32 + 8 * g + 4 * h)), v);
      }
  __syncthreads();
  constexpr int kEC = TL::kEC, kChunks = TM * TL::kCPR;
  T* out = reinterpret_cast<T*>(p.out);
  const bool vec = p.ldo % kEC == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll 6
  for (int it = 0; it < kChunks / kThreads; ++it) {
    const int q = it * kThreads + threadIdx.x;
    const int r = q / TL::kCPR, c = q % TL::kCPR;
    const int64_t i = row0 + r, j = col0 + c * kEC;
    if (i >= p.rows || j >= p.cols) continue;
    const uint4 val = *reinterpret_cast<const uint4*>(TL::chunk(r, c));
    T* dst = out + i * p.ldo + j;
    if (vec && j + kEC <= p.cols) {
      store16<false>(dst, val);
    } else {
      const T* vals = reinterpret_cast<const T*>(&val);
      for (int e = 0; e < kEC && j + e < p.cols; ++e) dst[e] = vals[e];
    }
  }
}

// dH's running sums: acc[split] (+)= dz (n_pad x piece) W^T (d_pad x piece)
// over the split's share of the piece's k-tiles.
struct XentDhArgs {
  const void *L, *R;
  int64_t ldl, ldr;  // bytes
  int ktiles, splits;
  int tiles_m, tiles_n;
  float* acc;        // [splits][n_pad][d_pad]
  int64_t n_pad, d_pad;
  int first;         // the first piece writes, the others add
};

template <typename T, int TM, int TN, int G>
__global__ void __launch_bounds__(kThreads, G) k_xent_dh(XentDhArgs p) {
  using A = Acc<T, TM, TN>;
  const int per = p.tiles_m * p.tiles_n;
  const int pos = xcd_order(blockIdx.x, per * p.splits);
  const int split = pos / per;
  int tm, tn;
  grouped_tile(pos % per, p.tiles_m, p.tiles_n, tm, tn);
  const int64_t row0 = (int64_t)tm * TM, col0 = (int64_t)tn * TN;
  const int kt0 = (int)((int64_t)p.ktiles * split / p.splits), kt1 = (int)((int64_t)p.ktiles * (split + 1) / p.splits);
  A acc;
  acc_zero(acc);
  mainloop<T, TM, TN, 0, G>(reinterpret_cast<const char*>(p.L) + row0 * p.ldl, p.ldl,
                            reinterpret_cast<const char*>(p.R) + col0 * p.ldr, p.ldr, kt0, kt1, acc, false, [] {},
                            [](int, const char*, const FragAddr&) {});
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int lr = lane & 31, h = lane >> 5;
  const int wr = (w >> 1) * (TM / 2), wc = (w & 1) * (TN / 2);
  float* out = p.acc + ((int64_t)split * p.n_pad + row0) * p.d_pad + col0;
#pragma unroll
  for (int fm = 0; fm < A::FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4* dst = reinterpret_cast<f32x4*>(out + (int64_t)(wr + fm * 32 + lr) * p.d_pad + wc + fn * 32 + 8 * g + 4 * h);
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc.v[fm][fn][4 * g + e];
        if (!p.first) v += *dst;
        *dst = v;
      }
}

// dH = the splits' sum, unscaled and rounded.
template <typename T>
__global__ void __launch_bounds__(256) k_xent_dh_out(const float* acc, int splits, int64_t n_pad, int64_t d_pad,
                                                     T* out, int64_t ldo, int cols, const float* gmax,
                                                     int32_t* d_status, int32_t status_bits) {
  const int64_t r = blockIdx.x;
  const float s = xent_unscale<T>(gmax);
  bool bad = false;
  for (int c = threadIdx.x; c < cols; c += 256) {
    float v = 0.f;
    for (int k = 0; k < splits; ++k) v += acc[((int64_t)k * n_pad + r) * d_pad + c];
    v *= s;
    bad |= !(fabsf(v) < kRoundsToInf<T>);
    out[r * ldo + c] = from_f32<T>(v);
  }
  if (d_status) report_status(d_status, status_bits, bad);
}

}  // namespace nsk

// ---------------------------------------------------------------------------
// Launchers, instantiated per operand type in kern_xent_*.hip.
// ---------------------------------------------------------------------------
namespace nsr {

using namespace nsk;

// Tile edges of the products: the edge that is fastest for the iteration's
// large products too (products.hpp).
template <typename T> inline constexpr int kXentEdge = sizeof(T) == 2 ? 192 : 128;
// Forward with at most kXentFewRows rows: short, wide tiles.
constexpr int kXentFewRows = 128;
template <typename T> inline constexpr int kXentFewM = sizeof(T) == 2 ? 128 : 64;
template <typename T> inline constexpr int kXentFewN = sizeof(T) == 2 ? 256 : 128;

template <typename T> hipError_t launch_xent_fwd(const XentArgs& a, bool few, hipStream_t s);
template <typename T> hipError_t launch_xent_dz(const XentArgs& a, hipStream_t s);
template <typename T> hipError_t launch_xent_dw(const XentDwArgs& a, hipStream_t s);
template <typename T> hipError_t launch_xent_dh(const XentDhArgs& a, hipStream_t s);

#define NS_XENT_LAUNCHERS(T)                                                                                        \
  template <>                                                                                                       \
  hipError_t launch_xent_fwd<T>(const XentArgs& a, bool few, hipStream_t s) {                                       \
    const dim3 grid((unsigned)((int64_t)a.tiles_m * a.tiles_n));                                                    \
    if (few)                                                                                                        \
      hipLaunchKernelGGL((k_xent_fwd<T, kXentFewM<T>, kXentFewN<T>, 1>), grid, dim3(kThreads), 0, s, a);            \
    else                                                                                                            \
      hipLaunchKernelGGL((k_xent_fwd<T, kXentEdge<T>, kXentEdge<T>, 1>), grid, dim3(kThreads), 0, s, a);            \
    return hipGetLastError();                                                                                       \
  }                                                                                                                 \
  template <>                                                                                                       \
  hipError_t launch_xent_dz<T>(const XentArgs& a, hipStream_t s) {                                                  \
    hipLaunchKernelGGL((k_xent_dz<T, kXentEdge<T>, kXentEdge<T>, 1>),                                               \
                       dim3((unsigned)((int64_t)a.tiles_m * a.tiles_n)), dim3(kThreads), 0, s, a);                  \
    return hipGetLastError();                                                                                       \
  }                                                                                                                 \
  template <>                                                                                                       \
  hipError_t launch_xent_dw<T>(const XentDwArgs& a, hipStream_t s) {                                                \
    hipLaunchKernelGGL((k_xent_dw<T, kXentEdge<T>, kXentEdge<T>, 1>),                                               \
                       dim3((unsigned)((int64_t)a.tiles_m * a.tiles_n)), dim3(kThreads), 0, s, a);                  \
    return hipGetLastError();                                                                                       \
  }                                                                                                                 \
  template <>                                                                                                       \
  hipError_t launch_xent_dh<T>(const XentDhArgs& a, hipStream_t s) {                                                \
    hipLaunchKernelGGL((k_xent_dh<T, kXentEdge<T>, kXentEdge<T>, 1>),                                               \
                       dim3((unsigned)((int64_t)a.tiles_m * a.tiles_n * a.splits)), dim3(kThreads), 0, s, a);       \
    return hipGetLastError();                                                                                       \
  }

}  // namespace nsr
