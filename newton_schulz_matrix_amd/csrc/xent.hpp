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
// One piece of dz (in both orientations) and transposed copies of that piece
// of W and of H are what is stored.
//
// Both are bound by the matrix cores (2 n v d forward, 4 n v d and the
// logits again backward) unless n is small, where reading W bounds them.
// The products run on the caller's type with fp32 accumulation; logits,
// maxima, sums and dH's running sum are fp32.  dz is rounded to the operands'
// type, because it is an operand itself: one rounding of half a step per
// term, of the size of the result's own (see xent_scale).
//
// Measured (MI355X, bf16): 8192 x 4096 x 128000 forward 6.9 ms, 1250 TFLOP/s,
// at a clock that power holds near 1.9 GHz; backward 4 pieces of 2.0 ms for
// dz and 3.4 ms for the gradients.  16384 x 768 x 50257: 1.1 ms and 4 x (0.50
// + 0.63) ms; products that short do not hide the writing of dz.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "norm.hpp"
#include "stream.hpp"

namespace nsk {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// ---------------------------------------------------------------------------
// Rows: targets and coefficients.
// ---------------------------------------------------------------------------
constexpr int kTargetNone = -1;  // ignored (or a padding row)
constexpr int kTargetBad = -2;   // outside the vocabulary

// Row i's target: an id, kTargetNone or kTargetBad.
struct XentTargets {
  const void* ids;
  int ids64;
  int64_t ignore_index, vocab;
  __device__ __forceinline__ int at(int64_t i) const {
    const int64_t id = ids64 ? reinterpret_cast<const int64_t*>(ids)[i]
                             : (int64_t) reinterpret_cast<const int32_t*>(ids)[i];
    return id == ignore_index ? kTargetNone : id >= 0 && id < vocab ? (int)id : kTargetBad;
  }
};

// What the products need beside the caller's own arrays, made by one kernel:
// the rows' targets and coefficients, and, tile by tile of 64 x 64, copies of
// H and of a piece of W: padded (an operand whose rows are not whole k-tiles
// or not aligned) and transposed.
struct XentRowArgs {
  XentTargets targets;
  int64_t n, n_pad;
  int32_t* tgt;        // n_pad
  const float* dloss;  // n, or null (forward)
  const float* lse;    // n (backward)
  float *coef, *lse_pad;  // n_pad (backward): dloss or 0, lse or 0
  float* gmax_parts;   // backward: max |coef| of each 256 rows, finite ones
  int32_t* d_status;
  int32_t index_bit;
};

struct XentCopyArgs {
  const void* src;        // rows x cols, row stride ld
  int64_t ld, rows;
  int cols;
  void* padded;           // rows x cols_k, zeros behind cols; or null
  int cols_k;
  void* transposed;       // cols_pad x ldt, zeros behind rows and cols; or null
  int masked;             // transposed: zeros for the rows without a coefficient
  int64_t ldt;
  int tiles_r, tiles_c;   // 64 x 64 tiles that cover the outputs
  __host__ __device__ int64_t blocks() const { return (int64_t)tiles_r * tiles_c; }
};

struct XentPrepArgs {
  XentRowArgs rows;
  int row_blocks;  // of 256 rows; then the tiles of H, then those of W
  XentCopyArgs h, w;
};

__device__ __forceinline__ void xent_rows_block(const XentRowArgs& p, int block) {
  const int64_t i = (int64_t)block * 256 + threadIdx.x;
  const int t = i < p.n ? p.targets.at(i) : kTargetNone;
  if (i < p.n_pad) p.tgt[i] = t;
  if (p.coef) {
    __shared__ uint32_t sh[4];
    const float g = t >= 0 ? p.dloss[i] : 0.f;
    if (i < p.n_pad) {
      p.coef[i] = g;
      p.lse_pad[i] = i < p.n ? p.lse[i] : 0.f;
    }
    // The maximum of non-negative floats is that of their bit patterns.  An
    // infinite or NaN coefficient goes into its own row's gradient, not into
    // the unit that all rows are held in.
    uint32_t m = __float_as_uint(fabsf(g));
    if (m >= 0x7f800000u) m = 0;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      const uint32_t o = __shfl_xor(m, off, 64);
      m = o > m ? o : m;
    }
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int k = 1; k < 4; ++k) m = sh[k] > m ? sh[k] : m;
      p.gmax_parts[block] = __uint_as_float(m);
    }
  }
  if (p.d_status) report_status(p.d_status, p.index_bit, t == kTargetBad);
}

// One 64 x 64 tile, read once in 16-byte vectors.  For the transpose a lane
// writes its vector's elements down a column of the transposed tile in LDS,
// whose rows are 64 elements and 16 bytes apart, and whole vectors leave.
//
// dW = dz^T H multiplies the zeros of a row without a gradient with that row
// of H, which may hold anything (padding positions): the transposed H has
// zeros there.
template <typename T>
__device__ __forceinline__ void xent_copy_tile(const XentCopyArgs& p, const XentRowArgs& rows, int tr, int tc) {
  constexpr int V = kVec<T>, C = 64 / V;  // vectors per tile row
  constexpr int kStride = 64 + V;
  __shared__ __attribute__((aligned(16))) T tile[64 * kStride];
  const int64_t r0 = (int64_t)tr * 64;
  const int c0 = tc * 64;
  typedef typename Vec16<sizeof(T)>::type vec_t;
  const T* src = reinterpret_cast<const T*>(p.src);
  u32x4_t v[64 * C / 256];
#pragma unroll
  for (int i = 0; i < 64 * C / 256; ++i) {
    const int q = i * 256 + threadIdx.x, r = q / C, c = q % C * V;
    v[i] = u32x4_t{0u, 0u, 0u, 0u};
    if (r0 + r < p.rows) {
      const T* s = src + (r0 + r) * p.ld + c0 + c;
      if (c0 + c + V <= p.cols) {
        v[i] = *reinterpret_cast<const vec_t*>(s);
      } else {
        T* e = reinterpret_cast<T*>(&v[i]);
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (c0 + c + k < p.cols) e[k] = s[k];
      }
    }
  }
  if (p.padded) {
    T* dst = reinterpret_cast<T*>(p.padded);
#pragma unroll
    for (int i = 0; i < 64 * C / 256; ++i) {
      const int q = i * 256 + threadIdx.x, r = q / C, c = q % C * V;
      if (r0 + r < p.rows && c0 + c < p.cols_k) *reinterpret_cast<u32x4_t*>(dst + (r0 + r) * p.cols_k + c0 + c) = v[i];
    }
  }
  if (p.transposed) {
    T* dst = reinterpret_cast<T*>(p.transposed);
    if (p.masked) {
#pragma unroll
      for (int i = 0; i < 64 * C / 256; ++i) {
        const int64_t row = r0 + (i * 256 + threadIdx.x) / C;
        if (row < p.rows && !(rows.targets.at(row) >= 0 && rows.dloss[row] != 0.f)) v[i] = u32x4_t{0u, 0u, 0u, 0u};
      }
    }
#pragma unroll
    for (int i = 0; i < 64 * C / 256; ++i) {
      const int q = i * 256 + threadIdx.x, r = q / C, c = q % C * V;
      const T* e = reinterpret_cast<const T*>(&v[i]);
#pragma unroll
      for (int k = 0; k < V; ++k) tile[(c + k) * kStride + r] = e[k];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 64 * C / 256; ++i) {
      const int q = i * 256 + threadIdx.x, c = q / C, r = q % C * V;
      *reinterpret_cast<uint4*>(dst + (int64_t)(c0 + c) * p.ldt + r0 + r) =
          *reinterpret_cast<const uint4*>(&tile[c * kStride + r]);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) k_xent_prep(XentPrepArgs p) {
  int64_t b = blockIdx.x;
  if (b < p.row_blocks) return xent_rows_block(p.rows, (int)b);
  b -= p.row_blocks;
  const XentCopyArgs& c = b < p.h.blocks() ? p.h : p.w;
  if (b >= p.h.blocks()) b -= p.h.blocks();
  xent_copy_tile<T>(c, p.rows, (int)(b / c.tiles_c), (int)(b % c.tiles_c));
}

// rows x cols zeros (dW when there is no row).
template <typename T>
__global__ void __launch_bounds__(256) k_xent_zero(T* dst, int64_t ld, int cols) {
  for (int c = threadIdx.x; c < cols; c += 256) dst[(int64_t)blockIdx.x * ld + c] = from_f32<T>(0.f);
}

// ---------------------------------------------------------------------------
// The products, each a persistent grid of at most one work-group per compute
// unit whose tiles run as one stream (stream.hpp).
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
  const float *coef, *lse, *gmax_parts;
  float* gmax;            // their maximum, for the kernels that follow
  int gmax_count;
  void *dz, *dzt;         // n_pad x ldz and ldz x n_pad
  int64_t ldz;
};

// The tiles of one work-group of a persistent grid: every gridDim.x-th of the
// list, offset so that work-groups of one XCD run neighbours.
struct TileRun {
  int first, count;
  __device__ __forceinline__ explicit TileRun(int total) {
    first = xcd_order(blockIdx.x, gridDim.x);
    count = first < total ? (total - first + (int)gridDim.x - 1) / (int)gridDim.x : 0;
  }
  __device__ __forceinline__ int at(int j) const { return first + j * (int)gridDim.x; }
};

// The logits' tiles, for the forward pass and for dz.
template <typename T, int TM, int TN, class Epilogue>
__device__ __forceinline__ void xent_logits(const XentArgs& p, const TileRun& run, Epilogue&& epi) {
  constexpr int BK = kRowBytes / sizeof(T);
  stream_tiles<T, TM, TN>(
      run.count, p.ldh, p.ldw, p.row_bytes,
      [&](int j) {
        int tm, tn;
        grouped_tile(run.at(j), p.tiles_m, p.tiles_n, tm, tn);
        const int64_t row0 = (int64_t)tm * TM, col0 = (int64_t)tn * TN;
        return StreamTile{reinterpret_cast<const char*>(p.H) + row0 * p.ldh,
                          reinterpret_cast<const char*>(p.W) + col0 * p.ldw,
                          (int)(p.n - row0 < TM ? p.n - row0 : TM),
                          (int)(p.v - col0 < TN ? p.v - col0 : TN),
                          0,
                          p.k / BK};
      },
      epi);
}

// Holds a value where it is until the wait before this point covers its load.
template <typename V>
__device__ __forceinline__ void pin(V& v) {
  asm volatile("" : "+v"(v));
}

// exp(z - ref).  The difference is taken first: folded into one fused
// multiply-add in base 2 (an operation less per logit) the exponent would be
// off by 2^-24 of ref, and a probability of 1 among logits of some thousands
// by parts in a thousand.
struct LogitExp {
  float ref;
  __device__ __forceinline__ float operator()(float z) const { return __builtin_amdgcn_exp2f((z - ref) * kLog2e); }
};

// Where a lane's values lie in a tile.
template <int TM, int TN>
struct LanePlace {
  int lr, h, wr, wc;
  __device__ __forceinline__ LanePlace() {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    lr = lane & 31;
    h = lane >> 5;
    wr = (w >> 1) * (TM / 2);
    wc = (w & 1) * (TN / 2);
  }
};

// -inf in the accumulators' columns from `cols` on, counted from the lane's
// first column: logits past the vocabulary.
template <typename T, int TM, int TN>
__device__ __forceinline__ void mask_columns(Acc<T, TM, TN>& acc, int cols) {
  using A = Acc<T, TM, TN>;
#pragma unroll
  for (int fm = 0; fm < A::FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        acc.v[fm][fn][e] = 32 * fn + 8 * (e >> 2) + (e & 3) >= cols ? -__builtin_inff() : acc.v[fm][fn][e];
}

// Forward: each wave owns TN / 2 columns of its rows, half of them in each
// half wave; a row's maximum and sum over them leave as one pair.
template <typename T, int TM, int TN>
struct FwdEpilogue {
  using A = Acc<T, TM, TN>;
  static constexpr int kStores = 0;  // the few there are may be skipped by a wave
  const XentArgs& p;
  const TileRun& run;
  LanePlace<TM, TN> at;
  int cur[A::FM], next[A::FM];
  __device__ __forceinline__ void load(int j) {
    int tm, tn;
    grouped_tile(run.at(j), p.tiles_m, p.tiles_n, tm, tn);
#pragma unroll
    for (int fm = 0; fm < A::FM; ++fm) {
      cur[fm] = next[fm];
      next[fm] = p.tgt[(int64_t)tm * TM + at.wr + fm * 32 + at.lr];
    }
  }
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int fm = 0; fm < A::FM; ++fm) pin(next[fm]);
  }
  __device__ __forceinline__ void store(int j, A& acc) {
    int tm, tn;
    grouped_tile(run.at(j), p.tiles_m, p.tiles_n, tm, tn);
    const int64_t row0 = (int64_t)tm * TM;
    const int col0 = tn * TN + at.wc + 4 * at.h;  // this lane's first column
    const int cols = (int)p.v - col0;             // and how many from there are in the vocabulary
    const float inf = __builtin_inff();
    if ((int64_t)(tn + 1) * TN > p.v) mask_columns(acc, cols);
#pragma unroll
    for (int fm = 0; fm < A::FM; ++fm) {
      const int64_t row = row0 + at.wr + fm * 32 + at.lr;
      const int t = cur[fm] - col0;  // the target's column in this lane's part
      if (__any(t >= 0 && t < TN / 2)) {
        float z = 0.f;
        bool mine = false;
#pragma unroll
        for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const bool hit = t == 32 * fn + 8 * (e >> 2) + (e & 3);
            z = hit ? acc.v[fm][fn][e] : z;
            mine |= hit;
          }
        if (mine) p.zt[row] = z;
      }
      float m = -inf;
#pragma unroll
      for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
        for (int e = 0; e < 16; ++e) m = fmaxf(m, acc.v[fm][fn][e]);
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      // A part without a finite logit (all columns past the vocabulary, or
      // all -inf) keeps m = -inf and a sum of zeros.
      const LogitExp exp_of{m == -inf ? 0.f : m};
      float s = 0.f;
#pragma unroll
      for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
        for (int e = 0; e < 16; ++e) s += exp_of(acc.v[fm][fn][e]);
      s += __shfl_xor(s, 32, 64);
      if (at.h == 0) p.parts[(int64_t)(2 * tn + (at.wc ? 1 : 0)) * p.n_pad + row] = float2{m, s};
    }
  }
};

template <typename T, int TM, int TN>
__global__ void __launch_bounds__(kThreads, 1) k_xent_fwd(XentArgs p) {
  const TileRun run(p.tiles_m * p.tiles_n);
  xent_logits<T, TM, TN>(p, run, FwdEpilogue<T, TM, TN>{p, run});
}

// Joins the parts of each row.
struct XentJoinArgs {
  const float2* parts;
  int count;
  int64_t n, part_stride, row_stride;  // part i of row r: parts[i part_stride + r row_stride]
  const float* zt;
  XentTargets targets;
  float *loss, *lse;
  int32_t* d_status;
  int32_t status_bits, index_bit;
};

struct PartJoin {
  float m = -__builtin_inff(), s = 0.f;
  __device__ __forceinline__ void add(float om, float os) {
    const float t = fmaxf(m, om);
    if (t == -__builtin_inff()) {  // both empty: zeros, or a NaN to keep
      s += os;
      return;
    }
    s = s * __builtin_amdgcn_exp2f((m - t) * kLog2e) + os * __builtin_amdgcn_exp2f((om - t) * kLog2e);
    m = t;
  }
  __device__ __forceinline__ void finish(const XentJoinArgs& p, int64_t row) const {
    const float lse = m + kLn2 * __builtin_amdgcn_logf(s);
    const int t = p.targets.at(row);
    const float loss = t >= 0 ? lse - p.zt[row] : 0.f;
    p.lse[row] = lse;
    p.loss[row] = t == kTargetBad ? __builtin_nanf("") : loss;
    if (p.d_status) {
      // A target's logit of -inf makes the loss infinite and leaves lse finite.
      const float inf = __builtin_inff();
      if (!(fabsf(lse) < inf && fabsf(loss) < inf)) atomicOr(p.d_status, p.status_bits);
      if (t == kTargetBad) atomicOr(p.d_status, p.index_bit);
    }
  }
};

// Many rows: 16 per block, 64 threads each.
static __global__ void __launch_bounds__(1024) k_xent_join(XentJoinArgs p) {
  __shared__ float2 sh[64][17];
  const int r = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int64_t row = (int64_t)blockIdx.x * 16 + r;
  PartJoin j;
  if (row < p.n) {
#pragma unroll 4
    for (int i = g; i < p.count; i += 64) {
      const float2 o = p.parts[(int64_t)i * p.part_stride + row * p.row_stride];
      j.add(o.x, o.y);
    }
  }
  sh[g][r] = float2{j.m, j.s};
  __syncthreads();
  if (g == 0 && row < p.n) {
    for (int i = 1; i < 64; ++i) j.add(sh[i][r].x, sh[i][r].y);
    j.finish(p, row);
  }
}

// Few rows: a block each.
static __global__ void __launch_bounds__(1024) k_xent_join_row(XentJoinArgs p) {
  __shared__ float2 sh[16];
  const int64_t row = blockIdx.x;
  PartJoin j;
#pragma unroll 4
  for (int i = threadIdx.x; i < p.count; i += 1024) {
    const float2 o = p.parts[(int64_t)i * p.part_stride + row * p.row_stride];
    j.add(o.x, o.y);
  }
  for (int off = 32; off > 0; off >>= 1) {
    const float om = __shfl_xor(j.m, off, 64), os = __shfl_xor(j.s, off, 64);
    j.add(om, os);
  }
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = float2{j.m, j.s};
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 16; ++i) j.add(sh[i].x, sh[i].y);
    j.finish(p, row);
  }
}

// ---------------------------------------------------------------------------
// Forward for a few rows (one token, or one per sequence): bound by reading W
// once, so no tiles: a wave takes R rows of W at a time, whole and in
// vectors at any alignment (no staging copies), the rows of H coming from the
// cache, and keeps each row's running maximum and sum until its last W row.
// One row against 128000 x 4096 bf16 takes 202 us, 5.2 TB/s, the rate of a
// large copy; in 128-byte columns of 256 rows, as the tiles read it, W comes
// at 4.6 TB/s.
// ---------------------------------------------------------------------------
constexpr int kDotRows = 8;  // R
struct XentDotArgs {
  const void *H, *W;
  int64_t ldh, ldw, n, v;  // elements
  int cols;
  int waves, groups;       // groups of R rows, dealt to the waves in turn
  XentTargets targets;
  float2* parts;           // [n][waves]
  float* zt;               // [n]
};

template <typename T, int N, int FORM>
__global__ void __launch_bounds__(256) k_xent_dot(XentDotArgs p) {
  constexpr int V = kVec<T>, R = kDotRows;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  if (wave >= p.waves) return;
  const T* H = reinterpret_cast<const T*>(p.H);
  const T* W = reinterpret_cast<const T*>(p.W);
  PartJoin run[N];
  int tgt[N];
#pragma unroll
  for (int i = 0; i < N; ++i) tgt[i] = i < p.n ? p.targets.at(i) : kTargetNone;
  for (int g = wave; g < p.groups; g += p.waves) {
    const int64_t v0 = (int64_t)g * R;
    const T* w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = W + (v0 + r < p.v ? v0 + r : p.v - 1) * p.ldw;
    float acc[R][N];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < N; ++i) acc[r][i] = 0.f;
    u32x4_t raw[R], next[R];
#pragma unroll
    for (int r = 0; r < R; ++r) raw[r] = issue16<FORM, T>(w[r], lane * V, p.cols);
    for (int c0 = 0; c0 < p.cols; c0 += 64 * V) {
      const int c = c0 + lane * V, cn = c0 + 64 * V < p.cols ? c + 64 * V : c;
#pragma unroll
      for (int r = 0; r < R; ++r) next[r] = issue16<FORM, T>(w[r], cn, p.cols);
      float h[N][V];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const T* row = H + (i < p.n ? i : 0) * p.ldh;
        unpack<T>(settle16<FORM, T>(issue16<FORM, T>(row, c, p.cols), row, c, p.cols), h[i]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x[V];
        unpack<T>(settle16<FORM, T>(raw[r], w[r], c, p.cols), x);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) acc[r][i] = fmaf(x[k], h[i][k], acc[r][i]);
        raw[r] = next[r];
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float m = -__builtin_inff();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        acc[r][i] = wave_row_sum<64>(acc[r][i]);
        if (v0 + r >= p.v) acc[r][i] = -__builtin_inff();
        if (lane == 0 && tgt[i] == v0 + r) p.zt[i] = acc[r][i];
        m = fmaxf(m, acc[r][i]);
      }
      const LogitExp exp_of{m == -__builtin_inff() ? 0.f : m};
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) s += exp_of(acc[r][i]);
      run[i].add(m, s);
    }
  }
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < p.n) p.parts[(int64_t)i * p.waves + wave] = float2{run[i].m, run[i].s};
  }
}

// 16-bit types hold dz in units of max|g|, so that the entries at the targets
// lie just below a power of two, where the type's relative step is finest.
// fp16: dz * 2^15 / max|g|, its largest entry just inside the type and
// probabilities down to 2^-39 of it still held; its operands end at 2^16, far
// from where the fp32 sums do.  bf16, whose operands reach as far as the sums:
// dz * 2^-24 / max|g|, so that 2^23 rows of the largest numbers still add up
// within fp32, with probabilities down to 2^-102 among its normal numbers.
// The products' results are taken back in fp32.  The scale stays between two
// powers of two, so that neither it nor its inverse is infinite or loses
// digits for the smallest and largest coefficients; results are taken back by
// what was applied.
template <typename T> inline constexpr float kDzUnit = __is_same(T, _Float16) ? 0x1p15f : 0x1p-24f;
constexpr float kDzScaleMin = 0x1p-126f, kDzScaleMax = 0x1p113f;
template <typename T>
__device__ __forceinline__ float xent_scale(const XentArgs& p) {
  if constexpr (sizeof(T) == 2) {
    uint32_t m = 0;
    for (int i = threadIdx.x & 63; i < p.gmax_count; i += 64) {
      const uint32_t o = __float_as_uint(p.gmax_parts[i]);
      m = o > m ? o : m;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      const uint32_t o = __shfl_xor(m, off, 64);
      m = o > m ? o : m;
    }
    const float g = __uint_as_float(m);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.gmax = g;
    return g > 0.f ? fminf(fmaxf(kDzUnit<T> / g, kDzScaleMin), kDzScaleMax) : 0.f;
  }
  return 1.f;
}
template <typename T>
__device__ __forceinline__ float xent_unscale(const float* gmax) {
  if constexpr (sizeof(T) == 2) {
    const float g = *gmax, scale = g > 0.f ? kDzUnit<T> / g : 1.f;
    return scale < kDzScaleMin ? 1.f / kDzScaleMin : scale > kDzScaleMax ? 1.f / kDzScaleMax : g / kDzUnit<T>;
  }
  return 1.f;
}

// Backward, first product: dz of one tile, stored in both orientations from
// the accumulators, at once: kept in registers and stored a block per step
// while the next tile's products run, the copies behind them waited for the
// stores (they complete in order) and a piece of 16384 x 768 x 12672 took 633
// us instead of 498.
template <typename T, int TM, int TN>
struct DzEpilogue {
  using A = Acc<T, TM, TN>;
  // Per 32 x 32 block, every one executed by every wave: 4 of dz^T, and 2 of
  // 16-bit dz rows or 4 of fp32 ones.
  static constexpr int kStores = A::FM * A::FN * (sizeof(T) == 2 ? 6 : 8);
  const XentArgs& p;
  const TileRun& run;
  float unit;
  LanePlace<TM, TN> at;
  int cur_t[A::FM], next_t[A::FM];
  float cur_c[A::FM], next_c[A::FM], cur_l[A::FM], next_l[A::FM];
  __device__ __forceinline__ void load(int j) {
    int tm, tn;
    grouped_tile(run.at(j), p.tiles_m, p.tiles_n, tm, tn);
#pragma unroll
    for (int fm = 0; fm < A::FM; ++fm) {
      cur_t[fm] = next_t[fm];
      cur_c[fm] = next_c[fm];
      cur_l[fm] = next_l[fm];
      const int64_t row = (int64_t)tm * TM + at.wr + fm * 32 + at.lr;
      next_t[fm] = p.tgt[row];
      next_c[fm] = p.coef[row];
      next_l[fm] = p.lse[row];
    }
  }
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int fm = 0; fm < A::FM; ++fm) {
      pin(next_t[fm]);
      pin(next_c[fm]);
      pin(next_l[fm]);
    }
  }
  __device__ __forceinline__ void store(int j, A& acc) {
    int tm, tn;
    grouped_tile(run.at(j), p.tiles_m, p.tiles_n, tm, tn);
    const int64_t row0 = (int64_t)tm * TM + at.wr;
    const int col0 = tn * TN + at.wc;
    const int cols = (int)p.v - col0 - 4 * at.h;  // columns of the piece from this lane's first
    T* dz = reinterpret_cast<T*>(p.dz);
    T* dzt = reinterpret_cast<T*>(p.dzt);
    const int q = at.lr & 3, i4 = at.lr & ~3;  // place in the quad, the quad's first row
    if ((int64_t)(tn + 1) * TN > p.v) mask_columns(acc, cols);
#pragma unroll
    for (int fm = 0; fm < A::FM; ++fm) {
      const float c = cur_c[fm] * unit;
      // A row without a gradient is exact zeros, whatever its logits: by a
      // mask, since a select became a branch around every conversion.
      const uint32_t keep = c == 0.f ? 0u : ~0u;
      const LogitExp p_of{cur_l[fm]};
      const int t = cur_t[fm] - p.v0 - col0 - 4 * at.h;
      T* row = dz + (row0 + fm * 32 + at.lr) * p.ldz + col0;
      T* col = dzt + (int64_t)(col0 + 4 * at.h + q) * p.n_pad + row0 + fm * 32 + i4;
      // Few parts hold a target; only those spend the comparisons.
      const bool hot = __any(t >= 0 && t < TN / 2);
#pragma unroll
      for (int fn = 0; fn < A::FN; ++fn) {
        f32x4 v[4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[g][e] = p_of(acc.v[fm][fn][4 * g + e]);
        if (hot) {
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[g][e] -= t == 32 * fn + 8 * g + e ? 1.f : 0.f;
        }
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[g][e] *= c;
        if constexpr (sizeof(T) == 2) {
          uint2 b[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            b[g] = pack_quad<T>(v[g]);
            b[g].x &= keep;
            b[g].y &= keep;
            *reinterpret_cast<uint2*>(col + (int64_t)(32 * fn + 8 * g) * p.n_pad) = transpose_quad(b[g]);
          }
#pragma unroll
          for (int g = 0; g < 4; g += 2)
            *reinterpret_cast<uint4*>(row + 32 * fn + 8 * (g + at.h)) = join_quads(b[g], b[g + 1]);
        } else {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[g][e] = __uint_as_float(__float_as_uint(v[g][e]) & keep);
            *reinterpret_cast<f32x4*>(row + 32 * fn + 8 * g + 4 * at.h) = v[g];
            *reinterpret_cast<f32x4*>(col + (int64_t)(32 * fn + 8 * g) * p.n_pad) = transpose_quad(v[g]);
          }
        }
      }
    }
  }
};

template <typename T, int TM, int TN>
__global__ void __launch_bounds__(kThreads, 1) k_xent_dz(XentArgs p) {
  const TileRun run(p.tiles_m * p.tiles_n);
  xent_logits<T, TM, TN>(p, run, DzEpilogue<T, TM, TN>{p, run, xent_scale<T>(p)});
}

// The gradients' products of one piece, in one launch: neither fills the
// compute units by itself (16384 x 768 against a piece of 10176: 212 tiles of
// 256 k-tiles for dW and 344 of 159 for dH, 301 and 250 us as two launches),
// so the work-groups with fewer tiles of dW take more of dH's.
//
// dW rows of the piece: dzt (piece x n_pad) times H^T (d_pad x n_pad).
struct XentDwArgs {
  const void *L, *R;
  int64_t ldl, ldr;  // bytes
  int k;
  int tiles_m, tiles_n;
  void* out;
  int64_t ldo, rows;  // valid rows of out
  int cols;           // and columns
  const float* gmax;
  int32_t* d_status;
  int32_t status_bits;
};

// Whether stored values are infinite or NaN, for a word of them at once: with
// the sign cleared, one more in the exponent carries into the sign's place
// exactly where the exponent was all ones.  A float test per value took 3 % of
// a step of 1000 x 1408 x 32003.
template <typename T> inline constexpr uint32_t kNonfiniteMask = sizeof(T) == 2 ? 0x80008000u : 0x80000000u;
template <typename T>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t word) {
  constexpr uint32_t one = __is_same(T, _Float16) ? 0x04000400u : __is_same(T, __bf16) ? 0x00800080u : 0x00800000u;
  return (word & ~kNonfiniteMask<T>) + one;
}
__device__ __forceinline__ uint32_t one_bits(float x) { return __float_as_uint(x); }
template <typename T>
__device__ __forceinline__ uint32_t one_bits(T x) {
  return __builtin_bit_cast(uint16_t, x);
}

template <typename T, int TM, int TN>
struct DwEpilogue {
  using A = Acc<T, TM, TN>;
  static constexpr int kStores = 0;  // rows and columns past the result store nothing
  const XentDwArgs& p;
  const TileRun& run;
  float scale;
  LanePlace<TM, TN> at;
  __device__ __forceinline__ void load(int) {}
  __device__ __forceinline__ void settle() {}
  __device__ __forceinline__ void store(int j, A& acc) {
    int tm, tn;
    grouped_tile(run.at(j), p.tiles_m, p.tiles_n, tm, tn);
    const int64_t row0 = (int64_t)tm * TM + at.wr;
    const int col0 = tn * TN + at.wc;
    constexpr int V = kVec<T>;
    T* out = reinterpret_cast<T*>(p.out);
    uint32_t found = 0;
#pragma unroll
    for (int fm = 0; fm < A::FM; ++fm) {
      const int64_t i = row0 + fm * 32 + at.lr;
      if (i >= p.rows) continue;
      T* row = out + i * p.ldo;
#pragma unroll
      for (int fn = 0; fn < A::FN; ++fn) {
        // 16-byte chunks of the row at any alignment; the row's last one may
        // be partial.
        auto put = [&](int c, const u32x4_t& q) {
          if (c + V <= p.cols) {
            *reinterpret_cast<typename Vec16<sizeof(T)>::type*>(row + c) = q;
#pragma unroll
            for (int k = 0; k < 4; ++k) found |= nonfinite_bits<T>(q[k]);
          } else {
            // Columns past the result may hold anything.
            const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
            for (int k = 0; k < V; ++k)
              if (c + k < p.cols) {
                row[c + k] = e[k];
                found |= nonfinite_bits<T>(one_bits(e[k]));
              }
          }
        };
        f32x4 v[4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[g][e] = scale * acc.v[fm][fn][4 * g + e];
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int g = 0; g < 4; g += 2) {
            const uint4 q = join_quads(pack_quad<T>(v[g]), pack_quad<T>(v[g + 1]));
            put(col0 + 32 * fn + 8 * (g + at.h), u32x4_t{q.x, q.y, q.z, q.w});
          }
        } else {
#pragma unroll
          for (int g = 0; g < 4; ++g) put(col0 + 32 * fn + 8 * g + 4 * at.h, __builtin_bit_cast(u32x4_t, v[g]));
        }
      }
    }
    if (p.d_status) report_status(p.d_status, p.status_bits, found & kNonfiniteMask<T>);
  }
};

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
  int extra;         // rounds that only the work-groups with fewer tiles of dW take part in
};
// dH's tiles of one work-group: `extra` rounds among the work-groups past the
// ones with a last tile of dW, then rounds among all.
struct DhRun {
  int first, step, rounds, base, count;
  __device__ __forceinline__ DhRun(int dw_tiles, int total, int extra) {
    const int w = xcd_order(blockIdx.x, gridDim.x), grid = (int)gridDim.x;
    const int busy = dw_tiles % grid;
    step = grid - busy;
    first = w - busy;
    const int shared = extra * step;
    rounds = 0;
    if (first >= 0 && first < total) {
      rounds = (total - first + step - 1) / step;
      rounds = rounds < extra ? rounds : extra;
    }
    base = shared + w;
    count = rounds + (base < total ? (total - base + grid - 1) / grid : 0);
  }
  __device__ __forceinline__ int at(int j) const {
    return j < rounds ? first + j * step : base + (j - rounds) * (int)gridDim.x;
  }
};

template <typename T, int TM, int TN>
struct DhEpilogue {
  using A = Acc<T, TM, TN>;
  static constexpr int kStores = A::FM * A::FN * 4;
  const XentDhArgs& p;
  const DhRun& run;
  int per;
  LanePlace<TM, TN> at;
  __device__ __forceinline__ void load(int) {}
  __device__ __forceinline__ void settle() {}
  __device__ __forceinline__ void store(int j, A& acc) {
    int tm, tn;
    grouped_tile(run.at(j) % per, p.tiles_m, p.tiles_n, tm, tn);
    float* out = p.acc + ((int64_t)(run.at(j) / per) * p.n_pad + (int64_t)tm * TM + at.wr + at.lr) * p.d_pad +
                 tn * TN + at.wc + 4 * at.h;
    if (!p.first) {
      // The loads of a block row go together.
#pragma unroll
      for (int fm = 0; fm < A::FM; ++fm) {
        f32x4 old[A::FN][4];
#pragma unroll
        for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            old[fn][g] = *reinterpret_cast<const f32x4*>(out + (int64_t)fm * 32 * p.d_pad + fn * 32 + 8 * g);
#pragma unroll
        for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc.v[fm][fn][4 * g + e] += old[fn][g][e];
      }
    }
#pragma unroll
    for (int fm = 0; fm < A::FM; ++fm)
#pragma unroll
      for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          f32x4* dst = reinterpret_cast<f32x4*>(out + (int64_t)fm * 32 * p.d_pad + fn * 32 + 8 * g);
          *dst = f32x4{acc.v[fm][fn][4 * g], acc.v[fm][fn][4 * g + 1], acc.v[fm][fn][4 * g + 2], acc.v[fm][fn][4 * g + 3]};
        }
  }
};

// dw.tiles_m or dh.tiles_m is 0 where that gradient is not wanted.
template <typename T, int TM, int TN>
__global__ void __launch_bounds__(kThreads, 1) k_xent_grads(XentDwArgs dw, XentDhArgs dh) {
  constexpr int BK = kRowBytes / sizeof(T);
  const int dw_tiles = dw.tiles_m * dw.tiles_n;
  {
    const TileRun run(dw_tiles);
    stream_tiles<T, TM, TN>(
        run.count, dw.ldl, dw.ldr, (uint32_t)(dw.k * sizeof(T)),
        [&](int j) {
          int tm, tn;
          grouped_tile(run.at(j), dw.tiles_m, dw.tiles_n, tm, tn);
          return StreamTile{reinterpret_cast<const char*>(dw.L) + (int64_t)tm * TM * dw.ldl,
                            reinterpret_cast<const char*>(dw.R) + (int64_t)tn * TN * dw.ldr, TM, TN, 0, dw.k / BK};
        },
        DwEpilogue<T, TM, TN>{dw, run, xent_unscale<T>(dw.gmax)});
  }
  // All reads of the stages are over before they are filled again.
  lds_barrier();
  const int per = dh.tiles_m * dh.tiles_n;
  const DhRun run(dw_tiles, per * dh.splits, dh.extra);
  stream_tiles<T, TM, TN>(
      run.count, dh.ldl, dh.ldr, (uint32_t)(dh.ktiles * BK * sizeof(T)),
      [&](int j) {
        const int i = run.at(j), split = i / per;
        int tm, tn;
        grouped_tile(i % per, dh.tiles_m, dh.tiles_n, tm, tn);
        const int kt0 = (int)((int64_t)dh.ktiles * split / dh.splits);
        const int kt1 = (int)((int64_t)dh.ktiles * (split + 1) / dh.splits);
        return StreamTile{reinterpret_cast<const char*>(dh.L) + (int64_t)tm * TM * dh.ldl,
                          reinterpret_cast<const char*>(dh.R) + (int64_t)tn * TN * dh.ldr, TM, TN, kt0, kt1 - kt0};
      },
      DhEpilogue<T, TM, TN>{dh, run, per});
}

// dH = the splits' sum, unscaled and rounded; rows without a gradient are
// zeros, whatever W holds.  A thread per 16 bytes of the row: few rows come
// with many splits, whose loads go eight at a time.
template <typename T>
__global__ void __launch_bounds__(64) k_xent_dh_out(const float* acc, int splits, int64_t n_pad, int64_t d_pad, T* out,
                                                    int64_t ldo, int cols, const float* coef, const float* gmax,
                                                    int32_t* d_status, int32_t status_bits) {
  constexpr int V = kVec<T>;
  const int64_t r = blockIdx.x;
  const int c = (blockIdx.y * 64 + threadIdx.x) * V;
  bool bad = false;
  if (c < cols) {
    f32x4 v[V / 4];
#pragma unroll
    for (int q = 0; q < V / 4; ++q) v[q] = f32x4{0.f, 0.f, 0.f, 0.f};
    const float* a = acc + r * d_pad + c;
    auto sum = [&](int k0, auto batch) {
      constexpr int B = decltype(batch)::value;
      f32x4 add[B][V / 4];
#pragma unroll
      for (int k = 0; k < B; ++k)
#pragma unroll
        for (int q = 0; q < V / 4; ++q) add[k][q] = reinterpret_cast<const f32x4*>(a + (k0 + k) * n_pad * d_pad)[q];
#pragma unroll
      for (int k = 0; k < B; ++k)
#pragma unroll
        for (int q = 0; q < V / 4; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[q][e] += add[k][q][e];
    };
    int k = 0;
    for (; k + 8 <= splits; k += 8) sum(k, std::integral_constant<int, 8>{});
    for (; k + 2 <= splits; k += 2) sum(k, std::integral_constant<int, 2>{});
    if (k < splits) sum(k, std::integral_constant<int, 1>{});
    const bool none = coef[r] == 0.f;
    const float s = xent_unscale<T>(gmax);
    T* row = out + r * ldo + c;
    u32x4_t packed;
    T* t = reinterpret_cast<T*>(&packed);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float x = none ? 0.f : v[k / 4][k % 4] * s;
      bad |= c + k < cols && !(fabsf(x) < kRoundsToInf<T>);
      t[k] = from_f32<T>(x);
    }
    if (c + V <= cols) {
      *reinterpret_cast<typename Vec16<sizeof(T)>::type*>(row) = packed;
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (c + k < cols) row[k] = t[k];
    }
  }
  if (d_status) report_status(d_status, status_bits, bad);
}

}  // namespace nsk

// ---------------------------------------------------------------------------
// Launchers, instantiated per operand type in kern_xent_*.hip.
// ---------------------------------------------------------------------------
namespace nsr {

using namespace nsk;

// Tile edges of the products: square tiles of the large or the small edge
// (choose_backward and xent_plan in train.hip choose); forward with few rows, 16-bit:
// short, wide tiles.
template <typename T> inline constexpr int kXentLarge = sizeof(T) == 2 ? 192 : 128;
template <typename T> inline constexpr int kXentSmall = sizeof(T) == 2 ? 128 : 64;
constexpr int kXentFewM = 128, kXentFewN = 256;
constexpr int kXentGroups = 256;  // one work-group per compute unit

template <typename T> hipError_t launch_xent_fwd(const XentArgs& a, int tm, hipStream_t s, int tn);
template <typename T> hipError_t launch_xent_dot(const XentDotArgs& a, hipStream_t s);
template <typename T> hipError_t launch_xent_dz(const XentArgs& a, int edge, hipStream_t s);
template <typename T> hipError_t launch_xent_grads(const XentDwArgs& a, const XentDhArgs& b, int edge, hipStream_t s);

inline dim3 xent_grid(int64_t tiles) { return dim3((unsigned)(tiles < kXentGroups ? tiles : kXentGroups)); }

// Rows of H that a build of k_xent_dot takes, for n of them.
inline int xent_dot_rows(int64_t n) { return n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : 8; }

template <typename T, int FORM>
void launch_dot(const XentDotArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.waves + 3) / 4));
  switch (xent_dot_rows(a.n)) {
    case 1: hipLaunchKernelGGL((k_xent_dot<T, 1, FORM>), grid, dim3(256), 0, s, a); break;
    case 2: hipLaunchKernelGGL((k_xent_dot<T, 2, FORM>), grid, dim3(256), 0, s, a); break;
    case 4: hipLaunchKernelGGL((k_xent_dot<T, 4, FORM>), grid, dim3(256), 0, s, a); break;
    default: hipLaunchKernelGGL((k_xent_dot<T, 8, FORM>), grid, dim3(256), 0, s, a);
  }
}

#define NS_XENT_LAUNCH(K, TM, TN, TILES, ...) \
  hipLaunchKernelGGL((K<T, TM, TN>), xent_grid(TILES), dim3(kThreads), 0, s, __VA_ARGS__)
#define NS_XENT_EDGE(K, TILES, ...)                                      \
  if (edge == kXentLarge<T>)                                             \
    NS_XENT_LAUNCH(K, kXentLarge<T>, kXentLarge<T>, TILES, __VA_ARGS__); \
  else                                                                   \
    NS_XENT_LAUNCH(K, kXentSmall<T>, kXentSmall<T>, TILES, __VA_ARGS__); \
  return hipGetLastError()

template <typename T>
hipError_t xent_fwd_of(const XentArgs& a, int edge, hipStream_t s, int tn) {
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
  if constexpr (sizeof(T) == 2) {
    if (edge != tn) {
      NS_XENT_LAUNCH(k_xent_fwd, kXentFewM, kXentFewN, tiles, a);
      return hipGetLastError();
    }
  }
  NS_XENT_EDGE(k_xent_fwd, tiles, a);
}
template <typename T>
hipError_t xent_dot_of(const XentDotArgs& a, hipStream_t s) {
  if (a.cols % kVec<T> == 0)
    launch_dot<T, kEven>(a, s);
  else if (a.cols > kVec<T>)
    launch_dot<T, kRagged>(a, s);
  else
    launch_dot<T, kTiny>(a, s);
  return hipGetLastError();
}
template <typename T>
hipError_t xent_dz_of(const XentArgs& a, int edge, hipStream_t s) {
  NS_XENT_EDGE(k_xent_dz, (int64_t)a.tiles_m * a.tiles_n, a);
}
template <typename T>
hipError_t xent_grads_of(const XentDwArgs& a, const XentDhArgs& b, int edge, hipStream_t s) {
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n + (int64_t)b.tiles_m * b.tiles_n * b.splits;
  NS_XENT_EDGE(k_xent_grads, tiles, a, b);
}

#define NS_XENT_LAUNCHERS(T)                                                                    \
  template <>                                                                                   \
  hipError_t launch_xent_fwd<T>(const XentArgs& a, int tm, hipStream_t s, int tn) {             \
    return xent_fwd_of<T>(a, tm, s, tn);                                                        \
  }                                                                                             \
  template <>                                                                                   \
  hipError_t launch_xent_dot<T>(const XentDotArgs& a, hipStream_t s) {                          \
    return xent_dot_of<T>(a, s);                                                                \
  }                                                                                             \
  template <>                                                                                   \
  hipError_t launch_xent_dz<T>(const XentArgs& a, int edge, hipStream_t s) {                    \
    return xent_dz_of<T>(a, edge, s);                                                           \
  }                                                                                             \
  template <>                                                                                   \
  hipError_t launch_xent_grads<T>(const XentDwArgs& a, const XentDhArgs& b, int edge, hipStream_t s) { \
    return xent_grads_of<T>(a, b, edge, s);                                                     \
  }

}  // namespace nsr
