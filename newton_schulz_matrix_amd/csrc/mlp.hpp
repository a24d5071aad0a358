// mlp.hpp - a gated feed-forward block, forward and backward.
//
//   a = x Wg^T,  b = x Wu^T,  h = act(a) b,  y = h Wd^T
//   dh = dy Wd,  da = dh b act'(a),  db = dh act(a)
//   dx = da Wg + db Wu,  dWg = da^T x,  dWu = db^T x,  dWd = dy^T h
//   (x, y: n x d;  a, b, h: n x f;  Wg, Wu: f x d;  Wd: d x f)
//
// Bound by the matrix cores (6 n d f forward, 12 n d f backward) unless n is
// small, where reading the weights bounds them.  The products run on the
// caller's type with fp32 accumulation, as streams of tiles (stream.hpp):
//
//   forward   one product for both projections: a tile's right-hand rows are
//             half rows of Wg and half the same rows of Wu, so each wave
//             holds a and b of the same columns and its epilogue makes h of
//             them.  Then y.
//   backward  dh, whose epilogue makes da, db and h again from the a and b
//             that forward left, and writes them as the last products read
//             them: da and db in rows for dx, all three transposed for the
//             weights' gradients.  Then those and dx in one launch.
//
// h, da and db are rounded to the operands' type, because they are operands
// themselves: half a step per term of the sums, of the size of the result's
// own rounding (bf16 results 0.0023 off instead of 0.0017).  Held as two numbers
// of that type each they would double the matrix work of y, dx and all weights'
// gradients.  a and b are left for backward in fp32 (or, at half the
// memory, rounded to the operands' type, which takes the gradients' error to
// 0.0035 in bf16).
//
// fp16 operands may lie outside the type's numbers where the results do not
// (see HeldRange): each product's epilogue also looks for the largest of what it
// leaves, and where that does not fit, the same tiles are made again in other
// units, which the next products' results are taken back by.
//
// A few rows go without tiles: a wave reads whole rows of the weights, and h
// stays in fp32.
//
// Measured (MI355X): 8192 x 4096 x 14336 in bf16 2.43 ms forward (1190
// TFLOP/s), 2.7 with a and b left, 5.3 backward (1090); 1003 x 2048 x 1407 in
// fp16 34, 38 and 86 us; 300 x 1000 x 2731 in fp32 73, 74 and 130 us; one row of
// 4096 x 14336 in bf16 65 us (5.4 TB/s), 48 rows 77.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "xent.hpp"

namespace nsk {

enum MlpAct { kSilu = 0, kGelu = 1, kGeluTanh = 2, kRelu = 3 };

// Value and slope of an activation.
template <int ACT>
struct Act {
  float value, slope;
  __device__ __forceinline__ explicit Act(float a) {
    if constexpr (ACT == kSilu) {
      const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * a));
      value = a * s;
      slope = s * fmaf(a, 1.f - s, 1.f);
    } else if constexpr (ACT == kGelu) {
      const float phi = fmaf(0.5f, erff(a * 0.70710678118654752f), 0.5f);
      value = a * phi;
      slope = fmaf(a * 0.39894228040143268f, __builtin_amdgcn_exp2f(-0.5f * kLog2e * a * a), phi);
    } else if constexpr (ACT == kGeluTanh) {
      // (1 + tanh(u)) / 2 = 1 / (1 + exp(-2 u)), u = c (a + k a^3).
      constexpr float c = 0.79788456080286536f, k = 0.044715f;
      const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-2.f * kLog2e * c * a * fmaf(k * a, a, 1.f)));
      value = a * s;
      // From |a| = 16 on s is 0 or 1 and so is the slope, but a^3 may be
      // infinite, which times that 0 would be a NaN.  A NaN stays one.
      const float t = a < -16.f ? -16.f : a > 16.f ? 16.f : a;
      slope = s * fmaf(2.f * t * (1.f - s), c * fmaf(3.f * k * t, t, 1.f), 1.f);
    } else {
      value = a < 0.f ? 0.f : a;  // a NaN stays one
      slope = a > 0.f ? 1.f : 0.f;
    }
  }
};

// Calls f(std::integral_constant<int, ACT>{}) for an activation known at run
// time (the same for a whole launch).
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case kSilu: f(std::integral_constant<int, kSilu>{}); break;
    case kGelu: f(std::integral_constant<int, kGelu>{}); break;
    case kGeluTanh: f(std::integral_constant<int, kGeluTanh>{}); break;
    default: f(std::integral_constant<int, kRelu>{});
  }
}

// ---------------------------------------------------------------------------
// The range of fp16 operands.
//
// h, da and db in fp16 are infinite past 65504 and lose digits below 2^-14, with
// x, weights and results well inside: |a|, |b| of 300 do for one, a dy of 1e-6
// for the other.  So they are held times a power of two, 2^held_exp, by which
// the products' fp32 results are taken back: h for y and da, db for dx in units
// of their row (a row's result does not depend on the others), for the weights'
// gradients, which add up over rows, in one unit each of da and db and of h.
// The unit is 1 while the largest magnitude is between 2^-10, from where on
// values of a sixteenth of it still have all their digits, and 65504; outside it
// takes that magnitude to [2^14, 2^15).
//
// The largest is known only when all tiles are made, so they are first made
// with the unit 1, which is nearly always right, and each wave leaves the
// largest magnitudes that it saw; a second launch of the same kernel then ends
// at once, or makes those tiles again that need it.  (1003 x 2048 x 1407: 2.7 us
// forward and 4.3 backward, of which the launches take 5; 8192 x 4096 x 14336
// 12 of 2440 and 25 of 5500.  Made again, all tiles: 25 and 32 us, 2.1 and 1.3 ms.)
// ---------------------------------------------------------------------------
template <typename T>
constexpr bool kRanged = __is_same(T, _Float16);

// Magnitudes of finite numbers as integers of the same order, infinities and
// NaN below all of them: they go into their own results only.
constexpr uint32_t kKeyZero = 0x01000000u;
__device__ __forceinline__ uint32_t range_key(float v) { return (__float_as_uint(v) << 1) + kKeyZero; }
constexpr uint32_t key_of(float v) { return (__builtin_bit_cast(uint32_t, v) << 1) + kKeyZero; }
constexpr uint32_t kKeyLeast = key_of(0x1p-10f), kKeyMost = key_of(65504.f);
__device__ __forceinline__ bool out_of_range(uint32_t key) { return key > kKeyZero && (key < kKeyLeast || key > kKeyMost); }
__device__ __forceinline__ int held_exp(uint32_t key) {
  if (!out_of_range(key)) return 0;
  // The magnitude is m 2^e with m in [1/2, 1).
  const int e = 15 - __builtin_amdgcn_frexp_expf(__uint_as_float((key - kKeyZero) >> 1));
  return e < 126 ? e : 126;
}
__device__ __forceinline__ float scaled(float v, int e) { return __builtin_amdgcn_ldexpf(v, e); }

// What the waves saw and the units that follow from it, in the workspace.
// Backward it is cleared before the tiles, and their waves take part in the
// maxima; forward, where a launch to clear it would cost as much as the check,
// each wave leaves its own parts (UpRange) and the second launch joins them.
constexpr int kRangeSlots = 64;  // words that the maxima of all are spread over (one took all atomics in turn)
struct HeldRange {
  uint32_t outside;        // whether any part of a row is out of range
  int32_t dz_exp, h_exp;   // held_exp of all da and db and of all h, left by the second launch
  uint32_t unused[61];
  uint32_t dz[kRangeSlots], h[kRangeSlots];
  uint32_t row[1];         // of each row of h (forward) or of da and db
};
constexpr int64_t kRangeWords = (sizeof(HeldRange) / 4) - 1;
__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }
// Ends a maximum here: left to the compiler it waits for its last term, with all
// the others kept in registers (49 of them spilled in dh's large tile).
__device__ __forceinline__ void settle_key(uint32_t& key) { asm volatile("" : "+v"(key)); }
// A row's part, whose two halves are in lanes lr and lr + 32.
__device__ __forceinline__ uint32_t row_part(uint32_t key) {
  const auto p = __builtin_amdgcn_permlane32_swap(key, key, false, false);
  return max_u32(p[0], p[1]);
}
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp_u32(uint32_t v) {
  return max_u32(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max_dpp_u32<0xB1>(v);
  v = max_dpp_u32<0x4E>(v);
  v = max_dpp_u32<0x141>(v);
  v = max_dpp_u32<0x140>(v);
  const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return row_part(max_u32(p[0], p[1]));
}
// held_exp of the largest of a wave's keys; nothing is moved between lanes
// where it is in range.
__device__ __forceinline__ int wave_held_exp(uint32_t key) {
  if (!__any(key > kKeyMost) && (__any(key >= kKeyLeast) || !__any(key > kKeyZero))) return 0;
  return __builtin_amdgcn_readfirstlane(held_exp(wave_max(key)));
}

// ---------------------------------------------------------------------------
// Copies of operands, padded or transposed, in 64 x 64 tiles (xent.hpp): all
// in one launch, or those that the projections' (dh's) tiles do not read
// beside these, where they leave compute units idle.
// ---------------------------------------------------------------------------
constexpr int kMlpCopies = 5;
struct MlpPrepArgs {
  XentCopyArgs copy[kMlpCopies];
  uint32_t* zero;  // words to clear (k_mlp_prep), in blocks behind the copies'
  int64_t zeros;
  __host__ __device__ int64_t zero_blocks() const { return (zeros + 1023) / 1024; }
  __host__ __device__ int64_t blocks() const {
    int64_t n = 0;
    for (const XentCopyArgs& c : copy) n += c.blocks();
    return n;
  }
};
template <typename T>
__device__ __forceinline__ void mlp_copy_block(const MlpPrepArgs& p, int64_t b, T* tile) {
#pragma unroll
  for (int i = 0; i < kMlpCopies; ++i) {
    const int64_t blocks = p.copy[i].blocks();
    if (b >= 0 && b < blocks)
      xent_copy_tile<T>(p.copy[i], XentRowArgs{}, (int)(b / p.copy[i].tiles_c), (int)(b % p.copy[i].tiles_c), tile);
    b -= blocks;
  }
}
template <typename T>
__global__ void __launch_bounds__(256) k_mlp_prep(MlpPrepArgs p) {
  __shared__ __attribute__((aligned(16))) T tile[kCopyTile<T>];
  if constexpr (kRanged<T>) {
    const int64_t copies = p.blocks();
    if (blockIdx.x >= copies) {
      const int64_t first = (blockIdx.x - copies) * 1024 + threadIdx.x;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (first + 256 * i < p.zeros) p.zero[first + 256 * i] = 0u;
      return;
    }
  }
  mlp_copy_block<T>(p, blockIdx.x, tile);
}

// ---------------------------------------------------------------------------
// Results stored from the accumulators.
// ---------------------------------------------------------------------------

// A lane's 16-byte chunk at column c of a caller's row, at any alignment; the
// row's last one may be partial.  Returns nonfinite_bits of what was stored.
template <typename T>
__device__ __forceinline__ uint32_t put_chunk(T* row, int c, int cols, const u32x4_t& q) {
  constexpr int V = kVec<T>;
  uint32_t found = 0;
  if (c + V <= cols) {
    *reinterpret_cast<typename Vec16<sizeof(T)>::type*>(row + c) = q;
#pragma unroll
    for (int k = 0; k < 4; ++k) found |= nonfinite_bits<T>(q[k]);
  } else {
    // Columns past the result may hold anything.
    const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (c + k < cols) {
        row[c + k] = e[k];
        found |= nonfinite_bits<T>(one_bits(e[k]));
      }
  }
  return found;
}

// A 32 x 32 block of a caller's matrix: lane (lr, h) gives row `row` (its
// lr), columns c0 + 8 g + 4 h + e in v[g][e].
template <typename T>
__device__ __forceinline__ uint32_t put_block(T* row, int c0, int cols, int h, const f32x4 (&v)[4]) {
  uint32_t found = 0;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
      const uint4 q = join_quads(pack_quad<T>(v[g]), pack_quad<T>(v[g + 1]));
      found |= put_chunk<T>(row, c0 + 8 * (g + h), cols, u32x4_t{q.x, q.y, q.z, q.w});
    }
  } else {
#pragma unroll
    for (int g = 0; g < 4; ++g) found |= put_chunk<T>(row, c0 + 8 * g + 4 * h, cols, __builtin_bit_cast(u32x4_t, v[g]));
  }
  return found;
}

// The same into a buffer of the workspace, whose rows are whole vectors.
template <typename T>
__device__ __forceinline__ void put_padded(T* row, int h, const f32x4 (&v)[4]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int g = 0; g < 4; g += 2)
      *reinterpret_cast<uint4*>(row + 8 * (g + h)) = join_quads(pack_quad<T>(v[g]), pack_quad<T>(v[g + 1]));
  } else {
#pragma unroll
    for (int g = 0; g < 4; ++g) *reinterpret_cast<f32x4*>(row + 8 * g + 4 * h) = v[g];
  }
}
// And transposed: col points at this lane's column of the quad (4 h + its
// place q) and the quad's first row.
template <typename T>
__device__ __forceinline__ void put_transposed(T* col, int64_t ld, const f32x4 (&v)[4]) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(col + (int64_t)(8 * g) * ld) = transpose_quad(pack_quad<T>(v[g]));
    else
      *reinterpret_cast<f32x4*>(col + (int64_t)(8 * g) * ld) = transpose_quad(v[g]);
  }
}

// ---------------------------------------------------------------------------
// Forward: both projections and the activation.
// ---------------------------------------------------------------------------
// What the waves of the first launch leave (fp16): whether a part of a row was
// out of range, for each wave, and the largest magnitudes of each part.
struct UpRange {
  uint32_t* outside;       // [waves]
  uint32_t* parts;         // [2 tiles_n][n]
};
struct MlpUpArgs {
  const void *X, *G, *U;   // n x k, f x k, f x k, rows of whole k-tiles
  int64_t ldx, ldw;        // row strides in bytes
  int ktiles;
  int64_t n, f;
  int tiles_m, tiles_n;    // tiles of TM rows and TN / 2 columns
  void* h;                 // tiles_m TM x ldh
  int64_t ldh;
  void *gate, *up;         // n x f, row stride lds, or null
  int64_t lds;
  int save32;              // they are fp32 and not T
  int act;
  int32_t* d_status;
  int32_t status_bits;
  HeldRange* range;        // fp16
  UpRange seen;
  MlpPrepArgs side;        // copies that go along
};

// Leaves one wave's a and b for the backward pass; returns whether any is not
// finite there.
template <typename S, int FM, int FH>
__device__ __forceinline__ bool save_projections(const f32x16 (&acc)[FM][2 * FH], S* gate, S* up, int64_t lds, int64_t rows,
                                                 int cols, int h) {
  uint32_t found = 0;
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) {
    if (fm * 32 >= rows) continue;
#pragma unroll
    for (int fn = 0; fn < FH; ++fn) {
      f32x4 a[4], b[4];
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          a[g][e] = acc[fm][fn][4 * g + e];
          b[g][e] = acc[fm][fn + FH][4 * g + e];
        }
      found |= put_block<S>(gate + fm * 32 * lds, 32 * fn, cols, h, a);
      found |= put_block<S>(up + fm * 32 * lds, 32 * fn, cols, h, b);
    }
  }
  return found & kNonfiniteMask<S>;
}

template <typename T, int TM, int TN, bool AGAIN>
struct UpEpilogue {
  using A = Acc<T, TM, TN>;
  static constexpr int FH = A::FN / 2;  // 32-column blocks of a, then as many of b
  static constexpr int kStores = A::FM * FH * (sizeof(T) == 2 ? 2 : 4);
  const MlpUpArgs& p;
  const TileRun& run;
  const uint32_t* row_keys;  // AGAIN: of the tile's rows, in LDS
  bool outside = false;      // whether the wave saw a part of a row that is out of range
  LanePlace<TM, TN> at;
  __device__ __forceinline__ UpEpilogue(const MlpUpArgs& p, const TileRun& run, const uint32_t* row_keys)
      : p(p), run(run), row_keys(row_keys) {}
  __device__ __forceinline__ void load(int) {}
  __device__ __forceinline__ void settle() {}
  __device__ __forceinline__ void store(int j, A& acc) {
    int tm, tn;
    grouped_tile(run.at(j), p.tiles_m, p.tiles_n, tm, tn);
    const int64_t row0 = (int64_t)tm * TM + at.wr + at.lr;
    const int64_t col0 = (int64_t)tn * (TN / 2) + at.wc / 2;
    const int cols = (int)(p.f - col0);  // of this wave's, those that exist
    if (cols < TN / 4) {
      // Columns past f are zeros whatever x holds: they are summed over next.
#pragma unroll
      for (int fm = 0; fm < A::FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int c = 32 * (fn % FH) + 8 * (e >> 2) + 4 * at.h + (e & 3);
            acc.v[fm][fn][e] = c < cols ? acc.v[fm][fn][e] : 0.f;
          }
    }
    if (p.gate) {
      const int64_t at0 = row0 * p.lds + col0;
      auto save = [&](auto s) {
        using S = decltype(s);
        return save_projections<S, A::FM, FH>(acc.v, reinterpret_cast<S*>(p.gate) + at0, reinterpret_cast<S*>(p.up) + at0,
                                              p.lds, p.n - row0, cols, at.h);
      };
      const bool bad = p.save32 ? save(float{}) : save(T{});
      if (p.d_status) report_status(p.d_status, p.status_bits, bad);
    }
    with_act(p.act, [&](auto act) {
#pragma unroll
      for (int fm = 0; fm < A::FM; ++fm) {
        T* row = reinterpret_cast<T*>(p.h) + (row0 + fm * 32) * p.ldh + col0;
        uint32_t key = 0;
        int unit = 0;
        if constexpr (AGAIN) unit = held_exp(row_keys[at.wr + at.lr + fm * 32]);
#pragma unroll
        for (int fn = 0; fn < FH; ++fn) {
          f32x4 v[4];
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e)
            {
              v[g][e] = Act<decltype(act)::value>(acc.v[fm][fn][4 * g + e]).value * acc.v[fm][fn + FH][4 * g + e];
              if constexpr (AGAIN)
                v[g][e] = scaled(v[g][e], unit);
              else if constexpr (kRanged<T>)
                key = max_u32(key, range_key(v[g][e]));
            }
          if constexpr (kRanged<T> && !AGAIN) settle_key(key);
          put_padded<T>(row + 32 * fn, at.h, v);
        }
        if constexpr (kRanged<T> && !AGAIN) {
          const int64_t r = row0 + fm * 32;
          key = row_part(key);
          if (r < p.n && at.h == 0) p.seen.parts[(2 * tn + (at.wc > 0)) * p.n + r] = key;
          outside |= __any(r < p.n && out_of_range(key));
        }
      }
    });
  }
};

template <typename T, int TM, int TN, class Epilogue>
__device__ __forceinline__ void up_tiles(const MlpUpArgs& p, const TileRun& run, Epilogue& epilogue) {
  // Wave w copies TN / 4 right-hand rows of a tile: even waves rows of Wg,
  // odd ones rows of Wu, for the columns of the waves w / 2 and w / 2 + 2.
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const char* W = reinterpret_cast<const char*>(w & 1 ? p.U : p.G);
  stream_tiles<T, TM, TN>(
      run.count, p.ldx, p.ldw, (uint32_t)(p.ktiles * kRowBytes),
      [&](int j) {
        int tm, tn;
        grouped_tile(run.at(j), p.tiles_m, p.tiles_n, tm, tn);
        const int64_t row0 = (int64_t)tm * TM, col0 = (int64_t)tn * (TN / 2) + (w >> 1) * (TN / 4);
        const int64_t left = p.f - col0;
        // The stream adds the wave's own offset to R and takes it off rows_r.
        const int own = w * (TN / 4);
        return StreamTile{reinterpret_cast<const char*>(p.X) + row0 * p.ldx, W + (col0 - own) * p.ldw,
                          (int)(p.n - row0 < TM ? p.n - row0 : TM), own + (int)(left < TN / 4 ? left : TN / 4), 0,
                          p.ktiles};
      },
      epilogue);
}

// The second launch (fp16): joins what the waves of the first saw, and makes
// those tiles again that have a row out of range, in its unit.
template <typename T, int TM, int TN>
__device__ __forceinline__ void up_again(const MlpUpArgs& p) {
  __shared__ uint32_t row_keys[TM];
  const int tiles = p.tiles_m * p.tiles_n;
  const TileRun run(tiles);
  uint32_t seen = 0;
  for (int i = threadIdx.x; i < (int)gridDim.x * (kThreads / 64); i += kThreads) seen |= p.seen.outside[i];
  const bool outside = __syncthreads_or(seen != 0);
  if (blockIdx.x == 0 && threadIdx.x == 0) p.range->outside = outside;
  if (!outside) return;
  for (int j = 0; j < run.count; ++j) {
    int tm, tn;
    grouped_tile(run.at(j), p.tiles_m, p.tiles_n, tm, tn);
    // Each row's parts, shared by kThreads / TM threads.
    const int r = threadIdx.x % TM;
    const int64_t row = (int64_t)tm * TM + r;
    if ((int)threadIdx.x < TM) row_keys[r] = 0;
    __syncthreads();
    uint32_t key = 0;
    if (row < p.n) {
#pragma unroll 16
      for (int i = threadIdx.x / TM; i < 2 * p.tiles_n; i += kThreads / TM) key = max_u32(key, p.seen.parts[i * p.n + row]);
      atomicMax(&row_keys[r], key);
    }
    __syncthreads();
    key = row_keys[r];
    if (tn == 0 && (int)threadIdx.x < TM && row < p.n) p.range->row[row] = key;
    if (!__syncthreads_or(out_of_range(key))) continue;
    TileRun one = run;
    one.first = run.at(j);
    one.count = 1;
    UpEpilogue<T, TM, TN, true> epilogue(p, one, row_keys);
    up_tiles<T, TM, TN>(p, one, epilogue);
    // All waves have read the keys.
    __syncthreads();
  }
}

template <typename T, int TM, int TN, bool AGAIN = false>
__global__ void __launch_bounds__(kThreads, 1) k_mlp_up(MlpUpArgs p) {
  if constexpr (AGAIN) {
    up_again<T, TM, TN>(p);
  } else {
    const int tiles = p.tiles_m * p.tiles_n;
    if ((int)blockIdx.x >= tiles) {
      // A work-group beyond the tiles (mlp_up_of).
      const int64_t blocks = p.side.blocks();
      for (int64_t b = blockIdx.x - tiles; b < blocks; b += gridDim.x - tiles) {
        mlp_copy_block<T>(p.side, b, reinterpret_cast<T*>(Stages<TM, TN>::s0()));
        __syncthreads();
      }
      return;
    }
    const TileRun run(tiles, (int)gridDim.x < tiles ? (int)gridDim.x : tiles);
    UpEpilogue<T, TM, TN, false> epilogue(p, run, nullptr);
    up_tiles<T, TM, TN>(p, run, epilogue);
    if constexpr (kRanged<T>) {
      if ((threadIdx.x & 63) == 0) p.seen.outside[blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6)] = epilogue.outside;
    }
  }
}

// ---------------------------------------------------------------------------
// One tile of a product whose epilogue moves as many bytes as its k-tiles:
// two work-groups share a compute unit, with two LDS stages each, so that one
// multiplies while the other loads and stores.  (dh as a stream of 192 x 192
// tiles, stream.hpp, whose one work-group does nothing else meanwhile, spent
// 640 of 1480 us on the epilogue at 8192 x 4096 x 14336; pairs of 128 tiles
// take 1345 us, and at 16384 x 768 x 2048 the backward pass takes 453 us
// instead of 528.  The projections' product, whose epilogue is shorter, lost
// by it: 1.60 -> 1.82 ms.)  Stages, fragments and steps are products.hpp's; the
// operands' resources end with their last valid rows as in stream.hpp.
// ---------------------------------------------------------------------------
template <int ROWS>
__device__ __forceinline__ void limit_rows(DmaLoader<ROWS>& l, const char* base, int64_t ld, int rows, uint32_t row_bytes) {
  const int left = rows - l.wave_row0;
  const uint32_t rec = left <= 0 ? 0 : (uint32_t)((left < ROWS / 4 ? left : ROWS / 4) - 1) * (uint32_t)ld + row_bytes;
  l.rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base) + l.wave_row0 * ld, (short)0, (int)rec, 0x00020000);
}

template <typename T, int TM, int TN>
__device__ __forceinline__ void pair_tile(const StreamTile& tile, int64_t ldl, int64_t ldr, Acc<T, TM, TN>& acc) {
  constexpr int FM = TM / 64, FN = TN / 64, kOffR = TM * kRowBytes;
  using S = Stages<TM, TN, 2>;
  static_assert(S::kCount == 2 && (TM + TN) * kRowBytes <= S::kBytes, "two stages of a tile");
  const int w = threadIdx.x >> 6;
  FragAddr fa;
  fa.init((w >> 1) * (TM / 2), (w & 1) * (TN / 2));
  DmaLoader<TM> la;
  DmaLoader<TN> lb;
  la.init(tile.L, ldl);
  lb.init(tile.R, ldr);
  const uint32_t row_bytes = (uint32_t)(tile.kts * kRowBytes);
  limit_rows(la, tile.L, ldl, tile.rows_l, row_bytes);
  limit_rows(lb, tile.R, ldr, tile.rows_r, row_bytes);
  const int last = tile.kts - 1;
  auto copy = [&](int kt, char* D) {
    la.issue(kt < last ? kt : last, D);
    lb.issue(kt < last ? kt : last, D + kOffR);
  };
  acc_zero(acc);
  copy(0, S::s0());
  copy(1, S::s1());
  __builtin_amdgcn_s_waitcnt(wait_vm(TM / 32 + TN / 32));
  lds_barrier();
  FragSets<FM, FN> fs;
  load_frags<FM, FN>(S::s0(), S::s0() + kOffR, fa, 0, fs.f0);
  load_frags<FM, FN>(S::s0(), S::s0() + kOffR, fa, 1, fs.f1);
  load_frags<FM, FN>(S::s0(), S::s0() + kOffR, fa, 2, fs.f2);
  load_frags<FM, FN>(S::s0(), S::s0() + kOffR, fa, 3, fs.f3);
  mma_frags<T, FM, FN>(fs.f0, acc.v);
  mma_frags<T, FM, FN>(fs.f1, acc.v);
  __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
  lds_barrier();
  // Step t: k-tile t + 2 into the stage of k-tile t, fragments of k-tile
  // t + 1.  Two steps at a time, so that each names its stages.
  auto step = [&](int t, char* D, const char* P) {
    const int kt = t + 2 < last ? t + 2 : last;
    pipe_step<T, TM, TN, 2>(nullptr, nullptr, la, lb, kt, 0, D, P, fa, fs, acc.v, [](int, const char*, const FragAddr&) {});
  };
  int t = 0;
  for (; t + 2 <= last; t += 2) {
    step(t, S::s0(), S::s1());
    step(t + 1, S::s1(), S::s0());
  }
  if (t < last) step(t, S::s0(), S::s1());
  mma_frags<T, FM, FN>(fs.f2, acc.v);
  mma_frags<T, FM, FN>(fs.f3, acc.v);
  // The last, repeated copies must land before the LDS is given away.
  __builtin_amdgcn_s_waitcnt(0);
}

// ---------------------------------------------------------------------------
// Backward: dh and what follows from it.
// ---------------------------------------------------------------------------
struct MlpDzArgs {
  const void *dY, *WT;     // n x k and f_pad x k (Wd transposed)
  int64_t ldy, ldw;        // bytes
  int ktiles;
  int64_t n, f;
  int tiles_m, tiles_n;
  const void *gate, *up;   // n x f, row stride lds
  int64_t lds;
  int save32;              // they are fp32 and not T
  void* dz;                // n_pad x 2 f_pad: da, db; row stride z_ld
  void* dzt;               // 2 f_pad x n_pad, row stride t_ld
  void* ht;                // f_pad x n_pad, row stride t_ld
  int64_t f_pad, z_ld, t_ld;
  int act;
  HeldRange* range;        // fp16
  MlpPrepArgs side;        // copies that go along
};

// Four columns of a caller's row as floats, at any alignment.
template <typename T>
__device__ __forceinline__ f32x4 load_quad(const T* s) {
  if constexpr (sizeof(T) == 2) {
    typedef uint32_t u32x2_a __attribute__((ext_vector_type(2), aligned(2)));
    typedef T h4 __attribute__((ext_vector_type(4)));
    const u32x2_a q = *reinterpret_cast<const u32x2_a*>(s);
    const h4 v = __builtin_bit_cast(h4, uint2{q[0], q[1]});
    return f32x4{to_f32<T>(v[0]), to_f32<T>(v[1]), to_f32<T>(v[2]), to_f32<T>(v[3])};
  } else {
    typedef float f32x4_a __attribute__((ext_vector_type(4), aligned(4)));
    const f32x4_a q = *reinterpret_cast<const f32x4_a*>(s);
    return f32x4{q[0], q[1], q[2], q[3]};
  }
}

template <typename T, int TM, int TN, bool AGAIN>
struct MlpDzEpilogue {
  using A = Acc<T, TM, TN>;
  // A wave with 64 rows of 16-bit results turns 32 columns of them in LDS, so
  // that its stores fill whole lines of the transposed rows (backward at
  // 8192 x 4096 x 14336 5427 to 5285 us, 16384 x 768 x 2048 480 to 453).  One
  // with 32 rows has but half a line of each column, and in fp32 a whole one,
  // without it.  (Loading a block's a and b before the stores of the one
  // before was no faster: 5443 against 5425, 457 against 455.)
  static constexpr bool kTurn = sizeof(T) == 2 && A::FM == 2;
  static constexpr int kTurnLd = 64 + 8;
  // Of 32 x 32.
  struct Saved {
    f32x4 a[4], b[4];
  };
  struct Block {
    f32x4 da[4], db[4], h[4];
  };
  const MlpDzArgs& p;
  LanePlace<TM, TN> at;
  int64_t row0, col0;
  int rows, cols;  // of this wave's part that exist
  bool whole;
  // The largest of each row's part of da and db and of h, as keys; AGAIN: the
  // units of the rows, of all da and db and of all h.
  uint32_t row_key[A::FM], h_key = 0;
  int row_exp[A::FM], dz_exp = 0, h_exp = 0;
  __device__ __forceinline__ MlpDzEpilogue(const MlpDzArgs& p, int tm, int tn) : p(p) {
    row0 = (int64_t)tm * TM + at.wr;
    col0 = (int64_t)tn * TN + at.wc;
    rows = (int)(p.n - row0 < TM / 2 ? p.n - row0 : TM / 2);
    cols = (int)(p.f - col0 < TN / 2 ? p.f - col0 : TN / 2);
    whole = rows == TM / 2 && cols == TN / 2;
#pragma unroll
    for (int fm = 0; fm < A::FM; ++fm) {
      row_key[fm] = 0;
      row_exp[fm] = 0;
      if constexpr (AGAIN)
        if (fm * 32 + at.lr < rows) row_exp[fm] = held_exp(p.range->row[row0 + fm * 32 + at.lr]);
    }
  }
  __device__ __forceinline__ bool exists(int fm, int fn, int g, int e) const {
    return fm * 32 + at.lr < rows && 32 * fn + 8 * g + 4 * at.h + e < cols;
  }
  __device__ __forceinline__ void fetch(int fm, int fn, Saved& o) const {
    const int64_t in = (row0 + fm * 32 + at.lr) * p.lds + col0 + 4 * at.h + 32 * fn;
    auto load = [&](auto s) {
      using S = decltype(s);
      const S *gate = reinterpret_cast<const S*>(p.gate) + in, *up = reinterpret_cast<const S*>(p.up) + in;
      if (whole) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          o.a[g] = load_quad<S>(gate + 8 * g);
          o.b[g] = load_quad<S>(up + 8 * g);
        }
      } else {
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool ok = exists(fm, fn, g, e);
            o.a[g][e] = ok ? to_f32<S>(gate[8 * g + e]) : 0.f;
            o.b[g][e] = ok ? to_f32<S>(up[8 * g + e]) : 0.f;
          }
      }
    };
    if (p.save32)
      load(float{});
    else
      load(T{});
  }
  template <int ACT>
  __device__ __forceinline__ void make(A& acc, int fm, int fn, Block& o) {
    Saved v;
    fetch(fm, fn, v);
    if (!whole) {
      // Outside they are operands of sums over rows or columns: zeros whatever
      // dy holds.
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc.v[fm][fn][4 * g + e] = exists(fm, fn, g, e) ? acc.v[fm][fn][4 * g + e] : 0.f;
    }
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const Act<ACT> s(v.a[g][e]);
        const float dh = acc.v[fm][fn][4 * g + e];
        o.da[g][e] = dh * v.b[g][e] * s.slope;
        o.db[g][e] = dh * s.value;
        o.h[g][e] = s.value * v.b[g][e];
        if constexpr (kRanged<T> && !AGAIN) {
          row_key[fm] = max_u32(row_key[fm], max_u32(range_key(o.da[g][e]), range_key(o.db[g][e])));
          h_key = max_u32(h_key, range_key(o.h[g][e]));
        }
      }
    if constexpr (kRanged<T> && !AGAIN) {
      settle_key(row_key[fm]);
      settle_key(h_key);
    }
    T* dz = reinterpret_cast<T*>(p.dz) + (row0 + fm * 32 + at.lr) * p.z_ld + col0 + 32 * fn;
    if constexpr (AGAIN) {
      f32x4 in_row[2][4];
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          in_row[0][g][e] = scaled(o.da[g][e], row_exp[fm]);
          in_row[1][g][e] = scaled(o.db[g][e], row_exp[fm]);
          o.da[g][e] = scaled(o.da[g][e], dz_exp);
          o.db[g][e] = scaled(o.db[g][e], dz_exp);
          o.h[g][e] = scaled(o.h[g][e], h_exp);
        }
      put_padded<T>(dz, at.h, in_row[0]);
      put_padded<T>(dz + p.f_pad, at.h, in_row[1]);
    } else {
      put_padded<T>(dz, at.h, o.da);
      put_padded<T>(dz + p.f_pad, at.h, o.db);
    }
  }
  // What the wave saw, once all its blocks are made.
  __device__ __forceinline__ void leave_keys() const {
    uint32_t key = 0;
    bool outside = false;
#pragma unroll
    for (int fm = 0; fm < A::FM; ++fm) {
      const uint32_t part = row_part(row_key[fm]);
      const bool valid = fm * 32 + at.lr < rows;
      if (valid && at.h == 0) atomicMax(&p.range->row[row0 + fm * 32 + at.lr], part);
      outside |= __any(valid && out_of_range(part));
      key = max_u32(key, part);
    }
    const uint32_t dz = wave_max(key), h = wave_max(h_key);
    if ((threadIdx.x & 63) == 0) {
      if (outside) atomicOr(&p.range->outside, 1u);
      atomicMax(&p.range->dz[blockIdx.x % kRangeSlots], dz);
      atomicMax(&p.range->h[blockIdx.x % kRangeSlots], h);
    }
  }
  // lds: the wave's own 3 x 32 rows of kTurnLd.
  __device__ __forceinline__ void store(A& acc, T* lds) {
    const int q = at.lr & 3, i4 = at.lr & ~3;  // place in the quad, the quad's first row
    T *dzt = reinterpret_cast<T*>(p.dzt), *ht = reinterpret_cast<T*>(p.ht);
    with_act(p.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      if constexpr (kTurn) {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int fn = 0; fn < A::FN; ++fn) {
#pragma unroll
          for (int fm = 0; fm < A::FM; ++fm) {
            Block o;
            make<ACT>(acc, fm, fn, o);
            T* turned = lds + (4 * at.h + q) * kTurnLd + fm * 32 + i4;
            put_transposed<T>(turned, kTurnLd, o.da);
            put_transposed<T>(turned + 32 * kTurnLd, kTurnLd, o.db);
            put_transposed<T>(turned + 64 * kTurnLd, kTurnLd, o.h);
          }
          wave_fence();
#pragma unroll
          for (int m = 0; m < 3; ++m) {
            T* out = m == 0 ? dzt : m == 1 ? dzt + p.f_pad * p.t_ld : ht;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int c = 8 * i + (lane >> 3), r = (lane & 7) * 8;
              *reinterpret_cast<uint4*>(out + (col0 + 32 * fn + c) * p.t_ld + row0 + r) =
                  *reinterpret_cast<const uint4*>(lds + (32 * m + c) * kTurnLd + r);
            }
          }
          wave_fence();
        }
      } else {
#pragma unroll
        for (int fm = 0; fm < A::FM; ++fm) {
#pragma unroll
          for (int fn = 0; fn < A::FN; ++fn) {
            Block o;
            make<ACT>(acc, fm, fn, o);
            const int64_t t = (col0 + 32 * fn + 4 * at.h + q) * p.t_ld + row0 + fm * 32 + i4;
            put_transposed<T>(dzt + t, p.t_ld, o.da);
            put_transposed<T>(dzt + t + p.f_pad * p.t_ld, p.t_ld, o.db);
            put_transposed<T>(ht + t, p.t_ld, o.h);
          }
        }
      }
    });
  }
  // What a wave wrote to LDS before is there for what it reads behind (and the
  // other way round): its LDS operations are carried out in order, so only
  // the compiler has to keep it.
  static __device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
};

template <typename T, int TM, int TN, bool AGAIN>
__device__ __forceinline__ void dz_tile(const MlpDzArgs& p, int tm, int tn, int dz_exp, int h_exp) {
  const int64_t row0 = (int64_t)tm * TM;
  const StreamTile tile{reinterpret_cast<const char*>(p.dY) + row0 * p.ldy,
                        reinterpret_cast<const char*>(p.WT) + (int64_t)tn * TN * p.ldw,
                        (int)(p.n - row0 < TM ? p.n - row0 : TM), TN, 0, p.ktiles};
  Acc<T, TM, TN> acc;
  pair_tile<T, TM, TN>(tile, p.ldy, p.ldw, acc);
  using Epilogue = MlpDzEpilogue<T, TM, TN, AGAIN>;
  char* lds = nullptr;
  if constexpr (Epilogue::kTurn) {
    // All waves' copies have landed and their reads are over.
    using S = Stages<TM, TN, 2>;
    static_assert(2 * 96 * Epilogue::kTurnLd * sizeof(T) <= S::kBytes, "two waves' turned columns in a stage");
    lds_barrier();
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lds = (w & 1 ? S::s1() : S::s0()) + (w >> 1) * (96 * Epilogue::kTurnLd * sizeof(T));
  }
  Epilogue epilogue(p, tm, tn);
  epilogue.dz_exp = dz_exp;
  epilogue.h_exp = h_exp;
  epilogue.store(acc, reinterpret_cast<T*>(lds));
  if constexpr (kRanged<T> && !AGAIN) epilogue.leave_keys();
}

// The second launch (fp16): leaves the units of all da and db and of all h for
// the products, and makes those tiles again that are out of range.
template <typename T, int TM, int TN>
__device__ __forceinline__ void dz_again(const MlpDzArgs& p) {
  static_assert(kRangeSlots == 64, "a lane each");
  const int lane = threadIdx.x & 63;
  const uint32_t dz_key = p.range->dz[lane], h_key = p.range->h[lane], outside = p.range->outside;
  const int dz_exp = wave_held_exp(dz_key), h_exp = wave_held_exp(h_key);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.range->dz_exp = dz_exp;
    p.range->h_exp = h_exp;
  }
  const bool all = dz_exp != 0 || h_exp != 0;
  if (!all && !outside) return;
  const int tiles = p.tiles_m * p.tiles_n;
  for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
    int tm, tn;
    grouped_tile(xcd_order(t, tiles), p.tiles_m, p.tiles_n, tm, tn);
    const int64_t row = (int64_t)tm * TM + threadIdx.x;
    const bool mine = (int)threadIdx.x < TM && row < p.n && out_of_range(p.range->row[row]);
    // Also a barrier behind the reads of the tile before.
    if (__syncthreads_or(mine) || all) dz_tile<T, TM, TN, true>(p, tm, tn, dz_exp, h_exp);
  }
}

template <typename T, int TM, int TN, bool AGAIN = false>
__global__ void __launch_bounds__(kThreads, 2) k_mlp_dz(MlpDzArgs p) {
  if constexpr (AGAIN) {
    dz_again<T, TM, TN>(p);
  } else {
    const int tiles = p.tiles_m * p.tiles_n;
    if ((int)blockIdx.x >= tiles)
      return mlp_copy_block<T>(p.side, blockIdx.x - tiles, reinterpret_cast<T*>(Stages<TM, TN, 2>::s0()));
    int tm, tn;
    grouped_tile(xcd_order(blockIdx.x, tiles), p.tiles_m, p.tiles_n, tm, tn);
    dz_tile<T, TM, TN, false>(p, tm, tn, 0, 0);
  }
}

// ---------------------------------------------------------------------------
// Products whose result is the caller's, each L R^T: up to kMlpProducts of one
// shape of operand rows (the weights' gradients), then one more (dx, or y
// alone), whose contraction may be split.
// ---------------------------------------------------------------------------
struct MlpProduct {
  const void *L, *R;
  int tiles_m, tiles_n;
  int64_t rows_l, rows_r;  // rows of L and R that may be read
  void* out;
  int64_t ldo, rows;       // row stride, valid rows
  int cols;                // and columns
};
constexpr int kMlpProducts = 3;
struct MlpGradArgs {
  MlpProduct w[kMlpProducts];
  int w_tiles[kMlpProducts];  // tiles up to and with product i
  int64_t w_ld;               // row stride of their operands, bytes
  int w_ktiles;
  MlpProduct x;
  int64_t x_ldl, x_ldr;
  int x_ktiles, splits;
  float* parts;               // splits > 1: [splits][x.tiles_m TM][x.tiles_n TN]
  int extra;                  // DhRun's
  const HeldRange* range;     // fp16: of x's rows and, with w, of its operands
  int32_t* d_status;
  int32_t status_bits;
};

// An accumulator's values times a power of two, per 32 rows.
template <typename T, int TM, int TN>
__device__ __forceinline__ void take_back(Acc<T, TM, TN>& acc, int fm, int held) {
  using A = Acc<T, TM, TN>;
#pragma unroll
  for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc.v[fm][fn][e] = scaled(acc.v[fm][fn][e], -held);
}

template <typename T, int TM, int TN>
__device__ __forceinline__ void product_store(const MlpProduct& o, int tm, int tn, const LanePlace<TM, TN>& at,
                                              const Acc<T, TM, TN>& acc, int32_t* d_status, int32_t bits) {
  using A = Acc<T, TM, TN>;
  const int64_t row0 = (int64_t)tm * TM + at.wr + at.lr;
  const int col0 = tn * TN + at.wc;
  uint32_t found = 0;
#pragma unroll
  for (int fm = 0; fm < A::FM; ++fm) {
    const int64_t row = row0 + fm * 32;
    if (row >= o.rows) continue;
    T* out = reinterpret_cast<T*>(o.out) + row * o.ldo;
#pragma unroll
    for (int fn = 0; fn < A::FN; ++fn) {
      f32x4 v[4];
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[g][e] = acc.v[fm][fn][4 * g + e];
      found |= put_block<T>(out, col0 + 32 * fn, o.cols, at.h, v);
    }
  }
  if (d_status) report_status(d_status, bits, found & kNonfiniteMask<T>);
}

template <typename T, int TM, int TN>
__device__ __forceinline__ StreamTile product_tile(const MlpProduct& o, int64_t ldl, int64_t ldr, int tm, int tn, int kt0,
                                                   int kts) {
  const int64_t l = o.rows_l - (int64_t)tm * TM, r = o.rows_r - (int64_t)tn * TN;
  return StreamTile{reinterpret_cast<const char*>(o.L) + (int64_t)tm * TM * ldl,
                    reinterpret_cast<const char*>(o.R) + (int64_t)tn * TN * ldr,
                    (int)(l < TM ? l : TM), (int)(r < TN ? r : TN), kt0, kts};
}

// Which of the weights' gradients tile i of their list is, and where in it.
struct WeightTile {
  int which, tm, tn;
  __device__ __forceinline__ WeightTile(const MlpGradArgs& p, int i) {
    which = i < p.w_tiles[0] ? 0 : i < p.w_tiles[1] ? 1 : 2;
    const int first = which == 0 ? 0 : which == 1 ? p.w_tiles[0] : p.w_tiles[1];
    const int m = which == 0 ? p.w[0].tiles_m : which == 1 ? p.w[1].tiles_m : p.w[2].tiles_m;
    const int n = which == 0 ? p.w[0].tiles_n : which == 1 ? p.w[1].tiles_n : p.w[2].tiles_n;
    grouped_tile(i - first, m, n, tm, tn);
  }
};

template <typename T, int TM, int TN>
struct WeightEpilogue {
  static constexpr int kStores = 0;  // rows and columns past the result store nothing
  const MlpGradArgs& p;
  const TileRun& run;
  int dz_exp, h_exp;  // fp16
  LanePlace<TM, TN> at;
  __device__ __forceinline__ void load(int) {}
  __device__ __forceinline__ void settle() {}
  __device__ __forceinline__ void store(int j, Acc<T, TM, TN>& acc) {
    const WeightTile t(p, run.at(j));
    if constexpr (kRanged<T>) {
      const int held = t.which == 2 ? h_exp : dz_exp;
      if (held != 0) {
#pragma unroll
        for (int fm = 0; fm < Acc<T, TM, TN>::FM; ++fm) take_back<T, TM, TN>(acc, fm, held);
      }
    }
    product_store<T, TM, TN>(p.w[t.which], t.tm, t.tn, at, acc, p.d_status, p.status_bits);
  }
};

template <typename T, int TM, int TN>
struct SplitEpilogue {
  using A = Acc<T, TM, TN>;
  static constexpr int kStores = 0;
  const MlpGradArgs& p;
  const DhRun& run;
  bool outside;  // fp16: whether rows have units of their own
  LanePlace<TM, TN> at;
  __device__ __forceinline__ void load(int) {}
  __device__ __forceinline__ void settle() {}
  __device__ __forceinline__ void store(int j, A& acc) {
    const int per = p.x.tiles_m * p.x.tiles_n, i = run.at(j);
    int tm, tn;
    grouped_tile(i % per, p.x.tiles_m, p.x.tiles_n, tm, tn);
    if constexpr (kRanged<T>) {
      if (outside) {
        const int64_t row = (int64_t)tm * TM + at.wr + at.lr;
#pragma unroll
        for (int fm = 0; fm < A::FM; ++fm)
          take_back<T, TM, TN>(acc, fm, row + fm * 32 < p.x.rows ? held_exp(p.range->row[row + fm * 32]) : 0);
      }
    }
    if (p.splits == 1) return product_store<T, TM, TN>(p.x, tm, tn, at, acc, p.d_status, p.status_bits);
    const int64_t ld = (int64_t)p.x.tiles_n * TN;
    float* out = p.parts + ((int64_t)(i / per) * p.x.tiles_m * TM + (int64_t)tm * TM + at.wr + at.lr) * ld + tn * TN +
                 at.wc + 4 * at.h;
#pragma unroll
    for (int fm = 0; fm < A::FM; ++fm) {
      // Rows past the result are not summed either.
      if ((int64_t)tm * TM + at.wr + at.lr + fm * 32 >= p.x.rows) continue;
#pragma unroll
      for (int fn = 0; fn < A::FN; ++fn)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<f32x4*>(out + (int64_t)fm * 32 * ld + fn * 32 + 8 * g) =
              f32x4{acc.v[fm][fn][4 * g], acc.v[fm][fn][4 * g + 1], acc.v[fm][fn][4 * g + 2], acc.v[fm][fn][4 * g + 3]};
    }
  }
};

template <typename T, int TM, int TN>
__global__ void __launch_bounds__(kThreads, 1) k_mlp_products(MlpGradArgs p) {
  const int w_tiles = p.w_tiles[kMlpProducts - 1];
  bool outside = false;
  int dz_exp = 0, h_exp = 0;
  if constexpr (kRanged<T>) {
    outside = p.range->outside != 0;
    if (w_tiles > 0) {
      dz_exp = p.range->dz_exp;
      h_exp = p.range->h_exp;
    }
  }
  if (w_tiles > 0) {
    const TileRun run(w_tiles);
    stream_tiles<T, TM, TN>(
        run.count, p.w_ld, p.w_ld, (uint32_t)(p.w_ktiles * kRowBytes),
        [&](int j) {
          const WeightTile t(p, run.at(j));
          return product_tile<T, TM, TN>(p.w[t.which], p.w_ld, p.w_ld, t.tm, t.tn, 0, p.w_ktiles);
        },
        WeightEpilogue<T, TM, TN>{p, run, dz_exp, h_exp});
    // All reads of the stages are over before they are filled again.
    lds_barrier();
  }
  const int per = p.x.tiles_m * p.x.tiles_n;
  const DhRun run(w_tiles, per * p.splits, p.extra);
  stream_tiles<T, TM, TN>(
      run.count, p.x_ldl, p.x_ldr, (uint32_t)(p.x_ktiles * kRowBytes),
      [&](int j) {
        const int i = run.at(j), split = i / per;
        int tm, tn;
        grouped_tile(i % per, p.x.tiles_m, p.x.tiles_n, tm, tn);
        const int kt0 = (int)((int64_t)p.x_ktiles * split / p.splits);
        const int kt1 = (int)((int64_t)p.x_ktiles * (split + 1) / p.splits);
        return product_tile<T, TM, TN>(p.x, p.x_ldl, p.x_ldr, tm, tn, kt0, kt1 - kt0);
      },
      SplitEpilogue<T, TM, TN>{p, run, outside});
}

// The splits' sum, rounded: a thread per 16 bytes of a row.
template <typename T>
__global__ void __launch_bounds__(64) k_mlp_join(const float* parts, int splits, int64_t rows_pad, int64_t cols_pad,
                                                 T* out, int64_t ldo, int cols, int32_t* d_status, int32_t status_bits) {
  constexpr int V = kVec<T>;
  const int64_t r = blockIdx.x;
  const int c = (blockIdx.y * 64 + threadIdx.x) * V;
  uint32_t found = 0;
  if (c < cols) {
    f32x4 v[V / 4];
#pragma unroll
    for (int q = 0; q < V / 4; ++q) v[q] = f32x4{0.f, 0.f, 0.f, 0.f};
    const float* a = parts + r * cols_pad + c;
    auto sum = [&](int k0, auto batch) {
      constexpr int B = decltype(batch)::value;
      f32x4 add[B][V / 4];
#pragma unroll
      for (int k = 0; k < B; ++k)
#pragma unroll
        for (int q = 0; q < V / 4; ++q) add[k][q] = reinterpret_cast<const f32x4*>(a + (k0 + k) * rows_pad * cols_pad)[q];
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
    u32x4_t packed;
    T* t = reinterpret_cast<T*>(&packed);
#pragma unroll
    for (int k2 = 0; k2 < V; ++k2) t[k2] = from_f32<T>(v[k2 / 4][k2 % 4]);
    found = put_chunk<T>(out + r * ldo, c, cols, packed);
  }
  if (d_status) report_status(d_status, status_bits, found & kNonfiniteMask<T>);
}

// ---------------------------------------------------------------------------
// Forward for a few rows: a wave reads whole rows of the weights, in vectors
// at any alignment, the rows of x or h coming from the cache.
// ---------------------------------------------------------------------------
constexpr int kMlpDotRows = 8;  // rows of weights that a wave has in flight
struct MlpDotUpArgs {
  const void *X, *G, *U;
  int64_t ldx, ldg, ldu, n, f;  // elements
  int d;
  float* h;                     // n x ldh, not rounded: it costs nothing here
  int64_t ldh;
  void *gate, *up;              // n x f, row stride lds, or null
  int64_t lds;
  int save32;                   // they are fp32 and not T
  int act;
  int32_t* d_status;
  int32_t status_bits;
};

// A vector's worth of T's of an fp32 row.
template <int FORM, typename T>
__device__ __forceinline__ void load_floats(const float* row, int c, int cols, float (&v)[kVec<T>]) {
  u32x4_t raw[kVec<T> / 4];
#pragma unroll
  for (int q = 0; q < kVec<T> / 4; ++q) raw[q] = issue16<FORM, float>(row, c + 4 * q, cols);
#pragma unroll
  for (int q = 0; q < kVec<T> / 4; ++q) {
    float part[4];
    unpack<float>(settle16<FORM, float>(raw[q], row, c + 4 * q, cols), part);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[4 * q + k] = part[k];
  }
}

// acc[r][i] = the wave's share of w[r] . x[i] over columns c0, c0 + step, ...;
// X is T or float.
template <typename T, int R, int N, int FORM, typename X>
__device__ __forceinline__ void dot_rows(const T* const (&w)[R], const X* x, int64_t ldx, int n, int cols, int first,
                                         int step, float (&acc)[R][N]) {
  constexpr int V = kVec<T>;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < N; ++i) acc[r][i] = 0.f;
  u32x4_t raw[R], next[R];
#pragma unroll
  for (int r = 0; r < R; ++r) raw[r] = issue16<FORM, T>(w[r], first + lane * V, cols);
  for (int c0 = first; c0 < cols; c0 += step) {
    const int c = c0 + lane * V, cn = c0 + step < cols ? c + step : c;
#pragma unroll
    for (int r = 0; r < R; ++r) next[r] = issue16<FORM, T>(w[r], cn, cols);
    float h[N][V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const X* row = x + (i < n ? i : 0) * ldx;
      if constexpr (std::is_same_v<X, T>)
        unpack<T>(settle16<FORM, T>(issue16<FORM, T>(row, c, cols), row, c, cols), h[i]);
      else
        load_floats<FORM, T>(row, c, cols, h[i]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v[V];
      unpack<T>(settle16<FORM, T>(raw[r], w[r], c, cols), v);
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) acc[r][i] = fmaf(v[k], h[i][k], acc[r][i]);
      raw[r] = next[r];
    }
  }
}

// A wave per kMlpDotRows / 2 columns of h.
template <typename T, int N, int FORM>
__global__ void __launch_bounds__(256) k_mlp_dot_up(MlpDotUpArgs p) {
  constexpr int V = kVec<T>, C = kMlpDotRows / 2;
  const int lane = threadIdx.x & 63;
  const int64_t c0 = ((int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * C;
  if (c0 >= p.f) return;
  const T* w[kMlpDotRows];
#pragma unroll
  for (int r = 0; r < C; ++r) {
    const int64_t row = c0 + r < p.f ? c0 + r : p.f - 1;
    w[r] = reinterpret_cast<const T*>(p.G) + row * p.ldg;
    w[C + r] = reinterpret_cast<const T*>(p.U) + row * p.ldu;
  }
  float acc[kMlpDotRows][N];
  dot_rows<T, kMlpDotRows, N, FORM>(w, reinterpret_cast<const T*>(p.X), p.ldx, (int)p.n, p.d, 0, 64 * V, acc);
  // Lane r N + i keeps column c0 + r of row i.
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int r = 0; r < C; ++r)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float s = wave_row_sum<64>(acc[r][i]), u = wave_row_sum<64>(acc[C + r][i]);
      a = lane == r * N + i ? s : a;
      b = lane == r * N + i ? u : b;
    }
  const int row = lane % N;
  const int64_t c = c0 + lane / N;
  bool bad = false;
  if (lane < C * N && row < p.n && c < p.f) {
    float h = 0.f;
    with_act(p.act, [&](auto act) { h = Act<decltype(act)::value>(a).value * b; });
    p.h[row * p.ldh + c] = h;
    if (p.gate) {
      auto save = [&](auto s) {
        using S = decltype(s);
        reinterpret_cast<S*>(p.gate)[row * p.lds + c] = from_f32<S>(a);
        reinterpret_cast<S*>(p.up)[row * p.lds + c] = from_f32<S>(b);
        bad = !(fabsf(a) < kRoundsToInf<S> && fabsf(b) < kRoundsToInf<S>);
      };
      if (p.save32)
        save(float{});
      else
        save(T{});
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
}

struct MlpDotDownArgs {
  const float* h;
  const void* W;
  int64_t ldh, ldw, n, d;  // elements
  int f;
  void* y;
  int64_t ldy;
  int32_t* d_status;
  int32_t status_bits;
};

// A block per kMlpDotRows columns of y: there are few of them and their rows
// are long, so the block's four waves share the columns of f.
template <typename T, int N, int FORM>
__global__ void __launch_bounds__(256) k_mlp_dot_down(MlpDotDownArgs p) {
  constexpr int V = kVec<T>, R = kMlpDotRows;
  __shared__ float sh[4][R * N];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c0 = (int64_t)blockIdx.x * R;
  const T* w[R];
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = reinterpret_cast<const T*>(p.W) + (c0 + r < p.d ? c0 + r : p.d - 1) * p.ldw;
  float acc[R][N];
  dot_rows<T, R, N, FORM>(w, p.h, p.ldh, (int)p.n, p.f, wave * 64 * V, 4 * 64 * V, acc);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float s = wave_row_sum<64>(acc[r][i]);
      if (lane == 0) sh[wave][r * N + i] = s;
    }
  __syncthreads();
  const int t = threadIdx.x, row = t % N;
  const int64_t c = c0 + t / N;
  bool bad = false;
  if (t < R * N && row < p.n && c < p.d) {
    const float y = (sh[0][t] + sh[1][t]) + (sh[2][t] + sh[3][t]);
    reinterpret_cast<T*>(p.y)[row * p.ldy + c] = from_f32<T>(y);
    bad = !(fabsf(y) < kRoundsToInf<T>);
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
}

}  // namespace nsk

// ---------------------------------------------------------------------------
// Launchers, instantiated per operand type in kern_mlp_*.hip.
// ---------------------------------------------------------------------------
namespace nsr {

using namespace nsk;

// Tiles, rows by right-hand rows.  The projections' right-hand rows are two a
// column.  16-bit products have short ones beside them, for few rows.
enum MlpTile { kTileLarge = 0, kTileSmall = 1, kTileShort = 2 };
struct TileShape {
  int m, n;
};
template <typename T>
constexpr TileShape up_shape(int tile) {
  if (sizeof(T) == 4) return tile == kTileLarge ? TileShape{128, 128} : TileShape{64, 128};
  return tile == kTileLarge ? TileShape{128, 256} : tile == kTileSmall ? TileShape{128, 128} : TileShape{64, 128};
}
template <typename T>
constexpr TileShape dz_shape(int tile) {
  if (sizeof(T) == 4) return tile == kTileLarge ? TileShape{128, 128} : TileShape{64, 64};
  return tile == kTileLarge ? TileShape{128, 128} : TileShape{64, 128};
}
template <typename T>
constexpr TileShape product_shape(int tile) {
  return tile == kTileLarge   ? TileShape{kXentLarge<T>, kXentLarge<T>}
         : tile == kTileSmall ? TileShape{kXentSmall<T>, kXentSmall<T>}
                              : TileShape{64, 128};
}

// again: the second launch for operands out of range (fp16).
template <typename T> hipError_t launch_mlp_up(const MlpUpArgs& a, int tile, bool again, hipStream_t s);
template <typename T> hipError_t launch_mlp_dz(const MlpDzArgs& a, int tile, bool again, hipStream_t s);
template <typename T> hipError_t launch_mlp_products(const MlpGradArgs& a, int tile, hipStream_t s);
template <typename T> hipError_t launch_mlp_dot_up(const MlpDotUpArgs& a, hipStream_t s);
template <typename T> hipError_t launch_mlp_dot_down(const MlpDotDownArgs& a, hipStream_t s);

#define NS_MLP_TILE(K, SHAPE, TILE, GRID) \
  hipLaunchKernelGGL((K<T, SHAPE<T>(TILE).m, SHAPE<T>(TILE).n>), GRID, dim3(kThreads), 0, s, a)
#define NS_MLP_PASS(K, SHAPE, TILE, AGAIN, GRID) \
  hipLaunchKernelGGL((K<T, SHAPE<T>(TILE).m, SHAPE<T>(TILE).n, AGAIN>), GRID, dim3(kThreads), 0, s, a)
template <typename T, bool AGAIN>
void mlp_up_pass(const MlpUpArgs& a, int tile, dim3 grid, hipStream_t s) {
  if (tile == kTileLarge)
    NS_MLP_PASS(k_mlp_up, up_shape, kTileLarge, AGAIN, grid);
  else if (tile == kTileSmall || sizeof(T) == 4)
    NS_MLP_PASS(k_mlp_up, up_shape, kTileSmall, AGAIN, grid);
  else
    NS_MLP_PASS(k_mlp_up, up_shape, kTileShort, AGAIN, grid);
}
template <typename T>
hipError_t mlp_up_of(const MlpUpArgs& a, int tile, bool again, hipStream_t s) {
  const dim3 tiles = xent_grid((int64_t)a.tiles_m * a.tiles_n);
  // With copies the tiles are fewer than the compute units; the others take
  // the copies.
  if (!again) mlp_up_pass<T, false>(a, tile, a.side.blocks() > 0 ? dim3(kXentGroups) : tiles, s);
  if constexpr (kRanged<T>) {
    if (again) mlp_up_pass<T, true>(a, tile, tiles, s);
  }
  return hipGetLastError();
}
template <typename T, bool AGAIN>
void mlp_dz_pass(const MlpDzArgs& a, int tile, dim3 grid, hipStream_t s) {
  if (tile == kTileLarge)
    NS_MLP_PASS(k_mlp_dz, dz_shape, kTileLarge, AGAIN, grid);
  else
    NS_MLP_PASS(k_mlp_dz, dz_shape, kTileSmall, AGAIN, grid);
}
template <typename T>
hipError_t mlp_dz_of(const MlpDzArgs& a, int tile, bool again, hipStream_t s) {
  const int64_t tiles = (int64_t)a.tiles_m * a.tiles_n;
  if (!again) mlp_dz_pass<T, false>(a, tile, dim3((unsigned)(tiles + a.side.blocks())), s);
  if constexpr (kRanged<T>) {
    if (again) mlp_dz_pass<T, true>(a, tile, dim3((unsigned)std::min<int64_t>(tiles, 2 * kXentGroups)), s);
  }
  return hipGetLastError();
}
template <typename T>
hipError_t mlp_products_of(const MlpGradArgs& a, int tile, hipStream_t s) {
  const dim3 grid = xent_grid(a.w_tiles[kMlpProducts - 1] + (int64_t)a.x.tiles_m * a.x.tiles_n * a.splits);
  if (tile == kTileLarge) {
    NS_MLP_TILE(k_mlp_products, product_shape, kTileLarge, grid);
  } else if (tile == kTileSmall) {
    NS_MLP_TILE(k_mlp_products, product_shape, kTileSmall, grid);
  } else {
    if constexpr (sizeof(T) == 2) NS_MLP_TILE(k_mlp_products, product_shape, kTileShort, grid);
  }
  return hipGetLastError();
}
#define NS_MLP_DOT(K, N, FORM) hipLaunchKernelGGL((K<T, N, FORM>), grid, dim3(256), 0, s, a)
#define NS_MLP_DOTS(K, COLS)                                                      \
  auto run = [&](auto form) {                                                     \
    constexpr int FORM = decltype(form)::value;                                   \
    switch (xent_dot_rows(a.n)) {                                                 \
      case 1: NS_MLP_DOT(K, 1, FORM); break;                                      \
      case 2: NS_MLP_DOT(K, 2, FORM); break;                                      \
      case 4: NS_MLP_DOT(K, 4, FORM); break;                                      \
      default: NS_MLP_DOT(K, 8, FORM);                                            \
    }                                                                             \
  };                                                                              \
  if ((COLS) % kVec<T> == 0)                                                      \
    run(std::integral_constant<int, kEven>{});                                    \
  else if ((COLS) > kVec<T>)                                                      \
    run(std::integral_constant<int, kRagged>{});                                  \
  else                                                                            \
    run(std::integral_constant<int, kTiny>{});                                    \
  return hipGetLastError()
template <typename T>
hipError_t mlp_dot_up_of(const MlpDotUpArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.f + 2 * kMlpDotRows - 1) / (2 * kMlpDotRows)));
  NS_MLP_DOTS(k_mlp_dot_up, a.d);
}
template <typename T>
hipError_t mlp_dot_down_of(const MlpDotDownArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.d + kMlpDotRows - 1) / kMlpDotRows));
  NS_MLP_DOTS(k_mlp_dot_down, a.f);
}

#define NS_MLP_LAUNCHERS(T)                                                          \
  template <>                                                                        \
  hipError_t launch_mlp_up<T>(const MlpUpArgs& a, int tile, bool again, hipStream_t s) { \
    return mlp_up_of<T>(a, tile, again, s);                                          \
  }                                                                                  \
  template <>                                                                        \
  hipError_t launch_mlp_dz<T>(const MlpDzArgs& a, int tile, bool again, hipStream_t s) { \
    return mlp_dz_of<T>(a, tile, again, s);                                          \
  }                                                                                  \
  template <>                                                                        \
  hipError_t launch_mlp_products<T>(const MlpGradArgs& a, int tile, hipStream_t s) { \
    return mlp_products_of<T>(a, tile, s);                                           \
  }                                                                                  \
  template <>                                                                        \
  hipError_t launch_mlp_dot_up<T>(const MlpDotUpArgs& a, hipStream_t s) {            \
    return mlp_dot_up_of<T>(a, s);                                                   \
  }                                                                                  \
  template <>                                                                        \
  hipError_t launch_mlp_dot_down<T>(const MlpDotDownArgs& a, hipStream_t s) {        \
    return mlp_dot_down_of<T>(a, s);                                                 \
  }

}  // namespace nsr
