// embed.hpp - embedding lookup with scaling, and its gradient by sorted
// tokens.
//
//   out_i = scale * T[id_i]          dT[v] = scale * sum_{i : id_i = v} dy_i
//
// An id outside the table reads and receives nothing: its output row is
// zero, and it sets a status bit.
//
// The gradient has no floating-point atomics: the positions of every id are
// first listed in order (k_embed_sort), and each table row is then summed
// from its list in fp32 and written once, the rows without a token as zeros
// in the same pass.  The order of every sum is fixed by the ids alone.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "norm.hpp"

namespace nsk {

__device__ __forceinline__ int64_t load_id(const void* ids, int ids64, int64_t i) {
  return ids64 ? reinterpret_cast<const int64_t*>(ids)[i] : (int64_t) reinterpret_cast<const int32_t*>(ids)[i];
}

struct EmbedArgs {
  const void* ids;
  int ids64;
  int64_t n;      // positions
  int64_t vocab;  // table rows
  int cols;
  const void* T;  // vocab x cols, row stride ldt
  void* out;      // n x cols, row stride ldo
  int64_t ldt, ldo;
  float scale;
  int32_t* d_status;
  int32_t index_bit, status_bits;
};

// One wave per position, four vectors per lane in flight.  Bound by memory:
// 32768 rows of 4096 16-bit columns from a table of 128000 take 75 us, 268 MB
// written and the distinct rows read.
template <typename IO, int FORM>
__global__ void __launch_bounds__(256) k_embed(EmbedArgs p) {
  constexpr int V = kVec<IO>, U = 4;
  const int lane = threadIdx.x & 63;
  bool bad = false, outside = false;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < p.n; i += (int64_t)gridDim.x * 4) {
    const int64_t id = load_id(p.ids, p.ids64, i);
    const bool in = id >= 0 && id < p.vocab;
    const IO* src = reinterpret_cast<const IO*>(p.T) + (in ? id : 0) * p.ldt;
    IO* dst = reinterpret_cast<IO*>(p.out) + i * p.ldo;
    outside |= !in;
    for (int c0 = lane * V; c0 < p.cols; c0 += 64 * V * U) {
      u32x4_t raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = issue16<FORM, IO>(src, c0 + u * 64 * V, p.cols);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 64 * V;
        if (c >= p.cols) continue;
        float f[V];
        unpack<IO>(settle16<FORM, IO>(raw[u], src, c, p.cols), f);
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = in ? f[k] * p.scale : 0.f;
        bad |= rounds_to_nonfinite<IO, V>(f);
        store16v<FORM, IO>(dst, c, p.cols, f);
      }
    }
  }
  if (p.d_status) {
    report_status(p.d_status, p.status_bits, bad);
    report_status(p.d_status, p.index_bit, outside);
  }
}

// ---------------------------------------------------------------------------
// Sorting: order[] lists the positions by id, equal ids by position; key[]
// holds their ids; start[v] is where id v's list begins (start[vocab]: the
// number of valid positions).
// ---------------------------------------------------------------------------
// Block b owns the ids [b R, (b + 1) R) and reads all ids: it counts the ids
// below its range (where its lists begin) and, per wave and id, those inside,
// which each wave also notes in LDS.  Then it places the positions.  Wave w
// reads the w-th sixteenth of the positions, so a list in (wave, position)
// order is in position order.  A wave whose notes do not fit (a block of very
// frequent ids) reads its share again instead.  No block waits for another,
// and the lists need no atomic whose order shows.
//
// The ids come from L2 once per block, about one block per compute unit: 16384
// of them take 12 us, 65536 28 us, beside 17 and 158 us for the sums of 768
// and 2048 columns.
constexpr int kSortWaves = 16;
constexpr int kSortMaxIds = 512;  // R: 16 x 512 counters take 32 KiB
constexpr int kSortNotes = 512;   // per wave; 32 KiB
constexpr int kNoteBits = 22;     // a note: the id's place in the range, and the position in the wave's share

struct SortArgs {
  const void* ids;
  int ids64;
  int64_t n, vocab;
  int per_block;  // R, a power of two, 64 .. kSortMaxIds
  int32_t *order, *key, *start;
  int32_t* d_status;
  int32_t index_bit;
};

static __global__ void __launch_bounds__(kSortWaves * 64) k_embed_sort(SortArgs p) {
  __shared__ int cnt[kSortWaves][kSortMaxIds];
  __shared__ uint32_t notes[kSortWaves][kSortNotes];
  __shared__ int scan[kSortMaxIds];
  __shared__ int sh[kSortWaves];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, R = p.per_block;
  const unsigned long long lower = (1ull << lane) - 1;
  const int64_t lo = (int64_t)blockIdx.x * R;
  const int64_t hi = lo + R < p.vocab ? lo + R : p.vocab;
  for (int i = threadIdx.x; i < kSortWaves * R; i += kSortWaves * 64) cnt[i / R][i % R] = 0;
  __syncthreads();
  const int64_t share = (p.n + kSortWaves * 64 - 1) / (kSortWaves * 64) * 64;
  const int64_t i0 = w * share < p.n ? w * share : p.n, i1 = i0 + share < p.n ? i0 + share : p.n;
  int below = 0, noted = 0;
  bool bad = false;
  constexpr int U = 8;
  auto fetch = [&](int64_t i, int64_t (&id)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = i + u * 64 + lane < i1 ? load_id(p.ids, p.ids64, i + u * 64 + lane) : p.vocab;
  };
  int64_t id[U], next[U];
  fetch(i0, id);
  for (int64_t i = i0; i < i1; i += 64 * U) {
    fetch(i + 64 * U, next);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      below += id[u] >= 0 && id[u] < lo;
      bad |= i + u * 64 + lane < i1 && (id[u] < 0 || id[u] >= p.vocab);
      const bool in = id[u] >= lo && id[u] < hi;
      const unsigned long long all = __ballot(in);
      if (all) {
        if (in) {
          const uint32_t local = (uint32_t)(id[u] - lo);
          atomicAdd(&cnt[w][local], 1);
          const int at = noted + __popcll(all & lower);
          if (at < kSortNotes) notes[w][at] = (local << kNoteBits) | (uint32_t)((i - i0 + u * 64 + lane) & ((1 << kNoteBits) - 1));
        }
        noted += __popcll(all);
      }
      id[u] = next[u];
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) below += __shfl_xor(below, off, 64);
  if (lane == 0) sh[w] = below;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int i = 0; i < kSortWaves; ++i) base += sh[i];
  // Inclusive scan over the ids' totals (R <= 512 <= the block's threads).
  int total = 0;
  if ((int)threadIdx.x < R) {
    for (int i = 0; i < kSortWaves; ++i) total += cnt[i][threadIdx.x];
    scan[threadIdx.x] = total;
  }
  __syncthreads();
  for (int off = 1; off < R; off <<= 1) {
    int add = 0;
    if ((int)threadIdx.x < R && (int)threadIdx.x >= off) add = scan[threadIdx.x - off];
    __syncthreads();
    if ((int)threadIdx.x < R) scan[threadIdx.x] += add;
    __syncthreads();
  }
  if ((int)threadIdx.x < R) {
    int at = base + scan[threadIdx.x] - total;
    if (lo + threadIdx.x < p.vocab) p.start[lo + threadIdx.x] = at;
    if (lo + threadIdx.x == p.vocab - 1) p.start[p.vocab] = at + total;
    for (int i = 0; i < kSortWaves; ++i) {
      const int c = cnt[i][threadIdx.x];
      cnt[i][threadIdx.x] = at;
      at += c;
    }
  }
  __syncthreads();
  // Places up to 64 positions of this wave: equal ids take consecutive places
  // in lane order.
  auto place = [&](int local, int64_t pos) {
    unsigned long long todo = __ballot(local >= 0);
    while (todo) {
      const int lead = __ffsll(todo) - 1;
      const int k = __builtin_amdgcn_readlane(local, lead);
      const unsigned long long same = __ballot(local == k);
      int at = 0;
      if (lane == lead) at = atomicAdd(&cnt[w][k], (int)__popcll(same));
      at = __builtin_amdgcn_readlane(at, lead);
      if (local == k) {
        at += __popcll(same & lower);
        p.order[at] = (int32_t)pos;
        p.key[at] = (int32_t)(lo + local);
      }
      todo &= ~same;
    }
  };
  if (noted <= kSortNotes && share <= (int64_t(1) << kNoteBits)) {
    for (int j = 0; j < noted; j += 64) {
      const uint32_t note = j + lane < noted ? notes[w][j + lane] : 0;
      place(j + lane < noted ? (int)(note >> kNoteBits) : -1, i0 + (note & ((1u << kNoteBits) - 1)));
    }
  } else {
    for (int64_t i = i0; i < i1; i += 64 * U) {
      fetch(i, id);
#pragma unroll
      for (int u = 0; u < U; ++u)
        place(id[u] >= lo && id[u] < hi ? (int)(id[u] - lo) : -1, i + u * 64 + lane);
    }
  }
  if (p.d_status && blockIdx.x == 0) report_status(p.d_status, p.index_bit, bad);
}

// ---------------------------------------------------------------------------
// Summing.  order[] is cut into chunks of equal length, one wave per chunk
// and slice of columns: the lists differ in length by orders of magnitude,
// the chunks do not.  A list inside one chunk is summed and written by its
// wave.  The pieces of a list that crosses chunk borders are written as fp32
// partial rows (a chunk has at most two: the list that enters it and the one
// that leaves it), and k_embed_join adds them up.
// ---------------------------------------------------------------------------
struct EmbedSumArgs {
  const void* dY;  // n x cols, row stride lddy
  void* dT;        // vocab x cols, row stride ldt
  int64_t n, vocab, lddy, ldt;
  int cols;
  const int32_t *order, *key, *start;
  float* partial;  // [chunks][2][cols_pad]: the entering and the leaving list's piece
  int cols_pad;    // cols in whole slices
  int chunk;       // a power of two
  int chunks;
  float scale;
  int accumulate;
  int32_t* d_status;
  int32_t status_bits;
};

// dT's row from a finished sum: scaled, added to what is there if asked, and
// rounded once.
template <typename IO, int U, int FORM>
__device__ __forceinline__ bool embed_finish(const EmbedSumArgs& p, int64_t v, int c0, float (&acc)[U][kVec<IO>]) {
  constexpr int V = kVec<IO>;
  IO* out = reinterpret_cast<IO*>(p.dT) + v * p.ldt;
  bool bad = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * 64 * V;
    if (c >= p.cols) continue;
    float old[V];
    if (p.accumulate) unpack<IO>(settle16<FORM, IO>(issue16<FORM, IO>(out, c, p.cols), out, c, p.cols), old);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      acc[u][k] *= p.scale;
      if (p.accumulate) acc[u][k] += old[k];
      bad |= c + k < p.cols && !(fabsf(acc[u][k]) < kRoundsToInf<IO>);
    }
    store16v<FORM, IO>(out, c, p.cols, acc[u]);
  }
  return bad;
}

template <int U, int V>
__device__ __forceinline__ void zero_acc(float (&acc)[U][V]) {
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int k = 0; k < V; ++k) acc[u][k] = 0.f;
}

// Rows with no position, kZeroRows ids per block.
constexpr int kZeroRows = 16;

// Blocks [0, chunks): the sums.  Blocks from there on: the zeros (none when
// adding to dT).  U vectors per lane and slice; B rows in flight.
template <typename IO, int U, int B, int FORM>
__global__ void __launch_bounds__(64) k_embed_sum(EmbedSumArgs p) {
  constexpr int V = kVec<IO>;
  const int lane = threadIdx.x;
  const int c0 = (blockIdx.y * U * 64 + lane) * V;
  if ((int)blockIdx.x >= p.chunks) {
    const int64_t v0 = (int64_t)(blockIdx.x - p.chunks) * kZeroRows;
    const int64_t vi = v0 + lane < p.vocab ? v0 + lane : p.vocab;
    const int bounds = lane <= kZeroRows ? p.start[vi] : 0;
    const float zero[V] = {};
#pragma unroll
    for (int r = 0; r < kZeroRows; ++r) {
      if (v0 + r >= p.vocab || __builtin_amdgcn_readlane(bounds, r) != __builtin_amdgcn_readlane(bounds, r + 1)) continue;
      IO* out = reinterpret_cast<IO*>(p.dT) + (v0 + r) * p.ldt;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 64 * V;
        if (c < p.cols) store16v<FORM, IO>(out, c, p.cols, zero);
      }
    }
    return;
  }
  const int total = p.start[p.vocab];
  const int s = blockIdx.x * p.chunk, e = s + p.chunk < total ? s + p.chunk : total;
  if (s >= e) return;
  const IO* dY = reinterpret_cast<const IO*>(p.dY);
  // The ids before and behind the chunk say whether a list enters or leaves.
  const int before = s > 0 ? p.key[s - 1] : -1, behind = e < total ? p.key[e] : -1;
  float acc[U][V];
  zero_acc<U, V>(acc);
  bool bad = false, entering = false;
  int current = -1;
  auto finish = [&](bool leaving) {
    if (entering || leaving) {
      float* out = p.partial + ((int64_t)blockIdx.x * 2 + (entering ? 0 : 1)) * p.cols_pad;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < V; k += 4)
          *reinterpret_cast<f32x4*>(out + c0 + u * 64 * V + k) =
              f32x4{acc[u][k], acc[u][k + 1], acc[u][k + 2], acc[u][k + 3]};
    } else {
      bad |= embed_finish<IO, U, FORM>(p, current, c0, acc);
    }
  };
  for (int b = s; b < e; b += 64) {
    const int at = b + lane < e ? b + lane : e - 1;
    const int pos = p.order[at], ids = p.key[at];
    const int m = e - b < 64 ? e - b : 64;
    if (b == s) {
      current = __builtin_amdgcn_readlane(ids, 0);
      entering = current == before;
    }
    for (int j = 0; j < m; j += B) {
      u32x4_t raw[B][U];
#pragma unroll
      for (int q = 0; q < B; ++q) {
        const IO* row = dY + (int64_t)__builtin_amdgcn_readlane(pos, j + q < m ? j + q : m - 1) * p.lddy;
#pragma unroll
        for (int u = 0; u < U; ++u) raw[q][u] = issue16<FORM, IO>(row, c0 + u * 64 * V, p.cols);
      }
#pragma unroll
      for (int q = 0; q < B; ++q) {
        if (j + q < m) {
          const int id = __builtin_amdgcn_readlane(ids, j + q);
          if (id != current) {
            finish(false);
            zero_acc<U, V>(acc);
            current = id;
            entering = false;
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float f[V];
            unpack<IO>(settle16<FORM, IO>(raw[q][u], dY + (int64_t)__builtin_amdgcn_readlane(pos, j + q) * p.lddy,
                                    c0 + u * 64 * V, p.cols), f);
#pragma unroll
            for (int k = 0; k < V; ++k) acc[u][k] += f[k];
          }
        }
      }
    }
  }
  finish(current == behind);
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
}

// Chunk c's wave joins the list that leaves c if it did not enter it: the
// leaving piece, then the entering pieces of the chunks it goes through.  One
// vector of columns per lane and sixteen pieces in flight: the longest list's
// latency is what this kernel takes (eight waves per list, joined in LDS, cost
// more in idle blocks than they saved).
template <typename IO, int FORM>
__global__ void __launch_bounds__(64) k_embed_join(EmbedSumArgs p) {
  constexpr int V = kVec<IO>, B = 16;
  const int total = p.start[p.vocab];
  const int64_t s = (int64_t)blockIdx.x * p.chunk, e = s + p.chunk;
  if (e >= total) return;
  const int id = p.key[e];
  if (p.key[e - 1] != id || (s > 0 && p.key[s - 1] == id)) return;
  const int c0 = (blockIdx.y * 64 + threadIdx.x) * V;
  const int last = (p.start[id + 1] - 1) / p.chunk;
  float acc[1][V];
  zero_acc<1, V>(acc);
  // Pieces 1 .. have their entering rows at even places; piece 0 is this
  // chunk's leaving row.
  const float* first = p.partial + ((int64_t)blockIdx.x * 2 + 1) * p.cols_pad + c0;
  const int pieces = last - (int)blockIdx.x + 1;
  for (int j = 0; j < pieces; j += B) {
    f32x4 raw[B][V / 4];
#pragma unroll
    for (int q = 0; q < B; ++q) {
      const int i = j + q < pieces ? j + q : pieces - 1;
      const float* part = i == 0 ? first : first + (2 * (int64_t)i - 1) * p.cols_pad;
#pragma unroll
      for (int k = 0; k < V / 4; ++k) raw[q][k] = *reinterpret_cast<const f32x4*>(part + 4 * k);
    }
#pragma unroll
    for (int q = 0; q < B; ++q) {
      if (j + q < pieces) {
#pragma unroll
        for (int k = 0; k < V; ++k) acc[0][k] += raw[q][k / 4][k % 4];
      }
    }
  }
  const bool bad = embed_finish<IO, 1, FORM>(p, id, c0, acc);
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
}

}  // namespace nsk
