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

// One wave per position.
template <typename IO, int V>
__global__ void __launch_bounds__(256) k_embed(EmbedArgs p) {
  const int lane = threadIdx.x & 63;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < p.n; i += (int64_t)gridDim.x * 4) {
    const int64_t id = load_id(p.ids, p.ids64, i);
    const bool in = id >= 0 && id < p.vocab;
    const IO* src = reinterpret_cast<const IO*>(p.T) + (in ? id : 0) * p.ldt;
    IO* dst = reinterpret_cast<IO*>(p.out) + i * p.ldo;
    bool bad = false;
    constexpr int U = 4;
    for (int c0 = lane * V; c0 < p.cols; c0 += 64 * V * U) {
      float f[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 64 * V;
        if (in && c < p.cols) load_vec<IO, V>(src + c, f[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 64 * V;
        if (c >= p.cols) continue;
#pragma unroll
        for (int k = 0; k < V; ++k) f[u][k] = in ? f[u][k] * p.scale : 0.f;
        bad |= rounds_to_nonfinite<IO, V>(f[u]);
        store_vec<IO, V>(dst + c, f[u]);
      }
    }
    if (p.d_status) {
      report_status(p.d_status, p.status_bits, bad);
      report_status(p.d_status, p.index_bit, !in);
    }
  }
}

// ---------------------------------------------------------------------------
// Sorting: order[] lists the positions by id, equal ids by position, and
// start[v] is where id v's list begins (start[vocab]: the valid positions).
// ---------------------------------------------------------------------------
// Block b owns the ids [b R, (b + 1) R).  It reads all ids twice: first it
// counts the ids below its range (where its lists begin) and, per wave and
// id, those inside; then it places the positions.  Wave w reads the w-th
// sixteenth of the positions, so a list in (wave, position) order is in
// position order.  No block waits for another, and the lists need no atomic
// whose order shows.
constexpr int kSortWaves = 16;
constexpr int kSortMaxIds = 512;  // R: 16 x 512 counters take 32 KiB

struct SortArgs {
  const void* ids;
  int ids64;
  int64_t n, vocab;
  int per_block;  // R, a power of two, 64 .. kSortMaxIds
  int32_t *order, *start;
  int32_t* d_status;
  int32_t index_bit;
};

static __global__ void __launch_bounds__(kSortWaves * 64) k_embed_sort(SortArgs p) {
  __shared__ int cnt[kSortWaves][kSortMaxIds];
  __shared__ int scan[kSortMaxIds];
  __shared__ int sh[kSortWaves];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, R = p.per_block;
  const int64_t lo = (int64_t)blockIdx.x * R;
  const int64_t hi = lo + R < p.vocab ? lo + R : p.vocab;
  for (int i = threadIdx.x; i < kSortWaves * R; i += kSortWaves * 64) cnt[i / R][i % R] = 0;
  __syncthreads();
  const int64_t share = (p.n + kSortWaves * 64 - 1) / (kSortWaves * 64) * 64;
  const int64_t i0 = w * share < p.n ? w * share : p.n, i1 = i0 + share < p.n ? i0 + share : p.n;
  int below = 0;
  bool bad = false;
  constexpr int U = 8;
  for (int64_t i = i0; i < i1; i += 64 * U) {
    int64_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = i + u * 64 + lane < i1 ? load_id(p.ids, p.ids64, i + u * 64 + lane) : p.vocab;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      below += id[u] >= 0 && id[u] < lo;
      if (id[u] >= lo && id[u] < hi) atomicAdd(&cnt[w][id[u] - lo], 1);
      bad |= i + u * 64 + lane < i1 && (id[u] < 0 || id[u] >= p.vocab);
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
  for (int64_t i = i0; i < i1; i += 64 * U) {
    int64_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = i + u * 64 + lane < i1 ? load_id(p.ids, p.ids64, i + u * 64 + lane) : p.vocab;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = id[u] >= lo && id[u] < hi;
      const int local = in ? (int)(id[u] - lo) : -1;
      unsigned long long todo = __ballot(in);
      while (todo) {
        const int lead = __ffsll(todo) - 1;
        const int key = __shfl(local, lead, 64);
        const unsigned long long same = __ballot(local == key);
        int at = 0;
        if (lane == lead) at = atomicAdd(&cnt[w][key], (int)__popcll(same));
        at = __shfl(at, lead, 64);
        if (local == key) p.order[at + __popcll(same & ((1ull << lane) - 1))] = (int32_t)(i + u * 64 + lane);
        todo &= ~same;
      }
    }
  }
  if (p.d_status && blockIdx.x == 0) report_status(p.d_status, p.index_bit, bad);
}

// ---------------------------------------------------------------------------
// Summing.
// ---------------------------------------------------------------------------
struct EmbedSumArgs {
  const void* dY;  // n x cols, row stride lddy
  void* dT;        // vocab x cols, row stride ldt
  int64_t n, vocab, lddy, ldt;
  int cols;
  const void* ids;
  int ids64;
  const int32_t *order, *start;
  float* partial;  // [n / chunk][cols]: sums of the aligned chunks of order[] that hold one id only
  int chunk;       // power of two, or 0: no partial sums
  float scale;
  int accumulate;
  int32_t* d_status;
  int32_t status_bits;
};

// acc += the rows order[s .. e) of dY, columns c0 + u * 64 V (+ V), in order.
template <typename IO, int V, int U>
__device__ __forceinline__ void sum_rows(const EmbedSumArgs& p, int s, int e, int c0, float (&acc)[U][V]) {
  const IO* dY = reinterpret_cast<const IO*>(p.dY);
  for (int b = s; b < e; b += 64) {
    const int lane = threadIdx.x & 63;
    const int mine = b + lane < e ? p.order[b + lane] : 0;
    const int m = e - b < 64 ? e - b : 64;
#pragma unroll 4
    for (int j = 0; j < m; ++j) {
      const IO* row = dY + (int64_t)__builtin_amdgcn_readlane(mine, j) * p.lddy;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * 64 * V;
        if (c < p.cols) {
          float f[V];
          load_vec<IO, V>(row + c, f);
#pragma unroll
          for (int k = 0; k < V; ++k) acc[u][k] += f[k];
        }
      }
    }
  }
}

// An id with thousands of positions would keep one wave busy long after the
// others; its list is cut at multiples of `chunk`, and the whole chunks are
// summed here by a wave each.
template <typename IO, int V, int U>
__global__ void __launch_bounds__(64) k_embed_chunks(EmbedSumArgs p) {
  const int s = blockIdx.x * p.chunk, e = s + p.chunk;
  if (e > p.start[p.vocab]) return;
  if (load_id(p.ids, p.ids64, p.order[s]) != load_id(p.ids, p.ids64, p.order[e - 1])) return;
  const int c0 = (blockIdx.y * U * 64 + (threadIdx.x & 63)) * V;
  float acc[U][V];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int k = 0; k < V; ++k) acc[u][k] = 0.f;
  sum_rows<IO, V, U>(p, s, e, c0, acc);
  float* out = p.partial + (int64_t)blockIdx.x * p.cols;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * 64 * V;
    if (c >= p.cols) continue;
#pragma unroll
    for (int k = 0; k < V; ++k) out[c + k] = acc[u][k];
  }
}

// One wave per table row and slice of U * 64 V columns.
constexpr int kEmbedRowsPerWave = 4;
template <typename IO, int V, int U>
__global__ void __launch_bounds__(256) k_embed_rows(EmbedSumArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t v0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * kEmbedRowsPerWave;
  if (v0 >= p.vocab) return;
  const int64_t vi = v0 + lane < p.vocab ? v0 + lane : p.vocab;
  const int bounds = lane <= kEmbedRowsPerWave ? p.start[vi] : 0;
  const int c0 = (blockIdx.y * U * 64 + lane) * V;
  bool bad = false;
  for (int r = 0; r < kEmbedRowsPerWave && v0 + r < p.vocab; ++r) {
    int s = __builtin_amdgcn_readlane(bounds, r);
    const int e = __builtin_amdgcn_readlane(bounds, r + 1);
    if (s == e && p.accumulate) continue;
    float acc[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < V; ++k) acc[u][k] = 0.f;
    if (p.chunk) {
      const int first = (s + p.chunk - 1) / p.chunk, last = e / p.chunk;
      if (first < last) {
        sum_rows<IO, V, U>(p, s, first * p.chunk, c0, acc);
#pragma unroll 4
        for (int q = first; q < last; ++q) {
          const float* part = p.partial + (int64_t)q * p.cols;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 64 * V;
            if (c < p.cols) {
#pragma unroll
              for (int k = 0; k < V; ++k) acc[u][k] += part[c + k];
            }
          }
        }
        s = last * p.chunk;
      }
    }
    sum_rows<IO, V, U>(p, s, e, c0, acc);
    IO* out = reinterpret_cast<IO*>(p.dT) + (v0 + r) * p.ldt;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * 64 * V;
      if (c >= p.cols) continue;
      float old[V];
      if (p.accumulate) load_vec<IO, V>(out + c, old);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        acc[u][k] *= p.scale;
        if (p.accumulate) acc[u][k] += old[k];
      }
      bad |= rounds_to_nonfinite<IO, V>(acc[u]);
      store_vec<IO, V>(out + c, acc[u]);
    }
  }
  if (p.d_status) report_status(p.d_status, p.status_bits, bad);
}

}  // namespace nsk
