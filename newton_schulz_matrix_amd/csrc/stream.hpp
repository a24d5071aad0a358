// stream.hpp - a persistent work-group's tiles as one stream of k-tiles.
//
// products.hpp's main loop fills its LDS stages at the start of a tile and
// lets them run dry before the epilogue, which costs about 8 us per tile of
// 192 x 192: little beside a contraction of 4096 (61 us), nearly as much as
// one of 768 (11 us).  Here the copies never stop: they run three k-tiles
// ahead of the products straight across tile borders, and a tile's epilogue,
// which works on the accumulators alone and touches no LDS stage, runs between the
// last products of its tile and the first of the next while those copies are
// in flight.  Stages, fragments and the steps themselves are products.hpp's.
#pragma once

#include <type_traits>

#include "products.hpp"

namespace nsk {

// One tile: its operands' first rows, how many of them are valid, and its
// k-tiles.  They are taken in groups of three, one per LDS stage, so that a
// tile always begins in the first stage and each step names its stages (with
// rotating stage pointers the compiler serialized copies and reads, 1.05 us
// per k-tile against 0.91; with a border for each of the three stages it
// spilled accumulators).  The up to two missing ones are loads past the end of
// an empty buffer resource, which give zeros and read no memory: a contraction
// of 4096 becomes 66 k-tiles instead of 64, where the drained pipeline took
// the time of eight.
struct StreamTile {
  const char *L, *R;
  int rows_l, rows_r;
  int kt0, kts;
  __device__ __forceinline__ int groups() const { return (kts + 2) / 3; }
};

template <typename T, int TM, int TN>
__device__ __forceinline__ void border_first(const DmaLoader<TM>& la, const DmaLoader<TN>& lb, int kt,
                                             char* __restrict__ D, const char* __restrict__ P, const FragAddr& fa,
                                             FragSets<TM / 64, TN / 64>& fs, f32x16 (&acc)[TM / 64][TN / 64]) {
  constexpr int FM = TM / 64, FN = TN / 64, kOffR = TM * kRowBytes;
  la.issue(kt, D);
  lb.issue(kt, D + kOffR);
  load_frags<FM, FN>(P, P + kOffR, fa, 0, fs.f0);
  load_frags<FM, FN>(P, P + kOffR, fa, 1, fs.f1);
  mma_frags<T, FM, FN>(fs.f2, acc);
  mma_frags<T, FM, FN>(fs.f3, acc);
}
// Waits until all but the `YOUNGER` latest memory operations (and the LDS
// reads) are done.  More than the counter holds are cut to 62: 63, its
// maximum, would not wait at all.
template <int YOUNGER>
__device__ __forceinline__ void wait_for_older() {
  __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(YOUNGER < 62 ? YOUNGER : 62));
}

// STORES: a lower bound on the epilogue's stores per wave, all of them issued
// after the border's copies.
template <typename T, int TM, int TN, int STORES>
__device__ __forceinline__ void border_second(const char* P, const FragAddr& fa, FragSets<TM / 64, TN / 64>& fs,
                                              f32x16 (&acc)[TM / 64][TN / 64]) {
  constexpr int FM = TM / 64, FN = TN / 64, kOffR = TM * kRowBytes;
  load_frags<FM, FN>(P, P + kOffR, fa, 2, fs.f2);
  load_frags<FM, FN>(P, P + kOffR, fa, 3, fs.f3);
  mma_frags<T, FM, FN>(fs.f0, acc);
  mma_frags<T, FM, FN>(fs.f1, acc);
  // The copies of the step before must have landed.  Memory operations
  // complete in order; younger than those copies are the border's own and the
  // epilogue's stores, which need not be waited for.
  wait_for_older<TM / 32 + TN / 32 + STORES>();
}

// pipe_step (products.hpp) for the first step after a border: the border's
// copies, for which it waits, are older than the epilogue's stores.
template <typename T, int TM, int TN, int STORES>
__device__ __forceinline__ void first_step(const DmaLoader<TM>& la, const DmaLoader<TN>& lb, int kt,
                                           char* __restrict__ D, const char* __restrict__ P, const FragAddr& fa,
                                           FragSets<TM / 64, TN / 64>& fs, f32x16 (&acc)[TM / 64][TN / 64]) {
  constexpr int FM = TM / 64, FN = TN / 64, kOffR = TM * kRowBytes;
  la.issue(kt, D);
  lb.issue(kt, D + kOffR);
  load_frags<FM, FN>(P, P + kOffR, fa, 0, fs.f0);
  load_frags<FM, FN>(P, P + kOffR, fa, 1, fs.f1);
  mma_frags<T, FM, FN>(fs.f2, acc);
  mma_frags<T, FM, FN>(fs.f3, acc);
  load_frags<FM, FN>(P, P + kOffR, fa, 2, fs.f2);
  load_frags<FM, FN>(P, P + kOffR, fa, 3, fs.f3);
  mma_frags<T, FM, FN>(fs.f0, acc);
  mma_frags<T, FM, FN>(fs.f1, acc);
  schedule_step<T, TM, TN, 1>();
  wait_for_older<TM / 32 + TN / 32 + STORES>();
  lds_barrier();
}

// Runs tiles 0 .. count - 1 of one work-group.  tile_of(j) gives tile j
// (uniform).  epi.load(j) puts the values loaded before into place and issues
// the loads that tile j's epilogue needs (called once more for the last tile,
// whose values it then puts into place), epi.settle() makes them final after
// a wait that covers them (they are issued before the border's copies), and
// epi.store(j, acc) is the epilogue, with at least kStores stores per wave.
template <typename T, int TM, int TN, class TileOf, class Epilogue>
__device__ __forceinline__ void stream_tiles(int count, int64_t ldl, int64_t ldr, uint32_t row_bytes, TileOf&& tile_of,
                                             Epilogue&& epi) {
  constexpr int FM = TM / 64, FN = TN / 64;
  constexpr int kOffR = TM * kRowBytes;
  constexpr int kDma = TM / 32 + TN / 32;
  using S = Stages<TM, TN, 1>;
  static_assert(S::kCount == 3, "the stream has three stages");
  constexpr int kStores = std::remove_reference_t<Epilogue>::kStores;
  if (count <= 0) return;
  const int w = threadIdx.x >> 6;
  const int wr = (w >> 1) * (TM / 2), wc = (w & 1) * (TN / 2);

  // Copy side: the tile being copied (c) and the one after it (n).
  //
  // An operand that is the caller's own matrix ends inside its last tile, so a
  // wave's resource ends with its last valid row (rec_l, rec_r bytes) and
  // nothing past it is read: a lane offset in an invalid row lies past the end
  // whether or not the hardware counts the scalar offset in its check, one in
  // a valid row never does.  What lands in LDS for the invalid rows reaches
  // only their own outputs.
  DmaLoader<TM> la;
  DmaLoader<TN> lb;
  struct Side {
    const char *L, *R;
    int rec_l, rec_r, kt, end, left;  // left: k-tiles to copy, the empty ones (from end on) included
  };
  auto side_of = [&](const StreamTile& t) {
    Side s;
    const int wl = la.wave_row0, wq = lb.wave_row0;
    const int left_l = t.rows_l - wl, left_r = t.rows_r - wq;
    s.L = t.L + wl * ldl;
    s.R = t.R + wq * ldr;
    s.rec_l = left_l <= 0 ? 0 : (int)((uint32_t)((left_l < TM / 4 ? left_l : TM / 4) - 1) * (uint32_t)ldl + row_bytes);
    s.rec_r = left_r <= 0 ? 0 : (int)((uint32_t)((left_r < TN / 4 ? left_r : TN / 4) - 1) * (uint32_t)ldr + row_bytes);
    s.kt = t.kt0;
    s.end = t.kt0 + t.kts;
    s.left = 3 * t.groups();
    return s;
  };
  // The loaders' lane offsets do not depend on the tile.
  la.init(nullptr, ldl);
  lb.init(nullptr, ldr);
  StreamTile tile = tile_of(0);
  Side c = side_of(tile), n;
  auto prepare_next = [&](int j) {
    if (j < count) {
      n = side_of(tile_of(j));
    } else {
      // Past the end: empty k-tiles, read by nobody.
      n = c;
      n.kt = n.end = 0;
      n.left = 1;
    }
  };
  prepare_next(1);
  // The next k-tile of the stream: selects, no branch, so that a step stays
  // one block to the scheduler.
  auto advance = [&] {
    const bool wrap = c.left == 0;
    c.L = wrap ? n.L : c.L;
    c.R = wrap ? n.R : c.R;
    c.rec_l = wrap ? n.rec_l : c.rec_l;
    c.rec_r = wrap ? n.rec_r : c.rec_r;
    c.kt = wrap ? n.kt : c.kt;
    c.end = wrap ? n.end : c.end;
    c.left = wrap ? n.left : c.left;
    const bool empty = c.kt >= c.end;
    la.rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(c.L), (short)0, empty ? 0 : c.rec_l, 0x00020000);
    lb.rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(c.R), (short)0, empty ? 0 : c.rec_r, 0x00020000);
    const int kt = c.kt;
    ++c.kt;
    --c.left;
    return kt;
  };
  auto copy = [&](char* D) {
    const int kt = advance();
    la.issue(kt, D);
    lb.issue(kt, D + kOffR);
  };

  FragAddr fa;
  fa.init(wr, wc);
  FragSets<FM, FN> fs;
  Acc<T, TM, TN> acc;
  acc_zero(acc);
  epi.load(0);
  copy(S::s0());
  copy(S::s1());
  copy(S::s2());
  __builtin_amdgcn_s_waitcnt(wait_vm(2 * kDma));
  epi.settle();
  lds_barrier();
  {
    const char* s0 = S::s0();
    load_frags<FM, FN>(s0, s0 + kOffR, fa, 0, fs.f0);
    load_frags<FM, FN>(s0, s0 + kOffR, fa, 1, fs.f1);
    load_frags<FM, FN>(s0, s0 + kOffR, fa, 2, fs.f2);
    load_frags<FM, FN>(s0, s0 + kOffR, fa, 3, fs.f3);
  }
  mma_frags<T, FM, FN>(fs.f0, acc.v);
  mma_frags<T, FM, FN>(fs.f1, acc.v);
  // All three k-tiles: the first step's wait counts an epilogue's stores,
  // and there has been none.
  __builtin_amdgcn_s_waitcnt(wait_vm_lgkm0(0));
  lds_barrier();

  // From the current k-tile (in stage D) to the next one of the tile (in P).
  auto step = [&](char* D, const char* P) {
    const int kt = advance();
    pipe_step<T, TM, TN, 1>(nullptr, nullptr, la, lb, kt, 0, D, P, fa, fs, acc.v, [](int, const char*, const FragAddr&) {});
  };
  for (int j = 0;; ++j) {
    first_step<T, TM, TN, kStores>(la, lb, advance(), S::s0(), S::s1(), fa, fs, acc.v);
    for (int g = tile.groups(); g > 1; --g) {
      step(S::s1(), S::s2());
      step(S::s2(), S::s0());
      step(S::s0(), S::s1());
    }
    step(S::s1(), S::s2());
    // The border: a step from this tile's last k-tile to the next tile's
    // first (past the end, a repeated one), in two halves around the
    // epilogue.
    const bool more = j + 1 < count;
    if (more) {
      tile = tile_of(j + 1);
      prepare_next(j + 2);
    }
    epi.load(more ? j + 1 : j);
    border_first<T, TM, TN>(la, lb, advance(), S::s2(), S::s0(), fa, fs, acc.v);
    epi.store(j, acc);
    // The waits after this count on the stores being issued by now.
    asm volatile("" ::: "memory");
    if (!more) break;
    acc_zero(acc);
    border_second<T, TM, TN, kStores>(S::s0(), fa, fs, acc.v);
    epi.settle();
    lds_barrier();
  }
  // The last, repeated copies must land before the LDS is given away.
  __builtin_amdgcn_s_waitcnt(0);
}

// ---------------------------------------------------------------------------
// Epilogue stores straight from the accumulators.  Lane (lr, h) of a 32 x 32
// block holds row lr, columns 8 g + 4 h .. + 3 for g = 0 .. 3.
// ---------------------------------------------------------------------------

// Two groups' 16-bit quads (columns 8 g .. and 8 (g + 1) ..) as one 16-byte
// chunk per lane: the halves of the wave trade quads, after which the lower
// half holds columns 8 g .. 8 g + 7 of its rows and the upper 8 g + 8 ...
__device__ __forceinline__ uint4 join_quads(uint2 even, uint2 odd) {
  auto a = __builtin_amdgcn_permlane32_swap(even.x, odd.x, false, false);
  auto b = __builtin_amdgcn_permlane32_swap(even.y, odd.y, false, false);
  return uint4{a[0], b[0], a[1], b[1]};
}

template <typename H>
__device__ __forceinline__ uint2 pack_quad(f32x4 v) {
  typedef H h4 __attribute__((ext_vector_type(4)));
  h4 o;
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = from_f32<H>(v[e]);
  return __builtin_bit_cast(uint2, o);
}

template <int CTRL>
__device__ __forceinline__ uint32_t quad_move(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, false);
}

// A 4 x 4 block transposed among the four lanes of a quad: lane q gives row q
// (four 16-bit columns) and gets column q (four rows).
__device__ __forceinline__ uint2 transpose_quad(uint2 v) {
  const bool high = threadIdx.x & 2, odd = threadIdx.x & 1;
  // Lanes 0 and 1 take columns 0, 1 of all rows, lanes 2 and 3 columns 2, 3.
  const uint32_t got = quad_move<0x4E>(high ? v.x : v.y);
  const uint32_t r0 = high ? got : v.x, r1 = high ? v.y : got;  // rows (0, 1) and (2, 3) of this lane's pair
  // Even lanes take the low columns of their own and their neighbour's row,
  // odd lanes the high ones (byte selects: as selects between shifts these
  // became branches).
  const uint32_t p0 = quad_move<0xB1>(r0), p1 = quad_move<0xB1>(r1);
  const uint32_t sel = odd ? 0x03020706u : 0x05040100u;
  return uint2{__builtin_amdgcn_perm(p0, r0, sel), __builtin_amdgcn_perm(p1, r1, sel)};
}

// The same for 32-bit columns.
__device__ __forceinline__ f32x4 transpose_quad(f32x4 v) {
  const bool high = threadIdx.x & 2, odd = threadIdx.x & 1;
  auto bits = [](float x) { return __float_as_uint(x); };
  const uint32_t g0 = quad_move<0x4E>(high ? bits(v[0]) : bits(v[2])), g1 = quad_move<0x4E>(high ? bits(v[1]) : bits(v[3]));
  // Pair (a, b): this lane's two columns of its own row and of the row two away.
  const uint32_t a0 = high ? g0 : bits(v[0]), a1 = high ? g1 : bits(v[1]);
  const uint32_t b0 = high ? bits(v[2]) : g0, b1 = high ? bits(v[3]) : g1;
  const uint32_t ga = quad_move<0xB1>(odd ? a0 : a1), gb = quad_move<0xB1>(odd ? b0 : b1);
  const uint32_t o0 = odd ? ga : a0, o1 = odd ? a1 : ga, o2 = odd ? gb : b0, o3 = odd ? b1 : gb;
  return f32x4{__uint_as_float(o0), __uint_as_float(o1), __uint_as_float(o2), __uint_as_float(o3)};
}

}  // namespace nsk
