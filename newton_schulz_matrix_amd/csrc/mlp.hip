// mlp.hip - C entry points of the gated feed-forward block (mlp.hpp): argument
// checks, workspace layout and kernel choice.
#include <math.h>
#include <stdio.h>

#include <algorithm>

#include "cost.hpp"
#include "host.hpp"
#include "mlp.hpp"

namespace {

constexpr int64_t kMaxMlpRows = 1 << 22, kMaxMlpCols = 1 << 20, kMaxMlpStride = 1 << 23;
// Elements of h at most: tiles are counted in 32 bits.
constexpr int64_t kMaxMlpInner = int64_t(1) << 40;
// Rows that go without tiles, and where tiles would need staging copies of
// the weights.
constexpr int64_t kMlpDotMost = 4, kMlpDotMostStaged = 8;

struct MlpPlan {
  int64_t n = 0, d = 0, f = 0;
  int es = 2, bk = 64;
  int64_t dk = 0, fk = 0;              // d and f in whole k-tiles
  bool stage_d = false, stage_f = false;  // operands of d or f columns need staging copies
  bool dot = false;
  // Forward.
  int up_tile = 0;                     // of the projections
  int64_t h_rows = 0, h_ld = 0;
  // y forward, the gradients backward: tile and its shape, splits of y or dx.
  int tile = 0;
  int64_t tm = 0, tn = 0;
  int splits = 1;
  // The copies that the projections (dh's product) do not read go along with
  // their tiles.
  bool side = false;
  // Backward: dh's tiles; the rows and columns that they cover, which the
  // gradients' contractions run over; d in whole 64s.
  int dz_tile = 0;
  int64_t n_pad = 0, f_pad = 0, d_pad = 0;
  // Row strides of buffers that are n_pad, 2 f_pad and d_pad wide (see skewed).
  int64_t t_ld = 0, z_ld = 0, d_ld = 0;
  // Buffers.
  char *Xs = nullptr, *Gs = nullptr, *Us = nullptr, *Ds = nullptr, *h = nullptr;
  char *Ys = nullptr, *dz = nullptr, *dzt = nullptr, *ht = nullptr, *WT = nullptr, *DT = nullptr, *XT = nullptr,
       *YT = nullptr;
  float* parts = nullptr;
  HeldRange* range = nullptr;  // fp16 (ranged)
  UpRange seen{};
  bool ranged = false;
  size_t total = 0;
};

// The row stride of a workspace buffer: an odd number of k-tiles (128 bytes).
// With rows a large power of two apart, a tile's rows meet in few memory
// channels.
int64_t skewed(int64_t width, int bk) {
  const int64_t k = (width + bk - 1) / bk;
  return (k % 2 ? k : k + 1) * bk;
}

bool mlp_shape_ok(int64_t n, int64_t d, int64_t f) {
  return n >= 0 && n <= kMaxMlpRows && d >= 1 && d <= kMaxMlpCols && f >= 1 && f <= kMaxMlpCols &&
         n <= kMaxMlpInner / f;
}

int64_t tiles_of(int64_t size, int64_t edge) { return (size + edge - 1) / edge; }

// Estimated times, as measured on MI355X: us per k-tile and fixed.  Tiles that
// share a compute unit (dh's) take `alone` per k-tile while there is one for
// each, and `ktile` for both of two.
struct TileCost {
  int tile;
  TileShape shape;
  double ktile, fixed, alone;
};
double tile_product_us(const TileCost& c, int64_t tiles, double ktiles) {
  if (c.alone == 0) return product_us(EdgeCost{0, c.ktile, c.fixed}, tiles, ktiles);
  if (tiles <= kXentGroups) return ktiles * c.alone + c.fixed;
  return (double)tiles_of(tiles, 2 * kXentGroups) * (ktiles * c.ktile + c.fixed);
}
template <typename T>
constexpr TileCost kUpCosts[3] = {{kTileLarge, up_shape<T>(kTileLarge), 0.82, 4.0, 0},
                                  {kTileSmall, up_shape<T>(kTileSmall), 0.52, 3.0, 0},
                                  {kTileShort, up_shape<T>(kTileShort), 0.36, 2.0, 0}};
template <>
constexpr TileCost kUpCosts<float>[3] = {{kTileLarge, up_shape<float>(kTileLarge), 2.10, 3.5, 0},
                                         {kTileSmall, up_shape<float>(kTileSmall), 1.06, 2.5, 0},
                                         {kTileSmall, up_shape<float>(kTileSmall), 1.06, 2.5, 0}};
template <typename T>
constexpr TileCost kDzCosts[2] = {{kTileLarge, dz_shape<T>(kTileLarge), 0.95, 6.0, 0.52},
                                  {kTileSmall, dz_shape<T>(kTileSmall), 0.55, 7.0, 0.36}};
template <>
constexpr TileCost kDzCosts<float>[2] = {{kTileLarge, dz_shape<float>(kTileLarge), 3.90, 9.0, 2.10},
                                         {kTileSmall, dz_shape<float>(kTileSmall), 1.00, 4.0, 0.53}};

constexpr double kCopyUs = 0.8;  // of a 64 x 64 tile

// The tile whose product of rows x cols over `ktiles` is estimated to end
// first; `per`: right-hand rows a column.
template <int N>
const TileCost& best_tile(const TileCost (&costs)[N], int64_t rows, int64_t cols, int per, double ktiles) {
  int best = 0;
  double least = 1e300;
  for (int i = 0; i < N; ++i) {
    const TileShape& s = costs[i].shape;
    const double us = tile_product_us(costs[i], tiles_of(rows, s.m) * tiles_of(cols, s.n / per), ktiles);
    if (us < least) {
      least = us;
      best = i;
    }
  }
  return costs[best];
}

// Whether `copies` 64 x 64 tiles of copies go along with a product's tiles of
// so many us on `slots` places for a work-group: where the idle ones get
// through them in that time.  (A launch of its own moves them faster, eight
// work-groups a compute unit, but nothing else runs meanwhile.  Along,
// 1003 x 2048 x 1407 in fp16, without its second launch, takes 33.5 us forward instead of 42.0 and
// 128 x 2048 x 5461 91.4 us backward instead of 99.3; with copies counted at
// 0.3 us, where there are few idle places for many, 128 x 2048 x 5461 takes
// 53.3 us forward instead of 42.2.)
bool goes_along(int64_t copies, int64_t tiles, int64_t slots, double us) {
  return copies > 0 && tiles < slots && (double)copies * kCopyUs <= (double)(slots - tiles) * us;
}

// y's tile and splits: few rows against a long contraction leave most compute
// units without a tile.
struct MlpChoice {
  int tile = kTileSmall;
  TileShape shape{};
  int splits = 1;
  double us = 1e300;
};
template <typename T>
MlpChoice choose_down(int64_t n, int64_t d, double ktiles) {
  MlpChoice best;
  const EdgeCost* edges = edge_costs(sizeof(T));
  const TileCost costs[3] = {{kTileLarge, product_shape<T>(kTileLarge), edges[0].ktile, edges[0].fixed, 0},
                             {kTileSmall, product_shape<T>(kTileSmall), edges[1].ktile, edges[1].fixed, 0},
                             {kTileShort, product_shape<T>(kTileShort), 0.36, 1.5, 0}};
  for (const TileCost& c : costs) {
    if (c.tile == kTileShort && (sizeof(T) == 4 || n > c.shape.m)) continue;
    const int64_t tiles = tiles_of(n, c.shape.m) * tiles_of(d, c.shape.n);
    for (int s : kXentSplits) {
      if (s > 1 && ktiles / s < 3) break;
      // fp32 sums written and read, and a launch.
      const double sums = s > 1 ? (double)s * n * tiles_of(d, c.shape.n) * c.shape.n * 8.0 / 4.5e6 + 5.0 : 0.0;
      const double us = tile_product_us(c, tiles * s, ktiles / s) + sums;
      if (us < best.us) best = {c.tile, c.shape, s, us};
    }
  }
  return best;
}

template <typename T>
MlpChoice choose_gradients(int64_t n, int64_t d, int64_t f, double kw, double kx) {
  MlpChoice best;
  for (int i = 0; i < 2; ++i) {
    const EdgeCost& c = edge_costs(sizeof(T))[i];
    const int64_t e = c.edge, m = tiles_of(n, e), t = tiles_of(d, e), ft = tiles_of(f, e);
    for (int s : kXentSplits) {
      if (s > 1 && kx / s < 3) break;
      const double sums = s > 1 ? (double)s * n * t * e * 8.0 / 4.5e6 + 5.0 : 0.0;
      const double us = sums + grad_rounds(c, 3 * ft * t, kw, m * t * s, kx / s).us;
      if (us < best.us) best = {i == 0 ? kTileLarge : kTileSmall, {(int)e, (int)e}, s, us};
    }
  }
  return best;
}

// The same for what a call leaves out: workspaces are planned with both
// gradients.
template <typename T>
MlpPlan mlp_plan_of(int64_t n, int64_t d, int64_t f, bool ranged, bool aligned, bool backward, void* ws) {
  MlpPlan p;
  p.n = n;
  p.d = d;
  p.f = f;
  p.es = sizeof(T);
  p.bk = kRowBytes / p.es;
  p.dk = round_to(d, p.bk);
  p.fk = round_to(f, p.bk);
  p.stage_d = !aligned || p.dk != d;
  p.stage_f = !aligned || p.fk != f;
  auto take_choice = [&](const MlpChoice& best) {
    p.tile = best.tile;
    p.tm = best.shape.m;
    p.tn = best.shape.n;
    p.splits = best.splits;
  };
  Carver c{reinterpret_cast<char*>(ws)};
  if (n == 0) return p;
  if (!backward) {
    p.dot = n <= (p.stage_d || p.stage_f ? kMlpDotMostStaged : kMlpDotMost);
    p.h_rows = n;
    p.h_ld = p.fk;
    if (!p.dot) {
      const TileCost& up = best_tile(kUpCosts<T>, n, f, 2, (double)p.dk / p.bk);
      p.up_tile = up.tile;
      p.h_rows = round_to(n, up.shape.m);
      p.h_ld = skewed(round_to(f, up.shape.n / 2), p.bk);
      take_choice(choose_down<T>(n, d, (double)p.fk / p.bk));
      if (p.stage_d) {
        p.Xs = c.take<char>(n * p.dk * p.es);
        p.Gs = c.take<char>(f * p.dk * p.es);
        p.Us = c.take<char>(f * p.dk * p.es);
      }
      if (p.stage_f) {
        p.Ds = c.take<char>(d * p.fk * p.es);
        p.side = goes_along(tiles_of(d, 64) * tiles_of(p.fk, 64), tiles_of(n, up.shape.m) * tiles_of(f, up.shape.n / 2),
                            kXentGroups, (double)p.dk / p.bk * up.ktile + up.fixed);
      }
      if (p.splits > 1) p.parts = c.take<float>(p.splits * round_to(n, p.tm) * round_to(d, p.tn));
    }
    p.h = c.take<char>(p.h_rows * p.h_ld * (p.dot ? 4 : p.es));
    p.ranged = ranged && !p.dot;
  } else {
    const TileCost& dz = best_tile(kDzCosts<T>, n, f, 1, (double)p.dk / p.bk);
    p.dz_tile = dz.tile;
    p.n_pad = round_to(n, dz.shape.m);
    p.f_pad = round_to(f, dz.shape.n);
    p.d_pad = round_to(d, 64);
    p.t_ld = skewed(p.n_pad, p.bk);
    p.z_ld = skewed(2 * p.f_pad, p.bk);
    p.d_ld = skewed(p.d_pad, p.bk);
    take_choice(choose_gradients<T>(n, d, f, (double)p.n_pad / p.bk, 2.0 * p.f_pad / p.bk));
    const int64_t d64 = p.d_pad / 64, n64 = tiles_of(p.n_pad, 64), f64 = tiles_of(p.f_pad, 64);
    p.side = goes_along((p.stage_d ? 1 : 2) * n64 * d64 + 2 * f64 * d64, p.n_pad / dz.shape.m * (p.f_pad / dz.shape.n),
                        2 * kXentGroups, (double)p.dk / p.bk * dz.alone + dz.fixed);
    if (p.stage_d) p.Ys = c.take<char>(n * p.dk * p.es);
    p.dz = c.take<char>(p.n_pad * p.z_ld * p.es);
    p.dzt = c.take<char>(2 * p.f_pad * p.t_ld * p.es);
    p.ht = c.take<char>(p.f_pad * p.t_ld * p.es);
    p.WT = c.take<char>(p.d_pad * p.z_ld * p.es);
    p.DT = c.take<char>(p.f_pad * p.d_ld * p.es);
    p.XT = c.take<char>(p.d_pad * p.t_ld * p.es);
    p.YT = c.take<char>(p.d_pad * p.t_ld * p.es);
    if (p.splits > 1) p.parts = c.take<float>(p.splits * round_to(n, p.tm) * round_to(d, p.tn));
    p.ranged = ranged;
  }
  if (p.ranged) {
    p.range = reinterpret_cast<HeldRange*>(c.take<uint32_t>(kRangeWords + n));
    if (!backward) {
      p.seen.outside = c.take<uint32_t>(kXentGroups * (kThreads / 64));
      p.seen.parts = c.take<uint32_t>(2 * tiles_of(f, up_shape<T>(p.up_tile).n / 2) * n);
    }
  }
  p.total = c.used;
  return p;
}

MlpPlan mlp_plan(int64_t n, int64_t d, int64_t f, ns_dtype dtype, bool aligned, bool backward, void* ws) {
  // bf16 and fp16 have the same tiles.
  return dtype == NS_FP32 ? mlp_plan_of<float>(n, d, f, false, aligned, backward, ws)
                          : mlp_plan_of<_Float16>(n, d, f, dtype == NS_FP16, aligned, backward, ws);
}

// A call's launches as text (see ns_plan_gated_mlp); the length that it needs
// without the NUL.
int describe_mlp(const MlpPlan& p, ns_dtype dtype, bool backward, char* buf, size_t len) {
  const char* op = dtype == NS_FP32 ? "f32" : dtype == NS_FP16 ? "f16" : "bf16";
  if (p.n == 0) return backward ? snprintf(buf, len, "zero<%s>", op) : snprintf(buf, len, "%s", "");
  if (p.dot) {
    const int64_t v = 16 / p.es;
    auto form = [&](int64_t cols) { return cols % v == 0 ? "even" : cols > v ? "ragged" : "tiny"; };
    const int rows = xent_dot_rows(p.n);
    return snprintf(buf, len, "dotup<%s,%d,%s> dotdown<%s,%d,%s>", op, rows, form(p.d), op, rows, form(p.f));
  }
  char split[32] = "";
  if (p.splits > 1) snprintf(split, sizeof split, " join<%s> splits=%d", op, p.splits);
  char first[32] = "";
  if (backward || p.stage_d || (p.stage_f && !p.side)) snprintf(first, sizeof first, "prep<%s> ", op);
  const bool half = p.es == 2;
  const TileShape up = half ? up_shape<_Float16>(p.up_tile) : up_shape<float>(p.up_tile);
  const TileShape dz = half ? dz_shape<_Float16>(p.dz_tile) : dz_shape<float>(p.dz_tile);
  const char* name = backward ? "dz" : "up";
  const TileShape& shape = backward ? dz : up;
  char tile[16], again[32] = "";
  snprintf(tile, sizeof tile, "%dx%d", shape.m, shape.n / (backward ? 1 : 2));
  if (p.ranged) snprintf(again, sizeof again, "again<%s,%s> ", op, tile);
  return snprintf(buf, len, "%s%s<%s,%s%s> %sproducts<%s,%dx%d>%s", first, name, op, tile, p.side ? ",copies" : "", again, op,
                  (int)p.tm, (int)p.tn, split);
}

// The products' copies take 16-byte chunks, swizzled by bits 4 to 6 of the
// address within a row: rows a multiple of 128 bytes apart.
bool operand_aligned(const void* p, int64_t ld, ns_dtype dtype) {
  return aligned16(p) && ld * bytes_of(dtype) % kRowBytes == 0;
}

// One operand's copies: padded to cols_k columns, transposed into dst_t (ldt
// wide, rows_pad of them filled, cols_pad rows of it), either null.
XentCopyArgs mlp_copy(const void* src, int64_t ld, int64_t rows, int64_t cols, char* padded, int64_t cols_k, char* dst_t,
                      int64_t rows_pad, int64_t cols_pad, int64_t ldt) {
  XentCopyArgs a{};
  if (!padded && !dst_t) return a;
  a.src = src;
  a.ld = ld;
  a.rows = rows;
  a.cols = (int)cols;
  a.padded = padded;
  a.cols_k = (int)cols_k;
  a.transposed = dst_t;
  a.ldt = ldt;
  a.tiles_r = (int)(round_to(dst_t ? rows_pad : rows, 64) / 64);
  a.tiles_c = (int)(round_to(std::max(dst_t ? cols_pad : 0, padded ? cols_k : 0), 64) / 64);
  return a;
}

template <typename T>
ns_status mlp_prep(const MlpPrepArgs& a, hipStream_t st) {
  const int64_t blocks = a.blocks() + a.zero_blocks();
  if (blocks == 0) return NS_OK;
  if (blocks >= int64_t(1) << 24) return NS_ERR_INVALID_ARG;  // a launch may not have 2^32 threads
  hipLaunchKernelGGL((k_mlp_prep<T>), dim3((unsigned)blocks), dim3(256), 0, st, a);
  return launched();
}

template <typename T>
ns_status mlp_join(const MlpPlan& p, int64_t rows_pad, int64_t cols_pad, void* out, int64_t ldo, int32_t* d_status,
                   int32_t bits, hipStream_t st) {
  constexpr int64_t kOutCols = 64 * kVec<T>;
  hipLaunchKernelGGL((k_mlp_join<T>), dim3((unsigned)p.n, (unsigned)((p.d + kOutCols - 1) / kOutCols)), dim3(64), 0, st,
                     p.parts, p.splits, rows_pad, cols_pad, reinterpret_cast<T*>(out), ldo, (int)p.d, d_status, bits);
  return launched();
}

struct MlpIn {
  const void *X, *G, *U, *D;
  int64_t ldx, ldg, ldu, ldd;
};

template <typename T>
ns_status mlp_forward(const MlpPlan& p, const MlpIn& in, int act, void* Y, int64_t ldy, void* gate, void* up, int64_t lds,
                      bool save32, int32_t* d_status, hipStream_t st) {
  const int32_t bits = (int32_t)(NS_ERR_NONFINITE | NS_STATUS_AT_OUTPUT);
  constexpr int64_t es = sizeof(T);
  if (p.dot) {
    float* h = reinterpret_cast<float*>(p.h);
    const MlpDotUpArgs a{in.X, in.G, in.U, in.ldx, in.ldg, in.ldu, p.n, p.f, (int)p.d, h,
                         p.h_ld, gate, up, lds,    save32, act,    d_status, bits};
    if (launch_mlp_dot_up<T>(a, st) != hipSuccess) return NS_ERR_HIP;
    const MlpDotDownArgs b{h, in.D, p.h_ld, in.ldd, p.n, p.d, (int)p.f, Y, ldy, d_status, bits};
    return launch_mlp_dot_down<T>(b, st) == hipSuccess ? NS_OK : NS_ERR_HIP;
  }
  MlpPrepArgs prep{};
  prep.copy[0] = mlp_copy(in.X, in.ldx, p.n, p.d, p.Xs, p.dk, nullptr, 0, 0, 0);
  prep.copy[1] = mlp_copy(in.G, in.ldg, p.f, p.d, p.Gs, p.dk, nullptr, 0, 0, 0);
  prep.copy[2] = mlp_copy(in.U, in.ldu, p.f, p.d, p.Us, p.dk, nullptr, 0, 0, 0);
  MlpUpArgs a{};
  (p.side ? a.side : prep).copy[3] = mlp_copy(in.D, in.ldd, p.d, p.f, p.Ds, p.fk, nullptr, 0, 0, 0);
  ns_status s = mlp_prep<T>(prep, st);
  if (s != NS_OK) return s;
  a.X = p.stage_d ? p.Xs : in.X;
  a.G = p.stage_d ? p.Gs : in.G;
  a.U = p.stage_d ? p.Us : in.U;
  a.ldx = (p.stage_d ? p.dk : in.ldx) * es;
  a.ldw = (p.stage_d ? p.dk : in.ldg) * es;
  a.ktiles = (int)(p.dk / p.bk);
  a.n = p.n;
  a.f = p.f;
  const TileShape up_tile = up_shape<T>(p.up_tile);
  a.tiles_m = (int)(p.h_rows / up_tile.m);
  a.tiles_n = (int)tiles_of(p.f, up_tile.n / 2);
  a.h = p.h;
  a.ldh = p.h_ld;
  a.gate = gate;
  a.up = up;
  a.lds = lds;
  a.save32 = save32;
  a.act = act;
  a.d_status = d_status;
  a.status_bits = bits;
  a.range = p.range;
  a.seen = p.seen;
  if (launch_mlp_up<T>(a, p.up_tile, false, st) != hipSuccess) return NS_ERR_HIP;
  if (p.ranged) {
    // a and b are saved and the copies made.
    a.gate = a.up = nullptr;
    if (launch_mlp_up<T>(a, p.up_tile, true, st) != hipSuccess) return NS_ERR_HIP;
  }
  MlpGradArgs g{};
  const int64_t tm = tiles_of(p.n, p.tm), tn = tiles_of(p.d, p.tn);
  g.x = MlpProduct{p.h, p.stage_f ? p.Ds : in.D, (int)tm, (int)tn, p.n, p.d, Y, ldy, p.n, (int)p.d};
  g.x_ldl = p.h_ld * es;
  g.x_ldr = (p.stage_f ? p.fk : in.ldd) * es;
  g.x_ktiles = (int)(p.fk / p.bk);
  g.splits = p.splits;
  g.parts = p.parts;
  g.range = p.range;
  g.d_status = d_status;
  g.status_bits = bits;
  if (launch_mlp_products<T>(g, p.tile, st) != hipSuccess) return NS_ERR_HIP;
  return p.splits > 1 ? mlp_join<T>(p, tm * p.tm, tn * p.tn, Y, ldy, d_status, bits, st) : NS_OK;
}

struct MlpOut {
  void *dX, *dG, *dU, *dD;
  int64_t lddx, lddg, lddu, lddd;
};

template <typename T>
ns_status mlp_backward(const MlpPlan& p, const MlpIn& in, const void* dY, int64_t lddy, const void* gate, const void* up,
                       int64_t lds, bool save32, int act, const MlpOut& out, int32_t* d_status, hipStream_t st) {
  const int32_t bits = (int32_t)(NS_ERR_NONFINITE | NS_STATUS_AT_OUTPUT);
  constexpr int64_t es = sizeof(T);
  const bool dw = out.dG || out.dU || out.dD;
  MlpPrepArgs prep{};
  MlpDzArgs a{};
  MlpPrepArgs& side = p.side ? a.side : prep;
  (p.stage_d ? prep : side).copy[0] = mlp_copy(dY, lddy, p.n, p.d, p.Ys, p.dk, dw ? p.YT : nullptr, p.n_pad, p.d_pad, p.t_ld);
  prep.copy[1] = mlp_copy(in.D, in.ldd, p.d, p.f, nullptr, 0, p.DT, p.d_pad, p.f_pad, p.d_ld);
  if (dw) side.copy[2] = mlp_copy(in.X, in.ldx, p.n, p.d, nullptr, 0, p.XT, p.n_pad, p.d_pad, p.t_ld);
  if (out.dX) {
    side.copy[3] = mlp_copy(in.G, in.ldg, p.f, p.d, nullptr, 0, p.WT, p.f_pad, p.d_pad, p.z_ld);
    side.copy[4] = mlp_copy(in.U, in.ldu, p.f, p.d, nullptr, 0, p.WT + p.f_pad * es, p.f_pad, p.d_pad, p.z_ld);
  }
  if (p.ranged) {
    prep.zero = reinterpret_cast<uint32_t*>(p.range);
    prep.zeros = kRangeWords + p.n;
  }
  ns_status s = mlp_prep<T>(prep, st);
  if (s != NS_OK) return s;
  // The gradients' tiles are square.
  const int64_t tm = tiles_of(p.n, p.tm), td = tiles_of(p.d, p.tm), tf = tiles_of(p.f, p.tm);
  a.dY = p.stage_d ? p.Ys : dY;
  a.WT = p.DT;
  a.ldy = (p.stage_d ? p.dk : lddy) * es;
  a.ldw = p.d_ld * es;
  a.ktiles = (int)(p.dk / p.bk);
  a.n = p.n;
  a.f = p.f;
  a.tiles_m = (int)(p.n_pad / dz_shape<T>(p.dz_tile).m);
  a.tiles_n = (int)(p.f_pad / dz_shape<T>(p.dz_tile).n);
  a.gate = gate;
  a.up = up;
  a.lds = lds;
  a.save32 = save32;
  a.dz = p.dz;
  a.dzt = p.dzt;
  a.ht = p.ht;
  a.f_pad = p.f_pad;
  a.z_ld = p.z_ld;
  a.t_ld = p.t_ld;
  a.act = act;
  a.range = p.range;
  if (launch_mlp_dz<T>(a, p.dz_tile, false, st) != hipSuccess) return NS_ERR_HIP;
  if (p.ranged && launch_mlp_dz<T>(a, p.dz_tile, true, st) != hipSuccess) return NS_ERR_HIP;
  MlpGradArgs g{};
  int tiles = 0;
  if (out.dG) tiles += (int)(tf * td);
  g.w[0] = MlpProduct{p.dzt, p.XT, (int)tf, (int)td, p.f_pad, p.d_pad, out.dG, out.lddg, p.f, (int)p.d};
  g.w_tiles[0] = tiles;
  if (out.dU) tiles += (int)(tf * td);
  g.w[1] = MlpProduct{p.dzt + p.f_pad * p.t_ld * es, p.XT, (int)tf, (int)td, p.f_pad, p.d_pad, out.dU, out.lddu, p.f,
                      (int)p.d};
  g.w_tiles[1] = tiles;
  if (out.dD) tiles += (int)(tf * td);
  g.w[2] = MlpProduct{p.YT, p.ht, (int)td, (int)tf, p.d_pad, p.f_pad, out.dD, out.lddd, p.d, (int)p.f};
  g.w_tiles[2] = tiles;
  g.w_ld = p.t_ld * es;
  g.w_ktiles = (int)(p.n_pad / p.bk);
  g.splits = p.splits;
  g.range = p.range;
  if (out.dX) {
    g.x = MlpProduct{p.dz, p.WT, (int)tm, (int)td, p.n, p.d_pad, out.dX, out.lddx, p.n, (int)p.d};
    g.x_ldl = g.x_ldr = p.z_ld * es;
    g.x_ktiles = (int)(2 * p.f_pad / p.bk);
    g.parts = p.parts;
    const EdgeCost* costs = edge_costs(p.es);
    g.extra = grad_rounds(costs[p.tile == kTileLarge ? 0 : 1], tiles, (double)g.w_ktiles, tm * td * p.splits,
                          (double)g.x_ktiles / p.splits)
                  .extra;
  }
  g.d_status = d_status;
  g.status_bits = bits;
  if (launch_mlp_products<T>(g, p.tile, st) != hipSuccess) return NS_ERR_HIP;
  return out.dX && p.splits > 1 ? mlp_join<T>(p, tm * p.tm, td * p.tm, out.dX, out.lddx, d_status, bits, st) : NS_OK;
}

bool stride_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= kMaxMlpStride; }

}  // namespace

extern "C" {

size_t ns_gated_mlp_workspace_size(int64_t rows, int64_t cols, int64_t inner, ns_dtype dtype, int32_t aligned,
                                   int32_t backward) {
  if (!mlp_shape_ok(rows, cols, inner) || !known(dtype)) return 0;
  return std::max(kAlignTo, mlp_plan(rows, cols, inner, dtype, aligned != 0, backward != 0, nullptr).total);
}

int64_t ns_plan_gated_mlp(int64_t rows, int64_t cols, int64_t inner, ns_dtype dtype, int32_t aligned, int32_t backward,
                          char* buf, size_t len) {
  if (!mlp_shape_ok(rows, cols, inner) || !known(dtype)) return -1;
  const MlpPlan p = mlp_plan(rows, cols, inner, dtype, aligned != 0, backward != 0, nullptr);
  return describe_mlp(p, dtype, backward != 0, buf, buf ? len : 0) + 1;
}

ns_status ns_gated_mlp(const void* X, int64_t ldx, const void* Wg, int64_t ldwg, const void* Wu, int64_t ldwu,
                       const void* Wd, int64_t ldwd, int64_t rows, int64_t cols, int64_t inner, ns_dtype dtype,
                       ns_activation activation, void* Y, int64_t ldy, void* gate, void* up, int64_t ldg,
                       ns_dtype save_dtype, int32_t* d_status, void* workspace, size_t workspace_bytes, ns_stream_t stream) {
  if (!mlp_shape_ok(rows, cols, inner)) return NS_ERR_INVALID_ARG;
  if (!stride_ok(ldx, cols) || !stride_ok(ldwg, cols) || !stride_ok(ldwu, cols) || !stride_ok(ldwd, inner) ||
      !stride_ok(ldy, cols) || ((gate || up) && !stride_ok(ldg, inner)))
    return NS_ERR_INVALID_ARG;
  if (activation < NS_SILU || activation > NS_RELU) return NS_ERR_INVALID_ARG;
  if (!known(dtype) || !(save_dtype == dtype || save_dtype == NS_FP32)) return NS_ERR_UNSUPPORTED_DTYPE;
  if (rows == 0) return NS_OK;
  if (!X || !Wg || !Wu || !Wd || !Y || !gate != !up) return NS_ERR_INVALID_ARG;
  // An operand whose rows are no whole k-tiles is copied wherever it starts.
  const int64_t bk = kRowBytes / bytes_of(dtype);
  const bool aligned = (cols % bk || (operand_aligned(X, ldx, dtype) && operand_aligned(Wg, ldwg, dtype) &&
                                      operand_aligned(Wu, ldwu, dtype) && ldwg == ldwu)) &&
                       (inner % bk || operand_aligned(Wd, ldwd, dtype));
  const MlpPlan p = mlp_plan(rows, cols, inner, dtype, aligned, false, workspace);
  if (!workspace_ok(workspace, workspace_bytes, p.total)) return NS_ERR_WORKSPACE;
  if (gate && gate == up) return NS_ERR_INVALID_ARG;
  const MlpIn in{X, Wg, Wu, Wd, ldx, ldwg, ldwu, ldwd};
  return with_type(dtype, [&](auto io) {
    return mlp_forward<decltype(io)>(p, in, (int)activation, Y, ldy, gate, up, ldg,
                                     save_dtype == NS_FP32, d_status, reinterpret_cast<hipStream_t>(stream));
  });
}

ns_status ns_gated_mlp_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* Wg, int64_t ldwg,
                                const void* Wu, int64_t ldwu, const void* Wd, int64_t ldwd, const void* gate,
                                const void* up, int64_t ldg, ns_dtype save_dtype, int64_t rows, int64_t cols, int64_t inner, ns_dtype dtype,
                                ns_activation activation, void* dX, int64_t lddx, void* dWg, int64_t lddwg, void* dWu,
                                int64_t lddwu, void* dWd, int64_t lddwd, int32_t* d_status, void* workspace,
                                size_t workspace_bytes, ns_stream_t stream) {
  if (!mlp_shape_ok(rows, cols, inner)) return NS_ERR_INVALID_ARG;
  if (!stride_ok(lddy, cols) || !stride_ok(ldx, cols) || !stride_ok(ldwg, cols) || !stride_ok(ldwu, cols) ||
      !stride_ok(ldwd, inner) || !stride_ok(ldg, inner) || (dX && !stride_ok(lddx, cols)) ||
      (dWg && !stride_ok(lddwg, cols)) || (dWu && !stride_ok(lddwu, cols)) || (dWd && !stride_ok(lddwd, inner)))
    return NS_ERR_INVALID_ARG;
  if (activation < NS_SILU || activation > NS_RELU) return NS_ERR_INVALID_ARG;
  if (!known(dtype) || !(save_dtype == dtype || save_dtype == NS_FP32)) return NS_ERR_UNSUPPORTED_DTYPE;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (rows == 0) {
    return with_type(dtype, [&](auto io) {
      using T = decltype(io);
      const struct {
        void* out;
        int64_t ld, rows, cols;
      } zeros[] = {{dWg, lddwg, inner, cols}, {dWu, lddwu, inner, cols}, {dWd, lddwd, cols, inner}};
      for (const auto& z : zeros)
        if (z.out)
          hipLaunchKernelGGL((k_xent_zero<T>), dim3((unsigned)z.rows), dim3(256), 0, st, reinterpret_cast<T*>(z.out), z.ld,
                             (int)z.cols);
      return dWg || dWu || dWd ? launched() : NS_OK;
    });
  }
  if (!dY || !X || !Wg || !Wu || !Wd || !gate || !up) return NS_ERR_INVALID_ARG;
  const MlpPlan p = mlp_plan(rows, cols, inner, dtype, operand_aligned(dY, lddy, dtype), true, workspace);
  if (!workspace_ok(workspace, workspace_bytes, p.total)) return NS_ERR_WORKSPACE;
  if (!dX && !dWg && !dWu && !dWd) return NS_OK;
  const void* outs[] = {dX, dWg, dWu, dWd};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (outs[i] && outs[i] == outs[j]) return NS_ERR_INVALID_ARG;
  const MlpIn in{X, Wg, Wu, Wd, ldx, ldwg, ldwu, ldwd};
  const MlpOut out{dX, dWg, dWu, dWd, lddx, lddwg, lddwu, lddwd};
  return with_type(dtype, [&](auto io) {
    return mlp_backward<decltype(io)>(p, in, dY, lddy, gate, up, ldg, save_dtype == NS_FP32, (int)activation, out,
                                      d_status, st);
  });
}

}  // extern "C"
