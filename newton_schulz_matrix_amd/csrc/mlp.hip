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

// The projections' tiles: us per k-tile and fixed, as EdgeCost.
template <int ES> constexpr EdgeCost kUpLargeCost = ES == 2 ? EdgeCost{0, 0.82, 4.0} : EdgeCost{0, 2.10, 3.5};
template <int ES> constexpr EdgeCost kUpSmallCost = ES == 2 ? EdgeCost{0, 0.52, 3.0} : EdgeCost{0, 1.06, 2.5};

struct MlpPlan {
  int64_t n = 0, d = 0, f = 0;
  int es = 2, bk = 64;
  int64_t dk = 0, fk = 0;              // d and f in whole k-tiles
  bool stage_d = false, stage_f = false;  // operands of d or f columns need staging copies
  bool dot = false;
  // Forward.
  bool up_large = false;
  int64_t up_m = 0, up_cols = 0;       // tile of the projections: rows and columns of h
  int64_t h_rows = 0, h_ld = 0;
  // y forward, dz and the gradients backward.
  int64_t edge = 0;
  int splits = 1;
  int64_t n_pad = 0, d_pad = 0, f_pad = 0, dt = 0;  // backward; dt: row stride of Wd^T
  // Buffers.
  char *Xs = nullptr, *Gs = nullptr, *Us = nullptr, *Ds = nullptr, *h = nullptr;
  char *Ys = nullptr, *dz = nullptr, *dzt = nullptr, *ht = nullptr, *WT = nullptr, *DT = nullptr, *XT = nullptr,
       *YT = nullptr;
  float* parts = nullptr;
  size_t total = 0;
};

bool mlp_shape_ok(int64_t n, int64_t d, int64_t f) {
  return n >= 0 && n <= kMaxMlpRows && d >= 1 && d <= kMaxMlpCols && f >= 1 && f <= kMaxMlpCols &&
         n <= kMaxMlpInner / f;
}

// y's edge and splits: few rows against a long contraction leave most compute
// units without a tile.
struct MlpChoice {
  int64_t edge = 0;
  int splits = 1;
  double us = 1e300;
};
MlpChoice choose_down(const EdgeCost& c, int64_t n, int64_t d, int64_t ktiles) {
  MlpChoice best;
  const int64_t m = (n + c.edge - 1) / c.edge, t = (d + c.edge - 1) / c.edge;
  for (int s : kXentSplits) {
    if (s > 1 && ktiles / s < 3) break;
    // fp32 sums written and read, and a launch.
    const double sums = s > 1 ? (double)s * m * t * c.edge * c.edge * 8.0 / 4.5e6 + 5.0 : 0.0;
    const double us = product_us(c, m * t * s, (double)ktiles / s) + sums;
    if (us < best.us) best = {c.edge, s, us};
  }
  return best;
}

MlpChoice choose_gradients(const EdgeCost& c, int64_t n, int64_t d, int64_t f, int64_t dk, int bk, bool dx, bool dw) {
  const int64_t e = c.edge, m = (n + e - 1) / e, t = (d + e - 1) / e, ft = (f + e - 1) / e;
  const double dz = product_us(c, m * ft, (double)dk / bk);
  const double kw = (double)m * e / bk, kx = 2.0 * ft * e / bk;
  MlpChoice best;
  for (int s : kXentSplits) {
    if (s > 1 && (!dx || kx / s < 3)) break;
    const double sums = s > 1 ? (double)s * m * t * e * e * 8.0 / 4.5e6 + 5.0 : 0.0;
    const double us = dz + sums + grad_rounds(c, dw ? 3 * ft * t : 0, kw, dx ? m * t * s : 0, kx / s).us;
    if (us < best.us) best = {e, s, us};
  }
  return best;
}

// The same for what a call leaves out: workspaces are planned with both
// gradients.
MlpPlan mlp_plan(int64_t n, int64_t d, int64_t f, ns_dtype dtype, bool aligned, bool backward, void* ws) {
  MlpPlan p;
  p.n = n;
  p.d = d;
  p.f = f;
  p.es = bytes_of(dtype);
  p.bk = kRowBytes / p.es;
  p.dk = round_to(d, p.bk);
  p.fk = round_to(f, p.bk);
  p.stage_d = !aligned || p.dk != d;
  p.stage_f = !aligned || p.fk != f;
  const EdgeCost* costs = edge_costs(p.es);
  Carver c{reinterpret_cast<char*>(ws)};
  if (n == 0) return p;
  if (!backward) {
    p.dot = n <= (p.stage_d || p.stage_f ? kMlpDotMostStaged : kMlpDotMost);
    p.h_rows = n;
    p.h_ld = p.fk;
    if (!p.dot) {
      auto us = [&](const EdgeCost& x, int64_t tm, int64_t cols) {
        return product_us(x, ((n + tm - 1) / tm) * ((f + cols - 1) / cols), (double)p.dk / p.bk);
      };
      const bool half = p.es == 2;
      const int64_t lm = half ? kUpLargeM<__bf16> : kUpLargeM<float>, lc = (half ? kUpLargeN<__bf16> : kUpLargeN<float>) / 2;
      const int64_t sm = half ? kUpSmallM<__bf16> : kUpSmallM<float>, sc = (half ? kUpSmallN<__bf16> : kUpSmallN<float>) / 2;
      p.up_large = us(half ? kUpLargeCost<2> : kUpLargeCost<4>, lm, lc) <= us(half ? kUpSmallCost<2> : kUpSmallCost<4>, sm, sc);
      p.up_m = p.up_large ? lm : sm;
      p.up_cols = p.up_large ? lc : sc;
      p.h_rows = round_to(n, p.up_m);
      p.h_ld = round_to(f, p.up_cols);
      const MlpChoice large = choose_down(costs[0], n, d, p.fk / p.bk), small = choose_down(costs[1], n, d, p.fk / p.bk);
      const MlpChoice& best = large.us <= small.us ? large : small;
      p.edge = best.edge;
      p.splits = best.splits;
      if (p.stage_d) {
        p.Xs = c.take<char>(n * p.dk * p.es);
        p.Gs = c.take<char>(f * p.dk * p.es);
        p.Us = c.take<char>(f * p.dk * p.es);
      }
      if (p.stage_f) p.Ds = c.take<char>(d * p.fk * p.es);
      if (p.splits > 1) p.parts = c.take<float>(p.splits * round_to(n, p.edge) * round_to(d, p.edge));
    }
    p.h = c.take<char>(p.h_rows * p.h_ld * p.es);
  } else {
    const MlpChoice large = choose_gradients(costs[0], n, d, f, p.dk, p.bk, true, true);
    const MlpChoice small = choose_gradients(costs[1], n, d, f, p.dk, p.bk, true, true);
    const MlpChoice& best = large.us <= small.us ? large : small;
    p.edge = best.edge;
    p.splits = best.splits;
    p.n_pad = round_to(n, p.edge);
    p.d_pad = round_to(d, p.edge);
    p.f_pad = round_to(f, p.edge);
    p.dt = round_to(d, 64);
    if (p.stage_d) p.Ys = c.take<char>(n * p.dk * p.es);
    p.dz = c.take<char>(2 * p.n_pad * p.f_pad * p.es);
    p.dzt = c.take<char>(2 * p.n_pad * p.f_pad * p.es);
    p.ht = c.take<char>(p.n_pad * p.f_pad * p.es);
    p.WT = c.take<char>(2 * p.d_pad * p.f_pad * p.es);
    p.DT = c.take<char>(p.f_pad * p.dt * p.es);
    p.XT = c.take<char>(p.d_pad * p.n_pad * p.es);
    p.YT = c.take<char>(p.d_pad * p.n_pad * p.es);
    if (p.splits > 1) p.parts = c.take<float>(p.splits * p.n_pad * p.d_pad);
  }
  p.total = c.used;
  return p;
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
  const char* prep = backward || p.stage_d || p.stage_f ? "prep" : "";
  char first[32] = "";
  if (*prep) snprintf(first, sizeof first, "prep<%s> ", op);
  if (!backward)
    return snprintf(buf, len, "%sup<%s,%dx%d> products<%s,%d>%s", first, op, (int)p.up_m, (int)p.up_cols, op, (int)p.edge,
                    split);
  return snprintf(buf, len, "%sdz<%s,%d> products<%s,%d>%s", first, op, (int)p.edge, op, (int)p.edge, split);
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
  int64_t blocks = 0;
  for (const XentCopyArgs& c : a.copy) blocks += c.blocks();
  if (blocks == 0) return NS_OK;
  if (blocks >= int64_t(1) << 31) return NS_ERR_INVALID_ARG;
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
    const MlpDotUpArgs a{in.X, in.G, in.U, in.ldx, in.ldg, in.ldu, p.n,      p.f, (int)p.d, p.h,
                         p.h_ld, gate, up, lds,    save32, act,    d_status, bits};
    if (launch_mlp_dot_up<T>(a, st) != hipSuccess) return NS_ERR_HIP;
    const MlpDotDownArgs b{p.h, in.D, p.h_ld, in.ldd, p.n, p.d, (int)p.f, Y, ldy, d_status, bits};
    return launch_mlp_dot_down<T>(b, st) == hipSuccess ? NS_OK : NS_ERR_HIP;
  }
  MlpPrepArgs prep{};
  prep.copy[0] = mlp_copy(in.X, in.ldx, p.n, p.d, p.Xs, p.dk, nullptr, 0, 0, 0);
  prep.copy[1] = mlp_copy(in.G, in.ldg, p.f, p.d, p.Gs, p.dk, nullptr, 0, 0, 0);
  prep.copy[2] = mlp_copy(in.U, in.ldu, p.f, p.d, p.Us, p.dk, nullptr, 0, 0, 0);
  prep.copy[3] = mlp_copy(in.D, in.ldd, p.d, p.f, p.Ds, p.fk, nullptr, 0, 0, 0);
  ns_status s = mlp_prep<T>(prep, st);
  if (s != NS_OK) return s;
  MlpUpArgs a{};
  a.X = p.stage_d ? p.Xs : in.X;
  a.G = p.stage_d ? p.Gs : in.G;
  a.U = p.stage_d ? p.Us : in.U;
  a.ldx = (p.stage_d ? p.dk : in.ldx) * es;
  a.ldw = (p.stage_d ? p.dk : in.ldg) * es;
  a.ktiles = (int)(p.dk / p.bk);
  a.n = p.n;
  a.f = p.f;
  a.tiles_m = (int)(p.h_rows / p.up_m);
  a.tiles_n = (int)(p.h_ld / p.up_cols);
  a.h = p.h;
  a.ldh = p.h_ld;
  a.gate = gate;
  a.up = up;
  a.lds = lds;
  a.save32 = save32;
  a.act = act;
  a.d_status = d_status;
  a.status_bits = bits;
  if (launch_mlp_up<T>(a, p.up_large, st) != hipSuccess) return NS_ERR_HIP;
  MlpGradArgs g{};
  const int64_t tm = (p.n + p.edge - 1) / p.edge, tn = (p.d + p.edge - 1) / p.edge;
  g.x = MlpProduct{p.h, p.stage_f ? p.Ds : in.D, (int)tm, (int)tn, p.n, p.d, Y, ldy, p.n, (int)p.d};
  g.x_ldl = p.h_ld * es;
  g.x_ldr = (p.stage_f ? p.fk : in.ldd) * es;
  g.x_ktiles = (int)(p.fk / p.bk);
  g.splits = p.splits;
  g.parts = p.parts;
  g.d_status = d_status;
  g.status_bits = bits;
  if (launch_mlp_products<T>(g, (int)p.edge, st) != hipSuccess) return NS_ERR_HIP;
  return p.splits > 1 ? mlp_join<T>(p, tm * p.edge, tn * p.edge, Y, ldy, d_status, bits, st) : NS_OK;
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
  prep.copy[0] = mlp_copy(dY, lddy, p.n, p.d, p.Ys, p.dk, dw ? p.YT : nullptr, p.n_pad, p.d_pad, p.n_pad);
  prep.copy[1] = mlp_copy(in.D, in.ldd, p.d, p.f, nullptr, 0, p.DT, p.dt, p.f_pad, p.dt);
  if (dw) prep.copy[2] = mlp_copy(in.X, in.ldx, p.n, p.d, nullptr, 0, p.XT, p.n_pad, p.d_pad, p.n_pad);
  if (out.dX) {
    prep.copy[3] = mlp_copy(in.G, in.ldg, p.f, p.d, nullptr, 0, p.WT, p.f_pad, p.d_pad, 2 * p.f_pad);
    prep.copy[4] = mlp_copy(in.U, in.ldu, p.f, p.d, nullptr, 0, p.WT + p.f_pad * es, p.f_pad, p.d_pad, 2 * p.f_pad);
  }
  ns_status s = mlp_prep<T>(prep, st);
  if (s != NS_OK) return s;
  const int64_t tm = p.n_pad / p.edge, td = p.d_pad / p.edge, tf = p.f_pad / p.edge;
  MlpDzArgs a{};
  a.dY = p.stage_d ? p.Ys : dY;
  a.WT = p.DT;
  a.ldy = (p.stage_d ? p.dk : lddy) * es;
  a.ldw = p.dt * es;
  a.ktiles = (int)(p.dk / p.bk);
  a.n = p.n;
  a.f = p.f;
  a.tiles_m = (int)tm;
  a.tiles_n = (int)tf;
  a.gate = gate;
  a.up = up;
  a.lds = lds;
  a.save32 = save32;
  a.dz = p.dz;
  a.dzt = p.dzt;
  a.ht = p.ht;
  a.n_pad = p.n_pad;
  a.f_pad = p.f_pad;
  a.act = act;
  if (launch_mlp_dz<T>(a, (int)p.edge, st) != hipSuccess) return NS_ERR_HIP;
  MlpGradArgs g{};
  int tiles = 0;
  if (out.dG) tiles += (int)(tf * td);
  g.w[0] = MlpProduct{p.dzt, p.XT, (int)tf, (int)td, p.f_pad, p.d_pad, out.dG, out.lddg, p.f, (int)p.d};
  g.w_tiles[0] = tiles;
  if (out.dU) tiles += (int)(tf * td);
  g.w[1] = MlpProduct{p.dzt + p.f_pad * p.n_pad * es, p.XT, (int)tf, (int)td, p.f_pad, p.d_pad, out.dU, out.lddu, p.f,
                      (int)p.d};
  g.w_tiles[1] = tiles;
  if (out.dD) tiles += (int)(tf * td);
  g.w[2] = MlpProduct{p.YT, p.ht, (int)td, (int)tf, p.d_pad, p.f_pad, out.dD, out.lddd, p.d, (int)p.f};
  g.w_tiles[2] = tiles;
  g.w_ld = p.n_pad * es;
  g.w_ktiles = (int)(p.n_pad / p.bk);
  g.splits = p.splits;
  if (out.dX) {
    g.x = MlpProduct{p.dz, p.WT, (int)tm, (int)td, p.n, p.d_pad, out.dX, out.lddx, p.n, (int)p.d};
    g.x_ldl = g.x_ldr = 2 * p.f_pad * es;
    g.x_ktiles = (int)(2 * p.f_pad / p.bk);
    g.parts = p.parts;
    const EdgeCost* costs = edge_costs(p.es);
    g.extra = grad_rounds(costs[p.edge == costs[0].edge ? 0 : 1], tiles, (double)g.w_ktiles, tm * td * p.splits,
                          (double)g.x_ktiles / p.splits)
                  .extra;
  }
  g.d_status = d_status;
  g.status_bits = bits;
  if (launch_mlp_products<T>(g, (int)p.edge, st) != hipSuccess) return NS_ERR_HIP;
  return out.dX && p.splits > 1 ? mlp_join<T>(p, p.n_pad, p.d_pad, out.dX, out.lddx, d_status, bits, st) : NS_OK;
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
  const bool aligned = operand_aligned(X, ldx, dtype) && operand_aligned(Wg, ldwg, dtype) &&
                       operand_aligned(Wu, ldwu, dtype) && operand_aligned(Wd, ldwd, dtype) && ldwg == ldwu;
  const MlpPlan p = mlp_plan(rows, cols, inner, dtype, aligned, false, workspace);
  if (!workspace_ok(workspace, workspace_bytes, p.total)) return NS_ERR_WORKSPACE;
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
  const MlpIn in{X, Wg, Wu, Wd, ldx, ldwg, ldwu, ldwd};
  const MlpOut out{dX, dWg, dWu, dWd, lddx, lddwg, lddwu, lddwd};
  return with_type(dtype, [&](auto io) {
    return mlp_backward<decltype(io)>(p, in, dY, lddy, gate, up, ldg, save_dtype == NS_FP32, (int)activation, out,
                                      d_status, st);
  });
}

}  // extern "C"
