// train.hip - C entry points of the operators at the two ends of a training
// step, beside the Muon step of the hidden matrices: embedding lookup and
// its gradient, layer norm forward and backward, and the output projection's
// softmax cross entropy with its gradients.  Argument checks, workspace
// layout and kernel choice; the kernels are in norm.hpp, embed.hpp and
// xent.hpp.
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <type_traits>

#include "../../include/nsortho.h"
#include "embed.hpp"
#include "norm.hpp"
#include "xent.hpp"

namespace {

using namespace nsk;
using namespace nsr;

constexpr size_t kAlignTo = 256;
inline size_t align_up_to(size_t x) { return (x + kAlignTo - 1) / kAlignTo * kAlignTo; }
inline int64_t round_to(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline bool known(ns_dtype d) { return d == NS_BF16 || d == NS_FP16 || d == NS_FP32; }
inline int bytes_of(ns_dtype d) { return d == NS_FP32 ? 4 : 2; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline ns_status launched() { return hipGetLastError() == hipSuccess ? NS_OK : NS_ERR_HIP; }
// Grids of the kernels that loop over their rows stay below this many blocks
// (a launch may not have 2^32 threads).
constexpr int64_t kMaxBlocks = 1 << 20;

// Buffers carved out of a workspace in order.
struct Carver {
  char* base;
  size_t used = 0;
  template <typename T>
  T* take(int64_t count) {
    char* p = base ? base + used : nullptr;
    used += align_up_to((size_t)count * sizeof(T));
    return reinterpret_cast<T*>(p);
  }
};

bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && have >= need && reinterpret_cast<uintptr_t>(ws) % kAlignTo == 0);
}

// Calls f(IO{}, PT{}) for a data type and a parameter type that is the same
// or fp32.
template <class F>
ns_status with_types(ns_dtype io, ns_dtype pt, F&& f) {
  if (io == NS_FP32) return f(float{}, float{});
  if (io == NS_BF16) return pt == NS_FP32 ? f(__bf16{}, float{}) : f(__bf16{}, __bf16{});
  return pt == NS_FP32 ? f(_Float16{}, float{}) : f(_Float16{}, _Float16{});
}
template <class F>
ns_status with_type(ns_dtype io, F&& f) {
  if (io == NS_FP32) return f(float{});
  if (io == NS_BF16) return f(__bf16{});
  return f(_Float16{});
}

// ---------------------------------------------------------------------------
// Layer norm.
// ---------------------------------------------------------------------------
constexpr int64_t kMaxNormCols = 1 << 24;
constexpr int kNormRegisterCols = 16384;  // the widest row that the kernels hold in registers
// Threads of the forward pass: as many as the chip holds at 64 registers
// each.  Blocks walk the rows beyond that.
constexpr int64_t kNormFwdThreads = 256 * 2048;
// Blocks of the backward pass, each of which leaves one partial row of dw
// and db.
constexpr int64_t kNormParts = 512;

// Calls f.template run<NV, TPR, FORM>() for a row width: as few threads per row as
// hold it in NV vectors each, so that a block works on many narrow rows and a
// row's sums stay within a wave up to 256 vectors (2048 16-bit columns).
// More vectors per thread would not leave registers for the backward's sums.
template <typename IO, int FORM, class F>
void norm_form(int64_t cols, F&& f) {
  const int64_t n = (cols + kVec<IO> - 1) / kVec<IO>;
  if (n <= 32) return f.template run<1, 32, FORM>();
  if (n <= 64) return f.template run<2, 32, FORM>();
  if (n <= 96) return f.template run<3, 32, FORM>();
  if (n <= 128) return f.template run<4, 32, FORM>();
  if (n <= 192) return f.template run<3, 64, FORM>();
  if (n <= 256) return f.template run<4, 64, FORM>();
  if (n <= 512) return f.template run<2, 256, FORM>();
  if (n <= 1024) return f.template run<4, 256, FORM>();
  if constexpr (sizeof(IO) == 4) {
    if (n > 2048) return f.template run<4, 1024, FORM>();
  }
  return f.template run<2, 1024, FORM>();
}
template <typename IO, class F>
void with_norm_form(int64_t cols, F&& f) {
  if (cols % kVec<IO> == 0)
    norm_form<IO, kEven>(cols, f);
  else
    norm_form<IO, kRagged>(cols, f);
}
// Rows of less than a vector or too long for registers take the kernels that
// go element by element.
template <typename IO>
bool norm_by_element(int64_t cols) {
  return cols < kVec<IO> || cols > kNormRegisterCols;
}

template <typename IO>
int norm_rows_per_block(int64_t cols) {
  const int64_t n = (cols + kVec<IO> - 1) / kVec<IO>;
  return n <= 128 ? kNormRows<32> : n <= 256 ? kNormRows<64> : 1;
}

template <typename IO, typename PT>
struct NormFwdRun {
  const NormFwdArgs& a;
  hipStream_t st;
  template <int NV, int TPR, int FORM>
  void run() const {
    const int64_t groups = (a.rows + kNormRows<TPR> - 1) / kNormRows<TPR>;
    const int64_t blocks = std::min<int64_t>(groups, kNormFwdThreads / kNormThreads<TPR>);
    hipLaunchKernelGGL((k_norm_fwd<IO, PT, NV, TPR, FORM>), dim3((unsigned)blocks), dim3(kNormThreads<TPR>), 0, st, a);
  }
};

template <typename IO, typename PT>
struct NormBwdRun {
  const NormBwdArgs& a;
  int64_t parts;
  hipStream_t st;
  template <int NV, int TPR, int FORM>
  void run() const {
    hipLaunchKernelGGL((k_norm_bwd<IO, PT, NV, TPR, FORM>), dim3((unsigned)parts), dim3(kNormThreads<TPR>), 0, st, a);
  }
};

// Partial rows of dw and db: one per block of the backward pass.
int64_t norm_parts(int64_t rows, int per_block) { return std::min((rows + per_block - 1) / per_block, kNormParts); }

bool norm_shape_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && rows < (int64_t(1) << 31) && cols >= 1 && cols <= kMaxNormCols;
}

// ---------------------------------------------------------------------------
// Embedding.
// ---------------------------------------------------------------------------
constexpr int64_t kMaxEmbedRows = int64_t(1) << 28;
constexpr int64_t kMaxEmbedCols = 1 << 23;
constexpr int64_t kMaxEmbedIds = int64_t(1) << 30;
// The gradient's sort reads all ids once per 512 table rows: at most about
// 2^40 bytes from L2, a fraction of a second.
constexpr int64_t kMaxEmbedSort = int64_t(1) << 46;

bool embed_shape_ok(int64_t n, int64_t vocab, int64_t cols) {
  return n >= 0 && n <= kMaxEmbedIds && vocab >= 1 && vocab <= kMaxEmbedRows && cols >= 1 && cols <= kMaxEmbedCols;
}

bool embed_grad_shape_ok(int64_t n, int64_t vocab, int64_t cols) {
  return embed_shape_ok(n, vocab, cols) && n <= kMaxEmbedSort / vocab;
}

// Ids per sorting block: about a block per compute unit (every block reads
// all ids, so fewer blocks read less), and at most the counters that fit.
int embed_ids_per_block(int64_t vocab) {
  int r = 64;
  while (r < kSortMaxIds && (int64_t)r * 256 < vocab) r *= 2;
  return r;
}

// Positions per chunk.  A wave adds up `chunk` rows, and the longest list,
// some twentieth of a text's positions, joins n / (20 chunk) pieces with four
// times as many in flight: balanced at chunk = sqrt(n / 160).
int embed_chunk(int64_t n) {
  int c = 8;
  while ((int64_t)c * c * 160 < n) c *= 2;
  return c;
}

struct EmbedPlan {
  int32_t *order, *key, *start;
  float* partial;
  int chunk, chunks;
  int64_t cols_pad;
  size_t total;
};

// Columns that one wave covers: one, two or four vectors per lane.
int64_t embed_slice(int64_t cols, int es) {
  const int64_t wave = 64 * 16 / es;
  return wave * (cols <= wave ? 1 : cols <= 2 * wave ? 2 : 4);
}

EmbedPlan embed_plan(int64_t n, int64_t vocab, int64_t cols, void* ws, int es) {
  EmbedPlan p;
  Carver c{reinterpret_cast<char*>(ws)};
  p.chunk = embed_chunk(n);
  p.chunks = (int)((n + p.chunk - 1) / p.chunk);
  p.order = c.take<int32_t>(n);
  p.key = c.take<int32_t>(n);
  p.start = c.take<int32_t>(vocab + 1);
  p.cols_pad = round_to(cols, embed_slice(cols, es));
  p.partial = c.take<float>(2 * p.chunks * p.cols_pad);
  p.total = c.used;
  return p;
}

// Calls f(std::integral_constant<int, FORM>{}) for a row width.
template <typename IO, class F>
void with_row_form(int64_t cols, F&& f) {
  if (cols % kVec<IO> == 0) return f(std::integral_constant<int, kEven>{});
  if (cols > kVec<IO>) return f(std::integral_constant<int, kRagged>{});
  return f(std::integral_constant<int, kTiny>{});
}

template <typename IO, int U, int B, int FORM>
void embed_sum(const EmbedSumArgs& a, hipStream_t st) {
  const unsigned slices = (unsigned)(a.cols_pad / (64 * kVec<IO> * U));
  const int64_t zeros = a.accumulate ? 0 : (a.vocab + kZeroRows - 1) / kZeroRows;
  if (a.chunks + zeros > 0)
    hipLaunchKernelGGL((k_embed_sum<IO, U, B, FORM>), dim3((unsigned)(a.chunks + zeros), slices), dim3(64), 0, st, a);
  if (a.chunks > 1)
    hipLaunchKernelGGL((k_embed_join<IO, FORM>), dim3((unsigned)a.chunks, slices * U), dim3(64), 0, st, a);
}

// ---------------------------------------------------------------------------
// Cross entropy.
// ---------------------------------------------------------------------------
constexpr int64_t kMaxXentRows = 1 << 23, kMaxXentVocab = 1 << 23, kMaxXentCols = 1 << 20;
// Elements of one piece of dz at most (16-bit: 512 MiB in each orientation).
constexpr int64_t kXentPieceElems = int64_t(1) << 28;
// Logits of one call at most: tiles are counted in 32 bits.
constexpr int64_t kMaxXentLogits = int64_t(1) << 42;
// Forward: up to kXentDotRows rows go without tiles (128000 x 4096 bf16: one
// row 202 us against 226 with tiles, eight 279 against 231), up to
// kXentDotRowsStaged where tiles would need staging copies of the operands,
// which cost more than the product; both were measured there only and serve
// every type and size.  Up to kXentFewRows take the short, wide tiles
// (16-bit).  Up to kXentJoinRows rows are joined by a block each.
constexpr int64_t kXentDotRows = 4, kXentDotRowsStaged = 8, kXentFewRows = kXentFewM, kXentJoinRows = 1024;
constexpr int64_t kXentDotWaves = 4096;  // sixteen per compute unit

// Estimated time of a product in us: rounds of tiles over the compute units,
// each of so many us per k-tile and a fixed part, as measured on MI355X with
// random operands.
// (Two or three of the smallest float tiles on a compute unit, with stages of
// 16 KB, gained 5 to 10 % where tiles filled them evenly and lost up to 30 %
// where they did not: 300 x 1000 x 8191 took 76 and 56 us against 59.)
struct EdgeCost {
  int edge;
  double ktile, fixed;
};
constexpr EdgeCost kXentCost16[2] = {{kXentLarge<_Float16>, 0.90, 3.0}, {kXentSmall<_Float16>, 0.52, 2.0}};
constexpr EdgeCost kXentCost32[2] = {{kXentLarge<float>, 2.10, 2.5}, {kXentSmall<float>, 0.53, 1.5}};
// k-tiles go in groups of three (stream.hpp).
double tile_us(const EdgeCost& c, double ktiles) { return ceil(ktiles / 3) * 3 * c.ktile + c.fixed; }
double product_us(const EdgeCost& c, int64_t tiles, double ktiles) {
  return (double)((tiles + kXentGroups - 1) / kXentGroups) * tile_us(c, ktiles);
}
const EdgeCost* edge_costs(int es) { return es == 2 ? kXentCost16 : kXentCost32; }

// The gradients' two products in one launch: dW's tiles go round the
// work-groups, so that some have one more than the others; those others take
// part in `extra` rounds of dH's tiles before all do.  The number of rounds
// that ends first.
struct GradRounds {
  int extra = 0;
  double us = 1e300;
};
GradRounds grad_rounds(const EdgeCost& c, int64_t dw_tiles, double dw_ktiles, int64_t dh_tiles, double dh_ktiles) {
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(kXentGroups, dw_tiles + dh_tiles));
  const int64_t busy = dw_tiles % grid, idle = grid - busy;
  const double one_w = tile_us(c, dw_ktiles), one_h = tile_us(c, dh_ktiles);
  const double before = (double)(dw_tiles / grid) * one_w;
  GradRounds best;
  for (int64_t e = 0; e == 0 || (busy && e <= one_w / one_h + 1 && (e - 1) * idle < dh_tiles); ++e) {
    if (before + e * one_h >= best.us) break;
    const int64_t left = std::max<int64_t>(0, dh_tiles - e * idle), r = (left + grid - 1) / grid;
    const double us = before + std::max(busy ? one_w + r * one_h : 0, (e + r) * one_h);
    if (us < best.us) best = {(int)e, us};
  }
  return best;
}

struct XentPlan {
  int64_t n = 0, d = 0, v = 0;
  int es = 2, bk = 64;
  int64_t k = 0;                   // d in whole k-tiles
  bool stage = false;              // H and W need staging copies
  int64_t n_pad = 0, tiles_m = 0;  // rows of the first product
  int64_t tm = 0, tn = 0;
  int64_t tiles_n = 0;             // forward: vocabulary tiles
  int64_t groups = 0, waves = 0;   // forward without tiles
  int64_t d_pad = 0, piece = 0;    // backward
  int splits = 1;
  // Buffers.
  int32_t* tgt = nullptr;
  char *Hs = nullptr, *Ws = nullptr;
  float2* parts = nullptr;
  float *zt = nullptr, *coef = nullptr, *lse = nullptr, *gmax = nullptr, *gmax_parts = nullptr,
        *acc = nullptr;
  char *dz = nullptr, *dzt = nullptr, *WT = nullptr, *HT = nullptr;
  size_t total = 0;
};

bool xent_shape_ok(int64_t n, int64_t d, int64_t v) {
  return n >= 0 && n <= kMaxXentRows && d >= 1 && d <= kMaxXentCols && v >= 1 && v <= kMaxXentVocab &&
         n <= kMaxXentLogits / v;
}

// The backward pass's piece of the vocabulary (in tiles) and dH's splits for
// one tile edge, and their estimated time.  Between the largest piece that is
// allowed and a sixteenth of it, the one whose products leave the fewest compute units idle in their last rounds; fewer, larger pieces touch
// dH's fp32 sums less often.
struct BackwardChoice {
  int64_t piece_tiles = 1;
  int splits = 1;
  double us = 1e300;
};
// dH's splits to choose from: few rows leave most compute units without a
// tile of dH (35 x 434 x 84115: 4 tiles of 1315 k-tiles, 140 us with 8 splits).
constexpr int kXentSplits[] = {1, 2, 3, 4, 5, 6, 7, 8, 12, 16, 24, 32, 48, 64};
BackwardChoice choose_backward(const EdgeCost& c, int64_t n, int64_t d, int64_t v, int64_t k, int bk) {
  const int64_t e = c.edge, m = std::max<int64_t>(1, (n + e - 1) / e), dt = (d + e - 1) / e, vt = (v + e - 1) / e;
  const int64_t most = std::max<int64_t>(1, std::min(vt, kXentPieceElems / (m * e * e)));
  const int64_t fewest = (vt + most - 1) / most;
  BackwardChoice best;
  for (int64_t pieces = fewest; pieces < fewest + 16 && pieces <= vt; ++pieces) {
    const int64_t q = (vt + pieces - 1) / pieces, count = (vt + q - 1) / q, rest = vt - (count - 1) * q;
    auto logits = [&](int64_t tiles) { return product_us(c, m * tiles, (double)k / bk) + 12.0; };
    const double base = (double)(count - 1) * logits(q) + logits(rest);
    for (int s : kXentSplits) {
      // Every split of every piece has its k-tiles (three at least).
      if (s > 1 && rest * e / bk / s < 3) break;
      const double sums = (double)s * m * dt * e * e * 8.0 / 4.5e6;  // fp32 read and written, in us
      if (base + (double)count * sums >= best.us) break;
      auto grads = [&](int64_t tiles) {
        return grad_rounds(c, tiles * dt, (double)m * e / bk, m * dt * s, (double)(tiles * e / bk) / s).us + sums;
      };
      const double us = base + (double)(count - 1) * grads(q) + grads(rest);
      if (us < best.us) best = {q, s, us};
    }
  }
  return best;
}

XentPlan xent_plan(int64_t n, int64_t d, int64_t v, ns_dtype dtype, bool aligned, bool backward, void* ws) {
  XentPlan p;
  p.n = n;
  p.d = d;
  p.v = v;
  p.es = bytes_of(dtype);
  p.bk = kRowBytes / p.es;
  p.k = round_to(d, p.bk);
  p.stage = p.k != d || !aligned;
  const EdgeCost* costs = edge_costs(p.es);
  Carver c{reinterpret_cast<char*>(ws)};
  if (!backward && n <= (p.stage ? kXentDotRowsStaged : kXentDotRows)) {
    p.groups = (v + kDotRows - 1) / kDotRows;
    const int64_t each = (p.groups + kXentDotWaves - 1) / kXentDotWaves;
    p.waves = (p.groups + each - 1) / each;
    p.zt = c.take<float>(n);
    p.parts = c.take<float2>(n * p.waves);
    p.total = c.used;
    return p;
  }
  if (!backward) {
    if (p.es == 2 && n <= kXentFewRows) {
      p.tm = kXentFewM;
      p.tn = kXentFewN;
    } else {
      auto us = [&](const EdgeCost& x) {
        const int64_t e = x.edge;
        return product_us(x, ((n + e - 1) / e) * ((v + e - 1) / e), (double)p.k / p.bk);
      };
      p.tm = p.tn = us(costs[0]) <= us(costs[1]) ? costs[0].edge : costs[1].edge;
    }
  } else {
    const BackwardChoice large = choose_backward(costs[0], n, d, v, p.k, p.bk);
    const BackwardChoice small = choose_backward(costs[1], n, d, v, p.k, p.bk);
    const bool l = large.us <= small.us;
    p.tm = p.tn = l ? costs[0].edge : costs[1].edge;
    p.piece = (l ? large : small).piece_tiles * p.tm;
    p.splits = (l ? large : small).splits;
  }
  p.n_pad = round_to(n, p.tm);
  p.tiles_m = p.n_pad / p.tm;
  p.tgt = c.take<int32_t>(p.n_pad);
  if (p.stage) p.Hs = c.take<char>(n * p.k * p.es);
  if (!backward) {
    p.tiles_n = (v + p.tn - 1) / p.tn;
    if (p.stage) p.Ws = c.take<char>(v * p.k * p.es);
    p.zt = c.take<float>(p.n_pad);
    p.parts = c.take<float2>(2 * p.tiles_n * p.n_pad);
  } else {
    p.d_pad = round_to(d, p.tm);
    if (p.stage) p.Ws = c.take<char>(std::min(p.piece, v) * p.k * p.es);
    p.coef = c.take<float>(p.n_pad);
    p.lse = c.take<float>(p.n_pad);
    p.gmax = c.take<float>(1);
    p.gmax_parts = c.take<float>((p.n_pad + 255) / 256);
    p.dz = c.take<char>(p.n_pad * p.piece * p.es);
    p.dzt = c.take<char>(p.n_pad * p.piece * p.es);
    p.WT = c.take<char>(p.d_pad * p.piece * p.es);
    p.HT = c.take<char>(p.d_pad * p.n_pad * p.es);
    p.acc = c.take<float>((int64_t)p.splits * p.n_pad * p.d_pad);
  }
  p.total = c.used;
  return p;
}

// A call's launches as text (see ns_plan_linear_cross_entropy); the length
// that it needs without the NUL.
int describe_xent(const XentPlan& p, ns_dtype dtype, bool backward, char* buf, size_t len) {
  const char* op = dtype == NS_FP32 ? "f32" : dtype == NS_FP16 ? "f16" : "bf16";
  const char* join = p.waves || p.n <= kXentJoinRows ? "joinrow" : "join";
  if (p.n == 0) return backward ? snprintf(buf, len, "zero<%s>", op) : snprintf(buf, len, "%s", "");
  if (p.waves) {
    const int64_t v = 16 / p.es;
    const char* form = p.d % v == 0 ? "even" : p.d > v ? "ragged" : "tiny";
    return snprintf(buf, len, "dot<%s,%d,%s> %s", op, xent_dot_rows(p.n), form, join);
  }
  if (!backward) return snprintf(buf, len, "prep<%s> fwd<%s,%dx%d> %s", op, op, (int)p.tm, (int)p.tn, join);
  return snprintf(buf, len, "prep<%s> dz<%s,%d> grads<%s,%d> dhout<%s> pieces=%d splits=%d", op, op, (int)p.tm, op,
                  (int)p.tm, op, (int)((p.v + p.piece - 1) / p.piece), p.splits);
}

// The products' copies take 16-byte chunks, swizzled by bits 4 to 6 of the
// address within a row: rows a multiple of 128 bytes apart.
bool xent_aligned(const void* H, int64_t ldh, const void* W, int64_t ldw, ns_dtype dtype) {
  const int64_t b = bytes_of(dtype);
  return aligned16(H) && aligned16(W) && ldh * b % kRowBytes == 0 && ldw * b % kRowBytes == 0;
}

// The copies of one operand (rows x d at src): padded when the products read
// a staging copy, transposed into dst_t (ldt wide) unless that is null.
XentCopyArgs xent_copy(const XentPlan& p, const void* src, int64_t ld, int64_t rows, char* padded, char* dst_t,
                       int64_t rows_pad, int64_t ldt) {
  XentCopyArgs a{};
  if (!padded && !dst_t) return a;
  a.src = src;
  a.ld = ld;
  a.rows = rows;
  a.cols = (int)p.d;
  a.padded = padded;
  a.cols_k = (int)p.k;
  a.transposed = dst_t;
  a.ldt = ldt;
  a.tiles_r = (int)((dst_t ? rows_pad : round_to(rows, 64)) / 64);
  a.tiles_c = (int)((dst_t ? p.d_pad : round_to(p.k, 64)) / 64);
  return a;
}

template <typename T>
ns_status xent_prep(const XentPrepArgs& a, hipStream_t st) {
  const int64_t blocks = a.row_blocks + a.h.blocks() + a.w.blocks();
  if (blocks == 0) return NS_OK;
  hipLaunchKernelGGL((k_xent_prep<T>), dim3((unsigned)blocks), dim3(256), 0, st, a);
  return launched();
}

template <typename T>
ns_status xent_forward(const XentPlan& p, const void* H, int64_t ldh, const void* W, int64_t ldw,
                       const XentTargets& targets, float* loss, float* lse, int32_t* d_status, hipStream_t st) {
  XentJoinArgs j{p.parts, 0,       p.n, 0,   0,        p.zt,
                 targets, loss, lse, d_status, (int32_t)(NS_ERR_NONFINITE | NS_STATUS_AT_OUTPUT),
                 (int32_t)NS_STATUS_BAD_INDEX};
  if (p.waves) {
    const XentDotArgs a{H, W, ldh, ldw, p.n, p.v, (int)p.d, (int)p.waves, (int)p.groups, targets, p.parts, p.zt};
    const hipError_t e = launch_xent_dot<T>(a, st);
    if (e != hipSuccess) return NS_ERR_HIP;
    j.count = (int)p.waves;
    j.part_stride = 1;
    j.row_stride = p.waves;
    hipLaunchKernelGGL(k_xent_join_row, dim3((unsigned)p.n), dim3(1024), 0, st, j);
    return launched();
  }
  XentPrepArgs prep{};
  prep.rows.targets = targets;
  prep.rows.n = p.n;
  prep.rows.n_pad = p.n_pad;
  prep.rows.tgt = p.tgt;
  prep.row_blocks = (int)((p.n_pad + 255) / 256);
  prep.h = xent_copy(p, H, ldh, p.n, p.Hs, nullptr, 0, 0);
  prep.w = xent_copy(p, W, ldw, p.v, p.Ws, nullptr, 0, 0);
  if (xent_prep<T>(prep, st) != NS_OK) return NS_ERR_HIP;
  XentArgs a{};
  a.H = p.stage ? p.Hs : H;
  a.W = p.stage ? p.Ws : W;
  a.ldh = (p.stage ? p.k : ldh) * (int64_t)sizeof(T);
  a.ldw = (p.stage ? p.k : ldw) * (int64_t)sizeof(T);
  a.row_bytes = (uint32_t)(p.k * sizeof(T));
  a.k = (int)p.k;
  a.n = p.n;
  a.v = p.v;
  a.tiles_m = (int)p.tiles_m;
  a.tiles_n = (int)p.tiles_n;
  a.tgt = p.tgt;
  a.n_pad = p.n_pad;
  a.parts = p.parts;
  a.zt = p.zt;
  const hipError_t e = launch_xent_fwd<T>(a, (int)p.tm, st, (int)p.tn);
  if (e != hipSuccess) return NS_ERR_HIP;
  j.count = (int)(2 * p.tiles_n);
  j.part_stride = p.n_pad;
  j.row_stride = 1;
  if (p.n <= kXentJoinRows)
    hipLaunchKernelGGL(k_xent_join_row, dim3((unsigned)p.n), dim3(1024), 0, st, j);
  else
    hipLaunchKernelGGL(k_xent_join, dim3((unsigned)((p.n + 15) / 16)), dim3(1024), 0, st, j);
  return launched();
}

template <typename T>
ns_status xent_backward(const XentPlan& p, const void* H, int64_t ldh, const void* W, int64_t ldw, XentRowArgs rows,
                        void* dH, int64_t lddh, void* dW, int64_t lddw, int32_t* d_status, hipStream_t st) {
  const int64_t edge = p.tm;
  XentPrepArgs prep{};
  prep.rows = rows;
  prep.row_blocks = (int)((p.n_pad + 255) / 256);
  prep.h = xent_copy(p, H, ldh, p.n, p.Hs, dW ? p.HT : nullptr, p.n_pad, p.n_pad);
  prep.h.masked = 1;
  for (int64_t v0 = 0; v0 < p.v; v0 += p.piece) {
    const int64_t rows_v = std::min(p.piece, p.v - v0), width = round_to(rows_v, edge);
    const T* w = reinterpret_cast<const T*>(W) + v0 * ldw;
    prep.w = xent_copy(p, w, ldw, rows_v, p.Ws, dH ? p.WT : nullptr, width, p.piece);
    if (xent_prep<T>(prep, st) != NS_OK) return NS_ERR_HIP;
    prep.row_blocks = 0;  // H and the rows once, W for every piece
    prep.h = XentCopyArgs{};
    XentArgs a{};
    a.H = p.stage ? p.Hs : H;
    a.W = p.stage ? p.Ws : reinterpret_cast<const char*>(w);
    a.ldh = (p.stage ? p.k : ldh) * (int64_t)sizeof(T);
    a.ldw = (p.stage ? p.k : ldw) * (int64_t)sizeof(T);
    a.row_bytes = (uint32_t)(p.k * sizeof(T));
    a.k = (int)p.k;
    a.n = p.n;
    a.v = rows_v;
    a.tiles_m = (int)p.tiles_m;
    a.tiles_n = (int)(width / edge);
    a.tgt = p.tgt;
    a.n_pad = p.n_pad;
    a.v0 = (int)v0;
    a.coef = p.coef;
    a.lse = p.lse;
    a.gmax = p.gmax;
    a.gmax_parts = p.gmax_parts;
    a.gmax_count = (int)((p.n_pad + 255) / 256);
    a.dz = p.dz;
    a.dzt = p.dzt;
    a.ldz = p.piece;
    hipError_t e = launch_xent_dz<T>(a, (int)edge, st);
    if (e != hipSuccess) return NS_ERR_HIP;
    XentDwArgs b{};
    b.gmax = p.gmax;
    b.d_status = d_status;
    b.status_bits = (int32_t)(NS_ERR_NONFINITE | NS_STATUS_AT_OUTPUT);
    if (dW) {
      b.L = p.dzt;
      b.R = p.HT;
      b.ldl = b.ldr = p.n_pad * (int64_t)sizeof(T);
      b.k = (int)p.n_pad;
      b.tiles_m = (int)(width / edge);
      b.tiles_n = (int)(p.d_pad / edge);
      b.out = reinterpret_cast<T*>(dW) + v0 * lddw;
      b.ldo = lddw;
      b.rows = rows_v;
      b.cols = (int)p.d;
    }
    XentDhArgs h{};
    if (dH) {
      h.L = p.dz;
      h.R = p.WT;
      h.ldl = h.ldr = p.piece * (int64_t)sizeof(T);
      h.ktiles = (int)(width / p.bk);
      h.splits = p.splits;
      h.tiles_m = (int)p.tiles_m;
      h.tiles_n = (int)(p.d_pad / edge);
      h.acc = p.acc;
      h.n_pad = p.n_pad;
      h.d_pad = p.d_pad;
      h.first = v0 == 0;
      const EdgeCost* costs = edge_costs(p.es);
      h.extra = grad_rounds(costs[edge == costs[0].edge ? 0 : 1], (int64_t)b.tiles_m * b.tiles_n, (double)b.k / p.bk,
                            (int64_t)h.tiles_m * h.tiles_n * h.splits, (double)h.ktiles / h.splits)
                    .extra;
    }
    if ((dW || dH) && (e = launch_xent_grads<T>(b, h, (int)edge, st)) != hipSuccess) return NS_ERR_HIP;
  }
  constexpr int64_t kOutCols = 64 * kVec<T>;
  if (dH)
    hipLaunchKernelGGL((k_xent_dh_out<T>), dim3((unsigned)p.n, (unsigned)((p.d + kOutCols - 1) / kOutCols)), dim3(64), 0, st, p.acc, p.splits, p.n_pad, p.d_pad,
                       reinterpret_cast<T*>(dH), lddh, (int)p.d, p.coef, p.gmax, d_status,
                       (int32_t)(NS_ERR_NONFINITE | NS_STATUS_AT_OUTPUT));
  return launched();
}

}  // namespace

extern "C" {

ns_status ns_layer_norm(const void* X, int64_t rows, int64_t cols, int64_t ldx, ns_dtype dtype, const void* weight,
                        const void* bias, ns_dtype param_dtype, float eps, void* Y, int64_t ldy, float* mean,
                        float* rstd, int32_t* d_status, ns_stream_t stream) {
  if (!norm_shape_ok(rows, cols) || ldx < cols || ldy < cols) return NS_ERR_INVALID_ARG;
  if (!(eps >= 0.f && isfinite(eps))) return NS_ERR_INVALID_ARG;
  if (!known(dtype) || !(param_dtype == dtype || param_dtype == NS_FP32)) return NS_ERR_UNSUPPORTED_DTYPE;
  if (rows == 0) return NS_OK;
  if (!X || !Y) return NS_ERR_INVALID_ARG;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const NormFwdArgs a{X,    Y,   weight,    bias, mean, rstd, rows, ldx, ldy, (int)cols,
                      eps, d_status, (int32_t)(NS_ERR_NONFINITE | NS_STATUS_AT_OUTPUT)};
  return with_types(dtype, param_dtype, [&](auto io, auto pt) {
    using IO = decltype(io);
    using PT = decltype(pt);
    if (norm_by_element<IO>(cols))
      hipLaunchKernelGGL((k_norm_fwd_long<IO, PT>), dim3((unsigned)std::min(rows, kMaxBlocks)), dim3(1024), 0, st, a);
    else
      with_norm_form<IO>(cols, NormFwdRun<IO, PT>{a, st});
    return launched();
  });
}

size_t ns_layer_norm_workspace_size(int64_t rows, int64_t cols) {
  if (!norm_shape_ok(rows, cols)) return 0;
  return std::max(kAlignTo, align_up_to((size_t)norm_parts(rows, 1) * 2 * cols * sizeof(float)));
}

ns_status ns_layer_norm_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, int64_t rows, int64_t cols,
                                 ns_dtype dtype, const float* mean, const float* rstd, const void* weight,
                                 ns_dtype param_dtype, void* dX, int64_t lddx, void* dweight, void* dbias,
                                 int32_t* d_status, void* workspace, size_t workspace_bytes, ns_stream_t stream) {
  if (!norm_shape_ok(rows, cols) || ldx < cols || lddy < cols || lddx < cols) return NS_ERR_INVALID_ARG;
  if (!known(dtype) || !(param_dtype == dtype || param_dtype == NS_FP32)) return NS_ERR_UNSUPPORTED_DTYPE;
  if (rows > 0 && (!dY || !X || !mean || !rstd || !dX)) return NS_ERR_INVALID_ARG;
  const bool params = dweight || dbias;
  if (rows == 0 && !params) return NS_OK;
  if (params && !workspace_ok(workspace, workspace_bytes, ns_layer_norm_workspace_size(rows, cols)))
    return NS_ERR_WORKSPACE;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const NormBwdArgs a{dY,   X,   weight, dX,   mean,      rstd,     params ? reinterpret_cast<float*>(workspace) : nullptr,
                      rows, lddy, ldx,    lddx, (int)cols, d_status, (int32_t)(NS_ERR_NONFINITE | NS_STATUS_AT_OUTPUT)};
  return with_types(dtype, param_dtype, [&](auto io, auto pt) {
    using IO = decltype(io);
    using PT = decltype(pt);
    const int64_t parts = norm_parts(rows, norm_rows_per_block<IO>(cols));
    if (rows > 0) {
      if (norm_by_element<IO>(cols)) {
        // The parameters' pass comes first: dX may be dY.
        if (params)
          hipLaunchKernelGGL((k_norm_cols<IO>), dim3((unsigned)((cols + 255) / 256), (unsigned)parts), dim3(256), 0, st,
                             a);
        hipLaunchKernelGGL((k_norm_bwd_long<IO, PT>), dim3((unsigned)std::min(rows, kMaxBlocks)), dim3(1024), 0, st, a);
      } else {
        with_norm_form<IO>(cols, NormBwdRun<IO, PT>{a, parts, st});
      }
    }
    if (params)
      hipLaunchKernelGGL((k_norm_join<PT>), dim3((unsigned)((2 * cols + 63) / 64)), dim3(1024), 0, st,
                         reinterpret_cast<const float*>(workspace), (int)(rows > 0 ? parts : 0), (int)cols,
                         reinterpret_cast<PT*>(dweight), reinterpret_cast<PT*>(dbias), d_status, a.status_bits);
    return launched();
  });
}

ns_status ns_embedding(const void* ids, int32_t ids64, int64_t n, const void* table, int64_t vocab, int64_t cols,
                       int64_t ldt, ns_dtype dtype, float scale, void* out, int64_t ldo, int32_t* d_status,
                       ns_stream_t stream) {
  if (!embed_shape_ok(n, vocab, cols) || ldt < cols || ldo < cols || !isfinite(scale)) return NS_ERR_INVALID_ARG;
  if (ids64 != 0 && ids64 != 1) return NS_ERR_INVALID_ARG;
  if (!known(dtype)) return NS_ERR_UNSUPPORTED_DTYPE;
  if (n == 0) return NS_OK;
  if (!ids || !table || !out) return NS_ERR_INVALID_ARG;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const EmbedArgs a{ids, ids64, n,        vocab,          (int)cols, table, out, ldt, ldo,
                    scale, d_status, (int32_t)NS_STATUS_BAD_INDEX, (int32_t)(NS_ERR_NONFINITE | NS_STATUS_AT_OUTPUT)};
  const dim3 grid((unsigned)std::min((n + 3) / 4, kMaxBlocks));
  return with_type(dtype, [&](auto io) {
    with_row_form<decltype(io)>(cols, [&](auto form) {
      hipLaunchKernelGGL((k_embed<decltype(io), decltype(form)::value>), grid, dim3(256), 0, st, a);
    });
    return launched();
  });
}

size_t ns_embedding_workspace_size(int64_t n, int64_t vocab, int64_t cols) {
  if (!embed_grad_shape_ok(n, vocab, cols)) return 0;
  // The same for every type: fp32's slices are the narrowest, 16-bit ones the widest.
  return std::max(embed_plan(n, vocab, cols, nullptr, 2).total, embed_plan(n, vocab, cols, nullptr, 4).total);
}

ns_status ns_embedding_backward(const void* ids, int32_t ids64, int64_t n, const void* dY, int64_t lddy, int64_t vocab,
                                int64_t cols, ns_dtype dtype, float scale, void* dT, int64_t ldt, int32_t accumulate,
                                int32_t* d_status, void* workspace, size_t workspace_bytes, ns_stream_t stream) {
  if (!embed_grad_shape_ok(n, vocab, cols) || lddy < cols || ldt < cols || !isfinite(scale)) return NS_ERR_INVALID_ARG;
  if ((ids64 != 0 && ids64 != 1) || (accumulate != 0 && accumulate != 1)) return NS_ERR_INVALID_ARG;
  if (!known(dtype)) return NS_ERR_UNSUPPORTED_DTYPE;
  if (!dT || (n > 0 && (!ids || !dY))) return NS_ERR_INVALID_ARG;
  const EmbedPlan p = embed_plan(n, vocab, cols, workspace, bytes_of(dtype));
  if (!workspace_ok(workspace, workspace_bytes, p.total)) return NS_ERR_WORKSPACE;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  const int per = embed_ids_per_block(vocab);
  const SortArgs s{ids, ids64, n, vocab, per, p.order, p.key, p.start, d_status, (int32_t)NS_STATUS_BAD_INDEX};
  hipLaunchKernelGGL(k_embed_sort, dim3((unsigned)((vocab + per - 1) / per)), dim3(kSortWaves * 64), 0, st, s);
  const EmbedSumArgs a{dY,      dT,        n,       vocab,    lddy,  ldt,        (int)cols, p.order, p.key,
                       p.start, p.partial, (int)p.cols_pad, p.chunk, p.chunks, scale, accumulate, d_status,
                       (int32_t)(NS_ERR_NONFINITE | NS_STATUS_AT_OUTPUT)};
  return with_type(dtype, [&](auto io) {
    using IO = decltype(io);
    with_row_form<IO>(cols, [&](auto form) {
      constexpr int FORM = decltype(form)::value;
      const int64_t vectors = embed_slice(cols, sizeof(IO)) / (64 * kVec<IO>);
      if (FORM == kTiny || vectors == 1)
        embed_sum<IO, 1, 8, FORM>(a, st);
      else if (vectors == 2)
        embed_sum<IO, 2, 8, FORM == kTiny ? kEven : FORM>(a, st);
      else
        embed_sum<IO, 4, 4, FORM == kTiny ? kEven : FORM>(a, st);
    });
    return launched();
  });
}

size_t ns_linear_cross_entropy_workspace_size(int64_t rows, int64_t cols, int64_t vocab, ns_dtype dtype,
                                              int32_t aligned, int32_t backward) {
  if (!xent_shape_ok(rows, cols, vocab) || !known(dtype)) return 0;
  return std::max(kAlignTo, xent_plan(rows, cols, vocab, dtype, aligned != 0, backward != 0, nullptr).total);
}

int64_t ns_plan_linear_cross_entropy(int64_t rows, int64_t cols, int64_t vocab, ns_dtype dtype, int32_t aligned,
                                     int32_t backward, char* buf, size_t len) {
  if (!xent_shape_ok(rows, cols, vocab) || !known(dtype)) return -1;
  const XentPlan p = xent_plan(rows, cols, vocab, dtype, aligned != 0, backward != 0, nullptr);
  return describe_xent(p, dtype, backward != 0, buf, buf ? len : 0) + 1;
}

ns_status ns_linear_cross_entropy(const void* H, int64_t ldh, const void* W, int64_t ldw, const void* targets,
                                  int32_t targets64, int64_t rows, int64_t cols, int64_t vocab, ns_dtype dtype,
                                  int64_t ignore_index, float* loss, float* lse, int32_t* d_status, void* workspace,
                                  size_t workspace_bytes, ns_stream_t stream) {
  if (!xent_shape_ok(rows, cols, vocab) || ldh < cols || ldw < cols) return NS_ERR_INVALID_ARG;
  if (ldh > kMaxXentCols * 8 || ldw > kMaxXentCols * 8) return NS_ERR_INVALID_ARG;
  if (targets64 != 0 && targets64 != 1) return NS_ERR_INVALID_ARG;
  if (!known(dtype)) return NS_ERR_UNSUPPORTED_DTYPE;
  if (rows == 0) return NS_OK;
  if (!H || !W || !targets || !loss || !lse) return NS_ERR_INVALID_ARG;
  const XentPlan p = xent_plan(rows, cols, vocab, dtype, xent_aligned(H, ldh, W, ldw, dtype), false, workspace);
  if (!workspace_ok(workspace, workspace_bytes, p.total)) return NS_ERR_WORKSPACE;
  const XentTargets t{targets, targets64, ignore_index, vocab};
  return with_type(dtype, [&](auto io) {
    return xent_forward<decltype(io)>(p, H, ldh, W, ldw, t, loss, lse, d_status, reinterpret_cast<hipStream_t>(stream));
  });
}

ns_status ns_linear_cross_entropy_backward(const void* H, int64_t ldh, const void* W, int64_t ldw, const void* targets,
                                           int32_t targets64, int64_t rows, int64_t cols, int64_t vocab, ns_dtype dtype,
                                           int64_t ignore_index, const float* lse, const float* dloss, void* dH,
                                           int64_t lddh, void* dW, int64_t lddw, int32_t* d_status, void* workspace,
                                           size_t workspace_bytes, ns_stream_t stream) {
  if (!xent_shape_ok(rows, cols, vocab) || ldh < cols || ldw < cols) return NS_ERR_INVALID_ARG;
  if (ldh > kMaxXentCols * 8 || ldw > kMaxXentCols * 8) return NS_ERR_INVALID_ARG;
  if ((dH && lddh < cols) || (dW && lddw < cols)) return NS_ERR_INVALID_ARG;
  if (targets64 != 0 && targets64 != 1) return NS_ERR_INVALID_ARG;
  if (!known(dtype)) return NS_ERR_UNSUPPORTED_DTYPE;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (rows == 0) {
    if (!dW) return NS_OK;
    return with_type(dtype, [&](auto io) {
      using T = decltype(io);
      hipLaunchKernelGGL((k_xent_zero<T>), dim3((unsigned)vocab), dim3(256), 0, st, reinterpret_cast<T*>(dW), lddw,
                         (int)cols);
      return launched();
    });
  }
  if (!H || !W || !targets || !lse || !dloss) return NS_ERR_INVALID_ARG;
  const XentPlan p = xent_plan(rows, cols, vocab, dtype, xent_aligned(H, ldh, W, ldw, dtype), true, workspace);
  if (!workspace_ok(workspace, workspace_bytes, p.total)) return NS_ERR_WORKSPACE;
  if (!dH && !dW) return NS_OK;
  XentRowArgs r{};
  r.targets = XentTargets{targets, targets64, ignore_index, vocab};
  r.n = rows;
  r.n_pad = p.n_pad;
  r.tgt = p.tgt;
  r.dloss = dloss;
  r.lse = lse;
  r.coef = p.coef;
  r.lse_pad = p.lse;
  r.gmax_parts = p.gmax_parts;
  r.d_status = d_status;
  r.index_bit = (int32_t)NS_STATUS_BAD_INDEX;
  return with_type(dtype, [&](auto io) {
    return xent_backward<decltype(io)>(p, H, ldh, W, ldw, r, dH, lddh, dW, lddw, d_status, st);
  });
}

}  // extern "C"
