// resnorm.hip - C entry points of the residual norms (resnorm.hpp): argument
// checks, workspace layout and kernel choice.
#include <math.h>

#include <algorithm>

#include "host.hpp"
#include "resnorm.hpp"

namespace {

using namespace nsk;

constexpr int64_t kMaxResNormCols = 1 << 24;
constexpr int kResNormRegisterCols = 8192;  // the widest row that the kernels hold in registers
constexpr int64_t kResNormFwdThreads = 256 * 2048;
// Blocks of the backward pass, each of which leaves partial rows of dw, dwb
// and the gate's gradient: two per compute unit (16384 x 768: one 56 us, two
// 43, four 52, for the partial rows), or the one that fits.
constexpr int64_t kResNormParts = 512;
constexpr int64_t kMaxJoinRows = 32768;  // of a launch's second dimension

// Calls f.template run<NV, TPR>() for a row width: rows of up to 128 vectors
// share a block, whose waves hold one or two each; wider ones have a block of
// their own with one vector per thread, or two where that was faster: fp32
// data, whose vectors are half as many values, and 16-bit data with 16-bit
// parameters (8192 x 4096 99 us against 104; with fp32 parameters, whose reads
// from LDS wait longer, 133 against 105).
template <typename IO, typename PT, class F>
auto resnorm_form(int64_t cols, F&& f) {
  const int64_t n = (cols + kVec<IO> - 1) / kVec<IO>;
  if (n <= 32) return f.template run<1, 32>();
  if (n <= 64) return f.template run<2, 32>();
  if (n <= 96) return f.template run<3, 32>();
  if (n <= 128) return f.template run<2, 64>();
  if (n <= 256) return f.template run<1, 256>();
  if constexpr (sizeof(IO) == 4) {
    if (n <= 512) return f.template run<2, 256>();
    if (n <= 1024) return f.template run<2, 512>();
    return f.template run<2, 1024>();
  } else {
    if constexpr (sizeof(PT) == 2) {
      if (n <= 512) return f.template run<2, 256>();
    } else {
      if (n <= 512) return f.template run<1, 512>();
    }
    return f.template run<1, 1024>();
  }
}
template <typename IO>
bool resnorm_by_element(int64_t cols) {
  return cols < kVec<IO> || cols > kResNormRegisterCols;
}

// Rows of less than a vector that a block sums columns over at a time, each of
// up to 256 / kResNormNarrow columns.
constexpr int kResNormNarrow = 32;
template <typename IO>
constexpr bool resnorm_narrow(int64_t cols) {
  static_assert(kVec<IO> <= 256 / kResNormNarrow, "a block's columns");
  return cols < kVec<IO>;
}

// Rows that a block works on at a time, and the blocks of the backward pass.
struct ResNormBlocks {
  int rows;
  int64_t parts;
};
struct ResNormBlocksOf {
  template <int NV, int TPR>
  ResNormBlocks run() const {
    return {kNormRows<TPR>, TPR == 1024 ? kResNormParts / 2 : kResNormParts};
  }
};
template <typename IO, typename PT>
ResNormBlocks resnorm_blocks(int64_t cols) {
  if (resnorm_by_element<IO>(cols)) return {resnorm_narrow<IO>(cols) ? kResNormNarrow : 1, kResNormParts};
  return resnorm_form<IO, PT>(cols, ResNormBlocksOf{});
}

template <typename IO, typename PT>
struct ResNormFwdRun {
  const ResNormFwdArgs& a;
  hipStream_t st;
  template <int NV, int TPR>
  void run() const {
    const int64_t groups = (a.rows + kNormRows<TPR> - 1) / kNormRows<TPR>;
    const dim3 blocks((unsigned)std::min<int64_t>(groups, kResNormFwdThreads / kNormThreads<TPR>)), threads(kNormThreads<TPR>);
    if (a.cols % kVec<IO> == 0)
      hipLaunchKernelGGL((k_resnorm_fwd<IO, PT, NV, TPR, kEven>), blocks, threads, 0, st, a);
    else
      hipLaunchKernelGGL((k_resnorm_fwd<IO, PT, NV, TPR, kRagged>), blocks, threads, 0, st, a);
  }
};

template <typename IO, typename PT>
struct ResNormBwdRun {
  const ResNormBwdArgs& a;
  int64_t blocks;
  hipStream_t st;
  template <int NV, int TPR>
  void run() const {
    const dim3 grid((unsigned)blocks), threads(kNormThreads<TPR>);
    if (a.cols % kVec<IO> == 0)
      hipLaunchKernelGGL((k_resnorm_bwd<IO, PT, NV, TPR, kEven>), grid, threads, 0, st, a);
    else
      hipLaunchKernelGGL((k_resnorm_bwd<IO, PT, NV, TPR, kRagged>), grid, threads, 0, st, a);
  }
};

bool resnorm_shape_ok(int64_t rows, int64_t cols, int64_t groups) {
  if (!(rows >= 0 && rows < (int64_t(1) << 31) && cols >= 1 && cols <= kMaxResNormCols)) return false;
  if (rows == 0) return groups >= 0 && groups < (int64_t(1) << 31);  // zeros for the gate's gradient
  return groups == 0 || (groups > 0 && groups <= rows && rows % groups == 0);
}

// How the backward pass cuts the rows (ResNormBwdArgs), for `groups` rows of
// the gate that are summed over.
struct ResNormCut {
  int64_t groups, group_rows, blocks;
  int split;
};
ResNormCut resnorm_cut(int64_t rows, int64_t groups, const ResNormBlocks& b) {
  ResNormCut c;
  c.groups = groups;
  c.group_rows = rows / groups;
  const int64_t most = (c.group_rows + b.rows - 1) / b.rows;  // no segment without rows
  c.split = (int)std::max<int64_t>(1, std::min(b.parts / groups, most));
  c.blocks = std::min(groups * c.split, b.parts);
  return c;
}

}  // namespace

extern "C" {

ns_status ns_residual_norm(const void* X, int64_t ldx, const void* Z, int64_t ldz, int64_t rows, int64_t cols,
                           ns_dtype dtype, const void* gate, int64_t groups, const void* branch_weight,
                           const void* weight, ns_dtype param_dtype, float scale, int32_t norm_branch, float eps,
                           void* S, int64_t lds, void* Y, int64_t ldy, float* branch_rstd, float* rstd,
                           int32_t* d_status, ns_stream_t stream) {
  if (!resnorm_shape_ok(rows, cols, gate ? groups : 0) || (gate && groups == 0)) return NS_ERR_INVALID_ARG;
  if (ldx < cols || (Z && (ldz < cols || lds < cols)) || (Y && ldy < cols)) return NS_ERR_INVALID_ARG;
  if (!(eps >= 0.f && isfinite(eps)) || !isfinite(scale) || (norm_branch != 0 && norm_branch != 1))
    return NS_ERR_INVALID_ARG;
  if (!known(dtype) || !(param_dtype == dtype || param_dtype == NS_FP32)) return NS_ERR_UNSUPPORTED_DTYPE;
  if (rows == 0) return NS_OK;
  // Without a block's output there is only the second norm.
  if (!Z && (gate || branch_weight || S || scale != 1.f || !Y)) return NS_ERR_INVALID_ARG;
  if (!X || (Z && !S) || (S && S == Y)) return NS_ERR_INVALID_ARG;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  ResNormFwdArgs a{};
  a.X = X;
  a.Z = Z;
  a.gate = gate;
  a.wb = branch_weight;
  a.w = weight;
  a.S = S;
  a.Y = Y;
  a.rb = branch_rstd;
  a.rs = rstd;
  a.rows = rows;
  a.ldx = ldx;
  a.ldz = ldz;
  a.lds = lds;
  a.ldy = ldy;
  a.gate_rows = gate ? (uint32_t)(rows / groups) : 1u;
  a.cols = (int)cols;
  a.scale = scale;
  a.eps = eps;
  a.norm_branch = norm_branch;
  a.d_status = d_status;
  a.status_bits = (int32_t)(NS_ERR_NONFINITE | NS_STATUS_AT_OUTPUT);
  return with_types(dtype, param_dtype, [&](auto io, auto pt) {
    using IO = decltype(io);
    using PT = decltype(pt);
    if (resnorm_by_element<IO>(cols))
      hipLaunchKernelGGL((k_resnorm_fwd_long<IO, PT>), dim3((unsigned)std::min(rows, kMaxBlocks)), dim3(1024), 0, st, a);
    else
      resnorm_form<IO, PT>(cols, ResNormFwdRun<IO, PT>{a, st});
    return launched();
  });
}

size_t ns_residual_norm_workspace_size(int64_t rows, int64_t cols) {
  if (!resnorm_shape_ok(rows, cols, 0)) return 0;
  const size_t parts = align_up_to((size_t)std::min(rows, kResNormParts) * 3 * partial_stride(cols) * sizeof(float));
  return std::max(kAlignTo, parts + align_up_to((size_t)rows * sizeof(float)));
}

ns_status ns_residual_norm_backward(const void* dS, int64_t ldds, const void* dY, int64_t lddy, const void* S,
                                    int64_t lds, const void* Z, int64_t ldz, int64_t rows, int64_t cols,
                                    ns_dtype dtype, const float* branch_rstd, const float* rstd, const void* gate,
                                    int64_t groups, const void* branch_weight, const void* weight,
                                    ns_dtype param_dtype, float scale, void* dX, int64_t lddx, void* dZ, int64_t lddz,
                                    void* dgate, void* dbranch_weight, void* dweight, int32_t* d_status,
                                    void* workspace, size_t workspace_bytes, ns_stream_t stream) {
  const bool gated = gate || dgate;
  if (!resnorm_shape_ok(rows, cols, gated ? groups : 0) || (gated && groups == 0)) return NS_ERR_INVALID_ARG;
  if ((dS && ldds < cols) || (dY && (lddy < cols || lds < cols)) || (Z && (ldz < cols || lddz < cols)) ||
      (dX && lddx < cols) || !isfinite(scale))
    return NS_ERR_INVALID_ARG;
  if (!known(dtype) || !(param_dtype == dtype || param_dtype == NS_FP32)) return NS_ERR_UNSUPPORTED_DTYPE;
  if (rows > 0) {
    if ((!dS && !dY) || (dY && (!S || !rstd)) || (Z && !dZ)) return NS_ERR_INVALID_ARG;
    // Without a block's output there is nothing that these would be gradients of.
    if (!Z && (dZ || gated || branch_weight || dbranch_weight || scale != 1.f || !dX)) return NS_ERR_INVALID_ARG;
    if (!dY && (weight || dweight)) return NS_ERR_INVALID_ARG;
  } else if (!dgate && !dbranch_weight && !dweight) {
    return NS_OK;
  }
  if (!workspace_ok(workspace, workspace_bytes, ns_residual_norm_workspace_size(rows, cols))) return NS_ERR_WORKSPACE;
  if (rows > 0 && dX && dX == dZ) return NS_ERR_INVALID_ARG;
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  ResNormBwdArgs a{};
  a.dS = dS;
  a.dY = dY;
  a.S = S;
  a.Z = Z;
  a.rb = branch_rstd;
  a.rs = rstd;
  a.gate = gate;
  a.wb = branch_weight;
  a.w = weight;
  a.dX = dX;
  a.dZ = dZ;
  a.rows = rows;
  a.ldds = ldds;
  a.lddy = lddy;
  a.lds = lds;
  a.ldz = ldz;
  a.lddx = lddx;
  a.lddz = lddz;
  a.gate_rows = gate && rows > 0 ? (uint32_t)(rows / groups) : 1u;
  a.cols = (int)cols;
  a.scale = scale;
  a.want_w = dweight != nullptr;
  a.want_wb = dbranch_weight != nullptr;
  a.d_status = d_status;
  a.status_bits = (int32_t)(NS_ERR_NONFINITE | NS_STATUS_AT_OUTPUT);
  // A gate of its own for each row has its gradient written with the row.
  const bool own_rows = dgate && rows > 0 && groups == rows && rows > 1;
  a.dgate_rows = own_rows ? dgate : nullptr;
  a.want_gate = dgate && !own_rows;
  a.e_gated = gate && groups > 1 && !a.want_gate;
  Carver carve{reinterpret_cast<char*>(workspace)};
  a.partial = carve.take<float>(std::min(rows, kResNormParts) * 3 * partial_stride(cols));
  a.c_row = carve.take<float>(rows);
  return with_types(dtype, param_dtype, [&](auto io, auto pt) {
    using IO = decltype(io);
    using PT = decltype(pt);
    ResNormCut cut{1, 0, 0, 1};
    if (rows > 0) {
      cut = resnorm_cut(rows, a.want_gate ? groups : 1, resnorm_blocks<IO, PT>(cols));
      a.groups = cut.groups;
      a.group_rows = cut.group_rows;
      a.split = cut.split;
      a.dgate = a.want_gate ? dgate : nullptr;
      if (resnorm_by_element<IO>(cols)) {
        const dim3 grid((unsigned)std::min(rows, kMaxBlocks));
        if (dY) hipLaunchKernelGGL((k_resnorm_rows_long<IO, PT>), grid, dim3(1024), 0, st, a);
        if (a.want_w || a.want_wb || a.want_gate) {
          const unsigned parts = (unsigned)cut.blocks;
          if (resnorm_narrow<IO>(cols))
            hipLaunchKernelGGL((k_resnorm_cols_long<IO, PT, kResNormNarrow>), dim3(1, parts), dim3(256), 0, st, a);
          else
            hipLaunchKernelGGL((k_resnorm_cols_long<IO, PT, 1>), dim3((unsigned)((cols + 255) / 256), parts), dim3(256), 0,
                               st, a);
        }
        if (dX || dZ) hipLaunchKernelGGL((k_resnorm_bwd_long<IO, PT>), grid, dim3(1024), 0, st, a);
      } else {
        resnorm_form<IO, PT>(cols, ResNormBwdRun<IO, PT>{a, cut.blocks, st});
      }
    }
    // Without rows the gradients are zeros; a gate then has no rows either
    // unless the caller says so.
    const bool join_gate = a.want_gate && (rows == 0 || cut.split > 1);
    if (dweight || dbranch_weight || join_gate) {
      ResNormJoinArgs j{a.partial, (int)cut.blocks, rows > 0 ? cut.split : 0, (int)cols, 0, dweight, dbranch_weight,
                        join_gate ? dgate : nullptr, d_status, a.status_bits};
      // More than one launch only for a gate that has no rows to sum over.
      const int64_t outputs = 2 + (join_gate ? groups : 0);
      for (; j.first < outputs; j.first += kMaxJoinRows)
        hipLaunchKernelGGL((k_resnorm_join<PT>),
                           dim3((unsigned)((cols + 31) / 32), (unsigned)std::min(outputs - j.first, kMaxJoinRows)), dim3(1024),
                           0, st, j);
    }
    return launched();
  });
}

}  // extern "C"
