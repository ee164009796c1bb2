// C ABI of the separate operators (grouped expert products, 8-bit row codes,
// combine): argument checks and launches.  Host code only; the kernels live
// in grouped.hip and rows.hip.  See include/moe.h for the contract.
#include "moe.h"

#include <algorithm>

#include "grouped.hpp"

namespace moe {
void set_last_hip_error(int e);
}

namespace {

constexpr int32_t kMaxRows = 33554432, kMaxDim = 1048576, kMaxK8 = 131071;

bool off16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u); }

template <class... P>
int check_aligned(P... p) {
  return (off16(p) || ...) ? MOE_ERR_ALIGN : MOE_OK;
}

int status(hipError_t e) {
  if (e == hipSuccess) return MOE_OK;
  moe::set_last_hip_error(int(e));
  return MOE_ERR_HIP;
}

bool dim_ok(int32_t v, int32_t lo, int32_t hi) { return v >= lo && v <= hi; }

int check_grouped(const moe_grouped_shape_t* s) {
  if (!s) return MOE_ERR_NULL;
  if (!dim_ok(s->rows, 0, kMaxRows) || !dim_ok(s->x_rows, 0, kMaxRows)) return MOE_ERR_SHAPE;
  if (!dim_ok(s->N, 1, kMaxDim) || !dim_ok(s->K, 1, kMaxDim)) return MOE_ERR_SHAPE;
  if (!dim_ok(s->E, 1, 256) || !dim_ok(s->row_div, 1, 256)) return MOE_ERR_SHAPE;
  if (s->x_dtype != MOE_F32 && s->x_dtype != MOE_BF16 && s->x_dtype != MOE_I8) return MOE_ERR_DTYPE;
  if (s->out_dtype != MOE_F32 && (s->out_dtype != MOE_BF16 || s->x_dtype == MOE_F32)) return MOE_ERR_DTYPE;
  if (s->x_dtype == MOE_I8 && s->K > kMaxK8) return MOE_ERR_SHAPE;
  return MOE_OK;
}

// With rows looked up through row_ids any x_rows and row_div go; without, row r is row r.
bool lookup_ok(const moe_grouped_shape_t* s, const int32_t* row_ids) {
  return row_ids || (s->x_rows == s->rows && s->row_div == 1);
}

moe::GroupedArgs grouped_args(const moe_grouped_shape_t* s) {
  moe::GroupedArgs a{};
  // ceil(2^(31 + l) / row_div) with row_div <= 2^l < 2 row_div: fits 32 bits and is exact for 31-bit dividends
  int l = 0;
  while ((1 << l) < s->row_div) ++l;
  a.div_mul = unsigned(((1ull << (31 + l)) + unsigned(s->row_div) - 1) / unsigned(s->row_div));
  a.div_shift = l;
  a.rows = s->rows; a.N = s->N; a.K = s->K; a.E = s->E; a.x_rows = s->x_rows; a.row_div = s->row_div;
  return a;
}

size_t workspace_need(const moe_grouped_shape_t* s) {
  const moe::GroupedArgs a = grouped_args(s);
  size_t n = moe::grouped_workspace(a, moe::GM_FORWARD, s->x_dtype, s->out_dtype);
  if (s->x_dtype != MOE_I8) {
    n = std::max(n, moe::grouped_workspace(a, moe::GM_GRAD_X, s->x_dtype, s->out_dtype));
    n = std::max(n, moe::grouped_workspace(a, moe::GM_GRAD_W, s->x_dtype, s->out_dtype));
  }
  return n;
}

int forward(const moe_grouped_shape_t* s, const void* x, const float* x_scale, const int32_t* row_ids,
            const int32_t* offsets, const int32_t* counts, const void* w, const float* w_scale, void* y,
            void* workspace, size_t ws_bytes, void* stream) {
  const bool i8 = s->x_dtype == MOE_I8;
  if (!lookup_ok(s, row_ids)) return MOE_ERR_SHAPE;
  if (s->rows == 0) return MOE_OK;
  if (!offsets || !w || !y || (!x && s->x_rows > 0) || (i8 && (!w_scale || (!x_scale && s->x_rows > 0))))
    return MOE_ERR_NULL;
  const size_t need = workspace_need(s);
  if (need > 0 && !workspace) return MOE_ERR_NULL;
  if (int rc = check_aligned(x, x_scale, row_ids, offsets, counts, w, w_scale, y, workspace)) return rc;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  moe::GroupedArgs a = grouped_args(s);
  a.x = x; a.x_scale = x_scale; a.row_ids = row_ids; a.offsets = offsets; a.counts = counts;
  a.w = w; a.w_scale = w_scale; a.out = y;
  return status(moe::launch_grouped(a, moe::GM_FORWARD, s->x_dtype, s->out_dtype, workspace,
                                    static_cast<hipStream_t>(stream)));
}

int check_combine(const moe_combine_shape_t* s) {
  if (!s) return MOE_ERR_NULL;
  if (!dim_ok(s->T, 0, 1048576) || !dim_ok(s->top_k, 1, 256) || !dim_ok(s->H, 1, kMaxDim) ||
      !dim_ok(s->rows, 0, kMaxRows) || long(s->T) * s->top_k > 16777216)
    return MOE_ERR_SHAPE;
  if (s->y_dtype != MOE_F32 && s->y_dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (s->out_dtype != MOE_F32 && s->out_dtype != MOE_BF16) return MOE_ERR_DTYPE;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_grouped_workspace_size(const moe_grouped_shape_t* s, size_t* bytes) {
  if (!s || !bytes) return MOE_ERR_NULL;
  if (int rc = check_grouped(s)) return rc;
  *bytes = workspace_need(s);
  return MOE_OK;
}

int moe_grouped_matmul(const moe_grouped_shape_t* s, const void* x, const int32_t* row_ids, const int32_t* offsets,
                       const int32_t* counts, const void* w, void* y, void* workspace, size_t ws_bytes,
                       void* stream) {
  if (int rc = check_grouped(s)) return rc;
  if (s->x_dtype == MOE_I8) return MOE_ERR_DTYPE;
  return forward(s, x, nullptr, row_ids, offsets, counts, w, nullptr, y, workspace, ws_bytes, stream);
}

int moe_grouped_matmul_i8(const moe_grouped_shape_t* s, const int8_t* xq, const float* x_scale,
                          const int32_t* row_ids, const int32_t* offsets, const int32_t* counts, const int8_t* wq,
                          const float* w_scale, void* y, void* workspace, size_t ws_bytes, void* stream) {
  if (int rc = check_grouped(s)) return rc;
  if (s->x_dtype != MOE_I8) return MOE_ERR_DTYPE;
  return forward(s, xq, x_scale, row_ids, offsets, counts, wq, w_scale, y, workspace, ws_bytes, stream);
}

int moe_grouped_matmul_backward(const moe_grouped_shape_t* s, const void* dy, const void* x, const int32_t* row_ids,
                                const int32_t* offsets, const int32_t* counts, const void* w, void* dx, void* dw,
                                void* workspace, size_t ws_bytes, void* stream) {
  if (int rc = check_grouped(s)) return rc;
  if (s->x_dtype == MOE_I8) return MOE_ERR_DTYPE;
  if (s->rows == 0 && !dw) return MOE_OK;       // dx is empty
  if (!dx && !dw) return MOE_ERR_NULL;
  if (dw && !lookup_ok(s, row_ids)) return MOE_ERR_SHAPE;
  if (!offsets || (s->rows > 0 && dx && !w) || (s->rows > 0 && (!dy || (dw && !x && s->x_rows > 0)))) return MOE_ERR_NULL;
  const size_t need = workspace_need(s);
  if (need > 0 && !workspace) return MOE_ERR_NULL;
  if (int rc = check_aligned(dy, x, row_ids, offsets, counts, w, dx, dw, workspace)) return rc;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  moe::GroupedArgs a = grouped_args(s);
  a.x = x; a.dy = dy; a.w = w; a.offsets = offsets; a.counts = counts; a.row_ids = row_ids;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (dx) {
    a.out = dx;
    if (int rc = status(moe::launch_grouped(a, moe::GM_GRAD_X, s->x_dtype, s->x_dtype, workspace, st))) return rc;
  }
  if (dw) {
    a.out = dw;
    if (int rc = status(moe::launch_grouped(a, moe::GM_GRAD_W, s->x_dtype, s->out_dtype, workspace, st))) return rc;
  }
  return MOE_OK;
}

int moe_quantize_rows(int32_t rows, int32_t cols, int32_t x_dtype, const void* x, int8_t* q, float* scale,
                      void* stream) {
  if (!dim_ok(rows, 0, kMaxRows) || !dim_ok(cols, 1, kMaxDim)) return MOE_ERR_SHAPE;
  if (x_dtype != MOE_F32 && x_dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scale) return MOE_ERR_NULL;
  if (int rc = check_aligned(x, q, scale)) return rc;
  const moe::QuantArgs a{x, q, scale, rows, cols};
  return status(moe::launch_quantize_rows(a, x_dtype, static_cast<hipStream_t>(stream)));
}

int moe_combine(const moe_combine_shape_t* s, const void* y, const int32_t* inv, const float* weights, void* out,
                void* stream) {
  if (int rc = check_combine(s)) return rc;
  if (s->T == 0) return MOE_OK;
  if (!inv || !out || (!y && s->rows > 0)) return MOE_ERR_NULL;
  if (int rc = check_aligned(y, inv, weights, out)) return rc;
  moe::CombineArgs a{};
  a.y = y; a.inv = inv; a.weights = weights; a.out = out;
  a.T = s->T; a.k = s->top_k; a.H = s->H; a.rows = s->rows;
  return status(moe::launch_combine(a, s->y_dtype, s->out_dtype, static_cast<hipStream_t>(stream)));
}

int moe_combine_backward(const moe_combine_shape_t* s, const void* dout, const void* y, const int32_t* inv,
                         const float* weights, void* dy, float* dweights, void* stream) {
  if (int rc = check_combine(s)) return rc;
  if (s->T == 0 || (s->rows == 0 && !dweights)) return MOE_OK;   // no gradient, or an empty dy
  if (!dy && !dweights) return MOE_ERR_NULL;
  if (!inv || !dout || (dweights && !y && s->rows > 0)) return MOE_ERR_NULL;
  if (int rc = check_aligned(dout, y, inv, weights, dy, dweights)) return rc;
  moe::CombineArgs a{};
  a.y = y; a.dout = dout; a.inv = inv; a.weights = weights; a.out = dy; a.dweights = dweights;
  a.T = s->T; a.k = s->top_k; a.H = s->H; a.rows = s->rows;
  return status(moe::launch_combine_backward(a, s->y_dtype, s->out_dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
