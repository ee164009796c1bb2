// Argument blocks and device helpers of the separate operators: the grouped
// expert products (grouped.hip) and the row operators (rows.hip).
#pragma once

#include "common.hpp"

namespace moe {

enum : int { DT_I8 = 5 };                       // MOE_I8
enum : int { GM_FORWARD = 0, GM_GRAD_X = 1, GM_GRAD_W = 2 };   // which product

struct GroupedArgs {
  const void* x;            // [x_rows, K] (forward, dw)
  const void* dy;           // [rows, N] (dx, dw)
  const void* w;            // [E, N, K] (forward, dx)
  void* out;                // y [rows, N], dx [rows, K] or dw [E, N, K]
  const int32_t* row_ids;   // [rows] or null
  const int32_t* offsets;   // [E + 1], or [E] with counts
  const int32_t* counts;    // [E] or null
  const float* x_scale;     // 8-bit: [x_rows]
  const float* w_scale;     // 8-bit: [E, N]
  int rows, N, K, E, x_rows, row_div;
};

// Expert e's segment [begin, begin + n) cut to [0, rows): whatever the tables
// hold, no row outside the buffers is touched.
struct Segment { int begin, n; };
__device__ __forceinline__ Segment segment_of(const GroupedArgs& a, int e) {
  const long b0 = a.offsets[e];
  const long n0 = a.counts ? long(a.counts[e]) : long(a.offsets[e + 1]) - b0;
  const long lo = b0 < 0 ? 0 : (b0 > a.rows ? a.rows : b0);
  const long end = b0 + (n0 < 0 ? 0 : n0);
  const long hi = end < lo ? lo : (end > a.rows ? a.rows : end);
  return Segment{int(lo), int(hi - lo)};
}

// Row of x that sorted row r reads, or -1 for a row of zeros.
__device__ __forceinline__ int source_row(const GroupedArgs& a, int r) {
  if (!a.row_ids) return r;
  const int id = a.row_ids[r];
  const int s = id / a.row_div;
  return id >= 0 && s < a.x_rows ? s : -1;
}

// Row tile `idx` of the list that holds ceil(n / tile) tiles for each
// expert's segment, in order: found by every wave for itself, four experts a
// lane, with a prefix sum over the lanes.  False past the end of the list.
struct RowTile {
  int e;         // expert
  int begin;     // first sorted row of the tile
  int n;         // rows from there to the end of the segment
  int in_seg;    // tile number within the segment
  int seg_n;     // rows of the whole segment
};
__device__ __forceinline__ bool find_row_tile(const GroupedArgs& a, long idx, int tile, RowTile& out) {
  const int lane = threadIdx.x & 63;
  Segment s[4];
  int t[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * lane + i;
    s[i] = e < a.E ? segment_of(a, e) : Segment{0, 0};
    t[i] = (s[i].n + tile - 1) / tile;
    sum += t[i];
  }
  long incl = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long v = __shfl_up(incl, d);
    if (lane >= d) incl += v;
  }
  const long first = incl - sum;
  const unsigned long long m = __ballot(first <= idx && idx < incl);
  if (m == 0) return false;
  const int src = __ffsll(m) - 1;
  int rem = int(idx - first), e = 4 * lane, begin = 0, n = 0;
  bool found = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (!found && rem < t[i]) {
      found = true;
      e = 4 * lane + i;
      begin = s[i].begin;
      n = s[i].n;
    } else if (!found) {
      rem -= t[i];
    }
  }
  auto bcast = [&](int v) { return __builtin_amdgcn_readfirstlane(__shfl(v, src)); };
  out.e = bcast(e);
  out.in_seg = bcast(rem);
  out.seg_n = bcast(n);
  out.begin = bcast(begin) + out.in_seg * tile;
  out.n = out.seg_n - out.in_seg * tile;
  return true;
}

struct QuantArgs {
  const void* x;
  int8_t* q;
  float* scale;
  int rows, cols;
};

struct CombineArgs {
  const void* y;            // [rows, H]
  const void* dout;         // [T, H] (gradients)
  const int32_t* inv;       // [T, k]
  const float* weights;     // [T, k] or null
  void* out;                // out [T, H] or dy [rows, H] (null: not formed)
  float* dweights;          // [T, k] or null
  int T, k, H, rows;
};

hipError_t launch_grouped(const GroupedArgs& a, int which, int in_dt, int out_dt, void* ws, hipStream_t st);
size_t grouped_workspace(const GroupedArgs& a, int which, int in_dt, int out_dt);
hipError_t launch_quantize_rows(const QuantArgs& a, int dt, hipStream_t st);
hipError_t launch_combine(const CombineArgs& a, int y_dt, int out_dt, hipStream_t st);
hipError_t launch_combine_backward(const CombineArgs& a, int y_dt, int out_dt, hipStream_t st);

}  // namespace moe
