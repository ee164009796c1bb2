// Argument blocks and device helpers of the separate operators: the grouped
// expert products (grouped.hip) and the row operators (rows.hip).
#pragma once

#include "common.hpp"

namespace moe {

enum : int { DT_I8 = 5 };                       // MOE_I8
enum : int { GM_FORWARD = 0, GM_GRAD_X = 1, GM_GRAD_W = 2 };   // which product

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

// Element types: how they lie in memory and what their products are summed in.
template <int DT> struct Elem;
template <> struct Elem<DT_F32> { typedef float type; typedef f32x16_t acc; };
template <> struct Elem<DT_BF16> { typedef uint16_t type; typedef f32x16_t acc; };
template <> struct Elem<DT_I8> { typedef int8_t type; typedef i32x16_t acc; };

__device__ __forceinline__ i32x16_t mfma32_i8(u32x4_t a, u32x4_t b, i32x16_t c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0,
                                               0, 0);
}

// acc += A x B over the values of q that 16 bytes a lane hold: lanes 0-31 the
// first 16 bytes of each row, lanes 32-63 the next.  fp32 takes four MFMAs of
// two values of q each.
template <int DT, class Acc>
__device__ __forceinline__ void mma16(u32x4_t a, u32x4_t b, Acc& c) {
  if constexpr (DT == DT_BF16) c = mfma32_bf16(a, b, c);
  else if constexpr (DT == DT_I8) c = mfma32_i8(a, b, c);
  else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[j]), __uint_as_float(b[j]), c, 0, 0, 0);
  }
}

// Two floats to bf16, to nearest even, by the hardware's conversion.
__device__ __forceinline__ uint32_t cvt_pk_bf16(float lo, float hi) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}

template <int OUT>
__device__ __forceinline__ void store_out(void* out, size_t i, float v) {
  if constexpr (OUT == DT_F32) reinterpret_cast<float*>(out)[i] = v;
  else reinterpret_cast<uint16_t*>(out)[i] = uint16_t(f32_to_bf16(v));
}

// 16 bytes from p, which needs the alignment of its elements only.
template <class T>
__device__ __forceinline__ u32x4_t load16(const T* p) {
  struct __attribute__((packed, aligned(sizeof(T)))) U { u32x4_t v; };
  return reinterpret_cast<const U*>(p)->v;
}
// Up to 16 bytes from p, which need not be aligned: the first n elements (all
// of a chunk's, or fewer at the end of a row), the others zero.
template <class T>
__device__ __forceinline__ u32x4_t load_chunk(const T* p, int n) {
  constexpr int C = 16 / sizeof(T);
  if (n >= C) return load16(p);
  u32x4_t v = {0, 0, 0, 0};
  if (n <= 0) return v;
  constexpr int PW = 4 / sizeof(T);             // elements per word
#pragma unroll
  for (int i = 0; i < C; ++i)
    if (i < n) {
      uint32_t b;
      if constexpr (sizeof(T) == 4) b = __float_as_uint(p[i]);
      else if constexpr (sizeof(T) == 2) b = uint32_t(p[i]);
      else b = uint32_t(uint8_t(p[i]));
      v[i / PW] |= b << ((i % PW) * 8 * int(sizeof(T)));
    }
  return v;
}

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
  const uint64_t* row_table;   // dw on large tiles: addresses of the rows of x in sorted order (workspace)
  float* parts;             // sums of tiles that are cut along the reduction (workspace)
  int max_parts;            // ... the most parts of a tile (large tiles), or the parts of every tile
  size_t part_size;         // ... values between the parts of a tile (the other kernel)
  int rows, N, K, E, x_rows, row_div;
  unsigned div_mul;         // n / row_div = mulhi(2 n, div_mul) >> div_shift for 0 <= n < 2^31
  int div_shift;
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

// Row of x that an entry of row_ids stands for, or -1 for a row of zeros.
__device__ __forceinline__ int source_of(const GroupedArgs& a, int id) {
  const int s = int(__umulhi(unsigned(id) << 1, a.div_mul) >> a.div_shift);
  return ((id >= 0) & (s < a.x_rows)) ? s : -1;
}

// Row of x that sorted row r reads, or -1.
__device__ __forceinline__ int source_row(const GroupedArgs& a, int r) {
  if (!a.row_ids) return r;
  return source_of(a, a.row_ids[r]);
}

// Scale of row src of x: x_scale (8-bit) or 1.  A row of zeros (src < 0) has
// -0 (no scale is passed on as -0): its product is 0 whatever w_scale holds.
template <int DT>
__device__ __forceinline__ float scale_of(const GroupedArgs& a, int src) {
  if (src < 0) return -0.f;
  if constexpr (DT != DT_I8) return 1.f;
  const uint32_t s = __float_as_uint(a.x_scale[src]);
  return __uint_as_float(s == 0x80000000u ? 0u : s);
}
__device__ __forceinline__ bool is_no_row(float scale) { return __float_as_uint(scale) == 0x80000000u; }

// The list that holds ceil(n / tile) row tiles for each expert's segment, in
// order.  Every wave looks it up for itself: four experts a lane, with a
// prefix sum over the lanes.
struct RowTile {
  int e;         // expert
  int begin;     // first sorted row of the tile
  int n;         // rows from there to the end of the segment
};
struct RowTiles {
  Segment s[4];  // segments of experts 4 lane .. 4 lane + 3
  int t[4];      // their tiles
  int first;     // tiles before them
  int sum;       // their sum
  int total;     // tiles of all experts

  __device__ __forceinline__ RowTiles(const GroupedArgs& a, int tile) {
    const int lane = threadIdx.x & 63;
    sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      s[i] = e < a.E ? segment_of(a, e) : Segment{0, 0};
      t[i] = (s[i].n + tile - 1) / tile;
      sum += t[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
    first = incl - sum;
    total = __builtin_amdgcn_readfirstlane(__shfl(incl, 63));
  }

  // Tile idx, 0 <= idx < total.
  __device__ __forceinline__ RowTile at(int idx, int tile) const {
    const int lane = threadIdx.x & 63;
    const int src = __ffsll(__ballot(first <= idx && idx < first + sum)) - 1;
    int rem = idx - first, e = 4 * lane, begin = 0, n = 0;
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
    const int done = bcast(rem) * tile;
    return RowTile{bcast(e), bcast(begin) + done, bcast(n) - done};
  }
};

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

// Few rows an expert, forward only (grouped_stream.hip).
hipError_t launch_grouped_stream(const GroupedArgs& a, int in_dt, int out_dt, hipStream_t st);
// Large tiles (grouped_tile.hip): which shapes they take, and their launch.
bool grouped_tile_fits(const GroupedArgs& a, int which, int in_dt);
size_t grouped_tile_workspace(const GroupedArgs& a, int which, int in_dt);
hipError_t launch_grouped_tile(const GroupedArgs& a, int which, int in_dt, int out_dt, void* ws, hipStream_t st);

hipError_t launch_grouped(const GroupedArgs& a, int which, int in_dt, int out_dt, void* ws, hipStream_t st);
size_t grouped_workspace(const GroupedArgs& a, int which, int in_dt, int out_dt);
hipError_t launch_quantize_rows(const QuantArgs& a, int dt, hipStream_t st);
hipError_t launch_combine(const CombineArgs& a, int y_dt, int out_dt, hipStream_t st);
hipError_t launch_combine_backward(const CombineArgs& a, int y_dt, int out_dt, hipStream_t st);

}  // namespace moe
