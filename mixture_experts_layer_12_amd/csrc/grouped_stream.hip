// Grouped expert products for few rows an expert (decode): a stream of weights.
// The forward product only: y[r, n] = sum_k x[row(r), k] w[e, n, k].
//
// What bounds it is reading each engaged expert's weights once, so nothing is
// staged: a wave loads 16 weight rows x 64 bytes of k straight into registers
// as one MFMA operand (lane l: row l % 16, 16 bytes at 16 (l / 16)) and the
// same bytes of up to 16 rows of x, which come from L2, as the other one.
// The waves of a work-group share 16 R weight rows and cut K between them, so
// that many loads are in flight for every row even when there are few tiles;
// their partial sums meet in LDS and are added in a fixed order.  A segment is
// taken 32 rows at a time (C = 1 or 2 column tiles of 16 rows): with more, the
// registers would leave room for too few waves to keep HBM busy.
// Rows of any alignment: 16-byte loads need none here.
// Measured, with cold weights: 64 tokens, top 6 of 64 experts of 1408 x 2048 in
// bf16 82 us (4.5 TB/s), in 8 bits 49; one token through 8 experts of 512 x 2048
// 8 us, what a bare read of those 17 MB takes.
#include <algorithm>
#include <type_traits>

#include "grouped.hpp"

namespace moe {

namespace {

constexpr int GS_ROWS = 32;              // sorted rows per item
// 16-byte loads that a lane has under way: more take registers from waves (eight tokens through 8 experts of
// 14336 x 4096: 12 loads 172 us, 18 175, 24 182)
constexpr int GS_LOADS = 12;

template <int DT> struct Small;
template <> struct Small<DT_F32> { typedef f32x4_t acc; };
template <> struct Small<DT_BF16> { typedef f32x4_t acc; };
template <> struct Small<DT_I8> { typedef i32x4_t acc; };

// One k-step of 64 bytes: acc (row 4 (l / 16) + i of the weights, column l % 16 of x) += w x.
template <int DT, class Acc>
__device__ __forceinline__ void mma16x16(u32x4_t w, u32x4_t x, Acc& c) {
  if constexpr (DT == DT_BF16) c = mfma_bf16(w, x, c);
  else if constexpr (DT == DT_I8)
    c = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, w), __builtin_bit_cast(i32x4_t, x), c, 0, 0, 0);
  else {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = mfma_f32(__uint_as_float(w[j]), __uint_as_float(x[j]), c);
  }
}

// R x 16 weight rows from n0, C x 16 rows of x; wave `wv` of W takes its share of K.
template <int DT, int OUT, int R, int C, int W>
__device__ __forceinline__ void stream_tile(const GroupedArgs& a, float* smem, int e, int row0, int rows, int n0) {
  typedef typename Elem<DT>::type T;
  typedef typename Small<DT>::acc Acc;
  constexpr int E16 = 16 / int(sizeof(T));                     // values per 16 bytes
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int l16 = lane & 15, g = lane >> 4;
  const T* const w = reinterpret_cast<const T*>(a.w) + size_t(e) * a.N * a.K;
  // rows of x that are not there read the weights: their sums are not stored (or replaced by zeros)
  const T* px[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int m = 16 * c + l16;
    const int src = m < rows ? source_row(a, row0 + m) : -1;
    px[c] = (src < 0 ? w : reinterpret_cast<const T*>(a.x) + size_t(src) * a.K) + g * E16;
  }
  const T* pw[R];                                // weight rows past N read the tile's first row
#pragma unroll
  for (int r = 0; r < R; ++r) pw[r] = w + size_t(n0 + 16 * r + l16 < a.N ? n0 + 16 * r + l16 : n0) * a.K + g * E16;
  Acc acc[R][C];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][c][i] = 0;

  constexpr int S = 4 * E16;                                   // values per k-step
  const int full = a.K / S;                                    // whole k-steps
  const int s_begin = int(long(full) * wv / W), s_end = int(long(full) * (wv + 1) / W);
  // groups of U k-steps, whose loads are all under way before the first product; in the last group the loads
  // past the end repeat the last step, and their products are left out
  constexpr int U = GS_LOADS / (R + C) < 8 ? GS_LOADS / (R + C) : 8;
  auto group = [&](int s, auto whole) {
    u32x4_t fw[U][R], fx[U][C];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const size_t at = size_t(decltype(whole)::value ? s + u : min(s + u, s_end - 1)) * S;
#pragma unroll
      for (int r = 0; r < R; ++r) fw[u][r] = load16(pw[r] + at);
#pragma unroll
      for (int c = 0; c < C; ++c) fx[u][c] = load16(px[c] + at);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (decltype(whole)::value || s + u < s_end) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int c = 0; c < C; ++c) mma16x16<DT>(fw[u][r], fx[u][c], acc[r][c]);
      }
  };
  int s = s_begin;
  for (; s + U <= s_end; s += U) group(s, std::true_type{});
  if (s < s_end) group(s, std::false_type{});
  if (wv == W - 1 && full * S < a.K) {                         // the end of the rows, past the last whole step
    const int left = a.K - full * S - g * E16;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const u32x4_t fw = load_chunk(pw[r] + size_t(full) * S, left);
#pragma unroll
      for (int c = 0; c < C; ++c) mma16x16<DT>(fw, load_chunk(px[c] + size_t(full) * S, left), acc[r][c]);
    }
  }

  // sums of the waves, in the order of the waves
  Acc* const part = reinterpret_cast<Acc*>(smem);              // [W][R * C][64]
  __syncthreads();                                             // the item before has been read
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < C; ++c) part[(wv * R * C + r * C + c) * 64 + lane] = acc[r][c];
  __syncthreads();
  for (int f = wv; f < R * C; f += W) {
    const int r = f / C, c = f % C;
    Acc v = part[f * 64 + lane];
#pragma unroll
    for (int q = 1; q < W; ++q) v += part[(q * R * C + f) * 64 + lane];
    const int m = 16 * c + l16, n = n0 + 16 * r + 4 * g;
    if (m >= rows || n >= a.N) continue;
    const int src = source_row(a, row0 + m);
    float o[4];
    if constexpr (DT == DT_I8) {
      const float xs = src < 0 ? 0.f : a.x_scale[src];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = n + i < a.N ? float(v[i]) * xs * a.w_scale[size_t(e) * a.N + n + i] : 0.f;
      if (src < 0) o[0] = o[1] = o[2] = o[3] = 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = src < 0 ? 0.f : v[i];
    }
    const size_t at = size_t(row0 + m) * a.N + n;
    if (a.N % 4 == 0) {
      if constexpr (OUT == DT_F32) *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(a.out) + at) = f32x4_t{o[0], o[1], o[2], o[3]};
      else
        *reinterpret_cast<u32x2_t*>(reinterpret_cast<uint16_t*>(a.out) + at) =
            u32x2_t{cvt_pk_bf16(o[0], o[1]), cvt_pk_bf16(o[2], o[3])};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < a.N) store_out<OUT>(a.out, at + i, o[i]);
    }
  }
}

// A work-group per (row tile, column tile) item, columns inner, dispatched as
// CUs fall free (resident ones with a fixed share of the items: 215 us for
// eight tokens through 8 experts of 14336 x 4096, against 183).
template <int DT, int OUT, int R, int W>
__global__ void __launch_bounds__(64 * W) grouped_stream_kernel(GroupedArgs a) {
  __shared__ __attribute__((aligned(16))) float smem[W * R * (GS_ROWS / 16) * 64 * 4];
  const int n_ct = (a.N + 16 * R - 1) / (16 * R);
  for (long item = blockIdx.x;; item += gridDim.x) {
    const RowTiles tiles(a, GS_ROWS);
    if (item >= long(tiles.total) * n_ct) return;
    const RowTile rt = tiles.at(int(item / n_ct), GS_ROWS);
    const int rows = min(rt.n, GS_ROWS), n0 = int(item % n_ct) * 16 * R;
    if (rows <= 16) stream_tile<DT, OUT, R, 1, W>(a, smem, rt.e, rt.begin, rows, n0);
    else stream_tile<DT, OUT, R, 2, W>(a, smem, rt.e, rt.begin, rows, n0);
  }
}

// Row tiles at most.
long stream_row_tiles(const GroupedArgs& a) { return long(a.rows) / GS_ROWS + std::min(a.E, a.rows); }

template <int DT, int OUT, int R>
hipError_t launch_r(const GroupedArgs& a, hipStream_t st) {
  const long n_items = stream_row_tiles(a) * ((a.N + 16 * R - 1) / (16 * R));
  hipLaunchKernelGGL((grouped_stream_kernel<DT, OUT, R, 4>), dim3(unsigned(std::min(n_items, 1L << 22))), dim3(64 * 4), 0,
                     st, a);
  return hipGetLastError();
}

template <int DT, int OUT>
hipError_t launch_stream(const GroupedArgs& a, hipStream_t st) {
  // Two tiles of weight rows a wave halve the reads of x, once there are work-groups enough without.
  if (stream_row_tiles(a) * ((a.N + 15) / 16) >= 2048) return launch_r<DT, OUT, 2>(a, st);
  return launch_r<DT, OUT, 1>(a, st);
}

}  // namespace

hipError_t launch_grouped_stream(const GroupedArgs& a, int in_dt, int out_dt, hipStream_t st) {
  if (in_dt == DT_F32) return launch_stream<DT_F32, DT_F32>(a, st);
  if (in_dt == DT_I8)
    return out_dt == DT_F32 ? launch_stream<DT_I8, DT_F32>(a, st) : launch_stream<DT_I8, DT_BF16>(a, st);
  return out_dt == DT_F32 ? launch_stream<DT_BF16, DT_F32>(a, st) : launch_stream<DT_BF16, DT_BF16>(a, st);
}

}  // namespace moe
