// Grouped expert products: one launch over the ragged segments of an
// expert-sorted order, in the three directions of a linear layer,
//   forward  y[r, n]     = sum_k x[row(r), k] w[e, n, k]
//   dx       dx[r, k]    = sum_n dy[r, n] w[e, n, k]
//   dw       dw[e, n, k] = sum_{r of e} dy[r, n] x[row(r), k]
// All three are C[m, n] = sum_q A(m, q) B(n, q) over MFMA tiles, m along the
// lanes' register rows and n, the contiguous direction of the output, along
// the lanes.  An operand either has its reduction index q contiguous in
// memory (x and w forward, dy for dx) or its output index (w for dx, both
// operands of dw); the second kind is staged as it lies and transposed on
// its way from LDS into registers.
#include <algorithm>
#include <type_traits>

#include "grouped.hpp"

namespace moe {

namespace {

// ------------------------------------------------- any size and alignment --
// Tiles of TILE x TILE, four waves in 2 x 2, 16384 / TILE bytes of q per stage
// for an operand that is contiguous along q and as many rows of q otherwise.
// The next stage's loads run while the present one is multiplied; they go
// through registers, where ends of rows are filled with zeros.  That chain of
// load, store to LDS, barrier and read bounds it, 2-4 us a stage: 333 tokens,
// top 3 of 7 fp32 experts of 1003 x 515 32.5 us; both gradients of 201 tokens,
// top 2 of 9 bf16 experts of 611 x 417 28.5 us.
constexpr int ATHREADS = 256;

template <int DT, int TILE>
struct Any {
  static constexpr int B = int(sizeof(typename Elem<DT>::type));
  static constexpr int STAGE = 16384 / TILE;              // bytes of q per stage
  static constexpr int Q = STAGE / B;                     // values
  // LDS row strides in bytes; the pads spread the rows of one read over the banks
  static constexpr int QROW = STAGE + 16;                 // q-contiguous: TILE rows
  static constexpr int MROW = TILE * B + 32;              // else: Q rows
  static constexpr int bytes(bool qc) { return qc ? TILE * QROW : Q * MROW; }
};

// One operand of the tile in LDS: 16 bytes of q (see mma16) for its 32 rows
// at `base` of k-step ks.
template <int DT, int TILE, bool QC>
__device__ __forceinline__ u32x4_t any_read(const uint8_t* s, int base, int ks) {
  constexpr int QROW = Any<DT, TILE>::QROW, MROW = Any<DT, TILE>::MROW;
  const int lane = threadIdx.x & 63, l32 = lane & 31, hi = lane >> 5;
  if constexpr (QC) {
    return *reinterpret_cast<const u32x4_t*>(s + (base + l32) * QROW + (2 * ks + hi) * 16);
  } else if constexpr (DT == DT_F32) {
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = *reinterpret_cast<const uint32_t*>(s + ((2 * ks + hi) * 4 + j) * MROW + (base + l32) * 4);
    return v;
  } else {
    // The transposing read hands the 16 lanes of a group a 4 x 16 block: lane
    // i gives the address of row i / 4, columns 4 (i % 4) .. +3, and receives
    // column i of the four rows.  Group g of the wave: columns 16 (g % 2),
    // rows of q 8 (g / 2) and on.
    static_assert(DT == DT_BF16, "transposed operands are fp32 or bf16");
    const int i = lane & 15, g = lane >> 4;
    const uint8_t* p = s + (ks * 16 + 8 * (g >> 1) + (i >> 2)) * MROW + (base + 16 * (g & 1) + 4 * (i & 3)) * 2;
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p));
    const s16x4_t up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * MROW));
    const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, up);
    return u32x4_t{a[0], a[1], b[0], b[1]};
  }
}

template <int DT, int OUT, int WHICH, int TILE>
__global__ void __launch_bounds__(ATHREADS) grouped_any_kernel(GroupedArgs a) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<DT>::acc Acc;
  typedef Any<DT, TILE> L;
  constexpr int C = 16 / int(sizeof(T));         // elements per 16-byte chunk
  constexpr int Q = L::Q, AT = TILE, MROW = L::MROW;
  constexpr int CPQ = L::STAGE / 16;             // chunks of a q-contiguous row
  constexpr int NB = TILE / 64;                  // 32 x 32 blocks of a wave along m and n
  constexpr bool AQ = WHICH != GM_GRAD_W;        // operand A contiguous along q
  constexpr bool BQ = WHICH == GM_FORWARD;
  __shared__ __attribute__((aligned(16))) uint8_t sa[L::bytes(AQ)];
  __shared__ __attribute__((aligned(16))) uint8_t sb[L::bytes(BQ)];
  __shared__ float row_scale[AT];

  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int wm = (wv >> 1) * (TILE / 2), wn = (wv & 1) * (TILE / 2);
  const int n_cols = WHICH == GM_FORWARD ? a.N : a.K;            // extent along n
  const int n_ct = (n_cols + AT - 1) / AT;
  const int n_mt = (a.N + AT - 1) / AT;                          // dw: tiles along m

  const RowTiles tiles(a, AT);
  const long n_tiles = n_ct * (WHICH == GM_GRAD_W ? long(a.E) * n_mt : long(tiles.total));
  for (long item = blockIdx.x; item < n_tiles * a.max_parts; item += gridDim.x) {
    const int part = int(item / n_tiles);         // each tile's reduction is cut into max_parts parts
    const long tile = item - part * n_tiles;
    int e, m0 = 0, m_end, row0 = 0, n_q;          // tile rows m0 .. m_end - 1; dw: first sorted row; extent of q
    const int n0 = int(tile % n_ct) * AT;
    if constexpr (WHICH == GM_GRAD_W) {
      const long r = tile / n_ct;
      m0 = int(r % n_mt) * AT;
      m_end = min(m0 + AT, a.N);
      e = int(r / n_mt);
      const Segment s = segment_of(a, e);
      row0 = s.begin;
      n_q = s.n;
    } else {
      const RowTile rt = tiles.at(int(tile / n_ct), AT);
      e = rt.e;
      m0 = rt.begin;
      m_end = m0 + min(rt.n, AT);
      n_q = WHICH == GM_FORWARD ? a.K : a.N;
    }
    const int stages = (n_q + Q - 1) / Q;
    const int q_begin = int(long(stages) * part / a.max_parts) * Q;
    const int q_end = min(int(long(stages) * (part + 1) / a.max_parts) * Q, n_q);
    const T* const w = reinterpret_cast<const T*>(a.w) + (WHICH == GM_GRAD_W ? 0 : size_t(e) * a.N * a.K);
    const T* const x = reinterpret_cast<const T*>(a.x);
    const T* const dy = reinterpret_cast<const T*>(a.dy);

    // q-contiguous operands: this thread's four rows (null: zeros)
    const T *pa[4], *pb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = tid / CPQ + i * (ATHREADS / CPQ);
      if constexpr (AQ) {
        const int m = m0 + r;
        const int src = m >= m_end ? -1 : (WHICH == GM_FORWARD ? source_row(a, m) : m);
        pa[i] = src < 0 ? nullptr : (WHICH == GM_FORWARD ? x + size_t(src) * a.K : dy + size_t(src) * a.N);
        if (WHICH == GM_FORWARD && tid % CPQ == 0) row_scale[r] = scale_of<DT>(a, src);
      }
      if constexpr (BQ) pb[i] = n0 + r < n_cols ? w + size_t(n0 + r) * a.K : nullptr;
    }
    u32x4_t ra[4], rb[4];
    auto load_q = [&](const T* const(&p)[4], int q0, u32x4_t(&v)[4]) {
      const int q = q0 + (tid % CPQ) * C;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = p[i] ? load_chunk(p[i] + q, n_q - q) : u32x4_t{0, 0, 0, 0};
    };
    constexpr int CPR = AT / C;                   // chunks per row of q
    auto load_m = [&](auto row_ptr, int col0, int cols, int q0, u32x4_t(&v)[4]) {
      const int c = col0 + (tid % CPR) * C;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = q0 + tid / CPR + i * (ATHREADS / CPR);
        const T* p = q < n_q ? row_ptr(q) : nullptr;
        v[i] = p ? load_chunk(p + c, cols - c) : u32x4_t{0, 0, 0, 0};
      }
    };
    auto load = [&](int q0) {
      if constexpr (AQ) load_q(pa, q0, ra);
      else
        load_m([&](int q) {                       // rows that stand for zeros add nothing, whatever dy holds there
          return source_row(a, row0 + q) < 0 ? (const T*)nullptr : dy + size_t(row0 + q) * a.N;
        }, m0, m_end, q0, ra);
      if constexpr (BQ) load_q(pb, q0, rb);
      else if constexpr (WHICH == GM_GRAD_X) load_m([&](int q) { return w + size_t(q) * a.K; }, n0, n_cols, q0, rb);
      else
        load_m([&](int q) {
          const int s = source_row(a, row0 + q);
          return s < 0 ? (const T*)nullptr : x + size_t(s) * a.K;
        }, n0, n_cols, q0, rb);
    };
    auto stage = [&](uint8_t* s, const u32x4_t(&v)[4], bool qc) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint8_t* p = qc ? s + (tid / CPQ + i * (ATHREADS / CPQ)) * L::QROW + (tid % CPQ) * 16
                        : s + (tid / CPR + i * (ATHREADS / CPR)) * MROW + (tid % CPR) * 16;
        *reinterpret_cast<u32x4_t*>(p) = v[i];
      }
    };

    Acc acc[NB][NB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;

    if (q_begin < q_end) load(q_begin);
    for (int q0 = q_begin; q0 < q_end; q0 += Q) {
      __syncthreads();                            // the stage before has been read
      stage(sa, ra, AQ);
      stage(sb, rb, BQ);
      __syncthreads();
      if (q0 + Q < q_end) load(q0 + Q);
#pragma unroll
      for (int ks = 0; ks < L::STAGE / 32; ++ks) {
        u32x4_t fa[NB], fb[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) fa[i] = any_read<DT, TILE, AQ>(sa, wm + 32 * i, ks);
#pragma unroll
        for (int j = 0; j < NB; ++j) fb[j] = any_read<DT, TILE, BQ>(sb, wn + 32 * j, ks);
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j) mma16<DT>(fa[i], fb[j], acc[i][j]);
      }
    }

    // register q of lane l: row 8 (q / 4) + 4 (l / 32) + q % 4, column l % 32
    const int l32 = lane & 31, hi = lane >> 5;
    const size_t out0 = WHICH == GM_GRAD_W ? size_t(e) * a.N * a.K : 0;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int n = n0 + wn + 32 * j + l32;
      if (n >= n_cols) continue;
      const float ws = DT == DT_I8 ? a.w_scale[size_t(e) * a.N + n] : 0.f;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int r = wm + 32 * i + 8 * (q >> 2) + 4 * hi + (q & 3);
          if (m0 + r >= m_end) continue;
          const size_t at = out0 + size_t(m0 + r) * n_cols + n;
          if (a.max_parts > 1) {                  // the sum as it is
            const auto sum = acc[i][j][q];
            a.parts[size_t(part) * a.part_size + at] = __builtin_bit_cast(float, sum);
            continue;
          }
          float v;
          if constexpr (DT == DT_I8) v = is_no_row(row_scale[r]) ? 0.f : float(acc[i][j][q]) * row_scale[r] * ws;
          else v = WHICH == GM_FORWARD && is_no_row(row_scale[r]) ? 0.f : acc[i][j][q];   // rows that stand for zeros
          store_out<OUT>(a.out, at, v);
        }
    }
    __syncthreads();                              // row_scale and the stages are free for the next item
  }
}

// Adds the parts of every output in order.  A work-group per tile of 64 rows
// and 64 columns (rows that belong to no expert keep what they hold); of dw,
// per 4096 values.
template <int DT, int OUT, int WHICH>
__global__ void __launch_bounds__(256) grouped_any_join_kernel(GroupedArgs a) {
  typedef typename std::conditional<DT == DT_I8, int, float>::type V;
  auto sum_at = [&](size_t at) {
    V v = 0;
    for (int p = 0; p < a.max_parts; ++p) v += reinterpret_cast<const V*>(a.parts)[size_t(p) * a.part_size + at];
    return v;
  };
  if constexpr (WHICH == GM_GRAD_W) {
    const size_t n = size_t(a.E) * a.N * a.K;
    for (size_t i = size_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += size_t(gridDim.x) * 256)
      store_out<OUT>(a.out, i, sum_at(i));
  } else {
    const int n_cols = WHICH == GM_FORWARD ? a.N : a.K, n_ct = (n_cols + 63) / 64;
    const RowTiles tiles(a, 64);
    for (long item = blockIdx.x; item < long(tiles.total) * n_ct; item += gridDim.x) {
      const RowTile rt = tiles.at(int(item / n_ct), 64);
      const int n = int(item % n_ct) * 64 + int(threadIdx.x & 63);
      if (n >= n_cols) continue;
      for (int r = threadIdx.x >> 6; r < min(rt.n, 64); r += 4) {
        const size_t at = size_t(rt.begin + r) * n_cols + n;
        const int src = WHICH == GM_FORWARD ? source_row(a, rt.begin + r) : 0;
        float v = float(sum_at(at));
        if constexpr (DT == DT_I8) v = v * (src < 0 ? 0.f : a.x_scale[src]) * a.w_scale[size_t(rt.e) * a.N + n];
        store_out<OUT>(a.out, at, src < 0 ? 0.f : v);
      }
    }
  }
}

// Tiles at most: every segment may end in a part of one.
long any_tiles(const GroupedArgs& a, int which, int tile) {
  const long n_ct = ((which == GM_FORWARD ? a.N : a.K) + tile - 1) / tile;
  return n_ct * (which == GM_GRAD_W ? long(a.E) * ((a.N + tile - 1) / tile)
                                    : long(a.rows) / tile + (a.E < a.rows ? a.E : a.rows));
}

// Small tiles until the large ones fill the CUs twice (999 rows of 515 fp32
// values by 1003 columns: 80 large tiles 49 us, 288 small ones 32).  Fewer
// small tiles than CUs are cut along the reduction, as long as each part has
// four stages at least, and a second kernel adds the parts.
struct AnyPlan { int tile, parts; size_t part_size; };
AnyPlan any_plan(const GroupedArgs& a, int which, int in_dt) {
  AnyPlan p{any_tiles(a, which, 128) < 512 ? 64 : 128, 1, 0};
  const long tiles = any_tiles(a, which, 64);
  if (p.tile == 128 || tiles >= 256) return p;
  const long n_q = which == GM_FORWARD ? a.K : (which == GM_GRAD_X ? a.N : a.rows);
  const long stage = 256 / (in_dt == DT_F32 ? 4 : (in_dt == DT_BF16 ? 2 : 1));
  const long parts = std::min(512 / std::max(tiles, 1L), (n_q + stage - 1) / stage / 4);
  if (parts < 2) return p;
  p.parts = int(parts);
  p.part_size = which == GM_GRAD_W ? size_t(a.E) * a.N * a.K : size_t(a.rows) * (which == GM_FORWARD ? a.N : a.K);
  return p;
}

template <int DT, int OUT, int WHICH>
hipError_t launch_any(const GroupedArgs& args, void* ws, hipStream_t st) {
  GroupedArgs a = args;
  const AnyPlan p = any_plan(a, WHICH, DT);
  a.parts = reinterpret_cast<float*>(ws);
  a.max_parts = p.parts;
  a.part_size = p.part_size;
  const dim3 grid(unsigned(std::min(any_tiles(a, WHICH, p.tile) * p.parts, 1L << 22)));
  if (p.tile == 64) hipLaunchKernelGGL((grouped_any_kernel<DT, OUT, WHICH, 64>), grid, dim3(ATHREADS), 0, st, a);
  else hipLaunchKernelGGL((grouped_any_kernel<DT, OUT, WHICH, 128>), grid, dim3(ATHREADS), 0, st, a);
  if (p.parts > 1) {
    const long n = WHICH == GM_GRAD_W ? long((p.part_size + 4095) / 4096) : any_tiles(a, WHICH, 64);
    hipLaunchKernelGGL((grouped_any_join_kernel<DT, OUT, WHICH>), dim3(unsigned(n)), dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace

namespace {
enum class Kind { stream, tile, any };
// Which kernels a shape takes.  A few rows an expert: the stream of weights
// (64 experts of 1408 x 2048 in bf16, 6 rows each 86 us against 95 on large
// tiles, 12 rows 98 against 94; in 8 bits, 12 rows 62 against 66); where the
// large tiles do not fit it pays for longer.
Kind kind_of(const GroupedArgs& a, int which, int in_dt) {
  const bool fits = grouped_tile_fits(a, which, in_dt);
  const long few = fits ? (in_dt == DT_I8 ? 12 : 6) : 32;
  if (which == GM_FORWARD && long(a.rows) <= std::max(16L, few * a.E)) return Kind::stream;
  if (!fits) return Kind::any;
  // The large tiles take one CU each; a call that gives them little to do is spread better by the small ones:
  // dw of few large tiles, which has no cuts along the rows there (both gradients of 1024 rows, 4 experts of 768 x 768,
  // 36 tiles: 27 us against 37 on large ones; of 1024 x 1536, 96 tiles: 58 against 48), or one round of short
  // reductions (2048 rows, 16 experts of 1024 x 512: 15 us against 20).
  const long n_cols = which == GM_FORWARD ? a.N : a.K, n_q = which == GM_FORWARD ? a.K : a.N;
  if (which == GM_GRAD_W) return long(a.E) * ((a.N + 255) / 256) * ((a.K + 255) / 256) < 64 ? Kind::any : Kind::tile;
  const long tiles = (long(a.rows) / 256 + std::min(a.E, a.rows)) * ((n_cols + 255) / 256);
  return tiles <= 256 && n_q * (in_dt == DT_I8 ? 1 : 2) < 16 * 128 ? Kind::any : Kind::tile;
}
}  // namespace

size_t grouped_workspace(const GroupedArgs& a, int which, int in_dt, int) {
  switch (kind_of(a, which, in_dt)) {
    case Kind::tile: return grouped_tile_workspace(a, which, in_dt);
    case Kind::any: {
      const AnyPlan p = any_plan(a, which, in_dt);
      return p.parts > 1 ? p.parts * p.part_size * 4 : 0;
    }
    default: return 0;
  }
}

hipError_t launch_grouped(const GroupedArgs& a, int which, int in_dt, int out_dt, void* ws, hipStream_t st) {
  if (which != GM_GRAD_W && a.rows == 0) return hipSuccess;
  switch (kind_of(a, which, in_dt)) {
    case Kind::stream: return launch_grouped_stream(a, in_dt, out_dt, st);
    case Kind::tile: return launch_grouped_tile(a, which, in_dt, out_dt, ws, st);
    default: break;
  }
  if (in_dt == DT_I8)
    return out_dt == DT_F32 ? launch_any<DT_I8, DT_F32, GM_FORWARD>(a, ws, st)
                            : launch_any<DT_I8, DT_BF16, GM_FORWARD>(a, ws, st);
  if (which == GM_FORWARD) {
    if (in_dt == DT_F32) return launch_any<DT_F32, DT_F32, GM_FORWARD>(a, ws, st);
    return out_dt == DT_F32 ? launch_any<DT_BF16, DT_F32, GM_FORWARD>(a, ws, st)
                            : launch_any<DT_BF16, DT_BF16, GM_FORWARD>(a, ws, st);
  }
  if (which == GM_GRAD_X)
    return in_dt == DT_F32 ? launch_any<DT_F32, DT_F32, GM_GRAD_X>(a, ws, st)
                           : launch_any<DT_BF16, DT_BF16, GM_GRAD_X>(a, ws, st);
  if (in_dt == DT_F32) return launch_any<DT_F32, DT_F32, GM_GRAD_W>(a, ws, st);
  return out_dt == DT_F32 ? launch_any<DT_BF16, DT_F32, GM_GRAD_W>(a, ws, st)
                          : launch_any<DT_BF16, DT_BF16, GM_GRAD_W>(a, ws, st);
}

}  // namespace moe
