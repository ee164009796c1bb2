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
#include "grouped.hpp"

namespace moe {

namespace {

// ------------------------------------------------- any size and alignment --
// 128 x 128 tiles, four waves of 64 x 64, 128 bytes of q per stage for an
// operand that is contiguous along q and as many rows of q otherwise.  The
// next stage's loads run while the present one is multiplied; they go through
// registers, where ends of rows are filled with zeros.
constexpr int AT = 128;
constexpr int ATHREADS = 256;

template <int DT> constexpr int kAnyQ = 128 / int(sizeof(typename Elem<DT>::type));   // values of q per stage
// LDS row strides in bytes; the pads spread the rows of one read over the banks
constexpr int kAnyQRow = 128 + 16;                                    // q-contiguous: AT rows
template <int DT> constexpr int kAnyMRow = AT * int(sizeof(typename Elem<DT>::type)) + 32;   // else: kAnyQ rows
template <int DT, bool QC> constexpr int kAnyBytes = QC ? AT * kAnyQRow : kAnyQ<DT>* kAnyMRow<DT>;

// One operand of the tile in LDS: 16 bytes of q (see mma16) for its 32 rows
// at `base` of k-step ks.
template <int DT, bool QC>
__device__ __forceinline__ u32x4_t any_read(const uint8_t* s, int base, int ks) {
  const int lane = threadIdx.x & 63, l32 = lane & 31, hi = lane >> 5;
  if constexpr (QC) {
    return *reinterpret_cast<const u32x4_t*>(s + (base + l32) * kAnyQRow + (2 * ks + hi) * 16);
  } else if constexpr (DT == DT_F32) {
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = *reinterpret_cast<const uint32_t*>(s + ((2 * ks + hi) * 4 + j) * kAnyMRow<DT> + (base + l32) * 4);
    return v;
  } else {
    // The transposing read hands the 16 lanes of a group a 4 x 16 block: lane
    // i gives the address of row i / 4, columns 4 (i % 4) .. +3, and receives
    // column i of the four rows.  Group g of the wave: columns 16 (g % 2),
    // rows of q 8 (g / 2) and on.
    static_assert(DT == DT_BF16, "transposed operands are fp32 or bf16");
    const int i = lane & 15, g = lane >> 4;
    const uint8_t* p = s + (ks * 16 + 8 * (g >> 1) + (i >> 2)) * kAnyMRow<DT> + (base + 16 * (g & 1) + 4 * (i & 3)) * 2;
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p));
    const s16x4_t up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * kAnyMRow<DT>));
    const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, up);
    return u32x4_t{a[0], a[1], b[0], b[1]};
  }
}

template <int DT, int OUT, int WHICH>
__global__ void __launch_bounds__(ATHREADS) grouped_any_kernel(GroupedArgs a, long n_items) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<DT>::acc Acc;
  constexpr int C = 16 / int(sizeof(T));         // elements per 16-byte chunk
  constexpr int Q = kAnyQ<DT>;
  constexpr bool AQ = WHICH != GM_GRAD_W;        // operand A contiguous along q
  constexpr bool BQ = WHICH == GM_FORWARD;
  __shared__ __attribute__((aligned(16))) uint8_t sa[kAnyBytes<DT, AQ>];
  __shared__ __attribute__((aligned(16))) uint8_t sb[kAnyBytes<DT, BQ>];
  __shared__ float row_scale[AT];

  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int wm = (wv >> 1) * 64, wn = (wv & 1) * 64;
  const int n_cols = WHICH == GM_FORWARD ? a.N : a.K;            // extent along n
  const int n_ct = (n_cols + AT - 1) / AT;
  const int n_mt = (a.N + AT - 1) / AT;                          // dw: tiles along m

  RowTiles tiles(a, AT);
  if constexpr (WHICH != GM_GRAD_W) n_items = long(tiles.total) * n_ct;
  for (long item = blockIdx.x; item < n_items; item += gridDim.x) {
    int e, m0 = 0, m_end, row0 = 0, n_q;          // tile rows m0 .. m_end - 1; dw: first sorted row; extent of q
    const int n0 = int(item % n_ct) * AT;
    if constexpr (WHICH == GM_GRAD_W) {
      const long r = item / n_ct;
      m0 = int(r % n_mt) * AT;
      m_end = min(m0 + AT, a.N);
      e = int(r / n_mt);
      const Segment s = segment_of(a, e);
      row0 = s.begin;
      n_q = s.n;
    } else {
      const RowTile rt = tiles.at(int(item / n_ct), AT);
      e = rt.e;
      m0 = rt.begin;
      m_end = m0 + min(rt.n, AT);
      n_q = WHICH == GM_FORWARD ? a.K : a.N;
    }
    const T* const w = reinterpret_cast<const T*>(a.w) + (WHICH == GM_GRAD_W ? 0 : size_t(e) * a.N * a.K);
    const T* const x = reinterpret_cast<const T*>(a.x);
    const T* const dy = reinterpret_cast<const T*>(a.dy);

    // q-contiguous operands: this thread's four rows (null: zeros)
    const T *pa[4], *pb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (tid >> 3) + 32 * i;
      if constexpr (AQ) {
        const int m = m0 + r;
        const int src = m >= m_end ? -1 : (WHICH == GM_FORWARD ? source_row(a, m) : m);
        pa[i] = src < 0 ? nullptr : (WHICH == GM_FORWARD ? x + size_t(src) * a.K : dy + size_t(src) * a.N);
        if (WHICH == GM_FORWARD && (tid & 7) == 0) row_scale[r] = src < 0 ? 0.f : (DT == DT_I8 ? a.x_scale[src] : 1.f);
      }
      if constexpr (BQ) pb[i] = n0 + r < n_cols ? w + size_t(n0 + r) * a.K : nullptr;
    }
    u32x4_t ra[4], rb[4];
    auto load_q = [&](const T* const(&p)[4], int q0, u32x4_t(&v)[4]) {
      const int q = q0 + (tid & 7) * C;
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
      else load_m([&](int q) { return dy + size_t(row0 + q) * a.N; }, m0, m_end, q0, ra);
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
        uint8_t* p = qc ? s + ((tid >> 3) + 32 * i) * kAnyQRow + (tid & 7) * 16
                        : s + (tid / CPR + i * (ATHREADS / CPR)) * kAnyMRow<DT> + (tid % CPR) * 16;
        *reinterpret_cast<u32x4_t*>(p) = v[i];
      }
    };

    Acc acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;

    if (n_q > 0) load(0);
    for (int q0 = 0; q0 < n_q; q0 += Q) {
      __syncthreads();                            // the stage before has been read
      stage(sa, ra, AQ);
      stage(sb, rb, BQ);
      __syncthreads();
      if (q0 + Q < n_q) load(q0 + Q);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        u32x4_t fa[2], fb[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) fa[i] = any_read<DT, AQ>(sa, wm + 32 * i, ks);
#pragma unroll
        for (int j = 0; j < 2; ++j) fb[j] = any_read<DT, BQ>(sb, wn + 32 * j, ks);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) mma16<DT>(fa[i], fb[j], acc[i][j]);
      }
    }

    // register q of lane l: row 8 (q / 4) + 4 (l / 32) + q % 4, column l % 32
    const int l32 = lane & 31, hi = lane >> 5;
    const size_t out0 = WHICH == GM_GRAD_W ? size_t(e) * a.N * a.K : 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = n0 + wn + 32 * j + l32;
      if (n >= n_cols) continue;
      const float ws = DT == DT_I8 ? a.w_scale[size_t(e) * a.N + n] : 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int r = wm + 32 * i + 8 * (q >> 2) + 4 * hi + (q & 3);
          if (m0 + r >= m_end) continue;
          float v;
          if constexpr (DT == DT_I8) v = float(acc[i][j][q]) * row_scale[r] * ws;
          else v = WHICH == GM_FORWARD && row_scale[r] == 0.f ? 0.f : acc[i][j][q];   // rows that stand for zeros
          store_out<OUT>(a.out, out0 + size_t(m0 + r) * n_cols + n, v);
        }
    }
    __syncthreads();                              // row_scale and the stages are free for the next item
  }
}

template <int DT, int OUT, int WHICH>
hipError_t launch_any(const GroupedArgs& a, hipStream_t st) {
  const long n_ct = ((WHICH == GM_FORWARD ? a.N : a.K) + AT - 1) / AT;
  // Row tiles: every segment may end in a part of one.
  const long n_rt = WHICH == GM_GRAD_W ? long(a.E) * ((a.N + AT - 1) / AT) : long(a.rows) / AT + a.E;
  const long n_items = n_rt * n_ct;
  const long grid = n_items < (1L << 22) ? n_items : (1L << 22);
  if (grid == 0) return hipSuccess;
  hipLaunchKernelGGL((grouped_any_kernel<DT, OUT, WHICH>), dim3(unsigned(grid)), dim3(ATHREADS), 0, st, a, n_items);
  return hipGetLastError();
}

}  // namespace

size_t grouped_workspace(const GroupedArgs& a, int which, int in_dt, int) {
  return grouped_tile_workspace(a, which, in_dt);
}

hipError_t launch_grouped(const GroupedArgs& a, int which, int in_dt, int out_dt, void* ws, hipStream_t st) {
  if (which != GM_GRAD_W && a.rows == 0) return hipSuccess;
  // few rows an expert: bound by the weights, which the stream reads at full rate
  if (which == GM_FORWARD && long(a.rows) <= 32L * a.E) return launch_grouped_stream(a, in_dt, out_dt, st);
  if (grouped_tile_fits(a, which, in_dt)) return launch_grouped_tile(a, which, in_dt, out_dt, ws, st);
  if (in_dt == DT_I8)
    return out_dt == DT_F32 ? launch_any<DT_I8, DT_F32, GM_FORWARD>(a, st) : launch_any<DT_I8, DT_BF16, GM_FORWARD>(a, st);
  if (which == GM_FORWARD) {
    if (in_dt == DT_F32) return launch_any<DT_F32, DT_F32, GM_FORWARD>(a, st);
    return out_dt == DT_F32 ? launch_any<DT_BF16, DT_F32, GM_FORWARD>(a, st)
                            : launch_any<DT_BF16, DT_BF16, GM_FORWARD>(a, st);
  }
  if (which == GM_GRAD_X)
    return in_dt == DT_F32 ? launch_any<DT_F32, DT_F32, GM_GRAD_X>(a, st)
                           : launch_any<DT_BF16, DT_BF16, GM_GRAD_X>(a, st);
  if (in_dt == DT_F32) return launch_any<DT_F32, DT_F32, GM_GRAD_W>(a, st);
  return out_dt == DT_F32 ? launch_any<DT_BF16, DT_F32, GM_GRAD_W>(a, st)
                          : launch_any<DT_BF16, DT_BF16, GM_GRAD_W>(a, st);
}

}  // namespace moe
