// Grouped expert products on large MFMA tiles, for bf16 and 8-bit operands
// whose rows are 16-byte aligned.  Same products and notation as grouped.hip:
// C[m, n] = sum_q A(m, q) B(n, q).
//
// A work-group owns a tile of 256 columns n and 256 (128, 64) rows m.  Eight
// waves, two on each SIMD, in 2 x 4: each accumulates 128 x 64 (64 x 64, 32 x
// 64) in 32 x 32 MFMAs held in registers; while one wave of a SIMD waits for
// LDS or at the stage barrier the other one multiplies.
// Operands go global -> LDS with direct-to-LDS loads of 16 bytes a lane, 128
// bytes of q per stage.  An operand that is contiguous along q is staged as
// 256 rows of 128 bytes; one that is contiguous along its output index as 64
// rows of q of 512 bytes, and transposed by the LDS reads.  The ring holds
// three stages of B, the operand that comes from HBM, and two of A, which
// neighbouring work-groups share in L2: after the barrier of stage t the
// loads of A (t + 2) and then of B (t + 3) are issued one by one between the
// MFMAs, and the next barrier waits for all but those last ones (loads
// complete in issue order).
// 16-byte chunks (32-byte pairs of them where reads transpose) are permuted
// within each staged row so that the rows one read touches lie on distinct
// banks.
#include "grouped.hpp"

namespace moe {

namespace {

typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(1))) void glb_void_t;

constexpr int GT_WAVES = 8;
constexpr int GT_N = 256;                       // columns per tile
constexpr int GT_STAGE = 128;                   // bytes of q per stage
constexpr int GT_SLOT = 256 * GT_STAGE;         // bytes of one operand's stage
constexpr int GT_LDS = 5 * GT_SLOT;             // A: slots 0, 1; B: slots 2, 3, 4

// 16 bytes of zeros: what lanes load that lie past the end of an operand.
__device__ const u32x4_t g_zeros = {0, 0, 0, 0};

template <int B, int E, class F>
__device__ __forceinline__ void for_range(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    for_range<B + 1, E>(f);
  }
}

template <int N>
__device__ __forceinline__ void wait_loads() {   // until at most N vector-memory operations are outstanding
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | (0xF << 8) | ((N >> 4) << 14));
}

// Barrier of the ring: this wave's LDS reads are done; loads stay in flight.
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_s_waitcnt((0x3F & 0xF) | (0x7 << 4) | (0x0 << 8) | ((0x3F >> 4) << 14));   // lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
}

// Position of 16-byte chunk c of staged row r: c ^ swz.
__device__ __forceinline__ int swz_q(int r) { return (r & 7) ^ ((r >> 3) & 1); }
__device__ __forceinline__ int swz_m(int r) { return ((r & 3) << 2) | ((r & 8) << 1); }

// This lane's number, computed where it is used: what the compiler derives
// from it (ends of rows, positions of outputs) is then not kept in registers
// through the main loop.
__device__ __forceinline__ int lane_here() {
  int l = int(threadIdx.x & 63);
  asm volatile("" : "+v"(l));
  return l;
}

// Values that the compiler shall take as they are: an address per stage that
// it would otherwise keep in many registers, one for each place it is used.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}
__device__ __forceinline__ const uint8_t* opaque_base(const uint8_t* p) {
  asm volatile("" : "+s"(p));
  return p;
}

// One operand's loads of a wave: LOADS instructions of 1 KiB per stage (8
// rows of 128 bytes, or 2 rows of q of 512).  Lane l of instruction i fills
// 16 bytes of staged row `row`, chunk `chunk` of that row in memory.
template <bool QC, int LOADS>
struct Share {
  __device__ __forceinline__ static int row(int wave, int i, int lane) {
    return (wave * LOADS + i) * (QC ? 8 : 2) + (QC ? lane >> 3 : lane >> 5);
  }
  __device__ __forceinline__ static int chunk(int wave, int i, int lane) {
    const int r = row(wave, i, lane);
    return QC ? (lane & 7) ^ swz_q(r) : (lane & 31) ^ swz_m(r);
  }
};

typedef __attribute__((address_space(3))) const uint8_t lds_byte_t;
typedef __attribute__((address_space(3))) const u32x4_t lds_u32x4_t;
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

// The transposing LDS read.  Its parameter is restrict so that the compiler
// does not take it to depend on the loads into LDS that are in flight (it
// would wait for all of them before each read): the stage barrier is what
// orders a slot's loads before its reads.
__device__ __forceinline__ u32x2_t read_transposed(lds_s16x4_t* __restrict__ p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}

// Offset within an operand's slot of this lane's part of a wave's first block
// (32 rows or columns from `base`) in the first k-step.
template <bool QC>
__device__ __forceinline__ uint32_t frag_offset(int base) {
  const int lane = threadIdx.x & 63;
  if constexpr (QC) {
    const int l32 = lane & 31, hi = lane >> 5;
    return uint32_t((base + l32) * GT_STAGE + ((hi ^ swz_q(l32)) << 4));
  } else {
    // transposing read: lane i of group g names row i / 4 of a 4 x 16 block, columns 4 (i % 4) and on, and
    // receives column i; the group's block is columns 16 (g % 2), rows 8 (g / 2) of the k-step's 16
    const int i = lane & 15, g = lane >> 4;
    const int r = 8 * (g >> 1) + (i >> 2);
    const int c = ((base + 16 * (g & 1)) >> 3) + ((i & 3) >> 1);
    return uint32_t(r * 512 + ((c ^ swz_m(r)) << 4) + ((i & 1) << 3));
  }
}
// 16 bytes of q (see mma16) of block `blk` of k-step ks, where `at` is the
// slot's offset plus frag_offset.  The swizzles exchange bits of the chunk
// number only, and a wave's blocks start at a multiple of their number, so the
// k-step (QC) or the block is an exclusive or of a few address bits.
template <bool QC>
__device__ __forceinline__ u32x4_t read_frag(lds_byte_t* ring, uint32_t at, int ks, int blk) {
  if constexpr (QC) {
    return *(lds_u32x4_t*)(ring + (at ^ uint32_t(ks << 5)) + blk * 32 * GT_STAGE);
  } else {
    lds_byte_t* p = ring + (at ^ uint32_t(blk << 6)) + ks * 16 * 512;
    const u32x2_t lo = read_transposed((lds_s16x4_t*)(p));
    const u32x2_t up = read_transposed((lds_s16x4_t*)(p + 4 * 512));     // 4 rows of q on: the same swizzle
    return u32x4_t{lo[0], lo[1], up[0], up[1]};
  }
}

template <int NI>
struct Frags { u32x4_t a[2][NI], b[2][2]; };    // [k-step parity][32-row block]

// acc[i][j] += the tile's products over n_q values of q (n_q * element size a
// multiple of 16).  `addr_a(i, t, ends)` and `addr_b` give this lane's address
// for load i of stage t; with `ends` true_type they replace chunks past the
// end of q by zeros.  `ahead(t)` is called well before the loads of B (t) are
// addressed, for every t in order.
template <int DT, bool AQ, bool BQ, int NI, class AddrA, class AddrB, class Ahead>
__device__ __forceinline__ void tile_products(uint8_t* smem, int n_q, AddrA addr_a, AddrB addr_b, Ahead ahead,
                                              typename Elem<DT>::acc (&acc)[NI][2]) {
  constexpr int Q = GT_STAGE / int(sizeof(typename Elem<DT>::type));   // values of q per stage
  const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int nk = (n_q + Q - 1) / Q, nk_full = n_q / Q;
  lds_byte_t* const ring = (lds_byte_t*)smem;
  const uint32_t off_a = frag_offset<AQ>((wv >> 2) * 32 * NI), off_b = frag_offset<BQ>((wv & 3) * 64);
  auto slot_a = [](int t) { return uint32_t(t & 1) * GT_SLOT; };
  auto slot_b = [](int t) { return uint32_t(2 + t % 3) * GT_SLOT; };

  auto load_a = [&](int t, auto i0, auto i1, auto ends) {
    for_range<decltype(i0)::value, decltype(i1)::value>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      __builtin_amdgcn_global_load_lds((glb_void_t*)addr_a(i, t, ends),
                                       (lds_void_t*)(smem + slot_a(t) + (wv * NI + i) * 1024), 16, 0, 0);
    });
  };
  auto load_b = [&](int t, auto i0, auto i1, auto ends) {
    for_range<decltype(i0)::value, decltype(i1)::value>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      __builtin_amdgcn_global_load_lds((glb_void_t*)addr_b(i, t, ends),
                                       (lds_void_t*)(smem + slot_b(t) + (wv * 4 + i) * 1024), 16, 0, 0);
    });
  };
  using I0 = std::integral_constant<int, 0>;
  using I2 = std::integral_constant<int, 2>;
  using I4 = std::integral_constant<int, 4>;
  using IA = std::integral_constant<int, NI>;
  using IA2 = std::integral_constant<int, (NI + 1) / 2>;
  using Yes = std::true_type;
  using No = std::false_type;

  Frags<NI> f;
  // Operand read r of a k-step, in the order in which its MFMAs need them: b0, a0, b1, a1, a2, ...
  auto read_one = [&](uint32_t at_a, uint32_t at_b, int ks, auto rc) {
    constexpr int r = decltype(rc)::value;
    const int p = ks & 1;
    if constexpr (r == 0) f.b[p][0] = read_frag<BQ>(ring, at_b, ks, 0);
    else if constexpr (r == 2) f.b[p][1] = read_frag<BQ>(ring, at_b, ks, 1);
    else if constexpr (r == 1) f.a[p][0] = read_frag<AQ>(ring, at_a, ks, 0);
    else f.a[p][r - 2] = read_frag<AQ>(ring, at_a, ks, r - 2);
  };
  auto read_step = [&](uint32_t at_a, uint32_t at_b, int ks) {
    for_range<0, NI + 2>([&](auto r) { read_one(at_a, at_b, ks, r); });
  };
  auto multiply = [&](int h) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) mma16<DT>(f.a[h][i], f.b[h][j], acc[i][j]);
  };
  // One k-step in a fixed order: the MFMAs of parity h, between them the reads of k-step ks of the slots
  // at_a / at_b, and after those, one to an MFMA, the loads 0 .. V - 1 that `load` issues.
  auto step = [&](int h, uint32_t at_a, uint32_t at_b, int ks, auto vc, auto load) {
    constexpr int M = NI * 2, R = NI + 2, V = decltype(vc)::value;
    constexpr int PER = (R + M - 1) / M > 1 ? (R + M - 1) / M : (R > M - V ? 2 : 1);   // reads after an MFMA
    for_range<0, M>([&](auto qc) {
      constexpr int q = decltype(qc)::value;
      mma16<DT>(f.a[h][q / 2], f.b[h][q % 2], acc[q / 2][q % 2]);
      for_range<(q * PER < R ? q * PER : R), ((q + 1) * PER < R ? (q + 1) * PER : R)>(
          [&](auto r) { read_one(at_a, at_b, ks, r); });
      if constexpr (q >= M - V) load(std::integral_constant<int, q - (M - V)>{});
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // Stage t with the stages it loads (up to t + 2) whole.
  auto steady = [&](int t) {
    const uint32_t at_a = opaque(slot_a(t) + off_a), at_b = opaque(slot_b(t) + off_b);
    auto one_a = [&](int t, auto ic) { load_a(t, ic, std::integral_constant<int, decltype(ic)::value + 1>{}, No{}); };
    auto one_b = [&](int t, auto ic) { load_b(t, ic, std::integral_constant<int, decltype(ic)::value + 1>{}, No{}); };
    step(0, at_a, at_b, 1, I2{}, [&](auto i) { one_b(t + 2, i); });
    step(1, at_a, at_b, 2, I2{}, [&](auto i) { one_b(t + 2, std::integral_constant<int, 2 + decltype(i)::value>{}); });
    step(0, at_a, at_b, 3, I0{}, [&](auto) {});
    wait_loads<4>();            // all but B (t + 2): stage t + 1 has landed (this wave's part)
    stage_barrier();
    __builtin_amdgcn_sched_barrier(0);
    ahead(t + 3);
    step(1, opaque(slot_a(t + 1) + off_a), opaque(slot_b(t + 1) + off_b), 0, IA{}, [&](auto i) { one_a(t + 2, i); });
  };
  // The same with the ends checked (the last stages, short reductions).
  auto tail = [&](int t) {
    const uint32_t at_a = opaque(slot_a(t) + off_a), at_b = opaque(slot_b(t) + off_b);
    multiply(0);
    read_step(at_a, at_b, 1);
    if (t + 2 < nk) load_b(t + 2, I0{}, I4{}, Yes{});
    multiply(1);
    read_step(at_a, at_b, 2);
    multiply(0);
    read_step(at_a, at_b, 3);
    const bool more = t + 1 < nk;
    if (more) {
      if (t + 2 < nk) wait_loads<4>();
      else wait_loads<0>();
      stage_barrier();
    }
    ahead(t + 3);
    multiply(1);
    if (more) {
      read_step(slot_a(t + 1) + off_a, slot_b(t + 1) + off_b, 0);
      if (t + 2 < nk) load_a(t + 2, I0{}, IA{}, Yes{});
    }
  };

  if (nk == 0) return;
  ahead(0);
  load_a(0, I0{}, IA{}, Yes{});
  load_b(0, I0{}, I4{}, Yes{});
  if (nk > 1) {
    ahead(1);
    load_b(1, I0{}, I4{}, Yes{});
    load_a(1, I0{}, IA{}, Yes{});
    ahead(2);
    wait_loads<4 + NI>();
  } else {
    wait_loads<0>();
  }
  stage_barrier();
  read_step(slot_a(0) + off_a, slot_b(0) + off_b, 0);
  int t = 0;
  for (; t + 2 < nk_full; ++t) steady(t);
  for (; t < nk; ++t) tail(t);
}

// Writes a wave's 32 NI x 64 part of a tile: rows from `row` (those below
// `end`), columns from `col` (below n_cols) of the row-major `out`.  `value(x,
// r, s)` makes the output of sum x in row r of the tile, s = `col_scale(n)`.
// The sums go through LDS, 32 rows at a time, so that a store instruction
// covers whole 128-byte lines (stored as they lie in registers, 64-byte pieces
// of bf16, the epilogue took longer than 8 stages of the main loop).  Rows of
// out that are not 16-byte aligned are stored element by element.
constexpr int GT_OUT_ROW = 64 * 4 + 16;           // bytes of a staged row: 64 columns, and a pad for the banks
constexpr int GT_OUT_WAVE = 32 * GT_OUT_ROW;
template <int OUT, int NI, class Acc, class Value, class Scale>
__device__ __forceinline__ void store_tile(uint8_t* smem, const Acc (&acc)[NI][2], void* out, int tile_row, int row,
                                           int end, int col, int n_cols, Scale col_scale, Value value) {
  constexpr int B = OUT == DT_F32 ? 4 : 2, C = 16 / B;
  constexpr int LPR = 64 / C, RPI = 64 / LPR;     // lanes per row and rows per store instruction
  const int lane = lane_here(), l32 = lane & 31, hi = lane >> 5;
  // register q of lane l: row 8 (q / 4) + 4 (l / 32) + q % 4 of a 32 x 32 block, column l % 32
  float s[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) s[j] = col + 32 * j + l32 < n_cols ? col_scale(col + 32 * j + l32) : 0.f;
  if (n_cols % C) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = col + 32 * j + l32;
      if (n >= n_cols) continue;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int r = 32 * i + 8 * (q >> 2) + 4 * hi + (q & 3);
          if (row + r < end) store_out<OUT>(out, size_t(row + r) * n_cols + n, value(acc[i][j][q], tile_row + r, s[j]));
        }
    }
    return;
  }
  uint8_t* const mine = smem + __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)) * GT_OUT_WAVE;
  const int cr = lane / LPR, cc = (lane % LPR) * C;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (row + 32 * i >= end) return;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int r = 8 * (q >> 2) + 4 * hi + (q & 3);
        const float v = value(acc[i][j][q], tile_row + 32 * i + r, s[j]);
        uint8_t* p = mine + r * GT_OUT_ROW + (32 * j + l32) * B;
        if constexpr (OUT == DT_F32) *reinterpret_cast<float*>(p) = v;
        else *reinterpret_cast<uint16_t*>(p) = uint16_t(f32_to_bf16(v));
      }
    // LDS serves a wave's accesses in order; the compiler has to keep it
    asm volatile("" ::: "memory");
#pragma unroll
    for (int k = 0; k < 32 / RPI; ++k) {
      const int r = k * RPI + cr;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(mine + r * GT_OUT_ROW + cc * B);
      if (row + 32 * i + r < end && col + cc < n_cols)
        *reinterpret_cast<u32x4_t*>(reinterpret_cast<uint8_t*>(out) + (size_t(row + 32 * i + r) * n_cols + col + cc) * B) = v;
    }
    asm volatile("" ::: "memory");
  }
}

// ------------------------------------------------------- forward and dx --
// Item list: (column group, row tile, column) over the row tiles that the
// segments fill.  Column groups are GT_CG tiles wide, row tiles go in order
// within a group and columns inside them, so that consecutive items share an
// expert's weights or a row tile; each XCD (work-group b runs on XCD b % 8)
// takes one contiguous eighth.
constexpr int GT_CG = 4;

// One tile: `rows` sorted rows from row0 (at most 64 NI), columns from n0.
template <int DT, int OUT, int WHICH, int NI>
__device__ __forceinline__ void rows_tile(const GroupedArgs& a, uint8_t* smem, int e, int row0, int rows, int n0) {
  typedef typename Elem<DT>::type T;
  constexpr int C = 16 / int(sizeof(T));
  constexpr bool BQ = WHICH == GM_FORWARD;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int n_cols = WHICH == GM_FORWARD ? a.N : a.K, n_q = WHICH == GM_FORWARD ? a.K : a.N;
  const uint8_t* const zeros = reinterpret_cast<const uint8_t*>(&g_zeros);
  const T* const w = reinterpret_cast<const T*>(a.w) + size_t(e) * a.N * a.K;

  // Rows without a source, and rows past the segment, load some row that exists (w's first, or the tile's
  // first of dy): their products are replaced or not stored.  Likewise the columns past the last.  Rows
  // found through row_ids may lie anywhere in x; all else is within 2^32 bytes of the tile's first row.
  typedef Share<true, NI> SA;
  typedef Share<BQ, 4> SB;
  const uint8_t* pa[NI];
  uint32_t oa[NI], ob[4];
  const uint8_t* const dy0 = reinterpret_cast<const uint8_t*>(reinterpret_cast<const T*>(a.dy) + size_t(row0) * a.N);
  const uint8_t* const w0 = reinterpret_cast<const uint8_t*>(w + (BQ ? size_t(n0) * a.K : size_t(n0)));
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = SA::row(wv, i, lane), c = SA::chunk(wv, i, lane) * 16;
    if constexpr (WHICH == GM_FORWARD) {
      const int src = r < rows ? source_row(a, row0 + r) : -1;
      pa[i] = reinterpret_cast<const uint8_t*>(src < 0 ? w : reinterpret_cast<const T*>(a.x) + size_t(src) * a.K) + c;
    } else {
      oa[i] = uint32_t(r < rows ? r : 0) * uint32_t(a.N * int(sizeof(T))) + c;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = SB::row(wv, i, lane), c = SB::chunk(wv, i, lane) * C;
    if constexpr (BQ) ob[i] = (uint32_t(n0 + r < n_cols ? r : 0) * uint32_t(a.K) + c) * uint32_t(sizeof(T));
    else ob[i] = (uint32_t(r) * uint32_t(a.K) + (n0 + c < n_cols ? c : 0)) * uint32_t(sizeof(T));
  }
  const size_t row_bytes = size_t(n_q) * sizeof(T);
  const size_t step_b = BQ ? GT_STAGE : size_t(64) * a.K * sizeof(T);
  auto addr_a = [&](int i, int t, auto ends) {
    const uint8_t* p;
    if constexpr (WHICH == GM_FORWARD) p = pa[i] + size_t(t) * GT_STAGE;
    else p = opaque_base(dy0 + size_t(t) * GT_STAGE) + oa[i];
    if constexpr (decltype(ends)::value)
      if (size_t(t) * GT_STAGE + SA::chunk(wv, i, lane_here()) * 16 >= row_bytes) p = zeros;
    return p;
  };
  auto addr_b = [&](int i, int t, auto ends) {
    const uint8_t* p = opaque_base(w0 + size_t(t) * step_b) + ob[i];
    if constexpr (decltype(ends)::value)
      if (BQ ? size_t(t) * GT_STAGE + SB::chunk(wv, i, lane_here()) * 16 >= row_bytes
             : t * 64 + SB::row(wv, i, lane_here()) >= n_q)
        p = zeros;
    return p;
  };

  typename Elem<DT>::acc acc[NI][2];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
  tile_products<DT, true, BQ, NI>(smem, n_q, addr_a, addr_b, [](int) {}, acc);

  // The rows' scales (8-bit), or 1; 0 for a row that stands for zeros.
  float* const row_scale = reinterpret_cast<float*>(smem + GT_WAVES * GT_OUT_WAVE);
  __syncthreads();
  if constexpr (WHICH == GM_FORWARD) {
    if (int(threadIdx.x) < 64 * NI) {
      const int r = threadIdx.x;
      const int src = r < rows ? source_row(a, row0 + r) : -1;
      row_scale[r] = src < 0 ? 0.f : (DT == DT_I8 ? a.x_scale[src] : 1.f);
    }
    __syncthreads();
  }
  const int m0 = (wv >> 2) * 32 * NI;
  store_tile<OUT, NI>(
      smem, acc, a.out, m0, row0 + m0, row0 + rows, n0 + (wv & 3) * 64, n_cols,
      [&](int n) { return DT == DT_I8 ? a.w_scale[size_t(e) * a.N + n] : 0.f; },
      [&](auto x, int r, float ws) {
        if constexpr (DT == DT_I8) return float(x) * row_scale[r] * ws;
        else return WHICH == GM_FORWARD && row_scale[r] == 0.f ? 0.f : float(x);
      });
}

template <int DT, int OUT, int WHICH>
__global__ void __launch_bounds__(64 * GT_WAVES) grouped_rows_kernel(GroupedArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[GT_LDS];
  constexpr int TM = 256;
  const int n_cols = WHICH == GM_FORWARD ? a.N : a.K;
  const int n_ct = (n_cols + GT_N - 1) / GT_N;
  const int xcd = blockIdx.x & 7;
  for (long it = blockIdx.x >> 3;; it += gridDim.x >> 3) {
    const RowTiles tiles(a, TM);                 // looked up anew per item: kept, it would cost registers below
    const long n_items = long(tiles.total) * n_ct;
    const long item = xcd * n_items / 8 + it;
    if (item >= (xcd + 1) * n_items / 8) return;
    const long per_group = long(tiles.total) * GT_CG;
    const int g = int(item / per_group);
    const int in_g = int(item - g * per_group);
    const int width = min(GT_CG, n_ct - g * GT_CG);
    const int n0 = (g * GT_CG + in_g % width) * GT_N;
    const RowTile rt = tiles.at(in_g / width, TM);
    // the last rows of a segment take the smallest tile that holds them
    if (rt.n > 128) rows_tile<DT, OUT, WHICH, 4>(a, smem, rt.e, rt.begin, min(rt.n, TM), n0);
    else if (rt.n > 64) rows_tile<DT, OUT, WHICH, 2>(a, smem, rt.e, rt.begin, rt.n, n0);
    else rows_tile<DT, OUT, WHICH, 1>(a, smem, rt.e, rt.begin, rt.n, n0);
    __syncthreads();                             // the ring is free for the next item
  }
}

template <int DT, int OUT, int WHICH>
hipError_t launch_rows(const GroupedArgs& a, hipStream_t st) {
  const long n_ct = ((WHICH == GM_FORWARD ? a.N : a.K) + GT_N - 1) / GT_N;
  const long n_items = (long(a.rows) / 256 + a.E) * n_ct;       // every segment may end in a part of a tile
  const long grid = (n_items < (1L << 20) ? n_items : (1L << 20)) + 7;
  hipLaunchKernelGGL((grouped_rows_kernel<DT, OUT, WHICH>), dim3(unsigned(grid / 8 * 8)), dim3(64 * GT_WAVES), 0, st, a);
  return hipGetLastError();
}

// -------------------------------------------------------------------- dw --
// One item per 256 x 256 tile of dw[e]; the reduction runs over e's rows.
// Experts' work differs with their rows, so each XCD takes an eighth of every
// expert's tiles, in order (they share panels of dy and x in that XCD's L2).
// LOOKUP: the rows of x are found through row_ids, which are read one stage
// before the loads that they address.
template <int OUT, bool LOOKUP>
__global__ void __launch_bounds__(64 * GT_WAVES) grouped_dw_kernel(GroupedArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[GT_LDS];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int n_mt = (a.N + 255) / 256, n_nt = (a.K + GT_N - 1) / GT_N;
  const long per_expert = long(n_mt) * n_nt, share = (per_expert + 7) / 8;
  const uint8_t* const zeros = reinterpret_cast<const uint8_t*>(&g_zeros);

  for (long it = blockIdx.x >> 3; it < share * a.E; it += gridDim.x >> 3) {
    const int e = __builtin_amdgcn_readfirstlane(int(it / share));
    const long tile = long(blockIdx.x & 7) * share + it % share;
    if (tile >= per_expert) continue;
    const int m0 = __builtin_amdgcn_readfirstlane(int(tile / n_nt)) * 256;
    const int n0 = __builtin_amdgcn_readfirstlane(int(tile % n_nt)) * GT_N;
    Segment seg = segment_of(a, e);
    seg.begin = __builtin_amdgcn_readfirstlane(seg.begin);
    const int n_q = __builtin_amdgcn_readfirstlane(seg.n);

    typedef Share<false, 4> S;
    // Each load fills two rows of q, so the wave's rows of a stage are eight entries of row_ids that all its
    // lanes share: scalar loads, which do not count among the vector loads that the stages wait for.
    int id[8];
    typedef const __attribute__((address_space(4))) int32_t const_i32_t;
    const_i32_t* const ids = (const_i32_t*)(a.row_ids);
    auto ahead = [&](int t) {
      if constexpr (LOOKUP) {
#pragma unroll
        for (int i = 0; i < 8; ++i) id[i] = ids[seg.begin + max(min(t * 64 + wv * 8 + i, n_q - 1), 0)];
      }
    };
    // columns past the last read the tile's first ones: their products are not stored
    const uint8_t* const dy0 = reinterpret_cast<const uint8_t*>(reinterpret_cast<const uint16_t*>(a.dy) +
                                                                size_t(seg.begin) * a.N + m0);
    const uint8_t* const x0 = reinterpret_cast<const uint8_t*>(reinterpret_cast<const uint16_t*>(a.x) +
                                                               (LOOKUP ? 0 : size_t(seg.begin) * a.K) + n0);
    uint32_t oa[4], ob[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = S::row(wv, i, lane), c = S::chunk(wv, i, lane) * 8;
      oa[i] = (uint32_t(r) * uint32_t(a.N) + (m0 + c < a.N ? c : 0)) * 2u;
      ob[i] = ((LOOKUP ? 0u : uint32_t(r) * uint32_t(a.K)) + (n0 + c < a.K ? c : 0)) * 2u;
    }
    const size_t step_a = size_t(64) * a.N * 2, step_b = size_t(64) * a.K * 2;
    auto addr_a = [&](int i, int t, auto ends) {
      const uint8_t* p = opaque_base(dy0 + size_t(t) * step_a) + oa[i];
      if constexpr (decltype(ends)::value)
        if (t * 64 + S::row(wv, i, lane_here()) >= n_q) p = zeros;
      return p;
    };
    auto addr_b = [&](int i, int t, auto ends) {
      const uint8_t* p;
      if constexpr (LOOKUP) {
        // selects between values that are there either way: no branches in the main loop
        const int s0 = source_of(a, id[2 * i]), s1 = source_of(a, id[2 * i + 1]);
        const uint64_t row = uint64_t(a.K) * 2u;
        const uint64_t r0 = uint64_t(x0) + uint64_t(unsigned(max(s0, 0))) * row;
        const uint64_t r1 = uint64_t(x0) + uint64_t(unsigned(max(s1, 0))) * row;
        const uint64_t p0 = s0 < 0 ? uint64_t(zeros) : r0, p1 = s1 < 0 ? uint64_t(zeros) : r1;
        const uint32_t o0 = s0 < 0 ? 0u : ob[i], o1 = s1 < 0 ? 0u : ob[i];
        const bool second = lane >= 32;
        p = reinterpret_cast<const uint8_t*>((second ? p1 : p0) + (second ? o1 : o0));
      } else {
        p = opaque_base(x0 + size_t(t) * step_b) + ob[i];
      }
      if constexpr (decltype(ends)::value)
        if (t * 64 + S::row(wv, i, lane_here()) >= n_q) p = zeros;
      return p;
    };

    f32x16_t acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
    tile_products<DT_BF16, false, false, 4>(smem, n_q, addr_a, addr_b, ahead, acc);

    __syncthreads();
    const int m = m0 + (wv >> 2) * 128;
    store_tile<OUT, 4>(
        smem, acc, reinterpret_cast<uint8_t*>(a.out) + size_t(e) * a.N * a.K * (OUT == DT_F32 ? 4 : 2), 0, m, a.N,
        n0 + (wv & 3) * 64, a.K, [](int) { return 0.f; }, [](float x, int, float) { return x; });
    __syncthreads();
  }
}

template <int OUT>
hipError_t launch_dw(const GroupedArgs& a, hipStream_t st) {
  const long per_expert = long((a.N + 255) / 256) * ((a.K + GT_N - 1) / GT_N);
  const long n_items = (per_expert + 7) / 8 * 8 * a.E;
  const long grid = n_items < (1L << 20) ? n_items : (1L << 20);
  if (a.row_ids)
    hipLaunchKernelGGL((grouped_dw_kernel<OUT, true>), dim3(unsigned(grid)), dim3(64 * GT_WAVES), 0, st, a);
  else
    hipLaunchKernelGGL((grouped_dw_kernel<OUT, false>), dim3(unsigned(grid)), dim3(64 * GT_WAVES), 0, st, a);
  return hipGetLastError();
}

}  // namespace

bool grouped_tile_fits(const GroupedArgs& a, int which, int in_dt) {
  if (in_dt == DT_I8) return a.K % 16 == 0;
  return in_dt == DT_BF16 && a.K % 8 == 0 && (which == GM_FORWARD || a.N % 8 == 0);
}

hipError_t launch_grouped_tile(const GroupedArgs& a, int which, int in_dt, int out_dt, hipStream_t st) {
  if (in_dt == DT_I8)
    return out_dt == DT_F32 ? launch_rows<DT_I8, DT_F32, GM_FORWARD>(a, st) : launch_rows<DT_I8, DT_BF16, GM_FORWARD>(a, st);
  if (which == GM_FORWARD)
    return out_dt == DT_F32 ? launch_rows<DT_BF16, DT_F32, GM_FORWARD>(a, st)
                            : launch_rows<DT_BF16, DT_BF16, GM_FORWARD>(a, st);
  if (which == GM_GRAD_X) return launch_rows<DT_BF16, DT_BF16, GM_GRAD_X>(a, st);
  return out_dt == DT_F32 ? launch_dw<DT_F32>(a, st) : launch_dw<DT_BF16>(a, st);
}

}  // namespace moe
