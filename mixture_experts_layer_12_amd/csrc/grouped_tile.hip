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
// neighbouring work-groups share in L2: the loads of B (t + 2) are issued one
// by one between the MFMAs of stage t, and those of A (t + 2) after the
// barrier at its end, which waits for all but the former (loads complete in
// issue order).
// Measured: 4096 tokens, top 2 of 8 experts of 14336 x 4096 in bf16 852-886 us
// (1.1 PF/s; MFMA busy for 60 % of the time at 1.65-1.75 GHz), in 8 bits 474;
// both gradients 1940-2001 us.  A stage takes 1.6 us, 1.17 if its MFMAs ran
// without a pause, 1.42 with all operands in cache.
// 16-byte chunks (32-byte pairs of them where reads transpose) are permuted
// within each staged row so that the rows one read touches lie on distinct
// banks.
#include <algorithm>

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

// One operand's loads: instruction i of the eight waves fills 64 staged rows of
// 128 bytes (8 a wave), or 16 rows of q of 512 bytes (2 a wave).  Lane l fills
// 16 bytes of staged row `row`, with chunk `chunk` of that row in memory.
template <bool QC>
struct Share {
  __device__ __forceinline__ static int row(int wave, int i, int lane) {
    return (i * GT_WAVES + wave) * (QC ? 8 : 2) + (QC ? lane >> 3 : lane >> 5);
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

__device__ __forceinline__ uint32_t slot_a(int t) { return uint32_t(t & 1) * GT_SLOT; }
__device__ __forceinline__ uint32_t slot_b(int t) { return uint32_t(2 + t % 3) * GT_SLOT; }
__device__ __forceinline__ void load_to_lds(const uint8_t* from, uint8_t* to) {   // `to` + 16 bytes a lane
  __builtin_amdgcn_global_load_lds((glb_void_t*)from, (lds_void_t*)to, 16, 0, 0);
}

// Tiles are addressed by an object `ad` with, for this lane,
//   a(i, t, ends), b(i, t, ends)  the address of load i of stage t; with `ends`
//             true_type chunks past the end of q are replaced by zeros
//   ahead(t)  called well before b(.., t, ..), for every t in order, and
//             between b(.., t - 1, ..) and a(.., t - 1, ..)
//   n_q       values of q (n_q * element size is a multiple of 16)

// The loads of stages 0 and 1 (ring slots 0 - 3): issued for the next tile
// before the outputs of the present one, which use slot 4 only, are written.
template <int DT, class Addr>
__device__ __forceinline__ void first_loads(uint8_t* smem, Addr& ad, int ni) {
  constexpr int Q = GT_STAGE / int(sizeof(typename Elem<DT>::type));
  const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int nk = (ad.n_q + Q - 1) / Q;
  ad.ahead(0);
  for (int t = 0; t < 2 && t < nk; ++t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) load_to_lds(ad.b(i, t, std::true_type{}), smem + slot_b(t) + (i * GT_WAVES + wv) * 1024);
    ad.ahead(t + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < ni) load_to_lds(ad.a(i, t, std::true_type{}), smem + slot_a(t) + (i * GT_WAVES + wv) * 1024);
  }
}

// acc[i][j] += the tile's products, once first_loads has been issued.
template <int DT, bool AQ, bool BQ, int NI, class Addr>
__device__ __forceinline__ void tile_products(uint8_t* smem, Addr& ad, typename Elem<DT>::acc (&acc)[NI][2]) {
  constexpr int Q = GT_STAGE / int(sizeof(typename Elem<DT>::type));   // values of q per stage
  const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int nk = (ad.n_q + Q - 1) / Q, nk_full = ad.n_q / Q;
  lds_byte_t* const ring = (lds_byte_t*)smem;
  const uint32_t off_a = frag_offset<AQ>((wv >> 2) * 32 * NI), off_b = frag_offset<BQ>((wv & 3) * 64);

  auto load_a = [&](int t, auto i0, auto i1, auto ends) {
    for_range<decltype(i0)::value, decltype(i1)::value>(
        [&](auto ic) { load_to_lds(ad.a(int(ic), t, ends), smem + slot_a(t) + (int(ic) * GT_WAVES + wv) * 1024); });
  };
  auto load_b = [&](int t, auto i0, auto i1, auto ends) {
    for_range<decltype(i0)::value, decltype(i1)::value>(
        [&](auto ic) { load_to_lds(ad.b(int(ic), t, ends), smem + slot_b(t) + (int(ic) * GT_WAVES + wv) * 1024); });
  };
  using I0 = std::integral_constant<int, 0>;
  using I2 = std::integral_constant<int, 2>;
  using I4 = std::integral_constant<int, 4>;
  using IA = std::integral_constant<int, NI>;
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
      for (int j = 0; j < 2; ++j) mma16<DT>(f.b[h][j], f.a[h][i], acc[i][j]);
  };
  // One k-step in a fixed order: the MFMAs of parity h, between them the reads of k-step ks of the slots
  // at_a / at_b, and after those, one to an MFMA, the loads 0 .. V - 1 that `load` issues.
  auto step = [&](int h, uint32_t at_a, uint32_t at_b, int ks, auto vc, auto load) {
    constexpr int M = NI * 2, R = NI + 2, V = decltype(vc)::value;
    constexpr int PER = (R + M - 1) / M > 1 ? (R + M - 1) / M : (R > M - V ? 2 : 1);   // reads after an MFMA
    for_range<0, M>([&](auto qc) {
      constexpr int q = decltype(qc)::value;
      mma16<DT>(f.b[h][q % 2], f.a[h][q / 2], acc[q / 2][q % 2]);
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
    ad.ahead(t + 3);
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
    ad.ahead(t + 3);
    multiply(1);
    if (more) {
      read_step(slot_a(t + 1) + off_a, slot_b(t + 1) + off_b, 0);
      if (t + 2 < nk) load_a(t + 2, I0{}, IA{}, Yes{});
    }
  };

  if (nk == 0) return;
  wait_loads<0>();              // stages 0 and 1 (and the stores of the tile before)
  stage_barrier();
  read_step(slot_a(0) + off_a, slot_b(0) + off_b, 0);
  int t = 0;
  for (; t + 2 < nk_full; ++t) steady(t);
  for (; t < nk; ++t) tail(t);
}

// Writes a wave's 32 NI x 64 part of a tile: rows from `row` (those below
// `end`), columns from `col` (below n_cols) of the row-major `out`.
// `value(acc, q, i, j, n, v)` makes the outputs v[0 .. 3] of columns n .. n + 3
// from the sums q .. q + 3 of block (i, j).  The MFMAs take B as their first
// operand, so that a lane holds four neighbouring columns of one row; 32 rows
// by 128 bytes at a time they go through LDS, so that a store instruction
// covers whole 128-byte lines.  16-byte units are permuted within the rows
// there (the lanes of one access lie 128 bytes apart).  Rows of out that are
// not 16-byte aligned are stored element by element.
constexpr int GT_OUT_WAVE = 32 * 128;             // bytes per wave, from slot 4 on
constexpr int GT_OUT = 4 * GT_SLOT;
static_assert(GT_WAVES * GT_OUT_WAVE <= GT_SLOT, "one slot");
template <int OUT, int NI, class Acc, class Value>
__device__ __forceinline__ void store_tile(uint8_t* smem, const Acc (&acc)[NI][2], void* out, int row, int end, int col,
                                           int n_cols, Value value) {
  constexpr int B = OUT == DT_F32 ? 4 : 2, C = 16 / B, HALVES = OUT == DT_F32 ? 2 : 1;
  uint8_t* const mine = smem + GT_OUT + __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)) * GT_OUT_WAVE;
  const int lane = lane_here(), l32 = lane & 31, hi = lane >> 5;
  uint8_t* const base = reinterpret_cast<uint8_t*>(out);
  // register q of lane l: column 8 (q / 4) + 4 (l / 32) + q % 4 of a 32 x 32 block, row l % 32
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int first = row + 32 * i;
    if (first >= end) return;
#pragma unroll
    for (int half = 0; half < HALVES; ++half) {
#pragma unroll
      for (int jj = 0; jj < 2 / HALVES; ++jj)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int j = half + jj;
          float v[4];
          value(acc[i][j], 4 * g, i, j, col + 32 * j + 8 * g + 4 * hi, v);
          if constexpr (OUT == DT_F32)
            *reinterpret_cast<f32x4_t*>(mine + l32 * 128 + (((2 * g + hi) ^ (l32 & 7)) << 4)) = f32x4_t{v[0], v[1], v[2], v[3]};
          else
            *reinterpret_cast<u32x2_t*>(mine + l32 * 128 + (((4 * j + g) ^ (l32 & 7)) << 4) + 8 * hi) =
                u32x2_t{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3])};
        }
      // LDS serves a wave's accesses in order; the compiler has to keep it
      asm volatile("" ::: "memory");
      const int c0 = col + 32 * half;              // the columns that are staged begin here
      if (n_cols % C == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = k * 8 + (lane >> 3), c = c0 + (lane & 7) * C;
          const u32x4_t v = *reinterpret_cast<const u32x4_t*>(mine + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
          if (first + r < end && c < n_cols)
            *reinterpret_cast<u32x4_t*>(base + (size_t(first + r) * n_cols + c) * B) = v;
        }
      } else {
        constexpr int LPR = 128 / B;               // a lane per element: 64 of bf16, 32 of fp32 in a row
        const int c = lane % LPR;
        if (c0 + c < n_cols)
          for (int r = lane / LPR; r < 32 && first + r < end; r += 64 / LPR) {
            const uint8_t* p = mine + r * 128 + (((c / C) ^ (r & 7)) << 4) + (c % C) * B;
            uint8_t* const q = base + (size_t(first + r) * n_cols + c0 + c) * B;
            if constexpr (OUT == DT_F32) *reinterpret_cast<float*>(q) = *reinterpret_cast<const float*>(p);
            else *reinterpret_cast<uint16_t*>(q) = *reinterpret_cast<const uint16_t*>(p);
          }
      }
      asm volatile("" ::: "memory");
    }
  }
}

// ------------------------------------------------------- forward and dx --
// Item list: (column group, row tile, column) over the row tiles that the
// segments fill.  Column groups are GT_CG tiles wide, row tiles go in order
// within a group and columns inside them, so that consecutive items share an
// expert's weights or a row tile; each XCD (work-group b runs on XCD b % 8)
// takes one contiguous eighth.  Work-groups are dispatched as CUs fall free:
// tiles of few rows take less time, and a fixed share for resident work-groups
// was 3 % slower for the 4096-token prompt.
// The items left over by the last whole round of an XCD's GT_P CUs, m of them,
// are cut along q into GT_P / m parts (whole stages, at least GT_MIN_PART of
// them); a second kernel adds the parts' sums in order.  That is also how a
// call with fewer tiles than CUs fills the chip.
constexpr int GT_P = 32;
constexpr int GT_CG = 4;
constexpr int GT_MIN_PART = 8;
constexpr int GT_MAXSPLIT = 4;

struct RowsItem {
  int e, row0, rows, n0;       // expert, first sorted row, rows (at most 256; 0: there is no item), first column
  int part, parts;             // the part-th of `parts` cuts along q
  int slot;                    // parts > 1: where its sums go
};

// An XCD's share of the list.
struct ListShare {
  long begin, n, whole;        // first item, items, items that are not cut
  int left, parts;             // the others, and the parts each is cut into
  __device__ __forceinline__ ListShare(long n_items, int xcd, int max_parts) {
    begin = xcd * n_items / 8;
    n = (xcd + 1) * n_items / 8 - begin;
    left = int(n % GT_P);
    parts = left ? min(GT_P / left, max_parts) : 1;
    if (parts < 2) left = 0, parts = 1;
    whole = n - left;
  }
};

template <int WHICH>
__device__ __forceinline__ RowsItem list_item(const GroupedArgs& a, const RowTiles& tiles, long item) {
  const int n_ct = ((WHICH == GM_FORWARD ? a.N : a.K) + GT_N - 1) / GT_N;
  const long per_group = long(tiles.total) * GT_CG;
  const int g = int(item / per_group), in_g = int(item - g * per_group);
  const int width = min(GT_CG, n_ct - g * GT_CG);
  const RowTile rt = tiles.at(in_g / width, 256);
  return RowsItem{rt.e, rt.begin, min(rt.n, 256), __builtin_amdgcn_readfirstlane((g * GT_CG + in_g % width) * GT_N), 0, 1, 0};
}

// The i-th piece of work of this work-group's XCD.
template <int WHICH>
__device__ __forceinline__ RowsItem rows_item(const GroupedArgs& a, long i) {
  const int n_ct = ((WHICH == GM_FORWARD ? a.N : a.K) + GT_N - 1) / GT_N, xcd = blockIdx.x & 7;
  const RowTiles tiles(a, 256);
  const ListShare s(long(tiles.total) * n_ct, xcd, a.max_parts);
  if (i >= s.whole + s.left * s.parts) return RowsItem{0, 0, 0, 0, 0, 1, 0};
  if (i < s.whole) return list_item<WHICH>(a, tiles, s.begin + i);
  const int u = int(i - s.whole), part = u / s.left;
  RowsItem it = list_item<WHICH>(a, tiles, s.begin + s.whole + (u - part * s.left));
  it.part = __builtin_amdgcn_readfirstlane(part);
  it.parts = __builtin_amdgcn_readfirstlane(s.parts);
  it.slot = __builtin_amdgcn_readfirstlane(xcd * GT_P + u);
  return it;
}

// Sums of a part: a tile of 256 columns.
__device__ __forceinline__ float* part_sums(const GroupedArgs& a, int slot) { return a.parts + size_t(slot) * (256 * GT_N); }

// Addresses of one tile.  Rows without a source, and rows past the segment,
// load some row that exists (w's first, or the tile's first of dy): their
// products are replaced or not stored.  Likewise the columns past the last.
// Rows found through row_ids may lie anywhere in x; all else is within 2^32
// bytes of the tile's first row.
template <int DT, int WHICH>
struct RowsAddr {
  typedef typename Elem<DT>::type T;
  static constexpr bool BQ = WHICH == GM_FORWARD;
  static constexpr int C = 16 / int(sizeof(T));
  const uint8_t* pa[WHICH == GM_FORWARD ? 4 : 1];
  uint32_t oa[4], ob[4];
  const uint8_t *dy0, *w0;
  size_t row_bytes, step_b;
  int n_q, wv;

  __device__ __forceinline__ void set(const GroupedArgs& a, const RowsItem& it) {
    const int lane = threadIdx.x & 63;
    wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int n_cols = WHICH == GM_FORWARD ? a.N : a.K;
    // this part's values of q: whole stages from t0 on, but for the end of the last part
    constexpr int Q = GT_STAGE / int(sizeof(T));
    const int all = WHICH == GM_FORWARD ? a.K : a.N, stages = (all + Q - 1) / Q;
    const int t0 = __builtin_amdgcn_readfirstlane(stages * it.part / it.parts);
    const int t1 = __builtin_amdgcn_readfirstlane(stages * (it.part + 1) / it.parts);
    n_q = min(all, t1 * Q) - t0 * Q;
    row_bytes = size_t(n_q) * sizeof(T);
    step_b = BQ ? GT_STAGE : size_t(64) * a.K * sizeof(T);
    const T* const w = reinterpret_cast<const T*>(a.w) + size_t(it.e) * a.N * a.K;
    w0 = reinterpret_cast<const uint8_t*>(w + (BQ ? size_t(it.n0) * a.K : size_t(it.n0))) + t0 * step_b;
    dy0 = reinterpret_cast<const uint8_t*>(reinterpret_cast<const T*>(a.dy) + size_t(it.row0) * a.N) + size_t(t0) * GT_STAGE;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = Share<true>::row(wv, i, lane), c = Share<true>::chunk(wv, i, lane) * 16;
      if constexpr (WHICH == GM_FORWARD) {
        const int src = r < it.rows ? source_row(a, it.row0 + r) : -1;
        pa[i] = reinterpret_cast<const uint8_t*>(src < 0 ? w : reinterpret_cast<const T*>(a.x) + size_t(src) * a.K) +
                size_t(t0) * GT_STAGE + c;
      } else {
        oa[i] = uint32_t(r < it.rows ? r : 0) * uint32_t(a.N * int(sizeof(T))) + c;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = Share<BQ>::row(wv, i, lane), c = Share<BQ>::chunk(wv, i, lane) * C;
      if constexpr (BQ) ob[i] = (uint32_t(it.n0 + r < n_cols ? r : 0) * uint32_t(a.K) + c) * uint32_t(sizeof(T));
      else ob[i] = (uint32_t(r) * uint32_t(a.K) + (it.n0 + c < n_cols ? c : 0)) * uint32_t(sizeof(T));
    }
  }
  template <class Ends>
  __device__ __forceinline__ const uint8_t* a(int i, int t, Ends) const {
    const uint8_t* p;
    if constexpr (WHICH == GM_FORWARD) p = pa[i] + size_t(t) * GT_STAGE;
    else p = opaque_base(dy0 + size_t(t) * GT_STAGE) + oa[i];
    if constexpr (Ends::value)
      if (size_t(t) * GT_STAGE + Share<true>::chunk(wv, i, lane_here()) * 16 >= row_bytes)
        p = reinterpret_cast<const uint8_t*>(&g_zeros);
    return p;
  }
  template <class Ends>
  __device__ __forceinline__ const uint8_t* b(int i, int t, Ends) const {
    const uint8_t* p = opaque_base(w0 + size_t(t) * step_b) + ob[i];
    if constexpr (Ends::value)
      if (BQ ? size_t(t) * GT_STAGE + Share<true>::chunk(wv, i, lane_here()) * 16 >= row_bytes
             : t * 64 + Share<false>::row(wv, i, lane_here()) >= n_q)
        p = reinterpret_cast<const uint8_t*>(&g_zeros);
    return p;
  }
  __device__ __forceinline__ void ahead(int) {}
};

template <int DT, int OUT, int WHICH, int NI>
__device__ __forceinline__ void rows_tile(const GroupedArgs& a, uint8_t* smem, RowsAddr<DT, WHICH>& ad, const RowsItem& it) {
  const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int n_cols = WHICH == GM_FORWARD ? a.N : a.K;
  float scale = 0.f;
  if (WHICH == GM_FORWARD && int(threadIdx.x) < it.rows) scale = scale_of<DT>(a, source_row(a, it.row0 + int(threadIdx.x)));
  typename Elem<DT>::acc acc[NI][2];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
  tile_products<DT, true, WHICH == GM_FORWARD, NI>(smem, ad, acc);

  float* const row_scale = reinterpret_cast<float*>(smem);
  stage_barrier();                               // every wave is through with the ring
  if (WHICH == GM_FORWARD && threadIdx.x < 256) row_scale[threadIdx.x] = scale;
  stage_barrier();
  const int m0 = (wv >> 2) * 32 * NI, c0 = it.n0 + (wv & 3) * 64;
  if (it.parts > 1) {                            // the sums as they are
    store_tile<DT_F32, NI>(smem, acc, part_sums(a, it.slot), m0, it.rows, (wv & 3) * 64, GT_N,
                           [](const auto& x, int q, int, int, int, float(&v)[4]) {
#pragma unroll
                             for (int t = 0; t < 4; ++t) {
                               const auto sum = x[q + t];
                               v[t] = __builtin_bit_cast(float, sum);
                             }
                           });
    return;
  }
  const int last = lane_here();
  float rs[NI], ws[2][16];                       // scales of the lane's rows and columns
  if constexpr (WHICH == GM_FORWARD)
#pragma unroll
    for (int i = 0; i < NI; ++i) rs[i] = row_scale[m0 + 32 * i + (last & 31)];
  if constexpr (DT == DT_I8)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int n = c0 + 32 * j + 8 * (q >> 2) + 4 * (last >> 5) + (q & 3);
        ws[j][q] = n < n_cols ? a.w_scale[size_t(it.e) * a.N + n] : 0.f;
      }
  store_tile<OUT, NI>(smem, acc, a.out, it.row0 + m0, it.row0 + it.rows, c0, n_cols,
                      [&](const auto& x, int q, int i, int j, int, float(&v)[4]) {
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                          if constexpr (DT == DT_I8) v[t] = is_no_row(rs[i]) ? 0.f : float(x[q + t]) * rs[i] * ws[j][q + t];
                          else if constexpr (WHICH == GM_FORWARD) v[t] = is_no_row(rs[i]) ? 0.f : x[q + t];
                          else v[t] = x[q + t];
                        }
                      });
}

template <int DT, int OUT, int WHICH>
__global__ void __launch_bounds__(64 * GT_WAVES) grouped_rows_kernel(GroupedArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[GT_LDS];
  for (long i = blockIdx.x >> 3;; i += gridDim.x >> 3) {
    const RowsItem it = rows_item<WHICH>(a, i);
    if (!it.rows) return;
    RowsAddr<DT, WHICH> ad;
    ad.set(a, it);
    // the last rows of a segment take the smallest tile that holds them
    first_loads<DT>(smem, ad, it.rows > 128 ? 4 : (it.rows > 64 ? 2 : 1));
    if (it.rows > 128) rows_tile<DT, OUT, WHICH, 4>(a, smem, ad, it);
    else if (it.rows > 64) rows_tile<DT, OUT, WHICH, 2>(a, smem, ad, it);
    else rows_tile<DT, OUT, WHICH, 1>(a, smem, ad, it);
    stage_barrier();                             // the ring is free for the next item
  }
}

// Adds the parts of the items that were cut, in order, and writes the outputs:
// a work-group per 16 rows of an item.
constexpr int GT_JOIN_ROWS = 16;
template <int DT, int OUT, int WHICH>
__global__ void __launch_bounds__(256) grouped_join_kernel(GroupedArgs a) {
  typedef typename std::conditional<DT == DT_I8, i32x4_t, f32x4_t>::type V;
  const int n_cols = WHICH == GM_FORWARD ? a.N : a.K, n_ct = (n_cols + GT_N - 1) / GT_N;
  const int chunk = blockIdx.x % (256 / GT_JOIN_ROWS), xcd = blockIdx.x / (256 / GT_JOIN_ROWS), u0 = blockIdx.y;
  const RowTiles t(a, 256);
  const ListShare s(long(t.total) * n_ct, xcd, a.max_parts);
  if (u0 >= s.left) return;
  const RowsItem it = list_item<WHICH>(a, t, s.begin + s.whole + u0);
  const int c = (threadIdx.x & 63) * 4, n = it.n0 + c;
  if (n >= n_cols) return;
  for (int r = chunk * GT_JOIN_ROWS + int(threadIdx.x >> 6); r < min(it.rows, (chunk + 1) * GT_JOIN_ROWS); r += 4) {
    V v = {0, 0, 0, 0};
    for (int p = 0; p < s.parts; ++p)
      v += *reinterpret_cast<const V*>(part_sums(a, xcd * GT_P + p * s.left + u0) + r * GT_N + c);
    float o[4];
    const int src = WHICH == GM_FORWARD ? source_row(a, it.row0 + r) : 0;
    const float xs = DT == DT_I8 && src >= 0 ? a.x_scale[src] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == DT_I8) o[i] = src >= 0 && n + i < n_cols ? float(v[i]) * xs * a.w_scale[size_t(it.e) * a.N + n + i] : 0.f;
      else o[i] = src < 0 ? 0.f : float(v[i]);
    }
    const size_t at = size_t(it.row0 + r) * n_cols + n;
    if (n_cols % 4 == 0) {
      if constexpr (OUT == DT_F32)
        *reinterpret_cast<f32x4_t*>(reinterpret_cast<float*>(a.out) + at) = f32x4_t{o[0], o[1], o[2], o[3]};
      else
        *reinterpret_cast<u32x2_t*>(reinterpret_cast<uint16_t*>(a.out) + at) =
            u32x2_t{cvt_pk_bf16(o[0], o[1]), cvt_pk_bf16(o[2], o[3])};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < n_cols) store_out<OUT>(a.out, at + i, o[i]);
    }
  }
}

// The most items a call can have (the host does not know the segments), and
// the most parts that an item of its shape is cut into (1: nothing is cut).
struct RowsPlan {
  long items;
  int max_parts;
};
RowsPlan rows_plan(const GroupedArgs& a, int which, int in_dt) {
  const long n_cols = which == GM_FORWARD ? a.N : a.K, n_q = which == GM_FORWARD ? a.K : a.N;
  const long stages = (n_q * (in_dt == DT_I8 ? 1 : 2) + GT_STAGE - 1) / GT_STAGE;
  RowsPlan p{(long(a.rows) / 256 + std::min(a.E, a.rows)) * ((n_cols + GT_N - 1) / GT_N), 1};
  // With many rounds the CUs that idle in the last one matter little, and the second launch and the parts' sums are
  // saved (9 rounds, 4096 tokens through 8 experts of 14336 x 4096: 870 us, 886 cut; in 8 bits 505 and 511; 3 rounds
  // and less: that prompt's gradients 2000 us, 2215 uncut; 64 experts of 1408 x 2048, 1024 tokens, 253 and 270).
  if (p.items <= GT_MAXSPLIT * 8 * GT_P) p.max_parts = int(std::max<long>(1, std::min<long>(stages / GT_MIN_PART, GT_P)));
  return p;
}

template <int DT, int OUT, int WHICH>
hipError_t launch_rows(const GroupedArgs& args, void* ws, hipStream_t st) {
  GroupedArgs a = args;
  const RowsPlan p = rows_plan(a, WHICH, DT);
  a.parts = reinterpret_cast<float*>(ws);
  a.max_parts = p.max_parts;
  const long grid = std::min<long>((p.items + 7) / 8 * 8 + (p.max_parts > 1 ? 8 * GT_P : 0), 1L << 20);
  hipLaunchKernelGGL((grouped_rows_kernel<DT, OUT, WHICH>), dim3(unsigned(grid)), dim3(64 * GT_WAVES), 0, st, a);
  if (p.max_parts > 1)
    hipLaunchKernelGGL((grouped_join_kernel<DT, OUT, WHICH>), dim3(8 * (256 / GT_JOIN_ROWS), GT_P / 2), dim3(256), 0, st, a);
  return hipGetLastError();
}

// -------------------------------------------------------------------- dw --
// One item per 256 x 256 tile of dw[e]; the reduction runs over e's rows.  A
// resident work-group (one per CU: the ring is all of its LDS) takes its items
// one after another, and while the outputs of one are written the first loads
// of the next are under way.
// Experts' work differs with their rows, so each XCD takes an eighth of every
// expert's tiles, in order (they share panels of dy and x in that XCD's L2).
constexpr int GT_GRID = 256;
struct DwItem {
  int e, m0, n0, begin, n;     // expert (-1: there is no item), tile of dw[e], e's segment
};

__device__ __forceinline__ DwItem dw_item(const GroupedArgs& a, long& it) {
  const int n_nt = (a.K + GT_N - 1) / GT_N;
  const long per_expert = long((a.N + 255) / 256) * n_nt, share = (per_expert + 7) / 8;
  for (; it < share * a.E; it += gridDim.x >> 3) {
    const long tile = long(blockIdx.x & 7) * share + it % share;
    if (tile >= per_expert) continue;
    const int e = int(it / share);
    const Segment s = segment_of(a, e);
    auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    return DwItem{uni(e), uni(int(tile / n_nt) * 256), uni(int(tile % n_nt) * GT_N), uni(s.begin), uni(s.n)};
  }
  return DwItem{-1, 0, 0, 0, 0};
}

// Entries of the table of row addresses, before its row of zeros (16-byte aligned).
constexpr int GT_TABLE_PAD = 64;
__host__ __device__ inline long zero_row_entry(const GroupedArgs& a) { return (long(a.rows) + GT_TABLE_PAD + 1) / 2 * 2; }

// LOOKUP: the rows of x are found through a table of their addresses (8 bytes
// a sorted row, see row_table_kernel).  Each load fills two rows of q, so a
// wave's rows of a stage are eight table entries that all its lanes share:
// scalar loads, a stage ahead, which do not count among the vector loads that
// the stages wait for.
template <bool LOOKUP>
struct DwAddr {
  uint32_t oa[4], ob[4];
  const uint8_t *dy0, *x0;
  size_t step_a, step_b;
  int n_q, wv, last;
  const uint64_t* table;
  uint64_t at[8], zero_row;
  uint32_t none;               // rows of the stage before at[]'s that have no source: they add nothing, whatever dy holds

  __device__ __forceinline__ void set(const GroupedArgs& a, const DwItem& it) {
    const int lane = threadIdx.x & 63;
    wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    n_q = it.n;
    last = (it.n + 63) / 64 - 1;
    step_a = size_t(64) * a.N * 2;
    step_b = size_t(64) * a.K * 2;
    dy0 = reinterpret_cast<const uint8_t*>(reinterpret_cast<const uint16_t*>(a.dy) + size_t(it.begin) * a.N + it.m0);
    x0 = reinterpret_cast<const uint8_t*>(reinterpret_cast<const uint16_t*>(a.x) + size_t(it.begin) * a.K + it.n0);
    table = a.row_table + it.begin + wv * 2;
    zero_row = reinterpret_cast<uint64_t>(a.row_table + zero_row_entry(a));
    none = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) at[i] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // columns past the last read the tile's first ones: their products are not stored
      const int r = Share<false>::row(wv, i, lane), c = Share<false>::chunk(wv, i, lane) * 8;
      oa[i] = (uint32_t(r) * uint32_t(a.N) + (it.m0 + c < a.N ? c : 0)) * 2u;
      const uint32_t col = it.n0 + c < a.K ? c : 0;
      ob[i] = LOOKUP ? (it.n0 + col) * 2u : (uint32_t(r) * uint32_t(a.K) + col) * 2u;
    }
  }
  template <class Ends>
  __device__ __forceinline__ const uint8_t* a(int i, int t, Ends) const {
    const uint8_t* p = opaque_base(dy0 + size_t(t) * step_a) + oa[i];
    if constexpr (LOOKUP)
      if (((threadIdx.x & 32) ? none >> (2 * i + 1) : none >> (2 * i)) & 1) p = reinterpret_cast<const uint8_t*>(&g_zeros);
    if constexpr (Ends::value)
      if (t * 64 + Share<false>::row(wv, i, lane_here()) >= n_q) p = reinterpret_cast<const uint8_t*>(&g_zeros);
    return p;
  }
  template <class Ends>
  __device__ __forceinline__ const uint8_t* b(int i, int t, Ends) const {
    const uint8_t* p;
    if constexpr (LOOKUP) p = reinterpret_cast<const uint8_t*>((threadIdx.x & 32) ? at[2 * i + 1] : at[2 * i]) + ob[i];
    else p = opaque_base(x0 + size_t(t) * step_b) + ob[i];
    if constexpr (Ends::value)
      if (t * 64 + Share<false>::row(wv, i, lane_here()) >= n_q) p = reinterpret_cast<const uint8_t*>(&g_zeros);
    return p;
  }
  __device__ __forceinline__ void ahead(int t) {
    if constexpr (LOOKUP) {
      typedef const __attribute__((address_space(4))) uint64_t const_u64_t;
      const_u64_t* const p = (const_u64_t*)(table) + max(min(t, last), 0) * 64;
      none = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) none |= (at[i] == zero_row ? 1u : 0u) << i;
#pragma unroll
      for (int i = 0; i < 4; ++i) at[2 * i] = p[16 * i], at[2 * i + 1] = p[16 * i + 1];
    }
  }
};

// Table of the addresses of the rows of x in sorted order, and a row of zeros
// behind it for rows without a source.  Entries past the last row (a stage
// reads whole blocks of 64) name the row of zeros as well.
__global__ void __launch_bounds__(256) row_table_kernel(GroupedArgs a, uint64_t* table, uint16_t* zero_row) {
  const long i = long(blockIdx.x) * 256 + threadIdx.x;
  if (i < zero_row_entry(a)) {
    const int src = i < a.rows ? source_row(a, int(i)) : -1;
    const uint16_t* p = src < 0 ? zero_row : reinterpret_cast<const uint16_t*>(a.x) + size_t(src) * a.K;
    table[i] = reinterpret_cast<uint64_t>(p);
  }
  if (i < a.K) zero_row[i] = 0;
}

template <int OUT, bool LOOKUP>
__global__ void __launch_bounds__(64 * GT_WAVES) grouped_dw_kernel(GroupedArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[GT_LDS];
  const int wv = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  long it = blockIdx.x >> 3;
  DwItem cur = dw_item(a, it);
  if (cur.e < 0) return;
  DwAddr<LOOKUP> ad;
  ad.set(a, cur);
  first_loads<DT_BF16>(smem, ad, 4);
  while (true) {
    it += gridDim.x >> 3;
    const DwItem next = dw_item(a, it);
    f32x16_t acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
    tile_products<DT_BF16, false, false, 4>(smem, ad, acc);
    stage_barrier();                             // every wave is through with the ring
    if (next.e >= 0) {
      ad.set(a, next);
      first_loads<DT_BF16>(smem, ad, 4);
    }
    const int m = cur.m0 + (wv >> 2) * 128;
    store_tile<OUT, 4>(smem, acc, reinterpret_cast<uint8_t*>(a.out) + size_t(cur.e) * a.N * a.K * (OUT == DT_F32 ? 4 : 2), m,
                       a.N, cur.n0 + (wv & 3) * 64, a.K, [](const auto& x, int q, int, int, int, float(&v)[4]) {
#pragma unroll
                         for (int t = 0; t < 4; ++t) v[t] = x[q + t];
                       });
    if (next.e < 0) return;
    cur = next;
  }
}

template <int OUT>
hipError_t launch_dw(const GroupedArgs& args, void* ws, hipStream_t st) {
  GroupedArgs a = args;
  const long per_expert = long((a.N + 255) / 256) * ((a.K + GT_N - 1) / GT_N);
  const long n_items = (per_expert + 7) / 8 * 8 * a.E;
  const dim3 grid(unsigned(n_items < GT_GRID ? n_items : GT_GRID));
  if (a.row_ids) {
    uint64_t* const table = reinterpret_cast<uint64_t*>(ws);
    const long entries = zero_row_entry(a);
    const long n = std::max(entries, long(a.K));
    hipLaunchKernelGGL(row_table_kernel, dim3(unsigned((n + 255) / 256)), dim3(256), 0, st, a, table,
                       reinterpret_cast<uint16_t*>(table + entries));
    a.row_table = table;
    hipLaunchKernelGGL((grouped_dw_kernel<OUT, true>), grid, dim3(64 * GT_WAVES), 0, st, a);
  } else {
    hipLaunchKernelGGL((grouped_dw_kernel<OUT, false>), grid, dim3(64 * GT_WAVES), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace

bool grouped_tile_fits(const GroupedArgs& a, int which, int in_dt) {
  if (in_dt == DT_I8) return a.K % 16 == 0;
  return in_dt == DT_BF16 && a.K % 8 == 0 && (which == GM_FORWARD || a.N % 8 == 0);
}

size_t grouped_tile_workspace(const GroupedArgs& a, int which, int in_dt) {
  if (!grouped_tile_fits(a, which, in_dt)) return 0;
  if (which != GM_GRAD_W)      // the parts' sums, a tile for each CU
    return rows_plan(a, which, in_dt).max_parts > 1 ? size_t(8 * GT_P) * 256 * GT_N * 4 : 0;
  return size_t(zero_row_entry(a)) * 8 + size_t(a.K) * 2;    // the rows' addresses and a row of zeros
}

hipError_t launch_grouped_tile(const GroupedArgs& a, int which, int in_dt, int out_dt, void* ws, hipStream_t st) {
  if (in_dt == DT_I8)
    return out_dt == DT_F32 ? launch_rows<DT_I8, DT_F32, GM_FORWARD>(a, ws, st)
                             : launch_rows<DT_I8, DT_BF16, GM_FORWARD>(a, ws, st);
  if (which == GM_FORWARD)
    return out_dt == DT_F32 ? launch_rows<DT_BF16, DT_F32, GM_FORWARD>(a, ws, st)
                            : launch_rows<DT_BF16, DT_BF16, GM_FORWARD>(a, ws, st);
  if (which == GM_GRAD_X) return launch_rows<DT_BF16, DT_BF16, GM_GRAD_X>(a, ws, st);
  return out_dt == DT_F32 ? launch_dw<DT_F32>(a, ws, st) : launch_dw<DT_BF16>(a, ws, st);
}

}  // namespace moe
