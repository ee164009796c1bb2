// Row operators beside the grouped products: 8-bit codes of each row, and the
// combine of the expert-sorted rows into tokens with its gradients.  All of
// them read and write each value once and are bound by HBM (or, for a few
// rows, by the launch).  Measured in bf16: combine of 4096 tokens, top 2, rows
// of 4096, 19 us (5.1 TB/s); gradients of 1024 tokens, top 6, rows of 2048,
// 10.7 us; codes of 4096 rows of 4096 22-24 us (2.1-2.3 TB/s: two passes over
// the registers and an exact rounding each), of one row 5-6 us.
#include "grouped.hpp"

namespace moe {

namespace {

// Eight values of a row from p, which need not be aligned: the first n, the
// others zero.  Rows of any length are read and written 16 bytes a lane; only
// the last piece of a row that is no multiple of eight goes by elements.
template <int DT>
__device__ __forceinline__ void load8(const void* base, size_t i, int n, float (&v)[8]) {
  if constexpr (DT == DT_F32) {
    const float* p = reinterpret_cast<const float*>(base) + i;
    struct __attribute__((packed, aligned(4))) U { f32x4_t v; };
    if (n >= 8) {
      const f32x4_t a = reinterpret_cast<const U*>(p)[0].v, b = reinterpret_cast<const U*>(p)[1].v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? p[j] : 0.f;
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + i;
    struct __attribute__((packed, aligned(2))) U { u32x4_t v; };
    if (n >= 8) {
      const u32x4_t a = reinterpret_cast<const U*>(p)->v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[2 * j] = bf16_lo(a[j]), v[2 * j + 1] = bf16_hi(a[j]);
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? bf16_to_f32(p[j]) : 0.f;
  }
}
template <int DT>
__device__ __forceinline__ void store8(void* base, size_t i, int n, const float (&v)[8]) {
  if constexpr (DT == DT_F32) {
    float* p = reinterpret_cast<float*>(base) + i;
    struct __attribute__((packed, aligned(4))) U { f32x4_t v; };
    if (n >= 8) {
      reinterpret_cast<U*>(p)[0].v = f32x4_t{v[0], v[1], v[2], v[3]};
      reinterpret_cast<U*>(p)[1].v = f32x4_t{v[4], v[5], v[6], v[7]};
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = v[j];
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + i;
    struct __attribute__((packed, aligned(2))) U { u32x4_t v; };
    if (n >= 8) {
      reinterpret_cast<U*>(p)->v = u32x4_t{cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]), cvt_pk_bf16(v[4], v[5]),
                                           cvt_pk_bf16(v[6], v[7])};
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = uint16_t(f32_to_bf16(v[j]));
  }
}

// ---------------------------------------------------------------- codes --
// scale = max |x| / 127; code = nearest integer of x / scale, ties to even.
// x * (1 / s) rounds to the right code or to a neighbour of it.  The
// remainder x - q s is exact in fp32 (x and s have 24 bits and |q| <= 127, and
// the remainder, a multiple of the smaller last place, is at most about s),
// and so is its double: comparing that with s decides the code exactly.
__device__ __forceinline__ int code_of(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float r2 = 2.f * fmaf(-q, s, x);
  const bool odd = (int(q) & 1) != 0;
  if (r2 > s || (r2 == s && odd)) q += 1.f;
  else if (r2 < -s || (r2 == -s && odd)) q -= 1.f;
  return int(fminf(fmaxf(q, -127.f), 127.f));
}

// A work-group per row.  The first QUANT_KEEP pieces of eight values of each
// thread stay in registers between the two passes (rows of up to 8192 values
// with 256 threads, 32768 with 1024); longer rows are read twice.
constexpr int QUANT_KEEP = 4;

template <int DT, int THREADS>
__global__ void __launch_bounds__(THREADS) quantize_rows_kernel(QuantArgs a) {
  __shared__ uint32_t part[THREADS / 64];
  const int tid = threadIdx.x;
  const int pieces = (a.cols + 7) / 8;
  for (long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const size_t base = size_t(r) * a.cols;
    float keep[QUANT_KEEP][8];
    // the bits of |x| order as integers, with infinities and NaN above all numbers
    uint32_t top = 0;
    auto widen = [&](const float (&v)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
    };
#pragma unroll
    for (int k = 0; k < QUANT_KEEP; ++k) {
      const int c = tid + k * THREADS;
      load8<DT>(a.x, base + 8 * size_t(c), a.cols - 8 * c, keep[k]);
    }
#pragma unroll
    for (int k = 0; k < QUANT_KEEP; ++k) widen(keep[k]);
    for (int c = tid + QUANT_KEEP * THREADS; c < pieces; c += THREADS) {
      float v[8];
      load8<DT>(a.x, base + 8 * size_t(c), a.cols - 8 * c, v);
      widen(v);
    }
    for (int d = 32; d; d >>= 1) top = max(top, uint32_t(__shfl_xor(int(top), d)));
    if ((tid & 63) == 0) part[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) top = max(top, part[w]);
    __syncthreads();
    const bool finite = top < 0x7f800000u;
    const float scale = finite ? __uint_as_float(top) / 127.0f : __uint_as_float(0x7fc00000u);
    if (tid == 0) a.scale[r] = scale;
    const bool coded = finite && scale > 0.f;
    // scales whose reciprocal would overflow: everything times 2^64, which is exact
    const float up = scale < 0x1p-100f ? 0x1p64f : 1.f;
    const float s = scale * up, inv = 1.f / s;
    auto put_codes = [&](const float (&v)[8], int c) {
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j >> 2] |= (coded ? uint32_t(code_of(v[j] * up, s, inv)) & 0xffu : 0u) << (8 * (j & 3));
      int8_t* p = a.q + base + 8 * size_t(c);
      const int n = a.cols - 8 * c;
      if (n >= 8) {
        struct __attribute__((packed)) U { u32x2_t v; };
        reinterpret_cast<U*>(p)->v = u32x2_t{w[0], w[1]};
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) p[j] = int8_t(w[j >> 2] >> (8 * (j & 3)));
      }
    };
#pragma unroll
    for (int k = 0; k < QUANT_KEEP; ++k)
      if (tid + k * THREADS < pieces) put_codes(keep[k], tid + k * THREADS);
    for (int c = tid + QUANT_KEEP * THREADS; c < pieces; c += THREADS) {
      float v[8];
      load8<DT>(a.x, base + 8 * size_t(c), a.cols - 8 * c, v);
      put_codes(v, c);
    }
  }
}

// -------------------------------------------------------------- combine --
// A thread per eight values of a token.  The rows of G assignments are looked
// up and loaded together (G = top_k up to 8): one after another each would
// wait for its own entry of inv and then for its row.  Dropped assignments
// load row 0, which counts as zeros.
template <int YT, int OT, int G>
__global__ void __launch_bounds__(256) combine_rows_kernel(CombineArgs a) {
  const int pieces = (a.H + 7) / 8;
  const long n = long(a.T) * pieces;
  for (long i = long(blockIdx.x) * 256 + threadIdx.x; i < n; i += long(gridDim.x) * 256) {
    const long t = i / pieces;
    const int h = int(i - t * pieces) * 8;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < a.k && a.rows > 0; j0 += G) {
      bool kept[G];
      int p[G];
      float w[G], v[G][8];
#pragma unroll
      for (int u = 0; u < G; ++u) {
        const int j = j0 + u < a.k ? j0 + u : a.k - 1;
        p[u] = a.inv[t * a.k + j];
        w[u] = a.weights ? a.weights[t * a.k + j] : 1.f;
        kept[u] = j0 + u < a.k && p[u] >= 0 && p[u] < a.rows;
      }
#pragma unroll
      for (int u = 0; u < G; ++u) load8<YT>(a.y, size_t(kept[u] ? p[u] : 0) * a.H + h, a.H - h, v[u]);
#pragma unroll
      for (int u = 0; u < G; ++u)
#pragma unroll
        for (int q = 0; q < 8; ++q) s[q] = kept[u] ? fmaf(w[u], v[u][q], s[q]) : s[q];
    }
    store8<OT>(a.out, size_t(t) * a.H + h, a.H - h, s);
  }
}

// A wave per assignment: its row of dy, and the dot product for its weight.
template <int YT, int OT>
__global__ void __launch_bounds__(256) combine_backward_kernel(CombineArgs a) {
  const int lane = threadIdx.x & 63;
  const long n = long(a.T) * a.k;
  for (long f = long(blockIdx.x) * 4 + (threadIdx.x >> 6); f < n; f += long(gridDim.x) * 4) {
    const int p = a.inv[f];
    const bool kept = p >= 0 && p < a.rows;
    const size_t drow = size_t(f / a.k) * a.H, row = kept ? size_t(p) * a.H : 0;
    const float w = a.weights ? a.weights[f] : 1.f;
    float dot = 0.f;
    if (kept) {
#pragma unroll 4
      for (int h = lane * 8; h < a.H; h += 64 * 8) {
        float g[8], v[8];
        load8<OT>(a.dout, drow + h, a.H - h, g);
        if (a.dweights) {
          load8<YT>(a.y, row + h, a.H - h, v);
#pragma unroll
          for (int q = 0; q < 8; ++q) dot = fmaf(g[q], v[q], dot);
        }
        if (a.out) {
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = w * g[q];
          store8<YT>(a.out, row + h, a.H - h, v);
        }
      }
    }
    if (a.dweights) {
      for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
      if (lane == 0) a.dweights[f] = dot;
    }
  }
}

unsigned grid_of(long n) { return unsigned(n < (1L << 22) ? n : (1L << 22)); }

template <int YT, int OT, int G = 8>
hipError_t combine(const CombineArgs& a, hipStream_t st) {
  if constexpr (G > 1)
    if (a.k < G) return combine<YT, OT, G - 1>(a, st);
  const dim3 grid(grid_of((long(a.T) * ((a.H + 7) / 8) + 255) / 256));
  hipLaunchKernelGGL((combine_rows_kernel<YT, OT, G>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}
template <int YT, int OT>
hipError_t combine_back(const CombineArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((combine_backward_kernel<YT, OT>), dim3(grid_of((long(a.T) * a.k + 3) / 4)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const QuantArgs& a, int dt, hipStream_t st) {
  const dim3 grid(grid_of(a.rows));
  const bool wide = a.cols > 256 * QUANT_KEEP * 8;      // a row that 256 threads do not hold
  if (dt == DT_F32) {
    if (wide) hipLaunchKernelGGL((quantize_rows_kernel<DT_F32, 1024>), grid, dim3(1024), 0, st, a);
    else hipLaunchKernelGGL((quantize_rows_kernel<DT_F32, 256>), grid, dim3(256), 0, st, a);
  } else {
    if (wide) hipLaunchKernelGGL((quantize_rows_kernel<DT_BF16, 1024>), grid, dim3(1024), 0, st, a);
    else hipLaunchKernelGGL((quantize_rows_kernel<DT_BF16, 256>), grid, dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs& a, int y_dt, int out_dt, hipStream_t st) {
  if (y_dt == DT_F32) return out_dt == DT_F32 ? combine<DT_F32, DT_F32>(a, st) : combine<DT_F32, DT_BF16>(a, st);
  return out_dt == DT_F32 ? combine<DT_BF16, DT_F32>(a, st) : combine<DT_BF16, DT_BF16>(a, st);
}

hipError_t launch_combine_backward(const CombineArgs& a, int y_dt, int out_dt, hipStream_t st) {
  if (y_dt == DT_F32)
    return out_dt == DT_F32 ? combine_back<DT_F32, DT_F32>(a, st) : combine_back<DT_F32, DT_BF16>(a, st);
  return out_dt == DT_F32 ? combine_back<DT_BF16, DT_F32>(a, st) : combine_back<DT_BF16, DT_BF16>(a, st);
}

}  // namespace moe
