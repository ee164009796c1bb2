// Row operators beside the grouped products: 8-bit codes of each row, and the
// combine of the expert-sorted rows into tokens with its gradients.  All of
// them read and write each value once and are bound by HBM (or, for a few
// rows, by the launch).
#include "grouped.hpp"

namespace moe {

namespace {

// ---------------------------------------------------------------- codes --
// scale = max |x| / 127; code = nearest integer of x / scale, ties to even.
// rint(x / s) alone can be off where the fp32 quotient rounds onto a half;
// the remainder x - q s is exact in fp32 (x and s have 24 bits and |q| <= 127,
// and the remainder, a multiple of the smaller last place, is at most about
// s / 2), and so is its double: comparing that with s decides the code exactly.
__device__ __forceinline__ int code_of(float x, float s) {
  float q = rintf(x / s);
  const float r2 = 2.f * fmaf(-q, s, x);
  const bool odd = (int(q) & 1) != 0;
  if (r2 > s || (r2 == s && odd)) q += 1.f;
  else if (r2 < -s || (r2 == -s && odd)) q -= 1.f;
  return int(fminf(fmaxf(q, -127.f), 127.f));
}

template <int DT>
__device__ __forceinline__ float elem(const void* p, size_t i) {
  if constexpr (DT == DT_F32) return reinterpret_cast<const float*>(p)[i];
  else return bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void put(void* p, size_t i, float v) {
  if constexpr (DT == DT_F32) reinterpret_cast<float*>(p)[i] = v;
  else reinterpret_cast<uint16_t*>(p)[i] = uint16_t(f32_to_bf16(v));
}

template <int DT>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantArgs a) {
  __shared__ uint32_t part[4];
  const int tid = threadIdx.x;
  for (long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const size_t base = size_t(r) * a.cols;
    // the bits of |x| order as integers, with infinities and NaN above all numbers
    uint32_t top = 0;
    for (int c = tid; c < a.cols; c += 256) top = max(top, __float_as_uint(elem<DT>(a.x, base + c)) & 0x7fffffffu);
    for (int d = 32; d; d >>= 1) top = max(top, uint32_t(__shfl_xor(int(top), d)));
    if ((tid & 63) == 0) part[tid >> 6] = top;
    __syncthreads();
    top = max(max(part[0], part[1]), max(part[2], part[3]));
    __syncthreads();
    const bool finite = top < 0x7f800000u;
    const float s = finite ? __uint_as_float(top) / 127.0f : __uint_as_float(0x7fc00000u);
    if (tid == 0) a.scale[r] = s;
    for (int c = tid; c < a.cols; c += 256)
      a.q[base + c] = finite && s > 0.f ? int8_t(code_of(elem<DT>(a.x, base + c), s)) : int8_t(0);
  }
}

// -------------------------------------------------------------- combine --
template <int YT, int OT>
__global__ void __launch_bounds__(256) combine_rows_kernel(CombineArgs a) {
  const long n = long(a.T) * a.H;
  for (long i = long(blockIdx.x) * 256 + threadIdx.x; i < n; i += long(gridDim.x) * 256) {
    const long t = i / a.H;
    const int h = int(i - t * a.H);
    float s = 0.f;
    for (int j = 0; j < a.k; ++j) {
      const int p = a.inv[t * a.k + j];
      if (p < 0 || p >= a.rows) continue;
      s = fmaf(a.weights ? a.weights[t * a.k + j] : 1.f, elem<YT>(a.y, size_t(p) * a.H + h), s);
    }
    put<OT>(a.out, i, s);
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
    if (kept)
      for (int h = lane; h < a.H; h += 64) {
        const float g = elem<OT>(a.dout, drow + h);
        if (a.out) put<YT>(a.out, row + h, w * g);
        if (a.dweights) dot = fmaf(g, elem<YT>(a.y, row + h), dot);
      }
    if (a.dweights) {
      for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
      if (lane == 0) a.dweights[f] = dot;
    }
  }
}

unsigned grid_of(long n) { return unsigned(n < (1L << 22) ? n : (1L << 22)); }

template <int YT, int OT>
hipError_t combine(const CombineArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((combine_rows_kernel<YT, OT>), dim3(grid_of((long(a.T) * a.H + 255) / 256)), dim3(256), 0, st, a);
  return hipGetLastError();
}
template <int YT, int OT>
hipError_t combine_back(const CombineArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((combine_backward_kernel<YT, OT>), dim3(grid_of((long(a.T) * a.k + 3) / 4)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const QuantArgs& a, int dt, hipStream_t st) {
  if (dt == DT_F32) hipLaunchKernelGGL(quantize_rows_kernel<DT_F32>, dim3(grid_of(a.rows)), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(quantize_rows_kernel<DT_BF16>, dim3(grid_of(a.rows)), dim3(256), 0, st, a);
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
