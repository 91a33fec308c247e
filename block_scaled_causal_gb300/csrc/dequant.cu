// MXFP8 rows back to values: element * 2^(scale - 127), exact in fp32 and rounded once to 16 bits.
//
// Memory-bound: 1 byte in, 2 out per element.  A thread takes 8 elements at a time, so that a warp's loads and stores are
// whole lines (16 elements, stored in two pieces of 16 bytes, took 13.6 us for 16.8 M elements in place of XX), DQ_ITEMS of them
// with all loads ahead of the first use.
#include "cache.cuh"

namespace bsc {
namespace {

constexpr int DQ_THREADS = 128, DQ_ITEMS = 4;

// Row r of the codes (in memory's order) has the scales of row scale_row(r).
__device__ __forceinline__ uint32_t scale_row(uint32_t r, int B, int S, int H, int layout) {
  const uint32_t x = r / H, h = r - x * H;
  uint32_t b, s;
  if (layout == 0) {
    b = x / S;
    s = x - b * S;
  } else {
    s = x / B;
    b = x - s * B;
  }
  return (b * H + h) * S + s;
}

template <int DT>
__global__ void __launch_bounds__(DQ_THREADS) dequantize_kernel(const uint8_t* x, const uint8_t* sc, void* y, int B, int S,
                                                                int H, int N, int layout, long long pieces) {
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const uint32_t per_row = N / 8;
  const bool in_order = H == 1 && (B == 1 || layout == 0);        // scales lie as their elements do
  uint2 v[DQ_ITEMS];
  float f[DQ_ITEMS];
  const long long block = (long long)blockIdx.x * (DQ_THREADS * DQ_ITEMS), i0 = block + threadIdx.x;
  const uint32_t row0 = (uint32_t)(block / per_row), p0 = (uint32_t)(block - (long long)row0 * per_row);   // below 2^31 rows
#pragma unroll
  for (int k = 0; k < DQ_ITEMS; ++k) {
    const long long i = i0 + k * DQ_THREADS;
    if (i >= pieces) break;
    v[k] = __ldcs(reinterpret_cast<const uint2*>(x) + i);
    long long at = i >> 2;
    if (!in_order) {
      const uint32_t p = p0 + threadIdx.x + k * DQ_THREADS, r = p / per_row;
      at = (long long)scale_row(row0 + r, B, S, H, layout) * (N / 32) + ((p - r * per_row) >> 2);
    }
    f[k] = scale_value(__ldca(sc + at));
  }
#pragma unroll
  for (int k = 0; k < DQ_ITEMS; ++k) {
    const long long i = i0 + k * DQ_THREADS;
    if (i >= pieces) break;
    uint32_t h[4], o[4];
    e4m3x4_to_f16(v[k].x, h[0], h[1]);
    e4m3x4_to_f16(v[k].y, h[2], h[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 y2 = __fmul2_rn(f16x2_to_f32(h[j]), make_float2(f[k], f[k]));
      o[j] = f32_to_act<DT>(y2.x, y2.y);
    }
    __stcs(reinterpret_cast<uint4*>(y) + i, make_uint4(o[0], o[1], o[2], o[3]));
  }
}

}  // namespace

cudaError_t launch_dequantize(const uint8_t* x, const uint8_t* sc, void* y, int B, int S, int H, int N, int layout, int dtype,
                              cudaStream_t st) {
  const long long pieces = (long long)B * S * H * (N / 8);
  const unsigned grid = (unsigned)((pieces + DQ_THREADS * DQ_ITEMS - 1) / (DQ_THREADS * DQ_ITEMS));
  return launch_early(dtype ? dequantize_kernel<1> : dequantize_kernel<0>, grid, DQ_THREADS, 0, st, 1, x, sc, y, B, S, H, N,
                      layout, pieces);
}

}  // namespace bsc
