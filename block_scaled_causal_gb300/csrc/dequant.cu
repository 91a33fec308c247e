// MXFP8 rows back to values: element * 2^(scale - 127), exact in fp32 and rounded once to 16 bits.
//
// Memory-bound: 1 byte in, 2 out per element.  A thread takes 8 elements at a time, so that a warp's loads and stores are
// whole lines, DQ_ITEMS of them with all loads ahead of the first use.  For 16.8 M elements of Q, cold: 9.9 us; with 16 elements
// per thread, stored in two pieces of 16 bytes, 13.6; with 8 items and 256 threads 12.2 (one wave and a little); of that 2 us were
// divisions for the scales' place.  33.6 M elements in one order with their scales: 15.6 us, 6.5 TB/s.
#include "cache.cuh"

namespace bsc {
namespace {

constexpr int DQ_THREADS = 128, DQ_ITEMS = 4;

// Division of numbers below 2^31 by d: with 2^(s-1) < d <= 2^s and m = ceil(2^(31+s) / d), which is below 2^32, n m differs
// from n 2^(31+s) / d by less than n d / d <= 2^31 <= 2^(31+s) / d, so n m >> (31 + s) is the whole quotient.
struct Divisor {
  uint32_t d, m;
  int s;
  explicit Divisor(uint32_t by) : d(by), s(0) {
    while ((1ull << s) < by) ++s;
    m = (uint32_t)(((1ull << (31 + s)) + by - 1) / by);
  }
  __device__ __forceinline__ uint32_t into(uint32_t n, uint32_t& rest) const {
    const uint32_t q = (uint32_t)(((unsigned long long)n * m) >> (31 + s));
    rest = n - q * d;
    return q;
  }
};

template <int DT>
__global__ void __launch_bounds__(DQ_THREADS) dequantize_kernel(const uint8_t* x, const uint8_t* sc, void* y, Divisor per_row,
                                                                Divisor heads, Divisor inner, int S, int sbhd, int in_order,
                                                                long long pieces) {
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  uint2 v[DQ_ITEMS];
  float f[DQ_ITEMS];
  const long long block = (long long)blockIdx.x * (DQ_THREADS * DQ_ITEMS), i0 = block + threadIdx.x;
  const uint32_t row0 = (uint32_t)(block / per_row.d), p0 = (uint32_t)(block - (long long)row0 * per_row.d);
#pragma unroll
  for (int k = 0; k < DQ_ITEMS; ++k) {
    const long long i = i0 + k * DQ_THREADS;
    if (i >= pieces) break;
    v[k] = __ldcs(reinterpret_cast<const uint2*>(x) + i);
    long long at = i >> 2;
    if (!in_order) {               // the row in memory's order is (b, s, h) or (s, b, h), its scales are those of (b, h, s)
      uint32_t p, h, minor;
      const uint32_t r = row0 + per_row.into(p0 + threadIdx.x + k * DQ_THREADS, p);
      const uint32_t major = inner.into(heads.into(r, h), minor);
      const uint32_t bb = sbhd ? minor : major, s = sbhd ? major : minor;
      at = (long long)((bb * heads.d + h) * S + s) * (per_row.d / 4) + (p >> 2);
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
  // with one head of one sequence (or whole sequences in order) the scales lie as their elements do
  return launch_early(dtype ? dequantize_kernel<1> : dequantize_kernel<0>, grid, DQ_THREADS, 0, st, 1, x, sc, y, Divisor(N / 8),
                      Divisor(H), Divisor(layout ? B : S), S, layout, (int)(H == 1 && (B == 1 || layout == 0)), pieces);
}

}  // namespace bsc
