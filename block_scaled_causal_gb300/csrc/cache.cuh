// What the kernels of the key/value cache share: element formats, scale rule, addresses, launch.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "bsc_internal.h"
#include "ptx.cuh"

namespace bsc {

constexpr int CACHE_FP8 = 0, CACHE_FP4 = 1;   // bsc_cache_format
constexpr int32_t CACHE_BAD_PAGE = 0x201, CACHE_BAD_LEN = 0x202;

// Bytes of one token's D elements of one head.
template <int FMT, int D>
constexpr int row_bytes() { return FMT == CACHE_FP4 ? D / 2 : D; }

// Largest binade of an element, and the significand (fp32 fraction bits) of its largest value:
// E4M3 448 = 1.75 * 2^8, E2M1 6 = 1.5 * 2^2.
template <int FMT>
struct Elem {
  static constexpr uint32_t emax = FMT == CACHE_FP4 ? 2u : 8u;
  static constexpr uint32_t top_frac = FMT == CACHE_FP4 ? 0x400000u : 0x600000u;
};

// The scale byte of a block from its absolute maximum (0xFF for NaN/Inf), and 2^-(byte - 127): the
// rule of e8m0_from_amax for either format.  `up` is ceil_carry's: 0 under the floor rule, else what carries a
// fraction above the largest element's into the exponent.  fp32-subnormal maxima clamp to byte 0.
template <int FMT>
__device__ __forceinline__ uint32_t ceil_carry(int ceil_rule) {
  return ceil_rule ? 0x7FFFFFu - Elem<FMT>::top_frac : 0u;
}
template <int FMT>
__device__ __forceinline__ uint32_t block_scale(float amax, uint32_t up, float& inv) {
  const uint32_t bits = __float_as_uint(amax);
  const uint32_t sb = max((bits + up) >> 23, Elem<FMT>::emax) - Elem<FMT>::emax;
  inv = __uint_as_float((254u - sb) << 23);   // sb <= 253: a normal fp32
  return bits >= 0x7F800000u ? 0xFFu : sb;
}

// 2^(byte - 127) in fp32; byte 0 is the fp32-subnormal 2^-127, byte 255 NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 0u ? __uint_as_float(0x00400000u) : byte == 255u ? __uint_as_float(0x7FC00000u)
                                                                  : __uint_as_float(byte << 23);
}

// E2M1: nearest even, saturated to +-6.
// Eight fp32 -> eight E2M1, the first in the lowest nibble.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{ .reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d}; }"
      : "=r"(r) : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}
// The four bytes (eight E2M1) of a word -> f16x2 each (exact), low nibble in the low half.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d; }"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}
// The four E4M3 of a word -> two f16x2 (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& h0, uint32_t& h1) {
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }" : "=r"(h0), "=r"(h1) : "r"(w));
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// The largest magnitude of values, NaN if any is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float amax8(const float2 (&f)[4]) {
  const float a = max3_nan(fabsf(f[0].x), fabsf(f[0].y), fabsf(f[1].x)), b = max3_nan(fabsf(f[1].y), fabsf(f[2].x), fabsf(f[2].y));
  return max_nan(max3_nan(a, b, fabsf(f[3].x)), fabsf(f[3].y));
}
// Eight fp32 of a block with scale byte sb, whose inverse is inv, as elements.
__device__ __forceinline__ uint2 quant8_e4m3(const float2 (&f)[4], float inv, uint32_t sb) {
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = __fmul2_rn(f[i], make_float2(inv, inv));
    r[i] = cvt_e4m3x2(y.x, y.y);
  }
  if (sb == 0xFFu) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  return make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
}
__device__ __forceinline__ uint32_t quant8_e2m1(const float2 (&f)[4], float inv, uint32_t sb) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __fmul2_rn(f[i], make_float2(inv, inv));
    y[2 * i] = p.x;
    y[2 * i + 1] = p.y;
  }
  return sb == 0xFFu ? 0x77777777u : cvt_e2m1x8(y);
}

// Activations: bf16 (DT = 0) or fp16 (DT = 1), two to a word.
template <int DT>
__device__ __forceinline__ float2 act_to_f32(uint32_t w) {
  if (DT == 0) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return f16x2_to_f32(w);
}
template <int DT>
__device__ __forceinline__ uint32_t f32_to_act(float lo, float hi) {
  if (DT == 0) return pack_bf16x2(lo, hi);
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The same with the type known at run time.
__device__ __forceinline__ float2 act_to_f32(uint32_t w, int fp16) { return fp16 ? act_to_f32<1>(w) : act_to_f32<0>(w); }
__device__ __forceinline__ uint32_t f32_to_act(float lo, float hi, int fp16) {
  return fp16 ? f32_to_act<1>(lo, hi) : f32_to_act<0>(lo, hi);
}

// Reports a code.  The status word keeps the first one it is given, whichever of the library's calls gave it.
__device__ __forceinline__ void report(int32_t* dev_status, int32_t code) {
  if (dev_status) atomicCAS(dev_status, 0, code);
}

// The page that holds position `pos` of sequence `b`, or -1 where there is none, and the row of that position and
// head in the page's [Hkv][page_size]; `bad` collects a status code.
__device__ __forceinline__ int cache_page(const CachePools& c, const CacheTable& pt, int b, long long pos, int h,
                                          uint32_t& row, int32_t& bad) {
  if (pos < 0) return -1;
  if (pos >= (long long)pt.max_pages * c.page_size) {   // < 2^31
    bad = CACHE_BAD_LEN;
    return -1;
  }
  const uint32_t lp = (uint32_t)pos / (uint32_t)c.page_size;
  row = (uint32_t)h * c.page_size + (uint32_t)pos - lp * c.page_size;
  const int page = __ldca(pt.table + b * pt.stride + lp);
  if (page < 0 || page >= c.num_pages) {
    bad = CACHE_BAD_PAGE;
    return -1;
  }
  return page;
}

// Programmatic dependence.  A cache kernel of at most one block per SM lets the next one of the stream be launched as soon
// as its own blocks run, and every one touches no memory before the one ahead of it has finished (but for the lengths
// that an attention's join reads, see there): of a step's write and attention, the second's launch is hidden behind
// the first.  (A token each, written and read back: 4.55 -> 3.7 us.  With larger grids the next kernel's waiting blocks
// are in the way: 8 ragged prompts written and read 35.0 -> 35.9 us, 368 blocks of attention 10.9 -> 11.4.)
//
// A kernel gives the signal after its own wait, never before: then all but one of the kernels ahead of a resident block have
// finished, and that one loads nothing through L1 that it stores, so no L1 can hold an old copy of what the block reads once
// its wait is over.  (The norm, which may store in place, loads its rows past L1 by cp.async.cg; rotations in place give no
// signal; the scores that a choice of pages keeps in its workspace are read by the cluster that wrote them, behind its
// barrier.)  Nor is anything read by ld.global.nc (__ldg), which may take it for constant while a kernel lives and
// promises nothing of stores made meanwhile: lengths, page ids, queries and scales come by ordinary loads (__ldca).
constexpr unsigned EARLY_BLOCKS = 152;
__device__ __forceinline__ void next_kernel_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A launch that may start early; cluster: blocks per cluster (1: none).
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int block, size_t smem, cudaStream_t st, int cluster,
                         const A&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace bsc
