// The key/value cache written and read back (memory-bound streaming kernels; layouts in bsc.h).
//
// Write: for each 32-element block along D, e = clamp(floor(log2 amax) - emax, -127, 127) (or the
// smallest e at which nothing saturates), elements round(x * 2^-e) to nearest even.  Read: element *
// 2^e.  Both take one warp to 16 tokens of one (sequence, KV head) and one of K and V, and issue all of a
// warp's loads before the first is used (4 KB of activations in flight per warp at D = 128).  Neighbouring warps
// take neighbouring heads, whose rows are neighbours in the activations; within a warp the 16 tokens'
// bytes are neighbours in the page.
//
// What bounds them.  Memory, once the instructions are few enough: 8 elements per lane and access (4 lanes to a
// block) took 950 warp instructions per warp in the write and 724 in the read, and both ran at the issue
// rate (22 and 17 us for 32K tokens of 4 heads, 85 MB); 16 elements per lane share the block's scale, addresses and
// shuffles.  Write then read of those, 4 bits, captured together: 34.6 -> 28.5 us (6.0 TB/s of 170 MB); of 8
// ragged prompts in 8 bits 38.9 -> 35.1 us; a read alone of 4 x 16K tokens of 16 heads 100.7 us (6.7 TB/s).
#include "cache.cuh"

namespace bsc {
namespace {

// Tokens per warp, warps per block: 32 tokens, or 2 or 8 warps, are within 2% on long prompts; 8 ragged prompts take
// 35.0 us with 16 and 4, 35.7 with 32, 37.1 and 35.8 with 2 and 8 warps.
constexpr int RW_TOKENS = 16, RW_WARPS = 4;

// Which piece of the work a warp has.
struct Piece {
  int b, t0, h, which;
};
__device__ __forceinline__ bool piece_of(const CacheRwArgs& a, Piece& p) {
  uint32_t i = blockIdx.x * RW_WARPS + (threadIdx.x >> 5);          // fewer than 2^31 warps: checked by the host
  const uint32_t tiles = ((uint32_t)a.T + RW_TOKENS - 1) / RW_TOKENS, H = a.c.Hkv;
  if (i >= 2u * a.B * tiles * H) return false;
  uint32_t next = i / H;
  p.h = (int)(i - next * H);
  p.which = (int)(next & 1u);
  i = next >> 1;
  next = i / tiles;
  p.t0 = (int)(i - next * tiles) * RW_TOKENS;
  p.b = (int)next;
  return true;
}

// Where a warp's rows are in the pools.  Lane r < 16 has row r's page (-1: none) and its row in the page; mostly
// they are neighbours in one page, and then `first` alone gives every address.
struct Rows {
  int page, page0;
  uint32_t row, row0;
  bool together;
  __device__ __forceinline__ void settle(int lane, int rows) {
    page0 = __shfl_sync(0xFFFFFFFFu, page, 0);
    row0 = __shfl_sync(0xFFFFFFFFu, row, 0);
    together = page0 >= 0 && __all_sync(0xFFFFFFFFu, lane >= rows || (page == page0 && row == row0 + lane));
  }
};

// Both kernels: a lane has two 8-element pieces, 16 elements apart, of one block of one row (two lanes to a block), so
// that a lane pair touches whole 32-byte sectors of the activations and the block's scale is worked out for 16
// elements at a time.
template <int FMT, int D, int DT>
__global__ void __launch_bounds__(RW_WARPS * 32) cache_write_kernel(const CacheRwArgs a) {
  constexpr int LPR = D / 16, RPI = 32 / LPR, NI = RW_TOKENS / RPI;   // lanes per row, rows per access, accesses
  constexpr int RB = row_bytes<FMT, D>(), NB = D / 32;
  Piece w;
  const bool mine = piece_of(a, w);
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  if (!mine) return;
  const int lane = threadIdx.x & 31, sub = lane / LPR, blk = lane % LPR >> 1, half = lane & 1;
  const long long len = __ldca(a.pt.seq_lens + w.b);
  const int n = a.first ? min(max(__ldca(a.first + w.b), 0), a.T) : a.T;
  const int rows = min(n - w.t0, RW_TOKENS);
  if (rows <= 0) return;

  const RowStrides& xs = a.xs[w.which];
  const uint16_t* x = reinterpret_cast<const uint16_t*>(a.x[w.which]) + w.b * xs.b + w.h * xs.h + blk * 32 + half * 8 +
                      (long long)(w.t0 + sub) * xs.t;
  uint4 v[NI][2];
  if (rows == RW_TOKENS) {
#pragma unroll
    for (int i = 0; i < NI; ++i, x += RPI * xs.t) {
      v[i][0] = __ldcs(reinterpret_cast<const uint4*>(x));
      v[i][1] = __ldcs(reinterpret_cast<const uint4*>(x + 16));
    }
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i, x += RPI * xs.t) {
      v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
      if (i * RPI + sub < rows) {
        v[i][0] = __ldcs(reinterpret_cast<const uint4*>(x));
        v[i][1] = __ldcs(reinterpret_cast<const uint4*>(x + 16));
      }
    }
  }
  Rows at{-1, -1, 0, 0, false};
  int32_t bad = 0;
  if (lane < rows) at.page = cache_page(a.c, a.pt, w.b, (len < 0 ? 0 : len) - n + w.t0 + lane, w.h, at.row, bad);
  if (bad) report(a.dev_status, bad);
  at.settle(lane, rows);

  constexpr int PB = RB / (D / 8);               // bytes of a piece: 4 or 8
  uint8_t* const pool = (w.which ? a.c.v : a.c.k) + blk * 4 * PB + half * 2 * PB;
  uint8_t* const pool_sc = (w.which ? a.c.v_sc : a.c.k_sc) + blk;
  const long long ps = w.which ? a.c.v_ps : a.c.k_ps, ps_sc = w.which ? a.c.v_sc_ps : a.c.k_sc_ps;
  uint8_t* const dst0 = pool + at.page0 * ps + (unsigned long long)(at.row0 + sub) * RB;
  uint8_t* const sc0 = pool_sc + at.page0 * ps_sc + (unsigned long long)(at.row0 + sub) * NB;
  const uint32_t up = ceil_carry<FMT>(a.rule);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (i * RPI >= rows) break;
    const int r = i * RPI + sub;
    // the block's maximum from bit patterns: without the sign they are in the values' order, NaN above Inf on top
    const uint32_t u[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
    uint32_t mx = u[0] & 0x7FFF7FFFu;
#pragma unroll
    for (int j = 1; j < 8; ++j) mx = __vmaxu2(mx, u[j] & 0x7FFF7FFFu);
    mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    float inv;
    const uint32_t sb = block_scale<FMT>(act_to_f32<DT>(max(mx & 0xFFFFu, mx >> 16)).x, up, inv);
    uint32_t q[2][2];                              // the two pieces' bytes
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p = __fmul2_rn(act_to_f32<DT>(u[4 * k + j]), make_float2(inv, inv));
        f[2 * j] = p.x;
        f[2 * j + 1] = p.y;
      }
      if (FMT == CACHE_FP4) {
        q[k][0] = sb == 0xFFu ? 0x77777777u : cvt_e2m1x8(f);
      } else {
        q[k][0] = sb == 0xFFu ? 0x7F7F7F7Fu : cvt_e4m3x2(f[0], f[1]) | (uint32_t)cvt_e4m3x2(f[2], f[3]) << 16;
        q[k][1] = sb == 0xFFu ? 0x7F7F7F7Fu : cvt_e4m3x2(f[4], f[5]) | (uint32_t)cvt_e4m3x2(f[6], f[7]) << 16;
      }
    }
    // the pair swaps its inner pieces: 0 2 | 1 3 becomes 0 1 | 2 3
#pragma unroll
    for (int k = 0; k < PB / 4; ++k) {
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, half ? q[0][k] : q[1][k], 1);
      q[0][k] = half ? got : q[0][k];
      q[1][k] = half ? q[1][k] : got;
    }
    uint8_t *dst = dst0 + i * RPI * RB, *sc = sc0 + i * RPI * NB;
    bool there = r < rows;
    if (!at.together) {
      const int pg = __shfl_sync(0xFFFFFFFFu, at.page, r);
      const uint32_t row = __shfl_sync(0xFFFFFFFFu, at.row, r);
      there = pg >= 0;
      dst = pool + pg * ps + (unsigned long long)row * RB;
      sc = pool_sc + pg * ps_sc + (unsigned long long)row * NB;
    }
    if (there) {
      if (FMT == CACHE_FP4) *reinterpret_cast<uint2*>(dst) = make_uint2(q[0][0], q[1][0]);
      else *reinterpret_cast<uint4*>(dst) = make_uint4(q[0][0], q[0][1], q[1][0], q[1][1]);
      if (half == 0) *sc = (uint8_t)sb;
    }
  }
}

template <int FMT, int D, int DT>
__global__ void __launch_bounds__(RW_WARPS * 32) cache_read_kernel(const CacheRwArgs a) {
  constexpr int LPR = D / 16, RPI = 32 / LPR, NI = RW_TOKENS / RPI;
  constexpr int RB = row_bytes<FMT, D>(), NB = D / 32, PB = RB / (D / 8);
  Piece w;
  const bool mine = piece_of(a, w);
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  if (!mine) return;
  const int lane = threadIdx.x & 31, sub = lane / LPR, blk = lane % LPR >> 1, half = lane & 1;
  const long long len = __ldca(a.pt.seq_lens + w.b), start = a.first ? __ldca(a.first + w.b) : 0;
  const int rows = min(a.T - w.t0, RW_TOKENS);
  Rows at{-1, -1, 0, 0, false};
  int32_t bad = 0;
  const long long pos = start + w.t0 + lane;
  if (lane < rows && pos < len) at.page = cache_page(a.c, a.pt, w.b, pos, w.h, at.row, bad);
  if (bad) report(a.dev_status, bad);
  at.settle(lane, rows);

  const uint8_t* const pool = (w.which ? a.c.v : a.c.k) + blk * 4 * PB + half * PB;
  const uint8_t* const pool_sc = (w.which ? a.c.v_sc : a.c.k_sc) + blk;
  const long long ps = w.which ? a.c.v_ps : a.c.k_ps, ps_sc = w.which ? a.c.v_sc_ps : a.c.k_sc_ps;
  uint2 v[NI][2];                                 // the two pieces' bytes
  uint32_t sb[NI];
  auto load = [&](int i, const uint8_t* src, const uint8_t* sc) {
    sb[i] = __ldca(sc);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (FMT == CACHE_FP4) v[i][k].x = __ldcs(reinterpret_cast<const uint32_t*>(src + 2 * k * PB));
      else v[i][k] = __ldcs(reinterpret_cast<const uint2*>(src + 2 * k * PB));
    }
  };
  uint32_t there = 0;                             // bit i: row i RPI + sub is held
  if (at.together && rows == RW_TOKENS) {
    const uint8_t* const src = pool + at.page0 * ps + (unsigned long long)(at.row0 + sub) * RB;
    const uint8_t* const sc = pool_sc + at.page0 * ps_sc + (unsigned long long)(at.row0 + sub) * NB;
    there = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < NI; ++i) load(i, src + i * RPI * RB, sc + i * RPI * NB);
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int pg = __shfl_sync(0xFFFFFFFFu, at.page, i * RPI + sub);
      const uint32_t row = __shfl_sync(0xFFFFFFFFu, at.row, i * RPI + sub);
      v[i][0] = v[i][1] = make_uint2(0, 0);
      sb[i] = 0;
      if (pg >= 0) {
        there |= 1u << i;
        load(i, pool + pg * ps + (unsigned long long)row * RB, pool_sc + pg * ps_sc + (unsigned long long)row * NB);
      }
    }
  }
  const RowStrides& xs = a.xs[w.which];
  uint16_t* x = reinterpret_cast<uint16_t*>(a.x[w.which]) + w.b * xs.b + w.h * xs.h + blk * 32 + half * 8 +
                (long long)(w.t0 + sub) * xs.t;
#pragma unroll
  for (int i = 0; i < NI; ++i, x += RPI * xs.t) {
    if (i * RPI >= rows) break;
    const float s = scale_value(sb[i]);
    const float2 s2 = make_float2(s, s);
    const bool held = (there >> i) & 1u;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t h[4];
      if (FMT == CACHE_FP4) {
        e2m1x8_to_f16(v[i][k].x, h);
      } else {
        e4m3x4_to_f16(v[i][k].x, h[0], h[1]);
        e4m3x4_to_f16(v[i][k].y, h[2], h[3]);
      }
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __fmul2_rn(f16x2_to_f32(h[j]), s2);
        o[j] = held ? f32_to_act<DT>(f.x, f.y) : 0u;           // the product is exact in fp32: one rounding
      }
      if (i * RPI + sub < rows) __stcs(reinterpret_cast<uint4*>(x + 16 * k), make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

using Kernel = void (*)(CacheRwArgs);
cudaError_t launch(Kernel k, const CacheRwArgs& a, cudaStream_t st) {
  const long long warps = 2LL * a.B * ((a.T + RW_TOKENS - 1LL) / RW_TOKENS) * a.c.Hkv;
  return launch_early(k, (unsigned)((warps + RW_WARPS - 1) / RW_WARPS), RW_WARPS * 32, 0, st, 1, a);
}

}  // namespace

cudaError_t launch_cache_write(const CacheRwArgs& a, int format, int D, int dtype, cudaStream_t st) {
  static const Kernel k[8] = {cache_write_kernel<0, 64, 0>,  cache_write_kernel<0, 64, 1>,
                              cache_write_kernel<0, 128, 0>, cache_write_kernel<0, 128, 1>,
                              cache_write_kernel<1, 64, 0>,  cache_write_kernel<1, 64, 1>,
                              cache_write_kernel<1, 128, 0>, cache_write_kernel<1, 128, 1>};
  return launch(k[format * 4 + (D == 128) * 2 + dtype], a, st);
}

cudaError_t launch_cache_read(const CacheRwArgs& a, int format, int D, int dtype, cudaStream_t st) {
  static const Kernel k[8] = {cache_read_kernel<0, 64, 0>,  cache_read_kernel<0, 64, 1>,
                              cache_read_kernel<0, 128, 0>, cache_read_kernel<0, 128, 1>,
                              cache_read_kernel<1, 64, 0>,  cache_read_kernel<1, 64, 1>,
                              cache_read_kernel<1, 128, 0>, cache_read_kernel<1, 128, 1>};
  return launch(k[format * 4 + (D == 128) * 2 + dtype], a, st);
}

}  // namespace bsc
