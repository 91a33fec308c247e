// The key/value cache written and read back (memory-bound streaming kernels; layouts in bsc.h).
//
// Write: for each 32-element block along D, e = clamp(floor(log2 amax) - emax, -127, 127) (or the
// smallest e at which nothing saturates), elements round(x * 2^-e) to nearest even.  Read: element *
// 2^e.  Both take one warp to 16 tokens of one (sequence, KV head) and one of K and V: a lane moves
// 16 bytes of activations per access, a 32-element block is 4 lanes, and all of a warp's loads are
// issued before the first is used (4 KB in flight per warp at D = 128).  Neighbouring warps take
// neighbouring heads, whose rows are neighbours in the activations; within a warp the 16 tokens'
// bytes are neighbours in the page.
#include "cache.cuh"

namespace bsc {
namespace {

constexpr int RW_TOKENS = 16;   // tokens per warp
constexpr int RW_WARPS = 4;

// Which piece of the work a warp has.
struct Piece {
  int b, t0, h, which;
};
__device__ __forceinline__ bool piece_of(const CacheRwArgs& a, Piece& p) {
  uint32_t i = blockIdx.x * RW_WARPS + (threadIdx.x >> 5);          // fewer than 2^31 warps: checked by the host
  const uint32_t tiles = (uint32_t)(a.T + RW_TOKENS - 1) / RW_TOKENS, H = a.c.Hkv;
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

template <int FMT, int D, int DT>
__global__ void __launch_bounds__(RW_WARPS * 32) cache_write_kernel(const CacheRwArgs a) {
  constexpr int LPR = D / 8, RPI = 32 / LPR, NI = RW_TOKENS / RPI;   // lanes per row, rows per access, accesses
  constexpr int RB = row_bytes<FMT, D>(), NB = D / 32;
  Piece w;
  if (!piece_of(a, w)) return;
  const int lane = threadIdx.x & 31, sub = lane / LPR, col = lane % LPR;
  const long long len = __ldg(a.pt.seq_lens + w.b);
  const int n = a.first ? min(max(__ldg(a.first + w.b), 0), a.T) : a.T;
  const int rows = min(n - w.t0, RW_TOKENS);
  if (rows <= 0) return;

  const RowStrides& xs = a.xs[w.which];
  const uint16_t* x = reinterpret_cast<const uint16_t*>(a.x[w.which]) + w.b * xs.b + w.h * xs.h + col * 8;
  uint4 v[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = i * RPI + sub;
    v[i] = r < rows ? __ldcs(reinterpret_cast<const uint4*>(x + (long long)(w.t0 + r) * xs.t)) : make_uint4(0, 0, 0, 0);
  }
  // lane r < 16 finds where row r goes: its page and its row in the page's [Hkv][page_size]
  int32_t bad = 0;
  int page = -1;
  uint32_t in_page = 0;
  if (lane < rows) page = cache_page(a.c, a.pt, w.b, (len < 0 ? 0 : len) - n + w.t0 + lane, w.h, in_page, bad);
  if (bad && a.dev_status) *a.dev_status = bad;

  uint8_t* const pool = (w.which ? a.c.v : a.c.k) + col * (RB / LPR);
  uint8_t* const pool_sc = w.which ? a.c.v_sc : a.c.k_sc;
  const long long ps = w.which ? a.c.v_ps : a.c.k_ps, ps_sc = w.which ? a.c.v_sc_ps : a.c.k_sc_ps;
  // the rows are mostly neighbours in one page: one address then, and constant steps
  const int page0 = __shfl_sync(0xFFFFFFFFu, page, 0);
  const uint32_t row0 = __shfl_sync(0xFFFFFFFFu, in_page, 0);
  const bool together = page0 >= 0 && __all_sync(0xFFFFFFFFu, lane >= rows || (page == page0 && in_page == row0 + lane));
  uint8_t* const dst0 = pool + page0 * ps + (unsigned long long)(row0 + sub) * RB;
  uint8_t* const sc0 = pool_sc + page0 * ps_sc + (unsigned long long)(row0 + sub) * NB;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (i * RPI >= rows) break;
    const int r = i * RPI + sub;
    // the block's maximum from bit patterns: without the sign they are in the values' order, NaN above Inf on top
    const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t mx = __vmaxu2(__vmaxu2(u[0] & 0x7FFF7FFFu, u[1] & 0x7FFF7FFFu), __vmaxu2(u[2] & 0x7FFF7FFFu, u[3] & 0x7FFF7FFFu));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
    const float am = act_to_f32<DT>(max(mx & 0xFFFFu, mx >> 16)).x;
    float inv;
    const uint32_t sb = block_scale<FMT>(am, a.rule, inv);
    // the row's scale word: each block's byte in its place, joined over the row's lanes
    uint32_t word = sb << (8 * (col >> 2));
#pragma unroll
    for (int o = 4; o < LPR; o <<= 1) word |= __shfl_xor_sync(0xFFFFFFFFu, word, o);
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = __fmul2_rn(act_to_f32<DT>(u[j]), make_float2(inv, inv));
      f[2 * j] = p.x;
      f[2 * j + 1] = p.y;
    }
    uint2 q;
    if (FMT == CACHE_FP4) {
      q.x = sb == 0xFFu ? 0x77777777u : cvt_e2m1x8(f);
    } else {
      q.x = cvt_e4m3x2(f[0], f[1]) | (uint32_t)cvt_e4m3x2(f[2], f[3]) << 16;
      q.y = cvt_e4m3x2(f[4], f[5]) | (uint32_t)cvt_e4m3x2(f[6], f[7]) << 16;
      if (sb == 0xFFu) q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    }
    uint8_t *dst = dst0 + i * RPI * RB, *sc = sc0 + i * RPI * NB;
    bool there = r < rows;
    if (!together) {
      const int pg = __shfl_sync(0xFFFFFFFFu, page, r);
      const uint32_t row = __shfl_sync(0xFFFFFFFFu, in_page, r);
      there = pg >= 0;
      dst = pool + pg * ps + (unsigned long long)row * RB;
      sc = pool_sc + pg * ps_sc + (unsigned long long)row * NB;
    }
    if (there) {
      if (FMT == CACHE_FP4) *reinterpret_cast<uint32_t*>(dst) = q.x;
      else *reinterpret_cast<uint2*>(dst) = q;
      if (col == 0) {
        if (NB == 4) *reinterpret_cast<uint32_t*>(sc) = word;
        else *reinterpret_cast<uint16_t*>(sc) = (uint16_t)word;
      }
    }
    __syncwarp();
  }
}

template <int FMT, int D, int DT>
__global__ void __launch_bounds__(RW_WARPS * 32) cache_read_kernel(const CacheRwArgs a) {
  constexpr int LPR = D / 8, RPI = 32 / LPR, NI = RW_TOKENS / RPI;
  constexpr int RB = row_bytes<FMT, D>(), NB = D / 32;
  Piece w;
  if (!piece_of(a, w)) return;
  const int lane = threadIdx.x & 31, sub = lane / LPR, col = lane % LPR;
  const long long len = __ldg(a.pt.seq_lens + w.b), start = a.first ? __ldg(a.first + w.b) : 0;
  const int rows = min(a.T - w.t0, RW_TOKENS);
  const uint8_t* const pool = w.which ? a.c.v : a.c.k;
  const uint8_t* const pool_sc = w.which ? a.c.v_sc : a.c.k_sc;
  const long long ps = w.which ? a.c.v_ps : a.c.k_ps, ps_sc = w.which ? a.c.v_sc_ps : a.c.k_sc_ps;

  // lane r < 16 finds row r: where its bytes are, and its scale word
  int32_t bad = 0;
  long long at = -1;
  uint32_t word = 0;
  if (lane < rows) {
    const long long pos = start + w.t0 + lane;
    uint32_t row = 0;
    const int page = pos < len ? cache_page(a.c, a.pt, w.b, pos, w.h, row, bad) : -1;
    if (page >= 0) {
      at = page * ps + (unsigned long long)row * RB;
      const uint8_t* const sc = pool_sc + page * ps_sc + (unsigned long long)row * NB;
      word = NB == 4 ? *reinterpret_cast<const uint32_t*>(sc) : *reinterpret_cast<const uint16_t*>(sc);
    }
  }
  if (bad && a.dev_status) *a.dev_status = bad;

  uint2 v[NI];
  long long src[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    src[i] = __shfl_sync(0xFFFFFFFFu, at, i * RPI + sub);
    v[i] = make_uint2(0, 0);
    if (src[i] >= 0) {
      if (FMT == CACHE_FP4)
        v[i].x = __ldcs(reinterpret_cast<const uint32_t*>(pool + src[i] + col * 4));
      else
        v[i] = __ldcs(reinterpret_cast<const uint2*>(pool + src[i] + col * 8));
    }
  }
  const RowStrides& xs = a.xs[w.which];
  uint16_t* const x = reinterpret_cast<uint16_t*>(a.x[w.which]) + w.b * xs.b + w.h * xs.h + col * 8;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    if (i * RPI >= rows) break;
    const int r = i * RPI + sub;
    const float s = scale_value((__shfl_sync(0xFFFFFFFFu, word, r) >> (8 * (col >> 2))) & 0xFFu);
    const float2 s2 = make_float2(s, s);
    uint32_t h[4];
    if (FMT == CACHE_FP4) {
      e2m1x8_to_f16(v[i].x, h);
    } else {
      e4m3x4_to_f16(v[i].x, h[0], h[1]);
      e4m3x4_to_f16(v[i].y, h[2], h[3]);
    }
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __fmul2_rn(f16x2_to_f32(h[j]), s2);
      o[j] = f32_to_act<DT>(f.x, f.y);           // the product is exact in fp32: one rounding
    }
    if (r < rows)
      __stcs(reinterpret_cast<uint4*>(x + (long long)(w.t0 + r) * xs.t),
             src[i] < 0 ? make_uint4(0, 0, 0, 0) : make_uint4(o[0], o[1], o[2], o[3]));
  }
}

using Kernel = void (*)(CacheRwArgs);
cudaError_t launch(Kernel k, const CacheRwArgs& a, cudaStream_t st) {
  const long long warps = 2LL * a.B * ((a.T + RW_TOKENS - 1) / RW_TOKENS) * a.c.Hkv;
  k<<<(unsigned)((warps + RW_WARPS - 1) / RW_WARPS), RW_WARPS * 32, 0, st>>>(a);
  return cudaGetLastError();
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
