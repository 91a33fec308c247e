// Rotary positions of Q and K: to 16 bits, to MXFP8 rows, and into the key/value cache.
//
// Pair i of a head's first `rot` elements, (x_i, x_{i + rot/2}) or, interleaved, (x_2i, x_2i+1), turns by the angle p f_i of
// its token's position p: (a, b) -> m (a cos - b sin, a sin + b cos).  The gradient turns by -p f_i.  Elements from `rot` on
// pass through.
//
// Angles.  f_i is held as a 64-bit fraction of a turn, so p * f_i mod 2^64 is the angle's fraction of a turn, exactly,
// whatever the position; its upper 32 bits (a step of 1.5e-9 radians) become an fp32 in [-1, 1) half turns for
// sincospif.  No table of positions is read and there is no longest one.  A block works out each of its tokens' cosines
// once, in shared memory, for all heads.
//
// What bounds it: memory, once those are shared by enough heads.  A lane has 8 neighbouring elements of one head (16
// bytes); D / 8 lanes are a head, and half pairs exchange their packed elements with the lane rot / 16 away.  Four
// neighbouring lanes are an MX block.  All loads of ROPE_BATCH heads are issued ahead of the first use.
#include "cache.cuh"

namespace bsc {
namespace {

constexpr int ROPE_THREADS = 128, ROPE_WARPS = ROPE_THREADS / 32, ROPE_BATCH = 4;
constexpr int MOST_TOKENS = 16, MOST_ANGLES = 1024;   // of a block
enum { TO_ACT, TO_MX, TO_CACHE };

template <int DT, bool INTER, int OUT, int FMT, int DC>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const RopeArgs a) {
  __shared__ __align__(16) float cosines[MOST_ANGLES], sines[MOST_ANGLES];
  __shared__ int page_of[MOST_TOKENS];           // TO_CACHE: the token's page, -1 where it has none; -2: not a token
  __shared__ uint32_t slot_of[MOST_TOKENS];
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const int tiles = (a.T + a.tt - 1) / a.tt, b = blockIdx.x / tiles, t0 = (blockIdx.x - b * tiles) * a.tt;
  const int tokens = min(a.tt, a.T - t0), P = a.rot / 2;
  // ---- the tokens' positions, pages and angles ----
  int n = 0;
  long long len = 0;
  if (OUT == TO_CACHE) {
    len = __ldca(a.pt.seq_lens + b);
    if (len < 0) len = 0;
    n = a.new_lens ? min(max(__ldca(a.new_lens + b), 0), a.T) : a.T;
    if (threadIdx.x < tokens) {
      const int t = t0 + threadIdx.x;
      const long long pos = len - n + t;
      uint32_t row = 0;
      int32_t bad = 0;
      int page = -2;
      if (t < n && pos >= 0) page = cache_page(a.c, a.pt, b, pos, 0, row, bad);
      if (bad) report(a.dev_status, bad);
      page_of[threadIdx.x] = page;
      slot_of[threadIdx.x] = row;
    }
  }
  for (int i = threadIdx.x; i < tokens * P; i += ROPE_THREADS) {
    const int tl = i / P, p = i - tl * P;
    long long pos = t0 + tl;
    if (OUT == TO_CACHE) pos += len - n;
    else if (a.pos) pos = a.pos_t ? __ldca(a.pos + b * a.pos_b + pos * a.pos_t) : __ldca(a.pos + b * a.pos_b) + pos;
    const unsigned long long turn = (unsigned long long)pos * __ldca(a.turns + p);
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    cosines[i] = c * a.magnitude;
    sines[i] = (a.inverse ? -s : s) * a.magnitude;
  }
  __syncthreads();

  // ---- the heads of all tokens, in memory's order: `heads` rows per token, q's then k's (then v's) ----
  const int D = DC ? DC : a.D, lpr = D / 8, rpw = 32 / lpr;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / lpr, chunk = lane - sub * lpr;
  const bool act = sub < rpw;
  const int heads = a.Hq + (OUT == TO_CACHE ? 2 : 1) * a.Hkv, rows = tokens * heads;
  const int half = a.rot / 16;                   // chunks of half the rotated part
  const bool turned = chunk < 2 * half, low = chunk < half;
  const int other = turned && !INTER ? (low ? lane + half : lane - half) : lane;
  const int angle = INTER ? chunk * 4 : (low ? chunk : chunk - half) * 8;
  const uint32_t up = OUT == TO_ACT ? 0u : ceil_carry<FMT>(a.rule);
  constexpr int STEP = ROPE_WARPS * ROPE_BATCH;
  for (int r0 = 0; r0 < rows; r0 += STEP * rpw) {
    uint4 x[ROPE_BATCH];
    int tok[ROPE_BATCH], head[ROPE_BATCH];
#pragma unroll
    for (int k = 0; k < ROPE_BATCH; ++k) {
      const int r = r0 + (k * ROPE_WARPS + warp) * rpw + sub;
      x[k] = make_uint4(0, 0, 0, 0);
      tok[k] = -1;
      head[k] = 0;
      if (act && r < rows) {
        tok[k] = r / heads;
        head[k] = r - tok[k] * heads;
        if (OUT == TO_CACHE && page_of[tok[k]] == -2 && head[k] >= a.Hq) tok[k] = -1;
      }
      if (tok[k] >= 0) {
        const int which = head[k] < a.Hq ? 0 : OUT == TO_CACHE && head[k] >= a.Hq + a.Hkv ? 2 : 1;
        const int h = head[k] - (which == 0 ? 0 : which == 1 ? a.Hq : a.Hq + a.Hkv);
        const RowStrides& s = a.xs[which];
        x[k] = __ldcs(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x[which]) + b * s.b +
                                                     (t0 + tok[k]) * s.t + h * s.h) + chunk);
      }
    }
#pragma unroll
    for (int k = 0; k < ROPE_BATCH; ++k) {
      uint32_t u[4] = {x[k].x, x[k].y, x[k].z, x[k].w}, o[4];
      if (!INTER)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = __shfl_sync(0xFFFFFFFFu, u[j], other);
      const int h = head[k], which = h < a.Hq ? 0 : OUT == TO_CACHE && h >= a.Hq + a.Hkv ? 2 : 1;
      const bool there = tok[k] >= 0;
      float f[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 p = act_to_f32<DT>(u[j]);
        f[2 * j] = p.x;
        f[2 * j + 1] = p.y;
      }
      if (there && turned && which != 2) {
        const float* const cs = cosines + tok[k] * P + angle;
        const float* const sn = sines + tok[k] * P + angle;
        if (INTER) {
          const float4 c = *reinterpret_cast<const float4*>(cs), s = *reinterpret_cast<const float4*>(sn);
          const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p = f[2 * j], q = f[2 * j + 1];
            f[2 * j] = p * cc[j] - q * ss[j];
            f[2 * j + 1] = p * ss[j] + q * cc[j];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 c = reinterpret_cast<const float4*>(cs)[i], s = reinterpret_cast<const float4*>(sn)[i];
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 pair = act_to_f32<DT>(o[2 * i + j / 2]);
              const float q = j & 1 ? pair.y : pair.x;
              f[4 * i + j] = f[4 * i + j] * cc[j] + (low ? -q : q) * ss[j];
            }
          }
        }
      }
      if (there && (OUT == TO_ACT || (OUT == TO_CACHE && which == 0))) {
        const RowStrides& s = a.ys[which];
        uint4 v = make_uint4(f32_to_act<DT>(f[0], f[1]), f32_to_act<DT>(f[2], f[3]), f32_to_act<DT>(f[4], f[5]),
                             f32_to_act<DT>(f[6], f[7]));
        if (OUT == TO_CACHE && page_of[tok[k]] == -2) v = make_uint4(0, 0, 0, 0);
        __stcs(reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.y[which]) + b * s.b + (t0 + tok[k]) * s.t +
                                        (h - (which ? a.Hq : 0)) * s.h) + chunk, v);
      }
      if (OUT != TO_ACT) {
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(f[i]) & 0x7FFFFFFFu);
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
        float inv;
        const uint32_t sb = block_scale<FMT>(__uint_as_float(am), up, inv);
        if (OUT == TO_MX && there) {
          const int H = which ? a.Hkv : a.Hq, hh = h - (which ? a.Hq : 0);
          const RowStrides& s = a.ys[which];
          __stcs(reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(a.y[which]) + b * s.b + (t0 + tok[k]) * s.t + hh * s.h) +
                     chunk, quant8_e4m3(f, inv, sb));
          if ((chunk & 3) == 0)
            a.sc[which][(((long long)b * H + hh) * a.T + t0 + tok[k]) * (D / 32) + (chunk >> 2)] = (uint8_t)sb;
        }
        if (OUT == TO_CACHE && there && which != 0) {
          const int page = page_of[tok[k]];
          if (page >= 0) {
            const int hh = h - a.Hq - (which == 2 ? a.Hkv : 0);
            const unsigned long long row = (unsigned long long)hh * a.c.page_size + slot_of[tok[k]];
            uint8_t* const dst = which == 2 ? a.c.v + page * a.c.v_ps : a.c.k + page * a.c.k_ps;
            uint8_t* const sc = which == 2 ? a.c.v_sc + page * a.c.v_sc_ps : a.c.k_sc + page * a.c.k_sc_ps;
            if (FMT == CACHE_FP4) {
              float y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = f[i] * inv;
              reinterpret_cast<uint32_t*>(dst + row * (D / 2))[chunk] = sb == 0xFFu ? 0x77777777u : cvt_e2m1x8(y);
            } else {
              reinterpret_cast<uint2*>(dst + row * D)[chunk] = quant8_e4m3(f, inv, sb);
            }
            if ((chunk & 3) == 0) sc[row * (D / 32) + (chunk >> 2)] = (uint8_t)sb;
          }
        }
      }
    }
  }
}

using Kernel = void (*)(RopeArgs);
// Tokens per block: enough for two batches of every thread, so that a block's angles and start are spread over its rows.
cudaError_t launch(Kernel k, RopeArgs a, int heads, cudaStream_t st) {
  const long long lanes = (long long)heads * (a.D / 8);
  long long tt = (2 * ROPE_BATCH * ROPE_THREADS + lanes - 1) / lanes;
  if (tt > MOST_TOKENS) tt = MOST_TOKENS;
  if (tt > MOST_ANGLES / (a.rot / 2)) tt = MOST_ANGLES / (a.rot / 2);
  if (tt > a.T) tt = a.T;
  a.tt = (int)tt;
  const long long grid = (long long)a.B * ((a.T + tt - 1) / tt);
  return launch_early(k, (unsigned)grid, ROPE_THREADS, 0, st, 1, a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, int interleaved, cudaStream_t st) {
  static const Kernel k[4] = {rope_kernel<0, false, TO_ACT, 0, 0>, rope_kernel<0, true, TO_ACT, 0, 0>,
                              rope_kernel<1, false, TO_ACT, 0, 0>, rope_kernel<1, true, TO_ACT, 0, 0>};
  return launch(k[dtype * 2 + interleaved], a, a.Hq + a.Hkv, st);
}
cudaError_t launch_rope_mx(const RopeArgs& a, int dtype, int interleaved, cudaStream_t st) {
  static const Kernel k[4] = {rope_kernel<0, false, TO_MX, CACHE_FP8, 128>, rope_kernel<0, true, TO_MX, CACHE_FP8, 128>,
                              rope_kernel<1, false, TO_MX, CACHE_FP8, 128>, rope_kernel<1, true, TO_MX, CACHE_FP8, 128>};
  return launch(k[dtype * 2 + interleaved], a, a.Hq + a.Hkv, st);
}
template <int FMT, int DC>
Kernel cache_kernel(int dtype, int interleaved) {
  static const Kernel k[4] = {rope_kernel<0, false, TO_CACHE, FMT, DC>, rope_kernel<0, true, TO_CACHE, FMT, DC>,
                              rope_kernel<1, false, TO_CACHE, FMT, DC>, rope_kernel<1, true, TO_CACHE, FMT, DC>};
  return k[dtype * 2 + interleaved];
}
cudaError_t launch_rope_cache(const RopeArgs& a, int format, int dtype, int interleaved, cudaStream_t st) {
  const Kernel k = format == CACHE_FP8 ? (a.D == 64 ? cache_kernel<CACHE_FP8, 64>(dtype, interleaved)
                                                    : cache_kernel<CACHE_FP8, 128>(dtype, interleaved))
                                       : (a.D == 64 ? cache_kernel<CACHE_FP4, 64>(dtype, interleaved)
                                                    : cache_kernel<CACHE_FP4, 128>(dtype, interleaved));
  return launch(k, a, a.Hq + 2 * a.Hkv, st);
}

}  // namespace bsc
