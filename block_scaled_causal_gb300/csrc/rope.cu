// Rotary positions of Q and K: to 16 bits, to MXFP8 rows, and into the key/value cache.
//
// Pair i of a head's first `rot` elements, (x_i, x_{i + rot/2}) or, interleaved, (x_2i, x_2i+1), turns by the angle p f_i of
// its token's position p: (a, b) -> m (a cos - b sin, a sin + b cos).  The gradient turns by -p f_i.  Elements from `rot` on
// pass through.
//
// Angles.  f_i is held as a 64-bit fraction of a turn, so p * f_i mod 2^64 is the angle's fraction of a turn, exactly,
// whatever the position: no table of positions is read and there is no longest one.  Its cosine and sine are rounded to fp32
// about once (turned()): what the MXFP8 forms' bytes are made from is as near as fp64 angles would leave it.
//
// Work.  A warp has one token: its cosines and sines are worked out once by its lanes and pass through shared memory into
// registers, then all heads of the token (or a share of them, where there are few tokens) go by.  A lane has 8 neighbouring
// elements of a head (16 bytes), D / 8 lanes are a head, and half pairs exchange their packed elements with the lane rot / 16
// away; four neighbouring lanes are an MX block.  From head to head an address moves by one addition.
//
// What bounds it: memory.  In 16 bits 32K tokens of 16 + 4 heads take 47.9 us cold (7.0 TB/s of 335 MB); to MXFP8 65536 tokens of
// 16 + 16 heads 131 us (93% of the copy rate), 8192 of them 19.0 (80%: 1.7 waves of warps, 2.7 instructions per clock; interleaved
// pairs, which exchange nothing, 18.8); prompts of 10K tokens into the cache 29.9 us for 173 MB.
// The loads of ROPE_BATCH heads are ahead of their first use, those of the first heads ahead of the angles (100.6 us for both
// directions, 102.4 behind them).  2 / 4 / 8 heads per batch: 116 / 104 / 114 us in a graph.
#include "cache.cuh"

namespace bsc {
namespace {

constexpr int ROPE_WARPS = 4, ROPE_BATCH = 4, MOST_PAIRS = 128;
enum { TO_ACT, TO_MX, TO_CACHE };

// Cosine and sine of 2 pi x / 2^64, times m + ml, rounded to fp32 about once (0.70 units of the last place in [1/2, 1) at most,
// 0.29 in root mean square over all angles, where one rounding has 0.29).  x is a quarter turn's number and an angle of half of
// one at most, |r| <= 2^29 with 2^-32 turns as the unit, in two pieces; theta = t + tl, |t| <= pi/4, z = t^2 (and zl):
//   sin theta = t + (t z P(z) + tl cos theta),  cos theta = w + (z^2 Q(z) + what w = 1 - z/2 and z have rounded away)
// with the Taylor series' P and Q (their next terms: 2^-29 and 2^-33); both sums stay in two parts up to the product with m.
// __fmul_rn: products whose rounding is taken up again must not become part of another operation.
__device__ __forceinline__ void turned(unsigned long long x, float m, float ml, float& c, float& s) {
  constexpr float UNIT = 6.2831853f * 0x1p-32f, UNIT_LOW = -1.7484556e-7f * 0x1p-32f;   // 2 pi 2^-32, and what is left of it
  const uint32_t y = (uint32_t)(x >> 32) + 0x20000000u;
  const int r = (int)(y & 0x3FFFFFFFu) - 0x20000000;
  const float h = (float)(r & ~63), l = (float)__funnelshift_r((uint32_t)x, (uint32_t)r, 6);   // 24 bits, the next 32
  float t = __fmul_rn(h, UNIT), tl = fmaf(l, UNIT * 0x1p-26f, fmaf(h, UNIT_LOW, fmaf(h, UNIT, -t)));
  const float sum = t + tl;
  tl -= sum - t;
  t = sum;
  const float z = __fmul_rn(t, t), zl = fmaf(t + t, tl, fmaf(t, t, -z)), w = fmaf(-0.5f, z, 1.f);
  const float p = fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6);
  const float q = fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24);
  const float cl = fmaf(z * z, q, fmaf(-0.5f, zl, fmaf(-0.5f, z, 1.f - w)));
  const float rest = fmaf(t * z, p, tl * w), sh = t + rest, sl = rest - (sh - t);
  const float cosine = fmaf(m, w, fmaf(m, cl, ml * w)), sine = fmaf(m, sh, fmaf(m, sl, ml * sh));
  const uint32_t quarter = y >> 30;
  c = quarter & 1 ? sine : cosine;
  s = quarter & 1 ? cosine : sine;
  c = __uint_as_float(__float_as_uint(c) ^ ((quarter + 1) & 2) << 30);
  s = __uint_as_float(__float_as_uint(s) ^ (quarter & 2) << 30);
}

// What a lane turns its 8 elements by: y = x c + o s, o being the partner chunk (or the pair's other element), signs in s.
template <bool INTER>
struct Turn {
  float2 c[4], s[4];
  __device__ __forceinline__ void load(const float* cosines, const float* sines, int angle, bool low) {
    if (INTER) {
      const float4 a = *reinterpret_cast<const float4*>(cosines + angle), b = *reinterpret_cast<const float4*>(sines + angle);
      c[0] = make_float2(a.x, a.x); c[1] = make_float2(a.y, a.y); c[2] = make_float2(a.z, a.z); c[3] = make_float2(a.w, a.w);
      s[0] = make_float2(-b.x, b.x); s[1] = make_float2(-b.y, b.y); s[2] = make_float2(-b.z, b.z); s[3] = make_float2(-b.w, b.w);
    } else {
      const float sign = low ? -1.f : 1.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 a = reinterpret_cast<const float4*>(cosines + angle)[i], b = reinterpret_cast<const float4*>(sines + angle)[i];
        c[2 * i] = make_float2(a.x, a.y); c[2 * i + 1] = make_float2(a.z, a.w);
        s[2 * i] = make_float2(sign * b.x, sign * b.y); s[2 * i + 1] = make_float2(sign * b.z, sign * b.w);
      }
    }
  }
};

// The next heads of a tensor, `step` elements apart from x on, of which the lane has the first `live`.
__device__ __forceinline__ void load_batch(uint4 (&v)[ROPE_BATCH], const uint16_t*& x, long long step, int live) {
#pragma unroll
  for (int k = 0; k < ROPE_BATCH; ++k) {
    v[k] = make_uint4(0, 0, 0, 0);
    if (k < live) v[k] = __ldcs(reinterpret_cast<const uint4*>(x));
    x += step;
  }
}
// One tensor's heads of a token for this lane: `rounds` of them, the first batch already in v and the next from x on;
// `emit(there, values)` for each in turn.  Whole warps call it with the same rounds.
template <int DT, bool INTER, bool TURN, class Emit>
__device__ __forceinline__ void heads_of(uint4 (&v)[ROPE_BATCH], const uint16_t* x, long long step, int rounds, int live, int other,
                                         bool in_rot, const Turn<INTER>& turn, Emit emit) {
  for (;;) {
#pragma unroll
    for (int k = 0; k < ROPE_BATCH; ++k) {
      if (k >= rounds) break;
      const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      float2 f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = act_to_f32<DT>(u[j]);
      if (TURN) {
        float2 o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = INTER ? make_float2(f[j].y, f[j].x) : act_to_f32<DT>(__shfl_sync(0xFFFFFFFFu, u[j], other));
        if (in_rot)
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = __ffma2_rn(f[j], turn.c[j], __fmul2_rn(o[j], turn.s[j]));
      }
      emit(k < live, f);
    }
    rounds -= ROPE_BATCH;
    live -= ROPE_BATCH;
    if (rounds <= 0) return;
    load_batch(v, x, step, live);
  }
}

// The scale byte of a block of four neighbouring lanes' elements.
template <int FMT>
__device__ __forceinline__ uint32_t chunk_scale(const float2 (&f)[4], uint32_t up, float& inv) {
  float am = amax8(f);
  am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
  am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
  return block_scale<FMT>(am, up, inv);
}
template <int DT>
__device__ __forceinline__ uint4 pack(const float2 (&f)[4]) {
  return make_uint4(f32_to_act<DT>(f[0].x, f[0].y), f32_to_act<DT>(f[1].x, f[1].y), f32_to_act<DT>(f[2].x, f[2].y),
                    f32_to_act<DT>(f[3].x, f[3].y));
}

// blockIdx.x: ROPE_WARPS tokens of the B x T, a warp each; blockIdx.y: a share of `per` heads of each token's list (q's, k's,
// then v's).
template <int DT, bool INTER, int OUT, int FMT, int DC>
__global__ void __launch_bounds__(ROPE_WARPS * 32, 8) rope_kernel(const RopeArgs a, int per) {
  __shared__ __align__(16) float cosines[ROPE_WARPS][MOST_PAIRS], sines[ROPE_WARPS][MOST_PAIRS];
  wait_for_last_kernel();
  if (a.may_signal) next_kernel_may_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t token = blockIdx.x * ROPE_WARPS + warp;
  if (token >= (uint32_t)a.B * a.T) return;
  const int b = token / a.T, t = token - b * a.T;

  const int D = DC ? DC : a.D, lpr = D / 8, rpw = 32 / lpr, sub = lane / lpr, chunk = lane - sub * lpr;
  const bool act = sub < rpw;
  const int half = a.rot / 16;                   // chunks of half the rotated part
  const bool in_rot = chunk < 2 * half, low = chunk < half;
  const int other = in_rot ? (low ? lane + half : lane - half) : lane;

  // ---- the heads: this block's share of [0, Hq + Hkv (+ Hkv)); those of tensor i are h0 .. h1 - 1 of it ----
  constexpr int TENSORS = OUT == TO_CACHE ? 3 : 2;
  const int total = a.Hq + (TENSORS - 1) * a.Hkv, from = blockIdx.y * per, to = min(from + per, total);
  const uint32_t up = OUT == TO_ACT ? 0u : ceil_carry<FMT>(a.rule);
  auto base_of = [&](int i) { return i == 0 ? 0 : i == 1 ? a.Hq : a.Hq + a.Hkv; };
  auto first_of = [&](int i) { return max(from - base_of(i), 0); };
  auto end_of = [&](int i) { return min(to - base_of(i), i == 0 ? a.Hq : a.Hkv); };
  auto live_of = [&](int i) {                    // heads of this lane
    const int first = first_of(i) + sub, h1 = end_of(i);
    return act && first < h1 ? (h1 - first + rpw - 1) / rpw : 0;
  };
  auto source = [&](int i) {
    return reinterpret_cast<const uint16_t*>(a.x[i]) + b * a.xs[i].b + t * a.xs[i].t + (first_of(i) + sub) * a.xs[i].h + chunk * 8;
  };
  // the first heads' loads start ahead of the angles
  const int start = from < a.Hq ? 0 : from < a.Hq + a.Hkv ? 1 : 2;
  uint4 v[ROPE_BATCH];
  const uint16_t* x = source(start);
  load_batch(v, x, rpw * a.xs[start].h, live_of(start));

  // ---- the token's position and page, its angles ----
  long long pos = t;
  bool real = true;                              // TO_CACHE: a token of the sequence
  int page = -1;
  uint32_t slot = 0;
  if (OUT == TO_CACHE) {
    const long long len = max(__ldca(a.pt.seq_lens + b), 0);
    const int n = a.new_lens ? min(max(__ldca(a.new_lens + b), 0), a.T) : a.T;
    pos = len - n + t;
    real = t < n && pos >= 0;
    if (real) {
      int32_t bad = 0;
      page = cache_page(a.c, a.pt, b, pos, 0, slot, bad);
      if (bad && lane == 0) report(a.dev_status, bad);
    }
  } else if (a.pos) {
    pos = a.pos_t ? __ldca(a.pos + b * a.pos_b + t * a.pos_t) : __ldca(a.pos + b * a.pos_b) + (long long)t;
  }
  const int P = a.rot / 2;
  for (int p = lane; p < P; p += 32) {
    float c, s;
    turned((unsigned long long)pos * __ldca(a.turns + p), a.magnitude, a.magnitude_low, c, s);
    cosines[warp][p] = c;
    sines[warp][p] = a.inverse ? -s : s;
  }
  __syncwarp();

  Turn<INTER> turn;
  turn.load(cosines[warp], sines[warp], !in_rot ? 0 : INTER ? chunk * 4 : (low ? chunk : chunk - half) * 8, low);

#pragma unroll
  for (int i = 0; i < TENSORS; ++i) {
    const int h0 = first_of(i), h1 = end_of(i);
    if (h0 >= h1 || (OUT == TO_CACHE && i != 0 && page < 0)) continue;
    const int H = i == 0 ? a.Hq : a.Hkv, first = h0 + sub, rounds = (h1 - h0 + rpw - 1) / rpw, live = live_of(i);
    const long long step = rpw * a.xs[i].h;
    if (i != start) {
      x = source(i);
      load_batch(v, x, step, live);
    }
    if (OUT == TO_ACT || (OUT == TO_CACHE && i == 0)) {
      uint16_t* y = reinterpret_cast<uint16_t*>(a.y[i]) + b * a.ys[i].b + t * a.ys[i].t + first * a.ys[i].h + chunk * 8;
      const long long y_step = rpw * a.ys[i].h;
      heads_of<DT, INTER, true>(v, x, step, rounds, live, other, in_rot, turn, [&](bool there, const float2 (&f)[4]) {
        if (there) __stcs(reinterpret_cast<uint4*>(y), real ? pack<DT>(f) : make_uint4(0, 0, 0, 0));
        y += y_step;
      });
    } else if (OUT == TO_MX) {
      uint8_t* y = reinterpret_cast<uint8_t*>(a.y[i]) + b * a.ys[i].b + t * a.ys[i].t + first * a.ys[i].h + chunk * 8;
      uint8_t* sc = a.sc[i] + (((long long)b * H + first) * a.T + t) * (D / 32) + (chunk >> 2);
      const long long y_step = rpw * a.ys[i].h, sc_step = (long long)rpw * a.T * (D / 32);
      heads_of<DT, INTER, true>(v, x, step, rounds, live, other, in_rot, turn, [&](bool there, const float2 (&f)[4]) {
        float inv;
        const uint32_t sb = chunk_scale<FMT>(f, up, inv);
        if (there) {
          __stcs(reinterpret_cast<uint2*>(y), quant8_e4m3(f, inv, sb));
          if ((chunk & 3) == 0) *sc = (uint8_t)sb;
        }
        y += y_step;
        sc += sc_step;
      });
    } else if constexpr (OUT == TO_CACHE) {
      constexpr int RB = row_bytes<FMT, DC>();
      const unsigned long long row = (unsigned long long)first * a.c.page_size + slot;
      uint8_t* y = (i == 2 ? a.c.v + page * a.c.v_ps : a.c.k + page * a.c.k_ps) + row * RB + chunk * (RB / lpr);
      uint8_t* sc = (i == 2 ? a.c.v_sc + page * a.c.v_sc_ps : a.c.k_sc + page * a.c.k_sc_ps) + row * (DC / 32) + (chunk >> 2);
      const long long y_step = (long long)rpw * a.c.page_size * RB, sc_step = (long long)rpw * a.c.page_size * (DC / 32);
      auto emit = [&](bool there, const float2 (&f)[4]) {
        float inv;
        const uint32_t sb = chunk_scale<FMT>(f, up, inv);
        if (there) {
          if (FMT == CACHE_FP4) *reinterpret_cast<uint32_t*>(y) = quant8_e2m1(f, inv, sb);
          else *reinterpret_cast<uint2*>(y) = quant8_e4m3(f, inv, sb);
          if ((chunk & 3) == 0) *sc = (uint8_t)sb;
        }
        y += y_step;
        sc += sc_step;
      };
      if (i == 1) heads_of<DT, INTER, true>(v, x, step, rounds, live, other, in_rot, turn, emit);
      else heads_of<DT, INTER, false>(v, x, step, rounds, live, other, in_rot, turn, emit);
    }
  }
}

using Kernel = void (*)(RopeArgs, int);
// A call in place loads what it stores through L1, so it does not let the next kernel start early (cache.cuh has why).  Loads past L1
// cost every call more: 32K tokens 100.3 -> 100.8 us, to MXFP8 38.6 -> 39.5, prompts into the cache 44.6 -> 45.9.
bool in_place(const RopeArgs& a) { return a.y[0] == a.x[0] || (a.x[1] && a.y[1] == a.x[1]); }
// Heads of a token are shared by several warps while the card has room for them at once; each works the angles out again (3063
// tokens of 25 heads, both directions: one warp 20.5 us, two 22.5, four 26.7).
cudaError_t launch(Kernel k, RopeArgs a, int heads, cudaStream_t st) {
  const long long tokens = (long long)a.B * a.T;
  const int rpw = 32 / (a.D / 8);
  int shares = 1;
  while (shares * 2 <= heads / rpw && tokens * shares * 2 <= 152 * 16) shares *= 2;
  int per = (heads + shares - 1) / shares;
  per = (per + rpw - 1) / rpw * rpw;
  const dim3 grid((unsigned)((tokens + ROPE_WARPS - 1) / ROPE_WARPS), (unsigned)((heads + per - 1) / per));
  a.may_signal = (long long)grid.x * grid.y <= EARLY_BLOCKS && !in_place(a);
  return launch_early(k, grid, ROPE_WARPS * 32, 0, st, 1, a, per);
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
