// Reading less of a long cache: bounds of each page's keys, and the pages that a query and KV head attends.
//
// Bounds.  For every page and KV head, min_d and max_d of its keys as 8-bit codes times one power of two 2^e, rounded
// outward: floor(min 2^-e), ceil(max 2^-e), e = floor(log2 max|K|) - 6.
//
// Score.  A head's largest possible q . K in the page is sum_d max(q_d, 0) max_d - max(-q_d, 0) min_d.  The heads that share
// the page's KV head are added up before the product: u_d = sum over heads of max(q_d, 0), l_d of max(-q_d, 0), both
// rounded to 0..127 with one power of two for the row, which changes no order.  Then
//   score = 2^e (u . max - l . min)
// is a whole number below 2^22 times a power of two, so it is exact in fp32: equal scores are equal, the choice depends on
// no order of summation, and four products are one instruction.
//
// Choice.  The first and the last pages, then the best scores, ties to the lower page; the list in ascending order, as
// slices (page, head) of the pools, so that the attention reads it as it reads a page table.
//
// What bounds it: latency for one sequence, else reading the bounds (2 D + 1 bytes per page and head against the
// page_size * 2 * (D / 2 + D / 32) or more of the page itself).
#include "cache.cuh"

namespace bsc {
namespace {

constexpr int BOUNDS_THREADS = 128;

// The page of a sequence's new tokens that block (b, i, h) takes, its tokens, and its id (-1: none).
template <int FMT, int D>
__global__ void __launch_bounds__(BOUNDS_THREADS) cache_bounds_kernel(const BoundsArgs a, int per_seq) {
  constexpr int LPR = D / 8, ROWS = BOUNDS_THREADS / LPR, RB = row_bytes<FMT, D>(), NB = D / 32;
  __shared__ float lo_s[BOUNDS_THREADS / 32][D], hi_s[BOUNDS_THREADS / 32][D];
  __shared__ float tops[BOUNDS_THREADS / 32];
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const int h = blockIdx.x % a.c.Hkv, x = blockIdx.x / a.c.Hkv, b = x / per_seq, i = x - b * per_seq;
  const int len = max(__ldca(a.pt.seq_lens + b), 0), ps = a.c.page_size;
  const int n = a.new_lens ? min(max(__ldca(a.new_lens + b), 0), a.T) : a.T;
  if (n == 0 || len == 0) return;
  const long long page_no = (long long)max(len - n, 0) / ps + i;
  if (page_no * ps >= len) return;
  uint32_t row;
  int32_t bad = 0;
  const int page = cache_page(a.c, a.pt, b, page_no * ps, h, row, bad);
  if (bad && threadIdx.x == 0) report(a.dev_status, bad);
  if (page < 0) return;
  const int tokens = (int)min((long long)ps, len - page_no * ps);
  const int chunk = threadIdx.x % LPR, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint8_t* const data = a.c.k + page * a.c.k_ps + (unsigned long long)row * RB + chunk * (RB / LPR);
  const uint8_t* const sc = a.c.k_sc + page * a.c.k_sc_ps + (unsigned long long)row * NB + chunk / 4;
  float lo[8], hi[8];
  bool odd = false;                              // a NaN, or a value beyond fp32
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo[j] = INFINITY;
    hi[j] = -INFINITY;
  }
#pragma unroll 4
  for (int t = threadIdx.x / LPR; t < tokens; t += ROWS) {
    uint32_t w[4];
    if (FMT == CACHE_FP4) {
      e2m1x8_to_f16(__ldca(reinterpret_cast<const uint32_t*>(data + (unsigned)t * RB)), w);
    } else {
      const uint2 y = __ldca(reinterpret_cast<const uint2*>(data + (unsigned)t * RB));
      e4m3x4_to_f16(y.x, w[0], w[1]);
      e4m3x4_to_f16(y.y, w[2], w[3]);
    }
    const float s = scale_value(__ldca(sc + (unsigned)t * NB));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = f16x2_to_f32(w[j]);
      const float v[2] = {f.x * s, f.y * s};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        odd |= !(fabsf(v[k]) < INFINITY);
        lo[2 * j + k] = fminf(lo[2 * j + k], v[k]);
        hi[2 * j + k] = fmaxf(hi[2 * j + k], v[k]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
#pragma unroll
    for (int o = 16; o >= LPR; o >>= 1) {
      lo[j] = fminf(lo[j], __shfl_xor_sync(0xFFFFFFFFu, lo[j], o));
      hi[j] = fmaxf(hi[j], __shfl_xor_sync(0xFFFFFFFFu, hi[j], o));
    }
    if (lane < LPR) {
      lo_s[warp][chunk * 8 + j] = lo[j];
      hi_s[warp][chunk * 8 + j] = hi[j];
    }
  }
  odd = __syncthreads_or(odd);
  float l = 0.f, m = 0.f;
  if (threadIdx.x < D) {
    l = lo_s[0][threadIdx.x];
    m = hi_s[0][threadIdx.x];
#pragma unroll
    for (int k = 1; k < BOUNDS_THREADS / 32; ++k) {
      l = fminf(l, lo_s[k][threadIdx.x]);
      m = fmaxf(m, hi_s[k][threadIdx.x]);
    }
  }
  float top = fmaxf(fabsf(l), fabsf(m));
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < BOUNDS_THREADS / 32; ++k) top = fmaxf(top, tops[k]);
  // the exponent field less 127 + 6, no lower than -100; above 100 the page counts as odd
  const int e = max((int)(__float_as_uint(top) >> 23) - 133, -100);
  odd |= e > 100;
  if (threadIdx.x < D) {
    const float f = odd ? 0.f : __uint_as_float((uint32_t)(127 - e) << 23);
    int8_t* const dst = a.codes + ((long long)page * a.c.Hkv + h) * (2 * D) + threadIdx.x;
    dst[0] = odd ? 0 : (int8_t)(int)floorf(l * f);
    dst[D] = odd ? 0 : (int8_t)(int)ceilf(m * f);
  }
  if (threadIdx.x == 0) a.exps[(long long)page * a.c.Hkv + h] = odd ? 0xFFu : (uint8_t)(e + 127);
}

// What a query row sees of its sequence: tokens (0: not a row), pages, and whether its positions pass the table's end.
struct Seen {
  int tokens, pages;
  bool past;
};
__device__ __forceinline__ Seen seen_by(const SelectArgs& a, int b, int t) {
  const int len = max(__ldca(a.pt.seq_lens + b), 0), cap = a.pt.max_pages * a.page_size;   // < 2^31
  const int n = a.new_lens ? min(max(__ldca(a.new_lens + b), 0), a.T) : a.T;
  long long v = t < n ? (long long)len - n + t + 1 : 0;
  if (v < 0) v = 0;
  Seen s;
  s.past = len > cap;
  s.tokens = (int)min(v, (long long)cap);
  s.pages = (s.tokens + a.page_size - 1) / a.page_size;
  return s;
}

// Scores of SCORE_PAGES pages for one query and KV head.  D / 16 lanes are a page: 16 minima and 16 maxima each.
constexpr int SCORE_THREADS = 128, SCORE_PAGES = 128;
template <int D, int DT>
__global__ void __launch_bounds__(SCORE_THREADS) cache_score_kernel(const SelectArgs a, int tiles) {
  constexpr int LPP = D / 16, PPW = 32 / LPP, WARPS = SCORE_THREADS / 32;
  __shared__ __align__(16) uint8_t codes[2][D];
  __shared__ float tops[WARPS];
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const uint32_t row = blockIdx.x / tiles, tile = blockIdx.x - row * tiles;
  const uint32_t bt = row / a.Hkv, h = row - bt * a.Hkv, b = bt / a.T, t = bt - b * a.T;
  const Seen seen = seen_by(a, b, t);
  const int first = tile * SCORE_PAGES, last = min(first + SCORE_PAGES, seen.pages);
  if (first >= last || seen.pages <= a.top) return;      // every page is taken: no score is read
  // ---- the row's codes ----
  const int G = a.Hq / a.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float u = 0.f, l = 0.f;
  if (threadIdx.x < D) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q) + b * a.qs.b + t * a.qs.t + (long long)h * G * a.qs.h + threadIdx.x;
    for (int g = 0; g < G; ++g) {
      const float f = act_to_f32<DT>((uint32_t)__ldca(q + g * a.qs.h)).x;
      u += f > 0.f ? f : 0.f;
      l += f < 0.f ? -f : 0.f;
      if (!(fabsf(f) < INFINITY)) u = INFINITY;
    }
  }
  float top = fmaxf(u, l);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < WARPS; ++k) top = fmaxf(top, tops[k]);
  // 2^(6 - floor(log2 top)); rows of nothing, and those with a NaN or an infinity, score 0 everywhere
  const int e = (int)(__float_as_uint(top) >> 23);
  const float f = e == 0 || e == 255 ? 0.f : __uint_as_float((uint32_t)min(max(260 - e, 1), 254) << 23);
  if (threadIdx.x < D) {
    codes[0][threadIdx.x] = f == 0.f ? 0 : (uint8_t)min(__float2int_rn(u * f), 127);
    codes[1][threadIdx.x] = f == 0.f ? 0 : (uint8_t)min(__float2int_rn(l * f), 127);
  }
  __syncthreads();
  const int part = lane % LPP;
  const uint4 cu = *reinterpret_cast<const uint4*>(codes[0] + part * 16), cl = *reinterpret_cast<const uint4*>(codes[1] + part * 16);
  // ---- the pages: all loads of a batch first ----
  constexpr int BATCH = 4;
  float* const out = a.scores + (long long)row * a.pt.max_pages;
  const int32_t* const table = a.pt.table + (long long)b * a.pt.stride;
  for (int p0 = first + warp * PPW; p0 < last; p0 += BATCH * WARPS * PPW) {
    int page[BATCH];
    uint32_t e8[BATCH];
    uint4 lo[BATCH], hi[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int p = p0 + k * WARPS * PPW + lane / LPP;
      page[k] = p < last ? __ldca(table + p) : -1;
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      lo[k] = hi[k] = make_uint4(0, 0, 0, 0);
      e8[k] = 0;
      if (page[k] >= 0 && page[k] < a.num_pages) {
        const long long at = (long long)page[k] * a.Hkv + h;
        lo[k] = __ldca(reinterpret_cast<const uint4*>(a.codes + at * (2 * D)) + part);
        hi[k] = __ldca(reinterpret_cast<const uint4*>(a.codes + at * (2 * D) + D) + part);
        e8[k] = __ldca(a.exps + at);
      } else {
        page[k] = -1;
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int p = p0 + k * WARPS * PPW + lane / LPP;
      int d = __dp4a((int)hi[k].x, (int)cu.x, 0), m = __dp4a((int)lo[k].x, (int)cl.x, 0);
      d = __dp4a((int)hi[k].y, (int)cu.y, d);
      m = __dp4a((int)lo[k].y, (int)cl.y, m);
      d = __dp4a((int)hi[k].z, (int)cu.z, d);
      m = __dp4a((int)lo[k].z, (int)cl.z, m);
      d = __dp4a((int)hi[k].w, (int)cu.w, d);
      m = __dp4a((int)lo[k].w, (int)cl.w, m);
      d -= m;
#pragma unroll
      for (int o = LPP / 2; o; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
      if (part == 0 && p < last) {
        if (page[k] < 0) report(a.dev_status, CACHE_BAD_PAGE);
        // a page that is not there comes last, one with a NaN first, so that it is met as it would be by reading all
        out[p] = page[k] < 0 ? -INFINITY : e8[k] == 0xFFu ? INFINITY : (float)d * scale_value(e8[k]);
      }
    }
  }
}

// The pages of one query and KV head.  A thread has a run of neighbouring pages, so that a scan over the threads gives
// the list's order.  The threshold, the key of the last page taken, is found two bits at a time: three counts of the
// keys at or above a trial value, over the block.
constexpr int SELECT_THREADS = 256, SELECT_WARPS = SELECT_THREADS / 32, HELD = 16;
__device__ __forceinline__ uint32_t key_of(float s) {                     // in the order of the floats
  const uint32_t u = __float_as_uint(s);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ int block_scan(int v, int* sums, int& all) {   // exclusive; sums[SELECT_WARPS] of its own
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) sums[warp] = s;
  __syncthreads();
  int before = 0;
  all = 0;
#pragma unroll
  for (int k = 0; k < SELECT_WARPS; ++k) {
    const int y = sums[k];
    if (k < warp) before += y;
    all += y;
  }
  return before + s - v;
}
__global__ void __launch_bounds__(SELECT_THREADS) cache_select_kernel(const SelectArgs a, int cols) {
  __shared__ int counts[2][SELECT_WARPS][3], scan[2][SELECT_WARPS];
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const uint32_t row = blockIdx.x, bt = row / a.Hkv, h = row - bt * a.Hkv, b = bt / a.T, t = bt - b * a.T;
  const Seen seen = seen_by(a, b, t);
  const int32_t* const table = a.pt.table + (long long)b * a.pt.stride;
  int32_t* const list = a.table + (long long)row * cols;
  int32_t* const blocks = a.blocks ? a.blocks + (long long)row * a.top : nullptr;
  const int n = seen.pages, k = min(n, a.top), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0 && seen.past) report(a.dev_status, CACHE_BAD_LEN);
  if (threadIdx.x == 0) a.lens[row] = k > 0 ? (k - 1) * a.page_size + seen.tokens - (n - 1) * a.page_size : 0;
  auto put = [&](int at, int p) {
    const int page = __ldca(table + p);
    list[at] = page >= 0 && page < a.num_pages ? page * a.pages_per_page + (int)h : -1;
    if (blocks) blocks[at] = p;
  };
  if (blocks)
    for (int i = k + threadIdx.x; i < a.top; i += SELECT_THREADS) blocks[i] = -1;
  if (n == k) {
    for (int i = threadIdx.x; i < k; i += SELECT_THREADS) put(i, i);
    return;
  }
  const float* const scores = a.scores + (long long)row * a.pt.max_pages;
  const int run = (n + SELECT_THREADS - 1) / SELECT_THREADS, p0 = threadIdx.x * run, p1 = min(p0 + run, n);
  auto key_at = [&](int p) {
    return p < a.first || p >= n - a.last ? 0xFFFFFFFFu : key_of(__ldca(scores + p));
  };
  uint32_t held[HELD];
  const bool fits = run <= HELD;
#pragma unroll
  for (int j = 0; j < HELD; ++j) held[j] = fits && p0 + j < p1 ? key_at(p0 + j) : 0u;
  // keys at or above x among the thread's; no page has key 0 (that of a NaN)
  auto count3 = [&](uint32_t x1, uint32_t x2, uint32_t x3, int& c1, int& c2, int& c3) {
    c1 = c2 = c3 = 0;
    if (fits) {
#pragma unroll
      for (int j = 0; j < HELD; ++j) {
        c1 += held[j] >= x1;
        c2 += held[j] >= x2;
        c3 += held[j] >= x3;
      }
    } else {
      for (int p = p0; p < p1; ++p) {
        const uint32_t y = key_at(p);
        c1 += y >= x1;
        c2 += y >= x2;
        c3 += y >= x3;
      }
    }
  };
  uint32_t cut = 0;                              // the largest value that at least k keys reach
  for (int bit = 30, turn = 0; bit >= 0; bit -= 2, turn ^= 1) {
    const uint32_t one = 1u << bit;
    int c1, c2, c3;
    count3(cut + one, cut + 2 * one, cut + 3 * one, c1, c2, c3);
    c1 = __reduce_add_sync(0xFFFFFFFFu, c1);
    c2 = __reduce_add_sync(0xFFFFFFFFu, c2);
    c3 = __reduce_add_sync(0xFFFFFFFFu, c3);
    if (lane == 0) {
      counts[turn][warp][0] = c1;
      counts[turn][warp][1] = c2;
      counts[turn][warp][2] = c3;
    }
    __syncthreads();
    c1 = c2 = c3 = 0;
#pragma unroll
    for (int w = 0; w < SELECT_WARPS; ++w) {
      c1 += counts[turn][w][0];
      c2 += counts[turn][w][1];
      c3 += counts[turn][w][2];
    }
    cut += c3 >= k ? 3 * one : c2 >= k ? 2 * one : c1 >= k ? one : 0u;
  }
  // ---- those above the cut, and the lowest of those at it ----
  int above = 0, equal = 0;
  auto each = [&](auto f) {
    if (fits) {
#pragma unroll
      for (int j = 0; j < HELD; ++j)
        if (p0 + j < p1) f(p0 + j, held[j]);
    } else {
      for (int p = p0; p < p1; ++p) f(p, key_at(p));
    }
  };
  each([&](int, uint32_t y) {
    above += y > cut;
    equal += y == cut;
  });
  int all_above, all;
  const int above_before = block_scan(above, scan[0], all_above);
  const int equal_before = block_scan(equal, scan[1], all);
  const int want = k - all_above;                // of those at the cut
  int at = above_before + min(equal_before, want), ties = equal_before;
  each([&](int p, uint32_t y) {
    if (y > cut || (y == cut && ties < want)) put(at++, p);
    ties += y == cut;
  });
}

}  // namespace

cudaError_t launch_cache_bounds(const BoundsArgs& a, int format, int D, cudaStream_t st) {
  const int per_seq = (a.T - 1) / a.c.page_size + 2;       // pages that T neighbouring tokens can touch
  const unsigned grid = (unsigned)a.B * per_seq * a.c.Hkv;
  const auto k = format == CACHE_FP4 ? (D == 128 ? cache_bounds_kernel<CACHE_FP4, 128> : cache_bounds_kernel<CACHE_FP4, 64>)
                                     : (D == 128 ? cache_bounds_kernel<CACHE_FP8, 128> : cache_bounds_kernel<CACHE_FP8, 64>);
  return launch_early(k, grid, BOUNDS_THREADS, 0, st, 1, a, per_seq);
}

cudaError_t launch_cache_select(const SelectArgs& a, int D, int dtype, cudaStream_t st) {
  const unsigned rows = (unsigned)a.B * a.T * a.Hkv;
  const int cols = a.top < a.pt.max_pages ? a.top : a.pt.max_pages;
  if (a.pt.max_pages > a.top) {
    const int tiles = (a.pt.max_pages + SCORE_PAGES - 1) / SCORE_PAGES;
    const auto k = D == 128 ? (dtype ? cache_score_kernel<128, 1> : cache_score_kernel<128, 0>)
                            : (dtype ? cache_score_kernel<64, 1> : cache_score_kernel<64, 0>);
    const cudaError_t e = launch_early(k, rows * tiles, SCORE_THREADS, 0, st, 1, a, tiles);
    if (e != cudaSuccess) return e;
  }
  return launch_early(cache_select_kernel, rows, SELECT_THREADS, 0, st, 1, a, cols);
}

}  // namespace bsc
