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
// What bounds it: latency.  512 pages of 4 KV heads: bounds of the newest page 4.4 us (of 32 prompts of 2048 tokens, 64 to a
// page, 15.6), choice 9.1 us cold (chains of length, page id, data; then rounds of barriers); 128 rows of up to 512 pages 12.1 us
// for 6.8 MB of bounds (2 D + 1 bytes per page and head, against 8.7 KB of a page of 64 tokens in 4 bits).
#include <cooperative_groups.h>

#include "cache.cuh"

namespace bsc {
namespace {

namespace cg = cooperative_groups;

constexpr int BOUNDS_THREADS = 128;

// Tokens of the i-th page that sequence b's new tokens touch (0: there is no such page), and its number in the sequence.
__device__ __forceinline__ int new_page(const BoundsArgs& a, int b, int i, long long& page_no) {
  const int len = max(__ldca(a.pt.seq_lens + b), 0), ps = a.c.page_size;
  const int n = a.new_lens ? min(max(__ldca(a.new_lens + b), 0), a.T) : a.T;
  page_no = (long long)((uint32_t)max(len - n, 0) / (uint32_t)ps) + i;
  return n == 0 ? 0 : (int)min(max(len - page_no * ps, 0LL), (long long)ps);
}

// Block (b, i, h): one head of the i-th page that sequence b's new tokens touch.
//
// Several sequences may have the page, with different numbers of tokens: the one with the most writes, and no other, so that
// codes and exponent are always of one block, and bound what every sequence has in the page.  Those with as many make the same
// bytes.  Nothing has more than a whole page, so only a sequence's last page looks for such a sequence; last pages are
// among the first blocks, so that their search is not what the call ends with (32 prompts of 2048 tokens 18.0 -> 15.7 us, 15.2
// without it).
template <int FMT, int D>
__global__ void __launch_bounds__(BOUNDS_THREADS) cache_bounds_kernel(const BoundsArgs a, int per_seq) {
  constexpr int LPR = D / 8, ROWS = BOUNDS_THREADS / LPR, RB = row_bytes<FMT, D>(), NB = D / 32;
  __shared__ float lo_s[BOUNDS_THREADS / 32][D], hi_s[BOUNDS_THREADS / 32][D];
  __shared__ float tops[BOUNDS_THREADS / 32];
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const int h = blockIdx.x % a.c.Hkv, x = blockIdx.x / a.c.Hkv, i = per_seq - 1 - x / a.B, b = x % a.B;
  const int ps = a.c.page_size;
  long long page_no;
  const int tokens = new_page(a, b, i, page_no);
  if (tokens == 0) return;
  // Ids of the pages that the call's sequences touch, from the j-th on, where they have more tokens than this block's.  The
  // first are on their way beside the block's own.  (A branch around all of it, for whole pages: 57 -> 53.6 us for 16000 of them.)
  const int all = tokens < ps ? a.B * per_seq : 0;
  constexpr int MET = 2;
  int32_t fuller[MET];
#pragma unroll
  for (int k = 0; k < MET; ++k) fuller[k] = -1;
  auto load_fuller = [&](uint32_t j) {
#pragma unroll
    for (int k = 0; k < MET; ++k, j += BOUNDS_THREADS) {
      fuller[k] = -1;
      if (j < (uint32_t)all) {
        const int other = j / (uint32_t)per_seq;
        long long no;
        if (new_page(a, other, (int)j - other * per_seq, no) > tokens && no < a.pt.max_pages)
          fuller[k] = __ldca(a.pt.table + other * a.pt.stride + no);
      }
    }
  };
  if (all) load_fuller(threadIdx.x);
  uint32_t row;
  int32_t bad = 0;
  const int page = cache_page(a.c, a.pt, b, page_no * ps, h, row, bad);
  if (bad && threadIdx.x == 0) report(a.dev_status, bad);
  if (page < 0) return;
  bool others = false;
  if (all)
    for (int j = threadIdx.x;;) {
#pragma unroll
      for (int k = 0; k < MET; ++k) others |= fuller[k] == page;
      if (j >= all - MET * BOUNDS_THREADS) break;
      j += MET * BOUNDS_THREADS;
      load_fuller(j);
    }
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
  constexpr int BATCH = 8;                       // tokens of a thread whose loads are all ahead of the first use (4: 8.1 us, 8: 4.4)
  for (int t0 = threadIdx.x / LPR; t0 < tokens; t0 += BATCH * ROWS) {
    uint2 y[BATCH];
    uint32_t e[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const unsigned t = min(t0 + i * ROWS, tokens - 1);          // the last token again: no bound moves
      if (FMT == CACHE_FP4) y[i].x = __ldca(reinterpret_cast<const uint32_t*>(data + t * RB));
      else y[i] = __ldca(reinterpret_cast<const uint2*>(data + t * RB));
      e[i] = __ldca(sc + t * NB);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      uint32_t w[4];
      if (FMT == CACHE_FP4) {
        e2m1x8_to_f16(y[i].x, w);
      } else {
        e4m3x4_to_f16(y[i].x, w[0], w[1]);
        e4m3x4_to_f16(y[i].y, w[2], w[3]);
      }
      const float s = scale_value(e[i]);
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
  if (__syncthreads_or(others)) return;
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

// The pages of one query and KV head: a cluster of blocks scores them, each block a run of pages, and the first block chooses.
//
// The scores pass through the first block's shared memory, or the workspace where a table has more pages than that holds.
// The threshold, the score of the last page taken, is found by histograms: the scores in question are spread evenly
// over 256 bins between their least and their largest, and those of the bin that holds the threshold are the next round's,
// until all of that bin are taken or all of them are equal.  Scores that are spread by chance take one to three rounds (a bin of
// 512 has a few), about 0.6 us each; a round takes at least the largest or the least away, and a bin is 1/255 of its round's
// range, so that no values of fp32 take more than 32.  (Two bits of the threshold at a time, sixteen counts of all scores, took
// 8 us for 512 pages.)  A thread then has a run of neighbouring pages, so that a scan over the threads gives the list's order.
constexpr int CHOOSE_THREADS = 256, CHOOSE_WARPS = CHOOSE_THREADS / 32, BINS = 256;
constexpr int HELD_PAGES = 10240;                // scores in shared memory at most: 40 KB
constexpr float FIRST_SCORE = 0x1p126f, LAST_SCORE = -0x1p126f;   // of a page with a NaN, of one that is not there

// Exclusive sums over the threads of two counts.
__device__ __forceinline__ void block_scan(int& x, int& y, int (&sums)[2][CHOOSE_WARPS]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, own_x = x, own_y = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ux = __shfl_up_sync(0xFFFFFFFFu, x, o), uy = __shfl_up_sync(0xFFFFFFFFu, y, o);
    if (lane >= o) {
      x += ux;
      y += uy;
    }
  }
  if (lane == 31) {
    sums[0][warp] = x;
    sums[1][warp] = y;
  }
  __syncthreads();
  x -= own_x;
  y -= own_y;
#pragma unroll
  for (int k = 0; k + 1 < CHOOSE_WARPS; ++k)
    if (k < warp) {
      x += sums[0][k];
      y += sums[1][k];
    }
}
// Floats as unsigned integers of the same order, and back.
__device__ __forceinline__ uint32_t key_of(float s) {
  const uint32_t u = __float_as_uint(s);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }

template <int D, int DT>
__global__ void __launch_bounds__(CHOOSE_THREADS) cache_choose_kernel(const SelectArgs a, int cols, int cs) {
  constexpr int LPP = D / 16, PPW = 32 / LPP;    // lanes per page (16 minima and 16 maxima each), pages per warp
  extern __shared__ float held[];                // scores, if they fit
  __shared__ __align__(16) uint8_t codes[2][D];
  __shared__ float tops[CHOOSE_WARPS];
  __shared__ uint32_t ends[2][CHOOSE_WARPS];
  __shared__ int bins[2][BINS], sums[2][CHOOSE_WARPS];
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const uint32_t row = blockIdx.x / cs, rank = blockIdx.x - row * cs;
  const uint32_t bt = row / a.Hkv, h = row - bt * a.Hkv, b = bt / a.T, t = bt - b * a.T;
  const Seen seen = seen_by(a, b, t);
  const int32_t* const table = a.pt.table + (long long)b * a.pt.stride;
  const int n = seen.pages, k = min(n, a.top), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool fits = a.pt.max_pages <= HELD_PAGES;
  float* scores = fits ? held : a.scores + (long long)row * a.pt.max_pages;

  // ---- scores: this block's run of the pages (where all are taken, none is needed) ----
  if (n > k) {
    const int G = a.Hq / a.Hkv;
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
    for (int i = 0; i < D / 32; ++i) top = fmaxf(top, tops[i]);
    // 2^(6 - floor(log2 top)); rows of nothing, and those with a NaN or an infinity, score 0 everywhere
    const int e = (int)(__float_as_uint(top) >> 23);
    const float f = e == 0 || e == 255 ? 0.f : __uint_as_float((uint32_t)min(max(260 - e, 1), 254) << 23);
    if (threadIdx.x < D) {
      codes[0][threadIdx.x] = f == 0.f ? 0 : (uint8_t)min(__float2int_rn(u * f), 127);
      codes[1][threadIdx.x] = f == 0.f ? 0 : (uint8_t)min(__float2int_rn(l * f), 127);
    }
    if (cs > 1) cg::this_cluster().sync();       // and the first block is there to be written to
    else __syncthreads();
    float* const out = fits && cs > 1 ? cg::this_cluster().map_shared_rank(held, 0) : scores;
    const int part = lane % LPP, each = (n + cs - 1) / cs, p_first = min((int)rank * each, n), p_last = min(p_first + each, n);
    const uint4 cu = *reinterpret_cast<const uint4*>(codes[0] + part * 16), cl = *reinterpret_cast<const uint4*>(codes[1] + part * 16);
    constexpr int BATCH = 4;                     // pages of a lane whose loads are all ahead of the first use
    for (int p0 = p_first + warp * PPW; p0 < p_last; p0 += BATCH * CHOOSE_WARPS * PPW) {
      int page[BATCH];
      uint32_t e8[BATCH];
      uint4 lo[BATCH], hi[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int p = p0 + i * CHOOSE_WARPS * PPW + lane / LPP;
        page[i] = p < p_last ? __ldca(table + p) : -1;
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
        e8[i] = 0;
        if (page[i] >= 0 && page[i] < a.num_pages) {
          const long long at = (long long)page[i] * a.Hkv + h;
          lo[i] = __ldca(reinterpret_cast<const uint4*>(a.codes + at * (2 * D)) + part);
          hi[i] = __ldca(reinterpret_cast<const uint4*>(a.codes + at * (2 * D) + D) + part);
          e8[i] = __ldca(a.exps + at);
        } else {
          page[i] = -1;
        }
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int p = p0 + i * CHOOSE_WARPS * PPW + lane / LPP;
        int d = __dp4a((int)hi[i].x, (int)cu.x, 0), m = __dp4a((int)lo[i].x, (int)cl.x, 0);
        d = __dp4a((int)hi[i].y, (int)cu.y, d);
        m = __dp4a((int)lo[i].y, (int)cl.y, m);
        d = __dp4a((int)hi[i].z, (int)cu.z, d);
        m = __dp4a((int)lo[i].z, (int)cl.z, m);
        d = __dp4a((int)hi[i].w, (int)cu.w, d);
        m = __dp4a((int)lo[i].w, (int)cl.w, m);
        d -= m;
#pragma unroll
        for (int o = LPP / 2; o; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
        if (part == 0 && p < p_last) {
          if (page[i] < 0) report(a.dev_status, CACHE_BAD_PAGE);
          // exponents that no bounds have (their buffer was never filled in) count as the nearest that they have: no score is
          // infinite or so small that a bin's width is not
          out[p] = page[i] < 0 ? LAST_SCORE : e8[i] == 0xFFu ? FIRST_SCORE : (float)d * scale_value(min(max(e8[i], 27u), 227u));
        }
      }
    }
  }
  if (cs > 1) cg::this_cluster().sync();
  else __syncthreads();
  if (rank != 0) return;

  int32_t* const list = a.table + (long long)row * cols;
  int32_t* const blocks = a.blocks ? a.blocks + (long long)row * a.top : nullptr;
  if (threadIdx.x == 0) {
    if (seen.past) report(a.dev_status, CACHE_BAD_LEN);
    a.lens[row] = k > 0 ? (k - 1) * a.page_size + seen.tokens - (n - 1) * a.page_size : 0;   // the last page is always listed
  }
  auto put = [&](int at, int p, int page) {
    list[at] = page >= 0 && page < a.num_pages ? page * a.pages_per_page + (int)h : -1;
    if (blocks) blocks[at] = p;
  };
  if (blocks)
    for (int i = k + threadIdx.x; i < a.top; i += CHOOSE_THREADS) blocks[i] = -1;
  if (n == k) {
    for (int i = threadIdx.x; i < k; i += CHOOSE_THREADS) put(i, i, __ldca(table + i));
    return;
  }

  // a thread's run of pages, the first two ids of it on their way
  const int run = (n + CHOOSE_THREADS - 1) / CHOOSE_THREADS, p0 = min((int)threadIdx.x * run, n), p1 = min(p0 + run, n);
  const int id0 = p0 < p1 ? __ldca(table + p0) : -1, id1 = p0 + 1 < p1 ? __ldca(table + p0 + 1) : -1;

  // ---- the threshold among pages [first, n - last): `want` of those with score `cut`, and all above it ----
  const int from = a.first, to = n - a.last;
  int want = k - a.first - a.last;
  float cut = INFINITY, base = 0.f, per = 0.f;   // the round before: bins of (score - base) * per
  bool whole = false;                            // all of `bin` is taken, and what lies above it
  float lo = -INFINITY, hi = INFINITY;
  int bin = 0;
  constexpr int MOST_ROUNDS = 64;                // never reached, unless another call writes to the workspace's scores meanwhile
  auto place_of = [](int bin) { return (bin & 7) * (BINS / 8) + (bin >> 3); };   // a lane's 8 bins in 8 places of one bank
  auto bin_of = [](float s, float base, float per) { return min((int)((s - base) * per), BINS - 1); };
  for (int round = 0; want > 0 && round < MOST_ROUNDS; ++round) {
    const int turn = round & 1;
    uint32_t least = 0xFFFFFFFFu, most = 0u;
    for (int p = from + threadIdx.x; p < to; p += CHOOSE_THREADS) {
      const float s = scores[p];
      if (s >= lo && s <= hi && bin_of(s, base, per) == bin) {
        least = min(least, key_of(s));
        most = max(most, key_of(s));
      }
    }
    least = __reduce_min_sync(0xFFFFFFFFu, least);
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) {
      ends[0][warp] = least;
      ends[1][warp] = most;
    }
    bins[turn][threadIdx.x] = 0;               // last read two rounds ago
    __syncthreads();
#pragma unroll
    for (int w = 0; w < CHOOSE_WARPS; ++w) {
      least = min(least, ends[0][w]);
      most = max(most, ends[1][w]);
    }
    lo = of_key(least);
    hi = of_key(most);
    if (least == most) {
      cut = lo;
      break;
    }
    base = lo;
    per = (float)(BINS - 1) / (hi - lo);
    for (int p = from + threadIdx.x; p < to; p += CHOOSE_THREADS) {
      const float s = scores[p];
      if (s >= lo && s <= hi) atomicAdd(&bins[turn][place_of(bin_of(s, base, per))], 1);
    }
    __syncthreads();
    // the bin of the want-th largest: every warp on its own, a lane with 8 bins, lane 0 the uppermost
    int c[8], mine = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = bins[turn][place_of(BINS - 1 - (lane * 8 + i))];
      mine += c[i];
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    const int who = __ffs(__ballot_sync(0xFFFFFFFFu, upto >= want)) - 1;
    int above = upto - mine, which = 0, in_it = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (in_it == 0) {
        if (above + c[i] >= want) {
          which = BINS - 1 - (lane * 8 + i);
          in_it = c[i];
        } else {
          above += c[i];
        }
      }
    bin = __shfl_sync(0xFFFFFFFFu, which, who);
    want -= __shfl_sync(0xFFFFFFFFu, above, who);
    if (want == __shfl_sync(0xFFFFFFFFu, in_it, who)) {
      whole = true;
      want = 0;
    }
  }

  // ---- the list ----
  // 2: taken, 1: of those with the threshold's score
  auto kind = [&](int p) {
    if (p < from || p >= to) return 2;
    const float s = scores[p];
    if (whole) return s > hi || (s >= lo && bin_of(s, base, per) >= bin) ? 2 : 0;
    return s > cut ? 2 : s == cut ? 1 : 0;
  };
  int at = 0, ties = 0;
  for (int p = p0; p < p1; ++p) {
    const int is = kind(p);
    at += is == 2;
    ties += is == 1;
  }
  block_scan(at, ties, sums);
  at += min(ties, want);
  for (int p = p0; p < p1; ++p) {
    const int is = kind(p);
    // (`at` stays below k unless another call writes to the workspace meanwhile)
    if ((is == 2 || (is == 1 && ties < want)) && at < k) put(at++, p, p == p0 ? id0 : p == p0 + 1 ? id1 : __ldca(table + p));
    ties += is == 1;
  }
}

}  // namespace

cudaError_t launch_cache_bounds(const BoundsArgs& a, int format, int D, cudaStream_t st) {
  const int per_seq = (int)((a.T - 1LL + a.c.page_size - 1) / a.c.page_size) + 1;   // pages that T neighbouring tokens can touch
  const unsigned grid = (unsigned)a.B * per_seq * a.c.Hkv;
  const auto k = format == CACHE_FP4 ? (D == 128 ? cache_bounds_kernel<CACHE_FP4, 128> : cache_bounds_kernel<CACHE_FP4, 64>)
                                     : (D == 128 ? cache_bounds_kernel<CACHE_FP8, 128> : cache_bounds_kernel<CACHE_FP8, 64>);
  return launch_early(k, grid, BOUNDS_THREADS, 0, st, 1, a, per_seq);
}

size_t cache_select_scores_bytes(int rows, int max_pages, int top) {
  return max_pages > top && max_pages > HELD_PAGES ? (size_t)rows * max_pages * 4 : 0;
}

cudaError_t launch_cache_select(const SelectArgs& a, int D, int dtype, cudaStream_t st) {
  const int rows = a.B * a.T * a.Hkv, cols = a.top < a.pt.max_pages ? a.top : a.pt.max_pages;
  const bool scored = a.pt.max_pages > a.top;
  // blocks of a row's cluster: while they all run at once (two to an SM) and each has CLUSTER_PAGES pages
  constexpr int CLUSTER_PAGES = 64, SMS = 152;
  int cs = 1;
  while (scored && cs < 8 && (long long)rows * cs * 2 <= 2 * SMS && a.pt.max_pages >= cs * 2 * CLUSTER_PAGES) cs *= 2;
  const size_t smem = scored && a.pt.max_pages <= HELD_PAGES ? (size_t)a.pt.max_pages * 4 : 0;
  const auto k = D == 128 ? (dtype ? cache_choose_kernel<128, 1> : cache_choose_kernel<128, 0>)
                          : (dtype ? cache_choose_kernel<64, 1> : cache_choose_kernel<64, 0>);
  return launch_early(k, (unsigned)(rows * cs), CHOOSE_THREADS, smem, st, cs, a, cols, cs);
}

}  // namespace bsc
