// Root-mean-square norm of rows, with the residual's addition, a 16-bit and/or MXFP8 output, and its gradients.
//
//   s = round(x + r),  rstd = (mean_n s_n^2 + eps)^(-1/2),  y_n = s_n rstd w_n
//   g = dy w,  c = rstd mean_n g_n s_n,  dx = rstd (g - s rstd c) + ds,  dw_n = sum over rows of dy_n s_n rstd
//
// Roundings.  s is the residual stream: the next layer adds to it and the gradients are taken at it, so it is held in the
// activations' type and y is the norm of what is held.  Everything between s and an output is fp32, rounded once.
//
// What bounds it: memory, if little else is done per row.  A block has every gridDim-th row (or group of rows): its threads
// keep their columns' weights (and dw's sums) in registers as fp32, and each copies its own pieces of the rows ahead into its
// own slots of a ring in shared memory (cp.async), so that nothing but a row's sum is shared and the bytes in flight are not
// held in registers.  Rows of up to 1024 elements belong to part of a warp, longer ones to a block.  FLAT rows are evenly
// spaced: addresses move by addition; heads of a slice take two divisions per row and tensor (262144 x 128 25.3 us against 23.8).
// bf16, fp32 weights: 16384 x 4096 with a residual 85.7 us (6.3 TB/s, 94% of the copy rate), its gradients with ds 89.6 (90%);
// 262144 x 128 23.8 and 49.0.  To MXFP8 latency bounds it: 41.4 us for 3 bytes per element (74%), DRAM at 48%, issue slots at 65%,
// 15 warps per SM that wait for their own last instructions (1.8 per issue) and for shared memory and shuffles (1.2), for memory 0.15.
#include <atomic>
#include <type_traits>

#include "cache.cuh"

namespace bsc {
namespace {

constexpr int SMS = 152;
constexpr int NARROW_THREADS = 128, WIDE_THREADS = 512;   // most threads of a block
// Threads per SM that the registers of V vectors (of 8 elements) per thread leave room for.
constexpr int threads_per_sm(int v) { return v < 4 ? 1024 : 512; }
constexpr int blocks_per_sm(int v, bool wide) { return threads_per_sm(v) / (wide ? WIDE_THREADS : NARROW_THREADS); }
// Rows in the ring, and its bytes per thread for `pieces` tensors and `scalars` fp32 of a row.
constexpr int stages(int v) { return v == 1 ? 4 : v == 2 ? 3 : 2; }
constexpr int ring_bytes(int v, int pieces, int scalars) { return stages(v) * (pieces * v * 16 + scalars * 4); }

template <int DT>
__device__ __forceinline__ void unpack8(const uint4& v, float2 (&f)[4]) {
  f[0] = act_to_f32<DT>(v.x);
  f[1] = act_to_f32<DT>(v.y);
  f[2] = act_to_f32<DT>(v.z);
  f[3] = act_to_f32<DT>(v.w);
}
template <int DT>
__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(f32_to_act<DT>(f[0].x, f[0].y), f32_to_act<DT>(f[1].x, f[1].y), f32_to_act<DT>(f[2].x, f[2].y),
                    f32_to_act<DT>(f[3].x, f[3].y));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Eight weights from the `at`-th on.
template <int DT>
__device__ __forceinline__ void load_weights(const void* w, int w32, int at, float2 (&f)[4]) {
  if (w32) {
    const float4 a = __ldca(reinterpret_cast<const float4*>(w) + 2 * at), b = __ldca(reinterpret_cast<const float4*>(w) + 2 * at + 1);
    f[0] = make_float2(a.x, a.y); f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y); f[3] = make_float2(b.z, b.w);
  } else {
    unpack8<DT>(__ldca(reinterpret_cast<const uint4*>(w) + at), f);
  }
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }

// Sum over the threads of a row: `tpr` lanes of a warp, or the block, whose warps' sums pass through `part` (two of them in
// turn, so that one barrier per row is enough).
template <bool WIDE>
__device__ __forceinline__ float row_sum(float v, int tpr, float* part) {
  if (WIDE) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int at = threadIdx.x & 15, warps = blockDim.x >> 5;    // at most 16: both halves of a warp add up the same
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = at < warps ? part[at] : 0.f;
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  } else {
    for (int o = tpr >> 1; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  return v;
}

// x^(-1/2), refined by one step so that it is within an ulp; where x is 0 or not finite, the limit as it stands.
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x);
  return x > 0.f && x < INFINITY ? fmaf(0.5f * r, fmaf(-x * r, r, 1.f), r) : r;
}

__device__ __forceinline__ long long row_at(const NormRows& s, long long row, int inner) {
  const long long o = row / inner;
  return o * s.outer + (row - o * inner) * s.inner;
}
// The rows that a thread meets, one after another: at its vector t of row `row`, and `rows_on` rows on.
template <bool FLAT>
struct Walk {
  uint16_t* p;
  long long step;
  __device__ __forceinline__ Walk(const void* base, const NormRows& s, long long row, long long rows_on, int t) {
    p = reinterpret_cast<uint16_t*>(const_cast<void*>(base)) + t * 8 + (FLAT ? row * s.outer : 0);
    step = FLAT ? rows_on * s.outer : 0;
  }
  // at the next row
  __device__ __forceinline__ uint4* next(const NormRows& s, long long row, int inner) {
    uint4* const at = reinterpret_cast<uint4*>(FLAT ? p : p + row_at(s, row, inner));
    if (FLAT) p += step;
    return at;
  }
};
// A thread's rows: the first, the step from one to the next, how many it has, and how many the block's first thread has (the
// rows of one warp end together: loops go by that).  Fewer than 2^31: the host checks rows, and a grid that is full has
// 152 blocks at least.
struct Rows {
  long long first, step;
  int count, rounds;
  __device__ __forceinline__ Rows(long long rows, int per_block, int group) {
    const long long block = (long long)blockIdx.x * per_block;
    step = (long long)gridDim.x * per_block;
    first = block + group;
    rounds = (int)((rows - block + step - 1) / step);          // no block is without a row
    count = first < rows ? (int)((rows - first + step - 1) / step) : 0;
  }
};

// RES: a residual is added (and the sum written, where it is asked for).
template <int DT, int V, bool WIDE, bool FLAT, bool RES>
__global__ void __launch_bounds__(WIDE ? WIDE_THREADS : NARROW_THREADS, blocks_per_sm(V, WIDE)) norm_kernel(const NormArgs a, int tpr) {
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float part[2][32];
  constexpr int STAGES = stages(V), PIECES = RES ? 2 : 1;
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const int threads = blockDim.x, t = WIDE ? threadIdx.x : threadIdx.x % tpr, nv = a.N / 8;
  const Rows rows(a.rows, WIDE ? 1 : NARROW_THREADS / tpr, WIDE ? 0 : threadIdx.x / tpr);
  uint4* const own = ring + threadIdx.x;                         // piece p of stage g: own[(g * PIECES * V + p) * threads]
  Walk<FLAT> xw(a.x, a.xs, rows.first, rows.step, t), rw(a.r, a.rs, rows.first, rows.step, t);
  Walk<FLAT> sw(a.s, a.ss, rows.first, rows.step, t), yw(a.y, a.ys, rows.first, rows.step, t);
  auto fetch = [&](int i, uint4* to) {                           // its i-th row
    if (i < rows.count) {
      const long long row = FLAT ? 0 : rows.first + i * rows.step;
      const uint4* const xp = xw.next(a.xs, row, a.inner);
      const uint4* const rp = RES ? rw.next(a.rs, row, a.inner) : nullptr;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * tpr + t < nv) {
          copy16(to + v * threads, xp + v * tpr);
          if (RES) copy16(to + (V + v) * threads, rp + v * tpr);
        }
    }
    copies_end();
  };
  const int stage = PIECES * V * threads;
  uint4 *from = own, *into = own;
#pragma unroll
  for (int g = 0; g < STAGES - 1; ++g) {
    fetch(g, into);
    into += stage;
  }
  float2 w[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v * tpr + t < nv) load_weights<DT>(a.w, a.w32, v * tpr + t, w[v]);
  const uint32_t up = ceil_carry<CACHE_FP8>(a.rule);
  const float inv_n = 1.f / (float)a.N;
  float* rstds = a.rstd + rows.first;
  for (int i = 0; i < rows.rounds; ++i) {
    const bool live = i < rows.count;
    const long long row = rows.first + i * rows.step;
    copies_wait<STAGES - 2>();
    uint4 s[V];
    float2 sum = both(0.f);
    uint4* const sp = a.s ? sw.next(a.ss, row, a.inner) : nullptr;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      s[v] = make_uint4(0, 0, 0, 0);
      if (v * tpr + t < nv && live) {
        s[v] = from[v * threads];
        float2 f[4];
        unpack8<DT>(s[v], f);
        if (RES) {
          float2 g[4];
          unpack8<DT>(from[(V + v) * threads], g);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = __fadd2_rn(f[j], g[j]);
          s[v] = pack8<DT>(f);
          unpack8<DT>(s[v], f);
        }
        if (a.s) __stcs(sp + v * tpr, s[v]);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = __ffma2_rn(f[j], f[j], sum);
      }
    }
    from = from == own + (STAGES - 1) * stage ? own : from + stage;
    fetch(i + STAGES - 1, into);                 // into the stage that was read before this one: its values are used
    into = into == own + (STAGES - 1) * stage ? own : into + stage;
    const float rstd = inverse_root(row_sum<WIDE>(sum.x + sum.y, tpr, part[i & 1]) * inv_n + a.eps);
    if (a.rstd) {
      if (t == 0 && live) *rstds = rstd;
      rstds += rows.step;
    }
    uint4* const yp = a.y ? yw.next(a.ys, row, a.inner) : nullptr;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = v * tpr + t;
      const bool mine = j < nv && live;
      float2 f[4];
      unpack8<DT>(s[v], f);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = __fmul2_rn(__fmul2_rn(f[k], both(rstd)), w[v][k]);
      if (a.y && mine) __stcs(yp + v * tpr, pack8<DT>(f));
      if (a.y8) {                    // 32 elements are four neighbouring lanes
        float am = amax8(f);
        am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
        am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
        float inv;
        const uint32_t sb = block_scale<CACHE_FP8>(am, up, inv);
        if (mine) {
          __stcs(reinterpret_cast<uint2*>(a.y8 + row * a.N) + j, quant8_e4m3(f, inv, sb));
          if ((t & 3) == 0) a.ysc[row * (a.N / 32) + (j >> 2)] = (uint8_t)sb;
        }
      }
    }
  }
}

// The gradients of a block's rows; dw's share of the block goes to partial[block][N].
template <int DT, int V, bool WIDE, bool FLAT>
__global__ void __launch_bounds__(WIDE ? WIDE_THREADS : NARROW_THREADS, blocks_per_sm(V, WIDE))
    norm_bwd_kernel(const NormBwdArgs a, int tpr) {
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float part[2][32];
  constexpr int STAGES = stages(V);
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const int threads = blockDim.x, t = WIDE ? threadIdx.x : threadIdx.x % tpr, nv = a.N / 8;
  const Rows rows(a.rows, WIDE ? 1 : NARROW_THREADS / tpr, WIDE ? 0 : threadIdx.x / tpr);
  const int stage = (a.ds ? 3 : 2) * V * threads;
  uint4* const own = ring + threadIdx.x;
  float* const own_rstd = reinterpret_cast<float*>(ring + STAGES * stage) + threadIdx.x;    // of stage g: [g * threads]
  Walk<FLAT> dw(a.dy, a.dys, rows.first, rows.step, t), sw(a.s, a.ss, rows.first, rows.step, t);
  Walk<FLAT> ew(a.ds, a.dss, rows.first, rows.step, t), ow(a.dx, a.dxs, rows.first, rows.step, t);
  const float* rstds = a.rstd + rows.first;
  auto fetch = [&](int i, int g) {               // its i-th row, into stage g
    if (i < rows.count) {
      const long long row = FLAT ? 0 : rows.first + i * rows.step;
      const uint4 *const dp = dw.next(a.dys, row, a.inner), *const sp = sw.next(a.ss, row, a.inner);
      const uint4* const ep = a.ds ? ew.next(a.dss, row, a.inner) : nullptr;
      uint4* const to = own + g * stage;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * tpr + t < nv) {
          copy16(to + v * threads, dp + v * tpr);
          copy16(to + (V + v) * threads, sp + v * tpr);
          if (a.ds) copy16(to + (2 * V + v) * threads, ep + v * tpr);
        }
      copy4(own_rstd + g * threads, rstds);
      rstds += rows.step;
    }
    copies_end();
  };
#pragma unroll
  for (int g = 0; g < STAGES - 1; ++g) fetch(g, g);
  float2 w[V][4], acc[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (v * tpr + t < nv) load_weights<DT>(a.w, a.w32, v * tpr + t, w[v]);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[v][k] = both(0.f);
  }
  const float inv_n = 1.f / (float)a.N;
  int g = 0;
  for (int i = 0; i < rows.rounds; ++i) {
    const bool live = i < rows.count;
    copies_wait<STAGES - 2>();
    const uint4* const from = own + g * stage;
    const float rs = live ? own_rstd[g * threads] : 0.f;
    constexpr bool KEPT = V == 1;                // dy and s stay in registers; more vectors are read again
    uint4 d0[KEPT ? V : 1], x0[KEPT ? V : 1];
    float2 sum = both(0.f);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * tpr + t < nv && live) {
        const uint4 dv = from[v * threads], xv = from[(V + v) * threads];
        if (KEPT) {
          d0[v] = dv;
          x0[v] = xv;
        }
        float2 d[4], x[4];
        unpack8<DT>(dv, d);
        unpack8<DT>(xv, x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 p = __fmul2_rn(d[k], __fmul2_rn(x[k], both(rs)));
          acc[v][k] = __fadd2_rn(acc[v][k], p);
          sum = __ffma2_rn(p, w[v][k], sum);
        }
      }
    const float c = row_sum<WIDE>(sum.x + sum.y, tpr, part[i & 1]) * inv_n;
    if (live) {
      uint4* const out = ow.next(a.dxs, rows.first + i * rows.step, a.inner);
      const float2 xc = both(-rs * c);           // times x it is no larger than g: rs^2 c may leave fp32's range where dx does not
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * tpr + t < nv) {
          float2 d[4], x[4], e[4];
          unpack8<DT>(KEPT ? d0[KEPT ? v : 0] : from[v * threads], d);
          unpack8<DT>(KEPT ? x0[KEPT ? v : 0] : from[(V + v) * threads], x);
#pragma unroll
          for (int k = 0; k < 4; ++k) e[k] = both(0.f);
          if (a.ds) unpack8<DT>(from[(2 * V + v) * threads], e);
#pragma unroll
          for (int k = 0; k < 4; ++k)     // rs (d w - x rs c) + e
            d[k] = __ffma2_rn(__ffma2_rn(x[k], xc, __fmul2_rn(d[k], w[v][k])), both(rs), e[k]);
          __stcs(out + v * tpr, pack8<DT>(d));
        }
    }
    fetch(i + STAGES - 1, g == 0 ? STAGES - 1 : g - 1);   // into the stage that was read before this one
    g = g + 1 == STAGES ? 0 : g + 1;
  }
  float* const out = a.partial + (long long)blockIdx.x * a.N;
  float2* const group = reinterpret_cast<float2*>(ring);           // narrow: over the ring, whose copies have landed
  const int groups = WIDE ? 1 : NARROW_THREADS / tpr;
  copies_wait<0>();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!WIDE) {                     // the block's rows' shares of these columns, in their order
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 4; ++k) group[threadIdx.x * 4 + k] = acc[v][k];
      __syncthreads();
      if (threadIdx.x < tpr)
        for (int q = 1; q < groups; ++q)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[v][k] = __fadd2_rn(acc[v][k], group[(q * tpr + t) * 4 + k]);
    }
    const int j = v * tpr + t;
    if (j < nv && (WIDE || threadIdx.x < tpr)) {
      float4* const dst = reinterpret_cast<float4*>(out) + 2 * j;
      dst[0] = make_float4(acc[v][0].x, acc[v][0].y, acc[v][1].x, acc[v][1].y);
      dst[1] = make_float4(acc[v][2].x, acc[v][2].y, acc[v][3].x, acc[v][3].y);
    }
  }
}

// dw = the blocks' shares summed, in their order: 32 columns per block, each warp every 16th share.
constexpr int DW_WARPS = 16;
__global__ void __launch_bounds__(DW_WARPS * 32) norm_dw_kernel(const float* partial, int parts, int N, void* dw, int dtype) {
  __shared__ float sums[DW_WARPS][32];
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (n < N) {
#pragma unroll 8
    for (int p = warp; p < parts; p += DW_WARPS) v += __ldcg(partial + (long long)p * N + n);
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || n >= N) return;
  for (int k = 1; k < DW_WARPS; ++k) v += sums[k][lane];
  if (dtype == 2) reinterpret_cast<float*>(dw)[n] = v;
  else if (dtype == 1) reinterpret_cast<__half*>(dw)[n] = __float2half_rn(v);
  else reinterpret_cast<__nv_bfloat16*>(dw)[n] = __float2bfloat16_rn(v);
}

// How a row is cut up: vectors of 8 elements per thread, threads per row, and whether a block has one row.
//
// Forward: four vectors a thread, which share the row's sum and addresses, but one while there are no more rows than SMs, so
// that a row has as many threads as it can use.  1 / 2 / 4 vectors, bf16 with fp32 weights, us: 262144 x 128 26.7 / 21.0 / 23.2
// (with a residual 49.3 / 48.5 / 44.3, to MXFP8 34.9 / 29.2 / 21.0), 131072 x 512 - / 48.3 / 44.6 (- / 95.0 / 87.0, - / 57.6 / 41.9),
// 16384 x 4096 44.7 / 45.4 / 46.0 (92.4 / 89.9 / 85.7, 58.4 / 50.7 / 41.7); one row of 2048 4.1 / - / 5.5.
// Gradients keep dw's sums beside the weights: four vectors where a row is part of a warp (262144 x 256 92.3 / 121 / 87.1; 600000 x
// 64, one per thread, 56.5 and two 76), else as few as a block of 512 threads has room for (16384 x 4096 90.1 / 94.2 / -).
struct Cut {
  int v, tpr;
  bool wide;
  int threads() const { return wide ? tpr : NARROW_THREADS; }
  int rows() const { return wide ? 1 : NARROW_THREADS / tpr; }     // of a block at a time
};
Cut cut_for(int nv, int v) {
  if (nv <= 32 * v) {
    int tpr = 4;
    while (tpr * v < nv) tpr *= 2;
    return {v, tpr, false};
  }
  return {v, ((nv + v - 1) / v + 31) / 32 * 32, true};
}
Cut cut_of(const NormArgs& a) {
  const int nv = a.N / 8;
  if (a.rows <= SMS) return cut_for(nv, nv <= WIDE_THREADS ? 1 : nv <= 2 * WIDE_THREADS ? 2 : 4);
  return cut_for(nv, nv <= 4 ? 1 : nv <= 8 ? 2 : 4);
}
Cut bwd_cut(int N) {
  const int nv = N / 8;
  return cut_for(nv, nv <= 8 ? 1 : nv <= 128 ? 4 : nv <= WIDE_THREADS ? 1 : nv <= 2 * WIDE_THREADS ? 2 : 4);
}
Cut cut_of(const NormBwdArgs& a) { return bwd_cut(a.N); }
// As many blocks as the card takes at once by registers and shared memory, or as there are rows for.
int blocks_for(long long rows, const Cut& c, int smem) {
  const int by_regs = threads_per_sm(c.v) / c.threads(), by_smem = 225 * 1024 / (smem + 1280);
  const long long want = (rows + c.rows() - 1) / c.rows(), most = (long long)SMS * (by_regs < by_smem ? by_regs : by_smem);
  return (int)(want < most ? want : most);
}
int smem_of(const Cut& c, int pieces, int scalars) { return c.threads() * ring_bytes(c.v, pieces, scalars); }
// The gradients' grid decides the order of dw's sums, so it goes by rows and N alone.
int bwd_blocks(long long rows, int N) {
  const Cut c = bwd_cut(N);
  return blocks_for(rows, c, smem_of(c, 3, 1));
}

template <class A>
cudaError_t go(void (*kernel)(A, int), int most_smem, const A& a, const Cut& c, int blocks, int smem, std::atomic<uint64_t>& opted,
               cudaStream_t st) {
  int dev = 0;                                 // the opt-in to more than 48 KB of shared memory, once per device
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!((opted.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
    if (e != cudaSuccess) return e;
    opted.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  return launch_early(kernel, (unsigned)blocks, c.threads(), smem, st, 1, a, c.tpr);
}
template <int DT, int V, bool WIDE, bool FLAT, bool RES>
cudaError_t run_norm(const NormArgs& a, const Cut& c, cudaStream_t st) {
  static std::atomic<uint64_t> opted{0};
  const int smem = smem_of(c, RES ? 2 : 1, 0);
  return go(norm_kernel<DT, V, WIDE, FLAT, RES>, (WIDE ? WIDE_THREADS : NARROW_THREADS) * ring_bytes(V, RES ? 2 : 1, 0), a, c,
            blocks_for(a.rows, c, smem), smem, opted, st);
}
template <int DT, int V, bool WIDE, bool FLAT>
cudaError_t run(const NormArgs& a, const Cut& c, cudaStream_t st) {
  return a.r ? run_norm<DT, V, WIDE, FLAT, true>(a, c, st) : run_norm<DT, V, WIDE, FLAT, false>(a, c, st);
}
template <int DT, int V, bool WIDE, bool FLAT>
cudaError_t run(const NormBwdArgs& a, const Cut& c, cudaStream_t st) {
  static std::atomic<uint64_t> opted{0};
  const int most = (WIDE ? WIDE_THREADS : NARROW_THREADS) * ring_bytes(V, 3, 1), group = NARROW_THREADS * 32;
  const int smem = smem_of(c, a.ds ? 3 : 2, 1);
  return go(norm_bwd_kernel<DT, V, WIDE, FLAT>, most, a, c, bwd_blocks(a.rows, a.N), WIDE || smem > group ? smem : group, opted,
            st);
}
template <int DT, bool FLAT, class A>
cudaError_t pick(const A& a, const Cut& c, cudaStream_t st) {
  if (c.wide)
    return c.v == 1 ? run<DT, 1, true, FLAT>(a, c, st) : c.v == 2 ? run<DT, 2, true, FLAT>(a, c, st) : run<DT, 4, true, FLAT>(a, c, st);
  if constexpr (std::is_same<A, NormArgs>::value)                // bwd_cut has no rows of part of a warp by two vectors
    if (c.v == 2) return run<DT, 2, false, FLAT>(a, c, st);
  return c.v == 1 ? run<DT, 1, false, FLAT>(a, c, st) : run<DT, 4, false, FLAT>(a, c, st);
}
template <class A>
cudaError_t pick(const A& a, int dtype, cudaStream_t st) {
  const Cut c = cut_of(a);
  if (dtype == 0) return a.inner == 1 ? pick<0, true>(a, c, st) : pick<0, false>(a, c, st);
  return a.inner == 1 ? pick<1, true>(a, c, st) : pick<1, false>(a, c, st);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, cudaStream_t st) { return pick(a, dtype, st); }

cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, cudaStream_t st) {
  const cudaError_t e = pick(a, dtype, st);
  if (e != cudaSuccess) return e;
  return launch_early(norm_dw_kernel, (unsigned)((a.N + 31) / 32), DW_WARPS * 32, 0, st, 1, (const float*)a.partial,
                      bwd_blocks(a.rows, a.N), a.N, a.dw, a.w32 ? 2 : dtype);
}

size_t norm_bwd_workspace_bytes(long long rows, int N) { return (size_t)bwd_blocks(rows, N) * N * 4; }

}  // namespace bsc
