// Root-mean-square norm of rows, with the residual's addition, a 16-bit and/or MXFP8 output, and its gradients.
//
//   s = round(x + r),  rstd = (mean_n s_n^2 + eps)^(-1/2),  y_n = s_n rstd w_n
//   g = dy w,  c = rstd mean_n g_n s_n,  dx = rstd (g - s rstd c) + ds,  dw_n = sum over rows of dy_n s_n rstd
//
// Roundings.  s is the residual stream: the next layer adds to it and the gradients are taken at it, so it is held in the
// activations' type and y is the norm of what is held.  Everything between s and an output is fp32, rounded once.
//
// What bounds it: memory.  A row is read once, kept in registers through the sum, and written once; a block walks over rows
// with the weights in registers and the next row's loads in flight.  Rows of up to 1024 elements belong to part of a
// warp, longer ones to a block.
#include <atomic>
#include <type_traits>

#include "cache.cuh"

namespace bsc {
namespace {

constexpr int SMS = 152;
constexpr int NARROW_THREADS = 128, WIDE_THREADS = 512;   // most threads of a block
// Threads per SM that the registers of V vectors per thread leave room for.
constexpr int threads_per_sm(int v) { return v < 4 ? 1024 : 512; }   // forward
constexpr int bwd_threads_per_sm(int v) { return v < 4 ? 1024 : 512; }
constexpr int blocks_per_sm(int threads, bool wide) { return threads / (wide ? WIDE_THREADS : NARROW_THREADS); }

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

// Eight weights as they are held: one or two 16-byte pieces.
template <int DT, bool W32>
struct Weights {
  uint4 v[W32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* w, int at) {
#pragma unroll
    for (int i = 0; i < (W32 ? 2 : 1); ++i) v[i] = __ldca(reinterpret_cast<const uint4*>(w) + (W32 ? 2 : 1) * at + i);
  }
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    if constexpr (W32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[2 * i] = make_float2(__uint_as_float(v[i].x), __uint_as_float(v[i].y));
        f[2 * i + 1] = make_float2(__uint_as_float(v[i].z), __uint_as_float(v[i].w));
      }
    } else {
      unpack8<DT>(v[0], f);
    }
  }
};

// Sum over the threads of a row: `tpr` lanes of a warp, or the block, whose warps' sums pass through `part` (two of them in
// turn, so that one barrier per row is enough).
template <bool WIDE>
__device__ __forceinline__ float row_sum(float v, int tpr, float* part) {
  if (WIDE) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  } else {
    for (int o = tpr >> 1; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  }
  return v;
}

__device__ __forceinline__ long long row_at(const NormRows& s, long long row, int inner) {
  if (inner == 1) return row * s.outer;
  const long long o = row / inner;
  return o * s.outer + (row - o * inner) * s.inner;
}

template <int DT, bool W32, int V, bool WIDE>
__global__ void __launch_bounds__(WIDE ? WIDE_THREADS : NARROW_THREADS, blocks_per_sm(threads_per_sm(V), WIDE))
    norm_kernel(const NormArgs a, int tpr) {
  __shared__ float part[32];
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const int rpb = WIDE ? 1 : NARROW_THREADS / tpr, t = WIDE ? threadIdx.x : threadIdx.x % tpr;
  const int nv = a.N / 8;
  // rows of one warp end together: the loop goes by the block's first row
  for (long long first = (long long)blockIdx.x * rpb; first < a.rows; first += (long long)gridDim.x * rpb) {
    const long long row = first + (WIDE ? 0 : threadIdx.x / tpr);
    const bool live = row < a.rows;
    uint4 x[V], r[V];
    Weights<DT, W32> w[V];
    const uint4* const xp = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) + row_at(a.xs, row, a.inner)) + t;
    const uint4* const rp = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.r) + row_at(a.rs, row, a.inner)) + t;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = make_uint4(0, 0, 0, 0);
      if (v * tpr + t < nv && live) {
        x[v] = __ldcs(xp + v * tpr);
        if (a.r) r[v] = __ldcs(rp + v * tpr);
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * tpr + t < nv) w[v].load(a.w, v * tpr + t);
    float2 sum = both(0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float2 f[4];
      unpack8<DT>(x[v], f);
      if (a.r && v * tpr + t < nv && live) {
        float2 g[4];
        unpack8<DT>(r[v], g);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __fadd2_rn(f[i], g[i]);
        x[v] = pack8<DT>(f);
        unpack8<DT>(x[v], f);
        if (a.s)
          __stcs(reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.s) + row_at(a.ss, row, a.inner)) + v * tpr + t, x[v]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) sum = __ffma2_rn(f[i], f[i], sum);
    }
    const float rstd = rsqrtf(row_sum<WIDE>(sum.x + sum.y, tpr, part) / (float)a.N + a.eps);
    if (a.rstd && t == 0 && live) a.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = v * tpr + t;
      const bool mine = j < nv && live;
      float2 f[4], g[4];
      unpack8<DT>(x[v], f);
      w[v].get(g);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __fmul2_rn(__fmul2_rn(f[i], both(rstd)), g[i]);
      if (a.y && mine)
        __stcs(reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.y) + row_at(a.ys, row, a.inner)) + j, pack8<DT>(f));
      if (a.y8) {                    // 32 elements are four neighbouring lanes
        float am = amax8(f);
        am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
        am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
        float inv;
        const uint32_t sb = block_scale<CACHE_FP8>(am, ceil_carry<CACHE_FP8>(a.rule), inv);
        if (mine) {
          __stcs(reinterpret_cast<uint2*>(a.y8 + row * a.N) + j, quant8_e4m3(f, inv, sb));
          if ((t & 3) == 0) a.ysc[row * (a.N / 32) + (j >> 2)] = (uint8_t)sb;
        }
      }
    }
    if (WIDE) __syncthreads();       // before the next row's sums are written
  }
}

// The gradients of a block's rows; dw's share of the block goes to partial[block][N].
//
// A block has every gridDim-th row (or group of rows), and every thread its own columns of them, so that dw's sums stay in
// registers.  Each thread copies its own pieces of the rows ahead into its own slots of a ring in shared memory
// (cp.async): nothing but the row's sum is shared, and the bytes in flight are not held in registers.
template <int V>
struct Ring {
  static constexpr int STAGES = V == 1 ? 4 : 2;
  static constexpr int THREAD_BYTES = STAGES * (3 * V * 16 + 4);
};
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
template <int DT, bool W32, int V, bool WIDE>
__global__ void __launch_bounds__(WIDE ? WIDE_THREADS : NARROW_THREADS, blocks_per_sm(bwd_threads_per_sm(V), WIDE))
    norm_bwd_kernel(const NormBwdArgs a, int tpr) {
  extern __shared__ __align__(16) uint4 ring[];
  __shared__ float part[2][32];
  constexpr int STAGES = Ring<V>::STAGES;
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const int threads = blockDim.x, rpb = WIDE ? 1 : NARROW_THREADS / tpr, t = WIDE ? threadIdx.x : threadIdx.x % tpr;
  const int nv = a.N / 8;
  const long long step = (long long)gridDim.x * rpb;
  const long long row0 = (long long)blockIdx.x * rpb + (WIDE ? 0 : threadIdx.x / tpr);
  uint4* const own = ring + threadIdx.x;                         // piece p of stage g: own[(g * 3 V + p) * threads]
  float* const own_rstd = reinterpret_cast<float*>(ring + STAGES * 3 * V * threads) + threadIdx.x;   // of stage g: [g * threads]
  auto at_row = [&](const void* p, const NormRows& rs, long long at) {
    return reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + row_at(rs, at, a.inner)) + t;
  };
  auto fetch = [&](long long at, int stage) {
    if (at < a.rows) {
      const uint4 *const dp = at_row(a.dy, a.dys, at), *const sp = at_row(a.s, a.ss, at), *const rp = at_row(a.ds, a.dss, at);
      uint4* const to = own + stage * 3 * V * threads;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * tpr + t < nv) {
          copy16(to + (3 * v) * threads, dp + v * tpr);
          copy16(to + (3 * v + 1) * threads, sp + v * tpr);
          if (a.ds) copy16(to + (3 * v + 2) * threads, rp + v * tpr);
        }
      copy4(own_rstd + stage * threads, a.rstd + at);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int g = 0; g < STAGES - 1; ++g) fetch(row0 + g * step, g);
  Weights<DT, W32> w[V];
  float2 acc[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (v * tpr + t < nv) w[v].load(a.w, v * tpr + t);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[v][i] = both(0.f);
  }
  const float inv_n = 1.f / (float)a.N;
  int turn = 0, stage = 0;
  long long row = row0;
  for (long long first = (long long)blockIdx.x * rpb; first < a.rows; first += step, row += step, turn ^= 1) {
    const bool live = row < a.rows;
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    const uint4* const from = own + stage * 3 * V * threads;
    const float rs = live ? own_rstd[stage * threads] : 0.f;
    float2 sum = both(0.f);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * tpr + t < nv && live) {
        float2 d[4], x[4], g[4];
        unpack8<DT>(from[(3 * v) * threads], d);
        unpack8<DT>(from[(3 * v + 1) * threads], x);
        w[v].get(g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 hat = __fmul2_rn(x[i], both(rs));
          acc[v][i] = __ffma2_rn(d[i], hat, acc[v][i]);
          sum = __ffma2_rn(__fmul2_rn(d[i], g[i]), hat, sum);
        }
      }
    const float c = row_sum<WIDE>(sum.x + sum.y, tpr, part[turn]) * inv_n;
    if (live) {
      uint4* const out = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.dx) + row_at(a.dxs, row, a.inner)) + t;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v * tpr + t < nv) {
          float2 d[4], x[4], g[4], e[4];
          unpack8<DT>(from[(3 * v) * threads], d);
          unpack8<DT>(from[(3 * v + 1) * threads], x);
          w[v].get(g);
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = both(0.f);
          if (a.ds) unpack8<DT>(from[(3 * v + 2) * threads], e);
#pragma unroll
          for (int i = 0; i < 4; ++i)     // rs (d g - x rs c) + e
            d[i] = __ffma2_rn(both(rs), __ffma2_rn(__fmul2_rn(x[i], both(rs)), both(-c), __fmul2_rn(d[i], g[i])), e[i]);
          __stcs(out + v * tpr, pack8<DT>(d));
        }
    }
    // the stage after the last one in flight is the one read before this: its values are used
    fetch(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
  float* const out = a.partial + (long long)blockIdx.x * a.N;
  float2* const group = reinterpret_cast<float2*>(ring);           // narrow: over the ring, whose copies have landed
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!WIDE) {                     // the block's rows' shares of these columns, in their order
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) group[threadIdx.x * 4 + i] = acc[v][i];
      __syncthreads();
      if (threadIdx.x < tpr)
        for (int k = 1; k < rpb; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[v][i] = __fadd2_rn(acc[v][i], group[(k * tpr + t) * 4 + i]);
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
struct Cut {
  int v, tpr;
  bool wide;
  int threads() const { return wide ? tpr : NARROW_THREADS; }
  int rows() const { return wide ? 1 : NARROW_THREADS / tpr; }     // of a block at a time
};
Cut cut_of(int N, bool bwd) {
  const int nv = N / 8;
  if (nv <= 128) {
    const int v = nv <= 4 ? 1 : nv <= 64 ? 2 : 4;
    int tpr = 4;
    while (tpr * v < nv) tpr *= 2;
    return {v, tpr, false};
  }
  const int v = bwd && nv <= WIDE_THREADS ? 1 : nv <= 2 * WIDE_THREADS ? 2 : 4;
  return {v, ((nv + v - 1) / v + 31) / 32 * 32, true};
}

int ring_bytes(const Cut& c) {
  return c.threads() * (c.v == 1 ? Ring<1>::THREAD_BYTES : c.v == 2 ? Ring<2>::THREAD_BYTES : Ring<4>::THREAD_BYTES);
}
// As many blocks as the card takes at once, by registers and shared memory.
int bwd_blocks(long long rows, int N) {
  const Cut c = cut_of(N, true);
  const int by_regs = bwd_threads_per_sm(c.v) / c.threads(), by_smem = 225 * 1024 / (ring_bytes(c) + 1280);
  const long long want = (rows + c.rows() - 1) / c.rows(), most = (long long)SMS * (by_regs < by_smem ? by_regs : by_smem);
  return (int)(want < most ? want : most);
}

template <int DT, bool W32, int V, bool WIDE>
cudaError_t go(const NormArgs& a, const Cut& c, cudaStream_t st) {
  const long long want = (a.rows + c.rows() - 1) / c.rows(), most = 1 << 22;
  return launch_early(norm_kernel<DT, W32, V, WIDE>, (unsigned)(want < most ? want : most), c.threads(), 0, st, 1, a, c.tpr);
}
template <int DT, bool W32, int V, bool WIDE>
cudaError_t go(const NormBwdArgs& a, const Cut& c, cudaStream_t st) {
  static std::atomic<uint64_t> opted{0};       // to more than 48 KB of shared memory, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!((opted.load(std::memory_order_relaxed) >> dev) & 1)) {
    const int most = (WIDE ? WIDE_THREADS : NARROW_THREADS) * Ring<V>::THREAD_BYTES;
    e = cudaFuncSetAttribute(norm_bwd_kernel<DT, W32, V, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    opted.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  return launch_early(norm_bwd_kernel<DT, W32, V, WIDE>, (unsigned)bwd_blocks(a.rows, a.N), c.threads(), ring_bytes(c), st, 1, a,
                      c.tpr);
}
template <int DT, bool W32, class A>
cudaError_t pick(const A& a, const Cut& c, cudaStream_t st) {
  if (!c.wide)
    return c.v == 1 ? go<DT, W32, 1, false>(a, c, st) : c.v == 2 ? go<DT, W32, 2, false>(a, c, st) : go<DT, W32, 4, false>(a, c, st);
  if constexpr (std::is_same<A, NormBwdArgs>::value)
    if (c.v == 1) return go<DT, W32, 1, true>(a, c, st);
  return c.v == 2 ? go<DT, W32, 2, true>(a, c, st) : go<DT, W32, 4, true>(a, c, st);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, int w32, cudaStream_t st) {
  const Cut c = cut_of(a.N, false);
  if (dtype == 0) return w32 ? pick<0, true>(a, c, st) : pick<0, false>(a, c, st);
  return w32 ? pick<1, true>(a, c, st) : pick<1, false>(a, c, st);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, int w32, cudaStream_t st) {
  const Cut c = cut_of(a.N, true);
  const cudaError_t e = dtype == 0 ? (w32 ? pick<0, true>(a, c, st) : pick<0, false>(a, c, st))
                                   : (w32 ? pick<1, true>(a, c, st) : pick<1, false>(a, c, st));
  if (e != cudaSuccess) return e;
  return launch_early(norm_dw_kernel, (unsigned)((a.N + 31) / 32), DW_WARPS * 32, 0, st, 1, (const float*)a.partial,
                      bwd_blocks(a.rows, a.N), a.N, a.dw, w32 ? 2 : dtype);
}

size_t norm_bwd_workspace_bytes(long long rows, int N) { return (size_t)bwd_blocks(rows, N) * N * 4; }

}  // namespace bsc
