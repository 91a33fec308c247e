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
#include "cache.cuh"

namespace bsc {
namespace {

constexpr int SMS = 152;
constexpr int NARROW_THREADS = 128, WIDE_THREADS = 512;   // most threads of a block

template <int DT>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = act_to_f32<DT>(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(f32_to_act<DT>(f[0], f[1]), f32_to_act<DT>(f[2], f[3]), f32_to_act<DT>(f[4], f[5]),
                    f32_to_act<DT>(f[6], f[7]));
}

// Eight weights as they are held: one or two 16-byte pieces.
template <int DT, bool W32>
struct Weights {
  uint4 v[W32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* w, int at) {
    if (W32) {
      v[0] = __ldca(reinterpret_cast<const uint4*>(w) + 2 * at);
      v[W32 ? 1 : 0] = __ldca(reinterpret_cast<const uint4*>(w) + 2 * at + 1);
    } else {
      v[0] = __ldca(reinterpret_cast<const uint4*>(w) + at);
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if (W32) {
      const uint4 a = v[0], b = v[W32 ? 1 : 0];
      const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
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
__global__ void __launch_bounds__(WIDE ? WIDE_THREADS : NARROW_THREADS) norm_kernel(const NormArgs a, int tpr) {
  __shared__ float part[2][32];
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const int rpb = WIDE ? 1 : NARROW_THREADS / tpr, t = WIDE ? threadIdx.x : threadIdx.x % tpr;
  const int nv = a.N / 8;
  const long long step = (long long)gridDim.x * rpb;
  long long row = (long long)blockIdx.x * rpb + (WIDE ? 0 : threadIdx.x / tpr);
  Weights<DT, W32> w[V];
  uint4 x[V], r[V];
  auto load = [&](long long at) {
    const uint4* const xp = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) + row_at(a.xs, at, a.inner));
    const uint4* const rp = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.r) + row_at(a.rs, at, a.inner));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = v * tpr + t;
      x[v] = make_uint4(0, 0, 0, 0);
      if (j < nv && at < a.rows) {
        x[v] = __ldcs(xp + j);
        if (a.r) r[v] = __ldcs(rp + j);
      }
    }
  };
  load(row);
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (v * tpr + t < nv) w[v].load(a.w, v * tpr + t);
  const uint32_t up = ceil_carry<CACHE_FP8>(a.rule);
  const float inv_n = 1.f / (float)a.N;
  int turn = 0;
  // rows of one warp end together: the loop goes by the block's first row
  for (long long first = (long long)blockIdx.x * rpb; first < a.rows; first += step, row += step, turn ^= 1) {
    const bool live = row < a.rows;
    uint4 s[V];
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[8];
      unpack8<DT>(x[v], f);
      s[v] = x[v];
      const int j = v * tpr + t;
      if (a.r && j < nv && live) {
        float g[8];
        unpack8<DT>(r[v], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += g[i];
        s[v] = pack8<DT>(f);
        unpack8<DT>(s[v], f);
        if (a.s)
          __stcs(reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.s) + row_at(a.ss, row, a.inner)) + j, s[v]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += f[i] * f[i];
    }
    load(row + step);
    const float rstd = rsqrtf(row_sum<WIDE>(sum, tpr, part[turn]) * inv_n + a.eps);
    if (a.rstd && t == 0 && live) a.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = v * tpr + t;
      const bool mine = j < nv && live;
      float f[8], g[8];
      unpack8<DT>(s[v], f);
      w[v].get(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * rstd * g[i];
      if (a.y && mine)
        __stcs(reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.y) + row_at(a.ys, row, a.inner)) + j, pack8<DT>(f));
      if (a.y8) {                    // 32 elements are four neighbouring lanes; NaN and Inf are above every finite pattern
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(f[i]) & 0x7FFFFFFFu);
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
        float inv;
        const uint32_t sb = block_scale<CACHE_FP8>(__uint_as_float(am), up, inv);
        if (mine) {
          __stcs(reinterpret_cast<uint2*>(a.y8 + row * a.N) + j, quant8_e4m3(f, inv, sb));
          if ((t & 3) == 0) a.ysc[row * (a.N / 32) + (j >> 2)] = (uint8_t)sb;
        }
      }
    }
  }
}

// The gradients of a block's rows; dw's share of the block goes to partial[block][N].
template <int DT, bool W32, int V, bool WIDE>
__global__ void __launch_bounds__(WIDE ? WIDE_THREADS : NARROW_THREADS) norm_bwd_kernel(const NormBwdArgs a, int tpr) {
  __shared__ float part[2][32];
  __shared__ float group[WIDE ? 1 : NARROW_THREADS * 8];
  wait_for_last_kernel();
  if (gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  const int rpb = WIDE ? 1 : NARROW_THREADS / tpr, t = WIDE ? threadIdx.x : threadIdx.x % tpr;
  const int nv = a.N / 8;
  const long long step = (long long)gridDim.x * rpb;
  long long row = (long long)blockIdx.x * rpb + (WIDE ? 0 : threadIdx.x / tpr);
  Weights<DT, W32> w[V];
  constexpr bool AHEAD = V < 4;                  // the next row's loads in flight: 4 vectors of three tensors leave no room
  uint4 dy[V], s[V], ds[V];
  float rstd = 0.f, acc[V][8];
  auto at_row = [&](const void* p, const NormRows& rs, long long at) {
    return reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + row_at(rs, at, a.inner));
  };
  auto load = [&](long long at) {
    const uint4 *const dp = at_row(a.dy, a.dys, at), *const sp = at_row(a.s, a.ss, at), *const rp = at_row(a.ds, a.dss, at);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = v * tpr + t;
      dy[v] = s[v] = ds[v] = make_uint4(0, 0, 0, 0);
      if (j < nv && at < a.rows) {
        dy[v] = __ldcs(dp + j);
        s[v] = __ldcs(sp + j);
        if (a.ds) ds[v] = __ldcs(rp + j);
      }
    }
    rstd = at < a.rows ? __ldca(a.rstd + at) : 0.f;
  };
  if (AHEAD) load(row);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (v * tpr + t < nv) w[v].load(a.w, v * tpr + t);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v][i] = 0.f;
  }
  const float inv_n = 1.f / (float)a.N;
  int turn = 0;
  for (long long first = (long long)blockIdx.x * rpb; first < a.rows; first += step, row += step, turn ^= 1) {
    const bool live = row < a.rows;
    if (!AHEAD) load(row);
    const float rs = rstd;
    uint4 dy0[V], s0[V], ds0[V];
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float d[8], x[8], g[8];
      dy0[v] = dy[v];
      s0[v] = s[v];
      ds0[v] = ds[v];
      unpack8<DT>(dy0[v], d);
      unpack8<DT>(s0[v], x);
      w[v].get(g);
      if (v * tpr + t < nv)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = d[i] * (x[i] * rs);
          acc[v][i] += p;
          sum += p * g[i];
        }
    }
    if (AHEAD) load(row + step);
    const float c = row_sum<WIDE>(sum, tpr, part[turn]) * inv_n;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = v * tpr + t;
      if (j >= nv || !live) continue;
      float d[8], x[8], g[8], e[8];
      unpack8<DT>(dy0[v], d);
      unpack8<DT>(s0[v], x);
      unpack8<DT>(ds0[v], e);
      w[v].get(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = rs * (d[i] * g[i] - x[i] * rs * c) + e[i];
      __stcs(reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.dx) + row_at(a.dxs, row, a.inner)) + j, pack8<DT>(d));
    }
  }
  float* const out = a.partial + (long long)blockIdx.x * a.N;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (!WIDE) {                     // the block's rows' shares of these columns, in their order
#pragma unroll
      for (int i = 0; i < 8; ++i) group[threadIdx.x * 8 + i] = acc[v][i];
      __syncthreads();
      if (threadIdx.x < tpr)
        for (int k = 1; k < rpb; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[v][i] += group[(k * tpr + t) * 8 + i];
      __syncthreads();
    }
    const int j = v * tpr + t;
    if (j < nv && (WIDE || threadIdx.x < tpr)) {
      float4* const dst = reinterpret_cast<float4*>(out) + 2 * j;
      dst[0] = make_float4(acc[v][0], acc[v][1], acc[v][2], acc[v][3]);
      dst[1] = make_float4(acc[v][4], acc[v][5], acc[v][6], acc[v][7]);
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
};
Cut cut_of(int N) {
  const int nv = N / 8;
  if (nv <= 128) {
    const int v = nv <= 32 ? 1 : nv <= 64 ? 2 : 4;
    int tpr = 4;
    while (tpr * v < nv) tpr *= 2;
    return {v, tpr, false};
  }
  const int v = nv <= WIDE_THREADS ? 1 : nv <= 2 * WIDE_THREADS ? 2 : 4;
  return {v, ((nv + v - 1) / v + 31) / 32 * 32, true};
}

int bwd_blocks(long long rows, int N) {
  const Cut c = cut_of(N);
  const int rpb = c.wide ? 1 : NARROW_THREADS / c.tpr;
  const long long want = (rows + rpb - 1) / rpb, most = (long long)SMS * (c.wide ? max(1, 1024 / c.tpr) : 8);
  return (int)(want < most ? want : most);
}

template <int DT, bool W32, int V, bool WIDE>
cudaError_t go(const NormArgs& a, const Cut& c, cudaStream_t st) {
  const int rpb = WIDE ? 1 : NARROW_THREADS / c.tpr, threads = WIDE ? c.tpr : NARROW_THREADS;
  const long long want = (a.rows + rpb - 1) / rpb, most = (long long)SMS * (2048 / threads);
  return launch_early(norm_kernel<DT, W32, V, WIDE>, (unsigned)(want < most ? want : most), threads, 0, st, 1, a, c.tpr);
}
template <int DT, bool W32, int V, bool WIDE>
cudaError_t go(const NormBwdArgs& a, const Cut& c, cudaStream_t st) {
  return launch_early(norm_bwd_kernel<DT, W32, V, WIDE>, (unsigned)bwd_blocks(a.rows, a.N), WIDE ? c.tpr : NARROW_THREADS, 0,
                      st, 1, a, c.tpr);
}
template <int DT, bool W32, class A>
cudaError_t pick(const A& a, const Cut& c, cudaStream_t st) {
  if (!c.wide)
    return c.v == 1 ? go<DT, W32, 1, false>(a, c, st) : c.v == 2 ? go<DT, W32, 2, false>(a, c, st) : go<DT, W32, 4, false>(a, c, st);
  return c.v == 1 ? go<DT, W32, 1, true>(a, c, st) : c.v == 2 ? go<DT, W32, 2, true>(a, c, st) : go<DT, W32, 4, true>(a, c, st);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, int w32, cudaStream_t st) {
  const Cut c = cut_of(a.N);
  if (dtype == 0) return w32 ? pick<0, true>(a, c, st) : pick<0, false>(a, c, st);
  return w32 ? pick<1, true>(a, c, st) : pick<1, false>(a, c, st);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, int w32, cudaStream_t st) {
  const Cut c = cut_of(a.N);
  const cudaError_t e = dtype == 0 ? (w32 ? pick<0, true>(a, c, st) : pick<0, false>(a, c, st))
                                   : (w32 ? pick<1, true>(a, c, st) : pick<1, false>(a, c, st));
  if (e != cudaSuccess) return e;
  return launch_early(norm_dw_kernel, (unsigned)((a.N + 31) / 32), DW_WARPS * 32, 0, st, 1, (const float*)a.partial,
                      bwd_blocks(a.rows, a.N), a.N, a.dw, w32 ? 2 : dtype);
}

size_t norm_bwd_workspace_bytes(long long rows, int N) { return (size_t)bwd_blocks(rows, N) * N * 4; }

}  // namespace bsc
