// Attention over the key/value cache: the plain kernel (one block per query row, fp32 throughout).
//
// For the query at position p: s_j = scale q . K_j over j <= p, O = sum exp(s_j - LSE) V_j, in one
// pass over the keys with a running maximum and sum.  A block takes 128 keys at a time: a thread per
// key for the scores, then a thread per output element for P V.
#include "cache.cuh"

namespace bsc {
namespace {

constexpr int AT = 128;

template <int FMT, int D>
__device__ __forceinline__ float element(const uint8_t* row, const uint8_t* sc, int d) {
  const float s = scale_value(sc[d >> 5]);
  uint32_t h[4];
  if (FMT == CACHE_FP4) {
    e2m1x8_to_f16((uint32_t)row[d >> 1], h);
    const float2 f = f16x2_to_f32(h[0]);
    return s * ((d & 1) ? f.y : f.x);
  }
  e4m3x4_to_f16((uint32_t)row[d], h[0], h[1]);
  return s * f16x2_to_f32(h[0]).x;
}

template <int FMT, int D, int DT>
__global__ void __launch_bounds__(AT) cache_attn_rows_kernel(const CacheAttnArgs a) {
  constexpr int RB = row_bytes<FMT, D>(), NB = D / 32;
  __shared__ float q[D], p[AT], red[AT / 32];
  __shared__ long long slots[AT];
  const int tid = threadIdx.x;
  const int hq = blockIdx.x % a.Hq, t = (blockIdx.x / a.Hq) % a.T, b = blockIdx.x / a.Hq / a.T;
  const int h = hq / (a.Hq / a.c.Hkv);
  const int n = a.new_lens ? min(max(__ldg(a.new_lens + b), 0), a.T) : a.T;
  const long long len = max(__ldg(a.pt.seq_lens + b), 0);
  const long long cap = (long long)a.pt.max_pages * a.c.page_size;
  if (len > cap && a.dev_status) *a.dev_status = CACHE_BAD_LEN;
  const long long lim = t < n ? min(len - n + t + 1, cap) : 0;   // keys j < lim
  if (tid < D) {
    const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + b * a.qs.b + t * a.qs.t + hq * a.qs.h;
    q[tid] = act_to_f32<DT>(src[tid]).x * a.scale_log2e;
  }
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (long long j0 = 0; j0 < lim; j0 += AT) {
    __syncthreads();
    int32_t bad = 0;
    long long sl = j0 + tid < lim ? cache_slot(a.c, a.pt, b, j0 + tid, bad) : -1;
    if (bad && a.dev_status) *a.dev_status = bad;
    slots[tid] = sl;
    float s = -INFINITY;
    if (sl >= 0) {
      const long long page = sl / a.c.page_size, in_page = (long long)h * a.c.page_size + sl % a.c.page_size;
      const uint8_t* row = a.c.k + page * a.c.k_ps + in_page * RB;
      const uint8_t* sc = a.c.k_sc + page * a.c.k_sc_ps + in_page * NB;
      s = 0.f;
      for (int d = 0; d < D; ++d) s += q[d] * element<FMT, D>(row, sc, d);
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float m2 = fmaxf(m, mx);
    const float keep = m2 == -INFINITY ? 1.f : exp2f(m - m2);
    p[tid] = sl >= 0 ? exp2f(s - m2) : 0.f;
    __syncthreads();
    acc *= keep;
    l *= keep;
    m = m2;
    for (int j = 0; j < AT; ++j) {
      if (slots[j] < 0) continue;
      l += p[j];
      if (tid < D) {
        const long long page = slots[j] / a.c.page_size;
        const long long in_page = (long long)h * a.c.page_size + slots[j] % a.c.page_size;
        acc += p[j] * element<FMT, D>(a.c.v + page * a.c.v_ps + in_page * RB, a.c.v_sc + page * a.c.v_sc_ps + in_page * NB,
                                      tid);
      }
    }
  }
  const bool none = m == -INFINITY && l == 0.f;
  if (tid < D) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(a.o) + b * a.os.b + t * a.os.t + hq * a.os.h;
    dst[tid] = (uint16_t)f32_to_act<DT>(none ? 0.f : acc / l, 0.f);
  }
  if (tid == 0 && a.lse) a.lse[((long long)b * a.Hq + hq) * a.T + t] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

size_t cache_attn_workspace_bytes(int, int, int, int, int) { return 0; }

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int format, int D, int dtype, cudaStream_t st) {
  using Kernel = void (*)(CacheAttnArgs);
  static const Kernel k[8] = {cache_attn_rows_kernel<0, 64, 0>,  cache_attn_rows_kernel<0, 64, 1>,
                              cache_attn_rows_kernel<0, 128, 0>, cache_attn_rows_kernel<0, 128, 1>,
                              cache_attn_rows_kernel<1, 64, 0>,  cache_attn_rows_kernel<1, 64, 1>,
                              cache_attn_rows_kernel<1, 128, 0>, cache_attn_rows_kernel<1, 128, 1>};
  k[format * 4 + (D == 128) * 2 + dtype]<<<(unsigned)(a.B * a.T * a.Hq), AT, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace bsc
