// C-ABI entry points: argument checks, tensor-map creation, launches.  See include/bsc.h.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "../../include/bsc.h"
#include "bsc_internal.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Device capability check, cached per device ordinal.
bsc_status check_device() {
  static std::mutex mu;
  static int cached[64];   // 0 unknown, 1 ok, 2 bad
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSC_ERR_CUDA;
  if (dev < 0 || dev >= 64) return BSC_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(mu);
  if (cached[dev] == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return BSC_ERR_CUDA;
    cached[dev] = (major == 10 && minor == 3) ? 1 : 2;
  }
  return cached[dev] == 1 ? BSC_OK : BSC_ERR_UNSUPPORTED;
}

// Common shape checks.  Returns BSC_OK with *empty set when there is nothing to do.
bsc_status check_shape(int B, int S, int H, int D, int layout, bool* empty) {
  *empty = false;
  if (B < 0 || S < 0 || H < 0 || D < 0) return BSC_ERR_SHAPE;
  if (layout != BSC_BSHD && layout != BSC_SBHD) return BSC_ERR_SHAPE;
  if (B == 0 || S == 0 || H == 0) {
    *empty = true;
    return BSC_OK;
  }
  if (D != 128 || S % 32 != 0) return BSC_ERR_UNSUPPORTED;
  // every index the kernels form fits in 64 bits; the grids (one CTA per 64 tokens of a (b, h) plane
  // at most) must fit their limits
  if ((long long)B * H * ((S + 63) / 64) >= (1LL << 31)) return BSC_ERR_UNSUPPORTED;
  return BSC_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// E4M3 [.., S, .., H, 128] operand as a 4-D map {D, H, S, B} with a 128-token x 128-byte box.
bool encode_tokens_map(CUtensorMap* m, const void* base, int B, int S, int H, int layout, bool swizzle) {
  auto enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[4] = {128, (cuuint64_t)H, (cuuint64_t)S, (cuuint64_t)B};
  const cuuint64_t sH = 128;
  const cuuint64_t sS = layout == BSC_BSHD ? (cuuint64_t)H * 128 : (cuuint64_t)B * H * 128;
  const cuuint64_t sB = layout == BSC_BSHD ? (cuuint64_t)S * H * 128 : (cuuint64_t)H * 128;
  const cuuint64_t strides[3] = {sH, sS, sB};
  const cuuint32_t box[4] = {128, 1, 128, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// BF16 [.., S, .., H, 128] tensor as a 4-D map {D, H, S, B} with a 128-token x 64-element box
// (128 bytes, the swizzle span): two boxes cover a row's 128 elements.
bool encode_bf16_tokens_map(CUtensorMap* m, const void* base, int B, int S, int H, int layout) {
  auto enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[4] = {128, (cuuint64_t)H, (cuuint64_t)S, (cuuint64_t)B};
  const cuuint64_t sH = 256;
  const cuuint64_t sS = layout == BSC_BSHD ? (cuuint64_t)H * 256 : (cuuint64_t)B * H * 256;
  const cuuint64_t sB = layout == BSC_BSHD ? (cuuint64_t)S * H * 256 : (cuuint64_t)H * 256;
  const cuuint64_t strides[3] = {sH, sS, sB};
  const cuuint32_t box[4] = {64, 1, 128, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// BF16 planes [planes][rows][128] (the backward's workspace) as a 3-D map with a 64-element x
// 128-row box and the 128-byte swizzle: two boxes cover a tile's 128 columns.
bool encode_bf16_planar_map(CUtensorMap* m, void* base, long long planes, int rows) {
  auto enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[3] = {128, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {256, (cuuint64_t)rows * 256};
  const cuuint32_t box[3] = {64, 128, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Transposed V bytes [rows = B*H*D][S] as a 2-D map with a 128-key x 128-row box.
bool encode_vt_map(CUtensorMap* m, const void* base, long long rows, int S) {
  auto enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)S, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)S};
  const cuuint32_t box[2] = {128, 128};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bsc_status from_cuda(cudaError_t e) { return e == cudaSuccess ? BSC_OK : BSC_ERR_CUDA; }

bsc_status quant_v_common(const void* v, int B, int S, int H, int D, bsc_layout layout, uint8_t* vt, uint8_t* vsc,
                          uint8_t* vtn, uint8_t* vtn_sc, bsc_stream_t stream, bool want_col, bool want_tn,
                          int rule = 0) {
  bool empty;
  bsc_status s = check_shape(B, S, H, D, layout, &empty);
  if (s != BSC_OK || empty) return s;
  if (!v || (want_col && (!vt || !vsc)) || (want_tn && (!vtn || !vtn_sc))) return BSC_ERR_NULL;
  if (!aligned16(v) || (want_col && (!aligned16(vt) || !aligned16(vsc))) ||
      (want_tn && (!aligned16(vtn) || !aligned16(vtn_sc))))
    return BSC_ERR_ALIGN;
  if ((s = check_device()) != BSC_OK) return s;
  return from_cuda(bsc::launch_quant_v(v, want_col ? vt : nullptr, want_col ? vsc : nullptr,
                                       want_tn ? vtn : nullptr, want_tn ? vtn_sc : nullptr, B, S, H, layout,
                                       reinterpret_cast<cudaStream_t>(stream), rule));
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether a product of sizes (each at least 1 and below 2^31) reaches 2^31.
bool reaches_2_31(std::initializer_list<long long> sizes) {
  long long product = 1;
  for (const long long s : sizes)
    if ((product *= s) >= (1LL << 31)) return true;
  return false;
}

// What the attention's grids and row numbers cannot hold: the rows of all tiles (the smallest of 8, 16 and 32 rows that takes
// a KV head's, else 32), or the chunks of 128 tokens of all tiles.  max_tokens 0: rows alone.
bool cache_attn_too_large(int B, int T, int Hq, int Hkv, long long max_tokens) {
  const long long rows = (long long)T * (Hq / Hkv);
  const int tile = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
  if (rows >= (1LL << 31)) return true;
  const long long tiles = (rows + tile - 1) / tile, chunks = (max_tokens + 127) / 128;
  return reaches_2_31({B, Hkv, tiles, tile}) || (chunks > 0 && reaches_2_31({B, Hkv, tiles, chunks}));
}

// The checks that the three cache calls share.  *empty: a problem without sequences, tokens or heads.
bsc_status check_cache(const bsc_mx_cache& c, int B, int T, int H, int dtype, long long table_stride, int max_pages,
                       bool* empty) {
  *empty = false;
  if (B < 0 || T < 0 || H < 0 || c.Hkv < 0 || c.D < 0 || c.num_pages < 0 || c.page_size < 0 || max_pages < 0)
    return BSC_ERR_SHAPE;
  if (c.format != BSC_CACHE_MXFP8 && c.format != BSC_CACHE_MXFP4) return BSC_ERR_UNSUPPORTED;
  if (dtype != BSC_BF16 && dtype != BSC_FP16) return BSC_ERR_UNSUPPORTED;
  if (B == 0 || T == 0 || H == 0) {
    *empty = true;
    return BSC_OK;
  }
  if (c.Hkv == 0 || c.num_pages == 0 || c.page_size == 0) return BSC_ERR_SHAPE;
  if ((c.D != 64 && c.D != 128) || c.page_size % 16 != 0) return BSC_ERR_UNSUPPORTED;
  if (B > 1 && table_stride < max_pages) return BSC_ERR_SHAPE;
  // positions are 32-bit, with room above the last for a tile's end and the tiles after it
  if ((long long)max_pages * c.page_size > BSC_CACHE_MAX_TOKENS) return BSC_ERR_UNSUPPORTED;
  // the attention addresses a page in 32-bit units of 16 bytes
  if ((long long)c.Hkv * c.page_size >= (1LL << 31) / c.D) return BSC_ERR_UNSUPPORTED;
  if (!c.k || !c.k_sc || !c.v || !c.v_sc) return BSC_ERR_NULL;
  if (!aligned16(c.k) || !aligned16(c.k_sc) || !aligned16(c.v) || !aligned16(c.v_sc)) return BSC_ERR_ALIGN;
  if (c.num_pages > 1) {
    const long long slots = (long long)c.Hkv * c.page_size;
    const long long data = slots * (c.format == BSC_CACHE_MXFP4 ? c.D / 2 : c.D), scales = slots * (c.D / 32);
    for (const long long s : {c.k_page_stride, c.k_sc_page_stride, c.v_page_stride, c.v_sc_page_stride}) {
      if (s % 16 != 0) return BSC_ERR_ALIGN;
      if (s >= (1LL << 36)) return BSC_ERR_UNSUPPORTED;
    }
    if (c.k_page_stride < data || c.v_page_stride < data || c.k_sc_page_stride < scales ||
        c.v_sc_page_stride < scales)
      return BSC_ERR_SHAPE;
  }
  return BSC_OK;
}

// Strides of an activation: 16-byte rows, and no two output rows in one place.
bsc_status check_strides(long long sb, long long st, long long sh, int B, int T, int H, bool output) {
  if ((B > 1 && sb % 8 != 0) || (T > 1 && st % 8 != 0) || (H > 1 && sh % 8 != 0)) return BSC_ERR_ALIGN;
  if (output && ((B > 1 && sb == 0) || (T > 1 && st == 0) || (H > 1 && sh == 0))) return BSC_ERR_SHAPE;
  return BSC_OK;
}

bsc::CachePools cache_pools(const bsc_mx_cache& c) {
  bsc::CachePools p{};
  p.k = c.k;
  p.k_sc = c.k_sc;
  p.v = c.v;
  p.v_sc = c.v_sc;
  p.k_ps = c.k_page_stride;
  p.k_sc_ps = c.k_sc_page_stride;
  p.v_ps = c.v_page_stride;
  p.v_sc_ps = c.v_sc_page_stride;
  p.num_pages = c.num_pages;
  p.page_size = c.page_size;
  p.Hkv = c.Hkv;
  return p;
}

}  // namespace

extern "C" {

int bsc_abi_version(void) { return 3; }

const char* bsc_status_string(bsc_status s) {
  switch (s) {
    case BSC_OK: return "BSC_OK";
    case BSC_ERR_NULL: return "BSC_ERR_NULL: a required pointer is NULL";
    case BSC_ERR_SHAPE: return "BSC_ERR_SHAPE: invalid sizes, head grouping or layout";
    case BSC_ERR_ALIGN: return "BSC_ERR_ALIGN: a pointer is not 16-byte aligned";
    case BSC_ERR_UNSUPPORTED: return "BSC_ERR_UNSUPPORTED: unsupported size, option or device";
    case BSC_ERR_CUDA: return "BSC_ERR_CUDA: a CUDA call failed";
    case BSC_ERR_DEVICE_TIMEOUT: return "BSC_ERR_DEVICE_TIMEOUT: a device-side wait gave up";
    case BSC_ERR_DEVICE_PAGE: return "BSC_ERR_DEVICE_PAGE: a page id or a length that the page table does not have";
  }
  return "unknown bsc_status";
}

bsc_status mxfp8_quantize_qk_rowwise(const void* x, int B, int S, int H, int D, bsc_layout layout, uint8_t* xq,
                                     uint8_t* xsc, bsc_stream_t stream) {
  bool empty;
  bsc_status s = check_shape(B, S, H, D, layout, &empty);
  if (s != BSC_OK || empty) return s;
  if (!x || !xq || !xsc) return BSC_ERR_NULL;
  if (!aligned16(x) || !aligned16(xq) || !aligned16(xsc)) return BSC_ERR_ALIGN;
  if ((s = check_device()) != BSC_OK) return s;
  return from_cuda(bsc::launch_quant_rowwise(x, xq, xsc, B, S, H, layout, reinterpret_cast<cudaStream_t>(stream)));
}

bsc_status mxfp8_quantize(const bsc_quant_params* p, bsc_stream_t stream) {
  if (!p) return BSC_ERR_NULL;
  if (p->rule != BSC_SCALE_FLOOR && p->rule != BSC_SCALE_CEIL) return BSC_ERR_UNSUPPORTED;
  const bsc_layout layout = (bsc_layout)p->layout;
  switch (p->kind) {
    case BSC_QUANT_ROWWISE: {
      bool empty;
      bsc_status s = check_shape(p->B, p->S, p->H, p->D, p->layout, &empty);
      if (s != BSC_OK || empty) return s;
      if (!p->x || !p->e4m3 || !p->sc) return BSC_ERR_NULL;
      if (!aligned16(p->x) || !aligned16(p->e4m3) || !aligned16(p->sc)) return BSC_ERR_ALIGN;
      if ((s = check_device()) != BSC_OK) return s;
      return from_cuda(bsc::launch_quant_rowwise(p->x, p->e4m3, p->sc, p->B, p->S, p->H, p->layout,
                                                 reinterpret_cast<cudaStream_t>(stream), p->rule));
    }
    case BSC_QUANT_V_COLWISE:
      return quant_v_common(p->x, p->B, p->S, p->H, p->D, layout, p->e4m3, p->sc, nullptr, nullptr, stream, true,
                            false, p->rule);
    case BSC_QUANT_V_TOKEN_NORM:
      return quant_v_common(p->x, p->B, p->S, p->H, p->D, layout, nullptr, nullptr, p->vtn_e4m3, p->vtn_sc, stream,
                            false, true, p->rule);
    case BSC_QUANT_V_FUSED:
      return quant_v_common(p->x, p->B, p->S, p->H, p->D, layout, p->e4m3, p->sc, p->vtn_e4m3, p->vtn_sc, stream,
                            true, true, p->rule);
    default:
      return BSC_ERR_UNSUPPORTED;
  }
}

bsc_status mxfp8_quantize_v_colwise(const void* v, int B, int S, int H, int D, bsc_layout layout, uint8_t* vt,
                                    uint8_t* vsc, bsc_stream_t stream) {
  return quant_v_common(v, B, S, H, D, layout, vt, vsc, nullptr, nullptr, stream, true, false);
}

bsc_status v_token_normalize(const void* v, int B, int S, int H, int D, bsc_layout layout, uint8_t* vtn,
                             uint8_t* vtn_sc, bsc_stream_t stream) {
  return quant_v_common(v, B, S, H, D, layout, nullptr, nullptr, vtn, vtn_sc, stream, false, true);
}

bsc_status mxfp8_quantize_v_fused(const void* v, int B, int S, int H, int D, bsc_layout layout, uint8_t* vt,
                                  uint8_t* vsc, uint8_t* vtn, uint8_t* vtn_sc, bsc_stream_t stream) {
  return quant_v_common(v, B, S, H, D, layout, vt, vsc, vtn, vtn_sc, stream, true, true);
}

bsc_status mxfp8_quantize_qkv(const bsc_qkv_quant_params* p, bsc_stream_t stream) {
  if (!p) return BSC_ERR_NULL;
  if (p->Hq < 0 || p->Hkv < 0) return BSC_ERR_SHAPE;
  if (p->rule != BSC_SCALE_FLOOR && p->rule != BSC_SCALE_CEIL) return BSC_ERR_UNSUPPORTED;
  bool empty;
  bsc_status s = check_shape(p->B, p->S, p->Hq, p->D, p->layout, &empty);
  if (s != BSC_OK) return s;
  if (!empty && p->Hkv == 0) return BSC_ERR_SHAPE;
  if (empty) return BSC_OK;
  if (p->Hq % p->Hkv != 0) return BSC_ERR_SHAPE;
  // one launch: V tiles plus Q's and K's 64-token chunks
  if ((long long)p->B * (p->Hq + 2LL * p->Hkv) * ((p->S + 63) / 64) >= (1LL << 31)) return BSC_ERR_UNSUPPORTED;
  const bool col = p->v_e4m3_t != nullptr || p->v_sc != nullptr;
  const bool tn = p->vtn_e4m3 != nullptr || p->vtn_sc != nullptr;
  if (!p->q || !p->k || !p->v || !p->q_e4m3 || !p->q_sc || !p->k_e4m3 || !p->k_sc) return BSC_ERR_NULL;
  if ((col && (!p->v_e4m3_t || !p->v_sc)) || (tn && (!p->vtn_e4m3 || !p->vtn_sc)) || (!col && !tn))
    return BSC_ERR_NULL;
  for (const void* ptr : {p->q, p->k, p->v, (const void*)p->q_e4m3, (const void*)p->q_sc, (const void*)p->k_e4m3,
                          (const void*)p->k_sc, (const void*)p->v_e4m3_t, (const void*)p->v_sc,
                          (const void*)p->vtn_e4m3, (const void*)p->vtn_sc})
    if (!aligned16(ptr)) return BSC_ERR_ALIGN;
  if ((s = check_device()) != BSC_OK) return s;
  bsc::QkvQuantArgs a{};
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.B = p->B;
  a.S = p->S;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.layout = p->layout;
  a.rule = p->rule;
  a.q8 = p->q_e4m3;
  a.q_sc = p->q_sc;
  a.k8 = p->k_e4m3;
  a.k_sc = p->k_sc;
  a.vt = p->v_e4m3_t;
  a.vsc = p->v_sc;
  a.vtn = p->vtn_e4m3;
  a.vtn_sc = p->vtn_sc;
  return from_cuda(bsc::launch_quant_qkv(a, reinterpret_cast<cudaStream_t>(stream)));
}

bsc_status mxfp8_causal_attn_fwd(const bsc_attn_fwd_params* p, bsc_stream_t stream) {
  if (!p) return BSC_ERR_NULL;
  if (p->Hq < 0 || p->Hkv < 0) return BSC_ERR_SHAPE;
  bool empty;
  bsc_status s = check_shape(p->B, p->S, p->Hq, p->D, p->layout, &empty);
  if (s != BSC_OK) return s;
  if (!empty && p->Hkv == 0) return BSC_ERR_SHAPE;
  if (empty) return BSC_OK;
  if (p->Hq % p->Hkv != 0) return BSC_ERR_SHAPE;
  if (p->p_terms != 1 && p->p_terms != 2) return BSC_ERR_UNSUPPORTED;
  if (p->leaky != 0 && p->leaky != 1) return BSC_ERR_UNSUPPORTED;
  // the kernel takes row maxima of the raw scores before scaling: a positive, finite scale only
  if (!(std::isfinite(p->softmax_scale) && p->softmax_scale > 0.f)) return BSC_ERR_UNSUPPORTED;
  const bool own = p->leaky == 0;
  if (!p->q || !p->q_sc || !p->k || !p->k_sc || !p->v_t || !p->v_sc || !p->lse) return BSC_ERR_NULL;
  if (!p->o && !p->o_e4m3) return BSC_ERR_NULL;
  if (p->o_e4m3 && !p->o_sc) return BSC_ERR_NULL;
  if (own && (!p->vtn || !p->vtn_sc)) return BSC_ERR_NULL;
  const void* ptrs[] = {p->q, p->q_sc, p->k, p->k_sc, p->v_t, p->v_sc, p->o, p->lse, p->dev_status,
                        p->o_e4m3, p->o_sc};
  for (const void* q : ptrs)
    if (!aligned16(q)) return BSC_ERR_ALIGN;
  if (own && (!aligned16(p->vtn) || !aligned16(p->vtn_sc))) return BSC_ERR_ALIGN;
  if ((s = check_device()) != BSC_OK) return s;

  bsc::AttnArgs a;
  std::memset(&a, 0, sizeof(a));
  if (!encode_tokens_map(&a.tm_q, p->q, p->B, p->S, p->Hq, p->layout, true) ||
      !encode_tokens_map(&a.tm_k, p->k, p->B, p->S, p->Hkv, p->layout, true) ||
      !encode_vt_map(&a.tm_v, p->v_t, (long long)p->B * p->Hkv * 128, p->S))
    return BSC_ERR_CUDA;
  a.q_sc = p->q_sc;
  a.k_sc = p->k_sc;
  a.v_sc = p->v_sc;
  a.vtn = own ? p->vtn : nullptr;
  a.vtn_sc = own ? p->vtn_sc : nullptr;
  a.o = p->o;
  a.o8 = p->o_e4m3;
  a.o_sc = p->o_sc;
  a.lse = p->lse;
  a.dev_status = p->dev_status;
  a.limit_ns = (unsigned long long)(p->wait_timeout_ms ? p->wait_timeout_ms : 2000u) * 1000000ull;
  a.B = p->B;
  a.S = p->S;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.layout = p->layout;
  a.scale_log2e = (float)((double)p->softmax_scale * 1.4426950408889634);
  a.p_terms = p->p_terms;
  a.leaky = p->leaky;
  a.inject_stall = p->debug_stall ? 1 : 0;
  return from_cuda(bsc::launch_attn_fwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t bf16_attn_bwd_workspace_bytes(int B, int S, int Hq, int Hkv) {
  if (B <= 0 || S <= 0 || Hq <= 0 || Hkv <= 0) return 0;
  return bsc::bwd_workspace_bytes(B, S, Hq, Hkv);
}

bsc_status bf16_attn_bwd(const bsc_attn_bwd_params* p, bsc_stream_t stream) {
  if (!p) return BSC_ERR_NULL;
  if (p->Hq < 0 || p->Hkv < 0) return BSC_ERR_SHAPE;
  bool empty;
  bsc_status s = check_shape(p->B, p->S, p->Hq, p->D, p->layout, &empty);
  if (s != BSC_OK) return s;
  if (!empty && p->Hkv == 0) return BSC_ERR_SHAPE;
  if (empty) return BSC_OK;
  if (p->Hq % p->Hkv != 0) return BSC_ERR_SHAPE;
  if (!(std::isfinite(p->softmax_scale) && p->softmax_scale > 0.f)) return BSC_ERR_UNSUPPORTED;
  if (!p->q || !p->q_sc || !p->k || !p->k_sc || !p->vtn || !p->vtn_sc || !p->o || !p->lse || !p->d_o || !p->dq ||
      !p->dk || !p->dv || !p->workspace)
    return BSC_ERR_NULL;
  const void* ptrs[] = {p->q,  p->q_sc, p->k,  p->k_sc, p->vtn,       p->vtn_sc,    p->o,
                        p->lse, p->d_o, p->dq, p->dk,   p->dv, p->workspace, p->dev_status};
  for (const void* q : ptrs)
    if (!aligned16(q)) return BSC_ERR_ALIGN;
  if (p->workspace_bytes < bf16_attn_bwd_workspace_bytes(p->B, p->S, p->Hq, p->Hkv)) return BSC_ERR_SHAPE;
  if ((s = check_device()) != BSC_OK) return s;

  bsc::BwdArgs a;
  std::memset(&a, 0, sizeof(a));
  const int Sp = (p->S + 127) / 128 * 128;
  const long long rq = (long long)p->B * p->Hq * Sp, rk = (long long)p->B * p->Hkv * Sp;
  uint8_t* ws = reinterpret_cast<uint8_t*>(p->workspace);
  a.ws = p->workspace;
  a.qh = reinterpret_cast<uint16_t*>(ws + 8 * rq);
  a.kh = a.qh + rq * 128;
  a.vh = a.kh + rk * 128;
  if (!encode_bf16_planar_map(&a.tm_qh, a.qh, (long long)p->B * p->Hq, Sp) ||
      !encode_bf16_planar_map(&a.tm_kh, a.kh, (long long)p->B * p->Hkv, Sp) ||
      !encode_bf16_planar_map(&a.tm_vh, a.vh, (long long)p->B * p->Hkv, Sp) ||
      !encode_bf16_tokens_map(&a.tm_do, p->d_o, p->B, p->S, p->Hq, p->layout))
    return BSC_ERR_CUDA;
  a.q8 = p->q;
  a.k8 = p->k;
  a.vtn = p->vtn;
  a.q_sc = p->q_sc;
  a.k_sc = p->k_sc;
  a.vtn_sc = p->vtn_sc;
  a.o = p->o;
  a.dO = p->d_o;
  a.lse = p->lse;
  a.dq = p->dq;
  a.dk = p->dk;
  a.dv = p->dv;
  a.Sp = Sp;
  a.dev_status = p->dev_status;
  a.limit_ns = (unsigned long long)(p->wait_timeout_ms ? p->wait_timeout_ms : 2000u) * 1000000ull;
  a.B = p->B;
  a.S = p->S;
  a.Hq = p->Hq;
  a.Hkv = p->Hkv;
  a.layout = p->layout;
  a.scale = p->softmax_scale;
  a.scale_log2e = (float)((double)p->softmax_scale * 1.4426950408889634);
  return from_cuda(bsc::launch_attn_bwd(a, reinterpret_cast<cudaStream_t>(stream)));
}

bsc_status mx_cache_write(const bsc_mx_cache_write_params* p, bsc_stream_t stream) {
  if (!p) return BSC_ERR_NULL;
  if (p->rule != BSC_SCALE_FLOOR && p->rule != BSC_SCALE_CEIL) return BSC_ERR_UNSUPPORTED;
  bool empty;
  bsc_status s = check_cache(p->cache, p->B, p->T, p->cache.Hkv, p->dtype, p->table_stride, p->max_pages, &empty);
  if (s != BSC_OK || empty) return s;
  if (reaches_2_31({2, p->B, (p->T + 15LL) / 16, p->cache.Hkv})) return BSC_ERR_UNSUPPORTED;   // warps
  if (!p->k || !p->v || !p->seq_lens || (p->max_pages > 0 && !p->page_table)) return BSC_ERR_NULL;
  if (!aligned16(p->k) || !aligned16(p->v) || !aligned4(p->page_table) || !aligned4(p->seq_lens) ||
      !aligned4(p->new_lens) || !aligned4(p->dev_status))
    return BSC_ERR_ALIGN;
  const int H = p->cache.Hkv;
  if ((s = check_strides(p->k_stride_b, p->k_stride_t, p->k_stride_h, p->B, p->T, H, false)) != BSC_OK) return s;
  if ((s = check_strides(p->v_stride_b, p->v_stride_t, p->v_stride_h, p->B, p->T, H, false)) != BSC_OK) return s;
  if ((s = check_device()) != BSC_OK) return s;
  bsc::CacheRwArgs a{};
  a.c = cache_pools(p->cache);
  a.pt = {p->page_table, p->table_stride, p->max_pages, p->seq_lens};
  a.x[0] = const_cast<void*>(p->k);
  a.x[1] = const_cast<void*>(p->v);
  a.xs[0] = {p->k_stride_b, p->k_stride_t, p->k_stride_h};
  a.xs[1] = {p->v_stride_b, p->v_stride_t, p->v_stride_h};
  a.B = p->B;
  a.T = p->T;
  a.rule = p->rule;
  a.first = p->new_lens;
  a.dev_status = p->dev_status;
  return from_cuda(bsc::launch_cache_write(a, p->cache.format, p->cache.D, p->dtype,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

bsc_status mx_cache_read(const bsc_mx_cache_read_params* p, bsc_stream_t stream) {
  if (!p) return BSC_ERR_NULL;
  bool empty;
  bsc_status s = check_cache(p->cache, p->B, p->T, p->cache.Hkv, p->dtype, p->table_stride, p->max_pages, &empty);
  if (s != BSC_OK || empty) return s;
  if (reaches_2_31({2, p->B, (p->T + 15LL) / 16, p->cache.Hkv})) return BSC_ERR_UNSUPPORTED;   // warps
  if (!p->k || !p->v || !p->seq_lens || (p->max_pages > 0 && !p->page_table)) return BSC_ERR_NULL;
  if (!aligned16(p->k) || !aligned16(p->v) || !aligned4(p->page_table) || !aligned4(p->seq_lens) ||
      !aligned4(p->starts) || !aligned4(p->dev_status))
    return BSC_ERR_ALIGN;
  const int H = p->cache.Hkv;
  if ((s = check_strides(p->k_stride_b, p->k_stride_t, p->k_stride_h, p->B, p->T, H, true)) != BSC_OK) return s;
  if ((s = check_strides(p->v_stride_b, p->v_stride_t, p->v_stride_h, p->B, p->T, H, true)) != BSC_OK) return s;
  if ((s = check_device()) != BSC_OK) return s;
  bsc::CacheRwArgs a{};
  a.c = cache_pools(p->cache);
  a.pt = {p->page_table, p->table_stride, p->max_pages, p->seq_lens};
  a.x[0] = p->k;
  a.x[1] = p->v;
  a.xs[0] = {p->k_stride_b, p->k_stride_t, p->k_stride_h};
  a.xs[1] = {p->v_stride_b, p->v_stride_t, p->v_stride_h};
  a.B = p->B;
  a.T = p->T;
  a.first = p->starts;
  a.dev_status = p->dev_status;
  return from_cuda(bsc::launch_cache_read(a, p->cache.format, p->cache.D, p->dtype,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

size_t mx_cache_attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D, long long max_tokens) {
  if (B <= 0 || T <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || max_tokens < 0) return 0;
  if (cache_attn_too_large(B, T, Hq, Hkv, 0)) return 0;     // refused by the call itself
  if (max_tokens > BSC_CACHE_MAX_TOKENS) max_tokens = BSC_CACHE_MAX_TOKENS;
  return bsc::cache_attn_workspace_bytes(B, T, Hq, Hkv, D, max_tokens);
}

bsc_status mx_cache_attn(const bsc_mx_cache_attn_params* p, bsc_stream_t stream) {
  if (!p) return BSC_ERR_NULL;
  bool empty;
  bsc_status s = check_cache(p->cache, p->B, p->T, p->Hq, p->dtype, p->table_stride, p->max_pages, &empty);
  if (s != BSC_OK || empty) return s;
  if (p->Hq % p->cache.Hkv != 0) return BSC_ERR_SHAPE;
  if (!(std::isfinite(p->softmax_scale) && p->softmax_scale > 0.f)) return BSC_ERR_UNSUPPORTED;
  if (cache_attn_too_large(p->B, p->T, p->Hq, p->cache.Hkv, (long long)p->max_pages * p->cache.page_size))
    return BSC_ERR_UNSUPPORTED;
  const size_t need = mx_cache_attn_workspace_bytes(p->B, p->T, p->Hq, p->cache.Hkv, p->cache.D,
                                                    (long long)p->max_pages * p->cache.page_size);
  if (!p->q || !p->o || !p->seq_lens || (p->max_pages > 0 && !p->page_table) || (need > 0 && !p->workspace)) return BSC_ERR_NULL;
  if (!aligned16(p->q) || !aligned16(p->o) || !aligned16(p->workspace) || !aligned4(p->page_table) ||
      !aligned4(p->seq_lens) || !aligned4(p->new_lens) || !aligned4(p->lse) || !aligned4(p->dev_status))
    return BSC_ERR_ALIGN;
  if ((s = check_strides(p->q_stride_b, p->q_stride_t, p->q_stride_h, p->B, p->T, p->Hq, false)) != BSC_OK) return s;
  if ((s = check_strides(p->o_stride_b, p->o_stride_t, p->o_stride_h, p->B, p->T, p->Hq, true)) != BSC_OK) return s;
  if (p->workspace_bytes < need) return BSC_ERR_SHAPE;
  if ((s = check_device()) != BSC_OK) return s;
  bsc::CacheAttnArgs a{};
  a.c = cache_pools(p->cache);
  a.pt = {p->page_table, p->table_stride, p->max_pages, p->seq_lens};
  a.q = p->q;
  a.o = p->o;
  a.lse = p->lse;
  a.qs = {p->q_stride_b, p->q_stride_t, p->q_stride_h};
  a.os = {p->o_stride_b, p->o_stride_t, p->o_stride_h};
  a.B = p->B;
  a.T = p->T;
  a.Hq = p->Hq;
  a.new_lens = p->new_lens;
  a.dev_status = p->dev_status;
  a.scale_log2e = (float)((double)p->softmax_scale * 1.4426950408889634);
  a.ws = p->workspace;
  a.fp16 = p->dtype == BSC_FP16;
  return from_cuda(bsc::launch_cache_attn(a, p->cache.format, p->cache.D, reinterpret_cast<cudaStream_t>(stream)));
}

bsc_status bsc_read_device_status(const int32_t* dev_status, bsc_stream_t stream) {
  if (!dev_status) return BSC_ERR_NULL;
  int32_t v = 0;
  if (cudaMemcpyAsync(&v, dev_status, sizeof(v), cudaMemcpyDeviceToHost, reinterpret_cast<cudaStream_t>(stream)) !=
          cudaSuccess ||
      cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return BSC_ERR_CUDA;
  return v == 0 ? BSC_OK : (v & ~0xFF) == 0x200 ? BSC_ERR_DEVICE_PAGE : BSC_ERR_DEVICE_TIMEOUT;
}

}  // extern "C"
