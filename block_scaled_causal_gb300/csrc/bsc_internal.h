// Internal launch interface shared by the C-ABI layer and the kernels (not part of the ABI).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace bsc {

// rule: 0 = OCP floor scale rule, 1 = ceil (no element saturates)
cudaError_t launch_quant_rowwise(const void* x, uint8_t* q, uint8_t* sc, int B, int S, int H, int layout,
                                 cudaStream_t st, int rule = 0);
// Q and K rowwise and V (columnwise and/or token-normalised) in one launch.
struct QkvQuantArgs {
  const void* q;
  const void* k;
  const void* v;
  int B, S, Hq, Hkv, layout, rule;
  uint8_t* q8;
  uint8_t* q_sc;
  uint8_t* k8;
  uint8_t* k_sc;
  uint8_t* vt;       // may be nullptr (no columnwise copy)
  uint8_t* vsc;
  uint8_t* vtn;      // may be nullptr (no token-normalised copy)
  uint8_t* vtn_sc;
  long long nv_blocks, nq_blocks;   // set by the launcher
};
cudaError_t launch_quant_qkv(QkvQuantArgs a, cudaStream_t st);
cudaError_t launch_quant_v(const void* v, uint8_t* vt, uint8_t* vsc, uint8_t* vtn, uint8_t* vtn_sc, int B, int S,
                           int H, int layout, cudaStream_t st, int rule = 0);

// Everything the attention kernel reads, by value (tensor maps must be 64-byte aligned).
struct AttnArgs {
  CUtensorMap tm_q;     // Q bytes, 4-D {D, Hq, S, B}, box {128,1,128,1}, 128-byte swizzle
  CUtensorMap tm_k;     // K bytes, 4-D {D, Hkv, S, B}, same box
  CUtensorMap tm_v;     // V columnwise bytes, 2-D {S, B*Hkv*D}, box {128,128}, 128-byte swizzle
  const uint8_t* q_sc;     // compact [B][Hq][S][4]
  const uint8_t* k_sc;     // compact [B][Hkv][S][4]
  const uint8_t* v_sc;     // compact [B][Hkv][S/32][128]
  const uint8_t* vtn;      // token-normalised V bytes, K's layout (unused when leaky)
  const uint8_t* vtn_sc;   // [B][Hkv][S]
  void* o;              // bf16 O, or nullptr
  uint8_t* o8;          // E4M3 O, or nullptr
  uint8_t* o_sc;        // compact [B][Hq][S][4] scales of the E4M3 O (with o8)
  float* lse;
  int32_t* dev_status;
  unsigned long long limit_ns;
  int B, S, Hq, Hkv, layout;
  float scale_log2e;
  int p_terms;
  int leaky;
  int inject_stall;
};

cudaError_t launch_attn_fwd(const AttnArgs& args, cudaStream_t st);

// Arguments of the backward kernels (prep, dQ, and dK/dV).
struct BwdArgs {
  CUtensorMap tm_qh;    // decoded Q, BF16 workspace planes [B*Hq][Sp][D], box {64,128,1}, 128-byte swizzle
  CUtensorMap tm_kh;    // decoded K, [B*Hkv][Sp][D], likewise
  CUtensorMap tm_vh;    // decoded token-normalised V, [B*Hkv][Sp][D], likewise
  CUtensorMap tm_do;    // dO bf16, 4-D {D, Hq, S, B}, box {64,1,128,1}, 128-byte swizzle
  const uint8_t* q8;    // Q bytes, `layout`, Hq heads
  const uint8_t* k8;    // K bytes, `layout`, Hkv heads
  const uint8_t* vtn;   // token-normalised V bytes, `layout`, Hkv heads
  const uint8_t* q_sc;  // compact [B][Hq][S][4]
  const uint8_t* k_sc;  // compact [B][Hkv][S][4]
  const uint8_t* vtn_sc;  // [B][Hkv][S]
  const void* o;        // bf16 O of the forward, Q's layout
  const void* dO;       // bf16 dO, Q's layout
  const float* lse;     // [B][Hq][S], natural log
  void* dq;             // bf16, Q's layout
  void* dk;             // bf16, K's layout
  void* dv;             // bf16, K's layout
  float* ws;            // workspace: Dlt [B][Hq][Sp], then LSE * log2(e) [B][Hq][Sp]
  uint16_t* qh;         // workspace: the BF16 planes behind tm_qh, tm_kh, tm_vh
  uint16_t* kh;
  uint16_t* vh;
  int32_t* dev_status;
  unsigned long long limit_ns;
  int B, S, Hq, Hkv, layout;
  int Sp;               // S rounded up to the 128-row tile
  float scale, scale_log2e;
};

// Workspace bytes of the backward: the statistics (2 x 4 B per query row) and the BF16 planes of
// Qh, Kh and Vt (256 B per row), rows padded to Sp.
size_t bwd_workspace_bytes(int B, int S, int Hq, int Hkv);

cudaError_t launch_attn_bwd(const BwdArgs& args, cudaStream_t st);

// The key/value cache.  Strides of the pools in bytes, of activations in elements.
struct CachePools {
  uint8_t* k;
  uint8_t* k_sc;
  uint8_t* v;
  uint8_t* v_sc;
  long long k_ps, k_sc_ps, v_ps, v_sc_ps;
  int num_pages, page_size, Hkv;
};
struct CacheTable {
  const int32_t* table;
  long long stride;
  int max_pages;
  const int32_t* seq_lens;
};
struct RowStrides {
  long long b, t, h;
};
struct CacheRwArgs {
  CachePools c;
  CacheTable pt;
  void* x[2];              // K and V activations (read by the write call, written by the read call)
  RowStrides xs[2];
  int B, T;
  int rule;
  const int32_t* first;    // write: new_lens (nullptr: T); read: starts (nullptr: 0)
  int32_t* dev_status;
};
cudaError_t launch_cache_write(const CacheRwArgs& a, int format, int D, int dtype, cudaStream_t st);
cudaError_t launch_cache_read(const CacheRwArgs& a, int format, int D, int dtype, cudaStream_t st);

// Root-mean-square norm.  Row r of a tensor starts at (r / inner) * outer + (r % inner) * NormRows::inner elements.
struct NormRows {
  long long outer, inner;
};
struct NormArgs {
  const void* x;
  const void* r;           // residual, or nullptr
  const void* w;
  void* y;                 // 16-bit output, or nullptr
  void* s;                 // x + residual, or nullptr
  float* rstd;             // or nullptr
  uint8_t* y8;             // MXFP8 output [rows][N], or nullptr
  uint8_t* ysc;            // [rows][N/32]
  NormRows xs, rs, ys, ss;
  long long rows;
  int inner, N, rule;
  int w32;                 // weights: 0 the activations' type, 1 fp32
  float eps;
};
cudaError_t launch_norm(const NormArgs& a, int dtype, cudaStream_t st);
struct NormBwdArgs {
  const void* dy;
  const void* s;
  const void* w;
  const float* rstd;
  const void* ds;          // gradient that reaches s by another way, or nullptr
  void* dx;
  void* dw;
  float* partial;          // workspace [blocks][N]
  NormRows dys, ss, dss, dxs;
  long long rows;
  int inner, N;
  int w32;
};
cudaError_t launch_norm_bwd(const NormBwdArgs& a, int dtype, cudaStream_t st);
size_t norm_bwd_workspace_bytes(long long rows, int N);

// MXFP8 rows back to values: codes in `layout`, scales [B][H][S][N/32].
cudaError_t launch_dequantize(const uint8_t* x, const uint8_t* sc, void* y, int B, int S, int H, int N, int layout, int dtype,
                              cudaStream_t st);

// Rotary positions.
struct RopeArgs {
  const void* x[3];        // q, k (nullptr: none), and v of the cache form
  RowStrides xs[3];
  void* y[2];              // 16-bit q and k (the cache form: q), or the E4M3 of the MXFP8 form
  RowStrides ys[2];
  uint8_t* sc[2];          // MXFP8 form: scales [B][H][T][D/32]
  const unsigned long long* turns;   // [rot/2], turns per token times 2^64
  float magnitude, magnitude_low;
  int rot, inverse;
  const int32_t* pos;      // nullptr: token t is at position t
  long long pos_b, pos_t;  // its strides; pos_t 0: of the first token
  int B, T, Hq, Hkv, D;    // Hkv 0: no k
  int rule;
  CachePools c;            // cache form
  CacheTable pt;
  const int32_t* new_lens;
  int32_t* dev_status;
  int may_signal;          // set by the launch: the next kernel may start while this one runs
};
cudaError_t launch_rope(const RopeArgs& a, int dtype, int interleaved, cudaStream_t st);
cudaError_t launch_rope_mx(const RopeArgs& a, int dtype, int interleaved, cudaStream_t st);
cudaError_t launch_rope_cache(const RopeArgs& a, int format, int dtype, int interleaved, cudaStream_t st);

// Bounds of the cache's pages, and the pages that every query and KV head attends.
struct BoundsArgs {
  CachePools c;
  CacheTable pt;
  int8_t* codes;           // [num_pages][Hkv][2][D]
  uint8_t* exps;           // [num_pages][Hkv]
  int B, T;
  const int32_t* new_lens; // may be nullptr
  int32_t* dev_status;
};
cudaError_t launch_cache_bounds(const BoundsArgs& a, int format, int D, cudaStream_t st);
struct SelectArgs {
  CacheTable pt;
  const int8_t* codes;
  const uint8_t* exps;
  const void* q;
  RowStrides qs;
  int B, T, Hq, Hkv, num_pages, page_size;
  const int32_t* new_lens; // may be nullptr
  int32_t* dev_status;
  int top, first, last;
  int pages_per_page;      // head slices of the pools from page to page: page p, head h is slice p * this + h
  int32_t* blocks;         // [B][T][Hkv][top], or nullptr
  float* scores;           // workspace of cache_select_scores_bytes(): [B T Hkv][max_pages], or unused
  int32_t* table;          // workspace [B T Hkv][top]: slices, in order
  int32_t* lens;           // workspace [B T Hkv]: tokens of the listed slices
};
cudaError_t launch_cache_select(const SelectArgs& a, int D, int dtype, cudaStream_t st);
size_t cache_select_scores_bytes(int rows, int max_pages, int top);

struct CacheAttnArgs {
  CachePools c;
  CacheTable pt;
  const void* q;
  void* o;
  float* lse;              // may be nullptr
  RowStrides qs, os;
  int B, T, Hq;
  int fp16;                // activations: 0 bf16, 1 fp16
  const int32_t* new_lens; // may be nullptr
  int32_t* dev_status;     // may be nullptr
  float scale_log2e;
  void* ws;
  // Selected pages: 0, or the KV heads; then "sequence" (b sel_T + t) sel_H + h has the pages of one query and KV head, T and
  // the cache's Hkv are 1, Hq counts the query heads of a KV head, and q, o and lse are addressed by (b, t, h).
  int sel_H, sel_T;
};
cudaError_t launch_cache_attn(const CacheAttnArgs& a, int format, int D, cudaStream_t st);
size_t cache_attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D, long long max_tokens);

}  // namespace bsc
