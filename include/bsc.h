/*
 * bsc.h - C ABI of the leak-free causal MXFP8 attention forward library (libbsc.so, sm_103a).
 *
 * The operation: "[PyTorch] Add causal MXFP8 attention without future-token leakage through V
 * scales" (TransformerEngine PR #3865), Description.  A columnwise MXFP8 V scale is shared by 32
 * consecutive tokens, so under an ordinary causal mask a later token of a query's own 32-token
 * block can change how earlier visible V values round.  The method attends keys of completed
 * 32-token blocks (j < 32*floor(i/32)) in MXFP8 with the columnwise V, attends the query's own
 * block (at most 32 keys, j <= i) on a token-normalised V copy (one power-of-two amplitude per
 * token), and merges the two partials through their log-sum-exps, so output row i never depends
 * on a token after i.
 *
 * Conventions for every call:
 *   - Every buffer is device memory owned by the caller.  The library never allocates, frees or
 *     synchronises; all work is enqueued on `stream` (NULL = the legacy default stream).
 *   - Arguments are checked before anything is enqueued; on any error nothing is launched.
 *   - Calls hold no state between invocations and may be made from several host threads.
 *   - Tokens S must be a multiple of 32 (whole MX blocks) and D must be 128.  B, S or H equal to 0
 *     is an empty problem: the call returns BSC_OK and launches nothing (pointers are not
 *     inspected).
 *   - Every pointer must be 16-byte aligned.
 *   - The current CUDA device must be compute capability 10.3 (GB300).
 *   - Inputs are assumed finite; a NaN/Inf V value in a later token can reach earlier rows
 *     through a 0 * NaN product inside the diagonal key tile.
 *
 * Data layouts (BSHD: [B][S][H][D]; SBHD: [S][B][H][D]; D fastest in both).  Every scale array is
 * compact, in the operation's natural order (no padding, no swizzle):
 *   x_bf16, v_bf16, o_bf16    bf16 in the given layout
 *   x_e4m3, vtn_e4m3          E4M3 bytes, same layout and strides as the bf16 input
 *   v_e4m3_t                  E4M3 bytes of V transposed, [B][H][D][S] (tokens in order)
 *   x_sc (Q, K and MXFP8 O)   one scale byte per (b, h, s, 32-element block c = d/32):
 *                             [B][H][S][D/32], byte ((b*H + h)*S + s)*4 + c
 *   v_sc                      one scale byte per (b, h, 32-token block, d):
 *                             [B][H][S/32][D], byte ((b*H + h)*(S/32) + s/32)*D + d
 *   vtn_sc                    one token amplitude per (b, h, s): [B][H][S], byte (b*H + h)*S + s
 *   lse                       fp32 [B][Hq][S], natural log
 * Scale bytes are E8M0: value 2^(byte-127), 0xFF = NaN.  The attention kernels permute scales
 * into the tensor cores' scale-factor order themselves.
 *
 * Quantisation rule (OCP MX, E4M3 elements): for a block with maximum magnitude amax, the scale
 * byte is clamp(floor(log2 amax) - 8 + 127, 0, 254) (0 for amax = 0); each element is x*2^-e
 * rounded to nearest even on the E4M3 grid and saturated to +-448; a block holding NaN/Inf gets
 * scale 0xFF and element bytes 0x7F.
 */
#ifndef BSC_H
#define BSC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Opaque stream handle: a cudaStream_t. */
typedef struct CUstream_st* bsc_stream_t;

typedef enum {
  BSC_OK = 0,
  BSC_ERR_NULL = 1,           /* a required pointer is NULL */
  BSC_ERR_SHAPE = 2,          /* negative size, Hq not a multiple of Hkv, bad layout code */
  BSC_ERR_ALIGN = 3,          /* a pointer is not 16-byte aligned */
  BSC_ERR_UNSUPPORTED = 4,    /* D != 128 (the cache calls: nor 64), S % 32 != 0, wrong device, unsupported option or size */
  BSC_ERR_CUDA = 5,           /* a CUDA runtime/driver call failed (launch, tensor map) */
  BSC_ERR_DEVICE_TIMEOUT = 6, /* a device-side wait gave up (see bsc_read_device_status) */
  BSC_ERR_DEVICE_PAGE = 7     /* a cache call met a page id or a length its page table does not have */
} bsc_status;

typedef enum { BSC_BSHD = 0, BSC_SBHD = 1 } bsc_layout;

/* Version of this ABI (bumped on any incompatible change). */
int bsc_abi_version(void);

/* Human-readable name of a status code (static storage). */
const char* bsc_status_string(bsc_status s);

/*
 * Rowwise MXFP8 quantisation of Q or K: one E8M0 scale per 32 consecutive elements along D of
 * each (b, s, h) row ("Q/K decoded from their rowwise MXFP8 bytes", PR #3865 Description).
 *   x_bf16 [in]  bf16 in `layout`;  x_e4m3 [out] same layout;  x_sc [out] [B][H][S][D/32].
 */
bsc_status mxfp8_quantize_qk_rowwise(const void* x_bf16, int B, int S, int H, int D, bsc_layout layout,
                                     uint8_t* x_e4m3, uint8_t* x_sc, bsc_stream_t stream);

/*
 * Columnwise MXFP8 quantisation of V: one E8M0 scale per 32 consecutive tokens of each (b, h, d)
 * ("A columnwise MXFP8 V scale is shared by 32 consecutive tokens", PR #3865 Description).
 *   v_bf16 [in] bf16 in `layout`;  v_e4m3_t [out] [B][H][D][S];  v_sc [out] [B][H][S/32][D].
 */
bsc_status mxfp8_quantize_v_colwise(const void* v_bf16, int B, int S, int H, int D, bsc_layout layout,
                                    uint8_t* v_e4m3_t, uint8_t* v_sc, bsc_stream_t stream);

/*
 * Token-normalised V copy: one power-of-two amplitude per (b, s, h) token row ("a
 * token-normalized copy of V (one power-of-two amplitude per token)", PR #3865 Description),
 * chosen by the same MX rule with the block spanning all D elements of the row.
 *   v_bf16 [in];  vtn_e4m3 [out] same layout as V;  vtn_sc [out] B*H*S bytes.
 */
bsc_status v_token_normalize(const void* v_bf16, int B, int S, int H, int D, bsc_layout layout,
                             uint8_t* vtn_e4m3, uint8_t* vtn_sc, bsc_stream_t stream);

/* Both V quantisations in one pass over V (one read); outputs as in the two calls above. */
bsc_status mxfp8_quantize_v_fused(const void* v_bf16, int B, int S, int H, int D, bsc_layout layout,
                                  uint8_t* v_e4m3_t, uint8_t* v_sc, uint8_t* vtn_e4m3, uint8_t* vtn_sc,
                                  bsc_stream_t stream);

/*
 * Scale rule of the quantisers.  FLOOR, used by every call above, is the OCP MX rule stated at
 * the top of this file.  CEIL rounds the scale up instead, e = ceil(log2(amax / 448)): the
 * smallest scale at which no element of the block saturates, one more than FLOOR exactly when
 * the significand of amax is above 1.75.  The pages say only that TE's MXFP8 attention reused
 * TE's existing quantisation kernels (PR #3865, base change list); CEIL is the "amax / scale
 * <= 448" reading of such a kernel, offered as a variant.
 */
typedef enum { BSC_SCALE_FLOOR = 0, BSC_SCALE_CEIL = 1 } bsc_scale_rule;
typedef enum {
  BSC_QUANT_ROWWISE = 0,      /* as mxfp8_quantize_qk_rowwise: x -> e4m3, sc */
  BSC_QUANT_V_COLWISE = 1,    /* as mxfp8_quantize_v_colwise: x -> e4m3 (the v_e4m3_t), sc */
  BSC_QUANT_V_TOKEN_NORM = 2, /* as v_token_normalize: x -> vtn_e4m3, vtn_sc */
  BSC_QUANT_V_FUSED = 3       /* as mxfp8_quantize_v_fused: all four outputs */
} bsc_quant_kind;
typedef struct {
  int kind;               /* bsc_quant_kind */
  const void* x;          /* [in] bf16 in `layout` */
  int B, S, H, D;
  int layout;             /* bsc_layout */
  int rule;               /* bsc_scale_rule */
  uint8_t* e4m3;          /* [out] rowwise bytes, or V columnwise bytes [B][H][D][S] */
  uint8_t* sc;            /* [out] [B][H][S][D/32] (rowwise) or [B][H][S/32][D] (V columnwise) */
  uint8_t* vtn_e4m3;      /* [out] token-normalised V bytes (token-norm and fused kinds) */
  uint8_t* vtn_sc;        /* [out] token amplitudes (token-norm and fused kinds) */
} bsc_quant_params;

/* Any of the four quantisations above with a chosen scale rule; layouts, sizes, ownership and
 * errors as in the matching call.  An unknown kind or rule is BSC_ERR_UNSUPPORTED. */
bsc_status mxfp8_quantize(const bsc_quant_params* p, bsc_stream_t stream);

/*
 * Every operand of the attention forward quantised in one launch: Q and K rowwise (as
 * mxfp8_quantize_qk_rowwise), V columnwise and token-normalised (as mxfp8_quantize_v_fused), each
 * tensor read once.  Outputs are byte-identical to those calls.  The pages quantise the three
 * operands in a separate step ahead of the attention and count it, with the launches, in a fixed
 * cost of about 1 ms at batch 1 (PR #3865, Performance); one launch for all three is this
 * library's form of that step.
 *   q [in] bf16 B x S x Hq x D in `layout`;  k, v [in] bf16 with Hkv heads;  Hq % Hkv == 0.
 *   q_e4m3, q_sc, k_e4m3, k_sc [out] as mxfp8_quantize_qk_rowwise for Q and K.
 *   v_e4m3_t, v_sc [out] as mxfp8_quantize_v_colwise; vtn_e4m3, vtn_sc [out] as v_token_normalize.
 *   Either V pair may be NULL (both pointers of the pair), not both.
 *   rule: bsc_scale_rule.  Errors as the calls above; an unknown rule is BSC_ERR_UNSUPPORTED.
 */
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  int B, S, Hq, Hkv, D;
  int layout;             /* bsc_layout */
  int rule;               /* bsc_scale_rule */
  uint8_t* q_e4m3;
  uint8_t* q_sc;
  uint8_t* k_e4m3;
  uint8_t* k_sc;
  uint8_t* v_e4m3_t;
  uint8_t* v_sc;
  uint8_t* vtn_e4m3;
  uint8_t* vtn_sc;
} bsc_qkv_quant_params;
bsc_status mxfp8_quantize_qkv(const bsc_qkv_quant_params* p, bsc_stream_t stream);

typedef struct {
  const uint8_t* q;       /* [in] Q E4M3 bytes, `layout`, Hq heads */
  const uint8_t* q_sc;    /* [in] Q scales [B][Hq][S][D/32] */
  const uint8_t* k;       /* [in] K E4M3 bytes, `layout`, Hkv heads */
  const uint8_t* k_sc;    /* [in] K scales [B][Hkv][S][D/32] */
  const uint8_t* v_t;     /* [in] V columnwise E4M3 bytes, [B][Hkv][D][S] */
  const uint8_t* v_sc;    /* [in] V columnwise scales [B][Hkv][S/32][D] */
  const uint8_t* vtn;     /* [in] token-normalised V bytes, `layout` (unused when leaky = 1) */
  const uint8_t* vtn_sc;  /* [in] token amplitudes [B][Hkv][S] (unused when leaky = 1) */
  void* o;                /* [out] bf16 O in `layout`, Hq heads (may be NULL when o_e4m3 is set) */
  float* lse;             /* [out] [B][Hq][S], ln sum_{j<=i} exp(softmax_scale * q_i . k_j) */
  int B, S, Hq, Hkv, D;
  int layout;             /* bsc_layout */
  float softmax_scale;    /* finite and > 0, else BSC_ERR_UNSUPPORTED */
  /* Number of E4M3 terms P is split into for the MXFP8 P.V of completed blocks (1 or 2).  Each
   * row's weights are quantised per 32-key block with a power-of-two scale chosen from that row's
   * own scores in that block (the block's largest weight lands in [128, 256)), so a scale never
   * depends on another row or on a key the row cannot see.  The second term is the E4M3 residual
   * at the same scale.  The own block is one BF16 term. */
  int p_terms;
  /* 0: the method.  1: ordinary (leaky) causal MXFP8 - the own block is attended with the
   * columnwise V as well; a control that shows the leak. */
  int leaky;
  /* Optional device int32 (may be NULL).  Left untouched on success; a device-side wait that
   * gives up writes 0x100 | site.  Clear it before the call when you intend to read it. */
  int32_t* dev_status;
  /* Wall-clock limit of any single device-side wait, milliseconds (0 = 2000). */
  uint32_t wait_timeout_ms;
  /* Test hook: 1 makes the MMA issuer wait on a barrier nothing arrives on, so the call ends
   * through the wait limit with dev_status set.  Must be 0 in normal use. */
  int debug_stall;
  /* Optional MXFP8 O ("FROST SDPA fp8: block-scaled O epilogues (NVFP4 / MXFP8) with an sf_o
   * output", cudnn-frontend PR #1088 and its follow-up #1180, Summary: FP8_E4M3 O with one UE8M0
   * scale per 32 head-dim elements; that page keeps the scales in its swizzled atom order, this
   * library in the compact order of Q's scales).  When o_e4m3 is not NULL the epilogue also
   * writes O as E4M3 bytes in `layout` (Hq heads) and
   * o_sc [B][Hq][S][D/32] like Q's scales, by the quantisation rule above applied to the fp32 O
   * before any BF16 rounding.  o_sc is required with o_e4m3. */
  uint8_t* o_e4m3;
  uint8_t* o_sc;
} bsc_attn_fwd_params;

/*
 * Leak-free causal MXFP8 attention forward (PR #3865 Description: completed-block MXFP8 part,
 * own-block part on the token-normalised V, log-sum-exp merge).  GQA: query head h reads
 * KV head h / (Hq/Hkv).  Returns BF16 O and/or MXFP8 O, and fp32 LSE.
 * Causality: for finite inputs, row i of every output is bit-for-bit independent of the tokens
 * after i.  V must be finite for that to hold inside a 128-token tile: the diagonal tile's MMAs
 * multiply the zero weights of a row's later keys with those keys' V, and 0 x NaN (or 0 x the NaN
 * that a non-finite V block encodes to) is NaN, so a non-finite V element of token j makes the
 * earlier rows of j's 128-token tile non-finite.  Rows of earlier tiles never read token j.
 */
bsc_status mxfp8_causal_attn_fwd(const bsc_attn_fwd_params* p, bsc_stream_t stream);

typedef struct {
  const uint8_t* q;       /* [in] Q E4M3 bytes, `layout`, Hq heads */
  const uint8_t* q_sc;    /* [in] Q scales [B][Hq][S][D/32] */
  const uint8_t* k;       /* [in] K E4M3 bytes, `layout`, Hkv heads */
  const uint8_t* k_sc;    /* [in] K scales [B][Hkv][S][D/32] */
  const uint8_t* vtn;     /* [in] token-normalised V bytes, `layout`, Hkv heads */
  const uint8_t* vtn_sc;  /* [in] token amplitudes [B][Hkv][S] */
  const void* o;          /* [in] bf16 O of the forward, `layout`, Hq heads */
  const float* lse;       /* [in] LSE of the forward, [B][Hq][S], natural log */
  const void* d_o;        /* [in] bf16 dO, `layout`, Hq heads */
  void* dq;               /* [out] bf16, `layout`, Hq heads */
  void* dk;               /* [out] bf16, `layout`, Hkv heads */
  void* dv;               /* [out] bf16, `layout`, Hkv heads */
  int B, S, Hq, Hkv, D;
  int layout;             /* bsc_layout */
  float softmax_scale;    /* finite and > 0, else BSC_ERR_UNSUPPORTED */
  int32_t* dev_status;    /* optional, as in bsc_attn_fwd_params */
  uint32_t wait_timeout_ms;
  /* [scratch] device memory of at least bf16_attn_bwd_workspace_bytes(B, S, Hq, Hkv) bytes,
   * 16-byte aligned, overlapping no other argument; owned by the caller, contents on entry
   * ignored, on return undefined.  The call first writes there, once, what both backward kernels
   * read: Qh, Kh and the token-normalised Vt decoded to BF16 (one plane per batch and head, rows
   * padded to a multiple of 128 with zeros) and the per-row statistics Dlt_i and LSE_i*log2(e).
   * NULL: BSC_ERR_NULL; workspace_bytes below the required size: BSC_ERR_SHAPE. */
  float* workspace;
  size_t workspace_bytes;
} bsc_attn_bwd_params;

/*
 * Backward of the leak-free attention on decoded operands ("[PyTorch] Add causal MXFP8 attention
 * without future-token leakage through V scales", PR #3865, Description, Backward: an FP16/BF16
 * backward on Q and K decoded from their rowwise MXFP8 bytes and V decoded from the
 * token-normalised copy, so no gradient depends on a future token).  With s = scale*Qh.Kh^T on
 * keys j <= i: P = exp(s - LSE), dV = P^T dO, dP = dO.Vt^T, Dlt_i = <dO_i, O_i>,
 * dS = P*(dP - Dlt), dQ = scale*dS.Kh, dK = scale*dS^T.Qh; GQA: dK, dV of a KV head sum over
 * the query heads that read it.  BF16 tensor-core MMAs (P and dS rounded to BF16), fp32
 * accumulation, BF16 outputs.  Uses no memory beyond its arguments and the caller's workspace.
 */
bsc_status bf16_attn_bwd(const bsc_attn_bwd_params* p, bsc_stream_t stream);

/*
 * Bytes of workspace bf16_attn_bwd needs: B * Sp * (8 * Hq + 256 * (Hq + 2 * Hkv)) with
 * Sp = 128 * ceil(S / 128) (fp32 statistics per query row, a BF16 row of D = 128 per query and
 * per key and value row); 0 if a size is not positive.  Host only, no CUDA call.
 */
size_t bf16_attn_bwd_workspace_bytes(int B, int S, int Hq, int Hkv);

/*
 * The backward of bf16_attn_bwd without caller scratch: `workspace` and `workspace_bytes` of *p are
 * ignored and the call uses a fixed device array of this library (bf16_attn_bwd_static_capacity()
 * bytes, taken when the library's module holding it is loaded), so it allocates nothing.  The
 * pages have no counterpart of this call; it is a packaging of the same computation.  The array is
 * shared by every call on a device: calls must not overlap in time (one stream, or synchronised).
 * A call that needs more than the capacity: BSC_ERR_SHAPE, nothing launched.  Other arguments and
 * errors as bf16_attn_bwd.
 */
bsc_status bf16_attn_bwd_static(const bsc_attn_bwd_params* p, bsc_stream_t stream);

/* Bytes of the fixed workspace of bf16_attn_bwd_static.  Host only, no CUDA call. */
size_t bf16_attn_bwd_static_capacity(void);

/*
 * The key/value cache for answering token by token: K and V of the tokens seen so far, block-scaled
 * in 8 or 4 bits, in pages; written as tokens arrive, read back, and attended.
 *
 * Both K and V are quantised rowwise, one E8M0 scale per 32 elements along D, by the rule at the
 * top of this file: a token's bytes depend on that token alone, so the cache grows without touching
 * what it holds and no scale covers a later token (a columnwise V scale covers 32 tokens and could
 * be written only when its block is complete).
 *   BSC_CACHE_MXFP8   E4M3 elements, one byte each, as everywhere in this library
 *   BSC_CACHE_MXFP4   OCP MX E2M1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two
 *                     per byte, the even element in the low nibble; the scale rule's 8 is 2 and its
 *                     448 is 6 here; a block holding NaN/Inf has scale 0xFF and nibbles 0x7
 * Pools: k, v [num_pages][Hkv][page_size][D bytes, or D/2] and k_sc, v_sc
 * [num_pages][Hkv][page_size][D/32], with a byte stride from page to page (a multiple of 16, at
 * least the page's own size), so K and V may be slices of one allocation.  page_size is a multiple
 * of 16; D is 64 or 128.  Pages of a sequence need not be neighbours or in order.
 *
 * Position p of sequence b is slot p % page_size of page page_table[b * table_stride + p / page_size];
 * entries past ceil(seq_lens[b] / page_size) are not read.  Two sequences may share pages (a common
 * prefix) as long as no call writes to a shared one: if one call writes a slot twice, what it holds
 * afterwards is unspecified.
 *
 * Activations (k, v, q, o) are bf16 or fp16 with element (b, t, h, d) at b*stride_b + t*stride_t +
 * h*stride_h + d: strides in elements, multiples of 8 (the stride of a dimension of size 1 is
 * ignored), so both of this library's layouts and slices of a fused projection are taken as they are.
 * Those pointers and the pools are 16-byte aligned; page_table, seq_lens, new_lens, starts, lse and
 * dev_status are 4-byte aligned.
 *
 * Lengths and page ids live on the device and cannot be checked before the launch.  A page id
 * outside [0, num_pages) is never followed: its tokens are not written, read as zeros, and are not
 * attended; a position past max_pages * page_size is treated the same way, a negative length as 0.
 * If dev_status is given and holds 0, it then receives 0x201 (page id) or 0x202 (length; either one where a call meets
 * both); it is left untouched otherwise, so a word shared by several calls keeps the first code.
 * bsc_read_device_status returns BSC_ERR_DEVICE_PAGE for both.
 *
 * Outputs, workspace and dev_status overlap no other argument.  Refused as BSC_ERR_UNSUPPORTED, because
 * positions, page rows and grids are counted in 32 bits: a page table of more than
 * BSC_CACHE_MAX_TOKENS positions (max_pages * page_size), a page of Hkv * page_size * D >= 2^31, a page stride of
 * 2^36 bytes or more; for writing and reading 2 * B * Hkv * ceil(T / 16) >= 2^31; for the attention
 * B * Hkv * ceil(T * (Hq/Hkv) / r) * max(r, ceil(max_pages * page_size / 128)) >= 2^31, r the smallest of 8, 16
 * and 32 rows that takes the T * (Hq/Hkv) query rows of a KV head, else 32.  page_table may be NULL where
 * max_pages is 0.
 */
#define BSC_CACHE_MAX_TOKENS (1LL << 30)
typedef enum { BSC_CACHE_MXFP8 = 0, BSC_CACHE_MXFP4 = 1 } bsc_cache_format;
typedef enum { BSC_BF16 = 0, BSC_FP16 = 1, BSC_FP32 = 2 } bsc_dtype;   /* BSC_FP32: weights of the norm only */
typedef struct {
  uint8_t* k;             /* [num_pages][Hkv][page_size][D or D/2] */
  uint8_t* k_sc;          /* [num_pages][Hkv][page_size][D/32] */
  uint8_t* v;
  uint8_t* v_sc;
  long long k_page_stride, k_sc_page_stride, v_page_stride, v_sc_page_stride;   /* bytes */
  int format;             /* bsc_cache_format */
  int num_pages, page_size, Hkv, D;
} bsc_mx_cache;

typedef struct {
  bsc_mx_cache cache;     /* [out] */
  const void* k;          /* [in] T tokens of each sequence, `dtype`, Hkv heads */
  const void* v;
  long long k_stride_b, k_stride_t, k_stride_h, v_stride_b, v_stride_t, v_stride_h;
  int B, T;
  int dtype;              /* bsc_dtype */
  int rule;               /* bsc_scale_rule */
  const int32_t* page_table;  /* [in] [B][max_pages], rows table_stride apart */
  long long table_stride;
  int max_pages;
  const int32_t* seq_lens;    /* [in] [B]: tokens of each sequence, the new ones included */
  const int32_t* new_lens;    /* [in] [B]: how many of the T tokens are real (clamped to [0, T]); NULL: all */
  int32_t* dev_status;        /* optional */
} bsc_mx_cache_write_params;

/* Quantises token t < n_b = new_lens[b] of sequence b into position seq_lens[b] - n_b + t.  Tokens
 * t >= n_b and negative positions are skipped; nothing else in the pools changes. */
bsc_status mx_cache_write(const bsc_mx_cache_write_params* p, bsc_stream_t stream);

typedef struct {
  bsc_mx_cache cache;     /* [in] */
  void* k;                /* [out] `dtype`, Hkv heads; a stride of 0 is refused (BSC_ERR_SHAPE) */
  void* v;
  long long k_stride_b, k_stride_t, k_stride_h, v_stride_b, v_stride_t, v_stride_h;
  int B, T;
  int dtype;              /* bsc_dtype */
  const int32_t* page_table;
  long long table_stride;
  int max_pages;
  const int32_t* seq_lens;    /* [in] [B] */
  const int32_t* starts;      /* [in] [B]: position of the first token read; NULL: 0 */
  int32_t* dev_status;        /* optional */
} bsc_mx_cache_read_params;

/* Token t of sequence b of the outputs is position starts[b] + t: element * 2^(scale - 127), rounded
 * once to nearest even in `dtype` (fp16 beyond 65504 is infinite); NaN where the scale is 0xFF.
 * Positions outside [0, seq_lens[b]) read as zeros. */
bsc_status mx_cache_read(const bsc_mx_cache_read_params* p, bsc_stream_t stream);

typedef struct {
  bsc_mx_cache cache;     /* [in] */
  const void* q;          /* [in] T queries of each sequence, `dtype`, Hq heads */
  void* o;                /* [out] `dtype`, Hq heads; a stride of 0 is refused (BSC_ERR_SHAPE) */
  float* lse;             /* [out] [B][Hq][T], natural log; may be NULL */
  long long q_stride_b, q_stride_t, q_stride_h, o_stride_b, o_stride_t, o_stride_h;
  int B, T, Hq;
  int dtype;              /* bsc_dtype */
  float softmax_scale;    /* finite and > 0, else BSC_ERR_UNSUPPORTED */
  const int32_t* page_table;
  long long table_stride;
  int max_pages;
  const int32_t* seq_lens;    /* [in] [B]: tokens held, the T new ones included */
  const int32_t* new_lens;    /* [in] [B]: how many of the T queries are real (clamped to [0, T]); NULL: all */
  int32_t* dev_status;        /* optional */
  /* [scratch] at least mx_cache_attn_workspace_bytes(...) bytes, 16-byte aligned, used by this call
   * alone until it has run; contents on entry ignored. */
  void* workspace;
  size_t workspace_bytes;
} bsc_mx_cache_attn_params;

/*
 * Attention of T new queries per sequence over the cache, causal: query t < n_b of sequence b is the
 * token at position p = seq_lens[b] - n_b + t and attends the positions j <= p (its own K and V are
 * written before the call).  GQA: query head h reads KV head h / (Hq/Hkv).  T = 1 is a decode step;
 * T > 1 checks a draft or takes a chunk of a prompt.  With Kc, Vc the values the cache stands for,
 *   s_j = softmax_scale * q . Kc_j,  O = sum_j exp(s_j - LSE) Vc_j,  LSE = ln sum_j exp(s_j).
 * Rows that attend nothing (t >= n_b, p < 0, an empty sequence) get O = 0 and LSE = -inf.
 * Row p is bit-for-bit independent of what positions after p hold, NaN and infinities included.
 * Sums run in fp32 over values that are lifted by powers of two, so finite Kc is taken up to 2^100 in magnitude, Vc
 * up to 2^100 where a row attends at most 1024 keys and up to 2^80 at any length, and s_j up to 2^120; beyond that rows
 * may come out infinite or NaN.  Scores, and the log-sum-exps by which the parts of a long sequence are weighed, are as
 * exact as fp32 is at their size.  A block of scale byte 0 (a maximum under 2^-118, or 2^-124 in 4 bits) may count as zeros,
 * and so do elements of q under 2^-39 of their row's largest (under 2^-29 of it they lose low bits).
 * A NaN block of K makes the rows that attend it NaN, one of V their columns of that block, a NaN code its column.
 * The result does not depend on the stream, on other calls or on timing (no atomics in it); it may differ in the
 * last bits with the batch's sizes, lengths and table, which decide how the keys are split.
 */
bsc_status mx_cache_attn(const bsc_mx_cache_attn_params* p, bsc_stream_t stream);

/* Bytes of workspace mx_cache_attn needs at these sizes, whatever the lengths are; max_tokens =
 * max_pages * page_size.  0 where it needs none (short tables; then workspace may be NULL) and if a
 * size is not positive.  Smaller sizes may need more than larger ones: ask for each that is used.
 * Host only, no CUDA call. */
size_t mx_cache_attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D, long long max_tokens);

/*
 * What stands ahead of the attention: the norm before the projections that make Q, K and V, and rotary positions.
 * The pages end at the attention's operands (PR #3865, Description); these calls make them.
 *
 * Root-mean-square norm of rows of N elements, with the residual's addition:
 *   s = x + residual, rounded to `dtype` (s = x where residual is NULL): the residual stream, which the next layer adds to
 *   rstd = (mean_n s_n^2 + eps)^(-1/2),  y_n = s_n * rstd * weight_n
 * in fp32, each output rounded once.  Rows are taken up to 2^56 in magnitude (a sum of squares beyond 3.4e38 is infinite), and
 * where eps is below 2^-126 their largest element is at least 2^-56 or 0 (smaller squares are lost).
 * y goes out in `dtype` (y), as MXFP8 rows (y_e4m3 [rows][N] and y_sc [rows][N/32], the quantisation rule at the top of
 * this file applied to the fp32 y), or both.  A row with a NaN or an infinity comes out as NaN where the formula says so (as
 * does a row of zeros with eps 0).  The order of a row's sum, and so its last bits, depends on N and on whether there are
 * more than 152 rows; on nothing else.
 *
 * Row r of x starts at element (r / inner) * stride + (r % inner) * inner_stride, and so for residual, y and sum: inner = 1
 * for evenly spaced rows, inner = the heads for the heads of a slice of a fused projection.  Strides are multiples of 8
 * (ignored where they do not count: a single row or group), an output's not 0.  N is a multiple of 8 (of 32 with
 * y_e4m3) and at most BSC_NORM_MAX_N, rows below BSC_NORM_MAX_ROWS.  Pointers are 16-byte aligned, rstd 4-byte.
 * y or sum may be x or residual itself (same strides); no other outputs overlap.  rows or N of 0: BSC_OK, nothing is done.
 */
#define BSC_NORM_MAX_N 16384
#define BSC_NORM_MAX_ROWS (1LL << 38)
typedef struct {
  const void* x;          /* [in] `dtype` */
  const void* residual;   /* [in] `dtype`, or NULL */
  const void* weight;     /* [in] [N], `weight_dtype`: `dtype` or BSC_FP32 */
  void* y;                /* [out] `dtype`, or NULL */
  void* sum;              /* [out] s, or NULL */
  float* rstd;            /* [out] [rows], or NULL */
  uint8_t* y_e4m3;        /* [out] [rows][N], or NULL */
  uint8_t* y_sc;          /* [out] [rows][N/32], with y_e4m3 */
  long long rows;
  long long x_stride, x_inner_stride, residual_stride, residual_inner_stride, y_stride, y_inner_stride, sum_stride,
      sum_inner_stride;
  int inner;              /* at least 1 */
  int N;
  int dtype;              /* bsc_dtype: BSC_BF16 or BSC_FP16 */
  int weight_dtype;
  int rule;               /* bsc_scale_rule of y_e4m3 */
  float eps;              /* finite and >= 0 */
} bsc_rms_norm_params;
bsc_status rms_norm(const bsc_rms_norm_params* p, bsc_stream_t stream);

/*
 * Gradients of rms_norm at s (the sum output, or x where there was no residual), with rstd of the forward call:
 *   g = dy * weight,  dx = rstd (g - s rstd mean_n(g s rstd)) + d_sum,  dweight_n = sum over rows of dy_n s_n rstd
 * dx is the gradient of x and of residual alike; d_sum (or NULL) is the gradient that reaches s by the residual stream.  fp32
 * inside; dx is `dtype`, dweight `weight_dtype`.  The rows are summed in an order that depends on rows and N alone: the
 * same inputs give the same bits.  dx may be dy, s or d_sum itself (same strides).  rows of 0 with N > 0: dweight is
 * not written.  workspace: rms_norm_bwd_workspace_bytes(rows, N) bytes, 16-byte aligned, used by this call alone until
 * it has run.  Strides and sizes as above.
 */
typedef struct {
  const void* dy;         /* [in] `dtype` */
  const void* s;          /* [in] `dtype` */
  const void* weight;
  const float* rstd;      /* [in] [rows] */
  const void* d_sum;      /* [in] `dtype`, or NULL */
  void* dx;               /* [out] `dtype` */
  void* dweight;          /* [out] [N], `weight_dtype` */
  long long rows;
  long long dy_stride, dy_inner_stride, s_stride, s_inner_stride, d_sum_stride, d_sum_inner_stride, dx_stride,
      dx_inner_stride;
  int inner, N, dtype, weight_dtype;
  void* workspace;
  size_t workspace_bytes;
} bsc_rms_norm_bwd_params;
bsc_status rms_norm_bwd(const bsc_rms_norm_bwd_params* p, bsc_stream_t stream);

/* Bytes of workspace rms_norm_bwd needs; 0 if a size is not positive or N is refused.  Host only, no CUDA call. */
size_t rms_norm_bwd_workspace_bytes(long long rows, int N);

/*
 * MXFP8 rows back to values: y = element * 2^(scale - 127), rounded once to nearest even in `dtype`; NaN where the scale is
 * 0xFF.  The way back from mxfp8_quantize_qk_rowwise, mxfp8_rope_quantize_qk and rms_norm's MXFP8 output (B = H = 1).
 *   x_e4m3 [in] [..][D] in `layout`, dense;  x_sc [in] [B][H][S][D/32];  y [out] `dtype`, laid out like x_e4m3.
 * D is a multiple of 32; any S.  B * S * H below 2^31, B * S * H * D below 2^40.
 */
bsc_status mxfp8_dequantize(const uint8_t* x_e4m3, const uint8_t* x_sc, int B, int S, int H, int D, bsc_layout layout, int dtype,
                            void* y, bsc_stream_t stream);

/*
 * Rotary positions.  The first `rot` elements of a head are rot/2 pairs; pair i of the token at position p turns by p f_i:
 *   (a, b) -> magnitude * (a cos(p f_i) - b sin(p f_i), a sin(p f_i) + b cos(p f_i))
 * Pairs are (x_i, x_{i + rot/2}), or (x_2i, x_{2i+1}) where `interleaved` is 1.  Elements from rot on pass through.
 *
 * f_i is given as turns per token, times 2^64 and rounded: a 64-bit fraction, so that the angle of any 32-bit position is
 * exact to 2^-33 turns without a table of positions.  bsc_rope_turns fills them in (host only, no CUDA call; the caller copies
 * them to the device once), rounded to nearest for base >= 1 (where f_i is a turn or more, its own last bits are lost):
 *   BSC_ROPE_PLAIN      f_i = base^(-2i/rot)
 *   BSC_ROPE_LINEAR     f_i / factor: positions are interpolated
 *   BSC_ROPE_BASE       base * factor^(rot/(rot-2)) in the place of base: the slowest pair is interpolated by factor, the
 *                       fastest not at all
 *   BSC_ROPE_BY_PARTS   f_i (k + (1 - k) / factor), k = clamp((original_length f_i / 2 pi - low_turns) / (high_turns -
 *                       low_turns), 0, 1): pairs that turn often in the trained length stay, slow ones are interpolated
 *                       (Peng et al., "YaRN: Efficient Context Window Extension of Large Language Models", 3.2); magnitude
 *                       0.1 ln(factor) + 1 (3.4), for every factor >= 1.  (k is linear in a pair's turns.  Where it is
 *                       linear in the pair's number i instead, as in some checkpoints, the caller fills in the turns.)
 * magnitude is 1 for the others.  base > 0, factor > 0 (>= 1 by parts), finite; by parts original_length > 0,
 * 0 <= low_turns < high_turns: else BSC_ERR_UNSUPPORTED.  rot is a multiple of 16 from 16 to 256.
 */
typedef enum { BSC_ROPE_PLAIN = 0, BSC_ROPE_LINEAR = 1, BSC_ROPE_BASE = 2, BSC_ROPE_BY_PARTS = 3 } bsc_rope_scaling;
typedef struct {
  int rot;
  int scaling;            /* bsc_rope_scaling */
  double base, factor;
  double original_length, low_turns, high_turns;   /* BSC_ROPE_BY_PARTS only */
} bsc_rope_config;
bsc_status bsc_rope_turns(const bsc_rope_config* c, unsigned long long* turns, float* magnitude);
/* The same magnitude in more bits than a float: its nearest float and what is left are a bsc_rope_angles' two. */
double bsc_rope_magnitude(const bsc_rope_config* c);

/* What a call rotates by. */
typedef struct {
  const unsigned long long* turns;   /* [in] device, [rot/2] */
  float magnitude;        /* finite */
  int rot;                /* a multiple of 16, at most D */
  int interleaved;        /* 0 or 1 */
  float magnitude_low;    /* added to magnitude, 2^-23 of it at most: what a float does not hold of the factor, or 0 */
} bsc_rope_angles;

/*
 * Q and K rotated in one launch.  Token t of sequence b is at position t (positions NULL), positions[b * position_stride_b]
 * + t (position_stride_t 0), or positions[b * position_stride_b + t * position_stride_t]; positions may be negative.
 * inverse 1 turns back: the gradients of q and k from those of the outputs.  fp32 inside, one rounding.
 * q, k: strides as in the cache calls (elements, multiples of 8), D a multiple of 16, at most 256.  k may be NULL (k_out
 * too), Hkv is then ignored.  q_out may be q and k_out k (same strides); no other overlap.  positions 4-byte aligned,
 * turns 8-byte.  B, T or Hq of 0: BSC_OK, nothing is done (to k neither).
 */
typedef struct {
  bsc_rope_angles angles;
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  long long q_stride_b, q_stride_t, q_stride_h, k_stride_b, k_stride_t, k_stride_h;
  long long q_out_stride_b, q_out_stride_t, q_out_stride_h, k_out_stride_b, k_out_stride_t, k_out_stride_h;
  const int32_t* positions;
  long long position_stride_b, position_stride_t;
  int B, T, Hq, Hkv, D;
  int dtype;              /* bsc_dtype */
  int inverse;
} bsc_rope_params;
bsc_status rope(const bsc_rope_params* p, bsc_stream_t stream);

/*
 * Q and K rotated and quantised rowwise to MXFP8 in one launch: the operands of mxfp8_causal_attn_fwd from the projections'
 * outputs.  The rotated values are quantised from fp32, without a rounding to 16 bits between (so a byte can differ
 * from that of rope followed by mxfp8_quantize_qk_rowwise).  D = 128; any T.
 *   q_e4m3, k_e4m3 [out] dense in `layout`;  q_sc [B][Hq][T][D/32], k_sc [B][Hkv][T][D/32].  Else as rope.
 */
typedef struct {
  bsc_rope_angles angles;
  const void* q;
  const void* k;
  long long q_stride_b, q_stride_t, q_stride_h, k_stride_b, k_stride_t, k_stride_h;
  uint8_t* q_e4m3;
  uint8_t* q_sc;
  uint8_t* k_e4m3;
  uint8_t* k_sc;
  const int32_t* positions;
  long long position_stride_b, position_stride_t;
  int B, T, Hq, Hkv, D;
  int dtype;
  int layout;             /* bsc_layout of the outputs */
  int rule;               /* bsc_scale_rule */
} bsc_rope_quant_params;
bsc_status mxfp8_rope_quantize_qk(const bsc_rope_quant_params* p, bsc_stream_t stream);

/*
 * mx_cache_write with K rotated on the way in, and the same tokens' Q rotated beside it, in one launch: what a decode step or
 * a chunk of a prompt needs ahead of mx_cache_attn.  Token t < n_b of sequence b is at position seq_lens[b] - n_b + t, where
 * its K and V are written and by which its Q and K turn.  K is quantised from the rotated fp32 values.  Rows of q_out with
 * t >= n_b or a negative position are zeros.  q_out may be q (same strides).  Checks and refusals as mx_cache_write, with
 * Hq a multiple of Hkv and B * T below 2^31.  Hq of 0: BSC_OK, nothing is done, to K and V neither.
 */
typedef struct {
  bsc_mx_cache cache;     /* [out] */
  bsc_rope_angles angles;
  const void* q;          /* [in] T tokens of each sequence, `dtype`, Hq heads */
  const void* k;          /* [in] likewise, Hkv heads */
  const void* v;
  void* q_out;            /* [out] `dtype`, Hq heads */
  long long q_stride_b, q_stride_t, q_stride_h, k_stride_b, k_stride_t, k_stride_h, v_stride_b, v_stride_t, v_stride_h;
  long long q_out_stride_b, q_out_stride_t, q_out_stride_h;
  int B, T, Hq;
  int dtype;
  int rule;
  const int32_t* page_table;
  long long table_stride;
  int max_pages;
  const int32_t* seq_lens;
  const int32_t* new_lens;
  int32_t* dev_status;
} bsc_mx_cache_write_rope_params;
bsc_status mx_cache_write_rope(const bsc_mx_cache_write_rope_params* p, bsc_stream_t stream);

/*
 * Reading less of a long cache.  Beside the pools the caller keeps bounds of every page's keys:
 *   codes [num_pages][Hkv][2][D]  int8, the minima and then the maxima along d, rounded outward
 *   exps  [num_pages][Hkv]        one byte e + 127 per page and head: a code stands for code * 2^e
 * with e = clamp(floor(log2 max|K|) - 6, -100, ...).  A page and head with a NaN, or a magnitude of 2^107 or more, has exps
 * 0xFF and codes 0.
 *
 * mx_cache_bounds makes the bounds of the pages that hold positions [seq_lens[b] - n_b, seq_lens[b]) of every sequence, from
 * all of a page's tokens below seq_lens[b]: after each write, with the write's lengths.  Nothing else changes.  It does not
 * read earlier bounds.  Where one call meets a page several times with different numbers of tokens (a shared prefix that ends
 * inside it), its bounds are those of the most tokens, which are bounds of the fewer ones too; a sequence that has the page,
 * but none of its new tokens in it, does not count.  codes 16-byte aligned.
 */
typedef struct {
  bsc_mx_cache cache;     /* [in]; k and k_sc are read */
  int8_t* codes;          /* [out] */
  uint8_t* exps;          /* [out] */
  int B, T;
  const int32_t* page_table;
  long long table_stride;
  int max_pages;
  const int32_t* seq_lens;
  const int32_t* new_lens;    /* [in] [B], clamped to [0, T]; NULL: T */
  int32_t* dev_status;        /* optional */
} bsc_mx_cache_bounds_params;
bsc_status mx_cache_bounds(const bsc_mx_cache_bounds_params* p, bsc_stream_t stream);

/*
 * Attention of T new queries per sequence over `top` pages each, chosen for every query and KV head by a score of the
 * pages' bounds.  Query t < n_b at position p sees the tokens at and before p, which lie in the pages 0 .. p / page_size.
 * With top pages or fewer all are attended: the result is mx_cache_attn's.  Else the first `first` and the last `last`
 * (the page of p among them), and of the others those with the largest
 *   score = 2^e (sum_d u_d max_d - l_d min_d),  u = sum over the KV head's query heads of max(q_d, 0), l of max(-q_d, 0),
 * u and l rounded to 0..127 with one power of two per query and KV head (the largest in [64, 128), 127 at most; less where it
 * is below 2^-121, since the power is 2^127 at most).  Scores are
 * exact in fp32; equal ones are taken in the pages' order.  An exps below 27 or from 228 to 254, which mx_cache_bounds does not
 * write, counts as 27 or 227.  A page whose exps is 0xFF scores above all others; one whose
 * id is out of range comes last and is not attended (0x201).  A query with a NaN or an infinity, or whose sums u and l pass
 * fp32's range or are all below 2^-126, scores every page 0.
 * O and LSE are those of mx_cache_attn over the tokens of the chosen pages.
 *   blocks [out] int32 [B][T][Hkv][top], or NULL: the chosen pages' numbers (position / page_size) in ascending order,
 *     then -1.
 * 1 <= last, 0 <= first, first + last <= top: else BSC_ERR_SHAPE.  The page strides of the four pools are the same whole
 * number of heads (page_size rows), num_pages times that number below 2^31: dense pools and slices of one [pages][2][Hkv]
 * allocation are; else BSC_ERR_UNSUPPORTED.  Also refused so: B * T * Hkv * max(max_pages, 128) or B * T * Hkv * top of
 * 2^31 or more, and what mx_cache_attn refuses at B * T * Hkv sequences of top pages.  Else as mx_cache_attn.
 */
typedef struct {
  bsc_mx_cache cache;     /* [in] */
  const int8_t* codes;    /* [in] */
  const uint8_t* exps;    /* [in] */
  const void* q;
  void* o;
  float* lse;             /* may be NULL */
  int32_t* blocks;        /* may be NULL */
  long long q_stride_b, q_stride_t, q_stride_h, o_stride_b, o_stride_t, o_stride_h;
  int B, T, Hq;
  int dtype;
  float softmax_scale;
  int top, first, last;
  const int32_t* page_table;
  long long table_stride;
  int max_pages;
  const int32_t* seq_lens;
  const int32_t* new_lens;
  int32_t* dev_status;
  void* workspace;        /* [scratch] 16-byte aligned, mx_cache_sparse_attn_workspace_bytes(...) bytes, of this call alone */
  size_t workspace_bytes;
} bsc_mx_cache_sparse_attn_params;
bsc_status mx_cache_sparse_attn(const bsc_mx_cache_sparse_attn_params* p, bsc_stream_t stream);

/* Bytes of workspace mx_cache_sparse_attn needs; 0 if a size is not positive or the sizes are refused.  Host only, no CUDA
 * call. */
size_t mx_cache_sparse_attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int page_size, int max_pages, int top);

/*
 * Synchronises `stream`, reads the int32 at `dev_status` and returns BSC_OK (0),
 * BSC_ERR_DEVICE_PAGE (0x2xx, the cache calls) or BSC_ERR_DEVICE_TIMEOUT (any other value).  The
 * only call that synchronises.
 */
bsc_status bsc_read_device_status(const int32_t* dev_status, bsc_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BSC_H */
