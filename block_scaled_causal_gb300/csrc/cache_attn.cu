// Attention over the key/value cache.
//
// For the query at position p: x_j = log2(e) scale q . K_j over j <= p, O = sum 2^(x_j - z) V_j with
// z = log2 sum 2^x_j, in one pass over the keys with a running reference m (weights 2^(x - m)).
//
// What bounds it.  A decode step reads every K and V byte once for the few query rows that share a KV
// head, so it is bound by memory if the decoding of elements keeps up: at D = 128 a token of one head is
// 136 bytes in 4 bits, so a full-rate stream leaves about 23 warp instructions per token and SM to decode
// 256 elements and do both products.  The layout below spends them.
//
// Products.  Scores are taken transposed, S^T = K Q^T, and O^T = V^T P^T, with 16-bit MMAs
// (mma.sync m16n8k16, fp32 accumulation): keys (then output columns) fill the 16-row side and 8 query
// rows the 8-column side, so a group of up to 8 rows wastes nothing and a K or V fragment is decoded once for
// 8 * NT rows.  The tensor pipe is not the bound (1 MMA per token and row group; 0.5 per clock and SM).
//   * K fragment: a lane holds D/4 neighbouring elements of two keys; the sum over d may run in any
//     order, so element 4i..4i+3 of each lane's run is k-step i and Q is laid out to match.
//   * V fragment: a register pairs two keys of one output column, so the packed bytes of two keys are
//     interleaved (2 logic operations per 4 pairs) before they are converted.
//   * P: the score fragment (keys x queries) becomes the P^T operand by one 8x8 transpose per 8 keys.
// E2M1 and E4M3 are exact in fp16, and so is their product with 2^(scale + OFF) while that is in fp16's
// range: scale exponents -16..11 (4 bits) or -19..2 (8 bits), block maxima from about 2^-14 or 2^-11
// to 2^13 or 2^11.  A key with a scale outside of that (or a NaN block) takes the scalar path below in
// fp32; keys are sorted one by one, by their own bytes, so a row never depends on a key it cannot see.
// Scale byte 0 (a zero block, or a maximum under 2^-117) counts as zero.
//
// Roundings.  Q is scaled per row by a power of two to [2^14, 2^15) and held in fp16: exact for 16-bit
// inputs down to 2^-29 of the row's maximum.  Scores, weights' sums and O are fp32.  Weights are rounded to
// fp16 for the second product (2^-12 relative at most, far under the output's own rounding), around 2^8
// at the reference so that only weights under 2^-22 of the largest lose relative precision.
//
// Work.  A warp takes 32 keys at a time through its own ring of shared-memory stages (cp.async, 16
// bytes per lane, rows permuted so that both fragments read without bank conflicts); a block is 4 warps on
// neighbouring 32-key tiles (a chunk, 128 keys).  The chunks of all (sequence, KV head, row tile) units form one
// list, which the blocks split into equal runs: a long sequence spreads over the card and ragged batches stay
// balanced, whatever the lengths, which only the device knows.  A run that covers a unit writes O; one
// that covers part of it writes (O, log-sum-exp) to the workspace, two slots per block at most, and a second
// kernel joins them in order.
#include "cache.cuh"

namespace bsc {
namespace {

constexpr int KT = 32, WARPS = 4, CHUNK = KT * WARPS, THREADS = WARPS * 32;
constexpr int SMS = 152;
constexpr float SLACK = 4.f;    // a reference moves when a score passes it by this much (log2)
constexpr float LIFT = 8.f;     // weights are 2^(x - m + LIFT)

template <int FMT, int D, int NT>
struct Cfg {
  static constexpr int RB = row_bytes<FMT, D>(), NB = D / 32;
  static constexpr int KE = D / 4, VE = D / 8;           // elements per lane and key of the K and V fragments
  static constexpr int KS = D / 16, MT = D / 16;         // k-steps of the scores, 16-row tiles of O^T
  static constexpr int ROWS = 8 * NT;
  static constexpr int OFF = FMT == CACHE_FP4 ? 2 : 5;   // elements are taken times 2^OFF
  static constexpr uint32_t LO = FMT == CACHE_FP4 ? 111u : 108u, HI = FMT == CACHE_FP4 ? 138u : 129u;
  static constexpr uint32_t SUB = 112u - OFF;            // fp16 exponent field = scale byte - SUB
  static constexpr int STAGE = 2 * KT * (RB + NB);       // K, V, K scales, V scales of 32 keys
  static constexpr int STAGES = FMT == CACHE_FP4 || D == 64 ? 3 : 2;
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int MERGE = WARPS * ROWS * (D + 4) * 4 + WARPS * ROWS * 8;
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;
  static constexpr int OCC = NT == 1 ? (STAGE * STAGES * WARPS > 56 * 1024 ? 3 : 4) : 2;   // blocks per SM
};

// Byte offset of 16-byte piece c of key k's row in a stage.  Rows of 32, 64 or 128 bytes lie in 128-byte
// lines whose 8 pieces are permuted by line: the K reads (8 lanes: two keys 4 apart, 4 pieces each)
// and the V reads (keys 0..3, the same piece) then touch 8 different pieces.
template <int RB>
__device__ __forceinline__ int piece_at(int k, int c) {
  if (RB == 128) return k * 128 + ((c ^ (2 * (k & 3) | ((k >> 2) & 1))) << 4);
  if (RB == 64) return (k >> 1) * 128 + ((((k & 1) * 4 + c) ^ (k & 6)) << 4);
  return (k >> 2) * 128 + ((((k & 3) * 2 + c) ^ (k & 4)) << 4);
}
// Key (0..15) of row s of a 16-key score tile: rows 2t, 2t+1 (one lane's pair after the transpose) are keys t, t+4.
__device__ __forceinline__ int key_of_row(int s) { return ((s & 7) >> 1) + 4 * (s & 1) + (s & 8); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four-byte add, each byte mod 256.
__device__ __forceinline__ uint32_t add4(uint32_t a, uint32_t b) {
  return ((a & 0x7F7F7F7Fu) + (b & 0x7F7F7F7Fu)) ^ ((a ^ b) & 0x80808080u);
}
// Whether every scale byte of a key is in [LO, HI] or 0 (bytes past D/32 of the word are in range).
template <class C>
__device__ __forceinline__ bool scales_in_range(uint32_t w) {
  const uint32_t above = add4(w, (128u - C::LO) * 0x01010101u);               // top bit: byte >= LO (of 0..235)
  const uint32_t beyond = add4(w, ((127u - C::HI) & 0xFFu) * 0x01010101u);    // top bit: byte > HI, or 0
  const uint32_t nonzero = ((w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | w;             // top bit: byte != 0
  return (((above & ~beyond) | ~nonzero) & 0x80808080u) == 0x80808080u;
}

// 2^(byte - 127 + OFF) in fp16 for bytes in range, 0 for byte 0: in both halves / for two bytes.
template <class C>
__device__ __forceinline__ uint32_t scale_f16(uint32_t byte) {
  return (uint32_t)max((int)byte - (int)C::SUB, 0) * 0x04000400u;
}
template <class C>
__device__ __forceinline__ uint32_t scales_f16x2(uint32_t lo, uint32_t hi) {
  return ((uint32_t)max((int)lo - (int)C::SUB, 0) << 10) | ((uint32_t)max((int)hi - (int)C::SUB, 0) << 26);
}

// One element of a row in shared memory, as the fp32 value it stands for times 2^OFF.
template <int FMT, class C>
__device__ __forceinline__ float element(const uint8_t* rows, int k, int d, float scale) {
  const int byte = FMT == CACHE_FP4 ? d >> 1 : d;
  const uint32_t w = rows[piece_at<C::RB>(k, byte >> 4) + (byte & 15)];
  float2 f;
  if (FMT == CACHE_FP4) {
    uint32_t h[4];
    e2m1x8_to_f16(w, h);
    f = f16x2_to_f32(h[0]);
    return (d & 1 ? f.y : f.x) * scale * (float)(1 << C::OFF);
  }
  uint32_t h0, h1;
  e4m3x4_to_f16(w, h0, h1);
  f = f16x2_to_f32(h0);
  return f.x * scale * (float)(1 << C::OFF);
}

// The list of chunks.  Sequence b has n_b = ceil(len_b / CHUNK) chunks per unit and U = Hkv * (row tiles) units.
__device__ __forceinline__ int seq_len(const CacheAttnArgs& a, int b) {
  const long long cap = (long long)a.pt.max_pages * a.c.page_size;   // < 2^31
  const int len = max(__ldg(a.pt.seq_lens + b), 0);
  return len > cap ? (int)cap : len;
}
__device__ __forceinline__ long long chunks_of(const CacheAttnArgs& a, int b, int U) {
  return b < a.B ? (long long)((seq_len(a, b) + CHUNK - 1) / CHUNK) * U : 0;
}
// Sum over the sequences before b (b = B: all of them).  Whole warps call it.
__device__ __forceinline__ long long chunks_before(const CacheAttnArgs& a, int b, int U) {
  long long s = 0;
  for (int i = threadIdx.x & 31; i < b; i += 32) s += chunks_of(a, i, U);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}
// The sequence that chunk x < total belongs to, and its first chunk.
__device__ __forceinline__ int seq_of_chunk(const CacheAttnArgs& a, long long x, int U, long long& base) {
  const int lane = threadIdx.x & 31;
  base = 0;
  for (int b0 = 0;; b0 += 32) {
    const long long n = chunks_of(a, b0 + lane, U);
    long long s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, base + s > x);
    if (hit) {
      const int l = __ffs(hit) - 1;
      base += __shfl_sync(0xFFFFFFFFu, s - n, l);
      return b0 + l;
    }
    base += __shfl_sync(0xFFFFFFFFu, s, 31);
    if (b0 + 32 >= a.B) return a.B;   // x is past the list
  }
}
// Blocks that share the list, the first chunk of block i, and the block that has chunk x.
__device__ __forceinline__ long long blocks_of(long long total, int grid) { return total < grid ? total : grid; }
__device__ __forceinline__ long long first_chunk(long long total, long long n, long long i) { return total * i / n; }
__device__ __forceinline__ long long block_of_chunk(long long total, long long n, long long x) {
  return ((x + 1) * n - 1) / total;
}

// A workspace slot: ROWS x D of O, then ROWS log-sum-exps (log2).
template <class C, int D>
constexpr int slot_floats() { return C::ROWS * (D + 1); }

template <int FMT, int D, int DT, int NT>
__global__ void __launch_bounds__(THREADS, Cfg<FMT, D, NT>::OCC) cache_attn_kernel(const CacheAttnArgs a, int row_tiles) {
  using C = Cfg<FMT, D, NT>;
  constexpr int RB = C::RB, NB = C::NB;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int G = a.Hq / a.c.Hkv, U = a.c.Hkv * row_tiles, page_size = a.c.page_size;
  const int R = a.T * G;

  const long long total = chunks_before(a, a.B, U);
  const long long nblk = blocks_of(total, gridDim.x);
  if (blockIdx.x >= nblk) return;
  long long x = first_chunk(total, nblk, blockIdx.x);
  const long long x_end = first_chunk(total, nblk, blockIdx.x + 1);
  long long base;
  int b = seq_of_chunk(a, x, U, base);

  uint8_t* const ring = smem + warp * C::STAGES * C::STAGE;
  const uint32_t ring_s = smem_u32(ring);

  while (x < x_end) {
    // ---- the next piece: chunks [c0, c1) of unit (b, h, rt) ----
    const int len = seq_len(a, b), n_chunks = (len + CHUNK - 1) / CHUNK;
    if (n_chunks == 0) {
      ++b;
      continue;
    }
    const long long rel = x - base;
    const int u = (int)(rel / n_chunks), c0 = (int)(rel - (long long)u * n_chunks);
    const int c1 = (int)min((long long)n_chunks, c0 + (x_end - x));
    const int h = u / row_tiles, rt = u - h * row_tiles;
    const int raw_len = max(__ldg(a.pt.seq_lens + b), 0);
    const int n_new = a.new_lens ? min(max(__ldg(a.new_lens + b), 0), a.T) : a.T;
    if (raw_len > len && tid == 0 && a.dev_status) *a.dev_status = CACHE_BAD_LEN;

    // ---- Q: lane (g, t) holds elements KE t .. KE t + KE - 1 of query row g of each 8-row tile ----
    uint32_t q[NT][C::KS][2];
    float c[NT][2];            // score -> log2 units, rows 2t and 2t + 1
    int lim[NT][2];            // keys j < lim are visible; rows that see nothing or do not exist: all
    int min_lim = len;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = rt * C::ROWS + nt * 8 + g, tq = r / G, hq = h * G + r - tq * G;
      float f[C::KE];
      float mx = 0.f;
      if (r < R) {
        const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + b * a.qs.b + tq * a.qs.t + hq * a.qs.h + t * C::KE;
#pragma unroll
        for (int i = 0; i < C::KE / 8; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 p = act_to_f32<DT>(w[j]);
            f[8 * i + 2 * j] = p.x;
            f[8 * i + 2 * j + 1] = p.y;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < C::KE; ++i) f[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < C::KE; ++i) mx = fmaxf(mx, fabsf(f[i]));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
      // the row's exponent, from -100 (tinier rows score nothing) to 128 (infinities)
      const int ex = max((int)(__float_as_uint(mx) >> 23) - 127, -100);
      const float up = __uint_as_float((uint32_t)(14 - ex + 127) << 23);
#pragma unroll
      for (int i = 0; i < C::KS; ++i) {
        q[nt][i][0] = pack_f16x2(f[4 * i] * up, f[4 * i + 1] * up);
        q[nt][i][1] = pack_f16x2(f[4 * i + 2] * up, f[4 * i + 3] * up);
      }
      const int ex_back = max(ex - 14 - C::OFF, -126);
      const float cg = fmaxf(a.scale_log2e * __uint_as_float((uint32_t)(ex_back + 127) << 23), 1.17549435e-38f);
      // first key past the row: position raw_len - n_new + tq sees itself
      int lg = len;
      if (r < R && tq < n_new) {
        const long long past = (long long)raw_len - n_new + tq + 1;
        if (past > 0 && past < len) lg = (int)past;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        c[nt][j] = __shfl_sync(0xFFFFFFFFu, cg, (2 * t + j) * 4);
        lim[nt][j] = __shfl_sync(0xFFFFFFFFu, lg, (2 * t + j) * 4);
        min_lim = min(min_lim, lim[nt][j]);
      }
    }
    min_lim = __reduce_min_sync(0xFFFFFFFFu, min_lim);

    // ---- the warp's tiles: keys (c0 + i) CHUNK + warp KT + [0, KT) ----
    const int k_first = c0 * CHUNK + warp * KT;
    const int last = min(c1 * CHUNK, len);
    const int n_tiles = k_first < last ? (last - k_first + CHUNK - 1) / CHUNK : 0;

    // page ids: lane 2 i + j has the 16-key group j of tile (window start) + i, for 16 tiles at a time
    int w_page = -1, w_off = 0;
    auto load_window = [&](int tile0) {
      const int i = tile0 + (lane >> 1), key = k_first + i * CHUNK + (lane & 1) * 16;
      w_page = -1;
      if (i < n_tiles && key < len) {
        const int lp = key / page_size;
        w_off = key - lp * page_size;
        w_page = __ldg(a.pt.table + b * a.pt.stride + lp);
        if (w_page < 0 || w_page >= a.c.num_pages) {
          w_page = -1;
          if (a.dev_status) *a.dev_status = CACHE_BAD_PAGE;
        }
      }
    };
    // bit i: the 16 keys of group i & 1 of window tile i >> 1 are there
    uint32_t present = 0;
    auto issue = [&](int tile) {
      if (tile < n_tiles) {
        const uint32_t dst = ring_s + (tile % C::STAGES) * C::STAGE;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int slot = (tile & 15) * 2 + j;
          const long long page = __shfl_sync(0xFFFFFFFFu, w_page, slot);
          const int off = __shfl_sync(0xFFFFFFFFu, w_off, slot);
          if (page >= 0) {
            const long long in_page = (long long)h * page_size + off;
            const uint8_t* ks = a.c.k + page * a.c.k_ps + in_page * RB;
            const uint8_t* vs = a.c.v + page * a.c.v_ps + in_page * RB;
#pragma unroll
            for (int i = 0; i < RB / 32; ++i) {   // 16 rows are RB pieces of 16 bytes
              const int p = i * 32 + lane, k = j * 16 + p / (RB / 16), at = piece_at<RB>(k, p % (RB / 16));
              cp16(dst + at, ks + p * 16);
              cp16(dst + KT * RB + at, vs + p * 16);
            }
            if (lane < 2 * NB) {                  // 16 keys' scales are NB pieces, K's then V's
              const bool v = lane >= NB;
              const int p = v ? lane - NB : lane;
              const uint8_t* src = (v ? a.c.v_sc + page * a.c.v_sc_ps : a.c.k_sc + page * a.c.k_sc_ps) + in_page * NB;
              cp16(dst + 2 * KT * RB + (v ? KT * NB : 0) + j * 16 * NB + p * 16, src + p * 16);
            }
          }
        }
      }
      cp_commit();
    };

    float acc[NT][C::MT][4], l[NT][2], m[NT][2], nm[NT][2];   // nm = LIFT - m (0 where m is -inf)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < C::MT; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
      l[nt][0] = l[nt][1] = nm[nt][0] = nm[nt][1] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
    }

    // a window is loaded when its first tile is issued; `present` follows two windows at most, so it is taken
    // tile by tile: ring_present keeps the two bits of each stage
    uint32_t ring_present = 0;
    auto advance = [&](int tile) {
      if ((tile & 15) == 0 && tile < n_tiles) {
        load_window(tile);
        present = __ballot_sync(0xFFFFFFFFu, w_page >= 0);
      }
      const int st = tile % C::STAGES;
      ring_present = (ring_present & ~(3u << (2 * st))) | (((present >> (2 * (tile & 15))) & 3u) << (2 * st));
      issue(tile);
    };
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) advance(i);

    for (int tile = 0; tile < n_tiles; ++tile) {
      cp_wait<C::STAGES - 2>();
      __syncwarp();
      const int st = tile % C::STAGES;
      const uint32_t there = (ring_present >> (2 * st)) & 3u;
      advance(tile + C::STAGES - 1);

      uint8_t* const stage = ring + st * C::STAGE;
      uint8_t* const vrows = stage + KT * RB;
      uint8_t* const ksc = stage + 2 * KT * RB;
      uint8_t* const vsc = ksc + KT * NB;
      const int k0 = k_first + tile * CHUNK;

      // ---- which keys the matrix path leaves out: `gone` (past the sequence, no page), `odd` (scales) ----
      const int valid = len - k0;
      uint32_t gone = (valid < KT ? 0xFFFFFFFFu << valid : 0u) | (there & 1 ? 0u : 0xFFFFu) |
                      (there & 2 ? 0u : 0xFFFF0000u);
      bool ok;
      if (NB == 4) {
        ok = scales_in_range<C>(reinterpret_cast<const uint32_t*>(ksc)[lane]) &
             scales_in_range<C>(reinterpret_cast<const uint32_t*>(vsc)[lane]);
      } else {
        ok = scales_in_range<C>(reinterpret_cast<const uint16_t*>(ksc)[lane] |
                                (uint32_t)reinterpret_cast<const uint16_t*>(vsc)[lane] << 16);
      }
      const uint32_t odd = __ballot_sync(0xFFFFFFFFu, !ok) & ~gone;
      const uint32_t left_out = gone | odd;

      // ---- scores ----
      float s[NT][2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const int ka = mt * 16 + key_of_row(g), kb = ka + 8;
        const uint32_t sa = scale_f16<C>(ksc[ka * NB + t * C::KE / 32]), sb = scale_f16<C>(ksc[kb * NB + t * C::KE / 32]);
        constexpr int LB = C::KE * RB / D;        // bytes of a lane's run: 8, 16 or 32
        uint32_t wa[LB / 4], wb[LB / 4];
        if (LB == 8) {
          const uint2 ua = *reinterpret_cast<const uint2*>(stage + piece_at<RB>(ka, t >> 1) + (t & 1) * 8);
          const uint2 ub = *reinterpret_cast<const uint2*>(stage + piece_at<RB>(kb, t >> 1) + (t & 1) * 8);
          wa[0] = ua.x; wa[1] = ua.y; wb[0] = ub.x; wb[1] = ub.y;
        } else {
#pragma unroll
          for (int i = 0; i < LB / 16; ++i) {
            const uint4 ua = *reinterpret_cast<const uint4*>(stage + piece_at<RB>(ka, t * (LB / 16) + i));
            const uint4 ub = *reinterpret_cast<const uint4*>(stage + piece_at<RB>(kb, t * (LB / 16) + i));
            wa[4 * i] = ua.x; wa[4 * i + 1] = ua.y; wa[4 * i + 2] = ua.z; wa[4 * i + 3] = ua.w;
            wb[4 * i] = ub.x; wb[4 * i + 1] = ub.y; wb[4 * i + 2] = ub.z; wb[4 * i + 3] = ub.w;
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[nt][mt][0] = s[nt][mt][1] = s[nt][mt][2] = s[nt][mt][3] = 0.f;
        if (FMT == CACHE_FP4) {
#pragma unroll
          for (int i = 0; i < LB / 4; ++i) {
            uint32_t ha[4], hb[4];
            e2m1x8_to_f16(wa[i], ha);
            e2m1x8_to_f16(wb[i], hb);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t a0 = mul_f16x2(ha[2 * j], sa), a1 = mul_f16x2(hb[2 * j], sb);
              const uint32_t a2 = mul_f16x2(ha[2 * j + 1], sa), a3 = mul_f16x2(hb[2 * j + 1], sb);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(s[nt][mt], a0, a1, a2, a3, q[nt][2 * i + j][0], q[nt][2 * i + j][1]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < LB / 4; ++i) {
            uint32_t ha[2], hb[2];
            e4m3x4_to_f16(wa[i], ha[0], ha[1]);
            e4m3x4_to_f16(wb[i], hb[0], hb[1]);
            const uint32_t a0 = mul_f16x2(ha[0], sa), a1 = mul_f16x2(hb[0], sb);
            const uint32_t a2 = mul_f16x2(ha[1], sa), a3 = mul_f16x2(hb[1], sb);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(s[nt][mt], a0, a1, a2, a3, q[nt][i][0], q[nt][i][1]);
          }
        }
      }

      // ---- scores of the odd keys, one at a time in fp32; then the masks ----
      for (uint32_t rest = odd; rest; rest &= rest - 1) {
        const int k = __ffs(rest) - 1;
        float dot[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) dot[nt] = 0.f;
        const float sc = scale_value(ksc[k * NB + t * C::KE / 32]);
#pragma unroll
        for (int i = 0; i < C::KS; ++i) {
          const int d = t * C::KE + 4 * i;
          const float e0 = element<FMT, C>(stage, k, d, sc), e1 = element<FMT, C>(stage, k, d + 1, sc);
          const float e2 = element<FMT, C>(stage, k, d + 2, sc), e3 = element<FMT, C>(stage, k, d + 3, sc);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 qa = f16x2_to_f32(q[nt][i][0]), qb = f16x2_to_f32(q[nt][i][1]);
            dot[nt] += qa.x * e0 + qa.y * e1 + qb.x * e2 + qb.y * e3;
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          dot[nt] += __shfl_xor_sync(0xFFFFFFFFu, dot[nt], 1);
          dot[nt] += __shfl_xor_sync(0xFFFFFFFFu, dot[nt], 2);
          const float s0 = __shfl_sync(0xFFFFFFFFu, dot[nt], 8 * t), s1 = __shfl_sync(0xFFFFFFFFu, dot[nt], 8 * t + 4);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int half = 0; half < 2; ++half)
              if (k == mt * 16 + half * 8 + key_of_row(g)) {
                s[nt][mt][2 * half] = s0;
                s[nt][mt][2 * half + 1] = s1;
              }
        }
      }
      if (gone != 0u || k0 + KT > min_lim) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int k = mt * 16 + half * 8 + key_of_row(g);
            const bool away = (gone >> k) & 1u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                if (away || k0 + k >= lim[nt][j]) s[nt][mt][2 * half + j] = -INFINITY;
          }
      }

      // ---- the reference: moved for a row when one of its own scores is SLACK above it ----
      float top[NT][2];
      bool climb = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          top[nt][j] = c[nt][j] * fmaxf(fmaxf(s[nt][0][j], s[nt][0][2 + j]), fmaxf(s[nt][1][j], s[nt][1][2 + j]));
          climb |= top[nt][j] > m[nt][j] + SLACK;
        }
      if (__any_sync(0xFFFFFFFFu, climb)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx = top[nt][j];
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
            if (mx > m[nt][j] + SLACK) {
              const float keep = ex2_approx(m[nt][j] - mx);   // 0 from -inf
              m[nt][j] = mx;
              nm[nt][j] = LIFT - mx;
              l[nt][j] *= keep;
#pragma unroll
              for (int i = 0; i < C::MT; ++i) {
                acc[nt][i][j] *= keep;
                acc[nt][i][2 + j] *= keep;
              }
            }
          }
      }

      // ---- weights ----
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[nt][mt][i] = ex2_approx(fmaf(s[nt][mt][i], c[nt][i & 1], nm[nt][i & 1]));
            l[nt][i & 1] += s[nt][mt][i];
          }

      // ---- odd keys' part of O in fp32, only for rows that see them; then they and absent keys become zeros ----
      if (left_out != 0u) {
        for (uint32_t rest = odd; rest; rest &= rest - 1) {
          const int k = __ffs(rest) - 1;
          // the lane that holds key k's weights for rows 2t, 2t + 1: row r of a 16-key tile with key_of_row(r) = k % 8
          const int src = ((k & 3) * 2 + ((k >> 2) & 1)) * 4 + t;
          const float sc = scale_value(vsc[k * NB + g * C::VE / 32]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float p[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float p0 = __shfl_sync(0xFFFFFFFFu, s[nt][0][j], src), p1 = __shfl_sync(0xFFFFFFFFu, s[nt][0][2 + j], src);
              const float p2 = __shfl_sync(0xFFFFFFFFu, s[nt][1][j], src), p3 = __shfl_sync(0xFFFFFFFFu, s[nt][1][2 + j], src);
              p[j] = k < 16 ? (k < 8 ? p0 : p1) : (k < 24 ? p2 : p3);
            }
            const bool sees0 = k0 + k < lim[nt][0], sees1 = k0 + k < lim[nt][1];
#pragma unroll
            for (int i = 0; i < C::MT; ++i) {
              const float e0 = element<FMT, C>(vrows, k, g * C::VE + 2 * i, sc);
              const float e1 = element<FMT, C>(vrows, k, g * C::VE + 2 * i + 1, sc);
              if (sees0) {
                acc[nt][i][0] += p[0] * e0;
                acc[nt][i][2] += p[0] * e1;
              }
              if (sees1) {
                acc[nt][i][1] += p[1] * e0;
                acc[nt][i][3] += p[1] * e1;
              }
            }
          }
        }
        __syncwarp();
        if ((left_out >> lane) & 1u) {
#pragma unroll
          for (int i = 0; i < RB / 16; ++i)
            *reinterpret_cast<uint4*>(vrows + piece_at<RB>(lane, i)) = make_uint4(0, 0, 0, 0);
          if (NB == 4)
            reinterpret_cast<uint32_t*>(vsc)[lane] = 0u;
          else
            reinterpret_cast<uint16_t*>(vsc)[lane] = 0;
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            if ((left_out >> (mt * 16 + half * 8 + key_of_row(g))) & 1u) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) s[nt][mt][2 * half] = s[nt][mt][2 * half + 1] = 0.f;
            }
        __syncwarp();
      }

      // ---- O^T += V^T P^T ----
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          pb[nt][0] = transpose8(pack_f16x2(s[nt][mt][0], s[nt][mt][1]));
          pb[nt][1] = transpose8(pack_f16x2(s[nt][mt][2], s[nt][mt][3]));
        }
        constexpr int VB = C::VE * RB / D;     // bytes of a lane's run: 4, 8 or 16
        const int kk = mt * 16 + t, blk = g * C::VE / 32;
        const uint32_t s01 = scales_f16x2<C>(vsc[kk * NB + blk], vsc[(kk + 4) * NB + blk]);
        const uint32_t s23 = scales_f16x2<C>(vsc[(kk + 8) * NB + blk], vsc[(kk + 12) * NB + blk]);
        uint32_t v[4][VB / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint8_t* src = vrows + piece_at<RB>(kk + 4 * i, g * VB / 16) + (g * VB) % 16;
          if (VB == 4) {
            v[i][0] = *reinterpret_cast<const uint32_t*>(src);
          } else if (VB == 8) {
            const uint2 y = *reinterpret_cast<const uint2*>(src);
            v[i][0] = y.x; v[i][1] = y.y;
          } else {
            const uint4 y = *reinterpret_cast<const uint4*>(src);
            v[i][0] = y.x; v[i][1] = y.y; v[i][2] = y.z; v[i][3] = y.w;
          }
        }
#pragma unroll
        for (int w = 0; w < VB / 4; ++w) {
          if (FMT == CACHE_FP4) {
            // even elements of two keys per byte, then odd ones
            uint32_t e01[4], o01[4], e23[4], o23[4];
            e2m1x8_to_f16((v[0][w] & 0x0F0F0F0Fu) | ((v[1][w] << 4) & 0xF0F0F0F0u), e01);
            e2m1x8_to_f16(((v[0][w] >> 4) & 0x0F0F0F0Fu) | (v[1][w] & 0xF0F0F0F0u), o01);
            e2m1x8_to_f16((v[2][w] & 0x0F0F0F0Fu) | ((v[3][w] << 4) & 0xF0F0F0F0u), e23);
            e2m1x8_to_f16(((v[2][w] >> 4) & 0x0F0F0F0Fu) | (v[3][w] & 0xF0F0F0F0u), o23);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t a0 = mul_f16x2(e01[j], s01), a1 = mul_f16x2(o01[j], s01);
              const uint32_t a2 = mul_f16x2(e23[j], s23), a3 = mul_f16x2(o23[j], s23);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][4 * w + j], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {      // elements 2j, 2j + 1 of both keys
              uint32_t e01, o01, e23, o23;
              e4m3x4_to_f16(__byte_perm(v[0][w], v[1][w], j ? 0x7362 : 0x5140), e01, o01);
              e4m3x4_to_f16(__byte_perm(v[2][w], v[3][w], j ? 0x7362 : 0x5140), e23, o23);
              const uint32_t a0 = mul_f16x2(e01, s01), a1 = mul_f16x2(o01, s01);
              const uint32_t a2 = mul_f16x2(e23, s23), a3 = mul_f16x2(o23, s23);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][2 * w + j], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
            }
          }
        }
      }
    }

    // ---- the four warps' parts joined in shared memory (over the rings, whose copies have all landed) ----
    cp_wait<0>();
    __syncthreads();
    float* const mo = reinterpret_cast<float*>(smem);                   // [warp][row][D + 4]
    float2* const ml = reinterpret_cast<float2*>(mo + WARPS * C::ROWS * (D + 4));   // [warp][row] reference, sum
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = l[nt][j];
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
        const int row = nt * 8 + 2 * t + j;
        if (g == 0) ml[warp * C::ROWS + row] = make_float2(m[nt][j], sum);
        float* const dst = mo + (warp * C::ROWS + row) * (D + 4) + g * C::VE;
#pragma unroll
        for (int i = 0; i < C::MT; ++i) *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(acc[nt][i][j], acc[nt][i][2 + j]);
      }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == n_chunks;
    float* const slot = reinterpret_cast<float*>(a.ws) +
                        (2LL * blockIdx.x + (c0 == 0 ? 1 : 0)) * slot_floats<C, D>();
    constexpr int LPR = D / 8;                 // threads per row, 8 columns each
    for (int i = tid; i < C::ROWS * LPR; i += THREADS) {
      const int row = i / LPR, d = (i % LPR) * 8, r = rt * C::ROWS + row;
      if (r >= R) continue;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, ml[w * C::ROWS + row].x);
      float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float2 part = ml[w * C::ROWS + row];
        if (part.x == -INFINITY && part.y == 0.f) continue;    // no key of this warp's
        const float f = part.x == -INFINITY ? 1.f : ex2_approx(part.x - mx);
        sum += f * part.y;
        const float4* src = reinterpret_cast<const float4*>(mo + (w * C::ROWS + row) * (D + 4) + d);
        const float4 y0 = src[0], y1 = src[1];
        o[0] += f * y0.x; o[1] += f * y0.y; o[2] += f * y0.z; o[3] += f * y0.w;
        o[4] += f * y1.x; o[5] += f * y1.y; o[6] += f * y1.z; o[7] += f * y1.w;
      }
      const int tq = r / G;
      const bool sees = tq < n_new && (long long)raw_len - n_new + tq >= 0;
      const bool none = !sees || sum == 0.f;
      const float inv = none ? 0.f : __fdividef(1.f, sum) * (1.f / (1 << C::OFF));
      const float z = none ? -INFINITY : mx - LIFT + __log2f(sum);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = none ? 0.f : o[j] * inv;
      if (whole) {
        const int hq = h * G + r - tq * G;
        uint16_t* dst = reinterpret_cast<uint16_t*>(a.o) + b * a.os.b + tq * a.os.t + hq * a.os.h + d;
        *reinterpret_cast<uint4*>(dst) = make_uint4(f32_to_act<DT>(o[0], o[1]), f32_to_act<DT>(o[2], o[3]),
                                                    f32_to_act<DT>(o[4], o[5]), f32_to_act<DT>(o[6], o[7]));
        if (d == 0 && a.lse) a.lse[((long long)b * a.Hq + hq) * a.T + tq] = z * 0.6931471805599453f;
      } else {
        float4* dst = reinterpret_cast<float4*>(slot + row * D + d);
        dst[0] = make_float4(o[0], o[1], o[2], o[3]);
        dst[1] = make_float4(o[4], o[5], o[6], o[7]);
        if (d == 0) slot[C::ROWS * D + row] = z;
      }
    }
    __syncthreads();

    x += c1 - c0;
    if (x == base + (long long)n_chunks * U) {
      base = x;
      ++b;
    }
  }
}

// Joins the parts of units that several blocks share, in their order along the keys, and writes the rows of
// sequences that hold nothing.  One block per unit; SPREAD: one block per row, its warps on every 8th part.
constexpr int JOIN_WARPS = 8;
template <int D, int DT, int NT, bool SPREAD>
__global__ void __launch_bounds__(JOIN_WARPS * 32) cache_attn_join_kernel(const CacheAttnArgs a, int row_tiles, int grid) {
  constexpr int ROWS = 8 * NT, SLOT = ROWS * (D + 1), PL = D / 32;    // columns per lane
  __shared__ float part_o[SPREAD ? JOIN_WARPS : 1][SPREAD ? D : 1];
  __shared__ float2 part_ml[JOIN_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.Hq / a.c.Hkv, U = a.c.Hkv * row_tiles, R = a.T * G;
  const int unit = SPREAD ? blockIdx.x / ROWS : blockIdx.x;
  const int b = unit / U, u = unit - b * U, h = u / row_tiles, rt = u - h * row_tiles;
  const int len = seq_len(a, b), n_chunks = (len + CHUNK - 1) / CHUNK;
  long long i0 = 0, i1 = -1;
  if (n_chunks > 0) {
    const long long total = chunks_before(a, a.B, U), n = blocks_of(total, grid);
    const long long x0 = chunks_before(a, b, U) + (long long)u * n_chunks;
    i0 = block_of_chunk(total, n, x0);
    i1 = block_of_chunk(total, n, x0 + n_chunks - 1);
    if (i0 == i1) return;               // one block had the whole unit and wrote it
  } else if (__ldg(a.pt.seq_lens + b) > 0 && threadIdx.x == 0 && a.dev_status) {
    *a.dev_status = CACHE_BAD_LEN;      // tokens, but a table without pages
  }
  const float* const ws = reinterpret_cast<const float*>(a.ws);
  const int row0 = SPREAD ? blockIdx.x % ROWS : warp, row_step = SPREAD ? ROWS : JOIN_WARPS;
  for (int row = row0; row < ROWS; row += row_step) {
    const int r = rt * ROWS + row;
    if (r >= R) return;                 // whole warps, and whole blocks where they meet below
    float m = -INFINITY, sum = 0.f, o[PL];
#pragma unroll
    for (int j = 0; j < PL; ++j) o[j] = 0.f;
    // block i0 holds the unit's first chunks in its odd slot, the others in their even one
    for (long long i = i0 + (SPREAD ? warp : 0); i <= i1; i += SPREAD ? JOIN_WARPS : 1) {
      const float* slot = ws + (2 * i + (i == i0 ? 1 : 0)) * SLOT;
      const float z = slot[ROWS * D + row];
      float v[PL];
#pragma unroll
      for (int j = 0; j < PL; ++j) v[j] = slot[row * D + lane * PL + j];
      if (z == -INFINITY) continue;
      const float m2 = z > m ? z : m, keep = m == -INFINITY ? 0.f : ex2_approx(m - m2), f = ex2_approx(z - m2);
      m = m2;
      sum = sum * keep + f;
#pragma unroll
      for (int j = 0; j < PL; ++j) o[j] = o[j] * keep + f * v[j];
    }
    if (SPREAD) {
      if (lane == 0) part_ml[warp] = make_float2(m, sum);
#pragma unroll
      for (int j = 0; j < PL; ++j) part_o[warp][lane * PL + j] = o[j];
      __syncthreads();
      if (warp != 0) return;
      m = -INFINITY;
#pragma unroll
      for (int w = 0; w < JOIN_WARPS; ++w) m = fmaxf(m, part_ml[w].x);
      sum = 0.f;
#pragma unroll
      for (int j = 0; j < PL; ++j) o[j] = 0.f;
#pragma unroll
      for (int w = 0; w < JOIN_WARPS; ++w) {
        const float2 y = part_ml[w];
        if (y.x == -INFINITY && y.y == 0.f) continue;
        const float f = ex2_approx(y.x - m);
        sum += f * y.y;
#pragma unroll
        for (int j = 0; j < PL; ++j) o[j] += f * part_o[w][lane * PL + j];
      }
    }
    const int tq = r / G, hq = h * G + r - tq * G;
    const bool none = sum == 0.f;
    uint16_t* dst = reinterpret_cast<uint16_t*>(a.o) + b * a.os.b + tq * a.os.t + hq * a.os.h + lane * PL;
#pragma unroll
    for (int j = 0; j < PL; j += 2)
      *reinterpret_cast<uint32_t*>(dst + j) = none ? 0u : f32_to_act<DT>(o[j] / sum, o[j + 1] / sum);
    if (lane == 0 && a.lse)
      a.lse[((long long)b * a.Hq + hq) * a.T + tq] = none ? -INFINITY : (m + __log2f(sum)) * 0.6931471805599453f;
  }
}

template <int FMT, int D, int DT, int NT>
cudaError_t launch(const CacheAttnArgs& a, cudaStream_t st) {
  using C = Cfg<FMT, D, NT>;
  const int rows = a.T * (a.Hq / a.c.Hkv), row_tiles = (rows + C::ROWS - 1) / C::ROWS;
  const long long units = (long long)a.B * a.c.Hkv * row_tiles;
  const long long chunks = ((long long)a.pt.max_pages * a.c.page_size + CHUNK - 1) / CHUNK;
  const long long grid = units * chunks < SMS * C::OCC ? units * chunks : SMS * C::OCC;
  if (grid > 0) {
    auto kernel = cache_attn_kernel<FMT, D, DT, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)grid, THREADS, C::SMEM, st>>>(a, row_tiles);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // few units: many parts each, a block per row
  if (units * C::ROWS <= SMS * 8)
    cache_attn_join_kernel<D, DT, NT, true><<<(unsigned)(units * C::ROWS), JOIN_WARPS * 32, 0, st>>>(a, row_tiles, (int)grid);
  else
    cache_attn_join_kernel<D, DT, NT, false><<<(unsigned)units, JOIN_WARPS * 32, 0, st>>>(a, row_tiles, (int)grid);
  return cudaGetLastError();
}

template <int FMT, int D, int DT>
cudaError_t pick(const CacheAttnArgs& a, cudaStream_t st) {
  return a.T * (a.Hq / a.c.Hkv) <= 8 ? launch<FMT, D, DT, 1>(a, st) : launch<FMT, D, DT, 2>(a, st);
}

}  // namespace

size_t cache_attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
  // two slots per block of the largest grid of either format
  const long long rows = (long long)T * ((Hq + Hkv - 1) / Hkv) <= 8 ? 8 : 16;
  const int occ = rows == 8 ? 4 : 2;
  return (size_t)2 * SMS * occ * rows * (D + 1) * 4;
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int format, int D, int dtype, cudaStream_t st) {
  using F = cudaError_t (*)(const CacheAttnArgs&, cudaStream_t);
  static const F f[8] = {pick<0, 64, 0>, pick<0, 64, 1>, pick<0, 128, 0>, pick<0, 128, 1>,
                         pick<1, 64, 0>, pick<1, 64, 1>, pick<1, 128, 0>, pick<1, 128, 1>};
  return f[format * 4 + (D == 128) * 2 + dtype](a, st);
}

}  // namespace bsc
