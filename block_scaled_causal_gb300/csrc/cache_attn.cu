// Attention over the key/value cache.
//
// For the query at position p: x_j = log2(e) scale q . K_j over j <= p, O = sum 2^(x_j - z) V_j with
// z = log2 sum 2^x_j, in one pass over the keys with a running reference m (weights 2^(x - m)).
//
// What bounds it.  A decode step reads every K and V byte once for the few query rows that share a KV
// head, so it is bound by memory if the decoding of elements keeps up: at D = 128 a token of one head is
// 136 bytes in 4 bits, so a full-rate stream leaves about 23 warp instructions per token and SM to decode
// 256 elements and do both products.  The layout below spends 21 (8 of them conversions and fp16 scalings), but 12
// warps per SM issue 2.2 per clock, so 4 bits run at half the copy rate (32 ragged sequences up to 16K, Hkv = 4:
// 34 us for 116 MB) and 8 bits, with twice the bytes per key, at all of it (16 x 16K, Hkv = 16: 162 to 165 us for 1.1
// GB).  Short work is bound by latency: 5.7 us for one sequence of 500 tokens, 13.4 us for one of 32K.
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
// to 2^13 or 2^11.  A key with a scale outside of that (or a NaN block, or, in tiles with keys that some row does
// not see, an E4M3 NaN code in V) takes the scalar path below in fp32; keys are sorted one by one, by their own
// bytes, so a row never depends on a key it cannot see.
// Scale byte 0 (a zero block, or a maximum under 2^-118) counts as zero.
//
// Roundings.  Q is scaled per row by a power of two to [2^14, 2^15) and held in fp16: exact for 16-bit
// inputs down to 2^-29 of the row's maximum.  Scores, weights' sums and O are fp32.  Weights are rounded to
// fp16 for the second product (2^-11 relative at most, and each weight on its own; the output's own rounding is
// 2^-8 or 2^-11 of the result), around 2^8 at the reference so that only weights under 2^-22 of the largest lose
// relative precision.
//
// Work.  A warp takes 32 keys at a time through its own ring of shared-memory stages (cp.async, 16
// bytes per lane, rows permuted so that both fragments read without bank conflicts); a block is 4 warps on
// neighbouring 32-key tiles (a chunk, 128 keys).  The chunks of all (sequence, KV head, row tile) units form one
// list, which the blocks split into equal runs: a long sequence spreads over the card and ragged batches stay
// balanced, whatever the lengths, which only the device knows.  A run that covers a unit writes O; one
// that covers part of it writes (O, log-sum-exp) to the workspace, two slots per block at most, and a second
// kernel joins them in order.  Short tables take a cluster per unit instead (plan() has the rule and both sides).
#include <atomic>
#include <cooperative_groups.h>

#include "cache.cuh"

namespace bsc {
namespace {

namespace cg = cooperative_groups;

constexpr int KT = 32, WARPS = 4, CHUNK = KT * WARPS, THREADS = WARPS * 32;
constexpr int SMS = 152;
constexpr int MIN_CHUNKS = 2;   // chunks a block takes at least, once there is one block per SM (see Share)
constexpr float SLACK = 4.f;    // a reference moves when a score passes it by this much (log2)
constexpr float LIFT = 8.f;     // a reference m gives weights 2^(x + r), r = LIFT - m
constexpr float UNSET = 3e38f;  // r of a row without a score yet: 2^(-inf + r) = 0, and any score moves it
constexpr float FAR = 1048576.f;   // |r| from which products are rounded first (tile_work): a unit is 1/8 there

// Blocks per SM.  Tiles of 8 rows: 3 blocks leave 168 registers, 4 leave 128 and fewer loads and conversions in flight.
// D = 128, G = 4, 4 bits, 4 blocks / 3: 64 x 6000 keys 50.3 / 48.1 us, 16 x 6000 20.2 / 19.1; but one sequence
// of 32K 12.7 / 13.7, whose 1024 chunks divide worse by 456.  In 8 bits shared memory holds 3 at most.  Larger tiles
// need up to 255 registers, and those of 32 rows at D = 128 spill 24 to 60 bytes beside.
constexpr int blocks_per_sm(int tile) { return tile == 8 ? 3 : 2; }

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
  // From four row tiles on, Q's fragments do not fit beside O in registers: shared memory, [tile][k-step][lane],
  // then c and lim of every row.
  static constexpr bool QS = NT >= 4;
  static constexpr int QF = QS ? NT * KS * 32 * 8 : 0;
  static constexpr int QBYTES = QS ? QF + ROWS * 8 : 0;
  static constexpr int MERGE = WARPS * ROWS * (D + 4) * 4 + WARPS * ROWS * 8;
  static constexpr int JOINED = MERGE + ROWS * D * 4 + ROWS * 8;   // and the block's own part, in the cluster form
  static constexpr int SMEM = RING + QBYTES > JOINED ? RING + QBYTES : JOINED;
  static constexpr int OCC = blocks_per_sm(ROWS);
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
// The same with nothing to add to.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

// Whether a row of E4M3 in shared memory has a NaN code (0x7F under the sign).
template <int RB>
__device__ __forceinline__ bool row_has_nan(const uint8_t* rows, int k) {
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < RB / 16; ++i) {
    const uint4 w = *reinterpret_cast<const uint4*>(rows + piece_at<RB>(k, i));
    any |= ((w.x & 0x7F7F7F7Fu) + 0x01010101u) | ((w.y & 0x7F7F7F7Fu) + 0x01010101u) |
           ((w.z & 0x7F7F7F7Fu) + 0x01010101u) | ((w.w & 0x7F7F7F7Fu) + 0x01010101u);
  }
  return (any & 0x80808080u) != 0u;
}

// 2^(byte - 127 + OFF) in fp16 for bytes in range, 0 for byte 0: in both halves / for two bytes.
template <class C>
__device__ __forceinline__ uint32_t scale_f16(uint32_t byte) {
  return (uint32_t)__viaddmax_s32_relu((int)byte, -(int)C::SUB, 0) * 0x04000400u;
}
template <class C>
__device__ __forceinline__ uint32_t scales_f16x2(uint32_t lo, uint32_t hi) {
  return __viaddmax_s16x2_relu(lo | hi << 16, (0x10000u - C::SUB) * 0x10001u, 0u) << 10;
}

// The elements of the 32-bit word at byte `at` of key k's row in shared memory, each as the fp32 value it stands
// for times 2^OFF.
template <int FMT, class C>
__device__ __forceinline__ void word_values(const uint8_t* rows, int k, int at, float scale, float (&v)[FMT == CACHE_FP4 ? 8 : 4]) {
  constexpr int N = FMT == CACHE_FP4 ? 4 : 2;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(rows + piece_at<C::RB>(k, at >> 4) + (at & 15));
  uint32_t h[4];
  if (FMT == CACHE_FP4) e2m1x8_to_f16(w, h);
  else e4m3x4_to_f16(w, h[0], h[1]);
  const float f = (float)(1 << C::OFF);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float2 y = f16x2_to_f32(h[i]);
    v[2 * i] = y.x * scale * f;
    v[2 * i + 1] = y.y * scale * f;
  }
}
// Whether a reference is one whose scores' products are rounded before they are compared (tile_work).
__device__ __forceinline__ bool is_far(float r) { return fabsf(r) >= FAR && r != UNSET; }
// Keeps the loads of a rarely taken loop from being gathered in registers ahead of it.
__device__ __forceinline__ void in_order() { asm volatile("" ::: "memory"); }

__device__ __forceinline__ uint32_t interleave_low(uint32_t x, uint32_t y) {    // low nibbles of x and y, byte by byte
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xCA;" : "=r"(r) : "r"(0x0F0F0F0Fu), "r"(x), "r"(y << 4));
  return r;
}
__device__ __forceinline__ uint32_t interleave_high(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xCA;" : "=r"(r) : "r"(0x0F0F0F0Fu), "r"(x >> 4), "r"(y));
  return r;
}
// Address `n` 16-byte units past row `row` of page `page`.
__device__ __forceinline__ const uint8_t* unit_at(const uint8_t* pool, uint32_t page_units, uint32_t page, uint32_t n) {
  return pool + ((unsigned long long)page * page_units + n) * 16;
}

// The list of chunks.  Sequence b has ceil(len_b / CHUNK) chunks per unit and U = Hkv * (row tiles) units; the host
// has checked that the longest list the page table allows has fewer than 2^31 chunks.
__device__ __forceinline__ int seq_len(const CacheAttnArgs& a, int b) {
  const int cap = a.pt.max_pages * a.c.page_size;   // < 2^31
  return min(max(__ldca(a.pt.seq_lens + b), 0), cap);
}
__device__ __forceinline__ uint32_t chunks_of(const CacheAttnArgs& a, int b, int U) {
  return b < a.B ? (uint32_t)((seq_len(a, b) + (CHUNK - 1)) / CHUNK) * U : 0u;
}
// Chunks of all sequences, and of those before b.  Whole warps call it.
__device__ __forceinline__ uint32_t chunks_of_all(const CacheAttnArgs& a, int U, int b, uint32_t& before) {
  uint32_t all = 0, first = 0;
  for (int i = threadIdx.x & 31; i < a.B; i += 32) {
    const uint32_t n = chunks_of(a, i, U);
    all += n;
    if (i < b) first += n;
  }
  before = __reduce_add_sync(0xFFFFFFFFu, first);
  return __reduce_add_sync(0xFFFFFFFFu, all);
}
// The sequence that chunk x of the list belongs to, and its first chunk.
__device__ __forceinline__ int seq_of_chunk(const CacheAttnArgs& a, uint32_t x, int U, uint32_t& base) {
  const int lane = threadIdx.x & 31;
  base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const uint32_t n = chunks_of(a, b0 + lane, U);
    uint32_t s = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, base + s > x);
    if (hit) {
      const int l = __ffs(hit) - 1;
      base += __shfl_sync(0xFFFFFFFFu, s - n, l);
      return b0 + l;
    }
    base += __shfl_sync(0xFFFFFFFFu, s, 31);
  }
  return a.B;   // past the list
}
// How the list is shared: n blocks, the first `more` of them with each + 1 chunks, the others with `each`.
// A block costs a prologue and a part to join, so a block per chunk is taken only while there are fewer chunks than
// SMs, and then MIN_CHUNKS chunks each until the grid is full (2 chunks at least: one sequence of 32K 12.7 us; 3 to 6:
// 14.5 and more).
struct Share {
  uint32_t n, each, more;
  __device__ __forceinline__ Share(uint32_t total, uint32_t grid) {
    n = total < SMS ? total : min(max(total / MIN_CHUNKS, (uint32_t)SMS), grid);
    n = min(n, grid);
    each = n ? total / n : 0;
    more = total - n * each;
  }
  __device__ __forceinline__ uint32_t first(uint32_t i) const { return i * each + min(i, more); }   // of block i
  __device__ __forceinline__ uint32_t block(uint32_t x) const {                                       // that has chunk x
    const uint32_t big = more * (each + 1);
    return x < big ? x / (each + 1) : more + (x - big) / each;
  }
};

// Where the rows of "sequence" b and query head 0 start in an activation, and in lse.
__device__ __forceinline__ long long rows_at(const CacheAttnArgs& a, const RowStrides& s, int b) {
  if (a.sel_H == 0) return b * s.b;
  const int x = b / a.sel_H, h = b - x * a.sel_H, bb = x / a.sel_T, t = x - bb * a.sel_T;
  return bb * s.b + t * s.t + (long long)h * a.Hq * s.h;
}
__device__ __forceinline__ long long lse_at(const CacheAttnArgs& a, int b, int hq, int tq) {
  if (a.sel_H == 0) return ((long long)b * a.Hq + hq) * a.T + tq;
  const int x = b / a.sel_H, h = b - x * a.sel_H, bb = x / a.sel_T, t = x - bb * a.sel_T;
  return (((long long)bb * a.sel_H + h) * a.Hq + hq) * a.sel_T + t;
}

// A workspace slot: ROWS x D of O, then ROWS log-sum-exps (log2).
template <class C, int D>
constexpr int slot_floats() { return C::ROWS * (D + 1); }

// A lane's place in a tile's rows: offsets in a stage of its K run, its V runs (keys t and t + 4), its scales.
struct Place {
  int lane, g, t, ko, vo0, vo4, kso, vso;
};
// One tile of 32 keys: scores, weights, and both products into acc, l and the references.  SPECIAL: some keys
// are left out (`gone`), need the scalar path (`odd`) or are hidden from some row, or some row's reference is `far`; a
// plain tile's code has none of that, and returns false with nothing changed but `far` where a reference gets there.  Both
// add the same things in the same order for the keys that a row sees.
template <int FMT, int D, int NT, bool SPECIAL, class QFrag, class COf, class LimOf>
__device__ __forceinline__ bool tile_work(uint8_t* const stage, const int k0, const uint32_t gone, const uint32_t odd,
                                          const Place& at, float (&acc)[NT][D / 16][4], float (&l)[NT][2],
                                          float (&ref)[NT][2], bool& far, QFrag q_frag, COf c_of, LimOf lim_of) {
  using C = Cfg<FMT, D, NT>;
  constexpr int RB = C::RB, NB = C::NB;
  constexpr int LB = C::KE * RB / D, VB = C::VE * RB / D;   // bytes of a lane's K run and of its V run
  const int lane = at.lane, g = at.g, t = at.t, ko = at.ko, vo0 = at.vo0, vo4 = at.vo4, kso = at.kso, vso = at.vso;
  uint8_t* const vrows = stage + KT * RB;
  uint8_t* const ksc = stage + 2 * KT * RB;
  uint8_t* const vsc = ksc + KT * NB;
  const uint32_t left_out = gone | odd;

  // ---- scores ----
  float s[NT][2][4];
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    const uint32_t sa = scale_f16<C>(stage[kso + mt * 16 * NB]), sb = scale_f16<C>(stage[kso + (mt * 16 + 8) * NB]);
    const uint8_t* const ra = stage + ko + mt * 16 * RB;
    const uint8_t* const rb = ra + 8 * RB;
    uint32_t wa[LB / 4], wb[LB / 4];
    if (LB == 8) {
      const uint2 ua = *reinterpret_cast<const uint2*>(ra), ub = *reinterpret_cast<const uint2*>(rb);
      wa[0] = ua.x; wa[1] = ua.y; wb[0] = ub.x; wb[1] = ub.y;
    } else {
#pragma unroll
      for (int i = 0; i < LB / 16; ++i) {   // the run's second piece is the first's neighbour: bit 4 of the offset
        const int flip = i ? ((ko & 16) ? -16 : 16) : 0;
        const uint4 ua = *reinterpret_cast<const uint4*>(ra + flip), ub = *reinterpret_cast<const uint4*>(rb + flip);
        wa[4 * i] = ua.x; wa[4 * i + 1] = ua.y; wa[4 * i + 2] = ua.z; wa[4 * i + 3] = ua.w;
        wb[4 * i] = ub.x; wb[4 * i + 1] = ub.y; wb[4 * i + 2] = ub.z; wb[4 * i + 3] = ub.w;
      }
    }
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
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 qb = q_frag(nt, 2 * i + j);
            if (2 * i + j == 0) mma_f16_first(s[nt][mt], a0, a1, a2, a3, qb.x, qb.y);
            else mma_f16(s[nt][mt], a0, a1, a2, a3, qb.x, qb.y);
          }
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
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 qb = q_frag(nt, i);
          if (i == 0) mma_f16_first(s[nt][mt], a0, a1, a2, a3, qb.x, qb.y);
          else mma_f16(s[nt][mt], a0, a1, a2, a3, qb.x, qb.y);
        }
      }
    }
  }

  // ---- scores of the odd keys, one at a time in fp32; then the masks ----
  if constexpr (SPECIAL) for (uint32_t rest = odd; rest; rest &= rest - 1) {
    const int k = __ffs(rest) - 1;
    float dot[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) dot[nt] = 0.f;
    const float sc = scale_value(ksc[k * NB + t * C::KE / 32]);
#pragma unroll
    for (int w = 0; w < LB / 4; ++w) {
      constexpr int PW = FMT == CACHE_FP4 ? 2 : 1;      // k-steps per word
      float e[4 * PW];
      word_values<FMT, C>(stage, k, t * LB + 4 * w, sc, e);
#pragma unroll
      for (int j = 0; j < PW; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 qf = q_frag(nt, w * PW + j);
          const float2 qa = f16x2_to_f32(qf.x), qb = f16x2_to_f32(qf.y);
          dot[nt] += qa.x * e[4 * j] + qa.y * e[4 * j + 1] + qb.x * e[4 * j + 2] + qb.y * e[4 * j + 3];
        }
      in_order();
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
  if constexpr (SPECIAL) {
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
            if (away || k0 + k >= lim_of(nt, j)) s[nt][mt][2 * half + j] = -INFINITY;
      }
  }

  // ---- the reference: moved for a row when one of its own scores is SLACK above it ----
  float top[NT][2];
  bool climb = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      top[nt][j] = __fmul_rn(c_of(nt, j), fmaxf(fmaxf(s[nt][0][j], s[nt][0][2 + j]), fmaxf(s[nt][1][j], s[nt][1][2 + j])));
      climb |= top[nt][j] + ref[nt][j] > LIFT + SLACK;
    }
  if (__any_sync(0xFFFFFFFFu, climb)) {
    bool away = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mx = top[nt][j];
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
        // from here on the new reference; mx + it <= LIFT also where bits are lost
        top[nt][j] = mx + ref[nt][j] > LIFT + SLACK ? __fsub_rd(LIFT, mx) : ref[nt][j];
        away |= is_far(top[nt][j]);
      }
    far = __any_sync(0xFFFFFFFFu, away);
    if (!SPECIAL && far) return false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (top[nt][j] != ref[nt][j]) {
          const float keep = ex2_approx(top[nt][j] - ref[nt][j]);   // 0 from UNSET
          ref[nt][j] = top[nt][j];
          l[nt][j] *= keep;
#pragma unroll
          for (int i = 0; i < C::MT; ++i) {
            acc[nt][i][j] *= keep;
            acc[nt][i][2 + j] *= keep;
          }
        }
  }

  // ---- weights ----
  // A reference holds its row's largest product as rounded, which is up to half a unit off.  Far out, where a unit is many
  // powers of two, that alone would take 2^(s c - round(s c)) out of fp16's range: there all products are rounded first.
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool rounded = SPECIAL && is_far(ref[nt][j]);
      const float c = rounded ? 1.f : c_of(nt, j), r = rounded ? 0.f : ref[nt][j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float& x = s[nt][i >> 1][2 * (i & 1) + j];
        if (rounded) x = __fadd_rn(__fmul_rn(x, c_of(nt, j)), ref[nt][j]);
        x = ex2_approx(fmaf(x, c, r));
        l[nt][j] += x;
      }
    }

  // ---- odd keys' part of O in fp32, only for rows that see them; then they and absent keys become zeros ----
  if constexpr (SPECIAL) if (left_out != 0u) {
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
        const bool sees0 = k0 + k < lim_of(nt, 0), sees1 = k0 + k < lim_of(nt, 1);
#pragma unroll
        for (int w = 0; w < VB / 4; ++w) {
          constexpr int PW = FMT == CACHE_FP4 ? 4 : 2;  // 16-row tiles per word
          float e[2 * PW];
          word_values<FMT, C>(vrows, k, g * VB + 4 * w, sc, e);
#pragma unroll
          for (int i = 0; i < PW; ++i) {
            if (sees0) {
              acc[nt][w * PW + i][0] += p[0] * e[2 * i];
              acc[nt][w * PW + i][2] += p[0] * e[2 * i + 1];
            }
            if (sees1) {
              acc[nt][w * PW + i][1] += p[1] * e[2 * i];
              acc[nt][w * PW + i][3] += p[1] * e[2 * i + 1];
            }
          }
          in_order();
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
    const uint8_t* const sv = stage + vso + mt * 16 * NB;
    const uint32_t s01 = scales_f16x2<C>(sv[0], sv[4 * NB]), s23 = scales_f16x2<C>(sv[8 * NB], sv[12 * NB]);
    uint32_t v[4][VB / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* src = vrows + (i & 1 ? vo4 : vo0) + (i >> 1) * 8 * RB + mt * 16 * RB;
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
        e2m1x8_to_f16(interleave_low(v[0][w], v[1][w]), e01);
        e2m1x8_to_f16(interleave_high(v[0][w], v[1][w]), o01);
        e2m1x8_to_f16(interleave_low(v[2][w], v[3][w]), e23);
        e2m1x8_to_f16(interleave_high(v[2][w], v[3][w]), o23);
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
  return true;
}

template <int FMT, int D, int NT, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, Cfg<FMT, D, NT>::OCC) cache_attn_kernel(const CacheAttnArgs a, int row_tiles,
                                                                                    int cluster_blocks) {
  const int cs = CLUSTER ? cluster_blocks : 0;
  using C = Cfg<FMT, D, NT>;
  constexpr int RB = C::RB, NB = C::NB;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int G = a.Hq / a.c.Hkv, U = a.c.Hkv * row_tiles, page_size = a.c.page_size;
  const int R = a.T * G;

  wait_for_last_kernel();
  // the joining kernel comes next in the list form; not before the wait, as it reads the lengths ahead of its own
  if (!CLUSTER || gridDim.x <= EARLY_BLOCKS) next_kernel_may_start();
  // List form (cs = 0): this block's run of the list.  Cluster form: unit blockIdx.x / cs, every cs-th chunk.
  uint32_t base = 0, x = 0, x_end = 1;
  const int unit = cs ? blockIdx.x / cs : 0, rank = cs ? blockIdx.x - unit * cs : 0;
  int b = cs ? unit / U : 0;
  if (cs == 0) {
    const Share share(chunks_of_all(a, U, 0, base), gridDim.x);
    if (blockIdx.x >= share.n) return;
    x = share.first(blockIdx.x);
    x_end = share.first(blockIdx.x + 1);
    b = seq_of_chunk(a, x, U, base);
  }

  // ---- what a lane's place fixes ----
  uint8_t* const ring = smem + warp * C::STAGES * C::STAGE;
  const uint32_t ring_s = smem_u32(ring);
  constexpr int PR = RB / 16, RPC = 32 / PR;      // pieces per row, rows per copy instruction
  const int to0 = piece_at<RB>(lane / PR, lane % PR), to1 = piece_at<RB>(lane / PR + RPC, lane % PR) - RPC * RB;
  constexpr int LB = C::KE * RB / D;              // bytes of a lane's K run: 8, 16 or 32
  constexpr int VB = C::VE * RB / D;              // of its V run: 4, 8 or 16
  const Place place{lane, g, t, piece_at<RB>(key_of_row(g), t * LB / 16) + t * LB % 16,
                    piece_at<RB>(t, g * VB / 16) + g * VB % 16, piece_at<RB>(t + 4, g * VB / 16) + g * VB % 16,
                    2 * KT * RB + key_of_row(g) * NB + t * C::KE / 32,
                    2 * KT * RB + KT * NB + t * NB + g * C::VE / 32};
  // pages of a multiple of 32 tokens: a tile lies in one page and is copied as a whole; else 16 keys at a time
  const bool one_page = page_size % KT == 0;
  const int sc_lanes = one_page ? 2 * NB : NB;    // pieces of scales per pool and copy
  const bool sc_v = lane >= sc_lanes;
  const int sc_p = sc_v ? lane - sc_lanes : lane;
  const uint8_t* const sc_pool = sc_v ? a.c.v_sc : a.c.k_sc;
  const uint32_t sc_units = (uint32_t)((sc_v ? a.c.v_sc_ps : a.c.k_sc_ps) >> 4);
  const uint32_t k_units = (uint32_t)(a.c.k_ps >> 4), v_units = (uint32_t)(a.c.v_ps >> 4);
  const uint32_t sc_to = 2 * KT * RB + (sc_v ? KT * NB : 0) + sc_p * 16;

  while (x < x_end) {
    // ---- the next piece: chunks c0, c0 + step, ... (count of them) of unit (b, h, rt) ----
    const int len = seq_len(a, b), n_chunks = (len + CHUNK - 1) / CHUNK;
    int u = unit - b * U, c0 = rank, count = n_chunks > rank ? (n_chunks - rank + cs - 1) / max(cs, 1) : 0;
    const int step = cs ? cs : 1;
    if (cs == 0) {
      if (n_chunks == 0) {
        ++b;
        continue;
      }
      u = (int)((x - base) / (uint32_t)n_chunks);
      c0 = (int)(x - base) - u * n_chunks;
      count = min(n_chunks - c0, (int)(x_end - x));
    }
    const int h = u / row_tiles, rt = u - h * row_tiles;
    const int raw_len = max(__ldca(a.pt.seq_lens + b), 0);
    const int n_new = a.new_lens ? min(max(__ldca(a.new_lens + b), 0), a.T) : a.T;
    if (raw_len > len && tid == 0) report(a.dev_status, CACHE_BAD_LEN);

    // ---- Q's loads start: lane (g, t) has elements KE t .. KE t + KE - 1 of query row g of each 8-row tile ----
    // (of all tiles, or each warp of its own where Q goes to shared memory)
    constexpr int NQ = C::QS ? NT / WARPS : NT;
    const int nt0 = C::QS ? warp * NQ : 0;
    uint4 q_in[NQ][C::KE / 8];
#pragma unroll
    for (int nt = 0; nt < NQ; ++nt) {
      const int r = rt * C::ROWS + (nt0 + nt) * 8 + g, tq = r / G, hq = h * G + r - tq * G;
      const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + rows_at(a, a.qs, b) + tq * a.qs.t + hq * a.qs.h + t * C::KE;
#pragma unroll
      for (int i = 0; i < C::KE / 8; ++i)
        q_in[nt][i] = r < R ? __ldca(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
    }

    // ---- the warp's tiles: keys (c0 + i step) CHUNK + warp KT + [0, KT); only the last can be past the end ----
    const int k_first = c0 * CHUNK + warp * KT, k_step = step * CHUNK;
    const int n_tiles = count - (count > 0 && k_first + (count - 1) * k_step >= len);

    // page ids: lane 2 i + j has the 16-key group j of tile (window start) + i, for 16 tiles at a time
    int w_page = -1;
    uint32_t w_row = 0, present = 0;      // row in the page's [Hkv][page_size]; bit l: lane l's group is there
    int st_in = 0, st_out = 0;
    uint32_t there[C::STAGES] = {};       // the two `present` bits of the tiles in flight, oldest first
    auto advance = [&](int tile) {        // copies of tile `tile` start; whole warps call it
      uint32_t bits = 0;
      if (tile < n_tiles) {
        if ((tile & 15) == 0) {
          const int i = tile + (lane >> 1), key = k_first + i * k_step + (lane & 1) * 16;
          w_page = -1;
          if (i < n_tiles && key < len) {
            const int lp = key / page_size;
            w_row = (uint32_t)(h * page_size + key - lp * page_size);
            w_page = __ldca(a.pt.table + b * a.pt.stride + lp);
            if (w_page < 0 || w_page >= a.c.num_pages) {
              w_page = -1;
              report(a.dev_status, CACHE_BAD_PAGE);
            }
          }
          present = __ballot_sync(0xFFFFFFFFu, w_page >= 0);
        }
        const int slot = (tile & 15) * 2;
        bits = (present >> slot) & 3u;
        const uint32_t dst = ring_s + st_in * C::STAGE;
        if (one_page) {
          const uint32_t page = __shfl_sync(0xFFFFFFFFu, (uint32_t)w_page, slot), row = __shfl_sync(0xFFFFFFFFu, w_row, slot);
          if (bits) {
            const uint8_t* const ks = unit_at(a.c.k, k_units, page, row * PR + lane);
            const uint8_t* const vs = unit_at(a.c.v, v_units, page, row * PR + lane);
#pragma unroll
            for (int i = 0; i < PR; ++i) {
              const int to = (i & 1 ? to1 : to0) + i * RPC * RB;
              cp16(dst + to, ks + i * 512);
              cp16(dst + KT * RB + to, vs + i * 512);
            }
            if (lane < 4 * NB) cp16(dst + sc_to, unit_at(sc_pool, sc_units, page, (row >> 4) * NB + sc_p));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t page = __shfl_sync(0xFFFFFFFFu, (uint32_t)w_page, slot + j);
            const uint32_t row = __shfl_sync(0xFFFFFFFFu, w_row, slot + j);
            if ((bits >> j) & 1u) {
              const uint8_t* const ks = unit_at(a.c.k, k_units, page, row * PR + lane);
              const uint8_t* const vs = unit_at(a.c.v, v_units, page, row * PR + lane);
#pragma unroll
              for (int i = 0; i < PR / 2; ++i) {
                const int to = (i & 1 ? to1 : to0) + i * RPC * RB + j * 16 * RB;
                cp16(dst + to, ks + i * 512);
                cp16(dst + KT * RB + to, vs + i * 512);
              }
              if (lane < 2 * NB)
                cp16(dst + sc_to + j * 16 * NB, unit_at(sc_pool, sc_units, page, (row >> 4) * NB + sc_p));
            }
          }
        }
      }
      cp_commit();
      st_in = st_in + 1 == C::STAGES ? 0 : st_in + 1;
#pragma unroll
      for (int i = 0; i + 1 < C::STAGES; ++i) there[i] = there[i + 1];
      there[C::STAGES - 1] = bits;
    };
#pragma unroll
    for (int i = 0; i < C::STAGES - 1; ++i) advance(i);

    // ---- Q scaled and in fp16 ----
    uint32_t q[NQ][C::KS][2];
    float c_own[NQ][2];        // score -> log2 units, rows 2t and 2t + 1
    int lim_own[NQ][2];        // keys j < lim are visible; rows that see nothing or do not exist: all
    int min_lim = len;
    uint2* const qs = reinterpret_cast<uint2*>(smem + C::RING);
    float* const c_all = reinterpret_cast<float*>(smem + C::RING + C::QF);
    int* const lims = reinterpret_cast<int*>(c_all + C::ROWS);
#pragma unroll
    for (int nt = 0; nt < NQ; ++nt) {
      const int r = rt * C::ROWS + (nt0 + nt) * 8 + g, tq = r / G;
      float mx = 0.f;
      float f[C::KE];
#pragma unroll
      for (int i = 0; i < C::KE / 8; ++i) {
        const uint32_t w[4] = {q_in[nt][i].x, q_in[nt][i].y, q_in[nt][i].z, q_in[nt][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 p = act_to_f32(w[j], a.fp16);
          f[8 * i + 2 * j] = p.x;
          f[8 * i + 2 * j + 1] = p.y;
        }
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
      // above 0, so that -inf stays -inf; in fp32's subnormals it is off by 2^-150 at most, scores then by under 2^-22
      const float cg = fmaxf(a.scale_log2e * __uint_as_float((uint32_t)(ex_back + 127) << 23), 1.4e-45f);
      // first key past the row: position raw_len - n_new + tq sees itself
      int lg = len;
      if (r < R && tq < n_new) {
        const long long past = (long long)raw_len - n_new + tq + 1;
        if (past > 0 && past < len) lg = (int)past;
      }
      min_lim = min(min_lim, lg);
      if (C::QS) {
#pragma unroll
        for (int i = 0; i < C::KS; ++i) qs[((nt0 + nt) * C::KS + i) * 32 + lane] = make_uint2(q[nt][i][0], q[nt][i][1]);
        if (t == 0) {
          c_all[(nt0 + nt) * 8 + g] = cg;
          lims[(nt0 + nt) * 8 + g] = lg;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          c_own[nt][j] = __shfl_sync(0xFFFFFFFFu, cg, (2 * t + j) * 4);
          lim_own[nt][j] = __shfl_sync(0xFFFFFFFFu, lg, (2 * t + j) * 4);
        }
      }
    }
    if (C::QS) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < C::ROWS; i += 32) min_lim = min(min_lim, lims[i + lane]);
    }
    min_lim = __reduce_min_sync(0xFFFFFFFFu, min_lim);
    auto q_frag = [&](int nt, int i) {
      return C::QS ? qs[(nt * C::KS + i) * 32 + lane] : make_uint2(q[C::QS ? 0 : nt][i][0], q[C::QS ? 0 : nt][i][1]);
    };
    auto c_of = [&](int nt, int j) { return C::QS ? c_all[nt * 8 + 2 * t + j] : c_own[C::QS ? 0 : nt][j]; };
    auto lim_of = [&](int nt, int j) { return C::QS ? lims[nt * 8 + 2 * t + j] : lim_own[C::QS ? 0 : nt][j]; };

    float acc[NT][C::MT][4], l[NT][2], ref[NT][2];   // weights are 2^(c s + ref)
    bool far = false;                                // some row's reference is FAR or more
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < C::MT; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
      l[nt][0] = l[nt][1] = 0.f;
      ref[nt][0] = ref[nt][1] = UNSET;
    }

    for (int tile = 0; tile < n_tiles; ++tile) {
      cp_wait<C::STAGES - 2>();
      __syncwarp();
      advance(tile + C::STAGES - 1);

      uint8_t* const stage = ring + st_out * C::STAGE;
      st_out = st_out + 1 == C::STAGES ? 0 : st_out + 1;
      const uint8_t* const ksc = stage + 2 * KT * RB;
      const uint8_t* const vsc = ksc + KT * NB;
      const int k0 = k_first + tile * k_step;

      // ---- which keys the matrix path leaves out: `gone` (past the sequence, no page), `odd` (scales) ----
      const int valid = len - k0;
      const uint32_t gone = (valid < KT ? 0xFFFFFFFFu << valid : 0u) | (there[0] & 1 ? 0u : 0xFFFFu) |
                            (there[0] & 2 ? 0u : 0xFFFF0000u);
      bool ok;
      if (NB == 4) {
        ok = scales_in_range<C>(reinterpret_cast<const uint32_t*>(ksc)[lane]) &
             scales_in_range<C>(reinterpret_cast<const uint32_t*>(vsc)[lane]);
      } else {
        ok = scales_in_range<C>(reinterpret_cast<const uint16_t*>(ksc)[lane] |
                                (uint32_t)reinterpret_cast<const uint16_t*>(vsc)[lane] << 16);
      }
      uint32_t odd = __ballot_sync(0xFFFFFFFFu, !ok) & ~gone;
      const bool masked = k0 + KT > min_lim;
      if ((gone | odd) != 0u || masked || far ||
          !tile_work<FMT, D, NT, false>(stage, k0, 0u, 0u, place, acc, l, ref, far, q_frag, c_of, lim_of)) {
        // a hidden key weighs 0, and 0 * NaN is NaN: where rows see different keys, NaN codes of V leave the matrix path too
        if (FMT == CACHE_FP8 && masked) odd |= __ballot_sync(0xFFFFFFFFu, row_has_nan<RB>(stage + KT * RB, lane)) & ~gone;
        tile_work<FMT, D, NT, true>(stage, k0, gone, odd, place, acc, l, ref, far, q_frag, c_of, lim_of);
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
        if (g == 0) ml[warp * C::ROWS + row] = make_float2(-ref[nt][j], sum);
        float* const dst = mo + (warp * C::ROWS + row) * (D + 4) + g * C::VE;
#pragma unroll
        for (int i = 0; i < C::MT; ++i) *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(acc[nt][i][j], acc[nt][i][2 + j]);
      }
    __syncthreads();
    const bool whole = cs == 1 || (cs == 0 && count == n_chunks);
    float* const slot = reinterpret_cast<float*>(a.ws) +
                        (2LL * blockIdx.x + (c0 == 0)) * slot_floats<C, D>();
    constexpr int LPR = D / 8;                 // threads per row, 8 columns each
    float* const co = reinterpret_cast<float*>(smem + C::MERGE);        // cluster form: [row][D], then (ref, sum) by row
    float2* const cl = reinterpret_cast<float2*>(co + C::ROWS * D);
    // Eight columns of a row from the weighted sum o, the sum of weights and their reference: O and its log-sum-exp
    // where the unit is complete, a part of it to the workspace otherwise.
    auto emit = [&](int row, int d, float (&o)[8], float mx, float sum) {
      const int r = rt * C::ROWS + row, tq = r / G;
      const bool sees = tq < n_new && (long long)raw_len - n_new + tq >= 0;
      const bool none = !sees || sum == 0.f;
      const float inv = none ? 0.f : __fdividef(1.f, sum) * (1.f / (1 << C::OFF));
      const float z = none ? -INFINITY : mx + __log2f(sum);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = none ? 0.f : o[j] * inv;
      if (whole || cs) {
        const int hq = h * G + r - tq * G;
        uint16_t* dst = reinterpret_cast<uint16_t*>(a.o) + rows_at(a, a.os, b) + tq * a.os.t + hq * a.os.h + d;
        *reinterpret_cast<uint4*>(dst) = make_uint4(f32_to_act(o[0], o[1], a.fp16), f32_to_act(o[2], o[3], a.fp16),
                                                    f32_to_act(o[4], o[5], a.fp16), f32_to_act(o[6], o[7], a.fp16));
        if (d == 0 && a.lse) a.lse[lse_at(a, b, hq, tq)] = z * 0.6931471805599453f;
      } else {
        float4* dst = reinterpret_cast<float4*>(slot + row * D + d);
        dst[0] = make_float4(o[0], o[1], o[2], o[3]);
        dst[1] = make_float4(o[4], o[5], o[6], o[7]);
        if (d == 0) slot[C::ROWS * D + row] = z;
      }
    };
    for (int i = tid; i < C::ROWS * LPR; i += THREADS) {
      const int row = i / LPR, d = (i % LPR) * 8, r = rt * C::ROWS + row;
      if (r >= R) continue;
      float mx = -UNSET;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, ml[w * C::ROWS + row].x);
      float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float2 part = ml[w * C::ROWS + row];     // (-UNSET, 0) where the warp had no key: weighs 0
        const float f = ex2_approx(part.x - mx);
        sum += f * part.y;
        const float4* src = reinterpret_cast<const float4*>(mo + (w * C::ROWS + row) * (D + 4) + d);
        const float4 y0 = src[0], y1 = src[1];
        o[0] += f * y0.x; o[1] += f * y0.y; o[2] += f * y0.z; o[3] += f * y0.w;
        o[4] += f * y1.x; o[5] += f * y1.y; o[6] += f * y1.z; o[7] += f * y1.w;
      }
      if (cs > 1) {                            // this block's part, for the cluster
        float4* const dst = reinterpret_cast<float4*>(co + row * D + d);
        dst[0] = make_float4(o[0], o[1], o[2], o[3]);
        dst[1] = make_float4(o[4], o[5], o[6], o[7]);
        if (d == 0) cl[row] = make_float2(mx, sum);
      } else {
        emit(row, d, o, mx, sum);
      }
    }
    if constexpr (CLUSTER) if (cs > 1) {
      // ---- the cluster's parts, each block taking every cs-th row from all blocks' shared memory ----
      cg::cluster_group cluster = cg::this_cluster();
      cluster.sync();
      for (int i = tid; i < C::ROWS * LPR; i += THREADS) {
        const int row = i / LPR, d = (i % LPR) * 8;
        if (row % cs != rank || rt * C::ROWS + row >= R) continue;
        float mx = -UNSET;
        for (int w = 0; w < cs; ++w) mx = fmaxf(mx, cluster.map_shared_rank(cl, w)[row].x);
        float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll 4
        for (int w = 0; w < cs; ++w) {
          const float2 part = cluster.map_shared_rank(cl, w)[row];
          const float f = ex2_approx(part.x - mx);
          sum += f * part.y;
          const float4* src = reinterpret_cast<const float4*>(cluster.map_shared_rank(co, w) + row * D + d);
          const float4 y0 = src[0], y1 = src[1];
          o[0] += f * y0.x; o[1] += f * y0.y; o[2] += f * y0.z; o[3] += f * y0.w;
          o[4] += f * y1.x; o[5] += f * y1.y; o[6] += f * y1.z; o[7] += f * y1.w;
        }
        emit(row, d, o, mx, sum);
      }
      cluster.sync();                          // no block leaves while another reads its memory
    }
    if (CLUSTER) return;
    __syncthreads();

    x += count;
    if (x == base + (uint32_t)n_chunks * U) {
      base = x;
      ++b;
    }
  }
}

// Joins the parts of units that several blocks share, in their order along the keys, and writes the rows of
// sequences that hold nothing.  A block has `rows_pb` (a power of two, at most ROWS and its warps) rows of one unit; its warps
// are spread over the rows, and over the parts of a row where there are more warps than rows.  The log-sum-exps
// come in first, all at once, then every part's O is loaded independently: two latencies, whatever the
// number of parts.  It is launched while the first kernel still runs (programmatic dependence) and waits for
// it before it touches the workspace or O; the lengths it reads ahead of that, which the first kernel allows by its signal:
// that comes after its own wait for whoever wrote them.  Alone and cold it takes 8 to 11 us, bound by latency
// (one part after another instead: 22 us).
constexpr int JOIN_WARPS = 16;
template <int D, int NT>
__global__ void __launch_bounds__(JOIN_WARPS * 32) cache_attn_join_kernel(const CacheAttnArgs a, int row_tiles, int grid,
                                                                          int rows_pb) {
  constexpr int ROWS = 8 * NT, SLOT = ROWS * (D + 1), PL = D / 32;    // columns per lane
  constexpr int MOST_PARTS = SMS * blocks_per_sm(ROWS);               // blocks of the largest grid
  __shared__ float zs[MOST_PARTS * (ROWS < JOIN_WARPS ? ROWS : JOIN_WARPS)];   // [row of the block][part]
  __shared__ __align__(16) float part_o[JOIN_WARPS][D];
  __shared__ float part_sum[JOIN_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.Hq / a.c.Hkv, U = a.c.Hkv * row_tiles, R = a.T * G;
  const int groups = ROWS / rows_pb, unit = blockIdx.x / groups, first_row = (blockIdx.x - unit * groups) * rows_pb;
  const int b = unit / U, u = unit - b * U, h = u / row_tiles, rt = u - h * row_tiles;
  const int len = seq_len(a, b), n_chunks = (len + CHUNK - 1) / CHUNK;
  const int left = R - rt * ROWS - first_row;         // rows of the block that exist
  bool mine = left > 0;
  uint32_t i0 = 0;
  int parts = 0;
  if (n_chunks > 0) {
    uint32_t x0;
    const Share share(chunks_of_all(a, U, b, x0), grid);
    x0 += (uint32_t)u * n_chunks;
    i0 = share.block(x0);
    parts = (int)(share.block(x0 + n_chunks - 1) - i0) + 1;
    if (parts == 1) mine = false;       // one block had the whole unit and wrote it
  }
  wait_for_last_kernel();
  if (!mine) return;
  // part i of a row: block i0 + i; the first one holds its share in its odd slot, the others in their even one
  const float* const ws = reinterpret_cast<const float*>(a.ws) + 2LL * i0 * SLOT;
  const int live = min(left, rows_pb);
  for (int i = threadIdx.x; i < parts * live; i += JOIN_WARPS * 32) {
    const int p = i / live, row = i - p * live;
    zs[row * parts + p] = __ldcg(ws + (2LL * p + (p == 0)) * SLOT + ROWS * D + first_row + row);
  }
  __syncthreads();
  const int ways = JOIN_WARPS / rows_pb, row = warp & (rows_pb - 1), way = warp / rows_pb;
  float m = -INFINITY, sum = 0.f, o[PL];
#pragma unroll
  for (int j = 0; j < PL; ++j) o[j] = 0.f;
  if (row < live) {
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, zs[row * parts + i]);
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
    const float* const src = ws + (first_row + row) * D + lane * PL;
#pragma unroll 8
    for (int i = way; i < parts; i += ways) {
      const float z = zs[row * parts + i];
      const float f = z == -INFINITY ? 0.f : m == -INFINITY ? z : ex2_approx(z - m);   // NaN stays NaN
      float v[PL];
      if (PL == 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(src + (2LL * i + (i == 0)) * SLOT));
        v[0] = y.x; v[1] = y.y; v[2] = y.z; v[3] = y.w;
      } else {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(src + (2LL * i + (i == 0)) * SLOT));
        v[0] = y.x; v[1] = y.y;
      }
      sum += f;
#pragma unroll
      for (int j = 0; j < PL; ++j) o[j] += f * v[j];
    }
  }
  if (ways > 1) {
#pragma unroll
    for (int j = 0; j < PL; ++j) part_o[warp][lane * PL + j] = o[j];
    if (lane == 0) part_sum[warp] = sum;
    __syncthreads();
    if (way != 0) return;
    for (int w = 1; w < ways; ++w) {
      sum += part_sum[w * rows_pb + row];
#pragma unroll
      for (int j = 0; j < PL; ++j) o[j] += part_o[w * rows_pb + row][lane * PL + j];
    }
  }
  if (row >= live) return;
  const int r = rt * ROWS + first_row + row, tq = r / G, hq = h * G + r - tq * G;
  const bool none = sum == 0.f;
  uint16_t* const dst = reinterpret_cast<uint16_t*>(a.o) + rows_at(a, a.os, b) + tq * a.os.t + hq * a.os.h + lane * PL;
  const float inv = 1.f / sum;
  uint32_t w[PL / 2];
#pragma unroll
  for (int j = 0; j < PL / 2; ++j) w[j] = none ? 0u : f32_to_act(o[2 * j] * inv, o[2 * j + 1] * inv, a.fp16);
  if (PL == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[PL / 2 - 1]);
  else *reinterpret_cast<uint32_t*>(dst) = w[0];
  if (lane == 0 && a.lse)
    a.lse[lse_at(a, b, hq, tq)] = none ? -INFINITY : (m + __log2f(sum)) * 0.6931471805599453f;
}

// How a call is cut up: the rows of a tile, and the blocks of a unit's cluster (1: a block), or 0 for the list.
struct Plan {
  int tile, cluster;
};
// A cluster joins its parts through shared memory: one launch, no workspace.  But a unit then has 8 blocks at most,
// whatever the others' lengths, so it is taken only where the longest sequence that the table allows is few
// chunks per block: CLUSTER_CHUNKS where the clusters leave more than half of the card idle, which the list would
// use, else CLUSTER_CHUNKS_FULL, or CLUSTER_CHUNKS_TILED where a larger tile would do.  D = 128, Hkv = 4, 4 bits,
// cluster / list in us: 4 rows, 1 x 500 tokens 5.6 / 7.3, 4 x 1000 6.4 / 8.2, 1 x 6000 9.9 / 10.5, 1 x 8000 11.3 / 10.8,
// 1 x 12000 14.1 / 9.9; 16 x 2000 9.6 / 13.4, 16 x 4000 13.5 / 16.3, 16 x 6000 17.8 / 19.4 (lengths spread from 1/8 of that:
// 16.1 / 15.6), 64 x 512 8.2 / 13.1, 64 x 1500 16.1 / 19.6 (spread: 14.8 / 16.0), 64 x 2000 20.0 / 22.6.
// 8 bits and heads of 64 take the same thresholds; they were not measured apart.
//
// Rows.  The smallest tile that takes all rows decodes each key once and is the best for long work.  A smaller one
// decodes keys again per tile, but each warp has fewer instructions per key tile and more warps fit, which
// wins while the card is not full: the smallest tile whose clusters all run at once is taken, else the smallest
// whose list has at most SMALL_LIST chunks.  D = 128, Hkv = 8, 4 bits, tiles of 8 / 16 / 32 in us: 16 rows, 4 x 1000
// tokens 8.3 / 10.3 / 12.2, 4 x 4000 16.5 / 14.0 / 17.0, 1 x 16000 15.6 / 16.9 / 20.4, 16 x 8000 57.9 / 47.4 / 66.5; 64
// rows, 4 x 512 8.5 / 11.2 / 14.8, 4 x 1000 17.2 / 13.7 / 16.1, 4 x 2000 23.1 / 21.9 / 20.3, 16 x 4000 112 / 85 / 72.
constexpr int CLUSTER_CHUNKS = 6, CLUSTER_CHUNKS_TILED = 8, CLUSTER_CHUNKS_FULL = 12, SMALL_LIST = 2304;
Plan plan(long long B, long long rows, int Hkv, long long max_tokens) {
  const int whole = rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
  const long long chunks = (max_tokens + CHUNK - 1) / CHUNK;
  for (int tile = 8; tile <= whole; tile *= 2) {
    const long long units = B * Hkv * ((rows + tile - 1) / tile), slots = SMS * blocks_per_sm(tile);
    int cs = 1;
    while (cs < 8 && cs < chunks && units * cs * 2 <= slots) cs *= 2;
    const int most = units * cs * 2 <= slots ? CLUSTER_CHUNKS : tile < whole ? CLUSTER_CHUNKS_TILED : CLUSTER_CHUNKS_FULL;
    if (chunks <= (long long)cs * most && (tile == whole || units <= slots)) return {tile, cs};
  }
  for (int tile = 8; tile < whole; tile *= 2)
    if (B * Hkv * ((rows + tile - 1) / tile) * chunks <= SMALL_LIST) return {tile, 0};
  return {whole, 0};
}

// units * ROWS and units * chunks are below 2^31: checked with the arguments for the tile that takes all rows, and a smaller
// one is chosen for few units or few chunks only.
template <int FMT, int D, int NT>
cudaError_t launch(const CacheAttnArgs& a, int cs, cudaStream_t st) {
  using C = Cfg<FMT, D, NT>;
  const int rows = a.T * (a.Hq / a.c.Hkv), row_tiles = (rows + C::ROWS - 1) / C::ROWS;
  const long long units = (long long)a.B * a.c.Hkv * row_tiles;
  const long long chunks = ((long long)a.pt.max_pages * a.c.page_size + CHUNK - 1) / CHUNK;
  {  // the opt-in to more than 48 KB of shared memory, once per device
    static std::atomic<uint64_t> opted{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!((opted.load(std::memory_order_relaxed) >> dev) & 1)) {
      e = cudaFuncSetAttribute(cache_attn_kernel<FMT, D, NT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(cache_attn_kernel<FMT, D, NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
      if (e != cudaSuccess) return e;
      opted.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
  }
  if (cs)
    return launch_early(cache_attn_kernel<FMT, D, NT, true>, (unsigned)(units * cs), THREADS, C::SMEM, st, cs, a, row_tiles,
                        cs);
  const long long grid = units * chunks < SMS * C::OCC ? units * chunks : SMS * C::OCC;   // no list without chunks: plan()
  const cudaError_t e =
      launch_early(cache_attn_kernel<FMT, D, NT, false>, (unsigned)grid, THREADS, C::SMEM, st, 1, a, row_tiles, 0);
  if (e != cudaSuccess) return e;
  // few units have many parts each: as many blocks per unit as the card takes at once
  int rows_pb = C::ROWS < JOIN_WARPS ? C::ROWS : JOIN_WARPS;
  while (rows_pb > 1 && units * (C::ROWS / rows_pb) * 2 <= SMS * 2) rows_pb /= 2;
  return launch_early(cache_attn_join_kernel<D, NT>, (unsigned)(units * (C::ROWS / rows_pb)), JOIN_WARPS * 32, 0, st, 1, a,
                      row_tiles, (int)grid, rows_pb);
}

template <int FMT, int D>
cudaError_t pick(const CacheAttnArgs& a, cudaStream_t st) {
  const Plan p = plan(a.B, (long long)a.T * (a.Hq / a.c.Hkv), a.c.Hkv, (long long)a.pt.max_pages * a.c.page_size);
  return p.tile == 8    ? launch<FMT, D, 1>(a, p.cluster, st)
         : p.tile == 16 ? launch<FMT, D, 2>(a, p.cluster, st)
                        : launch<FMT, D, 4>(a, p.cluster, st);
}

}  // namespace

size_t cache_attn_workspace_bytes(int B, int T, int Hq, int Hkv, int D, long long max_tokens) {
  const long long all = (long long)T * (Hq / Hkv);
  if (all <= 0) return 0;
  const Plan p = plan(B, all, Hkv, max_tokens);
  // two slots per block of the largest grid of either format
  return p.cluster ? 0 : (size_t)2 * SMS * blocks_per_sm(p.tile) * p.tile * (D + 1) * 4;
}

cudaError_t launch_cache_attn(const CacheAttnArgs& a, int format, int D, cudaStream_t st) {
  if (format == CACHE_FP4) return D == 128 ? pick<CACHE_FP4, 128>(a, st) : pick<CACHE_FP4, 64>(a, st);
  return D == 128 ? pick<CACHE_FP8, 128>(a, st) : pick<CACHE_FP8, 64>(a, st);
}

}  // namespace bsc
