// Linear attention with one decay per head, chunked form for prompts, on the
// 5th-generation tensor cores (tcgen05, accumulators in TMEM).
//
// A chunk is 128 tokens; b_i = sum of the decays' logarithms up to token i of
// the chunk, S the page [value][key] before it.  With A = Q K^T:
//   O  = E (Q S^T) + P V,   P_ij = A_ij 2^(b_i - b_j) for j <= i, else 0,  E_i = 2^b_i
//   S' = 2^b_C S + V^T K'',  K''_t = 2^(b_C - b_t) k_t.
// Four products of 128^3 a chunk, one unit (sequence or segment of it, head)
// after the other per CTA, one CTA per SM.
//
// Factors.  Exponents are sums inside 32-token blocks (bl: prefix sums; sums of the
// tokens behind) and of whole blocks, numbers of one sign.  P: in
// a chunk whose decay is above 2^-128 ("mild"), O = 2^(b_i - r) (Q (2^r S)^T + P' V)
// with P'_ij = A_ij 2^(r - b_j), r half the chunk's logarithm rounded to a whole
// number: every factor is within 2^+-64, one product per element of A and one
// per element of O.  Stronger decays take a row factor times a column factor off
// the diagonal blocks, both <= 1, and 2^(bl_i - bl_j) on them, and O = Q S^T is
// scaled by rows before P V joins it.  Those differences would lose their digits
// behind many resets (7e-4 of the factor after 28, summed in FP32): from a chunk's
// logarithm of -512 on (where FP32's sums are 2^-14 off) bl is summed in whole numbers
// and kept from the middle of the block's range: within +-2048, 2^-14 off, a
// difference 2^-13, the factor 8.5e-5, where P is rounded to 2^-9.  Logarithms below
// -128 (base 2) count as -128: subnormal factors are 0 either way, and a reset of -inf
// stays a number.
//
// Precision.  The page stays in FP32 registers.  K'' = factor * key is the one
// operand of the page's update that BF16 does not hold; it goes in three BF16
// parts, each the rounding of what the ones before leave, which hold its 24 bits:
// the update is exact to FP32's own rounding (one part would put 2^-9 into the
// page, two 2^-17).  What the page's own factor loses to rounding goes into the next
// chunk's (carried_factor), so a slow head's page does not drift.  P and the page's
// copy for Q S^T are rounded to BF16 once: they only feed an output that is itself
// rounded to BF16, and the FP32 sum keeps their errors at that size (outputs against
// 64 bits, 2-norm: 2.34e-3, of which the output's own rounding is 1.66e-3).  Second
// parts of both leave 1.66e-3 and take a third more products, the page's one after
// the other through one tile: 197 -> 261 us (16 prompts x 64 heads), 71 -> 92 (8
// ragged ones x 32), 415 -> 503 (256 suffixes) and 317 -> 379 (32749 tokens); of P
// alone 1.71e-3 to 2.05e-3 at 237, 80, 431 and 334 us.  Neither is kept.  Token by
// token (path 1) nothing is rounded but the output.
//
// Infinities and NaN.  P V multiplies the values of later tokens by zeros, and
// 0 * NaN is not 0.  So P V runs after the page's warps have read the chunk's
// update, where an odd value shows in every key of its column: they put zeros in
// V's place for it, and the outputs of the column are NaN from that token on.
// That costs 1-3% (1-3 us of 72 and 189, 12 of 407 where pages are carried);
// looking at V itself, by whichever warps, cost 4-25%: shared memory and
// instructions are what the kernel is short of.
//
// Roles (768 threads, 24 warps): TMA loads and stores (warp 0), MMA issue for the
// page (U; warp 1) and for the outputs (A, Q S^T, P V; warp 3), the work and its
// decay tables (warp 2); five warpgroups: P and O (4-11, 64 columns a warp), K''
// (12-19, 16 keys a warp), the page (20-23).  K'' is built transposed (lanes =
// keys) by transposing shared-memory matrix loads straight into TMEM, as the A
// operand: no shared memory is written for it.  P is written over A in TMEM.
//   TMEM columns: A / P 0 (P's halves at 0 and 64), O 128, U (the update) 256, K''
//   384 (2 x 48).
//   Shared memory: Q, K, V double-buffered (32 KiB tiles, 128-byte swizzle) and
//   the page's BF16 copy; O leaves through Q's tile.
//
// Split sequences.  A sequence much longer than an SM's share is cut into segments:
// chunk_kernel<false> sums each segment's own contribution to the page (from zeros),
// segment_kernel turns those into the pages the segments start from, and
// chunk_kernel<true> runs the segments side by side.
//
// What bounds it (GB300).  One sequence of 32749 tokens, 32 heads: 192 us for the
// pass with outputs = 3.5 us a chunk and SM, 5.7 TB/s (0.84 of the copy's rate),
// 109 us for the pass without (5.2 TB/s), 17 us between.  With keys and queries
// shared by 8 heads (16 sequences x 64 heads, 189-197 us) the bytes halve and the time
// does not: a chunk moves about 480 KB through shared memory (MMA operands 256 KB),
// 3.8k of its 5.3k cycles at 128 bytes a cycle, the tensor pipe is busy for 42-46%
// of the time and K'' takes one warpgroup pair 4.8k cycles.  What made it fast:
// roles short enough for the instruction cache (unrolled and each walking the work
// for itself 377 us, 7.9 warps waiting for instructions per issue; then 231), K''
// and the outputs over two warpgroups each (212), units dealt by length (190).
// Not kept, measured there: K'' in four parts from packed BF16 products (fewer
// instructions, a third more products for U: 205 us), the next tiles prefetched to
// L2 (205 us), one MMA warp for all products (211 us), the issue loops rolled (232
// us), the next keys loaded ahead (spills: 197-213 us), a third warpgroup for K''
// with 48 registers a thread (208-215 us).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_device.cuh"
#include "kda_host.h"
#include "kda_lin.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace lin {

constexpr int kChunk = 128;
constexpr int kThreads = 768;
constexpr int kHalf = 128 * 128;                 // bytes of a [128][64] BF16 tile
constexpr int kTile = 2 * kHalf;                 // bytes of a [128][128] BF16 tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -128.0f;               // of a decay's base-2 logarithm
constexpr float kMild = -128.0f;                 // a chunk's, for the one-factor form of P
constexpr float kManyDigits = -512.0f;           // a chunk's, from which bl is summed exactly
constexpr float kFixed = 262144.0f;              // 32 tokens of +-128, times 2^18, fit 31 bits

constexpr uint32_t kColA = 0, kColO = 128, kColU = 256, kColK = 384, kColsK = 48;

// One chunk of the CTA's work, as the table warp hands it to the other roles.
struct Info {
  int rows;            // tokens; 0: a unit without tokens, -1: no more
  int row, head;
  int first, last;     // of its unit
  const float *from;   // first: the page it starts from (NULL: zeros)
  float *to, *decay;   // last: where the page, and the unit's logarithm, go (or NULL)
};

// The chunk with its factors, for the roles that compute.
struct Table {
  float w[kChunk];     // K'': 2^(sum of the tokens behind, in the chunk)
  float x[kChunk];     // mild: 2^(ref - b); else bl (prefix sums in the block) - middle
  float total[4];      // the blocks' logarithms
  float middle[4];     // strong: half of that, or 0
  float sum;           // the chunk's
  float ref;           // mild: r, else 0
  uint32_t mild;
  Info info;
};
static_assert(sizeof(Table) % 16 == 0, "vector loads");

// The chunk for the roles that move data and issue.
struct Move {
  int rows, row, head;
};

constexpr int kInfos = 4;

struct Ctrl {
  Table tab[2];
  Move move[kInfos];
  uint64_t move_full[kInfos], move_empty[kInfos];
  uint64_t full_q[2], full_k[3], full_v[3];      // TMA landed
  uint64_t empty_k[3], empty_v[3];
  uint64_t st_full[2];                           // O staged in Q's tile (or written)
  uint64_t tab_full[2], tab_empty[2];
  uint64_t v_ok[2];                              // V there: zeros behind the end, finite
  uint64_t kq_full[4], kq_empty[4];              // K'' quarters in TMEM
  uint64_t u_full[2], u_empty[2];
  uint64_t a_full, p_full, qs_full, o_full, o_empty, s_full;
  uint32_t list[kList];                          // the CTA's first units, where sorted
  int found[kList];                              // the sequence of each that is a slot's, or -1
  uint32_t tmem, abort;
  uint8_t odd_row[2][kDim];                      // an odd column's first non-finite row
  uint8_t odd[2][4];                             // whether 32 columns of V have one
};

constexpr int kSmem = 7 * kTile + sizeof(Ctrl);
static_assert(kSmem <= 232448, "shared memory of one CTA");

// Without outputs A's and O's columns are free: the update has two accumulators
// and K'' four buffers; Q's tiles make a third buffer for K and V.
template <bool kOut>
struct Cols {
  static constexpr uint32_t kU = kOut ? 1 : 2, kKq = kOut ? 2 : 4, kBufs = kOut ? 2 : 3;
  __device__ static uint32_t u(uint32_t n) { return kOut || (n & 1) == 0 ? kColU : kColA; }
  __device__ static uint32_t kq(uint32_t b) {
    return b < 2 ? kColK + b * kColsK : kColO + (b - 2) * kColsK;
  }
};

__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
               : "memory");
}

__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

// 16 lanes x 16 columns: register 2 j + i holds lane row (laneid / 4 + 8 i) of
// column 4 j + laneid % 4.
__device__ __forceinline__ void tc_st_16x128(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
      : "memory");
}

// (shared-memory descriptor, as desc_k_major's) Rows along the contraction
// ("MN-major"): 8-row groups 1024 bytes apart, the
// next 64 columns a half tile further.
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (uint64_t(kHalf >> 4) << 16) |
         (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// FP32 accumulator, BF16 operands, M = N = 128; bit 16: B is MN-major.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (16u << 17) | (8u << 24);
constexpr uint32_t kIdescBmn = kIdesc | (1u << 16);

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// BF16 of both halves: low in the low half.
__device__ __forceinline__ uint32_t pack2(f32x2 v) {
  float lo, hi;
  unpair(v, lo, hi);
  return pack2(lo, hi);
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Byte offset of 16-byte group `group` (of 16) of row `row` in a [128][128] tile.
__device__ __forceinline__ uint32_t tile_at(int row, int group) {
  return static_cast<uint32_t>((group >> 3) * kHalf + row * 128 + (((group & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ f32x2 raw_pair(uint32_t lo, uint32_t hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}

// Notes the first row with an infinity or NaN (255: none) of each of a warp's 32
// columns of V, and puts zeros in their places.  A lane looks at 8 columns, every
// 8th row.
__device__ __forceinline__ void clear_odd(uint8_t *tile, int w4, int lane, int rows,
                                          uint8_t (&odd_row)[kDim]) {
  const int row = (lane & 4) + (lane >> 3);
  uint8_t *at = tile + tile_at(row, 4 * w4 + (lane & 3));
#pragma unroll 1
  for (int i = 0; i < 4; ++i, at += 4) {                // 2 columns at a time
    uint32_t first = 0xFFFFu;                           // a byte a column
#pragma unroll 1
    for (int k = 15; k >= 0; --k) {
      const uint32_t r = row + 8 * k;
      if (r >= static_cast<uint32_t>(rows)) continue;
      uint32_t *to = reinterpret_cast<uint32_t *>(at + 1024 * k);
      const uint32_t x = *to, lo = (x & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u,
                     hi = (x & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u;
      if (lo) first = (first & 0xFF00u) | r;
      if (hi) first = (first & 0xFFu) | r << 8;
      if (lo | hi) *to = x & ~(lo | hi);
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1)
      first = __vminu4(first, __shfl_xor_sync(0xffffffffu, first, o));
    if (lane < 4)
      *reinterpret_cast<uint16_t *>(odd_row + 32 * w4 + 8 * lane + 2 * i) = first;
  }
}

// P of a chunk with strong decays, 64 columns (`side`) of a warp's 32 rows: a row
// factor times f off the diagonal block, 2^(bl_i - bl_j) on it, zeros behind.
// x: this row's of the table.  Returns the row's factor of Q S^T.
__device__ __forceinline__ float strong_rows(const Table &tab, uint32_t col_a, int side, int w4,
                                             int lane, float x) {
  uint32_t a[32], r[16];
  const float bl = x + tab.middle[w4];                  // this row's prefix sum in its block
#pragma unroll 1
  for (int z = 0; z < 2; ++z) {
    const int J = 2 * side + z;
    tc_ld(col_a + 32 * z, a);
    tc_wait_ld(a);
    if (J < w4) {
      float sum = bl;                                   // and the blocks between
      for (int m = J + 1; m < w4; ++m) sum += tab.total[m];
      const float row = exp2_approx(sum), end = tab.x[32 * J + 31];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        r[j] = pack2(__uint_as_float(a[2 * j]) *
                         (row * exp2_approx(end - tab.x[32 * J + 2 * j])),
                     __uint_as_float(a[2 * j + 1]) *
                         (row * exp2_approx(end - tab.x[32 * J + 2 * j + 1])));
    } else {
      const int to = J == w4 ? lane : -1;               // the last column to keep
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float p = __uint_as_float(a[2 * j]) * exp2_approx(x - tab.x[32 * J + 2 * j]);
        const float q = __uint_as_float(a[2 * j + 1]) * exp2_approx(x - tab.x[32 * J + 2 * j + 1]);
        r[j] = pack2(2 * j <= to ? p : 0.0f, 2 * j + 1 <= to ? q : 0.0f);
      }
    }
    tc_st16(col_a + 16 * z, r);
  }
  float sum = bl;
  for (int m = 0; m < w4; ++m) sum += tab.total[m];
  return exp2_approx(sum);
}

// -------------------------------------------------------------- units, chunks

// A unit's rows, head and pages.
struct Unit {
  int row, n, head;
  const float *from;
  float *to, *decay;
};

// A segment's page in the workspace.  All segments but a sequence's last have
// seg_len rows, so first_row / seg_len tells them apart; the last ones (shorter:
// another sequence's first may start in the same seg_len rows) have pages of
// their own behind.
__device__ __forceinline__ int64_t ws_index(const PromptParams &p, int first_row, bool last, int h) {
  const int64_t at = first_row / p.seg_len + (last ? p.slots : 0);
  return at * p.heads + h;
}

// The items of work, each times the heads: first the slots, slot r for the
// segment of seg_len rows, not its sequence's last, that starts in rows r * seg_len
// .. (r + 1) * seg_len - 1 (at most one: it covers the last of them); then, with
// outputs, every sequence's last segment.  There are no more than the rows need,
// however long the longest sequence is.
template <bool kOut>
__device__ __forceinline__ int items_of(const PromptParams &p) {
  return p.slots + (kOut ? p.seqs : 0);
}

// Whether sequence s has slot r's segment, and which one that is.
__device__ __forceinline__ bool in_slot(const PromptParams &p, const Seq &s, int r, int *seg) {
  const int64_t end = static_cast<int64_t>(r + 1) * p.seg_len - 1;
  if (s.start > end) return false;
  const int64_t n = (end - s.start) / p.seg_len;
  *seg = static_cast<int>(n);
  return (n + 1) * p.seg_len < s.len;
}

__device__ __forceinline__ int segments_of(const PromptParams &p, const Seq &s) {
  return s.len > p.seg_len ? (s.len + p.seg_len - 1) / p.seg_len : 1;
}

// Puts this CTA's units in order: all units by length, the longest first, dealt
// to the CTAs forth and back, so that each gets long and short ones (8 ragged
// sequences x 32 heads: 86 -> 78 us; 16 x 64 heads 212 -> 197 us).  One thread an
// item ranks it by counting the longer ones; `keys` is scratch.  All threads call
// it.
template <bool kOut>
__device__ __forceinline__ void order_units(const PromptParams &p, int *keys, uint32_t *list) {
  const int items = items_of<kOut>(p), i = threadIdx.x;
  int key = -1;
  if (i < items) {
    Seq s;
    if (i < p.slots) {
      for (int b = 0, seg; b < p.seqs && key < 0; ++b)
        if (!resolve_seq(p, b, &s) && in_slot(p, s, i, &seg)) key = p.seg_len;
    } else if (!resolve_seq(p, i - p.slots, &s)) {
      key = s.len - (segments_of(p, s) - 1) * p.seg_len;
    }
    keys[i] = key;
  }
  __syncthreads();
  if (i < items) {
    uint32_t rank = 0;
#pragma unroll 8
    for (int j = 0; j < items; ++j) rank += keys[j] > key || (keys[j] == key && j < i);
    const uint32_t lo = rank * p.heads, units = static_cast<uint32_t>(items) * p.heads;
    for (uint32_t k = 0, base = 0; k < kList && base < units; ++k, base += gridDim.x) {
      const uint32_t r = base + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      if (r - lo < static_cast<uint32_t>(p.heads)) list[k] = i * p.heads + (r - lo);
    }
  }
  fence_proxy_async_smem();
}

// This CTA's k-th unit; -1: none this round (forth and back: the last round may
// pass over this CTA), -2: no more.
__device__ __forceinline__ int64_t unit_at(uint32_t k, int64_t units, const uint32_t *list) {
  const int64_t base = static_cast<int64_t>(k) * gridDim.x;
  if (base >= units) return -2;
  const int64_t place = base + (list && (k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  if (place >= units) return -1;
  return list ? list[k % kList] : place;
}

// Whether no sequence starts before the one before it ends, as far as this thread
// looks.  Otherwise two sequences may share rows, and split ones would then share
// pages of the workspace (their index goes by the row): such a call runs none of
// the sequences that it would split.  256 sequences: one load a thread.
__device__ __forceinline__ bool in_order(const PromptParams &p, int threads) {
  bool ok = true;
#pragma unroll 1
  for (int b = threadIdx.x; b < p.seqs; b += threads)
    ok = ok && __ldg(p.seq_starts + b) <= __ldg(p.seq_starts + b + 1);
  return ok;
}

// The sequences of this CTA's slot units (the host keeps them among the first
// kList).  All threads call it; `found` holds -1.
template <bool kOut>
__device__ __forceinline__ void find_slots(const PromptParams &p, const uint32_t *list, int *found) {
  const int64_t units = static_cast<int64_t>(items_of<kOut>(p)) * p.heads;
  for (uint32_t k = 0; k < kList; ++k) {
    const int64_t at = unit_at(k, units, list);
    if (at < 0 || at >= static_cast<int64_t>(p.slots) * p.heads) continue;
    for (int b = threadIdx.x; b < p.seqs; b += kThreads) {
      Seq s;
      int seg;
      if (!resolve_seq(p, b, &s) && in_slot(p, s, static_cast<int>(at / p.heads), &seg)) found[k] = b;
    }
  }
}

// Walks this CTA's units (a whole warp).
template <bool kOut>
struct Walk {
  const PromptParams &p;
  const uint32_t *list;    // NULL: every grid-th unit
  const int *found;
  bool ordered;            // else: split sequences are flagged
  uint32_t k;
  Unit unit;

  __device__ Walk(const PromptParams &p_, const uint32_t *list_, const int *found_, bool ordered_)
      : p(p_), list(list_), found(found_), ordered(ordered_), k(0) {}
  // The next unit that has work for this kernel.
  __device__ bool next(int lane) {
    const int64_t units = static_cast<int64_t>(items_of<kOut>(p)) * p.heads;   // < 2^31
    while (true) {
      const int64_t place = unit_at(k, units, list);
      if (place == -2) return false;
      ++k;
      if (place < 0) continue;
      const uint32_t at = static_cast<uint32_t>(place);
      const int item = at / p.heads;
      unit.head = at - static_cast<uint32_t>(item) * p.heads;
      const bool slot = item < p.slots;
      const int b = slot ? found[(k - 1) % kList] : item - p.slots;
      if (b < 0) continue;
      Seq s;
      int bad = resolve_seq(p, b, &s);
      if (!ordered && s.len > p.seg_len) bad |= KDA_DEVERR_SEQ;
      if (bad) {
        if (lane == 0 && p.err) atomicOr(p.err, bad);
        continue;
      }
      int seg;
      if (!slot || !in_slot(p, s, item, &seg)) seg = segments_of(p, s) - 1;
      unit.row = s.start + seg * p.seg_len;
      const int left = s.len - seg * p.seg_len;
      unit.n = left < p.seg_len ? left : p.seg_len;
      unit.from = nullptr;
      unit.to = unit.decay = nullptr;
      if (s.len > p.seg_len) {
        const int64_t page = ws_index(p, unit.row, !slot, unit.head);
        if (kOut) {
          unit.from = p.ws_state + page * kPage;
        } else {
          unit.to = p.ws_state + page * kPage;
          unit.decay = p.ws_decay + page;
        }
      } else if (s.src) {
        unit.from = page_of(p.state, s.src, p.heads, unit.head);
      }
      if (kOut && !slot && s.dst) unit.to = page_of(p.state, s.dst, p.heads, unit.head);
      return true;
    }
  }
};

// The next chunk of a role (a whole warp; m counts them).  False: no more.
__device__ __forceinline__ bool next_move(Ctrl &c, uint32_t &m, Move &move, int lane) {
  const uint32_t at = m % kInfos;
  if (!__all_sync(0xffffffffu, wait_phase(&c.move_full[at], (m / kInfos) & 1, &c.abort)))
    return false;
  move = c.move[at];
  __syncwarp();
  if (lane == 0) mbar_arrive(&c.move_empty[at]);
  ++m;
  return move.rows >= 0;
}
// The same with its factors: the table of chunk m, whose user gives it back.
__device__ __forceinline__ bool next_table(Ctrl &c, uint32_t m) {
  return __all_sync(0xffffffffu, wait_phase(&c.tab_full[m & 1], (m >> 1) & 1, &c.abort)) &&
         c.tab[m & 1].info.rows >= 0;
}

// -------------------------------------------------------------------- kernel

// A wait that ran out leaves the role's loop; whole warps leave together.
#define KDA_WAIT_WARP(bar, parity)                                                \
  if (!__all_sync(0xffffffffu, wait_phase(&(bar), (parity), &c.abort))) break

// TMEM, all 512 columns (one CTA per SM); one warp calls it.
__device__ __forceinline__ void take_tmem(uint32_t *to) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                   smem_addr(to))
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

// The CTA's end, for all threads: reports a wait that ran out, and frees TMEM.
__device__ __forceinline__ void leave(volatile uint32_t *abort_flag, uint32_t tmem, int warp,
                                      int32_t *err) {
  __syncthreads();
  if (*abort_flag) {
    // copies and products in flight end within microseconds: give them time
    // before the shared memory and TMEM go
    const uint64_t t0 = global_ns();
    for (int i = 0; i < 4096 && global_ns() - t0 < 200000ull; ++i) __nanosleep(1000);
    if (threadIdx.x == 0 && err) atomicOr(err, KDA_DEVERR_TIMEOUT);
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 3)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// kOut: outputs and last states.  Otherwise: each segment's own contribution
// to the page (from zeros) and its total decay, for every segment but a
// sequence's last.
template <bool kOut>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap map_q,
                 const __grid_constant__ CUtensorMap map_k,
                 const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ CUtensorMap map_o) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sq = smem, *sk = smem + (kOut ? 2 : 0) * kTile, *sv = smem + (kOut ? 4 : 3) * kTile,
          *ss = smem + 6 * kTile;
  Ctrl &c = *reinterpret_cast<Ctrl *>(smem + 7 * kTile);
  using C = Cols<kOut>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w4 = warp & 3;                           // TMEM lanes 32 w4 .. of this warp
  volatile uint32_t *abort_flag = &c.abort;

  if (warp == 3) take_tmem(&c.tmem);
  if (threadIdx.x == 0) {
    c.abort = 0;
    for (int i = 0; i < kInfos; ++i) {
      mbar_init(&c.move_full[i], 1);
      mbar_init(&c.move_empty[i], kOut ? 3 : 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.full_q[i], 1);
      mbar_init(&c.st_full[i], 8);
      mbar_init(&c.v_ok[i], 8);
      mbar_init(&c.tab_full[i], 1);
      mbar_init(&c.tab_empty[i], 20);
      mbar_init(&c.u_full[i], 1);
      mbar_init(&c.u_empty[i], 4);
    }
    mbar_init(&c.a_full, 1);
    mbar_init(&c.p_full, 8);
    mbar_init(&c.qs_full, 1);
    mbar_init(&c.o_full, 1);
    mbar_init(&c.o_empty, 8);
    for (uint32_t i = 0; i < C::kBufs; ++i) {
      mbar_init(&c.full_k[i], 1);
      mbar_init(&c.full_v[i], 1);
      mbar_init(&c.empty_k[i], kOut ? 9 : 16);
      mbar_init(&c.empty_v[i], kOut ? 2 : 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&c.kq_full[i], 8);
      mbar_init(&c.kq_empty[i], 1);
    }
    mbar_init(&c.s_full, 4);
    // a tile base that breaks the swizzle's 1024 bytes would give wrong data
    if (smem_addr(smem) & 1023u) c.abort = 1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const int64_t items = items_of<kOut>(p), all_units = items * p.heads;
  const bool sorted = all_units > gridDim.x && items <= kThreads &&
                      all_units <= static_cast<int64_t>(gridDim.x) * kList &&
                      (p.slots == 0 || p.seqs <= 64);      // (a slot looks at every sequence)
  if (threadIdx.x < kList) c.found[threadIdx.x] = -1;
  if (sorted) order_units<kOut>(p, reinterpret_cast<int *>(smem), c.list);
  // (without slots nothing is split)
  const bool ordered = p.slots == 0 || __syncthreads_and(in_order(p, kThreads));
  if (p.slots > 0 && ordered) {
    find_slots<kOut>(p, sorted ? c.list : nullptr, c.found);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;

  if (*abort_flag) {
    // nothing runs
  } else if (warp < 4) {
    // registers: 64, 64, 56 and 176 a thread (4 + 8 + 8 + 4 warps) are the 768 x 80
    // of the launch.  With 56 here the table warp spilled the decays it loads ahead,
    // and so waited for them (ragged prompts 79 -> 88 us); the page spills below 176.
    regs_dec<64>();
    if (warp == 0) {
      // ------------------------------------------------- TMA loads and stores
      Move info;
      uint32_t m = 0, n = 0, stored = 0;
      int row1 = 0, row2 = 0, head1 = 0, head2 = 0, rows1 = 0, rows2 = 0;  // the last two chunks
      // the stored-th chunk's outputs leave Q's tile, which is then free
      auto store = [&](int row, int head, int rows) {
        const int buf = stored & 1;
        if (!__all_sync(0xffffffffu, wait_phase(&c.st_full[buf], (stored >> 1) & 1, &c.abort)))
          return false;
        if (lane == 0 && rows == kChunk) {
          const uint8_t *tile = sq + buf * kTile;
          tma_store(&map_o, head * kDim, row, tile);
          tma_store(&map_o, head * kDim + 64, row, tile + kHalf);
          bulk_commit();
          bulk_wait_read(0);
        }
        __syncwarp();
        ++stored;
        return true;
      };
      bool ok = true;
      while (next_move(c, m, info, lane)) {
        if (info.rows == 0) continue;
        ok = false;
        const int buf = n % C::kBufs, boxes = (info.rows + 31) >> 5;
        const uint32_t parity = (n / C::kBufs & 1) ^ 1;
        const int xk = info.head / p.group * kDim, xv = info.head * kDim;
        // boxes of 32 rows x 64 columns, one a lane
        auto load = [&](uint8_t *tile, const CUtensorMap *map, int x, uint64_t *bar) {
          if (lane == 0) mbar_arrive_expect_tx(bar, boxes * 8192);
          __syncwarp();
          const int i = lane >> 1, t = lane & 1;
          if (i < boxes)
            tma_load(tile + buf * kTile + t * kHalf + i * 4096, map, x + 64 * t, info.row + 32 * i,
                     bar);
        };
        KDA_WAIT_WARP(c.empty_k[buf], parity);
        load(sk, &map_k, xk, &c.full_k[buf]);
        KDA_WAIT_WARP(c.empty_v[buf], parity);
        load(sv, &map_v, xv, &c.full_v[buf]);
        if (kOut) {
          if (n >= 2 && !store(row2, head2, rows2)) break;
          load(sq, &map_q, xk, &c.full_q[buf]);
          row2 = row1, head2 = head1, rows2 = rows1;
          row1 = info.row, head1 = info.head, rows1 = info.rows;
        }
        ++n;
        ok = true;
      }
      if (kOut && ok) {
        if (stored + 2 == n) ok = store(row2, head2, rows2);
        if (ok && stored < n) store(row1, head1, rows1);
      }
      if (lane == 0) bulk_wait_all();
    } else if (warp == 1) {
      // ------------------------------------------------------- MMA issue: U
      // The warp walks and waits as one; one elected thread issues.  Descriptors
      // are sums of a base and constants (addresses count 16 bytes).
      uint32_t quarter = 0;
      const bool leader = elect_one();
      const uint64_t v0 = desc_mn_major(smem_addr(sv));
      Move info;
      uint32_t m = 0, n = 0;
      while (next_move(c, m, info, lane)) {
        if (info.rows == 0) continue;
        const int buf = n % C::kBufs, quarters = (info.rows + 31) >> 5;
        // U = K''^T V, quarter by quarter of 32 tokens
        // (the first K'' also says that V is there)
        const uint32_t ub = n % C::kU, ur = n / C::kU & 1;
        KDA_WAIT_WARP(c.u_empty[ub], ur ^ 1);
        int i = 0;
        for (; i < quarters; ++i, ++quarter) {
          const uint32_t kb = quarter % C::kKq;
          KDA_WAIT_WARP(c.kq_full[kb], quarter / C::kKq & 1);
          tc_fence_after();
          if (leader) {
            const uint32_t a = tmem + C::kq(kb), u = tmem + C::u(n);
            const uint64_t v = v0 + buf * (kTile >> 4) + i * (4096 >> 4);
#pragma unroll
            for (int part = 0; part < 3; ++part)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                tc_mma_ts(u, a + part * 16 + j * 8, v + j * (2048 >> 4), kIdescBmn,
                          i + part + j > 0);
            tc_commit(&c.kq_empty[kb]);
            if (i == quarters - 1) {
              tc_commit(&c.u_full[ub]);
              tc_commit(&c.empty_v[buf]);
            }
          }
          __syncwarp();
        }
        if (i < quarters) break;
        ++n;
      }
    } else if (warp == 2) {
      // -------------------------------------- the work, and its decay tables
      Walk<kOut> it(p, sorted ? c.list : nullptr, c.found, ordered);
      Info next;
      int t = 0;                                           // tokens of the unit handed out
      bool unit = false;
      // the next chunk into `next`, and its decays (4 a lane)
      auto look = [&](float (&g)[4]) {
        if (!unit) {
          if (!it.next(lane)) {
            next = Info{-1};
            g[0] = g[1] = g[2] = g[3] = 0.0f;
            return;
          }
          next.head = it.unit.head;
          next.from = it.unit.from;
          next.to = it.unit.to;
          next.decay = it.unit.decay;
          t = 0;
        }
        const int left = it.unit.n - t;
        next.row = it.unit.row + t;
        next.rows = left < kChunk ? left : kChunk;
        next.first = t == 0;
        next.last = left <= kChunk;
        t += kChunk;
        unit = !next.last;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int x = 4 * lane + j;
          const int64_t at = p.decay_rows ? static_cast<int64_t>(next.row + x) * p.heads : 0;
          g[j] = x < next.rows ? __ldg(p.decay + at + next.head) : 0.0f;
        }
      };
      float ahead[4] = {};
      look(ahead);
      uint32_t m = 0;
      while (true) {
        KDA_WAIT_WARP(c.move_empty[m % kInfos], ((m / kInfos) & 1) ^ 1);
        if (lane == 0) {
          c.move[m % kInfos] = Move{next.rows, next.row, next.head};
          mbar_arrive(&c.move_full[m % kInfos]);
        }
        __syncwarp();
        const Info info = next;
        const int rows = info.rows, buf = m & 1;
        const uint32_t round = (m >> 1) & 1;
        ++m;
        float g[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          g[j] = ahead[j] * kLog2e;
          if (g[j] < kLowest) g[j] = kLowest;
        }
        if (rows >= 0) look(ahead);
        const float sum = (g[0] + g[1]) + (g[2] + g[3]);
        // sums of the lanes before and behind this one in its block of 8 lanes
        float before = sum, behind = sum;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          const float a = __shfl_up_sync(0xffffffffu, before, o, 8);
          const float b = __shfl_down_sync(0xffffffffu, behind, o, 8);
          if ((lane & 7) >= o) before += a;
          if ((lane & 7) + o < 8) behind += b;
        }
        const float total = __shfl_sync(0xffffffffu, before, 7, 8);
        before = __shfl_up_sync(0xffffffffu, before, 1, 8);
        behind = __shfl_down_sync(0xffffffffu, behind, 1, 8);
        if ((lane & 7) == 0) before = 0.0f;
        if ((lane & 7) == 7) behind = 0.0f;
        const float t0 = __shfl_sync(0xffffffffu, total, 0), t1 = __shfl_sync(0xffffffffu, total, 8),
                    t2 = __shfl_sync(0xffffffffu, total, 16), t3 = __shfl_sync(0xffffffffu, total, 24);
        const float all = (t0 + t1) + (t2 + t3);
        const bool mild = all > kMild && all <= 0.0f;    // (a reset is strong)
        const float ref = mild ? floorf(0.5f * all) : 0.0f;
        float4 x, w;
        x.x = before + g[0];
        x.y = x.x + g[1];
        x.z = x.y + g[2];
        x.w = x.z + g[3];
        const int block = lane >> 3;
        if (mild) {
          const float base =
              ref - (block == 0 ? 0.0f : block == 1 ? t0 : block == 2 ? t0 + t1 : t0 + t1 + t2);
          x.x = exp2_approx(base - x.x);
          x.y = exp2_approx(base - x.y);
          x.z = exp2_approx(base - x.z);
          x.w = exp2_approx(base - x.w);
        }
        behind += block == 3 ? 0.0f : block == 2 ? t3 : block == 1 ? t2 + t3 : t1 + (t2 + t3);
        const float s3 = behind, s2 = s3 + g[3], s1 = s2 + g[2], s0 = s1 + g[1];
        w.x = exp2_approx(s0);
        w.y = exp2_approx(s1);
        w.z = exp2_approx(s2);
        w.w = exp2_approx(s3);
        KDA_WAIT_WARP(c.tab_empty[buf], round ^ 1);
        Table &tab = c.tab[buf];
        reinterpret_cast<float4 *>(tab.x)[lane] = x;
        reinterpret_cast<float4 *>(tab.w)[lane] = w;
        if ((lane & 7) == 0) {
          tab.total[lane >> 3] = total;
          tab.middle[lane >> 3] = 0.0f;
        }
        if (lane == 1) {
          tab.sum = all;
          tab.ref = ref;
          tab.mild = mild;
          tab.info = info;
        }
        __syncwarp();
        if (kOut && __builtin_expect(all < kManyDigits, 0)) {
          // (a lane a token, from the decays again, in short loops: code that never runs
          // costs too, where it stands among the other)
#pragma unroll 1
          for (int i = 0; i < kChunk; i += 32) {
            const int64_t at =
                p.decay_rows ? static_cast<int64_t>(info.row + i + lane) * p.heads : 0;
            const float g = i + lane < rows ? __ldg(p.decay + at + info.head) * kLog2e : 0.0f;
            int upto = __float2int_rn(fminf(fmaxf(g, kLowest), -kLowest) * kFixed);
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
              const int before = __shfl_up_sync(0xffffffffu, upto, o);
              if (lane >= o) upto += before;
            }
            const int half = __shfl_sync(0xffffffffu, upto, 31) >> 1;
            float *to = tab.x + i + lane;
            if (*to == *to) *to = __int2float_rn(upto - half) * (1.0f / kFixed);  // (NaN stays)
            if (lane == 0) tab.middle[i >> 5] = __int2float_rn(half) * (1.0f / kFixed);
          }
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&c.tab_full[buf]);
        if (rows < 0) break;
      }
    } else if (kOut && warp == 3) {
      // ----------------------------------------- MMA issue: A, Q S^T and P V
      const bool leader = elect_one();
      const uint64_t q0 = desc_k_major(smem_addr(sq)), k0 = desc_k_major(smem_addr(sk)),
                     v0 = desc_mn_major(smem_addr(sv)), s0 = desc_mn_major(smem_addr(ss));
      Move info;
      uint32_t m = 0, n = 0;
      while (next_move(c, m, info, lane)) {
        if (info.rows == 0) continue;
        const int buf = n & 1, quarters = (info.rows + 31) >> 5;
        const uint32_t one = n & 1, two = (n >> 1) & 1;
        // A = Q K^T, over the P that the products before it have read
        KDA_WAIT_WARP(c.full_k[buf], two);
        KDA_WAIT_WARP(c.full_q[buf], two);
        tc_fence_after();
        if (leader) {
          const uint64_t q = q0 + buf * (kTile >> 4), k = k0 + buf * (kTile >> 4);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t off = ((j >> 2) * kHalf + (j & 3) * 32) >> 4;
            tc_mma_ss(tmem + kColA, q + off, k + off, kIdesc, j > 0);
          }
          tc_commit(&c.a_full);
          tc_commit(&c.empty_k[buf]);
        }
        __syncwarp();
        // O = Q S^T
        KDA_WAIT_WARP(c.s_full, one);
        KDA_WAIT_WARP(c.o_empty, one ^ 1);
        tc_fence_after();
        if (leader) {
          const uint64_t q = q0 + buf * (kTile >> 4);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            tc_mma_ss(tmem + kColO, q + (((j >> 2) * kHalf + (j & 3) * 32) >> 4),
                      s0 + j * (2048 >> 4), kIdescBmn, j > 0);
          tc_commit(&c.qs_full);
        }
        __syncwarp();
        // O += P V
        KDA_WAIT_WARP(c.v_ok[buf], two);
        KDA_WAIT_WARP(c.p_full, one);
        tc_fence_after();
        if (leader) {
          const uint64_t v = v0 + buf * (kTile >> 4);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < 2 * quarters)
              tc_mma_ts(tmem + kColO, tmem + kColA + (j >> 2) * 64 + (j & 3) * 8, v + j * (2048 >> 4), kIdescBmn, 1);
          tc_commit(&c.o_full);
          tc_commit(&c.empty_v[buf]);
        }
        __syncwarp();
        ++n;
      }
    }
    __syncwarp();
  } else if (kOut && warp < 12) {
    regs_dec<64>();
    // ------------------------------------------------------------------ P, O
    {
      uint32_t m = 0, n = 0;
      const int i = 32 * w4 + lane;                       // row of the chunk
      const int side = (warp - 4) >> 2;                   // columns 64 side .. of P and O
      const uint32_t lanes = static_cast<uint32_t>(32 * w4) << 16;
      const uint32_t col_a = tmem + lanes + kColA + 64 * side,
                     col_o = tmem + lanes + kColO + 64 * side;
      for (; next_table(c, m); ++m) {
        const Table &tab = c.tab[m & 1];
        const int rows = tab.info.rows, row = tab.info.row, head = tab.info.head;
        if (rows == 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.tab_empty[m & 1]);
          continue;
        }
        const int buf = n & 1;
        const uint32_t one = n & 1;
        uint32_t a[32], r[16];
        float of;                                         // O's factor
        KDA_WAIT_WARP(c.a_full, one);
        tc_fence_after();
        const float xi = tab.x[i];
        const bool mild = tab.mild;
        if (mild) {
          of = p.scale * rcp_approx(xi);
          // 32 columns at a time; P is written over the A that is read
#pragma unroll 1
          for (int z = 0; z < 2; ++z) {
            const int J = 2 * side + z;                   // block of 32 columns
            if (J <= w4) {
              const ulonglong2 *f = reinterpret_cast<const ulonglong2 *>(tab.x + 32 * J);
              tc_ld(col_a + 32 * z, a);
              tc_wait_ld(a);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const ulonglong2 ff = f[j];
                r[2 * j] = pack2(mul2(raw_pair(a[4 * j], a[4 * j + 1]), ff.x));
                r[2 * j + 1] = pack2(mul2(raw_pair(a[4 * j + 2], a[4 * j + 3]), ff.y));
              }
              if (J == w4) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  r[j] &= 2 * j + 1 <= lane ? 0xFFFFFFFFu : 2 * j <= lane ? 0xFFFFu : 0u;
              }
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) r[j] = 0;
            }
            tc_st16(col_a + 16 * z, r);
          }
        } else {
          of = p.scale;
          const float e = strong_rows(tab, col_a, side, w4, lane, xi);
          // O = E (Q S^T)
          KDA_WAIT_WARP(c.qs_full, one);
          tc_fence_after();
#pragma unroll 1
          for (int j = 0; j < 2; ++j) {
            tc_ld(col_o + 32 * j, a);
            tc_wait_ld(a);
#pragma unroll
            for (int m = 0; m < 32; ++m) a[m] = __float_as_uint(__uint_as_float(a[m]) * e);
            tc_st32(col_o + 32 * j, a);
          }
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&c.p_full);
          mbar_arrive(&c.tab_empty[m & 1]);
        }
        // the chunk's outputs: through Q's tile, or by rows where it is not full
        KDA_WAIT_WARP(c.o_full, one);
        tc_fence_after();
        const bool full = rows == kChunk;
        const uint32_t tile = smem_addr(sq + buf * kTile + side * kHalf) + i * 128;
        __nv_bfloat16 *to = p.output + static_cast<int64_t>(row + i) * p.o_stride + head * kDim + 64 * side;
        const f32x2 of2 = pair(of, of);
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          tc_ld(col_o + 32 * j, a);
          tc_wait_ld(a);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t v[4];
#pragma unroll
            for (int z = 0; z < 4; ++z)
              v[z] = pack2(mul2(raw_pair(a[8 * m + 2 * z], a[8 * m + 2 * z + 1]), of2));
            if (full) {
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                               tile + (((4 * j + m) ^ (lane & 7)) << 4)),
                           "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                           : "memory");
            } else if (i < rows) {
              reinterpret_cast<uint4 *>(to)[4 * j + m] = make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
        }
        if (*reinterpret_cast<const uint32_t *>(c.odd[buf])) {
          // columns with infinities or NaN in V: zeros stood in for them
#pragma unroll 1
          for (int x = 0; x < 64; ++x) {
            const int col = 64 * side + x;
            if (!c.odd[buf][col >> 5] || c.odd_row[buf][col] > i) continue;
            if (full)
              asm volatile("st.shared.b16 [%0], %1;" ::"r"(
                               tile + (((x >> 3) ^ (lane & 7)) << 4) + (x & 7) * 2),
                           "h"(static_cast<uint16_t>(0x7FFF))
                           : "memory");
            else if (i < rows)
              to[x] = __ushort_as_bfloat16(0x7FFF);
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&c.o_empty);
          mbar_arrive(&c.st_full[buf]);
        }
        ++n;
      }
    }
    __syncwarp();
  } else if (warp < 20) {
    regs_dec<56>();
    // ------------------------------------------------------------------- K''
    // Two warpgroups, 16 of the 32 keys each (without outputs: four, of which
    // two take the odd quarters).
    constexpr int kStep = kOut ? 1 : 2;
    const int half = (warp >> 2) & 1, first = kOut || warp < 12 ? 0 : 1;
    uint32_t m = 0, n = 0, done = 0;                       // done: quarters of the chunks before
    // this lane's row of the matrices that it addresses (token, 16-byte group)
    const uint32_t at_k =
        smem_addr(sk) + tile_at(8 * (lane >> 4) + (lane & 7), 4 * w4 + 2 * half + ((lane >> 3) & 1));
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * w4 + 16 * half) << 16);
    for (; next_table(c, m); ++m) {
      const Table &tab = c.tab[m & 1];
      const int rows = tab.info.rows, quarters = (rows + 31) >> 5;
      if (rows == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.tab_empty[m & 1]);
        continue;
      }
      const int buf = n % C::kBufs;
      const uint32_t two = n / C::kBufs & 1;
      KDA_WAIT_WARP(c.full_k[buf], two);
      int i = first;
#pragma unroll 1
      for (; i < quarters; i += kStep) {
        const uint32_t quarter = done + i, kb = quarter % C::kKq;
        // factors of the 8 tokens a lane sees: 8 j + 2 (lane % 4) + {0, 1}
        f32x2 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = reinterpret_cast<const f32x2 *>(tab.w + 32 * i + 8 * j)[lane & 3];
        uint32_t raw[8], hi[8], mid[8], lo[8];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t r[4];
          ldmatrix_x4_trans(at_k + buf * kTile + i * 4096 + x * 2048, r);
#pragma unroll
          for (int y = 0; y < 4; ++y) raw[4 * x + y] = r[y];
        }
        if (32 * i + 32 > rows) {
          const int valid = rows - 32 * i - 2 * (lane & 3);  // tokens behind it: any keys
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int j = y >> 1;
            raw[y] &= 8 * j + 1 < valid ? 0xFFFFFFFFu : 8 * j < valid ? 0xFFFFu : 0u;
          }
        }
        // three parts of 8 bits hold all 24
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const f32x2 v = mul2(raw_pair(raw[y] << 16, raw[y] & 0xFFFF0000u), w[y >> 1]);
          hi[y] = pack2(v);
          const f32x2 v1 = sub2(v, raw_pair(hi[y] << 16, hi[y] & 0xFFFF0000u));
          mid[y] = pack2(v1);
          lo[y] = pack2(sub2(v1, raw_pair(mid[y] << 16, mid[y] & 0xFFFF0000u)));
        }
        KDA_WAIT_WARP(c.kq_empty[kb], (quarter / C::kKq & 1) ^ 1);
        tc_fence_after();
        const uint32_t to = lanes + C::kq(kb);
        tc_st_16x128(to, hi);
        tc_st_16x128(to + 16, mid);
        tc_st_16x128(to + 32, lo);
        if (i == 0 && half == 0) {
          // the first K'' also says that V is there
          KDA_WAIT_WARP(c.full_v[buf], two);
          if (rows < 32 * quarters) {
            // rows behind the sequence's end become zeros: they are other rows of
            // the tensor (or stale), and 0 * NaN is not 0
            const int at = threadIdx.x & 127;
#pragma unroll 1
            for (int x = at; x < (32 * quarters - rows) * 16; x += 128)
              *reinterpret_cast<uint4 *>(sv + buf * kTile + tile_at(rows + (x >> 4), x & 15)) =
                  make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (kOut && lane == 0) mbar_arrive(&c.v_ok[buf]);
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.kq_full[kb]);
      }
      if (i < quarters) break;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&c.empty_k[buf]);
        mbar_arrive(&c.tab_empty[m & 1]);
      }
      done += quarters;
      ++n;
    }
    __syncwarp();
  } else {
    regs_inc<176>();
    // -------------------------------------------------------------- the page
    uint32_t m = 0, n = 0;
    const int d = 32 * w4 + lane;                          // key
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * w4) << 16);
    f32x2 s[kDim / 2];                                     // value rows 2 i, 2 i + 1
    float all = 0.0f, carry = 0.0f;                        // the unit's decay (logarithm)
    for (; next_table(c, m); ++m) {
      const Table &tab = c.tab[m & 1];
      const Info info = tab.info;
      const float total = tab.sum, ref = tab.ref;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.tab_empty[m & 1]);
      if (info.first) {
        all = carry = 0.0f;
        if (info.from) {
#pragma unroll
          for (int i = 0; i < kDim / 2; ++i)
            s[i] = pair(info.from[2 * i * kDim + d], info.from[(2 * i + 1) * kDim + d]);
        } else {
#pragma unroll
          for (int i = 0; i < kDim / 2; ++i) s[i] = 0;
        }
      }
      if (info.rows > 0) {
        const uint32_t one = n & 1;
        const float keep = carried_factor(total, carry);
        if (kOut) {
          // the page's copy for Q S^T; the product before has read the last one
          if (n > 0) KDA_WAIT_WARP(c.qs_full, one ^ 1);
          const float e = exp2_approx(ref);
          const f32x2 e2 = pair(e, e);
#pragma unroll
          for (int g = 0; g < 16; ++g)
            *reinterpret_cast<uint4 *>(ss + tile_at(d, g)) =
                make_uint4(pack2(mul2(s[4 * g], e2)), pack2(mul2(s[4 * g + 1], e2)),
                           pack2(mul2(s[4 * g + 2], e2)), pack2(mul2(s[4 * g + 3], e2)));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.s_full);
        }
        const f32x2 keep2 = pair(keep, keep);
        all += total;
        const uint32_t ub = n % C::kU, col_u = lanes + C::u(n);
        KDA_WAIT_WARP(c.u_full[ub], n / C::kU & 1);
        tc_fence_after();
        uint32_t u[32];
        f32x2 odd2 = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          tc_ld(col_u + 32 * j, u);
          tc_wait_ld(u);
#pragma unroll
          for (int m = 0; m < 16; ++m) {
            const f32x2 x = raw_pair(u[2 * m], u[2 * m + 1]);
            s[16 * j + m] = fma2(s[16 * j + m], keep2, x);
            if (kOut) odd2 = fma2(x, 0, odd2);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.u_empty[ub]);
        if (kOut) {
          // the update has read V, and shows whether there is an infinity or NaN in
          // it (a key's, or an overflow, finds none)
          const int buf = n & 1;
          float x, y;
          unpair(odd2, x, y);
          const bool odd = __any_sync(0xffffffffu, !(x + y == 0.0f));
          if (odd) {
            clear_odd(sv + buf * kTile, w4, lane, info.rows, c.odd_row[buf]);
            fence_proxy_async_smem();
          }
          if (lane == 0) c.odd[buf][w4] = odd;
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.v_ok[buf]);
        }
        ++n;
      }
      if (info.last && info.to) {
#pragma unroll
        for (int i = 0; i < kDim / 2; ++i) {
          float x, y;
          unpair(s[i], x, y);
          info.to[2 * i * kDim + d] = x;
          info.to[(2 * i + 1) * kDim + d] = y;
        }
        if (!kOut && threadIdx.x == 640) *info.decay = all;
      }
    }
    __syncwarp();
  }
  leave(&c.abort, tmem, warp, p.err);
}

// Self-test: the wait above running out, and the way out behind it.  A CTA of the
// chunked form's size takes TMEM and waits in its roles' manner, first for a phase
// that is complete, then for one that nothing completes.
__global__ void __launch_bounds__(kThreads, 1) wait_test_kernel(int32_t *err) {
  __shared__ struct { uint64_t complete, never; uint32_t tmem, abort; } c;
  const int warp = threadIdx.x >> 5;
  if (warp == 3) take_tmem(&c.tmem);
  if (threadIdx.x == 0) {
    c.abort = 0;
    mbar_init(&c.complete, 1);
    mbar_init(&c.never, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;
  if (threadIdx.x == 0) mbar_arrive(&c.complete);
  int passed = 0;
  while (true) {
    KDA_WAIT_WARP(c.complete, 0);
    ++passed;
    KDA_WAIT_WARP(c.never, 0);
    ++passed;
    break;
  }
  __syncwarp();
  leave(&c.abort, tmem, warp, __syncthreads_and(passed == 1) ? err : nullptr);
}
#undef KDA_WAIT_WARP

// The pages that the segments of split sequences start from, in place of their
// contributions: S_0 = the sequence's first page, S_(g+1) = 2^decay_g S_g + U_g.
// A block takes a sequence or, where there are fewer, a slot, and has work if the
// slot's segment is a sequence's first (200 short sequences beside a split one cost
// 100 us in blocks that find nothing).  Each thread walks 4 elements of a page over
// the segments, eight segments' loads in flight (one at a time, 19 segments of 32
// heads took 227 us instead of 15).
__global__ void __launch_bounds__(kSegmentThreads)
    segment_kernel(const __grid_constant__ PromptParams p) {
  constexpr int kBatch = 8;
  const int part = blockIdx.x % kSegmentBlocks, item = blockIdx.x / kSegmentBlocks;
  const int h = item % p.heads;
  Seq seq;
  if (!__syncthreads_and(in_order(p, kSegmentThreads))) return;
  if (p.seqs <= p.slots) {
    if (resolve_seq(p, item / p.heads, &seq) || seq.len <= p.seg_len) return;
  } else {
    __shared__ int found;
    if (threadIdx.x == 0) found = -1;
    __syncthreads();
    for (int b = threadIdx.x, seg; b < p.seqs; b += kSegmentThreads)
      if (!resolve_seq(p, b, &seq) && in_slot(p, seq, item / p.heads, &seg) && seg == 0) found = b;
    __syncthreads();
    if (found < 0) return;
    resolve_seq(p, found, &seq);
  }
  const int last = (seq.len + p.seg_len - 1) / p.seg_len - 1;
  const int at = part * kSegmentThreads + threadIdx.x;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (seq.src) s = reinterpret_cast<const float4 *>(page_of(p.state, seq.src, p.heads, h))[at];
  // (full segments' pages are heads apart)
  const int64_t first = ws_index(p, seq.start, false, h);
  float4 *ws = reinterpret_cast<float4 *>(p.ws_state + first * kPage) + at;
  const float *decay = p.ws_decay + first;
  const int64_t step = static_cast<int64_t>(p.heads) * (kPage / 4);
  float carry = 0.0f;
  for (int g = 0; g < last; g += kBatch) {
    float4 u[kBatch];
    float log2[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (g + i < last) {
        u[i] = ws[i * step];
        log2[i] = decay[i * p.heads];
      }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (g + i < last) {
        ws[i * step] = s;
        const float keep = carried_factor(log2[i], carry);
        s.x = __fmaf_rn(s.x, keep, u[i].x);
        s.y = __fmaf_rn(s.y, keep, u[i].y);
        s.z = __fmaf_rn(s.z, keep, u[i].z);
        s.w = __fmaf_rn(s.w, keep, u[i].w);
      }
    ws += kBatch * step;
    decay += kBatch * p.heads;
  }
  const int64_t end = ws_index(p, seq.start + last * p.seg_len, true, h);
  reinterpret_cast<float4 *>(p.ws_state + end * kPage)[at] = s;
}

// ---------------------------------------------------------------------- host

int launch_chunked(const PromptParams &p, int qk_heads, int dev, int sms, cudaStream_t stream) {
  CUtensorMap q, k, v, o;
  const int64_t kw = int64_t(qk_heads) * kDim, vw = int64_t(p.heads) * kDim;
  if (!rows_map(&q, p.q, kw, p.tokens, p.q_stride, 32, dev) ||
      !rows_map(&k, p.k, kw, p.tokens, p.k_stride, 32, dev) ||
      !rows_map(&v, p.v, vw, p.tokens, p.v_stride, 32, dev) ||
      !rows_map(&o, p.output, vw, p.tokens, p.o_stride, kChunk, dev))
    return KDA_ERR_LAUNCH;
  static std::atomic<bool> out_done[kMaxDevices], seg_done[kMaxDevices];
  if (!set_smem_limit_once(out_done, dev, reinterpret_cast<const void *>(chunk_kernel<true>),
                           kSmem) ||
      !set_smem_limit_once(seg_done, dev, reinterpret_cast<const void *>(chunk_kernel<false>),
                           kSmem))
    return KDA_ERR_LAUNCH;
  if (static_cast<int64_t>(p.slots) * p.heads > static_cast<int64_t>(kList) * sms)
    return KDA_ERR_SHAPE;  // (find_slots; not on a whole GPU)
  auto grid_of = [&](int64_t items) {
    return static_cast<int>(items * p.heads < sms ? items * p.heads : sms);
  };
  if (p.slots > 0) {
    chunk_kernel<false><<<grid_of(p.slots), kThreads, kSmem, stream>>>(p, q, k, v, o);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_LAUNCH;
    segment_kernel<<<(p.seqs < p.slots ? p.seqs : p.slots) * p.heads * kSegmentBlocks, kSegmentThreads, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_LAUNCH;
  }
  chunk_kernel<true><<<grid_of(static_cast<int64_t>(p.slots) + p.seqs), kThreads, kSmem, stream>>>(p, q, k, v, o);
  return cudaGetLastError() == cudaSuccess ? KDA_SUCCESS : KDA_ERR_LAUNCH;
}

}  // namespace lin
}  // namespace kda

extern "C" int kda_selftest_lin_wait_timeout(int32_t *err, void *stream) {
  if (!err) return KDA_ERR_NULL_POINTER;
  if (reinterpret_cast<uintptr_t>(err) & 3u) return KDA_ERR_ALIGNMENT;
  kda::lin::wait_test_kernel<<<1, kda::lin::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(err);
  return cudaGetLastError() == cudaSuccess ? KDA_SUCCESS : KDA_ERR_LAUNCH;
}
