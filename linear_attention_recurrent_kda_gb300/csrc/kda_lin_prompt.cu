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
// Factors.  Exponents are differences of sums; they are formed without
// cancellation from sums inside 32-token blocks: bl (prefix), f = 2^(suffix)
// and the blocks' totals.  Off the diagonal 2^(b_i - b_j) is a row factor times
// f_j, both <= 1; on it 2^(bl_i - bl_j).  Logarithms below -160 (in powers of
// two) count as -160: the factor is 0 in FP32 either way, and a reset of -inf
// stays a number.
//
// Precision.  The page stays in FP32 registers.  K'' = factor * key is the one
// FP32 operand of the page's update; it is split into three BF16 parts (what
// they leave is 2^-24 of it), so the update is exact to FP32's own rounding;
// one part would put 2^-9 into the page, two 2^-16.  P and the page's copy for
// Q S^T are rounded to BF16 once: they only feed an output that is itself
// rounded to BF16, and the FP32 sum keeps their errors at that size.
//
// Roles (512 threads, 16 warps): TMA loads (warp 0), MMA issue (1), decay
// tables (2), output stores (3); three warpgroups: P and O (4-7), K'' (8-11),
// the page (12-15).  K'' is built transposed (lanes = keys) by transposing
// shared-memory matrix loads straight into TMEM, as the A operand: no shared
// memory is written for it.  P is written over A in TMEM.
//   TMEM columns: A / P 0, O 128, U (the update) 256, K'' 384 (2 x 48).
//   Shared memory: Q, K, V double-buffered (32 KiB tiles, 128-byte swizzle) and
//   the page's BF16 copy; O leaves through Q's tile.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_device.cuh"
#include "kda_host.h"
#include "kda_lin.cuh"

namespace kda {
namespace lin {

constexpr int kChunk = 128;
constexpr int kThreads = 512;
constexpr int kHalf = 128 * 128;                 // bytes of a [128][64] BF16 tile
constexpr int kTile = 2 * kHalf;                 // bytes of a [128][128] BF16 tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -160.0f;               // of a decay's base-2 logarithm

constexpr uint32_t kColA = 0, kColO = 128, kColU = 256, kColK = 384, kColsK = 48;

struct Table {
  float bl[kChunk];    // prefix sums inside 32-token blocks (base-2 logarithms)
  float f[kChunk];     // 2^(sum of the tokens behind, in the block)
  float total[4];      // block totals
};

struct Ctrl {
  Table tab[2];
  uint64_t full_q[2], full_k[2], full_v[2];      // TMA landed
  uint64_t empty_q[2], empty_k[2], empty_v[2];
  uint64_t tab_full[2], tab_empty[2];
  uint64_t kq_full[2], kq_empty[2];              // K'' quarters in TMEM
  uint64_t v_ok[2];                              // V's rows behind the end are zeros
  uint64_t st_full[2];                           // O staged in Q's tile (or written)
  uint64_t a_full, p_full, qs_full, o_full, o_empty, u_full, u_empty, s_full;
  uint32_t tmem, abort;
};

constexpr int kSmem = 7 * kTile + sizeof(Ctrl);
static_assert(kSmem <= 232448, "shared memory of one CTA");

// ------------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D (TMEM) (+)= A B, both from shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same with A from TMEM.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Loads 32 columns of this warp's 32 lanes (and waits for them).
__device__ __forceinline__ void tc_ld32(uint32_t addr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tc_st32(uint32_t addr, const float (&v)[32]) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(addr)
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

// Shared-memory descriptors of 128-byte-swizzled BF16 tiles of 128-byte rows.
// Rows along the M / N extent ("K-major"): 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_k_major(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (uint64_t(1) << 16) |
         (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// Rows along the contraction ("MN-major"): 8-row groups 1024 bytes apart, the
// next 64 columns a half tile further.
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (uint64_t(kHalf >> 4) << 16) |
         (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// FP32 accumulator, BF16 operands, M = N = 128; bit 16: B is MN-major.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (16u << 17) | (8u << 24);
constexpr uint32_t kIdescBmn = kIdesc | (1u << 16);

__device__ __forceinline__ void tma_load(void *dst, const CUtensorMap *map, int x, int y,
                                         uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap *map, int x, int y, const void *src) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
      "r"(x), "r"(y), "r"(smem_addr(src))
      : "memory");
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float low_half(uint32_t r) { return __uint_as_float(r << 16); }
__device__ __forceinline__ float high_half(uint32_t r) { return __uint_as_float(r & 0xFFFF0000u); }

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

// -------------------------------------------------------------- units, chunks

struct Unit {
  int b, h, seg, segs;     // sequence, head, segment of its segments
  int row, n;              // first row, tokens
  int src, dst;
};

// Walks the chunks of this CTA's units, the same way in every role.
template <bool kOut>
struct Walk {
  const PromptParams &p;
  int64_t u;
  Unit unit;
  int chunk, chunks;       // of the unit

  __device__ explicit Walk(const PromptParams &p_) : p(p_), u(blockIdx.x), chunk(0), chunks(0) {
    u -= gridDim.x;
  }
  // The next unit that has work for this kernel.
  __device__ bool next_unit(bool report) {
    const int64_t units = static_cast<int64_t>(p.seqs) * p.segs * p.heads;
    for (u += gridDim.x; u < units; u += gridDim.x) {
      const int rest = static_cast<int>(u / p.heads);
      unit.h = static_cast<int>(u - static_cast<int64_t>(rest) * p.heads);
      unit.b = rest / p.segs;
      unit.seg = rest - unit.b * p.segs;
      Seq s;
      if (const int bad = resolve_seq(p, unit.b, &s)) {
        if (report && p.err) atomicOr(p.err, bad);
        continue;
      }
      unit.segs = s.len > p.seg_len ? (s.len + p.seg_len - 1) / p.seg_len : 1;
      if (unit.seg >= (kOut ? unit.segs : unit.segs - 1)) continue;
      unit.row = s.start + unit.seg * p.seg_len;
      const int left = s.len - unit.seg * p.seg_len;
      unit.n = left < p.seg_len ? left : p.seg_len;
      unit.src = s.src;
      unit.dst = s.dst;
      chunk = -1;
      chunks = (unit.n + kChunk - 1) / kChunk;
      return true;
    }
    return false;
  }
  __device__ bool next_chunk() { return ++chunk < chunks; }
  // The next chunk of this or a later unit.
  __device__ bool next() {
    while (true) {
      if (chunks && next_chunk()) return true;
      if (!next_unit(false)) return false;
    }
  }
  __device__ int rows() const {
    const int left = unit.n - chunk * kChunk;
    return left < kChunk ? left : kChunk;
  }
  __device__ int first_row() const { return unit.row + chunk * kChunk; }
};

// A segment's page in the workspace.  All segments but a sequence's last have
// seg_len rows, so first_row / seg_len tells them apart; the last ones (shorter:
// another sequence's first may start in the same seg_len rows) have pages of
// their own behind.
__device__ __forceinline__ int64_t ws_index(const PromptParams &p, int first_row, bool last, int h) {
  const int64_t at = first_row / p.seg_len + (last ? p.tokens / p.seg_len + 1 : 0);
  return at * p.heads + h;
}
__device__ __forceinline__ int64_t ws_index(const PromptParams &p, const Unit &u) {
  return ws_index(p, u.row, u.seg == u.segs - 1, u.h);
}

// -------------------------------------------------------------------- kernel

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
  uint8_t *sq = smem, *sk = smem + 2 * kTile, *sv = smem + 4 * kTile, *ss = smem + 6 * kTile;
  Ctrl &c = *reinterpret_cast<Ctrl *>(smem + 7 * kTile);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w4 = warp & 3;                           // TMEM lanes 32 w4 .. of this warp
  volatile uint32_t *abort_flag = &c.abort;

  if (warp == 3) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_addr(&c.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    c.abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.full_q[i], 1);
      mbar_init(&c.full_k[i], 1);
      mbar_init(&c.full_v[i], 1);
      mbar_init(&c.empty_q[i], 1);
      mbar_init(&c.empty_k[i], kOut ? 5 : 4);
      mbar_init(&c.empty_v[i], 1);
      mbar_init(&c.tab_full[i], 1);
      mbar_init(&c.tab_empty[i], kOut ? 12 : 8);
      mbar_init(&c.kq_full[i], 4);
      mbar_init(&c.kq_empty[i], 1);
      mbar_init(&c.v_ok[i], 4);
      mbar_init(&c.st_full[i], 4);
    }
    mbar_init(&c.a_full, 1);
    mbar_init(&c.p_full, 4);
    mbar_init(&c.qs_full, 1);
    mbar_init(&c.o_full, 1);
    mbar_init(&c.o_empty, 4);
    mbar_init(&c.u_full, 1);
    mbar_init(&c.u_empty, 4);
    mbar_init(&c.s_full, 4);
    // a tile base that breaks the swizzle's 1024 bytes would give wrong data
    if (smem_addr(smem) & 1023u) c.abort = 1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;

// A wait that ran out leaves the role's loop; whole warps leave together.
#define KDA_WAIT(bar, parity) \
  if (!mbar_wait(&(bar), (parity), abort_flag)) break
#define KDA_WAIT_WARP(bar, parity) \
  if (!__all_sync(0xffffffffu, mbar_wait(&(bar), (parity), abort_flag))) break

  if (*abort_flag) {
    // nothing runs
  } else if (warp < 4) {
    regs_dec<80>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ TMA loads
      Walk<kOut> it(p);
      for (uint32_t n = 0; it.next(); ++n) {
        const int buf = n & 1, boxes = (it.rows() + 31) >> 5, y = it.first_row();
        const uint32_t parity = ((n >> 1) & 1) ^ 1;
        const int xk = it.unit.h / p.group * kDim, xv = it.unit.h * kDim;
        KDA_WAIT(c.empty_k[buf], parity);
        mbar_arrive_expect_tx(&c.full_k[buf], boxes * 8192);
        for (int i = 0; i < boxes; ++i)
          for (int t = 0; t < 2; ++t)
            tma_load(sk + buf * kTile + t * kHalf + i * 4096, &map_k, xk + 64 * t, y + 32 * i,
                     &c.full_k[buf]);
        if (kOut) {
          KDA_WAIT(c.empty_q[buf], parity);
          mbar_arrive_expect_tx(&c.full_q[buf], boxes * 8192);
          for (int i = 0; i < boxes; ++i)
            for (int t = 0; t < 2; ++t)
              tma_load(sq + buf * kTile + t * kHalf + i * 4096, &map_q, xk + 64 * t, y + 32 * i,
                       &c.full_q[buf]);
        }
        KDA_WAIT(c.empty_v[buf], parity);
        mbar_arrive_expect_tx(&c.full_v[buf], boxes * 8192);
        for (int i = 0; i < boxes; ++i)
          for (int t = 0; t < 2; ++t)
            tma_load(sv + buf * kTile + t * kHalf + i * 4096, &map_v, xv + 64 * t, y + 32 * i,
                     &c.full_v[buf]);
      }
    } else if (warp == 1 && lane == 0) {
      // ------------------------------------------------------------ MMA issue
      Walk<kOut> it(p);
      bool more = it.next();
      uint32_t quarter = 0;
      auto issue_qk = [&](int buf) {
        const uint32_t q = smem_addr(sq + buf * kTile), k = smem_addr(sk + buf * kTile);
        for (int j = 0; j < 8; ++j) {
          const uint32_t off = (j >> 2) * kHalf + (j & 3) * 32;
          tc_mma_ss(tmem + kColA, desc_k_major(q + off), desc_k_major(k + off), kIdesc, j > 0);
        }
      };
      if (kOut && more) {
        do {
          KDA_WAIT(c.full_k[0], 0);
          KDA_WAIT(c.full_q[0], 0);
          tc_fence_after();
          issue_qk(0);
          tc_commit(&c.a_full);
          tc_commit(&c.empty_k[0]);
        } while (false);
      }
      for (uint32_t n = 0; more; ++n) {
        const int buf = n & 1, quarters = (it.rows() + 31) >> 5;
        const uint32_t one = n & 1, two = (n >> 1) & 1;
        const uint32_t v = smem_addr(sv + buf * kTile);
        if (kOut) {
          // O = Q S^T (unscaled)
          KDA_WAIT(c.s_full, one);
          if (n > 0) KDA_WAIT(c.o_empty, one ^ 1);
          tc_fence_after();
          const uint32_t q = smem_addr(sq + buf * kTile), s = smem_addr(ss);
          for (int j = 0; j < 8; ++j)
            tc_mma_ss(tmem + kColO, desc_k_major(q + (j >> 2) * kHalf + (j & 3) * 32),
                      desc_mn_major(s + j * 2048), kIdescBmn, j > 0);
          tc_commit(&c.qs_full);
        }
        // U = K''^T V, quarter by quarter of 32 tokens
        KDA_WAIT(c.full_v[buf], two);
        KDA_WAIT(c.v_ok[buf], two);
        if (n > 0) KDA_WAIT(c.u_empty, one ^ 1);
        int i = 0;
        for (; i < quarters; ++i, ++quarter) {
          const int kb = quarter & 1;
          KDA_WAIT(c.kq_full[kb], (quarter >> 1) & 1);
          tc_fence_after();
          for (int part = 0; part < 3; ++part)
            for (int j = 0; j < 2; ++j)
              tc_mma_ts(tmem + kColU, tmem + kColK + kb * kColsK + part * 16 + j * 8,
                        desc_mn_major(v + (2 * i + j) * 2048), kIdescBmn, i + part + j > 0);
          tc_commit(&c.kq_empty[kb]);
        }
        if (i < quarters) break;
        tc_commit(&c.u_full);
        if (kOut) {
          // O += P V
          KDA_WAIT(c.p_full, one);
          tc_fence_after();
          for (int j = 0; j < 2 * quarters; ++j)
            tc_mma_ts(tmem + kColO, tmem + kColA + j * 8, desc_mn_major(v + j * 2048), kIdescBmn, 1);
          tc_commit(&c.o_full);
        }
        tc_commit(&c.empty_v[buf]);
        more = it.next();
        if (kOut && more) {
          const int nb = (n + 1) & 1;
          const uint32_t np = ((n + 1) >> 1) & 1;
          KDA_WAIT(c.full_k[nb], np);
          KDA_WAIT(c.full_q[nb], np);
          tc_fence_after();
          issue_qk(nb);
          tc_commit(&c.a_full);
          tc_commit(&c.empty_k[nb]);
        }
      }
    } else if (warp == 2) {
      // --------------------------------------------------------- decay tables
      Walk<kOut> it(p);
      for (uint32_t n = 0; it.next(); ++n) {
        const int buf = n & 1, rows = it.rows();
        float g[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 4 * lane + j;
          g[j] = 0.0f;
          if (t < rows) {
            const int64_t at = p.decay_rows ? static_cast<int64_t>(it.first_row() + t) * p.heads : 0;
            g[j] = __ldg(p.decay + at + it.unit.h) * kLog2e;
            if (g[j] < kLowest) g[j] = kLowest;
          }
        }
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
        KDA_WAIT_WARP(c.tab_empty[buf], ((n >> 1) & 1) ^ 1);
        Table &tab = c.tab[buf];
        float4 bl, f;
        bl.x = before + g[0];
        bl.y = bl.x + g[1];
        bl.z = bl.y + g[2];
        bl.w = bl.z + g[3];
        const float s3 = behind, s2 = s3 + g[3], s1 = s2 + g[2], s0 = s1 + g[1];
        f.x = exp2_approx(s0);
        f.y = exp2_approx(s1);
        f.z = exp2_approx(s2);
        f.w = exp2_approx(s3);
        reinterpret_cast<float4 *>(tab.bl)[lane] = bl;
        reinterpret_cast<float4 *>(tab.f)[lane] = f;
        if ((lane & 7) == 0) tab.total[lane >> 3] = total;
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.tab_full[buf]);
      }
    } else if (kOut && warp == 3 && lane == 0) {
      // -------------------------------------------------------- output stores
      Walk<kOut> it(p);
      for (uint32_t n = 0; it.next(); ++n) {
        const int buf = n & 1;
        KDA_WAIT(c.st_full[buf], (n >> 1) & 1);
        if (it.rows() == kChunk) {
          for (int t = 0; t < 2; ++t)
            tma_store(&map_o, it.unit.h * kDim + 64 * t, it.first_row(), sq + buf * kTile + t * kHalf);
          bulk_commit();
          bulk_wait_read(0);
        }
        mbar_arrive(&c.empty_q[buf]);
      }
      bulk_wait_all();
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------------ P, O
    if (kOut) {
      Walk<kOut> it(p);
      const int i = 32 * w4 + lane;                       // row of the chunk
      const uint32_t lanes = static_cast<uint32_t>(32 * w4) << 16;
      for (uint32_t n = 0; it.next(); ++n) {
        const int buf = n & 1, rows = it.rows();
        const uint32_t one = n & 1;
        const Table &tab = c.tab[buf];
        KDA_WAIT_WARP(c.tab_full[buf], (n >> 1) & 1);
        KDA_WAIT_WARP(c.a_full, one);
        tc_fence_after();
        const float bl = tab.bl[i];
        float sum = bl;                                   // logarithm of the row factor
        // blocks J = w4 .. 0 need row factors from near to far; P is written
        // over A, so they go 0 .. w4: sum over the blocks between first
        for (int m = 1; m < w4; ++m) sum += tab.total[m];
        float v[32];
        uint32_t r[16];
        for (int J = 0; J < w4; ++J) {
          const float row = exp2_approx(sum);
          tc_ld32(tmem + lanes + kColA + 32 * J, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 f = reinterpret_cast<const float4 *>(tab.f + 32 * J)[j];
            r[2 * j] = pack2(v[4 * j] * (row * f.x), v[4 * j + 1] * (row * f.y));
            r[2 * j + 1] = pack2(v[4 * j + 2] * (row * f.z), v[4 * j + 3] * (row * f.w));
          }
          tc_st16(tmem + lanes + kColA + 16 * J, r);
          // next: one block fewer between
          sum = bl;
          for (int m = J + 2; m < w4; ++m) sum += tab.total[m];
        }
        tc_ld32(tmem + lanes + kColA + 32 * w4, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 o = reinterpret_cast<const float4 *>(tab.bl + 32 * w4)[j];
          float x[4] = {exp2_approx(bl - o.x), exp2_approx(bl - o.y), exp2_approx(bl - o.z),
                        exp2_approx(bl - o.w)};
#pragma unroll
          for (int m = 0; m < 4; ++m) x[m] = 4 * j + m <= lane ? v[4 * j + m] * x[m] : 0.0f;
          r[2 * j] = pack2(x[0], x[1]);
          r[2 * j + 1] = pack2(x[2], x[3]);
        }
        tc_st16(tmem + lanes + kColA + 16 * w4, r);
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = 0;
        for (int J = w4 + 1; J < 4; ++J) tc_st16(tmem + lanes + kColA + 16 * J, r);
        sum = bl;
        for (int m = 0; m < w4; ++m) sum += tab.total[m];
        const float e = exp2_approx(sum);
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.tab_empty[buf]);
        // O = E (Q S^T)
        KDA_WAIT_WARP(c.qs_full, one);
        tc_fence_after();
        for (int j = 0; j < 4; ++j) {
          tc_ld32(tmem + lanes + kColO + 32 * j, v);
#pragma unroll
          for (int m = 0; m < 32; ++m) v[m] *= e;
          tc_st32(tmem + lanes + kColO + 32 * j, v);
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.p_full);
        // the chunk's outputs
        KDA_WAIT_WARP(c.o_full, one);
        tc_fence_after();
        uint4 out[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          tc_ld32(tmem + lanes + kColO + 32 * j, v);
#pragma unroll
          for (int m = 0; m < 4; ++m)
            out[4 * j + m] = make_uint4(
                pack2(p.scale * v[8 * m], p.scale * v[8 * m + 1]),
                pack2(p.scale * v[8 * m + 2], p.scale * v[8 * m + 3]),
                pack2(p.scale * v[8 * m + 4], p.scale * v[8 * m + 5]),
                pack2(p.scale * v[8 * m + 6], p.scale * v[8 * m + 7]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.o_empty);
        if (rows == kChunk) {
          uint8_t *tile = sq + buf * kTile;
#pragma unroll
          for (int j = 0; j < 16; ++j) *reinterpret_cast<uint4 *>(tile + tile_at(i, j)) = out[j];
          fence_proxy_async_smem();
        } else if (i < rows) {
          uint4 *to = reinterpret_cast<uint4 *>(
              p.output + (it.first_row() + i) * p.o_stride + it.unit.h * kDim);
#pragma unroll
          for (int j = 0; j < 16; ++j) to[j] = out[j];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.st_full[buf]);
      }
    }
    __syncwarp();
  } else if (warp < 12) {
    regs_dec<96>();
    // ------------------------------------------------------------------- K''
    Walk<kOut> it(p);
    uint32_t quarter = 0;
    for (uint32_t n = 0; it.next(); ++n) {
      const int buf = n & 1, rows = it.rows(), quarters = (rows + 31) >> 5;
      const uint32_t two = (n >> 1) & 1;
      const Table &tab = c.tab[buf];
      KDA_WAIT_WARP(c.full_v[buf], two);
      if (rows < 32 * quarters) {
        // rows behind the sequence's end become zeros: they are other rows of
        // the tensor (or stale), and 0 * NaN is not 0
        const int at = threadIdx.x & 127;
        for (int x = at; x < (32 * quarters - rows) * 16; x += 128)
          *reinterpret_cast<uint4 *>(sv + buf * kTile + tile_at(rows + (x >> 4), x & 15)) =
              make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.v_ok[buf]);
      KDA_WAIT_WARP(c.tab_full[buf], two);
      KDA_WAIT_WARP(c.full_k[buf], two);
      const uint32_t k = smem_addr(sk + buf * kTile);
      int i = 0;
      for (; i < quarters; ++i, ++quarter) {
        const int kb = quarter & 1;
        // factors of the 8 tokens a lane sees: 8 j + 2 (lane % 4) + {0, 1}
        float sum = 0.0f;
        for (int m = i + 1; m < 4; ++m) sum += tab.total[m];
        const float block = exp2_approx(sum);
        float2 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[j] = reinterpret_cast<const float2 *>(tab.f + 32 * i + 8 * j)[lane & 3];
          f[j].x *= block;
          f[j].y *= block;
        }
        const int valid = rows - 32 * i - 2 * (lane & 3);   // token 8 j + e is live below it
        KDA_WAIT_WARP(c.kq_empty[kb], ((quarter >> 1) & 1) ^ 1);
        tc_fence_after();
        for (int half = 0; half < 2; ++half) {
          const int d0 = 32 * w4 + 16 * half;
          uint32_t hi[8], mid[8], lo[8];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t r[4];
            const int m = lane >> 3;
            ldmatrix_x4_trans(
                k + tile_at(32 * i + 16 * x + 8 * (m >> 1) + (lane & 7), d0 / 8 + (m & 1)), r);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int j = 2 * x + (y >> 1);
              float a = 8 * j < valid ? low_half(r[y]) * f[j].x : 0.0f;
              float b = 8 * j + 1 < valid ? high_half(r[y]) * f[j].y : 0.0f;
              const uint32_t h = pack2(a, b);
              a -= low_half(h);
              b -= high_half(h);
              const uint32_t s = pack2(a, b);
              a -= low_half(s);
              b -= high_half(s);
              hi[4 * x + y] = h;
              mid[4 * x + y] = s;
              lo[4 * x + y] = pack2(a, b);
            }
          }
          const uint32_t at = tmem + (static_cast<uint32_t>(d0) << 16) + kColK + kb * kColsK;
          tc_st_16x128(at, hi);
          tc_st_16x128(at + 16, mid);
          tc_st_16x128(at + 32, lo);
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
        mbar_arrive(&c.tab_empty[buf]);
      }
    }
    __syncwarp();
  } else {
    regs_inc<208>();
    // -------------------------------------------------------------- the page
    Walk<kOut> it(p);
    const int d = 32 * w4 + lane;                          // key
    const uint32_t lanes = static_cast<uint32_t>(32 * w4) << 16;
    uint32_t n = 0;
    bool ok = true;
    while (ok && it.next_unit(threadIdx.x == 384)) {
      float s[kDim];
      const float *from = nullptr;
      if (kOut) {
        if (it.unit.segs > 1)
          from = p.ws_state + ws_index(p, it.unit) * kPage;
        else if (it.unit.src)
          from = page_of(p.state, it.unit.src, p.heads, it.unit.h);
      }
      if (from) {
#pragma unroll
        for (int i = 0; i < kDim; ++i) s[i] = from[i * kDim + d];
      } else {
#pragma unroll
        for (int i = 0; i < kDim; ++i) s[i] = 0.0f;
      }
      float all = 0.0f;                                    // the unit's decay (logarithm)
      for (; it.next_chunk(); ++n) {
        ok = false;
        const int buf = n & 1;
        const uint32_t one = n & 1;
        const Table &tab = c.tab[buf];
        if (kOut) {
#pragma unroll
          for (int g = 0; g < 16; ++g)
            *reinterpret_cast<uint4 *>(ss + tile_at(d, g)) =
                make_uint4(pack2(s[8 * g], s[8 * g + 1]), pack2(s[8 * g + 2], s[8 * g + 3]),
                           pack2(s[8 * g + 4], s[8 * g + 5]), pack2(s[8 * g + 6], s[8 * g + 7]));
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.s_full);
        }
        KDA_WAIT_WARP(c.tab_full[buf], (n >> 1) & 1);
        const float total = (tab.total[0] + tab.total[1]) + (tab.total[2] + tab.total[3]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.tab_empty[buf]);
        const float keep = exp2_approx(total);
        all += total;
        KDA_WAIT_WARP(c.u_full, one);
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[32];
          tc_ld32(tmem + lanes + kColU + 32 * j, v);
#pragma unroll
          for (int m = 0; m < 32; ++m) s[32 * j + m] = __fmaf_rn(s[32 * j + m], keep, v[m]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.u_empty);
        ok = true;
      }
      if (!ok) break;
      float *to = nullptr;
      if (!kOut) {
        to = p.ws_state + ws_index(p, it.unit) * kPage;
        if (threadIdx.x == 384) p.ws_decay[ws_index(p, it.unit)] = all;
      } else if (it.unit.seg == it.unit.segs - 1 && it.unit.dst) {
        to = page_of(p.state, it.unit.dst, p.heads, it.unit.h);
      }
      if (to) {
#pragma unroll
        for (int i = 0; i < kDim; ++i) to[i * kDim + d] = s[i];
      }
    }
    __syncwarp();
  }
#undef KDA_WAIT_WARP
#undef KDA_WAIT

  __syncthreads();
  if (*abort_flag) {
    // copies and products in flight end within microseconds: give them time
    // before the shared memory and TMEM go
    const uint64_t t0 = global_ns();
    for (int i = 0; i < 4096 && global_ns() - t0 < 200000ull; ++i) __nanosleep(1000);
    if (threadIdx.x == 0 && p.err) atomicOr(p.err, KDA_DEVERR_TIMEOUT);
    __syncthreads();
  }
  tc_fence_after();
  if (warp == 3)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// The pages that the segments of split sequences start from, in place of their
// contributions: S_0 = the sequence's first page, S_(g+1) = 2^decay_g S_g + U_g.
// Each thread walks 4 elements of a page over the segments.
__global__ void __launch_bounds__(256) segment_kernel(const __grid_constant__ PromptParams p) {
  constexpr int kBlocks = kPage / (4 * 256);
  const int part = blockIdx.x % kBlocks, item = blockIdx.x / kBlocks;
  const int b = item / p.heads, h = item % p.heads;
  Seq seq;
  if (resolve_seq(p, b, &seq) || seq.len <= p.seg_len) return;
  const int segs = (seq.len + p.seg_len - 1) / p.seg_len;
  const int at = part * 256 + threadIdx.x;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (seq.src) s = reinterpret_cast<const float4 *>(page_of(p.state, seq.src, p.heads, h))[at];
  for (int g = 0; g < segs; ++g) {
    const int64_t page = ws_index(p, seq.start + g * p.seg_len, g == segs - 1, h);
    float4 *ws = reinterpret_cast<float4 *>(p.ws_state + page * kPage) + at;
    float4 u = s;
    if (g < segs - 1) u = *ws;
    *ws = s;
    if (g < segs - 1) {
      const float keep = exp2_approx(p.ws_decay[page]);
      s.x = __fmaf_rn(s.x, keep, u.x);
      s.y = __fmaf_rn(s.y, keep, u.y);
      s.z = __fmaf_rn(s.z, keep, u.z);
      s.w = __fmaf_rn(s.w, keep, u.w);
    }
  }
}

// ---------------------------------------------------------------------- host

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// BF16 rows [rows][width], `stride` elements apart, in boxes of 64 columns.
static bool rows_map(CUtensorMap *map, const void *base, int64_t width, int64_t rows,
                     int64_t stride, int box_rows) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, ones[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
                box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

int launch_chunked(const PromptParams &p, int qk_heads, int dev, int sms, cudaStream_t stream) {
  CUtensorMap q, k, v, o;
  const int64_t kw = int64_t(qk_heads) * kDim, vw = int64_t(p.heads) * kDim;
  if (!rows_map(&q, p.q, kw, p.tokens, p.q_stride, 32) ||
      !rows_map(&k, p.k, kw, p.tokens, p.k_stride, 32) ||
      !rows_map(&v, p.v, vw, p.tokens, p.v_stride, 32) ||
      !rows_map(&o, p.output, vw, p.tokens, p.o_stride, kChunk))
    return KDA_ERR_LAUNCH;
  static std::atomic<bool> out_done[kMaxDevices], seg_done[kMaxDevices];
  if (!set_smem_limit_once(out_done, dev, reinterpret_cast<const void *>(chunk_kernel<true>),
                           kSmem) ||
      !set_smem_limit_once(seg_done, dev, reinterpret_cast<const void *>(chunk_kernel<false>),
                           kSmem))
    return KDA_ERR_LAUNCH;
  const int64_t units = static_cast<int64_t>(p.seqs) * p.segs * p.heads;
  const int grid = units < sms ? static_cast<int>(units) : sms;
  if (p.segs > 1) {
    chunk_kernel<false><<<grid, kThreads, kSmem, stream>>>(p, q, k, v, o);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_LAUNCH;
    segment_kernel<<<p.seqs * p.heads * (kPage / 1024), 256, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return KDA_ERR_LAUNCH;
  }
  chunk_kernel<true><<<grid, kThreads, kSmem, stream>>>(p, q, k, v, o);
  return cudaGetLastError() == cudaSuccess ? KDA_SUCCESS : KDA_ERR_LAUNCH;
}

}  // namespace lin
}  // namespace kda
